"""Root-mean-square norm with residual and coded results against the oracle in 64
bits: every width class of the kernel, odd counts, strided rows, both kinds of weight,
values at the ends of the range, and rows that are not finite."""
import numpy as np
import pytest
import torch

from attention_parity import U, bf16, f64
from oracle.paged import norm_row
from paged_parity import check_bf16, check_codes

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")
EPS = 1e-6


def _check(label, x, weight, residual, out, got, eps=EPS, only=None):
    """got: the call's results; out: "bf16", "row" or "group"."""
    h = f64(x) if residual is None else f64(x) + f64(residual)
    w = f64(weight)
    got = list(got) if isinstance(got, tuple) else [got]
    if residual is not None:
        total = (x.float() + residual.float()).bfloat16()
        assert torch.equal(got[-1].cpu().view(torch.int16), total.view(torch.int16)), f"{label}: sum"
    for i in range(x.shape[0]) if only is None else only:
        want = norm_row(h[i], w, eps)
        err = 4 * U * np.abs(want) + 2.0 ** -149
        if out == "bf16":
            check_bf16(f"{label} row {i}", got[0][i], want, err)
            continue
        codes, scale = got[0][i].cpu().view(torch.uint8).numpy(), got[1][i].cpu().numpy()
        step = len(want) if out == "row" else 128
        for g, c in enumerate(range(0, len(want), step)):
            check_codes(f"{label} row {i} columns {c}..", codes[c:c + step], scale if out == "row" else scale[g], want[c:c + step],
                        err[c:c + step])


def _call(x, weight, residual, out, **kw):
    return S.rms_norm(x.cuda(), weight.cuda(), EPS, residual=None if residual is None else residual.cuda(),
                      coded=out != "bf16", group=128 if out == "group" else 0, **kw)


@pytest.mark.parametrize("out", ["bf16", "row", "group"])
@pytest.mark.parametrize("n,width", [(1, 8), (3, 64), (5, 136), (4, 512), (7, 520), (3, 1000), (2, 2048), (5, 2056), (3, 4096),
                                     (2, 4104), (3, 8192), (2, 8200), (1, 16384), (130, 512), (65, 1536)])
def test_norm(n, width, out):
    rng = np.random.default_rng(n * width)
    x, r = bf16(rng, n, width, scale=3.0), bf16(rng, n, width)
    w = (1 + 0.3 * bf16(rng, width).float()).bfloat16()
    for residual in (None, r):
        _check(f"{n}x{width} {out}", x, w, residual, out, _call(x, w, residual, out), only=range(min(n, 8)))
    w32 = torch.from_numpy(rng.standard_normal(width).astype(np.float32))
    _check(f"{n}x{width} {out} fp32 weight", x, w32, None, out, _call(x, w32, None, out), only=range(min(n, 8)))


@pytest.mark.parametrize("n", [3000, 9000])
@pytest.mark.parametrize("width", [72, 512, 1000, 4096])
def test_many_rows(n, width):
    rng = np.random.default_rng(width)
    x, r, w = bf16(rng, n, width), bf16(rng, n, width), bf16(rng, width)
    for out in ("bf16", "row", "group"):
        _check(f"{n}x{width} {out}", x, w, r, out, _call(x, w, r, out), only=[0, 1, n // 2, n - 1])


def test_strided_rows_and_given_outputs():
    rng = np.random.default_rng(3)
    wide, w = bf16(rng, 9, 640 + 64), bf16(rng, 640)
    x = wide[:, 64:]
    y = torch.full((9, 640), 7.0, dtype=torch.bfloat16, device="cuda")
    got = S.rms_norm(wide.cuda()[:, 64:], w.cuda(), EPS, out=y)
    assert got is y
    _check("strided", x, w, None, "bf16", y)
    r = bf16(rng, 9, 640)
    total = r.cuda()                                         # the residual itself takes the sum
    codes, scale = torch.empty(9, 640, dtype=torch.uint8, device="cuda"), torch.empty(9, 5, device="cuda")
    got = S.rms_norm(wide.cuda()[:, 64:], w.cuda(), EPS, residual=total, coded=True, group=128, out=(codes, scale), out_sum=total)
    assert got[0] is codes and got[1] is scale and got[2] is total
    _check("in place", x, w, r, "group", got)
    one = S.rms_norm(wide.cuda()[2:3, 64:], w.cuda(), EPS)
    assert torch.equal(one[0], y[2])
    assert S.rms_norm(wide.cuda()[:0, :640], w.cuda()).shape == (0, 640)
    bits = S.rms_norm(wide.cuda()[:, 64:].view(torch.int16), w.cuda().view(torch.int16), EPS)
    assert bits.dtype == torch.bfloat16 and torch.equal(bits, y)


def test_the_ends_of_the_range():
    rng = np.random.default_rng(4)
    w = torch.ones(1024).bfloat16()
    for scale in (1e30, 2.0 ** 126, 1e-30):                  # squares past fp32's range, either way
        x = bf16(rng, 4, 1024, scale=scale).clamp(-3e38, 3e38)
        for out in ("bf16", "row", "group"):
            got = S.rms_norm(x.cuda(), w.cuda(), 0.0, coded=out != "bf16", group=128 if out == "group" else 0)
            _check(f"{scale} {out}", x, w, None, out, got, eps=0.0)
    x = torch.zeros(3, 1024).bfloat16()
    x[1, 5] = -2.0
    codes, s = S.rms_norm(x.cuda(), w.cuda(), EPS, coded=True)
    assert s.cpu()[0] == 1 and s.cpu()[2] == 1 and (codes.cpu().view(torch.uint8)[0] == 0).all()
    _check("one value", x, w, None, "row", (codes, s))
    y = S.rms_norm(x.cuda(), w.cuda(), EPS)
    assert (y.cpu()[0] == 0).all()


def test_rows_that_are_not_finite():
    rng = np.random.default_rng(5)
    x, w = bf16(rng, 5, 512), bf16(rng, 512)
    clean = [_call(x, w, None, out) for out in ("bf16", "row", "group")]
    bad = x.clone()
    bad[1, 100], bad[3, 400] = float("inf"), float("nan")
    y, row, group = (_call(bad, w, None, out) for out in ("bf16", "row", "group"))
    ok = torch.tensor([0, 2, 4])
    assert torch.equal(y[ok], clean[0][ok])
    assert torch.equal(row[0][ok].view(torch.uint8), clean[1][0][ok].view(torch.uint8)) and torch.equal(row[1][ok], clean[1][1][ok])
    assert bool(y[3].isnan().all()) and bool(y[1, 100].isnan()) and bool((y[1, :100] == 0).all())   # inf / inf; finite / inf
    for r in (1, 3):
        assert bool(row[1][r].isnan()) and bool((row[0][r].view(torch.uint8) == 0x7f).all())
    assert group[1][1].isnan().tolist() == [True, False, False, False] and bool(group[1][3].isnan().all())
    assert bool((group[0][1, 128:].float() == 0).all()) and bool((group[0].view(torch.uint8)[1, :128] == 0x7f).all())


def test_the_same_bits_on_another_stream_and_in_graphs():
    rng = np.random.default_rng(6)
    x, r, w = bf16(rng, 33, 1000).cuda(), bf16(rng, 33, 1000).cuda(), bf16(rng, 1000).cuda()
    want = [t.clone() for t in S.rms_norm(x, w, EPS, residual=r, coded=True, group=128)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = S.rms_norm(x, w, EPS, residual=r, coded=True, group=128)
    side.synchronize()
    same = lambda a, b: all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(a, b))  # noqa: E731
    assert same(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = S.rms_norm(x, w, EPS, residual=r, coded=True, group=128)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert same(got, want)
        for t in got:
            t.view(torch.uint8).zero_()
    x.requires_grad_()
    assert not S.rms_norm(x, w, EPS).requires_grad


def test_refusals():
    rng = np.random.default_rng(7)
    x, w = bf16(rng, 3, 64).cuda(), bf16(rng, 64).cuda()
    for bad, text in [(dict(residual=x[:2]), "residual has shape"), (dict(weight=w[:32]), "weight has shape"),
                      (dict(weight=w.double()), "weight must be"), (dict(out_sum=x.clone()), "only for a residual"),
                      (dict(out=torch.empty(3, 64, device="cuda")), "out must be")]:
        with pytest.raises(ValueError, match=text):
            S.rms_norm(x, **(dict(weight=w) | bad))
    with pytest.raises(ValueError, match="contiguous"):
        S.rms_norm(bf16(rng, 64, 3).cuda().t(), w)
    with pytest.raises(ValueError, match="x must be"):
        S.rms_norm(x.float(), w)
    for bad in (dict(group=64, coded=True), dict(group=128), dict(eps=-1.0)):
        with pytest.raises((S.MisaError, ValueError)):
            S.rms_norm(x, w, **bad)
    with pytest.raises(S.MisaError, match="width"):
        S.rms_norm(bf16(rng, 3, 12).cuda(), bf16(rng, 12).cuda())
    with pytest.raises(S.MisaError, match="x_ld"):
        S.rms_norm(bf16(rng, 3, 68).cuda()[:, :64], w)
    with pytest.raises(S.MisaError, match="aligned"):
        S.rms_norm(bf16(rng, 3, 72).cuda()[:, 4:68], w)
