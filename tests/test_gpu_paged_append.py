"""Rows appended to paged caches (normed, rotated, coded) and rotated queries against
the oracle in 64 bits: every form of cache and of rotation, pages of 1 to 256 rows,
padding, places that do not exist, and what a call must leave as it was."""
import numpy as np
import pytest
import torch

from attention_parity import U, bf16, f64, gpu
from oracle.paged import norm_row, page_row, rotate_row
from paged_parity import check_bf16, check_codes, ints, rotation, tables

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")
EPS = 1e-6


def _cache(rng, rows, d, dr, fp8):
    if not fp8:
        return dict(C=bf16(rng, rows, d + dr), c_scale=None, rope=None)
    return dict(C=torch.from_numpy(rng.integers(0, 120, (rows, d)).astype(np.uint8)),
                c_scale=torch.from_numpy((1 + rng.random(rows)).astype(np.float32)), rope=bf16(rng, rows, dr) if dr else None)


def _want(x, d, dr, weight, rot, turn, at, pairs):
    """A row's values in float64 and how far their fp32 forms may be off."""
    v, tail = x[:d].copy(), x[d:].copy()
    err, terr = np.zeros(d), np.zeros(dr)
    if weight is not None:
        v = norm_row(v, weight, EPS)
        err = 4 * U * np.abs(v)
    if rot is not None:
        part, perr = (tail, terr) if dr else (v[at:at + 64], err[at:at + 64])
        mate = np.abs(part.reshape(32, 2)[:, ::-1].reshape(64)) if pairs else np.abs(np.roll(part, 32))
        merr = perr.reshape(32, 2)[:, ::-1].reshape(64) if pairs else np.roll(perr, 32)
        new, nerr = rotate_row(part, rot[turn], pairs), perr + merr + 2 * U * (np.abs(part) + mate)
        if dr:
            tail, terr = new, nerr
        else:
            v[at:at + 64], err[at:at + 64] = new, nerr
    return v, tail, err, terr


def _check(label, cache, before, x, seq, pos, table, page, d, dr, weight=None, rot=None, turn=None, at=None, pairs=False):
    rows = before["C"].shape[0]
    x, turn = f64(x), pos if turn is None else turn
    written = {}
    for i in range(len(x)):
        r = page_row(table, page, rows, int(seq[i]), int(pos[i]))
        if r >= 0 and (rot is None or 0 <= turn[i] < len(rot)):
            written[r] = i
    w, cs = None if weight is None else f64(weight), None if rot is None else f64(rot)
    got = {n: None if t is None else t.cpu() for n, t in cache.items()}
    for r, i in written.items():
        v, tail, err, terr = _want(x[i], d, dr, w, cs, int(turn[i]), at, pairs)
        where = f"{label} row {i} at {r}"
        if got["c_scale"] is None:
            check_bf16(where, got["C"][r, :d], v, err)
            check_bf16(where, got["C"][r, d:], tail, terr)
        else:
            check_codes(where, got["C"][r].view(torch.uint8).numpy(), got["c_scale"][r], v, err)
            if dr:
                check_bf16(where, got["rope"][r], tail, terr)
    keep = torch.ones(rows, dtype=torch.bool)
    keep[list(written)] = False
    for n, t in got.items():                                 # all other rows hold what they held
        if t is not None:
            bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]
            assert torch.equal(t[keep].view(bits), before[n][keep].view(bits)), f"{label}: {n} outside the appended rows"
    return written


def _places(rng, seqs, new, cap):
    """Rows of every sequence at consecutive positions, in random order."""
    first = rng.integers(0, cap - new + 1, seqs)
    seq, pos = np.repeat(np.arange(seqs), new), (first[:, None] + np.arange(new)).reshape(-1)
    order = rng.permutation(seqs * new)
    return seq[order], pos[order]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,dr,at", [(512, 64, 512), (128, 0, 0), (128, 0, 64), (512, 0, 448), (128, 64, 128)])
@pytest.mark.parametrize("seqs,new,page", [(1, 1, 1), (3, 7, 1), (2, 33, 16), (5, 3, 64), (1, 70, 256)])
def test_append(seqs, new, page, d, dr, at, fp8):
    rng = np.random.default_rng(seqs * new * page + d + at)
    per = -(-(new + 5) // page)
    table, pool = tables(rng, seqs, per)
    seq, pos = _places(rng, seqs, new, per * page)
    x, rot = bf16(rng, seqs * new, d + dr, scale=2.0), rotation(per * page)
    weight = (1 + 0.3 * bf16(rng, d).float()).bfloat16()
    for kw in (dict(), dict(weight=weight), dict(rot=rot), dict(weight=weight, rot=rot, pairs=True), dict(weight=weight.float(), rot=rot)):
        before = _cache(rng, pool * page, d, dr, fp8)
        cache = gpu(before)
        S.paged_append(x.cuda(), ints(seq), ints(pos), ints(table), page, eps=EPS, rot_at=at if "rot" in kw else None, **cache, **gpu(kw))
        n = _check(f"{sorted(kw)}", cache, before, x, seq, pos, table, page, d, dr, at=at, **kw)
        assert len(n) == seqs * new


def test_drafted_tokens_turn_by_their_depth():
    # places in the cache and positions in the text differ; strided rows out of a wider projection
    rng = np.random.default_rng(2)
    table, pool = tables(rng, 2, 3)
    seq, pos, turn = np.repeat([0, 1], 6), np.tile(np.arange(20, 26), 2), np.tile([20, 21, 21, 22, 22, 23], 2)
    wide, rot = bf16(rng, 12, 32 + 576 + 64), rotation(64)
    before = _cache(rng, pool * 16, 512, 64, True)
    cache = gpu(before)
    S.paged_append(wide.cuda()[:, 32:608], ints(seq), ints(pos), ints(table), 16, rot=rot.cuda(), turn=ints(turn), **cache)
    _check("turn", cache, before, wide[:, 32:608], seq, pos, table, 16, 512, 64, rot=rot, turn=turn, at=512)


@pytest.mark.parametrize("fp8", [False, True])
def test_places_that_do_not_exist_write_nothing(fp8):
    rng = np.random.default_rng(3)
    page, rows = 16, 5 * 16 + 7                              # the last page is cut short by the cache's end
    table = np.array([[0, -1, 5], [2, 1 << 27, 3]], dtype=np.int32)
    seq = np.array([0, 0, 0, 0, 0, 1, 1, 1, -1, 2, 1, 0, 1, 0, 1, 2 ** 31 - 1, -2 ** 31])
    pos = np.array([0, 17, 32, 38, 39, 3, 20, 47, 4, 4, 48, -1, 2 ** 31 - 1, -2 ** 31, 40, 3, 3])
    turn = np.array([0, 1, 2, 49, 4, 5, 6, 50, 8, 9, 10, 11, 12, 13, -1, 5, 5])
    x, rot, w = bf16(rng, len(seq), 576), rotation(50), bf16(rng, 512)
    for kw in (dict(), dict(rot=rot, turn=turn), dict(rot=rot)):
        before = _cache(rng, rows, 512, 64, fp8)
        cache = gpu(before)
        more = {n: ints(v) if n == "turn" else v.cuda() for n, v in kw.items()}
        S.paged_append(x.cuda(), ints(seq), ints(pos), ints(table), page, weight=w.cuda(), eps=EPS, **cache, **more)
        n = _check(str(sorted(kw)), cache, before, x, seq, pos, table, page, 512, 64, weight=w, at=512, **kw)
        assert len(n) == {(): 6, ("rot", "turn"): 4, ("rot",): 6}[tuple(sorted(kw))]


def test_rows_that_are_not_finite_and_zero():
    rng = np.random.default_rng(4)
    table, x = np.arange(4, dtype=np.int32)[None], bf16(rng, 4, 576)
    x[0, 5], x[1, 7], x[2, :512], x[3, 520] = float("nan"), float("-inf"), 0.0, float("inf")
    for weight in (None, bf16(rng, 512).cuda()):
        cache = gpu(_cache(rng, 4, 512, 64, True))
        S.paged_append(x.cuda(), ints([0] * 4), ints(range(4)), ints(table), 1, weight=weight, rot=rotation(4).cuda(), **cache)
        s, codes = cache["c_scale"].cpu(), cache["C"].cpu().view(torch.uint8)
        assert s.isnan().tolist() == [True, True, False, False] and bool((codes[:2] == 0x7f).all())
        assert s[2] == 1 and bool((codes[2] & 0x7f == 0).all())
        assert bool(cache["rope"][:3].isfinite().all()) and not bool(cache["rope"][3].isfinite().all())


def test_against_cache_write():
    # pages in order, nothing on the way: what misa_cache_write writes, bit for bit
    rng = np.random.default_rng(5)
    for d, dr in ((512, 64), (128, 0)):
        for fp8 in (False, True):
            before = _cache(rng, 96, d, dr, fp8)
            a, b, x = gpu(before), gpu(before), bf16(rng, 40, d + dr, scale=5.0).cuda()
            at = torch.from_numpy(rng.permutation(96)[:40].astype(np.int32)).cuda()
            S.cache_write(x, at, **a)
            S.paged_append(x, torch.zeros_like(at), at, ints(np.arange(6)[None]), 16, **b)
            for n in a:
                if a[n] is not None:
                    assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), (d, fp8, n)


def test_rows_far_into_a_long_cache():
    # a row whose byte offset passes 2^32
    rows, page = 4_200_000, 64
    C = torch.zeros(rows, 576, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(6)
    x, table = bf16(rng, 2, 576), np.array([[rows // page - 1, 0]], dtype=np.int32)
    S.paged_append(x.cuda(), ints([0, 0]), ints([63, 64]), ints(table), page, C)
    assert torch.equal(C[(rows // page - 1) * page + 63].cpu(), x[0]) and torch.equal(C[0].cpu(), x[1])
    assert int((C != 0).any(1).sum()) == 2


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (7, 5), (33, 16), (300, 3), (2, 129)])
def test_rotate(T, H, pairs):
    rng = np.random.default_rng(T + H)
    x, rot = bf16(rng, T, H, 192), rotation(1000)
    pos = rng.integers(0, 1000, T).astype(np.int32)
    q = bf16(rng, T, H, 576)
    to = q.cuda()
    got = S.rotate(x.cuda()[:, :, 128:], ints(pos), rot.cuda(), pairs=pairs, out=to[:, :, 512:])
    assert got.data_ptr() == to[:, :, 512:].data_ptr()
    assert torch.equal(to[:, :, :512].cpu(), q[:, :, :512])
    plain = S.rotate(x.cuda()[:, :, 128:].contiguous(), ints(pos), rot.cuda(), pairs=pairs)
    assert torch.equal(plain, to[:, :, 512:])
    own = x.cuda()[:, :, 128:].contiguous()
    S.rotate(own, ints(pos), rot.cuda(), pairs=pairs, out=own)            # in place
    assert torch.equal(own, plain)
    heads_first = x.cuda()[:, :, 128:].transpose(0, 1).contiguous().transpose(0, 1)  # [T, H, 64] with heads outermost
    assert torch.equal(S.rotate(heads_first, ints(pos), rot.cuda(), pairs=pairs), plain)
    xs, cs, out = f64(x[:, :, 128:]), f64(rot), f64(plain)
    for t in range(min(T, 10)):
        for h in range(min(H, 8)):
            part = xs[t, h]
            mate = np.abs(part.reshape(32, 2)[:, ::-1].reshape(64)) if pairs else np.abs(np.roll(part, 32))
            check_bf16(f"t={t} h={h}", torch.from_numpy(out[t, h]), rotate_row(part, cs[pos[t]], pairs), 2 * U * (np.abs(part) + mate))


def test_rotate_leaves_queries_without_a_position():
    rng = np.random.default_rng(8)
    x, rot = bf16(rng, 4, 3, 64).cuda(), rotation(10).cuda()
    pos = ints([3, -1, 10, 9])
    got, mine = S.rotate(x, pos, rot), x.clone()
    S.rotate(x, pos, rot, out=mine)
    assert bool((got[1:3] == 0).all()) and torch.equal(mine[1:3], x[1:3])
    assert torch.equal(mine[0], got[0]) and torch.equal(mine[3], got[3]) and not torch.equal(mine[0], x[0])
    assert S.rotate(x[:0], pos[:0], rot).shape == (0, 3, 64)


def test_graphs_and_streams():
    rng = np.random.default_rng(9)
    table, pool = tables(rng, 3, 2)
    x, w, rot = bf16(rng, 3, 576).cuda(), bf16(rng, 512).cuda(), rotation(32).cuda()
    seq, pos, t = ints([0, 1, 2]), ints([3, 17, 31]), ints(table)
    before = gpu(_cache(rng, pool * 16, 512, 64, True))
    a, b, c = ({n: v.clone() for n, v in before.items()} for _ in range(3))
    call = lambda k: S.paged_append(x, seq, pos, t, 16, weight=w, rot=rot, **k)  # noqa: E731
    call(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(b)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c)
    for _ in range(3):
        for n in c:
            c[n].copy_(before[n])
        g.replay()
        torch.cuda.synchronize()
        for n in a:
            assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)) and torch.equal(a[n].view(torch.uint8), c[n].view(torch.uint8))


def test_refusals():
    rng = np.random.default_rng(10)
    x, C, i = bf16(rng, 2, 576).cuda(), bf16(rng, 32, 576).cuda(), ints([0, 1])
    t, rot = ints([[0, 1]]), rotation(8).cuda()
    ok = dict(x=x, seq=i, pos=i, table=t, page=16, C=C)
    for bad, text in [(dict(x=x[:, :512]), "x has shape"), (dict(seq=i.long()), "seq must be"), (dict(pos=i[:1]), "pos has shape"),
                      (dict(table=t[0]), "2 dimensions"), (dict(weight=bf16(rng, 64).cuda()), "weight has shape"),
                      (dict(rot=rot[:, :32]), "rot "), (dict(rot_at=0), "only for a rotation"), (dict(pairs=True), "only for a rotation"),
                      (dict(rot=rot.double()), "rot must be"), (dict(x=x.t().contiguous().t()), "contiguous")]:
        with pytest.raises(ValueError, match=text):
            S.paged_append(**(ok | bad))
    for bad, text in [(dict(page=12), "power of two"), (dict(rot=rot, rot_at=0), "rot_at"), (dict(turn=i), "turn"),
                      (dict(weight=bf16(rng, 512).cuda(), eps=-1.0), "eps")]:
        with pytest.raises(S.MisaError, match=text):
            S.paged_append(**(ok | bad))
    assert torch.equal(C.cpu(), C.cpu())
    q = bf16(rng, 2, 3, 64).cuda()
    with pytest.raises(ValueError, match="shape"):
        S.rotate(q[:, :, :32].contiguous(), i, rot)
    with pytest.raises(ValueError, match="shape"):
        S.rotate(q, i, rot, out=q[:, :2])
    with pytest.raises(S.MisaError, match="x_h"):
        S.rotate(bf16(rng, 2, 3, 68).cuda()[:, :, :64], i, rot)
    with pytest.raises(S.MisaError, match="x_t"):
        S.rotate(q[:1].expand(2, 3, 64), i, rot)
