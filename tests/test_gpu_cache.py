"""Cache rows written and read on the GPU: codes, scales and read values equal
the oracle's exactly (a power-of-two scale leaves one rounding, and it is the
same one)."""
import numpy as np
import pytest
import torch

import oracle as O
from attention_parity import bf16, f64
from oracle.attention import code_row

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")


def _empty(rows, d, dr, fp8, fill=0x5a):
    """A cache whose bytes are all `fill`."""
    raw = lambda n, w, dt: torch.full((n, w), fill, dtype=torch.uint8, device="cuda").view(dt)  # noqa: E731
    if not fp8:
        return dict(C=raw(rows, 2 * (d + dr), torch.bfloat16), c_scale=None, rope=None)
    return dict(C=raw(rows, d, torch.uint8), c_scale=raw(rows, 4, torch.float32).view(-1),
                rope=raw(rows, 2 * dr, torch.bfloat16) if dr else None)


def _bytes(c):
    return [t.view(torch.uint8).clone() for t in c.values() if t is not None]


@pytest.mark.parametrize("d,dr", [(512, 64), (128, 0), (512, 0), (128, 64)])
@pytest.mark.parametrize("n", [1, 2, 7, 16, 33, 500])
@pytest.mark.parametrize("fp8", [True, False])
def test_write_then_read(d, dr, n, fp8):
    rng = np.random.default_rng(1000 * d + dr + n)
    rows = n + 13
    x = bf16(rng, n, d + dr) * torch.from_numpy(np.exp2(rng.integers(-30, 30, (n, 1)))).bfloat16()
    x[0, :d] = 0.0  # a zero row
    if n > 2:
        x[1, :5] = torch.tensor([448.0, -1.0, 2.0 ** -9, -2.0 ** -10, 3 * 2.0 ** -10])  # scale 1, ties at the bottom
        x[1, 5:d] = 0.25
        x[2, :d] = x[2, :d].sign() * 2.0 ** -133  # bf16's smallest
    slots = torch.from_numpy(rng.permutation(rows)[:n].astype(np.int32))
    if n > 4:
        slots[3] = -1
        slots[4] = rows  # past the cache
    c = _empty(rows, d, dr, fp8)
    before = {k: None if v is None else v.view(torch.uint8).clone() for k, v in c.items()}
    S.cache_write(x.cuda(), slots.cuda(), **c)
    live = [i for i in range(n) if 0 <= int(slots[i]) < rows]
    named = torch.tensor([int(slots[i]) for i in live], dtype=torch.long)
    rest = torch.ones(rows, dtype=torch.bool)
    rest[named] = False
    for k, v in c.items():  # rows that no slot names are as they were
        if v is not None:
            b, a = before[k].view(rows, -1).cpu(), v.view(torch.uint8).view(rows, -1).cpu()
            assert torch.equal(a[rest], b[rest]), k
    if fp8:
        for i in live:
            codes, scale = code_row(f64(x[i, :d]))
            assert float(c["c_scale"][int(slots[i])]) == scale, i
            assert np.array_equal(c["C"][int(slots[i])].cpu().numpy(), codes), i
            if dr:
                assert torch.equal(c["rope"][int(slots[i])].cpu(), x[i, d:]), i
    back = S.cache_read(slots.cuda(), **c).cpu()
    for i in range(n):
        if i not in live:
            assert (back[i] == 0).all()
        elif fp8:
            codes, scale = code_row(f64(x[i, :d]))
            assert np.array_equal(f64(back[i, :d]), O.decode_e4m3fn(codes) * scale), i  # exact in bf16
            assert torch.equal(back[i, d:], x[i, d:]), i
        else:
            assert torch.equal(back[i], x[i]), i


def test_every_bf16_value_is_coded_like_the_oracle():
    # each finite bf16 value beside a maximum that fixes the row's scale
    for top in (448.0, 450.0, 1.0, 1.7578125, 2.0 ** -125, 3.0e38):
        bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
        v = bits.view(torch.bfloat16)
        v = v[torch.isfinite(v) & (v.abs() <= top)]
        v = torch.cat([v, torch.zeros((-v.numel()) % 127, dtype=torch.bfloat16)]).view(-1, 127)
        x = torch.cat([v, torch.full((v.shape[0], 1), top, dtype=torch.bfloat16)], 1)
        c = _empty(x.shape[0], 128, 0, True)
        S.cache_write(x.cuda(), torch.arange(x.shape[0], dtype=torch.int32, device="cuda"), **c)
        for i in range(x.shape[0]):
            codes, scale = code_row(f64(x[i]))
            assert float(c["c_scale"][i]) == scale
            assert np.array_equal(c["C"][i].cpu().numpy(), codes), (top, i)


def test_rows_that_are_not_finite_read_back_as_nan():
    x = torch.ones(4, 576, dtype=torch.bfloat16)
    x[1, 7], x[2, 511], x[3, 575] = float("inf"), float("nan"), float("inf")  # the last one in the rotary part
    c = _empty(4, 512, 64, True)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    S.cache_write(x.cuda(), slots, **c)
    back = S.cache_read(slots, **c).cpu()
    assert torch.equal(back[0], x[0])
    assert back[1, :512].isnan().all() and back[2, :512].isnan().all()
    assert torch.equal(back[3], x[3]) and torch.equal(back[1, 512:], x[1, 512:])


def test_read_rounds_any_scale_once_from_fp32():
    rng = np.random.default_rng(5)
    codes = torch.from_numpy(rng.integers(0, 126, (64, 512)).astype(np.uint8))
    scale = torch.from_numpy((rng.random(64) * 3 - 1).astype(np.float32))
    rope = bf16(rng, 64, 64)
    slots = torch.tensor([5, 5, 63, 0, -7, 64, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    got = S.cache_read(slots.cuda(), codes.cuda(), scale.cuda(), rope.cuda()).cpu()
    dec = torch.from_numpy(O.decode_e4m3fn(codes.numpy())).float()
    want = torch.cat([(dec * scale[:, None]).bfloat16(), rope], 1)
    for i, s in enumerate([5, 5, 63, 0]):
        assert torch.equal(got[i], want[s])
    assert (got[4:] == 0).all()


def test_empty_calls():
    c = _empty(4, 512, 64, True)
    was = _bytes(c)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    S.cache_write(torch.empty(0, 576, dtype=torch.bfloat16, device="cuda"), none, **c)
    assert tuple(S.cache_read(none, **c).shape) == (0, 576)
    assert all(torch.equal(a, b) for a, b in zip(was, _bytes(c)))


def test_offsets_past_32_bits():
    # 4.3 GB of codes, 1.1 GB of rotary values: only rows at both ends are touched
    rows = (1 << 32) // 512 + 5
    C = torch.empty(rows, 512, dtype=torch.uint8, device="cuda")
    scale = torch.empty(rows, dtype=torch.float32, device="cuda")
    rope = torch.empty(rows, 64, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(3)
    x = bf16(rng, 3, 576)
    slots = torch.tensor([rows - 1, 0, rows - 3], dtype=torch.int32, device="cuda")
    S.cache_write(x.cuda(), slots, C, scale, rope)
    got = S.cache_read(slots, C, scale, rope).cpu()
    for i in range(3):
        codes, s = code_row(f64(x[i, :512]))
        assert np.array_equal(f64(got[i, :512]), O.decode_e4m3fn(codes) * s)
        assert torch.equal(got[i, 512:], x[i, 512:])
