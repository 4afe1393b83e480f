"""Caches read in long calls, where a wave takes several rows, at counts that
do not fill its last rows, with slots that name no row and slots that repeat."""
import pytest
import torch

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("d,dr,n", [(512, 64, 8193), (512, 64, 10007), (512, 0, 9001), (128, 0, 32769), (128, 0, 40003),
                                    (128, 64, 33333)])
def test_long_reads(d, dr, n, fp8):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    rows = n // 2
    slots = torch.randint(-3, rows + 3, (n,), generator=g, device="cuda").int()
    there = (slots >= 0) & (slots < rows)
    if fp8:
        codes = torch.randint(0, 256, (rows, d), generator=g, device="cuda", dtype=torch.uint8)
        codes[(codes & 0x7f) == 0x7f] = 0x38                   # (no NaN, which does not compare)
        scale = torch.exp2(torch.randint(-20, 20, (rows,), generator=g, device="cuda").float())
        rope = torch.randn(rows, dr, generator=g, device="cuda").bfloat16() if dr else None
        cache = dict(C=codes, c_scale=scale, rope=rope)
        want = (codes.view(torch.float8_e4m3fn).double() * scale.double()[:, None]).bfloat16()  # exact: powers of two
        if dr:
            want = torch.cat([want, rope], 1)
    else:
        want = torch.randn(rows, d + dr, generator=g, device="cuda").bfloat16()
        cache = dict(C=want)
    guard = torch.full((n + 64, d + dr), 7.0, dtype=torch.bfloat16, device="cuda")
    got = S.cache_read(slots, out=guard[:n], **cache)
    torch.cuda.synchronize()
    want = torch.where(there[:, None], want[slots.clamp(0, rows - 1).long()], torch.zeros((), dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(got, want)
    assert bool((guard[n:] == 7.0).all())                      # rows behind the last: as they were
