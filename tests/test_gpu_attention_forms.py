"""Latent and expanded attention on the GPU in every way that a call is cut
(16, 32, 64 and 128 rows a workgroup, keys in one share or split, expanded on
four and eight waves), with ragged lengths, padded queries and bad values; at
softmax scales from zero to large and of both signs; and calls that the binding
refuses. The sizes are the smallest that the cost model cuts in each way."""
import numpy as np
import pytest
import torch

from attention_parity import SM, bf16, check_rows, f64, gpu, latent_cache
from oracle.attention import latent_keys

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")


def _ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _check(label, got, lse, q, K, dv, rows_of, sm, only):
    check_rows(label, got, lse, q, lambda t, h: (K[rows_of(t)], K[rows_of(t)][:, :dv]), dv, sm=sm, only=only)


def _dirty(cache, rows, fp8, bad):
    """The cache with `bad` in every place of the given rows."""
    d = {n: (None if v is None else v.clone()) for n, v in cache.items()}
    if fp8:
        d["C"].view(torch.uint8)[rows] = 0x7f
        d["c_scale"][rows] = bad
        d["rope"][rows] = bad
    else:
        d["C"][rows] = bad
    return d


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,k", [(128, 40, 64), (16, 20, 3000), (260, 40, 64), (16, 40, 3000), (260, 100, 64), (64, 100, 3000), (100, 100, 8192)])
def test_lists(T, H, k, fp8):
    rng = np.random.default_rng(T + H + k)
    rows = 2 * k + 40
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    idx = 2 * rng.integers(0, k, (T, k)).astype(np.int32)     # even rows only; repeats, no order
    idx[rng.random((T, k)) < 0.3] = -1
    idx[1], idx[2, :k - 1] = -1, -1                            # no key; one at most
    idx[3, min(k - 1, 64):min(k - 1, 640)] = -1                # empty tiles
    base = 2 * rng.integers(0, 25, T).astype(np.int32)         # the last bases reach past the cache
    base[4] = -1
    args = dict(sm_scale=SM, idx=_ints(idx), base=_ints(base), with_lse=True)
    out, lse = S.latent_attention(q.cuda(), **gpu(cache), **args)
    _check(f"T={T} H={H} k={k}", out, lse, q, K, 512, lambda t: latent_keys(rows, None, idx[t], int(base[t])), SM,
           [0, 1, 2, 3, 4, T // 2, T - 1])
    d = _dirty(cache, torch.arange(rows) % 2 == 1, fp8, float("nan"))
    o2, z2 = S.latent_attention(q.cuda(), **gpu(d), **args)
    assert torch.equal(o2, out) and torch.equal(z2, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,rows", [(260, 3, 64), (128, 3, 400), (260, 20, 64), (32, 20, 3000), (32, 40, 3000), (520, 3, 64), (64, 40, 1000),
                                      (260, 3, 3000), (400, 33, 130)])
@pytest.mark.parametrize("order", ["causal", "any"])
def test_prefix(T, H, rows, fp8, order):
    # queries side by side share key tiles: with ends one apart, and with ends anywhere
    rng = np.random.default_rng(T + H + rows)
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    pos = (np.arange(T) % rows if order == "causal" else rng.integers(-1, rows + 2, T)).astype(np.int32)
    pos[1], pos[2], pos[T - 2] = -1, 2 ** 31 - 1, -2 ** 31
    args = dict(sm_scale=SM, pos=_ints(pos), with_lse=True)
    out, lse = S.latent_attention(q.cuda(), **gpu(cache), **args)
    _check(f"T={T} H={H} L={rows}", out, lse, q, K, 512, lambda t: latent_keys(rows, int(pos[t])), SM,
           [0, 1, 2, 3, T // 3, T // 2, T - 2, T - 1])
    cut = rows // 2 + 5                                        # a bad row: the queries that see it, and no other
    for bad in (float("nan"), float("inf")):
        d = _dirty(cache, torch.tensor([cut]), fp8, bad)
        o2, z2 = S.latent_attention(q.cuda(), **gpu(d), **args)
        sees = torch.from_numpy(pos >= cut)
        assert torch.equal(o2.cpu()[~sees], out.cpu()[~sees]) and torch.equal(z2.cpu()[~sees], lse.cpu()[~sees])
        assert bool(o2.cpu()[sees].isnan().all())


@pytest.mark.parametrize("T,H,L", [(300, 2, 64), (300, 2, 5000), (500, 256, 512), (500, 64, 3000)])
def test_expanded(T, H, L):
    rng = np.random.default_rng(T + H + L)
    q, kv, rope = bf16(rng, T, H, 192), bf16(rng, L, H, 256), bf16(rng, L, 64)
    pos = rng.integers(-1, L + 2, T).astype(np.int32)
    base = rng.integers(0, L + 1, T).astype(np.int32)
    base[:T // 2] = 0
    pos[1], base[3], base[T - 1] = 2 ** 31 - 1, -1, 2 ** 31 - 1
    out, lse = S.expanded_attention(q.cuda(), kv.cuda(), rope.cuda(), _ints(pos), SM, base=_ints(base), with_lse=True)
    kd, rd = f64(kv), f64(rope)

    def rows_of(t, h):
        r = latent_keys(L, int(pos[t]), None, int(base[t]))
        return np.concatenate([kd[r, h, :128], rd[r]], 1), kd[r, h, 128:]
    check_rows(f"T={T} H={H} L={L}", out, lse, q, rows_of, 128, only=[0, 1, 2, 3, T // 2 - 1, T // 2, T - 2, T - 1])


@pytest.mark.parametrize("sm", [0.0, -0.0, 1e-42, 1e-20, -0.07, 3.0])
@pytest.mark.parametrize("T,H,k", [(2, 20, 300), (260, 40, 64)])
def test_softmax_scales(T, H, k, sm):
    # a scale of zero weighs every key alike, whatever the scores are: here up to 2^122
    rng = np.random.default_rng(5)
    big = 2.0 ** 58 if abs(sm) < 1e-30 else 1.0
    K32, q = bf16(rng, 2 * k, 576, scale=big), bf16(rng, T, H, 576, scale=big)
    K = f64(K32)
    idx = np.stack([rng.permutation(2 * k)[:k] for _ in range(T)]).astype(np.int32)
    out, lse = S.latent_attention(q.cuda(), K32.cuda(), sm, idx=_ints(idx), with_lse=True)
    _check(f"sm={sm}", out, lse, q, K, 512, lambda t: idx[t], sm, [0, T - 1])
    kv, rope, qe = bf16(rng, k, 3, 256, scale=big), bf16(rng, k, 64, scale=big), bf16(rng, 40, 3, 192, scale=big)
    pos = np.arange(k - 40, k, dtype=np.int32)
    out, lse = S.expanded_attention(qe.cuda(), kv.cuda(), rope.cuda(), _ints(pos), sm, with_lse=True)
    kd, rd = f64(kv), f64(rope)
    check_rows(f"expanded sm={sm}", out, lse, qe,
               lambda t, h: (np.concatenate([kd[:pos[t] + 1, h, :128], rd[:pos[t] + 1]], 1), kd[:pos[t] + 1, h, 128:]), 128,
               sm=sm, only=[0, 39])


def test_one_rotary_row_at_the_end_of_its_tensor():
    # a single key whose rotary row is the last 64 values of a wider row
    rng = np.random.default_rng(6)
    q, kv, rows = bf16(rng, 3, 2, 192), bf16(rng, 1, 2, 256), bf16(rng, 1, 576)
    out = S.expanded_attention(q.cuda(), kv.cuda(), rows.cuda()[:, 512:], _ints([0, -1, 5]), SM)
    want = kv[0, :, 128:]
    assert torch.equal(out.cpu()[0], want) and torch.equal(out.cpu()[2], want) and not out.cpu()[1].any()


def test_two_streams_at_once():
    rng = np.random.default_rng(7)
    T, H, rows, k = 8, 64, 4000, 2000
    cache, _ = latent_cache(rng, rows, True)
    cache = gpu(cache)
    qs = [bf16(rng, T, H, 576).cuda() for _ in range(2)]
    idx = [_ints(rng.integers(0, rows, (T, k))) for _ in range(2)]
    ref = [S.latent_attention(q, sm_scale=SM, idx=i, **cache) for q, i in zip(qs, idx)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[j].append(S.latent_attention(qs[j], sm_scale=SM, idx=idx[j], **cache))
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(o, ref[j]) for o in outs[j])


def test_refused_arguments():
    dev = "cuda"
    q = torch.zeros(2, 4, 576, dtype=torch.bfloat16, device=dev)
    C = torch.zeros(8, 576, dtype=torch.bfloat16, device=dev)
    codes = torch.zeros(8, 512, dtype=torch.uint8, device=dev)
    scale, rope = torch.ones(8, device=dev), torch.zeros(8, 64, dtype=torch.bfloat16, device=dev)
    pos, idx = _ints([0, 1]), _ints([[0, 1], [2, -1]])
    att = lambda **kw: S.latent_attention(**{**dict(q=q, C=C, sm_scale=SM, pos=pos), **kw})  # noqa: E731
    bad = [
        dict(q=q.float()), dict(q=q[:, :, :512].contiguous()), dict(q=q[0]), dict(q=q.transpose(0, 1)),
        dict(C=C.half()), dict(C=C[:, :512]), dict(C=codes), dict(C=codes, c_scale=scale),
        dict(C=codes, c_scale=scale.double(), rope=rope), dict(C=codes, c_scale=scale[:4], rope=rope),
        dict(C=codes, c_scale=scale, rope=rope[:, ::2]), dict(pos=pos.long()), dict(pos=pos[:1]), dict(pos=None),
        dict(pos=None, idx=idx.long()), dict(pos=None, idx=idx[:1]), dict(pos=None, idx=idx.t()), dict(idx=idx),
        dict(base=pos.cpu()), dict(base=pos.long()), dict(sm_scale=float("nan")), dict(sm_scale=float("inf")),
        dict(out=torch.zeros(2, 4, 512, device=dev)), dict(out=torch.zeros(2, 4, 576, dtype=torch.bfloat16, device=dev)),
        dict(c_scale=scale), dict(rope=rope),
    ]
    for kw in bad:
        with pytest.raises((ValueError, S.MisaError)):
            att(**kw)
    qe = torch.zeros(2, 4, 192, dtype=torch.bfloat16, device=dev)
    kv = torch.zeros(8, 4, 256, dtype=torch.bfloat16, device=dev)
    exp = lambda **kw: S.expanded_attention(**{**dict(q=qe, kv=kv, rope=rope, pos=pos, sm_scale=SM), **kw})  # noqa: E731
    wide = torch.zeros(8, 68, dtype=torch.bfloat16, device=dev)
    for kw in [dict(q=qe.float()), dict(kv=kv[:, :3]), dict(kv=kv.transpose(0, 1)), dict(rope=rope[:7]), dict(rope=rope[:, ::2]),
               dict(rope=wide[:, 4:]), dict(rope=wide[:, :64]), dict(pos=pos[:1]), dict(base=idx), dict(sm_scale=float("nan")),
               dict(out=torch.zeros(2, 4, 128, device=dev))]:
        with pytest.raises((ValueError, S.MisaError)):
            exp(**kw)
    x = torch.zeros(2, 576, dtype=torch.bfloat16, device=dev)
    for kw in [dict(x=x.float()), dict(x=x[:, :512].contiguous()), dict(slots=pos.long()), dict(slots=pos[:1]), dict(slots=pos.cpu()),
               dict(c_scale=scale)]:
        with pytest.raises((ValueError, S.MisaError)):
            S.cache_write(**{**dict(x=x, slots=pos, C=C), **kw})
    for kw in [dict(slots=pos.long()), dict(slots=idx), dict(out=torch.zeros(2, 512, dtype=torch.bfloat16, device=dev))]:
        with pytest.raises((ValueError, S.MisaError)):
            S.cache_read(**{**dict(slots=pos, C=C), **kw})
    torch.cuda.synchronize()
    assert not C.any()
