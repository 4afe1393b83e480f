"""Latent attention on the GPU (absorbed and expanded form) against the
float64 oracle, at the sizes and masks where it can go wrong."""
import numpy as np
import pytest
import torch

from attention_parity import SM, bf16, check_expanded, check_latent, f64, gpu, latent_cache

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")


def _lists(rng, T, rows, k, fill=1.0):
    """k distinct rows of each query in ascending order, the tail -1 in part."""
    idx = np.full((T, k), -1, dtype=np.int32)
    for t in range(T):
        n = min(rows, k if fill == 1.0 else int(rng.integers(0, k + 1)))
        idx[t, :n] = np.sort(rng.permutation(rows)[:n])
    return idx


def _ints(a):
    return None if a is None else torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _latent(cache, q, **kw):
    return S.latent_attention(q.cuda(), sm_scale=SM, with_lse=True, **gpu(cache), **kw)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [1, 5, 16, 17, 32, 40, 64, 65, 128])
def test_lists_by_heads(H, fp8):
    rng = np.random.default_rng(H)
    T, rows, k = 3, 700, 333
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    idx = _lists(rng, T, rows, k)
    out, lse = _latent(cache, q, idx=_ints(idx))
    check_latent(f"H={H}", out, lse, q, K, idx=idx)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("k", [1, 2, 15, 16, 63, 64, 65, 127, 129, 1000, 2048])
def test_lists_by_length(k, fp8):
    rng = np.random.default_rng(k)
    T, H, rows = 4, 20, 2100
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    idx = _lists(rng, T, rows, k, fill=0.0)
    idx[0] = -1                       # a query without keys
    idx[1, :min(k, rows)] = np.sort(rng.permutation(rows)[:min(k, rows)])  # a full one
    out, lse = _latent(cache, q, idx=_ints(idx))
    check_latent(f"k={k}", out, lse, q, K, idx=idx)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [7, 16, 64, 128])
def test_many_queries_in_one_split(H, fp8):
    rng = np.random.default_rng(90 + H)
    T, rows, k = 520, 400, 70
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    idx = _lists(rng, T, rows, k, fill=0.0)
    out, lse = _latent(cache, q, idx=_ints(idx))
    check_latent(f"T={T}", out, lse, q, K, idx=idx, only=[0, 1, 2, 100, 255, 256, 257, 519])


@pytest.mark.parametrize("fp8", [False, True])
def test_lists_with_holes_repeats_any_order_and_bad_entries(fp8):
    rng = np.random.default_rng(8)
    T, H, rows, k = 5, 16, 300, 260
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    idx = rng.integers(0, rows, (T, k)).astype(np.int32)      # repeats, no order
    idx[rng.random((T, k)) < 0.4] = -1                        # holes
    idx[1, 64:192] = -1                                       # whole tiles of them
    idx[2, :] = -1
    idx[2, 200] = 17                                          # one key in the last tile
    idx[3, 3], idx[3, 70], idx[3, 71] = rows, 2 ** 31 - 1, -2 ** 31
    base = np.array([0, 0, 100, 0, 250], dtype=np.int32)      # and rows past the cache
    out, lse = _latent(cache, q, idx=_ints(idx), base=_ints(base))
    check_latent("holes", out, lse, q, K, idx=idx, base=base)
    base[0], base[1] = -1, -2 ** 31                           # no keys
    out, lse = _latent(cache, q, idx=_ints(idx), base=_ints(base))
    check_latent("base < 0", out, lse, q, K, idx=idx, base=base)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,rows", [(1, 1, 1), (1, 16, 64), (2, 5, 65), (4, 32, 1000), (9, 16, 130), (3, 128, 257),
                                      (70, 7, 300), (1, 128, 5000)])
def test_visible_prefix(T, H, rows, fp8):
    rng = np.random.default_rng(T * rows + H)
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    pos = rng.integers(-1, rows, T).astype(np.int32)
    pos[0] = rows - 1
    if T > 2:
        pos[1], pos[2] = -5, 2 ** 31 - 1                      # no key; all
    for base in (None, rng.integers(0, rows + 1, T).astype(np.int32)):
        out, lse = _latent(cache, q, pos=_ints(pos), base=_ints(base))
        check_latent(f"T={T} base={base is not None}", out, lse, q, K, pos=pos, base=base)


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_that_are_no_keys_do_not_matter(fp8):
    rng = np.random.default_rng(21)
    T, H, rows, k = 6, 16, 400, 100
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    idx = _lists(rng, T, 200, k, fill=0.0) * 2
    idx[idx < 0] = -1                                          # even rows only
    pos = np.array([130, 131, 132, 190, 10, -1], dtype=np.int32)
    ref = [_latent(cache, q, idx=_ints(idx)), _latent(cache, q, pos=_ints(pos))]
    for bad in (float("nan"), float("inf"), float("-inf")):
        dirty = {n: (None if v is None else v.clone()) for n, v in cache.items()}
        odd = torch.zeros(rows, dtype=torch.bool)
        odd[1::2] = True
        late = torch.arange(rows) > 190
        for rowset, which in ((odd, 0), (late, 1)):
            d = {n: (None if v is None else v.clone()) for n, v in dirty.items()}
            if fp8:
                d["C"].view(torch.uint8)[rowset] = 0x7f
                d["c_scale"][rowset] = bad
                d["rope"][rowset] = bad
            else:
                d["C"][rowset] = bad
            kw = dict(idx=_ints(idx)) if which == 0 else dict(pos=_ints(pos))
            got = _latent(d, q, **kw)
            assert torch.equal(got[0], ref[which][0]) and torch.equal(got[1], ref[which][1])


@pytest.mark.parametrize("fp8", [False, True])
def test_a_bad_key_reaches_the_queries_that_see_it_only(fp8):
    # queries of one tile with different ends: keys 131 and 140 hold NaN and infinities
    rng = np.random.default_rng(22)
    T, H, rows = 8, 4, 200
    cache, K = latent_cache(rng, rows, fp8)
    q = bf16(rng, T, H, 576)
    pos = np.array([128, 129, 130, 131, 139, 140, 150, 199], dtype=np.int32)
    clean = _latent(cache, q, pos=_ints(pos))
    if fp8:
        cache["c_scale"][131] = float("nan")
        cache["C"].view(torch.uint8)[140, 9] = 0x7f
    else:
        cache["C"][131, 100] = float("nan")
        cache["C"][140, 9] = float("inf")
    out, lse = _latent(cache, q, pos=_ints(pos))
    assert torch.equal(out[:3], clean[0][:3]) and torch.equal(lse[:3], clean[1][:3])
    assert lse[3:].isnan().all() and out[3:].isnan().all()


def test_large_scores_and_references_that_keep_rising():
    rng = np.random.default_rng(23)
    T, H, rows = 2, 16, 1500
    C = bf16(rng, rows, 576)
    q = bf16(rng, T, H, 576)
    C[:, 0] = torch.linspace(-300, 300, rows).bfloat16()       # scores climb along the row
    q[:, :, 0] = 8.0
    q[0, ::2, 0] = -8.0                                        # or fall
    cache = dict(C=C, c_scale=None, rope=None)
    pos = np.array([rows - 1, 700], dtype=np.int32)
    out, lse = _latent(cache, q, pos=_ints(pos))
    check_latent("rising", out, lse, q, f64(C), pos=pos)


def test_latent_offsets_past_32_bits():
    rows = (1 << 32) // 1152 + 100
    C = torch.zeros(rows, 576, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(4)
    tail = bf16(rng, 80, 576)
    C[rows - 80:] = tail.cuda()
    q = bf16(rng, 2, 16, 576)
    idx = np.stack([np.arange(rows - 80, rows), np.arange(rows - 1, rows - 81, -1)]).astype(np.int32)
    out, lse = S.latent_attention(q.cuda(), C, SM, idx=_ints(idx), with_lse=True)
    local = idx - (rows - 80)
    check_latent("far rows", out, lse, q, f64(tail), idx=local)
    base = np.full(2, rows - 80, dtype=np.int32)
    out, lse = S.latent_attention(q.cuda(), C, SM, pos=_ints([79, 40]), base=_ints(base), with_lse=True)
    check_latent("far prefix", out, lse, q, f64(tail), pos=np.array([79, 40]))


# ------------------------------------------------------------------ expanded

def _expanded(q, kv, rope, pos, base=None):
    return S.expanded_attention(q.cuda(), kv.cuda(), rope.cuda(), _ints(pos), SM, base=_ints(base), with_lse=True)


@pytest.mark.parametrize("T,H,L", [(1, 1, 1), (1, 3, 64), (5, 2, 65), (31, 1, 31), (32, 2, 200), (33, 1, 33), (127, 2, 127),
                                   (128, 1, 128), (129, 3, 129), (257, 2, 1000), (300, 1, 300), (64, 16, 700)])
def test_expanded_causal(T, H, L):
    rng = np.random.default_rng(T + L)
    q, kv, rope = bf16(rng, T, H, 192), bf16(rng, L, H, 256), bf16(rng, L, 64)
    pos = np.arange(L - T, L, dtype=np.int32) if L >= T else np.arange(T, dtype=np.int32)
    out, lse = _expanded(q, kv, rope, pos)
    only = sorted({0, 1, T // 2, T - 2, T - 1, 31, 32, 63, 64, 127, 128} & set(range(T)))
    check_expanded(f"T={T} L={L}", out, lse, q, kv, rope, pos, only=only)


def test_expanded_packed_sequences_padding_and_any_order():
    rng = np.random.default_rng(31)
    H, lens = 3, [1, 130, 64, 77]
    L = sum(lens)
    pos = np.concatenate([np.arange(n) for n in lens] + [[-1, -9, 5, 2 ** 31 - 1]]).astype(np.int32)
    base = np.concatenate([np.full(n, sum(lens[:i])) for i, n in enumerate(lens)] + [[0, 0, -1, 271]]).astype(np.int32)
    T = len(pos)
    q, kv, rope = bf16(rng, T, H, 192), bf16(rng, L, H, 256), bf16(rng, L, 64)
    out, lse = _expanded(q, kv, rope, pos, base)
    only = [0, 1, 2, 63, 64, 65, 127, 128, 129, 130, 131, 194, 195, 196, 270, T - 4, T - 3, T - 2, T - 1]
    check_expanded("packed", out, lse, q, kv, rope, pos, base, only=only)
    perm = rng.permutation(T)
    o2, l2 = _expanded(q[torch.from_numpy(perm)], kv, rope, pos[perm], base[perm])
    check_expanded("shuffled", o2, l2, q[torch.from_numpy(perm)], kv, rope, pos[perm], base[perm], only=range(0, T, 17))


def test_expanded_bad_keys_reach_the_queries_that_see_them_only():
    rng = np.random.default_rng(32)
    H, lens = 2, [70, 90, 40]
    L = sum(lens) + 30                                         # 30 rows of nobody behind the last sequence
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    base = np.concatenate([np.full(n, sum(lens[:i])) for i, n in enumerate(lens)]).astype(np.int32)
    T = len(pos)
    q, kv, rope = bf16(rng, T, H, 192), bf16(rng, L, H, 256), bf16(rng, L, 64)
    clean, zc = _expanded(q, kv, rope, pos, base)
    kv[200:] = float("nan")
    rope[200:] = float("inf")
    got = _expanded(q, kv, rope, pos, base)
    assert torch.equal(got[0], clean) and torch.equal(got[1], zc)
    kv[100, 1, 130] = float("nan")                             # a value of sequence 1, head 1
    kv[165, 0, 200] = float("-inf")                            # a value of sequence 2, head 0
    rope[20] = float("nan")                                    # a key of sequence 0
    out, lse = _expanded(q, kv, rope, pos, base)
    hit = torch.zeros(T, H, 128, dtype=torch.bool)
    hit[100:160, 1, 2] = True
    hit[165:200, 0, 72] = True
    hit[20:70] = True
    assert torch.equal(out.cpu()[~hit], clean.cpu()[~hit])
    assert out.cpu()[20:70].isnan().all() and out.cpu()[100:160, 1, 2].isnan().all()
    assert (out.cpu()[165:200, 0, 72] == float("-inf")).all()
    zhit = torch.zeros(T, H, dtype=torch.bool)
    zhit[20:70] = True
    assert torch.equal(lse.cpu()[~zhit], zc.cpu()[~zhit]) and lse.cpu()[zhit].isnan().all()


def test_expanded_strided_rotary_rows_and_long_context():
    rng = np.random.default_rng(33)
    T, H, L = 20, 2, 9000
    q, kv, rows = bf16(rng, T, H, 192), bf16(rng, L, H, 256), bf16(rng, L, 576)
    pos = np.arange(L - T, L, dtype=np.int32)
    rg = rows.cuda()
    out, lse = S.expanded_attention(q.cuda(), kv.cuda(), rg[:, 512:], _ints(pos), SM, with_lse=True)
    check_expanded("strided", out, lse, q, kv, rows[:, 512:], pos, only=[0, 7, 19])


def test_expanded_offsets_past_32_bits():
    H, L = 128, (1 << 32) // (128 * 512) + 200
    rng = np.random.default_rng(34)
    kv = torch.zeros(L, H, 256, dtype=torch.bfloat16, device="cuda")
    rope = torch.zeros(L, 64, dtype=torch.bfloat16, device="cuda")
    tk, tr = bf16(rng, 150, H, 256), bf16(rng, 150, 64)
    kv[L - 150:], rope[L - 150:] = tk.cuda(), tr.cuda()
    q = bf16(rng, 150, H, 192)
    pos, base = np.arange(150, dtype=np.int32), np.full(150, L - 150, dtype=np.int32)
    out, lse = S.expanded_attention(q.cuda(), kv, rope, _ints(pos), SM, base=_ints(base), with_lse=True)
    check_expanded("far", out, lse, q, tk, tr, pos, only=[0, 1, 75, 149])


# ------------------------------------------------------------------ calls

@pytest.mark.parametrize("form", ["lists", "prefix", "expanded"])
def test_same_bits_on_repeat_on_another_stream_and_without_lse(form):
    rng = np.random.default_rng(41)
    T, H, rows = 5, 16, 900
    cache, K = latent_cache(rng, rows, True)
    cache = gpu(cache)
    if form == "expanded":
        q = bf16(rng, T, H, 192).cuda()
        kv, rope = bf16(rng, rows, H, 256).cuda(), bf16(rng, rows, 64).cuda()
        pos = _ints(np.arange(rows - T, rows))
        call = lambda **kw: S.expanded_attention(q, kv, rope, pos, SM, **kw)  # noqa: E731
        width = 128
    else:
        q = bf16(rng, T, H, 576).cuda()
        kw0 = dict(idx=_ints(_lists(rng, T, rows, 500))) if form == "lists" else dict(pos=_ints([899, 800, 5, 0, 64]))
        call = lambda **kw: S.latent_attention(q, sm_scale=SM, **cache, **kw0, **kw)  # noqa: E731
        width = 512
    ref, z = call(with_lse=True)
    assert torch.equal(call(), ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, z2 = call(with_lse=True)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(z2, z)
    mine = torch.full((T, H, width), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")  # a workspace of NaN bytes
    got = call(out=mine, ws=ws)
    assert got is mine and torch.equal(mine, ref)
    assert bool((ws[-1024:] == 255).all())


@pytest.mark.parametrize("form", ["lists", "prefix", "expanded"])
def test_graph_replays_match_the_eager_call(form):
    rng = np.random.default_rng(42)
    T, H, rows = 3, 16, 700
    cache = gpu(latent_cache(rng, rows, True)[0])
    if form == "expanded":
        q = bf16(rng, T, H, 192).cuda()
        kv, rope = bf16(rng, rows, H, 256).cuda(), bf16(rng, rows, 64).cuda()
        ints = _ints(np.arange(rows - T, rows))
        call = lambda: S.expanded_attention(q, kv, rope, ints, SM, with_lse=True)  # noqa: E731
    else:
        q = bf16(rng, T, H, 576).cuda()
        ints = _ints(_lists(rng, T, rows, 300)) if form == "lists" else _ints([699, 3, 500])
        kw = dict(idx=ints) if form == "lists" else dict(pos=ints)
        call = lambda: S.latent_attention(q, sm_scale=SM, with_lse=True, **cache, **kw)  # noqa: E731
    ref = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = call()
    with torch.cuda.graph(g2):
        o2 = call()
    for i in range(4):
        for g, o in ((g1, o1), (g2, o2)):
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o[0], ref[0]) and torch.equal(o[1], ref[1]), i
        call()
        torch.cuda.synchronize()
    ints.zero_()                                               # new positions in the captured buffers
    g1.replay()
    want = call()
    torch.cuda.synchronize()
    assert torch.equal(o1[0], want[0]) and torch.equal(o1[1], want[1])


def test_empty_batch():
    C = torch.zeros(4, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(0, 16, 576, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out, lse = S.latent_attention(q, C, SM, pos=none, with_lse=True)
    assert tuple(out.shape) == (0, 16, 512) and tuple(lse.shape) == (0, 16)
    out = S.latent_attention(q, C, SM, idx=torch.empty(0, 5, dtype=torch.int32, device="cuda"))
    assert tuple(out.shape) == (0, 16, 512)
    kv = torch.zeros(4, 2, 256, dtype=torch.bfloat16, device="cuda")
    out = S.expanded_attention(torch.empty(0, 2, 192, dtype=torch.bfloat16, device="cuda"), kv, C[:, 512:], none, SM)
    assert tuple(out.shape) == (0, 2, 128)
