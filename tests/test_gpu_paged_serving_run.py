"""A speculative serving step with every operator of the paged caches as it is used:
the layer's input is normed and coded, drafted tokens' latents and indexer keys are
appended to their pages, queries are rotated, MISA-dagger selects committed tokens, the
tree attends to them and to its own ancestors; then the accepted branch is moved to
where the next step looks for it."""
import numpy as np
import pytest
import torch

from attention_parity import HALF, SM, U, bf16, f64
from oracle.paged import norm_row, page_row
from paged_parity import check_codes, check_tree, ints, random_trees, rotation, tables, words

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")
EPS = 1e-6


def _coded(rows, d, dr):
    return dict(C=torch.zeros(rows, d, dtype=torch.float8_e4m3fn, device="cuda"), c_scale=torch.ones(rows, device="cuda"),
                rope=torch.zeros(rows, dr, dtype=torch.bfloat16, device="cuda") if dr else None)


def test_speculative_steps():
    rng = np.random.default_rng(21)
    seqs, N, H, HI, width, page, cap = 3, 6, 16, 32, 640, 16, 160
    per = cap // page
    table, pool = tables(rng, seqs, per)
    lat, keys = _coded(pool * page, 512, 64), _coded(seqs * cap, 128, 0)      # indexer keys: a sequence's pages in order
    order = np.arange(seqs * per).reshape(seqs, per)
    t, o, rot = ints(table), ints(order), rotation(cap).cuda()
    w_in, w_lat = bf16(rng, width).cuda(), (1 + 0.2 * bf16(rng, 512).float()).bfloat16().cuda()
    proj = lambda n: bf16(rng, width, n, scale=width ** -0.5).cuda().float()  # noqa: E731
    W_lat, W_key, W_q, W_qi = proj(576), proj(128), proj(H * 576), proj(HI * 128)
    residual = bf16(rng, seqs * N, width).cuda()

    def layer_input(x, residual):
        codes, scale, total = S.rms_norm(x, w_in, EPS, residual=residual, coded=True, group=128)
        return (codes.float() * scale.repeat_interleave(128, 1)), codes, scale, total

    def append(h, seq, pos, turn):
        S.paged_append((h @ W_lat).bfloat16(), seq, pos, t, page, weight=w_lat, eps=EPS, rot=rot, turn=turn, **lat)
        S.paged_append((h @ W_key).bfloat16(), seq, pos, o, page, rot=rot, turn=turn, **keys)

    # the prompts
    prefix = np.array([100, 37, 129])
    for s, n in enumerate(prefix):
        h = layer_input(bf16(rng, n, width).cuda(), torch.zeros(n, width, dtype=torch.bfloat16, device="cuda"))[0]
        append(h, ints([s] * n), ints(range(n)), None)
    for step in range(2):
        mask = random_trees(rng, seqs, N)
        depth = np.array([[bin(m[0]).count("1") - 1 for m in mask[s]] for s in range(seqs)])
        x = bf16(rng, seqs * N, width).cuda()
        before = residual.clone()
        h, codes, scale, residual = layer_input(x, residual)
        for i in (0, seqs * N - 1):                          # the norm against its formula
            want = norm_row(f64(x[i]) + f64(before[i]), f64(w_in), EPS)
            for g in range(5):
                c = slice(128 * g, 128 * g + 128)
                check_codes(f"norm {i}", codes[i].cpu().view(torch.uint8).numpy()[c], scale[i, g], want[c], 4 * U * np.abs(want[c]) + 2.0 ** -149)
        seq = np.repeat(np.arange(seqs), N)
        pos, turn = (prefix[:, None] + np.arange(N)).reshape(-1), (prefix[:, None] + depth).reshape(-1)
        append(h, ints(seq), ints(pos), ints(turn))
        q = (h @ W_q).bfloat16().view(seqs * N, H, 576)
        S.rotate(q[:, :, 512:], ints(turn), rot, out=q[:, :, 512:])
        # the selection of each sequence's committed keys
        qi, w = (h @ W_qi).bfloat16().view(seqs * N, HI, 128), torch.from_numpy(rng.standard_normal((seqs * N, HI)).astype(np.float32)).cuda()
        k, lists = 24, []
        for s, n in enumerate(prefix):
            mine, rows = slice(s * N, s * N + N), slice(s * cap, s * cap + n)
            lists.append(S.hier_topk(qi[mine].contiguous(), w[mine].contiguous(), keys["C"][rows], ints([n - 1] * N), 32, 8, 48, k,
                                     keys["c_scale"][rows])[0])
        idx = torch.stack(lists)
        assert bool((idx >= 0).all()) and bool((idx < ints(prefix)[:, None, None]).all())
        K = f64(S.cache_read(ints(range(pool * page)), **lat))                # (exact: scales are powers of two)
        q4, m = q.view(seqs, N, H, 576), words(mask)
        out, lse = S.tree_attention(q4, ints(prefix), t, page, sm_scale=SM, mask=m, idx=idx, with_lse=True, **lat)
        check_tree("selected", out, lse, q4.cpu(), K, table, page, prefix, mask=mask, idx=idx.cpu().numpy())
        out, lse = S.tree_attention(q4, ints(prefix), t, page, sm_scale=SM, mask=m, with_lse=True, **lat)
        check_tree("all committed", out, lse, q4.cpu(), K, table, page, prefix, mask=mask)
        # the deepest branch is accepted: its rows move up behind the committed ones
        for s in range(seqs):
            leaf = int(depth[s].argmax())
            path = [b for b in range(N) if mask[s][leaf][0] >> b & 1]
            for cache, tb in ((lat, table), (keys, order)):
                frm = [page_row(tb, page, cache["C"].shape[0], s, prefix[s] + b) for b in path]
                to = [page_row(tb, page, cache["C"].shape[0], s, prefix[s] + i) for i in range(len(path))]
                rows = S.cache_read(ints(frm), **cache)
                S.cache_write(rows, ints(to), **cache)
                assert torch.equal(S.cache_read(ints(to), **cache), rows)     # the same values, whatever the scale
            prefix[s] += len(path)


def test_turned_keys_meet_turned_queries():
    # a key and a query of equal content score by the distance of their positions alone, to within the roundings of
    # the two rotated rows (half a step of each value, and the table's)
    rng = np.random.default_rng(22)
    n, page = 64, 16
    table = np.arange(8, dtype=np.int32)[None]
    rot = rotation(4096).cuda()
    x, qr = bf16(rng, 1, 576), bf16(rng, 1, 1, 64)
    x[:, :512] = 0
    lses = []
    for shift in (0, 1000, 4000):
        C = torch.zeros(8 * page, 576, dtype=torch.bfloat16, device="cuda")
        S.paged_append(x.cuda(), ints([0]), ints([0]), ints(table), page, C, rot=rot, turn=ints([5 + shift]))
        q = torch.zeros(1, 1, 1, 576, dtype=torch.bfloat16, device="cuda")
        S.rotate(qr.cuda(), ints([17 + shift]), rot, out=q.view(1, 1, 576)[:, :, 512:])
        lses.append(float(S.tree_attention(q, ints([0]), ints(table), page, C, 1.0, with_lse=True)[1]))
    bound = 1.01 * (2 * HALF + 2 ** -20) * 2 * float(x[:, 512:].double().norm() * qr.double().norm())
    assert max(lses) - min(lses) <= 2 * bound, (lses, bound)
