"""The cache, the selection and the attention together, as a serving step uses
them: keys and latents are coded as they are written, the block means are brought
up to date, MISA-dagger selects, and latent attention reads what was selected; and
a prompt whose latents are read back and expanded gives what the absorbed form
gives on the latents themselves."""
import numpy as np
import pytest
import torch

import oracle as O
from attention_parity import SM, bf16, check_latent, f64
from test_gpu_parity import check_hier

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparse_attention_indexer_block_amd")


def _coded(rows, d, dr):
    return dict(C=torch.zeros(rows, d, dtype=torch.float8_e4m3fn, device="cuda"),
                c_scale=torch.ones(rows, dtype=torch.float32, device="cuda"),
                rope=torch.zeros(rows, dr, dtype=torch.bfloat16, device="cuda") if dr else None)


def test_decode_steps_write_select_attend():
    rng = np.random.default_rng(7)
    L0, steps, T, H, HQ, B, A, kp, k = 900, 3, 1, 64, 16, 128, 8, 400, 130
    L = L0 + steps
    keys, lat = _coded(L, 128, 0), _coded(L, 512, 64)
    K, C = bf16(rng, L, 128), bf16(rng, L, 576)
    q, w, qa = bf16(rng, steps, H, 128), rng.standard_normal((steps, H)).astype(np.float32), bf16(rng, steps, HQ, 576)
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    S.cache_write(K[:L0].cuda(), ints(range(L0)), **keys)
    S.cache_write(C[:L0].cuda(), ints(range(L0)), **lat)
    kbar = torch.zeros((-(-L // B), 128), dtype=torch.float32, device="cuda")
    first = 0
    for i in range(steps):
        t = L0 + i
        S.cache_write(K[t:t + 1].cuda(), ints([t]), **keys)
        S.cache_write(C[t:t + 1].cuda(), ints([t]), **lat)
        n = t + 1
        M = -(-n // B)
        S.block_means_update(keys["C"][:n], B, kbar[:M], first, keys["c_scale"][:n])
        first = n // B
        pos = ints([t])
        idx, sc = S.hier_topk(q[i:i + 1].cuda(), torch.from_numpy(w[i:i + 1]).cuda(), keys["C"][:n], pos, B, A, kp, k,
                              keys["c_scale"][:n], kbar=kbar[:M])
        out, lse = S.latent_attention(qa[i:i + 1].cuda(), sm_scale=SM, idx=idx, with_lse=True, **lat)
        torch.cuda.synchronize()
        inp = dict(q=q[i:i + 1].view(torch.int16).numpy().view(np.uint16), w=w[i:i + 1],
                   K=keys["C"][:n].view(torch.uint8).cpu().numpy(), k_scale=keys["c_scale"][:n].cpu().numpy(),
                   pos=np.array([t], dtype=np.int32))
        check_hier(inp, B, A, kp, k, idx.cpu().numpy(), sc.cpu().numpy(), label=f"step {i}")
        rows = np.concatenate([O.decode_e4m3fn(lat["C"].view(torch.uint8).cpu().numpy()) *
                               lat["c_scale"].cpu().double().numpy()[:, None], f64(lat["rope"])], 1)
        check_latent(f"step {i}", out, lse, qa[i:i + 1], rows, idx=idx.cpu().numpy())


def test_expanded_prompt_equals_absorbed_prompt():
    # q_nope . (W_k c) = (W_k^T q_nope) . c and W_v sum p c = sum p (W_v c): the two forms agree up to the
    # roundings of the bf16 tensors between the steps (half a step 2^-8 each: the read rows are exact, the
    # expanded keys and values and the absorbed queries are rounded once, the weights and results once)
    rng = np.random.default_rng(8)
    T, H = 200, 4
    lat = _coded(T, 512, 64)
    x = bf16(rng, T, 576)
    slots = torch.from_numpy(rng.permutation(T).astype(np.int32)).cuda()
    S.cache_write(x.cuda(), slots, **lat)
    rows = S.cache_read(slots, **lat)                       # in the order of the tokens again
    wk = bf16(rng, H, 128, 512, scale=512 ** -0.5).cuda().float()
    wv = bf16(rng, H, 128, 512, scale=512 ** -0.5).cuda().float()
    q = bf16(rng, T, H, 192).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    c = rows[:, :512].float()
    kv = torch.cat([torch.matmul(c, wk.transpose(1, 2)).transpose(0, 1), torch.matmul(c, wv.transpose(1, 2)).transpose(0, 1)], 2)
    out = S.expanded_attention(q, kv.bfloat16().contiguous(), rows[:, 512:], pos, SM)
    qa = torch.cat([torch.matmul(q[:, :, :128].float().transpose(0, 1), wk).transpose(0, 1), q[:, :, 128:].float()], 2)
    # keys of token t are the rows slots[0..t] of the cache, as a list
    idx = torch.where(torch.arange(T, device="cuda")[None] <= pos[:, None], slots[None], -1).int().contiguous()
    low = S.latent_attention(qa.bfloat16().contiguous(), sm_scale=SM, idx=idx, **lat)
    absorbed = torch.matmul(low.float().transpose(0, 1), wv.transpose(1, 2)).transpose(0, 1)
    # bounds of the two sides' difference, from half steps b = 2^-8: scores (b sum|q||k| for the rounded keys,
    # b sum|qa||c| for the rounded queries), weights (twice that, and b each), values and results (b each)
    b = 2.0 ** -8
    qd, kd, vd = q.double(), kv[:, :, :128].double(), kv[:, :, 128:].double()
    s = torch.matmul(qd[:, :, :128].transpose(0, 1), kd.permute(1, 2, 0)) + \
        torch.matmul(qd[:, :, 128:].transpose(0, 1), rows[:, 512:].double().t()[None])
    seen = torch.arange(T, device="cuda")[None] <= pos[:, None]
    p = torch.softmax((s * SM).masked_fill(~seen, -float("inf")), 2)
    gk = torch.matmul(qd[:, :, :128].abs().transpose(0, 1), kd.abs().permute(1, 2, 0))
    ga = torch.matmul(qa[:, :, :512].double().abs().transpose(0, 1), rows[:, :512].double().abs().t()[None])
    ds = ((gk + ga) * (b * SM)).masked_fill(~seen, 0).amax(2, keepdim=True)          # [H, T, 1]
    spread = torch.matmul(p, vd.abs().transpose(0, 1))                               # sum p |v|
    lowmag = torch.matmul(torch.matmul(p, rows[:, :512].double().abs()), wv.double().abs().transpose(1, 2))
    tol = (torch.expm1(2 * ds) + 3 * b) * spread + 3 * b * lowmag
    diff = (out.double() - absorbed.double()).abs().transpose(0, 1)
    assert bool((diff <= tol).all()), float((diff / tol).max())
