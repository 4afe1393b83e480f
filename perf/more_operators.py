"""What is measured of the operators of a serving step over paged caches: the
norm that makes a layer's input (residual added, result coded), rows appended
to a paged cache (normed, rotated and coded on the way), the rotation of
queries, and latent attention of drafted tokens over such a cache.

run() computes each operator in its plain form (elementary torch operations in
32 bits; sums of squares, of which the coded values' scales depend, in 64), or
through the package's entry points when `own` is set. exact() computes the same
from the definitions in 64 bits.

Shapes: a latent row is 512 values followed by 64 rotary ones, an indexer key
128 values of which the first 64 are rotary. An 8-bit cache holds E4M3FN codes
with one power-of-two scale a row, and latents' rotary values in bf16. Position
j of sequence s lies in row table[s, j // page] * page + j % page of the cache.
"""
import math
import random

import torch

own = False

LATENT, ROTARY, KEY = 512, 64, 128
SM_SCALE = (128 + ROTARY) ** -0.5
EPS = 1e-6


# --------------------------------------------------------------------- cases

def listed():
    return [
        # the input of a layer of a decode batch, residual added, one scale a row: latency
        dict(name="norm_decode", op="norm", n=8, width=4096, residual=True, out="row"),
        # the same of a prompt, a scale for each 128 columns: bandwidth
        dict(name="norm_prefill", op="norm", n=16384, width=4096, residual=True, out="group"),
        # latents out of a wider projection (strided rows), an odd count, bf16 result
        dict(name="norm_latents", op="norm", n=5001, width=512, residual=False, out="bf16"),
        # a decode step of 32 sequences appends a latent each, normed, rotated and coded: latency
        dict(name="append_decode", op="append", kind="latent", seqs=32, new=1, page=64, fp8=True),
        # three prompts' latents to an 8-bit cache: bandwidth
        dict(name="append_prefill", op="append", kind="latent", seqs=3, new=5461, page=64, fp8=True),
        # indexer keys of five chunks of odd length to small pages, some tokens padding
        dict(name="append_keys", op="append", kind="key", seqs=5, new=1003, page=16, fp8=True),
        # queries of a drafted batch, every head
        dict(name="rotate_drafts", op="rotate", T=64, H=128, pairs=False),
        # queries of a prompt, neighbouring values paired
        dict(name="rotate_prefill", op="rotate", T=8192, H=64, pairs=True),
        # one token of one sequence, the 16 heads of one GPU out of several: latency
        dict(name="tree_one", op="tree", S=1, N=1, H=16, L=8191, k=0, page=64, fp8=True, tree=False, ragged=False),
        # a batch of drafted chains over contexts of different lengths, every head, 8-bit pages
        dict(name="tree_batch", op="tree", S=24, N=4, H=128, L=8000, k=0, page=64, fp8=True, tree=False, ragged=True),
        # trees of drafted tokens whose queries see a selection of the context and their ancestors
        dict(name="tree_selected", op="tree", S=8, N=7, H=64, L=32768, k=2048, page=64, fp8=True, tree=True, ragged=True),
        # two large trees over a long context: products
        dict(name="tree_large", op="tree", S=2, N=64, H=128, L=32000, k=0, page=16, fp8=False, tree=True, ragged=False),
    ]


def _spread(rng, lo, hi):
    """A whole number, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "rotate", "tree", "tree", "tree"])
    if op == "norm":
        width = 8 * _spread(rng, 8, 1024)
        return dict(op=op, n=_spread(rng, 1, min(16384, (1 << 26) // width)), width=width, residual=rng.random() < 0.6,
                    out=rng.choice(["bf16", "row", "group"]))
    if op == "append":
        seqs = _spread(rng, 1, 64)
        return dict(op=op, kind=rng.choice(["latent", "key"]), seqs=seqs, new=_spread(rng, 1, max(1, 16384 // seqs)),
                    page=rng.choice([1, 16, 32, 64, 128]), fp8=rng.random() < 0.7)
    if op == "rotate":
        H = rng.choice([1, 5, 8, 16, 20, 32, 64, 128])
        return dict(op=op, T=_spread(rng, 1, min(8192, (1 << 19) // H)), H=H, pairs=rng.random() < 0.5)
    H = rng.choice([1, 5, 8, 16, 20, 32, 40, 64, 128])
    S = _spread(rng, 1, 32)
    lists = rng.random() < 0.3
    L = _spread(rng, 1, 32768 if S <= 8 else 8192)
    k = _spread(rng, 1, 2048) if lists else 0
    most = 1.0e8  # rows times keys; the largest listed case has 5.2e8
    N = _spread(rng, 1, max(1, min(64, int(most / (S * H * (k + 64 if lists else L + 64))))))
    return dict(op=op, S=S, N=N, H=H, L=L, k=k, page=rng.choice([1, 16, 64, 128]), fp8=rng.random() < 0.5,
                tree=rng.random() < 0.6, ragged=rng.random() < 0.6)


# -------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rows_like(g, n, width):
    """Rows as a projection leaves them: a few columns that stand out, rows of differing size."""
    x = _normal(g, n, width)
    x *= torch.exp(0.4 * _normal(g, 1, width))
    return x * torch.exp(0.5 * _normal(g, n, 1))


def _rotation(positions):
    """Cosines and sines [positions, 32 + 32] of the rotary angles, which are formed in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, ROTARY, 2, device="cuda", dtype=torch.float64) / ROTARY)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


def _row_scale(x):
    """The smallest power of two (from 2^-126) that brings each row within 448, put together from its exponent; 1 for zeros."""
    top = x.abs().amax(-1)
    mant, ex = torch.frexp(top)
    ex = (ex - 9 + (mant > 0.875).int()).clamp(min=-126)
    return torch.where(top > 0, ((ex + 127) << 23).view(torch.float32), torch.ones_like(top))


def _cache(g, rows, kind, fp8):
    """A filled cache: {"C", "c_scale", "rope"}, with a spare row behind the last in the tensors of "spare"."""
    d, dr = (LATENT, ROTARY) if kind == "latent" else (KEY, 0)
    if not fp8:
        spare = dict(C=_normal(g, rows + 1, d + dr).bfloat16())
        return dict(C=spare["C"][:rows], c_scale=None, rope=None, spare=spare)
    x = _rows_like(g, rows + 1, d)
    scale = _row_scale(x)
    spare = dict(C=(x / scale[:, None]).to(torch.float8_e4m3fn), c_scale=scale,
                 rope=_normal(g, rows + 1, dr).bfloat16() if dr else None)
    return dict(C=spare["C"][:rows], c_scale=scale[:rows], rope=spare["rope"][:rows] if dr else None, spare=spare)


def _table(g, seqs, per):
    """Pages of the sequences, in any order, out of a pool with some to spare: table [seqs, per], pages of the pool."""
    pool = seqs * per + 3
    return torch.randperm(pool, generator=g, device="cuda")[:seqs * per].to(torch.int32).view(seqs, per), pool


def _lengths(case):
    """Committed tokens of each sequence."""
    cut = case["L"] * 3 // 4
    return [case["L"] - ((s * 40503 + 977) % (cut + 1) if case["ragged"] else 0) for s in range(case["S"])]


def _live(case, s):
    """Nodes of sequence s that are not padding."""
    return max(1, case["N"] - s % 3) if case["tree"] and case["ragged"] else case["N"]


def _trees(case, seed):
    """Masks [S, N] of the drafted nodes: itself and its ancestors; 0 for padding."""
    r, rows = random.Random(seed), []
    for s in range(case["S"]):
        mine = []
        for j in range(_live(case, s)):
            up = r.randint(-1, j - 1) if j else -1
            mine.append((mine[up] if up >= 0 else 0) | 1 << j)
        rows.append(mine + [0] * (case["N"] - len(mine)))
    return torch.tensor([[m - (1 << 64) if m >> 63 else m for m in row] for row in rows], dtype=torch.int64, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    st = dict(op=case["op"])
    if case["op"] == "norm":
        n, width = case["n"], case["width"]
        # one part of a wider projection's rows where there is no residual
        x = _rows_like(g, n, width if case["residual"] else width + ROTARY).bfloat16()
        st["x"] = x[:, :width]
        st["residual"] = _rows_like(g, n, width).bfloat16() if case["residual"] else None
        st["weight"] = (1.0 + 0.2 * _normal(g, width)).bfloat16()
        st["out"] = case["out"]
    elif case["op"] == "append":
        latent = case["kind"] == "latent"
        d, dr = (LATENT, ROTARY) if latent else (KEY, 0)
        seqs, new, page = case["seqs"], case["new"], case["page"]
        before = 512  # tokens that each sequence may have already
        per = -(-(before + new) // page)
        st["table"], pool = _table(g, seqs, per)
        st |= _cache(g, pool * page, case["kind"], case["fp8"])
        st["page"] = page
        st["x"] = _rows_like(g, seqs * new, d + dr).bfloat16()
        st["seq"] = torch.arange(seqs, device="cuda", dtype=torch.int32).repeat_interleave(new)
        first = torch.randint(0, before, (seqs, 1), generator=g, device="cuda", dtype=torch.int32)
        st["pos"] = (first + torch.arange(new, device="cuda", dtype=torch.int32)).view(-1)
        if not latent:  # every 50th token is padding
            st["pos"][torch.arange(seqs * new, device="cuda") % 50 == 49] = -1
        st["rot"] = _rotation(before + new)
        st["weight"] = (1.0 + 0.2 * _normal(g, d)).bfloat16() if latent else None
    elif case["op"] == "rotate":
        T, H = case["T"], case["H"]
        # the rotary columns of a query projection, to where the attention reads them
        st["x"] = _normal(g, T, H, 128 + ROTARY).bfloat16()[:, :, 128:]
        st["q"] = torch.zeros(T, H, LATENT + ROTARY, dtype=torch.bfloat16, device="cuda")
        st["pos"] = torch.randint(0, 16384, (T,), generator=g, device="cuda", dtype=torch.int32)
        st["rot"] = _rotation(16384)
        st["pairs"] = case["pairs"]
    else:
        S, N, H, page = case["S"], case["N"], case["H"], case["page"]
        per = -(-(case["L"] + N) // page)
        st["table"], pool = _table(g, S, per)
        st |= _cache(g, pool * page, "latent", case["fp8"])
        st["page"], st["longest"] = page, case["L"]
        st["q"] = _normal(g, S, N, H, LATENT + ROTARY).bfloat16()
        st["prefix"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        st["mask"] = _trees(case, seed) if case["tree"] else None
        st["idx"] = None
        if case["k"]:
            # up to k distinct committed positions of each query in ascending order, then -1
            k = case["k"]
            n = st["prefix"].long()[:, None, None]
            j = torch.arange(k, device="cuda")[None, None, :]
            step = (n // k).clamp(min=1)
            idx = j * step + torch.randint(0, 1 << 30, (S, N, k), generator=g, device="cuda") % step
            st["idx"] = torch.where((j < n) & (idx < n), idx, torch.full_like(idx, -1)).to(torch.int32).contiguous()
    return st


# ----------------------------------------------------------- the plain forms

def _plain_norm(h, weight):
    """h in 32 bits, normed; the mean square in 64, so that the coded rows' scales do not depend on the order of a sum."""
    r = (1.0 / torch.sqrt(h.double().square().mean(1, keepdim=True) + EPS)).float()
    return (h * r) * weight.float()


def _plain_norm_call(st):
    h = st["x"].float()
    res = {}
    if st["residual"] is not None:
        h = h + st["residual"].float()
        res["sum"] = h.bfloat16()
    y = _plain_norm(h, st["weight"])
    if st["out"] == "bf16":
        return res | {"y": y.bfloat16()}
    n, width = y.shape
    if st["out"] == "group":
        groups = -(-width // 128)
        wide = torch.nn.functional.pad(y, (0, groups * 128 - width)).view(n, groups, 128)
        scale = _row_scale(wide)
        codes = (wide / scale[:, :, None]).to(torch.float8_e4m3fn).view(n, groups * 128)[:, :width]
        return res | {"codes": codes.contiguous(), "scale": scale}
    scale = _row_scale(y)
    return res | {"codes": (y / scale[:, None]).to(torch.float8_e4m3fn), "scale": scale}


def _plain_rotation(x, at, rot, pairs):
    """The 64 values of x [T, 64] or [T, H, 64] rotated by the angles of positions `at` [T]."""
    x = x.float()
    cs = rot[at] if x.dim() == 2 else rot[at].unsqueeze(1)
    cos, sin = cs[..., :32], cs[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :32], x[..., 32:])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)


def _rows_of(st, seq, pos, rows):
    """Cache rows of positions; the spare row (index `rows`) where there is no position."""
    at = st["table"].long()[seq.long(), (pos.clamp(min=0) // st["page"]).long()] * st["page"] + pos % st["page"]
    return torch.where(pos < 0, torch.full_like(at, rows), at)


def _plain_append(st):
    spare, at = st["spare"], _rows_of(st, st["seq"], st["pos"], st["C"].shape[0])
    when = st["pos"].clamp(min=0).long()
    x = st["x"].float()
    if st["weight"] is not None:
        lat = _plain_norm(x[:, :LATENT], st["weight"])
        rot = _plain_rotation(x[:, LATENT:], when, st["rot"], False)
    else:
        lat = torch.cat([_plain_rotation(x[:, :ROTARY], when, st["rot"], False), x[:, ROTARY:]], 1)
        rot = None
    if st["c_scale"] is None:
        spare["C"][at] = (lat if rot is None else torch.cat([lat, rot], 1)).bfloat16()
        return
    scale = _row_scale(lat)
    spare["C"].view(torch.uint8)[at] = (lat / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    spare["c_scale"][at] = scale
    if rot is not None:
        spare["rope"][at] = rot.bfloat16()


def _plain_softmax(s, seen):
    """Weights and log-sum of each row over the keys it sees; zeros and -inf where it sees none."""
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total)), (top + torch.log(total)).squeeze(-1)


def _plain_rows(st, at):
    """Rows `at` of the latent cache in fp32."""
    if st["c_scale"] is None:
        return st["C"][at].float()
    codes = st["C"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    return torch.cat([codes * st["c_scale"][at][..., None], st["rope"][at].float()], -1)


def _masks(st):
    """[S, N, N]: whether node i sees node j, and [S, N]: whether node i is none of the padding."""
    S, N = st["q"].shape[:2]
    j = torch.arange(N, device=st["q"].device)
    if st["mask"] is None:
        return (j[None, :] <= j[:, None]).expand(S, N, N), torch.ones(S, N, dtype=torch.bool, device=j.device)
    return ((st["mask"][:, :, None] >> j) & 1).bool(), st["mask"] != 0


def _plain_tree(st):
    S, N, H, W = st["q"].shape
    page, n = st["page"], st["prefix"].long()
    nodes, live = _masks(st)
    at = lambda s, j: st["table"].long()[s, j // page] * page + j % page  # noqa: E731
    s_of = torch.arange(S, device=n.device)[:, None]
    drafted = at(s_of, n[:, None] + torch.arange(N, device=n.device))           # [S, N]
    q = st["q"].float()
    if st["idx"] is not None:
        idx = st["idx"].long()
        k = idx.shape[2]
        rows = torch.cat([at(s_of[:, :, None], idx.clamp(min=0)), drafted[:, None, :].expand(S, N, N)], 2)
        keys = _plain_rows(st, rows.view(S * N, k + N))
        seen = torch.cat([(idx >= 0) & live[:, :, None], nodes], 2).view(S * N, 1, k + N)
        s = torch.matmul(q.view(S * N, H, W), keys.transpose(1, 2)) * SM_SCALE
        p, lse = _plain_softmax(s, seen)
        return torch.matmul(p, keys[:, :, :LATENT]).bfloat16().view(S, N, H, LATENT), lse.view(S, N, H)
    L = st["longest"]
    j = torch.arange(L, device=n.device)[None, :].expand(S, L)
    keys = _plain_rows(st, torch.cat([at(s_of, j), drafted], 1))               # [S, L + N, 576]
    seen = torch.cat([(j < n[:, None])[:, None, :] & live[:, :, None], nodes], 2)
    s = (torch.matmul(q.view(S, N * H, W), keys.transpose(1, 2)) * SM_SCALE).view(S, N, H, L + N)
    p, lse = _plain_softmax(s, seen[:, :, None, :])
    out = torch.matmul(p.view(S, N * H, L + N), keys[:, :, :LATENT])
    return out.view(S, N, H, LATENT).bfloat16(), lse


# ------------------------------------------------------------------ one pass

def run(state):
    st = state
    cache = dict(C=st["C"], c_scale=st["c_scale"], rope=st["rope"]) if "C" in st else None
    if own:
        import sparse_attention_indexer_block_amd as S
        if st["op"] == "norm":
            got = S.rms_norm(st["x"], st["weight"], EPS, residual=st["residual"], coded=st["out"] != "bf16",
                             group=128 if st["out"] == "group" else 0)
            got = got if isinstance(got, tuple) else (got,)
            names = ("y",) if st["out"] == "bf16" else ("codes", "scale")
            return dict(zip(names + ("sum",), got))
        if st["op"] == "append":
            S.paged_append(st["x"], st["seq"], st["pos"], st["table"], st["page"], **cache, weight=st["weight"], eps=EPS,
                           rot=st["rot"])
        elif st["op"] == "rotate":
            S.rotate(st["x"], st["pos"], st["rot"], pairs=st["pairs"], out=st["q"][:, :, LATENT:])
        else:
            out, lse = S.tree_attention(st["q"], st["prefix"], st["table"], st["page"], sm_scale=SM_SCALE, **cache,
                                        mask=st["mask"], idx=st["idx"], longest=st["longest"], with_lse=True)
            return {"out": out, "lse": lse}
    else:
        if st["op"] == "norm":
            return _plain_norm_call(st)
        if st["op"] == "append":
            _plain_append(st)
        elif st["op"] == "rotate":
            st["q"][:, :, LATENT:] = _plain_rotation(st["x"], st["pos"].long(), st["rot"], st["pairs"]).bfloat16()
        else:
            out, lse = _plain_tree(st)
            return {"out": out, "lse": lse}
    if st["op"] == "rotate":
        return st["q"]
    return {n: t for n, t in (("rows", st["C"]), ("scale", st["c_scale"]), ("rope", st["rope"])) if t is not None}


# ---------------------------------------------------------------------- work

def work(case):
    if case["op"] == "norm":
        values = case["n"] * case["width"]
        coded = case["out"] != "bf16"
        scales = case["n"] * (-(-case["width"] // 128) if case["out"] == "group" else 1) if coded else 0
        return {"bytes": values * (2 + (4 if case["residual"] else 0) + (1 if coded else 2)) + 4 * scales + 2 * case["width"],
                "flops": 4 * values}
    if case["op"] == "append":
        d, dr = (LATENT, ROTARY) if case["kind"] == "latent" else (KEY, 0)
        n = case["seqs"] * case["new"]
        held = d + 4 + 2 * dr if case["fp8"] else 2 * (d + dr)
        return {"bytes": n * (2 * (d + dr) + held + 8 + 4 * ROTARY), "flops": n * (4 * d + 3 * ROTARY)}
    if case["op"] == "rotate":
        return {"bytes": case["T"] * (case["H"] * 4 * ROTARY + 4 + 4 * ROTARY), "flops": 3 * case["T"] * case["H"] * ROTARY}
    S, N, H = case["S"], case["N"], case["H"]
    row = LATENT + 4 + 2 * ROTARY if case["fp8"] else 2 * (LATENT + ROTARY)
    pairs = touched = 0
    for s, n in enumerate(_lengths(case)):
        nodes = _live(case, s)
        among = sum(sum(1.0 / i for i in range(1, j + 1)) for j in range(1, nodes + 1)) if case["tree"] else nodes * (nodes + 1) / 2
        mine = min(n, case["k"]) if case["k"] else n
        pairs += nodes * mine + among
        touched += min(n, nodes * mine) + nodes
    return {"bytes": touched * row + 4 * S * N * case["k"] + S * N * H * (2 * (LATENT + ROTARY) + 2 * LATENT + 4),
            "flops": 2 * pairs * H * (LATENT + ROTARY + LATENT)}


# --------------------------------------------------------------------- exact

def _two_to(e):
    """2 to the whole numbers e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(v):
    """The nearest value of E4M3FN, ties to the even code, of 64-bit values of at most 448."""
    a = v.abs()
    step = _two_to(torch.frexp(a.clamp(min=2.0 ** -6)).exponent - 4)
    return torch.sign(v) * torch.round(a / step) * step


def _wide_code(v):
    """Code values and scale of the last dimension's values, in 64 bits."""
    amax = v.abs().amax(-1)
    part, e = torch.frexp(amax / 448.0)
    e = torch.where(part == 0.5, e - 1, e).clamp(min=-126)
    s = torch.where(amax > 0, _two_to(e), torch.ones_like(amax))
    return _e4m3(v / s.unsqueeze(-1)), s


def _wide_norm(h, weight):
    ms = torch.einsum("ij,ij->i", h, h) / h.shape[1]
    return h / torch.sqrt(ms + EPS).unsqueeze(1) * weight.to(torch.float64)


def _wide_turn(x, rot, pairs):
    """Values x [..., 64] as 32 complex numbers times e^(i angle); rot [..., 64] in 64 bits."""
    turn = torch.complex(rot[..., :32], rot[..., 32:])
    if pairs:
        z = torch.view_as_complex(x.reshape(*x.shape[:-1], 32, 2).contiguous()) * turn
        return torch.view_as_real(z).reshape(x.shape)
    z = torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous()) * turn
    return torch.cat((z.real, z.imag), -1)


def exact(case, seed):
    st = prepare(case, seed)
    wide = torch.float64
    if case["op"] == "norm":
        h = st["x"].to(wide)
        res = {}
        if st["residual"] is not None:
            h = h + st["residual"].to(wide)
            res["sum"] = h
        y = _wide_norm(h, st["weight"])
        if case["out"] == "bf16":
            return {"y": y, **res}
        if case["out"] == "row":
            codes, scale = _wide_code(y)
            return {"codes": codes, "scale": scale, **res}
        parts = [_wide_code(y[:, c:c + 128]) for c in range(0, case["width"], 128)]
        return {"codes": torch.cat([c for c, _ in parts], 1), "scale": torch.stack([s for _, s in parts], 1), **res}
    if case["op"] == "rotate":
        out = st["q"].to(wide)
        out[:, :, LATENT:] = _wide_turn(st["x"].to(wide), st["rot"].to(wide)[st["pos"].long()].unsqueeze(1), case["pairs"])
        return out
    if case["op"] == "append":
        rows = st["C"].to(wide)
        keep = torch.nonzero(st["pos"] >= 0).flatten()
        pos, seq = st["pos"][keep].long(), st["seq"][keep].long()
        to = st["table"].long()[seq, torch.div(pos, case["page"], rounding_mode="floor")] * case["page"] + pos % case["page"]
        x, rot = st["x"][keep].to(wide), st["rot"].to(wide)[pos]
        if case["kind"] == "latent":
            main, turned = _wide_norm(x[:, :LATENT], st["weight"]), _wide_turn(x[:, LATENT:], rot, False)
        else:
            main, turned = torch.cat((_wide_turn(x[:, :ROTARY], rot, False), x[:, ROTARY:]), 1), x[:, :0]
        if not case["fp8"]:
            rows[to] = torch.cat((main, turned), 1)
            return {"rows": rows}
        codes, s = _wide_code(main)
        scale = st["c_scale"].to(wide)
        rows[to], scale[to] = codes, s
        if case["kind"] != "latent":
            return {"rows": rows, "scale": scale}
        rope = st["rope"].to(wide)
        rope[to] = turned
        return {"rows": rows, "scale": scale, "rope": rope}
    S, N, H = case["S"], case["N"], case["H"]
    out = torch.zeros(S, N, H, LATENT, dtype=wide, device="cuda")
    lse = torch.full((S, N, H), -math.inf, dtype=wide, device="cuda")
    table, lengths = st["table"].long(), _lengths(case)
    trees = _trees(case, seed).tolist() if case["tree"] else [[(2 << i) - 1 for i in range(N)]] * S

    def rows_at(s, where):  # 64-bit rows of positions of sequence s
        at = table[s, torch.div(where, case["page"], rounding_mode="floor")] * case["page"] + where % case["page"]
        if not case["fp8"]:
            return st["C"][at].to(wide)
        c = st["C"].view(torch.uint8)[at].view(torch.float8_e4m3fn).to(wide) * st["c_scale"][at].to(wide).unsqueeze(1)
        return torch.cat((c, st["rope"][at].to(wide)), 1)

    for s in range(S):
        if not case["k"]:
            before = rows_at(s, torch.arange(lengths[s], device="cuda"))
        drafted = rows_at(s, torch.arange(lengths[s], lengths[s] + N, device="cuda"))
        for i in range(N):  # one node at a time, over exactly the keys that it has
            bits = [j for j in range(N) if trees[s][i] >> j & 1]
            if not bits:
                continue
            mine = before if not case["k"] else rows_at(s, st["idx"][s, i][st["idx"][s, i] >= 0].long())
            q = st["q"][s, i].to(wide)
            ends = drafted[torch.tensor(bits, device="cuda")]
            a = torch.cat((torch.mm(q, mine.t()), torch.mm(q, ends.t())), 1) * SM_SCALE
            z = torch.logsumexp(a, 1)
            p = torch.exp(a - z.unsqueeze(1))
            lse[s, i] = z
            out[s, i] = torch.mm(p[:, :mine.shape[0]], mine[:, :LATENT]) + torch.mm(p[:, mine.shape[0]:], ends[:, :LATENT])
    return {"out": out, "lse": lse}
