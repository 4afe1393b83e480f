"""What is measured of the operators that serve latent attention: the two
that keep its caches (rows quantised as they are written, and read back) and
the two forms of the attention that reads them (absorbed, over one shared
latent vector a token; expanded, over per-head keys and values).

run() computes each operator in its plain form (elementary torch operations in
32 bits), or through the package's entry points when `own` is set. exact()
computes the same from the definitions in 64 bits.

Shapes: a latent row is 512 values followed by 64 rotary ones, an indexer key
128 values. An 8-bit cache holds E4M3FN codes with one power-of-two scale a
row, and the rotary values in bf16.
"""
import math

import torch

own = False

LATENT, ROTARY, KEY, NOPE, VALUE = 512, 64, 128, 128, 128
SM_SCALE = (NOPE + ROTARY) ** -0.5


# --------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 8 sequences appends one latent row each to an 8-bit cache: latency
        dict(name="write_decode", op="write", kind="latent", n=8, rows=16384, holes=1),
        # the prompt of a 16K prefill goes to the 8-bit latent cache at once: bandwidth
        dict(name="write_prefill", op="write", kind="latent", n=16384, rows=16384, holes=0),
        # indexer keys of a padded chunk: odd count, slots that hold no token
        dict(name="write_keys", op="write", kind="key", n=5001, rows=8192, holes=37),
        # the latents of one selection, for a reader that wants them in bf16
        dict(name="read_selection", op="read", kind="latent", n=2048, rows=32768, holes=9),
        # a whole 128K context read back before it is expanded into keys and values
        dict(name="read_context", op="read", kind="latent", n=131072, rows=131072, holes=0),
        # one token of one sequence, the 16 heads of one GPU out of several, selected keys: latency
        dict(name="latent_one", op="latent", T=1, H=16, L=32768, k=2048, fp8=True, lists=True, seqs=1),
        # a decode batch of 32 sequences with every head, selected keys of each sequence
        dict(name="latent_batch", op="latent", T=32, H=128, L=131072, k=2048, fp8=True, lists=True, seqs=32),
        # four draft tokens over a long context without a selection, odd length
        dict(name="latent_dense", op="latent", T=4, H=32, L=100003, k=0, fp8=False, lists=False, seqs=1),
        # a prefill chunk of a sparse layer: every query its own 2048 keys
        dict(name="latent_prefill", op="latent", T=2048, H=128, L=16384, k=2048, fp8=False, lists=True, seqs=1),
        # the prompt in expanded form, causal
        dict(name="expanded_prefill", op="expanded", T=8192, H=16, L=8192, seqs=1),
        # three packed prompts of odd lengths, with padded rows behind the last
        dict(name="expanded_packed", op="expanded", T=2987, H=5, L=2981, seqs=3),
        # the last chunk of a chunked prefill: few queries, long context
        dict(name="expanded_chunk", op="expanded", T=100, H=16, L=32768, seqs=1),
    ]


def _spread(rng, lo, hi):
    """A whole number, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "latent", "latent", "expanded", "expanded"])
    if op in ("write", "read"):
        n = _spread(rng, 1, 16384 if op == "write" else 131072)
        return dict(op=op, kind=rng.choice(["latent", "key"]), n=n, rows=n + _spread(rng, 8, 16384),
                    holes=rng.randint(0, n // 8))
    if op == "latent":
        lists = rng.random() < 0.7
        H = rng.choice([1, 5, 8, 16, 20, 32, 40, 64, 128])
        L = _spread(rng, 1, 65536)
        k = _spread(rng, 1, 2048) if lists else 0
        most = 2.0e8  # rows times keys; the largest listed case has 5.4e8
        T = _spread(rng, 1, max(1, min(1024, int(most / (H * (k or L))))))
        return dict(op=op, T=T, H=H, L=L, k=k, fp8=rng.random() < 0.5, lists=lists,
                    seqs=rng.choice([1, 1, min(T, 4)]))
    H = rng.choice([1, 3, 8, 16, 20])
    L = _spread(rng, 1, 16384)
    T = _spread(rng, 1, max(1, min(4096, int(5.0e8 / (H * L)))))
    return dict(op=op, T=T, H=H, L=L, seqs=rng.choice([1, 1, min(3, T, L)]))


# -------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rows_like(g, n, width):
    """Rows as a norm leaves them: unit values, a few columns that stand out, rows of differing size."""
    x = _normal(g, n, width)
    x *= torch.exp(0.4 * _normal(g, 1, width))
    return x * torch.exp(0.5 * _normal(g, n, 1))


def _slots(g, n, rows, holes):
    """Distinct rows in random order; `holes` of the entries name no row."""
    s = torch.randperm(rows, generator=g, device="cuda")[:n].to(torch.int32)
    if holes:
        s[torch.randperm(n, generator=g, device="cuda")[:holes]] = -1
    return s


def _row_scale(x):
    """The smallest power of two (from 2^-126) that brings each row within 448, put together from its exponent."""
    mant, ex = torch.frexp(x.abs().amax(1))
    ex = (ex - 9 + (mant > 0.875).int()).clamp(min=-126)
    return ((ex + 127) << 23).view(torch.float32)


def _coded(x):
    """Codes and scales of rows x, for a cache that is already there."""
    scale = _row_scale(x)
    return (x / scale[:, None]).to(torch.float8_e4m3fn), scale


def _cache(g, rows, kind, fp8):
    """A filled cache: {"C", "c_scale", "rope"}; bf16 rows are latent and rotary values side by side."""
    d, dr = (LATENT, ROTARY) if kind == "latent" else (KEY, 0)
    if not fp8:
        return dict(C=_normal(g, rows, d + dr).bfloat16(), c_scale=None, rope=None)
    # one spare row behind the last, so that a plain scatter has a place for rows without a slot
    codes, scale = _coded(_rows_like(g, rows + 1, d).bfloat16().float())
    rope = _normal(g, rows + 1, dr).bfloat16() if dr else None
    spare = dict(C=codes, c_scale=scale, rope=rope)
    return dict(C=codes[:rows], c_scale=scale[:rows], rope=None if rope is None else rope[:rows], spare=spare)


def _spans(T, L, seqs):
    """Query rows and keys of `seqs` sequences side by side: [(first row, rows, first key, keys)]."""
    cut = lambda n: [n * i // seqs for i in range(seqs + 1)]  # noqa: E731
    t, s = cut(T), cut(L)
    return [(t[i], t[i + 1] - t[i], s[i], s[i + 1] - s[i]) for i in range(seqs)]


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("write", "read"):
        d, dr = (LATENT, ROTARY) if case["kind"] == "latent" else (KEY, 0)
        st = _cache(g, case["rows"], case["kind"], True)
        st["slots"] = _slots(g, case["n"], case["rows"], case["holes"])
        if case["op"] == "write":
            st["x"] = _rows_like(g, case["n"], d + dr).bfloat16()
        st["op"] = case["op"]
        return st
    T, H, L = case["T"], case["H"], case["L"]
    st = dict(op=case["op"])
    spans = _spans(T, L, case["seqs"])
    base = torch.zeros(T, dtype=torch.int32)
    pos = torch.zeros(T, dtype=torch.int32)
    for t0, nt, s0, ns in spans:
        base[t0:t0 + nt] = s0
        # the last rows of the sequence; a span with more rows than keys starts with rows that see nothing
        pos[t0:t0 + nt] = torch.arange(ns - nt, ns, dtype=torch.int32)
    if case["op"] == "expanded":
        if T > L:  # padded rows behind the last sequence, instead of before each first
            for t0, nt, s0, ns in spans:
                pos[t0:t0 + nt] = torch.arange(nt, dtype=torch.int32)
                pos[t0 + ns:t0 + nt] = -1
        st["q"] = _normal(g, T, H, NOPE + ROTARY).bfloat16()
        st["kv"] = _normal(g, L, H, NOPE + VALUE).bfloat16()
        st["rope"] = _normal(g, L, ROTARY).bfloat16()
    else:
        st["q"] = _normal(g, T, H, LATENT + ROTARY).bfloat16()
        st |= _cache(g, L, "latent", case["fp8"])
        if case["lists"]:
            k = case["k"]
            n = (pos + 1).clamp(min=0).cuda()
            # up to k distinct visible keys of each query in ascending order, then -1: one key at a random place of
            # each of k equal stretches of the context, or every key where there are no more than k
            j = torch.arange(k, device="cuda")[None, :]
            step = (n[:, None].long() // max(1, k)).clamp(min=1)
            jitter = torch.randint(0, 1 << 30, (T, k), generator=g, device="cuda") % step
            idx = (j * step + jitter).to(torch.int32)
            idx = torch.where((j < n[:, None]) & (idx < n[:, None]), idx, torch.full_like(idx, -1))
            st["idx"], st["pos"] = idx.contiguous(), None
        else:
            st["idx"] = None
    st["base"] = base.cuda() if case["seqs"] > 1 else None
    if case["op"] == "expanded" or not case["lists"]:
        st["pos"] = pos.cuda()
    return st


# ----------------------------------------------------------- the plain forms

def _plain_write(st):
    d = st["C"].shape[1]
    x = st["x"].float()
    lat = x[:, :d]
    scale = _row_scale(lat)
    scale = torch.where(lat.abs().amax(1) > 0, scale, torch.ones_like(scale))
    codes = (lat / scale[:, None]).to(torch.float8_e4m3fn)
    spare = st["spare"]
    at = torch.where(st["slots"] < 0, spare["C"].shape[0] - 1, st["slots"]).long()
    spare["C"].view(torch.uint8)[at] = codes.view(torch.uint8)
    spare["c_scale"][at] = scale
    if st["rope"] is not None:
        spare["rope"][at] = st["x"][:, d:]


def _plain_read(st):
    at = st["slots"].clamp(min=0).long()
    x = st["C"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * st["c_scale"][at][:, None]
    if st["rope"] is not None:
        x = torch.cat([x, st["rope"][at].float()], 1)
    return torch.where((st["slots"] >= 0)[:, None], x, torch.zeros_like(x)).bfloat16()


def _plain_softmax(s, seen):
    """Weights and log-sum of each row over the keys it sees; zeros and -inf where it sees none."""
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total)), (top + torch.log(total)).squeeze(-1)


def _plain_rows(st):
    """The latent cache as fp32 rows [L, 576]."""
    if st["c_scale"] is None:
        return st["C"].float()
    return torch.cat([st["C"].float() * st["c_scale"][:, None], st["rope"].float()], 1)


def _plain_latent(st):
    rows = _plain_rows(st)
    L = rows.shape[0]
    q = st["q"].float()
    T, H, _ = q.shape
    base = torch.zeros(T, 1, dtype=torch.int64, device=q.device) if st["base"] is None else st["base"].long()[:, None]
    if st["idx"] is not None:
        at = torch.where(st["idx"] < 0, 0, st["idx"].long() + base)
        keys = rows[at]                                                   # [T, k, 576]
        s = torch.matmul(q, keys.transpose(1, 2)) * SM_SCALE
        p, lse = _plain_softmax(s, (st["idx"] >= 0)[:, None, :])
        return torch.matmul(p, keys[:, :, :LATENT]).bfloat16(), lse
    s = (torch.matmul(q.view(T * H, -1), rows.t()) * SM_SCALE).view(T, H, L)
    j = torch.arange(L, device=q.device)[None, :]
    seen = (j >= base) & (j <= base + st["pos"].long()[:, None])
    p, lse = _plain_softmax(s, seen[:, None, :])
    return torch.matmul(p.view(T * H, L), rows[:, :LATENT]).view(T, H, LATENT).bfloat16(), lse


def _plain_expanded(st):
    q, kv = st["q"].float(), st["kv"].float()
    T, H, _ = q.shape
    L = kv.shape[0]
    keys = torch.cat([kv[:, :, :NOPE], st["rope"].float()[:, None, :].expand(L, H, ROTARY)], 2)
    s = torch.matmul(q.transpose(0, 1), keys.permute(1, 2, 0)) * SM_SCALE  # [H, T, L]
    base = torch.zeros(T, 1, dtype=torch.int64, device=q.device) if st["base"] is None else st["base"].long()[:, None]
    j = torch.arange(L, device=q.device)[None, :]
    seen = (j >= base) & (j <= base + st["pos"].long()[:, None])
    p, lse = _plain_softmax(s, seen[None])
    out = torch.matmul(p, kv[:, :, NOPE:].transpose(0, 1))
    return out.transpose(0, 1).contiguous().bfloat16(), lse.t().contiguous()


# ------------------------------------------------------------------ one pass

def run(state):
    st = state
    if own:
        import sparse_attention_indexer_block_amd as S
        if st["op"] == "write":
            S.cache_write(st["x"], st["slots"], st["C"], st["c_scale"], st["rope"])
        elif st["op"] == "read":
            return S.cache_read(st["slots"], st["C"], st["c_scale"], st["rope"])
        elif st["op"] == "latent":
            out, lse = S.latent_attention(st["q"], st["C"], SM_SCALE, pos=st["pos"], idx=st["idx"],
                                          c_scale=st["c_scale"], rope=st["rope"], base=st["base"], with_lse=True)
            return {"out": out, "lse": lse}
        else:
            out, lse = S.expanded_attention(st["q"], st["kv"], st["rope"], st["pos"], SM_SCALE, base=st["base"],
                                            with_lse=True)
            return {"out": out, "lse": lse}
    else:
        if st["op"] == "write":
            _plain_write(st)
        elif st["op"] == "read":
            return _plain_read(st)
        elif st["op"] == "latent":
            out, lse = _plain_latent(st)
            return {"out": out, "lse": lse}
        else:
            out, lse = _plain_expanded(st)
            return {"out": out, "lse": lse}
    held = {"codes": st["C"], "scale": st["c_scale"]}
    if st["rope"] is not None:
        held["rope"] = st["rope"]
    return held


# ---------------------------------------------------------------------- work

def _visible(case):
    """Query-key pairs of one head."""
    pairs = 0
    for _, nt, _, ns in _spans(case["T"], case["L"], case["seqs"]):
        if case["op"] == "expanded" and case["T"] > case["L"]:
            pairs += sum(range(1, min(nt, ns) + 1))
        else:
            last, first = ns, ns - nt + 1
            lo = max(first, 1)
            n = [min(i, case["k"]) if case.get("lists") else i for i in range(lo, last + 1)]
            pairs += sum(n)
    return pairs


def work(case):
    if case["op"] in ("write", "read"):
        d, dr = (LATENT, ROTARY) if case["kind"] == "latent" else (KEY, 0)
        live = case["n"] - case["holes"]
        held, plain = d + 4 + 2 * dr, 2 * (d + dr)
        read_plain = live if case["op"] == "write" else case["n"]
        return {"bytes": live * held + read_plain * plain + 4 * case["n"], "flops": 2 * live * d}
    T, H, L = case["T"], case["H"], case["L"]
    pairs = _visible(case)
    if case["op"] == "latent":
        row = LATENT + 4 + 2 * ROTARY if case["fp8"] else 2 * (LATENT + ROTARY)
        touched = min(L, pairs) if case["lists"] else L
        lists = 4 * T * case["k"]
        return {"bytes": touched * row + lists + T * H * (2 * (LATENT + ROTARY) + 2 * LATENT + 4) + 4 * T,
                "flops": 2 * pairs * H * (LATENT + ROTARY + LATENT)}
    return {"bytes": L * (H * 2 * (NOPE + VALUE) + 2 * ROTARY) + T * H * (2 * (NOPE + ROTARY) + 2 * VALUE + 4) + 4 * T,
            "flops": 2 * pairs * H * (NOPE + ROTARY + VALUE)}


# --------------------------------------------------------------------- exact

def _two_to(e):
    """2 to the whole numbers e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(v):
    """The nearest value of E4M3FN, ties to the even code, of 64-bit values of at most 448."""
    a = v.abs()
    step = _two_to(torch.frexp(a.clamp(min=2.0 ** -6)).exponent - 4)
    return torch.sign(v) * torch.round(a / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    wide = torch.float64
    if case["op"] == "write":
        d = st["C"].shape[1]
        codes, scale = st["C"].to(wide), st["c_scale"].to(wide)
        rope = None if st["rope"] is None else st["rope"].to(wide)
        keep = torch.nonzero(st["slots"] >= 0).flatten()
        to = st["slots"][keep].long()
        x = st["x"][keep].to(wide)
        amax = x[:, :d].abs().max(1).values
        # the smallest power of two that brings the row within 448
        part, e = torch.frexp(amax / 448.0)
        e = torch.where(part == 0.5, e - 1, e).clamp(min=-126)
        s = torch.where(amax > 0, _two_to(e), torch.ones_like(amax))
        codes[to] = _e4m3(x[:, :d] / s[:, None])
        scale[to] = s
        out = {"codes": codes, "scale": scale}
        if rope is not None:
            rope[to] = x[:, d:]
            out["rope"] = rope
        return out
    if case["op"] == "read":
        out = torch.zeros(case["n"], st["C"].shape[1] + (0 if st["rope"] is None else ROTARY), dtype=wide, device="cuda")
        keep = torch.nonzero(st["slots"] >= 0).flatten()
        frm = st["slots"][keep].long()
        out[keep, :st["C"].shape[1]] = st["C"].to(wide)[frm] * st["c_scale"].to(wide)[frm].unsqueeze(1)
        if st["rope"] is not None:
            out[keep, st["C"].shape[1]:] = st["rope"].to(wide)[frm]
        return out
    T, H = case["T"], case["H"]
    dv = LATENT if case["op"] == "latent" else VALUE
    out = torch.zeros(T, H, dv, dtype=wide, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=wide, device="cuda")
    first = [0] * T if st["base"] is None else st["base"].tolist()
    if case["op"] == "latent":
        C = st["C"].to(wide)
        if st["c_scale"] is not None:
            C = torch.cat((C * st["c_scale"].to(wide).unsqueeze(1), st["rope"].to(wide)), 1)
        lists = None if st["idx"] is None else st["idx"].long()
        counts = None if lists is None else (lists >= 0).sum(1).tolist()
        last = None if lists is not None else st["pos"].tolist()
        for t in range(T):  # one query at a time, over exactly the keys that it has
            if lists is not None:
                if not counts[t]:
                    continue
                mine = C[lists[t, :counts[t]] + first[t]]
            else:
                if last[t] < 0:
                    continue
                mine = C[first[t]:first[t] + last[t] + 1]
            s = torch.mm(st["q"][t].to(wide), mine.t()) * SM_SCALE
            lse[t] = torch.logsumexp(s, 1)
            out[t] = torch.mm(torch.exp(s - lse[t].unsqueeze(1)), mine[:, :LATENT])
        return {"out": out, "lse": lse}
    last = st["pos"].tolist()
    rope = st["rope"].to(wide)
    block = 512
    for h in range(H):
        K = torch.cat((st["kv"][:, h, :NOPE].to(wide), rope), 1)
        V = st["kv"][:, h, NOPE:].to(wide)
        for t0 in range(0, T, block):
            t1 = min(T, t0 + block)
            lo = torch.tensor(first[t0:t1], device="cuda").unsqueeze(1)
            hi = lo + torch.tensor(last[t0:t1], device="cuda").unsqueeze(1)
            j = torch.arange(K.shape[0], device="cuda").unsqueeze(0)
            s = torch.mm(st["q"][t0:t1, h].to(wide), K.t()) * SM_SCALE
            s = s.masked_fill((j < lo) | (j > hi), -math.inf)
            z = torch.logsumexp(s, 1)
            lse[t0:t1, h] = z
            out[t0:t1, h] = torch.mm(torch.exp(s - z.unsqueeze(1)).nan_to_num(0.0), V)
    return {"out": out, "lse": lse}
