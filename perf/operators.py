"""Measured cases of the serving operators around the paged 8-bit key/value
cache: the step plan (block tables and slot maps), the query/key norm with
rotation and cache store, and the attention over the cache.

Each has a plain form in elementary torch operations (32 bits, rounded once at
the end) and the call a user makes of the library; ``own`` says which of the
two ``run`` takes.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
F8_MAX = 448.0                 # largest e4m3 value
EPS = 1e-6                     # of the RMS norm
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a small batch: pure latency
        dict(name="plan decode", op="plan", reqs=48, q_lo=1, q_hi=1, kv_lo=1, kv_hi=4096, page=64, mix=1),
        # chunked prefill mixed with decode and idle rows, small pages, many requests
        dict(name="plan mixed", op="plan", reqs=1023, q_lo=0, q_hi=257, kv_lo=0, kv_hi=5000, page=16, mix=2),
        # a long prefill wave: many tokens per request
        dict(name="plan prefill", op="plan", reqs=61, q_lo=900, q_hi=4096, kv_lo=0, kv_hi=100, page=32, mix=3),
        # one decode step: a token per request, most into pages already begun
        dict(name="store decode", op="store", reqs=64, q_lo=1, q_hi=1, kv_lo=1, kv_hi=4096, page=64, hq=32, hkv=8, d=128,
             rot=128, pairs="halves", dtype="bf16", mix=4),
        # a prefill wave of fresh requests
        dict(name="store prefill", op="store", reqs=6, q_lo=1500, q_hi=4096, kv_lo=0, kv_hi=0, page=64, hq=64, hkv=8,
             d=128, rot=128, pairs="halves", dtype="bf16", mix=5),
        # prefill chunks behind unaligned contexts: fp32, short heads, part of each head rotated, neighbour pairs
        dict(name="store ragged f32", op="store", reqs=19, q_lo=0, q_hi=301, kv_lo=0, kv_hi=999, page=16, hq=12, hkv=3,
             d=64, rot=32, pairs="neighbours", dtype="f32", mix=6),
        # a single user's decode step: few rows, so only the keys can be shared out
        dict(name="attn decode one", op="attn", reqs=1, q_lo=1, q_hi=1, kv_lo=2500, kv_hi=2500, page=64, hq=32, hkv=8,
             d=128, window=0, dtype="bf16", mix=7),
        # a full decode batch with long and short contexts: the cache is read once
        dict(name="attn decode batch", op="attn", reqs=128, q_lo=1, q_hi=1, kv_lo=1000, kv_hi=16384, page=64, hq=64,
             hkv=8, d=128, window=0, dtype="bf16", mix=8),
        # drafted tokens verified together: a few rows per request, odd group of heads, small pages
        dict(name="attn drafts", op="attn", reqs=31, q_lo=2, q_hi=5, kv_lo=200, kv_hi=6000, page=16, hq=28, hkv=4, d=128,
             window=0, dtype="bf16", mix=9),
        # prefill of two long prompts: matrix-product work
        dict(name="attn prefill", op="attn", reqs=2, q_lo=6000, q_hi=8192, kv_lo=0, kv_hi=0, page=64, hq=32, hkv=8,
             d=128, window=0, dtype="bf16", mix=10),
        # chunked prefill beside decode rows and idle ones, sliding window, short heads
        dict(name="attn chunks window", op="attn", reqs=24, q_lo=0, q_hi=700, kv_lo=1, kv_hi=5000, page=32, hq=16, hkv=4,
             d=64, window=1024, dtype="bf16", mix=11),
        # fp32 queries, one shared key head, wide heads, large pages
        dict(name="attn decode f32", op="attn", reqs=9, q_lo=1, q_hi=1, kv_lo=1, kv_hi=3000, page=128, hq=8, hkv=1, d=256,
             window=0, dtype="f32", mix=12),
    ]


def _log_int(rng, lo, hi):
    """An int of [lo, hi], spread over the logarithm where that spans more than a factor of ten."""
    if hi <= 10 * max(lo, 1):
        return rng.randint(lo, hi)
    v = math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1))) - 1
    return min(hi, max(lo, int(round(v))))


def _heads(rng, ds):
    while True:
        hkv = rng.choice([1, 2, 3, 4, 8])
        c = dict(hq=hkv * rng.choice([1, 2, 4, 5, 7, 8, 16]), hkv=hkv, d=rng.choice(ds))
        if c["hq"] <= 64 and 3072 not in (c["hq"] * c["d"], (c["hq"] + 2 * hkv) * c["d"]):
            return c


def draw(rng):
    op = rng.choice(["plan", "store", "attn", "attn"])
    mix = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        reqs = _log_int(rng, 1, 1500)
        q_hi = _log_int(rng, 1, max(1, min(4096, 120000 // reqs)))
        return dict(op=op, reqs=reqs, q_lo=rng.choice([0, 1, q_hi]), q_hi=q_hi, kv_lo=0, kv_hi=_log_int(rng, 1, 8000),
                    page=page, mix=mix)
    if op == "store":
        reqs = _log_int(rng, 1, 512)
        q_hi = _log_int(rng, 1, max(1, min(4096, 8000 // reqs)))
        c = dict(op=op, reqs=reqs, q_lo=rng.choice([0, 1, q_hi]), q_hi=q_hi, kv_lo=0, kv_hi=_log_int(rng, 1, 3000),
                 page=page, **_heads(rng, [64, 128, 256]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                 pairs=rng.choice(["halves", "neighbours"]), mix=mix)
        c["rot"] = c["d"] if rng.random() < 0.6 else 16 * rng.randint(0, c["d"] // 16)
        return c
    kind = rng.choice(["decode", "drafts", "prefill", "chunks"])
    c = dict(op=op, page=page, **_heads(rng, [64, 128, 256]), mix=mix)
    c["dtype"] = "f32" if rng.random() < 0.2 else "bf16"
    c["window"] = _log_int(rng, 1, 4000) if rng.random() < 0.25 else 0
    if kind in ("decode", "drafts"):
        hi = _log_int(rng, 20, 16384)
        # keys x heads x width stay below the listed batch's
        reqs = _log_int(rng, 1, max(1, min(256, 500000 * 1024 // (hi * c["hkv"] * c["d"]))))
        q = (1, 1) if kind == "decode" else (1, rng.randint(2, 8))
        c.update(reqs=reqs, q_lo=q[0], q_hi=q[1], kv_lo=rng.choice([0, hi // 4, hi]), kv_hi=hi)
    elif kind == "prefill":
        q_hi = _log_int(rng, 16, 4096)
        c.update(reqs=rng.randint(1, max(1, min(8, 6000 // q_hi))), q_lo=max(1, q_hi // 2), q_hi=q_hi, kv_lo=0, kv_hi=0)
    else:
        c.update(reqs=_log_int(rng, 2, 24), q_lo=0, q_hi=_log_int(rng, 16, 500), kv_lo=0, kv_hi=_log_int(rng, 16, 4000))
    for f in ("q_lo", "q_hi", "kv_lo", "kv_hi"):
        c[f] -= c[f] == 3072
    return c


def _lens(case):
    """(cached tokens, new tokens) of each request: a matter of the case alone."""
    rs = np.random.RandomState(case["mix"])

    def some(lo, hi):
        u = rs.rand(case["reqs"])
        if hi <= 10 * max(lo, 1):
            v = lo + np.floor(u * (hi - lo + 1))
        else:
            v = np.exp(np.log(lo + 1) + u * (np.log(hi + 1) - np.log(lo + 1))) - 1
        return np.clip(np.rint(v), lo, hi).astype(np.int64)

    q, kv = some(case["q_lo"], case["q_hi"]), some(case["kv_lo"], case["kv_hi"])
    if q.sum() == 0:
        q[0] = 1
    if case["op"] == "attn" and case["kv_hi"] > 0:    # kv counts the new tokens too
        kv = np.maximum(kv - q, 0)
    return kv, q


# ---------------------------------------------------------------- inputs
def _requests(case, seed):
    """The case's requests in this seed's order, with the pages they hold."""
    rs = np.random.RandomState(seed % (1 << 31))
    kv, q = _lens(case)
    order = rs.permutation(case["reqs"])
    kv, q = kv[order], q[order]
    P = case["page"]
    old, new = -(-kv // P), -(-(kv + q) // P)
    max_blocks = int(new.max()) + 1
    n_pages = int(new.sum()) + 5
    ids = rs.permutation(n_pages).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(q)])
    return dict(rs=rs, kv=kv, q=q, old=old, new=new, max_blocks=max_blocks, n_pages=n_pages, ids=ids, cu=cu,
                T=int(cu[-1]))


def _table(r, counts):
    """Block table whose row i holds the next counts[i] page ids; -1 behind them."""
    col = np.arange(r["max_blocks"])[None, :]
    begin = np.concatenate([[0], np.cumsum(counts)[:-1]])[:, None]
    return np.where(col < counts[:, None], r["ids"][np.minimum(begin + col, r["n_pages"] - 1)], -1).astype(np.int32)


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def _codes(shape, gen):
    """e4m3 codes of a cache in use (finite, most of the range taken)."""
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    for part in out.split(max(1, (1 << 27) // max(1, out[0].numel()))):
        part.copy_((torch.randn(part.shape, device=DEV, generator=gen) * 60).clamp_(-F8_MAX, F8_MAX)
                   .to(torch.float8_e4m3fn).view(torch.uint8))
    return out


def _cache(case, r, gen):
    n, h, P, D = r["n_pages"], case["hkv"], case["page"], case["d"]
    scale = lambda: torch.exp2(torch.randint(-7, -4, (n + 1, h), device=DEV, generator=gen).float())  # noqa: E731
    # one spare page behind the cache: the plain form stores what it has to drop there
    return dict(k=_codes((n + 1, h, P, D), gen), v=_codes((n + 1, h, P, D), gen), ks=scale(), vs=scale())


def _segments(case, r, table):
    """Slots, positions and segment leaders of the step's new tokens."""
    P = case["page"]
    req = np.repeat(np.arange(case["reqs"]), r["q"])
    pos = r["kv"][req] + np.arange(r["T"]) - r["cu"][req]
    slots = table[req, pos // P].astype(np.int64) * P + pos % P
    lead = np.flatnonzero((pos == r["kv"][req]) | (pos % P == 0))
    seg = np.full(min(r["T"], r["T"] // P + 2 * case["reqs"]), -1)
    seg[:len(lead)] = lead
    return slots, pos, seg


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = _requests(case, seed)
    s = dict(case=case, T=r["T"], n_pages=r["n_pages"], max_blocks=r["max_blocks"], kv=_dev(r["kv"]), q_len=_dev(r["q"]),
             cu=_dev(r["cu"]))
    if own:
        import routing_dispatch_grouped_amd as rdg
        s["rdg"] = rdg
        s["step"] = step = rdg.KvStep(case["reqs"], r["max_blocks"], case["page"], r["n_pages"], r["T"], DEV)
    if case["op"] == "plan":
        held = int(r["old"].sum())
        s["table"] = _dev(_table(r, r["old"]))
        s["free"], s["n_free"] = _dev(r["ids"][held:]), _dev(np.array([r["n_pages"] - held]))
        s["n_free_out"] = torch.zeros_like(s["n_free"])
        s["seg_cap"] = min(r["T"], r["T"] // case["page"] + 2 * case["reqs"])
        if own:
            step.block_table.copy_(s["table"])
        return s
    table = _table(r, r["new"])
    s["table"], s["kv_out"] = _dev(table), _dev(r["kv"] + r["q"])
    s.update(_cache(case, r, gen))
    dtype = DTYPES[case["dtype"]]
    hq, hkv, D = case["hq"], case["hkv"], case["d"]
    if case["op"] == "store":
        # activations with a few strong channels, as projections give them
        gain = torch.exp(0.7 * torch.randn(1, (hq + 2 * hkv) * D, device=DEV, generator=gen))
        s["qkv"] = (torch.randn(r["T"], (hq + 2 * hkv) * D, device=DEV, generator=gen) * gain).to(dtype)
        s["wq"] = 1 + 0.2 * torch.randn(D, device=DEV, generator=gen)
        s["wk"] = 1 + 0.2 * torch.randn(D, device=DEV, generator=gen)
        n_pos = int((r["kv"] + r["q"]).max())
        half = case["rot"] // 2
        freq = 10000.0 ** (-np.arange(half) / max(half, 1))
        angle = np.arange(n_pos)[:, None] * freq[None, :]
        s["cos_sin"] = _dev(np.concatenate([np.cos(angle), np.sin(angle)], 1), torch.float32)
        slots, pos, seg = _segments(case, r, table)
        s["slots"], s["pos"], s["seg"] = _dev(slots), _dev(pos), _dev(seg)
        s["q_out"] = torch.empty(r["T"], hq, D, dtype=dtype, device=DEV)
    else:
        s["q"] = (2 * torch.randn(r["T"], hq, D, device=DEV, generator=gen)).to(dtype)
        s["max_q"], s["max_kv"] = int(r["q"].max()), int((r["kv"] + r["q"]).max())
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(r["T"], hq, dtype=torch.float32, device=DEV)
    if own:
        n = r["n_pages"]
        s["cache"] = rdg.KvCache(s["k"][:n], s["v"][:n], s["ks"][:n], s["vs"][:n])
        step.block_table.copy_(s["table"])
        step.cu_q.copy_(s["cu"])
        step.kv_len.copy_(s["kv_out"])
        if case["op"] == "store":
            step.slots.copy_(s["slots"])
            step.positions.copy_(s["pos"])
            step.seg_tok.copy_(s["seg"])
        else:
            s["work"] = torch.empty(rdg.rdg_paged_attention_workspace_bytes(
                s["cache"], r["T"], case["reqs"], hq, s["max_q"], s["max_kv"], rdg_dtype(rdg, case)),
                dtype=torch.uint8, device=DEV)
    return s


def rdg_dtype(rdg, case):
    return rdg.RDG_BF16 if case["dtype"] == "bf16" else rdg.RDG_F32


# ---------------------------------------------------------------- one pass
def run(s):
    return {"plan": _plan, "store": _store, "attn": _attn}[s["case"]["op"]](s)


def _plan(s):
    if own:
        st = s["step"]
        s["rdg"].rdg_kv_plan(st, s["kv"], s["q_len"], s["free"], s["n_free"], s["n_free_out"])
        return dict(table=st.block_table, cu=st.cu_q, kv=st.kv_len, slots=st.slots, pos=st.positions, seg=st.seg_tok,
                    n_free=s["n_free_out"])
    P, T, R, B = s["case"]["page"], s["T"], s["case"]["reqs"], s["max_blocks"]
    kv, q = s["kv"], s["q_len"]
    old, new = (kv + P - 1) // P, (kv + q + P - 1) // P
    need = torch.where(new > B, 0, new - old)
    end = torch.cumsum(need, 0, dtype=torch.int32)
    ok = (new <= B) & ((need == 0) | (end <= s["n_free"]))
    begin = end - need
    n_free_out = s["n_free"] - torch.where(ok, end * (need > 0), 0).max()
    col = torch.arange(B, device=DEV, dtype=torch.int32)[None, :]
    fresh = ok[:, None] & (col >= old[:, None]) & (col < new[:, None])
    take = (s["n_free"] - 1 - begin[:, None] - (col - old[:, None])).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][take.long()], s["table"])
    cu = torch.zeros(R + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(q, 0, dtype=torch.int32)
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    req = torch.searchsorted(cu, t, right=True) - 1
    pos = kv[req] + t - cu[req]
    slots = torch.where(ok[req], table[req, (pos // P).long().clamp(max=B - 1)] * P + pos % P, -1)
    lead = ok[req] & ((pos == kv[req]) | (pos % P == 0))
    at = torch.where(lead, torch.cumsum(lead, 0) - 1, s["seg_cap"])
    seg = torch.full((s["seg_cap"] + 1,), -1, dtype=torch.int32, device=DEV).scatter(0, at, t)[:-1]
    seg = torch.where(torch.arange(s["seg_cap"], device=DEV) < lead.sum(), seg, -1)
    return dict(table=table, cu=cu, kv=kv + torch.where(ok, q, 0), slots=slots, pos=pos, seg=seg, n_free=n_free_out)


def _store(s):
    c = s["case"]
    n = s["n_pages"]
    if own:
        s["rdg"].rdg_qk_norm_rope_store(s["qkv"], c["hq"], c["hkv"], c["d"], s["wq"], s["wk"], EPS, s["cos_sin"], c["rot"],
                                        c["pairs"] == "neighbours", s["step"], s["cache"], s["q_out"])
        q = s["q_out"]
    else:
        T, hq, hkv, D, rot = s["T"], c["hq"], c["hkv"], c["d"], c["rot"]
        x = s["qkv"].float().view(T, hq + 2 * hkv, D)
        qk = x[:, :hq + hkv]
        qk = qk * torch.rsqrt((qk * qk).mean(-1, keepdim=True) + EPS)
        qk = qk * torch.cat([s["wq"].expand(hq, D), s["wk"].expand(hkv, D)])
        turn = s["cos_sin"][s["pos"].long()][:, None]
        cos, sin = turn[..., :rot // 2], turn[..., rot // 2:]
        if c["pairs"] == "halves":
            a, b = qk[..., :rot // 2], qk[..., rot // 2:rot]
            qk = torch.cat([a * cos - b * sin, b * cos + a * sin, qk[..., rot:]], -1)
        else:
            a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
            mixed = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
            qk = torch.cat([mixed, qk[..., rot:]], -1)
        q = qk[:, :hq].to(s["qkv"].dtype)
        _put(s, qk[:, hq:], s["k"], s["ks"])
        _put(s, x[:, hq + hkv:], s["v"], s["vs"])
    return dict(q=q, k=s["k"][:n].view(torch.float8_e4m3fn), ks=s["ks"][:n], v=s["v"][:n].view(torch.float8_e4m3fn),
                vs=s["vs"][:n])


def _put(s, x, codes, scales):
    """Rows x [T, heads, D] into their pages: one power-of-two scale for each page and head."""
    P, T, n = s["case"]["page"], s["T"], s["n_pages"]
    live = s["seg"] >= 0
    lead = s["seg"].clamp(min=0).long()
    first = s["slots"][lead].long()
    page, off = first // P, first % P
    row = torch.arange(P, device=DEV)[None, :]
    tok = lead[:, None] + row - off[:, None]                       # the token stored in each row of the page
    inside = (tok >= lead[:, None]) & (tok < T)
    tok = tok.clamp(0, T - 1)
    fresh = inside & (s["slots"][tok].long() == (page * P)[:, None] + row) & live[:, None]
    kept = (row < off[:, None]) & live[:, None]
    rows = torch.where(fresh[..., None, None], x[tok], 0.0).transpose(1, 2)   # [segments, heads, P, D]
    amax = rows.abs().amax((2, 3))
    mant, exp = torch.frexp(amax)                                  # amax = mant 2^exp, mant in [0.5, 1)
    new = torch.exp2((exp - 9 + (mant > 0.875)).float().clamp(-126, 127))
    new = torch.where(amax > 0, new, 2.0 ** -126)
    was = scales[page]
    now = torch.where(off[:, None] > 0, torch.maximum(was, new), new)
    have = codes[page].view(torch.float8_e4m3fn).float()
    again = have * (was / now)[..., None, None]
    put = torch.where(fresh[:, None, :, None], rows / now[..., None, None], again).clamp(-F8_MAX, F8_MAX)
    put = put.to(torch.float8_e4m3fn).view(torch.uint8)
    put = torch.where((fresh | kept)[:, None, :, None], put, codes[page])
    to = torch.where(live, page, n)
    codes[to] = put
    scales[to] = now


def _attn(s):
    c = s["case"]
    scale = c["d"] ** -0.5
    if own:
        s["rdg"].rdg_paged_attention(s["q"], s["step"], s["cache"], s["max_q"], s["max_kv"], scale, s["out"], s["lse"],
                                     s["work"], causal=True, window=c["window"])
        return dict(out=s["out"], lse=s["lse"])
    R, hq, hkv, D, P, T = c["reqs"], c["hq"], c["hkv"], c["d"], c["page"], s["T"]
    nb, mq = (s["max_kv"] + P - 1) // P, s["max_q"]
    L = nb * P
    cu, kv_out = s["cu"].long(), s["kv_out"].long()
    pages = s["table"][:, :nb].clamp(min=0).long()

    def rows(codes, scales):
        x = codes[pages].view(torch.float8_e4m3fn).float().mul_(scales[pages][..., None, None])
        return x.transpose(1, 2).reshape(R, hkv, L, D)

    k, v = rows(s["k"], s["ks"]), rows(s["v"], s["vs"])
    i, j = torch.arange(mq, device=DEV), torch.arange(L, device=DEV)
    v.masked_fill_((j[None, :] >= kv_out[:, None])[:, None, :, None], 0.0)
    tok = (cu[:-1, None] + i).clamp(max=T - 1)
    q = s["q"][tok].float().view(R, mq, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(R, hkv, -1, D)
    at = kv_out[:, None] - (cu[1:] - cu[:-1])[:, None] + i          # position of each query
    seen = (j <= at[..., None]) & (j < kv_out[:, None, None])       # [R, mq, L]
    if c["window"]:
        seen &= j > at[..., None] - c["window"]
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).view(R, hkv, hq // hkv, mq, L)
    p.masked_fill_(~seen[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, hkv, -1, L), v).view(R, hkv, hq // hkv, mq, D) / torch.where(total == 0, 1.0, total)
    lse = torch.log(total[..., 0]) + top[..., 0]
    t = torch.arange(T, device=DEV)
    req = torch.searchsorted(cu, t, right=True) - 1
    o = o.permute(0, 3, 1, 2, 4).reshape(R, mq, hq, D)[req, t - cu[req]]
    lse = lse.permute(0, 3, 1, 2).reshape(R, mq, hq)[req, t - cu[req]]
    return dict(out=o.to(s["q"].dtype), lse=lse)


# ---------------------------------------------------------------- work of one pass
def work(case):
    kv, q = _lens(case)
    T, R, P = int(q.sum()), case["reqs"], case["page"]
    old, new = -(-kv // P), -(-(kv + q) // P)
    if case["op"] == "plan":
        fresh = int((new - old).sum())
        segs = int(np.where(q > 0, (kv + q - 1) // P - kv // P + 1, 0).sum())
        # lengths in; sums and lengths out; page ids in and out; slot and position of each token; segments
        return dict(bytes=16 * R + 8 * fresh + 8 * T + 4 * segs, flops=0)
    hq, hkv, D = case["hq"], case["hkv"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "store":
        return dict(bytes=T * (hq + 2 * hkv) * D * e + T * hq * D * e + 2 * T * hkv * D + 8 * T + T * case["rot"] * 4,
                    flops=T * (hq + hkv) * (4 * D + 3 * case["rot"]))
    w = case["window"]
    keys, pairs = 0, 0
    for a, n in zip(kv.tolist(), q.tolist()):
        at = a + np.arange(n)
        seen = at + 1 if not w else np.minimum(at + 1, w)
        pairs += int(seen.sum())
        keys += 0 if n == 0 else (a + n if not w else min(a + n, w + n - 1))
    return dict(bytes=2 * T * hq * D * e + 4 * T * hq + 2 * keys * hkv * D + 4 * keys // P, flops=4 * D * hq * pairs)


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None                        # whole numbers only
    s = prepare(case, seed)
    return _exact_store(s) if case["op"] == "store" else _exact_attn(s)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def _exact_store(s):
    c = s["case"]
    T, hq, hkv, D, P, n = s["T"], c["hq"], c["hkv"], c["d"], c["page"], s["n_pages"]
    x = s["qkv"].double().view(T, hq + 2 * hkv, D)
    half = c["rot"] // 2
    turn = s["cos_sin"].double()[s["pos"].long()]
    z = torch.complex(turn[:, :half].contiguous(), turn[:, half:].contiguous())[:, None, :]

    def turned(y, w):
        y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / D + EPS) * w.double()
        r, rest = y[..., :c["rot"]], y[..., c["rot"]:]
        if c["pairs"] == "halves":
            a = torch.complex(r[..., :half].contiguous(), r[..., half:].contiguous()) * z
            return torch.cat([a.real, a.imag, rest], -1)
        a = torch.view_as_complex(r.reshape(T, -1, half, 2).contiguous()) * z
        return torch.cat([torch.view_as_real(a).flatten(-2), rest], -1)

    out = dict(q=turned(x[:, :hq], s["wq"]))
    slots, seg = s["slots"].tolist(), s["seg"].tolist()
    for name, sc, y in (("k", "ks", turned(x[:, hq:hq + hkv], s["wk"])), ("v", "vs", x[:, hq + hkv:])):
        values, scales = _values(s[name][:n]), s[sc][:n].double()
        for a in seg:
            if a < 0:
                break
            page, off = divmod(slots[a], P)
            m = 1
            while off + m < P and a + m < T and slots[a + m] == slots[a] + m:
                m += 1
            rows = y[a:a + m].transpose(0, 1)                       # [heads, m, D]
            fit = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((1, 2)) / F8_MAX)).clamp(-126, 127))
            now = torch.maximum(scales[page], fit) if off else fit
            values[page, :, :off] *= (scales[page] / now)[:, None, None]
            values[page, :, off:off + m] = rows / now[:, None, None]
            scales[page] = now
        out[name], out[sc] = values, scales
    return out


def _exact_attn(s):
    c = s["case"]
    P, hq, hkv, D = c["page"], c["hq"], c["hkv"], c["d"]
    cu, kv_out = s["cu"].tolist(), s["kv_out"].tolist()
    out = torch.zeros(s["T"], hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((s["T"], hq), -math.inf, dtype=torch.float64, device=DEV)
    for r in range(c["reqs"]):
        n, L = cu[r + 1] - cu[r], kv_out[r]
        if n == 0 or L == 0:
            continue
        pages = s["table"][r, :-(-L // P)].long()
        k = (_values(s["k"][pages]) * s["ks"][pages].double()[..., None, None]).transpose(0, 1).reshape(hkv, -1, D)[:, :L]
        v = (_values(s["v"][pages]) * s["vs"][pages].double()[..., None, None]).transpose(0, 1).reshape(hkv, -1, D)[:, :L]
        q = s["q"][cu[r]:cu[r + 1]].double()
        at = torch.arange(L - n, L, device=DEV)[:, None]
        j = torch.arange(L, device=DEV)[None, :]
        hidden = (j > at) if not c["window"] else (j > at) | (j <= at - c["window"])
        for h in range(hq):
            x = (q[:, h] @ k[h * hkv // hq].T / math.sqrt(D)).masked_fill(hidden, -math.inf)
            out[cu[r]:cu[r + 1], h] = torch.softmax(x, -1) @ v[h * hkv // hq]
            lse[cu[r]:cu[r + 1], h] = torch.logsumexp(x, -1)
    return dict(out=out, lse=lse)
