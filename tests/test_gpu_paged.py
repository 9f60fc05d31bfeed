"""The paged-cache operators on the GPU against the oracle: the step plan and
the hand-back of pages (exact), the query/key norm with rotation and store,
and the attention over the cache.

Tolerances, all derived:
  * plan, trim, codes and scales of operands that are neither normed nor rotated: equal.
  * q: half a bf16 step (2^-8 of the value), or nothing for fp32, plus the fp32
    arithmetic: the norm's sum of D squares, its root and division, two gains and
    the rotation's two products, under 32 roundings of 2^-24 of the pair's size.
  * codes of normed keys: half an e4m3 step (2^-4 of the value, 2^-10 of the
    scale below the normal range), widened by the same fp32 arithmetic.
  * attention: a logit is a sum of D products of exact operands, in fp32: off by at
    most (D + 4) 2^-24 of the sum of magnitudes, d; so each probability is off by a factor
    within 1 + 2 d + kv 2^-23 (the sum over kv keys, the running rescale), plus 2^-8 where
    it is rounded to bf16 (2^-9, against a sum that is not), and the output by that
    share of sum_j p_j |v_j|; then half a step of its own type.  A probability below fp32's
    range (2^-126 of the largest) counts as zero: kv 2^-126 of the largest value.
"""
import numpy as np
import pytest
import torch

import oracle
from harness import DEV, rdg
from oracle import paged

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def host(t):
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy().astype(np.int64)


# ---------------------------------------------------------------- plan
PLANS = {
    "decode": dict(kv=[5, 16, 0, 31, 32, 63], q=[1] * 6, P=16),
    "idle rows and empty requests": dict(kv=[0, 0, 17, 16, 0], q=[0, 3, 0, 0, 33], P=16),
    "one token in all": dict(kv=[0], q=[1], P=128),
    "no token": dict(kv=[3, 0], q=[0, 0], P=32),
    "long": dict(kv=[100, 0, 4000], q=[3000, 1, 129], P=64),
    "many": dict(kv=list(np.arange(700) % 90), q=list(np.arange(700) * 7 % 31), P=32),
    "most requests": dict(kv=[1] * 4096, q=[1] * 4096, P=16),
    "out of pages": dict(kv=[10, 20, 0, 16, 5], q=[40, 100, 30, 1, 3], P=16, spare=-9),
    "past the table": dict(kv=[10, 20, 60], q=[40, 100, 3], P=16, blocks=4),
    "past the tokens": dict(kv=[10, 20, 60], q=[40, 100, 3], P=16, t_cap=99),
    "negative": dict(kv=[10, -2, 60], q=[4, 1, -3], P=16),
    "huge": dict(kv=[10, 2 ** 31 - 1, 7], q=[4, 2 ** 31 - 1, 2], P=16, t_cap=50, blocks=9),
}


def plan_case(kv, q, P, spare=5, blocks=None, t_cap=None, seed=0):
    rng = np.random.default_rng(seed)
    kv, q = np.array(kv, np.int64), np.array(q, np.int64)
    held = [min(int(paged.pages_of(max(x, 0), P)), blocks or 10 ** 9) for x in kv]
    need = sum(int(paged.pages_of(a + b, P) - paged.pages_of(a, P)) for a, b in zip(kv, q)
               if a >= 0 and b >= 0 and a < 2 ** 30)
    need = min(need, 10000)
    B = blocks or max(int(paged.pages_of(a + b, P)) for a, b in zip(kv, q)) + 2
    n_pages = sum(held) + need + spare
    ids = rng.permutation(max(n_pages, 1))
    table, at = np.full((len(kv), B), -1), 0
    for r, n in enumerate(held):
        table[r, :n] = ids[at:at + n]
        at += n
    free = np.concatenate([ids[at:], np.full(n_pages - (n_pages - at), -1)])[:n_pages]
    return kv, q, table, free, n_pages - at, n_pages, int(q.sum()) + 3 if t_cap is None else t_cap


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", PLANS)
def test_plan_equals_the_oracle(name, in_place):
    m = rdg()
    P = PLANS[name]["P"]
    kv, q, table, free, n_free, n_pages, t_cap = plan_case(**PLANS[name])
    step = m.KvStep(len(kv), table.shape[1], P, n_pages, t_cap, DEV)
    for t in (step.slots, step.positions, step.seg_tok, step.cu_q):
        t.fill_(77)
    step.block_table.copy_(dev(table))
    n, out = dev([n_free]), dev([0])
    lens = dev(kv.astype(np.int32))
    if in_place:
        step.kv_len.copy_(lens)
        lens, out = step.kv_len, n
    m.rdg_kv_plan(step, lens, dev(q.astype(np.int32)), dev(free), n, out)
    code = m.rdg_check_status(step)
    want = paged.kv_plan(np.where(kv > 2 ** 30, -1, kv), np.where(q > 2 ** 30, -1, q), table, free, n_free, P, t_cap,
                         step.seg_tok.numel())
    for got, ref, what in zip((step.block_table, step.cu_q, step.kv_len, step.slots, step.positions, step.seg_tok, out),
                              want, ("table", "cu_q", "kv_len", "slots", "positions", "seg_tok", "n_free")):
        assert np.array_equal(host(got), np.ravel(ref).reshape(got.shape)), what
    assert code == want[-1]
    assert not host(step.work.view(torch.int32)).any()      # left as it was found


def test_plan_of_a_bad_table_names_the_request():
    m = rdg()
    kv, q, table, free, n_free, n_pages, t_cap = plan_case([5, 20, 9], [2, 2, 2], 16)
    table[1, 1] = n_pages + 7
    step = m.KvStep(3, table.shape[1], 16, n_pages, t_cap, DEV)
    step.block_table.copy_(dev(table))
    m.rdg_kv_plan(step, dev(kv), dev(q), dev(free), dev([n_free]), dev([0]))
    assert m.rdg_check_status(step) == (m.RDG_EDATA, 1)
    assert list(host(step.slots)[2:4]) == [-1, -1] and (host(step.slots)[4:6] >= 0).all()


@pytest.mark.parametrize("P,R", [(16, 5), (64, 300), (32, 4096)])
def test_steps_and_trims_in_a_row(P, R):
    """A serving loop's lengths: grow, drop drafted tokens, finish, reuse the pages; the
    state stays on the GPU and is compared with the oracle's after every call."""
    m = rdg()
    rng = np.random.default_rng(P)
    B = 6
    n_pages = R * 4
    step = m.KvStep(R, B, P, n_pages, R * 2 * P, DEV)
    table, free, n_free = np.full((R, B), -1), rng.permutation(n_pages), n_pages
    kv = np.zeros(R, int)
    d_free, d_n = dev(free), dev([n_free])
    for _ in range(5):
        q = np.minimum(rng.integers(0, 2 * P, R), B * P - kv)
        m.rdg_kv_plan(step, step.kv_len, dev(q), d_free, d_n, d_n)
        table, cu, kv, slots, pos, seg, n_free, status = paged.kv_plan(kv, q, table, free, n_free, P, R * 2 * P,
                                                                       step.seg_tok.numel())
        assert m.rdg_check_status(step) == status
        assert np.array_equal(host(step.block_table), table) and np.array_equal(host(step.slots), slots)
        assert host(d_n)[0] == n_free and np.array_equal(host(step.seg_tok), seg)
        keep = np.maximum(kv - rng.integers(0, 5, R), 0)
        keep[rng.random(R) < 0.3] = 0
        m.rdg_kv_trim(step, step.kv_len, dev(keep), d_free, d_n, d_n)
        table, kv, stack, n_free, status = paged.kv_trim(kv, keep, table, np.concatenate(
            [free[:n_free], np.full(n_pages - n_free, -1)]), n_free, P)
        free = np.concatenate([stack, np.full(n_pages - len(stack), -1)]).astype(int)
        assert m.rdg_check_status(step) == (0, 0)
        assert np.array_equal(host(step.kv_len), kv) and np.array_equal(host(step.block_table), table)
        assert host(d_n)[0] == n_free and np.array_equal(host(d_free)[:n_free], free[:n_free])


def test_trim_refuses_lengths_and_overfull_lists():
    m = rdg()
    step = m.KvStep(3, 4, 16, 6, 0, DEV)
    table = np.array([[0, 1, -1, -1], [2, -1, -1, -1], [3, 4, -1, -1]])
    step.block_table.copy_(dev(table))
    kv = dev([20, 9, 30])
    free = dev([5, -1, -1, -1, -1, -1])
    n, out = dev([1]), dev([0])
    m.rdg_kv_trim(step, kv, dev([16, 12, -1]), free, n, out)      # rows 1 and 2: out of range
    assert m.rdg_check_status(step) == (m.RDG_EDATA, 1)
    assert list(host(step.kv_len)) == [16, 9, 30] and list(host(free)[:2]) == [5, 1] and host(out)[0] == 2
    n.fill_(6)                                                     # a list that claims to be full
    before = host(step.block_table)
    m.rdg_kv_trim(step, kv, dev([0, 0, 0]), free, n, out)
    assert m.rdg_check_status(step) == (m.RDG_ECAPACITY, 5)
    assert np.array_equal(host(step.block_table), before) and host(out)[0] == 6 and list(host(step.kv_len)) == [20, 9, 30]


# ---------------------------------------------------------------- norm, rotation, store
def begin(m, kv, q, P, n_kv, D, seed, extra_pages=2):
    """A step over fresh tables, with a cache whose pages hold random codes, NaN codes too."""
    rng = np.random.default_rng(seed)
    kv, q = np.array(kv), np.array(q)
    new = paged.pages_of(kv + q, P)
    n_pages, B = int(new.sum()) + extra_pages, max(int(new.max()), 1)
    ids, at = rng.permutation(n_pages), 0
    table = np.full((len(kv), B), -1)
    for r, n in enumerate(new):
        table[r, :n] = ids[at:at + n]
        at += n
    step = m.KvStep(len(kv), B, P, n_pages, int(q.sum()), DEV)
    full = paged.kv_plan(kv, q, table, [], 0, P, int(q.sum()), step.seg_tok.numel())
    # every page is there already: the plan allots none and writes slots and segments
    held = paged.pages_of(kv, P)
    free = [table[r, b] for r in range(len(kv)) for b in range(held[r], new[r])][::-1]
    step.block_table.copy_(dev(np.where(np.arange(B)[None] < held[:, None], table, -1)))
    m.rdg_kv_plan(step, dev(kv), dev(q), dev(free if free else [0]), dev([len(free)]), dev([0]))
    assert m.rdg_check_status(step) == (0, 0) and full[-1][0] in (0, -2)
    assert np.array_equal(host(step.block_table), table)
    codes = lambda: rng.integers(0, 256, (n_pages, n_kv, P, D)).astype(np.uint8)  # noqa: E731
    scales = lambda: np.exp2(rng.integers(-9, -4, (n_pages, n_kv))).astype(np.float32)  # noqa: E731
    k, v, ks, vs = codes(), codes(), scales(), scales()
    cache = m.KvCache(dev(k, torch.uint8), dev(v, torch.uint8), dev(ks, torch.float32), dev(vs, torch.float32))
    return step, table, cache, (k, v, ks, vs)


STORES = [
    # kv, q, P, n_q, n_kv, D, rot, neighbours, dtype
    ([0], [1], 16, 1, 1, 64, 64, False, "bf16"),
    ([15, 16, 17, 0, 40], [1, 1, 1, 0, 1], 16, 4, 2, 128, 128, False, "bf16"),
    ([5, 0, 63, 64], [70, 130, 1, 2], 64, 7, 1, 128, 64, True, "bf16"),
    ([31, 0, 1], [33, 97, 64], 32, 5, 5, 64, 48, False, "f32"),
    ([100, 3], [30, 300], 128, 8, 2, 256, 256, False, "bf16"),
    ([0, 127, 130], [129, 2, 0], 128, 3, 3, 128, 32, True, "f32"),
    ([7], [1100], 16, 9, 3, 64, 16, True, "bf16"),
    ([2, 30], [50, 5], 16, 3, 1, 256, 0, False, "f32"),
    ([9], [1500], 64, 20, 4, 128, 96, False, "bf16"),
]


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("case", range(len(STORES)))
def test_store_equals_the_oracle(case, weights):
    m = rdg()
    kv, q, P, n_q, n_kv, D, rot, neighbours, dtype = STORES[case]
    rng = np.random.default_rng(100 + case)
    step, table, cache, (k, v, ks, vs) = begin(m, kv, q, P, n_kv, D, case)
    T, W = int(np.sum(q)), (n_q + 2 * n_kv) * D
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    wide = torch.from_numpy(rng.standard_normal((T, W + 16)) * np.exp(rng.standard_normal((T, 1)))).to(tt).to(DEV)
    qkv = wide[:, :W]                                       # tokens apart by more than their width
    wq, wk = (rng.uniform(0.5, 2, D).astype(np.float32) for _ in range(2))
    n_pos = int(np.max(np.array(kv) + q))
    ang = np.arange(n_pos)[:, None] * 100.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    q_wide = torch.full((T, n_q * D + 8), 9.0, dtype=tt, device=DEV)
    q_out = q_wide[:, :n_q * D]
    m.rdg_qk_norm_rope_store(qkv, n_q, n_kv, D, dev(wq, torch.float32) if weights else None,
                             dev(wk, torch.float32) if weights else None, 1e-5, dev(cs, torch.float32) if rot else None,
                             rot, neighbours, step, cache, q_out)
    assert m.rdg_check_status(step) == (0, 0)
    x = host(qkv).reshape(T, n_q + 2 * n_kv, D)
    pos = host(step.positions)

    def ref(y, w):
        y = paged.norm(y, w, 1e-5) if weights else y
        size = np.abs(y)
        if rot:
            turn = cs[pos][:, None].astype(np.float64)
            y = paged.rotate(y, turn[..., :rot // 2], turn[..., rot // 2:], neighbours)
            size = np.maximum(size, np.abs(y)).max(-1, keepdims=True) * np.ones(D)
        return y, size

    want, size = ref(x[:, :n_q], wq)
    err = np.abs(host(q_out).reshape(T, n_q, D) - want)
    assert (err <= (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(want) + 32 * EPS * size).all()
    assert (host(q_wide[:, n_q * D:]) == 9).all()

    slots, seg = host(step.slots), host(step.seg_tok)
    wv = paged.store(v, vs, slots, seg, x[:, n_q + n_kv:])
    assert np.array_equal(host(cache.v), wv[0]) and np.array_equal(host(cache.v_scale), wv[1])
    want, size = ref(x[:, n_q:n_q + n_kv], wk)
    wkc = paged.store(k, ks, slots, seg, want)
    if not weights and not rot:
        assert np.array_equal(host(cache.k), wkc[0]) and np.array_equal(host(cache.k_scale), wkc[1])
        return
    # rounded keys: a value within half a step of the exact one; a scale may differ only where the
    # largest value lies on the border of two (not in these inputs)
    assert np.array_equal(host(cache.k_scale), wkc[1])
    got, codes = host(cache.k), wkc[0]
    stored = np.zeros(k.shape, bool)
    for t, s in enumerate(slots):
        stored[s // P, :, s % P] = True
        scale = wkc[1][s // P][:, None]
        y = oracle.fp8_decode(got[s // P, :, s % P]) * scale
        half = np.maximum(np.abs(want[t]) * 2.0 ** -4, scale * 2.0 ** -10)
        assert (np.abs(y - want[t]) <= half + 32 * EPS * size[t] + 2.0 ** -4 * 32 * EPS * size[t]).all()
    assert np.array_equal(got[~stored], codes[~stored])


def test_store_scales_grow_and_odd_values():
    """Later tokens of a page with larger values: the older codes are rounded to the grown scale; with
    smaller ones the scale stays; zeros, infinities and NaN."""
    m = rdg()
    P, D = 16, 64
    step, table, cache, (k, v, ks, vs) = begin(m, [0], [9], P, 1, D, 5)
    rng = np.random.default_rng(6)
    rows = rng.standard_normal((9, 3 * D)).astype(np.float32)
    rows[0] = 0                                    # a first token of zeros
    rows[1] *= 1e-3
    rows[2] *= 40
    rows[3] *= 1e-6
    rows[4, D + 3], rows[4, D + 5], rows[4, 2 * D + 7] = np.inf, -np.inf, np.nan
    rows[5] *= 1e30
    rows[6] = 0
    rows[7] *= 1e-42                               # subnormal
    rows[8, D:] = 448 * 2.0 ** 100
    q_out = torch.empty(1, 1, D, device=DEV)
    for t in range(9):
        one = m.KvStep(1, step.max_blocks, P, step.n_pages, 1, DEV)
        one.block_table.copy_(step.block_table)
        m.rdg_kv_plan(one, dev([t]), dev([1]), dev([table[0, 0]]), dev([1 if t == 0 else 0]), dev([0]))
        m.rdg_qk_norm_rope_store(dev(rows[t:t + 1], torch.float32), 1, 1, D, None, None, 0.0, None, 0, False, one, cache,
                                 q_out)
        assert m.rdg_check_status(one) == (0, 0)
        slots = host(one.slots)
        k, ks = paged.store(k, ks, slots, [0], rows[t:t + 1, D:2 * D].reshape(1, 1, D))
        v, vs = paged.store(v, vs, slots, [0], rows[t:t + 1, 2 * D:].reshape(1, 1, D))
        assert np.array_equal(host(cache.k_scale), ks) and np.array_equal(host(cache.v_scale), vs), t
        assert np.array_equal(host(cache.k), k) and np.array_equal(host(cache.v), v), t
        assert np.array_equal(host(q_out)[0, 0], rows[t, :D].astype(np.float64))


def test_store_every_code():
    """All fp32 values on and beside the borders between codes, under scale 2^-3."""
    m = rdg()
    D = 256
    vals = oracle.fp8_decode(np.arange(0x7f))
    mid = (vals[1:] + vals[:-1]) / 2
    x = np.concatenate([vals, mid, np.nextafter(mid.astype(np.float32), np.float32(np.inf)),
                        np.nextafter(mid.astype(np.float32), np.float32(-np.inf))]).astype(np.float32) / 8
    x = np.concatenate([x, -x])
    x = np.concatenate([x, np.zeros(-len(x) % D, np.float32)]).reshape(-1, D)
    x[:, 0] = 56.0
    step, _, cache, (k, v, ks, vs) = begin(m, [0], [len(x)], 16, 1, D, 7)
    m.rdg_qk_norm_rope_store(dev(np.concatenate([x, x], 1), torch.float32), 0, 1, D, None, None, 0.0, None, 0, False,
                             step, cache, None)
    want = paged.store(k, ks, host(step.slots), host(step.seg_tok), x[:, None])
    assert np.array_equal(host(cache.k), want[0]) and np.array_equal(host(cache.k_scale), want[1])


def test_store_skips_tokens_without_a_slot_and_reports_positions():
    m = rdg()
    step, _, cache, (k, v, ks, vs) = begin(m, [0, 0], [3, 2], 16, 1, 64, 8)
    step.slots[:3] = -1
    step.seg_tok.fill_(-1)
    step.seg_tok[0] = 3
    step.positions[4] = 50
    x = torch.randn(5, 3 * 64, device=DEV)
    q = torch.empty(5, 1, 64, device=DEV)
    cs = torch.cat([torch.ones(4, 8), torch.zeros(4, 8)], 1).to(DEV)
    m.rdg_qk_norm_rope_store(x, 1, 1, 64, None, None, 0.0, cs, 16, False, step, cache, q)
    assert m.rdg_check_status(step) == (m.RDG_EDATA, 4)
    want = paged.store(v, vs, host(step.slots), [3], host(x).reshape(5, 3, 64)[:, 2:])
    assert np.array_equal(host(cache.v), want[0])
    # a segment whose slot lies outside the cache is reported and not stored
    before = host(cache.v)
    step.slots[3] = step.n_pages * 16
    step.positions.zero_()
    step.status.zero_()
    m.rdg_qk_norm_rope_store(x, 1, 1, 64, None, None, 0.0, cs, 16, False, step, cache, q)
    assert m.rdg_check_status(step) == (m.RDG_EDATA, 3)
    assert np.array_equal(host(cache.v), before)


def test_queries_alone():
    """n_kv = 0: heads normed and turned with no cache."""
    m = rdg()
    step = m.KvStep(1, 1, 16, 1, 5, DEV)
    step.positions.copy_(dev([0, 1, 2, 3, 4]))
    x = torch.randn(5, 3 * 128, device=DEV)
    w = torch.rand(128, device=DEV) + 0.5
    q = torch.empty(5, 3, 128, device=DEV)
    m.rdg_qk_norm_rope_store(x, 3, 0, 128, w, None, 1e-6, None, 0, False, step, None, q)
    want = paged.norm(host(x).reshape(5, 3, 128), host(w), 1e-6)
    assert (np.abs(host(q) - want) <= 32 * EPS * np.abs(want)).all()


# ---------------------------------------------------------------- attention
def values(codes, scales):
    return oracle.fp8_decode(codes) * np.asarray(scales, np.float64)[..., None, None]


def finite_codes(rng, shape):
    c = rng.integers(0, 256, shape).astype(np.uint8)
    return np.where((c & 0x7f) == 0x7f, 0x30, c).astype(np.uint8)


def attn_case(kv, q, P, n_q, n_kv, D, dtype, seed, q_gain=1.0):
    """kv: cached tokens with the new ones.  Rows that hold no token are NaN codes."""
    m = rdg()
    rng = np.random.default_rng(seed)
    kv, q = np.array(kv), np.array(q)
    nb = paged.pages_of(kv, P)
    n_pages, B = int(nb.sum()) + 2, max(int(nb.max()), 1)
    ids, at = rng.permutation(n_pages), 0
    table = np.full((len(kv), B), -1)
    k, v = (np.full((n_pages, n_kv, P, D), 0x7f, np.uint8) for _ in range(2))
    for r, n in enumerate(nb):
        table[r, :n] = ids[at:at + n]
        at += n
        for b in range(n):
            rows = min(P, kv[r] - b * P)
            for c in (k, v):
                c[table[r, b], :, :rows] = finite_codes(rng, (n_kv, rows, D))
    ks, vs = (np.exp2(rng.integers(-9, -5, (n_pages, n_kv))).astype(np.float32) for _ in range(2))
    T = int(q.sum())
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.from_numpy(q_gain * rng.standard_normal((T, n_q, D))).to(tt).to(DEV)
    step = m.KvStep(len(kv), B, P, n_pages, T, DEV)
    step.block_table.copy_(dev(table))
    step.cu_q.copy_(dev(np.concatenate([[0], np.cumsum(q)])))
    step.kv_len.copy_(dev(kv))
    cache = m.KvCache(dev(k, torch.uint8), dev(v, torch.uint8), dev(ks, torch.float32), dev(vs, torch.float32))
    return dict(m=m, step=step, cache=cache, x=x, kv=kv, q=q, table=table, k=k, v=v, ks=ks, vs=vs, dtype=dtype)


def call(c, scale, causal=True, window=0, out=None, max_q=None, max_kv=None, stream=None):
    m, x = c["m"], c["x"]
    T, n_q, D = x.shape
    max_q = max(int(c["q"].max()), 1) if max_q is None else max_q
    max_kv = max(int(c["kv"].max()), 1) if max_kv is None else max_kv
    dt = m.RDG_BF16 if c["dtype"] == "bf16" else m.RDG_F32
    n = m.rdg_paged_attention_workspace_bytes(c["cache"], T, len(c["kv"]), n_q, max_q, max_kv, dt)
    work = torch.full((n,), 255, dtype=torch.uint8, device=DEV)      # NaN where a part is not written
    out = torch.full_like(x, 7.0) if out is None else out
    lse = torch.full((T, n_q), 7.0, device=DEV)
    m.rdg_paged_attention(x, c["step"], c["cache"], max_q, max_kv, scale, out, lse, work, causal=causal, window=window,
                          stream=stream)
    return out, lse


def check(c, out, lse, scale, causal=True, window=0):
    D = c["x"].shape[2]
    k, v = values(c["k"], c["ks"]), values(c["v"], c["vs"])
    k, v = np.where(np.isnan(k), 0, k), np.where(np.isnan(v), 0, v)  # rows of no token
    want, wl, spread, size = paged.attention(host(c["x"]), host(c["step"].cu_q), c["kv"], c["table"], k, v, scale, causal,
                                             window)
    d = (D + 4) * EPS * size
    share = 2 * d + (int(c["kv"].max()) + 64) * 2 * EPS + (2.0 ** -8 if c["dtype"] == "bf16" else 3 * 2.0 ** -23)
    tol = share[..., None] * spread + (2.0 ** -8 if c["dtype"] == "bf16" else 4 * EPS) * np.abs(want)
    tol = tol + int(c["kv"].max()) * 2.0 ** -126 * np.abs(v).max()
    got, gl = host(out), host(lse)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / np.maximum(tol, 1e-30)).max())
    assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
    fin = ~np.isneginf(wl)
    lt = d + (int(c["kv"].max()) + 64) * 2 * EPS + 8 * EPS * np.abs(np.where(fin, wl, 0))
    assert (np.abs(gl[fin] - wl[fin]) <= lt[fin]).all()
    assert (got[~fin] == 0).all()


ATTNS = [
    # kv (with the new tokens), q, P, n_q, n_kv, D
    ([1], [1], 16, 1, 1, 64),
    ([1, 2, 15, 16, 17, 63, 64, 65], [1] * 8, 16, 8, 2, 128),
    ([255, 256, 257, 513, 0], [1, 1, 1, 1, 0], 64, 16, 1, 128),
    ([4097, 300], [1, 1], 32, 4, 2, 64),
    ([4200, 31], [1, 1], 128, 6, 2, 256),
    ([700, 9, 64, 0, 130], [5, 3, 4, 0, 1], 16, 28, 4, 128),
    ([200, 64], [17, 64], 32, 3, 1, 64),
    ([150, 90], [150, 33], 64, 8, 2, 128),
    ([333], [200], 16, 5, 5, 256),
    ([520, 77, 1], [300, 1, 1], 128, 4, 1, 128),
    ([2, 0, 3], [6, 4, 3], 16, 8, 4, 64),               # more queries than keys: the first see nothing
    ([600], [2], 64, 64, 1, 128),
    ([1300], [1300], 16, 2, 1, 64),                     # more than 1024 keys in one tile's walk
    ([3000, 40], [40, 40], 32, 8, 2, 128),              # few tiles: their keys are split too
    ([2100, 1, 0], [33, 1, 0], 128, 4, 1, 256),
]
# long and short requests together, for each width
MIXES = [([400, 70, 9, 0, 33, 1200], [150, 1, 9, 0, 3, 2], 16, 8, 2, D) for D in (64, 128, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(ATTNS)))
def test_attention_equals_the_oracle(case, dtype):
    c = attn_case(*ATTNS[case], dtype, 40 + case, q_gain=2.0)
    scale = 0.7 * c["x"].shape[2] ** -0.5
    out, lse = call(c, scale)
    assert c["m"].rdg_check_status(c["step"]) == (0, 0)
    check(c, out, lse, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 16, 65, 300])
@pytest.mark.parametrize("case", [1, 2, 3, 5, 7, 8, 10])
def test_attention_with_a_window(case, window, dtype):
    c = attn_case(*ATTNS[case], dtype, 60 + case)
    out, lse = call(c, 0.1, window=window)
    assert c["m"].rdg_check_status(c["step"]) == (0, 0)
    check(c, out, lse, 0.1, window=window)


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("case", range(len(MIXES)))
def test_mixed_batches(case, window):
    c = attn_case(*MIXES[case], "bf16", 70 + case)
    out, lse = call(c, 0.1, window=window)
    assert c["m"].rdg_check_status(c["step"]) == (0, 0)
    check(c, out, lse, 0.1, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_heads", [4, 16])
@pytest.mark.parametrize("window", [1 << 30, (1 << 31) - 1])
def test_windows_of_any_length(window, q_heads, dtype):
    """A window longer than any request hides nothing, also where a request has more rows than keys."""
    c = attn_case([2, 90, 0, 130], [9, 90, 3, 2], 16, q_heads, 2, 64, dtype, 73)
    out, lse = call(c, 0.1, window=window)
    assert c["m"].rdg_check_status(c["step"]) == (0, 0)
    check(c, out, lse, 0.1)


def test_more_requests_than_lanes():
    rng = np.random.default_rng(7)
    kv = rng.integers(0, 90, 150)
    q = np.minimum(kv, np.where(rng.random(150) < 0.1, 40, rng.integers(0, 3, 150)))
    c = attn_case(kv, q, 16, 4, 1, 64, "bf16", 71)
    out, lse = call(c, 0.1)
    check(c, out, lse, 0.1)


@pytest.mark.parametrize("D", [64, 128])
def test_long_prefill(D):
    """Enough rows for the 256-row tiles: two prompts, checked head by head in float64 on the GPU."""
    c = attn_case([2500, 1800], [2500, 1800], 64, 32, 8, D, "bf16", 72)
    out, lse = call(c, D ** -0.5)
    assert c["m"].rdg_check_status(c["step"]) == (0, 0)
    scale, t0 = D ** -0.5, 0
    for r, n in enumerate((2500, 1800)):
        pages = c["table"][r, :-(-n // 64)]
        hidden = torch.ones(n, n, dtype=torch.bool, device=DEV).triu_(1)
        for h in range(0, 32, 5):
            k, v = (torch.from_numpy(np.nan_to_num(values(a[pages, h // 4], s[pages, h // 4])).reshape(-1, D)[:n]).to(DEV)
                    for a, s in ((c["k"], c["ks"]), (c["v"], c["vs"])))
            x = c["x"][t0:t0 + n, h].double()
            s = (scale * x @ k.T).masked_fill_(hidden, -float("inf"))
            size = (scale * x.abs() @ k.abs().T).masked_fill_(hidden, 0).amax(-1)
            p = torch.softmax(s, -1)
            want, spread = p @ v, p @ v.abs()
            d = (D + 4) * EPS * size
            tol = (2 * d + (n + 64) * 2 * EPS + 2.0 ** -8)[:, None] * spread + 2.0 ** -8 * want.abs()
            assert ((out[t0:t0 + n, h].double() - want).abs() <= tol + n * 2.0 ** -126 * v.abs().max()).all()
            wl = torch.logsumexp(s, -1)
            assert ((lse[t0:t0 + n, h].double() - wl).abs() <= d + (n + 64) * 2 * EPS + 8 * EPS * wl.abs()).all()
        t0 += n


@pytest.mark.parametrize("case", [1, 5, 6, 8, 10])
def test_attention_without_a_causal_mask(case):
    c = attn_case(*ATTNS[case], "bf16", 80 + case)
    out, lse = call(c, 0.1, causal=False)
    check(c, out, lse, 0.1, causal=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kv,q,window", [([300, 70], [4, 9], 0), ([300, 70], [4, 9], 20), ([200, 90], [150, 90], 0),
                                         ([700], [300], 100)])
def test_nan_reaches_only_the_queries_that_see_it(kv, q, window, dtype):
    """NaN codes in cached tokens' keys and values: queries whose mask hides them
    are what they are without, the others are NaN."""
    c = attn_case(kv, q, 16, 8, 2, 64, dtype, 90)
    out, lse = call(c, 0.1, window=window)
    at = [(0, kv[0] - 2, "v"), (0, kv[0] - q[0] - 30, "v"), (0, kv[0] - 1, "k")]
    for r, key, what in at:
        page, row = c["table"][r, key // 16], key % 16
        d = 5
        (c["cache"].v if what == "v" else c["cache"].k)[page, 1, row, d] = 0xff
    bad, bad_lse = call(c, 0.1, window=window)
    assert torch.equal(bad[:, :4], out[:, :4])                       # the other key head
    pos = np.concatenate([a - n + np.arange(n) for a, n in zip(kv, q)])
    req = np.repeat(np.arange(len(kv)), q)
    nan_row, nan_d = np.zeros(len(pos), bool), np.zeros(len(pos), bool)
    for r, key, what in at:
        sees = (req == r) & (pos >= key) & ((pos < key + window) if window else True)
        if what == "k":
            nan_row |= sees
        else:
            nan_d |= sees
    got, ref = host(bad)[:, 4:], host(out)[:, 4:]
    want_nan = np.zeros(got.shape, bool)
    want_nan[nan_row] = True
    want_nan[nan_d, :, 5] = True
    assert np.array_equal(np.isnan(got), want_nan)
    assert np.array_equal(got[~want_nan], ref[~want_nan])
    assert np.array_equal(np.isnan(host(bad_lse)[:, 4:]), np.repeat(nan_row[:, None], 4, 1))


def test_attention_of_peaked_and_infinite_logits():
    c = attn_case([900, 65], [1, 1], 16, 4, 2, 128, "f32", 95, q_gain=60.0)
    out, lse = call(c, 1.0)
    check(c, out, lse, 1.0)
    c["x"][1, 2, 0] = float("inf")           # inf * code is +-inf (NaN for a zero code): no finite softmax
    out, lse = call(c, 1.0)
    assert torch.isnan(out[1, 2]).all() and torch.isfinite(out[0]).all() and torch.isfinite(out[1, [0, 1, 3]]).all()


def test_strides_streams_and_tight_bounds():
    """q and out inside wider rows, on another stream, bounds larger than the lengths."""
    c = attn_case([300, 64, 129], [3, 1, 2], 16, 6, 2, 128, "bf16", 96)
    ref, ref_lse = call(c, 0.1)
    T = c["x"].shape[0]
    wide = torch.randn(T, 9, 128, device=DEV).bfloat16()
    wide[:, 2:8] = c["x"]
    hold = torch.full((T, 8, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c["x"] = wide[:, 2:8]
    out, lse = call(c, 0.1, out=hold[:, 1:7], max_q=50, max_kv=1000, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert (host(hold[:, 0]) == 5).all() and (host(hold[:, 7]) == 5).all()
    c["x"] = wide[:, 2:8].contiguous()
    check(c, out, lse, 0.1)
    assert torch.equal(call(c, 0.1)[0], ref)                          # and again: the same bits


def test_bad_tables_and_lengths_are_reported():
    c = attn_case([100, 40], [1, 1], 16, 4, 2, 64, "bf16", 97)
    m = c["m"]
    ref, _ = call(c, 0.1)
    c["step"].block_table[1, 1] = 10 ** 6
    out, _ = call(c, 0.1)
    assert m.rdg_check_status(c["step"]) == (m.RDG_EDATA, 1)
    assert torch.equal(out[0], ref[0])
    c["step"].status.zero_()
    c["step"].block_table.copy_(dev(c["table"]))
    out, _ = call(c, 0.1, max_kv=64)                                  # request 0 is longer
    assert m.rdg_check_status(c["step"]) == (m.RDG_EDATA, 0)
    assert torch.equal(out[1], ref[1])


@pytest.mark.parametrize("q,max_q", [([2, 3], 2), ([9, 90], 40), ([90, 9], 40)])
def test_requests_past_max_q_are_left_out(q, max_q):
    """And nothing of them stays behind: the same buffers then give the right results."""
    c = attn_case([700, 700], q, 16, 4, 2, 64, "bf16", 99)
    m = c["m"]
    ref, _ = call(c, 0.1)
    out, _ = call(c, 0.1, max_q=max_q)
    long = 1 if q[1] > max_q else 0
    assert m.rdg_check_status(c["step"]) == (m.RDG_EDATA, long)
    t0 = q[0] if long else 0
    assert (out[t0:t0 + q[long]] == 7).all()
    keep = slice(0, q[0]) if long else slice(q[0], None)
    assert torch.equal(out[keep], ref[keep]) or torch.allclose(out[keep].float(), ref[keep].float(), atol=2.0 ** -7)
    assert torch.equal(call(c, 0.1)[0], ref)


@pytest.mark.parametrize("q", [1, 130])
def test_offsets_past_32_bits(q):
    """A cache of more than 4 GiB of codes whose requests live in its last pages."""
    m = rdg()
    P, n_kv, D = 128, 8, 256
    n_pages = (1 << 32) // (P * n_kv * D) + 40
    c = attn_case([300, 129], [q, 1], P, 8, n_kv, D, "bf16", 98)
    small = c["cache"]
    shape = (n_pages, n_kv, P, D)
    k, v = (torch.empty(shape, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.ones(shape[:2], device=DEV) for _ in range(2))
    move = n_pages - small.n_pages
    for big, part in ((k, small.k), (v, small.v), (ks, small.k_scale), (vs, small.v_scale)):
        big[move:] = part
    ref, ref_lse = call(c, 0.1)
    c["cache"] = m.KvCache(k, v, ks, vs)
    step = m.KvStep(2, c["step"].max_blocks, P, n_pages, q + 1, DEV)
    step.block_table.copy_(torch.where(c["step"].block_table < 0, -1, c["step"].block_table + move))
    step.cu_q.copy_(c["step"].cu_q)
    step.kv_len.copy_(c["step"].kv_len)
    c["step"] = step
    out, lse = call(c, 0.1)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    # and the store: the last tokens again, at 64-bit offsets
    x = torch.randn(1, (8 + 2 * n_kv) * D, device=DEV).bfloat16()
    one = m.KvStep(1, 1, P, n_pages, 1, DEV)
    one.slots.fill_(n_pages * P - 1)
    one.seg_tok[0] = 0
    m.rdg_qk_norm_rope_store(x, 8, n_kv, D, None, None, 0.0, None, 0, False, one, c["cache"],
                             torch.empty(1, 8, D, dtype=torch.bfloat16, device=DEV))
    want, scale = paged.store(host(k[-1:]), host(vs[-1:]), [P - 1], [0], host(x).reshape(1, -1, D)[:, 8 + n_kv:])
    assert np.array_equal(host(v[-1, :, P - 1]), want[0, :, P - 1])


def test_a_captured_step_replays():
    """Plan, store and attention recorded as one graph and replayed as a decode
    loop: each replay equals the same step run eagerly on a second state."""
    m = rdg()
    R, P, n_q, n_kv, D, B = 5, 16, 8, 2, 64, 6
    n_pages = R * B
    rng = np.random.default_rng(1)

    def state():
        step = m.KvStep(R, B, P, n_pages, R, DEV)
        return dict(step=step, cache=m.KvCache.empty(n_pages, n_kv, P, D, DEV), free=dev(np.arange(n_pages)),
                    n=dev([n_pages]), q=torch.empty(R, n_q, D, dtype=torch.bfloat16, device=DEV),
                    out=torch.zeros(R, n_q, D, dtype=torch.bfloat16, device=DEV),
                    lse=torch.zeros(R, n_q, device=DEV))

    ones = dev([1, 1, 0, 1, 1])
    x = torch.empty(R, (n_q + 2 * n_kv) * D, dtype=torch.bfloat16, device=DEV)
    cs = torch.rand(B * P, D, device=DEV)
    w = torch.rand(D, device=DEV)
    work = torch.empty(m.rdg_paged_attention_workspace_bytes(m.KvCache.empty(1, n_kv, P, D, DEV), R, R, n_q, 1, B * P,
                                                             m.RDG_BF16), dtype=torch.uint8, device=DEV)

    def step_of(s):
        m.rdg_kv_plan(s["step"], s["step"].kv_len, ones, s["free"], s["n"], s["n"])
        m.rdg_qk_norm_rope_store(x, n_q, n_kv, D, w, w, 1e-6, cs, D, False, s["step"], s["cache"], s["q"])
        m.rdg_paged_attention(s["q"], s["step"], s["cache"], 1, B * P, 0.125, s["out"], s["lse"], work)

    a, b = state(), state()
    x.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step_of(state())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_of(a)
    for i in range(40):
        x.copy_(torch.from_numpy(rng.standard_normal(x.shape)))
        graph.replay()
        torch.cuda.synchronize()
        step_of(b)
        for f in ("out", "lse", "n"):
            assert torch.equal(a[f], b[f]), (i, f)
        assert torch.equal(a["cache"].k, b["cache"].k) and torch.equal(a["step"].kv_len, b["step"].kv_len)
    assert m.rdg_check_status(a["step"]) == (0, 0) and host(a["step"].kv_len)[0] == 40
