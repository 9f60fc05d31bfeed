"""The paged-cache operators on the GPU at the ends of what they accept, against the oracle."""
import numpy as np
import pytest
import torch

from harness import DEV, rdg
from oracle import paged
from test_gpu_paged import ATTNS, EPS, MIXES, attn_case, begin, call, check, dev, host

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- plan
@pytest.mark.parametrize("bad_q", [-3, -(1 << 31), (1 << 30) + 1, (1 << 31) - 1])
def test_plan_keeps_the_cached_tokens_of_a_request_with_a_bad_length(bad_q):
    """In place, as a serving loop plans: the request keeps its length, table and pages, and its next step goes on."""
    m = rdg()
    P, n_pages = 16, 12
    step = m.KvStep(3, 6, P, n_pages, 60, DEV)
    free, n = dev(np.arange(n_pages)), dev([n_pages])
    m.rdg_kv_plan(step, step.kv_len, dev([10, 40, 5]), free, n, n)
    assert m.rdg_check_status(step) == (0, 0)
    table = host(step.block_table)
    m.rdg_kv_plan(step, step.kv_len, dev(np.array([1, bad_q, 2], np.int32)), free, n, n)
    assert m.rdg_check_status(step) == (m.RDG_EDATA, 1)
    assert list(host(step.kv_len)) == [11, 40, 7] and list(host(step.cu_q)) == [0, 1, 1, 3]
    assert np.array_equal(host(step.block_table), table) and host(n)[0] == n_pages - 5
    m.rdg_kv_plan(step, step.kv_len, dev([0, 9, 0]), free, n, n)
    assert m.rdg_check_status(step) == (0, 0)
    want = [table[1, 2] * P + 8 + i for i in range(8)] + [host(step.block_table)[1, 3] * P]
    assert list(host(step.slots)[:9]) == want and host(n)[0] == n_pages - 6
    m.rdg_kv_trim(step, step.kv_len, dev([0, 0, 0]), free, n, n)
    assert host(n)[0] == n_pages and sorted(host(free)) == list(range(n_pages))     # every page is back


@pytest.mark.parametrize("R,n_bad", [(5, 1), (5, 4), (300, 40), (4096, 1), (4096, 3000)])
def test_trim_keeps_ids_of_no_page_off_the_stack(R, n_bad):
    """Entries outside the cache are reported with the first request that has one and vanish; the other pages come back in
    their order, from one workgroup (5 requests) and from several; a plan then hands out pages of the cache only."""
    m = rdg()
    rng = np.random.default_rng(R + n_bad)
    P, B = 16, 6
    n_pages = R * B
    kv = rng.integers(1, B * P + 1, R)
    held = paged.pages_of(kv, P)
    ids = rng.permutation(n_pages)
    table = np.full((R, B), -1)
    at = np.concatenate([[0], np.cumsum(held)])
    for r in range(R):
        table[r, :held[r]] = ids[at[r]:at[r + 1]]
    keep = np.where(rng.random(R) < 0.5, 0, np.minimum(kv, rng.integers(0, B * P, R)))
    keep[0] = 0
    freed = [(r, b) for r in range(R) for b in range(paged.pages_of(keep[r], P), held[r])]
    for x in rng.permutation(len(freed))[:n_bad]:
        table[freed[x]] = rng.choice([-1, n_pages, (1 << 31) - 1, -(1 << 31)])
    free = np.concatenate([ids[at[-1]:], np.full(at[-1], -1)])
    n_free = n_pages - at[-1]
    step = m.KvStep(R, B, P, n_pages, 2 * R, DEV)
    step.block_table.copy_(dev(table))
    step.kv_len.copy_(dev(kv))
    d_free, d_n = dev(free), dev([n_free])
    m.rdg_kv_trim(step, step.kv_len, dev(keep), d_free, d_n, d_n)
    w_table, w_kv, w_free, w_n, status = paged.kv_trim(kv, keep, table, free, n_free, P)
    assert m.rdg_check_status(step) == status and status[0] == m.RDG_EDATA
    assert np.array_equal(host(step.block_table), w_table) and np.array_equal(host(step.kv_len), w_kv)
    assert host(d_n)[0] == w_n and np.array_equal(host(d_free)[:w_n], w_free)
    assert not host(step.work.view(torch.int32)).any()
    q = np.where(w_kv == 0, 2, 0)
    m.rdg_kv_plan(step, step.kv_len, dev(q), d_free, d_n, d_n)
    assert m.rdg_check_status(step) == (0, 0)
    want = paged.kv_plan(w_kv, q, w_table, w_free, w_n, P, 2 * R, step.seg_tok.numel(), n_pages)
    assert np.array_equal(host(step.block_table), want[0]) and np.array_equal(host(step.slots), want[3])


@pytest.mark.parametrize("R", [4, 300])
def test_plan_writes_no_id_of_no_page(R):
    """Ids outside the cache on the stack: their table entries are -1, their tokens have no slot, the first request is named
    (whichever workgroup comes first), and a trim hands every other page back."""
    m = rdg()
    rng = np.random.default_rng(R)
    P, B = 16, 4
    n_pages = 3 * R
    free = rng.permutation(n_pages)
    bad = rng.permutation(n_pages - 4)[:R // 4] + 4
    free[bad] = rng.choice([-1, n_pages, (1 << 31) - 1], len(bad))
    q = np.full(R, 40)
    step = m.KvStep(R, B, P, n_pages, int(q.sum()), DEV)
    step.block_table.fill_(1)                                    # of an earlier use
    d_free, d_n = dev(free), dev([n_pages])
    m.rdg_kv_plan(step, step.kv_len, dev(q), d_free, d_n, d_n)
    want = paged.kv_plan([0] * R, q, np.full((R, B), 1), free, n_pages, P, int(q.sum()), step.seg_tok.numel(), n_pages)
    for got, ref in zip((step.block_table, step.cu_q, step.kv_len, step.slots, step.positions, step.seg_tok, d_n), want):
        assert np.array_equal(host(got), np.ravel(ref).reshape(got.shape))
    assert m.rdg_check_status(step) == want[-1] and want[-1][0] == m.RDG_EDATA
    m.rdg_kv_trim(step, step.kv_len, dev([0] * R), d_free, d_n, d_n)
    good = np.sort(free[(free >= 0) & (free < n_pages)])
    assert host(d_n)[0] == len(good) and np.array_equal(np.sort(host(d_free)[:len(good)]), good)


# ---------------------------------------------------------------- norm, rotation, store
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 1023, 1024, 2500])
def test_store_of_keys_and_values_alone(T, dtype):
    """No query heads, around and past the number of tokens from which query waves take several heads."""
    m = rdg()
    P, n_kv, D = 64, 2, 64
    step, _, cache, (k, v, ks, vs) = begin(m, [9], [T], P, n_kv, D, T)
    x = torch.from_numpy(np.random.default_rng(T).standard_normal((T, 2 * n_kv * D))).to(DEV)
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    m.rdg_qk_norm_rope_store(x, 0, n_kv, D, None, None, 0.0, None, 0, False, step, cache, None)
    assert m.rdg_check_status(step) == (0, 0)
    rows, slots, seg = host(x).reshape(T, 2 * n_kv, D), host(step.slots), host(step.seg_tok)
    for codes, scales, was, part in ((cache.k, cache.k_scale, (k, ks), rows[:, :n_kv]),
                                     (cache.v, cache.v_scale, (v, vs), rows[:, n_kv:])):
        want = paged.store(*was, slots, seg, part)
        assert np.array_equal(host(codes), want[0]) and np.array_equal(host(scales), want[1])


@pytest.mark.parametrize("n_q", [1, 3, 40])
def test_queries_alone_of_many_tokens(n_q):
    m = rdg()
    T, D = 1300, 128
    step = m.KvStep(1, 1, 16, 1, T, DEV)
    x = torch.randn(T, n_q * D, device=DEV)
    w = torch.rand(D, device=DEV) + 0.5
    q = torch.empty(T, n_q, D, device=DEV)
    m.rdg_qk_norm_rope_store(x, n_q, 0, D, w, None, 1e-6, None, 0, False, step, None, q)
    want = paged.norm(host(x).reshape(T, n_q, D), host(w), 1e-6)
    assert (np.abs(host(q) - want) <= 32 * EPS * np.abs(want)).all()


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("max_kv", [1 << 30, 2147480000, 2147483000, (1 << 31) - 1])
def test_prefill_with_a_bound_of_any_size(max_kv):
    """max_kv far above every request: rows that fill the chip, whose keys are not split, and few rows, whose are."""
    c = attn_case([5000, 700], [1500, 548], 64, 32, 8, 64, "bf16", 110)
    ref, ref_lse = call(c, 0.1)
    out, lse = call(c, 0.1, max_kv=max_kv)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    c = attn_case([3000], [100], 64, 8, 2, 64, "bf16", 111)
    out, lse = call(c, 0.1, max_kv=max_kv)
    assert c["m"].rdg_check_status(c["step"]) == (0, 0)
    check(c, out, lse, 0.1)


LONG = [
    # kv, q, P, n_q, n_kv: few rows a request, whose keys one workgroup walks past the pages that a wave holds at a time
    ([9000, 4100, 300, 0], [1, 1, 1, 0], 64, 8, 2),
    ([4500, 2049, 70], [5, 3, 5], 16, 8, 2),
    ([2500, 1025, 1024], [9, 9, 1], 32, 4, 1),
    ([2500, 3100, 40], [16, 2, 16], 128, 8, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(LONG)))
def test_few_rows_with_a_bound_of_any_size(case, D, dtype):
    """A bound of 2^31 - 1 keys leaves each request one part."""
    c = attn_case(*LONG[case], D, dtype, 120 + case)
    for window in (0, 1500):
        out, lse = call(c, 0.1, window=window, max_kv=(1 << 31) - 1)
        assert c["m"].rdg_check_status(c["step"]) == (0, 0)
        check(c, out, lse, 0.1, window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_row_tiles_past_the_pages_held_at_a_time(D):
    """Long requests' tiles, unsplit under the same bound, whose keys pass two loads of pages."""
    c = attn_case([2600, 1100, 1024], [40, 100, 33], 16, 8, 2, D, "bf16", 125)
    for window in (0, 1500):
        out, lse = call(c, 0.1, window=window, max_kv=(1 << 31) - 1)
        assert c["m"].rdg_check_status(c["step"]) == (0, 0)
        check(c, out, lse, 0.1, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(MIXES)))
def test_mixed_batches_with_a_bound_of_any_size(case, dtype):
    c = attn_case(*MIXES[case], dtype, 130 + case)
    out, lse = call(c, 0.1, max_kv=(1 << 31) - 1)
    assert c["m"].rdg_check_status(c["step"]) == (0, 0)
    check(c, out, lse, 0.1)


def test_nan_past_the_pages_held_at_a_time():
    c = attn_case([2600], [16], 16, 4, 1, 64, "bf16", 140)
    ref, _ = call(c, 0.1, max_kv=(1 << 31) - 1)
    key = 2590                                                   # seen by the last ten queries
    c["cache"].v[c["table"][0, key // 16], 0, key % 16, 7] = 0x7f
    out, _ = call(c, 0.1, max_kv=(1 << 31) - 1)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[6:, :, 7] = True
    assert torch.equal(torch.isnan(out), want) and torch.equal(out[~want], ref[~want])


@pytest.mark.parametrize("case", range(len(ATTNS)))
def test_float_queries_without_a_causal_mask(case):
    c = attn_case(*ATTNS[case], "f32", 150 + case)
    out, lse = call(c, 0.1, causal=False)
    assert c["m"].rdg_check_status(c["step"]) == (0, 0)
    check(c, out, lse, 0.1, causal=False)


def test_many_float_requests_beside_a_long_one():
    """4096 requests under a bound of 4395 queries, all but one of a single token: the launch goes by the batch's
    tokens, not by requests times the bound, which no grid holds."""
    R, D = 4096, 64
    q = np.ones(R, int)
    q[1000] = 300
    kv = np.where(q > 1, 300, 1 + np.arange(R) % 37)
    c = attn_case(kv, q, 16, 64, 4, D, "f32", 160)
    out, lse = call(c, 0.1, max_q=4395)
    assert c["m"].rdg_check_status(c["step"]) == (0, 0)
    ref, ref_lse = call(c, 0.1, max_q=300)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    some = [0, 36, 999, 1000, 1001, 4095]
    few = dict(c, kv=kv[some], table=c["table"][some])
    t0 = np.concatenate([[0], np.cumsum(q)])
    rows = np.concatenate([np.arange(t0[r], t0[r + 1]) for r in some])
    few["x"], few["q"] = c["x"][rows], q[some]
    few["step"] = type("Step", (), dict(cu_q=dev(np.concatenate([[0], np.cumsum(q[some])]))))
    check(few, out[rows], lse[rows], 0.1)
