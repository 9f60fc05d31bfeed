"""Pins of the paged-cache oracle: its e4m3 encoder and page scale against
independent forms, the plan's invariants, and the attention's derivative
structure (a shift of all logits, a permutation of keys, one key)."""
import math

import numpy as np
import pytest

import oracle
from oracle import paged


def test_encoder_matches_the_layer_oracles():
    rng = np.random.default_rng(3)
    v = np.concatenate([rng.uniform(-460, 460, 2000), rng.uniform(-0.02, 0.02, 2000), oracle.fp8_decode(range(0x7f)),
                        [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 464.0, 1e30, -1e30]])
    v = v.astype(np.float32).astype(np.float64)
    assert np.array_equal(paged.encode(v), oracle.fp8_encode(np.clip(v, -448, 448)))
    assert paged.encode([np.nan])[0] == 0x7f
    assert list(paged.encode([np.inf, -np.inf])) == [0x7e, 0xfe]


def test_page_scale_is_the_smallest_that_holds():
    rng = np.random.default_rng(4)
    for amax in np.concatenate([np.exp(rng.uniform(-80, 80, 500)), 448 * np.exp2(np.arange(-20.0, 20))]):
        s = paged.page_scale(amax)
        assert math.log2(s) == int(math.log2(s)) and 448 * s >= amax and 448 * s / 2 < amax
    assert paged.page_scale(0.0) == 2.0 ** -126


@pytest.mark.parametrize("P", [16, 64])
def test_plan_gives_each_page_once_and_trim_takes_it_back(P):
    rng = np.random.default_rng(P)
    R, B, n_pages = 23, 12, 150
    table, free, n_free = np.full((R, B), -1), list(rng.permutation(n_pages)), n_pages
    kv = np.zeros(R, int)
    for step in range(6):
        q = rng.integers(0, 2 * P, R)
        t_cap = int(q.sum()) + 3
        before = kv
        table, cu, kv, slots, pos, seg, n_free, status = paged.kv_plan(kv, q, table, free, n_free, P, t_cap,
                                                                       t_cap // P + 2 * R)
        held = [table[r, b] for r in range(R) for b in range(paged.pages_of(kv[r], P))]
        assert len(set(held)) == len(held) and not set(held) & set(free[:n_free])
        assert len(held) + n_free == n_pages
        used = slots[slots >= 0]
        assert len(set(used)) == len(used) == (kv - before).sum()
        assert len(set(slots[s] // P for s in seg if s >= 0)) == (seg >= 0).sum() == len(set(used // P))
        keep = kv - rng.integers(0, 5, R).clip(max=kv)
        keep[rng.integers(0, R, 3)] = 0
        table, kv, free, n_free, status = paged.kv_trim(kv, keep, table, free + [-1] * (n_pages - len(free))
                                                        if len(free) < n_pages else free, n_free, P)
        assert status == (0, 0) and np.array_equal(kv, keep)
        assert sum(paged.pages_of(x, P) for x in kv) + n_free == n_pages


def test_rotation_and_norm():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((7, 3, 32))
    y = paged.norm(x, np.ones(32), 0.0)
    assert np.allclose((y ** 2).mean(-1), 1)
    ang = rng.uniform(0, 6, (7, 1, 8))
    for nb in (False, True):
        z = paged.rotate(y, np.cos(ang), np.sin(ang), nb)
        assert np.allclose((z ** 2).sum(-1), (y ** 2).sum(-1)) and np.array_equal(z[..., 16:], y[..., 16:])
        assert np.allclose(paged.rotate(z, np.cos(ang), -np.sin(ang), nb), y)


def test_attention_masks_and_lse():
    rng = np.random.default_rng(6)
    k, v = rng.standard_normal((4, 2, 16, 8)), rng.standard_normal((4, 2, 16, 8))
    table = np.array([[3, 1], [0, 2]])
    q = rng.standard_normal((5, 4, 8))
    out, lse, spread, _ = paged.attention(q, [0, 3, 5], [20, 1], table, k, v, 0.3)
    # the second request's first query has position -1: it sees nothing; its second one sees one key
    assert not out[3].any() and np.isneginf(lse[3]).all()
    assert np.allclose(out[4, :2], v[0, 0, 0]) and np.allclose(lse[4, 3], 0.3 * q[4, 3] @ k[0, 1, 0])
    # a window of one: each query sees its own position
    out1, _, _, _ = paged.attention(q, [0, 3, 5], [20, 1], table, k, v, 0.3, window=1)
    assert np.allclose(out1[2, 3], v[1, 1, 3])
    # lse is the derivative's normaliser: d lse / d (logit) sums to one, so a shift of all logits shifts it
    eps = 1e-6
    g = [(paged.attention(q + eps * np.eye(8)[d], [0, 3, 5], [20, 1], table, k, v, 0.3)[1][1, 0] - lse[1, 0]) / eps
         for d in range(8)]
    kk = np.concatenate([k[3, 0], k[1, 0]])[:19]
    p = np.exp(0.3 * kk @ q[1, 0] - lse[1, 0])
    assert np.isclose(p.sum(), 1) and np.allclose(g, 0.3 * p @ kk, atol=1e-5)
