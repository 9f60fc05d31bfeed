"""CPU oracle for the paged 8-bit key/value cache (test infrastructure: only
the test suite may import it; it shares no code with the library).

The definitions, written plainly in Python and numpy float64: the step plan
(pages and slots from the requests' lengths), the hand-back of pages, the
query/key norm with rotation, the store into e4m3 pages with one power-of-two
scale for each page and head, and the attention over such a cache.
"""
import math

import numpy as np

import oracle

OK, EDATA, ECAPACITY = 0, -6, -2


def pages_of(tokens, page_rows):
    return (tokens + page_rows - 1) // page_rows


def kv_plan(kv_len, q_len, table, free_list, n_free, page_rows, t_cap, seg_cap, n_pages=1 << 31):
    """One step: (table, cu_q, kv_len, slots, positions, seg_tok, n_free, status)."""
    P, table = page_rows, np.array(table)
    R, max_blocks = table.shape
    slots, positions = np.full(t_cap, -1), np.zeros(t_cap, int)
    segs, cu, out_len = [], [0], []
    bad = full = bad_page = None
    taken, left = 0, n_free
    stop = False            # a request ran out of pages: no later one gets any
    t = 0
    for r in range(R):
        kv, q = int(kv_len[r]), int(q_len[r])
        ok = True
        if kv < 0 or q < 0:
            bad = r if bad is None else bad
            kv, q, ok = max(kv, 0), 0, False
        need = pages_of(kv + q, P) - pages_of(kv, P)
        if ok and pages_of(kv + q, P) > max_blocks:
            need, ok = 0, False
            full = r if full is None else full
        if ok and t + q > t_cap:
            stop, ok = stop or need > 0, False
            full = r if full is None else full
        if ok and need > 0 and (stop or taken + need > n_free):
            stop, ok = True, False
            full = r if full is None else full
        if ok:
            for i in range(need):
                page = free_list[n_free - 1 - taken - i]
                table[r, pages_of(kv, P) + i] = page if 0 <= page < n_pages else -1
            taken += need
            left = n_free - taken
        for i in range(q):
            if t + i >= t_cap:
                break
            p = kv + i
            positions[t + i] = p
            if ok:
                page = table[r, p // P]
                if 0 <= page < n_pages:
                    slots[t + i] = page * P + p % P
                else:
                    bad_page = r if bad_page is None else bad_page
                if i == 0 or p % P == 0:
                    segs.append(t + i)
        t += q
        cu.append(min(t, t_cap))
        out_len.append(kv + q if ok else kv)
    seg = np.full(seg_cap, -1)
    seg[:len(segs)] = segs
    status = ((EDATA, bad) if bad is not None else (ECAPACITY, full) if full is not None else
              (EDATA, bad_page) if bad_page is not None else (OK, 0))
    return table, np.array(cu), np.array(out_len), slots, positions, seg, left, status


def kv_trim(kv_len, new_len, table, free_list, n_free, page_rows):
    """(table, kv_len, free_list, n_free, status); free_list has a place for every page."""
    P, table, free, n_pages = page_rows, np.array(table), list(free_list[:n_free]), len(free_list)
    R, max_blocks = table.shape
    before = np.array(table), np.array(kv_len), list(free)
    out, bad, bad_page, freed = [], None, None, 0
    for r in range(R):
        kv, to = int(kv_len[r]), int(new_len[r])
        if kv < 0 or kv > max_blocks * P or to < 0 or to > kv:
            bad = r if bad is None else bad
            out.append(kv)
            continue
        for b in range(pages_of(to, P), pages_of(kv, P)):
            if 0 <= table[r, b] < n_pages:
                free.append(table[r, b])
            else:
                bad_page = r if bad_page is None else bad_page
            table[r, b] = -1
            freed += 1
        out.append(to)
    if n_free + freed > n_pages:
        return before[0], before[1], before[2], n_free, (EDATA, bad) if bad is not None else (ECAPACITY, freed)
    bad = bad_page if bad is None else bad
    return table, np.array(out), free, len(free), (EDATA, bad) if bad is not None else (OK, 0)


def norm(x, weight, eps):
    x = np.asarray(x, np.float64)
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def rotate(x, cos, sin, neighbours):
    """x [..., head_dim], cos / sin [..., rot_dim / 2]: the pairs as complex numbers, turned."""
    x = np.array(x, np.float64)
    half = cos.shape[-1]
    turn = np.asarray(cos, np.float64) + 1j * np.asarray(sin, np.float64)
    a = slice(0, 2 * half, 2) if neighbours else slice(0, half)
    b = slice(1, 2 * half, 2) if neighbours else slice(half, 2 * half)
    z = (x[..., a] + 1j * x[..., b]) * turn
    x[..., a], x[..., b] = z.real, z.imag
    return x


def page_scale(amax):
    """The smallest 2^k, k in [-126, 127], with amax <= 448 * 2^k."""
    if not amax > 0:
        return 2.0 ** -126
    m, e = math.frexp(amax / 448.0)           # amax / 448 = m 2^e, m in [0.5, 1)
    return 2.0 ** min(127, max(-126, e - 1 if m == 0.5 else e))


def store(codes, scales, slots, seg_tok, rows):
    """rows [T, heads, head_dim] into copies of codes [pages, heads, P, head_dim] and scales [pages, heads]."""
    codes, scales = np.array(codes), np.array(scales, np.float64)
    P, T = codes.shape[2], len(slots)
    for lead in seg_tok:
        if lead < 0:
            continue
        page, off = divmod(int(slots[lead]), P)
        n = 1
        while off + n < P and lead + n < T and slots[lead + n] == slots[lead] + n:
            n += 1
        for h in range(codes.shape[1]):
            x = np.asarray(rows[lead:lead + n, h], np.float64)
            finite = np.abs(x[np.isfinite(x)])
            s = page_scale(finite.max() if finite.size else 0.0)
            if off:
                s = max(s, scales[page, h])
                if s > scales[page, h]:
                    old = oracle.fp8_decode(codes[page, h, :off]) * (scales[page, h] / s)
                    codes[page, h, :off] = encode(old)
            codes[page, h, off:off + n] = encode(x / s)
            scales[page, h] = s
    return codes, scales


def encode(x):
    """e4m3 codes, nearest even; infinities saturate, NaN is 0x7f."""
    x = np.asarray(x, np.float64)
    nan = np.isnan(x)
    v = np.where(nan, 0.0, np.clip(x, -448.0, 448.0))
    mag = np.abs(v)
    e = np.maximum(np.frexp(mag)[1] - 1, -6)
    step = np.exp2(e - 3.0)
    q = np.rint(mag / step) * step            # numpy rounds halves to even
    e = np.where(q > 0, np.maximum(np.frexp(q)[1] - 1, -6), -6)
    code = np.where(q < 2.0 ** -6, q * 512, (e + 7) * 8 + (q / np.exp2(e) - 1) * 8).astype(np.int64)
    return np.where(nan, 0x7f, np.where(np.signbit(v), 0x80, 0) | code).astype(np.uint8)


def attention(q, cu_q, kv_len, table, k, v, scale, causal=True, window=0):
    """q [T, n_q, D]; k, v [pages, heads, P, D] values.  Returns (out, lse, spread): spread is
    each element's sum_j p_j |v_j|, and the row's largest scale * sum_d |q_d k_jd| in lse's shape, for tolerances."""
    q = np.asarray(q, np.float64)
    T, n_q, D = q.shape
    heads, P = k.shape[1:3]
    out, spread = np.zeros((T, n_q, D)), np.zeros((T, n_q, D))
    lse, size = np.full((T, n_q), -np.inf), np.zeros((T, n_q))
    for r in range(len(kv_len)):
        n, kv = int(cu_q[r + 1] - cu_q[r]), int(kv_len[r])
        if kv == 0:
            continue
        blocks = table[r][:pages_of(kv, P)]
        for i in range(n):
            pos = kv - n + i
            hi = min(kv, pos + 1) if causal else kv
            lo = max(0, pos - window + 1) if window else 0
            if hi <= lo:
                continue
            t = int(cu_q[r]) + i
            for h in range(n_q):
                kh = h // (n_q // heads)
                kk = np.concatenate(list(k[blocks, kh]))[lo:hi]
                vv = np.concatenate(list(v[blocks, kh]))[lo:hi]
                x = scale * (kk @ q[t, h])
                top = x.max()
                p = np.exp(x - top)
                out[t, h] = p @ vv / p.sum()
                spread[t, h] = p @ np.abs(vv) / p.sum()
                lse[t, h] = top + math.log(p.sum())
                size[t, h] = scale * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, lse, spread, size
