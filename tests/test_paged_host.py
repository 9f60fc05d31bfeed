"""Host-side checks of the paged-cache entry points: struct layouts, size
queries, and every refusal, which comes before anything is enqueued."""
import ctypes

import pytest

A = 0x100000  # stand-in device address: 16-byte aligned, never dereferenced (each call fails its checks first)


def _rdg():
    import routing_dispatch_grouped_amd as rdg
    return rdg


def _step(n_req=3, max_blocks=8, page_rows=16, n_pages=40, t_cap=64, seg_cap=64, **null):
    rdg = _rdg()
    s = rdg.rdg_kv_step(n_req, max_blocks, page_rows, n_pages, t_cap, seg_cap, *([A] * 8))
    for f, v in null.items():
        setattr(s, f, v)
    return s


def _cache(n_pages=40, page_rows=16, n_kv=2, head_dim=128, **null):
    rdg = _rdg()
    c = rdg.rdg_kv_cache(n_pages, page_rows, n_kv, head_dim, A, A, A, A)
    for f, v in null.items():
        setattr(c, f, v)
    return c


def test_struct_layouts_match_the_header():
    rdg = _rdg()
    assert ctypes.sizeof(rdg.rdg_kv_cache) == 4 * 4 + 4 * 8
    assert ctypes.sizeof(rdg.rdg_kv_step) == 6 * 4 + 8 * 8
    assert rdg.rdg_kv_step.work.offset == 24 + 7 * 8


def test_size_queries():
    rdg = _rdg()
    L = rdg._lib
    assert L.rdg_kv_seg_cap(0, 5, 16) == 0
    assert L.rdg_kv_seg_cap(7, 100, 16) == 7            # a segment has a token
    assert L.rdg_kv_seg_cap(1000, 3, 64) == 15 + 6
    assert L.rdg_kv_seg_cap(10, 3, 48) == rdg.RDG_EINVAL
    c = _cache(n_kv=8)
    size = lambda *a: L.rdg_paged_attention_workspace_bytes(ctypes.byref(c), *a)  # noqa: E731
    assert size(0, 1, 32, 1, 100, rdg.RDG_BF16) == 0
    assert size(1, 1, 30, 1, 100, rdg.RDG_BF16) == 0    # 30 query heads over 8 key heads
    assert size(1, 1, 32, 1, 2500, rdg.RDG_BF16) >= 32 * 10 * 130 * 4
    assert L.rdg_kv_step_work_bytes() >= 8


def test_plan_refusals():
    rdg = _rdg()
    L = rdg._lib

    def plan(s, kv=A, q=A, free=A, n=A, out=A):
        return L.rdg_kv_plan(ctypes.byref(s), kv, q, free, n, out, None)

    for bad in (dict(n_req=-1), dict(max_blocks=0), dict(n_pages=0), dict(t_cap=-1), dict(page_rows=48),
                dict(page_rows=8), dict(n_pages=1 << 28), dict(max_blocks=1 << 27), dict(seg_cap=3),
                dict(status=None), dict(work=None), dict(cu_q=None), dict(block_table=None), dict(kv_len=None),
                dict(slots=None), dict(positions=A + 4), dict(seg_tok=None)):
        assert plan(_step(**bad)) == rdg.RDG_EINVAL, bad
    for arg in ("kv", "q", "free", "n", "out"):
        assert plan(_step(), **{arg: None}) == rdg.RDG_EINVAL, arg
    assert plan(_step(n_req=4097, t_cap=0, seg_cap=0)) == rdg.RDG_EUNSUPPORTED
    assert L.rdg_kv_plan(None, A, A, A, A, A, None) == rdg.RDG_EINVAL
    assert L.rdg_kv_trim(ctypes.byref(_step()), A, None, A, A, A, None) == rdg.RDG_EINVAL
    assert L.rdg_kv_trim(ctypes.byref(_step(n_req=5000)), A, A, A, A, A, None) == rdg.RDG_EUNSUPPORTED


def test_store_refusals():
    rdg = _rdg()
    L = rdg._lib

    def store(dt=rdg.RDG_BF16, stride=1024, T=4, n_q=4, n_kv=2, d=128, eps=1e-6, n_pos=99, rot=128, s=None, c=None,
              qkv=A, qo=A, qs=512, cs=A, wq=A, cache=True):
        c = c or _cache()
        return L.rdg_qk_norm_rope_store(qkv, dt, stride, T, n_q, n_kv, d, wq, A, eps, cs, n_pos, rot, 0,
                                        ctypes.byref(s or _step()), ctypes.byref(c) if cache else None, qo, qs, None)

    for bad in (dict(dt=rdg.RDG_FP8_E4M3), dict(stride=1016), dict(stride=1028), dict(T=-1), dict(T=65), dict(n_q=-1),
                dict(eps=-1.0), dict(eps=float("nan")), dict(n_pos=0), dict(rot=8), dict(rot=144), dict(rot=-16),
                dict(qkv=None), dict(qkv=A + 8), dict(qo=None), dict(qs=504), dict(cs=None), dict(cs=A + 4),
                dict(wq=A + 4), dict(cache=False), dict(c=_cache(n_kv=3)), dict(c=_cache(page_rows=32)),
                dict(c=_cache(n_pages=41)), dict(c=_cache(k=None)), dict(c=_cache(v=A + 1)),
                dict(s=_step(slots=None)), dict(s=_step(seg_tok=None)), dict(s=_step(positions=None)),
                dict(s=_step(status=None))):
        assert store(**bad) == rdg.RDG_EINVAL, bad
    assert store(d=96) == rdg.RDG_EUNSUPPORTED
    assert store(T=0, qkv=None, qo=None) == rdg.RDG_OK      # nothing to do, nothing launched


def test_attention_refusals():
    rdg = _rdg()
    L = rdg._lib

    def attn(dt=rdg.RDG_BF16, qs=512, T=4, n_q=4, mq=1, mk=100, scale=0.1, causal=1, window=0, s=None, c=None, q=A,
             out=A, os=512, work=A, wb=1 << 30):
        return L.rdg_paged_attention(q, dt, qs, T, n_q, ctypes.byref(s or _step()), ctypes.byref(c or _cache()), mq, mk,
                                     scale, causal, window, out, os, None, work, wb, None)

    for bad in (dict(dt=3), dict(qs=500), dict(qs=516), dict(os=256), dict(T=-1), dict(n_q=3), dict(n_q=0),
                dict(mq=-1), dict(mk=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(window=-1), dict(window=5, causal=0), dict(q=None), dict(q=A + 2),
                dict(out=None), dict(c=_cache(n_pages=39)), dict(c=_cache(page_rows=64)), dict(c=_cache(n_kv=0)),
                dict(c=_cache(v_scale=None)), dict(s=_step(cu_q=None)), dict(s=_step(kv_len=None)),
                dict(s=_step(block_table=None)), dict(s=_step(status=None)),
                dict(mk=4000, work=None), dict(mk=4000, wb=100), dict(mk=4000, work=A + 8)):
        assert attn(**bad) == rdg.RDG_EINVAL, bad
    assert attn(c=_cache(head_dim=80)) == rdg.RDG_EUNSUPPORTED
    for nothing in (dict(T=0), dict(mq=0), dict(s=_step(n_req=0))):
        assert attn(q=None, **nothing) == rdg.RDG_OK


def test_attention_refuses_more_rows_than_an_int_counts():
    rdg = _rdg()
    L = rdg._lib
    c = _cache()
    for T, n_q, most in ((1 << 29, 4, 0), (1 << 29, 2, 1)):
        assert (L.rdg_paged_attention_workspace_bytes(ctypes.byref(c), T, 2, n_q, 1, 4000, rdg.RDG_BF16) > 0) == most
    assert L.rdg_paged_attention(A, rdg.RDG_BF16, 512, 1 << 29, 4, ctypes.byref(_step()), ctypes.byref(c), 1, 100, 0.1, 1,
                                 0, A, 512, None, A, 1 << 30, None) == rdg.RDG_EINVAL


def test_binding_refuses_tensors_it_would_misread():
    import torch
    rdg = _rdg()
    i32 = dict(dtype=torch.int32)
    step = rdg.KvStep(2, 4, 16, 9, 32, "cpu")
    ok = [torch.zeros(2, **i32), torch.zeros(2, **i32), torch.zeros(9, **i32), torch.zeros(1, **i32),
          torch.zeros(1, **i32)]
    for at, wrong in ((0, torch.zeros(2)), (1, torch.zeros(3, **i32)), (2, torch.zeros(18, **i32)[::2]),
                      (3, torch.zeros(2, **i32))):
        args = list(ok)
        args[at] = wrong
        with pytest.raises(rdg.RdgError) as e:
            rdg.rdg_kv_plan(step, *args)
        assert e.value.code == rdg.RDG_EINVAL
    with pytest.raises(rdg.RdgError):
        rdg.rdg_kv_trim(step, ok[0], ok[1], torch.zeros(8, **i32), ok[3], ok[4])   # not room for every page
    with pytest.raises(rdg.RdgError):
        rdg.KvCache(torch.zeros(9, 2, 16, 64, dtype=torch.int8), torch.zeros(9, 2, 16, 64, dtype=torch.int8), None, None)
    with pytest.raises(rdg.RdgError):
        rdg.KvCache(torch.zeros(9, 2, 16, 64, dtype=torch.uint8), torch.zeros(9, 2, 64, 16, dtype=torch.uint8), None, None)
    cache = rdg.KvCache.empty(9, 2, 16, 64, "cpu")
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    for bad_q, bad_out in ((q.half(), q), (q.transpose(1, 2), q), (q, q.float()), (q, q[:4]), (q[..., :32], q)):
        with pytest.raises(rdg.RdgError) as e:
            rdg.rdg_paged_attention(bad_q, step, cache, 1, 10, 0.1, bad_out)
        assert e.value.code == rdg.RDG_EINVAL
    with pytest.raises(rdg.RdgError):
        rdg.rdg_qk_norm_rope_store(torch.zeros(5, 500, dtype=torch.bfloat16), 4, 2, 64, None, None, 0.0, None, 0, False,
                                   step, cache, q)
