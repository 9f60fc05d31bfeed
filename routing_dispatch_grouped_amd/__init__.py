"""Thin Python binding of librdg.so (include/rdg.h): argument marshalling only.

Every function carries the C entry point's name and forwards torch device
tensors as raw pointers plus torch's current HIP stream.  Nothing here
computes any step of the layer.  Importing fails loudly when the built
library is missing: there is no fallback path.
"""
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librdg.so")

RDG_OK, RDG_EINVAL, RDG_ECAPACITY, RDG_ETIMEOUT, RDG_EHIP, RDG_EUNSUPPORTED, RDG_EDATA = 0, -1, -2, -3, -4, -5, -6
RDG_F32, RDG_BF16, RDG_FP8_E4M3, RDG_FP8_E4M3_UE8M0 = 0, 1, 2, 3
RDG_CONTIGUOUS, RDG_MASKED = 0, 1
RDG_SCORE_SIGMOID, RDG_SCORE_SOFTMAX = 0, 1
RDG_ACT_NONE, RDG_ACT_RELU, RDG_ACT_SILU, RDG_ACT_GELU, RDG_ACT_GELU_TANH = 0, 1, 2, 3, 4


class RdgError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__("%s: %s (%d)" % (what, strerror(code), code))


class rdg_layout(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("n_local", ctypes.c_int32), ("block_m", ctypes.c_int32),
                ("m_max", ctypes.c_int32), ("m_cap", ctypes.c_int32), ("n_rows", ctypes.c_int32),
                ("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("masked_m", ctypes.c_void_p),
                ("pos", ctypes.c_void_p), ("row_src", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("work", ctypes.c_void_p), ("expert_load", ctypes.c_void_p)]


class rdg_kv_cache(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page_rows", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class rdg_kv_step(ctypes.Structure):
    _fields_ = [("n_req", ctypes.c_int32), ("max_blocks", ctypes.c_int32), ("page_rows", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("t_cap", ctypes.c_int32), ("seg_cap", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("seg_tok", ctypes.c_void_p),
                ("status", ctypes.c_void_p), ("work", ctypes.c_void_p)]


_NOT_BUILT = "%s is not built (run routing_dispatch_grouped_amd/_build.py or __graft_entry__.build()); there is no fallback implementation"
if not os.path.exists(LIB_PATH):
    raise ImportError(_NOT_BUILT % "librdg.so")

_lib = ctypes.CDLL(LIB_PATH)
_P, _I, _I64, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_LP = ctypes.POINTER(rdg_layout)
_CP, _SP = ctypes.POINTER(rdg_kv_cache), ctypes.POINTER(rdg_kv_step)

_SIGS = {
    "rdg_route": ([_P, _I, _I, _I, _I, _I, _F, _P, _P, _P], _I),
    "rdg_route_biased": ([_P, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P], _I),
    "rdg_eplb_place": ([_P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P], _I),
    "rdg_eplb_remap": ([_P, _P, _I, _I, _P, _P, _I, _I, _I, _I, _P, _P], _I),
    "rdg_tbo_split": ([_P, _I, _I], _I),
    "rdg_dispatch_workspace_bytes": ([_I, _I, _I], _SZ),
    "rdg_dispatch": ([_P, _P, _I, _I, _I, _P, _I, _LP, _P, _P, _P], _I),
    "rdg_dispatch_noalloc": ([_P, _P, _I, _I, _I, _P, _I, _LP, _P, _P, _P], _I),
    "rdg_layout_tables_bytes": ([_I], _SZ),
    "rdg_layout_dense": ([_I, _LP, _P], _I),
    "rdg_grouped_ffn": ([_LP, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "rdg_grouped_gate_up": ([_LP, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "rdg_grouped_down": ([_LP, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P], _I),
    "rdg_grouped_ffn_gather": ([_LP, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "rdg_grouped_gate_up_gather": ([_LP, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P], _I),
    "rdg_signal_rows": ([_LP, _I, _I, _I], _I),
    "rdg_signal_threshold": ([_I, _I], _I),
    "rdg_combine": ([_P, _I, _LP, _P, _I, _I, _I, _P, _P, _I, _P, _I, _I, _I64, _I, _P], _I),
    "rdg_combine_finish": ([_P, _I, _LP, _P, _I, _I, _I, _P, _P, _I, _P, _I, _P], _I),
    "rdg_quantize_fp8": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "rdg_quantize_fp8_ue8m0": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "rdg_fill_i32": ([_P, ctypes.c_int32, _I64, _P], _I),
    "rdg_packed_weight_bytes": ([_I, _I, _I, _I], _SZ),
    "rdg_pack_weights": ([_P, _I, _I, _I, _I, _P, _P], _I),
    "rdg_kv_step_work_bytes": ([], _SZ),
    "rdg_kv_seg_cap": ([_I, _I, _I], _I),
    "rdg_kv_plan": ([_SP, _P, _P, _P, _P, _P, _P], _I),
    "rdg_kv_trim": ([_SP, _P, _P, _P, _P, _P, _P], _I),
    "rdg_qk_norm_rope_store": ([_P, _I, _I64, _I, _I, _I, _I, _P, _P, _F, _P, _I, _I, _I, _SP, _CP, _P, _I64, _P], _I),
    "rdg_paged_attention_workspace_bytes": ([_CP, _I, _I, _I, _I, _I, _I], _SZ),
    "rdg_paged_attention": ([_P, _I, _I64, _I, _I, _SP, _CP, _I, _I, _F, _I, _I, _P, _I64, _P, _P, _SZ, _P], _I),
    "rdg_add_norm": ([_P, _I, _I64, _I, _I, _P, _P, _I, _I64, _P, _F, _P, _I64, _P, _P, _I, _P], _I),
    "rdg_linear_workspace_bytes": ([_I, _I, _I, _I], _SZ),
    "rdg_linear_workspace_bound": ([_I, _I, _I, _I], _SZ),
    "rdg_linear": ([_P, _P, _I, _I64, _I, _I, _I, _P, _P, _P, _I, _P, _I64, _P, _I, _I64, _P, _SZ, _P], _I),
    "rdg_route_topk": ([_P, _I, _I64, _I, _I, _I, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P], _I),
    "rdg_check_status": ([_P, _P, _P], _I),
    "rdg_strerror": ([_I], ctypes.c_char_p),
    "rdg_version": ([], _I),
}
for _name, (_args, _ret) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _ret


def strerror(code):
    return _lib.rdg_strerror(code).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc, what):
    if rc != RDG_OK:
        raise RdgError(rc, what)


# torch, its current-stream lookup and the part of the binding that is in C++ (it needs torch loaded; the calls that
# are marshalled here do without it), bound at the first call: the small calls of a decode step take as long on
# the host as on the GPU.
_torch = _stream_of = _device_of = _cpp = None


def _bind_torch():
    global _torch, _stream_of, _device_of
    import torch
    _stream_of, _device_of = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _torch = torch
    return torch


def _bind_cpp():
    global _cpp
    if _torch is None:
        _bind_torch()
    if not os.path.exists(os.path.join(_HERE, "_binding.so")):
        raise ImportError(_NOT_BUILT % "_binding.so")
    from . import _binding
    _cpp = _binding


def _raw_stream(stream):
    """The HIP stream as an integer (None: torch's current one)."""
    return _stream_of(_device_of()) if stream is None else stream.cuda_stream


# ------------------------------------------------------------------ layout
class Layout:
    """Device buffers of an rdg_layout, allocated with torch on ``device``."""

    def __init__(self, kind, n_local, T, K, device, block_m=128, m_max=0, m_cap=None, expert_load=None):
        import torch
        self.kind, self.n_local, self.T, self.K = kind, n_local, T, K
        n_rows = T * K
        if m_cap is None:
            m_cap = n_local * m_max if kind == RDG_MASKED else n_rows + n_local * (block_m - 1)
        i32 = dict(dtype=torch.int32, device=device)
        self.counts = torch.zeros(n_local, **i32)
        self.offsets = torch.zeros(n_local + 1, **i32)
        self.masked_m = torch.zeros(n_local, **i32)
        self.pos = torch.empty(max(n_rows, 1), **i32)
        self.row_src = torch.empty(max(m_cap, 1), **i32)
        self.status = torch.zeros(2, **i32)
        wb = rdg_dispatch_workspace_bytes(T, K, n_local)
        self.work = torch.zeros(max(wb, 256), dtype=torch.uint8, device=device)
        self.c = rdg_layout(kind, n_local, block_m, m_max, m_cap, n_rows,
                            self.counts.data_ptr(), self.offsets.data_ptr(), self.masked_m.data_ptr(),
                            self.pos.data_ptr(), self.row_src.data_ptr(), self.status.data_ptr(),
                            self.work.data_ptr(), expert_load.data_ptr() if expert_load is not None else None)
        self.expert_load = expert_load  # optional int64 [n_local] accumulated by rdg_dispatch
        self.m_cap = m_cap
        self.block_m = block_m
        self.m_max = m_max

    @property
    def ref(self):
        return ctypes.byref(self.c)


def _tensor(t, what, dtype, n):
    """The address of a tensor that the C call reads as it is: refuses another
    element type or number than the call assumes, and one that is not contiguous."""
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise RdgError(RDG_EINVAL, "%s: want a contiguous %s tensor of %d elements, got %s %s" %
                       (what, dtype, n, t.dtype, list(t.shape)))
    return t.data_ptr()


class KvCache:
    """A paged 8-bit key/value cache (rdg_kv_cache) over the caller's tensors:
    k, v [n_pages, n_kv, page_rows, head_dim] uint8, k_scale, v_scale [n_pages, n_kv] float32."""

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        if k.dim() != 4 or v.shape != k.shape:
            raise RdgError(RDG_EINVAL, "KvCache: k and v have to be [n_pages, n_kv, page_rows, head_dim]")
        n_pages, n_kv, page_rows, head_dim = k.shape
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_kv, self.page_rows, self.head_dim = n_pages, n_kv, page_rows, head_dim
        self.c = rdg_kv_cache(n_pages, page_rows, n_kv, head_dim, _tensor(k, "KvCache.k", torch.uint8, k.numel()),
                              _tensor(v, "KvCache.v", torch.uint8, k.numel()),
                              _tensor(k_scale, "KvCache.k_scale", torch.float32, n_pages * n_kv),
                              _tensor(v_scale, "KvCache.v_scale", torch.float32, n_pages * n_kv))
        self.ref = ctypes.byref(self.c)

    @classmethod
    def empty(cls, n_pages, n_kv, page_rows, head_dim, device):
        import torch
        code = dict(dtype=torch.uint8, device=device)
        scale = dict(dtype=torch.float32, device=device)
        shape = (n_pages, n_kv, page_rows, head_dim)
        return cls(torch.zeros(shape, **code), torch.zeros(shape, **code), torch.ones(shape[:2], **scale),
                   torch.ones(shape[:2], **scale))


class KvStep:
    """Device buffers of an rdg_kv_step, allocated with torch on ``device``."""

    def __init__(self, n_req, max_blocks, page_rows, n_pages, t_cap, device):
        import torch
        self.n_req, self.max_blocks, self.page_rows = n_req, max_blocks, page_rows
        self.n_pages, self.t_cap = n_pages, t_cap
        seg_cap = _lib.rdg_kv_seg_cap(t_cap, n_req, page_rows)
        _check(min(seg_cap, 0), "KvStep")
        i32 = dict(dtype=torch.int32, device=device)
        self.block_table = torch.full((n_req, max_blocks), -1, **i32)
        self.cu_q = torch.zeros(n_req + 1, **i32)
        self.kv_len = torch.zeros(n_req, **i32)
        self.slots = torch.full((t_cap,), -1, **i32)
        self.positions = torch.zeros(t_cap, **i32)
        self.seg_tok = torch.full((seg_cap,), -1, **i32)
        self.status = torch.zeros(2, **i32)
        self.work = torch.zeros(_lib.rdg_kv_step_work_bytes(), dtype=torch.uint8, device=device)
        self.c = rdg_kv_step(n_req, max_blocks, page_rows, n_pages, t_cap, seg_cap, self.block_table.data_ptr(),
                             self.cu_q.data_ptr(), self.kv_len.data_ptr(), self.slots.data_ptr(),
                             self.positions.data_ptr(), self.seg_tok.data_ptr(), self.status.data_ptr(),
                             self.work.data_ptr())
        self.ref = ctypes.byref(self.c)


# ------------------------------------------------------------------ entry points
def rdg_version():
    return _lib.rdg_version()


def rdg_dispatch_workspace_bytes(T, K, n_local):
    return int(_lib.rdg_dispatch_workspace_bytes(T, K, n_local))


def rdg_route(logits, n_group, topk_group, K, scale, topk_ids, topk_w, stream=None):
    B, N = logits.shape
    _check(_lib.rdg_route(_ptr(logits), B, N, n_group, topk_group, K, scale, _ptr(topk_ids), _ptr(topk_w),
                          _stream(stream)), "rdg_route")


def rdg_route_biased(logits, bias, n_group, topk_group, K, scale, topk_ids, topk_w, stream=None):
    B, N = logits.shape
    _check(_lib.rdg_route_biased(_ptr(logits), _ptr(bias), B, N, n_group, topk_group, K, scale, _ptr(topk_ids),
                                 _ptr(topk_w), _stream(stream)), "rdg_route_biased")


def rdg_eplb_place(load, n_groups, n_nodes, n_gpus, n_physical, r_max):
    """Host call on numpy arrays: load [n_logical] (converted to float64).
    Returns (phy2log [n_physical] int32, log2phy [n_logical, r_max] int32,
    n_replica [n_logical] int32, gpu_load [n_gpus] float64)."""
    import numpy as np
    load = np.ascontiguousarray(load, dtype=np.float64)
    n = load.shape[0]
    phy2log = np.empty(n_physical, np.int32)
    log2phy = np.empty((n, r_max), np.int32)
    n_replica = np.empty(n, np.int32)
    gpu_load = np.empty(n_gpus, np.float64)
    hp = lambda a: ctypes.c_void_p(a.ctypes.data)
    _check(_lib.rdg_eplb_place(hp(load), n, n_groups, n_nodes, n_gpus, n_physical, r_max, hp(phy2log), hp(log2phy),
                               hp(n_replica), hp(gpu_load)), "rdg_eplb_place")
    return phy2log, log2phy, n_replica, gpu_load


def rdg_tbo_split(seq_lens, decode=False):
    """Host call: seq_lens is a sequence of token counts.  Returns the number of
    sequences in the first micro-batch."""
    import numpy as np
    a = np.ascontiguousarray(seq_lens, dtype=np.int32)
    rc = _lib.rdg_tbo_split(ctypes.c_void_p(a.ctypes.data), a.shape[0], int(bool(decode)))
    if rc < 0:
        raise RdgError(rc, "rdg_tbo_split")
    return rc


def rdg_eplb_remap(ids, token_gidx, log2phy, n_replica, phys_begin, n_local, local_ids, stream=None):
    T, K = ids.shape
    n_logical, r_max = log2phy.shape
    _check(_lib.rdg_eplb_remap(_ptr(ids), _ptr(token_gidx), T, K, _ptr(log2phy), _ptr(n_replica), r_max,
                               n_logical, phys_begin, n_local, _ptr(local_ids), _stream(stream)),
           "rdg_eplb_remap")


def rdg_dispatch(x, x_scales, dtype, ids, layout, x_perm, x_perm_scales=None, stream=None):
    T, H = x.shape
    K = ids.shape[1]
    _check(_lib.rdg_dispatch(_ptr(x), _ptr(x_scales), dtype, T, H, _ptr(ids), K, layout.ref, _ptr(x_perm),
                             _ptr(x_perm_scales), _stream(stream)), "rdg_dispatch")


def rdg_layout_tables_bytes(n_local):
    return int(_lib.rdg_layout_tables_bytes(n_local))


def rdg_dispatch_noalloc(x, x_scales, dtype, ids, layout, x_perm, x_perm_scales=None, stream=None):
    """rdg_dispatch with its scratch in the library's static device array
    (layout.work then needs only rdg_layout_tables_bytes(n_local) bytes)."""
    T, H = x.shape
    K = ids.shape[1]
    _check(_lib.rdg_dispatch_noalloc(_ptr(x), _ptr(x_scales), dtype, T, H, _ptr(ids), K, layout.ref, _ptr(x_perm),
                                     _ptr(x_perm_scales), _stream(stream)), "rdg_dispatch_noalloc")


def rdg_layout_dense(T, layout, stream=None):
    _check(_lib.rdg_layout_dense(T, layout.ref, _stream(stream)), "rdg_layout_dense")


def rdg_grouped_ffn(layout, dtype, H, I, x_perm, x_perm_scales, W1, W3, W2, W1_s, W3_s, W2_s, h_ws, h_scales_ws,
                    y, signals=None, stream=None):
    _check(_lib.rdg_grouped_ffn(layout.ref, dtype, H, I, _ptr(x_perm), _ptr(x_perm_scales), _ptr(W1), _ptr(W3),
                                _ptr(W2), _ptr(W1_s), _ptr(W3_s), _ptr(W2_s), _ptr(h_ws), _ptr(h_scales_ws),
                                _ptr(y), _ptr(signals), _stream(stream)), "rdg_grouped_ffn")


def rdg_grouped_gate_up(layout, dtype, H, I, x_perm, x_perm_scales, W1, W3, W1_s, W3_s, h_ws, h_scales_ws,
                        stream=None):
    _check(_lib.rdg_grouped_gate_up(layout.ref, dtype, H, I, _ptr(x_perm), _ptr(x_perm_scales), _ptr(W1), _ptr(W3),
                                    _ptr(W1_s), _ptr(W3_s), _ptr(h_ws), _ptr(h_scales_ws), _stream(stream)),
           "rdg_grouped_gate_up")


def rdg_grouped_ffn_gather(layout, dtype, H, I, x, x_scales, K, W1, W3, W2, W1_s, W3_s, W2_s, h_ws, h_scales_ws,
                           y, signals=None, stream=None):
    _check(_lib.rdg_grouped_ffn_gather(layout.ref, dtype, H, I, _ptr(x), _ptr(x_scales), K, _ptr(W1), _ptr(W3),
                                       _ptr(W2), _ptr(W1_s), _ptr(W3_s), _ptr(W2_s), _ptr(h_ws), _ptr(h_scales_ws),
                                       _ptr(y), _ptr(signals), _stream(stream)), "rdg_grouped_ffn_gather")


def rdg_grouped_gate_up_gather(layout, dtype, H, I, x, x_scales, K, W1, W3, W1_s, W3_s, h_ws, h_scales_ws,
                               stream=None):
    _check(_lib.rdg_grouped_gate_up_gather(layout.ref, dtype, H, I, _ptr(x), _ptr(x_scales), K, _ptr(W1), _ptr(W3),
                                           _ptr(W1_s), _ptr(W3_s), _ptr(h_ws), _ptr(h_scales_ws), _stream(stream)),
           "rdg_grouped_gate_up_gather")


def rdg_grouped_down(layout, dtype, H, I, h_ws, h_scales_ws, W2, W2_s, y, signals=None, stream=None):
    _check(_lib.rdg_grouped_down(layout.ref, dtype, H, I, _ptr(h_ws), _ptr(h_scales_ws), _ptr(W2), _ptr(W2_s),
                                 _ptr(y), _ptr(signals), _stream(stream)), "rdg_grouped_down")


def rdg_signal_rows(layout, dtype, H, I):
    r = _lib.rdg_signal_rows(layout.ref, dtype, H, I)
    _check(min(r, 0), "rdg_signal_rows")
    return r


def rdg_signal_threshold(H, dtype):
    r = _lib.rdg_signal_threshold(H, dtype)
    _check(min(r, 0), "rdg_signal_threshold")
    return r


def rdg_combine(y, y_dtype, layout, topk_w, T, K, H, shared_out, out, out_dtype, signals=None, signal_rows=0,
                threshold=0, timeout_us=0, max_blocks=0, stream=None):
    _check(_lib.rdg_combine(_ptr(y), y_dtype, layout.ref, _ptr(topk_w), T, K, H, _ptr(shared_out), _ptr(out),
                            out_dtype, _ptr(signals), signal_rows, threshold, timeout_us, max_blocks,
                            _stream(stream)), "rdg_combine")


def rdg_combine_finish(y, y_dtype, layout, topk_w, T, K, H, shared_out, out, out_dtype, signals, signal_rows,
                       stream=None):
    _check(_lib.rdg_combine_finish(_ptr(y), y_dtype, layout.ref, _ptr(topk_w), T, K, H, _ptr(shared_out),
                                   _ptr(out), out_dtype, _ptr(signals), signal_rows, _stream(stream)),
           "rdg_combine_finish")


def rdg_quantize_fp8(src, src_dtype, block_rows, q, scales, stream=None):
    rows, cols = src.shape
    _check(_lib.rdg_quantize_fp8(_ptr(src), src_dtype, rows, cols, block_rows, _ptr(q), _ptr(scales),
                                 _stream(stream)), "rdg_quantize_fp8")


def rdg_quantize_fp8_ue8m0(src, src_dtype, block_rows, q, scales, stream=None):
    rows, cols = src.shape
    _check(_lib.rdg_quantize_fp8_ue8m0(_ptr(src), src_dtype, rows, cols, block_rows, _ptr(q), _ptr(scales),
                                       _stream(stream)), "rdg_quantize_fp8_ue8m0")


def rdg_pack_weights(W, dtype, W_packed, stream=None):
    """W: [n_mat, rows, cols] (or [rows, cols]) device tensor; W_packed: same byte size."""
    shape = tuple(W.shape)
    n_mat, rows, cols = (1,) + shape if len(shape) == 2 else shape
    _check(_lib.rdg_pack_weights(_ptr(W), dtype, n_mat, rows, cols, _ptr(W_packed), _stream(stream)),
           "rdg_pack_weights")


def rdg_fill_i32(p, value, stream=None):
    _check(_lib.rdg_fill_i32(_ptr(p), value, p.numel(), _stream(stream)), "rdg_fill_i32")


def rdg_kv_plan(step, kv_len, q_len, free_list, n_free, n_free_out, stream=None):
    """kv_len, q_len [n_req], free_list [>= n_free], n_free, n_free_out [1]: int32 device tensors."""
    i32, R = (_torch or _bind_torch()).int32, step.n_req
    _check(_lib.rdg_kv_plan(step.ref, _tensor(kv_len, "rdg_kv_plan: kv_len", i32, R),
                            _tensor(q_len, "rdg_kv_plan: q_len", i32, R),
                            _tensor(free_list, "rdg_kv_plan: free_list", i32, free_list.numel()),
                            _tensor(n_free, "rdg_kv_plan: n_free", i32, 1),
                            _tensor(n_free_out, "rdg_kv_plan: n_free_out", i32, 1), _raw_stream(stream)),
           "rdg_kv_plan")


def rdg_kv_trim(step, kv_len, new_len, free_list, n_free, n_free_out, stream=None):
    """kv_len, new_len [n_req], free_list [n_pages], n_free, n_free_out [1]: int32 device tensors."""
    i32, R = (_torch or _bind_torch()).int32, step.n_req
    _check(_lib.rdg_kv_trim(step.ref, _tensor(kv_len, "rdg_kv_trim: kv_len", i32, R),
                            _tensor(new_len, "rdg_kv_trim: new_len", i32, R),
                            _tensor(free_list, "rdg_kv_trim: free_list", i32, step.n_pages),
                            _tensor(n_free, "rdg_kv_trim: n_free", i32, 1),
                            _tensor(n_free_out, "rdg_kv_trim: n_free_out", i32, 1), _raw_stream(stream)),
           "rdg_kv_trim")


def _rows(t, what, heads, head_dim):
    """(dtype code, tokens, token stride) of [T, heads * head_dim] or [T, heads, head_dim] rows; tokens may be apart."""
    torch = _torch or _bind_torch()
    dt, shape, stride = t.dtype, t.shape, t.stride()
    code = RDG_BF16 if dt is torch.bfloat16 else RDG_F32 if dt is torch.float32 else None
    if len(shape) == 3:
        fits = shape[1] == heads and shape[2] == head_dim and stride[2] == 1 and (stride[1] == head_dim or heads == 1)
    else:
        fits = len(shape) == 2 and shape[1] == heads * head_dim and stride[1] == 1
    if code is None or not fits:
        raise RdgError(RDG_EINVAL, "%s: want bfloat16 or float32 rows of %d heads of %d, got %s %s with strides %s" %
                       (what, heads, head_dim, dt, list(shape), list(stride)))
    T = shape[0]
    return code, T, stride[0] if T > 1 else heads * head_dim


def rdg_qk_norm_rope_store(qkv, n_q, n_kv, head_dim, q_weight, k_weight, eps, cos_sin, rot_dim, neighbours, step, cache,
                           q_out, stream=None):
    """qkv [T, (n_q + 2 n_kv) * head_dim] (token stride free), q_out [T, n_q, head_dim], weights [head_dim] float32
    or None, cos_sin [n_pos, rot_dim] float32 or None; cache None with n_kv = 0."""
    f32 = (_torch or _bind_torch()).float32
    dt, T, stride = _rows(qkv, "rdg_qk_norm_rope_store: qkv", n_q + 2 * n_kv, head_dim)
    q_stride, q_ptr, n_pos, cs_ptr = 0, None, 0, None
    if n_q > 0:
        q_dt, q_T, q_stride = _rows(q_out, "rdg_qk_norm_rope_store: q_out", n_q, head_dim)
        if q_dt != dt or q_T != T:
            raise RdgError(RDG_EINVAL, "rdg_qk_norm_rope_store: q_out differs from qkv in type or tokens")
        q_ptr = q_out.data_ptr()
    wq = None if q_weight is None else _tensor(q_weight, "rdg_qk_norm_rope_store: q_weight", f32, head_dim)
    wk = None if k_weight is None else _tensor(k_weight, "rdg_qk_norm_rope_store: k_weight", f32, head_dim)
    if rot_dim:
        n_pos = cos_sin.shape[0]
        cs_ptr = _tensor(cos_sin, "rdg_qk_norm_rope_store: cos_sin", f32, n_pos * rot_dim)
    _check(_lib.rdg_qk_norm_rope_store(qkv.data_ptr(), dt, stride, T, n_q, n_kv, head_dim, wq, wk, eps, cs_ptr, n_pos,
                                       rot_dim, 1 if neighbours else 0, step.ref, None if cache is None else cache.ref,
                                       q_ptr, q_stride, _raw_stream(stream)), "rdg_qk_norm_rope_store")


def rdg_paged_attention_workspace_bytes(cache, T, n_req, n_q, max_q, max_kv, dtype):
    return int(_lib.rdg_paged_attention_workspace_bytes(cache.ref, T, n_req, n_q, max_q, max_kv, dtype))


def rdg_paged_attention(q, step, cache, max_q, max_kv, scale, out, lse=None, work=None, causal=True, window=0,
                        stream=None):
    """q, out [T, n_q, head_dim] (token strides free), lse [T, n_q] float32 or None; work: a uint8 tensor of
    rdg_paged_attention_workspace_bytes."""
    n_q = q.shape[1]
    dt, T, q_stride = _rows(q, "rdg_paged_attention: q", n_q, cache.head_dim)
    out_dt, out_T, out_stride = _rows(out, "rdg_paged_attention: out", n_q, cache.head_dim)
    if out_dt != dt or out_T != T:
        raise RdgError(RDG_EINVAL, "rdg_paged_attention: out differs from q in type or tokens")
    lse_ptr = None if lse is None else _tensor(lse, "rdg_paged_attention: lse", (_torch or _bind_torch()).float32, T * n_q)
    work_ptr, work_bytes = (None, 0) if work is None else (work.data_ptr(), work.nbytes)
    _check(_lib.rdg_paged_attention(q.data_ptr(), dt, q_stride, T, n_q, step.ref, cache.ref, max_q, max_kv, scale,
                                    1 if causal else 0, window, out.data_ptr(), out_stride, lse_ptr, work_ptr, work_bytes,
                                    _raw_stream(stream)), "rdg_paged_attention")


def _answer(call, r):
    """Raises what a function of _binding answered: the C call's error code, or the text of a refusal."""
    if isinstance(r, str):
        raise RdgError(RDG_EINVAL, "%s: %s" % (call, r))
    raise RdgError(r, call)


def rdg_add_norm(x, weight, eps, out=None, residual=None, residual_out=None, q=None, q_scales=None,
                 q_dtype=RDG_FP8_E4M3, stream=None):
    """x, out [T, H], residual, residual_out [T, H] of one type (row strides free), weight [H] float32 or None,
    q [T, H] uint8 and q_scales [T, H/128] float32."""
    if _cpp is None:
        _bind_cpp()
    r = _cpp.add_norm(x, weight, eps, out, residual, residual_out, q, q_scales, q_dtype, _device_of(),
                      _stream_of if stream is None else stream.cuda_stream)
    if r is not None:
        _answer("rdg_add_norm", r)


def rdg_linear_workspace_bytes(T, N, K, dtype):
    return int(_lib.rdg_linear_workspace_bytes(T, N, K, dtype))


def rdg_linear_workspace_bound(T, N, K, dtype):
    """Bytes that do for every call of up to T tokens."""
    return int(_lib.rdg_linear_workspace_bound(T, N, K, dtype))


def rdg_linear(x, x_scales, dtype, W, W_scales, out, bias=None, act=RDG_ACT_NONE, residual=None, work=None, stream=None):
    """x [T, K] (row stride free; fp8 codes as uint8 or float8_e4m3fn) with x_scales [T, K/128] float32, W [N, K] packed
    with W_scales [ceil(N/128), K/128], out, residual [T, N] bfloat16 or float32 (row strides free), bias [N] float32;
    work: a uint8 tensor of rdg_linear_workspace_bytes, or rdg_linear_workspace_bound of the most tokens."""
    if _cpp is None:
        _bind_cpp()
    r = _cpp.linear(x, x_scales, dtype, W, W_scales, out, bias, act, residual, work, _device_of(),
                    _stream_of if stream is None else stream.cuda_stream)
    if r is not None:
        _answer("rdg_linear", r)


def rdg_route_topk(logits, score, n_group, topk_group, group_best, K, renorm, scale, topk_ids, topk_w, bias=None,
                   stream=None):
    """logits [B, N] bfloat16 or float32 (row stride free), topk_ids [B, K] int32, topk_w [B, K] float32, bias [N] float32
    or None."""
    if _cpp is None:
        _bind_cpp()
    r = _cpp.route_topk(logits, score, n_group, topk_group, group_best, K, 1 if renorm else 0, scale, topk_ids, topk_w,
                        bias, _device_of(), _stream_of if stream is None else stream.cuda_stream)
    if r is not None:
        _answer("rdg_route_topk", r)


def rdg_check_status(layout_or_status, stream=None):
    """Waits for the stream; returns (code, detail)."""
    st = layout_or_status.status if isinstance(layout_or_status, (Layout, KvStep)) else layout_or_status
    host = (ctypes.c_int32 * 2)()
    rc = _lib.rdg_check_status(_ptr(st), host, _stream(stream))
    if rc in (RDG_EINVAL, RDG_EHIP):  # the query itself failed (device codes are -2, -3 and -6)
        raise RdgError(rc, "rdg_check_status")
    return int(host[0]), int(host[1])
