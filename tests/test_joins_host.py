"""Host-side checks of the joins of a decoder layer: size queries and every
refusal, which comes before anything is enqueued."""
import pytest

A = 0x100000  # stand-in device address: 16-byte aligned, never dereferenced (each call fails its checks first)


def _rdg():
    import routing_dispatch_grouped_amd as rdg
    return rdg


def _norm(**change):
    rdg = _rdg()
    a = dict(x=A, x_dtype=rdg.RDG_BF16, x_stride=256, T=4, H=256, residual=A, residual_out=A, res_dtype=rdg.RDG_BF16,
             res_stride=256, weight=A, eps=1e-6, out=2 * A, out_stride=256, q=3 * A, q_scales=A, q_dtype=rdg.RDG_FP8_E4M3)
    a.update(change)
    return rdg._lib.rdg_add_norm(*a.values(), None)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(H=0), dict(H=252), dict(H=136), dict(x_dtype=2), dict(x=None), dict(x=A + 8), dict(x_stride=255),
    dict(x_stride=260), dict(x_stride=-256), dict(res_dtype=3), dict(res_dtype=-1), dict(residual=A + 4), dict(res_stride=248),
    dict(residual=None), dict(residual_out=A + 2), dict(weight=A + 4), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(out=None, q=None), dict(out=A), dict(out=2 * A + 8), dict(out_stride=128), dict(q=A + 8),
    dict(q_scales=None), dict(q_scales=A + 4), dict(q_dtype=0), dict(q_dtype=1),
    # an output over an input's other rows, or over another output
    dict(res_dtype=0), dict(res_stride=264), dict(residual_out=5 * A, out=A, out_stride=264), dict(out=A, residual_out=A), dict(q=A),
    dict(q=2 * A), dict(x=4 * A, residual_out=5 * A, out=A, res_stride=512)])
def test_norm_refusals(change):
    assert _norm(**change) == _rdg().RDG_EINVAL


def test_norm_sizes():
    rdg = _rdg()
    assert _norm(T=0) == rdg.RDG_OK
    assert _norm(T=0, x=None, q_scales=None) == rdg.RDG_OK
    big = dict(H=32896, x_stride=32896, res_stride=32896, out_stride=32896)
    assert _norm(**big) == rdg.RDG_EUNSUPPORTED


def _linear(**change):
    rdg = _rdg()
    a = dict(x=A, x_scales=A, dtype=rdg.RDG_FP8_E4M3, x_stride=256, T=4, N=48, K=256, W=A, W_scales=A, bias=A, act=1,
             residual=A, res_stride=48, out=2 * A, out_dtype=rdg.RDG_BF16, out_stride=48, work=A, work_bytes=1 << 40)
    a.update(change)
    return rdg._lib.rdg_linear(*a.values(), None)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(N=0), dict(N=24), dict(K=0), dict(K=192), dict(dtype=4), dict(dtype=-1), dict(x=None), dict(x=A + 8),
    dict(x_stride=128), dict(x_stride=264), dict(x_scales=None), dict(x_scales=A + 4), dict(W=None), dict(W=A + 8), dict(W_scales=None),
    dict(W_scales=A + 4), dict(bias=A + 4), dict(act=-1), dict(act=5), dict(residual=A + 8), dict(res_stride=40), dict(res_stride=52),
    dict(out=None), dict(out=A + 4), dict(out_stride=32), dict(out_dtype=2), dict(out=A), dict(x=4 * A, out=A, residual=None),
    dict(residual=2 * A, res_stride=64)])
def test_linear_refusals(change):
    assert _linear(**change) == _rdg().RDG_EINVAL


def test_linear_sizes():
    rdg = _rdg()
    assert _linear(T=0) == rdg.RDG_OK
    assert _linear(dtype=rdg.RDG_F32) == rdg.RDG_EUNSUPPORTED       # fp32 operands, bf16 out
    size = rdg.rdg_linear_workspace_bytes
    assert size(0, 256, 256, rdg.RDG_BF16) == 0
    assert size(8, 250, 256, rdg.RDG_BF16) == 0 and size(8, 256, 100, rdg.RDG_BF16) == 0


def test_linear_checks_its_workspace():
    rdg = _rdg()
    # a small product over a long reduction, where the work is shared along it
    for T, N, K in ((1, 16, 7168), (64, 256, 7168), (128, 256, 16384), (300, 512, 16384), (1000, 1024, 8192)):
        for dtype in (rdg.RDG_BF16, rdg.RDG_FP8_E4M3, rdg.RDG_FP8_E4M3_UE8M0):
            need = rdg.rdg_linear_workspace_bytes(T, N, K, dtype)
            a = dict(T=T, N=N, K=K, dtype=dtype, x_stride=K, res_stride=N, out_stride=N)
            if need:
                assert _linear(work_bytes=need - 1, **a) == rdg.RDG_EINVAL
                assert _linear(work=None, work_bytes=need, **a) == rdg.RDG_EINVAL
                assert _linear(work=A + 8, work_bytes=need, **a) == rdg.RDG_EINVAL


def _route(**change):
    rdg = _rdg()
    a = dict(logits=A, dtype=rdg.RDG_F32, stride=64, B=4, N=64, score=rdg.RDG_SCORE_SOFTMAX, bias=None, n_group=8,
             topk_group=2, group_best=1, K=8, renorm=1, scale=1.0, ids=A, w=A)
    a.update(change)
    return rdg._lib.rdg_route_topk(*a.values(), None)


@pytest.mark.parametrize("change", [
    dict(B=-1), dict(N=0), dict(N=1032, stride=1032), dict(n_group=0), dict(n_group=6), dict(dtype=2), dict(score=2), dict(score=-1),
    dict(topk_group=0), dict(topk_group=9), dict(group_best=0), dict(group_best=3), dict(K=0), dict(K=17), dict(K=33, topk_group=8),
    dict(logits=None), dict(ids=None), dict(w=None), dict(stride=63)])
def test_route_refusals(change):
    assert _route(**change) == _rdg().RDG_EINVAL


def test_route_of_no_tokens():
    assert _route(B=0, logits=None) == _rdg().RDG_OK


def test_binding_refusals(monkeypatch):
    """Types, shapes and strides that the C call cannot see."""
    import torch
    rdg = _rdg()
    rdg._bind_torch()
    monkeypatch.setattr(rdg, "_device_of", lambda: -1)   # where the tensors here are
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt)  # noqa: E731
    x = e(4, 256)
    f32 = torch.float32

    def refused(call):
        with pytest.raises(rdg.RdgError) as err:
            call()
        assert err.value.code == rdg.RDG_EINVAL and "device" not in str(err.value)

    refused(lambda: rdg.rdg_add_norm(x.half(), None, 1e-6, out=x))
    refused(lambda: rdg.rdg_add_norm(e(4, 2, 128), None, 1e-6, out=x))
    refused(lambda: rdg.rdg_add_norm(x, e(256), 1e-6, out=x))                       # a gain in bf16
    refused(lambda: rdg.rdg_add_norm(x, None, 1e-6, out=e(4, 128)))
    refused(lambda: rdg.rdg_add_norm(x, None, 1e-6, out=e(4, 256, dt=f32)))
    refused(lambda: rdg.rdg_add_norm(x, None, 1e-6, out=x, residual=x, residual_out=e(4, 256, dt=f32)))
    refused(lambda: rdg.rdg_add_norm(x, None, 1e-6, out=x, residual=x, residual_out=e(4, 512)[:, :256]))
    refused(lambda: rdg.rdg_add_norm(x, None, 1e-6, out=x, residual_out=x))
    refused(lambda: rdg.rdg_add_norm(e(256, 4).T, None, 1e-6, out=x))
    refused(lambda: rdg.rdg_add_norm(x, None, 1e-6, q=e(4, 256, dt=torch.uint8), q_scales=e(4, 1, dt=f32)))
    w, out = e(48, 256), e(4, 48)
    refused(lambda: rdg.rdg_linear(x, None, rdg.RDG_F32, w, None, out))
    refused(lambda: rdg.rdg_linear(x, None, rdg.RDG_BF16, e(48, 128), None, out))
    refused(lambda: rdg.rdg_linear(x, None, rdg.RDG_BF16, w, None, e(5, 48)))
    refused(lambda: rdg.rdg_linear(x, None, rdg.RDG_BF16, w, None, out, bias=e(48)))
    refused(lambda: rdg.rdg_linear(x, None, rdg.RDG_BF16, w, None, out, residual=e(4, 48, dt=f32)))
    u8 = torch.uint8
    refused(lambda: rdg.rdg_linear(e(4, 256, dt=u8), e(4, 1, dt=f32), rdg.RDG_FP8_E4M3, e(48, 256, dt=u8), e(1, 2, dt=f32), out))
    refused(lambda: rdg.rdg_linear(e(4, 256, dt=u8), e(4, 2, dt=f32), rdg.RDG_FP8_E4M3, e(48, 256, dt=u8), e(2, 2, dt=f32), out))
    ids, tw = e(4, 2, dt=torch.int32), e(4, 2, dt=f32)
    refused(lambda: rdg.rdg_route_topk(e(4, 16).half(), 0, 1, 1, 1, 2, 1, 1.0, ids, tw))
    refused(lambda: rdg.rdg_route_topk(e(4, 16), 0, 1, 1, 1, 2, 1, 1.0, ids.long(), tw))
    refused(lambda: rdg.rdg_route_topk(e(4, 16), 0, 1, 1, 1, 4, 1, 1.0, ids, tw))
    refused(lambda: rdg.rdg_route_topk(e(4, 16), 0, 1, 1, 1, 2, 1, 1.0, ids, tw, bias=e(16)))


def test_tensors_of_another_device_are_refused(monkeypatch):
    import torch
    rdg = _rdg()
    rdg._bind_torch()
    monkeypatch.setattr(rdg, "_device_of", lambda: 0)
    x = torch.empty(4, 256, dtype=torch.bfloat16)
    with pytest.raises(rdg.RdgError, match="device"):
        rdg.rdg_add_norm(x, None, 1e-6, out=x)
    with pytest.raises(rdg.RdgError, match="device"):
        rdg.rdg_linear(x, None, rdg.RDG_BF16, torch.empty(16, 256, dtype=torch.bfloat16), None, torch.empty(4, 16))
    with pytest.raises(rdg.RdgError, match="device"):
        rdg.rdg_route_topk(x, 0, 1, 1, 1, 2, 1, 1.0, torch.empty(4, 2, dtype=torch.int32), torch.empty(4, 2))


def test_what_is_no_tensor_is_refused(monkeypatch):
    import torch
    rdg = _rdg()
    rdg._bind_torch()
    monkeypatch.setattr(rdg, "_device_of", lambda: -1)
    x, f32 = torch.empty(4, 256), torch.float32
    many = torch.empty(1, 256).expand(1 << 31, 256)   # one row more than 32 bits count
    for call in (lambda: rdg.rdg_add_norm(None, None, 1e-6, out=x),
                 lambda: rdg.rdg_add_norm(x, None, 1e-6, out=x.numpy()),
                 lambda: rdg.rdg_add_norm(x, None, "eps", out=x),
                 lambda: rdg.rdg_add_norm(x, None, 1e-6, q=torch.empty(4, 256, dtype=torch.uint8)),
                 lambda: rdg.rdg_add_norm(many, None, 1e-6, out=many),
                 lambda: rdg.rdg_linear(x, None, 9, x, None, x),
                 lambda: rdg.rdg_linear(x, None, rdg.RDG_F32, x.to_sparse(), None, torch.empty(4, 4)),
                 lambda: rdg.rdg_linear(x, None, rdg.RDG_F32, x, None, torch.empty(4, 4), act=None),
                 lambda: rdg.rdg_linear(x, None, rdg.RDG_F32, x, None, torch.empty(4, 4), act=1 << 40),
                 lambda: rdg.rdg_route_topk(many, 0, 1, 1, 1, 2, 1, 1.0, x.int(), x),
                 lambda: rdg.rdg_route_topk(x, 0, 1, 1, 1, -1, 1, 1.0, torch.empty(4, 2, dtype=torch.int32),
                                            torch.empty(4, 2, dtype=f32))):
        with pytest.raises(rdg.RdgError) as err:
            call()
        assert err.value.code == rdg.RDG_EINVAL
