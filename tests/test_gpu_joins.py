"""The joins of a decoder layer on the GPU against the oracle: the residual's
addition with the norm and its 8-bit output, the matrix product with its epilogue,
and routing by scores; then a run of them together.

Tolerances, all derived (u = 2^-24, half an fp32 step):
  * sum x + r: one rounding, u of it; half a step of its type more where it is stored.
  * y: at most H/8 + 32 fp32 roundings in a sum of squares of one sign (a thread's chain of at most 32, then a tree
    and a chain over the waves: 64 covers them), halved by the root, and under 8 more: 64 u of |y|;
    half a step of its type where it is stored.
  * block scales: the same share of amax / 448 and one division: 66 u; a power of two is the oracle's
    for some amax within 64 u of the oracle's.
  * codes: half an e4m3 step, 2^-4 of the value and 2^-10 of the scale below the normal range, 132 u besides.
  * products: K exact products (bf16, fp8; one rounding each for fp32) summed in fp32 in any order: (K + 8) u of
    the sum of magnitudes d, twice for fp8 whose partial sums are scaled; activations have slopes under 1.2 and
    values off by at most 512 u (an exponential's argument of at most 128 rounded four times); half a step of out's type.
  * operands of small whole numbers and scales of powers of two: every sum is exact, so equal.
  * routing: ids equal; weights K + 4 roundings.
"""
import numpy as np
import pytest
import torch

from harness import DEV, rdg
from oracle import joins

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF, "f32": F32}
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def f64(t):
    return t.detach().cpu().double().numpy()


def spaced(rows, cols, dtype, gap):
    """[rows, cols] uninitialised, gap elements between rows."""
    return torch.full((rows, cols + gap), 7.0, dtype=dtype, device=DEV)[:, :cols]


# ---------------------------------------------------------------- norm
def norm_case(T, H, dtype, res, seed=0, gap=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 131 * T + H)
    n = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    x = spaced(T, H, TYPES[dtype], gap)
    x.copy_(n(T, H) * torch.exp(n(1, H)))
    r = None
    if res:
        r = spaced(T, H, TYPES[res], gap)
        r.copy_(3 * n(T, H))
    return x, r, 1 + 0.2 * n(H)


def check_codes(q, qs, y, pow2):
    T, H = y.shape
    q, qs = q.view(torch.float8_e4m3fn).double().cpu().numpy().reshape(T, -1, 128), f64(qs)
    y = y.reshape(T, -1, 128)
    amax = np.abs(y).max(2)
    if pow2:
        lo, hi = (joins.block_scale(amax * (1 + s * 64 * U), True) for s in (-1, 1))
        assert ((qs == lo) | (qs == hi)).all()
    else:
        want = joins.block_scale(amax, False)
        assert (np.abs(qs - want) <= 66 * U * want).all()
    err = np.abs(q * qs[..., None] - y)
    assert (err <= (2.0 ** -4 + 132 * U) * np.abs(y) + 2.0 ** -10 * qs[..., None] * (1 + 132 * U)).all()


SIZES = [(1, 8), (1, 128), (3, 512), (5, 520), (4, 640), (2, 1024), (7, 1032), (3, 2048), (2, 2056), (33, 4096), (2, 4104),
         (1, 7168), (70, 7168), (5, 8192), (3, 8200), (2, 16384), (2, 16392), (3, 32768), (9000, 128), (2500, 1280)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("f32", ""), ("bf16", "f32"), ("f32", "bf16"), ("bf16", ""), ("f32", "f32")])
def test_norm(T, H, dtype, res):
    m = rdg()
    gap = 8 if T % 2 else 0
    x, r, w = norm_case(T, H, dtype, res, gap=gap)
    w = None if T == 5 else w
    out = spaced(T, H, x.dtype, 2 * gap)
    r_out = None if r is None else spaced(T, H, r.dtype, gap)
    coded = H % 128 == 0
    s, y = joins.add_norm(f64(x), None if r is None else f64(r), None if w is None else f64(w), 1e-6)
    for pow2 in (False, True) if coded else (False,):
        q = torch.empty(T, H, dtype=torch.uint8, device=DEV) if coded else None
        qs = torch.empty(T, H // 128, device=DEV) if coded else None
        m.rdg_add_norm(x, w, 1e-6, out=out, residual=r, residual_out=r_out, q=q, q_scales=qs,
                       q_dtype=m.RDG_FP8_E4M3_UE8M0 if pow2 else m.RDG_FP8_E4M3)
        assert (np.abs(f64(out) - y) <= (64 * U + HALF[x.dtype]) * np.abs(y)).all()
        if r is not None:
            assert (np.abs(f64(r_out) - s) <= (U + HALF[r.dtype]) * np.abs(s)).all()
        if coded:
            check_codes(q, qs, y, pow2)
    for t in (x, r, out, r_out):
        if gap and t is not None:
            rest = t.as_strided((T, t.stride(0) - H), (t.stride(0), 1), t.storage_offset() + H)
            assert (rest == 7).all()


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("H", [128, 896, 7168])
def test_norm_codes_are_the_quantisers(H, pow2):
    m = rdg()
    x, r, w = norm_case(37, H, "f32", "bf16", seed=3)
    x[5] = 0
    r[5] = 0
    out, q, qs = torch.empty_like(x), torch.empty(37, H, dtype=torch.uint8, device=DEV), torch.empty(37, H // 128, device=DEV)
    m.rdg_add_norm(x, w, 1e-6, out=out, residual=r, q=q, q_scales=qs, q_dtype=m.RDG_FP8_E4M3_UE8M0 if pow2 else m.RDG_FP8_E4M3)
    q2, qs2 = torch.empty_like(q), torch.empty_like(qs)
    (m.rdg_quantize_fp8_ue8m0 if pow2 else m.rdg_quantize_fp8)(out, m.RDG_F32, 1, q2, qs2)
    assert torch.equal(q, q2) and torch.equal(qs, qs2)
    assert (q[5] == 0).all() and (qs[5] == 1).all()


def test_norm_in_place():
    m = rdg()
    for dtype, res in (("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")):
        x, r, w = norm_case(19, 2304, dtype, res)
        out, r_out = torch.empty_like(x), torch.empty_like(r)
        m.rdg_add_norm(x, w, 1e-6, out=out, residual=r, residual_out=r_out)
        x2, r2 = x.clone(), r.clone()
        m.rdg_add_norm(x2, w, 1e-6, out=x2, residual=r2, residual_out=r2)
        assert torch.equal(x2, out) and torch.equal(r2, r_out)
        if dtype == res:  # the sum in x's place
            x3 = x.clone()
            m.rdg_add_norm(x3, w, 1e-6, out=out, residual=r, residual_out=x3)
            assert torch.equal(x3, r_out)


def test_norm_rows_that_are_not_finite():
    """Each such row by itself: its neighbours, also in the same workgroup, keep their results."""
    m = rdg()
    for H in (256, 1024, 7168):
        x, _, w = norm_case(9, H, "f32", "")
        want, q0, qs0 = torch.empty_like(x), torch.empty(9, H, dtype=torch.uint8, device=DEV), torch.empty(9, H // 128, device=DEV)
        m.rdg_add_norm(x, w, 1e-6, out=want, q=q0, q_scales=qs0)
        y = x.clone()
        y[1, 3], y[4, 130], y[6] = float("nan"), float("inf"), 1e30
        out, q, qs = torch.empty_like(x), torch.empty_like(q0), torch.empty_like(qs0)
        m.rdg_add_norm(y, w, 1e-6, out=out, q=q, q_scales=qs)
        assert out[1].isnan().all() and (q[1] == 0x7f).all() and (qs[1] == 1).all()
        assert out[4, 130].isnan() and (out[4].nan_to_num(0) == 0).all() and q[4, 130] == 0x7f
        assert (out[6] == 0).all() and (qs[6] == 1).all()
        for i in (0, 2, 3, 5, 7, 8):
            assert torch.equal(out[i], want[i]) and torch.equal(q[i], q0[i]) and torch.equal(qs[i], qs0[i])
    # an infinity that the gain makes: the largest code of its block's scale
    x, w = torch.ones(1, 256, device=DEV), torch.ones(256, device=DEV)
    w[7], w[200] = float("inf"), -float("inf")
    out, q, qs = torch.empty_like(x), torch.empty(1, 256, dtype=torch.uint8, device=DEV), torch.empty(1, 2, device=DEV)
    m.rdg_add_norm(x, w, 0.0, out=out, q=q, q_scales=qs)
    v = q.view(torch.float8_e4m3fn).float()
    assert v[0, 7] == 448 and v[0, 200] == -448 and torch.isfinite(qs).all()


def test_norm_of_no_rows():
    m = rdg()
    x = torch.empty(0, 256, dtype=BF, device=DEV)
    m.rdg_add_norm(x, None, 1e-6, out=torch.empty_like(x))
    torch.cuda.synchronize()


# ---------------------------------------------------------------- linear
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def act_code(act):
    m = rdg()
    return [m.RDG_ACT_NONE, m.RDG_ACT_RELU, m.RDG_ACT_SILU, m.RDG_ACT_GELU, m.RDG_ACT_GELU_TANH][ACTS.index(act)]


def linear_case(T, N, K, kind, whole, seed=0, gap=0):
    """dict of device operands and their float64 values.  whole: small whole numbers, scales of powers of two."""
    m = rdg()
    g = torch.Generator(device=DEV).manual_seed(seed + T + 7 * N + 13 * K)
    dt = dict(bf16=m.RDG_BF16, f32=m.RDG_F32, fp8=m.RDG_FP8_E4M3, e8m0=m.RDG_FP8_E4M3_UE8M0)[kind]
    if whole:
        draw = lambda *s: torch.randint(-3, 4, s, device=DEV, generator=g).float()  # noqa: E731
    else:
        draw = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    x, w = draw(T, K), draw(N, K)
    c = dict(kind=dt, xs=None, ws=None)
    nat = {"bf16": BF, "f32": F32}.get(kind, torch.float8_e4m3fn)
    xq = torch.empty(T, K + gap, dtype=nat, device=DEV)[:, :K]
    xq.copy_(x)
    wq = w.to(nat)
    xv, wv = f64(xq.float()), f64(wq.float())
    if nat is torch.float8_e4m3fn:
        e = lambda *s: torch.exp2(torch.randint(-2, 3, s, device=DEV, generator=g).float())  # noqa: E731
        r = lambda *s: e(*s) if whole or kind == "e8m0" else 0.25 + torch.rand(*s, device=DEV, generator=g)  # noqa: E731
        c["xs"], c["ws"] = r(T, K // 128), r(-(-N // 128), K // 128)
        xv = xv * f64(c["xs"]).repeat(128, 1)
        wv = wv * f64(c["ws"]).repeat(128, 1).repeat(128, 0)[:N]
    packed = torch.empty_like(wq)
    m.rdg_pack_weights(wq, dt, packed)
    c.update(x=xq, w=packed, xv=xv, wv=wv, g=g)
    return c


def work_for(T, N, K, dt):
    m = rdg()
    n = m.rdg_linear_workspace_bytes(T, N, K, dt)
    return torch.full((n,), 0xff, dtype=torch.uint8, device=DEV) if n else None  # NaN wherever a part is not written


def run_linear(c, out_dtype, act="none", bias=None, residual=None, gap=0):
    m = rdg()
    T, K = c["x"].shape
    N = c["w"].shape[0]
    out = spaced(T, N, out_dtype, gap)
    m.rdg_linear(c["x"], c["xs"], c["kind"], c["w"], c["ws"], out, bias=bias, act=act_code(act), residual=residual,
                 work=work_for(T, N, K, c["kind"]))
    if gap:
        assert (out.as_strided((T, gap), (N + gap, 1), out.storage_offset() + N) == 7).all()
    return out


SHAPES = [(1, 16, 128), (1, 64, 7168), (3, 48, 256), (16, 128, 384), (17, 80, 512), (32, 256, 2048), (33, 144, 128), (61, 272, 640),
          (64, 512, 1024), (65, 16, 1024), (100, 2112, 256), (128, 256, 4096), (129, 528, 128), (200, 1040, 896), (255, 256, 7168),
          (257, 272, 256), (300, 4096, 384), (513, 784, 1152), (1000, 160, 2304), (2049, 2064, 128)]


@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8", "e8m0"])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_linear_of_whole_numbers_is_exact(T, N, K, kind):
    gap = 16 if T % 2 else 0
    c = linear_case(T, N, K, kind, True, gap=gap)
    out = run_linear(c, F32, gap=gap // 4)
    assert np.array_equal(f64(out), c["xv"] @ c["wv"].T)


# larger tiles, splits, whole rounds of 256 x 256 tiles with others behind them, an odd number of stages (every plan: test_gpu_joins_edges)
LARGE = [(2300, 9232, 640), (4000, 5136, 256), (2048, 9216, 384), (700, 4112, 2048), (1100, 2064, 4096), (129, 7184, 3968),
         (64, 7184, 7168), (1000, 272, 16384), (300, 4112, 512), (500, 12304, 1152), (4097, 4112, 128), (100, 18432, 2048),
         (260, 784, 7168), (900, 1040, 14336)]
# tiles of 64, 80 and 96 features, whose waves load unlike numbers of pieces: cut tiles, splits, tiles across two scale blocks
LARGE += [(33, 24560, 640), (40, 24560, 1152), (49, 18416, 896), (64, 16368, 1152), (100, 9200, 1152), (64, 10256, 7168),
          (100, 2064, 7168), (250, 4112, 3968)]
# sixteen splits
LARGE += [(37, 528, 7168), (64, 272, 14336), (100, 48, 3968)]


@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8", "e8m0"])
@pytest.mark.parametrize("T,N,K", LARGE)
def test_linear_of_whole_numbers_at_larger_sizes(T, N, K, kind):
    c = linear_case(T, N, K, kind, True, gap=16)
    x, w = (torch.from_numpy(c[v]).to(DEV) for v in ("xv", "wv"))
    want = x @ w.T                             # float64
    assert torch.equal(run_linear(c, F32, gap=4).double(), want)
    if kind != "f32":                          # the kernels of 16-bit outputs, with the whole epilogue
        bias, res = torch.arange(N, device=DEV).float() - N // 2, spaced(T, N, BF, 8)
        res.copy_(torch.randint(-9, 10, (T, N), device=DEV, generator=c["g"]))
        got = run_linear(c, BF, "relu", bias, res, gap=8)
        assert torch.equal(got, ((want + bias).clamp(min=0) + res.double()).float().to(BF))


@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("fp8", "bf16"), ("fp8", "f32"),
                                      ("e8m0", "bf16"), ("e8m0", "f32")])
@pytest.mark.parametrize("T,N,K,act,bias,res", [
    (1, 96, 7168, "silu", 1, 0), (5, 256, 128, "none", 0, 1), (31, 208, 1024, "gelu", 1, 1), (64, 128, 2048, "relu", 1, 0),
    (130, 400, 512, "gelu_tanh", 0, 1), (333, 528, 1536, "silu", 1, 1), (700, 272, 256, "gelu", 1, 0)])
def test_linear_epilogue(T, N, K, act, bias, res, kind, out):
    c = linear_case(T, N, K, kind, False)
    n = lambda *s: torch.randn(*s, device=DEV, generator=c["g"])  # noqa: E731
    b = 3 * n(N) if bias else None
    r = None
    if res:
        r = spaced(T, N, TYPES[out], 16)
        r.copy_(2 * n(T, N))
    got = f64(run_linear(c, TYPES[out], act, b, r, gap=8))
    want, y, size = joins.linear(c["xv"], c["wv"], None if b is None else f64(b), act, None if r is None else f64(r))
    tol = 1.2 * (2 if kind in ("fp8", "e8m0") else 1) * (K + 8) * U * size + 512 * U * np.abs(joins.activate(y, act)) + 2 * U * np.abs(want)
    tol = tol + HALF[TYPES[out]] * (np.abs(want) + tol) + 2.0 ** -133
    err = np.abs(got - want)
    assert (err <= tol).all(), (err / tol).max()


def test_linear_residual_in_place_and_repeatable():
    m = rdg()
    for kind, T, N, K in (("bf16", 3, 256, 4096), ("bf16", 300, 512, 1024), ("fp8", 70, 384, 2048), ("e8m0", 260, 512, 512)):
        c = linear_case(T, N, K, kind, False)
        r = torch.randn(T, N, device=DEV, generator=c["g"]).to(BF)
        want = run_linear(c, BF, "silu", None, r)
        for _ in range(3):
            out = r.clone()
            m.rdg_linear(c["x"], c["xs"], c["kind"], c["w"], c["ws"], out, act=m.RDG_ACT_SILU, residual=out,
                         work=work_for(T, N, K, c["kind"]))
            assert torch.equal(out, want)


def test_linear_rows_do_not_touch_each_other():
    """NaN and infinities in one token's row reach no other row."""
    for kind, T, N, K in (("bf16", 40, 256, 512), ("bf16", 300, 272, 256), ("f32", 40, 64, 256)):
        c = linear_case(T, N, K, kind, False)
        want = run_linear(c, F32)
        c["x"][7, 5], c["x"][T - 1, K - 1] = float("nan"), float("inf")
        got = run_linear(c, F32)
        keep = [t for t in range(T) if t not in (7, T - 1)]
        assert torch.equal(got[keep], want[keep]) and got[7].isnan().all() and not got[T - 1].isfinite().any()


def test_linear_of_no_tokens():
    m = rdg()
    m.rdg_linear(torch.empty(0, 128, dtype=BF, device=DEV), None, m.RDG_BF16, torch.empty(16, 128, dtype=BF, device=DEV), None,
                 torch.empty(0, 16, dtype=BF, device=DEV))
    torch.cuda.synchronize()


def test_linear_output_past_32_bit_offsets():
    """An output whose last rows lie more than 2^32 bytes behind its first, rows far apart."""
    T, N, K = 300, 256, 128
    c = linear_case(T, N, K, "bf16", True)
    gap = 8_000_000
    buf = torch.empty(T * (N + gap), dtype=BF, device=DEV)
    out = buf.as_strided((T, N), (N + gap, 1))
    m = rdg()
    m.rdg_linear(c["x"], None, c["kind"], c["w"], None, out, work=work_for(T, N, K, c["kind"]))
    want = torch.from_numpy(c["xv"] @ c["wv"].T).to(BF)
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("T,N,stride", [(40, 256, 1 << 22), (40, 256, (1 << 22) - 8), (250, 272, (1 << 22) - 8), (300, 64, (1 << 22) + 8)])
def test_linear_of_rows_far_apart(T, N, stride):
    """x with 8 MiB from row to row: just below and just beyond the offsets that the tiles' loads hold."""
    m, K = rdg(), 256
    c = linear_case(T, N, K, "bf16", True)
    x = torch.empty(T * stride, dtype=BF, device=DEV).as_strided((T, K), (stride, 1))
    x.copy_(c["x"])
    out = torch.empty(T, N, device=DEV)
    m.rdg_linear(x, None, c["kind"], c["w"], None, out, work=work_for(T, N, K, c["kind"]))
    assert np.array_equal(f64(out), c["xv"] @ c["wv"].T)


# ---------------------------------------------------------------- routing
def route(logits, score, bias=None, group=1, keep=1, best=1, K=2, renorm=True, scale=1.0):
    m = rdg()
    B = logits.shape[0]
    ids = torch.full((B, K), -7, dtype=torch.int32, device=DEV)
    w = torch.full((B, K), -7.0, device=DEV)
    m.rdg_route_topk(logits, m.RDG_SCORE_SOFTMAX if score == "softmax" else m.RDG_SCORE_SIGMOID, group, keep, best, K, renorm,
                     scale, ids, w, bias=bias)
    return ids, w


def check_route(logits, score, bias=None, group=1, keep=1, best=1, K=2, renorm=True, scale=1.0):
    ids, w = route(logits, score, bias, group, keep, best, K, renorm, scale)
    want_ids, want = joins.route_topk(logits.float().cpu().numpy(), score, None if bias is None else bias.cpu().numpy(), group, keep,
                                      best, K, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    # scores below fp32's normal range have steps of 2^-149; a weight has a rounding or two of such scores
    assert (np.abs(f64(w) - want) <= (K + 4) * U * want + 2.0 ** -147 * abs(scale)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B,N,K,group,keep,best", [
    (5, 1, 1, 1, 1, 1), (70, 3, 3, 1, 1, 1), (33, 8, 2, 1, 1, 1), (1, 9, 4, 3, 2, 2), (50, 16, 4, 4, 2, 1), (31, 17, 17, 1, 1, 1),
    (9, 32, 8, 8, 3, 2), (17, 33, 5, 1, 1, 1), (12, 60, 4, 1, 1, 1), (7, 64, 6, 64, 9, 2), (6, 65, 32, 1, 1, 1), (21, 100, 7, 10, 4, 2),
    (19, 160, 6, 8, 3, 1), (40, 256, 8, 8, 4, 2), (3, 257, 8, 1, 1, 1), (6, 384, 8, 4, 1, 1), (5, 512, 10, 16, 5, 2), (4, 1000, 32, 40, 9, 2),
    (3, 1024, 8, 1, 1, 1), (2, 1024, 5, 1024, 7, 1)])
def test_route(B, N, K, group, keep, best, score):
    g = torch.Generator(device=DEV).manual_seed(B + N)
    n = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    logits = spaced(B, N, F32, 3)
    logits.copy_(2 * n(B, N))
    check_route(logits, score, None, group, keep, best, K, True, 2.5)
    check_route(logits, score, 0.1 * n(N), group, keep, best, K, False, 1.0)
    # bf16 logits tie often
    check_route((2 * n(B, N)).to(BF), score, None, group, keep, best, K, False, 0.5)
    check_route((2 * n(B, N)).to(BF), score, torch.round(4 * n(N)) / 4, group, keep, best, K, True)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("N,group,keep,K", [(256, 8, 4, 8), (64, 1, 1, 6), (160, 8, 3, 6), (48, 16, 5, 4), (1024, 4, 2, 8)])
def test_route_by_sigmoid_is_rdg_route(N, group, keep, K, biased):
    m = rdg()
    g = torch.Generator(device=DEV).manual_seed(N)
    logits = 3 * torch.randn(301, N, device=DEV, generator=g)
    logits[3] = 0
    logits[4, ::3] = 100
    bias = 0.3 * torch.randn(N, device=DEV, generator=g)
    ids, w = torch.empty(301, K, dtype=torch.int32, device=DEV), torch.empty(301, K, device=DEV)
    if biased:
        m.rdg_route_biased(logits, bias, group, keep, K, 2.5, ids, w)
    else:
        m.rdg_route(logits, group, keep, K, 2.5, ids, w)
    ids2, w2 = route(logits, "sigmoid", bias if biased else None, group, keep, 2, K, True, 2.5)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,group,keep", [(8, 1, 1), (40, 1, 1), (64, 8, 3), (256, 8, 2)])
def test_route_of_masked_and_broken_logits(N, group, keep, score):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(F32).min
    g = torch.Generator(device=DEV).manual_seed(N)
    logits = torch.randn(9, N, device=DEV, generator=g)
    logits[0] = -inf                    # nothing left
    logits[1] = low
    logits[2] = nan
    logits[3, 1:] = -inf                # one expert left
    logits[4, ::2] = nan
    logits[5, 3] = inf
    logits[6, 3], logits[6, 5], logits[6, 0] = inf, inf, nan
    logits[7, N // 2:] = low
    logits[8] = torch.linspace(-900, 0, N, device=DEV)  # scores below fp32's range
    for bias in (None, 0.2 * torch.randn(N, device=DEV, generator=g)):
        for renorm in (True, False):
            check_route(logits, score, bias, group, keep, 2, 4, renorm, 1.5)
    if score == "softmax":
        ids, w = route(logits, score, None, group, keep, 2, 4, True)
        assert ids[0].tolist() == [0, 1, 2, 3] and (w[0] == 0).all() and w[3].tolist() == [1, 0, 0, 0]
    # a bias that switches experts off, or means nothing
    bias = torch.zeros(N, device=DEV)
    bias[::2], bias[1] = -inf, nan
    check_route(logits, score, bias, group, keep, 1, 4, True)


@pytest.mark.parametrize("N,group,keep,K", [(16, 8, 3, 4), (32, 4, 2, 8), (64, 32, 5, 8), (256, 8, 2, 8), (512, 256, 9, 12), (96, 48, 48, 32)])
def test_route_of_biases_that_force_and_forbid(N, group, keep, K):
    """Infinite biases of both signs, also both within a group of two."""
    inf = float("inf")
    g = torch.Generator(device=DEV).manual_seed(N)
    bias = 0.1 * torch.randn(N, device=DEV, generator=g)
    bias[3], bias[2], bias[N - 2], bias[N - 1], bias[N // 2:N // 2 + 2] = inf, -inf, inf, inf, -inf
    for score in ("softmax", "sigmoid"):
        for best in (1, 2):
            check_route(torch.randn(37, N, device=DEV, generator=g), score, bias, group, keep, best, K, True)


def test_route_of_no_tokens():
    route(torch.empty(0, 16, device=DEV), "softmax")
    torch.cuda.synchronize()


# ---------------------------------------------------------------- together
class Block:
    """norm -> 8-bit projection with activation -> projection back onto the residual stream -> norm in both forms ->
    router product -> routing -> 8-bit experts' dispatch."""

    def __init__(self, T, H=512, F=1024, N=32, K=4, seed=0):
        m = rdg()
        self.m, self.T, self.H, self.F, self.N, self.K = m, T, H, F, N, K
        g = torch.Generator(device=DEV).manual_seed(seed)
        n = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
        self.x, self.r = n(T, H).to(BF), (2 * n(T, H)).to(BF)
        self.gain = 1 + 0.1 * n(H)
        self.up = (n(F, H) * H ** -0.5)
        self.upq, self.ups = torch.empty(F, H, dtype=torch.uint8, device=DEV), torch.empty(F // 128, H // 128, device=DEV)
        m.rdg_quantize_fp8(self.up, m.RDG_F32, 128, self.upq, self.ups)
        self.up_p = torch.empty_like(self.upq)
        m.rdg_pack_weights(self.upq, m.RDG_FP8_E4M3, self.up_p)
        self.down, self.router = (n(H, F) * F ** -0.5).to(BF), (n(N, H) * H ** -0.5).to(BF)
        self.down_p, self.router_p = torch.empty_like(self.down), torch.empty_like(self.router)
        m.rdg_pack_weights(self.down, m.RDG_BF16, self.down_p)
        m.rdg_pack_weights(self.router, m.RDG_BF16, self.router_p)
        self.bias = 0.2 * n(F)
        e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
        self.q, self.qs, self.r1, self.h, self.r2 = e(T, H, dt=torch.uint8), e(T, H // 128, dt=F32), e(T, H), e(T, F), e(T, H)
        self.n2, self.q2, self.qs2 = e(T, H), e(T, H, dt=torch.uint8), e(T, H // 128, dt=F32)
        self.logits, self.ids, self.w = e(T, N, dt=F32), e(T, K, dt=torch.int32), e(T, K, dt=F32)
        size = max(m.rdg_linear_workspace_bytes(T, F, H, m.RDG_FP8_E4M3), m.rdg_linear_workspace_bytes(T, H, F, m.RDG_BF16),
                   m.rdg_linear_workspace_bytes(T, N, H, m.RDG_BF16))
        self.work = e(max(size, 16), dt=torch.uint8)
        self.layout = m.Layout(m.RDG_CONTIGUOUS, N, T, K, DEV, block_m=16)

    def run(self):
        m = self.m
        m.rdg_add_norm(self.x, self.gain, 1e-6, residual=self.r, residual_out=self.r1, q=self.q, q_scales=self.qs)
        m.rdg_linear(self.q, self.qs, m.RDG_FP8_E4M3, self.up_p, self.ups, self.h, bias=self.bias, act=m.RDG_ACT_SILU, work=self.work)
        m.rdg_linear(self.h, None, m.RDG_BF16, self.down_p, None, self.r2, residual=self.r1, work=self.work)
        m.rdg_add_norm(self.r2, self.gain, 1e-6, out=self.n2, q=self.q2, q_scales=self.qs2, q_dtype=m.RDG_FP8_E4M3_UE8M0)
        m.rdg_linear(self.n2, None, m.RDG_BF16, self.router_p, None, self.logits, work=self.work)
        m.rdg_route_topk(self.logits, m.RDG_SCORE_SOFTMAX, 1, 1, 1, self.K, True, 1.0, self.ids, self.w)
        m.rdg_dispatch(self.q2, self.qs2, m.RDG_FP8_E4M3_UE8M0, self.ids, self.layout, None)

    def results(self):
        return [t.clone() for t in (self.r1, self.q, self.qs, self.h, self.r2, self.n2, self.q2, self.qs2, self.logits, self.ids, self.w,
                                    self.layout.counts, self.layout.pos)]


@pytest.mark.parametrize("T", [1, 50, 300])
def test_run_together(T):
    b = Block(T)
    b.run()
    s, y = joins.add_norm(f64(b.x), f64(b.r), f64(b.gain), 1e-6)
    check_codes(b.q, b.qs, y, False)
    # each stage from what the one before it stored
    codes = lambda q, s, rows: f64(q.view(torch.float8_e4m3fn).float()) * f64(s).repeat(128, 1).repeat(rows, 0)[:q.shape[0]]  # noqa: E731
    h, z, size = joins.linear(codes(b.q, b.qs, 1), codes(b.upq, b.ups, 128), f64(b.bias), "silu", None)
    assert (np.abs(f64(b.h) - h) <= 2.5 * (b.H + 8) * U * size + (512 * U + 2.0 ** -8) * np.abs(h)).all()
    r2, _, size = joins.linear(f64(b.h), f64(b.down), None, "none", f64(b.r1))
    assert (np.abs(f64(b.r2) - r2) <= 1.1 * (b.F + 8) * U * size + (2 * U + 2.0 ** -8) * np.abs(r2)).all()
    _, n2 = joins.add_norm(f64(b.r2), None, f64(b.gain), 1e-6)
    check_codes(b.q2, b.qs2, n2, True)
    logits, _, size = joins.linear(f64(b.n2), f64(b.router), None, "none", None)
    assert (np.abs(f64(b.logits) - logits) <= 1.1 * (b.H + 8) * U * size).all()
    ids, w = joins.route_topk(b.logits.cpu().numpy(), "softmax", None, 1, 1, 1, b.K, True, 1.0)
    assert np.array_equal(b.ids.cpu().numpy(), ids)
    assert b.m.rdg_check_status(b.layout) == (0, 0)
    assert np.array_equal(b.layout.counts.cpu().numpy(), np.bincount(ids.ravel(), minlength=b.N))


@pytest.mark.parametrize("T", [4, 200])
def test_captured_and_replayed(T):
    """Several replays, new inputs and eager work between them, each equal to the eager run."""
    b = Block(T, seed=5)
    b.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        b.run()
    other = Block(T, seed=6)
    for i in range(5):
        b.x.copy_(torch.randn(T, b.H, device=DEV, generator=torch.Generator(device=DEV).manual_seed(i)))
        graph.replay()
        got = b.results()
        other.run()
        torch.cuda.synchronize()
        b.run()
        for u, v in zip(got, b.results()):
            assert torch.equal(u, v)


def test_two_streams_with_workspaces_of_their_own():
    blocks = [Block(200, seed=s) for s in (7, 8)]
    want = []
    for b in blocks:
        b.run()
        want.append(b.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(4):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.run()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        for u, v in zip(b.results(), w):
            assert torch.equal(u, v)


def test_two_graphs_that_share_a_workspace():
    """Captured apart, replayed in turn on one stream: what one leaves in the workspace does not reach the other."""
    blocks = [Block(60, seed=s) for s in (11, 12)]
    size = max(b.work.numel() for b in blocks)
    shared = torch.empty(size, dtype=torch.uint8, device=DEV)
    want, graphs = [], []
    for b in blocks:
        b.work = shared
        b.run()
        want.append(b.results())
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run()
        graphs.append(g)
    for i in range(6):
        graphs[i % 2].replay()
        shared.fill_(0xff)
        graphs[(i + 1) % 2].replay()
        for b, w in zip(blocks, want):
            for u, v in zip(b.results(), w):
                assert torch.equal(u, v)


def test_two_threads_on_streams_of_their_own():
    """The binding lets go of the interpreter during a call: two threads call at once."""
    import threading
    blocks = [Block(100, seed=s) for s in (21, 22)]
    want = []
    for b in blocks:
        b.run()
        want.append(b.results())
    torch.cuda.synchronize()
    failed = []

    def serve(b):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    b.run()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=serve, args=(b,)) for b in blocks]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for b, w in zip(blocks, want):
        for u, v in zip(b.results(), w):
            assert torch.equal(u, v)
