// C ABI of the joins of a decoder layer (include/rdg.h): the norm with the residual's
// addition, the matrix product with its epilogue, and routing by scores.  Argument checks, then
// enqueue.
#include <math.h>

#include "rdg_internal.h"

using namespace rdg;

namespace {

// InvalidConfiguration: sizes whose grid no launch holds.
inline int hip_rc(hipError_t e) {
    return e == hipSuccess ? RDG_OK : e == hipErrorInvalidConfiguration ? RDG_EUNSUPPORTED : RDG_EHIP;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows of n elements of esz bytes every `stride` elements, each on 16 bytes; at most 2^61 bytes in all, so
// that offsets fit.
inline bool rows_ok(const void* p, int64_t stride, int64_t n, int64_t rows, int esz) {
    return p != nullptr && aligned16(p) && stride >= n && stride < (int64_t)1 << 28 && stride * esz % 16 == 0 && rows < (int64_t)1 << 31;
}

// An output may lie where an input lies only as the same rows: the same type, and the same stride beyond one row.
inline bool apart_or_same(const void* to, const void* from, bool same_type, int64_t to_stride, int64_t from_stride, int T) {
    return to == nullptr || to != from || (same_type && (to_stride == from_stride || T == 1));
}

inline bool is_fp8(int dtype) { return dtype == RDG_FP8_E4M3 || dtype == RDG_FP8_E4M3_UE8M0; }
inline bool is_float(int dtype) { return dtype == RDG_F32 || dtype == RDG_BF16; }
inline int size_of(int dtype) { return dtype == RDG_F32 ? 4 : dtype == RDG_BF16 ? 2 : 1; }

bool linear_sizes_ok(int T, int N, int K, int dtype) {
    return T >= 0 && N >= 16 && N % 16 == 0 && K >= 128 && K % 128 == 0 && (is_float(dtype) || is_fp8(dtype));
}

}  // namespace

extern "C" {

int rdg_add_norm(const void* x, int x_dtype, int64_t x_stride, int T, int H, const void* residual, void* residual_out,
                 int res_dtype, int64_t res_stride, const float* weight, float eps, void* out, int64_t out_stride,
                 uint8_t* q, float* q_scales, int q_dtype, rdg_stream_t stream) {
    if (T < 0 || H < 8 || H % 8 != 0 || !is_float(x_dtype) || !(eps >= 0.0f) || isinf(eps)) return RDG_EINVAL;
    if (H > kNormMax) return RDG_EUNSUPPORTED;
    if (T == 0) return RDG_OK;
    if (out == nullptr && q == nullptr) return RDG_EINVAL;
    if (q != nullptr && (H % 128 != 0 || !is_fp8(q_dtype))) return RDG_EINVAL;
    if (residual == nullptr ? residual_out != nullptr : !is_float(res_dtype)) return RDG_EINVAL;
    if (!rows_ok(x, x_stride, H, T, size_of(x_dtype))) return RDG_EINVAL;
    if (residual != nullptr && !rows_ok(residual, res_stride, H, T, size_of(res_dtype))) return RDG_EINVAL;
    if (residual_out != nullptr && !aligned16(residual_out)) return RDG_EINVAL;
    if (out != nullptr && !rows_ok(out, out_stride, H, T, size_of(x_dtype))) return RDG_EINVAL;
    if (q != nullptr && (!aligned16(q) || q_scales == nullptr || !aligned16(q_scales))) return RDG_EINVAL;
    if (weight != nullptr && !aligned16(weight)) return RDG_EINVAL;
    // two outputs in one place, or one that would run over an input's other rows
    if (residual_out != nullptr && residual_out == out) return RDG_EINVAL;
    if (q != nullptr && (q == x || q == residual || q == residual_out || q == out)) return RDG_EINVAL;
    const bool alike = residual != nullptr && res_dtype == x_dtype;
    if (!apart_or_same(residual_out, x, alike, res_stride, x_stride, T) || !apart_or_same(out, x, true, out_stride, x_stride, T) ||
        !apart_or_same(out, residual, alike, out_stride, res_stride, T))
        return RDG_EINVAL;
    AddNormCall a{};
    a.x = x, a.residual = residual, a.residual_out = residual_out, a.weight = weight, a.out = out, a.q = q;
    a.q_scales = q_scales, a.x_stride = x_stride, a.res_stride = res_stride, a.out_stride = out_stride, a.eps = eps;
    a.T = T, a.H = H, a.x_bf16 = x_dtype == RDG_BF16, a.res_bf16 = res_dtype == RDG_BF16;
    a.pow2 = q_dtype == RDG_FP8_E4M3_UE8M0;
    return hip_rc(launch_add_norm(a, stream));
}

size_t rdg_linear_workspace_bytes(int T, int N, int K, int dtype) {
    return linear_sizes_ok(T, N, K, dtype) && T > 0 ? linear_work_bytes(linear_plan(T, N, K, dtype), T) : 0;
}

// For the tests, not in rdg.h: kernel, splits and features of a call's two parts.
void rdg_linear_plan_of(int T, int N, int K, int dtype, int* parts) {
    const LinearPlan p = linear_plan(T, N, K, dtype);
    const LinearPart* of[2] = {&p.first, &p.rest};
    for (int i = 0; i < 2; ++i) parts[3 * i] = of[i]->kernel, parts[3 * i + 1] = of[i]->splits, parts[3 * i + 2] = of[i]->features;
}

size_t rdg_linear_workspace_bound(int T, int N, int K, int dtype) {
    return linear_sizes_ok(T, N, K, dtype) ? linear_work_bound(T, N, K, dtype) : 0;
}

int rdg_linear(const void* x, const float* x_scales, int dtype, int64_t x_stride, int T, int N, int K, const void* W,
               const float* W_scales, const float* bias, int act, const void* residual, int64_t res_stride, void* out,
               int out_dtype, int64_t out_stride, void* work, size_t work_bytes, rdg_stream_t stream) {
    if (!linear_sizes_ok(T, N, K, dtype) || !is_float(out_dtype)) return RDG_EINVAL;
    if (act < RDG_ACT_NONE || act > RDG_ACT_GELU_TANH) return RDG_EINVAL;
    if (dtype == RDG_F32 && out_dtype != RDG_F32) return RDG_EUNSUPPORTED;
    if (T == 0) return RDG_OK;
    if (!rows_ok(x, x_stride, K, T, size_of(dtype)) || !rows_ok(out, out_stride, N, T, size_of(out_dtype))) return RDG_EINVAL;
    if (W == nullptr || !aligned16(W)) return RDG_EINVAL;
    if (is_fp8(dtype) && (x_scales == nullptr || W_scales == nullptr || !aligned16(x_scales) || !aligned16(W_scales)))
        return RDG_EINVAL;
    if (bias != nullptr && !aligned16(bias)) return RDG_EINVAL;
    if (residual != nullptr && !rows_ok(residual, res_stride, N, T, size_of(out_dtype))) return RDG_EINVAL;
    if (out == x || out == W || !apart_or_same(out, residual, true, out_stride, res_stride, T)) return RDG_EINVAL;
    const LinearPlan plan = linear_plan(T, N, K, dtype);
    const size_t need = linear_work_bytes(plan, T);
    if (need > 0 && (work == nullptr || !aligned16(work) || work_bytes < need)) return RDG_EINVAL;
    LinearCall a{};
    a.x = x, a.w = W, a.x_scales = x_scales, a.w_scales = W_scales, a.bias = bias, a.residual = residual, a.out = out;
    a.parts = static_cast<float*>(work);
    a.x_stride = x_stride, a.res_stride = res_stride, a.out_stride = out_stride;
    a.T = T, a.N = N, a.K = K, a.dtype = dtype, a.act = act, a.out_bf16 = out_dtype == RDG_BF16;
    return hip_rc(launch_linear(a, plan, stream));
}

int rdg_route_topk(const void* logits, int dtype, int64_t logit_stride, int B, int N, int score, const float* bias,
                   int n_group, int topk_group, int group_best, int K, int renorm, float scale, int32_t* topk_ids,
                   float* topk_w, rdg_stream_t stream) {
    if (B < 0 || N < 1 || N > 1024 || n_group < 1 || N % n_group != 0 || !is_float(dtype)) return RDG_EINVAL;
    if (score != RDG_SCORE_SOFTMAX && score != RDG_SCORE_SIGMOID) return RDG_EINVAL;
    if (topk_group < 1 || topk_group > n_group || (group_best != 1 && group_best != 2)) return RDG_EINVAL;
    if (K < 1 || K > 32 || K > topk_group * (N / n_group)) return RDG_EINVAL;
    if (B == 0) return RDG_OK;
    if (logits == nullptr || topk_ids == nullptr || topk_w == nullptr) return RDG_EINVAL;
    if (logit_stride < N || logit_stride >= (int64_t)1 << 28) return RDG_EINVAL;
    RouteCall a{};
    a.logits = logits, a.bias = bias, a.ids = topk_ids, a.w = topk_w, a.stride = logit_stride, a.scale = scale;
    a.B = B, a.N = N, a.n_group = n_group, a.topk_group = topk_group, a.group_best = group_best, a.K = K;
    a.softmax = score == RDG_SCORE_SOFTMAX, a.bf16 = dtype == RDG_BF16, a.renorm = renorm != 0;
    return hip_rc(launch_route_topk(a, stream));
}

}  // extern "C"
