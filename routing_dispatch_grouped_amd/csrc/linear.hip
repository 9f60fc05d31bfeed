// Matrix product with bias, activation and residual in its epilogue:
//
//   out[t, f] = act(sum_k x[t, k] W[f, k] + bias[f]) + residual[t, f]
//
// products summed in fp32; fp8 partial sums of 128 are scaled by their
// activation and weight block scales in fp32; one rounding at the end.
//
// Design: a workgroup has 16 * FPW weight rows and 16 * NR tokens; its four
// waves take the reduction's 128-element blocks in turn (wave w blocks w, w + 4, ...), so
// that the weights stream through in order, and add their sums in LDS in wave order.
#include "linear.h"

namespace rdg {
namespace {

template <int DT, int FPW, int NR>
__global__ __launch_bounds__(256) void k_linear_rows(LinearCall a) {
    using O = LinOp<DT>;
    using op_t = typename O::op_t;
    constexpr int STEPS = 128 / O::KS;              // matrix steps of a 128-element block
    constexpr int U = STEPS > 4 ? 4 : STEPS;        // in flight
    __shared__ f32x4_t part[4][FPW * NR][kWave];
    const int wv = threadIdx.x / kWave, lane = lane_id();
    const int groups = a.N / 16, panels = (groups + FPW - 1) / FPW;
    const int panel = (int)(blockIdx.x % panels);
    const int64_t t0 = (int64_t)(blockIdx.x / panels) * (16 * NR);
    const int nkb = a.K / 128;
    // rows past the last: the last one again, not stored
    const uint8_t* w[FPW];
#pragma unroll
    for (int i = 0; i < FPW; ++i) {
        const int g = panel * FPW + i < groups ? panel * FPW + i : groups - 1;
        w[i] = static_cast<const uint8_t*>(a.w) + (int64_t)g * (a.K / O::KS) * O::BLK;
    }
    const uint8_t* x[NR];
    const float* xs[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        int64_t t = t0 + j * 16 + (lane & 15);
        t = t < a.T ? t : a.T - 1;
        x[j] = static_cast<const uint8_t*>(a.x) + t * a.x_stride * O::ESZ;
        xs[j] = DT == RDG_FP8_E4M3 ? a.x_scales + t * nkb : nullptr;
    }
    const float* ws[FPW];
#pragma unroll
    for (int i = 0; i < FPW; ++i) {
        const int g = panel * FPW + i < groups ? panel * FPW + i : groups - 1;
        ws[i] = DT == RDG_FP8_E4M3 ? a.w_scales + (int64_t)(g / 8) * nkb : nullptr;
    }
    f32x4_t acc[FPW][NR];
#pragma unroll
    for (int i = 0; i < FPW; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    for (int kb = wv; kb < nkb; kb += 4) {
#pragma unroll
        for (int s0 = 0; s0 < STEPS; s0 += U) {
            op_t rw[U][FPW], rx[U][NR];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t step = (int64_t)kb * STEPS + s0 + u;
#pragma unroll
                for (int i = 0; i < FPW; ++i) rw[u][i] = O::load_w(w[i] + step * O::BLK, lane);
#pragma unroll
                for (int j = 0; j < NR; ++j) rx[u][j] = O::load_x(x[j], (int)step * O::KS, lane);
            }
            if constexpr (DT == RDG_FP8_E4M3) {
#pragma unroll
                for (int j = 0; j < NR; ++j) {
                    const float sx = xs[j][kb];
#pragma unroll
                    for (int i = 0; i < FPW; ++i) acc[i][j] += O::mma(f32x4_t{0.f, 0.f, 0.f, 0.f}, rw[0][i], rx[0][j]) * (sx * ws[i][kb]);
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < FPW; ++i)
#pragma unroll
                        for (int j = 0; j < NR; ++j) acc[i][j] = O::mma(acc[i][j], rw[u][i], rx[u][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < FPW; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j) part[wv][i * NR + j][lane] = acc[i][j];
    __syncthreads();
    // lane l of a 16 x 16 tile: token l % 16, features 4 (l / 16) .. + 3
    for (int c = wv; c < FPW * NR; c += 4) {
        const int i = c / NR, j = c % NR;
        const int64_t t = t0 + j * 16 + (lane & 15);
        const int f = (panel * FPW + i) * 16 + (lane >> 4) * 4;
        if (t >= a.T || f >= a.N) continue;
        f32x4_t v = part[0][c][lane];
#pragma unroll
        for (int u = 1; u < 4; ++u) v += part[u][c][lane];
        finish4(a, v, t, f);
    }
}

template <int DT, int FPW, int NR>
hipError_t launch_rows(const LinearCall& a, hipStream_t s) {
    const int64_t panels = (a.N / 16 + FPW - 1) / FPW;
    const int64_t blocks = panels * (((int64_t)a.T + 16 * NR - 1) / (16 * NR));
    if (!grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
    k_linear_rows<DT, FPW, NR><<<(unsigned)blocks, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const LinearCall& a, hipStream_t s) {
    if (a.T <= 16) return launch_rows<DT, 1, 1>(a, s);
    if (a.T <= 32) return launch_rows<DT, 1, 2>(a, s);
    return launch_rows<DT, 2, 4>(a, s);
}

}  // namespace

hipError_t launch_linear(const LinearCall& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    if (a.dtype != RDG_F32 && a.T > 256) return launch_linear_tiled(a, s);
    switch (a.dtype) {
        case RDG_F32: return launch_dt<RDG_F32>(a, s);
        case RDG_BF16: return launch_dt<RDG_BF16>(a, s);
        default: return launch_dt<RDG_FP8_E4M3>(a, s);
    }
}

size_t linear_workspace_bytes(int T, int N, int K, int dtype) { return 0; }

}  // namespace rdg
