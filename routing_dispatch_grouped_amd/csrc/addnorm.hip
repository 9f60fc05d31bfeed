// The residual's addition with the root-mean-square norm and its 8-bit output, in
// one pass over the rows.
//
//   s = x + r                                   r' = s rounded to the residual's type
//   y = s / sqrt(mean(s^2) + eps) * g           out = y rounded to x's type
//   scale = amax / 448 of y's 1 x 128 blocks, or the smallest power of two not below it
//   code = RNE_e4m3(clamp(y / scale, -448, 448))
//
// s, the sum of squares and y are fp32; the norm takes s before it is rounded
// to the residual's type, and the codes take y before it is rounded to x's.
//
// Bound by HBM for many rows, by latency for few.  A row lies in the registers
// of NT threads, V vectors of 8 elements each, between its one read and its one
// write.  Up to 1024 elements a row is within a wave (up to 512 with a vector a lane, several short rows to a wave), so
// that its sum needs no LDS; beyond, as few vectors a thread as 1024 threads allow: 64 bf16 rows of 7168 with residual, output
// and codes 4.5 us, with 256 threads of 4 vectors 5.9 (512 rows 8.3 and 9.8; 16384 rows the same).  Rows
// of up to 4096 take 256 threads: 1087 fp32 rows of 1536 4.0 us, with 1024 threads 5.1.  The workgroups that the chip
// holds at a time walk over the rows with their weights in registers.
//
// Measured: 16384 bf16 rows of 7168 with residual and codes 166 us, 4.98 TB/s (a large copy has 4.8 to 5.1);
// 100000 rows of 128 with output and codes 19.3 us (one row a wave: 48.8); one row of 7168 2.9 us of latency.
#include <type_traits>

#include "vec8.h"

namespace rdg {
namespace {

constexpr float kE4m3Max = 448.0f;

// e4m3 codes of x / s; infinities saturate, NaN becomes 0x7f.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float s) {
    float v[8];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        nan |= x[i] != x[i];
        v[i] = fminf(fmaxf(x[i] / s, -kE4m3Max), kE4m3Max);
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
        w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], w[h], true);
    }
    if (nan) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (x[i] != x[i]) w[i / 4] = (w[i / 4] & ~(0xffu << (8 * (i & 3)))) | (0x7fu << (8 * (i & 3)));
    }
    return make_uint2(w[0], w[1]);
}

// XB: x and out are bf16 (else fp32).  RES: 0 no residual, 1 fp32, 2 bf16.  NT: threads of a row, V: vectors of a thread.
template <bool XB, int RES, int NT, int V>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_add_norm(AddNormCall a) {
    constexpr int ROWS = NT < 256 ? 256 / NT : 1;  // rows a workgroup
    __shared__ float part[2][NT < kWave ? 1 : NT / kWave];
    const int tid = (int)threadIdx.x % NT;
    const int nv = a.H / 8;
    float g[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = tid + j * NT;
        if (a.weight != nullptr && i < nv) {
            load8<false>(a.weight, 8 * i, g[j]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[j][e] = 1.0f;
        }
    }
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * ROWS; first < a.T; first += (int64_t)gridDim.x * ROWS) {
        // rows past the last: the last one again, not stored (the exchanges take every lane of the wave)
        const int64_t at = first + threadIdx.x / NT;
        const bool live = ROWS == 1 || at < a.T;
        const int64_t row = live ? at : a.T - 1;
        float s[V][8];
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * NT;
            if (i < nv) {
                load8<XB>(a.x, row * a.x_stride + 8 * i, s[j]);
                if constexpr (RES != 0) {
                    float r[8];
                    load8<RES == 2>(a.residual, row * a.res_stride + 8 * i, r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[j][e] += r[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) s[j][e] = 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(s[j][e], s[j][e], sum);
        sum = across<(NT < kWave ? NT : kWave)>(sum, [](float p, float q) { return p + q; });
        if constexpr (NT > kWave) {
            // two slots in turn: a wave writes the next row's before the others have read this one's
            if (lane_id() == 0) part[turn][tid / kWave] = sum;
            __syncthreads();
            sum = 0.0f;
#pragma unroll
            for (int w = 0; w < NT / kWave; ++w) sum += part[turn][w];
            turn ^= 1;
        }
        const float inv = 1.0f / sqrtf(sum / (float)a.H + a.eps);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * NT;
            if (i >= nv || !live) continue;  // the lanes of a 128-block are all here or all not
            if constexpr (RES != 0) {
                if (a.residual_out != nullptr) store8<RES == 2>(a.residual_out, row * a.res_stride + 8 * i, s[j]);
            }
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = s[j][e] * inv * g[j][e];
            if (a.out != nullptr) store8<XB>(a.out, row * a.out_stride + 8 * i, y);
            if (a.q != nullptr) {
                float amax = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float m = fabsf(y[e]);
                    amax = fmaxf(amax, m < __builtin_inff() ? m : 0.0f);
                }
                amax = across<16>(amax, [](float p, float q) { return fmaxf(p, q); });
                const float scale = fp8_block_scale(amax, a.pow2);
                *reinterpret_cast<uint2*>(a.q + row * a.H + 8 * i) = encode8(y, scale);
                if (i % 16 == 0) a.q_scales[row * (a.H / 128) + i / 16] = scale;
            }
        }
    }
}

template <bool XB, int RES>
hipError_t launch(const AddNormCall& a, hipStream_t s) {
    const int nv = a.H / 8;
    auto go = [&](auto nt, auto v) {
        constexpr int NT = decltype(nt)::value, V = decltype(v)::value;
        constexpr int ROWS = NT < 256 ? 256 / NT : 1;
        const int64_t groups = ((int64_t)a.T + ROWS - 1) / ROWS;
        const int64_t most = 256 * (2048 / (NT < 256 ? 256 : NT));
        k_add_norm<XB, RES, NT, V><<<(unsigned)(groups < most ? groups : most), NT < 256 ? 256 : NT, 0, s>>>(a);
        return hipGetLastError();
    };
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I4 = std::integral_constant<int, 4>;
    if (nv <= 16) return go(std::integral_constant<int, 16>{}, I1{});
    if (nv <= 32) return go(std::integral_constant<int, 32>{}, I1{});
    if (nv <= 64) return go(std::integral_constant<int, 64>{}, I1{});
    if (nv <= 128) return go(std::integral_constant<int, 64>{}, I2{});
    if (nv <= 256) return go(std::integral_constant<int, 256>{}, I1{});
    if (nv <= 512) return go(std::integral_constant<int, 256>{}, I2{});
    if (nv <= 1024) return go(std::integral_constant<int, 1024>{}, I1{});
    if (nv <= 2048) return go(std::integral_constant<int, 1024>{}, I2{});
    return go(std::integral_constant<int, 1024>{}, I4{});
}

}  // namespace

hipError_t launch_add_norm(const AddNormCall& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    const int res = a.residual == nullptr ? 0 : a.res_bf16 ? 2 : 1;
    if (a.x_bf16) return res == 0 ? launch<true, 0>(a, s) : res == 1 ? launch<true, 1>(a, s) : launch<true, 2>(a, s);
    return res == 0 ? launch<false, 0>(a, s) : res == 1 ? launch<false, 1>(a, s) : launch<false, 2>(a, s);
}

}  // namespace rdg
