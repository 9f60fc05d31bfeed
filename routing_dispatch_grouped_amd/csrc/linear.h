// Matrix product with bias, activation and residual in its epilogue: operands
// of the matrix instructions and the epilogue, shared by its kernels.
#pragma once
#include "vec8.h"

namespace rdg {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// Per type: the reduction elements KS of a matrix instruction, the bytes BLK of a packed
// 16-row weight tile (pack.hip) and the instruction.
template <int DT>
struct LinOp;

template <>
struct LinOp<RDG_F32> {
    using op_t = float;
    static constexpr int KS = 4, ESZ = 4, BLK = 256;
    __device__ static op_t load_w(const uint8_t* tile, int lane) { return reinterpret_cast<const float*>(tile)[lane]; }
    __device__ static op_t stream_w(const uint8_t* tile, int lane) {
        return __builtin_nontemporal_load(reinterpret_cast<const float*>(tile) + lane);
    }
    __device__ static op_t load_x(const uint8_t* row, int k, int lane) {
        return reinterpret_cast<const float*>(row)[k + (lane >> 4)];
    }
    __device__ static f32x4_t mma(f32x4_t c, op_t a, op_t b) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }
};

template <>
struct LinOp<RDG_BF16> {
    using op_t = bf16x8_t;
    static constexpr int KS = 32, ESZ = 2, BLK = 1024;
    __device__ static op_t load_w(const uint8_t* tile, int lane) {
        return *reinterpret_cast<const bf16x8_t*>(tile + lane * 16);
    }
    __device__ static op_t stream_w(const uint8_t* tile, int lane) {
        return __builtin_nontemporal_load(reinterpret_cast<const bf16x8_t*>(tile + lane * 16));
    }
    __device__ static op_t load_x(const uint8_t* row, int k, int lane) {
        return *reinterpret_cast<const bf16x8_t*>(row + (int64_t)(k + (lane >> 4) * 8) * 2);
    }
    __device__ static f32x4_t mma(f32x4_t c, op_t a, op_t b) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

template <>
struct LinOp<RDG_FP8_E4M3> {
    using op_t = i32x8_t;
    static constexpr int KS = 128, ESZ = 1, BLK = 2048;  // a step is one block of 128 with its scales
    __device__ static op_t join(i32x4_t a, i32x4_t b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }
    __device__ static op_t load_w(const uint8_t* tile, int lane) {
        return join(*reinterpret_cast<const i32x4_t*>(tile + lane * 16), *reinterpret_cast<const i32x4_t*>(tile + 1024 + lane * 16));
    }
    __device__ static op_t stream_w(const uint8_t* tile, int lane) {
        return join(__builtin_nontemporal_load(reinterpret_cast<const i32x4_t*>(tile + lane * 16)),
                    __builtin_nontemporal_load(reinterpret_cast<const i32x4_t*>(tile + 1024 + lane * 16)));
    }
    __device__ static op_t load_x(const uint8_t* row, int k, int lane) {
        const i32x4_t* p = reinterpret_cast<const i32x4_t*>(row + k + (lane >> 4) * 32);
        return join(p[0], p[1]);
    }
    // The matrix core adds e4m3 products eight at a time (consecutive elements), each cut to a multiple of 2^-13 of the
    // power of two of the largest of them; the sums of eight, and the running sum, are added as fp32 holds them.
    // So a sum loses up to 7 * 2^-13 of each eight's largest product, on even terms 1.5e-5 of itself, and 1.2% of the results in
    // bf16, whose half step is 2^-9, are the neighbour of the value's own rounding.
    __device__ static f32x4_t mma(f32x4_t c, op_t a, op_t b) {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 127, 0, 127);
    }
    // The same from bf16 operands, which hold every code: products of 8 bits, added as fp32 holds them (1e-7 of the sum).  On the
    // tiles it costs half the rate and the conversions: 64 tokens on 18432 features of K = 7168 28 -> 46 us, 4001
    // tokens 424 .. 468 -> 940.  Taken where the output is fp32, and by the kernel for few tokens.
    // widen: elements 8 c .. 8 c + 7 of the lane's 32, as they are in bf16
    __device__ static bf16x8_t widen(op_t a, int c) {
        typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
        bf16x8_t r;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)a[2 * c + h], 1.0f, false);
            const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)a[2 * c + h], 1.0f, true);
            r[4 * h] = lo[0], r[4 * h + 1] = lo[1], r[4 * h + 2] = hi[0], r[4 * h + 3] = hi[1];
        }
        return r;
    }
    __device__ static f32x4_t mma_wide(f32x4_t c, op_t a, op_t b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(a, i), widen(b, i), c, 0, 0, 0);
        return c;
    }
};

// The kernels of a LinearPart.
enum { kRows, kTile256, kTile128, kTile128x64, kTile64x32, kTile96x64, kTile80x64, kTile64x64 };  // k_linear_rows, or the tile of k_linear_tiled

// The activations, in fp32 by the instructions for 2^v and 1 / v (each good to an ulp; results below 2^-126 come out as 0).
// An exponential's argument is rounded a few times, at most 3 * 128 u of its value where it is 2^-128, u = 2^-24.
__device__ __forceinline__ float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float one_over(float v) { return __builtin_amdgcn_rcpf(v); }

// y / (1 + exp(-u)), by the exponential of -|u|, which does not overflow
__device__ __forceinline__ float times_sigmoid(float y, float u) {
    const float e = exp2_of(fabsf(u) * -1.44269504088896341f);
    return y * ((u < 0.0f ? e : 1.0f) * one_over(1.0f + e));
}

// y Phi(y) = y - y Phi(-y), Phi(-|y|) = erfc(w) / 2 with w = |y| / sqrt(2).  erfc(w) = t exp(-w^2) g(t), t = 1 / (1 + w / 2):
// the form of Press et al., Numerical Recipes, in base 2:
// log2 g is smooth on 0 < t <= 1, and the polynomial of degree 9 through it at 4000 Chebyshev nodes by least squares is off
// by 7e-8 (evaluated in fp32 by 3e-7, relative to erfc).  Past |y| = 40 Phi(-|y|) is 0 in fp32, and |y| counts as 40 where it
// would be inf * 0.
__device__ __forceinline__ float gelu(float y) {
    constexpr float c[10] = {-1.82572699f, 1.4422425f, 0.544218361f, 0.117095776f, -0.201445639f,
                             0.276221722f, -1.4883672f, 2.03882122f, -1.14183986f, 0.238780305f};
    const float m = fminf(fabsf(y), 40.0f);
    const float t = one_over(fmaf(m, 0.35355339059327376f, 1.0f));
    float g = c[9];
#pragma unroll
    for (int i = 8; i >= 0; --i) g = fmaf(g, t, c[i]);
    const float phi = 0.5f * t * exp2_of(fmaf(m * m, -0.72134752044448170f, g));
    return y < 0.0f ? y * phi : y - m * phi;
}

template <int M>
__device__ __forceinline__ void activate(float (&v)[M], int act) {
    switch (act) {
        case RDG_ACT_RELU:
#pragma unroll
            for (int e = 0; e < M; ++e) v[e] = v[e] < 0.0f ? 0.0f : v[e];
            break;
        case RDG_ACT_SILU:
#pragma unroll
            for (int e = 0; e < M; ++e) v[e] = times_sigmoid(v[e], v[e]);
            break;
        case RDG_ACT_GELU:
#pragma unroll
            for (int e = 0; e < M; ++e) v[e] = gelu(v[e]);
            break;
        case RDG_ACT_GELU_TANH:  // y (1 + tanh(u / 2)) / 2, u = 2 sqrt(2 / pi) (y + 0.044715 y^3)
#pragma unroll
            for (int e = 0; e < M; ++e) v[e] = times_sigmoid(v[e], 1.5957691216057308f * (v[e] + 0.044715f * v[e] * v[e] * v[e]));
            break;
        default: break;
    }
}

// Features f..f+3 of token t: bias, activation, residual, one rounding to out's type.
__device__ __forceinline__ void finish4(const LinearCall& a, f32x4_t v, int64_t t, int f) {
    if (a.bias != nullptr) v += *reinterpret_cast<const f32x4_t*>(a.bias + f);
    if (a.act != RDG_ACT_NONE) {
        float y[4] = {v[0], v[1], v[2], v[3]};
        activate(y, a.act);
        v = f32x4_t{y[0], y[1], y[2], y[3]};
    }
    if (a.out_bf16) {
        if (a.residual != nullptr) {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.residual) + t * a.res_stride + f);
            v[0] += __uint_as_float(u.x << 16), v[1] += __uint_as_float(u.x & 0xffff0000u);
            v[2] += __uint_as_float(u.y << 16), v[3] += __uint_as_float(u.y & 0xffff0000u);
        }
        typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
        *reinterpret_cast<bf16x4_t*>(static_cast<uint16_t*>(a.out) + t * a.out_stride + f) =
            __builtin_convertvector(v, bf16x4_t);
    } else {
        if (a.residual != nullptr)
            v += *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(a.residual) + t * a.res_stride + f);
        *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + t * a.out_stride + f) = v;
    }
}

// Features f..f+7 of token t: as finish4.
__device__ __forceinline__ void finish8(const LinearCall& a, float (&v)[8], int64_t t, int f) {
    if (a.bias != nullptr) {
        float bias[8];
        load8<false>(a.bias, f, bias);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += bias[e];
    }
    activate(v, a.act);
    if (a.residual != nullptr) {
        float r[8];
        if (a.out_bf16) load8<true>(a.residual, t * a.res_stride + f, r);
        else load8<false>(a.residual, t * a.res_stride + f, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += r[e];
    }
    if (a.out_bf16) store8<true>(a.out, t * a.out_stride + f, v);
    else store8<false>(a.out, t * a.out_stride + f, v);
}

}  // namespace rdg
