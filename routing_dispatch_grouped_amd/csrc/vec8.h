// Eight consecutive elements of a row in a lane (bf16: 16 bytes, fp32: 32), and
// exchanges among the lanes of a wave in the vector unit.
#pragma once
#include "rdg_internal.h"

namespace rdg {

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&x)[8]) {
    if constexpr (BF16) {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    } else {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = f[0], b = f[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&x)[8]) {
    if constexpr (BF16) {
        bf16x8_t b;
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = (__bf16)x[j];
        *reinterpret_cast<bf16x8_t*>(static_cast<uint16_t*>(p) + i) = b;
    } else {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// The value of another lane: DPP controls that pair lanes inside quads, eights and
// rows of 16 (once the lanes of a quad agree, a mirrored eight pairs its quads, and so on).
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;

template <int CTRL>
__device__ __forceinline__ uint32_t lane_of(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float lane_of(float x) {
    return __uint_as_float(lane_of<CTRL>(__float_as_uint(x)));
}
template <int CTRL>
__device__ __forceinline__ double lane_of(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    return __longlong_as_double((int64_t)(lane_of<CTRL>((uint32_t)u) | ((uint64_t)lane_of<CTRL>((uint32_t)(u >> 32)) << 32)));
}

// Both values of a pair of lanes 16 (32) apart, in the same order in both.
template <int APART>
__device__ __forceinline__ void pair_of(uint32_t x, uint32_t& a, uint32_t& b) {
    static_assert(APART == 16 || APART == 32, "rows of 16 lanes, halves of the wave");
    if constexpr (APART == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        a = r[0], b = r[1];
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        a = r[0], b = r[1];
    }
}
template <int APART>
__device__ __forceinline__ void pair_of(float x, float& a, float& b) {
    uint32_t u, v;
    pair_of<APART>(__float_as_uint(x), u, v);
    a = __uint_as_float(u), b = __uint_as_float(v);
}
template <int APART>
__device__ __forceinline__ void pair_of(double x, double& a, double& b) {
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    uint32_t l0, l1, h0, h1;
    pair_of<APART>((uint32_t)u, l0, l1);
    pair_of<APART>((uint32_t)(u >> 32), h0, h1);
    a = __longlong_as_double((int64_t)(l0 | ((uint64_t)h0 << 32)));
    b = __longlong_as_double((int64_t)(l1 | ((uint64_t)h1 << 32)));
}

// op over each aligned set of LANES lanes (8, 16, 32 or 64), left in all of them: the same tree
// in every lane, so the same bits for a commutative op.
template <int LANES, class T, class Op>
__device__ __forceinline__ T across(T x, Op op) {
    static_assert(LANES == 8 || LANES == 16 || LANES == 32 || LANES == 64, "lanes of a set");
    x = op(x, lane_of<kSwap1>(x));
    x = op(x, lane_of<kSwap2>(x));
    x = op(x, lane_of<kMirror8>(x));
    if constexpr (LANES >= 16) x = op(x, lane_of<kMirror16>(x));
    if constexpr (LANES >= 32) {
        T a, b;
        pair_of<16>(x, a, b);
        x = op(a, b);
    }
    if constexpr (LANES >= 64) {
        T a, b;
        pair_of<32>(x, a, b);
        x = op(a, b);
    }
    return x;
}

}  // namespace rdg
