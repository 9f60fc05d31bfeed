// Routing scores, shared by the routers: the sigmoid and the exponential in fp64,
// and the order of fp32 scores as unsigned integers.
#pragma once
#include "rdg_internal.h"

#pragma clang fp contract(off)

namespace rdg {

// The score: sigmoid in fp64, rounded once to fp32.  Every step is one IEEE
// double operation so the value is identical wherever it is evaluated:
//   x clamped to [-87, 87]; z = -x; n = rint(z * log2(e));
//   r = z - n*ln2 with ln 2 split in a 42-bit head (exact products) and a tail;
//   e^r by its degree-13 Taylor series (Horner, fma, 1/k! rounded to double);
//   e^z = e^r * 2^n exactly; score = (float)(1 / (1 + e^z)).
// The truncation error of the series for |r| <= ln2/2 is below 2^-55.
constexpr double kLog2e = 0x1.71547652b82fep+0;   // double nearest 1/ln 2
constexpr double kLn2Hi = 0x1.62e42fefa3800p-1;   // double ln 2, 42 significant bits
constexpr double kLn2Lo = 0x1.ef00000000000p-45;  // double ln 2 minus the head
constexpr double kInvFact[14] = {
    0x1.0000000000000p+0,  0x1.0000000000000p+0,  0x1.0000000000000p-1,  0x1.5555555555555p-3,
    0x1.5555555555555p-5,  0x1.1111111111111p-7,  0x1.6c16c16c16c17p-10, 0x1.a01a01a01a01ap-13,
    0x1.a01a01a01a01ap-16, 0x1.71de3a556c734p-19, 0x1.27e4fb7789f5cp-22, 0x1.ae64567f544e4p-26,
    0x1.1eed8eff8d898p-29, 0x1.6124613a86d09p-33};

// e^z for z in [-800, 87] (0 below what fp64 holds).
__device__ __forceinline__ double exp64(double z) {
    double n = __builtin_rint(z * kLog2e);
    double r = __builtin_fma(-n, kLn2Hi, z);
    r = __builtin_fma(-n, kLn2Lo, r);
    double p = kInvFact[13];
#pragma unroll
    for (int k = 12; k >= 0; --k) p = __builtin_fma(p, r, kInvFact[k]);
    return __builtin_ldexp(p, (int)n);
}

__device__ __forceinline__ float score_sigmoid(float xf) {
    xf = fminf(fmaxf(xf, -87.0f), 87.0f);
    return (float)(1.0 / (1.0 + exp64(-(double)xf)));
}

// fp32 -> uint32 whose unsigned order is the numeric order (negative values
// have every bit flipped, non-negative ones the sign bit); never 0 for a
// finite value
__device__ __forceinline__ uint32_t ordered_bits(float v) {
    const uint32_t u = __float_as_uint(v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

}  // namespace rdg
