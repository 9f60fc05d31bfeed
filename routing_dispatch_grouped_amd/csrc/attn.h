// What the two attention kernels share: the call, the rows' key ranges, and
// the 8-bit codes' way into MFMA operands.
#pragma once
#include "rdg_internal.h"

namespace rdg {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr float kLn2 = 0.6931471805599453f;
// The running maximum is raised only when a row outgrows it by more than this
// (base-2 exponent): probabilities then reach 2^8 instead of 1, at the same
// relative precision, and the output is rescaled a few times instead of at most tiles.
// Relative error of bf16 outputs against 64 bits: 0.0017 to 0.0021, where rounding
// an exact result costs 0.0017.
constexpr float kSlack = 8.0f;

// k_attn_rows workgroups for each key head and chunk.
inline int row_tiles(const AttnCall& a) { return a.row_places > 0 ? a.row_places : a.R; }

// A request's queries and keys.  Query i has position kv - n + i.
struct ReqSpan {
    int t0, n, kv;
};

__device__ __forceinline__ ReqSpan req_span(const AttnCall& a, int r) {
    ReqSpan s;
    int t0 = a.cu_q[r], t1 = a.cu_q[r + 1], kv = a.kv_len[r];
    // offsets and lengths that the buffers cannot hold are cut to what they can
    t0 = t0 < 0 ? 0 : t0 > a.T ? a.T : t0;
    t1 = t1 < t0 ? t0 : t1 > a.T ? a.T : t1;
    const int most = a.kv_cap;
    if (kv < 0 || kv > most) {
        if (threadIdx.x == 0) set_status(a.status, RDG_EDATA, r);
        kv = kv < 0 ? 0 : most;
    }
    s.t0 = t0;
    s.n = t1 - t0;
    s.kv = kv;
    // grids and parts are sized for max_q queries: a longer request is left out
    if (s.n > a.max_q) {
        if (threadIdx.x == 0) set_status(a.status, RDG_EDATA, r);
        s.n = 0;
    }
    return s;
}

// Row tiles of `rows` rows by place: request r's have the places from
// floor(cu_q[r] * group / rows) + r on, as many as it can need, whatever its
// neighbours' lengths, so T * group / rows + R places hold every request's.  The
// request of a place (wave-uniform; -1: none), and the first place of its tiles:
__device__ __forceinline__ int request_of_place(const AttnCall& a, int place, int rows) {
    int r = -1;
    for (int b = 0; b < a.R; b += kWave) {
        const int i = b + lane_id();
        bool before = false;
        if (i < a.R) {
            const int t = a.cu_q[i];
            before = (int64_t)(t < 0 ? 0 : t) * a.group / rows + i <= place;
        }
        r += __popcll(__ballot(before));
    }
    return __builtin_amdgcn_readfirstlane(r);
}
__device__ __forceinline__ int first_place(const AttnCall& a, const ReqSpan& s, int r, int rows) {
    return (int)((int64_t)s.t0 * a.group / rows + r);
}

// Keys [lo, hi) that query i of the request sees (hi <= lo: none).
__device__ __forceinline__ int key_hi(const AttnCall& a, const ReqSpan& s, int i) {
    if (!a.causal) return s.kv;
    const int pos = s.kv - s.n + i;
    return pos < 0 ? 0 : pos + 1;
}
__device__ __forceinline__ int key_lo(const AttnCall& a, const ReqSpan& s, int i) {
    if (a.window == 0) return 0;
    const int lo = s.kv - s.n + i - a.window + 1;
    return lo < 0 ? 0 : lo;
}

// The keys of a tile of rows [row0, row1) of one request and key head (row =
// query * group + head of the group): [begin, end) holds every key that any of them
// sees, begin a multiple of the 64-key blocks; it is cut into chunks of `chunk` keys.
struct TileKeys {
    int begin, end, chunks;
};
__device__ __forceinline__ TileKeys tile_keys(const AttnCall& a, const ReqSpan& s, int row0, int row1, int chunk) {
    TileKeys k;
    k.begin = key_lo(a, s, row0 / a.group) & ~63;
    k.end = key_hi(a, s, (row1 - 1) / a.group);
    k.chunks = k.end > k.begin ? (k.end - k.begin + chunk - 1) / chunk : 1;
    return k;
}

// The first part of head h of a request's query i among the short requests' parts.
__device__ __forceinline__ int64_t row_part(const AttnCall& a, const ReqSpan& s, int r, int i, int h) {
    const int64_t place = a.row_place > 0 ? (int64_t)r * a.row_place + i : s.t0 + i;
    return (place * a.n_q + h) * a.row_chunks;
}

// Page of a key, made safe: ids outside the cache are reported and read page 0.
__device__ __forceinline__ int page_of(const AttnCall& a, int r, int key) {
    int page = a.block_table[(int64_t)r * a.max_blocks + (key >> a.page_shift)];
    if ((unsigned)page >= (unsigned)a.n_pages) {
        set_status(a.status, RDG_EDATA, r);
        page = 0;
    }
    return page;
}

// A stored scale as the power of two that it is (its exponent alone counts).
__device__ __forceinline__ float pow2_scale(float s) { return __uint_as_float(__float_as_uint(s) & 0x7f800000u); }

// 8 codes -> 8 bf16 values, times a power of two: exact.
__device__ __forceinline__ bf16x8_t codes_to_bf16(uint32_t w0, uint32_t w1, float s0, float s1) {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s0, false);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s0, true);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s1, false);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s1, true);
    return bf16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Bytes of four dwords, transposed: out[b] holds byte b of r[0..3].
__device__ __forceinline__ void transpose4(const uint32_t (&r)[4], uint32_t (&out)[4]) {
    const uint32_t a = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u), b = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u);
    const uint32_t c = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u), d = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
    out[0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    out[1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    out[2] = __builtin_amdgcn_perm(d, c, 0x05040100u);
    out[3] = __builtin_amdgcn_perm(d, c, 0x07060302u);
}

// Reductions across the wave's halves and quarters, in the vector unit
// (v_permlane*_swap with one value as both operands leaves both sides' values).
__device__ __forceinline__ float max_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float max_quarters(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_quarters(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// NaN in V.  0 * NaN would carry a key's NaN into rows that do not see it, so in
// tiles that some row does not see whole, NaN codes go into the product as zeros;
// where there were any, the rows that do see them get their NaN at the end.
// 0x80 in each byte of w that is a NaN code (0x7f or 0xff):
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t without_nan(uint32_t w, uint32_t nan) { return w & ~((nan >> 7) * 0xffu); }

// Elements d..d+3 of a finished row: acc / total, 0 and -inf where it sees no key.
template <bool BF16>
__device__ __forceinline__ void store_part(const AttnCall& a, int t, int h, int d, int D, float4 acc, float total,
                                           float top, bool none) {
    const float inv = 1.0f / total;
    const float v[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
    const int64_t at = (int64_t)t * a.out_stride + (int64_t)h * D + d;
    if constexpr (BF16) {
        typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
        bf16x4_t b;
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = none ? (__bf16)0.0f : (__bf16)v[i];
        *reinterpret_cast<bf16x4_t*>(static_cast<uint16_t*>(a.out) + at) = b;
    } else {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) =
            none ? make_float4(0, 0, 0, 0) : make_float4(v[0], v[1], v[2], v[3]);
    }
    if (a.lse && d == 0)
        a.lse[(int64_t)t * a.n_q + h] = none ? -__builtin_inff() : (top + __builtin_amdgcn_logf(total)) * kLn2;
}

}  // namespace rdg
