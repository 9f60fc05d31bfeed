// Query/key norm for each head with the position rotation, and the store of
// the step's keys and values into the 8-bit paged cache, in one pass over the
// projections.
//
//   y = x / sqrt(mean(x^2) + eps) * w          (q and k heads, over head_dim)
//   (a, b) -> (a cos - b sin, b cos + a sin)   (the first rot_dim elements)
//   page scale s = smallest 2^k with amax <= 448 * 2^k over the page's rows
//   code = RNE_e4m3(clamp(y / s, -448, 448))
//
// All in fp32, rounded once: q to its type, k and v to their codes.  With
// power-of-two scales a division by s is exact, so the code is the nearest one to
// the fp32 value, and when later tokens of a page need a larger scale its
// older codes move by a power of two, which rounds only those that fall below
// e4m3's normal range.
//
// Bound by HBM: each projection is read once and q, the codes and the scales
// written once.  A head vector lies in head_dim / 8 lanes (8 elements each,
// 16-byte loads of bf16), so the norm's sum is a few lane exchanges and the
// rotation's partner is in the same wave.  The grid holds two kinds of
// workgroup: query workgroups, whose waves take a token's cos/sin once for
// several heads, and page workgroups, one per (page touched, head, k or v),
// which keep the page's new rows in registers between the maximum and the
// rounding.
//
// Measured: 17614 tokens of 64 / 8 heads of 128, bf16: 148 us, 4.7 TB/s, what a large copy
// reaches on the card.  64 tokens of 32 / 8 heads into begun pages: 6.3 us of
// latency (segment, slots, rows and scale are read one after the other).
#include "vec8.h"

namespace rdg {
namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.0f;

// cos and sin of this lane's 8 elements (elements past rot_dim: not used).
struct Turn {
    float c[8], s[8];
};

__device__ __forceinline__ Turn load_turn(const QkStoreCall& a, int pos, int j) {
    Turn t;
    const int half = a.rot_dim / 2, e = 8 * j;
    if (e < a.rot_dim) {
        const float* row = a.cos_sin + (int64_t)pos * a.rot_dim;
        if (!a.neighbours) {
            const int k = e < half ? e : e - half;
            load8<false>(row, k, t.c);
            load8<false>(row, half + k, t.s);
        } else {
            const float4 c = *reinterpret_cast<const float4*>(row + e / 2);
            const float4 s = *reinterpret_cast<const float4*>(row + half + e / 2);
            t.c[0] = t.c[1] = c.x, t.c[2] = t.c[3] = c.y, t.c[4] = t.c[5] = c.z, t.c[6] = t.c[7] = c.w;
            t.s[0] = t.s[1] = s.x, t.s[2] = t.s[3] = s.y, t.s[4] = t.s[5] = s.z, t.s[6] = t.s[7] = s.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) t.c[i] = 1.0f, t.s[i] = 0.0f;
    }
    return t;
}

// Norm over the LPV lanes of a head vector.
template <int LPV>
__device__ __forceinline__ void norm8(float (&x)[8], const float (&w)[8], float eps) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int off = LPV / 2; off >= 1; off >>= 1) ss += __shfl_xor(ss, off);
    const float inv = 1.0f / sqrtf(ss * (1.0f / (8 * LPV)) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
}

// Rotation; j = the lane's place in its head vector.  Every lane of the wave
// takes part in the exchange.
template <int LPV>
__device__ __forceinline__ void rotate8(float (&x)[8], const Turn& t, int j, int rot_dim, bool neighbours) {
    if (rot_dim == 0) return;
    if (!neighbours) {
        const int step = rot_dim / 16;  // lanes between an element and its partner
        const int src = j < step ? lane_id() + step : j < 2 * step ? lane_id() - step : lane_id();
        const float sign = j < step ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float o = __shfl(x[i], src);
            if (j < 2 * step) x[i] = x[i] * t.c[i] + sign * (o * t.s[i]);
        }
    } else if (8 * j < rot_dim) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float u = x[i], v = x[i + 1];
            x[i] = u * t.c[i] - v * t.s[i];
            x[i + 1] = v * t.c[i] + u * t.s[i];
        }
    }
}

__device__ __forceinline__ int checked_pos(const QkStoreCall& a, int t) {
    if (a.rot_dim == 0) return 0;
    const int p = a.positions[t];
    if ((unsigned)p < (unsigned)a.n_pos) return p;
    set_status(a.status, RDG_EDATA, t);
    return p < 0 ? 0 : a.n_pos - 1;
}

// e4m3 codes of x / 2^k; infinities saturate, NaN becomes 0x7f (the conversion
// gives NaN either sign: both mean NaN, one is stored).
__device__ __forceinline__ uint2 encode8(const float (&x)[8], int k) {
    float v[8];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        nan |= x[i] != x[i];
        v[i] = fminf(fmaxf(__builtin_amdgcn_ldexpf(x[i], -k), -kE4m3Max), kE4m3Max);
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

__device__ __forceinline__ void decode8(uint2 c, float (&x)[8]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(c.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(c.x, true);
    const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8(c.y, false), e = __builtin_amdgcn_cvt_pk_f32_fp8(c.y, true);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = d.x, x[5] = d.y, x[6] = e.x, x[7] = e.y;
}

// Exponent of the smallest power of two s with amax <= 448 s.  An all-zero
// block takes the smallest scale, so that it never holds later rows back.
__device__ __forceinline__ int scale_exp(float amax) {
    return amax > 0.0f ? e8m0_of(fp8_block_scale(amax, true)) - 127 : -126;
}

// Query workgroups: one (token, heads_per_wave heads) item per wave.
template <int D, bool BF16>
__device__ void query_part(const QkStoreCall& a, int64_t item) {
    constexpr int LPV = D / 8, VPW = kWave / LPV;  // lanes per vector, vectors per wave and pass
    if (item >= a.q_items) return;
    const int t = (int)(item / a.q_chunks), h0 = (int)(item % a.q_chunks) * a.q_passes * VPW;
    const int j = lane_id() % LPV, v = lane_id() / LPV;
    const Turn turn = load_turn(a, checked_pos(a, t), j);
    float w[8];
    if (a.q_weight) load8<false>(a.q_weight, 8 * j, w);
    const int64_t row = (int64_t)t * a.row_stride, out = (int64_t)t * a.q_stride;
    for (int p = 0; p < a.q_passes; ++p) {
        const int h = h0 + p * VPW + v;
        if (h0 + p * VPW >= a.n_q) break;
        const int hc = h < a.n_q ? h : a.n_q - 1;  // every lane takes part in the exchanges
        float x[8];
        load8<BF16>(a.qkv, row + (int64_t)hc * D + 8 * j, x);
        if (a.q_weight) norm8<LPV>(x, w, a.eps);
        rotate8<LPV>(x, turn, j, a.rot_dim, a.neighbours);
        if (h < a.n_q) store8<BF16>(a.q_out, out + (int64_t)h * D + 8 * j, x);
    }
}

// Page workgroups: the rows of one segment, head and operand.
template <int D, bool BF16, int NP>
__device__ void page_part(const QkStoreCall& a, int item) {
    constexpr int LPV = D / 8, RPP = kThreads / LPV;  // rows per pass
    __shared__ float red[kThreads / kWave];
    const int P = a.page_rows;
    const int seg = item / (2 * a.n_kv), h = item % (2 * a.n_kv);
    const bool is_k = h < a.n_kv;
    const int head = is_k ? h : h - a.n_kv;
    const int lead = a.seg_tok[seg];
    if (lead < 0) return;
    if (lead >= a.T) {
        if (threadIdx.x == 0) set_status(a.status, RDG_EDATA, lead);
        return;
    }
    const int slot = a.slots[lead];
    if (slot < 0 || (int64_t)slot >= (int64_t)a.n_pages * P) {
        if (threadIdx.x == 0) set_status(a.status, RDG_EDATA, lead);
        return;
    }
    const int page = slot / P, off = slot % P;  // P is a power of two, but not the compiler's to know
    // new rows: the tokens behind the leader whose slots follow its own
    int m = 0;
    for (int b = 0; b < P - off; b += kWave) {
        const int i = b + lane_id();
        const bool next = i < P - off && lead + i < a.T && a.slots[lead + i] == slot + i;
        const uint64_t gap = ~__ballot(next);
        const int run = gap ? __builtin_ctzll(gap) : kWave;
        m += run;
        if (run < kWave) break;
    }
    const int j = threadIdx.x % LPV, row0 = threadIdx.x / LPV;
    float w[8];
    const bool norm = is_k && a.k_weight;
    if (norm) load8<false>(a.k_weight, 8 * j, w);
    const int64_t col = (int64_t)(a.n_q + h) * D + 8 * j;

    float x[NP][8];
    float amax = 0.0f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int i = p * RPP + row0 - off;
        if (i >= 0 && i < m) load8<BF16>(a.qkv, (int64_t)(lead + i) * a.row_stride + col, x[p]);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) x[p][e] = 0.0f;
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int i = p * RPP + row0 - off;
        const bool fresh = i >= 0 && i < m;
        if (__ballot(fresh) == 0) continue;  // the same for the whole wave
        if (norm) norm8<LPV>(x[p], w, a.eps);
        if (is_k && a.rot_dim) {
            const Turn turn = load_turn(a, fresh ? checked_pos(a, lead + i) : 0, j);
            rotate8<LPV>(x[p], turn, j, a.rot_dim, a.neighbours);
        }
        if (fresh) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = fabsf(x[p][e]);
                amax = f < __builtin_inff() ? fmaxf(amax, f) : amax;  // infinities and NaN do not set the scale
            }
        }
    }
    amax = wave_max_f32(amax);
    if (lane_id() == 0) red[threadIdx.x / kWave] = amax;
    float* scale = (is_k ? a.k_scale : a.v_scale) + (int64_t)page * a.n_kv + head;
    int old_k = -126;
    if (off > 0) {
        old_k = e8m0_of(fabsf(*scale)) - 127;
        old_k = old_k < -126 ? -126 : old_k > 127 ? 127 : old_k;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / kWave; ++i) amax = fmaxf(amax, red[i]);
    const int new_k = scale_exp(amax);
    const int k = new_k > old_k ? new_k : old_k;
    uint8_t* codes = (is_k ? a.k_codes : a.v_codes) + ((int64_t)page * a.n_kv + head) * P * D + 8 * j;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int row = p * RPP + row0, i = row - off;
        uint2* to = reinterpret_cast<uint2*>(codes + (int64_t)row * D);
        if (i >= 0 && i < m) {
            *to = encode8(x[p], k);
        } else if (i < 0 && k > old_k && row < P) {
            float y[8];
            decode8(*to, y);
            *to = encode8(y, k - old_k);
        }
    }
    if (threadIdx.x == 0) *scale = __uint_as_float((uint32_t)(k + 127) << 23);
}

template <int D, bool BF16, int NP>
__global__ __launch_bounds__(kThreads) void k_qk_store(QkStoreCall a) {
    // the page workgroups first: their work takes longest
    if ((int)blockIdx.x < a.page_items) page_part<D, BF16, NP>(a, blockIdx.x);
    else query_part<D, BF16>(a, (int64_t)((int)blockIdx.x - a.page_items) * (kThreads / kWave) + threadIdx.x / kWave);
}

template <int D, bool BF16>
hipError_t launch_d(const QkStoreCall& a, unsigned grid, hipStream_t s) {
    constexpr int RPP = kThreads / (D / 8);
    const int np = a.page_rows <= RPP ? 1 : a.page_rows / RPP;
    if constexpr (D == 256) {
        if (np == 16) {
            k_qk_store<D, BF16, 16><<<grid, kThreads, 0, s>>>(a);
            return hipGetLastError();
        }
    }
    if constexpr (D >= 128) {
        if (np == 8) {
            k_qk_store<D, BF16, 8><<<grid, kThreads, 0, s>>>(a);
            return hipGetLastError();
        }
    }
    switch (np) {
        case 1: k_qk_store<D, BF16, 1><<<grid, kThreads, 0, s>>>(a); break;
        case 2: k_qk_store<D, BF16, 2><<<grid, kThreads, 0, s>>>(a); break;
        case 4: k_qk_store<D, BF16, 4><<<grid, kThreads, 0, s>>>(a); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_store(QkStoreCall a, int head_dim, bool bf16, int seg_cap, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    const int vpw = kWave * 8 / head_dim, groups = (a.n_q + vpw - 1) / vpw;
    // A wave keeps its token's turn for up to four groups of heads where tokens alone fill
    // the chip: 64 / 8 heads of 128, 2048 tokens 17.7 us (one group a wave: 20.3), 4096 31.9
    // (40.6), 17614 148 (200); at 1024 and fewer they are level (11.6 and 11.9).
    a.q_passes = a.T >= 1024 && groups > 1 ? (groups < 4 ? groups : 4) : 1;
    a.q_chunks = (groups + a.q_passes - 1) / a.q_passes;
    a.q_items = (int64_t)a.T * a.q_chunks;
    const int64_t pages = (int64_t)seg_cap * 2 * a.n_kv, q_blocks = (a.q_items + 3) / 4;
    if (!grid_fits(pages + q_blocks, kThreads)) return hipErrorInvalidConfiguration;
    if (pages + q_blocks == 0) return hipSuccess;  // neither queries nor keys and values: an empty grid is an error
    a.page_items = (int)pages;
    const unsigned grid = (unsigned)(pages + q_blocks);
    switch (head_dim) {
        case 64: return bf16 ? launch_d<64, true>(a, grid, s) : launch_d<64, false>(a, grid, s);
        case 128: return bf16 ? launch_d<128, true>(a, grid, s) : launch_d<128, false>(a, grid, s);
        default: return bf16 ? launch_d<256, true>(a, grid, s) : launch_d<256, false>(a, grid, s);
    }
}

}  // namespace rdg
