// Attention over the 8-bit paged cache, many query rows per request: prefill and
// prefill chunks in bf16.  The same mathematics as attn.hip's k_attn_rows (one
// pass, running maximum and sum in fp32); here the work is matrix products,
// 4 * head_dim flops per (query row, key), bound by the bf16 matrix rate and by
// the exponentials beside it.
//
// A workgroup takes 32 * RB rows per wave of one key head -- rows are (query, head
// of the group), so grouped heads share the tile -- and walks its keys in 64-key
// tiles.  The tile's codes become bf16 once for all waves, on their way into
// LDS: K by rows, V by columns, with each 16-key step's keys in the order in
// which S^T = K Q^T (v_mfma_f32_32x32x16_bf16) leaves them in a lane, so that the
// probabilities go from its result registers into O^T = V^T P^T's operand with no
// exchange.  A row is a lane of the result: maximum and sum over keys are
// in-lane but for one exchange between the wave's halves, and rescaling O^T is
// one factor per lane.  16-byte pieces are swizzled by row, so that reads and
// writes of 8 lanes fall into different banks.
//
// The next tile's codes are loaded before a tile's products and converted after
// them into the other LDS buffer: one barrier per tile.  Workgroup b works on
// key head b % n_kv, so with 8 heads each XCD's L2 holds the keys of one; row tiles run
// from a request's last to its first, longest work first.
#include <type_traits>

#include "attn.h"

namespace rdg {
namespace {

constexpr int kTile = 64;

template <int D>
struct TileLds {
    uint16_t k[2][kTile * D];
    uint16_t v[2][D * kTile];
    int nan;  // whether a masked tile's V held NaN
};

// Swizzles: the 16-byte piece that holds piece c of a K row / of a V^T row.
__device__ __forceinline__ int k_piece(int key, int c) { return c ^ (key & 7); }
__device__ __forceinline__ int v_piece(int d, int c) { return c ^ ((d & 7) ^ ((d >> 3) & 3)); }

template <int D, int NW>
__global__ __launch_bounds__(NW * kWave, 1) void k_attn_tiles(AttnCall a) {
    constexpr int BM = 32 * NW;
    constexpr int KS = D / 16, DB = D / 32;  // reduction steps of S^T, 32-row blocks of O^T
    // Staging: the first half of the waves loads V, the second K.
    constexpr int HT = NW / 2 * kWave;
    constexpr int KU = kTile * D / 16 / HT;  // 16-code K units per thread
    constexpr int VU = 8 * D / 4 / HT > 0 ? 8 * D / 4 / HT : 1;  // (8 keys x 4 columns) V units per thread
    constexpr bool kAllV = 8 * D / 4 >= HT;
    constexpr int RAW = 4 * KU > 8 * VU ? 4 * KU : 8 * VU;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    auto& lds = *reinterpret_cast<TileLds<D>*>(lds_raw);

    const int tid = (int)threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int col = lane & 31, half = lane >> 5;
    int id = (int)blockIdx.x;
    const int head = id % a.n_kv;
    id /= a.n_kv;
    const int slot = a.tile_slots - 1 - id % a.tile_slots, chunk = id / a.tile_slots;
    // request r's tiles have the places from floor(cu_q[r] * group / BM) + r on:
    // as many as it can need, whatever its neighbours' lengths
    int r = -1;
    for (int b = 0; b < a.R; b += kWave) {
        const int i = b + lane;
        bool before = false;
        if (i < a.R) {
            const int t = a.cu_q[i];
            before = (int64_t)(t < 0 ? 0 : t) * a.group / BM + i <= slot;
        }
        r += __popcll(__ballot(before));
    }
    r = __builtin_amdgcn_readfirstlane(r);
    if (r < 0) return;
    const ReqSpan s = req_span(a, r);
    const int G = a.group, rows = s.n * G;
    const int row0 = (slot - (int)((int64_t)s.t0 * G / BM + r)) * BM;
    if (s.n <= a.n_most || row0 < 0 || row0 >= rows) return;
    const int row1 = row0 + BM < rows ? row0 + BM : rows;
    const TileKeys keys = tile_keys(a, s, row0, row1, a.tile_chunk);
    if (chunk >= keys.chunks) return;
    const int any_lo = key_lo(a, s, row0 / G), any_hi = keys.end;
    const int wg_all_lo = key_lo(a, s, (row1 - 1) / G), wg_all_hi = key_hi(a, s, row0 / G);
    const int k0 = keys.begin + chunk * a.tile_chunk;
    const int k1 = any_hi < k0 + a.tile_chunk ? any_hi : k0 + a.tile_chunk;
    const int tiles = k1 > k0 ? (k1 - k0 + kTile - 1) / kTile : 0;

    // this wave's rows: one per lane of either half
    const int first = row0 + wave * 32, row = first + col;
    const int row_c = row < rows ? row : rows - 1;
    const int lo = key_lo(a, s, row_c / G), hi = key_hi(a, s, row_c / G);
    const int i0 = (first < rows ? first : rows - 1) / G, i1 = (first + 31 < rows ? first + 31 : rows - 1) / G;
    const int all_lo = key_lo(a, s, i1), all_hi = key_hi(a, s, i0);
    bf16x8_t q[KS];
    {
        const uint16_t* p = static_cast<const uint16_t*>(a.q) + (int64_t)(s.t0 + row_c / G) * a.q_stride +
                            (int64_t)(head * G + row_c % G) * D + 8 * half;
#pragma unroll
        for (int x = 0; x < KS; ++x) q[x] = *reinterpret_cast<const bf16x8_t*>(p + 16 * x);
    }

    // pages and scales of 16-key groups: lane l holds group 64 b + l of this chunk
    const bool stage_v = wave < NW / 2;
    const int st = tid - (stage_v ? 0 : HT);  // place among the threads that stage this operand
    const uint8_t* codes = stage_v ? a.v_codes : a.k_codes;
    const float* scales = stage_v ? a.v_scale : a.k_scale;
    int page = 0;
    float page_scale = 1.0f;
    const auto load_pages = [&](int b) {
        const int key = k0 + (b * kWave + lane) * 16;
        page = 0;
        page_scale = 1.0f;
        if (key < k1) {
            page = page_of(a, r, key);
            page_scale = pow2_scale(scales[(int64_t)page * a.n_kv + head]);
        }
    };
    const int in_page = (1 << a.page_shift) - 1;
    // first code of key `key` of this chunk's 16-key group g, and its scale
    const auto group_row = [&](int g, int key) -> const uint8_t* {
        const int pg = __shfl(page, g & (kWave - 1));
        return codes + ((((int64_t)pg * a.n_kv + head) << a.page_shift) + (key & in_page)) * D;
    };
    uint32_t raw[RAW];
    float raw_scale[KU > VU ? KU : VU];
    const auto load_tile = [&](int t) {  // V waves: tile t; K waves: tile t
        const int t0 = k0 + t * kTile;
        if (stage_v) {
#pragma unroll
            for (int u = 0; u < VU; ++u) {
                const int x = st + u * HT, c = (x / (D / 4)) & 7, dq = x % (D / 4);
                raw_scale[u] = __shfl(page_scale, (t * 4 + c / 2) & (kWave - 1));
                const uint8_t* p = group_row(t * 4 + c / 2, t0 + 16 * (c / 2) + 4 * (c & 1)) + 4 * dq;
                if (kAllV || x < 8 * D / 4) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        raw[8 * u + i] = *reinterpret_cast<const uint32_t*>(p + (8 * (i / 4) + (i & 3)) * D);
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                const int x = st + u * HT, key = x / (D / 16), c = x % (D / 16);
                raw_scale[u] = __shfl(page_scale, (t * 4 + key / 16) & (kWave - 1));
                const uint4 w = *reinterpret_cast<const uint4*>(group_row(t * 4 + key / 16, t0 + key) + 16 * c);
                raw[4 * u] = w.x, raw[4 * u + 1] = w.y, raw[4 * u + 2] = w.z, raw[4 * u + 3] = w.w;
            }
        }
    };
    const auto store_tile = [&](int t, uint16_t* to_k, uint16_t* to_v) {
        if (stage_v) {
            const int t0 = k0 + t * kTile;
            const bool masked = t0 < wg_all_lo || t0 + kTile > wg_all_hi;
            uint32_t saw = 0;
#pragma unroll
            for (int u = 0; u < VU; ++u) {
                const int x = st + u * HT, c = (x / (D / 4)) & 7, dq = x % (D / 4);
                if (kAllV || x < 8 * D / 4) {
                    if (masked) {
                        // keys that no row sees may hold anything
                        const int key = t0 + 16 * (c / 2) + 4 * (c & 1);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int j = key + 8 * (i / 4) + (i & 3);
                            if (j < any_lo || j >= any_hi) raw[8 * u + i] = 0;
                            const uint32_t nan = nan_bytes(raw[8 * u + i]);
                            raw[8 * u + i] = without_nan(raw[8 * u + i], nan);
                            saw |= nan;
                        }
                    }
                    const uint32_t in0[4] = {raw[8 * u], raw[8 * u + 1], raw[8 * u + 2], raw[8 * u + 3]};
                    const uint32_t in1[4] = {raw[8 * u + 4], raw[8 * u + 5], raw[8 * u + 6], raw[8 * u + 7]};
                    uint32_t x0[4], x1[4];
                    transpose4(in0, x0);
                    transpose4(in1, x1);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int d = 4 * dq + b;
                        *reinterpret_cast<bf16x8_t*>(to_v + d * kTile + 8 * v_piece(d, c)) =
                            codes_to_bf16(x0[b], x1[b], raw_scale[u], raw_scale[u]);
                    }
                }
            }
            if (saw) lds.nan = 1;
        } else {
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                const int x = st + u * HT, key = x / (D / 16), c = x % (D / 16);
                uint16_t* to = to_k + key * D;
                *reinterpret_cast<bf16x8_t*>(to + 8 * k_piece(key, 2 * c)) =
                    codes_to_bf16(raw[4 * u], raw[4 * u + 1], raw_scale[u], raw_scale[u]);
                *reinterpret_cast<bf16x8_t*>(to + 8 * k_piece(key, 2 * c + 1)) =
                    codes_to_bf16(raw[4 * u + 2], raw[4 * u + 3], raw_scale[u], raw_scale[u]);
            }
        }
    };
    // What a wave has staged: K waves run one tile ahead of V waves.
    const int ahead = stage_v ? 0 : 1;
    const auto fetch = [&](int t) {
        if (t < tiles) {
            if ((t & 15) == 0) load_pages(t / 16);
            load_tile(t);
        }
    };

    f32x16_t o[DB];
    float m = -__builtin_inff(), l = 0.0f;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] = 0.0f;
    const float scale = a.scale_log2;

    // LDS places of this lane's operand pieces: the swizzle touches only the low
    // three bits of a piece's number, so four of each, the rest are offsets.
    int k_at[4], v_at[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        k_at[x] = col * D + 8 * k_piece(col, 2 * x + half);
        v_at[x] = col * kTile + 8 * v_piece(col, 2 * x + half);
    }
    // operand y of the logits of keys 32 kb ..
    const auto k_frag = [&](const uint16_t* k, int kb, int y) {
        return *reinterpret_cast<const bf16x8_t*>(k + k_at[y & 3] + kb * 32 * D + (y / 4) * 64);
    };
    const auto v_frag = [&](const uint16_t* v, int db, int x) {
        return *reinterpret_cast<const bf16x8_t*>(v + v_at[x] + db * 32 * kTile);
    };
    const auto logits = [&](f32x16_t (&sc)[2], const uint16_t* k) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[kb][i] = 0.0f;
#pragma unroll
            for (int y = 0; y < KS; ++y)
                sc[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k_frag(k, kb, y), q[y], sc[kb], 0, 0, 0);
        }
    };
    // One tile: its softmax beside the next tile's logits, then its V product.
    const auto tile = [&](f32x16_t (&sc)[2], f32x16_t (&next)[2], int t, auto parity) {
        constexpr int B = decltype(parity)::value;
        const uint16_t *k_next = lds.k[1 - B], *v_now = lds.v[B];
        const int t0 = k0 + t * kTile;
        fetch(t + 1 + ahead);
        if (t0 < all_lo || t0 + kTile > all_hi) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = t0 + kb * 32 + 8 * (i / 4) + 4 * half + (i & 3);
                    if (key < lo || key >= hi) sc[kb][i] = -__builtin_inff();
                }
        }
        // eight groups of KG products and four exponentials, operands one group ahead
        constexpr int KG = KS / 4;
        bf16x8_t kf[KG];
#pragma unroll
        for (int x = 0; x < KG; ++x) kf[x] = k_frag(k_next, 0, x);
        float top = -__builtin_inff();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[kb][i]);
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m_new = fmaxf(m, top * scale);
        if (__any(m_new > m)) {
            const float shrink = __builtin_amdgcn_exp2f(m - (m_new == -__builtin_inff() ? 0.0f : m_new));
            l *= shrink;
#pragma unroll
            for (int db = 0; db < DB; ++db) o[db] *= shrink;
            m = m_new;
        }
        const float ref = m == -__builtin_inff() ? 0.0f : m;
        float sum = 0.0f;
        bf16x8_t p[4], vf[2];
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            __builtin_amdgcn_sched_barrier(0);
            const int kb = g / 4, y0 = (g & 3) * KG;
            if ((g & 3) == 0)
#pragma unroll
                for (int i = 0; i < 16; ++i) next[kb][i] = 0.0f;
            bf16x8_t ahead_f[KG];
            if (g < 7) {
#pragma unroll
                for (int x = 0; x < KG; ++x) ahead_f[x] = k_frag(k_next, (g + 1) / 4, ((g + 1) & 3) * KG + x);
            } else {
                vf[0] = v_frag(v_now, 0, 0);
                vf[1] = v_frag(v_now, 0, 1);
            }
            // past the last tile: of an old buffer, not used
#pragma unroll
            for (int x = 0; x < KG; ++x)
                next[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[x], q[y0 + x], next[kb], 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = __builtin_amdgcn_exp2f(fmaf(sc[kb][4 * (g & 3) + i], scale, -ref));
                sum += e;
                p[g / 2][4 * (g & 1) + i] = (__bf16)e;
            }
            // summed here and not behind the loop, where 32 exponentials would have to be kept
            asm volatile("" : "+v"(sum));
            if (g < 7) {
#pragma unroll
                for (int x = 0; x < KG; ++x) kf[x] = ahead_f[x];
            }
        }
        l += sum;
#pragma unroll
        for (int g = 0; g < 2 * DB; ++g) {
            __builtin_amdgcn_sched_barrier(0);
            bf16x8_t f0, f1;
            if (g + 1 < 2 * DB) {
                f0 = v_frag(v_now, (g + 1) / 2, 2 * ((g + 1) & 1));
                f1 = v_frag(v_now, (g + 1) / 2, 2 * ((g + 1) & 1) + 1);
            }
            o[g / 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[0], p[2 * (g & 1)], o[g / 2], 0, 0, 0);
            o[g / 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[1], p[2 * (g & 1) + 1], o[g / 2], 0, 0, 0);
            if (g + 1 < 2 * DB) vf[0] = f0, vf[1] = f1;
        }
        __builtin_amdgcn_sched_barrier(0);
        // K waves: into the buffer that this tile's logits came from
        if (t + 1 + ahead < tiles) store_tile(t + 1 + ahead, lds.k[B], lds.v[1 - B]);
        __syncthreads();
    };

    if (tid == 0) lds.nan = 0;
    __syncthreads();
    fetch(0);
    if (tiles > 0) store_tile(0, lds.k[0], lds.v[0]);
    if (!stage_v) {
        fetch(1);
        if (tiles > 1) store_tile(1, lds.k[1], lds.v[1]);
    }
    __syncthreads();
    if (tiles > 0) {
        f32x16_t s0[2], s1[2];
        logits(s0, lds.k[0]);
        __syncthreads();  // the first tile's buffer takes the third tile
        for (int t = 0; t < tiles; t += 2) {
            tile(s0, s1, t, std::integral_constant<int, 0>{});
            if (t + 1 < tiles) tile(s1, s0, t + 1, std::integral_constant<int, 1>{});
        }
    }

    if (lds.nan) {
        for (int t = 0; t < tiles; ++t) {
            const int t0 = k0 + t * kTile;
            if (t0 >= wg_all_lo && t0 + kTile <= wg_all_hi) continue;
            for (int j = t0; j < t0 + kTile && j < any_hi; ++j) {
                const int pg = page_of(a, r, j);
                const uint8_t* p = a.v_codes + ((((int64_t)pg * a.n_kv + head) << a.page_shift) + (j & in_page)) * D;
                if (j < lo || j >= hi) continue;
#pragma unroll
                for (int db = 0; db < DB; ++db)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if ((p[db * 32 + 8 * (i / 4) + 4 * half + (i & 3)] & 0x7f) == 0x7f) o[db][i] = __builtin_nanf("");
            }
        }
    }

    const float total = l + __shfl_xor(l, 32);
    if (row >= rows) return;
    const int i = row / G, h = head * G + row % G;
    const bool none = hi <= lo;
    const int64_t at = ((int64_t)(s.t0 + i) * a.n_q + h) * a.max_chunks + chunk;
    if (keys.chunks > 1 && half == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(m, total);
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = db * 32 + 8 * j + 4 * half;
            const float4 v = make_float4(o[db][4 * j], o[db][4 * j + 1], o[db][4 * j + 2], o[db][4 * j + 3]);
            if (keys.chunks == 1) store_part<true>(a, s.t0 + i, h, d, D, v, total, m, none);
            else *reinterpret_cast<float4*>(a.part_o + at * D + d) = v;
        }
}

template <int D, int NW>
hipError_t launch(const AttnCall& a, hipStream_t s) {
    constexpr size_t bytes = sizeof(TileLds<D>);
    static_assert(bytes <= 160 * 1024, "LDS");
    const int64_t grid = (int64_t)a.n_kv * a.tile_slots * a.tile_chunks;
    if (grid >= (int64_t)1 << 31) return hipErrorInvalidConfiguration;
    if (bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_attn_tiles<D, NW>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != hipSuccess) return e;
    }
    k_attn_tiles<D, NW><<<(unsigned)grid, NW * kWave, bytes, s>>>(a);
    return hipGetLastError();
}

}  // namespace

// a.tile_rows = attn_tile_rows(head_dim)
hipError_t launch_attn_tiles(const AttnCall& a, int head_dim, hipStream_t s) {
    switch (head_dim) {
        case 64: return launch<64, 8>(a, s);
        case 128: return launch<128, 8>(a, s);
        default: return launch<256, 4>(a, s);
    }
}

}  // namespace rdg
