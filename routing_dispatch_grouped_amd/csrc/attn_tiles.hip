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
#include "attn.h"

namespace rdg {
namespace {

constexpr int kTile = 64;

template <int D, int NW, int RB>
struct TileLds {
    uint16_t k[2][kTile * D];
    uint16_t v[2][D * kTile];
    int nan[3];
};

// Swizzles: the 16-byte piece that holds piece c of a K row / of a V^T row.
__device__ __forceinline__ int k_piece(int key, int c) { return c ^ (key & 7); }
__device__ __forceinline__ int v_piece(int d, int c) { return c ^ ((d & 7) ^ ((d >> 3) & 3)); }

template <int D, int NW, int RB>
__global__ __launch_bounds__(NW * kWave, 1) void k_attn_tiles(AttnCall a) {
    constexpr int NT = NW * kWave, BM = 32 * RB * NW;
    constexpr int KS = D / 16, DB = D / 32;                     // reduction steps of S, 32-row blocks of O^T
    constexpr int KU = kTile * D / 16 / NT;                     // 16-code K units per thread
    constexpr int VUNITS = 8 * D / 4, VU = (VUNITS + NT - 1) / NT;  // (8 keys x 4 columns) V units
    static_assert(KU >= 1 || kTile * D / 16 < NT, "");
    constexpr int KUN = KU >= 1 ? KU : 1;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    auto& lds = *reinterpret_cast<TileLds<D, NW, RB>*>(lds_raw);

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

    // this wave's rows
    bf16x8_t q[RB][KS];
    int lo[RB], hi[RB], all_lo[RB], all_hi[RB], see_lo[RB], see_hi[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int first = row0 + (wave * RB + rb) * 32, row = first + col;
        const bool live = row < rows;
        const int row_c = live ? row : rows - 1, i = row_c / G, h = head * G + row_c % G;
        lo[rb] = key_lo(a, s, i);
        hi[rb] = key_hi(a, s, i);
        const int i0 = (first < rows ? first : rows - 1) / G, i1 = (first + 31 < rows ? first + 31 : rows - 1) / G;
        see_lo[rb] = key_lo(a, s, i0), see_hi[rb] = key_hi(a, s, i1);
        all_lo[rb] = key_lo(a, s, i1), all_hi[rb] = key_hi(a, s, i0);
        if (first >= rows) see_hi[rb] = 0;
        const uint16_t* p = static_cast<const uint16_t*>(a.q) + (int64_t)(s.t0 + i) * a.q_stride + (int64_t)h * D + 8 * half;
#pragma unroll
        for (int x = 0; x < KS; ++x) q[rb][x] = *reinterpret_cast<const bf16x8_t*>(p + 16 * x);
    }

    // pages and scales of 16-key groups: lane l holds group 64 b + l of this chunk
    int page = 0;
    float ks = 1.0f, vs = 1.0f;
    const auto load_pages = [&](int b) {
        const int key = k0 + (b * kWave + lane) * 16;
        page = 0;
        ks = vs = 1.0f;
        if (key < k1) {
            page = page_of(a, r, key);
            ks = pow2_scale(a.k_scale[(int64_t)page * a.n_kv + head]);
            vs = pow2_scale(a.v_scale[(int64_t)page * a.n_kv + head]);
        }
    };
    uint4 kreg[KUN];
    float kscale[KUN], vscale[VU];
    uint32_t vreg[VU][8];
    const int in_page = (1 << a.page_shift) - 1;
    const auto load_tile = [&](int t) {
        const int t0 = k0 + t * kTile;
#pragma unroll
        for (int u = 0; u < KUN; ++u) {
            const int x = tid + u * NT, key = x / (D / 16), c = x % (D / 16);
            const int g = (t * 4 + key / 16) & (kWave - 1);
            const int pg = __shfl(page, g);
            kscale[u] = __shfl(ks, g);
            if (kTile * D / 16 >= NT || x < kTile * D / 16)
                kreg[u] = *reinterpret_cast<const uint4*>(
                    a.k_codes + (((((int64_t)pg * a.n_kv + head) << a.page_shift) + ((t0 + key) & in_page)) * D + 16 * c));
        }
#pragma unroll
        for (int u = 0; u < VU; ++u) {
            const int x = tid + u * NT, c = x / (D / 4), dq = x % (D / 4);
            const int g = (t * 4 + c / 2) & (kWave - 1);
            const int pg = __shfl(page, g);
            vscale[u] = __shfl(vs, g);
            const int key = t0 + 16 * (c / 2) + 4 * (c & 1);
            if (VUNITS % NT == 0 || x < VUNITS) {
                const uint8_t* p =
                    a.v_codes + (((((int64_t)pg * a.n_kv + head) << a.page_shift) + (key & in_page)) * D + 4 * dq);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    vreg[u][i] = *reinterpret_cast<const uint32_t*>(p + (8 * (i / 4) + (i & 3)) * D);
            }
        }
    };
    const auto store_tile = [&](int t) {
        const int t0 = k0 + t * kTile, buf = t & 1;
        const bool masked = t0 < wg_all_lo || t0 + kTile > wg_all_hi;
        bool nan = false;
#pragma unroll
        for (int u = 0; u < KUN; ++u) {
            const int x = tid + u * NT, key = x / (D / 16), c = x % (D / 16);
            if (kTile * D / 16 >= NT || x < kTile * D / 16) {
                uint16_t* row = lds.k[buf] + key * D;
                *reinterpret_cast<bf16x8_t*>(row + 8 * k_piece(key, 2 * c)) =
                    codes_to_bf16(kreg[u].x, kreg[u].y, kscale[u], kscale[u]);
                *reinterpret_cast<bf16x8_t*>(row + 8 * k_piece(key, 2 * c + 1)) =
                    codes_to_bf16(kreg[u].z, kreg[u].w, kscale[u], kscale[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < VU; ++u) {
            const int x = tid + u * NT, c = x / (D / 4), dq = x % (D / 4);
            if (VUNITS % NT == 0 || x < VUNITS) {
                if (masked) {
                    // keys that no row sees may hold anything; NaN in the others is marked
                    const int key = t0 + 16 * (c / 2) + 4 * (c & 1);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int j = key + 8 * (i / 4) + (i & 3);
                        if (j < any_lo || j >= any_hi) vreg[u][i] = 0;
                        nan |= has_nan(vreg[u][i]);
                    }
                }
                const uint32_t in0[4] = {vreg[u][0], vreg[u][1], vreg[u][2], vreg[u][3]};
                const uint32_t in1[4] = {vreg[u][4], vreg[u][5], vreg[u][6], vreg[u][7]};
                uint32_t x0[4], x1[4];
                transpose4(in0, x0);
                transpose4(in1, x1);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int d = 4 * dq + b;
                    *reinterpret_cast<bf16x8_t*>(lds.v[buf] + d * kTile + 8 * v_piece(d, c)) =
                        codes_to_bf16(x0[b], x1[b], vscale[u], vscale[u]);
                }
            }
        }
        if (nan) lds.nan[t % 3] = 1;
        if (tid == 0) lds.nan[(t + 1) % 3] = 0;
    };

    f32x16_t o[RB][DB];
    float m[RB], l[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        m[rb] = -__builtin_inff();
        l[rb] = 0.0f;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[rb][db][i] = 0.0f;
    }
    const float c = a.scale_log2;
    if (tid == 0) lds.nan[0] = 0;
    __syncthreads();
    if (tiles > 0) {
        load_pages(0);
        load_tile(0);
        store_tile(0);
    }
    __syncthreads();
    for (int t = 0; t < tiles; ++t) {
        const int t0 = k0 + t * kTile, buf = t & 1;
        if (t + 1 < tiles) {
            if (((t + 1) & 15) == 0) load_pages((t + 1) / 16);
            load_tile(t + 1);
        }
        bool any = false;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) any |= t0 < see_hi[rb] && t0 + kTile > see_lo[rb];
        if (any) {
            f32x16_t sc[RB][2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
                for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) sc[rb][kb][i] = 0.0f;
                const int key = kb * 32 + col;
                const uint16_t* row = lds.k[buf] + key * D;
#pragma unroll
                for (int x = 0; x < KS; ++x) {
                    const bf16x8_t kf = *reinterpret_cast<const bf16x8_t*>(row + 8 * k_piece(key, 2 * x + half));
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb)
                        sc[rb][kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, q[rb][x], sc[rb][kb], 0, 0, 0);
                }
            }
            bf16x8_t p[RB][4];
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                if (t0 < all_lo[rb] || t0 + kTile > all_hi[rb]) {
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int key = t0 + kb * 32 + 8 * (i / 4) + 4 * half + (i & 3);
                            if (key < lo[rb] || key >= hi[rb]) sc[rb][kb][i] = -__builtin_inff();
                        }
                }
                float top = -__builtin_inff();
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[rb][kb][i]);
                top = fmaxf(top, __shfl_xor(top, 32));
                const float m_new = fmaxf(m[rb], top * c);
                if (__any(m_new > m[rb])) {
                    const float shrink = __builtin_amdgcn_exp2f(m[rb] - (m_new == -__builtin_inff() ? 0.0f : m_new));
                    l[rb] *= shrink;
#pragma unroll
                    for (int db = 0; db < DB; ++db) o[rb][db] *= shrink;
                    m[rb] = m_new;
                }
                const float ref = m[rb] == -__builtin_inff() ? 0.0f : m[rb];
                float sum = 0.0f;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float e = __builtin_amdgcn_exp2f(fmaf(sc[rb][kb][i], c, -ref));
                        sum += e;
                        p[rb][2 * kb + i / 8][i & 7] = (__bf16)e;
                    }
                l[rb] += sum;
            }
            const bool nan = lds.nan[t % 3] != 0;
#pragma unroll
            for (int db = 0; db < DB; ++db) {
                const int d = db * 32 + col;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    bf16x8_t vf = *reinterpret_cast<const bf16x8_t*>(lds.v[buf] + d * kTile + 8 * v_piece(d, 2 * x + half));
                    if (nan) {
                        const bf16x8_t where = take_nan(vf);
#pragma unroll
                        for (int rb = 0; rb < RB; ++rb) {
                            bf16x8_t seen;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int key = t0 + 16 * x + 8 * (i / 4) + 4 * half + (i & 3);
                                seen[i] = key >= lo[rb] && key < hi[rb] ? (__bf16)1.0f : (__bf16)0.0f;
                            }
                            f32x16_t n;
#pragma unroll
                            for (int i = 0; i < 16; ++i) n[i] = 0.0f;
                            n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(where, seen, n, 0, 0, 0);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (n[i] > 0.0f) o[rb][db][i] = __builtin_nanf("");
                        }
                    }
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb)
                        o[rb][db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, p[rb][x], o[rb][db], 0, 0, 0);
                }
            }
        }
        if (t + 1 < tiles) store_tile(t + 1);
        __syncthreads();
    }

#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int row = row0 + (wave * RB + rb) * 32 + col;
        const float total = l[rb] + __shfl_xor(l[rb], 32);
        if (row >= rows) continue;
        const int i = row / G, h = head * G + row % G;
        const bool none = hi[rb] <= lo[rb];
        const int64_t at = ((int64_t)(s.t0 + i) * a.n_q + h) * a.max_chunks + chunk;
        if (keys.chunks > 1 && half == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(m[rb], total);
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = db * 32 + 8 * j + 4 * half;
                const float4 v = make_float4(o[rb][db][4 * j], o[rb][db][4 * j + 1], o[rb][db][4 * j + 2], o[rb][db][4 * j + 3]);
                if (keys.chunks == 1) store_part<true>(a, s.t0 + i, h, d, D, v, total, m[rb], none);
                else *reinterpret_cast<float4*>(a.part_o + at * D + d) = v;
            }
    }
}

template <int D, int NW, int RB>
hipError_t launch(const AttnCall& a, hipStream_t s) {
    constexpr size_t bytes = sizeof(TileLds<D, NW, RB>);
    static_assert(bytes <= 160 * 1024, "LDS");
    const int64_t grid = (int64_t)a.n_kv * a.tile_slots * a.tile_chunks;
    if (grid >= (int64_t)1 << 31) return hipErrorInvalidConfiguration;
    if (bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_attn_tiles<D, NW, RB>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != hipSuccess) return e;
    }
    k_attn_tiles<D, NW, RB><<<(unsigned)grid, NW * kWave, bytes, s>>>(a);
    return hipGetLastError();
}

}  // namespace

// a.tile_rows = attn_tile_rows(head_dim)
hipError_t launch_attn_tiles(const AttnCall& a, int head_dim, hipStream_t s) {
    switch (head_dim) {
        case 64: return launch<64, 8, 1>(a, s);
        case 128: return launch<128, 8, 1>(a, s);
        default: return launch<256, 4, 1>(a, s);
    }
}

}  // namespace rdg
