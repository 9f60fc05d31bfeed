// Attention over the 8-bit paged cache, many query rows per request: prefill and
// prefill chunks in bf16.  The same mathematics as attn_rows.h (one
// pass, running maximum and sum in fp32); here the work is matrix products,
// 4 * head_dim flops per (query row, key), bound by the bf16 matrix rate and by
// the exponentials beside it.
//
// A workgroup takes 32 rows per wave of one key head -- rows are (query, head of the
// group), so grouped heads share the tile -- and walks its keys in 64-key tiles.
// The tile's codes become bf16 once for all waves, on their way into LDS: K
// by rows, V by columns, with each 16-key step's keys in the order in which S^T =
// K Q^T (v_mfma_f32_32x32x16_bf16) leaves them in a lane, so that the
// probabilities go from its result registers into O^T = V^T P^T's operand with
// no exchange.  A row is a lane of the result: maximum and sum over keys are
// in-lane but for one swap of the wave's halves, and rescaling O^T is one
// factor per lane.  16-byte pieces are swizzled by row, so that 16 lanes' reads fall
// into the 64 different banks.
//
// A step interleaves, in program order, the exponentials of tile t with the
// products of S(t + 1), and then the products of O(t) with the conversion of K(t + 2)
// and V(t + 1): the matrix and vector units overlap within a wave, and one
// barrier a step suffices.  Loads from the cache run one step further ahead and
// stay in flight across it.  Workgroup b works on key head b % n_kv, so with 8 heads
// each XCD's L2 holds the keys of one; row tiles run from a request's last to
// its first, longest work first.
//
// Measured (784 GFLOP: two causal prompts of 6045 and 7691 tokens, 32 / 8 heads of 128):
// 800 us (785 to 850 with the card's clocks), 1.0 PFLOP/s, 0.6 of what a large bf16
// library product reaches on the card.  The matrix units are busy 49% of the time and the vector units 48% (of a
// tile's 200 vector instructions per lane, 32 are exponentials), both at once
// 18%: what is left is mostly issue and LDS latency at two waves a SIMD.
// Without the interleaving it took 1174 us; halves of the workgroup in
// opposite phases with two barriers a step 833, two 128-row workgroups per
// CU 852.
// Registers: the eight-wave form of width 128 takes all 256 of a lane, the four-wave one
// and the mixed launch spill 36 bytes a lane besides.  Width 256 takes 256 and
// 255 accumulator registers at one wave a SIMD: a prompt of 3400 tokens, 64 / 4 heads, 379
// GFLOP in 548 us, 0.7 PFLOP/s.
#include <type_traits>

#include "attn_rows.h"

namespace rdg {
namespace {

constexpr int kTile = 64;

template <int D>
struct TileLds {
    uint16_t k[2][kTile * D];
    uint16_t v[2][D * kTile];
    int nan;  // whether a masked tile's V held NaN
};

// Barrier for LDS alone: loads from memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    __builtin_amdgcn_sched_barrier(0);
}

// Swizzles: the 16-byte piece that holds piece c of a K row / of a V^T row.
template <int D>
__device__ __forceinline__ int k_piece(int key, int c) {
    return c ^ (D == 64 ? (key >> 1) & 7 : key & 15);
}
__device__ __forceinline__ int v_piece(int d, int c) { return c ^ (((d >> 1) & 7) ^ ((d >> 4) & 1)); }

// Workgroup `id` of NW waves.
template <int D, int NW>
__device__ __forceinline__ void attn_tiles(const AttnCall& a, int id, TileLds<D>& lds) {
    // One 32-row block a wave.  Two halve the LDS reads per product, but at one wave a
    // SIMD (512 registers) the copies between the register files ate that: the prompts
    // above took 965 us so, 815 then with eight waves of one block each.
    constexpr int NT = NW * kWave, BM = 32 * NW;
    constexpr int KS = D / 16, DB = D / 32;  // reduction steps of S^T, 32-row blocks of O^T
    // Staging, per thread: KU pieces of 16 K codes, VU of 8 keys x 4 columns of V.
    constexpr int KP = kTile * D / 16, VP = 8 * D / 4;
    constexpr int KU = (KP + NT - 1) / NT, VU = (VP + NT - 1) / NT;
    const int tid = (int)threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int col = lane & 31, half = lane >> 5;
    const int head = id % a.n_kv;
    id /= a.n_kv;
    const int slot = a.tile_slots - 1 - id % a.tile_slots, chunk = id / a.tile_slots;
    const int r = request_of_place(a, slot, BM);
    if (r < 0) return;
    const ReqSpan s = req_span(a, r);
    const int G = a.group, rows = s.n * G;
    const int row0 = (slot - first_place(a, s, r, BM)) * BM;
    if (s.n <= a.n_most || row0 < 0 || row0 >= rows) return;
    const int row1 = row0 + BM < rows ? row0 + BM : rows;
    const TileKeys keys = tile_keys(a, s, row0, row1, a.tile_chunk);
    if (chunk >= keys.chunks) return;
    const int any_lo = key_lo(a, s, row0 / G), any_hi = keys.end;
    const int wg_all_lo = key_lo(a, s, (row1 - 1) / G), wg_all_hi = key_hi(a, s, row0 / G);
    const int k0 = keys.begin + chunk * a.tile_chunk;
    const int k1 = any_hi < k0 + a.tile_chunk ? any_hi : k0 + a.tile_chunk;
    const int tiles = k1 > k0 ? (k1 - k0 + kTile - 1) / kTile : 0;

    // this wave's rows: a block of 32, one per lane of either half
    int lo, hi, all_lo, all_hi;
    bf16x8_t q[KS];
    {
        const int first = row0 + wave * 32, row = first + col;
        const int i = (row < rows ? row : rows - 1) / G, h = head * G + (row < rows ? row : rows - 1) % G;
        lo = key_lo(a, s, i);
        hi = key_hi(a, s, i);
        all_lo = key_lo(a, s, (first + 31 < rows ? first + 31 : rows - 1) / G);
        all_hi = key_hi(a, s, (first < rows ? first : rows - 1) / G);
        const uint16_t* p = static_cast<const uint16_t*>(a.q) + (int64_t)(s.t0 + i) * a.q_stride + (int64_t)h * D + 8 * half;
#pragma unroll
        for (int x = 0; x < KS; ++x) q[x] = *reinterpret_cast<const bf16x8_t*>(p + 16 * x);
    }

    // pages and scales of 16-key groups: lane l holds group 64 b + l of this chunk
    int page = 0;
    float ks = 1.0f, vs = 1.0f;
    const auto load_pages = [&](int b) {
        const int key = k0 + (b * kWave + lane) * 16;
        page = 0;  // past the last key: page 0, whose codes are not used
        ks = vs = 1.0f;
        if (key < k1) {
            page = page_of(a, r, key);
            ks = pow2_scale(a.k_scale[(int64_t)page * a.n_kv + head]);
            vs = pow2_scale(a.v_scale[(int64_t)page * a.n_kv + head]);
        }
    };
    const int in_page = (1 << a.page_shift) - 1;
    const auto row_at = [&](const uint8_t* codes, int g, int key) -> const uint8_t* {
        const int pg = __shfl(page, g & (kWave - 1));
        return codes + ((((int64_t)pg * a.n_kv + head) << a.page_shift) + (key & in_page)) * D;
    };
    uint4 kraw[2][KU];  // the second set for the first tile only
    uint32_t vraw[2][VU][8];
    float vscale[2][VU];
    // Loads of one step: V of tile t - 1, then K of tile t, whose pages may be the next set.
    const auto fetch = [&](int t, auto set) {
        constexpr int F = decltype(set)::value;
#pragma unroll
        for (int u = 0; u < VU; ++u) {
            const int x = tid + u * NT, c = (x / (D / 4)) & 7, dq = x % (D / 4), g = (t - 1) * 4 + c / 2;
            vscale[F][u] = __shfl(vs, g & (kWave - 1));
            const uint8_t* p = row_at(a.v_codes, g, k0 + (t - 1) * kTile + 16 * (c / 2) + 4 * (c & 1)) + 4 * dq;
#pragma unroll
            for (int i = 0; i < 8; ++i) vraw[F][u][i] = *reinterpret_cast<const uint32_t*>(p + (8 * (i / 4) + (i & 3)) * D);
        }
        if ((t & 15) == 0) load_pages(t / 16);
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            const int x = tid + u * NT, key = (x / (D / 16)) & (kTile - 1), c = x % (D / 16), g = t * 4 + key / 16;
            kraw[F][u] = *reinterpret_cast<const uint4*>(row_at(a.k_codes, g, k0 + t * kTile + key) + 16 * c);
        }
    };
    // V codes of tile t before their conversion: keys that no row sees may hold
    // anything, and a NaN that only some see is kept out of the product.
    const auto clean = [&](int t, auto set) {
        constexpr int F = decltype(set)::value;
        const int t0 = k0 + t * kTile;
        if (t0 >= wg_all_lo && t0 + kTile <= wg_all_hi) return;
        uint32_t saw = 0;
#pragma unroll
        for (int u = 0; u < VU; ++u) {
            const int x = tid + u * NT, c = (x / (D / 4)) & 7, key = t0 + 16 * (c / 2) + 4 * (c & 1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = key + 8 * (i / 4) + (i & 3);
                if (j < any_lo || j >= any_hi) vraw[F][u][i] = 0;
                const uint32_t nan = nan_bytes(vraw[F][u][i]);
                vraw[F][u][i] = without_nan(vraw[F][u][i], nan);
                saw |= nan;
            }
        }
        if (saw) lds.nan = 1;
    };
    const auto stage_k = [&](uint16_t* to_k, int t, int u, auto set) {  // unit u of tile t, whose pages are the ones held
        constexpr int F = decltype(set)::value;
        const int x = tid + u * NT, key = (x / (D / 16)) & (kTile - 1), c = x % (D / 16);
        const float scale = __shfl(ks, (t * 4 + key / 16) & (kWave - 1));
        if (KP % NT == 0 || x < KP) {
            uint16_t* row = to_k + key * D;
            *reinterpret_cast<bf16x8_t*>(row + 8 * k_piece<D>(key, 2 * c)) =
                codes_to_bf16(kraw[F][u].x, kraw[F][u].y, scale, scale);
            *reinterpret_cast<bf16x8_t*>(row + 8 * k_piece<D>(key, 2 * c + 1)) =
                codes_to_bf16(kraw[F][u].z, kraw[F][u].w, scale, scale);
        }
    };
    const auto stage_v = [&](uint16_t* to_v, int u, auto set) {
        constexpr int F = decltype(set)::value;
        const int x = tid + u * NT, c = (x / (D / 4)) & 7, dq = x % (D / 4);
        const uint32_t in0[4] = {vraw[F][u][0], vraw[F][u][1], vraw[F][u][2], vraw[F][u][3]};
        const uint32_t in1[4] = {vraw[F][u][4], vraw[F][u][5], vraw[F][u][6], vraw[F][u][7]};
        uint32_t x0[4], x1[4];
        transpose4(in0, x0);
        transpose4(in1, x1);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int d = 4 * dq + b;
            if (VP % NT == 0 || x < VP)
                *reinterpret_cast<bf16x8_t*>(to_v + d * kTile + 8 * v_piece(d, c)) =
                    codes_to_bf16(x0[b], x1[b], vscale[F][u], vscale[F][u]);
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
    // bits of a piece's number, so a few places and offsets give them all.
    constexpr int KA = D == 64 ? 4 : 8;
    int k_at[KA], v_at[4];
#pragma unroll
    for (int x = 0; x < KA; ++x) k_at[x] = col * D + 8 * k_piece<D>(col, 2 * x + half);
#pragma unroll
    for (int x = 0; x < 4; ++x) v_at[x] = col * kTile + 8 * v_piece(col, 2 * x + half);
    // operand y of the logits of keys 32 kb .., operand x of output block db
    const auto k_frag = [&](const uint16_t* k, int kb, int y) {
        return *reinterpret_cast<const bf16x8_t*>(k + k_at[y % KA] + kb * 32 * D + (y / KA) * KA * 16);
    };
    const auto v_frag = [&](const uint16_t* v, int db, int x) {
        return *reinterpret_cast<const bf16x8_t*>(v + v_at[x] + db * 32 * kTile);
    };
    // A tile's logits: what the mask hides, then the largest of each row.
    const auto mask = [&](f32x16_t (&sc)[2], int t) {
        const int t0 = k0 + t * kTile;
        if (t0 >= all_lo && t0 + kTile <= all_hi) return;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int key = t0 + kb * 32 + 8 * (i / 4) + 4 * half + (i & 3);
                if (key < lo || key >= hi) sc[kb][i] = -__builtin_inff();
            }
    };
    const auto row_top = [&](f32x16_t (&sc)[2]) {
        float top = -__builtin_inff();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[kb][i]);
        return max_halves(top) * scale;
    };
    const auto raise = [&](float top) {
        if (__any(top > m + kSlack)) {
            const float m_new = fmaxf(m, top);
            const float shrink = __builtin_amdgcn_exp2f(m - (m_new == -__builtin_inff() ? 0.0f : m_new));
            l *= shrink;
#pragma unroll
            for (int db = 0; db < DB; ++db) o[db] *= shrink;
            m = m_new;
        }
    };
    // One tile: its probabilities beside the next tile's logits; then its V product
    // beside the next maximum and the staging of K(t + 2) and V(t + 1).
    const auto tile = [&](f32x16_t (&sc)[2], f32x16_t (&next)[2], int t, auto parity) {
        constexpr int B = decltype(parity)::value;
        constexpr int KG = KS / 4;
        const std::integral_constant<int, 0> set0;
        const uint16_t *k_next = lds.k[1 - B], *v_now = lds.v[B];
        bf16x8_t p[4];
        float sum = 0.0f;
        const float ref = m == -__builtin_inff() ? 0.0f : m;
        __builtin_amdgcn_s_setprio(1);
        // Nine steps: the products of group g - 1, with their operands read two
        // steps before, beside the exponentials of group g.
        bf16x8_t kf[3][KG], vf[4][2];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int x = 0; x < KG; ++x) kf[g][x] = k_frag(k_next, 0, g * KG + x);
#pragma unroll
        for (int g = 0; g < 9; ++g) {
            __builtin_amdgcn_sched_barrier(0);
            if (g > 0) {
                const int w = g - 1, kb = w / 4;
                if (g + 1 < 8) {
#pragma unroll
                    for (int x = 0; x < KG; ++x) kf[(g + 1) % 3][x] = k_frag(k_next, (g + 1) / 4, ((g + 1) & 3) * KG + x);
                } else {
                    vf[g - 7][0] = v_frag(v_now, 0, 2 * (g - 7));
                    vf[g - 7][1] = v_frag(v_now, 0, 2 * (g - 7) + 1);
                }
                // past the last tile: of an old buffer, not used
                if ((w & 3) == 0)
#pragma unroll
                    for (int i = 0; i < 16; ++i) next[kb][i] = 0.0f;
#pragma unroll
                for (int x = 0; x < KG; ++x)
                    next[kb] =
                        __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[w % 3][x], q[(w & 3) * KG + x], next[kb], 0, 0, 0);
            }
            if (g < 8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f(fmaf(sc[g / 4][4 * (g & 3) + i], scale, -ref));
                    sum += e;
                    p[g / 2][4 * (g & 1) + i] = (__bf16)e;
                }
                // summed here and not behind the loop, where all the exponentials would have to be kept
                asm volatile("" : "+v"(sum));
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        l += sum;
        if (t + 1 < tiles) {
            mask(next, t + 1);
            clean(t + 1, set0);
        }
        __builtin_amdgcn_s_setprio(0);
        float top;
        constexpr int G2 = 2 * DB;
#pragma unroll
        for (int g = 0; g < G2; ++g) {
            __builtin_amdgcn_sched_barrier(0);
            if (g + 2 < G2) {
                vf[(g + 2) & 3][0] = v_frag(v_now, (g + 2) / 2, 2 * (g & 1));
                vf[(g + 2) & 3][1] = v_frag(v_now, (g + 2) / 2, 2 * (g & 1) + 1);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
                o[g / 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[g & 3][x], p[2 * (g & 1) + x], o[g / 2], 0, 0, 0);
            // staged past the last tile: never read
#pragma unroll
            for (int u = 0; u < VU; ++u)
                if (g == u % G2) stage_v(lds.v[1 - B], u, set0);
#pragma unroll
            for (int u = 0; u < KU; ++u)
                if (g == (1 + u) % G2) stage_k(lds.k[B], t + 2, u, set0);
            if (g == G2 - 1) top = row_top(next);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (t + 1 < tiles) raise(top);
        fetch(t + 3, set0);
        lds_barrier();
    };

    if (tid == 0) lds.nan = 0;
    __syncthreads();
    if (tiles > 0) {
        f32x16_t s0[2], s1[2];
        const std::integral_constant<int, 0> even;
        const std::integral_constant<int, 1> odd;
        fetch(0, odd);
        fetch(1, even);
        clean(0, even);
#pragma unroll
        for (int u = 0; u < KU; ++u) stage_k(lds.k[0], 0, u, odd);
#pragma unroll
        for (int u = 0; u < KU; ++u) stage_k(lds.k[1], 1, u, even);
#pragma unroll
        for (int u = 0; u < VU; ++u) stage_v(lds.v[0], u, even);
        fetch(2, even);
        lds_barrier();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s0[kb][i] = 0.0f;
#pragma unroll
            for (int y = 0; y < KS; ++y) {
                const bf16x8_t f = k_frag(lds.k[0], kb, y);
                s0[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, q[y], s0[kb], 0, 0, 0);
            }
        }
        mask(s0, 0);
        raise(row_top(s0));
        lds_barrier();  // the first tile's K buffer takes the third tile
        for (int t = 0;;) {
            tile(s0, s1, t, even);
            if (++t >= tiles) break;
            tile(s1, s0, t, odd);
            if (++t >= tiles) break;
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
                        if ((p[db * 32 + 8 * (i / 4) + 4 * half + (i & 3)] & 0x7f) == 0x7f)
                            o[db][i] = __builtin_nanf("");
            }
        }
    }

    const int row = row0 + wave * 32 + col;
    const float total = sum_halves(l);
    if (row >= rows) return;
    const int i = row / G, h = head * G + row % G;
    const bool none = hi <= lo;
    const int64_t at = ((int64_t)(s.t0 + i) * a.n_q + h) * a.tile_chunks + chunk;
    if (keys.chunks > 1 && half == 0) *reinterpret_cast<float2*>(a.tile_ml + 2 * at) = make_float2(m, total);
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = db * 32 + 8 * j + 4 * half;
            const float4 v = make_float4(o[db][4 * j], o[db][4 * j + 1], o[db][4 * j + 2], o[db][4 * j + 3]);
            if (keys.chunks == 1) store_part<true>(a, s.t0 + i, h, d, D, v, total, m, none);
            else *reinterpret_cast<float4*>(a.tile_o + at * D + d) = v;
        }
}

template <int D, int NW>
__global__ __launch_bounds__(NW * kWave, NW == 4 && D < 256 ? 2 : 1) void k_attn_tiles(AttnCall a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    attn_tiles<D, NW>(a, (int)blockIdx.x, *reinterpret_cast<TileLds<D>*>(lds_raw));
}

// A mixed batch in one launch: the long requests' tiles, then the short ones'
// rows, which fill the CUs beside them (one after the other they took 28 + 9 us
// of a window-1024 batch of 24 chunks and decode rows).
template <int D>
__global__ __launch_bounds__(4 * kWave, D < 256 ? 2 : 1) void k_attn_mixed(AttnCall a, int tile_blocks) {
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    const int id = (int)blockIdx.x;
    if (id < tile_blocks) attn_tiles<D, 4>(a, id, *reinterpret_cast<TileLds<D>*>(lds_raw));
    else attn_rows<D, 1, 4>(a, id - tile_blocks, *reinterpret_cast<RowsLds<D, 4>*>(lds_raw));
}

int64_t tile_blocks(const AttnCall& a) { return (int64_t)a.n_kv * a.tile_slots * a.tile_chunks; }

template <int D, int NW>
hipError_t launch(const AttnCall& a, hipStream_t s) {
    static_assert(sizeof(TileLds<D>) <= 160 * 1024, "LDS");
    const int64_t grid = tile_blocks(a);
    if (!grid_fits(grid, NW * kWave)) return hipErrorInvalidConfiguration;
    k_attn_tiles<D, NW><<<(unsigned)grid, NW * kWave, sizeof(TileLds<D>), s>>>(a);
    return hipGetLastError();
}

template <int D>
hipError_t launch_mixed(const AttnCall& a, hipStream_t s) {
    constexpr size_t bytes = sizeof(TileLds<D>) > sizeof(RowsLds<D, 4>) ? sizeof(TileLds<D>) : sizeof(RowsLds<D, 4>);
    const int64_t tiles = tile_blocks(a), grid = tiles + (int64_t)a.n_kv * row_tiles(a) * a.row_chunks;
    if (!grid_fits(grid, 4 * kWave)) return hipErrorInvalidConfiguration;
    k_attn_mixed<D><<<(unsigned)grid, 4 * kWave, bytes, s>>>(a, (int)tiles);
    return hipGetLastError();
}

template <int D>
hipError_t launch_d(const AttnCall& a, hipStream_t s) {
    if (a.n_most > 0) return launch_mixed<D>(a, s);
    if constexpr (D < 256) {
        if (a.tile_rows == 256) return launch<D, 8>(a, s);
    }
    return launch<D, 4>(a, s);
}

}  // namespace

// With short requests too (n_most > 0): 128-row tiles and 64-row workgroups.
hipError_t launch_attn_tiles(const AttnCall& a, int head_dim, hipStream_t s) {
    switch (head_dim) {
        case 64: return launch_d<64>(a, s);
        case 128: return launch_d<128>(a, s);
        default: return launch_d<256>(a, s);
    }
}

}  // namespace rdg
