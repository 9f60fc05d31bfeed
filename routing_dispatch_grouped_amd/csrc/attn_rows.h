// Attention over the 8-bit paged cache, few query rows per request: decode,
// drafted tokens, fp32 queries.
//
//   o_i = sum_j softmax_j(scale * q_i . k_j) v_j     lse_i = log sum_j exp(scale * q_i . k_j)
//
// over the keys that query i sees, in one pass with a running maximum and sum
// (fp32, base-2 exponents).  Bound by HBM: every code is read once, 2 * head_dim
// bytes per key and key head, and the G = n_q / n_kv query heads of a key head
// share the read: the rows of a tile are (query token, head of the group).
//
// A wave computes
//   S^T = K Q^T   16 keys x 16 rows per v_mfma_f32_16x16x32_bf16
//   O^T = V^T P^T 16 columns x 16 rows, 32 keys per MFMA
// The order of the reduction index is free, so a lane's 16 consecutive K codes
// serve two MFMA steps, and the keys that S^T leaves in a lane (4 of each 16)
// are the ones that its P^T operand holds, with V's 4-byte columns transposed by
// byte permutes to match: probabilities never leave their lane.  The codes
// become bf16 exactly, times their page's power of two
// (v_cvt_scalef32_pk_bf16_fp8).  fp32 queries and probabilities go in as three
// bf16 parts each, which carries 24 bits.
//
// A workgroup's waves are RT row tiles x KG key groups (4 x 1, 3 x 1, 2 x 2 or 1 x
// 4): the key groups take the step_keys blocks of one chunk of one request's
// keys in turn and join in LDS; a key group's row tiles share its loads.
// Codes come in as contiguous KiB per instruction (16-key groups of a page
// lie together), one step ahead in registers -- 16 KB a wave at head_dim 128 --
// and pass to their operand lanes through LDS.  With operand-shaped loads straight into the
// registers, 16 rows x 64 bytes an instruction, for each row tile by itself, 35 rows a
// request cost the L1 8.1 million accesses, now 1.4; 16 requests of 64 rows took 53 us, with
// one set of such loads for all row tiles 46, now 41; the decode batch below 272, now 265.
// Four row tiles in one wave's registers spilled: 50 us for 35 rows a request, 39 so.
// Chunks of one row are joined by a second launch, in chunk order, so results
// do not depend on scheduling.  (The last workgroup to finish joining them itself,
// by a counter: 10.3 against 10.5 us for one request, 48 against 40 where 35
// rows have 10 parts.)
//
// Measured, head_dim 128: 128 requests of 1000 to 16384 tokens, 64 / 8 heads: 265 us, 5.2
// TB/s of codes (reads alone reach 6.4 on the card, non-temporal ones 7.2), of 1000 to 131000 5.6; one request of
// 2500 tokens: 7.5 us and 4 for the join, all latency.  fp32, whose three parts a side make
// three products of one: four prompts of 2048, 32 / 8 heads, 456 us, 0.9 PFLOP/s of bf16
// products, 0.56 of what a large library one reaches.
#pragma once
#include "attn.h"

namespace rdg {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// Keys per wave and step: 64, or 32 of wide heads, whose codes in flight would
// else take 128 registers.
template <int D>
constexpr int step_keys() {
    return D == 256 ? 32 : 64;
}

template <int D>
struct VWords {
    static constexpr int n = D / 64;  // dwords of V per key and lane (D / 16 codes)
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x, w[1] = u.y;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    }
}

// x as NS bf16 parts that sum to it (NS = 1: x rounded).
template <int NS>
__device__ __forceinline__ void split_bf16(float x, __bf16 (&part)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        part[i] = (__bf16)x;
        if (i + 1 < NS) x -= (float)part[i];
    }
}

// NS = 1: bf16 queries and output; 3: fp32.  RT: 16-row tiles per workgroup.
template <int RT>
constexpr int key_groups() {
    return RT == 1 ? 4 : RT == 2 ? 2 : 1;
}

template <int D, int RT>
struct RowsLds {
    // the codes of a step (RT > 1: of two) of each key group; then the parts to be joined
    static constexpr int KG = key_groups<RT>();
    static constexpr int kCodes = KG * (RT > 1 ? 2 : 1) * 2 * step_keys<D>() * D, kParts = RT * KG * 16 * (D + 4) * 4;
    uint8_t raw[kCodes > kParts ? kCodes : kParts];
    float m[RT][KG][16], l[RT][KG][16];
};

// Workgroup `id` of RT * key_groups<RT>() waves.
template <int D, int NS, int RT>
__device__ __forceinline__ void attn_rows(const AttnCall& a, int id, RowsLds<D, RT>& lds) {
    constexpr int KJ = D / 64, W = VWords<D>::n, U = D / 16;
    constexpr int KG = key_groups<RT>(), kBlock = step_keys<D>(), GP = kBlock / 16;  // 16-key groups of a step
    auto& lds_raw = lds.raw;
    auto& lds_m = lds.m;
    auto& lds_l = lds.l;
    auto& lds_o = *reinterpret_cast<float(*)[RT][KG][16][D + 4]>(lds_raw);
    const int lane = lane_id(), w_id = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int rt = w_id / KG, wave = w_id % KG;  // row tile, key group
    const int col = lane & 15, g4 = lane >> 4;
    const int head = id % a.n_kv;
    id /= a.n_kv;
    // bf16 requests have one tile at most here; tiles of longer fp32 ones go by place
    int r, chunk, place = 0;
    if (NS > 1 && a.row_places > 0) {
        place = id % a.row_places;
        chunk = id / a.row_places;
        r = request_of_place(a, place, 16 * RT);
        if (r < 0) return;
    } else {
        r = id % a.R;
        chunk = id / a.R;
    }
    const ReqSpan s = req_span(a, r);
    const int G = a.group, rows = s.n * G;
    const int first = NS > 1 && a.row_places > 0 ? (place - first_place(a, s, r, 16 * RT)) * 16 * RT : 0;
    if (first < 0 || first >= rows || s.n > a.n_most) return;
    const int last = first + 16 * RT < rows ? first + 16 * RT - 1 : rows - 1;
    const TileKeys keys = tile_keys(a, s, first, last + 1, a.chunk);
    const int chunks = keys.chunks;
    if (chunk >= chunks) return;
    const int k0 = keys.begin + chunk * a.chunk;
    // this wave's rows (none: those of the last row, not stored), keys that every one
    // of them sees, and that any does
    const int row0 = first + rt * 16;
    const int i_first = (row0 < rows ? row0 : rows - 1) / G, i_last = (row0 + 15 < rows ? row0 + 15 : rows - 1) / G;
    const int all_lo = key_lo(a, s, i_last), all_hi = key_hi(a, s, i_first);
    const int any_lo = key_lo(a, s, i_first), any_hi = key_hi(a, s, i_last);
    // one row tile: this wave's last key; more: the workgroup's, whose waves step together
    const int end = RT > 1 ? keys.end : any_hi;
    const int k1 = end < k0 + a.chunk ? end : k0 + a.chunk;

    // queries: lane (row col, reduction group g4)
    bf16x8_t q[2 * KJ][NS];
    int hi, lo;
    {
        const int row = row0 + col;
        const bool live = row < rows;
        const int i = live ? row / G : 0, h = head * G + (live ? row % G : 0);
        hi = key_hi(a, s, live ? i : i_last);
        lo = key_lo(a, s, live ? i : i_last);
        const int64_t at = (int64_t)(s.t0 + i) * a.q_stride + (int64_t)h * D + 16 * g4;
#pragma unroll
        for (int j = 0; j < KJ; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if constexpr (NS == 1) {
                    bf16x8_t v = *reinterpret_cast<const bf16x8_t*>(static_cast<const uint16_t*>(a.q) + at + 64 * j + 8 * e);
                    q[2 * j + e][0] = v;
                } else {
                    const float* f = static_cast<const float*>(a.q) + at + 64 * j + 8 * e;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        __bf16 part[NS];
                        split_bf16<NS>(f[c], part);
#pragma unroll
                        for (int n = 0; n < NS; ++n) q[2 * j + e][n][c] = part[n];
                    }
                }
            }
    }

    // page and scales of this wave's 16-key groups, one per lane: those of kHeld steps (1024 keys) from `step` on
    constexpr int kHeld = kWave / GP;
    int my_page = 0;
    float my_ks = 1.0f, my_vs = 1.0f;
    const auto load_pages = [&](int step) {
        const int key = k0 + ((step + lane / GP) * KG + wave) * kBlock + lane % GP * 16;
        my_page = 0;
        my_ks = my_vs = 1.0f;
        if (key < k1) {
            my_page = page_of(a, r, key);
            my_ks = pow2_scale(a.k_scale[(int64_t)my_page * a.n_kv + head]);
            my_vs = pow2_scale(a.v_scale[(int64_t)my_page * a.n_kv + head]);
        }
    };

    f32x4_t o[U];
    float m = -__builtin_inff(), l = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) o[u] = f32x4_t{0, 0, 0, 0};

    // The key group's waves share the loads -- 16-key groups are contiguous, so
    // each instruction reads a KiB in a row -- and pass the codes on through LDS;
    // K's 16-byte pieces are swizzled by row and V's rows interleaved, so that
    // the operands' reads fall into different banks.
    constexpr int PK = kBlock * D / 16, ST = RT * kWave, NP = (2 * PK + ST - 1) / ST;
    constexpr int kBufs = RT > 1 ? 2 : 1;  // a wave on its own reads what it wrote in order
    const int in_page = (1 << a.page_shift) - 1;
    uint4 kreg[GP][KJ];
    uint32_t vreg[GP][4][W];
    u32x4_t stg[NP];
    uint8_t* const lds_codes = lds_raw + wave * (kBufs * 2 * kBlock * D);
    const auto k_place = [&](int key, int piece) {
        const int turn = D == 64 ? (key >> 2) & 3 : D == 128 ? (key >> 1) & 7 : key & 15;
        return key * D + 16 * (piece ^ turn);
    };
    const auto v_row = [&](int key) { return (key & ~15) | ((key & 3) << 2) | ((key >> 2) & 3); };
    const auto fetch = [&](int step, int held) {  // held: the step's first group among those held
        const int kb = k0 + (step * KG + wave) * kBlock;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int u = rt * kWave + p * ST;  // of the wave's first lane: one 16-key group for all
            if (2 * PK % ST == 0 || u < 2 * PK) {
                const int y = u % PK, g = y / D, page = __builtin_amdgcn_readlane(my_page, held + g);
                const uint8_t* from = (u < PK ? a.k_codes : a.v_codes) +
                    ((((int64_t)page * a.n_kv + head) << a.page_shift) + ((kb + 16 * g) & in_page)) * D + y % D * 16;
                stg[p] = *reinterpret_cast<const u32x4_t*>(from + 16 * lane);
                __builtin_amdgcn_sched_barrier(0x38f);  // loads in the order of their use: the waits then go one by one
            }
        }
    };
    const auto pass_on = [&](int step) {
        uint8_t* buf = lds_codes + step % kBufs * (2 * kBlock * D);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int u = rt * kWave + p * ST, y = u % PK + lane, key = y / (D / 16), piece = y % (D / 16);
            if (2 * PK % ST == 0 || u < 2 * PK)
                *reinterpret_cast<u32x4_t*>(buf + (u < PK ? k_place(key, piece) : kBlock * D + v_row(key) * D + 16 * piece)) =
                    stg[p];
        }
    };
    const auto take_k = [&](int step) {
        const uint8_t* buf = lds_codes + step % kBufs * (2 * kBlock * D);
#pragma unroll
        for (int t = 0; t < GP; ++t)
#pragma unroll
            for (int j = 0; j < KJ; ++j)
                kreg[t][j] = *reinterpret_cast<const uint4*>(buf + k_place(16 * t + col, 4 * j + g4));
    };
    const auto take_v = [&](int step) {
        const uint8_t* buf = lds_codes + step % kBufs * (2 * kBlock * D) + kBlock * D;
#pragma unroll
        for (int t = 0; t < GP; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load_words<W>(buf + v_row(16 * t + 4 * g4 + i) * D + col * (D / 16), vreg[t][i]);
    };

    const int span = k1 - k0 - (RT > 1 ? 0 : wave * kBlock);
    const int steps = span > 0 ? (span + KG * kBlock - 1) / (KG * kBlock) : 0;
    const float c = a.scale_log2;
    uint32_t saw_nan = 0;
    // kHeld steps at a time.  The loads do not run ahead from one such run into the next: holding two
    // sets of pages for that takes registers that four row tiles of 128 do not have at three waves a SIMD.
    for (int s0 = 0, s1; s0 < steps; s0 = s1) {
        s1 = s0 + kHeld < steps ? s0 + kHeld : steps;
        load_pages(s0);
        fetch(s0, 0);
        if constexpr (RT > 1) {
            pass_on(s0);
            if (s0 + 1 < s1) fetch(s0 + 1, GP);
            __syncthreads();
        }
        for (int step = s0; step < s1; ++step) {
            const int kb = k0 + (step * KG + wave) * kBlock, held = (step - s0) * GP;
            if constexpr (RT == 1) {
                pass_on(step);
                if (step + 1 < s1) fetch(step + 1, held + GP);
            }
            take_k(step);
            f32x4_t sc[GP];
#pragma unroll
            for (int t = 0; t < GP; ++t) {
                const float ks = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_ks), held + t));
                sc[t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
                    const bf16x8_t k_lo = codes_to_bf16(kreg[t][j].x, kreg[t][j].y, ks, ks);
                    const bf16x8_t k_hi = codes_to_bf16(kreg[t][j].z, kreg[t][j].w, ks, ks);
#pragma unroll
                        for (int n = NS - 1; n >= 0; --n) {  // small parts first
                            sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k_lo, q[2 * j][n], sc[t], 0, 0, 0);
                            sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k_hi, q[2 * j + 1][n], sc[t], 0, 0, 0);
                        }
                }
            }
            take_v(step);
            const bool masked = kb < all_lo || kb + kBlock > all_hi;
            if (masked) {
#pragma unroll
                    for (int t = 0; t < GP; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = kb + 16 * t + 4 * g4 + i;
                            if (key < lo || key >= hi) sc[t][i] = -__builtin_inff();
                        }
                // keys that no row sees may hold anything
#pragma unroll
                for (int t = 0; t < GP; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = kb + 16 * t + 4 * g4 + i;
                        const bool any = key >= any_lo && key < any_hi;
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            vreg[t][i][w] = any ? vreg[t][i][w] : 0;
                            const uint32_t nan = nan_bytes(vreg[t][i][w]);
                            vreg[t][i][w] = without_nan(vreg[t][i][w], nan);
                            saw_nan |= nan;
                        }
                    }
            }
            bf16x8_t p[GP / 2][NS];
            {
                float top = -__builtin_inff();
#pragma unroll
                for (int t = 0; t < GP; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[t][i]);
                top = max_quarters(top);
                const float m_new = fmaxf(m, top * c);
                if (__any(m_new > m + kSlack)) {
                    const float shrink = __builtin_amdgcn_exp2f(m - (m_new == -__builtin_inff() ? 0.0f : m_new));
                    l *= shrink;
#pragma unroll
                    for (int u = 0; u < U; ++u) o[u] *= shrink;
                    m = m_new;
                }
                const float ref = m == -__builtin_inff() ? 0.0f : m;
                float sum = 0.0f;
#pragma unroll
                for (int t = 0; t < GP; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float e = __builtin_amdgcn_exp2f(fmaf(sc[t][i], c, -ref));
                        sum += e;
                        __bf16 part[NS];
                        split_bf16<NS>(e, part);
#pragma unroll
                        for (int n = 0; n < NS; ++n) p[t / 2][n][(t & 1) * 4 + i] = part[n];
                    }
                l += sum;
            }
            // O^T += V^T P^T; column of output tile u in lane col: col * U + u
#pragma unroll
            for (int t2 = 0; t2 < GP / 2; ++t2) {
                const float va = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_vs), held + 2 * t2));
                const float vb = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_vs), held + 2 * t2 + 1));
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    uint32_t in[4], x[4], y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) in[i] = vreg[2 * t2][i][w];
                    transpose4(in, x);
#pragma unroll
                    for (int i = 0; i < 4; ++i) in[i] = vreg[2 * t2 + 1][i][w];
                    transpose4(in, y);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const bf16x8_t v = codes_to_bf16(x[b], y[b], va, vb);
                        const int u = 4 * w + b;
#pragma unroll
                            for (int n = NS - 1; n >= 0; --n)
                                o[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[t2][n], o[u], 0, 0, 0);
                    }
                }
            }
            if constexpr (RT > 1) {
                if (step + 1 < s1) pass_on(step + 1);
                if (step + 2 < s1) fetch(step + 2, held + 2 * GP);
                __syncthreads();
            }
        }
        __builtin_amdgcn_s_waitcnt(0x0f70);  // no load is in flight here: says so, else the next ones wait for the scales
    }

    if (__any(saw_nan != 0)) {
        for (int step = 0; step < steps; ++step) {
            const int kb = k0 + (step * KG + wave) * kBlock;
            if (kb >= all_lo && kb + kBlock <= all_hi) continue;
            for (int j = kb; j < kb + kBlock && j < any_hi; ++j) {
                const int page = page_of(a, r, j);
                const uint8_t* p = a.v_codes +
                    ((((int64_t)page * a.n_kv + head) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * D;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const uint32_t nan = nan_bytes(*reinterpret_cast<const uint32_t*>(p + (4 * g4 + i) * U + 4 * w));
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                if (j >= lo && j < hi && (nan >> (8 * b + 7) & 1))
                                    o[4 * w + b][i] = __builtin_nanf("");
                    }
            }
        }
    }

    const float sum = sum_quarters(l);
    if constexpr (KG == 1) {  // no other wave has a part of these rows: out of the registers
        const int row = row0 + col;
        if (row >= rows) return;
        const int i = row / G, h = head * G + row % G;
        const bool none = key_hi(a, s, i) <= key_lo(a, s, i);
        const int64_t at = row_part(a, s, r, i, h) + chunk;
        if (chunks > 1 && g4 == 0) *reinterpret_cast<float2*>(a.row_ml + 2 * at) = make_float2(m, sum);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int u = 0; u < U; u += 4) {
                const int d = (4 * g4 + x) * U + u;
                const float4 v = make_float4(o[u][x], o[u + 1][x], o[u + 2][x], o[u + 3][x]);
                if (chunks == 1) store_part<NS == 1>(a, s.t0 + i, h, d, D, v, sum, m, none);
                else *reinterpret_cast<float4*>(a.row_o + at * D + d) = v;
            }
        return;
    }
    // the key groups' parts, joined in LDS where their codes were
    __syncthreads();
    if (lane < 16) {
        lds_m[rt][wave][col] = m;
        lds_l[rt][wave][col] = sum;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < U; u += 4)
            *reinterpret_cast<float4*>(&lds_o[rt][wave][col][(4 * g4 + i) * U + u]) =
                make_float4(o[u][i], o[u + 1][i], o[u + 2][i], o[u + 3][i]);
    __syncthreads();
    constexpr int TPR = D / 4;  // threads per row
    for (int x = threadIdx.x; x < 16 * RT * TPR; x += RT * KG * kWave) {
        const int rr = (x / TPR) & 15, ty = x / (16 * TPR), d = (x % TPR) * 4, row = first + x / TPR;
        if (row >= rows) break;
        float top = lds_m[ty][0][rr];
#pragma unroll
        for (int w = 1; w < KG; ++w) top = fmaxf(top, lds_m[ty][w][rr]);
        const float ref = top == -__builtin_inff() ? 0.0f : top;
        float total = 0.0f;
        float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < KG; ++w) {
            const float f = __builtin_amdgcn_exp2f(lds_m[ty][w][rr] - ref);
            total = fmaf(f, lds_l[ty][w][rr], total);
            const float4 v = *reinterpret_cast<const float4*>(&lds_o[ty][w][rr][d]);
            acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
        }
        const int i = row / G, h = head * G + row % G;
        if (chunks == 1) {
            const bool none = key_hi(a, s, i) <= key_lo(a, s, i);
            store_part<NS == 1>(a, s.t0 + i, h, d, D, acc, total, top, none);
        } else {
            const int64_t at = row_part(a, s, r, i, h) + chunk;
            *reinterpret_cast<float4*>(a.row_o + at * D + d) = acc;
            if (d == 0) *reinterpret_cast<float2*>(a.row_ml + 2 * at) = make_float2(top, total);
        }
    }
}

}  // namespace
}  // namespace rdg
