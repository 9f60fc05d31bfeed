// Matrix product with its epilogue for more than a few tokens: a workgroup has a tile of TF features x TT
// tokens and walks over its share of the reduction in stages of 128 bytes of each row.
//
//   acc[f, t] = sum_k W[f, k] x[t, k]    (fp8: sum over blocks of 128 of (sum of the block) * W_scale * x_scale)
//   out = act(acc + bias) + residual, or, with the reduction split, parts that k_linear_join adds in their order
//
// Features are the matrix instruction's rows and tokens its columns, so that a lane's four sums are neighbours in the
// packed weights' order.  WF x WT waves have NF x NTK tiles of 16 x 16 each.
//
// Operands go from memory straight to LDS, into a ring of NB stages: up to NB - 1 stages are under way during the
// products, a few loads at a time between matrix instructions (all at once they would hold up the wave's own).  A packed
// weight tile is in the order of the lanes, so that its reads meet no bank twice; a token's row is 128 bytes, whose 16-byte
// pieces are swapped (piece_slot).  One meeting of the workgroup a stage: behind it the next stage is there for
// all and the oldest place is free.  The loop's body is there twice, without and, for the last NB stages, with tests for
// the end.
//
// Large tiles are bound by the matrix core (256 x 256: bf16 8192 x 7168 x 8192 677 .. 711 us from card to card, 1.4 PFLOP/s, its
// units 72% busy at 1.8 GHz; e8m0 4001 x 18432 x 7168 415 .. 437 us, 2.5 PFLOP/s; fp32 scales 467 .. 493: the sums'
// multiplications are nearly as many cycles as the products), small ones by the lines that a compute unit has under way or by L2 (4096 tokens on 256
// features of K = 7168: 24.4 us, 3.7 million lines from L2, 23 TB/s), with few tokens by memory (linear.hip).
// Tiles lie in bands of four by features on each XCD: 8192 x 7168 x 8192 686 us, with bands of one 792, of two 708, of
// eight 695, of all features 743; 4096 x 18432 x 7168 800, 807, 807, 833 and 921.
//
// Not kept: the 32 x 32 x 16 instruction and raised wave priority around the products (slower), a ring of 6
// stages for 128 x 64 (no gain).
#include <type_traits>
#include <utility>

#include "linear.h"

namespace rdg {
namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// What a kernel does with its operands: bf16; e4m3 with fp32 scales (each partial product of 128
// is scaled into the sum); e4m3 with power-of-two scales (the matrix core applies them); e4m3 with either,
// its products from bf16 operands; fp32.
using Yes = std::true_type;
using No = std::false_type;
enum { kBf16 = 0, kFp8 = 1, kE8m0 = 2, kFp8Wide = 3, kF32 = 4 };

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 (4) bytes a lane from base + off + IMM straight to lds + IMM + 16 (4) * lane (base and lds wave-uniform); with
// TEST where `now` < `end`; with ONCE past the caches.  The compiler does not count these loads: meet() below waits for
// them.  The branch is in the assembly, as the compiler would move matrix instructions past one of its own.  A load into
// LDS comes an instruction behind the write of m0 at the earliest: the branch, or an s_nop.
#define RDG_M0 "s_mov_b32 m0, %2\n\t"
#define RDG_LOAD(how) "global_load_lds_dwordx4 %0, %1 offset:%3" how
#define RDG_UNLESS "s_cmp_ge_i32 %4, %5\n\ts_cbranch_scc1 1f\n\t"
#define RDG_WAIT "s_nop 0\n\t"
template <int IMM, bool TEST, bool ONCE>
__device__ __forceinline__ void dma16(int now, int end, const uint8_t* base, uint32_t off, uint32_t lds) {
    if constexpr (TEST && ONCE)
        asm volatile(RDG_M0 RDG_UNLESS RDG_LOAD(" nt\n1:") ::"v"(off), "s"(base), "s"(lds), "n"(IMM), "s"(now), "s"(end) : "memory", "m0", "scc");
    else if constexpr (TEST)
        asm volatile(RDG_M0 RDG_UNLESS RDG_LOAD("\n1:") ::"v"(off), "s"(base), "s"(lds), "n"(IMM), "s"(now), "s"(end) : "memory", "m0", "scc");
    else if constexpr (ONCE)
        asm volatile(RDG_M0 RDG_WAIT RDG_LOAD(" nt") ::"v"(off), "s"(base), "s"(lds), "n"(IMM) : "memory", "m0");
    else
        asm volatile(RDG_M0 RDG_WAIT RDG_LOAD("") ::"v"(off), "s"(base), "s"(lds), "n"(IMM) : "memory", "m0");
}
#undef RDG_M0
#undef RDG_LOAD
#undef RDG_UNLESS
#undef RDG_WAIT
__device__ __forceinline__ void dma4(int now, int end, const void* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_cmp_ge_i32 %3, %4\n\ts_cbranch_scc1 1f\n\tglobal_load_lds_dword %0, %1\n1:" ::"v"(off), "s"(base),
                 "s"(lds), "s"(now), "s"(end)
                 : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

// Waits until at most P * min(MOST, left) of the wave's loads are outstanding (none for left <= 0), and for
// its LDS reads; a wave that has P - 1 loads a stage (`fewer`, where they are not EVEN): as many of those.
template <int P, int MOST, bool TEST, bool EVEN>
__device__ __forceinline__ void wait_loads(int left, int fewer) {
    static_assert(MOST >= 0 && MOST <= 4 && P * MOST < 64, "vmcnt is six bits");
    if constexpr (!EVEN && TEST) {  // (the last stages only: all waves as those with fewer)
        wait_loads<P - 1, MOST, true, true>(left, 0);
    } else if constexpr (!EVEN) {
        asm volatile("s_cmp_eq_u32 %0, 0\n\ts_cbranch_scc1 1f\n\ts_waitcnt vmcnt(%1)\n1:\ts_waitcnt vmcnt(%2) lgkmcnt(0)" ::"s"(fewer),
                     "n"((P - 1) * MOST), "n"(P * MOST)
                     : "memory", "scc");
    } else if constexpr (MOST == 0 || !TEST) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(P * MOST) : "memory");
    } else if constexpr (MOST <= 2) {
        asm volatile("s_cmp_ge_i32 %0, %1\n\ts_cbranch_scc1 2f\n\ts_cmp_ge_i32 %0, 1\n\ts_cbranch_scc1 1f\n\ts_waitcnt vmcnt(0)\n"
                     "1:\ts_waitcnt vmcnt(%2)\n2:\ts_waitcnt vmcnt(%3) lgkmcnt(0)" ::"s"(left), "n"(MOST), "n"(P), "n"(P * MOST)
                     : "memory", "scc");
    } else {
        asm volatile("s_cmp_ge_i32 %0, %1\n\ts_cbranch_scc1 4f\n\ts_cmp_ge_i32 %0, 3\n\ts_cbranch_scc1 3f\n\ts_cmp_ge_i32 %0, 2\n\t"
                     "s_cbranch_scc1 2f\n\ts_cmp_ge_i32 %0, 1\n\ts_cbranch_scc1 1f\n\ts_waitcnt vmcnt(0)\n1:\ts_waitcnt vmcnt(%2)\n"
                     "2:\ts_waitcnt vmcnt(%3)\n3:\ts_waitcnt vmcnt(%4)\n4:\ts_waitcnt vmcnt(%5) lgkmcnt(0)" ::"s"(left), "n"(MOST), "n"(P),
                     "n"(2 * P), "n"(3 * P), "n"(P * MOST)
                     : "memory", "scc");
    }
}

// LDS place of 16-byte piece c of tile row r (rows of 128 bytes).  A read's 16 rows are served
// 16 lanes at a time, a mix of two pieces: pieces next to each other for bf16, two apart for e4m3 (fp32: one
// piece, read by fours of a lane each).
template <bool NEXT>
__device__ __forceinline__ int piece_slot(int r, int c) {
    return c ^ ((r & 7) ^ (((r >> 3) & 1) << (NEXT ? 1 : 0)));
}

// f(0), f(1), .. f(N - 1) with compile-time arguments.
template <int N, class F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
    each_of<N>(f, std::make_integer_sequence<int, N>{});
}

// ONCE: no other workgroup reads the weights.
template <int KIND, int WF, int WT, int NF, int NTK, int NB, bool ONCE>
__global__ __launch_bounds__(WF * WT * 64, 2) void k_linear_tiled(LinearCall a, int f_tiles, int t_tiles, int splits) {
    constexpr bool FP8 = KIND == kFp8 || KIND == kE8m0 || KIND == kFp8Wide, F32 = KIND == kF32, BF16 = KIND == kBf16;
    constexpr int NW = WF * WT, TF = WF * NF * 16, TT = WT * NTK * 16;
    constexpr int WB = TF * 128, XB = TT * 128, STAGE = WB + XB;    // bytes of a stage: 128 of each row
    // KiB loads a wave and stage, the weights' first; where x's cannot be shared out evenly the last waves have one less
    constexpr int WL = WB / 1024 / NW, XL = (XB / 1024 + NW - 1) / NW, PIECES = WL + XL, FULL = XB / 1024 - (XL - 1) * NW;
    constexpr int ESZ = FP8 ? 1 : F32 ? 4 : 2, S = FP8 ? 1 : F32 ? 8 : 2;  // matrix steps of a stage
    // fp8: scales of SC stages at a time, [token][stage], then [128 features][stage]
    constexpr int SC = 8, SB = (TT * SC + 64) * 4;
    constexpr int OUT_ROW = NF * 16 + 4;                            // floats; 32 token rows a wave in the epilogue
    constexpr int LDS_LOOP = NB * STAGE + (FP8 ? 2 * SB : 0), LDS_OUT = NW * 32 * OUT_ROW * 4;
    static_assert(WL % 2 == 0 && WL * 1024 * NW == WB && NTK % 2 == 0, "shape");
    // the scales' loads of a chunk are issued 3 stages before its first use
    static_assert(!FP8 || (128 % (NF * 16) == 0 && (SC - 3) * NW > TT * SC / 64 && NB <= 5), "shape");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS_LOOP > LDS_OUT ? LDS_LOOP : LDS_OUT];
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
    const int wf = wv / WT, wt = wv % WT;

    // XCD b % 8 takes a contiguous share of the tiles, ordered in bands of 4 feature tiles that are
    // walked along the tokens: the tiles that run together on an XCD share their operands in its L2.
    const int tiles = f_tiles * t_tiles, n = tiles * splits, xcd = blockIdx.x % 8, q8 = n / 8, r8 = n % 8;
    const int job = xcd * q8 + (xcd < r8 ? xcd : r8) + blockIdx.x / 8;
    const int split = job / tiles, item = job % tiles;
    const int band = item / (4 * t_tiles), in_band = item % (4 * t_tiles);
    const int wide = f_tiles - 4 * band < 4 ? f_tiles - 4 * band : 4;
    const int ft = 4 * band + in_band % wide;
    const int64_t t0 = (int64_t)(in_band / wide) * TT;
    const int g0 = ft * (TF / 16), groups = a.N / 16;
    const int row_bytes = a.K * ESZ, nkb = a.K / 128;
    // this split's blocks of 128 elements: kb0 .. kb1 - 1, in stages
    const int kb0 = (int)((int64_t)nkb * split / splits), kb1 = (int)((int64_t)nkb * (split + 1) / splits);
    const int nst = (kb1 - kb0) * ESZ;
    const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr_t)lds;

    // rows past the last: the last one again, not stored
    const uint8_t* wsrc[WL / 2];
#pragma unroll
    for (int i = 0; i < WL / 2; ++i) {
        const int g = g0 + wv * (WL / 2) + i;
        wsrc[i] = static_cast<const uint8_t*>(a.w) + (int64_t)(g < groups ? g : groups - 1) * 16 * row_bytes + (int64_t)kb0 * 2048 * ESZ;
    }
    const int rows = a.T - t0 < TT ? (int)(a.T - t0) : TT;
    const uint8_t* xsrc = static_cast<const uint8_t*>(a.x) + t0 * a.x_stride * ESZ + (int64_t)kb0 * 128 * ESZ;
    const uint32_t woff = lane * 16;
    constexpr bool EVEN = FULL == NW;
    const int fewer = EVEN ? 0 : (FULL - 1 - wv) >> 31;  // all bits: this wave has XL - 1 pieces of x
    auto x_piece = [&](int i) { return EVEN ? wv * XL + i : wv + i * NW; };
    uint32_t xoff[XL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int r = x_piece(i) * 8 + lane / 8;
        xoff[i] = (uint32_t)(r < rows ? r : rows - 1) * (uint32_t)(a.x_stride * ESZ) + piece_slot<BF16>(r, lane % 8) * 16;
    }
    // piece p of stage st; with TEST if there is such a stage
    auto request = [&](int st, int place, auto pc, auto test) {
        constexpr bool TEST = decltype(test)::value;
        constexpr int p = decltype(pc)::value;
        const uint32_t to = base + place;
        if constexpr (p < WL)
            dma16<p % 2 * 1024, TEST, ONCE>(st, nst, wsrc[p / 2] + (int64_t)st * 2048, woff, to + (wv * WL + p / 2 * 2) * 1024);
        else if constexpr (p < PIECES) {
            constexpr bool SOME = !EVEN && p == PIECES - 1;  // not every wave's: a stage past the end for the others
            dma16<0, TEST || SOME, false>(SOME ? __builtin_amdgcn_readfirstlane(st | (fewer & 1 << 30)) : st, nst, xsrc + (int64_t)st * 128, xoff[p - WL],
                                   to + WB + x_piece(p - WL) * 1024);
        }
    };
    // piece `slot` of the scales of stages SC c .. (past the end the last stage's again): 8 tokens, or, behind
    // the tokens', the tile's blocks of 128 features; no piece for a slot beyond
    auto request_scales = [&](int c, int slot) {
        constexpr int XP = TT * SC / 64;
        const bool of_w = slot >= XP;
        const int first = of_w ? g0 / 8 : slot * 8, most = of_w ? (a.N - 1) / 128 : rows - 1;
        const int r = first + lane / SC, kb = kb0 + c * SC + lane % SC;
        dma4(slot > XP ? nst : c * SC, nst, of_w ? a.w_scales : a.x_scales + t0 * nkb, ((r < most ? r : most) * nkb + (kb < nkb ? kb : nkb - 1)) * 4,
             base + NB * STAGE + (c & 1) * SB + (of_w ? XP : slot) * 256);
    };

    f32x4_t acc[NF][NTK];
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < NTK; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // fragments: a wave's items are (step s, weight tile i), NTK matrix instructions each.  Weight
    // fragments are read AHEAD items before their use, token fragments a step before; fp32's, whose steps are short, both
    // AHEAD steps where a step is an item (DEEP).
    using op_t = typename LinOp<FP8 ? RDG_FP8_E4M3 : F32 ? RDG_F32 : RDG_BF16>::op_t;
    constexpr bool DEEP = F32 && NF == 1;
    constexpr int NI = S * NF, AHEAD = DEEP ? 3 : FP8 || NF < 4 ? 1 : 3, RPI = (2 * PIECES + NI - 1) / NI;
    constexpr int EARLY = AHEAD * RPI < PIECES ? AHEAD * RPI : PIECES;  // pieces issued between the meeting and the stage's end
    constexpr int SETS = DEEP ? AHEAD + 1 : S > 1 ? 2 : 1;
    static_assert((AHEAD <= NF || DEEP) && (NI % (AHEAD + 1) == 0 || NI == 1), "this stage's fragments are read before the meeting");
    static_assert(NI * RPI >= PIECES, "items");
    op_t fa[AHEAD + 1], fb[SETS][NTK];
    float sx[NTK], sw = 1.0f;
    const int wl = wf * NF * 2048 + lane * (F32 ? 4 : 16);
    int xl[F32 ? 8 : 2];
#pragma unroll
    for (int h = 0; h < (F32 ? 8 : 2); ++h) {
        const int piece = FP8 ? (lane >> 4) * 2 + h : F32 ? h : h * 4 + (lane >> 4);
        xl[h] = WB + wt * NTK * 2048 + (lane & 15) * 128 + piece_slot<BF16>(lane & 15, piece) * 16 + (F32 ? (lane >> 4) * 4 : 0);
    }
    auto read_a = [&](int place, int it) {
        const uint8_t* p = lds + (wl + place) + (it % NF) * 2048;
        if constexpr (FP8)
            fa[it % (AHEAD + 1)] = LinOp<RDG_FP8_E4M3>::join(*reinterpret_cast<const i32x4_t*>(p), *reinterpret_cast<const i32x4_t*>(p + 1024));
        else
            fa[it % (AHEAD + 1)] = *reinterpret_cast<const op_t*>(p + (it / NF) * (F32 ? 256 : 1024));
    };
    auto read_b = [&](int place, int s, int j) {
        if constexpr (FP8)
            fb[0][j] = LinOp<RDG_FP8_E4M3>::join(*reinterpret_cast<const i32x4_t*>(lds + (xl[0] + place) + j * 2048),
                                                 *reinterpret_cast<const i32x4_t*>(lds + (xl[1] + place) + j * 2048));
        else
            fb[s % SETS][j] = *reinterpret_cast<const op_t*>(lds + (xl[s] + place) + j * 2048);
    };
    const int w_block = (g0 + wf * NF) / 8 - g0 / 8;
    auto read_scales = [&](int st, float (&x)[NTK], float& w) {
        const float* p = reinterpret_cast<const float*>(lds + NB * STAGE + (st / SC & 1) * SB);
#pragma unroll
        for (int j = 0; j < NTK; ++j) x[j] = p[(wt * NTK * 16 + j * 16 + (lane & 15)) * SC + st % SC];
        w = p[TT * SC + w_block * SC + st % SC];
    };
    // In stage st: stage st + 1 has landed for every wave, and every wave has stage st's fragments in
    // registers, so that its place is free.
    auto meet = [&](int st, auto test) {
        __builtin_amdgcn_sched_barrier(0);
        wait_loads<PIECES, NB - 2, decltype(test)::value, EVEN>(nst - 2 - st, __builtin_amdgcn_readfirstlane(fewer));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };

    // the first NB - 1 stages, and what of the next one stage 0 takes as issued
    each<PIECES>([&](auto p) { request(0, 0, p, Yes{}); });
    if (FP8) {
#pragma unroll
        for (int i = 0; i < SC; ++i) request_scales(0, i * NW + wv);
    }
    each<NB - 2>([&](auto b) { each<PIECES>([&](auto p) { request(decltype(b)::value + 1, (decltype(b)::value + 1) * STAGE, p, Yes{}); }); });
    meet(-1, Yes{});
    each<EARLY>([&](auto p) { request(NB - 1, (NB - 1) * STAGE, p, Yes{}); });
#pragma unroll
    for (int s = 0; s < (DEEP ? AHEAD : 1); ++s)
#pragma unroll
        for (int j = 0; j < NTK; ++j) read_b(0, s, j);
    if (FP8) read_scales(0, sx, sw);
#pragma unroll
    for (int it = 0; it < AHEAD; ++it) read_a(0, it);
    __builtin_amdgcn_sched_barrier(0);

    f32x4_t part[2][2];  // fp8 with fp32 scales: products of two token tiles, and the two before
    int here = 0;        // place of stage st in LDS
    auto stage = [&](int st, auto test) {
        const int next = here + STAGE == NB * STAGE ? 0 : here + STAGE, before = here == 0 ? (NB - 1) * STAGE : here - STAGE;
        float f[NTK], next_sx[NTK], next_sw = 1.0f;
        int ex[NTK], ew = 0;
        if constexpr (KIND == kFp8 || KIND == kFp8Wide) {
#pragma unroll
            for (int j = 0; j < NTK; ++j) f[j] = sx[j] * sw;
        }
        if constexpr (KIND == kE8m0) {
#pragma unroll
            for (int j = 0; j < NTK; ++j) ex[j] = e8m0_of(sx[j]);
            ew = e8m0_of(sw);
        }
        each<NI>([&](auto itc) {
            constexpr int it = decltype(itc)::value, s = it / NF, i = it % NF;
            if constexpr (FP8 && it == 0) request_scales(st / SC + 1, st % SC * NW + wv);
            const op_t w = fa[it % (AHEAD + 1)];
            if (it + AHEAD < NI) read_a(here, it + AHEAD);
            if constexpr (DEEP) {
                if constexpr (it + AHEAD < NI) {
#pragma unroll
                    for (int j = 0; j < NTK; ++j) read_b(here, it + AHEAD, j);
                }
            } else if constexpr (s + 1 < S) {  // in the step's last items, all in one where it has fewer than NTK
                if constexpr (NF < NTK) {
                    if constexpr (i == NF - 1) {
#pragma unroll
                        for (int j = 0; j < NTK; ++j) read_b(here, s + 1, j);
                    }
                } else if constexpr (i >= NF - NTK) {
                    read_b(here, s + 1, i - (NF - NTK));
                }
            }
            if constexpr (it == NI - AHEAD) {
                meet(st, test);
                if constexpr (FP8) {
                    read_scales(st + 1, next_sx, next_sw);
                } else if constexpr (!DEEP) {
#pragma unroll
                    for (int j = 0; j < NTK; ++j) read_b(next, 0, j);
                }
            }
            // loads a few at a time, the last stages but one's: all at once they would hold up the wave's own instructions
            each<RPI>([&](auto r) {
                if constexpr (it >= NI - AHEAD)
                    request(st + NB, here, std::integral_constant<int, (it - (NI - AHEAD)) * RPI + decltype(r)::value>{}, test);
                else
                    request(st + NB - 1, before, std::integral_constant<int, EARLY + it * RPI + decltype(r)::value>{}, test);
            });
            // (behind the last stage the first fragments are read from a place that holds none, and not used)
            if (it + AHEAD >= NI) read_a(next, it + AHEAD - NI);
            if constexpr (DEEP && it + AHEAD >= NI) {
#pragma unroll
                for (int j = 0; j < NTK; ++j) read_b(next, it + AHEAD - NI, j);
            }
            if constexpr (BF16 || F32) {
#pragma unroll
                for (int j = 0; j < NTK; ++j)
                    acc[i][j] = LinOp<F32 ? RDG_F32 : RDG_BF16>::mma(acc[i][j], w, fb[s % SETS][j]);
            } else if constexpr (KIND == kE8m0) {
#pragma unroll
                for (int j = 0; j < NTK; ++j) {
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, fb[0][j], acc[i][j], 0, 0, 0, ew, 0, ex[j]);
                    if (it == NI - 1) {
                        __builtin_amdgcn_sched_barrier(0);
                        read_b(next, 0, j);  // in its predecessor's place, used for the last time
                    }
                }
            } else {
                // two products at a time, and behind them the two before them into the sum
#pragma unroll
                for (int h = 0; h < NTK / 2; ++h) {
                    const int now = it * (NTK / 2) + h, then = now - 1;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const f32x4_t z = {0.f, 0.f, 0.f, 0.f};
                        part[now % 2][u] = KIND == kFp8Wide ? LinOp<RDG_FP8_E4M3>::mma_wide(z, w, fb[0][2 * h + u]) : LinOp<RDG_FP8_E4M3>::mma(z, w, fb[0][2 * h + u]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    if (it == NI - 1) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) read_b(next, 0, 2 * h + u);
                    }
                    if (now > 0) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int jb = then % (NTK / 2) * 2 + u;
                            acc[then / (NTK / 2)][jb] += part[then % 2][u] * f[jb];
                        }
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (KIND == kFp8 || KIND == kFp8Wide) {
            constexpr int last = NI * (NTK / 2) - 1;
#pragma unroll
            for (int u = 0; u < 2; ++u) acc[NF - 1][NTK - 2 + u] += part[last % 2][u] * f[NTK - 2 + u];
        }
        if constexpr (FP8) {
#pragma unroll
            for (int j = 0; j < NTK; ++j) sx[j] = next_sx[j];
            sw = next_sw;
        }
        here = next;
    };
    int st = 0;
    if constexpr (F32) {
        // sums of 512 products each, then their sum: the rounding errors of one long chain of fp32 products grow with its
        // length (K = 4096: 1.1e-6 of the result in one chain, 4e-7 in eights)
        f32x4_t total[NF][NTK];
        auto flush = [&](bool first) {
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int j = 0; j < NTK; ++j) {
                    total[i][j] = first ? acc[i][j] : total[i][j] + acc[i][j];
                    acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                }
        };
        flush(true);
        while (st < nst) {
            const int stop = st + 16 < nst ? st + 16 : nst, free = stop < nst - NB ? stop : nst - NB;
            for (; st < free; ++st) stage(st, No{});
            for (; st < stop; ++st) stage(st, Yes{});
            flush(false);
        }
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int j = 0; j < NTK; ++j) acc[i][j] = total[i][j];
    } else {
        for (; st < nst - NB; ++st) stage(st, No{});
        for (; st < nst; ++st) stage(st, Yes{});
    }

    // ---------------------------------------------------------------- epilogue
    // Each wave turns its sums over in LDS (its own part; no wave reads operands any more), two token
    // tiles at a time, and stores 8 features a lane: whole rows of its features.  The residual of these rows is asked for
    // first, all at once, and bias and activation are done in place in LDS by a loop of their own, whose code
    // is there once.
    constexpr int LPR = NF * 2, RPP = 64 / LPR, PASSES = 32 / RPP;  // lanes a row, rows a pass
    float* tile = reinterpret_cast<float*>(lds) + wv * 32 * OUT_ROW;
    const int f = (g0 + wf * NF) * 16 + lane % LPR * 8;
    const bool whole = splits == 1, added = whole && a.residual != nullptr && f < a.N;
    auto place = [&](int p) { return tile + (p * RPP + lane / LPR) * OUT_ROW + lane % LPR * 8; };
    float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (whole && a.bias != nullptr && f < a.N) load8<false>(a.bias, f, bias);
#pragma unroll
    for (int half = 0; half < NTK / 2; ++half) {
        const int64_t first = t0 + (wt * NTK + half * 2) * 16 + lane / LPR;
        uint4 held[PASSES][2];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            held[p][0] = held[p][1] = make_uint4(0u, 0u, 0u, 0u);
            const int64_t t = first + p * RPP;
            if (added && t < a.T) {
                const uint4* r = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.residual) +
                                                                (t * a.res_stride + f) * (a.out_bf16 ? 2 : 4));
                held[p][0] = r[0];
                if (!a.out_bf16) held[p][1] = r[1];
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < NF; ++i)
                *reinterpret_cast<f32x4_t*>(tile + (u * 16 + (lane & 15)) * OUT_ROW + i * 16 + (lane >> 4) * 4) = acc[i][half * 2 + u];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (whole && (a.bias != nullptr || a.act != RDG_ACT_NONE)) {
#pragma unroll 1
            for (int p = 0; p < PASSES; ++p) {
                float v[8];
                load8<false>(place(p), 0, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += bias[e];
                activate(v, a.act);
                store8<false>(place(p), 0, v);  // read by this lane alone
            }
        }
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int64_t t = first + p * RPP;
            float v[8];
            load8<false>(place(p), 0, v);
            if (t < a.T && f < a.N) {
                if (!whole) {
                    store8<false>(a.parts, ((int64_t)split * a.T + t) * a.N + f, v);
                } else if (a.out_bf16) {
                    float r[8];
                    load8<true>(&held[p][0], 0, r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += r[e];
                    store8<true>(a.out, t * a.out_stride + f, v);
                } else {
                    float r[8];
                    load8<false>(&held[p][0], 0, r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += r[e];
                    store8<false>(a.out, t * a.out_stride + f, v);
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
}

// The splits' sums in their order, and the epilogue: 8 features a thread, all its loads asked for at once.
template <int SPLITS>
__global__ __launch_bounds__(256) void k_linear_join(LinearCall a) {
    const int per_row = a.N / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)a.T * per_row;
    if (i >= all) return;
    float p[SPLITS][8];
#pragma unroll
    for (int s = 0; s < SPLITS; ++s) load8<false>(a.parts, ((int64_t)s * all + i) * 8, p[s]);
#pragma unroll
    for (int s = 1; s < SPLITS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) p[0][e] += p[s][e];
    finish8(a, p[0], i / per_row, (int)(i % per_row) * 8);
}

template <int KIND, int WF, int WT, int NF, int NTK, int NB>
hipError_t launch(const LinearCall& a, int splits, hipStream_t s) {
    constexpr int TF = WF * NF * 16, TT = WT * NTK * 16;
    const int64_t f_tiles = (a.N + TF - 1) / TF, t_tiles = ((int64_t)a.T + TT - 1) / TT, all = f_tiles * t_tiles * splits;
    const int64_t join = ((int64_t)a.T * (a.N / 8) + 255) / 256;
    if (!grid_fits(all, WF * WT * 64) || !grid_fits(join, 256)) return hipErrorInvalidConfiguration;
    // weights that no other workgroup reads pass the caches.  us from memory, and with the same weights over again, past the
    // caches and through them: 64 tokens, 18432 features, K = 7168 in e8m0 28.8, 27.1 and 29.7, 26.8, in bf16 50.8, 49.5 and
    // 53.7, 44.5; 24576 features 59.5, 58.5 and 65.7, 65.0.  A layer's weights come from memory, as the other layers' have passed
    // since; weights that the last cache keeps (256 MiB) pay up to a fifth (7168 features 26.2 and 20.9).  With a second
    // tile of tokens it would cost: 256 tokens of 7168 x 7168 51.5 -> 55.7.
    if (NF <= 2 && t_tiles == 1)
        k_linear_tiled<KIND, WF, WT, NF, NTK, NB, (NF <= 2)><<<(unsigned)all, WF * WT * 64, 0, s>>>(a, (int)f_tiles, 1, splits);
    else
        k_linear_tiled<KIND, WF, WT, NF, NTK, NB, false><<<(unsigned)all, WF * WT * 64, 0, s>>>(a, (int)f_tiles, (int)t_tiles, splits);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || splits == 1) return err;
    if (splits == 2) k_linear_join<2><<<(unsigned)join, 256, 0, s>>>(a);
    else if (splits == 4) k_linear_join<4><<<(unsigned)join, 256, 0, s>>>(a);
    else if (splits == 8) k_linear_join<8><<<(unsigned)join, 256, 0, s>>>(a);
    else k_linear_join<16><<<(unsigned)join, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

template <int KIND>
static hipError_t launch_kind(const LinearCall& a, const LinearPart& p, hipStream_t s) {
    // (fp32 has no plans of these: 256 x 256 would keep two sets of sums)
    if constexpr (KIND != kF32) {
        // (products of widened operands need registers for them, so half the tokens)
        if (p.kernel == kTile256) return launch<KIND, 2, 4, 8, KIND == kFp8Wide ? 2 : 4, 2>(a, p.splits, s);
        if (p.kernel == kTile96x64) return launch<KIND, 6, 1, 1, 4, 5>(a, p.splits, s);
        if (p.kernel == kTile80x64) return launch<KIND, 5, 1, 1, 4, 5>(a, p.splits, s);
        if (p.kernel == kTile64x64) return launch<KIND, 4, 1, 1, 4, 5>(a, p.splits, s);
    }
    switch (p.kernel) {
        case kTile128: return launch<KIND, 2, 4, 4, 2, 4>(a, p.splits, s);
        case kTile128x64: return launch<KIND, 4, 2, 2, 2, 5>(a, p.splits, s);
        default: return launch<KIND, 4, 1, 1, 2, 4>(a, p.splits, s);
    }
}

hipError_t launch_linear_tiled(const LinearCall& a, const LinearPart& p, hipStream_t s) {
    switch (a.dtype) {
        case RDG_F32: return launch_kind<kF32>(a, p, s);
        case RDG_BF16: return launch_kind<kBf16>(a, p, s);
        case RDG_FP8_E4M3: return a.out_bf16 ? launch_kind<kFp8>(a, p, s) : launch_kind<kFp8Wide>(a, p, s);
        default: return a.out_bf16 ? launch_kind<kE8m0>(a, p, s) : launch_kind<kFp8Wide>(a, p, s);
    }
}

}  // namespace rdg
