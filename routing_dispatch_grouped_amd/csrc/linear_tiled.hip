// Matrix product with its epilogue for many tokens: tiles of TF features x TT tokens.
#include <type_traits>
#include <utility>

#include "linear.h"

namespace rdg {
namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// s_waitcnt immediates (vmcnt in bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8).
constexpr int kWaitVm0 = (7 << 4) | (15 << 8);
constexpr int kWaitLgkm0 = 15 | (3 << 14) | (7 << 4);

// What a kernel does with its operands: bf16; e4m3 with fp32 scales (each partial product of 128
// is scaled into the sum); e4m3 with power-of-two scales (the matrix core applies them).
enum { kBf16 = 0, kFp8 = 1, kE8m0 = 2 };

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 (4) bytes a lane from base + off + IMM straight to lds + IMM + 16 (4) * lane (base and lds wave-uniform).
// The compiler does not count these loads; meet() below waits for them.
template <int IMM>
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1 offset:%3" ::"v"(off), "s"(base), "s"(lds), "n"(IMM) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
#pragma clang diagnostic pop

// LDS place of 16-byte piece c of tile row r (rows of 128 bytes).  A read's 16 rows are served
// 16 lanes at a time, a mix of two pieces: pieces next to each other for bf16, two apart for e4m3.
template <bool FP8>
__device__ __forceinline__ int piece_slot(int r, int c) {
    return c ^ ((r & 7) ^ (((r >> 3) & 1) << (FP8 ? 0 : 1)));
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

template <int KIND, int WF, int WT, int NF, int NTK>
__global__ __launch_bounds__(WF * WT * 64, 1) void k_linear_tiled(LinearCall a, int f_tiles, int t_tiles) {
    constexpr bool FP8 = KIND != kBf16;
    constexpr int NW = WF * WT, TF = WF * NF * 16, TT = WT * NTK * 16;
    constexpr int WB = TF * 128, XB = TT * 128, STAGE = WB + XB;  // bytes of a stage: 128 of each row
    constexpr int PIECES = STAGE / 1024 / NW, WL = WB / 1024 / NW;  // KiB loads a wave and stage, the weights' first
    constexpr int ESZ = FP8 ? 1 : 2, S = FP8 ? 1 : 2;             // matrix steps of a stage
    // fp8: scales of SC stages at a time, [token][stage], then [128 features][stage]
    constexpr int SC = 8, FB = TF / 128, SB = (TT * SC + 64) * 4;
    constexpr int OUT_ROW = NF * 16 + 4;                          // floats; 32 token rows a wave in the epilogue
    constexpr int LDS_LOOP = 2 * STAGE + (FP8 ? 2 * SB : 0), LDS_OUT = NW * 32 * OUT_ROW * 4;
    static_assert(WL % 2 == 0 && (!FP8 || (NF == 8 && SC * NW > TT * SC / 64)), "shape");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS_LOOP > LDS_OUT ? LDS_LOOP : LDS_OUT];
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
    const int wf = wv / WT, wt = wv % WT;

    // XCD b % 8 takes a contiguous share of the tiles, ordered in bands of 4 feature tiles that are
    // walked along the tokens: the tiles that run together on an XCD share their operands in its L2.
    const int n = f_tiles * t_tiles, xcd = blockIdx.x % 8, q8 = n / 8, r8 = n % 8;
    const int item = xcd * q8 + (xcd < r8 ? xcd : r8) + blockIdx.x / 8;
    const int band = item / (4 * t_tiles), in_band = item % (4 * t_tiles);
    const int wide = f_tiles - 4 * band < 4 ? f_tiles - 4 * band : 4;
    const int ft = 4 * band + in_band % wide;
    const int64_t t0 = (int64_t)(in_band / wide) * TT;
    const int g0 = ft * (TF / 16), groups = a.N / 16;
    const int row_bytes = a.K * ESZ, nst = row_bytes / 128, nkb = a.K / 128;
    const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr_t)lds;

    // rows past the last: the last one again, not stored
    const uint8_t* wsrc[WL / 2];
#pragma unroll
    for (int i = 0; i < WL / 2; ++i) {
        const int g = g0 + wv * (WL / 2) + i;
        wsrc[i] = static_cast<const uint8_t*>(a.w) + (int64_t)(g < groups ? g : groups - 1) * 16 * row_bytes;
    }
    const int rows = a.T - t0 < TT ? (int)(a.T - t0) : TT;
    const uint8_t* xsrc = static_cast<const uint8_t*>(a.x) + t0 * a.x_stride * ESZ;
    const uint32_t woff = lane * 16;
    uint32_t xoff[PIECES - WL];
#pragma unroll
    for (int i = 0; i < PIECES - WL; ++i) {
        const int r = (wv * (PIECES - WL) + i) * 8 + lane / 8;
        xoff[i] = (uint32_t)(r < rows ? r : rows - 1) * (uint32_t)(a.x_stride * ESZ) + piece_slot<FP8>(r, lane % 8) * 16;
    }
    // piece p of stage st
    auto request = [&](int st, int buf, auto pc) {
        constexpr int p = decltype(pc)::value;
        const uint32_t to = base + buf * STAGE;
        if constexpr (p < WL)
            dma16<p % 2 * 1024>(wsrc[p / 2] + (int64_t)st * 2048, woff, to + (wv * WL + p / 2 * 2) * 1024);
        else if constexpr (p < PIECES)
            dma16<0>(xsrc + (int64_t)st * 128, xoff[p - WL], to + WB + (wv * (PIECES - WL) + p - WL) * 1024);
    };
    // piece `slot` (64 in all, the last ones alike) of the scales of stages SC c .. (past the end the last
    // stage's again): 8 tokens, or the tile's blocks of 128 features
    auto request_scales = [&](int c, int slot) {
        constexpr int XP = TT * SC / 64;
        const bool of_w = slot >= XP;
        const int first = of_w ? ft * FB : slot * 8, most = of_w ? (a.N - 1) / 128 : rows - 1;
        const int r = first + lane / SC, kb = c * SC + lane % SC;
        dma4(of_w ? a.w_scales : a.x_scales + t0 * nkb, ((r < most ? r : most) * nkb + (kb < nkb ? kb : nkb - 1)) * 4,
             base + 2 * STAGE + (c & 1) * SB + (of_w ? XP : slot) * 256);
    };

    f32x4_t acc[NF][NTK];
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < NTK; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // fragments: a wave's items are (step s, weight tile i), NTK matrix instructions each.  Weight
    // fragments are read AHEAD items before their use, token fragments a step before.
    using op_t = typename LinOp<FP8 ? RDG_FP8_E4M3 : RDG_BF16>::op_t;
    constexpr int NI = S * NF, AHEAD = FP8 ? 1 : 3, RPI = FP8 ? 2 : 1;
    op_t fa[AHEAD + 1], fb[S][NTK];
    float sx[2][NTK], sw[2];
    const uint8_t* wl = lds + wf * NF * 2048 + lane * 16;
    const uint8_t* xl[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int piece = FP8 ? (lane >> 4) * 2 + h : h * 4 + (lane >> 4);
        xl[h] = lds + WB + wt * NTK * 2048 + (lane & 15) * 128 + piece_slot<FP8>(lane & 15, piece) * 16;
    }
    auto read_a = [&](int buf, int it) {
        const uint8_t* p = wl + buf * STAGE + (it % NF) * 2048;
        if constexpr (FP8)
            fa[it % (AHEAD + 1)] = LinOp<RDG_FP8_E4M3>::join(*reinterpret_cast<const i32x4_t*>(p), *reinterpret_cast<const i32x4_t*>(p + 1024));
        else
            fa[it % (AHEAD + 1)] = *reinterpret_cast<const bf16x8_t*>(p + (it / NF) * 1024);
    };
    auto read_b = [&](int buf, int s, int j) {
        if constexpr (FP8)
            fb[0][j] = LinOp<RDG_FP8_E4M3>::join(*reinterpret_cast<const i32x4_t*>(xl[0] + buf * STAGE + j * 2048),
                                                   *reinterpret_cast<const i32x4_t*>(xl[1] + buf * STAGE + j * 2048));
        else
            fb[s][j] = *reinterpret_cast<const bf16x8_t*>(xl[s] + buf * STAGE + j * 2048);
    };
    auto read_scales = [&](int st, int set) {
        const float* p = reinterpret_cast<const float*>(lds + 2 * STAGE + (st / SC & 1) * SB);
#pragma unroll
        for (int j = 0; j < NTK; ++j) sx[set][j] = p[(wt * NTK * 16 + j * 16 + (lane & 15)) * SC + st % SC];
        sw[set] = p[TT * SC + wf * SC + st % SC];
    };
    // Every wave's loads have landed, and every wave has its fragments in registers.
    auto meet = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(kWaitVm0 & kWaitLgkm0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };

    each<PIECES>([&](auto p) { request(0, 0, p); });
    if (FP8) {
#pragma unroll
        for (int i = 0; i < SC; ++i) request_scales(0, i * NW + wv);
    }
    meet();
    if (nst > 1) each<AHEAD * RPI>([&](auto p) { request(1, 1, p); });
#pragma unroll
    for (int j = 0; j < NTK; ++j) read_b(0, 0, j);
    if (FP8) read_scales(0, 0);
#pragma unroll
    for (int it = 0; it < AHEAD; ++it) read_a(0, it);
    __builtin_amdgcn_sched_barrier(0);

    f32x4_t part[2][2];  // fp8 with fp32 scales: products of two token tiles, and the two before
    // left: stages behind this one, 2 for two and more.  (No branch inside: the compiler would move the matrix
    // instructions past it.)
    auto stage = [&](int st, auto bufc, auto leftc) {
        constexpr int buf = decltype(bufc)::value, left = decltype(leftc)::value;
        float f[NTK];
        int ex[NTK], ew = 0;
        if constexpr (KIND == kFp8) {
#pragma unroll
            for (int j = 0; j < NTK; ++j) f[j] = sx[buf][j] * sw[buf];
        }
        if constexpr (KIND == kE8m0) {
#pragma unroll
            for (int j = 0; j < NTK; ++j) ex[j] = e8m0_of(sx[buf][j]);
            ew = e8m0_of(sw[buf]);
        }
        each<NI>([&](auto itc) {
            constexpr int it = decltype(itc)::value, s = it / NF, i = it % NF;
            if constexpr (FP8 && it == 0 && left > 0) request_scales(st / SC + 1, st % SC * NW + wv);
            if (it + AHEAD < NI) read_a(buf, it + AHEAD);
            if (s + 1 < S && i >= NF - NTK) read_b(buf, s + 1, i - (NF - NTK));
            if (it == NI - AHEAD) {
                // behind the meeting the next stage has landed and this one's place is free
                meet();
                if constexpr (FP8) {
                    if constexpr (left > 0) read_scales(st + 1, buf ^ 1);
                } else if constexpr (left > 0) {
#pragma unroll
                    for (int j = 0; j < NTK; ++j) read_b(buf ^ 1, 0, j);
                }
            }
            // the next loads a few at a time: all at once they would hold up the wave's own instructions
            if constexpr (it >= NI - AHEAD) {
                if constexpr (left > 1)
                    each<RPI>([&](auto r) { request(st + 2, buf, std::integral_constant<int, (it - (NI - AHEAD)) * RPI + decltype(r)::value>{}); });
            } else if constexpr (left > 0 && (it + AHEAD) * RPI < PIECES) {
                each<RPI>([&](auto r) { request(st + 1, buf ^ 1, std::integral_constant<int, (it + AHEAD) * RPI + decltype(r)::value>{}); });
            }
            if (left > 0 && it + AHEAD >= NI) read_a(buf ^ 1, it + AHEAD - NI);
            const op_t w = fa[it % (AHEAD + 1)];
            if constexpr (KIND == kBf16) {
#pragma unroll
                for (int j = 0; j < NTK; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, fb[s][j], acc[i][j], 0, 0, 0);
            } else if constexpr (KIND == kE8m0) {
#pragma unroll
                for (int j = 0; j < NTK; ++j) {
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, fb[0][j], acc[i][j], 0, 0, 0, ew, 0, ex[j]);
                    if (left > 0 && it == NI - 1) {
                        __builtin_amdgcn_sched_barrier(0);
                        read_b(buf ^ 1, 0, j);  // in its predecessor's place, used for the last time
                    }
                }
            } else {
                // two products at a time, and behind them the two before them into the sum
#pragma unroll
                for (int h = 0; h < NTK / 2; ++h) {
                    const int now = it * (NTK / 2) + h, before = now - 1;
#pragma unroll
                    for (int u = 0; u < 2; ++u) part[now % 2][u] = LinOp<RDG_FP8_E4M3>::mma(f32x4_t{0.f, 0.f, 0.f, 0.f}, w, fb[0][2 * h + u]);
                    __builtin_amdgcn_sched_barrier(0);
                    if (left > 0 && it == NI - 1) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) read_b(buf ^ 1, 0, 2 * h + u);
                    }
                    if (now > 0) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int jb = before % (NTK / 2) * 2 + u;
                            acc[before / (NTK / 2)][jb] += part[before % 2][u] * f[jb];
                        }
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (KIND == kFp8) {
            constexpr int last = NI * (NTK / 2) - 1;
#pragma unroll
            for (int u = 0; u < 2; ++u) acc[NF - 1][NTK - 2 + u] += part[last % 2][u] * f[NTK - 2 + u];
        }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    int st = 0;
    for (; st + 3 < nst; st += 2) {
        stage(st, I0{}, I2{});
        stage(st + 1, I1{}, I2{});
    }
    if (!FP8 || nst % 2 == 0) {  // two stages left (bf16: K is a multiple of 128)
        stage(st, I0{}, I1{});
        stage(st + 1, I1{}, I0{});
    } else if (nst > 1) {
        stage(st, I0{}, I2{});
        stage(st + 1, I1{}, I1{});
        stage(st + 2, I0{}, I0{});
    } else {
        stage(st, I0{}, I0{});
    }

    // ---------------------------------------------------------------- epilogue
    // Each wave turns its sums over in LDS (its own part; no wave reads operands any more), two token
    // tiles at a time, and stores 8 features a lane: whole rows of its features.
    constexpr int LPR = NF * 2, RPP = 64 / LPR;  // lanes a row, rows a pass
    float* tile = reinterpret_cast<float*>(lds) + wv * 32 * OUT_ROW;
    const int f = (g0 + wf * NF) * 16 + lane % LPR * 8;
    float bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = 0.0f;
    if (a.bias != nullptr && f < a.N) load8<false>(a.bias, f, bias);
#pragma unroll
    for (int half = 0; half < NTK / 2; ++half) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < NF; ++i)
                *reinterpret_cast<f32x4_t*>(tile + (u * 16 + (lane & 15)) * OUT_ROW + i * 16 + (lane >> 4) * 4) = acc[i][half * 2 + u];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll 1
        for (int p = 0; p < 32 / RPP; ++p) {
            const int row = p * RPP + lane / LPR;
            const int64_t t = t0 + (wt * NTK + half * 2) * 16 + row;
            float v[8];
            load8<false>(tile + row * OUT_ROW, lane % LPR * 8, v);
            if (t < a.T && f < a.N) finish8(a, v, bias, t, f);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
}

template <int KIND, int WF, int WT, int NF, int NTK>
hipError_t launch(const LinearCall& a, hipStream_t s) {
    constexpr int TF = WF * NF * 16, TT = WT * NTK * 16;
    const int64_t f_tiles = (a.N + TF - 1) / TF, t_tiles = ((int64_t)a.T + TT - 1) / TT;
    if (!grid_fits(f_tiles * t_tiles, WF * WT * 64)) return hipErrorInvalidConfiguration;
    k_linear_tiled<KIND, WF, WT, NF, NTK><<<(unsigned)(f_tiles * t_tiles), WF * WT * 64, 0, s>>>(a, (int)f_tiles, (int)t_tiles);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_tiled(const LinearCall& a, hipStream_t s) {
    if (a.dtype == RDG_BF16) return launch<kBf16, 2, 4, 8, 4>(a, s);
    return a.dtype == RDG_FP8_E4M3 ? launch<kFp8, 2, 4, 8, 4>(a, s) : launch<kE8m0, 2, 4, 8, 4>(a, s);
}

}  // namespace rdg
