// Matrix product with its epilogue for many tokens: tiles of TF features x TT tokens.
#include <type_traits>

#include "linear.h"

namespace rdg {
namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// s_waitcnt immediates (vmcnt in bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8).
constexpr int kWaitVm0 = (7 << 4) | (15 << 8);
constexpr int kWaitLgkm0 = 15 | (3 << 14) | (7 << 4);

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 bytes a lane from src straight to lds + 16 * lane (lds wave-uniform).
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "memory", "m0");
}
#pragma clang diagnostic pop

// Place of 16-byte piece c of tile row r (rows of 128 bytes).
__device__ __forceinline__ int piece_slot(int r, int c) { return c ^ ((r & 7) ^ ((r >> 3) & 1)); }

template <int WF, int WT, int NF, int NTK>
__global__ __launch_bounds__(WF * WT * 64, 1) void k_linear_tiled(LinearCall a, int f_tiles, int t_tiles) {
    constexpr int NW = WF * WT, TF = WF * NF * 16, TT = WT * NTK * 16;
    constexpr int WB = TF * 128, XB = TT * 128, STAGE = WB + XB;  // bytes of a stage: 64 elements of each row
    constexpr int WL = WB / 1024 / NW, XL = XB / 1024 / NW;       // KiB loads a wave and stage
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
    const int n = f_tiles * t_tiles, b = blockIdx.x, xcd = b % 8, q8 = n / 8, r8 = n % 8;
    const int item = xcd * q8 + (xcd < r8 ? xcd : r8) + b / 8;
    const int tt = item % t_tiles, ft = item / t_tiles;
    const int64_t t0 = (int64_t)tt * TT;
    const int g0 = ft * (TF / 16), groups = a.N / 16;
    const int nst = a.K / 64;
    const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr_t)lds;

    const uint8_t* wsrc[WL / 2];
#pragma unroll
    for (int i = 0; i < WL / 2; ++i) {
        const int g = g0 + wv * (WL / 2) + i;
        wsrc[i] = static_cast<const uint8_t*>(a.w) + (int64_t)(g < groups ? g : groups - 1) * (a.K / 32) * 1024 + lane * 16;
    }
    const uint8_t* xsrc[XL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int r = (wv * XL + i) * 8 + lane / 8;
        const int64_t t = t0 + r < a.T ? t0 + r : a.T - 1;
        xsrc[i] = static_cast<const uint8_t*>(a.x) + t * a.x_stride * 2 + piece_slot(r, lane % 8) * 16;
    }
    auto request = [&](int st, int buf) {
        const uint32_t to = base + buf * STAGE;
#pragma unroll
        for (int i = 0; i < WL; ++i)
            dma16(wsrc[i / 2] + (int64_t)st * 2048 + (i % 2) * 1024, to + (wv * WL + i) * 1024);
#pragma unroll
        for (int i = 0; i < XL; ++i) dma16(xsrc[i] + (int64_t)st * 128, to + WB + (wv * XL + i) * 1024);
    };
    const int wf = wv / WT, wt = wv % WT;
    // the lane's places: weight tile i, step s at (wf NF + i) 2048 + s 1024 + lane 16; token tile j likewise 16 rows of 128
    const int wo = wf * NF * 2048 + lane * 16;
    int xo[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) xo[s] = WB + wt * NTK * 2048 + (lane & 15) * 128 + piece_slot(lane & 15, s * 4 + (lane >> 4)) * 16;

    f32x4_t acc[NF][NTK];
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < NTK; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    constexpr int AHEAD = 3, NI = 2 * NF;
    bf16x8_t fa[AHEAD + 1], fb[2][NTK];
    auto read_a = [&](int buf, int it) {  // item it = step * NF + i
        fa[it % (AHEAD + 1)] = *reinterpret_cast<const bf16x8_t*>(lds + buf * STAGE + wo + (it % NF) * 2048 + (it / NF) * 1024);
    };
    auto read_b = [&](int buf, int s, int j) {
        fb[s][j] = *reinterpret_cast<const bf16x8_t*>(lds + buf * STAGE + xo[s] + j * 2048);
    };
    auto meet = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(kWaitVm0 & kWaitLgkm0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    request(0, 0);
    meet();
    if (nst > 1) request(1, 1);
#pragma unroll
    for (int j = 0; j < NTK; ++j) read_b(0, 0, j);
#pragma unroll
    for (int it = 0; it < AHEAD; ++it) read_a(0, it);
    __builtin_amdgcn_sched_barrier(0);
    auto stage = [&](int st, auto bufc) {
        constexpr int buf = decltype(bufc)::value;
#pragma unroll
        for (int it = 0; it < NI; ++it) {
            const int s = it / NF, i = it % NF;
            if (it + AHEAD < NI) read_a(buf, it + AHEAD);
            if (s == 0 && i >= NF - NTK) read_b(buf, 1, i - (NF - NTK));
            if (it == NI - AHEAD) {
                // every fragment of this stage is in registers: once all waves are here, the next
                // stage has landed and this one's place is free
                meet();
                if (st + 2 < nst) request(st + 2, buf);
#pragma unroll
                for (int j = 0; j < NTK; ++j) read_b(buf ^ 1, 0, j);
            }
            if (it + AHEAD >= NI) read_a(buf ^ 1, it + AHEAD - NI);
#pragma unroll
            for (int j = 0; j < NTK; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[it % (AHEAD + 1)], fb[s][j], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // an even number of stages (K is a multiple of 128); behind the last one the first fragments are read again from
    // the other place, and not used
    for (int st = 0; st < nst; st += 2) {
        stage(st, std::integral_constant<int, 0>{});
        stage(st + 1, std::integral_constant<int, 1>{});
    }
#pragma unroll
    for (int j = 0; j < NTK; ++j) {
        const int64_t t = t0 + (wt * NTK + j) * 16 + (lane & 15);
        if (t >= a.T) continue;
#pragma unroll
        for (int i = 0; i < NF; ++i) {
            const int g = g0 + wf * NF + i;
            if (g < groups) finish4(a, acc[i][j], t, g * 16 + (lane >> 4) * 4);
        }
    }
}

template <int WF, int WT, int NF, int NTK>
hipError_t launch(const LinearCall& a, hipStream_t s) {
    constexpr int TF = WF * NF * 16, TT = WT * NTK * 16;
    const int64_t f_tiles = (a.N + TF - 1) / TF, t_tiles = ((int64_t)a.T + TT - 1) / TT;
    if (!grid_fits(f_tiles * t_tiles, WF * WT * 64)) return hipErrorInvalidConfiguration;
    k_linear_tiled<WF, WT, NF, NTK><<<(unsigned)(f_tiles * t_tiles), WF * WT * 64, 0, s>>>(a, (int)f_tiles, (int)t_tiles);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_tiled(const LinearCall& a, hipStream_t s) { return launch<2, 4, 8, 4>(a, s); }

}  // namespace rdg
