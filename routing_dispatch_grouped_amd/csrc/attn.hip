// Launches of the few-row attention (attn_rows.h), and the join of split rows.
#include "attn_rows.h"

namespace rdg {
namespace {

template <int D, int NS, int RT>
__global__ __launch_bounds__((RT * key_groups<RT>() * kWave), D < 256 && NS == 1 ? 2 : 1) void k_attn_rows(AttnCall a) {
    __shared__ __attribute__((aligned(16))) RowsLds<D, RT> lds;
    attn_rows<D, NS, RT>(a, (int)blockIdx.x, lds);
}

// The chunks of each row, joined in order: one wave per row, a workgroup's four
// waves (and blockIdx.y) taking a token's heads in turn.  Rows of requests with up to n_most queries were split by
// k_attn_rows, the others by k_attn_tiles.
constexpr int kJoinWaves = kJoinThreads / kWave;

template <int D, bool BF16>
__global__ __launch_bounds__(kJoinThreads) void k_attn_join(AttnCall a) {
    const int lane = lane_id(), t = (int)blockIdx.x;
    int r = -1;  // the last request that begins at or before the token
    for (int b = 0; b < a.R; b += kWave) r += __popcll(__ballot(b + lane < a.R && a.cu_q[b + lane] <= t));
    if (r < 0) return;
    const ReqSpan s = req_span(a, r);
    const int i = t - s.t0;
    if (i < 0 || i >= s.n) return;
    const bool few = s.n <= a.n_most;
    if ((few ? a.row_chunks : a.tile_chunks) == 1) return;
    const int per = few ? a.rows_per_tile : a.tile_rows;
    const float *part_o = few ? a.row_o : a.tile_o, *part_ml = few ? a.row_ml : a.tile_ml;
    for (int h = (int)blockIdx.y * kJoinWaves + (int)threadIdx.x / kWave; h < a.n_q; h += (int)gridDim.y * kJoinWaves) {
        const int row = i * a.group + h % a.group;
        const int row0 = row / per * per, row1 = row0 + per < s.n * a.group ? row0 + per : s.n * a.group;
        const int chunks = tile_keys(a, s, row0, row1, few ? a.chunk : a.tile_chunk).chunks;
        if (chunks == 1) continue;
        const int64_t at = few ? row_part(a, s, r, i, h) : ((int64_t)t * a.n_q + h) * a.tile_chunks;
        float top = -__builtin_inff();
        for (int c = lane; c < chunks; c += kWave) top = fmaxf(top, part_ml[2 * (at + c)]);
        top = wave_max_f32(top);
        const float ref = top == -__builtin_inff() ? 0.0f : top;
        float total = 0.0f;
        float acc[D / kWave];
#pragma unroll
        for (int e = 0; e < D / kWave; ++e) acc[e] = 0.0f;
#pragma unroll 4
        for (int c = 0; c < chunks; ++c) {
            const float2 ml = *reinterpret_cast<const float2*>(part_ml + 2 * (at + c));
            const float f = __builtin_amdgcn_exp2f(ml.x - ref);
            total = fmaf(f, ml.y, total);
#pragma unroll
            for (int e = 0; e < D / kWave; ++e) acc[e] = fmaf(f, part_o[(at + c) * D + e * kWave + lane], acc[e]);
        }
        const bool none = key_hi(a, s, i) <= key_lo(a, s, i);
        const float inv = none ? 0.0f : 1.0f / total;
        const int64_t out = (int64_t)t * a.out_stride + (int64_t)h * D;
#pragma unroll
        for (int e = 0; e < D / kWave; ++e) {
            const float v = none ? 0.0f : acc[e] * inv;
            if constexpr (BF16) static_cast<__bf16*>(a.out)[out + e * kWave + lane] = (__bf16)v;
            else static_cast<float*>(a.out)[out + e * kWave + lane] = v;
        }
        if (a.lse && lane == 0)
            a.lse[(int64_t)t * a.n_q + h] = none ? -__builtin_inff() : (top + __builtin_amdgcn_logf(total)) * kLn2;
    }
}

template <int D, int NS, int RT>
hipError_t launch_rows(const AttnCall& a, hipStream_t s) {
    constexpr int threads = RT * key_groups<RT>() * kWave;
    const int64_t grid = (int64_t)a.n_kv * row_tiles(a) * a.row_chunks;
    if (!grid_fits(grid, threads)) return hipErrorInvalidConfiguration;
    k_attn_rows<D, NS, RT><<<(unsigned)grid, threads, 0, s>>>(a);
    return hipGetLastError();
}

template <int D, int NS>
hipError_t launch_d(const AttnCall& a, int rt, hipStream_t s) {
    switch (rt) {
        case 1: return launch_rows<D, NS, 1>(a, s);
        case 2: return launch_rows<D, NS, 2>(a, s);
        case 3: return launch_rows<D, NS, 3>(a, s);
        default: return launch_rows<D, NS, 4>(a, s);
    }
}

template <int D>
hipError_t join_d(const AttnCall& a, bool bf16, hipStream_t s) {
    // many tokens fill the chip by themselves, and in a mixed batch most have nothing to join
    const int groups = (a.n_q + kJoinWaves - 1) / kJoinWaves;
    const dim3 grid(a.T, a.T >= 1024 && groups > 2 ? 2 : groups);
    if (bf16) k_attn_join<D, true><<<grid, kJoinThreads, 0, s>>>(a);
    else k_attn_join<D, false><<<grid, kJoinThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_rows(const AttnCall& a, int head_dim, bool bf16, hipStream_t s) {
    const int rt = a.rows_per_tile / 16;
    switch (head_dim) {
        case 64: return bf16 ? launch_d<64, 1>(a, rt, s) : launch_d<64, 3>(a, rt, s);
        case 128: return bf16 ? launch_d<128, 1>(a, rt, s) : launch_d<128, 3>(a, rt, s);
        default: return bf16 ? launch_d<256, 1>(a, rt, s) : launch_d<256, 3>(a, rt, s);
    }
}

hipError_t launch_attn_join(const AttnCall& a, int head_dim, bool bf16, hipStream_t s) {
    switch (head_dim) {
        case 64: return join_d<64>(a, bf16, s);
        case 128: return join_d<128>(a, bf16, s);
        default: return join_d<256>(a, bf16, s);
    }
}

}  // namespace rdg
