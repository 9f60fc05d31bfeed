// Matrix product with bias, activation and residual in its epilogue:
//
//   out[t, f] = act(sum_k x[t, k] W[f, k] + bias[f]) + residual[t, f]
//
// products summed in fp32; fp8 partial sums of 128 are scaled by their
// activation and weight block scales in fp32; one rounding at the end.
//
// Here: which kernel runs, and the kernel for few tokens, bound by reading the weights.
// (linear_tiled.hip: for more tokens.)
#include <type_traits>

#include "linear.h"

namespace rdg {
namespace {

// A workgroup has 16 weight rows and 16 tokens; its waves take the reduction's 128-element blocks
// in turn (wave w blocks w, w + NW, ...), so that the weights stream through in order, and add their sums in LDS in wave
// order.  One token, 10240 features of K = 7168 in bf16: 25.0 to 26.6 us with the weights from memory (5.5 to 5.9 TB/s), 23.1 to
// 25.6 with the same 147 MB over again, some of which the last cache holds.  Over again: 24.6 with 16 waves, 25.4 with 4 or 8, 28
// with two weight tiles a wave; 16 tokens on 256 features of K = 4096: 7.9 us against 10.9.  Loading the next block
// during the products, 24.1 us at 16 waves for twice the registers, gained nothing elsewhere.
// A token tile's loads touch 16 rows, so their time grows with the tokens: rows_us below.
// e4m3 products are taken from bf16 operands (LinOp::mma_wide): one token on 18432 features of K = 7168 takes 21.7 us either
// way, eight tokens 24.7 and 24.6.
constexpr int NW = 16;

template <int DT>
__global__ __launch_bounds__(NW * 64) void k_linear_rows(LinearCall a) {
    using O = LinOp<DT>;
    using op_t = typename O::op_t;
    constexpr int STEPS = 128 / O::KS, U = STEPS > 4 ? 8 : STEPS;  // matrix steps of a block, and those in flight
    constexpr bool FP8 = DT == RDG_FP8_E4M3;
    __shared__ f32x4_t part[NW][kWave];
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
    const int nkb = a.K / 128;
    // XCD b % 8 takes a contiguous share; the token tiles of 16 weight rows lie together in it
    const int t_tiles = (int)(((int64_t)a.T + 15) / 16);
    const int n = gridDim.x, xcd = blockIdx.x % 8, q8 = n / 8, r8 = n % 8;
    const int item = xcd * q8 + (xcd < r8 ? xcd : r8) + blockIdx.x / 8;
    const int group = item / t_tiles;
    const int64_t t0 = (int64_t)(item % t_tiles) * 16;
    const uint8_t* w = static_cast<const uint8_t*>(a.w) + (int64_t)group * (a.K / O::KS) * O::BLK;
    // tokens past the last: the last one again, not stored
    const int64_t mine = t0 + (lane & 15), t = mine < a.T ? mine : a.T - 1;
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + t * a.x_stride * O::ESZ;
    const float* ws = FP8 ? a.w_scales + (int64_t)(group / 8) * nkb : nullptr;
    const float* xs = FP8 ? a.x_scales + t * nkb : nullptr;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    auto walk = [&](auto once) {
        for (int kb = wv; kb < nkb; kb += NW) {
#pragma unroll
            for (int s0 = 0; s0 < STEPS; s0 += U) {
                op_t rw[U], rx[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t step = (int64_t)kb * STEPS + s0 + u;
                    if constexpr (decltype(once)::value) rw[u] = O::stream_w(w + step * O::BLK, lane);
                    else rw[u] = O::load_w(w + step * O::BLK, lane);
                    rx[u] = O::load_x(x, (int)step * O::KS, lane);
                }
                if constexpr (FP8) {
                    const float scale = xs[kb] * ws[kb];
                    const f32x4_t z = {0.f, 0.f, 0.f, 0.f};
                    acc += O::mma_wide(z, rw[0], rx[0]) * scale;
                } else {
#pragma unroll
                    for (int u = 0; u < U; ++u) acc = O::mma(acc, rw[u], rx[u]);
                }
            }
        }
    };
    // weights that no other workgroup reads stream past the caches
    if (t_tiles == 1) walk(std::true_type{});
    else walk(std::false_type{});
    part[wv][lane] = acc;
    __syncthreads();
    // lane l of a 16 x 16 tile: token l % 16, features 4 (l / 16) .. + 3
    if (wv != 0 || mine >= a.T) return;
    f32x4_t v = part[0][lane];
#pragma unroll
    for (int u = 1; u < NW; ++u) v += part[u][lane];
    finish4(a, v, mine, group * 16 + (lane >> 4) * 4);
}

template <int DT>
hipError_t launch_rows(const LinearCall& a, hipStream_t s) {
    const int64_t blocks = (int64_t)(a.N / 16) * (((int64_t)a.T + 15) / 16);
    if (!grid_fits(blocks, NW * 64)) return hipErrorInvalidConfiguration;
    k_linear_rows<DT><<<(unsigned)blocks, NW * 64, 0, s>>>(a);
    return hipGetLastError();
}

// ---------------------------------------------------------------- which kernel
// The expected time of each kernel and split in us, and the least of them.  Constants measured over 461 sizes each of
// bf16 and of fp8 (1 .. 5000 tokens, 64 .. 32768 features, K of 256 .. 14336, weights from memory), before the join asked for all
// splits at once and 16 splits came; the choice took on average 1% longer than the best of all at each size, 1.23 times at
// worst (64 tokens, 2048 features, K = 7168, bf16: 13.5 us).  With both, at 25 sizes of up to 32 tokens and 48 of up to 1250,
// all three types: 8% longer at worst (16 tokens, 7168 features, K = 2048, bf16: 9.7 us, k_linear_rows 9.0; 182 tokens, 192
// features, K = 11648: 10.0, 64 x 32 with 8 splits 9.3), 2% or less at all but four.
// e4m3 to fp32 is planned with the costs of e4m3 to bf16, whose products take half the time.
constexpr int kCus = 256;
constexpr float kStart = 2.0f, kMore = 1.5f;            // launch, first loads, last stores; one launch more
constexpr float kRowsRead = 6.7e6f, kTilesRead = 7.5e6f;  // bytes/us at which weights come from memory
constexpr float kJoin = 3.0f, kJoinRate = 3.6e6f;       // the join's launch; splits' sums, written and read
// With few tokens a stage takes the time in which a CU gets its 128-byte lines: it has some 500 of them under way at
// a time, for a latency that grows with the weights under way on the whole chip.  So the tile is best whose workgroups
// just fill the CUs: 64 tokens, 18432 features, K = 7168 in bf16, of 128 features on 144 CUs 60.4 us, of 80 on 231
// 49.6; 16384 features in e8m0, of 128 35.4 us, of 64 28.3.  Weights that pass the caches
// (k_linear_tiled's ONCE) take less.
constexpr int kFewTokens = 160;
constexpr float kLine = 0.00168f, kUnderWay = 8.0e-6f;  // us a line; us a feature of the tile and workgroup of the chip
constexpr float kLineOnce = 0.0015f, kUnderWayOnce = 7.9e-6f;
constexpr float kFewFp8 = 0.045f, kFewFp8Once = 0.03f;  // the scales' lines

struct TileCost {
    int kernel, features, tokens;
    int per_cu;           // workgroups a CU holds (LDS)
    float alone, loaded;  // us a stage of 128 bytes of each row and workgroup: one round of workgroups, and more
    float tile;           // us a tile besides
};
// 256 x 256 is bound by the matrix core; the smaller the tile, the more bytes it loads for its products, and the less
// of the chip a small problem leaves idle.
constexpr TileCost kBf16Cost[] = {{kTile256, 256, 256, 1, 1.2f, 1.4f, 6.0f},      {kTile128, 128, 128, 1, 0.383f, 0.5f, 1.9f},
                                  {kTile128x64, 128, 64, 1, 0.275f, 0.36f, 1.95f}, {kTile64x32, 64, 32, 3, 0.141f, 0.135f, 0.93f},
                                  {kTile96x64, 96, 64, 1, 0.23f, 0.34f, 1.5f},    {kTile80x64, 80, 64, 1, 0.21f, 0.27f, 1.2f},
                                  {kTile64x64, 64, 64, 1, 0.18f, 0.22f, 1.3f}};
constexpr TileCost kFp8Cost[] = {{kTile256, 256, 256, 1, 1.3f, 1.5f, 7.0f},       {kTile128, 128, 128, 1, 0.596f, 0.63f, 2.25f},
                                 {kTile128x64, 128, 64, 1, 0.417f, 0.40f, 1.6f},  {kTile64x32, 64, 32, 3, 0.236f, 0.178f, 1.0f},
                                 {kTile96x64, 96, 64, 1, 0.42f, 0.45f, 2.2f},     {kTile80x64, 80, 64, 1, 0.38f, 0.40f, 2.15f},
                                 {kTile64x64, 64, 64, 1, 0.362f, 0.34f, 1.8f}};
constexpr TileCost kF32Cost[] = {{kTile128, 128, 128, 1, 1.92f, 1.92f, 2.0f},
                                 {kTile128x64, 128, 64, 1, 1.08f, 1.08f, 1.3f},
                                 {kTile64x32, 64, 32, 3, 0.39f, 0.30f, 0.8f}};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int size_of(int dtype) { return dtype == RDG_F32 ? 4 : dtype == RDG_BF16 ? 2 : 1; }

// A wave's 2048 elements (16 waves of 128) take a time that grows with the tokens of its tile; or the weights' reading and
// a round's start.
float rows_us(int T, int N, int K, int dtype) {
    const float per = dtype == RDG_F32 ? 5.0f : dtype == RDG_BF16 ? 1.5f : 0.48f;
    const float token = dtype == RDG_F32 ? 0.6f : dtype == RDG_BF16 ? 0.125f : 0.106f;
    const int64_t rounds = ceil_div((int64_t)(N / 16) * ceil_div(T, 16), kCus);
    const float us = K / 2048.0f * (per + token * (T < 16 ? T : 16)) * rounds;
    const float read_us = (float)N * K * size_of(dtype) / kRowsRead + 0.33f * rounds;
    return kStart + 0.3f + (us > read_us ? us : read_us);
}

float tiles_us(const TileCost& c, int splits, int T, int N, int K, int dtype) {
    const int stages = (int)ceil_div(K / 128, splits) * size_of(dtype);
    const int64_t f_jobs = ceil_div(N, c.features) * splits, rounds = ceil_div(f_jobs * ceil_div(T, c.tokens), kCus);
    const int64_t full = rounds / c.per_cu, rest = rounds % c.per_cu;
    auto round_us = [&](int64_t workgroups) {
        const float loaded = c.loaded * workgroups;
        float stage = rounds == 1 || loaded < c.alone ? c.alone : loaded;
        if (T <= kFewTokens && dtype != RDG_F32) {
            // (a token past the last costs half a line)
            const float lines = workgroups * (c.features + (c.tokens + (T < c.tokens ? T : c.tokens)) * 0.5f);
            const int64_t chip = kCus * workgroups;
            const bool once = T <= c.tokens && c.tokens <= 64;
            const float under_way = (float)c.features * (f_jobs < chip ? f_jobs : chip);
            const float few = lines * (once ? kLineOnce : kLine) + under_way * (once ? kUnderWayOnce : kUnderWay) +
                              (dtype == RDG_BF16 ? 0.0f : once ? kFewFp8Once : kFewFp8);
            stage = stage > few ? stage : few;
        }
        return stages * stage + c.tile;
    };
    const float us = full * round_us(c.per_cu) + (rest ? round_us(rest) : 0.0f);
    const float read_us = (float)N * K * size_of(dtype) / kTilesRead;
    return kStart + (us > read_us ? us : read_us) + (splits > 1 ? kJoin + (float)splits * T * N * 8 / kJoinRate : 0.0f);
}

const TileCost* costs(int dtype, int& kinds) {
    kinds = dtype == RDG_F32 ? 3 : 7;
    return dtype == RDG_F32 ? kF32Cost : dtype == RDG_BF16 ? kBf16Cost : kFp8Cost;
}

// The most tiles whose reduction is split so often, which also bounds the workspace: 256 MiB.  (16 splits beyond one round:
// 128 x 512 x 7168 fp8 9.8 us, 8 8.6; within one 64 x 256 x 14336 bf16 9.2 and 10.9.)
constexpr int kMostSplits = 16;
constexpr int most_tiles(int splits) { return (splits > 8 ? kCus : 4 * kCus) / splits; }

// One kernel for all features.
LinearPart plan_part(int T, int N, int K, int dtype, float& least) {
    int kinds;
    const TileCost* cost = costs(dtype, kinds);
    LinearPart best{kRows, 1, N};
    // (Beyond 32 tokens the tiles are always faster.)  At near equal times the rows, one launch that needs no workspace.
    // us from memory, and over again, for the rows and for the best of the tiles:
    //   bf16  1 x 10240 x 7168  25.3, 24.8  27.4, 26.1     4 x 10240 x 7168  27.5, 26.1  27.4, 26.1
    //         1 x  7168 x 8192  21.4, 20.0  22.0, 20.8     2 x  1536 x 7168   8.3,  7.4   8.6,  8.3
    //   e8m0  8 x 18432 x 7168  24.2, 23.5  25.6, 24.9     1 x  7168 x 18432 22.9, 20.8  24.9, 23.5
    //   fp32  1 x  7168 x 2048  16.0, 14.1  16.5, 15.4
    least = T <= 32 ? 0.97f * rows_us(T, N, K, dtype) : 3e38f;
    for (int i = 0; i < kinds; ++i) {
        const int64_t tiles = ceil_div(N, cost[i].features) * ceil_div(T, cost[i].tokens);
        for (int splits = 1; splits <= kMostSplits && splits <= K / 128; splits *= 2) {
            if (splits > 1 && tiles > most_tiles(splits)) break;
            const float us = tiles_us(cost[i], splits, T, N, K, dtype);
            if (us < least) least = us, best = LinearPart{cost[i].kernel, splits, N};
        }
    }
    return best;
}

hipError_t launch_part(const LinearCall& a, const LinearPart& p, hipStream_t s) {
    // the tiles address their token rows (at most 256) and their scales with 32 bits
    const bool near = a.x_stride * size_of(a.dtype) * 256 < (int64_t)1 << 31;
    if (p.kernel != kRows && near) return launch_linear_tiled(a, p, s);
    switch (a.dtype) {
        case RDG_F32: return launch_rows<RDG_F32>(a, s);
        case RDG_BF16: return launch_rows<RDG_BF16>(a, s);
        default: return launch_rows<RDG_FP8_E4M3>(a, s);
    }
}

size_t part_bytes(const LinearPart& p, int T) { return p.splits > 1 ? (size_t)p.splits * T * p.features * 4 : 0; }

}  // namespace

// Two where the last round of 256 x 256 tiles would leave much of the chip idle: whole rounds of them, and smaller tiles or
// splits for the features behind.  bf16, 8192 x 7168 x 8192 (3.5 rounds) 686 us against 707; 2048 x 9216 x 7168
// (1.1 rounds) 196 against 276.
LinearPlan linear_plan(int T, int N, int K, int dtype) {
    float least, rest_us;
    LinearPlan p{plan_part(T, N, K, dtype, least), LinearPart{kRows, 1, 0}};
    if (dtype == RDG_F32) return p;
    const int64_t t_tiles = ceil_div(T, 256), rounds = ceil_div(N, 256) * t_tiles / kCus;
    const int64_t features = rounds * kCus / t_tiles * 256;
    if (features == 0 || features >= N) return p;
    const TileCost& c = dtype == RDG_BF16 ? kBf16Cost[0] : kFp8Cost[0];
    const LinearPart rest = plan_part(T, N - (int)features, K, dtype, rest_us);
    if (tiles_us(c, 1, T, (int)features, K, dtype) + rest_us + kMore - kStart < least)
        p = LinearPlan{LinearPart{kTile256, 1, (int)features}, rest};
    return p;
}

hipError_t launch_linear(const LinearCall& a, const LinearPlan& p, hipStream_t s) {
    LinearCall b = a;
    b.N = p.first.features;
    hipError_t err = launch_part(b, p.first, s);
    if (err != hipSuccess || p.rest.features == 0) return err;
    // the features behind: a multiple of 256 of them are done
    const int64_t n = b.N;
    const int osz = a.out_bf16 ? 2 : 4;
    b.N = p.rest.features;
    b.w = static_cast<const uint8_t*>(a.w) + n * a.K * size_of(a.dtype);
    b.out = static_cast<uint8_t*>(a.out) + n * osz;
    if (a.w_scales) b.w_scales = a.w_scales + n / 128 * (a.K / 128);
    if (a.bias) b.bias = a.bias + n;
    if (a.residual) b.residual = static_cast<const uint8_t*>(a.residual) + n * osz;
    return launch_part(b, p.rest, s);
}

size_t linear_work_bytes(const LinearPlan& p, int T) {
    // the parts' launches run one after the other, and only the second has splits
    const size_t first = part_bytes(p.first, T), rest = part_bytes(p.rest, T);
    return first > rest ? first : rest;
}

// Of every kind of tile and number of splits the outputs of the most tiles that may have so many, but no more than there are.
size_t linear_work_bound(int T, int N, int K, int dtype) {
    int kinds;
    const TileCost* cost = costs(dtype, kinds);
    int64_t most = 0;
    for (int i = 0; i < kinds; ++i)
        for (int splits = 2; splits <= kMostSplits && splits <= K / 128; splits *= 2) {
            const int64_t held = (int64_t)most_tiles(splits) * cost[i].features * cost[i].tokens, outputs = (int64_t)T * N;
            const int64_t bytes = 4 * splits * (held < outputs ? held : outputs);
            most = most > bytes ? most : bytes;
        }
    return (size_t)most;
}

}  // namespace rdg
