// Routing to experts by softmax or sigmoid scores: optional selection bias, groups
// ranked by their best expert or the sum of their two best, top-K, weights
// renormalised or as they are.
//
//   p_e = exp(l_e - max l) / sum_e exp(l_e - max l)   or   1 / (1 + exp(-l_e))
//   c_e = p_e + bias_e                                (the choice; p_e without a bias)
//   keep the topk_group groups of the largest best c (or sum of the two best), then the K
//   largest c among their experts; ties to the lower index
//   w_k = p / (sum of the K chosen p) * scale, or p * scale
//
// p is computed in fp64 and rounded once to fp32, so that which of two near
// scores is larger does not depend on how a sum was ordered; c, the groups' sums
// and the weights are fp32.
//
// Bound by latency and the vector unit: a row is at most 4 KiB.  A token has
// SEG lanes (8, 16, 32 or 64, the fewest that hold its experts one each), so
// that few experts do not leave most of a wave idle, and VPL experts a lane
// from 65 experts on: expert e on lane e % 64.  Each of the K rounds is a maximum of
// ordered score bits across the token's lanes in the vector unit, and a ballot
// for the lowest expert that holds it.
#include "score.h"
#include "vec8.h"

#pragma clang fp contract(off)

namespace rdg {
namespace {

constexpr int kThreads = 256;

template <int SEG, int VPL>
__global__ __launch_bounds__(kThreads) void k_route_topk(RouteCall a) {
    constexpr int PER = kThreads / SEG;  // tokens a workgroup
    static_assert(VPL == 1 || SEG == kWave, "several experts a lane only in whole waves");
    __shared__ float choice_lds[PER][SEG * VPL];
    __shared__ float plain_lds[PER][SEG * VPL];
    __shared__ float rank_lds[PER][SEG * VPL];
    const int slot = threadIdx.x / SEG, sub = threadIdx.x % SEG, first = lane_id() / SEG * SEG;
    // past the last token: the last one again, not stored (the exchanges take every lane of the wave)
    const int64_t at = (int64_t)blockIdx.x * PER + slot;
    const bool live = at < a.B;
    const int64_t t = live ? at : a.B - 1;
    float* ch = choice_lds[slot];
    float* pl = plain_lds[slot];

    // NaN counts as -inf, +inf as the largest finite value
    float x[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = sub + SEG * v;
        x[v] = -__builtin_inff();
        if (e < a.N) {
            const int64_t i = t * a.stride + e;
            const float l = a.bf16 ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[i]) : static_cast<const float*>(a.logits)[i];
            x[v] = l != l ? -__builtin_inff() : fminf(l, 3.402823466e38f);
        }
    }
    float p[VPL];
    if (a.softmax) {
        float top = x[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) top = fmaxf(top, x[v]);
        top = across<SEG>(top, [](float q, float r) { return fmaxf(q, r); });
        double e[VPL], sum = 0.0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            // a row of nothing but -inf has no scores: all 0
            e[v] = x[v] == -__builtin_inff() ? 0.0 : exp64(fmax((double)x[v] - (double)top, -800.0));
            sum += e[v];
        }
        sum = across<SEG>(sum, [](double q, double r) { return q + r; });
#pragma unroll
        for (int v = 0; v < VPL; ++v) p[v] = sum > 0.0 ? (float)(e[v] / sum) : 0.0f;
    } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) p[v] = score_sigmoid(x[v]);
    }

    uint32_t key[VPL];  // 0: no candidate (any longer)
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = sub + SEG * v;
        float c = p[v];
        if (a.bias != nullptr && e < a.N) {
            c += a.bias[e];
            if (c != c) c = -__builtin_inff();
            pl[e] = p[v];
        }
        key[v] = e < a.N ? ordered_bits(c) : 0u;
        if (a.n_group > 1 && e < a.N) ch[e] = c;
    }
    if (a.n_group > 1) {
        const int gs = a.N / a.n_group;
        float* rank = rank_lds[slot];
        __syncthreads();
        for (int g = sub; g < a.n_group; g += SEG) {
            float best = -__builtin_inff(), next = best;
            for (int i = g * gs; i < (g + 1) * gs; ++i) {
                const float c = ch[i];
                next = fmaxf(next, fminf(best, c));
                best = fmaxf(best, c);
            }
            rank[g] = a.group_best == 2 && gs >= 2 ? best + next : best;
        }
        __syncthreads();
        // kept: fewer than topk_group groups are better (larger, or as large with a lower index)
        for (int g = sub; g < a.n_group; g += SEG) {
            const uint32_t mine = ordered_bits(rank[g]);
            int better = 0;
            for (int h = 0; h < a.n_group; ++h) {
                const uint32_t other = ordered_bits(rank[h]);
                better += other > mine || (other == mine && h < g);
            }
            ch[g] = better < a.topk_group ? 1.0f : 0.0f;  // the choices are in registers
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = sub + SEG * v;
            if (e < a.N && ch[e / gs] == 0.0f) key[v] = 0u;
        }
    } else if (a.bias != nullptr) {
        __syncthreads();
    }

    const uint64_t seg_mask = SEG == 64 ? ~0ull : ((1ull << (SEG & 63)) - 1) << first;
    float sum = 0.0f, my_p = 0.0f;
    int my_id = 0;
    for (int k = 0; k < a.K; ++k) {
        uint32_t m = key[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) m = key[v] > m ? key[v] : m;
        m = across<SEG>(m, [](uint32_t q, uint32_t r) { return q > r ? q : r; });
        int e = -1;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const uint64_t have = __ballot(key[v] == m) & seg_mask;
            if (e < 0 && have != 0) e = __ffsll((unsigned long long)have) - 1 - first + SEG * v;
        }
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (sub + SEG * v == e) key[v] = 0u;
        // without a bias the choice is the score: back from its ordered bits
        const float pe = a.bias != nullptr ? pl[e] : __uint_as_float(m & 0x7fffffffu);
        sum += pe;
        if (sub == k) my_id = e, my_p = pe;
    }
    if (live && sub < a.K) {
        const float w = !a.renorm ? my_p : sum > 0.0f ? my_p / sum : 0.0f;
        a.ids[t * a.K + sub] = my_id;
        a.w[t * a.K + sub] = w * a.scale;
    }
}

template <int SEG, int VPL>
hipError_t launch(const RouteCall& a, hipStream_t s) {
    constexpr int PER = kThreads / SEG;
    const int64_t blocks = ((int64_t)a.B + PER - 1) / PER;
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    k_route_topk<SEG, VPL><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route_topk(const RouteCall& a, hipStream_t s) {
    if (a.B == 0) return hipSuccess;
    // a lane holds the K-th choice until the end, so the lanes are no fewer than K (K <= N)
    if (a.N <= 8) return launch<8, 1>(a, s);
    if (a.N <= 16) return launch<16, 1>(a, s);
    if (a.N <= 32) return launch<32, 1>(a, s);
    if (a.N <= 64) return launch<64, 1>(a, s);
    if (a.N <= 128) return launch<64, 2>(a, s);
    if (a.N <= 256) return launch<64, 4>(a, s);
    if (a.N <= 512) return launch<64, 8>(a, s);
    return launch<64, 16>(a, s);
}

}  // namespace rdg
