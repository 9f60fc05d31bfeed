// Group-limited top-k gating, one wavefront per token.
//
// What it computes (DeepEP deep-dive, section on DeepSeek-V3's
// group-limited gating: the router keeps the best expert groups first and
// then the top-K experts inside them; same page, EP section: the token's
// output is the routing-weighted sum over its K experts).  Scores are
// sigmoids of the logits, a group's score is the sum of its two best scores,
// the K weights are renormalised to sum to `scale`, and every tie goes to the
// lower index.
//
// With a selection bias (a variant not on the pages: a per-expert correction
// added for the choice only), groups and experts are chosen by the fp32 sums
// score + bias, and the weights still renormalise the plain scores.
//
// Design for CDNA4: a token's N <= 1024 choosing scores sit in LDS (one
// wave's private slice) and in registers (N/64 per lane, expert e on lane
// e % 64).  Group g's score is computed by lane g % 64; each of the
// topk_group + K selection rounds is one 64-lane max-reduction of a 64-bit
// key (ordered score bits << 32 | ~index) -- the fp32 bits mapped so that
// unsigned order is numeric order, and ~index makes the lower index win a
// tie.
#include "vec8.h"

#pragma clang fp contract(off)

namespace rdg {
namespace {

// The score: sigmoid in fp64, rounded once to fp32.  Every step is one IEEE
// double operation so the value is identical wherever it is evaluated:
//   x clamped to [-87, 87]; z = -x; n = rint(z * log2(e));
//   r = z - n*ln2 with ln 2 split in a 42-bit head (exact products) and a tail;
//   e^r by its degree-13 Taylor series (Horner, fma, 1/k! rounded to double);
//   e^z = e^r * 2^n exactly; score = (float)(1 / (1 + e^z)).
// The truncation error of the series for |r| <= ln2/2 is below 2^-55.
constexpr double kLog2e = 0x1.71547652b82fep+0;   // double nearest 1/ln 2
constexpr double kLn2Hi = 0x1.62e42fefa3800p-1;   // double ln 2, 42 significant bits
constexpr double kLn2Lo = 0x1.ef00000000000p-45;  // double ln 2 minus the head
constexpr double kInvFact[14] = {
    0x1.0000000000000p+0,  0x1.0000000000000p+0,  0x1.0000000000000p-1,  0x1.5555555555555p-3,
    0x1.5555555555555p-5,  0x1.1111111111111p-7,  0x1.6c16c16c16c17p-10, 0x1.a01a01a01a01ap-13,
    0x1.a01a01a01a01ap-16, 0x1.71de3a556c734p-19, 0x1.27e4fb7789f5cp-22, 0x1.ae64567f544e4p-26,
    0x1.1eed8eff8d898p-29, 0x1.6124613a86d09p-33};

// e^z for z in [-800, 87] (0 below what fp64 holds).
__device__ __forceinline__ double exp64(double z) {
    double n = __builtin_rint(z * kLog2e);
    double r = __builtin_fma(-n, kLn2Hi, z);
    r = __builtin_fma(-n, kLn2Lo, r);
    double p = kInvFact[13];
#pragma unroll
    for (int k = 12; k >= 0; --k) p = __builtin_fma(p, r, kInvFact[k]);
    return __builtin_ldexp(p, (int)n);
}

__device__ __forceinline__ float score_sigmoid(float xf) {
    xf = fminf(fmaxf(xf, -87.0f), 87.0f);
    return (float)(1.0 / (1.0 + exp64(-(double)xf)));
}

// fp32 -> uint32 whose unsigned order is the numeric order (negative values
// have every bit flipped, non-negative ones the sign bit); never 0 for a
// finite value
__device__ __forceinline__ uint32_t ordered_bits(float v) {
    const uint32_t u = __float_as_uint(v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint64_t make_key(float score, int idx) {
    return ((uint64_t)ordered_bits(score) << 32) | (uint32_t)(0xffffffffu - (uint32_t)idx);
}
__device__ __forceinline__ int key_index(uint64_t key) { return (int)(0xffffffffu - (uint32_t)key); }

template <int VPL>
__global__ __launch_bounds__(256) void k_route(const float* __restrict__ logits, const float* __restrict__ bias,
                                               int B, int N, int n_group, int topk_group, int K, float scale,
                                               int32_t* __restrict__ ids, float* __restrict__ w) {
    __shared__ float lds[4][64 * VPL];   // choosing scores
    __shared__ float plain_lds[4][64 * VPL];  // plain scores (weights), with a bias
    __shared__ uint8_t gsel_lds[4][64 * VPL];
    const int wv = threadIdx.x / kWave, lane = lane_id();
    const int t = blockIdx.x * 4 + wv;
    if (t >= B) return;  // the wave is idle; nothing below synchronises across waves
    float* s_lds = lds[wv];
    float* p_lds = plain_lds[wv];
    const float* row = logits + (size_t)t * N;

    float s[VPL];  // choosing scores
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        int e = lane + kWave * v;
        const float plain = e < N ? score_sigmoid(row[e]) : 0.0f;
        s[v] = bias && e < N ? plain + bias[e] : plain;
        if (e < N) {
            s_lds[e] = s[v];
            if (bias) p_lds[e] = plain;
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");

    // group score: sum of the group's two largest scores (with multiplicity);
    // lane l owns groups l, l+64, ... (n_group <= N <= 64*VPL, so VPL slots suffice)
    const int gs = N / n_group;
    uint64_t gkey[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int g = lane + kWave * j;
        gkey[j] = 0ull;
        if (g < n_group) {
            float a = -__builtin_inff(), b = -__builtin_inff();
            for (int i = g * gs; i < (g + 1) * gs; ++i) {
                const float v = s_lds[i];
                if (v > a) {
                    b = a;
                    a = v;
                } else if (v > b) {
                    b = v;
                }
            }
            gkey[j] = make_key(gs >= 2 ? a + b : a, g);
        }
    }
    // keep topk_group groups; the kept set is a byte per group in LDS
    uint8_t* gsel = gsel_lds[wv];
    for (int g = lane; g < n_group; g += kWave) gsel[g] = 0;
    for (int r = 0; r < topk_group; ++r) {
        uint64_t best = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) best = gkey[j] > best ? gkey[j] : best;
        const int g = key_index(wave_max_u64(best));
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (lane + kWave * j == g) gkey[j] = 0ull;
        if (lane == 0) gsel[g] = 1;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    // top-K experts of the kept groups
    uint64_t key[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        int e = lane + kWave * v;
        bool cand = e < N && gsel[e / gs];
        key[v] = cand ? make_key(s[v], e) : 0ull;
    }
    float my_s = 0.0f;
    int my_id = 0;
    for (int k = 0; k < K; ++k) {
        uint64_t best = 0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) best = key[v] > best ? key[v] : best;
        uint64_t m = wave_max_u64(best);
        int e = key_index(m);
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (lane + kWave * v == e) key[v] = 0ull;
        if (lane == k) my_id = e;
    }
    // renormalise the plain scores: fp32 sum in slot order, then
    // w_k = s_k / sum * scale
    if (lane < K) my_s = bias ? p_lds[my_id] : s_lds[my_id];
    float sum = 0.0f;
    for (int k = 0; k < K; ++k) sum += __shfl(my_s, k);
    if (lane < K) {
        ids[(size_t)t * K + lane] = my_id;
        w[(size_t)t * K + lane] = (my_s / sum) * scale;
    }
}

// ---------------------------------------------------------------------------
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
// Bound by the vector unit for many tokens: the fp64 exponentials, and the rounds in which one
// expert after the other is taken.  Up to 32 experts a token has SEG lanes (8, 16 or 32, the fewest that
// hold its experts one each); beyond, a wave with VPL experts a lane, expert e on lane e % 64.
// A round is a maximum of ordered score bits across the token's lanes, in the vector unit, and a ballot for
// the lowest expert that holds it.
//
// Measured: 16384 tokens of 160 experts, 3 of 8 groups, 6 chosen 15.6 us; of 256 experts, 8 chosen 13.7; sigmoid, 4 of 8
// groups by their two best, biased 19.2 (k_route 40.4); 32768 tokens of 8 experts 3.0; 128 of 256 4.0.
constexpr int kTopkThreads = 256;

// The logits of token t that lane `first` of STEP lanes holds, -inf past the last; NaN counts as -inf, +inf as the
// largest finite value.  All are requested before the first is looked at.
template <int STEP, int VPL>
__device__ __forceinline__ void topk_logits(const RouteCall& a, int64_t t, int first, float (&x)[VPL]) {
    uint32_t u[VPL];
    if (a.bf16) {
        const uint16_t* row = static_cast<const uint16_t*>(a.logits) + t * a.stride;
#pragma unroll
        for (int v = 0; v < VPL; ++v) u[v] = row[first + STEP * v < a.N ? first + STEP * v : a.N - 1];
#pragma unroll
        for (int v = 0; v < VPL; ++v) u[v] <<= 16;
    } else {
        const uint32_t* row = static_cast<const uint32_t*>(a.logits) + t * a.stride;
#pragma unroll
        for (int v = 0; v < VPL; ++v) u[v] = row[first + STEP * v < a.N ? first + STEP * v : a.N - 1];
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const float l = __uint_as_float(u[v]);
        x[v] = first + STEP * v < a.N && l == l ? fminf(l, 3.402823466e38f) : -__builtin_inff();
    }
}

// The scores of a token's logits, spread over LANES lanes.
template <int LANES, int VPL>
__device__ __forceinline__ void topk_scores(bool softmax, const float (&x)[VPL], float (&p)[VPL]) {
    if (!softmax) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) p[v] = score_sigmoid(x[v]);
        return;
    }
    float top = x[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v) top = fmaxf(top, x[v]);
    top = across<LANES>(top, [](float q, float r) { return fmaxf(q, r); });
    // a row of nothing but -inf has no scores: exp(-inf) everywhere
    const double shift = fmaxf(top, -3.402823466e38f);
    double e[VPL], sum = 0.0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        e[v] = exp64(__builtin_fmax((double)x[v] - shift, -800.0));
        sum += e[v];
    }
    sum = across<LANES>(sum, [](double q, double r) { return q + r; });
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) p[v] = (float)(e[v] * inv);
}

__device__ __forceinline__ uint32_t topk_key(float c) { return ordered_bits(c == c ? c : -__builtin_inff()); }
__device__ __forceinline__ float topk_value(uint32_t key) {  // of a key that is not 0
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// The largest of the wave's values, in a scalar register: each row of 16 shifted over itself, then row by row
// into the last lane.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x) {
    auto with = [&](uint32_t y) { x = y > x ? y : x; };
    with(lane_of<0x111>(x));  // row_shr:1, 0 comes in
    with(lane_of<0x112>(x));
    with(lane_of<0x114>(x));
    with(lane_of<0x118>(x));
    with(lane_of<0x142>(x));  // row_bcast:15
    with(lane_of<0x143>(x));  // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)x, kWave - 1);
}

__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ void topk_store(const RouteCall& a, int64_t t, int k, int id, float p, float sum) {
    const float w = !a.renorm ? p : sum > 0.0f ? p / sum : 0.0f;
    a.ids[t * a.K + k] = id;
    a.w[t * a.K + k] = w * a.scale;
}

// A group's rank from its two largest choices; +inf and -inf together count as the larger.
__device__ __forceinline__ float group_rank(const RouteCall& a, int gs, float best, float next) {
    const float sum = best + next;
    return a.group_best == 2 && gs >= 2 && sum == sum ? sum : best;
}

// Up to 32 experts: SEG lanes a token.
template <int SEG>
__global__ __launch_bounds__(kTopkThreads) void k_route_few(RouteCall a) {
    constexpr int PER = kTopkThreads / SEG;  // tokens a workgroup
    __shared__ float choice_lds[PER][SEG], plain_lds[PER][SEG], rank_lds[PER][SEG];
    const int slot = threadIdx.x / SEG, sub = threadIdx.x % SEG, first = lane_id() / SEG * SEG;
    // past the last token: the last one again, not stored (the exchanges take every lane of the wave)
    const int64_t at = (int64_t)blockIdx.x * PER + slot;
    const bool live = at < a.B, mine = sub < a.N;
    const int64_t t = live ? at : a.B - 1;
    float* pl = plain_lds[slot];
    float x[1], p[1];
    topk_logits<SEG>(a, t, sub, x);
    topk_scores<SEG>(a.softmax, x, p);
    float c = p[0];
    if (a.bias != nullptr && mine) {
        c += a.bias[sub];
        pl[sub] = p[0];
    }
    uint32_t key = mine ? topk_key(c) : 0u;  // 0: no candidate (any longer)
    if (a.n_group > 1) {
        // group `sub`: its rank; kept where fewer than topk_group groups are better (larger, or as large with a lower index)
        const int gs = a.N / a.n_group;
        float* ch = choice_lds[slot];
        float* rank = rank_lds[slot];
        if (mine) ch[sub] = topk_value(key);
        wave_lds_fence();
        uint32_t own = 0u;
        if (sub < a.n_group) {
            float best = -__builtin_inff(), next = best;
            for (int i = sub * gs; i < (sub + 1) * gs; ++i) {
                next = fmaxf(next, fminf(best, ch[i]));
                best = fmaxf(best, ch[i]);
            }
            rank[sub] = group_rank(a, gs, best, next);
            own = ordered_bits(rank[sub]);
        }
        wave_lds_fence();
        int better = 0;
        for (int h = 0; h < a.n_group; ++h) {
            const uint32_t other = ordered_bits(rank[h]);
            better += other > own || (other == own && h < sub);
        }
        const uint64_t kept = __ballot(better < a.topk_group && sub < a.n_group);
        if (mine && !(kept >> (first + sub / gs) & 1)) key = 0u;
    }
    wave_lds_fence();
    const uint64_t seg_mask = ((1ull << SEG) - 1) << first;
    float sum = 0.0f, my_p = 0.0f;
    int my_id = 0;
    for (int k = 0; k < a.K; ++k) {
        const uint32_t m = across<SEG>(key, [](uint32_t q, uint32_t r) { return q > r ? q : r; });
        const int e = __ffsll((unsigned long long)(__ballot(key == m) & seg_mask)) - 1 - first;
        if (sub == e) key = 0u;
        const float pe = a.bias != nullptr ? pl[e] : topk_value(m);
        sum += pe;
        if (sub == k) my_id = e, my_p = pe;
    }
    if (live && sub < a.K) topk_store(a, t, sub, my_id, my_p, sum);
}

// More experts: a wave a token.
template <int VPL>
__global__ __launch_bounds__(kTopkThreads) void k_route_wave(RouteCall a) {
    constexpr int WAVES = kTopkThreads / kWave;
    // lanes that hold their experts in descending order offer one at a time; for more than 4 that costs more than it saves
    constexpr bool SORTED = VPL <= 4;
    __shared__ float choice_lds[WAVES][kWave * VPL], plain_lds[WAVES][kWave * VPL];
    __shared__ uint2 chosen_lds[WAVES][32];
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
    const int64_t t = (int64_t)blockIdx.x * WAVES + wv;
    if (t >= a.B) return;  // nothing below synchronises across waves
    float* pl = plain_lds[wv];
    float x[VPL], p[VPL];
    topk_logits<kWave>(a, t, lane, x);
    topk_scores<kWave>(a.softmax, x, p);
    uint32_t key[VPL];  // 0: no candidate (any longer)
    if (a.bias != nullptr) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = lane + kWave * v;
            key[v] = topk_key(p[v] + a.bias[e < a.N ? e : a.N - 1]);
            pl[e] = p[v];
        }
    } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) key[v] = topk_key(p[v]);
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) key[v] = lane + kWave * v < a.N ? key[v] : 0u;
    if (a.n_group > 1) {
        float* ch = choice_lds[wv];
#pragma unroll
        for (int v = 0; v < VPL; ++v) ch[lane + kWave * v] = topk_value(key[v]);
        wave_lds_fence();
        const int gs = a.N / a.n_group;
        // e / gs: e + 1/2 is at least gs / 2 parts in 1024 gs from a multiple of gs, more than fp32 loses
        const float per_gs = 1.0f / gs;
        auto group_of = [&](int e) { return (int)((e + 0.5f) * per_gs); };
        auto merge = [](float& best, float& next, float b2, float n2) {
            next = fmaxf(fmaxf(next, n2), fminf(best, b2));
            best = fmaxf(best, b2);
        };
        if (a.n_group <= 8) {
            // eight lanes a group
            const int g = lane / 8;
            float best = -__builtin_inff(), next = best;
            if (g < a.n_group)
                for (int i = g * gs + lane % 8; i < (g + 1) * gs; i += 8) merge(best, next, ch[i], -__builtin_inff());
            merge(best, next, lane_of<kSwap1>(best), lane_of<kSwap1>(next));
            merge(best, next, lane_of<kSwap2>(best), lane_of<kSwap2>(next));
            merge(best, next, lane_of<kMirror8>(best), lane_of<kMirror8>(next));
            const uint32_t own = ordered_bits(group_rank(a, gs, best, next));
            int better = 0;
            for (int h = 0; h < a.n_group; ++h) {
                const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)own, h * 8);
                better += other > own || (other == own && h < g);
            }
            const uint64_t kept = __ballot(better < a.topk_group);
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (!(kept >> (group_of(lane + kWave * v) * 8 & 63) & 1)) key[v] = 0u;
        } else {
            // a lane a group; the choices are in registers, so their ranks and then who is kept take their place
            float rank[VPL];
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                const int g = lane + kWave * v;
                float best = -__builtin_inff(), next = best;
                if (g < a.n_group)
                    for (int i = g * gs; i < (g + 1) * gs; ++i) merge(best, next, ch[i], -__builtin_inff());
                rank[v] = group_rank(a, gs, best, next);
            }
            wave_lds_fence();
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (lane + kWave * v < a.n_group) ch[lane + kWave * v] = rank[v];
            wave_lds_fence();
            int better[VPL];
#pragma unroll
            for (int v = 0; v < VPL; ++v) better[v] = 0;
            for (int h = 0; h < a.n_group; ++h) {
                const uint32_t other = ordered_bits(ch[h]);
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    const uint32_t own = ordered_bits(rank[v]);
                    better[v] += other > own || (other == own && h < lane + kWave * v);
                }
            }
            wave_lds_fence();
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (lane + kWave * v < a.n_group) ch[lane + kWave * v] = better[v] < a.topk_group ? 1.0f : 0.0f;
            wave_lds_fence();
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                const int e = lane + kWave * v;
                if (e < a.N && ch[group_of(e)] == 0.0f) key[v] = 0u;
            }
        }
    }
    wave_lds_fence();

    uint32_t slots = 0;  // SORTED: which of the lane's experts key[0], key[1], .. belong to, a byte each
    if constexpr (SORTED) {
        uint32_t s[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v) s[v] = v;
        auto order = [&](int i) {  // neighbours, as large ones staying: the lower expert first
            const bool swap = key[i + 1] > key[i];
            const uint32_t k = key[i], q = s[i];
            key[i] = swap ? key[i + 1] : k, key[i + 1] = swap ? k : key[i + 1];
            s[i] = swap ? s[i + 1] : q, s[i + 1] = swap ? q : s[i + 1];
        };
#pragma unroll
        for (int n = VPL - 1; n > 0; --n)
#pragma unroll
            for (int i = 0; i < n; ++i) order(i);
#pragma unroll
        for (int v = 0; v < VPL; ++v) slots |= s[v] << (8 * v);
    }
    uint2* chosen = chosen_lds[wv];  // expert and key
    float sum = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        uint32_t m = key[0];
        if constexpr (!SORTED) {
#pragma unroll
            for (int v = 1; v < VPL; ++v) m = key[v] > m ? key[v] : m;
        }
        m = wave_max_u32(m);
        // the lowest expert that holds m; the lane that holds it notes it and goes on to its next
        if constexpr (SORTED) {
            bool mine = key[0] == m;
            const uint64_t have = __ballot(mine);
            if (have & (have - 1)) {  // a tie of several lanes
                int e = kWave * VPL;
                for (uint64_t h = have; h != 0; h &= h - 1) {
                    const int l = __builtin_ctzll(h), at = (__builtin_amdgcn_readlane((int)slots, l) & 255) * kWave + l;
                    e = at < e ? at : e;
                }
                mine = lane == e % kWave;
            }
            if (mine) {
                chosen[k] = make_uint2((slots & 255) * kWave + lane, m);
#pragma unroll
                for (int v = 0; v + 1 < VPL; ++v) key[v] = key[v + 1];
                key[VPL - 1] = 0u;
                slots >>= 8;
            }
        } else {
            int e = 0;
#pragma unroll
            for (int v = VPL - 1; v >= 0; --v) {
                const uint64_t have = __ballot(key[v] == m);
                if (have != 0) e = __builtin_ctzll(have) + kWave * v;
            }
            if (lane == 0) chosen[k] = make_uint2(e, m);
#pragma unroll
            for (int v = 0; v < VPL; ++v) key[v] = lane + kWave * v == e ? 0u : key[v];
        }
        sum += topk_value(m);
    }
    wave_lds_fence();
    if (lane < a.K) {
        const uint2 own = chosen[lane];
        float p_own = topk_value(own.y);  // without a bias the choice is the score
        if (a.bias != nullptr) {
            p_own = pl[own.x];
            sum = 0.0f;
            if (a.renorm)
                for (int k = 0; k < a.K; ++k) sum += pl[chosen[k].x];
        }
        topk_store(a, t, lane, (int)own.x, p_own, sum);
    }
}

template <class Kernel>
hipError_t launch_topk(Kernel kernel, int tokens, const RouteCall& a, hipStream_t s) {
    const int64_t blocks = ((int64_t)a.B + tokens - 1) / tokens;
    if (!grid_fits(blocks, kTopkThreads)) return hipErrorInvalidConfiguration;
    kernel<<<(unsigned)blocks, kTopkThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const float* logits, const float* bias, int B, int N, int n_group, int topk_group, int K,
                        float scale, int32_t* ids, float* w, hipStream_t s) {
    if (B == 0) return hipSuccess;
    dim3 grid((B + 3) / 4), block(256);
    if (N <= 64)
        k_route<1><<<grid, block, 0, s>>>(logits, bias, B, N, n_group, topk_group, K, scale, ids, w);
    else if (N <= 256)
        k_route<4><<<grid, block, 0, s>>>(logits, bias, B, N, n_group, topk_group, K, scale, ids, w);
    else
        k_route<16><<<grid, block, 0, s>>>(logits, bias, B, N, n_group, topk_group, K, scale, ids, w);
    return hipGetLastError();
}

hipError_t launch_route_topk(const RouteCall& a, hipStream_t s) {
    if (a.B == 0) return hipSuccess;
    // lane k holds the k-th choice until the end: the lanes are no fewer than K (K <= N)
    if (a.N <= 8) return launch_topk(k_route_few<8>, kTopkThreads / 8, a, s);
    if (a.N <= 16) return launch_topk(k_route_few<16>, kTopkThreads / 16, a, s);
    if (a.N <= 32) return launch_topk(k_route_few<32>, kTopkThreads / 32, a, s);
    if (a.N <= 64) return launch_topk(k_route_wave<1>, kTopkThreads / kWave, a, s);
    if (a.N <= 128) return launch_topk(k_route_wave<2>, kTopkThreads / kWave, a, s);
    if (a.N <= 192) return launch_topk(k_route_wave<3>, kTopkThreads / kWave, a, s);
    if (a.N <= 256) return launch_topk(k_route_wave<4>, kTopkThreads / kWave, a, s);
    if (a.N <= 512) return launch_topk(k_route_wave<8>, kTopkThreads / kWave, a, s);
    return launch_topk(k_route_wave<16>, kTopkThreads / kWave, a, s);
}

}  // namespace rdg
