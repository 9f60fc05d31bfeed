// Step plan of the paged key/value cache: block tables and slot maps built on
// the GPU from the requests' lengths, and the pages handed back.
//
// With P = page_rows, request r holds ceil(kv_r / P) pages and needs
//   need_r = ceil((kv_r + q_r) / P) - ceil(kv_r / P)
// more.  An exclusive scan of need over the requests gives each its place on
// the stack of free pages, one of q gives cu_q, and one of the pages that the
// new tokens touch gives each request's first segment.  Every new page starts
// with exactly one new token (its position is a multiple of P), so the
// per-token pass writes the block table too.
//
// Bound by latency: a step writes 8 bytes per token and reads 8 per request,
// a few microseconds' worth of one launch.  Every workgroup therefore scans
// all the requests by itself in LDS (16 bytes a request) instead of waiting
// for another launch or workgroup, and then expands its own 1024 tokens.
// The last workgroup to finish (a ticket in S.work) writes what a caller may
// pass as input and output at once: kv_len, the free count, the status.
//
// Measured: 48 decode requests 5.3 us, 1023 mixed ones with 44 thousand tokens 9.0
// (15.6 with a thread's lengths and page ids loaded one after the other), 146
// thousand prefill tokens of 61 requests 7.4.  An empty launch takes 3.4.  The hand-back:
// 120 pages of 48 requests 5.2, 17607 of 1024 5.9, 12910 of 4096 13.1 (a thread reads 16
// requests' lengths one after the other).
#include "rdg_internal.h"

namespace rdg {
namespace {

constexpr int kThreads = 256;
constexpr int kTokPerThread = 4;
constexpr uint32_t kSat = 1u << 30;

// Saturating sum of values <= 2^30: associative, so lengths of any size scan
// without wrapping.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) {
    const uint32_t s = a + b;
    return s < kSat ? s : kSat;
}

// Exclusive saturating scan of one value per thread over the workgroup; part
// holds one word per wave.  The total is left in *total.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* part, uint32_t* total) {
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    uint32_t inc = v;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const uint32_t o = __shfl_up(inc, off);
        if (lane >= off) inc = sat_add(inc, o);
    }
    __syncthreads();  // part may still be read from the scan before
    if (lane == kWave - 1) part[wave] = inc;
    uint32_t exc = __shfl_up(inc, 1);
    if (lane == 0) exc = 0;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) {
        if (w < wave) before = sat_add(before, part[w]);
        all = sat_add(all, part[w]);
    }
    *total = all;
    return sat_add(before, exc);
}

// The same of two values at once; part holds two words per wave.
__device__ __forceinline__ void block_scan2(uint32_t u, uint32_t v, uint32_t* part, uint32_t* u_before, uint32_t* v_before,
                                            uint32_t* u_all, uint32_t* v_all) {
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    uint32_t a = u, b = v;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const uint32_t oa = __shfl_up(a, off), ob = __shfl_up(b, off);
        if (lane >= off) {
            a = sat_add(a, oa);
            b = sat_add(b, ob);
        }
    }
    __syncthreads();  // part may still be read from the scan before
    if (lane == kWave - 1) {
        part[wave] = a;
        part[kThreads / kWave + wave] = b;
    }
    a = __shfl_up(a, 1);
    b = __shfl_up(b, 1);
    if (lane == 0) a = b = 0;
    __syncthreads();
    uint32_t ua = 0, va = 0, ub = 0, vb = 0;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) {
        const uint32_t x = part[w], y = part[kThreads / kWave + w];
        if (w < wave) {
            ub = sat_add(ub, x);
            vb = sat_add(vb, y);
        }
        ua = sat_add(ua, x);
        va = sat_add(va, y);
    }
    *u_before = sat_add(ub, a);
    *v_before = sat_add(vb, b);
    *u_all = ua;
    *v_all = va;
}

// Last i in [0, n) with begin[i] <= t (begin[0] = 0, ascending).
__device__ __forceinline__ int find_row(const uint32_t* begin, int n, uint32_t t) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (begin[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// True in every thread of the last workgroup of the grid to get here; the
// ticket is then 0 again for the next launch.  READS: the last workgroup reads
// what the others have written.
template <bool READS>
__device__ __forceinline__ bool last_block(int32_t* ticket) {
    __shared__ int last;
    // every wave has used what it read, and what it noted has been noted: the
    // ticket orders nothing else, so without READS it needs no fence
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (threadIdx.x == 0) {
        last = 1;
        if (gridDim.x > 1) {
            if (READS) __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
            last = __hip_atomic_fetch_add(ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
            if (last) __hip_atomic_store(ticket, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (READS) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        }
    }
    __syncthreads();
    return last != 0;
}

// work[1]: kMaxRequests less the first request with a page id outside the cache; 0: none.
__device__ __forceinline__ void note_bad(int32_t* work, int r) {
    __hip_atomic_fetch_max(work + 1, kMaxRequests - r, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ void write_status(int32_t* status, int32_t* work, int code, int detail) {
    const int bad = __hip_atomic_load(work + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (bad != 0) {
        __hip_atomic_store(work + 1, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (code == RDG_OK) {
            code = RDG_EDATA;
            detail = kMaxRequests - bad;
        }
    }
    status[0] = code;
    status[1] = detail;
}

struct Lens {
    int kv, q;
    bool bad;
};

// A request's lengths, made safe: with one of them out of range it has no new
// tokens and is reported.  Its cached ones stay, unless theirs is the bad length.
__device__ __forceinline__ Lens lens_of(const int32_t* kv_len, const int32_t* q_len, int r) {
    Lens l = {kv_len[r], q_len[r], false};
    const bool bad_kv = l.kv < 0 || l.kv > (int)kSat;
    if (bad_kv || l.q < 0 || l.q > (int)kSat) {
        l.bad = true;
        l.kv = bad_kv ? 0 : l.kv;
        l.q = 0;
    }
    return l;
}

// PER: consecutive requests per thread, whose lengths are loaded together.
template <int PER>
__global__ __launch_bounds__(kThreads) void k_kv_plan(rdg_kv_step S, int shift, const int32_t* kv_len,
                                                      const int32_t* q_len, const int32_t* __restrict__ free_list,
                                                      const int32_t* n_free, int32_t* n_free_out) {
    extern __shared__ uint32_t lds[];
    __shared__ uint32_t part[2 * kThreads / kWave];
    __shared__ uint32_t used;        // pages taken
    __shared__ uint32_t failed[2];   // first request that did not fit / had bad lengths
    const int R = S.n_req, P1 = S.page_rows - 1, tid = (int)threadIdx.x;
    uint32_t* cu = lds;                        // [R + 1] first token
    int32_t* page0 = (int32_t*)(lds + R + 1);  // [R] place on the free stack, -1: not admitted
    uint32_t* seg0 = lds + 2 * R + 1;          // [R] first segment
    int32_t* kv0 = (int32_t*)(lds + 3 * R + 1);  // [R] cached tokens
    if (tid == 0) {
        used = 0;
        failed[0] = failed[1] = 0xffffffffu;
        cu[0] = 0;
    }
    const int r0 = tid * PER;
    Lens len[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        len[i] = {0, 0, false};
        if (r0 + i < R) len[i] = lens_of(kv_len, q_len, r0 + i);
    }
    int nf = n_free[0];
    nf = nf < 0 ? 0 : nf > S.n_pages ? S.n_pages : nf;

    uint32_t q_sum = 0, need_sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const Lens l = len[i];
        const int old_b = (l.kv + P1) >> shift, new_b = (int)(((uint32_t)l.kv + l.q + P1) >> shift);
        q_sum = sat_add(q_sum, l.q);
        need_sum = sat_add(need_sum, new_b > S.max_blocks ? 0 : new_b - old_b);
    }
    uint32_t n_tok, n_seg, all;
    uint32_t tok, pg;
    block_scan2(q_sum, need_sum, part, &tok, &pg, &n_tok, &all);
    uint32_t seg_sum = 0, seg[PER], took = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = r0 + i;
        const Lens l = len[i];
        seg[i] = seg_sum;
        if (r >= R) continue;
        const int old_b = (l.kv + P1) >> shift, new_b = (int)(((uint32_t)l.kv + l.q + P1) >> shift);
        const bool fits = new_b <= S.max_blocks;
        const uint32_t need = fits ? new_b - old_b : 0;
        const uint32_t begin = pg;
        tok = sat_add(tok, l.q);
        pg = sat_add(pg, need);
        const bool ok = !l.bad && fits && tok <= (uint32_t)S.t_cap && (need == 0 || pg <= (uint32_t)nf);
        cu[r + 1] = tok;
        kv0[r] = l.kv;
        page0[r] = ok ? (need ? (int)begin : 0) : -1;
        if (ok && l.q > 0) seg_sum += ((l.kv + l.q - 1) >> shift) - (l.kv >> shift) + 1;
        if (ok && need) took = pg;  // ascending over the requests
        if (!ok) atomicMin(&failed[l.bad ? 1 : 0], (uint32_t)r);
    }
#pragma unroll
    for (int off = kWave / 2; off >= 1; off >>= 1) {
        const uint32_t o = __shfl_xor(took, off);
        took = o > took ? o : took;
    }
    if (lane_id() == 0) atomicMax(&used, took);
    const uint32_t seg_before = block_scan(seg_sum, part, &n_seg);
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (r0 + i < R) seg0[r0 + i] = seg[i] + seg_before;
    __syncthreads();

    // tokens: kTokPerThread consecutive ones per thread
    const uint32_t total = n_tok < (uint32_t)S.t_cap ? n_tok : (uint32_t)S.t_cap;
    const int t0 = ((int)blockIdx.x * kThreads + tid) * kTokPerThread;
    if (t0 < S.t_cap) {
        int32_t slot[kTokPerThread], pos[kTokPerThread], req[kTokPerThread], page[kTokPerThread];
        bool stored[kTokPerThread], fresh[kTokPerThread];
        int r = (uint32_t)t0 < total ? find_row(cu, R, t0) : 0;
#pragma unroll
        for (int i = 0; i < kTokPerThread; ++i) {
            const uint32_t t = t0 + i;
            stored[i] = fresh[i] = false;
            pos[i] = 0;
            page[i] = -1;
            if (t < total) {
                while (cu[r + 1] <= t) ++r;
                const int kv = kv0[r], base = page0[r];
                pos[i] = kv + (int)(t - cu[r]);
                stored[i] = base >= 0;
                if (stored[i]) {  // the four tokens' loads are in flight together
                    const int blk = pos[i] >> shift, back = blk - ((kv + P1) >> shift);
                    fresh[i] = back >= 0;
                    page[i] = fresh[i] ? free_list[nf - 1 - base - back] : S.block_table[(int64_t)r * S.max_blocks + blk];
                }
            }
            req[i] = r;
        }
#pragma unroll
        for (int i = 0; i < kTokPerThread; ++i) {
            slot[i] = -1;
            if (!stored[i]) continue;
            const int blk = pos[i] >> shift, kv = kv0[req[i]];
            const bool starts = (pos[i] & P1) == 0;
            const bool in_cache = (unsigned)page[i] < (unsigned)S.n_pages;
            if (fresh[i] && starts) S.block_table[(int64_t)req[i] * S.max_blocks + blk] = in_cache ? page[i] : -1;
            if (in_cache) slot[i] = (page[i] << shift) + (pos[i] & P1);
            else note_bad(S.work, req[i]);
            if (pos[i] == kv || starts) {
                const uint32_t place = seg0[req[i]] + (blk - (kv >> shift));
                if (place < (uint32_t)S.seg_cap) S.seg_tok[place] = t0 + i;
            }
        }
        if (t0 + kTokPerThread <= S.t_cap) {
            *reinterpret_cast<int4*>(S.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4*>(S.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
            for (int i = 0; t0 + i < S.t_cap; ++i) {
                S.slots[t0 + i] = slot[i];
                S.positions[t0 + i] = pos[i];
            }
        }
    }
    for (int s = (int)n_seg + (int)blockIdx.x * kThreads + tid; s < S.seg_cap; s += (int)gridDim.x * kThreads)
        S.seg_tok[s] = -1;

    if (!last_block<false>(S.work)) return;
    for (int r = tid; r < R; r += kThreads) {
        const Lens l = lens_of(kv_len, q_len, r);
        S.cu_q[r + 1] = (int)(cu[r + 1] < (uint32_t)S.t_cap ? cu[r + 1] : (uint32_t)S.t_cap);
        S.kv_len[r] = page0[r] >= 0 ? l.kv + l.q : l.kv;
    }
    if (tid == 0) {
        S.cu_q[0] = 0;
        n_free_out[0] = nf - (int)used;
        const bool bad = failed[1] != 0xffffffffu, full = failed[0] != 0xffffffffu;
        write_status(S.status, S.work, bad ? RDG_EDATA : full ? RDG_ECAPACITY : RDG_OK,
                     bad ? (int)failed[1] : full ? (int)failed[0] : 0);
    }
}

// Pages behind the new lengths, in request and block order, onto the stack.
__global__ __launch_bounds__(kThreads) void k_kv_trim(rdg_kv_step S, int shift, const int32_t* new_len,
                                                      const int32_t* kv_len, int32_t* __restrict__ free_list,
                                                      const int32_t* n_free, int32_t* n_free_out) {
    extern __shared__ uint32_t lds[];
    __shared__ uint32_t part[kThreads / kWave];
    __shared__ uint32_t failed;
    const int R = S.n_req, P1 = S.page_rows - 1, tid = (int)threadIdx.x;
    uint32_t* begin = lds;  // [R] first freed page of each request
    if (tid == 0) failed = 0xffffffffu;
    int nf = n_free[0];
    nf = nf < 0 ? 0 : nf > S.n_pages ? S.n_pages : nf;
    const int limit = S.max_blocks << shift;
    const int per = (R + kThreads - 1) / kThreads;
    const int r0 = tid * per < R ? tid * per : R, r1 = r0 + per < R ? r0 + per : R;
    __syncthreads();
    uint32_t sum = 0;
    for (int r = r0; r < r1; ++r) {
        const int kv = kv_len[r], to = new_len[r];
        uint32_t n = 0;
        if (kv < 0 || kv > limit || to < 0 || to > kv) atomicMin(&failed, (uint32_t)r);
        else n = ((kv + P1) >> shift) - ((to + P1) >> shift);
        begin[r] = sum;
        sum = sat_add(sum, n);
    }
    uint32_t total;
    const uint32_t before = block_scan(sum, part, &total);
    for (int r = r0; r < r1; ++r) begin[r] = sat_add(begin[r], before);
    __syncthreads();
    const bool fits = total <= (uint32_t)(S.n_pages - nf);
    if (fits) {
        for (uint32_t e = blockIdx.x * kThreads + tid; e < total; e += gridDim.x * kThreads) {
            const int r = find_row(begin, R, e);
            int32_t* entry = S.block_table + (int64_t)r * S.max_blocks + ((new_len[r] + P1) >> shift) + (e - begin[r]);
            const int page = *entry;
            if ((unsigned)page >= (unsigned)S.n_pages) note_bad(S.work, r);
            free_list[nf + e] = page;
            *entry = -1;
        }
    }
    if (!last_block<true>(S.work)) return;
    uint32_t freed = fits ? total : 0;
    const int bad_page = __hip_atomic_load(S.work + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();  // read by all before write_status clears it
    if (bad_page != 0) {  // ids that no page has: the others move up, in their order
        freed = 0;
        for (uint32_t e0 = 0; e0 < total; e0 += kThreads) {
            const uint32_t e = e0 + tid;
            const int page = e < total ? free_list[nf + e] : -1;
            const bool in_cache = (unsigned)page < (unsigned)S.n_pages;
            uint32_t n;
            const uint32_t at = block_scan(in_cache ? 1 : 0, part, &n);
            if (in_cache) free_list[nf + freed + at] = page;
            freed += n;
        }
    }
    for (int r = tid; r < R; r += kThreads) {
        const int kv = kv_len[r], to = new_len[r];
        S.kv_len[r] = (!fits || kv < 0 || kv > limit || to < 0 || to > kv) ? kv : to;
    }
    if (tid == 0) {
        n_free_out[0] = nf + (int)freed;
        const bool bad = failed != 0xffffffffu;
        write_status(S.status, S.work, bad ? RDG_EDATA : fits ? RDG_OK : RDG_ECAPACITY,
                     bad ? (int)failed : fits ? 0 : (int)total);
    }
}

inline int log2_of(int p) { return p == 16 ? 4 : p == 32 ? 5 : p == 64 ? 6 : 7; }

}  // namespace

hipError_t launch_kv_plan(const rdg_kv_step& S, const int32_t* kv_len, const int32_t* q_len, const int32_t* free_list,
                          const int32_t* n_free, int32_t* n_free_out, hipStream_t s) {
    const int per_block = kThreads * kTokPerThread;
    const int blocks = S.t_cap > 0 ? (S.t_cap + per_block - 1) / per_block : 1;
    const size_t bytes = sizeof(uint32_t) * (4 * (size_t)S.n_req + 1);
    const int shift = log2_of(S.page_rows);
    if (S.n_req <= kThreads)
        k_kv_plan<1><<<blocks, kThreads, bytes, s>>>(S, shift, kv_len, q_len, free_list, n_free, n_free_out);
    else if (S.n_req <= 4 * kThreads)
        k_kv_plan<4><<<blocks, kThreads, bytes, s>>>(S, shift, kv_len, q_len, free_list, n_free, n_free_out);
    else
        k_kv_plan<16><<<blocks, kThreads, bytes, s>>>(S, shift, kv_len, q_len, free_list, n_free, n_free_out);
    return hipGetLastError();
}

hipError_t launch_kv_trim(const rdg_kv_step& S, const int32_t* new_len, const int32_t* kv_len, int32_t* free_list,
                          const int32_t* n_free, int32_t* n_free_out, hipStream_t s) {
    const int64_t most = (int64_t)S.n_req * S.max_blocks;
    const int blocks = (int)(most >= 64 * 2048 ? 64 : (most + 2047) / 2048);
    k_kv_trim<<<blocks < 1 ? 1 : blocks, kThreads, sizeof(uint32_t) * (size_t)S.n_req, s>>>(
        S, log2_of(S.page_rows), new_len, kv_len, free_list, n_free, n_free_out);
    return hipGetLastError();
}

}  // namespace rdg
