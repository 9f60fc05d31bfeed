// C ABI of the paged key/value cache (include/rdg.h): argument checks, the
// choice of kernels, then enqueue.
#include <math.h>

#include "rdg_internal.h"

using namespace rdg;

namespace {

// InvalidConfiguration: sizes whose grid no launch holds.
inline int hip_rc(hipError_t e) {
    return e == hipSuccess ? RDG_OK : e == hipErrorInvalidConfiguration ? RDG_EUNSUPPORTED : RDG_EHIP;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool page_rows_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }

int page_shift_of(int p) { return p == 16 ? 4 : p == 32 ? 5 : p == 64 ? 6 : 7; }

// The fields of a step that every call reads.
bool step_ok(const rdg_kv_step* S) {
    if (S == nullptr) return false;
    if (S->n_req < 0 || S->max_blocks < 1 || S->n_pages < 1 || S->t_cap < 0 || S->seg_cap < 0) return false;
    if (!page_rows_ok(S->page_rows)) return false;
    if ((int64_t)S->n_pages * S->page_rows >= (int64_t)1 << 31) return false;
    if ((int64_t)S->max_blocks * S->page_rows > (int64_t)1 << 30 || S->t_cap > 1 << 30) return false;
    return S->status != nullptr;
}

int cache_rc(const rdg_kv_cache* C) {
    if (C == nullptr || C->n_pages < 1 || C->n_kv < 1 || !page_rows_ok(C->page_rows)) return RDG_EINVAL;
    if ((int64_t)C->n_pages * C->page_rows >= (int64_t)1 << 31) return RDG_EINVAL;
    if (C->head_dim != 64 && C->head_dim != 128 && C->head_dim != 256) return RDG_EUNSUPPORTED;
    return RDG_OK;
}

int cache_buffers_rc(const rdg_kv_cache* C) {
    if (!C->k || !C->v || !C->k_scale || !C->v_scale || !aligned16(C->k) || !aligned16(C->v)) return RDG_EINVAL;
    return RDG_OK;
}

// How attention shares out its work.  Times in us at head_dim 128, each as it is
// against the value named.
//
// Keys at least in a k_attn_rows chunk, one 64-key step of each of four waves.  512: two
// requests of 3 queries, 5000 keys, 8 heads a key head 14.8 against 17.5; 31 requests
// of 35 rows 39.8 against 46.8.
constexpr int kChunkMin = 256;
constexpr int kWaveKeys = 1024;  // keys whose pages the lanes of a k_attn_rows wave hold at a time
// k_attn_rows workgroups wanted, four per CU.  31 requests of 35 rows 39.8, with 512 46.9,
// with 2048 44.5; 16 requests of 64 rows 40.6, 40.3 and 49.1; 64 requests of one row 64,
// 62 and 62.
constexpr int kRowUnits = 1024;
// Bytes of parts that k_attn_rows may leave to be joined; where the longest chunks below come to more,
// they grow.  That many parts are 4000 workgroups of 64 rows and more, so the chip stays
// full, but a chunk is also the longest walk beside a batch's long requests.  One chunk of 4096
// tokens and 31 decode rows of up to 4000 keys under a bound of 32768, 64 / 8 heads: 384, with 128
// MiB 402, unbounded (4.2 GiB) 384; four fp32 prompts of 2048, whose rows fill the chip: 456
// without parts, 690 with 4.2 GiB of them.
constexpr size_t kRowParts = (size_t)256 << 20;
// k_attn_tiles workgroups wanted, two per CU; above it rows go in tiles of 256, below
// half of it keys are split.  Prompts of 32 / 8 heads: 1000 tokens 33, with 256 33, with 1024
// 47; 2000 tokens 63, 67 and 83; 4000 tokens 163, 153 and 159; 300 tokens on
// 6000 58, 61 and 66; four times 400 on 3000 99, 100 and 132.
constexpr int kTileUnits = 512;
// Keys: fewer do not pay for the parts' way through memory.  1024: 800 tokens on up to
// 4000, 8 heads sharing one of 256, 45 against 51; 300 on 6000, 58 against 56.
constexpr int kTileChunkMin = 512;
// The longest request a block table can list (step_ok): bounds and windows above it say no
// more, and key positions, and a position and a chunk of keys together, stay within an int.
constexpr int kMaxKeys = 1 << 30;

// How a call's work is split.  span: the longest run of keys that one request's
// queries see together.
struct AttnPlan {
    int rt;  // 16-row tiles per workgroup of k_attn_rows
    int n_most, row_places, chunk, row_chunks;
    int tile_rows, tile_slots, tile_chunk, tile_chunks;  // tile_slots 0: no k_attn_tiles
    // workspace: parts of the short requests' rows by request (row_place each) or by token (0), then the long ones' by token
    int row_place;
    size_t row_bytes, tile_bytes;
};

// Bytes of the parts of every head of `places` tokens, fp32 row, maximum and sum each.
size_t parts_bytes(int64_t places, int n_q, int head_dim, int chunks) {
    return chunks > 1 ? align256(sizeof(float) * (size_t)places * n_q * (head_dim + 2) * chunks) : 0;
}

// Parts of `chunk` keys that a run of span keys can have, from the 64-key block it begins in.
int chunks_of(int64_t span, int chunk) {
    const int64_t keys = span + 63 < kMaxKeys ? span + 63 : kMaxKeys, n = (keys + chunk - 1) / chunk;
    return n < 1 ? 1 : (int)n;
}

// Chunks that a run of span keys fills `room` times at most.
void coarsen(int* chunk, int* chunks, int span, int64_t room) {
    if (*chunks <= room) return;
    const int64_t keys = span + 63 < kMaxKeys ? span + 63 : kMaxKeys;
    *chunk = (int)(((keys + room - 1) / room + kChunkMin - 1) / kChunkMin * kChunkMin);
    *chunks = chunks_of(span, *chunk);
}

AttnPlan plan_attn(int T, int R, int n_kv, int group, int head_dim, bool bf16, int max_q, int span) {
    AttnPlan p = {};
    // Requests of more than 64 rows (query x head of the group) go to
    // k_attn_tiles, whose workgroups share the conversion of the codes (35 rows a request
    // 34 us there and 39 here, but 64 rows 75 against 41 and 32 rows 185 against 133).
    const bool tiles = bf16 && (int64_t)max_q * group > 64;
    p.n_most = max_q;
    if (tiles) {
        p.n_most = 64 / group;
        // no request is that short if even max_q for all the others leaves more
        if ((int64_t)T - (int64_t)(R - 1) * max_q > p.n_most) p.n_most = 0;
        // Tiles of 256 rows convert each key's codes half as often: two prompts of 7000 tokens,
        // 32 / 8 heads, 796 us, with 128 rows 831; one of 8000 516 and 555.  Tiles of 128 fill the
        // chip sooner and waste less on short requests: one prompt of 1000 33, with 256 rows 46;
        // four times 400 tokens on 3000 99 and 139.
        const auto units_of = [&](int bm) { return (double)n_kv * ceil((double)T * group / bm); };
        p.tile_rows = head_dim == 256 || p.n_most > 0 || units_of(256) < kTileUnits ? 128 : 256;
        p.tile_slots = (int)((int64_t)T * group / p.tile_rows + R);
        const double units = units_of(p.tile_rows);
        double want = span + 64.0;
        if (units < kTileUnits / 2) want = ceil(span * units / kTileUnits / 64) * 64;
        if (want < kTileChunkMin) want = kTileChunkMin;
        if (want > kMaxKeys) want = kMaxKeys;
        p.tile_chunk = (int)((want + 63) / 64) * 64;
        p.tile_chunks = chunks_of(span, p.tile_chunk);
        p.tile_bytes = parts_bytes(T, n_kv * group, head_dim, p.tile_chunks);
    }
    if (p.n_most > 0) {
        const int64_t rows = (int64_t)p.n_most * group;
        p.rt = rows <= 64 && !tiles ? (int)((rows + 15) / 16) : 4;
        // one tile a request, or places for the tiles of all (see request_of_place)
        if (rows > 16 * p.rt) p.row_places = (int)((int64_t)T * group / (16 * p.rt) + R);
        const int most = kWaveKeys * (p.rt == 1 ? 4 : p.rt == 2 ? 2 : 1);
        const double units = (double)n_kv * (p.row_places > 0 ? p.row_places : R);
        double want = ceil(span * units / kRowUnits / kChunkMin) * kChunkMin;
        if (want < kChunkMin) want = kChunkMin;
        p.chunk = want > most ? most : (int)want;
        p.row_chunks = chunks_of(span, p.chunk);
        // Beside long requests most tokens are not the short ones': those then have n_most places a request.
        const int64_t by_request = (int64_t)R * p.n_most, places = by_request < T ? by_request : T;
        p.row_place = by_request < T ? p.n_most : 0;
        const size_t room = kRowParts / (sizeof(float) * (size_t)places * n_kv * group * (head_dim + 2));
        coarsen(&p.chunk, &p.row_chunks, span, room > 0 ? (int64_t)room : 1);
        p.row_bytes = parts_bytes(places, n_kv * group, head_dim, p.row_chunks);
    }
    return p;
}

int key_span(int max_q, int max_kv, int window) {
    const int64_t w = window > 0 ? (int64_t)window + max_q : max_kv;
    return w < max_kv ? (int)w : max_kv;
}

}  // namespace

extern "C" {

size_t rdg_kv_step_work_bytes(void) { return 16; }

int rdg_kv_seg_cap(int t_cap, int n_req, int page_rows) {
    if (t_cap < 0 || n_req < 0 || !page_rows_ok(page_rows)) return RDG_EINVAL;
    const int64_t n = t_cap / page_rows + 2 * (int64_t)n_req;
    return n < t_cap ? (int)n : t_cap;
}

int rdg_kv_plan(const rdg_kv_step* S, const int32_t* kv_len, const int32_t* q_len, const int32_t* free_list,
                const int32_t* n_free, int32_t* n_free_out, rdg_stream_t stream) {
    if (!step_ok(S) || !S->work || !n_free || !n_free_out || !S->cu_q) return RDG_EINVAL;
    if (S->n_req > 0 && (!kv_len || !q_len || !free_list || !S->block_table || !S->kv_len)) return RDG_EINVAL;
    if (S->t_cap > 0 && (!S->slots || !S->positions || !aligned16(S->slots) || !aligned16(S->positions)))
        return RDG_EINVAL;
    if (S->seg_cap < rdg_kv_seg_cap(S->t_cap, S->n_req, S->page_rows) || (S->seg_cap > 0 && !S->seg_tok))
        return RDG_EINVAL;
    if (S->n_req > kMaxRequests) return RDG_EUNSUPPORTED;
    return hip_rc(launch_kv_plan(*S, kv_len, q_len, free_list, n_free, n_free_out, stream));
}

int rdg_kv_trim(const rdg_kv_step* S, const int32_t* kv_len, const int32_t* new_len, int32_t* free_list,
                const int32_t* n_free, int32_t* n_free_out, rdg_stream_t stream) {
    if (!step_ok(S) || !S->work || !n_free || !n_free_out) return RDG_EINVAL;
    if (S->n_req > 0 && (!kv_len || !new_len || !free_list || !S->block_table || !S->kv_len)) return RDG_EINVAL;
    if (S->n_req > kMaxRequests) return RDG_EUNSUPPORTED;
    return hip_rc(launch_kv_trim(*S, new_len, kv_len, free_list, n_free, n_free_out, stream));
}

int rdg_qk_norm_rope_store(const void* qkv, int dtype, int64_t qkv_stride, int T, int n_q, int n_kv, int head_dim,
                           const float* q_weight, const float* k_weight, float eps, const float* cos_sin, int n_pos,
                           int rot_dim, int neighbours, const rdg_kv_step* S, const rdg_kv_cache* C, void* q_out,
                           int64_t q_stride, rdg_stream_t stream) {
    if (dtype != RDG_F32 && dtype != RDG_BF16) return RDG_EINVAL;
    if (T < 0 || n_q < 0 || n_kv < 0 || n_q > 4096 || n_kv > 4096 || !(eps >= 0.0f) || !step_ok(S)) return RDG_EINVAL;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return RDG_EUNSUPPORTED;
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0) return RDG_EINVAL;
    const int vec = dtype == RDG_BF16 ? 8 : 4;
    if (T > 0) {
        if (T > S->t_cap || !qkv || !aligned16(qkv) || qkv_stride < (int64_t)(n_q + 2 * n_kv) * head_dim ||
            qkv_stride % vec != 0)
            return RDG_EINVAL;
        if (rot_dim > 0 && (!cos_sin || !aligned16(cos_sin) || n_pos < 1 || !S->positions)) return RDG_EINVAL;
        if (n_q > 0 && (!q_out || !aligned16(q_out) || q_stride < (int64_t)n_q * head_dim || q_stride % vec != 0))
            return RDG_EINVAL;
        if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight))) return RDG_EINVAL;
    }
    QkStoreCall a = {};
    if (n_kv > 0) {
        const int rc = cache_rc(C);
        if (rc != RDG_OK) return rc;
        if (C->n_kv != n_kv || C->head_dim != head_dim || C->page_rows != S->page_rows || C->n_pages != S->n_pages)
            return RDG_EINVAL;
        if (T > 0 && (cache_buffers_rc(C) != RDG_OK || !S->slots || !S->seg_tok)) return RDG_EINVAL;
        a.k_codes = C->k, a.v_codes = C->v, a.k_scale = C->k_scale, a.v_scale = C->v_scale;
    }
    a.qkv = qkv, a.q_out = q_out, a.q_weight = q_weight, a.k_weight = k_weight, a.cos_sin = cos_sin;
    a.positions = S->positions, a.slots = S->slots, a.seg_tok = S->seg_tok, a.status = S->status;
    a.row_stride = qkv_stride, a.q_stride = q_stride, a.eps = eps;
    a.T = T, a.n_q = n_q, a.n_kv = n_kv, a.rot_dim = rot_dim, a.n_pos = n_pos, a.n_pages = S->n_pages;
    a.page_rows = S->page_rows, a.neighbours = neighbours != 0;
    return hip_rc(launch_qk_store(a, head_dim, dtype == RDG_BF16, n_kv > 0 ? S->seg_cap : 0, stream));
}

size_t rdg_paged_attention_workspace_bytes(const rdg_kv_cache* C, int T, int n_req, int n_q, int max_q, int max_kv,
                                           int dtype) {
    if (cache_rc(C) != RDG_OK || T <= 0 || n_req <= 0 || n_q < C->n_kv || n_q % C->n_kv != 0 || max_q <= 0 ||
        max_kv <= 0 || (int64_t)T * n_q >= (int64_t)1 << 31)
        return 0;
    if (max_q > T) max_q = T;
    if (max_kv > kMaxKeys) max_kv = kMaxKeys;
    const AttnPlan p = plan_attn(T, n_req, C->n_kv, n_q / C->n_kv, C->head_dim, dtype == RDG_BF16, max_q, max_kv);
    return p.row_bytes + p.tile_bytes;
}

int rdg_paged_attention(const void* q, int dtype, int64_t q_stride, int T, int n_q, const rdg_kv_step* S,
                        const rdg_kv_cache* C, int max_q, int max_kv, float scale, int causal, int window, void* out,
                        int64_t out_stride, float* lse, void* work, size_t work_bytes, rdg_stream_t stream) {
    if (dtype != RDG_F32 && dtype != RDG_BF16) return RDG_EINVAL;
    if (!step_ok(S) || T < 0 || n_q < 1 || max_q < 0 || max_kv < 0 || window < 0) return RDG_EINVAL;
    if (window > 0 && !causal) return RDG_EINVAL;
    if (window > kMaxKeys) window = kMaxKeys;
    if (max_kv > kMaxKeys) max_kv = kMaxKeys;
    if (!(scale > 0.0f) || !(scale < INFINITY)) return RDG_EINVAL;
    int rc = cache_rc(C);
    if (rc != RDG_OK) return rc;
    if (n_q % C->n_kv != 0 || n_q > 4096 || C->page_rows != S->page_rows || C->n_pages != S->n_pages) return RDG_EINVAL;
    if ((int64_t)T * n_q >= (int64_t)1 << 31) return RDG_EINVAL;
    if (T == 0 || S->n_req == 0 || max_q == 0) return RDG_OK;
    if (max_q > T) max_q = T;
    const int D = C->head_dim, vec = dtype == RDG_BF16 ? 8 : 4;
    if (!q || !out || !aligned16(q) || !aligned16(out) || cache_buffers_rc(C) != RDG_OK) return RDG_EINVAL;
    if (q_stride < (int64_t)n_q * D || q_stride % vec != 0 || out_stride < (int64_t)n_q * D || out_stride % vec != 0)
        return RDG_EINVAL;
    if (!S->block_table || !S->cu_q || !S->kv_len) return RDG_EINVAL;
    AttnCall a = {};
    a.q = q, a.out = out, a.lse = lse, a.block_table = S->block_table, a.cu_q = S->cu_q, a.kv_len = S->kv_len;
    a.k_codes = C->k, a.v_codes = C->v, a.k_scale = C->k_scale, a.v_scale = C->v_scale, a.status = S->status;
    a.q_stride = q_stride, a.out_stride = out_stride, a.scale_log2 = scale * 1.4426950408889634f;
    a.T = T, a.R = S->n_req, a.n_q = n_q, a.n_kv = C->n_kv, a.group = n_q / C->n_kv;
    a.max_blocks = S->max_blocks, a.n_pages = C->n_pages, a.page_shift = page_shift_of(C->page_rows);
    const int64_t table = (int64_t)S->max_blocks * C->page_rows;
    a.kv_cap = table < max_kv ? (int)table : max_kv;
    a.max_q = max_q, a.window = window, a.causal = causal != 0;
    const bool bf16 = dtype == RDG_BF16;
    // The workspace is sized for all max_kv keys.  A window leaves a shorter run,
    // which may be cut finer than the workspace holds parts for: then coarser.
    const int span = key_span(max_q, max_kv, window);
    const AttnPlan most = plan_attn(T, a.R, a.n_kv, a.group, D, bf16, max_q, max_kv);
    AttnPlan p = plan_attn(T, a.R, a.n_kv, a.group, D, bf16, max_q, span);
    const size_t need = most.row_bytes + most.tile_bytes;
    if (need > 0 && (!work || !aligned16(work) || work_bytes < need)) return RDG_EINVAL;
    if (p.tile_slots > 0) coarsen(&p.tile_chunk, &p.tile_chunks, span, most.tile_chunks);
    if (p.n_most > 0) coarsen(&p.chunk, &p.row_chunks, span, most.row_chunks);
    a.n_most = p.n_most, a.rows_per_tile = 16 * p.rt, a.row_places = p.row_places, a.chunk = p.chunk;
    a.row_chunks = p.row_chunks, a.tile_rows = p.tile_rows, a.tile_slots = p.tile_slots;
    a.tile_chunk = p.tile_chunk, a.tile_chunks = p.tile_chunks;
    a.row_place = p.row_place;
    if (p.row_chunks > 1) {
        const int64_t places = p.row_place > 0 ? (int64_t)a.R * p.row_place : T;
        a.row_o = static_cast<float*>(work);
        a.row_ml = a.row_o + (size_t)places * n_q * D * p.row_chunks;
    }
    if (p.tile_chunks > 1) {
        a.tile_o = reinterpret_cast<float*>(static_cast<char*>(work) + most.row_bytes);
        a.tile_ml = a.tile_o + (size_t)T * n_q * D * p.tile_chunks;
    }
    const bool join = p.row_chunks > 1 || p.tile_chunks > 1;
    if (join && !grid_fits(T, kJoinThreads)) return RDG_EUNSUPPORTED;  // before anything is enqueued
    hipError_t e = p.tile_slots > 0 ? launch_attn_tiles(a, D, stream) : launch_attn_rows(a, D, bf16, stream);
    if (e == hipSuccess && join) e = launch_attn_join(a, D, bf16, stream);
    return hip_rc(e);
}

}  // extern "C"
