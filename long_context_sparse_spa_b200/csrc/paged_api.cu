// Host side of the paged KV cache entry points: argument validation and launches.  Nothing here
// allocates device memory or reads it.
#include <climits>

#include "paged.cuh"

namespace spa {
namespace {

// Checks a cache's description; SPA_OK with *noop when it holds no sequence.
spa_status check_kv(const spa_paged_kv& kv, bool* noop, PagedView* v) {
    *noop = false;
    if (kv.format != SPA_KV_BF16 && kv.format != SPA_KV_INT4) return SPA_ERR_INVALID_ARG;
    if (kv.B < 0 || kv.Hkv <= 0 || kv.num_pages < 0 || kv.max_pages < 0 || kv.page <= 0) return SPA_ERR_INVALID_ARG;
    if (kv.B == 0) {
        *noop = true;
        return SPA_OK;
    }
    if (kv.d != 64 && kv.d != 128) return SPA_ERR_UNSUPPORTED_SHAPE;
    if (kv.page < 16 || kv.page > 1024 || (kv.page & (kv.page - 1))) return SPA_ERR_UNSUPPORTED_SHAPE;
    if (kv.B > 65535 || kv.Hkv > 65535) return SPA_ERR_UNSUPPORTED_SHAPE;
    int shift = 0;
    while ((1 << shift) < kv.page) ++shift;
    // rows of the pool are counted in 32 bits (more would not fit a GPU)
    if ((long long)kv.num_pages * kv.Hkv > (0xfffffffell >> shift)) return SPA_ERR_UNSUPPORTED_SHAPE;
    // lengths are 32-bit: tokens that a page table can name must be too
    if (((long long)kv.max_pages << shift) > INT_MAX - 4096) return SPA_ERR_UNSUPPORTED_SHAPE;
    if (!kv.kv_len || (kv.max_pages > 0 && !kv.page_table) || (kv.num_pages > 0 && !kv.data)) return SPA_ERR_INVALID_ARG;
    if (!aligned16(kv.data)) return SPA_ERR_UNSUPPORTED_SHAPE;
    v->data = static_cast<uint8_t*>(kv.data);
    v->page_table = kv.page_table;
    v->kv_len = kv.kv_len;
    v->num_pages = kv.num_pages;
    v->Hkv = kv.Hkv;
    v->page_shift = shift;
    v->d = kv.d;
    v->B = kv.B;
    v->max_pages = kv.num_pages > 0 ? kv.max_pages : 0;   // without a page nothing is looked up: a length above 0 is an error
    v->int4 = kv.format == SPA_KV_INT4;
    v->row_bytes = paged_row_bytes(v->int4, kv.d);
    return SPA_OK;
}

// rows [T, heads, d] with strides: 16-byte loads of whole 8-channel pieces
spa_status check_rows(const void* p, int64_t tok, int64_t head) {
    if (!p) return SPA_ERR_INVALID_ARG;
    if (!aligned16(p) || tok % 8 || head % 8) return SPA_ERR_UNSUPPORTED_SHAPE;
    if (tok < 0 || head < 0) return SPA_ERR_INVALID_ARG;
    return SPA_OK;
}

// whether out [T, Hq, d] of `bytes` per element reaches into the stretch of rows [T, heads, d] at p
bool overlaps(const void* out, size_t bytes, int T, int Hq, int d, const uint16_t* p, int heads, int64_t tok, int64_t head) {
    const uintptr_t o = reinterpret_cast<uintptr_t>(out), r = reinterpret_cast<uintptr_t>(p);
    const uintptr_t o1 = o + uintptr_t(T) * Hq * d * bytes, r1 = r + 2 * (uintptr_t(T - 1) * tok + uintptr_t(heads - 1) * head + d);
    return o < r1 && r < o1;
}

}  // namespace
}  // namespace spa

using namespace spa;

extern "C" {

size_t spa_paged_row_bytes(int format, int d) {
    if ((format != SPA_KV_BF16 && format != SPA_KV_INT4) || d <= 0) return 0;
    return size_t(paged_row_bytes(format == SPA_KV_INT4, d));
}

spa_status spa_paged_append(const spa_paged_append_args* a, void* ws, size_t ws_bytes, void* stream) {
    if (!a) return SPA_ERR_INVALID_ARG;
    PagedAppendParams p{};
    bool noop;
    spa_status s = check_kv(a->kv, &noop, &p.kv);
    if (s != SPA_OK) return s;
    if (a->T < 0 || (a->q && (a->Hq <= 0 || a->Hq > 65535))) return SPA_ERR_INVALID_ARG;
    if (noop || a->T == 0) return SPA_OK;
    if (!a->seq_start && a->T != a->kv.B) return SPA_ERR_INVALID_ARG;
    s = check_rows(a->k, a->k_token_stride, a->k_head_stride);
    if (s == SPA_OK) s = check_rows(a->v, a->v_token_stride, a->v_head_stride);
    if (s == SPA_OK && a->q) s = check_rows(a->q, a->q_token_stride, a->q_head_stride);
    if (s != SPA_OK) return s;
    if (a->q && (!a->q_out || a->q_out == a->q)) return SPA_ERR_INVALID_ARG;
    if (a->q && !aligned16(a->q_out)) return SPA_ERR_UNSUPPORTED_SHAPE;
    const int d = a->kv.d, Hkv = a->kv.Hkv;
    if (a->q && (overlaps(a->q_out, 2, a->T, a->Hq, d, a->q, a->Hq, a->q_token_stride, a->q_head_stride) ||
                 overlaps(a->q_out, 2, a->T, a->Hq, d, a->k, Hkv, a->k_token_stride, a->k_head_stride) ||
                 overlaps(a->q_out, 2, a->T, a->Hq, d, a->v, Hkv, a->v_token_stride, a->v_head_stride)))
        return SPA_ERR_INVALID_ARG;
    if (a->rot < 0 || a->rot > a->kv.d || (a->rot > 0 && !a->inv_freq)) return SPA_ERR_INVALID_ARG;
    if (a->rot % 16) return SPA_ERR_UNSUPPORTED_SHAPE;
    if (ws && ws_bytes < kWsHeader) return SPA_ERR_WORKSPACE_TOO_SMALL;
    p.T = a->T;
    p.Hq = a->Hq;
    p.seq_start = a->seq_start;
    p.positions = a->positions;
    p.k = a->k;
    p.v = a->v;
    p.q = a->q;
    p.k_tok = a->k_token_stride;
    p.k_head = a->k_head_stride;
    p.v_tok = a->v_token_stride;
    p.v_head = a->v_head_stride;
    p.q_tok = a->q_token_stride;
    p.q_head = a->q_head_stride;
    p.q_out = a->q_out;
    p.inv_freq = a->inv_freq;
    p.rot = a->rot;
    p.interleaved = a->interleaved;
    p.status = static_cast<uint32_t*>(ws);
    return launch_paged_append(p, static_cast<cudaStream_t>(stream));
}

spa_status spa_paged_gather(const spa_paged_gather_args* a, void* ws, size_t ws_bytes, void* stream) {
    if (!a) return SPA_ERR_INVALID_ARG;
    PagedGatherParams p{};
    bool noop;
    const spa_status s = check_kv(a->kv, &noop, &p.kv);
    if (s != SPA_OK) return s;
    if (a->N < 0) return SPA_ERR_INVALID_ARG;
    if (noop || a->N == 0) return SPA_OK;
    if (!a->K || !a->V) return SPA_ERR_INVALID_ARG;
    if (!aligned16(a->K) || !aligned16(a->V)) return SPA_ERR_UNSUPPORTED_SHAPE;
    if (ws && ws_bytes < kWsHeader) return SPA_ERR_WORKSPACE_TOO_SMALL;
    p.N = a->N;
    p.start = a->start;
    p.K = a->K;
    p.V = a->V;
    p.status = static_cast<uint32_t*>(ws);
    return launch_paged_gather(p, static_cast<cudaStream_t>(stream));
}

static bool chunk_taken(const spa_paged_attend_args* a) {
    return a->kv.Hkv > 0 && paged_chunk_taken(a->seq_start, a->idx, a->T, a->Hq, a->kv.Hkv, a->kv.B,
                                              a->sm_scale);
}

size_t spa_paged_attend_workspace_bytes(const spa_paged_attend_args* a) {
    if (!a || a->kv.d <= 0 || a->kv.Hkv <= 0 || a->kv.B <= 0 || a->T < 0) return 0;
    if (a->Hq <= 0 || a->Hq % a->kv.Hkv) return 0;     // (no heads per kv head to divide by)
    if (chunk_taken(a)) return kWsHeader + paged_chunk_scratch_bytes(a->kv.d);
    const bool sparse = a->idx != nullptr;
    const int heads = sparse && a->collapse == SPA_COLLAPSE_NONE ? 1 : a->Hq / a->kv.Hkv;
    return kWsHeader + paged_attend_scratch_bytes(a->kv.d, a->T, a->kv.B, heads, sparse);
}

spa_status spa_paged_attend(const spa_paged_attend_args* a, void* ws, size_t ws_bytes, void* stream) {
    if (!a) return SPA_ERR_INVALID_ARG;
    PagedAttendParams p{};
    bool noop;
    spa_status s = check_kv(a->kv, &noop, &p.kv);
    if (s != SPA_OK) return s;
    if (a->T < 0 || a->Hq <= 0 || a->Hq % a->kv.Hkv) return SPA_ERR_INVALID_ARG;
    if (noop || a->T == 0) return SPA_OK;
    if (!a->seq_start && a->T != a->kv.B) return SPA_ERR_INVALID_ARG;
    if (!a->out || !ws || (a->idx == nullptr) != (a->count == nullptr)) return SPA_ERR_INVALID_ARG;
    s = check_rows(a->q, a->q_token_stride, a->q_head_stride);
    if (s != SPA_OK) return s;
    // (channels of a query tile's rows, 256 tokens of all heads, are counted in 32 bits)
    if (a->Hq / a->kv.Hkv > 16 || a->Hq > 65535) return SPA_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(a->out) || !aligned16(a->out_f32) || !aligned16(ws)) return SPA_ERR_UNSUPPORTED_SHAPE;
    if (a->idx) {
        if (a->T > a->kv.B || a->cap < 0 || a->unit_tokens <= 0) return SPA_ERR_INVALID_ARG;
        if (a->collapse != SPA_COLLAPSE_NONE && a->collapse != SPA_COLLAPSE_GROUP_MEAN) return SPA_ERR_INVALID_ARG;
    }
    if (ws_bytes < spa_paged_attend_workspace_bytes(a)) return SPA_ERR_WORKSPACE_TOO_SMALL;
    if (overlaps(a->out, 2, a->T, a->Hq, a->kv.d, a->q, a->Hq, a->q_token_stride, a->q_head_stride) ||
        (a->out_f32 && overlaps(a->out_f32, 4, a->T, a->Hq, a->kv.d, a->q, a->Hq, a->q_token_stride, a->q_head_stride)))
        return SPA_ERR_INVALID_ARG;
    uint8_t* const w = static_cast<uint8_t*>(ws);
    p.T = a->T;
    p.Hq = a->Hq;
    p.seq_start = a->seq_start;
    p.q = a->q;
    p.q_tok = a->q_token_stride;
    p.q_head = a->q_head_stride;
    p.idx = a->idx;
    p.count = a->count;
    p.cap = a->cap;
    p.collapse = a->collapse;
    p.unit_tokens = a->idx ? a->unit_tokens : 1;
    p.sm_scale = a->sm_scale;
    p.out = a->out;
    p.out_f32 = a->out_f32;
    p.lse = a->lse;
    p.status = reinterpret_cast<uint32_t*>(w);
    paged_carve(p, w + kWsHeader);
    if (chunk_taken(a)) return launch_paged_chunk(p, static_cast<cudaStream_t>(stream));
    return launch_paged_attend(p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
