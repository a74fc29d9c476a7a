// Declarations shared by the paged KV cache kernels (paged.cu, paged_attend.cu) and their host side.
#pragma once
#include "internal.cuh"
#include "paged_map.h"

namespace spa {

struct PagedAppendParams {
    PagedView kv;
    int T, Hq;
    const int32_t* seq_start;   // [B + 1] or null
    const int32_t* positions;   // [T] or null
    const uint16_t *k, *v, *q;  // q null: keys and values only
    long long k_tok, k_head, v_tok, v_head, q_tok, q_head;   // strides in elements
    uint16_t* q_out;            // [T, Hq, d]
    const float* inv_freq;      // [rot / 2]
    int rot, interleaved;
    uint32_t* status;
};
spa_status launch_paged_append(const PagedAppendParams& p, cudaStream_t st);

struct PagedGatherParams {
    PagedView kv;
    int N;
    const int32_t* start;       // [B] or null
    uint16_t *K, *V;            // [B, Hkv, N, d]
    uint32_t* status;
};
spa_status launch_paged_gather(const PagedGatherParams& p, cudaStream_t st);

struct PagedAttendParams {
    PagedView kv;
    int T, Hq;
    const int32_t* seq_start;
    const uint16_t* q;
    long long q_tok, q_head;
    const int32_t* idx;         // null: every cached token
    const int32_t* count;
    int cap, collapse, unit_tokens;
    float sm_scale;
    uint16_t* out;              // [T, Hq, d]
    float* out_f32;
    float* lse;                 // [T, Hq]
    int* arrived;               // [2 * SMs]: finished shares of the split unit that starts in a CTA; 0 between calls
    float* partials;            // [2 * CTAs] shares of split units
    uint32_t* status;
    uint32_t spin;              // tries of a bounded wait
    int stall;                  // test hook (spa_test_stall): what a wait is for never starts
};
spa_status launch_paged_attend(const PagedAttendParams& p, cudaStream_t st);
size_t paged_attend_scratch_bytes(int d, int T, int B, int heads, bool sparse);
// paged_chunk.cu: more than 32 rows per sequence and kv head on average.  16 sequences of 4096, 32 / 8 heads, mma.sync
// and tcgen05: 4-bit 72 and 95 us at 32 rows, 118 and 95 at 36; bf16 95 and 106 us at 32 rows, 165 and 107 at 36.
// All rows of a call go the same way: 64 sequences of 4096 with one token and one with 1024 take 512 us in one call, in
// two calls 91 and 122; measured with equal sequences only, the rule is wrong for such a batch.
inline bool paged_chunk_taken(const void* seq_start, const void* idx, int T, int Hq, int Hkv, int B,
                              float sm_scale) {
    return seq_start && !idx && sm_scale > 0.f && (long long)T * (Hq / Hkv) > 32ll * B;
}
spa_status launch_paged_chunk(const PagedAttendParams& p, cudaStream_t st);
size_t paged_chunk_scratch_bytes(int d);
// The workspace after its header: arrival counters, 0 between calls, then the shares of split units, of no meaning
// between calls.  Both kernels have their counters in the same place, so that a workspace that is large enough serves
// calls of either in turn.
inline size_t paged_counter_bytes() { return align_up(size_t(device_info().num_sms) * 2 * sizeof(int), 256); }
inline void paged_carve(PagedAttendParams& p, uint8_t* scratch) {
    p.arrived = reinterpret_cast<int*>(scratch);
    p.partials = reinterpret_cast<float*>(scratch + paged_counter_bytes());
}
constexpr int kPagedMaxUnits = 512;   // sequences, or supports, of one launch: 4 bytes of shared memory each

}  // namespace spa
