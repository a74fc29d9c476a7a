// Exact softmax attention over a paged KV cache, bf16 or 4-bit: decode (one query per sequence), a few
// drafted or chunked queries per sequence (causal among themselves), or decode restricted to supports.
//
// Work split: a unit is one tile of up to 32 (query, head) rows that share the keys of one (sequence,
// kv head), or one support.  Its keys are cut into tiles of TILE tokens; the tiles of all units form one
// list (each unit charged kSeg tiles for its start-up and merge), split evenly over the CTAs (one per
// SM; two for 4-bit rows and up to eight rows of a unit).  Inside a CTA the warps take a unit's tiles round-robin; each warp copies its tiles into its own
// ring with bulk asynchronous copies, one per run of tokens that lie together on a page.
//
// Math per 16 tokens on tensor cores (mma.sync m16n8k16, fp32 accumulation), transposed so that tokens
// fill the 16-row side and heads the 8-column side:
//   4-bit keys: S = sum_g s_g (sum_{c in g} q_c u_c - 8 sum_{c in g} q_c), u the code 0..15.
//     A nibble masked out of its word is an fp16 denormal, u * 2^-24 in bits 0-3 and u * 2^-20 in bits
//     4-7: one AND per two codes makes the A operand, exactly.  q is scaled by a power of two into
//     fp16's range (and by 1/16 for the second kind), exactly above 2^-24 of its largest channel; the
//     group scale multiplies in fp32, and the -8 terms are one more product, scales times three bf16
//     terms of the sums.
//   4-bit values: with 2^e the power of two of the token's largest s, r_g = s_g 2^-e and P = p 2^e, O += V^T P^T
//     with V = (u - 8) r_g, one fp16 FMA per two codes after the AND.  V has 3 + 8 bits and is exact (a group's
//     scale below 2^-11 of its token's largest: within 2^-19 of that); only the weight is rounded, to fp16's 11
//     bits, three more than the outputs have.  A transposing ldmatrix over 16-bit units (four codes of a token)
//     pairs tokens for the A operand.  So that P fits fp16 whatever the scales are, the running reference of the
//     softmax is the maximum of (logit + e), not of the logit; P <= 2^15, and l = sum p is kept in fp32.
//   bf16 rows: S = K Q^T, O += V^T P^T with P = hi + lo bf16 (about 16 bits).
// The m16 rows of a tile are a permutation of its tokens (tau) that keeps the shared-memory reads free
// of bank conflicts for the rows' strides; a softmax does not see the order.
//
// At the end of its share of a unit a CTA merges its warps in shared memory and writes the output, or a
// partial (o, m, l) if the unit is split; the last CTA of a split unit to finish merges its partials in the
// order of the CTAs, so equal calls give equal bits.
//
// Measured on B200: 4-bit, 4 sequences of 128K, 32 query / 4 kv heads, d = 128 (302 MB): 81 us, 3.7 TB/s.  60 % of the
// issue slots and 52 % of the ALU pipe are used; 15 warps per SM do not hide the chain of the unpacking (about 630
// instructions per 32 tokens and 8 heads), and copying alone takes 66 us with the start and the merge, 20 above the
// bytes' time.  bf16, 64K: 94 us, 5.7 TB/s; bound by memory.  One sequence of 4096 tokens and one kv head: 10.8 us, a
// chain of lookups, one copy, one tile and two merges.
#include "paged.cuh"
#include "warp_mma.cuh"

#include <cuda_fp16.h>

#include <type_traits>

namespace spa {
namespace {

constexpr int kRowsMax = 32;              // (query, head) rows of a unit
constexpr int kSeg = 32;                  // tiles charged to a unit for its start-up and merge
constexpr int kShare = 16;                // least weighted tiles of a CTA's share
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFloorV = 8.077935669463161e-28f;   // 2^-90: least value scale that the reference follows (l = sum P / 2^e)
constexpr float kBase = 9.f;              // weights are 2^9 at the reference, and at most 2^(9 + kSlack)
constexpr float kSlack = 6.f;             // the reference moves only when it is exceeded by this (log2)
constexpr uint32_t kWaitLimit = 1u << 22, kStallLimit = 1u << 10;   // tries of a wait; with the test hook

// floats of one share of a split unit
__host__ __device__ constexpr int paged_rec_floats(int d, int rows) { return rows * (d + 2); }

template <int D, bool INT4, int NT>
struct Geo {
    static constexpr int ROWB = INT4 ? D + 16 : 4 * D;
    static constexpr int TILE = INT4 ? 32 : 16;           // tokens per warp step
    static constexpr int MT = TILE / 16;
    static constexpr int STAGES = 3;
    static constexpr int WARPS = INT4 && NT == 2 ? 12 : 8;
    static constexpr int CTAS = INT4 && NT == 1 ? 2 : 1;  // per SM
    // more than one column tile: the queries' operand fragments lie in shared memory, not in registers
    static constexpr bool QS = NT > 1;
    static constexpr int QBYTES = QS ? NT * (D / 16 + 3) * 256 : 0;
    // shared-memory row stride: bf16 rows are copied one by one and padded (a multiple of 128 bytes would put
    // the eight rows of a fragment on the same banks)
    static constexpr int SROW = INT4 ? ROWB : ROWB + 16;
    static constexpr int RING = WARPS * STAGES * TILE * SROW;
    // the warps' parts, their factors and (M, L); the merge of shares puts a factor of each over the parts
    static constexpr int MERGE = WARPS * NT * 8 * (D + 2) * 4 + NT * 8 * (WARPS + 2) * 4;
    static constexpr int PREP = INT4 ? WARPS * TILE * 8 : 0;   // (e, 2^-e) of each token's largest value scale
    static constexpr int SMEM = (RING > MERGE ? RING : MERGE) + PREP + QBYTES;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {   // of a number and a NaN the number
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.u32 [%0], {%1,%2};\n" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;\n" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ void sts128_zero(uint32_t a) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};\n" ::"r"(a), "r"(0) : "memory");
}

// Row r (0..7) of a 16-row tile is token tau(r), row r + 8 token tau(r) + 8.  Keys are read two (d = 128:
// 16 bytes a lane) or four rows (d = 64) at a time, which must lie on different banks: rows of 144 and 528
// bytes step by 4 banks, so d = 128 and bf16 want neighbours 4 apart, {0,4,1,5,2,6,3,7}; rows of 80 bytes step
// by 20, so d = 64 wants {0,2,4,6,1,3,5,7}.  Transposing loads take any order of the eight.
template <int D, bool INT4>
__device__ __forceinline__ int tau(int r) {
    return INT4 && D == 64 ? int((0x75316420u >> (4 * r)) & 15u) : int((0x73625140u >> (4 * r)) & 15u);
}
// the row that holds token n (0..7)
template <int D, bool INT4>
__device__ __forceinline__ int tau_inv(int n) {
    return INT4 && D == 64 ? int((0x73625140u >> (4 * n)) & 15u) : int((0x75316420u >> (4 * n)) & 15u);
}

struct Unit {
    int b, g, h0;       // sequence, kv head, first query head
    int row0;           // first query row of q / out
    int nq;             // query tokens
    int heads;          // query heads per token
    int lim0;           // keys the first query token may see (the i-th: lim0 + i)
    int len;            // tokens of the sequence
    int u;              // support, or -1
    int ntok;           // tokens to visit (dense: keys of the last query; support: entries * unit_tokens)
};

struct SeqGeo { int n, len, row0; };
__device__ __forceinline__ SeqGeo seq_geo(const PagedAttendParams& p, int b, bool* bad) {
    SeqGeo s;
    s.len = paged_len(p.kv, p.kv.kv_len[b], bad);
    if (!p.seq_start) {
        s.n = b < p.T ? 1 : 0;
        s.row0 = b;
    } else {
        const long long a = p.seq_start[b], e = p.seq_start[b + 1];
        if (!paged_rows_ok(a, e, p.T)) { *bad = true; s.n = 0; s.row0 = 0; }
        else { s.n = int(e - a); s.row0 = int(a); }
    }
    return s;
}

// Query row of a sequence's one new token, or -1: it has none, or (an error with supports) several.
__device__ __forceinline__ int one_row(const PagedAttendParams& p, int b, bool* bad) {
    if (!p.seq_start) return b;
    const int a = p.seq_start[b], e = p.seq_start[b + 1];
    if (paged_rows_ok(a, e, p.T) && e - a == 1) return a;
    if (e != a) *bad = true;
    return -1;
}

// tokens that support u names, or -1: its sequence has no query
__device__ __forceinline__ int support_tokens(const PagedAttendParams& p, int u, bool* bad) {
    if (one_row(p, u / (p.collapse == SPA_COLLAPSE_GROUP_MEAN ? p.kv.Hkv : p.Hq), bad) < 0) return -1;
    int c = p.count[u];
    c = c < 0 ? 0 : c > p.cap ? p.cap : c;
    const long long n = (long long)c * p.unit_tokens;
    return n > 0x3fffffff ? 0x3fffffff : int(n);
}

// Weighted tiles of one kv head of a sequence: sum over its query tiles of (tiles + kSeg).
template <int TILE>
__device__ __forceinline__ long long head_weight(const SeqGeo& s, int TQ) {
    long long w = 0;
    const int nj = (s.n + TQ - 1) / TQ;
    for (int j = 0; j < nj; ++j) {
        const int lim = paged_tile_limit(s.len, s.n, TQ, j);
        if (lim > 0) w += (lim + TILE - 1) / TILE + kSeg;
    }
    return w;
}

template <int D, bool INT4, int NT>
__global__ void __launch_bounds__(Geo<D, INT4, NT>::WARPS * 32, Geo<D, INT4, NT>::CTAS)
paged_attend_kernel(PagedAttendParams p, int g0, int groups, int TQ) {
    using G_ = Geo<D, INT4, NT>;
    constexpr int kWarps = G_::WARPS, kThreads = kWarps * 32, ROWS = NT * 8;
    constexpr int TILE = G_::TILE, ROWB = G_::ROWB, SROW = G_::SROW, STAGES = G_::STAGES, MT = G_::MT;
    constexpr int KS = D / 16;                 // k-steps of S, and 16-channel tiles of O
    constexpr int DT = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* const ring = smem;
    uint32_t* const s_prefix = reinterpret_cast<uint32_t*>(smem + G_::SMEM);   // [groups + 1]
    const uint32_t prep = smem_u32(smem + G_::SMEM - G_::PREP - G_::QBYTES + (INT4 ? (threadIdx.x >> 5) * TILE * 8 : 0));
    // per column tile: KS k-steps of (b0, b1) by lane, then (qz0, qz1), (hs0, hs1) and the two columns' limits
    constexpr bool QS = G_::QS;
    const uint32_t qs = smem_u32(smem + G_::SMEM - G_::QBYTES) + (threadIdx.x & 31) * 8;
    __shared__ uint64_t s_full[kWarps][STAGES];
    __shared__ uint32_t s_vmask[kWarps][STAGES];
    __shared__ long long s_wsum[kWarps];
    __shared__ int s_last;
    __shared__ long long s_seg[3];       // the unit's first and last weighted tile, and where this CTA goes on

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r8 = lane >> 2, t4 = lane & 3;
    if (lane < STAGES) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(smem_u32(&s_full[warp][lane])));
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    }
    pdl_enter();
    const bool sparse = p.idx != nullptr;
    const int G = p.Hq / p.kv.Hkv;

    // ---- weighted tile prefix over the groups [g0, g0 + groups): sequences (all kv heads), or supports
    long long running = 0;
    bool empties = false;     // some query of the launch sees nothing
    for (int base = 0; base < groups; base += kThreads) {
        const int u = base + tid;
        long long t = 0;
        if (u < groups) {
            if (sparse) {
                bool bad = false;
                const int n = support_tokens(p, g0 + u, &bad);
                t = n > 0 ? (n + TILE - 1) / TILE + kSeg : 0;
                empties |= n == 0;
                if (bad && blockIdx.x == 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
            } else {
                bool bad = false;
                const SeqGeo s = seq_geo(p, g0 + u, &bad);
                t = head_weight<TILE>(s, TQ) * p.kv.Hkv;
                empties |= s.n > 0 && paged_tile_limit(s.len, s.n, TQ, 0) == 0;
                if (bad && blockIdx.x == 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
            }
        }
        long long incl = t;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += x;
        }
        if (lane == 31) s_wsum[warp] = incl;
        __syncthreads();
        long long before = running, tot = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += s_wsum[w];
            tot += s_wsum[w];
        }
        if (u < groups) s_prefix[u] = uint32_t(before + incl - t);
        running += tot;
        __syncthreads();
    }
    if (tid == 0) s_prefix[groups] = uint32_t(running);
    empties = __syncthreads_or(empties);
    // Starts out of order can make sequences overlap, and their tiles more than the host counted and the prefix holds.
    if (running > 0xffffffffll) {
        if (blockIdx.x == 0 && tid == 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
        running = 0;
    }
    const long long TT = running;
    const int cta = blockIdx.x;
    // CTAs with work: none gets less than about kShare tiles, since every share of a unit is merged
    const long long shares = (TT + kShare - 1) / kShare;
    const int GC = int(shares < (long long)gridDim.x ? shares : (long long)gridDim.x);

    // ---- units without a key: out = 0, lse = -inf
    auto write_empty = [&](int row0, int nrow, int h0, int nh) {
        for (int i = tid; i < nrow * nh * D; i += kThreads) {
            const int c = i % D, h = (i / D) % nh, q = i / (D * nh);
            const size_t o = (size_t(row0 + q) * p.Hq + h0 + h) * D + c;
            p.out[o] = 0;
            if (p.out_f32) p.out_f32[o] = 0.f;
            if (p.lse && c == 0) p.lse[size_t(row0 + q) * p.Hq + h0 + h] = -INFINITY;
        }
    };
    for (int u = cta; empties && u < groups; u += gridDim.x) {
        if (sparse) {
            if (s_prefix[u + 1] != s_prefix[u]) continue;
            const bool grp = p.collapse == SPA_COLLAPSE_GROUP_MEAN;
            const int per = grp ? p.kv.Hkv : p.Hq;
            bool bad = false;
            const int row = one_row(p, (g0 + u) / per, &bad);
            if (row >= 0) write_empty(row, 1, ((g0 + u) % per) * (grp ? G : 1), grp ? G : 1);
        } else {
            bool bad = false;
            const SeqGeo s = seq_geo(p, g0 + u, &bad);
            // query tiles whose last query sees no key
            const int nj = (s.n + TQ - 1) / TQ;
            for (int j = 0; j < nj && paged_tile_limit(s.len, s.n, TQ, j) == 0; ++j)
                write_empty(s.row0 + j * TQ, min(TQ, s.n - j * TQ), 0, p.Hq);
        }
    }
    if (cta >= GC) return;

    const long long x0 = TT * cta / GC, x1 = TT * (cta + 1) / GC;
    int grp;
    {
        int lo = 0, hi = groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_prefix[mid] <= x0) lo = mid; else hi = mid;
        }
        grp = lo;
    }
    const float sl2 = p.sm_scale * kLog2e;
    uint32_t phases = 0;      // parity of each stage's barrier
    bool failed = false;      // a wait of this warp gave up: it copies nothing more
    uint8_t* const my_ring = ring + size_t(warp) * STAGES * TILE * SROW;

    long long x = x0;
    while (x < x1) {
        while (s_prefix[grp + 1] <= x) ++grp;
        // ---- the unit at weighted tile x
        Unit un;
        long long u_lo;       // first weighted tile of the unit
        int tiles;
        bool bad = false;
        if (sparse) {
            const bool gm = p.collapse == SPA_COLLAPSE_GROUP_MEAN;
            const int per = gm ? p.kv.Hkv : p.Hq;
            un.b = (g0 + grp) / per;
            const int r = g0 + grp - un.b * per;
            un.g = gm ? r : r / G;
            un.h0 = gm ? r * G : r;
            un.heads = gm ? G : 1;
            un.row0 = one_row(p, un.b, &bad);
            un.nq = 1;
            un.len = paged_len(p.kv, p.kv.kv_len[un.b], &bad);
            un.lim0 = un.len;
            un.u = g0 + grp;
            un.ntok = support_tokens(p, g0 + grp, &bad);
            u_lo = s_prefix[grp];
            tiles = (un.ntok + TILE - 1) / TILE;
        } else {
            const SeqGeo s = seq_geo(p, g0 + grp, &bad);
            const long long hw = (s_prefix[grp + 1] - s_prefix[grp]) / p.kv.Hkv;
            long long rem = x - s_prefix[grp];
            un.g = int(rem / hw);
            rem -= un.g * hw;
            u_lo = s_prefix[grp] + un.g * hw;
            int j = 0, lim;
            for (;;) {
                lim = paged_tile_limit(s.len, s.n, TQ, j);
                const long long w = lim > 0 ? (lim + TILE - 1) / TILE + kSeg : 0;
                if (rem < w) break;
                rem -= w;
                u_lo += w;
                ++j;
            }
            un.b = g0 + grp;
            un.h0 = un.g * G;
            un.heads = G;
            un.row0 = s.row0 + j * TQ;
            un.nq = min(TQ, s.n - j * TQ);
            un.len = s.len;
            un.lim0 = lim - un.nq + 1;
            un.u = -1;
            un.ntok = lim;
            tiles = (lim + TILE - 1) / TILE;
        }
        const long long u_hi = u_lo + kSeg + tiles;
        const long long seg_end = x1 < u_hi ? x1 : u_hi;
        const int a = int(x - u_lo) - kSeg > 0 ? int(x - u_lo) - kSeg : 0;
        const int bnd = int(seg_end - u_lo) - kSeg > 0 ? int(seg_end - u_lo) - kSeg : 0;
        if (a >= bnd) {       // only the unit's fixed cost lies in this CTA's range
            x = seg_end;
            continue;
        }
        if (tid == 0) {       // kept in shared memory over the tile loop
            s_seg[0] = u_lo;
            s_seg[1] = u_hi;
            s_seg[2] = seg_end;
        }
        const int nrow = un.nq * un.heads;

        // ---- copying: lane i fetches the i-th run of R tokens of a tile
        const int ut = p.unit_tokens;
        int rsh = !INT4 ? 0 : min(5, p.kv.page_shift);   // R = 1 << rsh
        if (sparse) rsh = min(rsh, __ffs(ut) - 1);
        const int R = 1 << rsh;
        constexpr int kTileSh = TILE == 32 ? 5 : 4;
        const int runsh = kTileSh - rsh;
        const int n_my = a + warp < bnd && !failed ? (bnd - a - warp + kWarps - 1) / kWarps : 0;
        const int persh = 5 - runsh;            // tiles whose runs the lanes hold at once (a batch): lane i has run
        const int my_tile = lane >> runsh, my_run = lane & ((1 << runsh) - 1);   // my_run of the batch's tile my_tile
        // first token of this lane's run in batch k of my tiles, or -1
        auto token_of = [&](int k) -> int {
            const int j = (k << persh) + my_tile;
            if (j >= n_my) return -1;
            const int i = (a + warp + j * kWarps) * TILE + my_run * R;
            if (i >= un.ntok) return -1;
            if (!sparse) return i;
            const int e = ut == 1 ? i : i / ut;
            const long long n = (long long)__ldg(p.idx + size_t(un.u) * p.cap + e) * ut + (i - e * ut);
            return n >= 0 && n < un.len ? int(n) : -1;
        };
        auto page_of = [&](int n) -> int {
            const long long s = paged_slot(p.kv, un.b, n);
            return s < 0 ? -1 : __ldg(p.kv.page_table + s);
        };
        // the batch in hand: address and bytes of this lane's run
        const uint8_t* src = nullptr;
        int valid = 0;
        auto take = [&](int n, int pid) {
            valid = 0;                          // tokens of the run that exist
            if (n < 0) return;
            const long long off = paged_row(p.kv, pid, un.g, n);
            if (off < 0) {
                raise_status(p.status, SPA_ERR_INVALID_ARG);
                return;
            }
            valid = min(R, un.len - n);
            if (!sparse) valid = min(valid, un.ntok - n);
            src = p.kv.data + off;
        };
        constexpr uint32_t kFull = TILE == 32 ? 0xffffffffu : (1u << TILE) - 1u;
        int fill = 0;                           // the stage that is filled next
        uint32_t ragged = 0;                    // runs of the batch in hand that are not whole
        auto issue = [&](int j) {               // tile j of mine, which is in the batch in hand
            const int stage = fill;
            fill = fill + 1 == STAGES ? 0 : fill + 1;
            if (p.stall) return;
            const uint32_t bar = smem_u32(&s_full[warp][stage]);
            const uint32_t dst = smem_u32(my_ring + size_t(stage) * TILE * SROW);
            const int slot = j & ((1 << persh) - 1);
            const bool mine = my_tile == slot;
            uint32_t all = kFull;
            if ((ragged >> (slot << runsh)) & ((2u << ((1 << runsh) - 1)) - 1u)) {
                const uint32_t mask =
                    mine && valid > 0 ? (valid >= 32 ? 0xffffffffu : ((1u << valid) - 1u)) << (my_run * R) : 0u;
                all = __reduce_or_sync(0xffffffffu, mask);
                // tokens that do not exist: nothing of them may reach an operand as NaN or infinity
                if (mine)
                    for (int i = valid; i < R; ++i) {
                        const uint32_t row = dst + (my_run * R + i) * SROW;
                        if (INT4) sts128_zero(row + D);
                        else
                            for (int c = 0; c < 4 * D; c += 16) sts128_zero(row + c);
                    }
                asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
            }
            if (lane == 0) {
                s_vmask[warp][stage] = all;
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar),
                             "r"(uint32_t(__popc(all) * ROWB))
                             : "memory");
            }
            __syncwarp();
            if (mine && valid > 0)
                asm volatile(
                    "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                        dst + my_run * R * SROW),
                    "l"(src), "r"(uint32_t(valid * ROWB)), "r"(bar)
                    : "memory");
        };

        // tokens are looked up two batches ahead of their copies and pages one ahead
        int n1 = token_of(0), pg1 = page_of(n1), n2 = token_of(1);
        int issued = 0;
        auto advance = [&]() {                  // the next tile, if any, on its way
            if (issued >= n_my) return;
            if ((issued & ((1 << persh) - 1)) == 0) {
                take(n1, pg1);
                ragged = __ballot_sync(0xffffffffu, valid != R);
                n1 = n2;
                pg1 = page_of(n1);
                n2 = token_of((issued >> persh) + 2);
            }
            issue(issued++);
        };
#pragma unroll 1
        for (int j = 0; j < STAGES - 1; ++j) advance();
        // ---- queries as the B operand of S (column n = r8 of column tile nt), zero beyond nrow
        constexpr int NR = QS ? 1 : NT;         // column tiles held in registers
        uint32_t qb[KS][NR][2];
        float hs[NR][2];                        // logit scale (log2 units) of this lane's two columns
        uint32_t qz[NR][2];                     // 4-bit: -8 sum q of each group in three bf16 terms, as a B operand
        int lim[NR][2];                         // keys that this lane's columns may see
        qz[0][0] = qz[0][1] = 0;
        for (int tile = QS ? warp : 0; tile < NT; tile += QS ? kWarps : 1) {   // QS: a warp per column tile
            constexpr int nt = 0;
            const int row = tile * 8 + r8;
            const bool v = row < nrow;
            const uint16_t* src =
                p.q + (v ? (un.row0 + row / un.heads) * p.q_tok + (un.h0 + row % un.heads) * p.q_head : 0);
            if constexpr (INT4) {
                // lane t4's channels: D/16 consecutive ones of each of the 4 groups
                constexpr int E = D / 16;
                float f[4][E], z[4];
                float top = 0.f;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
#pragma unroll
                    for (int e = 0; e < E; e += 4) {
                        uint2 w = make_uint2(0, 0);
                        if (v) w = __ldg(reinterpret_cast<const uint2*>(src + g * (D / 4) + t4 * E + e));
                        f[g][e] = bf_lo(w.x);
                        f[g][e + 1] = bf_hi(w.x);
                        f[g][e + 2] = bf_lo(w.y);
                        f[g][e + 3] = bf_hi(w.y);
                    }
#pragma unroll
                    for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(f[g][e]));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // power of two that brings the largest channel to [2^13, 2^14)
                int ex = 13 - (int(__float_as_uint(top) >> 23) - 127);
                ex = ex > 100 ? 100 : ex < -100 ? -100 : ex;
                const float up = __uint_as_float(uint32_t(127 + ex) << 23);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float sum = 0.f;
                    auto half_of = [&](int e, float mul) {   // rounded once; below 2^-24 of the top it may round
                        const __half h = __float2half_rn(f[g][e] * up * mul);
                        return h;
                    };
                    auto pair = [&](int e0, int e1, float mul) -> uint32_t {
                        const __half2 h = __halves2half2(half_of(e0, mul), half_of(e1, mul));
                        sum += (__low2float(h) + __high2float(h)) / mul;
                        return *reinterpret_cast<const uint32_t*>(&h);
                    };
                    if constexpr (D == 128) {   // word of 8 nibbles: (0,4) (1,5)*16, then (2,6) (3,7)*16
                        qb[2 * g][nt][0] = pair(0, 4, 1.f);
                        qb[2 * g][nt][1] = pair(1, 5, 0.0625f);
                        qb[2 * g + 1][nt][0] = pair(2, 6, 1.f);
                        qb[2 * g + 1][nt][1] = pair(3, 7, 0.0625f);
                    } else {                    // two bytes: (0,2) (1,3)*16
                        qb[g][nt][0] = pair(0, 2, 1.f);
                        qb[g][nt][1] = pair(1, 3, 0.0625f);
                    }
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    z[g] = sum * -4.76837158203125e-07f;   // -8 * 2^-24: the codes' unit
                }
                // rows k = 0-3 take the first terms of the four groups, 4-7 the second, 8-11 the third
                {
                    const float z0 = t4 & 1 ? z[2] : z[0], z1 = t4 & 1 ? z[3] : z[1];
                    uint32_t h, m, l;
                    split_bf16(z0, z1, h, m);
                    const float2 fh = bf16x2_to_float2(h);
                    split_bf16(z0 - fh.x, z1 - fh.y, m, l);
                    qz[nt][0] = t4 < 2 ? h : m;
                    qz[nt][1] = t4 < 2 ? l : 0u;
                }
                const float mine = sl2 * __uint_as_float(uint32_t(127 + 24 - ex) << 23);
                hs[nt][0] = __shfl_sync(0xffffffffu, mine, 8 * t4);
                hs[nt][1] = __shfl_sync(0xffffffffu, mine, 8 * t4 + 4);
            } else {
                // lane t4's channels: 8 consecutive ones of every 32: pairs (0,1) (2,3), then (4,5) (6,7)
#pragma unroll
                for (int g = 0; g < D / 32; ++g) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (v) w = __ldg(reinterpret_cast<const uint4*>(src + g * 32 + t4 * 8));
                    qb[2 * g][nt][0] = w.x;
                    qb[2 * g][nt][1] = w.y;
                    qb[2 * g + 1][nt][0] = w.z;
                    qb[2 * g + 1][nt][1] = w.w;
                }
                hs[nt][0] = hs[nt][1] = sl2;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = tile * 8 + 2 * t4 + e;
                lim[nt][e] = col < nrow ? un.lim0 + col / un.heads : un.ntok;
            }
            if constexpr (QS) {
                const uint32_t at = qs + tile * (KS + 3) * 256;
#pragma unroll
                for (int k = 0; k < KS; ++k) sts64(at + k * 256, qb[k][0][0], qb[k][0][1]);
                sts64(at + KS * 256, qz[0][0], qz[0][1]);
                sts64(at + KS * 256 + 256, __float_as_uint(hs[0][0]), __float_as_uint(hs[0][1]));
                sts64(at + KS * 256 + 512, uint32_t(lim[0][0]), uint32_t(lim[0][1]));
            }
        }
        if constexpr (QS) __syncthreads();
        auto q_frag = [&](int k, int nt) -> uint2 {
            if constexpr (QS) return lds64(qs + (nt * (KS + 3) + k) * 256);
            else return make_uint2(qb[k][nt][0], qb[k][nt][1]);
        };
        auto q_zero = [&](int nt) -> uint2 {
            if constexpr (QS) return lds64(qs + (nt * (KS + 3) + KS) * 256);
            else return make_uint2(qz[nt][0], qz[nt][1]);
        };
        auto q_scale = [&](int nt) -> float2 {
            if constexpr (QS) {
                const uint2 v = lds64(qs + (nt * (KS + 3) + KS + 1) * 256);
                return make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
            } else {
                return make_float2(hs[nt][0], hs[nt][1]);
            }
        };
        auto q_lim = [&](int nt) -> int2 {
            if constexpr (QS) {
                const uint2 v = lds64(qs + (nt * (KS + 3) + KS + 2) * 256);
                return make_int2(int(v.x), int(v.y));
            } else {
                return make_int2(lim[nt][0], lim[nt][1]);
            }
        };

        // ---- state of this warp: per column the reference m (-inf: no key yet), the sum l, and O^T
        float top_r[NT][2], off_r[NT][2], l_r[NT][2], acc[DT][NT][4];   // m + kSlack and kBase - m
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            top_r[nt][0] = top_r[nt][1] = -INFINITY;
            off_r[nt][0] = off_r[nt][1] = 0.f;
            l_r[nt][0] = l_r[nt][1] = 0.f;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) acc[dt][nt][0] = acc[dt][nt][1] = acc[dt][nt][2] = acc[dt][nt][3] = 0.f;
        }

        int drain = 0;
        // bounded wait for the copies into a stage; for the whole warp
        auto landed = [&](int stage) -> bool {
            const uint32_t bar = smem_u32(&s_full[warp][stage]);
            const uint32_t par = (phases >> stage) & 1u;
            uint32_t ok = 0;
            for (uint32_t it = 0; !ok && it < p.spin; ++it)
                asm volatile(
                    "{\n .reg .pred q;\n mbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\n selp.u32 "
                    "%0, 1, 0, q;\n}\n"
                    : "=r"(ok)
                    : "r"(bar), "r"(par)
                    : "memory");
            return __all_sync(0xffffffffu, ok != 0);
        };
        for (int j = 0; j < n_my; ++j) {
            advance();
            const int stage = drain;
            drain = drain + 1 == STAGES ? 0 : drain + 1;
            if (!landed(stage)) {               // the copy never landed: results are undefined
                raise_status(p.status, SPA_ERR_TIMEOUT);
                failed = true;
                for (int k = j + 1; k < issued; ++k) {   // what else is in flight lands first, or has as long to
                    landed(drain);
                    drain = drain + 1 == STAGES ? 0 : drain + 1;
                }
                break;
            }
            phases ^= 1u << stage;
            const uint32_t st = smem_u32(my_ring + size_t(stage) * TILE * SROW);
            const uint32_t vmask = s_vmask[warp][stage];
            const int n0 = (a + warp + j * kWarps) * TILE;
            const bool edge = vmask != (TILE == 32 ? 0xffffffffu : (1u << TILE) - 1u) ||
                              (!sparse && n0 + TILE > un.lim0);

            // Values that are not finite among tokens that only some queries see (else a zero weight is enough)
            bool poison = false;
            if (edge && un.nq > 1) {
                auto inf2 = [](uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; };
                if constexpr (INT4) {
                    const uint2 v = lds64(st + lane * SROW + D + 8);
                    poison = inf2(v.x) || inf2(v.y);
                } else {
                    for (int i = lane; i < TILE * (D / 8); i += 32) {
                        const uint4 v = lds128(st + (i / (D / 8)) * SROW + 2 * D + (i % (D / 8)) * 16);
                        poison |= inf2(v.x) || inf2(v.y) || inf2(v.z) || inf2(v.w);
                    }
                }
                poison = __any_sync(0xffffffffu, poison);
            }
            if constexpr (INT4) {
                // One token per lane: the power of two 2^e of its largest value scale that is a number, and the scales
                // times 2^-e (in [0, 2)) as fp16 * 2^15, exactly above 2^-32, stored by token pairs over the scales
                // themselves.
                const uint32_t row = st + lane * SROW + D + 8;
                const uint2 v = lds64(row);
                const uint32_t m2 = max_bf16x2(max_bf16x2(v.x, v.y), 0u);
                const uint32_t m = max_bf16x2(m2, __byte_perm(m2, m2, 0x1032));
                const float top = fmaxf(__uint_as_float(m & 0x7f800000u), kFloorV);
                const float iv = __frcp_rn(top);
                sts64(prep + lane * 8, __float_as_uint(float(int(__float_as_uint(top) >> 23) - 127)), __float_as_uint(iv));
                const uint32_t h01 = pack_f16(bf_lo(v.x) * iv * 32768.f, bf_hi(v.x) * iv * 32768.f);
                const uint32_t h23 = pack_f16(bf_lo(v.y) * iv * 32768.f, bf_hi(v.y) * iv * 32768.f);
                // rows 2i and 2i + 1 of a 16-row tile are a pair; the partner's token
                const int rho = tau_inv<D, INT4>(lane & 7), mate = (lane & ~7) + tau<D, INT4>(rho ^ 1);
                const uint32_t o01 = __shfl_sync(0xffffffffu, h01, mate), o23 = __shfl_sync(0xffffffffu, h23, mate);
                // the first token's row takes groups 0 and 1 of both, the second's groups 2 and 3
                if (rho & 1) sts64(row, __byte_perm(o23, h23, 0x5410), __byte_perm(o23, h23, 0x7632));
                else sts64(row, __byte_perm(h01, o01, 0x5410), __byte_perm(h01, o01, 0x7632));
                __syncwarp();
            }
            // ---- 16 tokens at a time; EDGE: some of them are not to be seen by some column
            auto step = [&](int mt, auto edge_c) {
                constexpr bool EDGE = decltype(edge_c)::value;
                const int tk = mt * 16 + tau<D, INT4>(r8);
                float s[NT][4];
                float lgv[2] = {0.f, 0.f}, inv[2] = {1.f, 1.f};   // 4-bit: of this lane's two tokens
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
                if constexpr (INT4) {
                    const uint32_t ra = st + tk * SROW, rb = ra + 8 * SROW;
                    const uint2 sa = lds64(ra + D), sb = lds64(rb + D);
                    {
                        // start value sum_g s_g (-8 sum q): scales (rows) by the terms of the sums
                        const uint32_t z0 = t4 & 1 ? sa.y : sa.x, z1 = t4 & 1 ? sb.y : sb.x;
                        const uint32_t f[4] = {z0, z1, z0, z1};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint2 z = q_zero(nt);
                            mma16816(s[nt], f, z.x, z.y);
                        }
                    }
                    {
                        const uint2 wa = lds64(prep + tk * 8), wb = lds64(prep + tk * 8 + 64);
                        lgv[0] = __uint_as_float(wa.x); inv[0] = __uint_as_float(wa.y);
                        lgv[1] = __uint_as_float(wb.x); inv[1] = __uint_as_float(wb.y);
                    }
                    uint32_t ka[4], kb[4];
                    if constexpr (D == 128) {
                        const uint4 wa = lds128(ra + 16 * t4), wb = lds128(rb + 16 * t4);
                        ka[0] = wa.x; ka[1] = wa.y; ka[2] = wa.z; ka[3] = wa.w;
                        kb[0] = wb.x; kb[1] = wb.y; kb[2] = wb.z; kb[3] = wb.w;
                    } else {
                        const uint2 wa = lds64(ra + 8 * t4), wb = lds64(rb + 8 * t4);
                        ka[0] = __byte_perm(wa.x, 0, 0x4140); ka[1] = __byte_perm(wa.x, 0, 0x4342);
                        ka[2] = __byte_perm(wa.y, 0, 0x4140); ka[3] = __byte_perm(wa.y, 0, 0x4342);
                        kb[0] = __byte_perm(wb.x, 0, 0x4140); kb[1] = __byte_perm(wb.x, 0, 0x4342);
                        kb[2] = __byte_perm(wb.y, 0, 0x4140); kb[3] = __byte_perm(wb.y, 0, 0x4342);
                    }
                    const float fa[4] = {bf_lo(sa.x), bf_hi(sa.x), bf_lo(sa.y), bf_hi(sa.y)};
                    const float fb[4] = {bf_lo(sb.x), bf_hi(sb.x), bf_lo(sb.y), bf_hi(sb.y)};
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const uint32_t f0[4] = {ka[g] & 0x000f000fu, kb[g] & 0x000f000fu, ka[g] & 0x00f000f0u,
                                                kb[g] & 0x00f000f0u};
                        const uint32_t ha = ka[g] >> 8, hb = kb[g] >> 8;
                        [[maybe_unused]] const uint32_t f1[4] = {ha & 0x000f000fu, hb & 0x000f000fu, ha & 0x00f000f0u,
                                                                 hb & 0x00f000f0u};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            if constexpr (D == 128) {
                                const uint2 qa = q_frag(2 * g, nt), qc = q_frag(2 * g + 1, nt);
                                mma_f16(d, f0, qa.x, qa.y);
                                mma_f16(d, f1, qc.x, qc.y);
                            } else {
                                const uint2 qa = q_frag(g, nt);
                                mma_f16(d, f0, qa.x, qa.y);
                            }
                            s[nt][0] = fmaf(fa[g], d[0], s[nt][0]);
                            s[nt][1] = fmaf(fa[g], d[1], s[nt][1]);
                            s[nt][2] = fmaf(fb[g], d[2], s[nt][2]);
                            s[nt][3] = fmaf(fb[g], d[3], s[nt][3]);
                        }
                    }
                } else {
                    const uint32_t ra = st + tk * SROW, rb = ra + 8 * SROW;
#pragma unroll
                    for (int g = 0; g < D / 32; ++g) {
                        const uint4 wa = lds128(ra + g * 64 + t4 * 16), wb = lds128(rb + g * 64 + t4 * 16);
                        const uint32_t f0[4] = {wa.x, wb.x, wa.y, wb.y}, f1[4] = {wa.z, wb.z, wa.w, wb.w};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint2 qa = q_frag(2 * g, nt), qc = q_frag(2 * g + 1, nt);
                            mma16816(s[nt], f0, qa.x, qa.y);
                            mma16816(s[nt], f1, qc.x, qc.y);
                        }
                    }
                }
                // ---- the reference follows logit + the value scale's e
                bool up = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 h = q_scale(nt);
                    [[maybe_unused]] const int2 li = q_lim(nt);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[nt][e] = fmaf(s[nt][e], e & 1 ? h.y : h.x, lgv[e >> 1]);
                        if constexpr (EDGE) {
                            const int tok = tk + (e >> 1) * 8;
                            const bool see = ((vmask >> tok) & 1u) && (sparse || n0 + tok < (e & 1 ? li.y : li.x));
                            s[nt][e] = see ? s[nt][e] : -INFINITY;
                        }
                    }
                    up |= fmaxf(s[nt][0], s[nt][2]) > top_r[nt][0] || fmaxf(s[nt][1], s[nt][3]) > top_r[nt][1];
                }
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float old = top_r[nt][e] - kSlack;
                            float mx = fmaxf(old, fmaxf(s[nt][e], s[nt][e + 2]));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                            const float f = mx == -INFINITY ? 1.f : ex2(old - mx);
                            top_r[nt][e] = mx + kSlack;
                            off_r[nt][e] = mx == -INFINITY ? 0.f : kBase - mx;
                            l_r[nt][e] *= f;
#pragma unroll
                            for (int dt = 0; dt < DT; ++dt) {
                                acc[dt][nt][e] *= f;
                                acc[dt][nt][e + 2] *= f;
                            }
                        }
                }
                // With such values: one product per query token, with what it does not see taken as 0 (0 * NaN would
                // reach its sum).
                auto edge_product = [&](const uint32_t (&f)[4], int dt, auto product) {
                    const int ka = n0 + mt * 16 + tau<D, INT4>(2 * t4), kb = n0 + mt * 16 + tau<D, INT4>(2 * t4 + 1);
                    for (int i = 0; i < un.nq; ++i) {
                        const int sees = un.lim0 + i;
                        const uint32_t mlo = (ka < sees ? 0xffffu : 0u) | (kb < sees ? 0xffff0000u : 0u);
                        const uint32_t mhi = (ka + 8 < sees ? 0xffffu : 0u) | (kb + 8 < sees ? 0xffff0000u : 0u);
                        const uint32_t fi[4] = {f[0] & mlo, f[1] & mlo, f[2] & mhi, f[3] & mhi};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float o[4] = {0.f, 0.f, 0.f, 0.f};
                            product(nt, o, fi);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if ((nt * 8 + 2 * t4 + (e & 1)) / un.heads == i) acc[dt][nt][e] += o[e];
                        }
                    }
                };
                (void)edge_product;
                // ---- weights and O^T += V^T P^T
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[nt][e] = ex2(s[nt][e] + off_r[nt][e & 1]);
                        l_r[nt][e & 1] = INT4 ? fmaf(s[nt][e], inv[e >> 1], l_r[nt][e & 1]) : l_r[nt][e & 1] + s[nt][e];
                    }
                if constexpr (INT4) {
                    uint32_t b0[NT], b1[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        b0[nt] = movm_t(pack_f16(s[nt][0], s[nt][1]));
                        b1[nt] = movm_t(pack_f16(s[nt][2], s[nt][3]));
                    }
                    // This lane's codes belong to one group (d = 128) or two (d = 64: codes 0, 1 and 2, 3 of a
                    // unit).  Its r_g * 2^15 for the token pairs of k = 2 t4, 2 t4 + 1 and the same + 8 lie where
                    // the two tokens had their value scales: groups 0, 1 in the first token's row, 2, 3 in the
                    // second's.
                    constexpr int NG = D == 128 ? 1 : 2;
                    uint32_t rg[2][NG], nl[2][NG], nh[2][NG];   // r, and -8 r in the units of the two kinds of codes
                    {
                        const int g0 = D == 128 ? r8 & 3 : 2 * (r8 & 1);
                        const uint32_t at = st + (mt * 16 + tau<D, INT4>(2 * t4 + (g0 >> 1))) * SROW + D + 8 + (g0 & 1) * 4;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if constexpr (NG == 1) {
                                rg[h][0] = lds32(at + h * 8 * SROW);
                            } else {
                                const uint2 w = lds64(at + h * 8 * SROW);
                                rg[h][0] = w.x;
                                rg[h][1] = w.y;
                            }
#pragma unroll
                            for (int i = 0; i < NG; ++i) {
                                nl[h][i] = mul_f16x2(rg[h][i], 0x80408040u);   // -8 * 2^-21
                                nh[h][i] = mul_f16x2(rg[h][i], 0x84008400u);   // -8 * 2^-17
                            }
                        }
                    }
                    // 16-bit units of V transposed: matrices (chunk q, tokens 0-7), (chunk q, tokens 8-15), ...
                    const uint32_t vb =
                        st + (mt * 16 + tau<D, INT4>(lane & 7) + ((lane >> 3) & 1) * 8) * SROW + D / 2 + (lane >> 4) * 16;
#pragma unroll
                    for (int qq = 0; qq < D / 64; ++qq) {
                        uint32_t x[4];
                        ldsm_x4_t(vb + qq * 32, x[0], x[1], x[2], x[3]);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {       // codes 2e and 2e + 1 of the units
                                // a code in bits 3-6 is u * 2^-21 as fp16, in bits 7-10 u * 2^-17 (bit 10 is the
                                // exponent's lowest, whose step is the denormals'): products stay above 2^-6 r, exact
                                const uint32_t lo = e ? x[2 * q] >> 5 : x[2 * q] << 3;
                                const uint32_t hi = e ? x[2 * q + 1] >> 5 : x[2 * q + 1] << 3;
                                const int i = NG == 1 ? 0 : e;
                                const uint32_t f[4] = {fma_f16x2(lo & 0x00780078u, rg[0][i], nl[0][i]),
                                                       fma_f16x2(lo & 0x07800780u, rg[0][i], nh[0][i]),
                                                       fma_f16x2(hi & 0x00780078u, rg[1][i], nl[1][i]),
                                                       fma_f16x2(hi & 0x07800780u, rg[1][i], nh[1][i])};
                                const int dt = (2 * qq + q) * 2 + e;
                                if (!EDGE || !poison) {
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt) mma_f16(acc[dt][nt], f, b0[nt], b1[nt]);
                                } else {
                                    edge_product(f, dt, [&](int nt, float (&o)[4], const uint32_t (&fi)[4]) {
                                        mma_f16(o, fi, b0[nt], b1[nt]);
                                    });
                                }
                            }
                        }
                    }
                } else {
                    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        split_bf16(s[nt][0], s[nt][1], ph[nt][0], pl[nt][0]);
                        split_bf16(s[nt][2], s[nt][3], ph[nt][1], pl[nt][1]);
                        ph[nt][0] = movm_t(ph[nt][0]);
                        ph[nt][1] = movm_t(ph[nt][1]);
                        pl[nt][0] = movm_t(pl[nt][0]);
                        pl[nt][1] = movm_t(pl[nt][1]);
                    }
                    // V^T tile dt: a0 = channels 0-7 x k 0-7, a1 = channels 8-15 x k 0-7, a2, a3 = k 8-15
                    const int mat = lane >> 3;
                    const int tv = mt * 16 + tau<D, INT4>(lane & 7) + (mat >> 1) * 8;
                    const uint32_t vb = st + tv * SROW + 2 * D + (mat & 1) * 16;
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) {
                        uint32_t f[4];
                        ldsm_x4_t(vb + dt * 32, f[0], f[1], f[2], f[3]);
                        if (!EDGE || !poison) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816(acc[dt][nt], f, ph[nt][0], ph[nt][1]);
                                mma16816(acc[dt][nt], f, pl[nt][0], pl[nt][1]);
                            }
                        } else {
                            edge_product(f, dt, [&](int nt, float (&o)[4], const uint32_t (&fi)[4]) {
                                mma16816(o, fi, ph[nt][0], ph[nt][1]);
                                mma16816(o, fi, pl[nt][0], pl[nt][1]);
                            });
                        }
                    }
                }
            };
            if (edge) {
#pragma unroll 1
                for (int mt = 0; mt < MT; ++mt) step(mt, std::true_type{});
            } else {
#pragma unroll 1
                for (int mt = 0; mt < MT; ++mt) step(mt, std::false_type{});
            }
            if constexpr (INT4) asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // the pair scales
            __syncwarp();   // every lane has read the stage before it is filled again
        }

        // ---- merge the warps in shared memory (the ring is free: all copies of this segment have landed)
        __syncthreads();
        float* const mg = reinterpret_cast<float*>(smem);       // [warp][row][D + 2]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_r[nt][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                float* const rec = mg + (warp * ROWS + nt * 8 + 2 * t4 + e) * (D + 2);
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    if constexpr (INT4) {   // tile dt: chunk dt / 2, codes 2 (dt % 2) and the next of its units
                        const int q = dt >> 1, e2 = 2 * (dt & 1);
                        const int c0 = D == 128 ? 32 * (r8 & 3) + 2 * q + (r8 >> 2) + 8 * e2
                                                : 16 * (2 * (r8 & 1) + (dt & 1)) + 4 * q + (r8 >> 1);
                        rec[c0] = acc[dt][nt][e] * 64.f;        // values were held times 2^-6 and 2^-2
                        rec[c0 + 8] = acc[dt][nt][e + 2] * 4.f;
                    } else {
                        rec[dt * 16 + r8] = acc[dt][nt][e];
                        rec[dt * 16 + r8 + 8] = acc[dt][nt][e + 2];
                    }
                }
                if (r8 == 0) {
                    rec[D] = top_r[nt][e] - kSlack;
                    rec[D + 1] = l;
                }
            }
        __syncthreads();
        const bool whole = a == 0 && bnd == int(s_seg[1] - s_seg[0]) - kSeg;
        // four channels of a row
        auto store = [&](int row, int c, float L, float4 o) {
            const float il = L == 0.f ? 0.f : 1.f / L;   // L == 0: nothing seen
            const size_t at = (size_t(un.row0 + row / un.heads) * p.Hq + un.h0 + row % un.heads) * D + c;
            o = make_float4(o.x * il, o.y * il, o.z * il, o.w * il);
            const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
            *reinterpret_cast<uint2*>(p.out + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            if (p.out_f32) *reinterpret_cast<float4*>(p.out_f32 + at) = o;
        };
        auto store_lse = [&](int row, float M, float L) {
            if (p.lse)
                p.lse[size_t(un.row0 + row / un.heads) * p.Hq + un.h0 + row % un.heads] =
                    L == 0.f ? -INFINITY : (M - kBase + log2f(L)) * kLn2;
        };
        // per row: the factor of every warp's (later: every share's) part, and the row's (M, L)
        float* const fac = mg + kWarps * ROWS * (D + 2);
        float* const ml = fac + ROWS * kWarps;
        if (tid < nrow) {
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mg[(w * ROWS + tid) * (D + 2) + D]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* rec = mg + (w * ROWS + tid) * (D + 2);
                const float f = rec[D] == -INFINITY ? 0.f : ex2(rec[D] - M);
                fac[tid * kWarps + w] = f;
                L += rec[D + 1] * f;   // a warp that saw only NaN has m = -inf and keeps its NaN here
            }
            ml[2 * tid] = M;
            ml[2 * tid + 1] = L;
        }
        __syncthreads();
        // A unit's first share goes to slot 2c + 1 of its CTA, later shares to slot 2c.  A slot holds O [ROWS][D],
        // then (M, L) [ROWS].
        constexpr int REC = paged_rec_floats(D, ROWS);
        float* const part = p.partials + size_t(2 * cta + (a == 0 ? 1 : 0)) * REC;
        for (int i = tid; i < nrow * (D / 4); i += kThreads) {
            const int row = i / (D / 4), c = 4 * (i % (D / 4));
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2* rec = reinterpret_cast<const float2*>(mg + (w * ROWS + row) * (D + 2) + c);
                const float f = fac[row * kWarps + w];
                const float2 u = rec[0], v = rec[1];
                o = make_float4(fmaf(u.x, f, o.x), fmaf(u.y, f, o.y), fmaf(v.x, f, o.z), fmaf(v.y, f, o.w));
            }
            if (whole) store(row, c, ml[2 * row + 1], o);
            else *reinterpret_cast<float4*>(part + row * D + c) = o;
        }
        if (tid < nrow) {
            if (whole) store_lse(tid, ml[2 * tid], ml[2 * tid + 1]);
            else *reinterpret_cast<float2*>(part + ROWS * D + 2 * tid) = make_float2(ml[2 * tid], ml[2 * tid + 1]);
        }
        if (!whole) {
            // the last CTA of a split unit to get here merges its shares, in the order of the CTAs
            const long long tt = s_prefix[groups];
            const int lo = paged_tile_owner(s_seg[0] + kSeg, tt, GC), hi = paged_tile_owner(s_seg[1] - 1, tt, GC);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int n = atomicAdd(p.arrived + lo, 1);
                s_last = n == hi - lo;
                if (n == hi - lo) p.arrived[lo] = 0;   // ready for the next call
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                const float* const base = p.partials + size_t(2 * lo + 1) * REC;   // slot of CTA lo, then 2k
                const int n = hi - lo + 1;
                float* const fs = mg;                      // [nrow][n]
                auto slot = [&](int k) { return k == 0 ? base : base + size_t(2 * k - 1) * REC; };
                for (int row = warp; row < nrow; row += kWarps) {
                    float M = -INFINITY, L = 0.f;
                    for (int k0 = 0; k0 < n; k0 += 32) {   // running (M, L) over 32 shares at a time
                        const int k = k0 + lane;
                        float2 v = make_float2(-INFINITY, 0.f);
                        if (k < n) v = __ldcg(reinterpret_cast<const float2*>(slot(k) + ROWS * D + 2 * row));
                        float m = v.x;
#pragma unroll
                        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        m = fmaxf(m, M);
                        float l = v.y * (v.x == -INFINITY ? 0.f : ex2(v.x - m));
#pragma unroll
                        for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                        L = (M == -INFINITY ? 0.f : L * ex2(M - m)) + l;
                        M = m;
                        if (k < n) fs[row * n + k] = v.x;
                    }
                    __syncwarp();
                    for (int k = lane; k < n; k += 32) {
                        const float m = fs[row * n + k];
                        fs[row * n + k] = m == -INFINITY ? 0.f : ex2(m - M);
                    }
                    if (lane == 0) {
                        ml[2 * row + 1] = L;
                        store_lse(row, M, L);
                    }
                }
                __syncthreads();
                for (int i = tid; i < nrow * (D / 4); i += kThreads) {
                    const int row = i / (D / 4), c = 4 * (i % (D / 4));
                    const float* const f = fs + row * n;
                    const int at = row * D + c;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int k = 0; k < n; ++k) {
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(slot(k) + at));
                        o = make_float4(fmaf(v.x, f[k], o.x), fmaf(v.y, f[k], o.y), fmaf(v.z, f[k], o.z),
                                        fmaf(v.w, f[k], o.w));
                    }
                    store(row, c, ml[2 * row + 1], o);
                }
            }
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // before the ring is copied into again
        __syncthreads();
        if (bad && tid == 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
        x = s_seg[2];
        __syncthreads();
    }
}

}  // namespace

// Column tiles of 8 (query, head) rows of a unit, and query tokens of a unit: one query per unit where there
// are no more tokens than sequences, else as many as a sequence has on average, up to 32 rows.
static void paged_shape(int T, int B, int heads, bool sparse, int* nt, int* TQ) {
    int rows = heads;
    if (!sparse && T > B) {
        const long long avg = ((long long)T * heads + B - 1) / B;
        rows = avg > kRowsMax ? kRowsMax : avg > heads ? int(avg) : heads;
    }
    *nt = (rows + 7) / 8;
    *TQ = sparse || T <= B ? 1 : paged_tokens_per_tile(*nt * 8, heads);
}

// two shares for each of up to two CTAs per SM
size_t paged_attend_scratch_bytes(int d, int T, int B, int heads, bool sparse) {
    const size_t grid = size_t(device_info().num_sms) * 2;
    int nt, TQ;
    paged_shape(T, B, heads, sparse, &nt, &TQ);
    return paged_counter_bytes() + align_up(2 * grid * paged_rec_floats(d, nt * 8) * 4, 256);
}

spa_status launch_paged_attend(const PagedAttendParams& args, cudaStream_t st) {
    PagedAttendParams p = args;
    p.stall = (test_stall_bits() & SPA_TEST_STALL_PAGED_COPY) != 0;
    p.spin = p.stall ? kStallLimit : kWaitLimit;
    const int G = p.Hq / p.kv.Hkv;
    const int sms = device_info().num_sms;
    const bool sparse = p.idx != nullptr;
    const int heads = sparse && p.collapse == SPA_COLLAPSE_NONE ? 1 : G;
    const long long all = !sparse ? p.kv.B : (long long)p.kv.B * (p.collapse == SPA_COLLAPSE_GROUP_MEAN ? p.kv.Hkv : p.Hq);
    int nt, TQ;
    paged_shape(p.T, p.kv.B, heads, sparse, &nt, &TQ);
    // the prefix of a launch's groups lies in shared memory, so a launch takes at most kPagedMaxUnits of them
    // (and the weighted tiles of a launch are counted in 32 bits: a sequence's queries times its length bound them)
    const long long tiles = (((long long)p.kv.max_pages << p.kv.page_shift) + 15) / 16 + kSeg;
    const long long most = sparse ? ((long long)p.cap * p.unit_tokens + 15) / 16 + kSeg
                                  : tiles * p.kv.Hkv * ((p.T + TQ - 1) / TQ);
    long long step = kPagedMaxUnits;
    if (!sparse && most + tiles * p.kv.Hkv * step > 0xffffffffll) step = (0xffffffffll - most) / (tiles * p.kv.Hkv);
    if (sparse && most * step > 0xffffffffll) step = 0xffffffffll / most;
    if (step < 1) return SPA_ERR_UNSUPPORTED_SHAPE;
    for (long long g0 = 0; g0 < all; g0 += step) {
        const int groups = int(all - g0 < step ? all - g0 : step);
#define SPA_PA(DD, I4, NTT)                                                                                      \
    if (p.kv.d == DD && (p.kv.int4 != 0) == I4 && nt == NTT) {                                                   \
        using G_ = Geo<DD, I4, NTT>;                                                                             \
        constexpr size_t kMost = G_::SMEM + size_t(kPagedMaxUnits + 1) * 4;                                      \
        static_assert(kMost + 1024 <= 227 * 1024, "paged attention: shared memory over the per-CTA limit");       \
        SPA_CUDA_TRY(set_func_attr(reinterpret_cast<const void*>(paged_attend_kernel<DD, I4, NTT>),              \
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMost)));                   \
        SPA_CUDA_TRY(launch_pdl(paged_attend_kernel<DD, I4, NTT>, dim3(sms * G_::CTAS), dim3(G_::WARPS * 32),    \
                                G_::SMEM + size_t(groups + 1) * 4, st, p, int(g0), groups, TQ));                 \
    }
#define SPA_PN(DD, I4) SPA_PA(DD, I4, 1) SPA_PA(DD, I4, 2) SPA_PA(DD, I4, 3) SPA_PA(DD, I4, 4)
        SPA_PN(64, false) SPA_PN(64, true) SPA_PN(128, false) SPA_PN(128, true)
#undef SPA_PN
#undef SPA_PA
    }
    return SPA_OK;
}

}  // namespace spa
