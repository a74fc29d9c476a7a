// Exact softmax attention over a paged KV cache, bf16 or 4-bit: decode (one query per sequence), a few
// drafted or chunked queries per sequence (causal among themselves), or decode restricted to supports.
//
// Work split: a unit is one tile of up to 16 (query, head) rows that share the keys of one (sequence,
// kv head), or one support.  Its keys are cut into tiles of TILE tokens; the tiles of all units form one
// list (each unit charged kSeg tiles for its start-up and merge), split evenly over the CTAs (one per
// SM).  Inside a CTA the warps take a unit's tiles round-robin; each warp copies its tiles into its own
// ring with bulk asynchronous copies, one per run of tokens that lie together on a page.
//
// Math per 16 tokens on tensor cores (mma.sync m16n8k16, fp32 accumulation), transposed so that tokens
// fill the 16-row side and heads the 8-column side:
//   4-bit keys: S = sum_g s_g (sum_{c in g} q_c u_c - 8 sum_{c in g} q_c), u the code 0..15.
//     A nibble masked out of its word is an fp16 denormal, u * 2^-24 in bits 0-3 and u * 2^-20 in bits
//     4-7: one AND per two codes makes the A operand, exactly.  q is scaled by a power of two into
//     fp16's range (and by 1/16 for the second kind), exactly above 2^-24 of its largest channel; the
//     -8 is the accumulator's start value, and the group scale multiplies in fp32.
//   4-bit values: O += V^T W^T with W = p * s_g in fp16 (11 bits), V = u - 8 centred exactly in fp16.
//     So that W fits fp16 whatever the scales are, the running reference of the softmax is the maximum
//     of (logit + log2 of the token's largest value scale), not of the logit; p and l are relative to it
//     in fp32, and W <= 2^15.
//   bf16 rows: S = K Q^T, O += V^T P^T with P = hi + lo bf16 (about 16 bits).
// The m16 rows of a tile are a permutation of its tokens (tau) that keeps the shared-memory reads free
// of bank conflicts for the rows' strides; a softmax does not see the order.
//
// At the end of its share of a unit a CTA merges its warps in shared memory and writes the output, or a
// partial (o, m, l) if the unit is split; a second kernel merges partials in a fixed order.
#include "paged.cuh"
#include "warp_mma.cuh"

#include <cuda_fp16.h>

namespace spa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRowsMax = 16;              // (query, head) rows of a unit
constexpr int kSeg = 8;                   // tiles charged to a unit for its start-up and merge
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFloorV = 8.077935669463161e-28f;   // 2^-90: least value scale that the reference follows
constexpr float kBase = 9.f;              // weights are 2^9 at the reference, and at most 2^(9 + kSlack)
constexpr float kSlack = 6.f;             // the reference moves only when it is exceeded by this (log2)
constexpr uint32_t kWaitLimit = 1u << 22;

template <int D, bool INT4>
struct Geo {
    static constexpr int ROWB = INT4 ? D + 16 : 4 * D;
    static constexpr int TILE = INT4 ? 32 : 16;           // tokens per warp step
    static constexpr int MT = TILE / 16;
    static constexpr int STAGES = INT4 ? 4 : 3;
    // shared-memory row stride: bf16 rows are copied one by one and padded (a multiple of 128 bytes would put
    // the eight rows of a fragment on the same banks)
    static constexpr int SROW = INT4 ? ROWB : ROWB + 16;
    static constexpr int RING = kWarps * STAGES * TILE * SROW;
    static constexpr int MERGE = kWarps * kRowsMax * (D + 2) * 4;
    static constexpr int SMEM = RING > MERGE ? RING : MERGE;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                        const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
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
__device__ __forceinline__ void sts128_zero(uint32_t a) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};\n" ::"r"(a), "r"(0) : "memory");
}

// Row r (0..7) of a 16-row tile is token tau(r), row r + 8 token tau(r) + 1 (4-bit) or tau(r) + 8 (bf16).
// 4-bit: {0,4,2,6,12,8,14,10}; bf16: {0,4,1,5,2,6,3,7}.
template <bool INT4>
__device__ __forceinline__ int tau(int r) {
    return INT4 ? int((0xAE8C6240u >> (4 * r)) & 15u) : int((0x73625140u >> (4 * r)) & 15u);
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
        if (a < 0 || e > p.T || e < a) { *bad = true; s.n = 0; s.row0 = 0; }
        else { s.n = int(e - a); s.row0 = int(a); }
    }
    return s;
}

__device__ __forceinline__ int support_tokens(const PagedAttendParams& p, int u) {
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
__global__ void __launch_bounds__(kThreads, 1) paged_attend_kernel(PagedAttendParams p, int g0, int groups, int TQ) {
    using G_ = Geo<D, INT4>;
    constexpr int TILE = G_::TILE, ROWB = G_::ROWB, SROW = G_::SROW, STAGES = G_::STAGES, MT = G_::MT;
    constexpr int KS = D / 16;                 // k-steps of S, and 16-channel tiles of O
    constexpr int DT = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* const ring = smem;
    long long* const s_prefix = reinterpret_cast<long long*>(smem + G_::SMEM);   // [groups + 1]
    __shared__ uint64_t s_full[kWarps][STAGES];
    __shared__ uint32_t s_vmask[kWarps][STAGES];
    __shared__ long long s_wsum[kWarps];

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
    for (int base = 0; base < groups; base += kThreads) {
        const int u = base + tid;
        long long t = 0;
        if (u < groups) {
            if (sparse) {
                const int n = support_tokens(p, g0 + u);
                t = n > 0 ? (n + TILE - 1) / TILE + kSeg : 0;
            } else {
                bool bad = false;
                const SeqGeo s = seq_geo(p, g0 + u, &bad);
                t = head_weight<TILE>(s, TQ) * p.kv.Hkv;
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
        if (u < groups) s_prefix[u] = before + incl - t;
        running += tot;
        __syncthreads();
    }
    if (tid == 0) s_prefix[groups] = running;
    __syncthreads();
    const long long TT = running;
    const int cta = blockIdx.x;
    const int GC = int(TT < (long long)gridDim.x ? TT : (long long)gridDim.x);   // CTAs with work

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
    for (int u = cta; u < groups; u += gridDim.x) {
        if (sparse) {
            if (s_prefix[u + 1] != s_prefix[u]) continue;
            const bool grp = p.collapse == SPA_COLLAPSE_GROUP_MEAN;
            const int per = grp ? p.kv.Hkv : p.Hq;
            write_empty((g0 + u) / per, 1, ((g0 + u) % per) * (grp ? G : 1), grp ? G : 1);
        } else {
            bool bad = false;
            const SeqGeo s = seq_geo(p, g0 + u, &bad);
            // query tiles whose last query sees no key
            const int nj = (s.n + TQ - 1) / TQ;
            for (int j = 0; j < nj && paged_tile_limit(s.len, s.n, TQ, j) == 0; ++j)
                write_empty(s.row0 + j * TQ, min(TQ, s.n - j * TQ), 0, p.Hq);
        }
    }
    if (tid == 0) p.split[cta] = make_int4(-1, -1, -1, -1);
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
    const int page = 1 << p.kv.page_shift;
    uint32_t phases = 0;      // parity of each stage's barrier
    bool failed = false;      // a wait gave up: the rest of this CTA's waits are short
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
            un.row0 = un.b;
            un.nq = 1;
            un.len = paged_len(p.kv, p.kv.kv_len[un.b], &bad);
            un.lim0 = un.len;
            un.u = g0 + grp;
            un.ntok = support_tokens(p, g0 + grp);
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
        const long long x_next = seg_end;
        if (a >= bnd) {       // only the unit's fixed cost lies in this CTA's range
            x = x_next;
            continue;
        }
        const int nrow = un.nq * un.heads;

        // ---- queries as the B operand of S (column n = r8 of column tile nt), zero beyond nrow
        uint32_t qb[KS][NT][2];
        float hs[NT][2];                        // logit scale (log2 units) of this lane's two columns
        float q0[INT4 ? 4 : 1][NT][2];          // 4-bit: start values -8 sum q of each group
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = nt * 8 + r8;
            const bool v = row < nrow;
            const uint16_t* src =
                p.q + (v ? (un.row0 + row / un.heads) * p.q_tok + (un.h0 + row % un.heads) * p.q_head : 0);
            if constexpr (INT4) {
                // lane t4's channels: D/16 consecutive ones of each of the 4 groups
                constexpr int E = D / 16;
                float f[4][E];
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
                    const float s8 = sum * -4.76837158203125e-07f;   // -8 * 2^-24: the codes' unit
                    q0[g][nt][0] = __shfl_sync(0xffffffffu, s8, 8 * t4);
                    q0[g][nt][1] = __shfl_sync(0xffffffffu, s8, 8 * t4 + 4);
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
        }
        int lim[NT][2];                         // keys that this lane's columns may see
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = nt * 8 + 2 * t4 + e;
                lim[nt][e] = row < nrow ? un.lim0 + row / un.heads : un.ntok;
            }

        // ---- copying: lane i fetches the i-th run of R tokens of a tile
        const int ut = p.unit_tokens;
        int R = !INT4 ? 1 : TILE < page ? TILE : page;
        if (sparse) while (ut % R) R >>= 1;
        const int runs = TILE / R;
        const int n_my = a + warp < bnd ? (bnd - a - warp + kWarps - 1) / kWarps : 0;
        // first token of this lane's run of the j-th of my tiles, or -1
        auto token_of = [&](int j) -> long long {
            if (j >= n_my || lane >= runs) return -1;
            const long long i = (long long)(a + warp + j * kWarps) * TILE + lane * R;
            if (i >= un.ntok) return -1;
            if (!sparse) return i;
            const long long e = i / ut;
            const long long n = (long long)__ldg(p.idx + size_t(un.u) * p.cap + e) * ut + (i - e * ut);
            return n >= 0 && n < un.len ? n : -1;
        };
        auto page_of = [&](long long n) -> int {
            const long long s = paged_slot(p.kv, un.b, n);
            return s < 0 ? -1 : __ldg(p.kv.page_table + s);
        };
        auto issue = [&](int j, long long n, int pid) {
            const int stage = j % STAGES;
            const uint32_t bar = smem_u32(&s_full[warp][stage]);
            const uint32_t dst = smem_u32(my_ring + size_t(stage) * TILE * SROW);
            int valid = 0;                      // tokens of the run that exist
            long long off = -1;
            if (n >= 0) {
                off = paged_row(p.kv, pid, un.g, n);
                if (off < 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
                else {
                    const long long left = un.len - n;
                    valid = left < R ? int(left) : R;
                    if (!sparse) {
                        const long long vis = un.ntok - n;
                        valid = vis < valid ? int(vis) : valid;
                    }
                }
            }
            const uint32_t mask =
                valid > 0 ? (valid >= 32 ? 0xffffffffu : ((1u << valid) - 1u)) << (lane * R) : 0u;
            const uint32_t all = __reduce_or_sync(0xffffffffu, mask);
            const uint32_t full = TILE == 32 ? 0xffffffffu : (1u << TILE) - 1u;
            if (all != full) {
                // tokens that do not exist: nothing of them may reach an operand as NaN or infinity
                if (lane < runs)
                    for (int i = valid; i < R; ++i) {
                        const uint32_t row = dst + (lane * R + i) * SROW;
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
            if (valid > 0)
                asm volatile(
                    "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                        dst + lane * R * SROW),
                    "l"(p.kv.data + off), "r"(uint32_t(valid * ROWB)), "r"(bar)
                    : "memory");
        };

        // ---- state of this warp: per column the reference m, the sum l, and O^T
        float m_r[NT][2], l_r[NT][2], acc[DT][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m_r[nt][0] = m_r[nt][1] = -INFINITY;
            l_r[nt][0] = l_r[nt][1] = 0.f;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) acc[dt][nt][0] = acc[dt][nt][1] = acc[dt][nt][2] = acc[dt][nt][3] = 0.f;
        }

        // tokens are looked up two tiles ahead of their copy and pages one ahead
        long long n1;
        int pg1;
#pragma unroll
        for (int j = 0; j < STAGES - 1; ++j)
            if (j < n_my) {
                const long long n = token_of(j);
                issue(j, n, page_of(n));
            }
        n1 = token_of(STAGES - 1);
        pg1 = page_of(n1);
        long long n2 = token_of(STAGES);
        for (int j = 0; j < n_my; ++j) {
            if (j + STAGES - 1 < n_my) {
                issue(j + STAGES - 1, n1, pg1);
                n1 = n2;
                pg1 = page_of(n1);
                n2 = token_of(j + STAGES + 1);
            }
            const int stage = j % STAGES;
            {
                const uint32_t bar = smem_u32(&s_full[warp][stage]);
                const uint32_t par = (phases >> stage) & 1u;
                auto poll = [&](uint32_t limit) -> bool {
                    uint32_t ok = 0;
                    for (uint32_t it = 0; !ok && it < limit; ++it)
                        asm volatile(
                            "{\n .reg .pred q;\n mbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\n selp.u32 "
                            "%0, 1, 0, q;\n}\n"
                            : "=r"(ok)
                            : "r"(bar), "r"(par)
                            : "memory");
                    return ok != 0;
                };
                if (!poll(failed ? 1024u : kWaitLimit)) {   // the copy never landed: results are undefined
                    raise_status(p.status, SPA_ERR_TIMEOUT);
                    if (!failed) poll(kWaitLimit);          // a last chance for what is in flight
                    failed = true;
                }
                phases ^= 1u << stage;
                __syncwarp();
            }
            const uint32_t st = smem_u32(my_ring + size_t(stage) * TILE * SROW);
            const uint32_t vmask = s_vmask[warp][stage];
            const int n0 = (a + warp + j * kWarps) * TILE;
            const bool edge = vmask != (TILE == 32 ? 0xffffffffu : (1u << TILE) - 1u) ||
                              (!sparse && n0 + TILE > un.lim0);

            // ---- logits (in units of this kernel's q) and value scales
            float s[MT][NT][4];
            uint32_t vs[MT][2][2];              // 4-bit: the value scales of this lane's two tokens
            float lgv[MT][2];                   // log2 of the largest of them
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int tk = mt * 16 + tau<INT4>(r8);
                if constexpr (INT4) {
                    const uint32_t ra = st + tk * SROW, rb = ra + SROW;
                    const uint4 sa = lds128(ra + D), sb = lds128(rb + D);
                    vs[mt][0][0] = sa.z; vs[mt][0][1] = sa.w;
                    vs[mt][1][0] = sb.z; vs[mt][1][1] = sb.w;
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
                    for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const uint32_t f0[4] = {ka[g] & 0x000f000fu, kb[g] & 0x000f000fu, ka[g] & 0x00f000f0u,
                                                kb[g] & 0x00f000f0u};
                        const uint32_t ha = ka[g] >> 8, hb = kb[g] >> 8;
                        const uint32_t f1[4] = {ha & 0x000f000fu, hb & 0x000f000fu, ha & 0x00f000f0u,
                                                hb & 0x00f000f0u};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float c[4] = {q0[g][nt][0], q0[g][nt][1], q0[g][nt][0], q0[g][nt][1]};
                            float d[4];
                            if constexpr (D == 128) {
                                mma_f16(d, f0, qb[2 * g][nt][0], qb[2 * g][nt][1], c);
                                mma_f16(d, f1, qb[2 * g + 1][nt][0], qb[2 * g + 1][nt][1], d);
                            } else {
                                mma_f16(d, f0, qb[g][nt][0], qb[g][nt][1], c);
                            }
                            s[mt][nt][0] = fmaf(fa[g], d[0], s[mt][nt][0]);
                            s[mt][nt][1] = fmaf(fa[g], d[1], s[mt][nt][1]);
                            s[mt][nt][2] = fmaf(fb[g], d[2], s[mt][nt][2]);
                            s[mt][nt][3] = fmaf(fb[g], d[3], s[mt][nt][3]);
                        }
                    }
                    // largest value scale of each token; scales are not negative, so their bits order them
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t m2 = __vmaxu2(vs[mt][e][0] & 0x7fff7fffu, vs[mt][e][1] & 0x7fff7fffu);
                        const uint32_t m1 = max(m2 << 16, m2 & 0xffff0000u);
                        lgv[mt][e] = lg2(fmaxf(__uint_as_float(m1), kFloorV));
                    }
                } else {
                    const uint32_t ra = st + tk * SROW, rb = ra + 8 * SROW;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
#pragma unroll
                    for (int g = 0; g < D / 32; ++g) {
                        const uint4 wa = lds128(ra + g * 64 + t4 * 16), wb = lds128(rb + g * 64 + t4 * 16);
                        const uint32_t f0[4] = {wa.x, wb.x, wa.y, wb.y}, f1[4] = {wa.z, wb.z, wa.w, wb.w};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816(s[mt][nt], f0, qb[2 * g][nt][0], qb[2 * g][nt][1]);
                            mma16816(s[mt][nt], f1, qb[2 * g + 1][nt][0], qb[2 * g + 1][nt][1]);
                        }
                    }
                    lgv[mt][0] = lgv[mt][1] = 0.f;
                }
            }
            // ---- logits in log2 units, masked; the reference follows logit + log2 of the value scale
            bool up = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int tk = mt * 16 + tau<INT4>(r8);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = s[mt][nt][e] * hs[nt][e & 1];
                        if (edge) {
                            const int tok = tk + (e >> 1) * (INT4 ? 1 : 8);
                            const bool see = ((vmask >> tok) & 1u) && (sparse || n0 + tok < lim[nt][e & 1]);
                            v = see ? v : -INFINITY;
                        }
                        s[mt][nt][e] = v;
                        up |= v + lgv[mt][e >> 1] > m_r[nt][e & 1] + kSlack;
                    }
            }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = m_r[nt][e];
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            mx = fmaxf(mx, fmaxf(s[mt][nt][e] + lgv[mt][0], s[mt][nt][e + 2] + lgv[mt][1]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float f = mx == -INFINITY ? 1.f : ex2(m_r[nt][e] - mx);
                        m_r[nt][e] = mx;
                        l_r[nt][e] *= f;
#pragma unroll
                        for (int dt = 0; dt < DT; ++dt) {
                            acc[dt][nt][e] *= f;
                            acc[dt][nt][e + 2] *= f;
                        }
                    }
            }
            // ---- weights and O^T += V^T W^T
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float m = m_r[nt][e & 1];   // still -inf: every logit is -inf, or NaN (kept)
                        const float pr = ex2(s[mt][nt][e] - (m == -INFINITY ? 0.f : m) + kBase);
                        s[mt][nt][e] = pr;
                        l_r[nt][e & 1] += pr;
                    }
                if constexpr (INT4) {
                    // value codes of this lane's fragment row for the tokens of k = 2 t4, 2 t4 + 1 (+ 8)
                    const int ta = mt * 16 + tau<INT4>(2 * t4), tb = mt * 16 + tau<INT4>(2 * t4 + 1);
                    const uint32_t vb = st + D / 2 + r8 * (D / 16);
                    uint32_t va[2], vbw[2], vc[2], vd[2];
                    if constexpr (D == 128) {
                        uint2 w;
                        w = lds64(vb + ta * SROW); va[0] = w.x; va[1] = w.y;
                        w = lds64(vb + tb * SROW); vbw[0] = w.x; vbw[1] = w.y;
                        w = lds64(vb + (ta + 1) * SROW); vc[0] = w.x; vc[1] = w.y;
                        w = lds64(vb + (tb + 1) * SROW); vd[0] = w.x; vd[1] = w.y;
                    } else {
                        va[0] = lds32(vb + ta * SROW); vbw[0] = lds32(vb + tb * SROW);
                        vc[0] = lds32(vb + (ta + 1) * SROW); vd[0] = lds32(vb + (tb + 1) * SROW);
                    }
                    constexpr int BPG = D / 64;   // bytes, and 16-channel tiles, per group
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint32_t b0[NT], b1[NT];
                        const uint32_t sa = vs[mt][0][g >> 1], sb = vs[mt][1][g >> 1];
                        const float fa = g & 1 ? bf_hi(sa) : bf_lo(sa), fb = g & 1 ? bf_hi(sb) : bf_lo(sb);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float w[4] = {s[mt][nt][0] * fa, s[mt][nt][1] * fa, s[mt][nt][2] * fb, s[mt][nt][3] * fb};
                            if (edge) {   // a masked token's scale may be NaN: its weight is 0, not 0 * NaN
#pragma unroll
                                for (int e = 0; e < 4; ++e) w[e] = s[mt][nt][e] == 0.f ? 0.f : w[e];
                            }
                            b0[nt] = movm_t(pack_f16(w[0], w[1]));
                            b1[nt] = movm_t(pack_f16(w[2], w[3]));
                        }
#pragma unroll
                        for (int i = 0; i < BPG; ++i) {
                            const int by = g * BPG + i;          // byte of the row's share
                            const uint32_t sel = uint32_t(by & 3) | (uint32_t(4 + (by & 3)) << 8);
                            const uint32_t lo = __byte_perm(va[by >> 2], vbw[by >> 2], sel);
                            const uint32_t hi = __byte_perm(vc[by >> 2], vd[by >> 2], sel);
                            // u * 2^-24 (or 2^-20) minus 8 of the same unit: exact
                            const uint32_t f[4] = {sub_f16x2(lo & 0x000f000fu, 0x00080008u),
                                                   sub_f16x2(lo & 0x00f000f0u, 0x00800080u),
                                                   sub_f16x2(hi & 0x000f000fu, 0x00080008u),
                                                   sub_f16x2(hi & 0x00f000f0u, 0x00800080u)};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma_f16(acc[by][nt], f, b0[nt], b1[nt], acc[by][nt]);
                        }
                    }
                } else {
                    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        split_bf16(s[mt][nt][0], s[mt][nt][1], ph[nt][0], pl[nt][0]);
                        split_bf16(s[mt][nt][2], s[mt][nt][3], ph[nt][1], pl[nt][1]);
                        ph[nt][0] = movm_t(ph[nt][0]);
                        ph[nt][1] = movm_t(ph[nt][1]);
                        pl[nt][0] = movm_t(pl[nt][0]);
                        pl[nt][1] = movm_t(pl[nt][1]);
                    }
                    // V^T tile dt: a0 = channels 0-7 x k 0-7, a1 = channels 8-15 x k 0-7, a2, a3 = k 8-15
                    const int mat = lane >> 3;
                    const int tk = mt * 16 + tau<INT4>(lane & 7) + (mat >> 1) * 8;
                    const uint32_t vb = st + tk * SROW + 2 * D + (mat & 1) * 16;
                    if (!edge || un.nq == 1) {
#pragma unroll
                        for (int dt = 0; dt < DT; ++dt) {
                            uint32_t f[4];
                            ldsm_x4_t(vb + dt * 32, f[0], f[1], f[2], f[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816(acc[dt][nt], f, ph[nt][0], ph[nt][1]);
                                mma16816(acc[dt][nt], f, pl[nt][0], pl[nt][1]);
                            }
                        }
                    } else {
                        // Tokens that some of the queries do not see: one product per query token, with the
                        // values it does not see taken as 0 (0 * NaN would reach its sum).
                        const int ka = n0 + mt * 16 + tau<INT4>(2 * t4), kb = n0 + mt * 16 + tau<INT4>(2 * t4 + 1);
                        for (int i = 0; i < un.nq; ++i) {
                            const int sees = un.lim0 + i;
                            const uint32_t mlo = (ka < sees ? 0xffffu : 0u) | (kb < sees ? 0xffff0000u : 0u);
                            const uint32_t mhi = (ka + 8 < sees ? 0xffffu : 0u) | (kb + 8 < sees ? 0xffff0000u : 0u);
#pragma unroll
                            for (int dt = 0; dt < DT; ++dt) {
                                uint32_t f[4];
                                ldsm_x4_t(vb + dt * 32, f[0], f[1], f[2], f[3]);
                                f[0] &= mlo; f[1] &= mlo; f[2] &= mhi; f[3] &= mhi;
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float o[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma16816(o, f, ph[nt][0], ph[nt][1]);
                                    mma16816(o, f, pl[nt][0], pl[nt][1]);
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if ((nt * 8 + 2 * t4 + (e & 1)) / un.heads == i) acc[dt][nt][e] += o[e];
                                }
                            }
                        }
                    }
                }
            }
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
                float* const rec = mg + (warp * kRowsMax + nt * 8 + 2 * t4 + e) * (D + 2);
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    // codes are in units of 2^-24, and of 2^-20 in the upper eight channels
                    rec[dt * 16 + r8] = acc[dt][nt][e] * (INT4 ? 16777216.f : 1.f);
                    rec[dt * 16 + r8 + 8] = acc[dt][nt][e + 2] * (INT4 ? 1048576.f : 1.f);
                }
                if (r8 == 0) {
                    rec[D] = m_r[nt][e];
                    rec[D + 1] = l;
                }
            }
        __syncthreads();
        const bool whole = a == 0 && bnd == tiles;
        // a unit's first share goes to slot 2c + 1 of its CTA, later shares to slot 2c
        float* const part = p.partials + size_t(2 * cta + (a == 0 ? 1 : 0)) * kRowsMax * (D + 2);
        for (int i = tid; i < nrow * D; i += kThreads) {
            const int row = i / D, c = i % D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mg[(w * kRowsMax + row) * (D + 2) + D]);
            float L = 0.f, O = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* rec = mg + (w * kRowsMax + row) * (D + 2);
                const float f = rec[D] == -INFINITY ? 0.f : ex2(rec[D] - M);
                L += rec[D + 1] * f;
                O += rec[c] * f;
            }
            if (whole) {
                const float val = L == 0.f ? 0.f : O / L;
                const size_t orow = size_t(un.row0 + row / un.heads) * p.Hq + un.h0 + row % un.heads;
                const __nv_bfloat16 bv = __float2bfloat16_rn(val);
                p.out[orow * D + c] = *reinterpret_cast<const uint16_t*>(&bv);
                if (p.out_f32) p.out_f32[orow * D + c] = val;
                if (p.lse && c == 0) p.lse[orow] = L == 0.f ? -INFINITY : (M - kBase + log2f(L)) * kLn2;
            } else {
                part[row * (D + 2) + c] = O;
                if (c == 0) {
                    part[row * (D + 2) + D] = M;
                    part[row * (D + 2) + D + 1] = L;
                }
            }
        }
        if (!whole && a == 0 && tid == 0)
            p.split[cta] = make_int4(un.row0, un.h0, un.heads | (nrow << 8),
                                     paged_tile_owner(u_hi - 1, TT, GC));
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // before the ring is copied into again
        __syncthreads();
        if (bad && tid == 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
        x = x_next;
    }
}

// Merge of a split unit's partials, in the order of their CTAs: block (c, row) takes row `row` of the unit
// that starts in CTA c and goes on past it.
template <int D>
__global__ void __launch_bounds__(D) paged_combine_kernel(PagedAttendParams p) {
    pdl_enter();
    const int c0 = blockIdx.x, row = blockIdx.y, c = threadIdx.x;
    const int4 s = p.split[c0];
    const int heads = s.z & 255, nrow = s.z >> 8, hi = s.w;
    if (s.x < 0 || row >= nrow) return;
    const size_t rec = D + 2;
    const float* const first = p.partials + (size_t(2 * c0 + 1) * kRowsMax + row) * rec;
    auto slot = [&](int k) { return k == c0 ? first : p.partials + (size_t(2 * k) * kRowsMax + row) * rec; };
    float M = -INFINITY;
    for (int k = c0; k <= hi; ++k) M = fmaxf(M, __ldcg(slot(k) + D));
    float L = 0.f, O = 0.f;
#pragma unroll 4
    for (int k = c0; k <= hi; ++k) {
        const float* r = slot(k);
        const float m = __ldcg(r + D);
        const float f = m == -INFINITY ? 0.f : ex2(m - M);
        L += __ldcg(r + D + 1) * f;
        O += __ldcg(r + c) * f;
    }
    const float val = L == 0.f ? 0.f : O / L;
    const size_t orow = size_t(s.x + row / heads) * p.Hq + s.y + row % heads;
    const __nv_bfloat16 bv = __float2bfloat16_rn(val);
    p.out[orow * D + c] = *reinterpret_cast<const uint16_t*>(&bv);
    if (p.out_f32) p.out_f32[orow * D + c] = val;
    if (p.lse && c == 0) p.lse[orow] = L == 0.f ? -INFINITY : (M - kBase + log2f(L)) * kLn2;
}

}  // namespace

size_t paged_attend_scratch_bytes(int d) {
    const size_t grid = device_info().num_sms;
    return align_up(grid * sizeof(int4), 256) + align_up(2 * grid * kRowsMax * (d + 2) * 4, 256);
}

spa_status launch_paged_attend(const PagedAttendParams& p, cudaStream_t st) {
    const int G = p.Hq / p.kv.Hkv;
    const int grid = device_info().num_sms;
    const bool sparse = p.idx != nullptr;
    const int heads = sparse && p.collapse == SPA_COLLAPSE_NONE ? 1 : G;
    if (heads > kRowsMax) return SPA_ERR_UNSUPPORTED_SHAPE;
    const long long all = !sparse ? p.kv.B : (long long)p.T * (p.collapse == SPA_COLLAPSE_GROUP_MEAN ? p.kv.Hkv : p.Hq);
    // one query tile per token when there are no more tokens than sequences, else as many as fill 16 rows
    const int TQ = sparse || p.T <= p.kv.B ? 1 : paged_tokens_per_tile(kRowsMax, G);
    const int nt = TQ * heads > 8 ? 2 : 1;
    // the prefix of a launch's groups lies in shared memory, so a launch takes at most kPagedMaxUnits of them
    for (long long g0 = 0; g0 < all; g0 += kPagedMaxUnits) {
        const int groups = int(all - g0 < kPagedMaxUnits ? all - g0 : kPagedMaxUnits);
#define SPA_PA(DD, I4, NTT)                                                                                      \
    if (p.kv.d == DD && (p.kv.int4 != 0) == I4 && nt == NTT) {                                                   \
        constexpr size_t kMost = Geo<DD, I4>::SMEM + size_t(kPagedMaxUnits + 1) * 8;                             \
        SPA_CUDA_TRY(set_func_attr(reinterpret_cast<const void*>(paged_attend_kernel<DD, I4, NTT>),              \
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMost)));                   \
        SPA_CUDA_TRY(launch_pdl(paged_attend_kernel<DD, I4, NTT>, dim3(grid), dim3(kThreads),                    \
                                Geo<DD, I4>::SMEM + size_t(groups + 1) * 8, st, p, int(g0), groups, TQ));        \
    }
        SPA_PA(64, false, 1) SPA_PA(64, false, 2) SPA_PA(64, true, 1) SPA_PA(64, true, 2)
        SPA_PA(128, false, 1) SPA_PA(128, false, 2) SPA_PA(128, true, 1) SPA_PA(128, true, 2)
#undef SPA_PA
        const dim3 rows(grid, nt * 8);
        if (p.kv.d == 64) SPA_CUDA_TRY(launch_pdl(paged_combine_kernel<64>, rows, dim3(64), 0, st, p));
        else SPA_CUDA_TRY(launch_pdl(paged_combine_kernel<128>, rows, dim3(128), 0, st, p));
    }
    return SPA_OK;
}

}  // namespace spa
