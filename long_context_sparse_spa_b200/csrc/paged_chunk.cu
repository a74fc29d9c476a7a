// Exact softmax attention of many new tokens per sequence over a paged KV cache, 4-bit or bf16 (a prefill chunk
// against its cached prefix, drafted tokens of a large batch) on tcgen05 tensor cores.
//
// A unit is up to 256 (query token, head) rows that share one (sequence, kv head): two tiles of 128 rows.
// Per 128 cached tokens and row tile, 4-bit rows:
//   S = Q K^T        fp16 x fp16, fp32 in TMEM; K = scale * (code - 8) has at most 8 + 3 significant bits,
//                    so it is exact in fp16 once a power of two per 64 tokens (per token where some queries
//                    do not see all of them, or where their scales lie more than 2^11 apart) brings the scales
//                    into range; a group whose scale is below 2^-11 of its own token's largest is off by up to
//                    2^-19 of that largest;
//                    Q is scaled by a power of two per row (exact above 2^-24 of the row's largest channel)
//   P = 2^(logit + log2(V's power of two) - reference) in fp16, at most 2^15, from registers to TMEM over S
//   O += P V         P as the TMEM operand, V exact in fp16 like K; fp32 in TMEM
// with the online softmax's reference per row following (logit + V's power of two); it moves, and O is
// rescaled through TMEM, only when it is exceeded by 2^6.  l is summed in fp32.
// bf16 rows: S = Q K^T and O += P V in bf16, fp32 in TMEM, with P = hi + lo (about 16 bits): two products per
// weight, both parts over their logits in TMEM.
//
// Warps: 0-3 and 4-7 softmax of row tile 0 and 1 (a thread is a row); 8-15 unpack the cache (8-11 keys, 12-15
// values; a thread has half of a token's codes); 16 and 17 issue the MMAs of row tile 0 and 1; 18 copies raw
// rows, up to three steps of 64 tokens ahead, one bulk copy per run of tokens that lie together on a page.  (bf16:
// 8-15 copy the rows to their swizzled places themselves, 16 bytes a copy, three steps in flight.)  The K and V tiles
// are double-buffered.  A row tile's chain S(t) -> P(t) -> O += P V, S(t+1) is in issue order, so an observed S(t)
// also means that P(t-1) V is complete and O may be read and rescaled; while one row tile is in its softmax the
// tensor cores work for the other.
//
// Units are split evenly over the SMs by 128-token tiles as in paged_attend.cu; the last CTA of a split
// unit merges its shares in the order of the CTAs.
//
// Measured on B200, 1024 new tokens at 28672, 32 query / 8 kv heads, d = 128 (472 GFLOP; 293 us at the measured
// bf16 rate): 662 us, 713 TFLOP/s.  It is bound by the chain of one row tile (about 6300 clocks per 128 tokens:
// products 1500, exponentials 2050 at 16 a clock for both row tiles together, TMEM reads and barriers): the tensor pipe
// is used 34 % of the time, the issue slots 51 %.  When the kernel took 667 us it took 426 without the exponentials, 577
// without the unpacking, 518 with one product in eight.  Steps that counted: four to eight unpacking warps 1128 -> 892,
// the weights' product not waiting for the next keys -> 805, loops over 32 columns kept rolled (the roles share the
// instruction cache) -> 666.  The same from bf16 pages (708 GFLOP with the weights' two parts, 439 us at that rate):
// 697 us, where the mma.sync kernel takes 3509.
#include "paged.cuh"
#include "tc.cuh"

#include <cuda_fp16.h>

namespace spa {
namespace {

using namespace tc;

constexpr int kKeys = 128;                // tokens per tile
constexpr int kHalf = 64;                 // tokens per unpacking step
constexpr int kUnpack = 8;                // unpacking warps
constexpr int kThreads = (8 + kUnpack + 3) * 32;
constexpr int kSegC = 6;                  // tiles charged to a unit
constexpr int kChunkUnits = 256;          // sequences of a launch: 4 bytes of shared memory each
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kBase = 9.f, kSlack = 6.f;
constexpr int kSpread = 11;               // powers of two over which scales in the same units are exact
constexpr uint32_t kSpin = 1u << 22, kStallSpin = 1u << 10;   // tries of a wait; with the test hook

template <int D, bool INT4>
struct ChunkShared {
    static constexpr int kSlabs = D / 64;
    static constexpr int kTile = kSlabs * kSlab;       // 128 rows of D fp16
    uint8_t q[2][kTile];
    uint8_t k[2][kTile];
    uint8_t v[2][kTile];
    static constexpr int ROWB = D + 16;
    uint8_t raw[3][INT4 ? kHalf * ROWB : 16];
    uint64_t raw_full[3], raw_empty[3];
    uint32_t raw_valid[3][2];                          // tokens of the step that exist
    uint32_t raw_end;                                  // steps copied before a wait of the copying warp gave up
    uint64_t s_full[2], p_full[2][2], pv_half[2];      // by row tile (and half of the tokens)
    uint64_t k_full[2], v_full[2], k_empty[2], v_empty[2], o_done, q_full;
    alignas(16) uint32_t pw[4][4];                     // the powers of two of tile t (slot t % 4) by 32 tokens: power_word
    alignas(16) int8_t ek1[4][kKeys];                  // ... by token
    alignas(16) int8_t ev1[4][kKeys];
    uint32_t poison[4][4][4];                          // 4-bit, tile t: tokens whose values of group g are not finite
    // bf16, tile t (one that not all queries see whole): by token, a bit for each channel whose value is not finite,
    // and whether a warp found one in a half
    alignas(16) uint8_t bad[INT4 ? 1 : 4][INT4 ? 1 : kKeys][D / 8];
    uint32_t any_bad[INT4 ? 1 : 4][2][kUnpack / 2];
    uint32_t tmem_base;
    int fail;                                          // a bounded wait gave up
    int last;
    alignas(16) uint32_t valid[4][4];                  // tile t: tokens that exist
    long long wsum[kThreads / 32];
};

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
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
__device__ __forceinline__ bool elect_one() {          // one lane of a converged warp
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc));
}
// Instruction descriptor of kind::f16 with fp16 A and B, fp32 D; B K- or MN-major
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
    return (1u << 4) | (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};\n" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// 16 columns of this thread's TMEM lane, not to be used before ld_wait
__device__ __forceinline__ void ld16_begin(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void ld_wait(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}
// Fp16 pairs of scales s, and -8 s in the units of the two kinds of codes below.
struct Scale2 {
    uint32_t s, lo, hi;
};
__device__ __forceinline__ Scale2 scale2(float a, float b) {
    Scale2 r;
    r.s = pack_f16(a, b);
    r.lo = mul_f16x2(r.s, 0x80408040u);                // -8 * 2^-21
    r.hi = mul_f16x2(r.s, 0x84008400u);                // -8 * 2^-17
    return r;
}
// Eight codes of a word as (u - 8) s, in the order 0 4 1 5 2 6 3 7.  A code in bits 3-6 is the fp16
// denormal u * 2^-21, in bits 7-10 u * 2^-17 (bit 10 is the exponent's lowest, whose step is the denormals'):
// even codes come times 2^-21, odd ones times 2^-17.  (u - 8) s has at most 3 + 8 bits, the lowest of them
// 2^-7 of s's power of two; with that power at least 2^4 it is not below 2^-24, fp16's last place, and the result
// is exact.  The largest scale has 2^15, so scales may lie 2^kSpread apart; a smaller one is off by up to 2^-4.
__device__ __forceinline__ uint4 unpack8(uint32_t w, const Scale2& a, const Scale2& b) {
    const uint32_t x = w << 3, y = w >> 5;
    return make_uint4(fma_f16x2(x & 0x00780078u, a.s, a.lo), fma_f16x2(x & 0x07800780u, a.s, a.hi),
                      fma_f16x2(y & 0x00780078u, b.s, b.lo), fma_f16x2(y & 0x07800780u, b.s, b.hi));
}

// paired fp32 arithmetic (one instruction for two lanes of a 64-bit register pair)
__device__ __forceinline__ void ffma2(float& r0, float& r1, float b, float c) {   // r * b + c
    asm("{\n .reg .b64 a, x, y;\n mov.b64 a, {%0, %1};\n mov.b64 x, {%2, %2};\n mov.b64 y, {%3, %3};\n"
        " fma.rn.f32x2 a, a, x, y;\n mov.b64 {%0, %1}, a;\n}\n"
        : "+f"(r0), "+f"(r1)
        : "f"(b), "f"(c));
}
__device__ __forceinline__ void fadd2(float& r0, float& r1, float a0, float a1) {
    asm("{\n .reg .b64 a, x;\n mov.b64 a, {%0, %1};\n mov.b64 x, {%2, %3};\n add.f32x2 a, a, x;\n mov.b64 {%0, %1}, a;\n}\n"
        : "+f"(r0), "+f"(r1)
        : "f"(a0), "f"(a1));
}
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {   // of a number and a NaN the number
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Whether one of four bf16 scales is not zero and its bits are at most `limit` (the same in both halves): less one as
// 16-bit integers, zeros are the largest (NaNs are above any scale).
__device__ __forceinline__ bool any_below(uint32_t a, uint32_t b, uint32_t limit) {
    uint32_t m;
    asm("{\n .reg .b32 x, y;\n add.u16x2 x, %1, %3;\n add.u16x2 y, %2, %3;\n min.u16x2 x, x, y;\n min.u16x2 %0, x, %4;\n}\n"
        : "=r"(m)
        : "r"(a), "r"(b), "r"(0xffffffffu), "r"(limit));
    return m != limit;
}
// the powers of two of 64 tokens' keys and values, and whether 32 of them have their own instead
__device__ __forceinline__ uint32_t power_word(int ek, int ev, bool own) {
    return (uint32_t(ek) & 0xffu) | (uint32_t(ev) & 0xffu) << 8 | (own ? 1u << 16 : 0u);
}

// floats of one share of a split unit: O [D / 4][256][4], then m, l and four words of poisoned groups (4-bit: the
// first) or channels of each row
__host__ __device__ constexpr int chunk_rec_floats(int d) { return 256 * (d + 6); }

struct SeqG { int n, len, row0; };
__device__ __forceinline__ SeqG seq_geo(const PagedAttendParams& p, int b, bool* bad) {
    SeqG s;
    s.len = paged_len(p.kv, p.kv.kv_len[b], bad);
    const long long a = p.seq_start[b], e = p.seq_start[b + 1];
    if (!paged_rows_ok(a, e, p.T)) { *bad = true; s.n = 0; s.row0 = 0; }
    else { s.n = int(e - a); s.row0 = int(a); }
    return s;
}
__device__ __forceinline__ long long head_weight(const SeqG& s, int TQ) {
    long long w = 0;
    const int nj = (s.n + TQ - 1) / TQ;
    for (int j = 0; j < nj; ++j) {
        const int lim = paged_tile_limit(s.len, s.n, TQ, j);
        if (lim > 0) w += (lim + kKeys - 1) / kKeys + kSegC;
    }
    return w;
}

template <int D, bool INT4>
__global__ void __launch_bounds__(kThreads, 1) paged_chunk_kernel(PagedAttendParams p, int g0, int groups, int TQ) {
    using SH = ChunkShared<D, INT4>;
    static_assert(offsetof(SH, valid) % 16 == 0 && offsetof(SH, pw) % 16 == 0 && offsetof(SH, raw) % 16 == 0 && SH::ROWB % 16 == 0 && offsetof(SH, ek1) % 16 == 0 &&
                  sizeof(SH) % 8 == 0, "alignment of shared accesses");
    constexpr int NW = INT4 ? 1 : D / 32;              // words of poisoned groups or channels
    constexpr int WORDS = D / 8;                       // 16-byte pieces of an operand row, code words of a row
    extern __shared__ __align__(1024) uint8_t dyn[];
    SH& sh = *reinterpret_cast<SH*>(dyn);
    uint32_t* const s_prefix = reinterpret_cast<uint32_t*>(dyn + sizeof(SH));   // [groups + 1]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.Hq / p.kv.Hkv;

    if (warp == 0) tmem_alloc(&sh.tmem_base, 512);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            for (int h = 0; h < 2; ++h) mbar_init(&sh.p_full[i][h], 128);
            mbar_init(&sh.pv_half[i], 1);
            mbar_init(&sh.k_full[i], kUnpack);         // 4 warps x 2 steps
            mbar_init(&sh.v_full[i], kUnpack);
            mbar_init(&sh.k_empty[i], 2);              // both row tiles are through with it
            mbar_init(&sh.v_empty[i], 2);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], kUnpack);
        }
        mbar_init(&sh.o_done, 2);
        mbar_init(&sh.q_full, 256);
        sh.fail = 0;
        sh.raw_end = 0xffffffffu;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    pdl_enter();

    // ---- weighted tile prefix over the sequences
    long long running = 0;
    bool empties = false;
    for (int base = 0; base < groups; base += kThreads) {
        const int u = base + tid;
        long long t = 0;
        if (u < groups) {
            bool bad = false;
            const SeqG s = seq_geo(p, g0 + u, &bad);
            t = head_weight(s, TQ) * p.kv.Hkv;
            empties |= s.n > 0 && paged_tile_limit(s.len, s.n, TQ, 0) == 0;
            if (bad && blockIdx.x == 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
        }
        long long incl = t;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += x;
        }
        if (lane == 31) sh.wsum[warp] = incl;
        __syncthreads();
        long long before = running, tot = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += sh.wsum[w];
            tot += sh.wsum[w];
        }
        if (u < groups) s_prefix[u] = uint32_t(before + incl - t);
        running += tot;
        __syncthreads();
    }
    if (tid == 0) s_prefix[groups] = uint32_t(running);
    tc_fence_before();
    empties = __syncthreads_or(empties);               // (also: barriers initialised, TMEM allocated)
    tc_fence_after();
    // Starts out of order can make sequences overlap, and their tiles more than the host counted and the prefix holds.
    if (running > 0xffffffffll) {
        if (blockIdx.x == 0 && tid == 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
        running = 0;
    }
    const long long TT = running;
    const int cta = blockIdx.x;
    const long long shares = (TT + kSegC) / (kSegC + 1);
    const int GC = int(shares < (long long)gridDim.x ? shares : (long long)gridDim.x);
    const uint32_t tmem = sh.tmem_base;

    // ---- query tiles that see no key: out = 0, lse = -inf
    for (int u = cta; empties && u < groups; u += gridDim.x) {
        bool bad = false;
        const SeqG s = seq_geo(p, g0 + u, &bad);
        for (int j = 0; j * TQ < s.n && paged_tile_limit(s.len, s.n, TQ, j) == 0; ++j) {
            const int rows = min(TQ, s.n - j * TQ) * p.Hq;
            const size_t r0 = size_t(s.row0 + j * TQ) * p.Hq;
            for (int i = tid; i < rows * D; i += kThreads) {
                p.out[r0 * D + i] = 0;
                if (p.out_f32) p.out_f32[r0 * D + i] = 0.f;
                if (p.lse && i % D == 0) p.lse[r0 + i / D] = -INFINITY;
            }
        }
    }

    // bounded wait on a barrier's phase; on expiry, or once another thread's has expired, false
    auto wait = [&](uint64_t* bar, uint32_t par) -> bool {
        for (uint32_t it = 0; !mbar_try_wait(bar, par); ++it) {
            if (it >= p.spin || ((it & 255u) == 255u && *reinterpret_cast<volatile int*>(&sh.fail))) {
                if (it >= p.spin) raise_status(p.status, SPA_ERR_TIMEOUT);
                *reinterpret_cast<volatile int*>(&sh.fail) = 1;
                return false;
            }
        }
        return true;
    };

    const long long x0 = cta < GC ? TT * cta / GC : 0, x1 = cta < GC ? TT * (cta + 1) / GC : 0;
    int grp = 0;
    {
        int lo = 0, hi = groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_prefix[mid] <= x0) lo = mid; else hi = mid;
        }
        grp = lo;
    }
    const float sl2 = p.sm_scale * kLog2e;
    // uses of the barriers so far, by role: tiles filled / consumed over all segments, and segments
    uint32_t raw_done = 0;                             // steps of 64 tokens
    uint32_t tiles_done = 0, tiles1_done = 0, segs = 0;   // (tiles1: those in which row tile 1 took part)

    long long x = x0;
    while (x < x1) {
        while (s_prefix[grp + 1] <= x) ++grp;
        bool bad = false;
        const SeqG sq = seq_geo(p, g0 + grp, &bad);
        const long long hw = (s_prefix[grp + 1] - s_prefix[grp]) / p.kv.Hkv;
        long long rem = x - s_prefix[grp];
        const int g = int(rem / hw);
        rem -= g * hw;
        long long u_lo = s_prefix[grp] + g * hw;
        int j = 0, lim;
        for (;;) {
            lim = paged_tile_limit(sq.len, sq.n, TQ, j);
            const long long w = lim > 0 ? (lim + kKeys - 1) / kKeys + kSegC : 0;
            if (rem < w) break;
            rem -= w;
            u_lo += w;
            ++j;
        }
        const int nq = min(TQ, sq.n - j * TQ), nrow = nq * G, ntile = nrow > 128 ? 2 : 1;
        const int lim0 = lim - nq + 1;                 // keys the first query token sees
        const int row0 = sq.row0 + j * TQ;
        const int tiles = (lim + kKeys - 1) / kKeys;
        const long long u_hi = u_lo + kSegC + tiles;
        const long long seg_end = x1 < u_hi ? x1 : u_hi;
        const int a = int(x - u_lo) - kSegC > 0 ? int(x - u_lo) - kSegC : 0;
        const int bnd = int(seg_end - u_lo) - kSegC > 0 ? int(seg_end - u_lo) - kSegC : 0;
        if (a >= bnd) {
            x = seg_end;
            continue;
        }
        const int nt = bnd - a;
        const uint32_t base = tiles_done;              // tile index of this segment's first tile, over the kernel
        const uint32_t base1 = tiles1_done, base_raw = raw_done;
        raw_done += uint32_t(2 * nt);
        tiles_done += uint32_t(nt);
        if (ntile == 2) tiles1_done += uint32_t(nt);

        if (warp >= 8 && warp < 8 + kUnpack) {
            // (The two formats part inside the role: as two branches of this chain the 4-bit kernel came out 4 % slower.)
            if constexpr (!INT4) {
                // ================================================================ bf16 rows
                // Warps 8-11 copy the keys and 12-15 the values of 64 tokens at a time to their swizzled places, 16 bytes a
                // copy, three steps in flight.  A lane looks up the page of one run of tokens, a step ahead.
                constexpr int CH = D / 8, PER = kHalf * CH / 128;  // pieces of a row, and of a thread's step
                const bool isv = warp >= 12;
                const int ut = (tid - 256) & 127, c = ut % CH;     // this thread's piece, of tokens ut / CH + k (128 / CH)
                const int rsh = min(6, p.kv.page_shift), R = 1 << rsh, runs = kHalf >> rsh;
                const int32_t* const pt = p.kv.page_table + (long long)(g0 + grp) * p.kv.max_pages;
                const int steps = 2 * nt;
                auto page_of = [&](int h) -> int {                 // (lim <= len: inside the table)
                    const int n = a * kKeys + h * kHalf + lane * R;
                    return h < steps && lane < runs && n < lim ? __ldg(pt + (n >> p.kv.page_shift)) : -1;
                };
                auto place = [&](int h, int k) -> uint8_t* {       // of piece k of step h
                    const int r = (h & 1) * kHalf + ut / CH + k * (128 / CH);
                    uint8_t* const tile = isv ? sh.v[(base + uint32_t(h >> 1)) & 1] : sh.k[(base + uint32_t(h >> 1)) & 1];
                    return tile + (c >> 3) * kSlab + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                };
                auto finish = [&](int h) {                         // step h has landed
                    const uint32_t T = base + uint32_t(h >> 1);
                    if (isv && (a + (h >> 1) + 1) * kKeys > lim0) {
                        // Tokens that some of the unit's queries do not see: values that are not finite are taken as 0 (0 * NaN
                        // would reach every query) and noted for those that do see them.
                        bool found = false;
#pragma unroll
                        for (int k = 0; k < PER; ++k) {
                            uint4* const at = reinterpret_cast<uint4*>(place(h, k));
                            const uint4 w = *at;
                            uint32_t u4[4] = {w.x, w.y, w.z, w.w}, bits = 0;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if ((u4[i] & 0x7f80u) == 0x7f80u) { bits |= 1u << (2 * i); u4[i] &= 0xffff0000u; }
                                if ((u4[i] & 0x7f800000u) == 0x7f800000u) { bits |= 2u << (2 * i); u4[i] &= 0xffffu; }
                            }
                            sh.bad[T & 3][(h & 1) * kHalf + ut / CH + k * (128 / CH)][c] = uint8_t(bits);
                            if (bits) *at = make_uint4(u4[0], u4[1], u4[2], u4[3]);
                            found |= bits != 0;
                        }
                        found = __any_sync(0xffffffffu, found);
                        if (lane == 0) sh.any_bad[T & 3][h & 1][warp - 12] = found;
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive(isv ? &sh.v_full[T & 1] : &sh.k_full[T & 1]);
                };
                int pid = page_of(0), h = 0;
                for (; h < steps; ++h) {
                    const uint32_t T = base + uint32_t(h >> 1);
                    const int n = a * kKeys + h * kHalf + lane * R;
                    int rows = lane < runs ? min(max(lim - n, 0), R) : 0;
                    long long off = rows > 0 ? paged_row(p.kv, pid, g, n) : -1;
                    if (rows > 0 && off < 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
                    if (off < 0) off = rows = 0;
                    pid = page_of(h + 1);
                    if ((h & 1) == 0 && T >= 2 &&              // the tile two back has been read
                        !__all_sync(0xffffffffu, wait(isv ? &sh.v_empty[T & 1] : &sh.k_empty[T & 1], ((T >> 1) - 1) & 1)))
                        break;
                    if (warp == 8) {                           // tokens of the step that exist
                        const unsigned long long m =
                            rows > 0 ? (rows >= 64 ? ~0ull : (1ull << rows) - 1) << (lane * R & 63) : 0ull;
                        const uint32_t m0 = __reduce_or_sync(0xffffffffu, uint32_t(m));
                        const uint32_t m1 = __reduce_or_sync(0xffffffffu, uint32_t(m >> 32));
                        if (lane == 0) {
                            sh.valid[T & 3][2 * (h & 1)] = m0;
                            sh.valid[T & 3][2 * (h & 1) + 1] = m1;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < PER; ++k) {
                        const int tok = ut / CH + k * (128 / CH), run = tok >> rsh, i = tok & (R - 1);
                        const long long o = __shfl_sync(0xffffffffu, off, run);
                        const bool there = i < __shfl_sync(0xffffffffu, rows, run);
                        const uint8_t* const src = p.kv.data + (there ? o + i * (4 * D) + (isv ? 2 * D : 0) + c * 16 : 0);
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(place(h, k))), "l"(src),
                                     "r"(there ? 16 : 0)       // (zeros where there is no token)
                                     : "memory");
                    }
                    asm volatile("cp.async.commit_group;\n" ::: "memory");
                    if (h >= 2) {
                        asm volatile("cp.async.wait_group 2;\n" ::: "memory");
                        finish(h - 2);
                    }
                }
                asm volatile("cp.async.wait_group 0;\n" ::: "memory");
                if (h == steps) {
                    finish(h - 2);                             // (steps is even)
                    finish(h - 1);
                }
                __syncwarp();
            } else {
                // ================================================================ unpacking
                // Keys and values have their own warps, which meet only at the raw rows, three steps deep.
                const bool isv = warp >= 12;
                const int ut = (tid - 256) & 127, part = ut >> 6, tok = ut & 63;
                constexpr int ROWB = SH::ROWB;
                const int steps = 2 * nt;
                for (int h = 0; h < steps; ++h) {
                    const uint32_t T = base + uint32_t(h >> 1);        // tile over the kernel
                    const int stage = T & 1, half = h & 1;
                    const uint32_t S = base_raw + uint32_t(h), slot = S % 3;
                    if (!__all_sync(0xffffffffu, wait(&sh.raw_full[slot], (S / 3) & 1))) break;
                    const uint8_t* raw = sh.raw[slot];
                    // powers of two: the largest scale (that is a number) of the 64 tokens to [2^15, 2^16)
                    auto top = [](uint32_t w) -> uint32_t { return max(w & 0x7fffu, (w >> 16) & 0x7fffu); };   // of two bf16
                    uint32_t kmx, vmx;
                    {
                        const uint4 s0 = *reinterpret_cast<const uint4*>(raw + lane * ROWB + D);
                        const uint4 s1 = *reinterpret_cast<const uint4*>(raw + (lane + 32) * ROWB + D);
                        kmx = top(max_bf16x2(max_bf16x2(max_bf16x2(s0.x, s0.y), max_bf16x2(s1.x, s1.y)), 0u));
                        vmx = top(max_bf16x2(max_bf16x2(max_bf16x2(s0.z, s0.w), max_bf16x2(s1.z, s1.w)), 0u));
                        if (isv) kmx = 0;                      // (only the key warps of part 0 need both)
                        else if (part) vmx = 0;
                    }
                    auto expo = [](uint32_t m) { return min(max(int(m >> 7) - 127, -70), 127) - 15; };
                    const uint8_t* row = raw + tok * ROWB;
                    const uint4 all = *reinterpret_cast<const uint4*>(row + D);
                    // A tile that some queries do not see whole: every token has its own powers of two, so that what a
                    // query does not see cannot push what it sees out of fp16's range.  So have the 32 tokens of a warp
                    // where one has a scale too far below the 64 tokens' largest to be exact in its units: a token of
                    // large keys or values and little weight must not blur the others.  (Keys and values each by
                    // themselves; the warps of both parts find the same.)
                    const bool edge = (a + (h >> 1) + 1) * kKeys > lim0;
                    int ek = 0, ev = 0;
                    bool kown = edge, vown = edge;
                    if (!edge) {
                        auto below = [](int e) { return uint32_t(((e + 15 + 127 - kSpread) << 7) - 1) * 0x10001u; };
                        if (!isv) {
                            ek = expo(__reduce_max_sync(0xffffffffu, kmx));
                            kown = __any_sync(0xffffffffu, any_below(all.x, all.y, below(ek)));
                        }
                        if (isv || part == 0) {
                            ev = expo(__reduce_max_sync(0xffffffffu, vmx));
                            vown = __any_sync(0xffffffffu, any_below(all.z, all.w, below(ev)));
                        }
                    }
                    if (!isv && part == 0 && lane == 0) sh.pw[T & 3][(half * kHalf + tok) >> 5] = power_word(ek, ev, kown || vown);
                    if (kown) ek = expo(top(max_bf16x2(max_bf16x2(all.x, all.y), 0u)));
                    if (vown) ev = expo(top(max_bf16x2(max_bf16x2(all.z, all.w), 0u)));
                    if (!isv && part == 0) {
                        sh.ek1[T & 3][half * kHalf + tok] = int8_t(ek);
                        sh.ev1[T & 3][half * kHalf + tok] = int8_t(ev);
                    }
                    const uint2 sc = isv ? make_uint2(all.z, all.w) : make_uint2(all.x, all.y);
                    const float mul = pow2i(isv ? -ev : -ek);
                    float f[4] = {bf_lo(sc.x) * mul, bf_hi(sc.x) * mul, bf_lo(sc.y) * mul, bf_hi(sc.y) * mul};
                    const int r = half * kHalf + tok;      // row of the operand tile
                    if (isv && edge) {
                        // Tokens that some of the unit's queries do not see: a group that is not finite is taken as 0
                        // (0 * NaN would reach every query) and noted for those that do see it.
                        const int n = (a + (h >> 1)) * kKeys + r;
#pragma unroll
                        for (int gr = 0; gr < 4; ++gr) {
                            const bool nan = n < lim && !(fabsf(f[gr]) <= 3.402823466e38f);
                            const uint32_t m = __ballot_sync(0xffffffffu, nan);
                            if (lane == 0 && part == 0) sh.poison[T & 3][gr][r >> 5] = m;
                            if (nan) f[gr] = 0.f;
                        }
                    }
                    if (!isv && part == 0 && lane == 0) sh.valid[T & 3][r >> 5] = sh.raw_valid[slot][tok >> 5];
                    if (half == 0 && T >= 2) {             // the tile two back has been read
                        if (!__all_sync(0xffffffffu,
                                        wait(isv ? &sh.v_empty[stage] : &sh.k_empty[stage], ((T >> 1) - 1) & 1)))
                            break;
                    }
                    uint8_t* dst = isv ? sh.v[stage] : sh.k[stage];
                    const uint32_t* codes = reinterpret_cast<const uint32_t*>(row + (isv ? D / 2 : 0));
                    // scale pairs of a word's code pairs (0,4) (1,5) and (2,6) (3,7), for the words that differ in them
                    Scale2 s2[4];
                    if (D == 128) {
                        if (isv) {                         // word 2 r + hh: groups 2 hh and 2 hh + 1
                            s2[0] = s2[2] = scale2(f[0], f[1]);
                            s2[1] = s2[3] = scale2(f[2], f[3]);
                        } else {                           // word 4 t + g: group g
#pragma unroll
                            for (int gr = 0; gr < 4; ++gr) s2[gr] = scale2(f[gr], f[gr]);
                        }
                    } else {
                        if (isv) {                         // word r: groups 0 and 2, then 1 and 3
                            s2[0] = scale2(f[0], f[2]);
                            s2[1] = scale2(f[1], f[3]);
                        } else {                           // word 2 t + i: groups 2 i and 2 i + 1
                            s2[0] = scale2(f[0], f[1]);
                            s2[1] = scale2(f[2], f[3]);
                        }
                    }
                    // piece of the operand row: keys in word order; values so that a 64-channel slab is hh
                    uint8_t* const out = dst + r * 128;
#pragma unroll
                    for (int w4 = 0; w4 < WORDS / 8; ++w4) {
                        const int at = part * (WORDS / 8) + w4;
                        const uint4 w = *reinterpret_cast<const uint4*>(codes + 4 * at);
                        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int wi = 4 * at + i;
                            uint4 o;
                            int c;
                            if constexpr (D == 128) {
                                o = unpack8(ws[i], s2[i], s2[i]);
                                c = isv ? (i & 1) * 8 + (wi >> 1) : wi;
                            } else {
                                o = isv ? unpack8(ws[i], s2[0], s2[1]) : unpack8(ws[i], s2[i & 1], s2[i & 1]);
                                c = wi;
                            }
                            *reinterpret_cast<uint4*>(out + (c >> 3) * kSlab + (((c & 7) ^ (r & 7)) << 4)) = o;
                        }
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        arrive(&sh.raw_empty[slot]);
                        arrive(isv ? &sh.v_full[stage] : &sh.k_full[stage]);
                    }
                }
            }
        } else if (warp == 8 + kUnpack || warp == 8 + kUnpack + 1) {
            // ================================================================ MMA issue
            // A warp per row tile, so that neither waits for the other's weights (one warp for both: 696 us, where two took
            // 667).  The whole warp runs the loop, so that descriptors stay in uniform registers; one elected lane issues.
            constexpr uint32_t kIdS = INT4 ? idesc_f16(128, kKeys, false) : idesc_bf16(128, kKeys, false);
            constexpr uint32_t kIdO = INT4 ? idesc_f16(128, D, true) : idesc_bf16(128, D, true);
            const uint64_t dq0 = sw128_desc(smem_u32(sh.q[0]), 16, 1024);
            const uint64_t dk0 = sw128_desc(smem_u32(sh.k[0]), 16, 1024);
            const uint64_t dv0 = sw128_desc(smem_u32(sh.v[0]), kSlab, 1024);
            constexpr uint64_t kTile16 = SH::kTile >> 4;       // a stage's or row tile's step in a descriptor
            // S of row tile i against a tile's keys; O += P V over 64 tokens
            const int i = warp - (8 + kUnpack);
            const bool solo = ntile == 1;              // row tile 0 stands for both
            const bool part = i < ntile;
            const bool leader = elect_one();           // one thread issues and commits: a commit tracks its own thread's MMAs
            auto s_mma = [&](uint32_t T) {
                const uint64_t dq = dq0 + uint32_t(i) * kTile16;
                const uint64_t dk = dk0 + (T & 1) * kTile16;
                const uint32_t dst = tmem + i * 128;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t off = uint64_t(((kk >> 2) * kSlab + (kk & 3) * 32) >> 4);
                        umma_bf16(dst, dq + off, dk + off, kIdS, kk > 0);
                    }
                    umma_commit(&sh.s_full[i]);
                }
                __syncwarp();
            };
            auto pv_mma = [&](uint32_t T, int h, bool first) {
                const uint64_t dv = dv0 + (T & 1) * kTile16 + uint64_t(h * ((kHalf * 128) >> 4));
                const uint32_t src = tmem + i * 128 + h * 64, dst = tmem + 256 + i * 128;
                const uint32_t acc0 = !first || h > 0 ? 1u : 0u;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kHalf / 16; ++kk) {
                        const uint64_t dk16 = dv + uint64_t((kk * 2048) >> 4);
                        if constexpr (INT4) {
                            umma_ts(dst, src + kk * 8, dk16, kIdO, kk > 0 ? 1u : acc0);
                        } else {                       // of 32 tokens the high parts, then the low parts
                            umma_ts(dst, src + (kk >> 1) * 32 + (kk & 1) * 8, dk16, kIdO, kk > 0 ? 1u : acc0);
                            umma_ts(dst, src + (kk >> 1) * 32 + (kk & 1) * 8 + 16, dk16, kIdO, 1u);
                        }
                    }
                    if (h == 0) umma_commit(&sh.pv_half[i]);
                }
                __syncwarp();
            };
            auto commit = [&](uint64_t* bar) {
                if (leader) {
                    umma_commit(bar);
                    if (solo) umma_commit(bar);
                }
                __syncwarp();
            };
            auto all = [&](bool v) { return __all_sync(0xffffffffu, v) != 0; };
            // (a warp without a row tile waits for the queries all the same: it must not run ahead of a phase)
            bool live = all(wait(&sh.q_full, segs & 1)) && part && all(wait(&sh.k_full[base & 1], (base >> 1) & 1));
            if (live && !p.stall) {
                tc_fence_after();
                s_mma(base);
                commit(&sh.k_empty[base & 1]);
            }
            // Half by half: O takes the first half's weights while the softmax is at the second.  (Logits by halves too,
            // N = 64, so that the next tile's begin as early, take half as many products again, about 73 clocks each at
            // either width: slower.)
            for (int t = 0; live && t < nt; ++t) {
                const uint32_t T = base + uint32_t(t);
                live = all(wait(&sh.v_full[T & 1], (T >> 1) & 1));
                for (int h = 0; live && h < 2; ++h) {
                    live = all(wait(&sh.p_full[i][h], ((i ? base1 : base) + uint32_t(t)) & 1));
                    if (!live) break;
                    tc_fence_after();
                    pv_mma(T, h, t == 0);
                }
                if (!live) break;
                commit(&sh.v_empty[T & 1]);
                if (t + 1 < nt) {
                    live = all(wait(&sh.k_full[(T + 1) & 1], ((T + 1) >> 1) & 1));
                    if (!live) break;
                    tc_fence_after();
                    s_mma(T + 1);
                    commit(&sh.k_empty[(T + 1) & 1]);
                }
            }
            if (part) commit(&sh.o_done);
            if (part && !live) wait(&sh.o_done, segs & 1);   // what was issued before a wait gave up
            __syncwarp();
        } else if (INT4 && warp == 8 + kUnpack + 2) {
            // ================================================================ raw rows
            constexpr int ROWB = SH::ROWB;
            const int rsh = min(6, p.kv.page_shift), R = 1 << rsh, runs = kHalf >> rsh;   // runs of R tokens per step
            const int32_t* const pt = p.kv.page_table + (long long)(g0 + grp) * p.kv.max_pages;
            const int steps = 2 * nt;
            // page of this lane's run of step h (lim <= len: inside the table)
            auto page_of = [&](int h) -> int {
                const int n = a * kKeys + h * kHalf + lane * R;
                return h < steps && lane < runs && n < lim ? __ldg(pt + (n >> p.kv.page_shift)) : -1;
            };
            int pid = page_of(0);
            for (int h = 0; h < steps && sh.raw_end == 0xffffffffu; ++h) {
                const uint32_t S = base_raw + uint32_t(h), slot = S % 3;
                const int n = a * kKeys + h * kHalf + lane * R;
                int rows = lane < runs ? min(max(lim - n, 0), R) : 0;
                const long long off = rows > 0 ? paged_row(p.kv, pid, g, n) : -1;
                if (rows > 0 && off < 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
                if (off < 0) rows = 0;
                pid = page_of(h + 1);
                if (S >= 3 && !__all_sync(0xffffffffu, wait(&sh.raw_empty[slot], (S / 3 - 1) & 1))) {
                    if (lane == 0) sh.raw_end = S;     // nothing is copied any more, in later segments either
                    break;
                }
                const uint32_t dst = smem_u32(sh.raw[slot]) + lane * R * ROWB;
                uint32_t m0 = 0, m1 = 0;               // this lane's tokens among the step's 64
                if (rows > 0) {
                    const unsigned long long m = (rows >= 64 ? ~0ull : (1ull << rows) - 1) << (lane * R & 63);
                    m0 = uint32_t(m);
                    m1 = uint32_t(m >> 32);
                }
                m0 = __reduce_or_sync(0xffffffffu, m0);
                m1 = __reduce_or_sync(0xffffffffu, m1);
                if ((m0 & m1) != 0xffffffffu && lane < runs) {   // tokens that do not exist: scales of zero
                    for (int i = rows; i < R; ++i)
                        *reinterpret_cast<uint4*>(sh.raw[slot] + (lane * R + i) * ROWB + D) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                }
                if (lane == 0) {
                    sh.raw_valid[slot][0] = m0;
                    sh.raw_valid[slot][1] = m1;
                }
                __syncwarp();                          // the zeros and the masks before the arrival
                if (lane == 0)
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(
                                     smem_u32(&sh.raw_full[slot])),
                                 "r"(uint32_t((__popc(m0) + __popc(m1)) * ROWB))
                                 : "memory");
                __syncwarp();
                if (rows > 0)
                    asm volatile(
                        "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
                        "l"(p.kv.data + off), "r"(uint32_t(rows * ROWB)), "r"(smem_u32(&sh.raw_full[slot]))
                        : "memory");
            }
            __syncwarp();
        } else if (warp < 8) {
            // ================================================================ softmax
            const int rt = warp >> 2, r = (warp & 3) * 32 + lane, row = rt * 128 + r;
            const bool have = row < nrow;
            const uint32_t t_s = tmem + rt * 128 + (uint32_t((warp & 3) * 32) << 16);
            const uint32_t t_o = t_s + 256;
            const int lim_r = have ? lim0 + row / G : lim;
            float hrow;
            if (!INT4 && rt < ntile) {
                const uint16_t* src = p.q + (have ? (row0 + row / G) * p.q_tok + (g * G + row % G) * p.q_head : 0);
                hrow = sl2;
#pragma unroll
                for (int c = 0; c < WORDS; ++c)
                    *reinterpret_cast<uint4*>(sh.q[rt] + (c >> 3) * kSlab + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                        have ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            if (INT4 && rt < ntile) {
                // this row of Q: its largest channel to [2^13, 2^14), pieces and order as the keys'
                const uint16_t* src = p.q + (have ? (row0 + row / G) * p.q_tok + (g * G + row % G) * p.q_head : 0);
                uint4 w[WORDS];
                uint32_t mx = 0;
#pragma unroll
                for (int c = 0; c < WORDS; ++c) {
                    w[c] = have ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
                    const uint32_t u4[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = max(mx, max(u4[i] & 0x7fffu, (u4[i] >> 16) & 0x7fffu));
                }
                int ex = 13 - (int(mx >> 7) - 127);
                ex = ex > 100 ? 100 : ex < -100 ? -100 : ex;
                const float up = pow2i(ex);
                hrow = sl2 * pow2i(-ex) * 2097152.f;       // 2^21: the unit of the even codes
                auto chan = [&](int ch) -> float {         // channel ch of the row, scaled
                    const uint4 v = w[ch >> 3];
                    const uint32_t u = (ch & 7) < 2 ? v.x : (ch & 7) < 4 ? v.y : (ch & 7) < 6 ? v.z : v.w;
                    return (ch & 1 ? bf_hi(u) : bf_lo(u)) * up;
                };
#pragma unroll
                for (int c = 0; c < WORDS; ++c) {
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {          // codes i and i + 4 of the key word c
                        int c0, c1;
                        if (D == 128) {
                            c0 = 32 * (c & 3) + 8 * (c >> 2) + i;
                            c1 = c0 + 4;
                        } else {
                            c0 = 16 * (2 * (c & 1)) + 4 * (c >> 1) + i;
                            c1 = c0 + 16;
                        }
                        // odd codes are held 2^4 times the even ones
                        o[i] = (i & 1) ? pack_f16(chan(c0) * 0.0625f, chan(c1) * 0.0625f) : pack_f16(chan(c0), chan(c1));
                    }
                    *reinterpret_cast<uint4*>(sh.q[rt] + (c >> 3) * kSlab + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
                fence_async_smem();
            }
            tc_fence_before();
            arrive(&sh.q_full);

            auto n0_of = [&](int t) { return (a + t) * kKeys; };
            float m = -INFINITY, l = 0.f;
            uint32_t nan[NW] = {};                         // groups (bf16: channels) of V that are not finite in a token it sees
            // values of tile t are unpacked once P(t) V is complete, which S(t + 1) shows
            auto poisoned = [&](int t) {
                if (n0_of(t) + kKeys <= lim0) return;
                const int seen = lim_r - n0_of(t);
                const int slot = (base + uint32_t(t)) & 3;
                if constexpr (INT4) {
#pragma unroll
                    for (int gr = 0; gr < 4; ++gr)
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const int c = seen - 32 * w;
                            const uint32_t vis = c >= 32 ? 0xffffffffu : c <= 0 ? 0u : (1u << c) - 1u;
                            if (sh.poison[slot][gr][w] & vis) nan[0] |= 1u << gr;
                        }
                } else {
                    uint32_t any = 0;
                    for (int i = 0; i < kUnpack; ++i) any |= sh.any_bad[slot][i >> 2][i & 3];
                    if (!any) return;
#pragma unroll 1
                    for (int i = 0; i < seen && i < kKeys; ++i)
#pragma unroll
                        for (int w = 0; w < NW; ++w) nan[w] |= *reinterpret_cast<const uint32_t*>(&sh.bad[slot][i][4 * w]);
                }
            };
            bool ok = rt < ntile;
            for (int t = 0; ok && t < nt; ++t) {
                const uint32_t T = base + uint32_t(t), Ti = (rt ? base1 : base) + uint32_t(t);
                ok = __all_sync(0xffffffffu, wait(&sh.s_full[rt], Ti & 1));
                if (!ok) break;
                tc_fence_after();
                const int n0 = n0_of(t);
                const uint4 vd = *reinterpret_cast<const uint4*>(sh.valid[T & 3]);
                const uint32_t vm[4] = {vd.x, vd.y, vd.z, vd.w};
                bool edge = n0 + kKeys > lim0;
                const bool gaps = (vm[0] & vm[1] & vm[2] & vm[3]) != 0xffffffffu;
                const int seen = lim_r - n0;               // columns below this one are seen
                float cs[2] = {hrow, hrow}, ev[2] = {0.f, 0.f};
                if constexpr (INT4) {
                    const uint4 pw = *reinterpret_cast<const uint4*>(sh.pw[T & 3]);
                    edge |= (pw.x | pw.y | pw.z | pw.w) >> 16 != 0;    // powers of two by token
                    cs[0] = hrow * pow2i(int8_t(pw.x));
                    cs[1] = hrow * pow2i(int8_t(pw.z));
                    ev[0] = float(int8_t(pw.x >> 8));
                    ev[1] = float(int8_t(pw.z >> 8));
                }
                // logits + V's power of two of 32 tokens, for tiles with tokens that are not seen or do not exist
                auto masked = [&](int q4, float (&v)[32]) {
#pragma unroll
                    for (int i4 = 0; i4 < 8; ++i4) {
                        if constexpr (!INT4) {
#pragma unroll
                            for (int i = 4 * i4; i < 4 * i4 + 4; ++i)
                                v[i] = ((vm[q4] >> i) & 1u) && q4 * 32 + i < seen ? v[i] * hrow : -INFINITY;
                            continue;
                        }
                        const char4 e = reinterpret_cast<const char4*>(sh.ek1[T & 3])[q4 * 8 + i4];
                        const char4 f = reinterpret_cast<const char4*>(sh.ev1[T & 3])[q4 * 8 + i4];
                        const int ee[4] = {e.x, e.y, e.z, e.w}, ff[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int i = 4 * i4 + k;
                            v[i] = ((vm[q4] >> i) & 1u) && q4 * 32 + i < seen
                                       ? fmaf(v[i], hrow * pow2i(ee[k]), float(ff[k]))
                                       : -INFINITY;
                        }
                    }
                };
                // The reference of the warp's rows up to `top` where that exceeds it by 2^kSlack, with l and O.  What has
                // been issued into O is complete before: of the tile before, shown by S(t); at the second half, this
                // tile's first.
                auto follow = [&](float top, int h) {
                    if (h == 1) {
                        ok = __all_sync(0xffffffffu, wait(&sh.pv_half[rt], Ti & 1)) && ok;
                        tc_fence_after();
                    }
                    const float mn = top > m + kSlack ? top : m;
                    const float f = mn == -INFINITY ? 1.f : ex2_approx(m - mn);
                    m = mn;
                    l *= f;
                    if (t > 0 || h == 1) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float v[32];
                            tmem_ld32(t_o + c, v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] *= f;
                            tmem_st32(t_o + c, v);
                        }
                        tmem_wait_st();
                    }
                };
                auto done = [&](int h) {               // the weights of a half are stored
                    tmem_wait_st();
                    tc_fence_before();
                    arrive(&sh.p_full[rt][h]);
                };
                // (the loops over 32 columns are not unrolled: the warps' roles share the instruction cache)
                auto top_of = [&](int q0, int q1) -> float {
                    float top = -INFINITY;
#pragma unroll 1
                    for (int q4 = q0; q4 < q1; ++q4) {
                        float v[32];
                        tmem_ld32(t_s + q4 * 32, v);
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        if (edge || gaps) masked(q4, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], v[i]);
                        const float x4 = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        top = fmaxf(top, edge || gaps ? x4 : fmaf(x4, q4 < 2 ? cs[0] : cs[1], q4 < 2 ? ev[0] : ev[1]));
                    }
                    return top;
                };
                if constexpr (!INT4) {
                    // The maximum first, then the weights as two bf16 numbers of 32 tokens at a time, over their logits.
                    if (edge && t > 0) poisoned(t - 1);
                    const float top = top_of(0, 4);
                    if (__any_sync(0xffffffffu, top > m + kSlack)) follow(top, 0);
                    const float ref = m == -INFINITY ? 0.f : kBase - m;
                    float sum[2] = {0.f, 0.f};
#pragma unroll 1
                    for (int q4 = 0; q4 < 4; ++q4) {
                        float v[32];
                        tmem_ld32(t_s + q4 * 32, v);
                        float c = hrow;
                        if (edge || gaps) {
                            masked(q4, v);
                            c = 1.f;
                        }
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x0 = v[2 * i], x1 = v[2 * i + 1];
                            ffma2(x0, x1, c, ref);
                            x0 = ex2_approx(x0);
                            x1 = ex2_approx(x1);
                            hi[i] = pack_bf16(x0, x1);
                            lo[i] = pack_bf16(x0 - bf_lo(hi[i]), x1 - bf_hi(hi[i]));
                            fadd2(sum[0], sum[1], x0, x1);
                        }
                        tmem_st16(t_s + q4 * 32, hi);
                        tmem_st16(t_s + q4 * 32 + 16, lo);
                        if (q4 & 1) done(q4 >> 1);
                    }
                    l += sum[0] + sum[1];
                } else if (edge || gaps) {
                    if (t > 0) poisoned(t - 1);
                    const float top = top_of(0, 4);
                    if (__any_sync(0xffffffffu, top > m + kSlack)) follow(top, 0);
                    const float ref = m == -INFINITY ? 0.f : kBase - m;
#pragma unroll 1
                    for (int q4 = 0; q4 < 4; ++q4) {
                        float v[32];
                        tmem_ld32(t_s + q4 * 32, v);
                        masked(q4, v);
                        uint32_t o[16];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            v[i] = ex2_approx(v[i] + ref);
                            const int e = sh.ev1[T & 3][q4 * 32 + i];
                            l = fmaf(v[i], pow2i(-e), l);
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = pack_f16(v[2 * i], v[2 * i + 1]);
                        tmem_st16(t_s + (q4 >> 1) * 64 + (q4 & 1) * 16, o);
                    }
                    done(0);
                    done(1);
                } else {
                    // One pass: the weights of 64 columns are computed for the reference as it is; only if one of them
                    // reaches 2^15 (in fp16: none is lost as long as it is below 2^16) is the maximum looked for, the
                    // reference moved and the half done again.  A row without a reference starts with the maximum.
                    if (__any_sync(0xffffffffu, m == -INFINITY)) {
                        const float top = top_of(0, 2);
                        if (__any_sync(0xffffffffu, top > m + kSlack)) follow(top, 0);
                    }
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        const float c = h ? cs[1] : cs[0], e = h ? ev[1] : ev[0];
                        uint32_t o[2][16];
                        float sum[2];
#pragma unroll 1
                        for (int turn = 0;; ++turn) {
                            const float off = e + (m == -INFINITY ? 0.f : kBase - m);
                            uint32_t hm = 0;
                            sum[0] = sum[1] = 0.f;
                            // 16 columns at a time, the next ones on their way
                            float v[2][16];
                            ld16_begin(t_s + h * 64, v[0]);
                            ld_wait(v[0]);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                float (&x)[16] = v[q & 1];
                                if (q < 3) ld16_begin(t_s + h * 64 + (q + 1) * 16, v[(q + 1) & 1]);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    ffma2(x[2 * i], x[2 * i + 1], c, off);
                                    x[2 * i] = ex2_approx(x[2 * i]);
                                    x[2 * i + 1] = ex2_approx(x[2 * i + 1]);
                                    uint32_t& w = o[q >> 1][(q & 1) * 8 + i];
                                    w = pack_f16(x[2 * i], x[2 * i + 1]);
                                    hm = max_f16x2(hm, w);
                                    fadd2(sum[0], sum[1], x[2 * i], x[2 * i + 1]);
                                }
                                if (q < 3) ld_wait(v[(q + 1) & 1]);
                            }
                            const bool over = (hm & 0x7fffu) >= 0x7800u || (hm >> 16) >= 0x7800u;
                            if (turn || !__any_sync(0xffffffffu, over)) break;
                            follow(top_of(2 * h, 2 * h + 2), h);
                        }
                        tmem_st16(t_s + h * 64, o[0]);
                        tmem_st16(t_s + h * 64 + 16, o[1]);
                        l = fmaf(sum[0] + sum[1], ex2_approx(-e), l);
                        done(h);
                    }
                }
            }

            // ---- output, or a share of a split unit
            constexpr int REC = chunk_rec_floats(D);
            const bool whole = a == 0 && bnd == tiles;
            const bool in = rt < ntile;
            ok = __all_sync(0xffffffffu, wait(&sh.o_done, segs & 1)) && ok;
            tc_fence_after();
            if (in && ok) poisoned(nt - 1);
            // 32 columns of this row: column 64 hh + 8 r + q of O is channel 64 hh + r + 32 (q % 2) + 8 (q / 2), held
            // times 2^-21, or 2^-17 where its code is odd (q / 2 odd)
            auto put = [&](int n, const float (&o)[32], float L) {
                if constexpr (!INT4) {                 // column n of O is channel n
                    const float il = L == 0.f ? 0.f : 1.f / L;
                    const size_t at = (size_t(row0 + row / G) * p.Hq + g * G + row % G) * D + n;
                    uint32_t nb = 0;
#pragma unroll
                    for (int w = 0; w < NW; ++w)
                        if (n == 32 * w) nb = nan[w];
#pragma unroll
                    for (int q = 0; q < 32; q += 4) {
                        auto val = [&](int k) { return (nb >> (q + k)) & 1u ? __uint_as_float(0x7fc00000u) : o[q + k] * il; };
                        const float4 y = make_float4(val(0), val(1), val(2), val(3));
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
                        *reinterpret_cast<uint2*>(p.out + at + q) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                        if (p.out_f32) *reinterpret_cast<float4*>(p.out_f32 + at + q) = y;
                    }
                    if (p.lse && n == 0)
                        p.lse[size_t(row0 + row / G) * p.Hq + g * G + row % G] =
                            L == 0.f ? -INFINITY : (m - kBase + log2f(L)) * kLn2;
                    return;
                }
                const float il = (L == 0.f ? 0.f : 1.f / L) * 2097152.f;
                const int hh = n >> 6, r8 = (n & 63) >> 3;             // four r from r8 on
                const size_t at = (size_t(row0 + row / G) * p.Hq + g * G + row % G) * D;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int ch = 64 * hh + r8 + 32 * (q & 1) + 8 * (q >> 1);
                    const bool bad = (nan[0] >> (ch / (D / 4))) & 1u;
                    const float f = bad ? __uint_as_float(0x7fc00000u) : (q >> 1) & 1 ? il * 0.0625f : il;
                    const float4 y = make_float4(o[q] * f, o[8 + q] * f, o[16 + q] * f, o[24 + q] * f);
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
                    *reinterpret_cast<uint2*>(p.out + at + ch) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                    if (p.out_f32) *reinterpret_cast<float4*>(p.out_f32 + at + ch) = y;
                }
                if (p.lse && n == 0)
                    p.lse[size_t(row0 + row / G) * p.Hq + g * G + row % G] =
                        L == 0.f ? -INFINITY : (m - kBase + log2f(L)) * kLn2;
            };
            float* const part = p.partials + size_t(2 * cta + (a == 0 ? 1 : 0)) * REC;
            if (in) {
#pragma unroll 1
                for (int n = 0; n < D; n += 32) {
                    float o[32];
                    tmem_ld32(t_o + n, o);
                    if (whole) {
                        if (have && ok) put(n, o, l);
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; c += 4)
                            reinterpret_cast<float4*>(part)[((n + c) / 4) * 256 + row] =
                                make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                    }
                }
                if (!whole) {
                    part[256 * D + row] = m;
                    part[256 * D + 256 + row] = l;
#pragma unroll
                    for (int w = 0; w < NW; ++w) part[256 * D + (2 + w) * 256 + row] = __uint_as_float(nan[w]);
                }
            }
            tc_fence_before();
            if (!whole) {
                const int lo = paged_tile_owner(u_lo + kSegC, TT, GC), hi = paged_tile_owner(u_hi - 1, TT, GC);
                __threadfence();
                asm volatile("bar.sync 1, 256;\n" ::: "memory");
                if (tid == 0) {
                    const int n = atomicAdd(p.arrived + lo, 1);
                    sh.last = n == hi - lo;
                    if (n == hi - lo) p.arrived[lo] = 0;
                }
                asm volatile("bar.sync 1, 256;\n" ::: "memory");
                if (sh.last && have) {
                    __threadfence();
                    const float* const b0 = p.partials + size_t(2 * lo + 1) * REC;
                    auto slot = [&](int k) { return k == 0 ? b0 : b0 + size_t(2 * k - 1) * REC; };
                    const int n = hi - lo + 1;
                    float M = -INFINITY, L = 0.f;
                    for (int k = 0; k < n; ++k) M = fmaxf(M, __ldcg(slot(k) + 256 * D + row));
                    for (int k = 0; k < n; ++k) {
                        const float mk = __ldcg(slot(k) + 256 * D + row);
                        L += (mk == -INFINITY ? 0.f : ex2_approx(mk - M)) * __ldcg(slot(k) + 256 * D + 256 + row);
                    }
                    m = M;
                    for (int k = 0; k < n; ++k)
#pragma unroll
                        for (int w = 0; w < NW; ++w) nan[w] |= __float_as_uint(__ldcg(slot(k) + 256 * D + (2 + w) * 256 + row));
#pragma unroll 1
                    for (int nn = 0; nn < D; nn += 32) {
                        float o[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0.f;
                        for (int k = 0; k < n; ++k) {
                            const float mk = __ldcg(slot(k) + 256 * D + row);
                            const float f = mk == -INFINITY ? 0.f : ex2_approx(mk - M);
#pragma unroll
                            for (int c = 0; c < 32; c += 4) {
                                const float4 v = __ldcg(reinterpret_cast<const float4*>(slot(k)) + ((nn + c) / 4) * 256 + row);
                                o[c] = fmaf(v.x, f, o[c]);
                                o[c + 1] = fmaf(v.y, f, o[c + 1]);
                                o[c + 2] = fmaf(v.z, f, o[c + 2]);
                                o[c + 3] = fmaf(v.w, f, o[c + 3]);
                            }
                        }
                        put(nn, o, L);
                    }
                }
                asm volatile("bar.sync 1, 256;\n" ::: "memory");
            }
        }
        ++segs;
        if (bad && tid == 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
        x = seg_end;
    }
    tc_fence_before();
    __syncthreads();
    if (sh.fail) {                                     // a wait gave up: what is in flight ends first, or has as long to
        auto drain = [&](uint64_t* bar, uint32_t par) {
            for (uint32_t it = 0; it < kSpin && !mbar_try_wait(bar, par); ++it) {
            }
        };
        if (warp == 8 + kUnpack && segs) drain(&sh.o_done, (segs - 1) & 1);
        if (INT4 && warp == 8 + kUnpack + 2) {
            const uint32_t n = min(sh.raw_end, raw_done);
            for (uint32_t S = n > 3 ? n - 3 : 0; S < n; ++S) drain(&sh.raw_full[S % 3], (S / 3) & 1);
        }
        __syncthreads();
    }
    if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace

size_t paged_chunk_scratch_bytes(int d) {
    const size_t grid = device_info().num_sms;         // two shares for each CTA
    return paged_counter_bytes() + align_up(2 * grid * chunk_rec_floats(d) * 4, 256);
}

spa_status launch_paged_chunk(const PagedAttendParams& args, cudaStream_t st) {
    PagedAttendParams p = args;
    p.stall = (test_stall_bits() & SPA_TEST_STALL_PAGED_CHUNK) != 0;
    p.spin = p.stall ? kStallSpin : kSpin;
    const int sms = device_info().num_sms;
    const int TQ = paged_tokens_per_tile(256, p.Hq / p.kv.Hkv);
    // the prefix of a launch's sequences lies in shared memory, in 32 bits: a sequence's query tiles times its
    // tiles bound its part
    const long long tiles = (((long long)p.kv.max_pages << p.kv.page_shift) + kKeys - 1) / kKeys + kSegC;
    const long long most = tiles * p.kv.Hkv * (((long long)p.T + TQ - 1) / TQ);
    long long step = kChunkUnits;
    if (most + tiles * p.kv.Hkv * step > 0xffffffffll) step = (0xffffffffll - most) / (tiles * p.kv.Hkv);
    if (step < 1) return SPA_ERR_UNSUPPORTED_SHAPE;
    for (int g0 = 0; g0 < p.kv.B; g0 += int(step)) {
        const int groups = p.kv.B - g0 < step ? p.kv.B - g0 : int(step);
#define SPA_PC(DD, I4)                                                                                          \
    if (p.kv.d == DD && (p.kv.int4 != 0) == I4) {                                                               \
        constexpr size_t kMost = sizeof(ChunkShared<DD, I4>) + size_t(kChunkUnits + 1) * 4;                      \
        static_assert(kMost <= 227 * 1024, "paged chunk: shared memory over the per-CTA limit");                 \
        SPA_CUDA_TRY(set_func_attr(reinterpret_cast<const void*>(paged_chunk_kernel<DD, I4>),                    \
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMost)));                   \
        SPA_CUDA_TRY(launch_pdl(paged_chunk_kernel<DD, I4>, dim3(sms), dim3(kThreads),                           \
                                sizeof(ChunkShared<DD, I4>) + size_t(groups + 1) * 4, st, p, g0, groups, TQ));    \
    }
        SPA_PC(64, false) SPA_PC(64, true) SPA_PC(128, false) SPA_PC(128, true)
#undef SPA_PC
    }
    return SPA_OK;
}

}  // namespace spa
