// Paged KV cache: appending new keys and values with the position rotation on the way, in bf16 or
// quantised to 4 bits, and reading rows back as dense bf16.  The method pages have no counterpart;
// the cache feeds the same attention and selection as the dense [B, Hkv, N, d] one.
//
// Append, per new token t of sequence b at position n (its slot in the cache):
//   the rotation turns channel pairs (x, y) of q and k by the angle a_i = pos * inv_freq[i]:
//     x' = x cos a_i - y sin a_i,  y' = y cos a_i + x sin a_i;
//   a bf16 cache takes k' and v rounded once; a 4-bit cache takes, per group of d/4 channels,
//     s = amax / 7 rounded up to bf16,  code = rint(x / s) + 8, x / s in [-7, 7].
//   Rounding the scale up keeps every quotient within [-7, 7], so no code clamps and the error of a
//   value is at most s/2.  Codes are taken from the rotated keys in fp32, not from their bf16 rounding.
//   A group that holds a NaN or an infinity gets the scale NaN: it reads back as NaN, never as a number.
// Angles and their sine and cosine are computed in fp64 (a position of 10^6 leaves fp32 only 0.06 rad),
// the rotation itself in fp32 without contraction.
//
// Each row of d channels is held by d/8 lanes, 8 channels (16 bytes) each; pair partners and group
// maxima are exchanged by shuffles, so a row is read once.
//
// Measured on B200: append of 4096 tokens (32 query, 8 kv heads, d = 128) in 4 bits about 34 us and 8 us for reading
// them back, 88 + 22 MB; the append uses 75 % of the issue slots (rotation and quantisation of 16-byte pieces).  Gather
// of 28672 4-bit tokens of 8 heads to bf16 (150 MB) 29.4 us, 5.1 TB/s: its warps wait for shared memory, through which
// the rows go in and out, twice as long as for DRAM.  Gather of 42 MB of bf16 rows 11.1 us, 3.8 TB/s (6.8 us where they
// lie in L2): it waits for its loads, four of 16 bytes to a lane.
#include <climits>

#include "paged.cuh"

namespace spa {
namespace {

constexpr int kThreads = 256;
constexpr int kAppTok = 8;   // most tokens per CTA
constexpr int kAppCtas = 6;  // CTAs per SM
// Passes whose loads are in flight besides the current one.  More of them cost registers, and so resident CTAs:
// 1 with 6 CTAs per SM, 2 with 4 and 3 with 4 took 39.7, 39.2 and 41.4 us for 4096 tokens in 4 bits (with the
// read-back) and 11.5, 12.5 and 12.4 us for seven bf16 prompts.
constexpr int kAppAhead = 1;

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ float f4(const float4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// sin and cos of an angle of up to about 2^31 in fp64: the nearest multiple of pi/2 is taken off in two parts
// with fused multiply-adds (Cody and Waite, "Software Manual for the Elementary Functions", 1980), so the
// functions see |r| <= pi/4 whatever the position is.
__device__ __forceinline__ void angle_sincos(double a, double* sn, double* cs) {
    const double k = rint(a * 0.63661977236758134);
    const double r = fma(-k, 6.123233995736766e-17, fma(-k, 1.5707963267948966, a));
    double s, c;
    sincos(r, &s, &c);
    const int q = int((long long)k & 3);
    const double x = q & 1 ? c : s, y = q & 1 ? s : c;
    *sn = q & 2 ? -x : x;
    *cs = (q + 1) & 2 ? -y : y;
}

// ------------------------------------------------------------------ append
template <int D, bool INT4>
__global__ void __launch_bounds__(kThreads, kAppCtas) paged_append_kernel(PagedAppendParams p, int tok_per_cta) {
    constexpr int LPR = D / 8;              // lanes per row
    constexpr int RPP = kThreads / LPR;     // rows per pass
    constexpr int GL = LPR / 4;             // lanes per quantisation group
    __shared__ __align__(16) float s_cos[kAppTok][64], s_sin[kAppTok][64];
    __shared__ long long s_row[kAppTok];    // byte offset of the token's row of kv head 0, or -1
    __shared__ int s_pos[kAppTok];
    __shared__ __align__(16) uint8_t s_val[INT4 ? RPP : 1][INT4 ? D / 2 : 16];
    pdl_enter();
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * tok_per_cta;
    const int nt = min(tok_per_cta, p.T - t0);
    const int Hkv = p.kv.Hkv, Hq = p.q ? p.Hq : 0;
    const int rows = Hq + 2 * Hkv;          // rows of a token: queries, keys, values
    const int c = tid % LPR;                // this lane's 8 channels: [8c, 8c + 8)
    const int total = nt * rows;
    const long long head_bytes = (long long)p.kv.row_bytes << p.kv.page_shift;
    // A cursor over the CTA's rows, RPP at a time: token t, row r of the token.
    struct Cursor { int t, r; };
    auto step = [&](Cursor& u) {
        u.r += RPP;
        while (u.r >= rows) { u.r -= rows; ++u.t; }
    };
    auto fetch = [&](const Cursor& u) -> uint4 {
        if (u.t >= nt) return make_uint4(0, 0, 0, 0);
        const int kv = u.r - Hq;
        const uint16_t* src = kv < 0     ? p.q + (t0 + u.t) * p.q_tok + u.r * p.q_head
                              : kv < Hkv ? p.k + (t0 + u.t) * p.k_tok + kv * p.k_head
                                         : p.v + (t0 + u.t) * p.v_tok + (kv - Hkv) * p.v_head;
        return __ldg(reinterpret_cast<const uint4*>(src) + c);
    };
    Cursor now{0, tid / LPR}, next;
    while (now.r >= rows) { now.r -= rows; ++now.t; }
    next = now;
    // the rows of the next passes are always on their way, the first ones before the token is looked up
    uint4 ahead[kAppAhead];
#pragma unroll
    for (int i = 0; i < kAppAhead; ++i) {
        ahead[i] = fetch(next);
        step(next);
    }
    // starts out of order are reported once (by the warps, if there are any, that look up no token)
    if (p.seq_start && blockIdx.x == 0)
        for (int k = kThreads - 1 - tid; k < p.kv.B; k += kThreads)
            if (!paged_rows_ok(p.seq_start[k], p.seq_start[k + 1], p.T)) raise_status(p.status, SPA_ERR_INVALID_ARG);
    if (tid < 32 * nt) {                    // a warp per token
        const int lane = tid & 31, i = tid >> 5, t = t0 + i;
        int b = -1;
        if (!p.seq_start || p.kv.B > 1024) {
            b = paged_seq_of(p.seq_start, p.kv.B, t);
            if (b >= 0 && p.seq_start && !paged_rows_ok(p.seq_start[b], p.seq_start[b + 1], p.T)) b = -1;
        }
        if (b < 0 && p.seq_start) {
            // the first sequence that the attention too takes the row for (the loads do not wait for one another; many
            // starts only where they are out of order, or for a row of nobody)
            int first = INT_MAX;
            for (int k = lane; k < p.kv.B; k += 32) {
                const int a = p.seq_start[k], e = p.seq_start[k + 1];
                if (a <= t && t < e && paged_rows_ok(a, e, p.T)) first = min(first, k);
            }
            first = __reduce_min_sync(0xffffffffu, first);
            if (first < INT_MAX) b = first;
        }
        if (lane == 0) {
            long long row = -1;
            int rope = 0;
            if (b >= 0) {
                // slot of the token: the last of the sequence's new tokens is token kv_len[b] - 1
                const long long left = p.seq_start ? (long long)p.seq_start[b + 1] - t : 1;
                const long long n = (long long)p.kv.kv_len[b] - left;
                const long long slot = paged_slot(p.kv, b, n);
                if (slot >= 0) row = paged_row(p.kv, p.kv.page_table[slot], 0, n);
                if (row < 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
                rope = p.positions ? p.positions[t] : int(n);
            }
            s_row[i] = row;
            s_pos[i] = rope;
        }
    }
    __syncthreads();
    const int half = p.rot / 2;
    for (int i = tid; i < nt * half; i += kThreads) {
        const int t = i / half, f = i - t * half;
        if (s_row[t] < 0) continue;
        double sn, cs;
        angle_sincos(double(s_pos[t]) * double(p.inv_freq[f]), &sn, &cs);
        s_cos[t][f] = float(cs);
        s_sin[t][f] = float(sn);
    }
    __syncthreads();

    const int hc = p.rot / 16;              // lanes per half of the rotated channels
    const bool turn = p.interleaved ? 8 * c < p.rot : c < 2 * hc;
    const int mate = !turn ? c : c < hc ? c + hc : c - hc;        // the lane with the pair partners
    const int f0 = p.interleaved ? 4 * c : (c < hc ? c : c - hc) * 8;
    for (int base = 0; base < total; base += kAppAhead * RPP) {   // same trip count for every lane: shuffles below
#pragma unroll
        for (int pass = 0; pass < kAppAhead; ++pass) {
            if (base + pass * RPP >= total) break;                // (uniform)
            const uint4 w = ahead[pass];
            ahead[pass] = fetch(next);
            step(next);
            const int t = min(now.t, nt - 1), kv = now.r - Hq;
            const int kind = kv < 0 ? 0 : kv < Hkv ? 1 : 2, h = kv < 0 ? now.r : kv < Hkv ? kv : kv - Hkv;
            const bool live = now.t < nt && s_row[t] >= 0;
            step(now);
            float x[8] = {bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y), bf_lo(w.z), bf_hi(w.z), bf_lo(w.w), bf_hi(w.w)};
            if (p.rot > 0 && __any_sync(0xffffffffu, kind < 2)) {
                if (p.interleaved) {
                    if (kind < 2 && turn) {
                        const float4 cs = *reinterpret_cast<const float4*>(&s_cos[t][f0]);
                        const float4 sn = *reinterpret_cast<const float4*>(&s_sin[t][f0]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float a = x[2 * j], b = x[2 * j + 1];
                            x[2 * j] = __fsub_rn(__fmul_rn(a, f4(cs, j)), __fmul_rn(b, f4(sn, j)));
                            x[2 * j + 1] = __fadd_rn(__fmul_rn(b, f4(cs, j)), __fmul_rn(a, f4(sn, j)));
                        }
                    }
                } else {
                    const int src = (tid & 31) - c + mate;
                    const uint32_t flip = c < hc ? 0x80008000u : 0u;   // x cos - y sin, or x cos + y sin
                    uint4 o;
                    o.x = __shfl_sync(0xffffffffu, w.x, src) ^ flip;
                    o.y = __shfl_sync(0xffffffffu, w.y, src) ^ flip;
                    o.z = __shfl_sync(0xffffffffu, w.z, src) ^ flip;
                    o.w = __shfl_sync(0xffffffffu, w.w, src) ^ flip;
                    if (kind < 2 && turn) {
                        const float y[8] = {bf_lo(o.x), bf_hi(o.x), bf_lo(o.y), bf_hi(o.y),
                                            bf_lo(o.z), bf_hi(o.z), bf_lo(o.w), bf_hi(o.w)};
#pragma unroll
                        for (int j4 = 0; j4 < 8; j4 += 4) {
                            const float4 cs = *reinterpret_cast<const float4*>(&s_cos[t][f0 + j4]);
                            const float4 sn = *reinterpret_cast<const float4*>(&s_sin[t][f0 + j4]);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                x[j4 + j] = __fadd_rn(__fmul_rn(x[j4 + j], f4(cs, j)), __fmul_rn(y[j4 + j], f4(sn, j)));
                        }
                    }
                }
            }
            if ((kind == 0 || !INT4) && live) {
                const uint4 o = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                           pack_bf16(x[6], x[7]));
                uint8_t* dst = kind == 0 ? reinterpret_cast<uint8_t*>(p.q_out + (size_t(t0 + t) * p.Hq + h) * D)
                                         : p.kv.data + s_row[t] + h * head_bytes + (kind == 2 ? 2 * D : 0);
                reinterpret_cast<uint4*>(dst)[c] = o;
            }
            if (INT4 && __any_sync(0xffffffffu, kind > 0)) {
                // group maximum; an element that is not finite (its magnitude's bits are the largest) poisons the group
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
#pragma unroll
                for (int off = 1; off < GL; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
                // up to bf16: the scale must not be below amax / 7, so that no code clamps
                const bool fin = top < 0x7f800000u;
                const uint32_t sb =
                    fin ? (__float_as_uint(__fdiv_rn(__uint_as_float(top), 7.f)) + 0xffffu) & 0xffff0000u : 0x7fc00000u;
                const float s = __uint_as_float(sb);
                // rint(x / s) + 8 in the low bits of y + (1.5 * 2^23 + 8), y = x * (1 / s): y is off by less than
                // 2^-20, so only where it is that near to a border is the quotient itself needed
                const float rs = __frcp_rn(s);
                uint32_t nib = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float y = x[j] * rs;
                    float z = __fadd_rn(y, 12582920.f);
                    if (!(fabsf(__fsub_rn(y, __fsub_rn(z, 12582920.f))) < 0.49999f))
                        z = __fadd_rn(fin && s > 0.f ? __fdiv_rn(x[j], s) : 0.f, 12582920.f);
                    nib |= (__float_as_uint(z) & 15u) << (4 * j);
                }
                uint8_t* dst = p.kv.data + (live ? s_row[t] + h * head_bytes : 0);
                const int g = c / GL;
                if (live && kind > 0 && c % GL == 0)
                    reinterpret_cast<uint16_t*>(dst + D)[(kind == 2 ? 4 : 0) + g] = uint16_t(sb >> 16);
                if (kind == 1 && live) {
                    if constexpr (D == 128) {   // a lane's 8 channels are one lane-of-a-quad's share of its group
                        *reinterpret_cast<uint32_t*>(dst + (c % 4) * 16 + g * 4) = nib;
                    } else {
                        *reinterpret_cast<uint16_t*>(dst + (c % 2) * 16 + g * 2) = uint16_t(nib);
                        *reinterpret_cast<uint16_t*>(dst + (c % 2) * 16 + 8 + g * 2) = uint16_t(nib >> 16);
                    }
                }
                if (__any_sync(0xffffffffu, kind == 2)) {
                    // channels 16 i + r and 16 i + r + 8 share byte r * D/16 + (c / 2): an even lane joins its
                    // neighbour's codes to its own; the bytes go through shared memory and out in 16-byte stores
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, nib, 1);
                    const uint32_t even = (nib & 0x0f0f0f0fu) | (other & 0x0f0f0f0fu) << 4;      // r = 0, 2, 4, 6
                    const uint32_t odd = ((nib >> 4) & 0x0f0f0f0fu) | (other & 0xf0f0f0f0u);     // r = 1, 3, 5, 7
                    uint8_t* sv = s_val[tid / LPR];
                    if (c % 2 == 0) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            sv[2 * r * (D / 16) + c / 2] = uint8_t(even >> (8 * r));
                            sv[(2 * r + 1) * (D / 16) + c / 2] = uint8_t(odd >> (8 * r));
                        }
                    }
                    __syncwarp();
                    if (kind == 2 && live && c < D / 32)
                        *reinterpret_cast<uint4*>(dst + D / 2 + 16 * c) = *reinterpret_cast<const uint4*>(sv + 16 * c);
                    __syncwarp();
                }
            }
        }
    }
}

// ------------------------------------------------------------------ gather
// One warp per 16 tokens of one (sequence, kv head), without block barriers: the lanes look up the rows,
// keep 5 (d = 128) 16-byte loads each in flight into the warp's shared memory, and write dense rows.
constexpr int kGatTok = 16, kGatWarps = 4;

template <int D, bool INT4>
__global__ void __launch_bounds__(kGatWarps * 32) paged_gather_kernel(PagedGatherParams p) {
    constexpr int ROWB = INT4 ? D + 16 : 4 * D;
    constexpr int LPR = D / 8;
    // the unpacked rows go out by way of shared memory too, so that a warp's stores are whole rows
    constexpr int OROW = 2 * D + 16;
    __shared__ __align__(16) uint8_t s_in[INT4 ? kGatWarps : 1][INT4 ? kGatTok * ROWB : 16];
    __shared__ __align__(16) uint8_t s_out[INT4 ? kGatWarps : 1][INT4 ? kGatTok * OROW : 16];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = blockIdx.y, b = blockIdx.z;
    const long long i0 = ((long long)blockIdx.x * kGatWarps + warp) * kGatTok;
    if (i0 >= p.N) return;
    bool bad = false;
    const int len = paged_len(p.kv, p.kv.kv_len[b], &bad);
    const long long first = p.start ? p.start[b] : 0;
    long long row = -1;                     // of token i0 + lane (lanes 0-15)
    {
        const long long i = i0 + lane, n = first + i;
        if (lane < kGatTok && i < p.N && n >= 0 && n < len) {
            row = paged_row(p.kv, p.kv.page_table[paged_slot(p.kv, b, n)], g, n);
            bad |= row < 0;
        }
        if (bad || first < 0) raise_status(p.status, SPA_ERR_INVALID_ARG);
    }
    uint16_t* const outs[2] = {p.K, p.V};
    const size_t out0 = (size_t(b) * p.kv.Hkv + g) * p.N + i0;
    if constexpr (INT4) {
        constexpr int CH = ROWB / 16, NL = (kGatTok * CH + 31) / 32;
        uint4 w[NL];
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int i = lane + 32 * j, t = min(i / CH, kGatTok - 1), ch = i - t * CH;
            const long long r = __shfl_sync(0xffffffffu, row, t);
            w[j] = make_uint4(0, 0, 0, 0);
            if (i < kGatTok * CH && r >= 0) w[j] = __ldg(reinterpret_cast<const uint4*>(p.kv.data + r) + ch);
        }
#pragma unroll
        for (int j = 0; j < NL; ++j)
            if (lane + 32 * j < kGatTok * CH) reinterpret_cast<uint4*>(s_in[warp])[lane + 32 * j] = w[j];
        __syncwarp();
        // A lane takes one group (d/4 channels) of a token's key and value.  A code u in the low bits of bf16 128 is
        // 128 + u; minus 136 it is u - 8, both exact, and the product with the scale is rounded once.
        auto value2 = [](uint32_t nib2, uint32_t s2) -> uint32_t {   // two codes in bits 0-3 and 16-19
            uint32_t r;
            asm("{\n .reg .b32 t;\n sub.rn.bf16x2 t, %1, %2;\n mul.rn.bf16x2 %0, t, %3;\n}\n"
                : "=r"(r)
                : "r"((nib2 & 0x000f000fu) | 0x43004300u), "r"(0x43084308u), "r"(s2));
            return r;
        };
        const int gr = lane & 3;
#pragma unroll
        for (int isv = 0; isv < 2; ++isv) {
#pragma unroll
            for (int t0 = 0; t0 < kGatTok; t0 += 8) {
                const int t = t0 + (lane >> 2);
                const uint8_t* src = s_in[warp] + t * ROWB;
                const uint32_t sc = reinterpret_cast<const uint16_t*>(src + D)[isv * 4 + gr], s2 = sc | sc << 16;
                uint32_t o[D / 8];                     // the group's channel pairs
                if (!isv) {
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) { // eight codes: channels 8 q .. 8 q + 7
                        const uint32_t w =
                            D == 128 ? *reinterpret_cast<const uint32_t*>(src + q * 16 + gr * 4)
                                     : *reinterpret_cast<const uint16_t*>(src + q * 16 + gr * 2) |
                                           uint32_t(*reinterpret_cast<const uint16_t*>(src + q * 16 + 8 + gr * 2)) << 16;
                        uint32_t v[4];                 // codes k and k + 4
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = value2(w >> (4 * k), s2);
                        o[4 * q] = __byte_perm(v[0], v[1], 0x5410);
                        o[4 * q + 1] = __byte_perm(v[2], v[3], 0x5410);
                        o[4 * q + 2] = __byte_perm(v[0], v[1], 0x7632);
                        o[4 * q + 3] = __byte_perm(v[2], v[3], 0x7632);
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {      // channels 2 r, 2 r + 1 of every eight
                        const uint8_t* b0 = src + D / 2 + 2 * r * (D / 16) + gr * (D / 64);
                        const uint32_t x = D == 128 ? *reinterpret_cast<const uint16_t*>(b0) : *b0;
                        const uint32_t y = D == 128 ? *reinterpret_cast<const uint16_t*>(b0 + D / 16) : *(b0 + D / 16);
                        const uint32_t w = x | y << 16;
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) o[4 * k + r] = value2(w >> (4 * k), s2);
                    }
                }
#pragma unroll
                for (int q = 0; q < D / 32; ++q)
                    *reinterpret_cast<uint4*>(s_out[warp] + t * OROW + gr * (D / 2) + 16 * q) =
                        make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kGatTok * LPR / 32; ++j) {
                const int i = lane + 32 * j, t = i / LPR, c = i - t * LPR;
                const bool live = __shfl_sync(0xffffffffu, int(row >= 0), t);
                const uint4 v = *reinterpret_cast<const uint4*>(s_out[warp] + t * OROW + 16 * c);
                if (live) reinterpret_cast<uint4*>(outs[isv] + (out0 + t) * D)[c] = v;
            }
            __syncwarp();
        }
    } else {
        constexpr int CH = 2 * LPR, NL = kGatTok * CH / 32;    // pieces of a row, loads per lane
#pragma unroll
        for (int j0 = 0; j0 < NL; j0 += 4) {
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = lane + 32 * (j0 + j), t = i / CH, r = i - t * CH;
                const long long at = __shfl_sync(0xffffffffu, row, t);
                if (at >= 0) w[j] = __ldg(reinterpret_cast<const uint4*>(p.kv.data + at) + r);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = lane + 32 * (j0 + j), t = i / CH, r = i - t * CH, isv = r / LPR;
                const long long at = __shfl_sync(0xffffffffu, row, t);
                if (at >= 0) reinterpret_cast<uint4*>(outs[isv] + (out0 + t) * D)[r - isv * LPR] = w[j];
            }
        }
    }
}

}  // namespace

spa_status launch_paged_append(const PagedAppendParams& p, cudaStream_t st) {
    // tokens per CTA: as few as give one wave of resident CTAs (a decode step has one token per sequence)
    const int wave = device_info().num_sms * kAppCtas, want = (p.T + wave - 1) / wave;
    const int tok = want < 1 ? 1 : want > kAppTok ? kAppTok : want;
    const dim3 grid((p.T + tok - 1) / tok);
#define SPA_APP(DD, I4)                                                                                   \
    if (p.kv.d == DD && (p.kv.int4 != 0) == I4)                                                           \
        SPA_CUDA_TRY(launch_pdl(paged_append_kernel<DD, I4>, grid, dim3(kThreads), 0, st, p, tok));
    SPA_APP(64, false) SPA_APP(64, true) SPA_APP(128, false) SPA_APP(128, true)
#undef SPA_APP
    return SPA_OK;
}

spa_status launch_paged_gather(const PagedGatherParams& p, cudaStream_t st) {
    constexpr int kPer = kGatTok * kGatWarps;
    const dim3 grid((p.N + kPer - 1) / kPer, p.kv.Hkv, p.kv.B);
#define SPA_GAT(DD, I4)                                                                       \
    if (p.kv.d == DD && (p.kv.int4 != 0) == I4)                                               \
        SPA_CUDA_TRY(launch_pdl(paged_gather_kernel<DD, I4>, grid, dim3(kGatWarps * 32), 0, st, p));
    SPA_GAT(64, false) SPA_GAT(64, true) SPA_GAT(128, false) SPA_GAT(128, true)
#undef SPA_GAT
    return SPA_OK;
}

}  // namespace spa
