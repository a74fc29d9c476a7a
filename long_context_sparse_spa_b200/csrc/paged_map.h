// Index arithmetic of the paged KV cache, shared by its kernels and by a CPU test that checks every
// access against its buffer: no CUDA type or builtin here.  Everything that a kernel reads from
// device memory (page numbers, lengths, sequence starts) may hold any bits; each function answers
// with an index inside its buffer or with -1.
#pragma once
#include <cstdint>

#if defined(__CUDACC__)
#define SPA_HD __host__ __device__ __forceinline__
#else
#define SPA_HD inline
#endif

namespace spa {

struct PagedView {
    uint8_t* data;              // [num_pages][Hkv][page][row_bytes]
    const int32_t* page_table;  // [B][max_pages]
    const int32_t* kv_len;      // [B]
    int num_pages, Hkv, page_shift, d;
    int B, max_pages;
    int int4;                   // 4-bit rows, else bf16
    int row_bytes;
};

// bytes of one token of one kv head: d/2 + d/2 bytes of codes and 2 x 4 bf16 scales, or 2 x d bf16
SPA_HD int paged_row_bytes(bool int4, int d) { return int4 ? d + 16 : 4 * d; }

// tokens of a sequence that its page table can hold; a length outside [0, that] is an error and is clamped
SPA_HD int paged_len(const PagedView& v, int len, bool* bad) {
    const long long cap = (long long)v.max_pages << v.page_shift;
    if (len < 0) { *bad = true; return 0; }
    if (len > cap) { *bad = true; return int(cap); }
    return len;
}

// index into page_table of token n of sequence b, or -1
SPA_HD long long paged_slot(const PagedView& v, int b, long long n) {
    if (b < 0 || b >= v.B || n < 0 || (n >> v.page_shift) >= v.max_pages) return -1;
    return (long long)b * v.max_pages + (n >> v.page_shift);
}

// byte offset in data of token n (of any sequence) on page `pid` for kv head g, or -1 for a bad page number
SPA_HD long long paged_row(const PagedView& v, int pid, int g, long long n) {
    if (pid < 0 || pid >= v.num_pages) return -1;
    const long long in_page = n & ((1ll << v.page_shift) - 1);
    return ((((long long)pid * v.Hkv + g) << v.page_shift) + in_page) * v.row_bytes;
}

// whether [a, e), a sequence's start and the next one's, are rows of T; where not, the sequence has no new tokens
SPA_HD bool paged_rows_ok(long long a, long long e, int T) { return a >= 0 && a <= e && e <= T; }

// sequence whose rows [seq_start[b], seq_start[b + 1]) hold token t, or -1 (rows before the first or
// behind the last sequence); seq_start null: one token per sequence
SPA_HD int paged_seq_of(const int32_t* seq_start, int B, int t) {
    if (!seq_start) return t < B ? t : -1;
    int lo = 0, hi = B;   // the last b with seq_start[b] <= t, if any
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq_start[mid] <= t) lo = mid; else hi = mid;
    }
    return seq_start[lo] <= t && t < seq_start[lo + 1] ? lo : -1;
}

// ------------------------------------------------------------------ 4-bit rows
// A row of d values has 4 groups of d/4 consecutive channels with one bf16 scale each; the value of a
// code c is scale * (c - 8).  Codes are laid out as the attention's mma fragments read them:
//   keys    lane t of a quad (t = 0..3) holds d/16 consecutive channels of every group:
//           group g, t, e: byte t * d/8 + g * d/32 + e / 2, nibble e % 2
//   values  fragment row r (r = 0..7) holds channels 16 i + r (low nibble) and 16 i + r + 8 (high):
//           byte r * d/16 + g * d/64 + i
SPA_HD int int4_key_nibble(int d, int ch) {
    const int g = ch / (d / 4), j = ch % (d / 4), t = j / (d / 16), e = j % (d / 16);
    return 2 * (t * (d / 8) + g * (d / 32) + e / 2) + e % 2;
}
SPA_HD int int4_value_nibble(int d, int ch) {
    const int g = ch / (d / 4), j = ch % (d / 4);
    return 2 * ((j % 8) * (d / 16) + g * (d / 64) + j / 16) + (j % 16) / 8;
}

// ------------------------------------------------------------------ work split of the attention
// Owner, of G CTAs, of (weighted) tile x when TT tiles are split as [TT*c/G, TT*(c+1)/G).
SPA_HD int paged_tile_owner(long long x, long long TT, int G) { return int(((x + 1) * G - 1) / TT); }

// Query tokens per query tile when a tile holds up to `rows` (query, head) rows of G heads each.
SPA_HD int paged_tokens_per_tile(int rows, int G) { return rows / G > 0 ? rows / G : 1; }

// Keys that the last query of query tile j (TQ tokens each) of n queries may see, in a sequence of len tokens.
SPA_HD int paged_tile_limit(int len, int n, int TQ, int j) {
    long long last = (long long)(j + 1) * TQ;
    if (last > n) last = n;
    const long long lim = (long long)len - n + last;
    return lim < 0 ? 0 : int(lim);
}

}  // namespace spa
