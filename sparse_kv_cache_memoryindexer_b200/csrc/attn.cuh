// Attention over a paged cache with a sliding window and first tokens that stay visible, and the same
// together with a query's Top-k entries (hyper.ai summary, "Method": the chosen entries are concatenated
// with the sliding window's for core attention).
//
// Query token i of sequence b stands at p = cache_len[b] + i and sees key j < cache_len[b] + n_b iff
//     j <= p and (window = 0 or j > p - window or j < n_sink).
// Head hq reads key/value head hq / (Hq / H).  o = sum_j softmax_j(scale q . k_j) v_j, and
// lse = log sum_j exp(scale q . k_j); a query that sees nothing gets o = 0, lse = -inf.
// An E4M3 page and head carries one scale for its keys and one for its values: the former multiplies
// the score, the latter the probability.
//
// This file: the arguments, and what the kernels share.
#pragma once
#include "kv_append.cuh"

namespace lsa {

struct AttnArgs {
    const void *q;             // [N][Hq][D], q_stride elements from one token to the next
    int64_t q_stride;
    const int64_t *q_offsets;  // [B + 1]
    const int32_t *cache_len;  // [B] tokens before this call's
    const int32_t *page_table; // [B][max_pages]
    const void *k_cache, *v_cache;  // [n_pages][H][page][D]
    const float *k_scale, *v_scale; // [n_pages][H], E4M3 only
    void *out;                 // [N][Hq][D]
    float *lse;                // [N][Hq] or null
    int64_t N, n_pages;
    int B, max_pages, Hq, H, D, page, window, n_sink;
    float scale;
    // the Top-k entries of each query token (k = 0: none)
    const int32_t *topk_idx;   // [N][k]
    const int32_t *idx, *count;
    const int64_t *seq_offsets;
    const uint8_t *hot_kv, *win_kv;  // rows of row_bytes: [2][H][D], keys then values
    int64_t total_S, row_bytes;
    int k, W;
};

// The keys a query position sees, in the order [first tokens][window]: key number t is position t for
// t < sinks, else lo + (t - sinks).
struct Span {
    int64_t lo;   // first position of the window
    int64_t sinks;
    int64_t total;
};

__host__ __device__ __forceinline__ Span visible_span(int64_t p, int window, int n_sink)
{
    Span s;
    s.lo = (window > 0 && p + 1 > window) ? p + 1 - window : 0;
    s.sinks = s.lo < n_sink ? s.lo : n_sink;
    s.total = s.sinks + (p + 1 - s.lo);
    return s;
}

// A page scale must be finite, >= 0; a value scale's reciprocal and its product with a long sum are formed
// in fp32, so one that is not zero lies in [2^-100, 2^120].
__device__ __forceinline__ bool good_scale(float s) { return s == 0.f || (s >= 7.8886090522101181e-31f && s <= 1.329227995784916e36f); }

// Row of entry e of sequence b (null: flagged).
__device__ __forceinline__ const uint8_t *entry_row(const AttnArgs &A, int b, int32_t e)
{
    const int64_t off = __ldg(A.seq_offsets + b), S = __ldg(A.seq_offsets + b + 1) - off;
    if (off < 0 || S < 0 || off + S > A.total_S) {
        flag(ERRF_OFFSETS);
        return nullptr;
    }
    if (e >= S) {
        if (e - S < A.W) return A.win_kv + ((int64_t)b * A.W + (e - S)) * A.row_bytes;
        flag(ERRF_INDEX);
        return nullptr;
    }
    const int32_t cnt = __ldg(A.count + b);
    if (cnt < 0 || cnt > S) {
        flag(ERRF_COUNT);
        return nullptr;
    }
    int64_t lo = 0, hi = cnt;  // first slot whose entry is >= e
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (__ldg(A.idx + off + mid) < e) lo = mid + 1;
        else hi = mid;
    }
    if (lo < cnt && __ldg(A.idx + off + lo) == e) return A.hot_kv + (off + lo) * A.row_bytes;
    flag(ERRF_INDEX);
    return nullptr;
}

}  // namespace lsa
