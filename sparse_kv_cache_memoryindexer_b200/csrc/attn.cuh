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
#include <atomic>

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
    int B, max_pages, Hq, H, D, page, page_shift, window, n_sink;
    float scale;
    // the Top-k entries of each query token (k = 0: none)
    const int32_t *topk_idx;   // [N][k]
    const int32_t *idx, *count;
    const int64_t *seq_offsets;
    const uint8_t *hot_kv, *win_kv;  // rows of row_bytes: [2][H][D], keys then values
    int64_t total_S, row_bytes;
    int k, W;
};

// Raises a kernel's limit of dynamic shared memory, once per device (the attribute stays): done holds a bit for each
// of the first 64 devices.
template <typename K>
inline cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

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

// A page scale: zero, or in [2^-100, 2^120] (finite with room for a code's 448).
__device__ __forceinline__ bool good_scale(float s) { return s == 0.f || (s >= 7.8886090522101181e-31f && s <= 1.329227995784916e36f); }

// Value scales that the kernels' one reference serves.  A key's weight in the value product is p vs, in the softmax sum p;
// the kernels hold p' = 2^(s + log2 vs - m'), m' the running maximum of s + log2 vs, and add p' / vs to the sum.  With
// scales in [2^-64, 2^40] a key that counts in the sum has a p' above fp32's least normal (104 binades apart, and the
// factor 2^15 or 2^7 of p' leaves it 37 or 29 more), and 2^31 of the largest p' / vs (2^79) stay below 2^128.  What lies
// outside is rare, and rows that it touches are done again by attend_row, which keeps the two maxima apart:
//   - a scale outside (values beyond 2^48 or whose largest is below 2^-55): every row of the tile that met it;
//   - a scale of zero counts as 2^-64 in the sum and as nothing in the value product, which is right unless its keys set m'
//     (then the others' p' may have vanished).  Such a key's p' / vs is 2^64 times the factor of p', so only rows whose sum
//     comes to that are concerned (from_zero), in a tile that met a scale of zero.
// Both are looked at where a page's scale is read and at a tile's end, not for every key: a running maximum of the
// zero-scale keys in the loops cost 6 %.
__device__ __forceinline__ bool usual_value_scale(float s) { return s >= 5.421010862427522e-20f && s <= 1.099511627776e12f; }
constexpr float ZERO_LV = -64.f, ZERO_INV = 18446744073709551616.f;  // log2 and reciprocal that a scale of zero counts with
constexpr uint32_t MET_ZERO = 1u, MET_ODD = 2u;                      // what a tile's pages held

__device__ __forceinline__ uint32_t met_of(float s) { return s == 0.f ? MET_ZERO : (good_scale(s) ? MET_ODD : 0u); }

// The sum l of a row (or of a part) whose tile met `met`, as it is handed on: NaN for an odd scale; negative where the
// maximum may be that of a key with a scale of zero (factor: of p').
__device__ __forceinline__ float marked_sum(float l, uint32_t met, float factor)
{
    if (met & MET_ODD) return NAN;
    return (met & MET_ZERO) && l >= 0.5f * ZERO_INV * factor ? -l : l;
}

// Key and value rows of one cached token of head h, with their page's scales (false: the page is bad, flagged).
template <int CT>
__device__ __forceinline__ bool cached_rows(const AttnArgs &A, int b, int h, int64_t pos, const uint8_t *&k,
                                            const uint8_t *&v, float &ks, float &vs)
{
    const int32_t page = page_of(A.page_table, A.max_pages, A.n_pages, b, pos / A.page);
    if (page < 0) return false;
    const int64_t ph = (int64_t)page * A.H + h;
    const int64_t e = (ph * A.page + pos % A.page) * A.D;
    constexpr int bytes = CT == DT_F32 ? 4 : (CT == DT_BF16 ? 2 : 1);
    k = (const uint8_t *)A.k_cache + e * bytes;
    v = (const uint8_t *)A.v_cache + e * bytes;
    ks = vs = 1.f;
    if constexpr (CT == DT_FP8) {
        ks = __ldg(A.k_scale + ph);
        vs = __ldg(A.v_scale + ph);
        if (!good_scale(ks) || !good_scale(vs)) {
            flag(ERRF_SCALE);
            return false;
        }
    }
    return true;
}

constexpr int ATTN_MAX_D = 128;

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// Key and value rows of Top-k entry e of sequence b, head h (false: none, flagged where the entry is nowhere).
template <int CT>
__device__ __forceinline__ bool listed_rows(const AttnArgs &A, int b, int h, int32_t e, const uint8_t *&k, const uint8_t *&v)
{
    const int64_t off = __ldg(A.seq_offsets + b), S = __ldg(A.seq_offsets + b + 1) - off;
    if (e < 0 || off < 0 || S < 0 || off + S > A.total_S) return false;
    const uint8_t *row = nullptr;
    if (e >= S) {
        if (e - S < A.W) row = A.win_kv + ((int64_t)b * A.W + (e - S)) * A.row_bytes;
    } else {
        const int cnt = __ldg(A.count + b);
        int at = 0;
        for (int c = cnt >= 0 && cnt <= S ? cnt : 0; c > 1;) {  // last place of the ascending list whose entry is <= e
            const int half = c >> 1;
            at += __ldg(A.idx + off + at + half) <= e ? half : 0;
            c -= half;
        }
        if (cnt > 0 && cnt <= S && __ldg(A.idx + off + at) == e) row = A.hot_kv + (off + at) * A.row_bytes;
    }
    if (!row) {
        flag(ERRF_INDEX);
        return false;
    }
    constexpr int bytes = CT == DT_F32 ? 4 : 2;
    k = row + (int64_t)h * A.D * bytes;
    v = k + (int64_t)A.H * A.D * bytes;
    return true;
}

// One query row (token n, head hq) by one warp, key by key in fp32: 32 keys at a time, a key per lane for the
// scores, D / 32 dimensions per lane for the values.  The way out for rows whose tile met an infinity or NaN: a
// matrix product carries one from a key that a row must not see into that row as 0 x inf.  Such a row comes out
// as NaN, so a row that is not finite is done again here, over its own keys alone.  So are rows of E4M3 caches that met
// unusual value scales (usual_value_scale): the softmax sum is relative to the largest score (m), the value product to the
// largest score + log2 vs (mo), whatever the scales.  And fp32 rows that are not finite: the split into two tf32 parts
// makes NaN of an infinity (and of a number next to fp32's largest) that the row does see (CORE: with its Top-k entries).
// qs: the warp's D floats of shared memory.
template <int QT, int CT, bool CORE = false>
__device__ __forceinline__ void attend_row(const AttnArgs &A, int b, int64_t pos, int64_t n, int hq, float *qs)
{
    const int lane = threadIdx.x & 31;
    const int h = hq / (A.Hq / A.H), D = A.D, per = D / 32;
    for (int i = lane; i < D; i += 32) qs[i] = load_elem<QT>(A.q, n * A.q_stride + (int64_t)hq * D + i);
    __syncwarp();
    const Span sp = visible_span(pos, A.window, A.n_sink);
    // (a position behind the page table's end, from a bad length, has no keys: the search does not go there)
    const int64_t total = sp.sinks + max((int64_t)0, min(pos + 1, (int64_t)A.max_pages * A.page) - sp.lo);
    const float sl2 = A.scale * 1.4426950408889634f;  // scores in log2 units
    float m = -INFINITY, l = 0.f, mo = -INFINITY, acc[ATTN_MAX_D / 32];
#pragma unroll
    for (int i = 0; i < ATTN_MAX_D / 32; i++) acc[i] = 0.f;
    // (the cached keys, then the Top-k list's: each from a number of its own that is a multiple of 32)
    const int64_t cached = (total + 31) & ~(int64_t)31, keys = CORE ? cached + A.k : total;
#pragma unroll 1
    for (int64_t t0 = 0; t0 < keys; t0 += 32) {
        const int64_t t = t0 + lane;
        const uint8_t *kr = nullptr, *vr = nullptr;
        float ks = 1.f, vs = 1.f;
        bool there = false;
        if (t < total) there = cached_rows<CT>(A, b, h, t < sp.sinks ? t : sp.lo + (t - sp.sinks), kr, vr, ks, vs);
        if constexpr (CORE) {
            if (t >= cached && t < keys) there = listed_rows<CT>(A, b, h, __ldg(A.topk_idx + n * A.k + (t - cached)), kr, vr);
        }
        if (!there || vs == 0.f) vr = nullptr;  // (a bad scale, NaN among them, must not meet its weight of zero)
        float s = -INFINITY;
        if (there) {
            float d = 0.f;
#pragma unroll 4
            for (int i = 0; i < D; i++) d += qs[i] * load_elem<CT>(kr, i);
            s = d * (sl2 * ks);
        }
        const float mx = warp_max(s), mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
        const float p = there ? exp2f(s - ref) : 0.f;
        const float f = exp2f(m - ref);
        l = l * f + p;
        m = mn;
        float w = p, fo = f;  // weight in the value product, and what brings that to its new maximum
        if constexpr (CT == DT_FP8) {
            const float y = vr ? s + log2f(vs) : -INFINITY, on = fmaxf(mo, warp_max(y)), oref = on == -INFINITY ? 0.f : on;
            w = vr ? exp2f(y - oref) : 0.f;
            fo = exp2f(mo - oref);
            mo = on;
        }
#pragma unroll
        for (int i = 0; i < ATTN_MAX_D / 32; i++) acc[i] *= fo;
        const int many = (int)min((int64_t)32, keys - t0);
#pragma unroll 1
        for (int j = 0; j < many; j++) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            const uint8_t *rj = (const uint8_t *)__shfl_sync(0xffffffffu, (unsigned long long)vr, j);
            if (!rj) continue;
#pragma unroll
            for (int i = 0; i < ATTN_MAX_D / 32; i++)
                if (i < per) acc[i] += wj * load_elem<CT>(rj, lane + 32 * i);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    // (no key with a value: the sums of values are zero, whatever the maxima)
    const float back = CT == DT_FP8 ? (mo == -INFINITY ? 1.f : exp2f(mo - m)) : 1.f;
#pragma unroll
    for (int i = 0; i < ATTN_MAX_D / 32; i++)
        if (i < per) store_elem<QT>(A.out, (n * A.Hq + hq) * D + lane + 32 * i, acc[i] * inv * back);
    if (A.lse && lane == 0) A.lse[n * A.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    __syncwarp();
}

}  // namespace lsa
