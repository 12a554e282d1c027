// Core attention for few query rows: decode steps, small groups of tokens, every type and head size.
//
// A tile is 16 query rows of one sequence and key/value head (rows are token-major, the G = Hq / H heads
// of a group inside a token); its keys come in aligned chunks of 16 positions (E4M3: 32, in two halves), so
// 16 positions lie in one page and their rows are contiguous.  With so few rows the time goes into reading keys and values once
// (HBM), so the kernel is built around loads in flight: every warp walks chunks of its own with its own
// ring of stages (cp.async, 16 bytes a lane), the 16 rows of the tile in its registers, and never waits
// for another warp until the tile's end, where the warps' running maxima, sums and outputs are joined.
// The products are warp MMAs: 16 rows are one m16 tile, and the tensor pipe is far from its limit here
// (32 MMAs for the 8 KB of a bf16 chunk), so nothing is gained by staging them through TMEM.
//   bf16 cache:  m16n8k16 bf16, probabilities rounded to bf16 (their sum is taken before that): the product takes both
//                operands in the values' type, and a second product for the rest of each probability would double it.  Costs
//                2^-8 of a weight at most: output error 2.0e-3 to 2.3e-3 (2-norm) where the result's rounding has 1.7e-3.
//   E4M3 cache:  codes decoded exactly to f16; the query row is brought to f16 by a power of two of its
//                own, its largest element to [2^8, 2^9).  f16 steps by 2^-24 at least, so a bf16 element keeps its eight bits
//                down to 2^-17; from 2^25 below the largest they are lost, from 2^33 below the element is.  A page's
//                value scale vs enters the exponent: p' = 2^(s + log2 vs - m'), with m' the running maximum
//                of s + log2 vs, so p' is rounded to f16 relative to what it adds to the output; the softmax sum
//                takes p' / vs in fp32 (unusual scales: see usual_value_scale).  p' is kept 2^15 times larger (below
//                f16's largest), so that only weights under 2^-29 of the largest are subnormal and lose bits.
//   fp32 cache:  m16n8k8 tf32 with both operands split into two parts, x = hi + lo, three products
//                (the fourth, lo lo, is below 2^-22 of the product, as is what the rounding of each lo leaves): there is no
//                MMA in fp32.  Output error 7.7e-7 (2-norm) where sums in fp32 have 4.2e-7.  The split has no infinities: see attend_row.
//
// Measured: 32 users over a window of 4096, 8 heads of 128 in bf16: 96 us, 5.4 TB/s, bound by HBM; 8 histories of up
// to 131071 tokens in E4M3: 242 us (231-248 by box), 4.4 TB/s, bound by instruction issue; Top-2048 and a window of 512 for
// 32 users, 64 heads on 2: 42 us, bound by the 16-row tiles, which read a group's rows once for every 16 heads.
//
// Work is shared in one of two ways.  Tiles of bounded length (a window, a Top-k list) go to a cluster of up to
// eight CTAs each, which share its chunks and join their sums through distributed shared memory: one launch.
// Otherwise the chunks of all tiles of all sequences form one range that the CTAs share evenly (a tile's start and end, about
// as long as a dozen chunks, are not counted: a CTA whose share is many short sequences takes longer); a CTA's part of a tile that it does not hold whole goes to the workspace and k_attn_join adds the parts
// in order.  A CTA leaves at most two parts.
//
// The Top-k entries' rows are looked up by the CTA that reads them, before it reads: the sequence's ascending fetch
// list (or every 2^i-th of a long one) is copied into the ring's space and searched there.  Searching it in global
// memory, 32 unrelated addresses an instruction, took 20 us of 55 (32 tokens, 2048 of 8847 entries each).
#pragma once
#include "attn.cuh"
#include "pdl.cuh"

namespace lsa {

namespace few {

constexpr int WARPS = 4;
constexpr int ROWS = 16;
constexpr int JOIN_ROWS = 4;       // rows of a tile per CTA of k_attn_join

template <int CT, int D>
struct Cfg {
    static constexpr int EB = CT == DT_F32 ? 4 : (CT == DT_BF16 ? 2 : 1);
    static constexpr int RB = D * EB;               // bytes of a key or value row
    static constexpr int KEYS = CT == DT_FP8 ? 32 : 16;  // positions of a chunk: one or two halves of 16
    static constexpr int KH = KEYS / 16;
    static constexpr int CHUNK = 2 * KEYS * RB;     // keys, then values
    static constexpr int STAGES = 3;
    static constexpr int RING = WARPS * STAGES * CHUNK;
    static constexpr float SHIFT = CT == DT_FP8 ? 15.f : 0.f;  // probabilities are kept 2^SHIFT times larger
    static constexpr int NT = D / 8;                // n-tiles of the value product
    static constexpr int QREGS = CT == DT_F32 ? D / 2 : D / 4;  // query fragment registers
    static constexpr int OFF_MET = RING + 2 * WARPS * ROWS * 4 + WARPS * STAGES * 32;
    static constexpr int SMEM = OFF_MET + (CT == DT_FP8 ? WARPS * 4 : 0);
};

// 16-byte piece of a row that holds piece c of row `row`: chosen for each access pattern below so that the
// eight lanes of a phase fall on different banks.
template <int CT, int D>
__device__ __forceinline__ int swz(int row, int c)
{
    if constexpr (CT == DT_BF16) return D >= 64 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
    else if constexpr (CT == DT_F32 || D == 128) return c ^ ((((row >> 1) & 3) << 1) ^ ((row & 1) << 2));
    else if constexpr (D == 64) return c ^ (((row >> 1) & 1) << 1);
    else return c;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo, both tf32 (hi is x without its low bits' rounding; lo the rest, rounded).
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo)
{
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
}
__device__ __forceinline__ void mma_3xtf32(float (&d)[4], const float (&a)[4], float b0, float b1)
{
    uint32_t ah[4], al[4], bh0, bl0, bh1, bl1;
#pragma unroll
    for (int i = 0; i < 4; i++) split_tf32(a[i], ah[i], al[i]);
    split_tf32(b0, bh0, bl0);
    split_tf32(b1, bh1, bl1);
    mma_tf32(d, al, bh0, bh1);
    mma_tf32(d, ah, bl0, bl1);
    mma_tf32(d, ah, bh0, bh1);
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ bool finite4(const float4 &v)
{
    return fabsf(v.x) <= 3.4028235e38f && fabsf(v.y) <= 3.4028235e38f && fabsf(v.z) <= 3.4028235e38f && fabsf(v.w) <= 3.4028235e38f;
}

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t at_rank(uint32_t a, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t a, uint32_t rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at_rank(a, rank)));
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a, uint32_t rank)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at_rank(a, rank)));
    return v;
}

// Four E4M3 codes to two pairs of f16 (exact; a NaN code stays NaN).
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t codes, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(codes));
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack_b16x2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Dimension that k-step ks of the score product puts in slot e of the lanes of column c (E4M3: the order of
// the dimensions in the contraction is free, this one lets a lane read its codes 16 bytes at a time).
template <int D>
__device__ __forceinline__ int e4m3_dim(int ks, int c, int e)
{
    return D >= 64 ? 16 * (c + 4 * (ks / 4)) + 4 * (ks % 4) + e : 8 * c + 4 * ks + e;
}

// Dimension of accumulator element e (0: first column, 1: second) of n-tile t of the value product.
template <int CT>
__device__ __forceinline__ int out_dim(int t, int c, int e)
{
    if constexpr (CT == DT_BF16) return 8 * t + 2 * c + e;
    else return 32 * (t / 4) + 4 * (2 * c + e) + t % 4;
}

// Query fragments of rows r and r + 8 (null: a row that is not there), and the factor of each row's scores.
template <int CT, int D>
__device__ __forceinline__ void load_q(const void *const (&row)[2], int c, uint32_t (&q)[Cfg<CT, D>::QREGS], float (&f)[2])
{
    f[0] = f[1] = 1.f;
    if constexpr (CT == DT_BF16) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ks++)
#pragma unroll
            for (int i = 0; i < 4; i++) {  // a0: row r, k 2c; a1: row r + 8; a2, a3: k 2c + 8
                const uint32_t *p = (const uint32_t *)row[i & 1];
                q[4 * ks + i] = p ? __ldg(p + (16 * ks + 8 * (i >> 1) + 2 * c) / 2) : 0u;
            }
    } else if constexpr (CT == DT_FP8) {
        float mx[2] = {0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < D / 16; ks++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t *p = (const uint32_t *)row[i & 1];
                const uint32_t w = p ? __ldg(p + e4m3_dim<D>(ks, c, 2 * (i >> 1)) / 2) : 0u;
                q[4 * ks + i] = w;
                mx[i & 1] = fmaxf(mx[i & 1], fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xFFFF0000u))));
            }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            // 2^(8 - exponent of the row's largest): its element comes to [2^8, 2^9)
            int e = 8 - ((int)(__float_as_uint(mx[i]) >> 23) - 127);
            e = e > 120 ? 120 : (e < -120 ? -120 : e);
            const float up = __uint_as_float((uint32_t)(e + 127) << 23);
            f[i] = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
            for (int ks = 0; ks < D / 16; ks++)
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    uint32_t &w = q[4 * ks + 2 * k + i];
                    w = pack_f16x2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
                }
        }
    } else {
#pragma unroll
        for (int ks = 0; ks < D / 8; ks++)  // k-steps of 8: slots c and c + 4 are dimensions 2 (ks % 2) + {0, 1} of the lane's four
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float *p = (const float *)row[i & 1];
                q[4 * ks + i] = p ? __float_as_uint(__ldg(p + 16 * (ks / 2) + 4 * c + 2 * (ks % 2) + (i >> 1))) : 0u;
            }
    }
}

// s0, s1 += query rows . keys 0 .. 7, 8 .. 15 at shared address kb.
template <int CT, int D>
__device__ __forceinline__ void scores(uint32_t kb, const uint32_t (&q)[Cfg<CT, D>::QREGS], float (&s0)[4], float (&s1)[4])
{
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    if constexpr (CT == DT_BF16) {
        // matrices of ldmatrix: keys 0-7 and dims 0-7, keys 0-7 and dims 8-15, then keys 8-15
        const int row = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < D / 16; ks++) {
            uint32_t b[4];
            ldsm4(b, kb + (uint32_t)(row * Cfg<CT, D>::RB + swz<CT, D>(row, 2 * ks + half) * 16));
            const uint32_t a[4] = {q[4 * ks], q[4 * ks + 1], q[4 * ks + 2], q[4 * ks + 3]};
            mma_bf16(s0, a, b[0], b[1]);
            mma_bf16(s1, a, b[2], b[3]);
        }
    } else if constexpr (CT == DT_FP8) {
#pragma unroll
        for (int hh = 0; hh < (D >= 64 ? D / 64 : 1); hh++) {
            uint32_t w[2][4];
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int row = r + 8 * j;
                if constexpr (D >= 64) {
                    const uint4 v = lds128(kb + (uint32_t)(row * D + swz<CT, D>(row, c + 4 * hh) * 16));
                    w[j][0] = v.x; w[j][1] = v.y; w[j][2] = v.z; w[j][3] = v.w;
                } else {
                    const uint2 v = lds64(kb + (uint32_t)(row * D + c * 8));
                    w[j][0] = v.x; w[j][1] = v.y;
                }
            }
#pragma unroll
            for (int t = 0; t < (D >= 64 ? 4 : 2); t++) {
                const int ks = 4 * hh + t;
                const uint32_t a[4] = {q[4 * ks], q[4 * ks + 1], q[4 * ks + 2], q[4 * ks + 3]};
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    uint32_t b0, b1;
                    e4m3x4_to_f16x2(w[j][t], b0, b1);
                    mma_f16(j ? s1 : s0, a, b0, b1);
                }
            }
        }
    } else {
#pragma unroll
        for (int g = 0; g < D / 16; g++) {
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int row = r + 8 * j;
                const uint4 v = lds128(kb + (uint32_t)(row * Cfg<CT, D>::RB + swz<CT, D>(row, 4 * g + c) * 16));
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    const int ks = 2 * g + t;
                    const float a[4] = {__uint_as_float(q[4 * ks]), __uint_as_float(q[4 * ks + 1]),
                                        __uint_as_float(q[4 * ks + 2]), __uint_as_float(q[4 * ks + 3])};
                    mma_3xtf32(j ? s1 : s0, a, __uint_as_float(t ? v.z : v.x), __uint_as_float(t ? v.w : v.y));
                }
            }
        }
    }
}

// acc += p (16 rows x 16 keys, as the score product leaves them) . values at shared address vb.
template <int CT, int D>
__device__ __forceinline__ void values(uint32_t vb, const float (&p0)[4], const float (&p1)[4], float (&acc)[Cfg<CT, D>::NT][4])
{
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    if constexpr (CT == DT_BF16) {
        const uint32_t a[4] = {pack_b16x2(p0[0], p0[1]), pack_b16x2(p0[2], p0[3]), pack_b16x2(p1[0], p1[1]),
                               pack_b16x2(p1[2], p1[3])};
        const int row = lane & 15;
#pragma unroll
        for (int t = 0; t < D / 16; t++) {  // keys 0-7, 8-15 of dims 16t .. + 7, then of dims 16t + 8 .. + 15
            uint32_t b[4];
            ldsm4t(b, vb + (uint32_t)(row * Cfg<CT, D>::RB + swz<CT, D>(row, 2 * t + (lane >> 4)) * 16));
            mma_bf16(acc[2 * t], a, b[0], b[1]);
            mma_bf16(acc[2 * t + 1], a, b[2], b[3]);
        }
    } else if constexpr (CT == DT_FP8) {
        const uint32_t a[4] = {pack_f16x2(p0[0], p0[1]), pack_f16x2(p0[2], p0[3]), pack_f16x2(p1[0], p1[1]),
                               pack_f16x2(p1[2], p1[3])};
#pragma unroll
        for (int blk = 0; blk < D / 32; blk++) {
            uint32_t w[4];  // keys 2c, 2c + 1, 2c + 8, 2c + 9 of dims 32 blk + 4r .. + 3
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int row = 2 * c + (j & 1) + 8 * (j >> 1);
                w[j] = lds32(vb + (uint32_t)(row * D + swz<CT, D>(row, 2 * blk + (r >> 2)) * 16 + (r & 3) * 4));
            }
            // pairs of codes (key, key + 1) for dims 0, 1 and 2, 3 of the four
            const uint32_t x0 = __byte_perm(w[0], w[1], 0x5140), x1 = __byte_perm(w[0], w[1], 0x7362);
            const uint32_t y0 = __byte_perm(w[2], w[3], 0x5140), y1 = __byte_perm(w[2], w[3], 0x7362);
            uint32_t b[8];
            e4m3x4_to_f16x2(x0, b[0], b[2]);
            e4m3x4_to_f16x2(y0, b[1], b[3]);
            e4m3x4_to_f16x2(x1, b[4], b[6]);
            e4m3x4_to_f16x2(y1, b[5], b[7]);
#pragma unroll
            for (int t = 0; t < 4; t++) mma_f16(acc[4 * blk + t], a, b[2 * t], b[2 * t + 1]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; j++) {  // k-step j: slots c, c + 4 are keys 8j + 2c, + 1
            const float a[4] = {j ? p1[0] : p0[0], j ? p1[2] : p0[2], j ? p1[1] : p0[1], j ? p1[3] : p0[3]};
#pragma unroll
            for (int blk = 0; blk < D / 32; blk++) {
                const int row = 8 * j + 2 * c;
                const uint4 x = lds128(vb + (uint32_t)(row * Cfg<CT, D>::RB + swz<CT, D>(row, 8 * blk + r) * 16));
                const uint4 y = lds128(vb + (uint32_t)((row + 1) * Cfg<CT, D>::RB + swz<CT, D>(row + 1, 8 * blk + r) * 16));
                mma_3xtf32(acc[4 * blk], a, __uint_as_float(x.x), __uint_as_float(y.x));
                mma_3xtf32(acc[4 * blk + 1], a, __uint_as_float(x.y), __uint_as_float(y.y));
                mma_3xtf32(acc[4 * blk + 2], a, __uint_as_float(x.z), __uint_as_float(y.z));
                mma_3xtf32(acc[4 * blk + 3], a, __uint_as_float(x.w), __uint_as_float(y.w));
            }
        }
    }
}

// Rows of the Top-k entries [first, first + many) of query token n, sequence b, into rows[0, many): a row's number in
// hot_kv, or ~ its number in win_kv, or NO_ROW (none, or flagged).  list: `cap` words of shared memory, free for now.
constexpr int32_t NO_ROW = INT32_MIN;

__device__ __forceinline__ void find_rows(const AttnArgs &A, int b, int n, int first, int many, int32_t *rows, int32_t *list, int cap)
{
    constexpr int T = 32 * WARPS, M = 8;  // M entries of a thread side by side
    const int64_t off = __ldg(A.seq_offsets + b), S = __ldg(A.seq_offsets + b + 1) - off;
    int cnt = __ldg(A.count + b);
    if (off < 0 || S < 0 || off + S > A.total_S) {
        if (threadIdx.x == 0) flag(ERRF_OFFSETS);
        for (int i = threadIdx.x; i < many; i += T) rows[i] = NO_ROW;
        __syncthreads();
        return;
    }
    if (cnt < 0 || cnt > S) {
        if (threadIdx.x == 0) flag(ERRF_COUNT);
        cnt = 0;
    }
    const int32_t *idx = A.idx + off;
    int sh = 0;
    while (((cnt - 1) >> sh) + 1 > cap - 4) sh++;
    const int m = cnt > 0 ? ((cnt - 1) >> sh) + 1 : 0;
    // (a whole list keeps its place in a 16-byte word, so that all but its ends come 16 bytes at a time)
    if (sh == 0) list += ((uintptr_t)idx & 15) >> 2;
    const uint32_t la = (uint32_t)__cvta_generic_to_shared(list);
    const int head = sh == 0 ? min(m, (int)((16 - ((uintptr_t)idx & 15)) & 15) >> 2) : m, body = (m - head) >> 2;
    for (int i = threadIdx.x; i < head; i += T) cp_async4(la + 4 * i, idx + ((int64_t)i << sh), 4);
    for (int i = threadIdx.x; i < body; i += T) cp_async16(la + 4 * (head + 4 * i), idx + head + 4 * i, 16);
    for (int i = head + 4 * body + threadIdx.x; i < m; i += T) cp_async4(la + 4 * i, idx + i, 4);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    for (int i0 = threadIdx.x; i0 < many; i0 += M * T) {
        int32_t e[M];
        int at[M];  // last place of the list whose entry is <= e
#pragma unroll
        for (int x = 0; x < M; x++) {
            const int i = i0 + x * T;
            e[x] = i < many && first + i < A.k ? __ldg(A.topk_idx + (int64_t)n * A.k + first + i) : -1;
            at[x] = 0;
        }
        for (int c = m; c > 1;) {
            const int half = c >> 1;
#pragma unroll
            for (int x = 0; x < M; x++) at[x] += list[at[x] + half] <= e[x] ? half : 0;
            c -= half;
        }
#pragma unroll
        for (int x = 0; x < M; x++) {
            int32_t row = NO_ROW;
            if (e[x] >= S) {
                if (e[x] - S < A.W) row = ~(int32_t)(b * A.W + (e[x] - S));
            } else if (e[x] >= 0 && cnt > 0) {
                int slot = at[x] << sh;
                for (int c = min(cnt - slot, 1 << sh); c > 1;) {  // (only where the list was thinned)
                    const int half = c >> 1;
                    slot += __ldg(idx + slot + half) <= e[x] ? half : 0;
                    c -= half;
                }
                if ((sh == 0 ? list[slot] : __ldg(idx + slot)) == e[x]) row = (int32_t)(off + slot);
            }
            if (row == NO_ROW && e[x] >= 0) flag(ERRF_INDEX);
            if (i0 + x * T < many) rows[i0 + x * T] = row;
        }
    }
    __syncthreads();
}

// --------------------------------------------------------------------------------------- the work

// What the tiles of one sequence share.  Chunks are numbered [first tokens][window]: chunk u < sc is positions
// KEYS u .., the others KEYS (wc0 + u - sc) .., up to `chunks`; then the chunks of the Top-k list.
struct Seq {
    int off, n;     // first query token, query tokens
    int len;        // tokens before this call's
    int tiles;      // tiles of 16 rows
    int sc, wc0;
    int chunks;     // of the cache
    int total;      // with the Top-k list's
};

__device__ __forceinline__ int tiles_per_token(const AttnArgs &A) { return (A.Hq / A.H + ROWS - 1) / ROWS; }

template <bool CORE, int KEYS>
__device__ __forceinline__ Seq load_seq(const AttnArgs &A, int b)
{
    Seq s = {};
    const int64_t lo = __ldg(A.q_offsets + b), hi = __ldg(A.q_offsets + b + 1);
    if (lo < 0 || hi < lo || hi > A.N) {
        flag(ERRF_OFFSETS);
        return s;
    }
    s.off = (int)lo;
    s.n = (int)(hi - lo);
    if (s.n == 0) return s;
    s.len = __ldg(A.cache_len + b);
    const int G = A.Hq / A.H;
    s.tiles = CORE ? s.n * tiles_per_token(A) : (int)(((int64_t)s.n * G + ROWS - 1) / ROWS);
    const int limit = A.max_pages << A.page_shift;  // (below 2^31)
    if (s.len < 0) {
        flag(ERRF_COUNT);
        s.len = -s.n;  // every query stands before position 0: nothing to see
    } else if ((int64_t)s.len + s.n > limit) {
        flag(ERRF_COUNT);
        s.len = min(s.len, 0x7FFFFFFF - (1 << 25));  // (positions stay in 32 bits)
    }
    const int last = min(s.len + s.n, limit) - 1;
    const Span first = visible_span(max(s.len, 0), A.window, A.n_sink);
    s.wc0 = (int)(first.lo / KEYS);
    s.sc = min((int)((first.sinks + KEYS - 1) / KEYS), s.wc0);
    const int wend = last < 0 ? 0 : last / KEYS + 1;
    s.sc = min(s.sc, (limit + KEYS - 1) / KEYS);
    s.chunks = s.sc + max(0, wend - s.wc0);
    s.total = max(1, s.chunks + (CORE ? (A.k + KEYS - 1) / KEYS : 0));  // (a tile without keys still writes its rows)
    return s;
}

// One tile: 16 rows of a sequence and head.
struct Tile {
    int n0;          // CORE: its token; else the sequence's first token
    int p_lo, p_hi;  // positions of its first and last row's tokens
    int row0;        // first row (token-major within the sequence; CORE: first head of the group)
    int rows;
};

template <bool CORE>
__device__ __forceinline__ Tile make_tile(const AttnArgs &A, const Seq &s, int tile)
{
    Tile t;
    const int G = A.Hq / A.H;
    if constexpr (CORE) {
        const int tpt = tiles_per_token(A);
        t.n0 = s.off + tile / tpt;
        t.row0 = (tile % tpt) * ROWS;
        t.rows = min(ROWS, G - t.row0);
        t.p_lo = t.p_hi = s.len + tile / tpt;
    } else {
        t.n0 = s.off;
        t.row0 = tile * ROWS;
        t.rows = (int)min((int64_t)ROWS, (int64_t)s.n * G - t.row0);
        t.p_lo = s.len + t.row0 / G;
        t.p_hi = s.len + (t.row0 + t.rows - 1) / G;
    }
    return t;
}

// Token of row i of the tile, its position, and its head in the group.
template <bool CORE>
__device__ __forceinline__ void tile_row(const AttnArgs &A, const Seq &s, const Tile &t, int i, int &n, int &pos, int &g)
{
    if constexpr (CORE) {
        n = t.n0;
        pos = t.p_lo;
        g = t.row0 + i;
    } else {
        const int G = A.Hq / A.H, R = t.row0 + i;
        n = t.n0 + R / G;
        pos = s.len + R / G;
        g = R % G;
    }
}

// A part in the workspace: maxima and sums of 16 rows (of 2^(x - max)), then the sums of values.  E4M3: a sum is negative
// where the maximum is that of a key with a value scale of zero, NaN where a scale is unusual (marked_sum).
template <int D>
constexpr size_t part_floats() { return 2 * ROWS + (size_t)ROWS * D; }

template <int CT>
__device__ __forceinline__ float sum_of(float l) { return CT == DT_FP8 ? fabsf(l) : l; }
// The part (m, l) sets the maximum M, perhaps with a key whose value scale is zero.
template <int CT>
__device__ __forceinline__ bool from_zero(float l, float m, float M) { return CT == DT_FP8 && l < 0.f && m == M; }

// Chunks [u0, u1) of tile `tile` and head h of sequence b, by the whole CTA.  part: where to leave the sums (null:
// the outputs are written; with CLUSTER, together with the cluster's other CTAs, which have the tile's other chunks).
template <int QT, int CT, int D, bool CORE, bool CLUSTER>
__device__ __forceinline__ void do_tile(const AttnArgs &A, const Seq &s, int b, int tile, int h, int u0, int u1, float *part,
                                        uint8_t *smem)
{
    using C = Cfg<CT, D>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    uint8_t *ring = smem + warp * C::STAGES * C::CHUNK;
    const uint32_t ring_a = (uint32_t)__cvta_generic_to_shared(ring);
    float *ml = (float *)(smem + C::RING);
    constexpr int KEYS = C::KEYS, KH = C::KH;
    struct Meta { float sc[2][2]; uint32_t live, pad[3]; };  // key and value scale of each half; which keys are there
    Meta *meta = (Meta *)(ml + 2 * WARPS * ROWS) + warp * C::STAGES;
    const uint32_t meta_a = (uint32_t)__cvta_generic_to_shared(meta);
    // E4M3: whether the warp met unusual value scales
    uint32_t *met = (uint32_t *)(smem + C::OFF_MET) + warp;
    if constexpr (CT == DT_FP8) {
        if (lane == 0) *met = 0;
    }

    int32_t *entries = (int32_t *)(smem + C::SMEM);  // CORE: rows of the part's Top-k entries

    const Tile t = make_tile<CORE>(A, s, tile);
    const int G = A.Hq / A.H;
    const int low = A.window > 0 ? max(0, t.p_lo + 1 - A.window) : 0;  // first window key of the first row

    // the chunks of this tile among [u0, u1): [u0, min(u1, sc)) and [max(u0, a), min(u1, z)), then the Top-k list's
    // (first tokens that reach into the window's chunks: none of those is skipped)
    const int a = A.n_sink > s.wc0 * KEYS ? s.sc : max(s.sc, s.sc + low / KEYS - s.wc0);
    const int z = t.p_hi < 0 ? 0 : min(s.chunks, s.sc + t.p_hi / KEYS - s.wc0 + 1);
    const int e0 = t.p_hi < 0 ? 0 : max(0, min(u1, s.sc) - u0);
    const int b0 = max(u0, a), e1 = t.p_hi < 0 ? 0 : max(0, min(u1, z) - b0);
    const int c0 = max(u0, s.chunks), e2 = CORE ? max(0, u1 - c0) : 0;
    const int count = e0 + e1 + e2;
    auto chunk_of = [&](int i) -> int { return i < e0 ? u0 + i : (i < e0 + e1 ? b0 + (i - e0) : c0 + (i - e0 - e1)); };
    auto pos_of = [&](int u) -> int { return (u < s.sc ? u : s.wc0 + (u - s.sc)) * KEYS; };

    uint32_t q[C::QREGS];
    float qf[2];
    int rpos[2];
    {
        const void *rows[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            rows[i] = nullptr;
            rpos[i] = -1;
            if (r + 8 * i < t.rows) {
                int n, g;
                tile_row<CORE>(A, s, t, r + 8 * i, n, rpos[i], g);
                constexpr int qb = QT == DT_F32 ? 4 : 2;
                rows[i] = (const uint8_t *)A.q + (n * A.q_stride + (int64_t)(h * G + g) * D) * qb;
            }
        }
        load_q<CT, D>(rows, c, q, qf);
    }
    const float sl2 = A.scale * 1.4426950408889634f;
    const float sf[2] = {sl2 * qf[0], sl2 * qf[1]};

    float acc[C::NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < C::NT; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[i][e] = 0.f;

    // 16 rows are RB pieces of 16 bytes for the keys and as many for the values; piece lane + 32 x goes to lane, and
    // XH values of x are a half of a chunk.  The swizzle repeats every 8 rows, i.e. every REP values of x.
    constexpr int XH = C::RB / 32, REP = C::RB >= 64 ? C::RB / 64 : 1, PR = C::RB / 16;
    uint32_t so[REP];
#pragma unroll
    for (int x = 0; x < REP; x++) {
        const int piece = lane + 32 * x, row = piece / PR;
        so[x] = (uint32_t)(row * C::RB + swz<CT, D>(row, piece % PR) * 16);
    }
    auto dst = [&](int x) -> uint32_t { return so[x % REP] + (uint32_t)(x / REP) * (uint32_t)(REP * 512); };

    // what the loads of the CTA's i-th chunk need from memory first: its page, or its entries' rows (a lane each)
    auto look = [&](int i) -> int32_t {
        if (i >= count) return -1;
        const int u = chunk_of(i);
        if (CORE && u >= s.chunks) return entries[(u - c0) * KEYS + (lane & 15)];
        // (lanes 0-15 for the first half, the others for the second; its page may lie behind the table's end: not used)
        const int at = (pos_of(u) + (KH > 1 ? lane & 16 : 0)) >> A.page_shift;
        return __ldg(A.page_table + (int64_t)b * A.max_pages + (KH > 1 ? min(at, A.max_pages - 1) : at));
    };
    // (the last position to load: a length that is flagged may put rows behind the page table's end)
    const int p_end = min(t.p_hi, (A.max_pages << A.page_shift) - 1);
    // start the loads of the CTA's i-th chunk (warp w takes w, w + WARPS, ..)
    auto issue = [&](int i, int stage, int32_t found) {
        const uint32_t kb = ring_a + (uint32_t)stage * C::CHUNK, vb = kb + KEYS * C::RB;
        const int u = chunk_of(i);
        if (!CORE || u < s.chunks) {
            uint32_t live = 0;
#pragma unroll
            for (int hf = 0; hf < KH; hf++) {
                const int p0 = pos_of(u) + 16 * hf;
                int page = KH > 1 ? __shfl_sync(0xffffffffu, found, 16 * hf) : found;
                if (KH > 1 && (p0 > p_end || (p0 + 15 < low && p0 >= A.n_sink))) {
                    page = -1;  // (a half that no row sees: its page is not looked at)
                } else if (page < 0 || page >= A.n_pages) {
                    if (lane == 0) flag(ERRF_PAGE);
                    page = -1;
                }
                const int64_t ph = (int64_t)max(page, 0) * A.H + h;
                const int64_t byte = ((ph << A.page_shift) + (p0 & ((1 << A.page_shift) - 1))) * C::RB + lane * 16;
                const uint8_t *kp = (const uint8_t *)A.k_cache + byte, *vp = (const uint8_t *)A.v_cache + byte;
                if (page >= 0 && p0 + 15 <= p_end && (p0 >= low || p0 + 16 <= A.n_sink)) {
#pragma unroll
                    for (int x = 0; x < XH; x++) cp_async16(kb + dst(hf * XH + x), kp + 512 * x, 16);
#pragma unroll
                    for (int x = 0; x < XH; x++) cp_async16(vb + dst(hf * XH + x), vp + 512 * x, 16);
                } else {  // keys that no row of the tile sees come in as zeros
#pragma unroll
                    for (int x = 0; x < XH; x++) {
                        const int pos = p0 + (lane + 32 * x) / PR;
                        const bool see = page >= 0 && pos <= p_end && (pos >= low || pos < A.n_sink);
                        cp_async16(kb + dst(hf * XH + x), see ? kp + 512 * x : (const uint8_t *)A.k_cache, see ? 16 : 0);
                        cp_async16(vb + dst(hf * XH + x), see ? vp + 512 * x : (const uint8_t *)A.v_cache, see ? 16 : 0);
                    }
                }
                if constexpr (CT == DT_FP8) {
                    if (lane < 2)
                        cp_async4(meta_a + (uint32_t)stage * 32 + hf * 8 + lane * 4, (lane ? A.v_scale : A.k_scale) + ph, page >= 0 ? 4 : 0);
                }
                if (page >= 0) live |= 0xFFFFu << (16 * hf);
            }
            if (lane == 0) meta[stage].live = live;
        } else {
            const uint32_t live = __ballot_sync(0xffffffffu, found != NO_ROW) & 0xFFFFu;
#pragma unroll
            for (int x = 0; x < XH; x++) {
                const int piece = lane + 32 * x, pc = piece % PR;
                const int32_t row = __shfl_sync(0xffffffffu, found, piece / PR);
                const uint8_t *p = (row >= 0 ? A.hot_kv + row * A.row_bytes : A.win_kv + (int64_t)~row * A.row_bytes) +
                                   (int64_t)h * C::RB + pc * 16;
                const bool there = row != NO_ROW;
                cp_async16(kb + dst(x), there ? p : A.hot_kv, there ? 16 : 0);
                cp_async16(vb + dst(x), there ? p + (int64_t)A.H * C::RB : A.hot_kv, there ? 16 : 0);
            }
            if (lane == 0) meta[stage].live = live;
        }
    };

    if constexpr (CORE) {
        if (e2 > 0) find_rows(A, b, t.n0, (c0 - s.chunks) * KEYS, e2 * KEYS, entries, (int32_t *)smem, C::RING / 4);
    }
    float last_vs[KH], lv[KH], inv_vs[KH];
#pragma unroll
    for (int hf = 0; hf < KH; hf++) {
        last_vs[hf] = inv_vs[hf] = 1.f;
        lv[hf] = 0.f;
    }
    {
        int32_t f[C::STAGES - 1];  // (the first look-ups together)
#pragma unroll
        for (int st = 0; st < C::STAGES - 1; st++) f[st] = look(warp + st * WARPS);
#pragma unroll
        for (int st = 0; st < C::STAGES - 1; st++) {
            if (warp + st * WARPS < count) issue(warp + st * WARPS, st, f[st]);
            cp_commit();
        }
    }
    int32_t next = look(warp + (C::STAGES - 1) * WARPS);
    int stage = 0, fill = C::STAGES - 1;
#pragma unroll 1
    for (int i = warp; i < count; i += WARPS) {
        if (i + (C::STAGES - 1) * WARPS < count) issue(i + (C::STAGES - 1) * WARPS, fill, next);
        cp_commit();
        next = look(i + C::STAGES * WARPS);
        cp_wait<C::STAGES - 1>();
        __syncwarp();
        const uint32_t kb = ring_a + (uint32_t)stage * C::CHUNK, vb = kb + KEYS * C::RB;
        const int u = chunk_of(i);
        const bool listed = CORE && u >= s.chunks;
        uint32_t live = meta[stage].live;
        float ks[KH];
#pragma unroll
        for (int hf = 0; hf < KH; hf++) {
            ks[hf] = 1.f;
            if constexpr (CT == DT_FP8) {
                ks[hf] = meta[stage].sc[hf][0];
                const float vs = meta[stage].sc[hf][1];
                if ((live >> (16 * hf) & 1) && (!good_scale(ks[hf]) || !good_scale(vs))) {
                    if (lane == 0) flag(ERRF_SCALE);
                    live &= ~(0xFFFFu << (16 * hf));
                }
                // (a half that is not there has come in with scales of zero, which are not a page's)
                if ((live >> (16 * hf) & 1) && vs != last_vs[hf]) {
                    last_vs[hf] = vs;
                    if (usual_value_scale(vs)) {
                        lv[hf] = log2f(vs);
                        inv_vs[hf] = 1.f / vs;
                    } else {
                        lv[hf] = vs > 0.f ? log2f(vs) : ZERO_LV;
                        inv_vs[hf] = vs > 0.f ? 1.f / vs : ZERO_INV;
                        if (lane == 0) *met |= met_of(vs);
                    }
                }
            }
        }
        float x[2 * KH][4];
#pragma unroll
        for (int j = 0; j < 2 * KH; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) x[j][e] = 0.f;
#pragma unroll
        for (int hf = 0; hf < KH; hf++) scores<CT, D>(kb + hf * 16 * C::RB, q, x[2 * hf], x[2 * hf + 1]);
        const int p0 = pos_of(u);
        const bool whole = live == (KH > 1 ? 0xFFFFFFFFu : 0xFFFFu) &&
                           (listed || (p0 + KEYS - 1 <= t.p_lo && (A.window == 0 || p0 > t.p_hi - A.window || p0 + KEYS <= A.n_sink)));
#pragma unroll
        for (int j = 0; j < 2 * KH; j++) {
            const float fa = sf[0] * ks[j / 2], fb = sf[1] * ks[j / 2];
#pragma unroll
            for (int e = 0; e < 4; e++) x[j][e] = CT == DT_FP8 ? fmaf(x[j][e], e < 2 ? fa : fb, lv[j / 2]) : x[j][e] * (e < 2 ? fa : fb);
        }
        if (!whole) {
#pragma unroll
            for (int j = 0; j < 2 * KH; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int key = 8 * j + 2 * c + (e & 1), pos = p0 + key, me = rpos[e >> 1];
                    const bool see = (live >> key & 1) &&
                                     (listed || (pos <= me && (A.window == 0 || pos > me - A.window || pos < A.n_sink)));
                    if (!see) x[j][e] = -INFINITY;
                }
        }
        bool moved = false;
        float f[2];
#pragma unroll
        for (int i2 = 0; i2 < 2; i2++) {
            float mx = fmaxf(fmaxf(x[0][2 * i2], x[0][2 * i2 + 1]), fmaxf(x[1][2 * i2], x[1][2 * i2 + 1]));
            if constexpr (KH > 1) mx = fmaxf(mx, fmaxf(fmaxf(x[2][2 * i2], x[2][2 * i2 + 1]), fmaxf(x[3][2 * i2], x[3][2 * i2 + 1])));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[i2], mx);
            const float ref = mn == -INFINITY ? 0.f : mn;
            f[i2] = exp2_fast(m[i2] - ref);
            moved |= mn != m[i2];
            m[i2] = mn;
            l[i2] *= f[i2];
#pragma unroll
            for (int hf = 0; hf < KH; hf++) {
                float sum = 0.f;
#pragma unroll
                for (int j = 2 * hf; j < 2 * hf + 2; j++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        float &v = x[j][2 * i2 + e];
                        v = exp2_fast(v - (ref - C::SHIFT));
                        sum += v;
                    }
                l[i2] = fmaf(sum, inv_vs[hf], l[i2]);
            }
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int i2 = 0; i2 < C::NT; i2++) {
                acc[i2][0] *= f[0];
                acc[i2][1] *= f[0];
                acc[i2][2] *= f[1];
                acc[i2][3] *= f[1];
            }
        }
        // (a value scale of zero: the keys have had their share of the softmax sum and add nothing)
#pragma unroll
        for (int hf = 0; hf < KH; hf++)
            if ((live >> (16 * hf) & 0xFFFFu) && !(CT == DT_FP8 && last_vs[hf] == 0.f)) values<CT, D>(vb + hf * 16 * C::RB, x[2 * hf], x[2 * hf + 1], acc);
        __syncwarp();
        stage = stage + 1 == C::STAGES ? 0 : stage + 1;
        fill = fill + 1 == C::STAGES ? 0 : fill + 1;
    }
    cp_wait<0>();
    __syncwarp();

    // join the warps: maxima, then every warp's sums brought to the common maximum
#pragma unroll
    for (int i = 0; i < 2; i++) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if (c == 0) {
            if constexpr (CT == DT_FP8) l[i] = marked_sum(l[i], *met, 32768.f);
            ml[warp * ROWS + r + 8 * i] = m[i];
            ml[(WARPS + warp) * ROWS + r + 8 * i] = l[i];
        }
    }
    __syncthreads();
    float *os = (float *)smem + warp * ROWS * D;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        float M = ml[r + 8 * i];
#pragma unroll
        for (int w = 1; w < WARPS; w++) M = fmaxf(M, ml[w * ROWS + r + 8 * i]);
        const float f = m[i] == -INFINITY ? 0.f : exp2_fast(m[i] - M);
#pragma unroll
        for (int nt = 0; nt < C::NT; nt++)
#pragma unroll
            for (int e = 0; e < 2; e++) os[(r + 8 * i) * D + out_dim<CT>(nt, c, e)] = acc[nt][2 * i + e] * f;
    }
    __syncthreads();
    constexpr int GROUPS = D / 4;  // four dimensions of a row each
    uint32_t bad = 0;              // rows of this thread's that are not finite
    // (again: the row's maximum may be that of a key with a value scale of zero)
    auto write = [&](int row, int d, float4 o, float M, float L, bool again) {
        int n, pos, g;
        tile_row<CORE>(A, s, t, row, n, pos, g);
        const int64_t at = (int64_t)n * A.Hq + h * G + g;
        const float inv = L == 0.f ? 0.f : 1.f / L;
        o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
        if (again || !finite4(o)) bad |= 1u << row;
        if constexpr (QT == DT_F32)
            *(float4 *)((float *)A.out + at * D + d) = o;
        else
            *(uint2 *)((__nv_bfloat16 *)A.out + at * D + d) = make_uint2(pack_b16x2(o.x, o.y), pack_b16x2(o.z, o.w));
        if (A.lse && d == 0) A.lse[at] = L == 0.f ? -INFINITY : (M - C::SHIFT + log2f(L)) * 0.6931471805599453f;
    };
    // the CTA's own sums, for the cluster: maxima, sums, outputs (behind the warps' outputs)
    float *own = (float *)smem + WARPS * ROWS * D;
    static_assert(((WARPS + 1) * ROWS * D + 2 * ROWS) * 4 <= C::RING, "the joined sums fit in the ring");
    const uint32_t ranks = CLUSTER ? cluster_size() : 1u;
    for (int i = tid; i < ROWS * GROUPS; i += 32 * WARPS) {
        const int row = i / GROUPS, d = (i % GROUPS) * 4;
        if (row >= t.rows) continue;
        float M = ml[row], L = 0.f;
        bool zero = false;
#pragma unroll
        for (int w = 1; w < WARPS; w++) M = fmaxf(M, ml[w * ROWS + row]);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; w++) {
            const float mw = ml[w * ROWS + row], lw = ml[(WARPS + w) * ROWS + row];
            L += sum_of<CT>(lw) * (mw == -INFINITY ? 0.f : exp2_fast(mw - M));
            zero |= from_zero<CT>(lw, mw, M);
            const float4 v = *(const float4 *)((const float *)smem + (w * ROWS + row) * D + d);
            o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
        }
        if (part || ranks > 1) {
            float *to = part ? part : own;
            if (d == 0) {
                to[row] = M;
                to[ROWS + row] = zero ? -L : L;
            }
            *(float4 *)(to + 2 * ROWS + row * D + d) = o;
        } else {
            write(row, d, o, M, L, zero);
        }
    }
    if (CLUSTER && ranks > 1) {
        cluster_sync();
        const uint32_t own_a = (uint32_t)__cvta_generic_to_shared(own), me = cluster_rank(), per = ROWS / ranks;
        for (int i = tid; i < (int)per * GROUPS; i += 32 * WARPS) {
            const int row = (int)(me * per) + i / GROUPS, d = (i % GROUPS) * 4;
            if (row >= t.rows) continue;
            float M = -INFINITY, L = 0.f;
            bool zero = false;
            for (uint32_t w = 0; w < ranks; w++) M = fmaxf(M, ld_cluster(own_a + row * 4, w));
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (uint32_t w = 0; w < ranks; w++) {
                const float mw = ld_cluster(own_a + row * 4, w), f = mw == -INFINITY ? 0.f : exp2_fast(mw - M);
                const float4 v = ld_cluster4(own_a + (2 * ROWS + row * D + d) * 4, w);
                const float lw = ld_cluster(own_a + (ROWS + row) * 4, w);
                L = fmaf(sum_of<CT>(lw), f, L);
                zero |= from_zero<CT>(lw, mw, M);
                o.x = fmaf(v.x, f, o.x); o.y = fmaf(v.y, f, o.y); o.z = fmaf(v.z, f, o.z); o.w = fmaf(v.w, f, o.w);
            }
            write(row, d, o, M, L, zero);
        }
        cluster_sync();  // (nobody leaves, or writes its ring, while the others read its sums)
    }
    __syncthreads();  // the ring is free again
    if constexpr (!CORE || CT == DT_F32) {
        // rows of several tokens: one that is not finite may have met another's key; fp32 rows that are not finite; rows
        // with unusual value scales (see attend_row)
        if (!part && (t.p_lo != t.p_hi || CT != DT_BF16)) {
            bad = __reduce_or_sync(0xffffffffu, bad);
            uint32_t *rows = (uint32_t *)smem;
            if (lane == 0) rows[warp] = bad;
            __syncthreads();
            bad = rows[0] | rows[1] | rows[2] | rows[3];
            static_assert(WARPS == 4, "the line above");
            __syncthreads();
            for (int row = warp; row < t.rows; row += WARPS) {
                if (!(bad >> row & 1)) continue;
                int n, pos, g;
                tile_row<CORE>(A, s, t, row, n, pos, g);
                attend_row<QT, CT, CORE>(A, b, pos, n, h * G + g, (float *)smem + warp * ATTN_MAX_D);
            }
            __syncthreads();
        }
    }
}

// Sum over the block of v, and the sum over the threads before this one.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *warp_sums, int64_t &before)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int64_t total = 0, base = 0;
    for (int w = 0; w < warps; w++) {
        if (w == warp) base = total;
        total += warp_sums[w];
    }
    before = base + x - v;
    return total;
}

// Chunks of sequence b's tiles, of all heads.
__device__ __forceinline__ int64_t seq_cost(const AttnArgs &A, const Seq &s) { return (int64_t)s.tiles * A.H * s.total; }

// Range of CTA c of `ctas` among `total` chunks.
__device__ __forceinline__ int64_t range_start(int64_t total, int c, int ctas) { return total * c / ctas; }
// CTA whose range holds chunk x.
__device__ __forceinline__ int cta_of(int64_t total, int64_t x, int ctas) { return (int)(((x + 1) * ctas - 1) / total); }

// CTAs that share the work: no more than leave 128 keys to each.
template <int KEYS>
__device__ __forceinline__ int sharing_ctas(int64_t total, int grid)
{
    const int64_t c = total / (128 / KEYS);
    return c < 1 ? 1 : (c < grid ? (int)c : grid);
}

template <int CT, int D>
constexpr int CTAS_PER_SM = Cfg<CT, D>::SMEM <= 74 * 1024 ? 3 : (Cfg<CT, D>::SMEM <= 112 * 1024 ? 2 : 1);

template <int QT, int CT, int D, bool CORE, bool SPLIT>
__global__ void __launch_bounds__(32 * WARPS, CTAS_PER_SM<CT, D>) k_attn_few(const AttnArgs A, float *parts)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t sums[WARPS];
    __shared__ int found;
    __shared__ int64_t found_before;
    if constexpr (!SPLIT) {
        // one cluster per tile and head; tiles of sequence b are numbered from off_b G / 16 + b (CORE: off_b tiles a
        // token), so that ranges of ragged sequences do not meet
        const int G = A.Hq / A.H;
        const uint32_t Z = cluster_size(), z = cluster_rank();
        const int64_t x = blockIdx.x / Z;
        if (threadIdx.x == 0) found = -1;
        __syncthreads();
        for (int b = threadIdx.x; b < A.B; b += blockDim.x) {
            const int64_t lo = __ldg(A.q_offsets + b), hi = __ldg(A.q_offsets + b + 1);
            if (lo < 0 || hi < lo || hi > A.N) flag(ERRF_OFFSETS);
            else if (hi > lo && (CORE ? lo * tiles_per_token(A) : lo * G / ROWS + b) <= x) atomicMax(&found, b);
        }
        __syncthreads();
        const int b = found;
        if (b < 0) return;  // (the whole cluster)
        const Seq s = load_seq<CORE, Cfg<CT, D>::KEYS>(A, b);
        const int64_t tile = x - (CORE ? (int64_t)s.off * tiles_per_token(A) : (int64_t)s.off * G / ROWS + b);
        if (tile >= s.tiles) return;
        const int u0 = (int)((int64_t)s.total * z / Z), u1 = (int)((int64_t)s.total * (z + 1) / Z);
        do_tile<QT, CT, D, CORE, true>(A, s, b, (int)tile, blockIdx.y, u0, u1, nullptr, smem);
    } else {
        pdl_trigger();
        if (threadIdx.x == 0) found = -1;
        int64_t total = 0, mine = 0, before = 0;  // (of the last group of sequences: the only one up to 128)
        for (int b0 = 0; b0 < A.B; b0 += blockDim.x) {
            const int b = b0 + threadIdx.x;
            mine = b < A.B ? seq_cost(A, load_seq<CORE, Cfg<CT, D>::KEYS>(A, b)) : 0;
            total += block_scan(mine, sums, before);
        }
        const int ctas = sharing_ctas<Cfg<CT, D>::KEYS>(total, gridDim.x);
        if (total == 0 || (int)blockIdx.x >= ctas) return;
        int64_t x = range_start(total, blockIdx.x, ctas);
        const int64_t end = range_start(total, blockIdx.x + 1, ctas);
        // the sequence that holds x
        if (A.B > (int)blockDim.x) {
            int64_t base = 0;
            for (int b0 = 0; b0 < A.B; b0 += blockDim.x) {
                const int b = b0 + threadIdx.x;
                mine = b < A.B ? seq_cost(A, load_seq<CORE, Cfg<CT, D>::KEYS>(A, b)) : 0;
                const int64_t sum = block_scan(mine, sums, before);
                before += base;
                if (base + sum > x) {
                    if (mine > 0 && before <= x && x < before + mine) {
                        found = b;
                        found_before = before;
                    }
                    break;  // (the same for every thread)
                }
                base += sum;
            }
        } else if (mine > 0 && before <= x && x < before + mine) {
            found = threadIdx.x;
            found_before = before;
        }
        __syncthreads();
        int b = found;
        if (b < 0) return;
        int64_t seq_start = found_before;
        Seq s = load_seq<CORE, Cfg<CT, D>::KEYS>(A, b);
        while (x < end) {
            while (x >= seq_start + seq_cost(A, s)) {
                seq_start += seq_cost(A, s);
                if (++b >= A.B) return;
                s = load_seq<CORE, Cfg<CT, D>::KEYS>(A, b);
            }
            const int64_t rel = x - seq_start;
            const int64_t item = rel / s.total;
            const int u0 = (int)(rel % s.total);
            const int u1 = (int)min((int64_t)s.total, u0 + (end - x));
            float *part = nullptr;
            if (u0 > 0 || u1 < s.total) part = parts + (size_t)(2 * blockIdx.x + (u0 > 0 ? 0 : 1)) * part_floats<D>();
            // heads inside tiles: neighbouring CTAs then read neighbouring heads of the same pages
            do_tile<QT, CT, D, CORE, false>(A, s, b, (int)(item / A.H), (int)(item % A.H), u0, u1, part, smem);
            x += u1 - u0;
        }
    }
}

// Joins the parts of the tiles that k_attn_few split.  Grid: (tile numbers as in the unsplit launch, heads,
// groups of JOIN_ROWS rows); split_grid: CTAs that k_attn_few was launched with; shift: its
// Cfg::SHIFT.
template <int QT, int CT, int D, bool CORE>
__global__ void __launch_bounds__(32 * JOIN_ROWS) k_attn_join(const AttnArgs A, const float *parts, int split_grid, float shift)
{
    __shared__ int64_t sums[JOIN_ROWS];
    __shared__ int found;
    __shared__ int64_t found_before;
    const int G = A.Hq / A.H;
    const int64_t x = blockIdx.x;
    if (threadIdx.x == 0) found = -1;
    __syncthreads();
    int64_t total = 0;
    // the sequence of this tile (the last whose tile numbers start at or before x), and the chunks before it
    for (int b0 = 0; b0 < A.B; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        Seq s = {};
        if (b < A.B) s = load_seq<CORE, Cfg<CT, D>::KEYS>(A, b);
        const bool mine = s.n > 0 && (CORE ? (int64_t)s.off * tiles_per_token(A) : (int64_t)s.off * G / ROWS + b) <= x;
        if (mine) atomicMax(&found, b);
        int64_t before;
        const int64_t sum = block_scan(seq_cost(A, s), sums, before);
        if (mine && found == b) found_before = total + before;
        total += sum;
        __syncthreads();
    }
    pdl_wait();  // (before any return: this launch must not end before the one whose parts it joins)
    const int b = found;
    if (b < 0) return;
    const Seq s = load_seq<CORE, Cfg<CT, D>::KEYS>(A, b);
    const int64_t tile = x - (CORE ? (int64_t)s.off * tiles_per_token(A) : (int64_t)s.off * G / ROWS + b);
    if (tile >= s.tiles) return;
    const int h = blockIdx.y, ctas = sharing_ctas<Cfg<CT, D>::KEYS>(total, split_grid);
    const int64_t start = found_before + (tile * A.H + h) * s.total;
    const int c0 = cta_of(total, start, ctas), c1 = cta_of(total, start + s.total - 1, ctas);
    if (c0 == c1) return;  // written whole
    const Tile t = make_tile<CORE>(A, s, (int)tile);
    const int row = blockIdx.z * JOIN_ROWS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= t.rows) return;
    constexpr size_t PF = part_floats<D>();
    auto part = [&](int cta) { return parts + (size_t)(2 * cta + (cta == c0 ? 1 : 0)) * PF; };
    float M = -INFINITY;
    for (int i = c0 + lane; i <= c1; i += 32) M = fmaxf(M, part(i)[row]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    constexpr int PER = D / 32;
    float acc[PER], L = 0.f;
    bool zero = false;
#pragma unroll
    for (int e = 0; e < PER; e++) acc[e] = 0.f;
#pragma unroll 4
    for (int i = c0; i <= c1; i++) {
        const float *p = part(i);
        const float m = p[row], f = m == -INFINITY ? 0.f : exp2_fast(m - M);
        L = fmaf(sum_of<CT>(p[ROWS + row]), f, L);
        zero |= from_zero<CT>(p[ROWS + row], m, M);
#pragma unroll
        for (int e = 0; e < PER; e++) acc[e] = fmaf(p[2 * ROWS + row * D + lane + 32 * e], f, acc[e]);
    }
    int n, pos, g;
    tile_row<CORE>(A, s, t, row, n, pos, g);
    const int64_t at = (int64_t)n * A.Hq + h * G + g;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    bool bad = zero;
#pragma unroll
    for (int e = 0; e < PER; e++) {
        const float v = acc[e] * inv;
        bad |= !(fabsf(v) <= 3.4028235e38f);
        store_elem<QT>(A.out, at * D + lane + 32 * e, v);
    }
    if (A.lse && lane == 0) A.lse[at] = L == 0.f ? -INFINITY : (M - shift + log2f(L)) * 0.6931471805599453f;
    if constexpr (!CORE || CT == DT_F32) {
        __shared__ float qs[JOIN_ROWS][ATTN_MAX_D];
        if ((t.p_lo != t.p_hi || CT != DT_BF16) && __any_sync(0xffffffffu, bad))
            attend_row<QT, CT, CORE>(A, b, pos, n, h * G + g, qs[threadIdx.x >> 5]);
    }
}

// CTAs of a launch that is split over keys, and the parts they may leave.
constexpr int SPLIT_CTAS = 3 * 148;
inline size_t parts_bytes(int D) { return (size_t)2 * SPLIT_CTAS * (2 * ROWS + (size_t)ROWS * D) * sizeof(float); }

// Tiles of at most this many keys go to clusters, the others are split over the grid.  Measured (split : cluster, us, 8 heads
// of 128 in bf16, a step, L2 cold):
//   keys                               512       1000        2000       4000       8000
//   1 user                           19 : 12    21 : 14    23 : 14    27 : 18    29 : 23
//   32 users                         33 : 26    45 : 39    70 : 64   115 : 109  195 : 189
//   100 users                        72 : 64   106 : 92   168 : 147  311 : 281  583 : 537
//   32 users, one of that length,
//   the others of 100 keys                      27 : 25    31 : 33    33 : 53    39 : 90
// Clusters lead while lengths are alike, and lose to the even shares by what lengths differ: the more, the longer they are.
// A length is not known here, only its bound, hence the limit.  E4M3 likewise (32 users 27 : 25, 29 : 35, 35 : 55, 43 : 96 in
// the last row); fp32 at D = 128, one CTA an SM, is within 6 % either way over windows (32 users of 4000: 428 : 443), but
// its Top-k lists lose by clusters of eight, which do not fill the SMs (8 users, Top-2048: 74 : 104).
constexpr int64_t CLUSTER_KEYS = 4096;

template <int QT, int CT, int D, bool CORE>
cudaError_t launch(const AttnArgs &A, void *workspace, int sms, cudaStream_t st, int *launches)
{
    using C = Cfg<CT, D>;
    constexpr int KEYS = C::KEYS;
    float *parts = (float *)workspace;
    const int G = A.Hq / A.H, tpt = (G + ROWS - 1) / ROWS;
    const int64_t tiles = CORE ? A.N * tpt : A.N * G / ROWS + A.B;
    if (tiles * 8 >= (int64_t)1 << 31 || A.H > 65535) return cudaErrorInvalidConfiguration;
    // chunks of a tile at most, and tiles, were the tokens shared evenly by the sequences
    const int64_t limit = (int64_t)A.max_pages * A.page, n = A.N / A.B;
    const int64_t seen = A.window > 0 && A.window + n < limit ? A.window + n : limit;
    const int64_t list = CORE ? (A.k + KEYS - 1) / KEYS : 0;
    const int64_t chunks = seen / KEYS + 2 + (A.window > 0 ? (A.n_sink < limit ? A.n_sink : limit) / KEYS + 1 : 0) + list;
    const int64_t likely = CORE ? tiles : A.B * ((n * G + ROWS - 1) / ROWS > 0 ? (n * G + ROWS - 1) / ROWS : 1);
    const size_t smem = C::SMEM + (CORE ? (size_t)list * KEYS * 4 : 0);
    constexpr size_t most_smem = C::SMEM + (CORE ? LSA_MAX_TOPK * 4 : 0);
    const int per_sm = std::max(1, std::min(CTAS_PER_SM<CT, D>, (int)(227 * 1024 / (smem + 1024))));
    cudaLaunchAttribute attr[1];
    cudaError_t e;
    if (chunks * KEYS <= CLUSTER_KEYS) {
        // as many CTAs a tile as leave each one chunk a warp and run at once
        int Z = 1;
        while (Z < 8 && 2 * Z * WARPS <= chunks + WARPS - 1 && 2 * Z * likely * A.H <= per_sm * sms) Z *= 2;
        // (not where the last of several waves would leave more than a quarter of the CTAs' time unused: 64 users, 8 heads of
        // 64, 512 tiles on 444 places: 2000 keys 74 : 73, 4000 keys 119 : 129, E4M3 94 : 109; up to 1024 keys the second
        // launch costs more than that)
        const int64_t ctas = Z * likely * A.H, slots = (int64_t)per_sm * sms;
        if (chunks * KEYS <= 1024 || ctas <= slots || 4 * ctas >= 3 * ((ctas + slots - 1) / slots) * slots) {
            auto kernel = k_attn_few<QT, CT, D, CORE, false>;
            static std::atomic<uint64_t> done{0};
            e = allow_smem(kernel, most_smem, done);
            if (e != cudaSuccess) return e;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(tiles * Z), (unsigned)A.H);
            cfg.blockDim = dim3(32 * WARPS);
            cfg.dynamicSmemBytes = smem;
            cfg.stream = st;
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)Z;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaLaunchKernelEx(&cfg, kernel, A, parts);
            ++*launches;
            return e;
        }
    }
    auto kernel = k_attn_few<QT, CT, D, CORE, true>;
    static std::atomic<uint64_t> done{0};
    e = allow_smem(kernel, most_smem, done);
    if (e != cudaSuccess) return e;
    const int grid = std::min(per_sm * sms, SPLIT_CTAS);
    k_attn_few<QT, CT, D, CORE, true><<<grid, 32 * WARPS, smem, st>>>(A, parts);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
    cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)tiles, (unsigned)A.H, ROWS / JOIN_ROWS), dim3(32 * JOIN_ROWS), 0, st, attr);
    e = cudaLaunchKernelEx(&cfg, k_attn_join<QT, CT, D, CORE>, A, (const float *)parts, grid, C::SHIFT);
    ++*launches;
    return e;
}

template <int QT, int CT, bool CORE>
cudaError_t launch_d(const AttnArgs &A, void *workspace, int sms, cudaStream_t st, int *launches)
{
    if (A.D == 32) return launch<QT, CT, 32, CORE>(A, workspace, sms, st, launches);
    if (A.D == 64) return launch<QT, CT, 64, CORE>(A, workspace, sms, st, launches);
    return launch<QT, CT, 128, CORE>(A, workspace, sms, st, launches);
}

}  // namespace few

}  // namespace lsa
