// int4_mv.cuh -- products of a few tokens with a 4-bit weight that has one
// scale per group of input rows and output column,
//
//   y[t, n] = sum_k x[t, k] q[k, n] s[k / group, n],
//
// for the weights' layout of the layer: q [K, N / 2] bytes, two's-complement
// nibbles, the even column in the low one.  Used by the matrix-vector
// operator and by the layer's experts when their scales are grouped.
//
// With a handful of tokens the weight's bytes bound the product (one multiply
// per half byte and token), so every weight byte goes from global memory
// straight to the registers of the one warp that needs it, and the work per
// weight is kept small enough to run beside the loads:
//
// - mma.sync.m16n8k16 (f16 in, fp32 sums): weights as the 16-row operand, up
//   to 8 tokens as the 8 columns.  tcgen05 would take its weight operand from
//   shared memory, a round trip for widened weights that nothing is gained
//   from at 8 columns.
// - A thread holds 16 neighbouring columns of 8 neighbouring rows (an 8-byte
//   load per row, 64 bytes of a row per warp).  The operand wants pairs along
//   K, so two rows' words are interleaved by one byte permutation per four
//   columns, and each pair of nibbles is then one AND (with the sign bit
//   flipped) away: u = q + 8 in [0, 15] left where it lies in the f16's low
//   bits is the subnormal u 2^-24 (or 16 u 2^-24 one nibble up), exact in the
//   tensor core.  No conversion instruction, 0.75 per weight in all.
// - The bias 8 leaves through the sum's start value: each 32-row block starts
//   at -8 sum(x) (2^-24), from the tokens' block sums kept beside them.
// - The block's fp32 sum is multiplied by the group's scale and added to the
//   column's total in fp32: the weights are never rounded to a product.
// - Tokens are f16 in shared memory: f16 rows as they are, bf16 rows divided
//   by a power of two that brings the largest of the slice to [2^14, 2^15)
//   (exact for values down to 2^-31 of it, others round at 2^-39 of it).
//   A row with an infinity or a NaN gives NaN (inf times the bias).
//
// A CTA takes 256 columns (two groups of 128) and a slice of K, four warps of
// each column half on a quarter of the slice; the quarters are added through
// shared memory and the slices of a cluster through distributed shared
// memory, always in the same order.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "schedule.cuh"
#include "sm.cuh"

namespace l4moe {
namespace mv {

constexpr unsigned kErrF16Range = 1u << 4;  // DEV_ERR_F16_RANGE of the layer's error word

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCols = 256;       // columns of a CTA: two halves of 128
constexpr int kQuarters = 4;     // warps of a half, each on a quarter of a chunk
constexpr int kBlock = 32;       // rows of a block (scale groups are multiples of it)
constexpr int kChunk = 1024;     // rows of x staged at a time
constexpr int kXStride = kChunk + 32;  // halves; 64 bytes past a multiple of 128: the two
                                       // tokens of a quarter-warp's load use other banks

// A warp's ring of weight blocks: 8 bytes per row and lane, each lane's own,
// then the block's scales of the warp's 128 columns.
template <int NT8, typename ST>
struct Cfg {
    static constexpr int WORDS = 8 * 32 * 8;
    static constexpr int STAGE = WORDS + 128 * (int)sizeof(ST);
    // two CTAs per SM want at most 113 KB each
    static constexpr int STAGES = (NT8 == 2 && sizeof(ST) == 4) ? 3 : 4;
    static constexpr int X = (int)sizeof(__half) * NT8 * 8 * kXStride;
    static constexpr int BIAS = (int)sizeof(float) * (kChunk / kBlock) * NT8 * 8;
    static constexpr int RING = kWarps * STAGES * STAGE;
    static constexpr int RED = (int)sizeof(float) * kQuarters * NT8 * 8 * kCols;  // over all of it
    static constexpr int SMEM = X + BIAS + RING > RED ? X + BIAS + RING : RED;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1, float c0, float c1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mma_f16_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (x & mask) ^ flip in one instruction: two nibbles with their sign bit flipped.
__device__ __forceinline__ uint32_t and_xor(uint32_t x, uint32_t mask, uint32_t flip) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(x), "r"(mask), "r"(flip));
    return r;
}

// A weight matrix as a warp sees it.
template <typename ST>
struct Weight {
    const uint8_t* q;      // [K, row_bytes]
    const ST* s;           // [groups, N]
    long long row_bytes;   // N / 2
    int N;                 // columns of a row of scales
    int K, group;
};

// Issue one block's loads into a stage: this lane's 8 rows of 8 bytes (16
// columns), and its part of the scales of the warp's columns.  Rows past K
// and columns past the limit are zeros.  VEC: asynchronous copies (rows of a
// multiple of 16 columns); else plain loads, byte by byte.
template <typename ST, bool VEC>
__device__ __forceinline__ void issue_block(uint8_t* stage, const Weight<ST>& W, int row, int col, int limit, int lane) {
    const int t = lane & 3, g = lane >> 2;
    const int r0 = row + 8 * t;
    const ST* s = W.s + (long long)(row / W.group) * W.N;
    constexpr int WORDS = Cfg<1, ST>::WORDS;
    constexpr int SB = 4 * (int)sizeof(ST);  // scale bytes of a lane: 4 columns
    if constexpr (VEC) {
        const bool in = col < limit;
        const uint8_t* p = W.q + (in ? r0 * W.row_bytes + (col >> 1) : 0);
        const uint32_t dst = op::smem_u32(stage) + lane * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool ok = in && r0 + i < W.K;
            op::cp_async<8>(dst + i * 256, ok ? p + i * W.row_bytes : W.q, ok);
        }
        op::cp_async<SB>(op::smem_u32(stage) + WORDS + g * 16 * (int)sizeof(ST) + t * SB, in ? s + col + 4 * t : W.s, in);
    } else {
        const int nb = min(8, (limit - col + 1) >> 1);  // limit and col are even: whole bytes
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t lo = 0u, hi = 0u;
            if (r0 + i < W.K) {
                const uint8_t* p = W.q + (r0 + i) * W.row_bytes + (col >> 1);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (b < nb) lo |= (uint32_t)__ldg(p + b) << (8 * b);
                    if (4 + b < nb) hi |= (uint32_t)__ldg(p + 4 + b) << (8 * b);
                }
            }
            reinterpret_cast<uint2*>(stage)[i * 32 + lane] = make_uint2(lo, hi);
        }
        ST* d = reinterpret_cast<ST*>(stage + WORDS) + g * 16 + t * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = col + 4 * t + j;
            ST v;
            if (c < limit) v = s[c];
            else memset(&v, 0, sizeof v);
            d[j] = v;
        }
    }
}

// Column (of a thread's 16) that accumulator tile i holds in its first row
// (c0, c1); its second row (c2, c3) is two columns on.  Odd tiles hold 16
// times their sum.
__device__ __forceinline__ constexpr int tile_col(int i) { return (i >> 1) * 4 + (i & 1); }

// acc += one block: 32 rows of x (f16, xs + 8 t of this thread's token g) and
// this thread's words; bias: the block's -8 2^-24 sum(x) per token.
template <int NT8>
__device__ __forceinline__ void block_fma(float (&acc)[NT8][8][4], const uint2 (&w)[8], const float (&sc)[16],
                                          const __half* xs, const float* bias, int g, int t) {
    uint32_t b[NT8][4];
    float2 c0[NT8];
#pragma unroll
    for (int n = 0; n < NT8; ++n) {
        const uint4 v = *reinterpret_cast<const uint4*>(xs + (n * 8 + g) * kXStride + 8 * t);
        b[n][0] = v.x, b[n][1] = v.y, b[n][2] = v.z, b[n][3] = v.w;
        c0[n] = *reinterpret_cast<const float2*>(bias + n * 8 + 2 * t);
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // columns 4 h .. 4 h + 3: half (h & 1) of word h / 2
        uint32_t u[4];             // rows (0,1), (2,3), (4,5), (6,7) interleaved
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint32_t r0 = h < 2 ? w[2 * p].x : w[2 * p].y, r1 = h < 2 ? w[2 * p + 1].x : w[2 * p + 1].y;
            u[p] = __byte_perm(r0, r1, (h & 1) ? 0x7632 : 0x5410);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t mask = s ? 0x00f000f0u : 0x000f000fu, flip = s ? 0x00800080u : 0x00080008u;
            uint32_t a[8];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                a[2 * p] = and_xor(u[p], mask, flip);
                a[2 * p + 1] = and_xor(u[p] >> 8, mask, flip);
            }
            const float sa = sc[4 * h + s], sb = sc[4 * h + s + 2];
#pragma unroll
            for (int n = 0; n < NT8; ++n) {
                float d[4];
                const float k = s ? 16.f : 1.f;
                mma_f16(d, a[0], a[1], a[2], a[3], b[n][0], b[n][1], k * c0[n].x, k * c0[n].y);
                mma_f16_add(d, a[4], a[5], a[6], a[7], b[n][2], b[n][3]);
                float(&o)[4] = acc[n][2 * h + s];
                o[0] = fmaf(sa, d[0], o[0]);
                o[1] = fmaf(sa, d[1], o[1]);
                o[2] = fmaf(sb, d[2], o[2]);
                o[3] = fmaf(sb, d[3], o[3]);
            }
        }
    }
}

// The blocks a warp takes of a slice, in order: its quarter of every chunk.
struct Blocks {
    int row0, k1, quarter, b, b1;  // chunk's first row; block and end of the quarter

    __device__ __forceinline__ void start(int row) {
        row0 = row;
        const int nblk = (min(kChunk, k1 - row0) + kBlock - 1) / kBlock;
        b = nblk * quarter / kQuarters;
        b1 = nblk * (quarter + 1) / kQuarters;
    }
    __device__ __forceinline__ bool done() const { return row0 >= k1; }
    // to the next block that exists, chunk by chunk
    __device__ __forceinline__ void settle() {
        while (row0 < k1 && b >= b1) start(row0 + kChunk);
    }
    __device__ __forceinline__ void next() {
        ++b;
        settle();
    }
    __device__ __forceinline__ int row() const { return row0 + b * kBlock; }
};

// The f16 a value is staged as, and the power of two a bf16 row is
// multiplied with (f16 rows: 1).
__device__ __forceinline__ float row_factor(float amax) {
    if (!(amax > 0.f) || !(amax < INFINITY)) return 1.0f;
    const int e = (int)((__float_as_uint(amax) >> 23) & 0xffu) - 127;  // -127 for subnormals
    const int p = min(14 - e, 126);
    return __uint_as_float((uint32_t)(p + 127) << 23);
}

// Stage rows [row0, row0 + rows) of nt tokens (rows of x, ldx apart) as f16,
// zeros up to a whole number of blocks, and each block's bias.  bf16 rows are
// multiplied by factor[token]; where the chunk is the whole slice (own), the
// factor is found here.  A warp per token, 8 neighbouring values per lane.
// Tokens past nt are left as they are: a token is a column of the products,
// and what such columns hold reaches no other.
template <int NT8, typename XT>
__device__ __forceinline__ void stage_x(__half* xs, float* bias, const XT* x, long long ldx, int nt, int row0, int rows,
                                        float* factor, bool own) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int span = (rows + kBlock - 1) / kBlock * kBlock;
    const bool vec = (ldx & 7) == 0;  // rows (and so 8 values) start on 16 bytes
    constexpr int PASSES = kChunk / 256;
    for (int tok = warp; tok < nt; tok += kWarps) {
        const XT* xr = x + tok * ldx + row0;
        float v[PASSES][8];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int r = p * 256 + lane * 8;
            if (vec && r + 8 <= rows) {
                XT tmp[8];
                *reinterpret_cast<uint4*>(tmp) = *reinterpret_cast<const uint4*>(xr + r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[p][j] = to_f32(tmp[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[p][j] = r + j < rows ? to_f32(xr[r + j]) : 0.f;
            }
        }
        float f = 1.f;
        if constexpr (!std::is_same<XT, __half>::value) {
            if (own) {
                float m = 0.f;
#pragma unroll
                for (int p = 0; p < PASSES; ++p)
#pragma unroll
                    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[p][j]));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                f = row_factor(m);
                if (lane == 0) factor[tok] = f;
            } else {
                f = factor[tok];
            }
        }
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int r = p * 256 + lane * 8;
            __half2 h[4];
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = __floats2half2_rn(v[p][2 * j] * f, v[p][2 * j + 1] * f);
                const float2 b = __half22float2(h[j]);
                s += b.x + b.y;
            }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            if (r < span) {
                *reinterpret_cast<uint4*>(xs + tok * kXStride + r) = *reinterpret_cast<const uint4*>(h);
                if ((lane & 3) == 0) bias[(r / kBlock) * NT8 * 8 + tok] = s * -0x1p-21f;  // -8 2^-24
            }
        }
    }
}

// The sums of this CTA's slice [k0, k1) of K, left in smem as [token][256
// columns] fp32 (column c of half c / 128 is col0 + c or col1 + c - 128) for
// the nt tokens.  limit0 / limit1: the first column of each half that does
// not exist.  factor: smem, one per token; set by the caller for slices of
// more than one chunk of bf16 tokens.  before_x: called once the first
// weight loads are on their way, before x is read.
template <int NT8, typename XT, typename ST, bool VEC, typename F>
__device__ __forceinline__ void slice_sums(uint8_t* smem, const Weight<ST>& W, int col0, int limit0, int col1, int limit1,
                                           const XT* x, long long ldx, int nt, int k0, int k1, float* factor,
                                           F&& before_x) {
    using C = Cfg<NT8, ST>;
    __half* xs = reinterpret_cast<__half*>(smem);
    float* bias = reinterpret_cast<float*>(smem + C::X);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int half = warp & 1, quarter = warp >> 1;
    const int col = (half ? col1 : col0) + 16 * g, limit = half ? limit1 : limit0;
    uint8_t* ring = smem + C::X + C::BIAS + warp * (C::STAGES * C::STAGE);
    Blocks ahead{0, k1, quarter, 0, 0};  // the next block to load
    ahead.start(k0);
    ahead.settle();
    int put = 0, get = 0;
    auto issue = [&] {
        if (!ahead.done()) {
            issue_block<ST, VEC>(ring + put * C::STAGE, W, ahead.row(), col, limit, lane);
            ahead.next();
        }
        op::cp_commit();  // (an empty group where nothing is left keeps the count)
        put = put + 1 == C::STAGES ? 0 : put + 1;
    };
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) issue();
    before_x();
    float acc[NT8][8][4];
#pragma unroll
    for (int n = 0; n < NT8; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[n][i][c] = 0.f;
    const bool own = k1 - k0 <= kChunk;
    for (int row0 = k0; row0 < k1; row0 += kChunk) {
        if (row0 > k0) __syncthreads();  // the last chunk's x has been read
        stage_x<NT8>(xs, bias, x, ldx, nt, row0, min(kChunk, k1 - row0), factor, own);
        __syncthreads();
        Blocks cur{0, k1, quarter, 0, 0};
        cur.start(row0);
        for (int b = cur.b; b < cur.b1; ++b) {
            op::cp_wait<C::STAGES - 2>();
            __syncwarp();  // the scales are other lanes' copies
            const uint8_t* stage = ring + get * C::STAGE;
            get = get + 1 == C::STAGES ? 0 : get + 1;
            uint2 w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = reinterpret_cast<const uint2*>(stage)[i * 32 + lane];
            float sc[16];
            const ST* sp = reinterpret_cast<const ST*>(stage + C::WORDS) + g * 16;
            constexpr int V = 16 / (int)sizeof(ST);
#pragma unroll
            for (int i = 0; i < 16 / V; ++i) {
                ST tmp[V];
                *reinterpret_cast<uint4*>(tmp) = reinterpret_cast<const uint4*>(sp)[i];
#pragma unroll
                for (int j = 0; j < V; ++j) sc[i * V + j] = to_f32(tmp[j]);
            }
            __syncwarp();  // every lane has read the stage that the next copies overwrite one turn on
            issue();
            block_fma<NT8>(acc, w, sc, xs + b * kBlock, bias + b * NT8 * 8, g, t);
        }
    }
    op::cp_wait<0>();
    __syncthreads();
    // the quarters' sums, in their order
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int n = 0; n < NT8; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int tok = n * 8 + 2 * t + (c & 1), f = half * 128 + 16 * g + tile_col(i) + (c & 2);
                if (tok < nt)
                    red[(quarter * NT8 * 8 + tok) * kCols + f] = acc[n][i][c] * ((i & 1) ? 0x1p20f : 0x1p24f);
            }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * kCols; i += kThreads) {
        float v = red[i];
#pragma unroll
        for (int q = 1; q < kQuarters; ++q) v += red[q * NT8 * 8 * kCols + i];
        if constexpr (!std::is_same<XT, __half>::value) v *= 1.0f / factor[i / kCols];
        red[i] = v;  // read and written by this thread alone
    }
}

// Sum over the cluster's slices of smem float i, slice order.
__device__ __forceinline__ float cluster_total(const float* red, int i, int slices) {
    if (slices == 1) return red[i];
    const uint32_t at = op::smem_u32(red + i);
    float v = 0.f;
    for (int r = 0; r < slices; ++r) v += op::ld_cluster_f32(op::mapa(at, (uint32_t)r));
    return v;
}

// Each token's largest magnitude over a slice -> factor (bf16 tokens).
template <typename XT>
__device__ __forceinline__ void slice_factors(float* factor, const XT* x, long long ldx, int nt, int k0, int k1) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int tok = warp; tok < nt; tok += kThreads / 32) {
        float m = 0.f;
        for (int k = k0 + lane; k < k1; k += 32) {
            m = fmaxf(m, fabsf(to_f32(x[tok * ldx + k])));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) factor[tok] = row_factor(m);
    }
}

// Rows [k0, k1) of slice r of S: whole blocks, as even as they come.
__host__ __device__ __forceinline__ int slice_row(int K, int r, int S) {
    const int blocks = (K + kBlock - 1) / kBlock;
    const int k = (int)((long long)blocks * r / S) * kBlock;
    return k < K ? k : K;
}

// Slices of K for a launch of `tiles` tiles: enough CTAs for two on every SM
// (what their registers and shared memory allow), a block at least for each
// quarter, at most a portable cluster.
__host__ __forceinline__ int slices(long long tiles, int K, int sms) {
    const int blocks = (K + kBlock - 1) / kBlock;
    int S = 1;
    while (S < 8 && tiles * S < 2LL * sms && blocks >= 2 * S * kQuarters) S *= 2;
    return S;
}

// ------------------------------------------------------------ the operator
// y [T, N] = x [T, K] W.  Grid: (column tiles, token tiles, slices), the
// slices of a tile one cluster.
template <int NT8, typename XT, typename ST, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) int4_matvec_kernel(const XT* __restrict__ x, int T, Weight<ST> W,
                                                               XT* __restrict__ y) {
    op::pdl_enter();
    extern __shared__ __align__(16) uint8_t mv_smem[];
    __shared__ float factor[NT8 * 8];
    const int S = gridDim.z, slice = blockIdx.z;
    const int col0 = blockIdx.x * kCols;
    const int t0 = blockIdx.y * NT8 * 8, nt = min(NT8 * 8, T - t0);
    const int k0 = slice_row(W.K, slice, S), k1 = slice_row(W.K, slice + 1, S);
    const XT* xt = x + (long long)t0 * W.K;
    slice_sums<NT8, XT, ST, VEC>(mv_smem, W, col0, W.N, col0 + 128, W.N, xt, W.K, nt, k0, k1, factor, [&] {
        if constexpr (!std::is_same<XT, __half>::value) {
            if (k1 - k0 > kChunk) {  // several chunks share one factor
                slice_factors(factor, xt, W.K, nt, k0, k1);
                __syncthreads();
            }
        }
    });
    float* red = reinterpret_cast<float*>(mv_smem);
    if (S > 1) op::cluster_sync();
    else __syncthreads();
    const int items = nt * kCols;
    const int i0 = (int)((long long)items * slice / S), i1 = (int)((long long)items * (slice + 1) / S);
    for (int i = i0 + threadIdx.x; i < i1; i += kThreads) {
        const int tok = i / kCols, n = col0 + i % kCols;
        if (n >= W.N) continue;
        const float v = cluster_total(red, i, S);
        XT* o = y + (long long)(t0 + tok) * W.N + n;
        if constexpr (std::is_same<XT, __half>::value) *o = __float2half_rn(v);
        else *o = __float2bfloat16_rn(v);
    }
    if (S > 1) op::cluster_sync();  // the sums stay until every CTA of the cluster has read them
}

// ----------------------------------------------------------- the layer's experts
// The codes and scales of every expert and of the shared one (index E), by
// value: the launch carries them, so there is no table to upload or to keep.
struct Experts {
    const uint8_t* q[kMaxGroups];
    const void* s[kMaxGroups];
};

// A launch's rows and outputs for its routed experts and the shared one.
struct Rows {
    const __half* x[2];      // operand rows: routed (slot order), shared (token order)
    int K[2], N[2];          // the weights' rows and columns
    const float* scale[2];   // gate/up: what multiplies a row's sums (null: 1)
    __half* h[2];            // gate/up: hidden rows [., N / 2]
    float* part[2];          // down: fp32 rows [., N], routed at the row's entry (perm)
    const int32_t* perm;
    unsigned* err;
};

// Which group and rows unit u of the work list is: units are the groups'
// tiles of 8 rows, in the list's order.  All threads; false past the list.
__device__ __forceinline__ bool find_unit(const GroupTable* tab, int u, int& group, int& row) {
    __shared__ int s_group, s_row;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x, n = tab->num_groups;
        int base = 0, found = -1, at = 0;
        for (int g0 = 0; g0 < n && found < 0; g0 += 32) {
            const int tiles = g0 + lane < n ? (tab->rows[g0 + lane] + 7) >> 3 : 0;
            int incl = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const bool here = u < base + incl && u >= base + incl - tiles;
            const unsigned who = __ballot_sync(0xffffffffu, here);
            if (who) {
                const int l = __ffs(who) - 1;
                found = g0 + l;
                at = u - base - __shfl_sync(0xffffffffu, incl - tiles, l);
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            s_group = found;
            s_row = at * 8;
        }
    }
    __syncthreads();
    group = s_group;
    row = s_row;
    return group >= 0;
}

// Gate/up: h = silu(c a_gate) (c a_up), c the row's scale (its sigmoid gate).
// Down: the fp32 sums, un-permuted.  Grid: (column tiles, units, slices); a
// gate/up tile is 128 hidden columns (gate in the first half, up in the
// second), a down tile 256 columns.
template <typename ST, bool GATE_UP>
__global__ void __launch_bounds__(kThreads, 2) experts_kernel(const GroupTable* tab, int num_experts, int group_rows,
                                                           const __grid_constant__ Experts E, const Rows R) {
    op::pdl_enter();
    extern __shared__ __align__(16) uint8_t mv_smem[];
    int grp, row;
    if (!find_unit(tab, blockIdx.y, grp, row)) return;
    const int expert = tab->expert[grp], sh = expert == num_experts ? 1 : 0;
    const int nt = min(8, tab->rows[grp] - row), row0 = tab->row0[grp] + row;
    const int K = R.K[sh], N = R.N[sh];
    const int F = N / 2;
    const int col0 = blockIdx.x * (GATE_UP ? 128 : kCols);
    if (col0 >= (GATE_UP ? F : N)) return;
    const int S = gridDim.z, slice = blockIdx.z;
    const int k0 = slice_row(K, slice, S), k1 = slice_row(K, slice + 1, S);
    const Weight<ST> W{E.q[expert], static_cast<const ST*>(E.s[expert]), N / 2, N, K, group_rows};
    slice_sums<1, __half, ST, true>(mv_smem, W, col0, GATE_UP ? F : N, GATE_UP ? F + col0 : col0 + 128, N,
                                    R.x[sh] + (long long)row0 * K, K, nt, k0, k1, nullptr, [] {});
    const float* red = reinterpret_cast<const float*>(mv_smem);
    if (S > 1) op::cluster_sync();
    else __syncthreads();
    const int width = GATE_UP ? 128 : kCols, items = nt * width;
    const int i0 = (int)((long long)items * slice / S), i1 = (int)((long long)items * (slice + 1) / S);
    for (int i = i0 + threadIdx.x; i < i1; i += kThreads) {
        const int tok = i / width, c = i % width;
        if (GATE_UP) {
            if (col0 + c >= F) continue;
            const float g = R.scale[sh] ? R.scale[sh][row0 + tok] : 1.0f;
            const float a = g * cluster_total(red, tok * kCols + c, S), b = g * cluster_total(red, tok * kCols + 128 + c, S);
            const float hv = __fdividef(a, 1.0f + __expf(-a)) * b;
            if (!(fabsf(hv) < 65520.0f)) atomicOr(R.err, kErrF16Range);  // rounds to infinity in f16
            R.h[sh][(long long)(row0 + tok) * F + col0 + c] = __float2half_rn(hv);
        } else {
            if (col0 + c >= N) continue;
            const int orow = sh ? row0 + tok : R.perm[row0 + tok];
            R.part[sh][(long long)orow * N + col0 + c] = cluster_total(red, i, S);
        }
    }
    if (S > 1) op::cluster_sync();
}

}  // namespace mv
}  // namespace l4moe
