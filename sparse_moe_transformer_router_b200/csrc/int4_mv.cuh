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
//   by a power of two that brings the largest of a quarter slice to [2^14, 2^15)
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
constexpr int kQuarters = 4;     // warps of a half, each on a quarter of the slice
constexpr int kBlock = 32;       // rows of a block (scale groups are multiples of it)
constexpr int kPiece = 512;      // rows of x a quarter stages at a time
constexpr int kXStride = kPiece + 32;  // halves; 64 bytes past a multiple of 128: the two
                                       // tokens of a quarter-warp's load use other banks

// A warp's ring of weight blocks: 32 rows of 64 bytes (its 128 columns), then
// their scales.  Each quarter has its part of x and of the block sums.
template <int NT8, typename ST>
struct Cfg {
    static constexpr int WORDS = kBlock * 64;
    static constexpr int STAGE = WORDS + 128 * (int)sizeof(ST);
    // up to 8 tokens two CTAs share an SM (128 registers a thread, 113 KB
    // each); for 16 tokens the sums alone take 64, and one CTA has it
    static constexpr int PER_SM = NT8 == 1 ? 2 : 1;
    static constexpr int STAGES = NT8 == 1 ? 4 : 6;
    static constexpr int X = (int)sizeof(__half) * NT8 * 8 * kXStride;       // of a quarter
    static constexpr int BIAS = (int)sizeof(float) * (kPiece / kBlock) * NT8 * 8;
    static constexpr int RING = kWarps * STAGES * STAGE;
    static constexpr int RED = (int)sizeof(float) * kQuarters * NT8 * 8 * kCols;  // over all of it
    static constexpr int USED = kQuarters * (X + BIAS) + RING;
    static constexpr int SMEM = USED > RED ? USED : RED;
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

// Where a stage holds the 8 bytes of columns 16 g .. 16 g + 15 of row 8 t + i:
// two rows to a 128-byte line, so that the 16 lanes of half a warp (4 values
// of g, 4 of t) read 32 different banks.
__device__ __forceinline__ int word_at(int i, int g, int t) {
    return ((t >> 1) * 8 + i) * 128 + (t & 1) * 64 + ((((g >> 1) ^ (t & 2)) & 3) << 4) + (g & 1) * 8;
}

// A weight matrix's blocks as one lane loads them.  VEC (rows of a multiple
// of 32 columns): asynchronous 16-byte copies, lane l 16 bytes of rows l / 4,
// l / 4 + 8, ... and its four columns' scales; else plain loads of the lane's
// own words, byte by byte.  What lies past K or past the columns' limit is
// not loaded: x is zero there and such columns are not stored, and no nibble
// is an infinity or a NaN.
template <typename ST, bool VEC>
struct Loader {
    const uint8_t* q;     // VEC: this lane's 16 bytes of row 0; else the matrix
    const ST* s;          // this lane's 4 scales of the current group (VEC), or of row 0's columns
    long long row_bytes;
    int N, K, group, col, limit;
    int row, end;         // next block's row, end of the quarter
    int left;             // rows until the next group
    bool fresh;           // the next block is this warp's first of its group

    __device__ __forceinline__ void start(const Weight<ST>& W, int c0, int lim, int r0, int r1, int lane) {
        row_bytes = W.row_bytes, N = W.N, K = W.K, group = W.group;
        row = r0, end = r1, limit = lim;
        const int grp = r0 / group;
        left = group - (r0 - grp * group);
        fresh = true;
        if constexpr (VEC) {
            col = c0 + (lane & 3) * 32;
            q = W.q + (long long)(r0 + (lane >> 2)) * row_bytes + (col >> 1);
            s = W.s + (long long)grp * N + c0 + lane * 4;
            limit = lim - c0;
        } else {
            col = c0 + 16 * (lane >> 2);
            q = W.q;
            s = W.s + (long long)grp * N;
        }
    }
    __device__ __forceinline__ void issue(uint8_t* stage, int lane) {
        constexpr int WORDS = Cfg<1, ST>::WORDS;
        if constexpr (VEC) {
            const uint32_t base = op::smem_u32(stage);
            if ((lane & 3) * 32 < limit) {
                const uint32_t dst = base + (lane >> 2) * 128 + (lane & 3) * 16;
                const uint8_t* p = q;
                const bool whole = row + kBlock <= K;
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // t = i: line half i & 1, lines from (i / 2) 8, chunks swapped by i & 2
                    if (whole || row + i * 8 + (lane >> 2) < K)
                        op::cp_async<16>((dst + (i >> 1) * 1024 + (i & 1) * 64) ^ ((i & 2) * 16), p);
                    p += 8 * row_bytes;
                }
            }
            if (fresh && lane * 4 < limit)
                op::cp_async<4 * (int)sizeof(ST)>(base + WORDS + lane * 4 * (int)sizeof(ST), s);
            q += kBlock * row_bytes;
        } else {
            const int t = lane & 3, g = lane >> 2;
            const int nb = min(8, (limit - col + 1) >> 1);  // limit and col are even: whole bytes
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t lo = 0u, hi = 0u;
                if (row + 8 * t + i < K) {
                    const uint8_t* p = q + (row + 8 * t + i) * row_bytes + (col >> 1);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (b < nb) lo |= (uint32_t)__ldg(p + b) << (8 * b);
                        if (4 + b < nb) hi |= (uint32_t)__ldg(p + 4 + b) << (8 * b);
                    }
                }
                *reinterpret_cast<uint2*>(stage + word_at(i, g, t)) = make_uint2(lo, hi);
            }
            ST* d = reinterpret_cast<ST*>(stage + WORDS) + g * 16 + t * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (fresh && col + 4 * t + j < limit) d[j] = s[col + 4 * t + j];
        }
        row += kBlock;
        left -= kBlock;
        fresh = left == 0;
        if (fresh) {
            left = group;
            s += N;
        }
    }
};

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
// multiplied by factor[token]; where the piece is all of the quarter (own),
// the factor is found here.  The quarter's two warps (half = 0, 1) take the
// tokens in turn, 8 neighbouring values per lane.  Tokens past nt are left as
// they are: a token is a column of the products, and what such a column holds
// reaches no other.
template <int NT8, typename XT>
__device__ __forceinline__ void stage_x(__half* xs, float* bias, const XT* x, long long ldx, int nt, int row0, int rows,
                                        float* factor, bool own, int half, int lane) {
    const int span = (rows + kBlock - 1) / kBlock * kBlock;
    const bool vec = (ldx & 7) == 0;  // rows (and so 8 values) start on 16 bytes
    constexpr int PASSES = kPiece / 256;
#pragma unroll 2
    for (int tok = half; tok < nt; tok += 2) {
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

// Each token's factor over rows [r0, r1) (bf16 tokens, more than one piece).
template <typename XT>
__device__ __forceinline__ void find_factors(float* factor, const XT* x, long long ldx, int nt, int r0, int r1, int half,
                                             int lane) {
    for (int tok = half; tok < nt; tok += 2) {
        float m = 0.f;
#pragma unroll 8
        for (int k = r0 + lane; k < r1; k += 32) m = fmaxf(m, fabsf(to_f32(x[tok * ldx + k])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) factor[tok] = row_factor(m);
    }
}

// The sums of this CTA's slice [k0, k1) of K, left in smem as [token][256
// columns] fp32 (column c of half c / 128 is col0 + c or col1 + c - 128) for
// the nt tokens.  limit0 / limit1: the first column of each half that does
// not exist.  before_x: called once the first weight loads are on their way,
// before x is read.
template <int NT8, typename XT, typename ST, bool VEC, typename F>
__device__ __forceinline__ void slice_sums(uint8_t* smem, const Weight<ST>& W, int col0, int limit0, int col1, int limit1,
                                           const XT* x, long long ldx, int nt, int k0, int k1, F&& before_x) {
    using C = Cfg<NT8, ST>;
    constexpr bool BF = !std::is_same<XT, __half>::value;
    __shared__ float s_factor[kQuarters][NT8 * 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int half = warp & 1, quarter = warp >> 1;
    __half* xs = reinterpret_cast<__half*>(smem + quarter * (C::X + C::BIAS));
    float* bias = reinterpret_cast<float*>(smem + quarter * (C::X + C::BIAS) + C::X);
    uint8_t* ring = smem + kQuarters * (C::X + C::BIAS) + warp * (C::STAGES * C::STAGE);
    const int nblk = (k1 - k0 + kBlock - 1) / kBlock;
    const int r0 = k0 + nblk * quarter / kQuarters * kBlock;
    const int r1 = min(k1, k0 + nblk * (quarter + 1) / kQuarters * kBlock);
    Loader<ST, VEC> ld;
    ld.start(W, half ? col1 : col0, half ? limit1 : limit0, r0, r1, lane);
    int put = 0, get = 0;
    auto issue = [&] {
        if (ld.row < r1) ld.issue(ring + put * C::STAGE, lane);
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
    const bool own = r1 - r0 <= kPiece;
    if (BF && !own) find_factors(s_factor[quarter], x, ldx, nt, r0, r1, half, lane);  // (a token's warp reads it back)
    const int words = word_at(0, g, t);
    float sc[16];
    int left = 0;  // rows that the scales at hand still cover
    for (int row0 = r0; row0 < r1; row0 += kPiece) {
        const int rows = min(kPiece, r1 - row0);
        if (row0 > r0) op::pair_sync(1 + quarter);  // the last piece of x has been read
        else __syncwarp();
        stage_x<NT8>(xs, bias, x, ldx, nt, row0, rows, s_factor[quarter], own, half, lane);
        op::pair_sync(1 + quarter);
        for (int b = 0; b * kBlock < rows; ++b) {
            op::cp_wait<C::STAGES - 2>();
            __syncwarp();  // the copies are other lanes'
            const uint8_t* stage = ring + get * C::STAGE;
            get = get + 1 == C::STAGES ? 0 : get + 1;
            uint2 w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint2*>(stage + words + i * 128);
            if (left == 0) {  // a group's first block brings its scales
                const ST* sp = reinterpret_cast<const ST*>(stage + C::WORDS) + g * 16;
                constexpr int V = 16 / (int)sizeof(ST);
#pragma unroll
                for (int i = 0; i < 16 / V; ++i) {
                    ST tmp[V];
                    *reinterpret_cast<uint4*>(tmp) = reinterpret_cast<const uint4*>(sp)[i];
#pragma unroll
                    for (int j = 0; j < V; ++j) sc[i * V + j] = to_f32(tmp[j]);
                }
                left = W.group - (row0 + b * kBlock) % W.group;
            }
            left -= kBlock;
            // (the copies issued here go to the stage read one turn ago: every
            // lane has passed this turn's __syncwarp since)
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
        for (int c = 0; c < 4; ++c) {
            const int tok = n * 8 + 2 * t + (c & 1);
            if (tok < nt) {
                const float f = BF && r0 < r1 ? 1.0f / s_factor[quarter][tok] : 1.0f;
                float* o = red + (quarter * NT8 * 8 + tok) * kCols + half * 128 + 16 * g + (c & 2);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[tile_col(i)] = acc[n][i][c] * ((i & 1) ? 0x1p20f : 0x1p24f) * f;
            }
        }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * kCols; i += kThreads) {
        float v = red[i];
#pragma unroll
        for (int q = 1; q < kQuarters; ++q) v += red[q * NT8 * 8 * kCols + i];
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

// First row of slice r of 2^lg: whole blocks, as even as they come.
__host__ __device__ __forceinline__ int slice_row(int K, int r, int lg) {
    const int blocks = (K + kBlock - 1) / kBlock;  // K <= 2^30: blocks * 8 fits
    const int k = ((blocks * r) >> lg) * kBlock;
    return k < K ? k : K;
}

// Slices of K (a power of two) for a launch of `tiles` tiles: a CTA for every
// SM, a block at least for each quarter, at most a portable cluster.
__host__ __forceinline__ int slices(long long tiles, int K, int sms) {
    const int blocks = (K + kBlock - 1) / kBlock;
    int S = 1;
    while (S < 8 && tiles * S < sms && blocks >= 2 * S * kQuarters) S *= 2;
    return S;
}

// ------------------------------------------------------------ the operator
// y [T, N] = x [T, K] W.  Grid: (column tiles, token tiles, slices), the
// slices of a tile one cluster.
template <int NT8, typename XT, typename ST, bool VEC>
__global__ void __launch_bounds__(kThreads, Cfg<NT8, ST>::PER_SM) int4_matvec_kernel(const XT* __restrict__ x, int T, Weight<ST> W,
                                                               XT* __restrict__ y) {
    op::pdl_enter();
    extern __shared__ __align__(128) uint8_t mv_smem[];
    const int S = gridDim.z, slice = blockIdx.z, lg = __ffs(S) - 1;
    const int col0 = blockIdx.x * kCols;
    const int t0 = blockIdx.y * NT8 * 8, nt = min(NT8 * 8, T - t0);
    const int k0 = slice_row(W.K, slice, lg), k1 = slice_row(W.K, slice + 1, lg);
    const XT* xt = x + (long long)t0 * W.K;
    slice_sums<NT8, XT, ST, VEC>(mv_smem, W, col0, W.N, col0 + 128, W.N, xt, W.K, nt, k0, k1, [] {});
    float* red = reinterpret_cast<float*>(mv_smem);
    if (S > 1) op::cluster_sync();
    else __syncthreads();
    const int items = nt * kCols;
    const int i0 = (items >> lg) * slice, i1 = i0 + (items >> lg);  // items is a multiple of 8
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
    extern __shared__ __align__(128) uint8_t mv_smem[];
    int grp, row;
    if (!find_unit(tab, blockIdx.y, grp, row)) return;
    const int expert = tab->expert[grp], sh = expert == num_experts ? 1 : 0;
    const int nt = min(8, tab->rows[grp] - row), row0 = tab->row0[grp] + row;
    const int K = R.K[sh], N = R.N[sh];
    const int F = N / 2;
    const int col0 = blockIdx.x * (GATE_UP ? 128 : kCols);
    if (col0 >= (GATE_UP ? F : N)) return;
    const int S = gridDim.z, slice = blockIdx.z, lg = __ffs(S) - 1;
    const int k0 = slice_row(K, slice, lg), k1 = slice_row(K, slice + 1, lg);
    const Weight<ST> W{E.q[expert], static_cast<const ST*>(E.s[expert]), N / 2, N, K, group_rows};
    slice_sums<1, __half, ST, true>(mv_smem, W, col0, GATE_UP ? F : N, GATE_UP ? F + col0 : col0 + 128, N,
                                    R.x[sh] + (long long)row0 * K, K, nt, k0, k1, [] {});
    const float* red = reinterpret_cast<const float*>(mv_smem);
    if (S > 1) op::cluster_sync();
    else __syncthreads();
    const int width = GATE_UP ? 128 : kCols, items = nt * width;
    const int i0 = (items >> lg) * slice, i1 = i0 + (items >> lg);  // items is a multiple of 8
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
