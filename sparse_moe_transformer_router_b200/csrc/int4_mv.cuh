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
// per half byte and token), so every weight byte is read once, by the one
// warp that needs it, and the work per weight is kept small enough to run
// beside the loads:
//
// - mma.sync.m16n8k16 (f16 in, fp32 sums): weights as the 16-row operand, up
//   to 8 tokens as the 8 columns.  tcgen05 would take its weight operand from
//   shared memory, a round trip for widened weights that nothing is gained
//   from at 8 columns.
// - A warp takes blocks of 32 rows by 128 columns through a ring of its own
//   in shared memory, filled by asynchronous 16-byte copies.  The operand
//   wants pairs along K: a transposing matrix load of 16-bit units, four
//   columns each, returns two rows' units in one register.  Each pair of
//   nibbles is then one AND (with the sign bit flipped) away: u = q + 8 in
//   [0, 15] left where it lies in the f16's low bits is the subnormal u 2^-24
//   (or 16 u 2^-24 one nibble up), exact in the tensor core.  No conversion
//   instruction, 0.625 per weight in all.
// - The bias 8 leaves as -8 sum(x) (2^-24) times the group's scale, once for
//   each run of a group's blocks; the sums are two products with a constant.
// - The block's fp32 sum is multiplied by the group's scale and added to the
//   column's total in fp32: the weights are never rounded to a product.
// - Tokens come along in the ring, f16 rows as they are, bf16 rows divided (on
//   their way to the product) by a power of two that brings the largest of a
//   warp's rows to [2^14, 2^15)
//   (exact for values down to 2^-31 of it, others round at 2^-39 of it).
//   A row with an infinity or a NaN gives NaN (inf times the bias).
//
// A CTA of four warps takes 128 columns and a slice of K, each warp a quarter
// of the slice; the quarters are added through shared memory and the slices
// of a cluster through distributed shared memory, always in the same order.
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

constexpr int kWarps = 4;        // of a CTA, each on a quarter of the CTA's slice of K
constexpr int kThreads = 32 * kWarps;
constexpr int kCols = 128;       // columns of a CTA: two halves of 64
constexpr int kHalf = kCols / 2;
constexpr int kBlock = 32;       // rows of a block (scale groups are multiples of it)

// A warp's ring of blocks: 32 rows of 64 bytes of the weight, the scales of
// the columns, 64 bytes (32 rows) of each token.
template <int NT8, typename ST>
struct Cfg {
    static constexpr int WORDS = kBlock * 64;
    static constexpr int XOFF = WORDS + kCols * (int)sizeof(ST);
    static constexpr int STAGE = XOFF + NT8 * 8 * 64;
    static constexpr int STAGES = 4;
    static constexpr int RING = STAGES * STAGE;
    // CTAs that share an SM: the registers' limit (up to 8 tokens 128 a
    // thread, 16 tokens 168)
    static constexpr int PER_SM = NT8 == 1 ? 4 : 3;
    static constexpr int RED = (int)sizeof(float) * kWarps * NT8 * 8 * kCols;  // over all of it
    static constexpr int SMEM = kWarps * RING > RED ? kWarps * RING : RED;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

// Where a stage holds the 16 bytes of columns 32 c .. 32 c + 31 of row r (or of
// rows 8 c .. 8 c + 7 of token r): the eight rows of a matrix load lie in
// different banks.
__device__ __forceinline__ constexpr int chunk_at(int r, int c) { return r * 64 + ((c ^ ((r >> 1) & 3)) << 4); }

// The 128 columns of a CTA: two runs of 64, each with the first column that
// does not exist.
struct Columns {
    int col0, col1, limit0, limit1;
    __device__ __forceinline__ int first(int second) const { return second ? col1 : col0; }
    __device__ __forceinline__ int end(int second) const { return second ? limit1 : limit0; }
};

// A weight matrix's blocks as one lane loads them.  VEC (rows of a multiple
// of 32 columns): asynchronous 16-byte copies, lane l 16 bytes of rows l / 4,
// l / 4 + 8, ... and its four columns' scales; else plain loads, byte by
// byte.  What lies past K or past the columns' limit is not loaded: x is zero
// there and such columns are not stored, and no nibble is an infinity or a
// NaN.
template <typename ST, bool VEC>
struct Loader {
    const uint8_t* q;     // VEC: this lane's 16 bytes of its first row; else this lane's row
    const ST* s;          // VEC: this lane's 4 scales of the next block; else the row of scales
    long long row_bytes;
    int N, group;
    int left;             // rows until the next group
    int rows;             // rows of K left from the next block on
    bool in, in_s;        // VEC: this lane's columns exist

    __device__ __forceinline__ void start(const Weight<ST>& W, const Columns& C, int row, int lane) {
        row_bytes = W.row_bytes, N = W.N, group = W.group;
        const int grp = row / group;
        left = 0;
        first = group - (row - grp * group);
        rows = W.K - row;
        s = W.s + (long long)grp * N;
        if constexpr (VEC) {
            const int col = C.first(lane & 2) + (lane & 1) * 32;
            in = col < C.end(lane & 2);
            q = W.q + (long long)(row + (lane >> 2)) * row_bytes + (col >> 1);
            const int cs = C.first(lane & 16) + (lane & 15) * 4;
            in_s = cs < C.end(lane & 16);
            s += cs;
        } else {
            q = W.q + (long long)(row + lane) * row_bytes;
        }
    }
    int first;            // rows until the first change of group
    __device__ __forceinline__ void issue(uint32_t stage, uint8_t* generic, const Columns& C, int lane) {
        constexpr int WORDS = Cfg<1, ST>::WORDS;
        const bool fresh = left == 0;  // this warp's first block of its group: its scales too
        if constexpr (VEC) {
            const uint32_t dst = stage + chunk_at(lane >> 2, lane & 3);
            const long long step = 8 * row_bytes;
            const uint8_t *p1 = q + step, *p2 = p1 + step, *p3 = p2 + step;
            if (in) {
                if (rows >= kBlock) {
                    op::cp_async<16>(dst, q);
                    op::cp_async<16>(dst + 512, p1);
                    op::cp_async<16>(dst + 1024, p2);
                    op::cp_async<16>(dst + 1536, p3);
                } else {
                    const int n = rows - (lane >> 2);
                    if (n > 0) op::cp_async<16>(dst, q);
                    if (n > 8) op::cp_async<16>(dst + 512, p1);
                    if (n > 16) op::cp_async<16>(dst + 1024, p2);
                    if (n > 24) op::cp_async<16>(dst + 1536, p3);
                }
            }
            q = p3 + step;
            if (fresh && in_s) op::cp_async<4 * (int)sizeof(ST)>(stage + WORDS + lane * 4 * (int)sizeof(ST), s);
        } else {
            if (lane < rows) {  // the 64 bytes of the lane's row; col and limit are even: whole bytes
                for (int c = 0; c < 4; ++c) {
                    const int col = C.first(c & 2) + (c & 1) * 32;
                    const int nb = min(16, (C.end(c & 2) - col) >> 1);
                    const uint8_t* p = q + (col >> 1);
                    uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int b = 0; b < 16; ++b)
                        if (b < nb) v[b >> 2] |= (uint32_t)__ldg(p + b) << (8 * (b & 3));
                    *reinterpret_cast<uint4*>(generic + chunk_at(lane, c)) = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
            q += kBlock * row_bytes;
            ST* d = reinterpret_cast<ST*>(generic + WORDS) + lane * 4;
            const int cs = C.first(lane & 16) + (lane & 15) * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (fresh && cs + j < C.end(lane & 16)) d[j] = s[cs + j];
        }
        rows -= kBlock;
        if (fresh) left = first, first = group;
        left -= kBlock;
        if (left == 0) s += N;
    }
};

// The token rows of a CTA: rows of x, ld apart, from row0 on, or those that
// slot row0 + token of perm names (entry / k).
template <typename XT>
struct Tokens {
    const XT* x;
    long long ld;
    int row0;
    const int32_t* perm;
    int k;
    __device__ __forceinline__ const XT* row(int token) const {
        const int r = perm ? perm[row0 + token] / k : row0 + token;
        return x + r * ld;
    }
};

// The tokens' rows as one lane loads them: 8 values (16 bytes) of tokens
// l / 4, l / 4 + 8.  Rows past the slice's end are zeros; tokens past nt are
// not loaded (a token is a column of the products, and what such a column
// holds reaches no other).
template <int NT8, typename XT>
struct XLoader {
    const XT* x[NT8];  // this lane's 8 values of tokens l / 4, l / 4 + 8 in the next block
    int rows;          // rows left from this lane's on
    bool vec;          // rows (and so 8 values) start on 16 bytes

    __device__ __forceinline__ void start(const Tokens<XT>& X, int nt, int row, int end, int lane) {
        vec = (X.ld & 7) == 0;
#pragma unroll
        for (int n = 0; n < NT8; ++n) {
            const int tok = n * 8 + (lane >> 2);
            x[n] = X.row(tok < nt ? tok : 0) + row + (lane & 3) * 8;
        }
        rows = end - row - (lane & 3) * 8;
    }
    __device__ __forceinline__ void issue(uint32_t at, uint8_t* generic, int nt, int lane) {
#pragma unroll
        for (int n = 0; n < NT8; ++n) {
            const int off = n * 8 * 64 + chunk_at(lane >> 2, lane & 3);
            if ((lane >> 2) + 8 * n < nt) {
                const XT* p = x[n];
                if (vec) {
                    op::cp_async16_zero(at + off, p, rows > 0);  // 8 values or none: rows of a multiple of 8
                } else {
                    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < rows) w[j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[j] << (16 * (j & 1));
                    *reinterpret_cast<uint4*>(generic + off) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            x[n] += kBlock;
        }
        rows -= kBlock;
    }
};

// Column (of the warp's 128) that accumulator tile i of lane group g holds in
// its first row (c0, c1); its second row (c2, c3) is two columns on.  Odd
// tiles hold 16 times their sum.
__device__ __forceinline__ constexpr int tile_col(int i, int g) { return (i >> 1) * 32 + 4 * g + (i & 1); }

// acc += one block: the warp's stage (rows_at: this lane's address of a matrix
// load of the weight, x_at: of the tokens); sc: the scales of the lane's
// columns; f: what the lane's tokens (column l / 4 of each 8) are multiplied
// with as they become f16.  b8 += -8 2^-24 sum(x) of the lane's two tokens: a
// product with rows of that constant (an f16 subnormal).
template <int NT8, bool BF>
__device__ __forceinline__ void block_fma(float (&acc)[NT8][8][4], float (&b8)[NT8][4], uint32_t rows_at, uint32_t x_at,
                                          const float (&sc)[16], const float (&f)[NT8]) {
    constexpr uint32_t kMinus8 = 0x80088008u;
    uint32_t b[NT8][4];
#pragma unroll
    for (int n = 0; n < NT8; ++n) {
        op::ldmatrix(b[n], x_at + n * 8 * 64);
        if constexpr (BF) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2 h = __floats2half2_rn(__uint_as_float(b[n][j] << 16) * f[n],
                                                    __uint_as_float(b[n][j] & 0xffff0000u) * f[n]);
                b[n][j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // columns 32 h .. 32 h + 31, four of them this lane's
        uint32_t u[4];             // rows 2 t + (0, 1), then 8, 16 and 24 on
        op::ldmatrix_trans(u, rows_at ^ (h * 16));
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
                mma_f16(d, a[0], a[1], a[2], a[3], b[n][0], b[n][1]);
                mma_f16_add(d, a[4], a[5], a[6], a[7], b[n][2], b[n][3]);
                float(&o)[4] = acc[n][2 * h + s];
                o[0] = fmaf(sa, d[0], o[0]);
                o[1] = fmaf(sa, d[1], o[1]);
                o[2] = fmaf(sb, d[2], o[2]);
                o[3] = fmaf(sb, d[3], o[3]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT8; ++n) {
        mma_f16_add(b8[n], kMinus8, kMinus8, kMinus8, kMinus8, b[n][0], b[n][1]);
        mma_f16_add(b8[n], kMinus8, kMinus8, kMinus8, kMinus8, b[n][2], b[n][3]);
    }
}

// The bias of some blocks of one group: acc += scale * b8 (16 times that on
// odd tiles).
template <int NT8>
__device__ __forceinline__ void bias_fma(float (&acc)[NT8][8][4], const float (&sc)[16], const float (&b8)[NT8][4]) {
#pragma unroll
    for (int n = 0; n < NT8; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float k = (i & 1) ? 16.f : 1.f, bx = k * b8[n][0], by = k * b8[n][1];
            const float sa = sc[4 * (i >> 1) + (i & 1)], sb = sc[4 * (i >> 1) + (i & 1) + 2];
            float(&o)[4] = acc[n][i];
            o[0] = fmaf(sa, bx, o[0]);
            o[1] = fmaf(sa, by, o[1]);
            o[2] = fmaf(sb, bx, o[2]);
            o[3] = fmaf(sb, by, o[3]);
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

// 8 values of a row of x from row r on (rows from `rows` on are zeros), as
// 16 bytes of its type.
template <typename XT>
__device__ __forceinline__ uint4 load_x8(const XT* xr, int r, int rows, bool vec) {
    if (vec && r + 8 <= rows) return *reinterpret_cast<const uint4*>(xr + r);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    const uint16_t* p = reinterpret_cast<const uint16_t*>(xr + r);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (r + j < rows) w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The largest magnitude among 8 bf16 values and m.
__device__ __forceinline__ float absmax8(uint4 v, float m) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        m = fmaxf(m, fabsf(__uint_as_float(w[j] << 16)));
        m = fmaxf(m, fabsf(__uint_as_float(w[j] & 0xffff0000u)));
    }
    return m;
}
__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// Lane tok: the factor of bf16 token tok over rows [r0, r1).  One warp, with
// eight 16-byte loads of a lane on their way at once.
__device__ __forceinline__ float find_factors(const Tokens<__nv_bfloat16>& X, int nt, int r0, int r1, int lane) {
    const bool vec = (X.ld & 7) == 0;
    const int rows = r1 - r0, per = (rows + 255) >> 8;  // loads of 256 rows per token
    float mine = 1.f, m = 0.f;
    int tok = 0, p = 0, tok_j = 0, p_j = 0;  // the next load's token and pass; the next one's to use
    for (int i0 = 0; i0 < nt * per; i0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = make_uint4(0u, 0u, 0u, 0u);
            const int r = p * 256 + lane * 8;
            if (tok < nt && r < rows) v[j] = load_x8(X.row(tok) + r0, r, rows, vec);
            if (++p == per) p = 0, ++tok;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m = absmax8(v[j], m);
            if (++p_j == per) {
                m = warp_max(m);
                if (lane == tok_j) mine = row_factor(m);
                m = 0.f;
                p_j = 0, ++tok_j;
            }
        }
    }
    return mine;
}

// The sums of this CTA's slice [k0, k1) of K, left in smem as [token][128
// columns] fp32 for the nt tokens.  tokens(): the token rows, asked for once
// the first weight loads are on their way.
template <int NT8, typename XT, typename ST, bool VEC, typename F>
__device__ __forceinline__ void slice_sums(uint8_t* smem, const Weight<ST>& W, const Columns& C, int nt, int k0, int k1,
                                           F&& tokens) {
    using Cf = Cfg<NT8, ST>;
    constexpr bool BF = !std::is_same<XT, __half>::value;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + warp * Cf::RING;
    const int nblk = (k1 - k0 + kBlock - 1) / kBlock;
    const int r0 = k0 + nblk * warp / kWarps * kBlock;
    const int r1 = min(k1, k0 + nblk * (warp + 1) / kWarps * kBlock);
    Loader<ST, VEC> ld;
    ld.start(W, C, r0, lane);
    const int blocks = nblk * (warp + 1) / kWarps - nblk * warp / kWarps;
    const uint32_t ring0 = op::smem_u32(ring);
#pragma unroll
    for (int i = 0; i < Cf::STAGES - 1; ++i)
        if (i < blocks) ld.issue(ring0 + i * Cf::STAGE, ring + i * Cf::STAGE, C, lane);
    const Tokens<XT> X = tokens();
    XLoader<NT8, XT> xl;
    xl.start(X, nt, r0, r1, lane);
#pragma unroll
    for (int i = 0; i < Cf::STAGES - 1; ++i)
        if (i < blocks) xl.issue(ring0 + i * Cf::STAGE + Cf::XOFF, ring + i * Cf::STAGE + Cf::XOFF, nt, lane);
    // the first stages are one group; empty groups keep the count of the later ones
#pragma unroll
    for (int i = 0; i < Cf::STAGES - 1; ++i) op::cp_commit();
    float factors = 1.f, f[NT8];
    if constexpr (BF) {
        if (blocks > 0) factors = find_factors(X, nt, r0, r1, lane);
    }
    float acc[NT8][8][4], b8[NT8][4];  // b8: the bias not yet added, of the scales at hand
#pragma unroll
    for (int n = 0; n < NT8; ++n) {
        f[n] = __shfl_sync(0xffffffffu, factors, n * 8 + g);
        b8[n][0] = b8[n][1] = b8[n][2] = b8[n][3] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[n][i][c] = 0.f;
    }
    // a matrix load's addresses: row l % 8 of row group l / 8 of the weight; token l % 8, rows 8 (l / 8) on
    const uint32_t rows0 = ring0 + chunk_at(lane, 0), x0 = ring0 + Cf::XOFF + chunk_at(lane & 7, lane >> 3);
    const uint32_t sc0 = ring0 + Cf::WORDS + 4 * g * (int)sizeof(ST);
    float sc[16];
    int left = 0, next = W.group - r0 % W.group;  // rows that the scales at hand still cover; of the next ones
    for (int i0 = 0; i0 < blocks; i0 += Cf::STAGES) {
#pragma unroll
        for (int j = 0; j < Cf::STAGES; ++j) {
            if (i0 + j >= blocks) break;
            op::cp_wait<Cf::STAGES - 2>();
            __syncwarp();  // the copies are other lanes'
            if (left == 0) {  // a group's first block brings its scales
                if (i0 + j > 0) bias_fma<NT8>(acc, sc, b8);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    ST v[4];
                    op::lds<4 * (int)sizeof(ST)>(v, sc0 + j * Cf::STAGE + 32 * h * (int)sizeof(ST));
#pragma unroll
                    for (int c = 0; c < 4; ++c) sc[4 * h + c] = to_f32(v[c]);
                }
#pragma unroll
                for (int n = 0; n < NT8; ++n) b8[n][0] = b8[n][1] = b8[n][2] = b8[n][3] = 0.f;
                left = next;
                next = W.group;
            }
            left -= kBlock;
            // (these copies go to the stage read one turn ago: every lane has
            // passed this turn's __syncwarp since)
            constexpr int LAST = Cf::STAGES - 1;
            const int to = (j + LAST) % Cf::STAGES * Cf::STAGE;
            if (i0 + j + LAST < blocks) {
                ld.issue(ring0 + to, ring + to, C, lane);
                xl.issue(ring0 + to + Cf::XOFF, ring + to + Cf::XOFF, nt, lane);
            }
            op::cp_commit();
            block_fma<NT8, BF>(acc, b8, rows0 + j * Cf::STAGE, x0 + j * Cf::STAGE, sc, f);
        }
    }
    if (blocks > 0) bias_fma<NT8>(acc, sc, b8);
    op::cp_wait<0>();
    __syncthreads();
    // the quarters' sums, in their order
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int n = 0; n < NT8; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int tok = n * 8 + 2 * t + (c & 1);
            float inv = 1.f;
            if constexpr (BF) inv = 1.0f / __shfl_sync(0xffffffffu, factors, tok);
            if (tok < nt) {
                float* o = red + (warp * NT8 * 8 + tok) * kCols + (c & 2);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[tile_col(i, g)] = acc[n][i][c] * ((i & 1) ? 0x1p20f : 0x1p24f) * inv;
            }
        }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * kCols; i += kThreads) {
        float v = red[i];
#pragma unroll
        for (int q = 1; q < kWarps; ++q) v += red[q * NT8 * 8 * kCols + i];
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

// Slices of K (a power of two) for a launch of `tiles` tiles: as many CTAs as
// the SMs hold at once (per_sm each), a block at least for each warp, at most
// a portable cluster.
__host__ __forceinline__ int slices(long long tiles, int K, int sms, int per_sm) {
    const int blocks = (K + kBlock - 1) / kBlock;
    int S = 1;
    while (S < 8 && 2 * tiles * S <= (long long)per_sm * sms && blocks >= 2 * S * kWarps) S *= 2;
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
    const Columns C{col0, col0 + kHalf, W.N, W.N};
    slice_sums<NT8, XT, ST, VEC>(mv_smem, W, C, nt, k0, k1, [&] { return Tokens<XT>{x, W.K, t0, nullptr, 1}; });
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
    const void* x[2];        // operand rows: routed (slot order, or x itself: gather), shared (token order)
    int K[2], N[2];          // the weights' rows and columns
    const float* scale[2];   // gate/up: what multiplies a row's sums (null: 1)
    __half* h[2];            // gate/up: hidden rows [., N / 2]
    float* part[2];          // down: fp32 rows [., N], routed at the row's entry (perm)
    const int32_t* perm;
    int k;
    bool gather;             // routed operand row = x[perm[slot] / k]
    int shared_rows;         // > 0: the shared expert's rows, its units the first ones (it is not in the list)
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
// gate/up tile is 64 hidden columns (gate in the first half, up in the
// second), a down tile 128 columns.
template <typename XT, typename ST, bool GATE_UP>
__global__ void __launch_bounds__(kThreads, Cfg<1, ST>::PER_SM) experts_kernel(const GroupTable* tab, int num_experts,
                                                                              int group_rows,
                                                                              const __grid_constant__ Experts E,
                                                                              const Rows R) {
    extern __shared__ __align__(128) uint8_t mv_smem[];
    // the shared expert's units come first and read nothing that the routing
    // before this launch writes: they need not wait for it
    const int shared_units = (R.shared_rows + 7) >> 3;
    const bool early = GATE_UP && (int)blockIdx.y < shared_units;
    if (!early) op::pdl_wait();
    op::pdl_launch();
    int expert, sh, nt, row0;
    if ((int)blockIdx.y < shared_units) {
        expert = num_experts, sh = 1;
        row0 = blockIdx.y * 8;
        nt = min(8, R.shared_rows - row0);
    } else {
        int grp, row;
        if (!find_unit(tab, blockIdx.y - shared_units, grp, row)) return;
        expert = tab->expert[grp], sh = expert == num_experts ? 1 : 0;
        nt = min(8, tab->rows[grp] - row), row0 = tab->row0[grp] + row;
    }
    const int K = R.K[sh], N = R.N[sh];
    const int F = N / 2;
    const int col0 = blockIdx.x * (GATE_UP ? kHalf : kCols);
    if (col0 >= (GATE_UP ? F : N)) return;
    const int S = gridDim.z, slice = blockIdx.z, lg = __ffs(S) - 1;
    const int k0 = slice_row(K, slice, lg), k1 = slice_row(K, slice + 1, lg);
    const Weight<ST> W{E.q[expert], static_cast<const ST*>(E.s[expert]), N / 2, N, K, group_rows};
    const Columns C{col0, GATE_UP ? F + col0 : col0 + kHalf, GATE_UP ? F : N, N};
    slice_sums<1, XT, ST, true>(mv_smem, W, C, nt, k0, k1, [&] {
        return Tokens<XT>{static_cast<const XT*>(R.x[sh]), K, row0, GATE_UP && R.gather && !sh ? R.perm : nullptr, R.k};
    });
    const float* red = reinterpret_cast<const float*>(mv_smem);
    if (S > 1) op::cluster_sync();
    else __syncthreads();
    const int width = GATE_UP ? kHalf : kCols, items = nt * width;
    const int i0 = (items >> lg) * slice, i1 = i0 + (items >> lg);  // items is a multiple of 8
    for (int i = i0 + threadIdx.x; i < i1; i += kThreads) {
        const int tok = i / width, c = i % width;
        if (GATE_UP) {
            if (col0 + c >= F) continue;
            const float g = R.scale[sh] ? R.scale[sh][row0 + tok] : 1.0f;
            const float a = g * cluster_total(red, tok * kCols + c, S), b = g * cluster_total(red, tok * kCols + kHalf + c, S);
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
