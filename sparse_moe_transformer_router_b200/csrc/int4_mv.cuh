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
// - A warp takes 128 columns by 64 rows at a time through a ring of its own in
//   shared memory, filled by TMA: one lane's few instructions bring the
//   weight's box, the scales of the groups that begin there and the tokens'
//   rows.  Copies issued by every lane (cp.async) compete with the arithmetic
//   for issue slots: with the arithmetic taken out, 5120 x 202048 streams in
//   87 us by TMA and in 95 to 97 by cp.async (floor 81).
// - The operand wants pairs along K: a transposing matrix load of 16-bit
//   units, four columns each, returns two rows' units in one register.  Each
//   pair of nibbles is then one AND (with the sign bit flipped) away: u = q + 8
//   in [0, 15] left where it lies in the f16's low bits is the subnormal u
//   2^-24 (or 16 u 2^-24 one nibble up), exact in the tensor core.  No
//   conversion instruction, 0.625 logic instructions per weight in all.
// - The bias 8 leaves through the sums' start value, -8 sum(x) (2^-24): two
//   products with a constant per 32 rows, in the layout the others start from.
// - The block's fp32 sum is multiplied by the group's scale and added to the
//   column's total in fp32: the weights are never rounded to a product.
// - Tokens come along in the ring, f16 rows as they are, bf16 rows multiplied
//   (on their way to the product) by a power of two that brings the largest of
//   a warp's rows to [2^14, 2^15): exact for values down to 2^-31 of it, others
//   round at 2^-39 of it.  A row with an infinity or a NaN gives NaN (inf times
//   the bias).
//
// A CTA has four warps.  As an operator (and for the down product) it takes
// 128 columns and a slice of K, each warp a quarter of the slice; for gate/up
// it takes the 128 gate columns and the 128 up columns of the same hidden
// values, each by two warps with half of the slice.  The warps' sums are added
// through shared memory and the slices of a cluster through distributed shared
// memory, always in the same order.  Every wait for a copy gives up after a
// second: the sums become NaN (and the layer's error word gets a bit).
//
// What bounds it: loads and arithmetic of nearly the same length that overlap
// in part.  5120 x 202048 takes 87 us with the arithmetic taken out, 97 with
// the loads taken out, 110 together.  A scheduler issues a logic instruction
// every other cycle and an m16n8k16 product every eight (measured), and per 32
// rows x 128 columns a warp needs 80 and 18 of them beside 32 fp32 FMAs.
// Measured on one B200 (device time, three weights in turn):
//   1 x 5120 x 202048, groups of 128   110 us   4.8 TB/s   0.74 of the copy rate
//     (at 1965 MHz; a second of such calls on end, replayed or not, brings the
//     power cap, 1700 MHz and 125 to 127 us)
//   1 x 5120 x 16384                    16 us   2.7 TB/s   (1 x 512 x 128 alone takes 3.9 us)
//   16 x 8192 x 5120, groups of 64      15 us   1.5 TB/s   (two token columns: twice the products)
//   8 x 5120 x 16384 bf16               21 us   2.0 TB/s
//   16 x 5120 x 16384 bf16              43 us   1.0 TB/s   (each warp of each column tile finds the rows'
//     powers of two and converts them again; 256 CTAs for 444 places; some registers spill)
// The layer's figures stand at experts_kernel.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "schedule.cuh"
#include "sm.cuh"

namespace l4moe {
namespace mv {

constexpr unsigned kErrTimeout = 1u << 0;   // DEV_ERR_TIMEOUT_PRODUCER of the layer's error word
constexpr unsigned kErrF16Range = 1u << 4;  // DEV_ERR_F16_RANGE

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kCols = 128;       // columns of a warp
constexpr int kBlock = 32;       // rows that share a scale at least (scale groups are multiples of it)
constexpr int kRows = 64;        // rows of a stage
constexpr int kStages = 2;       // of a warp's ring
constexpr int kXRow = 2 * kRows; // bytes of a token's row in a stage

// A warp's ring.  Stage: the weight's 64 rows of 64 bytes, the tokens' 64
// values, two rows of scales (of the group of each 32 rows, where it begins).
template <int NT8, typename ST>
struct Cfg {
    static constexpr int XOFF = kRows * 64;
    static constexpr int SOFF = XOFF + NT8 * 8 * kXRow;
    static constexpr int STAGE = (SOFF + 2 * kCols * (int)sizeof(ST) + 1023) / 1024 * 1024;  // the swizzles' period
    // CTAs that share an SM: the registers' limit (up to 8 tokens 128 a
    // thread, 16 tokens 168).  Four with two stages each beat three with
    // three (1 x 5120 x 202048: 111 against 118 us): the arithmetic wants the warps
    static constexpr int PER_SM = NT8 == 1 ? 4 : 3;
    static constexpr int STAGES = kStages;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int RED = (int)sizeof(float) * kWarps * NT8 * 8 * kCols;  // over the rings
    static constexpr int SMEM = (kWarps * RING > RED ? kWarps * RING : RED) + 1024;  // and room to align them
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
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

// A weight matrix: its codes and scales behind tensor maps (boxes of 64 rows by
// 64 bytes and of one row by 128 columns), or, for sizes that those do not
// take, in memory.
template <typename ST>
struct Weight {
    const CUtensorMap *qm, *sm;
    const uint8_t* q;      // [K, N / 2]
    const ST* s;           // [groups, N]
    int N, K, group;
};

// Where a stage holds the 16 bytes of columns 32 c .. 32 c + 31 of row r, and
// values 8 c .. 8 c + 7 of token t (TMA's 64- and 128-byte swizzles): the
// eight rows of a matrix load lie in different banks.
__device__ __forceinline__ constexpr int chunk_at(int r, int c) { return r * 64 + ((c ^ ((r >> 1) & 3)) << 4); }
__device__ __forceinline__ constexpr int token_at(int t, int c) { return t * kXRow + ((c ^ (t & 7)) << 4); }

// The token rows of a CTA: rows of x, ld apart, from row0 on, or those that
// slot row0 + token of perm names (entry / k).
template <typename XT>
struct Tokens {
    const CUtensorMap* map;  // boxes of one row by 64 values
    const XT* x;
    long long ld;
    int row0;
    const int32_t* perm;
    int k;
    __device__ __forceinline__ int at(int token) const { return perm ? perm[row0 + token] / k : row0 + token; }
    __device__ __forceinline__ const XT* row(int token) const { return x + at(token) * ld; }
};

// Column (of the warp's 128) that accumulator tile i of lane group g holds in
// its first row (c0, c1); its second row (c2, c3) is two columns on.  Odd
// tiles hold 16 times their sum.
__device__ __forceinline__ constexpr int tile_col(int i, int g) { return (i >> 1) * 32 + 4 * g + (i & 1); }

// acc += 32 rows of the warp's stage (rows_at: this lane's address of a matrix
// load of the weight, x_at: of the tokens); sc: the scales of the lane's
// columns; f: what the lane's tokens (column l / 4 of each 8) are multiplied
// with as they become f16.  The sums start at -8 2^-24 sum(x): products of the
// tokens with rows of that constant (an f16 subnormal).
template <int NT8, bool BF>
__device__ __forceinline__ void block_fma(float (&acc)[NT8][8][4], uint32_t rows_at, uint32_t x_at, const float (&sc)[16], const float (&f)[NT8]) {
    constexpr uint32_t kMinus8 = 0x80088008u;
    uint32_t b[NT8][4];
#pragma unroll
    for (int n = 0; n < NT8; ++n) {
        op::ldmatrix(b[n], x_at + n * 8 * kXRow);
        if constexpr (BF) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2 h = __floats2half2_rn(__uint_as_float(b[n][j] << 16) * f[n],
                                                    __uint_as_float(b[n][j] & 0xffff0000u) * f[n]);
                b[n][j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
    // the sums' start values (on even tiles, 16 times that on odd ones)
    float c0[2][NT8][4];
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < NT8; ++n) {
        mma_f16(c0[0][n], kMinus8, kMinus8, kMinus8, kMinus8, b[n][0], b[n][1], zero);
        mma_f16_add(c0[0][n], kMinus8, kMinus8, kMinus8, kMinus8, b[n][2], b[n][3]);
#pragma unroll
        for (int c = 0; c < 4; ++c) c0[1][n][c] = 16.f * c0[0][n][c];
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
                mma_f16(d, a[0], a[1], a[2], a[3], b[n][0], b[n][1], c0[s][n]);
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

// Lane tok: the factor of bf16 token tok over rows [r0, r1).  One warp; B: the
// 16-byte loads of a lane (256 rows of a token each) on their way at once.
template <int B>
__device__ __forceinline__ float find_factors(const Tokens<__nv_bfloat16>& X, int nt, int r0, int r1, int lane) {
    const bool vec = (X.ld & 7) == 0;
    const int rows = r1 - r0, per = (rows + 255) >> 8;  // loads per token
    const __nv_bfloat16* src = X.row(0) + r0;
    float mine = 1.f, m = 0.f;
    int left = nt * per, p = 0, tok_j = 0, p_j = 0;  // loads left; the next load's pass; the next one's to use
    while (left > 0) {
        uint4 v[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            v[j] = make_uint4(0u, 0u, 0u, 0u);
            if (j < left) {
                const int r = p * 256 + lane * 8;
                if (r < rows) v[j] = load_x8(src, r, rows, vec);
                if (++p == per) p = 0, src += X.ld;
            }
        }
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (j >= left) break;
            m = absmax8(v[j], m);
            if (++p_j == per) {
                m = warp_max(m);
                if (lane == tok_j) mine = row_factor(m);
                m = 0.f;
                p_j = 0, ++tok_j;
            }
        }
        left -= B;
    }
    return mine;
}

// 16 bytes from any address of a matrix that ends at `end`: whole words,
// shifted together, or byte by byte where those would reach past the end.
__device__ __forceinline__ uint4 load_any16(const uint8_t* p, const uint8_t* end) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(a & ~uintptr_t(3));
    uint32_t v[4] = {0u, 0u, 0u, 0u};
    if (reinterpret_cast<const uint8_t*>(w + 5) <= end) {
        uint32_t r[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) r[i] = __ldg(w + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(r[i], r[i + 1], (uint32_t)(a & 3) * 8);
    } else {
#pragma unroll
        for (int b = 0; b < 16; ++b)
            if (p + b < end) v[b >> 2] |= (uint32_t)__ldg(p + b) << (8 * (b & 3));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// One stage's plain loads, for sizes that tensor maps do not take: lane l rows
// l and l + 32 of the weight (what lies past a row's end belongs to columns
// that are not stored), tokens and scales element by element, zeros past K.
template <int NT8, typename XT, typename ST>
__device__ __forceinline__ void load_plain(uint8_t* stage, const Weight<ST>& W, int col0, const Tokens<XT>& X, int nt,
                                           int row, int end, bool s0, bool s1, int grp, int lane) {
    using Cf = Cfg<NT8, ST>;
    const uint8_t* wend = W.q + (long long)W.K * (W.N / 2);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = lane + 32 * h;
        const uint8_t* p = W.q + (long long)(row + r) * (W.N / 2) + (col0 >> 1);
        uint4 v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[c] = make_uint4(0u, 0u, 0u, 0u);
            if (row + r < W.K && col0 + 32 * c < W.N) v[c] = load_any16(p + 16 * c, wend);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(stage + chunk_at(r, c)) = v[c];
    }
    for (int i = lane; i < nt * 8; i += 32) {
        const int t = i >> 3, c = i & 7;
        *reinterpret_cast<uint4*>(stage + Cf::XOFF + token_at(t, c)) =
            load_x8(X.row(t) + row, c * 8, end - row, false);
    }
    ST* d = reinterpret_cast<ST*>(stage + Cf::SOFF);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h ? !s1 : !s0) continue;
        const ST* s = W.s + (long long)(grp + h) * W.N + col0;  // (grp: the first half's)
        for (int c = lane; c < kCols; c += 32)
            if (col0 + c < W.N) d[h * kCols + c] = s[c];
    }
}

// First row of slice r of 2^lg: whole blocks, as even as they come.
__host__ __device__ __forceinline__ int slice_row(int K, int r, int lg) {
    const int blocks = (K + kBlock - 1) / kBlock;  // K <= 2^30: blocks * 8 fits
    const int k = ((blocks * r) >> lg) * kBlock;
    return k < K ? k : K;
}

// Rows [r0, r1) of part `part` of PARTS of the slice [k0, k1): whole blocks (of
// the last one what K leaves); the number of blocks.
__host__ __device__ __forceinline__ int part_rows(int k0, int k1, int part, int PARTS, int& r0, int& r1) {
    const int nblk = (k1 - k0 + kBlock - 1) / kBlock;
    const int b0 = nblk * part / PARTS, blocks = nblk * (part + 1) / PARTS - b0;
    r0 = k0 + b0 * kBlock;
    r1 = k1 < r0 + blocks * kBlock ? k1 : r0 + blocks * kBlock;
    return blocks;
}

// The scales that come with a warp's stages, from row r0 (a multiple of kBlock)
// on: a half of a stage brings the scales of the group that begins there (the
// warp's first half always does).
struct ScaleRows {
    int group, grp, left, next;  // the latest group; its rows that are left; the next one's rows
    __host__ __device__ __forceinline__ ScaleRows(int r0, int group_) : group(group_) {
        grp = r0 / group;
        left = 0, next = group - (r0 - grp * group);
        --grp;
    }
    // The next stage, at `row` of rows that end at r1: whether its halves bring
    // scales; those are the rows first(s1) and grp of the scales.
    __host__ __device__ __forceinline__ void stage(int row, int r1, bool& s0, bool& s1) {
        s0 = left == 0;
        if (s0) left = next, next = group, ++grp;
        left -= kBlock;
        s1 = left == 0 && row + kBlock < r1;  // (the last stage's second half may have no rows, and no group)
        if (s1) left = group, ++grp;
        left -= kBlock;
    }
    __host__ __device__ __forceinline__ int first(bool s1) const { return grp - (s1 ? 1 : 0); }
};

// Stage i of a warp is load i of its ring: slot i % STAGES, the barrier's phase
// of this parity.
template <int STAGES>
__host__ __device__ __forceinline__ uint32_t stage_parity(int i) { return (uint32_t)(i / STAGES) & 1u; }

// After the wait for stage `at` of `stages` gave up: wait(slot, parity) for
// every copy that is on its way.
template <int STAGES, typename W>
__host__ __device__ __forceinline__ void drain(int at, int stages, W&& wait) {
    for (int i = at; i < at + STAGES && i < stages; ++i) wait(i % STAGES, stage_parity<STAGES>(i));
}

// This warp's sums over part `part` of PARTS of the slice [k0, k1) of K, for
// the 128 columns from col0 on and nt tokens, left in red [warp][token][128]
// (over the rings: all warps are through with theirs).  tokens(): the token
// rows, asked for once the first weight loads are on their way.  ring: this
// warp's, 1024-byte aligned; bar: its barriers, initialised.  False: a copy
// did not come (the sums are NaN).
template <int NT8, int PARTS, typename XT, typename ST, bool TMA, typename F>
__device__ __forceinline__ bool warp_sums(uint8_t* ring, uint64_t* bar, float* red, const Weight<ST>& W, int col0, int nt,
                                          int k0, int k1, int part, F&& tokens) {
    using Cf = Cfg<NT8, ST>;
    constexpr bool BF = !std::is_same<XT, __half>::value;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    int r0, r1;
    const int blocks = part_rows(k0, k1, part, PARTS, r0, r1);
    const int stages = (blocks + 1) >> 1;
    const uint32_t ring0 = op::smem_u32(ring), bar0 = op::smem_u32(bar);

    // ---- loads: the next stage's row and the scales that come with it
    int lrow = r0;
    ScaleRows scales(r0, W.group);
    int xrow = 0;  // this lane's token's row (lanes below nt)
    Tokens<XT> X{};
    auto issue_w = [&](int s, uint32_t at) {  // the weight's and the scales' part of stage s
        bool s0, s1;
        scales.stage(lrow, r1, s0, s1);
        if constexpr (TMA) {
            if (lane == 0) {
                const uint32_t b = bar0 + s * 8;
                op::mbar_expect(b, kRows * 64 + nt * kXRow + ((s0 ? 1 : 0) + (s1 ? 1 : 0)) * kCols * (int)sizeof(ST));
                op::tma_2d(at, W.qm, b, col0 >> 1, lrow);
                if (s0) op::tma_2d(at + Cf::SOFF, W.sm, b, col0, scales.first(s1));
                if (s1) op::tma_2d(at + Cf::SOFF + kCols * (int)sizeof(ST), W.sm, b, col0, scales.grp);
            }
        } else {
            load_plain<NT8, XT, ST>(ring + (at - ring0), W, col0, X, nt, lrow, r1, s0, s1, scales.first(s1), lane);
        }
    };
    auto issue_x = [&](int s, uint32_t at) {
        if constexpr (TMA) {
            if (lane < nt) op::tma_2d(at + Cf::XOFF + lane * kXRow, X.map, bar0 + s * 8, lrow, xrow);
        }
        lrow += kRows;
    };
    const int pre = min(stages, Cf::STAGES);
    if constexpr (!TMA) X = tokens();
#pragma unroll
    for (int s = 0; s < Cf::STAGES; ++s)
        if (s < pre) {
            issue_w(s, ring0 + s * Cf::STAGE);
            lrow += kRows;
        }
    lrow = r0;
    if constexpr (TMA) {
        X = tokens();
        if (lane < nt) xrow = X.at(lane);
    }
#pragma unroll
    for (int s = 0; s < Cf::STAGES; ++s)
        if (s < pre) issue_x(s, ring0 + s * Cf::STAGE);

    float factors = 1.f, f[NT8];
    if constexpr (BF) {
        // up to two loads a lane (512 values) nothing is gained from eight at
        // once, and the extra steps show: always 2 against always 8, 1 x 512 x
        // 128 3.86 and 4.03 us, 1 x 8192 x 5120 11.9 and 12.1; above, 8 x 5120
        // x 16384 22.3 and 20.9, 16 x 5120 x 16384 47.0 and 42.0
        if (blocks > 0)
            factors = nt * (r1 - r0) <= 512 ? find_factors<2>(X, nt, r0, r1, lane) : find_factors<8>(X, nt, r0, r1, lane);
    }
    float acc[NT8][8][4];
#pragma unroll
    for (int n = 0; n < NT8; ++n) {
        f[n] = __shfl_sync(0xffffffffu, factors, n * 8 + g);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[n][i][c] = 0.f;
    }
    // a matrix load's addresses: row l % 8 of row group l / 8 of the weight; token l % 8, values 8 (l / 8) on
    const uint32_t rows0 = ring0 + chunk_at(lane, 0), x0 = ring0 + Cf::XOFF + token_at(lane & 7, lane >> 3);
    const uint32_t sc0 = ring0 + Cf::SOFF + 4 * g * (int)sizeof(ST);
    float sc[16];
    int left = 0, next = W.group - r0 % W.group;  // rows that the scales at hand still cover; of the next ones
    bool ok = true;
    for (int i0 = 0; i0 < stages && ok; i0 += Cf::STAGES) {
#pragma unroll
        for (int s = 0; s < Cf::STAGES; ++s) {
            if (i0 + s >= stages) break;
            if constexpr (TMA) {
                ok = __all_sync(0xffffffffu, op::mbar_wait(bar0 + s * 8, stage_parity<Cf::STAGES>(i0)));
                if (!ok) {  // let what is on its way arrive before the memory is used again
                    drain<Cf::STAGES>(i0 + s, stages,
                                      [&](int slot, uint32_t parity) { op::mbar_wait(bar0 + slot * 8, parity); });
                    break;
                }
            } else {
                __syncwarp();
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (2 * (i0 + s) + h >= blocks) break;
                if (left == 0) {  // a group's first rows bring its scales
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        ST v[4];
                        op::lds<4 * (int)sizeof(ST)>(v, sc0 + s * Cf::STAGE + (h * kCols + 32 * q) * (int)sizeof(ST));
#pragma unroll
                        for (int c = 0; c < 4; ++c) sc[4 * q + c] = to_f32(v[c]);
                    }
                    left = next;
                    next = W.group;
                }
                left -= kBlock;
                block_fma<NT8, BF>(acc, rows0 + s * Cf::STAGE + h * kBlock * 64,
                                   (x0 + s * Cf::STAGE) ^ (h * 64), sc, f);
            }
            if (lrow < r1) {  // a stage still to load
                __syncwarp();  // every lane has read the stage
                issue_w(s, ring0 + s * Cf::STAGE);
                issue_x(s, ring0 + s * Cf::STAGE);
            }
        }
    }
    const float bad = ok ? 0.f : __int_as_float(0x7fffffff);
    __syncthreads();
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
                for (int i = 0; i < 8; ++i)
                    o[tile_col(i, g)] = acc[n][i][c] * ((i & 1) ? 0x1p20f : 0x1p24f) * inv + bad;
            }
        }
    __syncthreads();
    return ok;
}

// Sum of element i (of [token][128]) over the PARTS warps from `first` on and
// the cluster's slices, in their order: own(i) leaves the CTA's sum in place,
// total(i) is read after the cluster's barrier.
template <int NT8, int PARTS>
__device__ __forceinline__ void join_parts(float* red, int first, int nt) {
    constexpr int STRIDE = NT8 * 8 * kCols;
    float* r = red + first * STRIDE;
    for (int i = threadIdx.x; i < nt * kCols; i += kThreads) {
        float v = r[i];
#pragma unroll
        for (int q = 1; q < PARTS; ++q) v += r[q * STRIDE + i];
        r[i] = v;  // read and written by this thread alone
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

// This warp's ring and barriers in a kernel's shared memory; all threads.
template <int NT8, typename ST>
__device__ __forceinline__ uint8_t* rings(uint8_t* smem, uint64_t (&bar)[kWarps][kStages]) {
    using Cf = Cfg<NT8, ST>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) {
        for (int s = 0; s < Cf::STAGES; ++s) op::mbar_init(op::smem_u32(&bar[warp][s]), 1);
        op::fence_mbar_init();
    }
    __syncwarp();
    return smem + ((1024u - (op::smem_u32(smem) & 1023u)) & 1023u);
}

// Slices of K (a power of two) for a launch of `tiles` tiles: as many CTAs as
// the SMs hold at once (per_sm each), two at least for each warp (a stage), at most
// a portable cluster.
__host__ __forceinline__ int slices(long long tiles, int K, int sms, int per_sm) {
    const int blocks = (K + kBlock - 1) / kBlock;
    int S = 1;
    while (S < 8 && 2 * tiles * S <= (long long)per_sm * sms && blocks >= 4 * S * kWarps) S *= 2;
    return S;
}

// ------------------------------------------------------------ the operator
// y [T, N] = x [T, K] W.  Grid: (column tiles, token tiles, slices), the
// slices of a tile one cluster.
template <int NT8, typename XT, typename ST, bool TMA>
__global__ void __launch_bounds__(kThreads, Cfg<NT8, ST>::PER_SM) int4_matvec_kernel(
    const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap sm,
    const __grid_constant__ CUtensorMap xm, const XT* __restrict__ x, int T, Weight<ST> W, XT* __restrict__ y) {
    extern __shared__ __align__(16) uint8_t mv_smem[];
    __shared__ uint64_t bar[kWarps][kStages];
    uint8_t* base = rings<NT8, ST>(mv_smem, bar);
    op::pdl_enter();
    const int warp = threadIdx.x >> 5;
    const int S = gridDim.z, slice = blockIdx.z, lg = __ffs(S) - 1;
    const int col0 = blockIdx.x * kCols;
    const int t0 = blockIdx.y * NT8 * 8, nt = min(NT8 * 8, T - t0);
    W.qm = &qm;
    W.sm = &sm;
    float* red = reinterpret_cast<float*>(base);
    warp_sums<NT8, kWarps, XT, ST, TMA>(base + warp * Cfg<NT8, ST>::RING, bar[warp], red, W, col0, nt,
                                        slice_row(W.K, slice, lg), slice_row(W.K, slice + 1, lg), warp,
                                        [&] { return Tokens<XT>{&xm, x, W.K, t0, nullptr, 1}; });
    join_parts<NT8, kWarps>(red, 0, nt);
    if (S > 1) op::cluster_sync();
    else __syncthreads();
    const int items = nt * kCols >> lg;  // nt * 128 is a multiple of 8
    for (int i = items * slice + threadIdx.x; i < items * (slice + 1); i += kThreads) {
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
// A launch's experts, rows and outputs, for its routed experts [0] and the
// shared one [1].
struct Rows {
    CUtensorMap xm[2];       // operand rows: routed (slot order, or by gather), shared (token order)
    const CUtensorMap* qm;   // codes of experts 0 .. E - 1 and of the shared one (E), then
    const CUtensorMap* sm;   // their scales
    int K[2], N[2];          // the weights' rows and columns
    const float* scale[2];   // gate/up: what multiplies a row's sums (null: 1)
    __half* h[2];            // gate/up: hidden rows [., N / 2]
    float* part[2];          // down: fp32 rows [., N], routed at the row's entry (perm)
    const int32_t* perm;
    int k;
    bool gather;             // routed operand row = x[perm[slot] / k]
    int shared_rows;         // > 0: the shared expert's rows; its units are the first ones and not in the list
    const int4* units;       // the other units as (expert, first slot, rows, -), rows = 0 past the last; null: by tab
    const GroupTable* tab;
    int num_experts, group;
    unsigned* err;
};

// The group and first row of unit u of a work list: units are the groups'
// tiles of 8 rows, in the list's order.  One warp; group < 0 past the list.
__device__ __forceinline__ int2 find_unit(const GroupTable* tab, int u) {
    const int lane = threadIdx.x & 31, n = tab->num_groups;
    int base = 0;
    for (int g0 = 0; g0 < n; g0 += 32) {
        const int tiles = g0 + lane < n ? (tab->rows[g0 + lane] + 7) >> 3 : 0;
        int incl = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned who = __ballot_sync(0xffffffffu, u < base + incl);
        if (who) {
            const int l = __ffs(who) - 1;
            return make_int2(g0 + l, (u - base - __shfl_sync(0xffffffffu, incl - tiles, l)) * 8);
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return make_int2(-1, 0);
}

// Gate/up: h = silu(c a_gate) (c a_up), c the row's scale (its sigmoid gate).
// Down: the fp32 sums, un-permuted.  Grid: (column tiles, units, slices); a
// tile is 128 hidden columns (gate/up) or 128 columns (down).
//
// Bound like the operator: by the weights' bytes, then by the logic that
// widens them.  8 rows of an expert at a time; more rows of one expert
// read its weights again.  Layer of width 5120 and 8192, one B200, device time
// of a whole forward: one token, 128 experts, groups of 128: 53 us (131 MB,
// 2.5 TB/s); sixteen tokens, 16 experts, groups of 32: 195 to 201 us (800 MB,
// 4.0 to 4.1 TB/s).  Between events, which keep the launches from overlapping:
// routing 17, gate/up 29, down 23 us and 15, 127, 72 us.
template <typename ST, bool GATE_UP>
__global__ void __launch_bounds__(kThreads, Cfg<1, ST>::PER_SM) experts_kernel(const __grid_constant__ Rows R) {
    extern __shared__ __align__(16) uint8_t mv_smem[];
    __shared__ uint64_t bar[kWarps][kStages];
    uint8_t* base = rings<1, ST>(mv_smem, bar);
    const int warp = threadIdx.x >> 5;
    // the shared expert's units come first: their weights are on their way
    // before what the launch before this one writes is waited for
    const int shared_units = (R.shared_rows + 7) >> 3;
    const bool first = (int)blockIdx.y < shared_units;
    if (!first) op::pdl_wait();
    op::pdl_launch();
    int expert, sh, nt, row0;
    if (first) {
        expert = R.num_experts, sh = 1;
        row0 = blockIdx.y * 8;
        nt = min(8, R.shared_rows - row0);
    } else if (R.units) {
        const int4 u = __ldg(R.units + (blockIdx.y - shared_units));
        expert = u.x, row0 = u.y, nt = u.z, sh = 0;
        if (nt == 0) return;
    } else {
        const int2 at = find_unit(R.tab, blockIdx.y);
        if (at.x < 0) return;
        expert = R.tab->expert[at.x], sh = expert == R.num_experts ? 1 : 0;
        nt = min(8, R.tab->rows[at.x] - at.y), row0 = R.tab->row0[at.x] + at.y;
    }
    const int K = R.K[sh], N = R.N[sh], width = GATE_UP ? N / 2 : N;
    const int c0 = blockIdx.x * kCols;
    if (c0 >= width) {
        if (first) op::pdl_wait();
        return;
    }
    const int S = gridDim.z, slice = blockIdx.z, lg = __ffs(S) - 1;
    const int k0 = slice_row(K, slice, lg), k1 = slice_row(K, slice + 1, lg);
    const Weight<ST> W{R.qm + expert, R.sm + expert, nullptr, nullptr, N, K, R.group};
    constexpr int PARTS = GATE_UP ? kWarps / 2 : kWarps;
    const int side = warp / PARTS;  // gate/up: 0 gate, 1 up
    float* red = reinterpret_cast<float*>(base);
    const bool ok = warp_sums<1, PARTS, __half, ST, true>(
        base + warp * Cfg<1, ST>::RING, bar[warp], red, W, side * width + c0, nt, k0, k1, warp - side * PARTS, [&] {
            if (first) op::pdl_wait();
            return Tokens<__half>{&R.xm[sh], nullptr, K, row0, GATE_UP && R.gather && !sh ? R.perm : nullptr, R.k};
        });
    if (!ok && (threadIdx.x & 31) == 0) atomicOr(R.err, kErrTimeout);
    join_parts<1, PARTS>(red, 0, nt);
    if (GATE_UP) join_parts<1, PARTS>(red, PARTS, nt);
    if (S > 1) op::cluster_sync();
    else __syncthreads();
    const int items = nt * kCols >> lg;  // nt * 128 is a multiple of 8
    for (int i = items * slice + threadIdx.x; i < items * (slice + 1); i += kThreads) {
        const int tok = i / kCols, c = c0 + i % kCols, row = row0 + tok;
        if (c >= width) continue;
        if (GATE_UP) {
            const float g = R.scale[sh] ? R.scale[sh][row] : 1.0f;
            const float a = g * cluster_total(red, i, S), b = g * cluster_total(red, PARTS * 8 * kCols + i, S);
            const float hv = __fdividef(a, 1.0f + __expf(-a)) * b;
            if (!(fabsf(hv) < 65520.0f)) atomicOr(R.err, kErrF16Range);  // rounds to infinity in f16
            R.h[sh][(long long)row * width + c] = __float2half_rn(hv);
        } else {
            const int orow = sh ? row : R.perm[row];
            R.part[sh][(long long)orow * width + c] = cluster_total(red, i, S);
        }
    }
    if (S > 1) op::cluster_sync();
}

}  // namespace mv
}  // namespace l4moe
