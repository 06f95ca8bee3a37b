// route_group.cuh -- the routing of a small batch (up to 16 tokens) for the
// products that gather their rows themselves (int4_mv.cuh): logits, top-k
// selection, gates, counts, offsets, slots and the list of the experts in use.
//
// The router is x (16 rows, padded) times W_router [d, E], bound by reading
// W_router and by the chain of short steps after it.  One cluster of 8 CTAs
// shares K: every warp takes 16-row steps of W_router through a ring of its
// own (asynchronous copies) into mma.sync m16n8k16 with fp32 sums, the
// tokens' rows as the other operand straight from global memory; the warps'
// sums are added through shared memory, the CTAs' through distributed shared
// memory by the CTA that then selects the token's experts, and the first CTA
// makes the slots.  All sums in a fixed order.  The tokens' rows are not
// copied into expert order; each is written once as f16, times a power of two
// where f16's range asks for it.
//
// Far from its floor (0.2 us for the 1.3 MB of W_router at d 5120, 128
// experts): the timeline of the layer shows 17 us for one token and 15 us for
// sixteen tokens and 16 experts, the events' own time included.  It took the
// place of the one-launch routing of the other layers, whose last CTA converts
// and copies every row; with that change and the shared expert's products
// beside it the whole layer went from 87 to 65 us and from 299 to 234 us.
// Clusters of 16 CTAs (the non-portable size) were not tried.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "permute.cuh"
#include "sm.cuh"
#include "topk.cuh"

namespace l4moe {
namespace rg {

constexpr int kTokens = 16;
constexpr int kCtas = 8;       // one cluster
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kStep = 16;      // rows of W_router per step
constexpr int kBlockCols = 128;  // experts per warp
constexpr int kPitch = kBlockCols * 2 + 16;  // bytes: a matrix load's eight rows lie in different banks
constexpr int kStage = kStep * kPitch;
constexpr int kStages = 3;
constexpr int kRing = kStages * kStage;
constexpr int kMaxEntries = kTokens * kMaxTopK;

// Dynamic shared memory: the warps' rings, then (in the same place) their
// sums [warp group][T][E].
__host__ __device__ constexpr size_t smem_bytes() {
    const size_t ring = (size_t)kWarps * kRing, red = sizeof(float) * kWarps * kTokens * kBlockCols;
    return ring > red ? ring : red;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// E a multiple of 8, d of 16, T <= 16.  Grid: one cluster of kCtas.  units
// [max_units] receives tiles of 8 rows of the experts in use (expert, first
// slot, rows, 0), rows = 0 past the last.  x16 [T][d]: the rows in f16, each
// divided by its scale (a power of two), which tokscale gets and gslot holds
// with the gate.
__global__ void __launch_bounds__(kThreads) route_group_kernel(
    const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ Wr, const float* __restrict__ bias, int T,
    int d, int E, int k, int32_t* __restrict__ idx, float* __restrict__ gate, float* __restrict__ lmax,
    float* __restrict__ margin, int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
    int32_t* __restrict__ perm, float* __restrict__ gslot, int4* __restrict__ units, int max_units,
    __half* __restrict__ x16, float* __restrict__ tokscale) {
    op::pdl_enter();
    extern __shared__ __align__(128) uint8_t rg_smem[];
    __shared__ int32_t s_ent[kMaxEntries];   // selected expert of entry n = t * k + j (first CTA)
    __shared__ float s_gate[kMaxEntries];
    __shared__ int32_t s_rank[kMaxEntries];
    __shared__ int32_t s_rows[256], s_off[256];
    __shared__ float s_scale[kTokens];       // first CTA: every token's scale
    __shared__ float s_max[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x;
    const int nb = (E + kBlockCols - 1) / kBlockCols;  // 1 or 2 blocks of experts
    const int groups = kWarps / nb, group = warp / nb, block = warp - group * nb;
    const int c0 = block * kBlockCols, cols = min(kBlockCols, E - c0);
    const int g = lane >> 2, t4 = lane & 3;

    op::cluster_arrive();  // (the first CTA's shared memory is written below: it must have started)
    // ------------------------------------------------ this warp's share of the sums
    {
        uint8_t* ring = rg_smem + warp * kRing;
        const uint32_t ring0 = op::smem_u32(ring);
        const int steps = d / kStep, stride = kCtas * groups;
        int next = rank + kCtas * group;  // the next step to load
        const int chunks = cols / 8;      // 16-byte pieces of a row
        auto issue = [&](int stage) {
            if (next < steps) {
                const __nv_bfloat16* src = Wr + (size_t)next * kStep * E + c0;
                for (int i = lane; i < kStep * chunks; i += 32) {
                    const int r = i / chunks, c = i - r * chunks;
                    op::cp_async16(ring0 + stage * kStage + r * kPitch + c * 16, src + (size_t)r * E + c * 8);
                }
            }
            next += stride;
            op::cp_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue(i);
        op::cluster_wait();
        // while they come: the rows of tokens rank and rank + 8 in f16
        for (int t = rank; t < T; t += kCtas) {
            const uint4* src = reinterpret_cast<const uint4*>(x + (size_t)t * d);
            const int n = d / 8;
            float m = 0.f;
            for (int i = tid; i < n; i += kThreads) m = absmax_vec(src[i], m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            __syncthreads();  // s_max has been read
            if (lane == 0) s_max[warp] = m;
            __syncthreads();
            m = s_max[lane & (kWarps - 1)];
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float sc = f16_row_scale(m), r = 1.0f / sc;
            for (int i = tid; i < n; i += kThreads)
                reinterpret_cast<uint4*>(x16 + (size_t)t * d)[i] = cvt_row_vec(src[i], __nv_bfloat16{}, __half{}, r);
            if (tid == 0) {
                tokscale[t] = sc;
                op::st_cluster_u32(op::mapa(op::smem_u32(s_scale + t), 0u), __float_as_uint(sc));
            }
        }
        float acc[kBlockCols / 8][4];
#pragma unroll
        for (int i = 0; i < kBlockCols / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        auto load_x = [&](uint32_t (&a)[4], int s) {
            const __nv_bfloat16* p = x + (size_t)s * kStep + 2 * t4;
            const bool in = s < steps, lo = in && g < T, hi = in && g + 8 < T;
            a[0] = lo ? *reinterpret_cast<const uint32_t*>(p + (size_t)g * d) : 0u;
            a[1] = hi ? *reinterpret_cast<const uint32_t*>(p + (size_t)(g + 8) * d) : 0u;
            a[2] = lo ? *reinterpret_cast<const uint32_t*>(p + (size_t)g * d + 8) : 0u;
            a[3] = hi ? *reinterpret_cast<const uint32_t*>(p + (size_t)(g + 8) * d + 8) : 0u;
        };
        uint32_t a[4], an[4];
        const int first = rank + kCtas * group;
        load_x(a, first);
        int get = 0, put = kStages - 1;
        // a matrix load: rows 0-7 and 8-15 of tile 2 j, then of tile 2 j + 1
        const uint32_t at = ring0 + (((lane >> 3) & 1) * 8 + (lane & 7)) * kPitch + (lane >> 4) * 16;
        for (int s = first; s < steps; s += stride) {
            load_x(an, s + stride);
            op::cp_wait<kStages - 2>();
            __syncwarp();
            issue(put);
#pragma unroll
            for (int j = 0; j < kBlockCols / 16; ++j) {
                if (j * 16 >= cols) break;
                uint32_t b[4];
                op::ldmatrix_trans(b, at + get * kStage + j * 32);
                mma_bf16(acc[2 * j], a, b[0], b[1]);
                mma_bf16(acc[2 * j + 1], a, b[2], b[3]);  // (past the last tile: not stored)
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = an[i];
            put = get;
            get = get + 1 == kStages ? 0 : get + 1;
        }
        op::cp_wait<0>();
        __syncthreads();
        float* red = reinterpret_cast<float*>(rg_smem);  // [group][T][E]
#pragma unroll
        for (int i = 0; i < kBlockCols / 8; ++i) {
            if (i * 8 >= cols) break;
            float* o = red + ((size_t)group * T + g) * E + c0 + i * 8 + 2 * t4;
            if (g < T) *reinterpret_cast<float2*>(o) = make_float2(acc[i][0], acc[i][1]);
            if (g + 8 < T) *reinterpret_cast<float2*>(o + 8 * E) = make_float2(acc[i][2], acc[i][3]);
        }
        __syncthreads();
        for (int i = tid; i < T * E; i += kThreads) {
            float v = red[i];
            for (int q = 1; q < groups; ++q) v += red[(size_t)q * T * E + i];
            red[i] = v;  // read and written by this thread alone
        }
    }
    op::cluster_sync();

    // ------------------------------------------------ selection: CTA r has tokens r and r + 8
    const float* sums = reinterpret_cast<const float*>(rg_smem);
    const int t = rank + kCtas * warp;
    if (warp < 2 && t < T) {
        TopK tk;
        tk.init();
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            if (e < E) {
                uint32_t v[kCtas];
                const uint32_t from = op::smem_u32(sums + t * E + e);
#pragma unroll
                for (int r = 0; r < kCtas; ++r) v[r] = op::ld_cluster_u32(op::mapa(from, (uint32_t)r));
                float l = 0.f;
#pragma unroll
                for (int r = 0; r < kCtas; ++r) l += __uint_as_float(v[r]);
                tk.offer(l + (bias ? bias[e] : 0.f), e);
            }
        }
        // the lanes' lists joined: k + 1 rounds take the first head in (value, index) order
        TopK sel;
        sel.init();
        int pos = 0;
#pragma unroll
        for (int j = 0; j <= kMaxTopK; ++j) {
            if (j > k) break;
            float hv = tk.value(pos);
            int hi = pos <= kMaxTopK ? tk.index(pos) : -1, hl = lane;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float ov = __shfl_xor_sync(0xffffffffu, hv, o);
                const int oi = __shfl_xor_sync(0xffffffffu, hi, o), ol = __shfl_xor_sync(0xffffffffu, hl, o);
                if (topk_before(ov, oi, hv, hi)) hv = ov, hi = oi, hl = ol;
            }
            sel.set(j, hv, hi);
            if (hl == lane && hi >= 0) ++pos;
        }
        if (lane == 0) {
            sel.fill_empty(k);
#pragma unroll
            for (int j = 0; j < kMaxTopK; ++j) {
                if (j < k) {
                    const int n = t * k + j;
                    const float gt = 1.0f / (1.0f + expf(-sel.value(j)));
                    idx[n] = sel.index(j);
                    lmax[n] = sel.value(j);
                    gate[n] = gt;
                    op::st_cluster_u32(op::mapa(op::smem_u32(s_ent + n), 0u), (uint32_t)sel.index(j));
                    op::st_cluster_u32(op::mapa(op::smem_u32(s_gate + n), 0u), __float_as_uint(gt));
                }
            }
            margin[t] = sel.value(k - 1) - sel.value(k);
        }
    }
    op::cluster_sync();
    if (rank != 0 || warp != 0) return;

    // ------------------------------------------------ slots (one warp)
    const int Tv = T * k;
    for (int e = lane; e < 256; e += 32) s_rows[e] = 0;
    __syncwarp();
    for (int n0 = 0; n0 < Tv; n0 += 32) {
        const int n = n0 + lane, e = n < Tv ? s_ent[n] : -1;
        const unsigned peers = __match_any_sync(0xffffffffu, e);
        const int below = __popc(peers & ((1u << lane) - 1u));
        if (e >= 0) s_rank[n] = s_rows[e] + below;  // entries of e before these 32, then among them
        __syncwarp();
        if (e >= 0 && below == 0) s_rows[e] += __popc(peers);
        __syncwarp();
    }
    int base = 0, used = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane, rows = e < E ? s_rows[e] : 0;
        int incl = rows;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const int off = base + incl - rows;
        const unsigned some = __ballot_sync(0xffffffffu, rows > 0);
        if (e < E) {
            s_off[e] = off;
            offsets[e] = off;
            counts[e] = rows;
        }
        const unsigned big = __ballot_sync(0xffffffffu, rows > 8);  // (at most 16 rows: two tiles)
        if (rows > 0) {
            const unsigned lower = (1u << lane) - 1u;
            const int at = used + __popc(some & lower) + __popc(big & lower);
            units[at] = make_int4(e, off, min(rows, 8), 0);
            if (rows > 8) units[at + 1] = make_int4(e, off + 8, rows - 8, 0);
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
        used += __popc(some) + __popc(big);
    }
    for (int i = used + lane; i < max_units; i += 32) units[i] = make_int4(0, 0, 0, 0);
    if (lane == 0) offsets[E] = base;
    __syncwarp();
    for (int n = lane; n < Tv; n += 32) {
        const int slot = s_off[s_ent[n]] + s_rank[n];
        perm[slot] = n;
        gslot[slot] = s_gate[n] * s_scale[n / k];
    }
}

}  // namespace rg
}  // namespace l4moe
