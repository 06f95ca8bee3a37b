// router_loss.cuh -- the losses that train a router next to the task's own,
// the per-expert counts of its choices, and the gradient of the logits.
//
// For T rows of E logits l (one row per token), a row counts when the mask
// keeps it and it holds a logit other than -inf; n = counted rows.
//   c_e  = number of entries (t, j), j < k, that choose expert e
//   f_e  = c_e / (k n)
//   p_te = softmax_e(l_t), or sigma(l_te) / sum_j sigma(l_tj)   (the score)
//   P_e  = (1 / n) sum_t p_te
//   balance = E sum_e f_e P_e          (1 where every expert is equally used)
//   z       = (1 / n) sum_t lse(l_t)^2
//   loss    = wb balance + wz z
// The choices are the layer's (topk.cuh): the k largest logits, the lower
// index first among equal ones, NaN never before a number; or they are given
// (entries outside [0, E) choose nothing: dropped tokens).  The counts have
// no derivative, so with a_e = wb E f_e / n and u the gradient of the loss
//   dl_te = u (p_te s_te (a_e - sum_j a_j p_tj) + (2 wz / n) lse_t softmax_te)
// with s = 1 for softmax and 1 - sigma(l_te) for the sigmoid score.  Rows
// that do not count have a gradient of zero, whatever they hold.
//
// Both passes read each logit once and are bound by that read (and the
// gradient's write) for long batches and by the launches for short ones.  A
// row is spread over L lanes of a warp, 8 neighbouring experts to a lane (one
// 16-byte load of a 16-bit row), so its sums and choices are butterflies of
// log2 L shuffles and small rows share a warp.  Sums are fp32, always in the
// same order.
//
// For long rows the arithmetic bounds both: 400 warp instructions per row
// of 256 in the values' pass and 240 in the gradient's (counted by a profiler
// for sigmoid and four choices: exponentials, reciprocals, keys and choices), where HBM delivers the
// 512 bytes in about 90 cycles of a scheduler.  Measured on one B200 (device time of values and
// gradient together): 65536 x 256 bf16, sigmoid, four choices: 59 to
// 60 us; 16384 x 128 fp32 18 us; 4096 x 16 bf16 7 us and 64 x 4 fp32
// 5 us (two launches).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "sm.cuh"

namespace l4moe {

constexpr int kLossThreads = 512;
constexpr int kLossWarps = kLossThreads / 32;
constexpr int kLossCluster = 8;  // blocks that add up through distributed shared memory
constexpr int kGradThreads = 256;
constexpr int kLossMaxExperts = 256;
constexpr int kLossMaxK = 4;
constexpr int kLossPer = 8;  // experts per lane

// Words (4 bytes) of the result: loss, balance, z, counted rows; counts [E]
// (int32); a_e [E]; 2 wz / n.
__host__ __device__ constexpr size_t loss_result_words(int E) { return 4 + 2 * (size_t)E + 1; }

// Words of one block's partial sums: P [E], counts [E], z, rows.
__host__ __device__ constexpr size_t loss_partial_words(int E) { return 2 * (size_t)E + 2; }

__device__ __forceinline__ void loss_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void loss_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void loss_store(__half* p, float v) { *p = __float2half_rn(v); }

// The hardware's 2^y, 1 / y and log2 y: within 2 ulp (the logarithm of values
// near 1: 2^-22 off at most, which is what the fp32 sum that it is taken of is
// off by itself); tiny values are zero.  Their errors are those of a few more
// fp32 steps, and they keep the division and logf's slow paths out of the rows.
__device__ __forceinline__ float hw_exp2(float y) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    return r;
}
__device__ __forceinline__ float hw_rcp(float y) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    return r;
}
__device__ __forceinline__ float hw_log2(float y) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    return r;
}

// e^x for logits of type IT: 2^(x log2 e) (off by 2 + 1.2 |x| ulp, most of it
// the product's rounding) where the logits and their gradient are 16-bit
// values, CUDA's expf for fp32.
template <typename IT>
__device__ __forceinline__ float loss_exp(float x) {
    if constexpr (sizeof(IT) == 2) return hw_exp2(x * 1.44269504f);
    else return expf(x);
}

// This lane's kLossPer logits of a row as they lie in memory.
template <typename IT>
struct Raw {
    static constexpr int W = kLossPer * (int)sizeof(IT) / 4;
    uint32_t w[W];

    // vec: E % 8 == 0 and aligned rows (a lane's experts are all there or none is)
    __device__ __forceinline__ void load(const IT* row, int e0, int E, bool vec) {
        if (vec) {
            if (e0 < E) {
#pragma unroll
                for (int q = 0; q < W / 4; ++q) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + e0) + q);
                    w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
                }
            }
        } else if constexpr (sizeof(IT) == 2) {
            const uint16_t* p = reinterpret_cast<const uint16_t*>(row + e0);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                w[i] = e0 + 2 * i < E ? p[2 * i] : 0u;
                if (e0 + 2 * i + 1 < E) w[i] |= (uint32_t)p[2 * i + 1] << 16;
            }
        } else {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(row + e0);
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = e0 + i < E ? p[i] : 0u;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0u;
    }
    // As fp32, -inf past the row's end (full: no lane of the warp reaches it).
    __device__ __forceinline__ void widen(float (&v)[kLossPer], int e0, int E, bool full) const {
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) {
            float f;
            if constexpr (std::is_same<IT, float>::value) f = __uint_as_float(w[i]);
            else if constexpr (std::is_same<IT, __nv_bfloat16>::value)
                f = __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
            else f = __half2float(__ushort_as_half((unsigned short)((i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu)));
            v[i] = f;
        }
        if (!full) {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) v[i] = e0 + i < E ? v[i] : -INFINITY;
        }
    }
};

template <int L>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Lanes of this lane's row among the warp's.
template <int L>
__device__ __forceinline__ unsigned row_lanes() {
    const unsigned lane = threadIdx.x & 31u;
    return L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1u) << (lane & ~(unsigned)(L - 1));
}

// One row: ex ~ its softmax (times inv: exactly that), sg ~ the score's shares
// (times iw), q = 1 - sigma (the sigmoid score), lse.
template <typename IT, int L, bool SIG>
struct RowStats {
    float ex[kLossPer], sg[kLossPer], q[kLossPer], inv, iw, lse;

    // The usual rows: the sum of e^l is in (1e-12, 1e20) in all of the warp's
    // rows, so nothing need be subtracted first, and sigma(l) = e^l / (1 +
    // e^l) takes no exponential of its own.  The bounds leave fp32's range to
    // what the gradient multiplies with: its factors (those of 2^31 rows are
    // near 1e-10, a loss scale of f16 is 65536) times the sum or 1 / the sum.
    // False, for the whole warp: not usual (a NaN, +inf, nothing above -inf, ...).
    __device__ __forceinline__ bool usual(const float (&v)[kLossPer]) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) {
            ex[i] = loss_exp<IT>(v[i]);
            s += ex[i];
        }
        s = row_sum<L>(s);
        if (__any_sync(0xffffffffu, !(s > 1e-12f && s < 1e20f))) return false;
        inv = hw_rcp(s);
        lse = hw_log2(s) * 0.693147181f;
        if constexpr (SIG) {
            float w = 0.f;
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) {
                q[i] = hw_rcp(1.0f + ex[i]);
                sg[i] = ex[i] * q[i];
                w += sg[i];
            }
            iw = hw_rcp(row_sum<L>(w));
        } else {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) sg[i] = ex[i];
            iw = inv;
        }
        return true;
    }

    // Any row that holds something above -inf.
    __device__ __forceinline__ void general(const float (&v)[kLossPer]) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) m = fmaxf(m, v[i]);  // NaN is passed over and comes back in the sum
        m = row_max<L>(m);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) {
            ex[i] = expf(v[i] - m);
            s += ex[i];
        }
        s = row_sum<L>(s);
        lse = m + logf(s);
        inv = 1.0f / s;
        iw = inv;
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) sg[i] = ex[i];
        if constexpr (SIG) {
            float w = 0.f, sv[kLossPer];
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) {
                const float t = expf(-fabsf(v[i])), r = 1.0f / (1.0f + t);
                sv[i] = v[i] >= 0.f ? r : t * r;
                q[i] = v[i] >= 0.f ? t * r : r;
                if (v[i] != v[i]) sv[i] = q[i] = v[i];
                w += sv[i];
            }
            w = row_sum<L>(w);
            // logits all below -30: sigma(l) = e^l to 2^-43, so the shares are
            // the softmax's (the sum of the sigmas may underflow there)
            if (!(m < -30.f)) {
                iw = 1.0f / w;
#pragma unroll
                for (int i = 0; i < kLossPer; ++i) sg[i] = sv[i];
            }
        }
    }

    // Whether the row counts, and its statistics; kept: the mask's word.
    // clean: no NaN in the warp's rows.  A row that does not count is given
    // zeros for logits, so that what it holds cannot matter.
    __device__ __forceinline__ bool compute(float (&v)[kLossPer], bool kept, int e0, int E, bool& clean) {
        clean = true;
        if (usual(v)) return kept;
        clean = false;
        bool some = false;
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) some |= v[i] != -INFINITY;
        const unsigned who = __ballot_sync(0xffffffffu, some);  // (every lane votes, kept or not)
        const bool counted = kept && (who & row_lanes<L>()) != 0u;
        if (!counted) {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) v[i] = e0 + i < E ? 0.f : -INFINITY;
        }
        if (!usual(v)) general(v);
        return counted;
    }
};

// A logit as an unsigned number in the order of the choice: numbers by value
// (-0 as +0), then NaN (1); 0 is kept for "taken" and for lanes past the row.
__device__ __forceinline__ uint32_t choice_key(float v) {
    if (v != v) return 1u;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int L>
__device__ __forceinline__ uint32_t row_umax(uint32_t v) {
    if constexpr (L == 32) return __reduce_max_sync(0xffffffffu, v);
    else {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
}

// a >= b
__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}

// Counts the k choices of a row (its first lane adds to `counts` when the row
// is counted), `key` holding a 32-bit key per expert whose low 10 bits are
// 1023 - expert: the largest key is the next choice.
template <int L>
__device__ __forceinline__ void count_keys(uint32_t (&key)[kLossPer], int k, bool adds, int* counts) {
    if (k <= 2) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < kLossPer; ++i) best = max(best, key[i]);
        best = row_umax<L>(best);
        if (adds) atomicAdd(counts + (1023 - (int)(best & 1023u)), 1);
        if (k == 2) {
            const uint32_t first = best;
            best = 0u;
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) best = max(best, key[i] == first ? 0u : key[i]);
            best = row_umax<L>(best);
            if (adds) atomicAdd(counts + (1023 - (int)(best & 1023u)), 1);
        }
        return;
    }
    // the lane's four largest in order (two fours sorted, the larger of the
    // opposite pairs, sorted again), then each choice takes a lane's first
#pragma unroll
    for (int q = 0; q < 8; q += 4) {
        order(key[q], key[q + 1]);
        order(key[q + 2], key[q + 3]);
        order(key[q], key[q + 2]);
        order(key[q + 1], key[q + 3]);
        order(key[q + 1], key[q + 2]);
    }
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = max(key[i], key[7 - i]);
    order(h[0], h[2]);
    order(h[1], h[3]);
    order(h[0], h[1]);
    order(h[2], h[3]);
    for (int j = 0; j < k; ++j) {
        const uint32_t best = row_umax<L>(h[0]);
        const bool mine = best == h[0];
        h[0] = mine ? h[1] : h[0];
        h[1] = mine ? h[2] : h[1];
        h[2] = mine ? h[3] : h[2];
        h[3] = mine ? 0u : h[3];
        if (adds) atomicAdd(counts + (1023 - (int)(best & 1023u)), 1);
    }
}

// Counts the k choices of a row of 16-bit logits: value and index fit one
// 32-bit key.  clean: no NaN in the warp's rows.
template <typename IT, int L>
__device__ __forceinline__ void count_choices16(const Raw<IT>& raw, const float (&v)[kLossPer], bool clean, int e0, int E,
                                                int k, bool adds, int* counts) {
    uint32_t key[kLossPer];
    if (clean) {
#pragma unroll
        for (int i = 0; i < kLossPer / 2; ++i) {
            uint32_t w;  // + 0: -0 becomes +0
            if constexpr (std::is_same<IT, __half>::value) {
                const __half2 z = __hadd2(*reinterpret_cast<const __half2*>(&raw.w[i]), __half2{__half(0.f), __half(0.f)});
                w = *reinterpret_cast<const uint32_t*>(&z);
            } else {
                const __nv_bfloat162 z =
                    __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&raw.w[i]), __floats2bfloat162_rn(0.f, 0.f));
                w = *reinterpret_cast<const uint32_t*>(&z);
            }
            // both halves as unsigned numbers in the order of their values
            const uint32_t neg = (w >> 15) & 0x00010001u;
            w ^= (neg * 0xffffu) | 0x80008000u;
            key[2 * i] = w << 16;
            key[2 * i + 1] = w & 0xffff0000u;
        }
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) key[i] |= (uint32_t)(1023 - (e0 + i));
        if (E < L * kLossPer) {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) key[i] = e0 + i < E ? key[i] : 0u;
        }
    } else {
        // (a widened 16-bit value's key: its low 13 bits carry nothing)
#pragma unroll
        for (int i = 0; i < kLossPer; ++i)
            key[i] = e0 + i < E ? (choice_key(v[i]) & ~1023u) | (uint32_t)(1023 - (e0 + i)) : 0u;
    }
    count_keys<L>(key, k, adds, counts);
}

// The same of fp32 logits: the largest value, then the lowest index that holds it.
template <int L>
__device__ __forceinline__ void count_choices32(const float (&v)[kLossPer], int e0, int E, int k, bool adds, int* counts) {
    uint32_t key[kLossPer];
#pragma unroll
    for (int i = 0; i < kLossPer; ++i) key[i] = e0 + i < E ? choice_key(v[i]) : 0u;
    for (int j = 0; j < k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < kLossPer; ++i) best = max(best, key[i]);
        best = row_umax<L>(best);
        uint32_t at = 0u;  // kLossMaxExperts - index: the largest is the lowest index
#pragma unroll
        for (int i = kLossPer - 1; i >= 0; --i)
            if (key[i] == best) at = (uint32_t)(kLossMaxExperts - (e0 + i));
        const int e = kLossMaxExperts - (int)row_umax<L>(at);
#pragma unroll
        for (int i = 0; i < kLossPer; ++i)
            if (e0 + i == e) key[i] = 0u;
        if (adds) atomicAdd(counts + e, 1);
    }
}

// The result from the totals P [E], c [E], z and n (shared memory).  All
// threads of a block; at most 1024.
__device__ __forceinline__ void write_result(const float* P, const int* c, float z, long long rows, int E, int k,
                                             float wb, float wz, float* result) {
    __shared__ float s_red[32];
    const int tid = threadIdx.x;
    const float n = rows > 0 ? (float)rows : 1.0f, per = 1.0f / n, perk = per / (float)k;
    float bal = 0.f;
    for (int e = tid; e < E; e += blockDim.x) {
        const float f = (float)c[e] * perk;
        bal = fmaf(f, P[e] * per, bal);
        reinterpret_cast<int*>(result)[4 + e] = c[e];
        result[4 + E + e] = wb * (float)E * f * per;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bal += __shfl_xor_sync(0xffffffffu, bal, o);
    if ((tid & 31) == 0) s_red[tid >> 5] = bal;
    __syncthreads();
    if (tid < 32) {
        float b = tid < (int)(blockDim.x >> 5) ? s_red[tid] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
        if (tid == 0) {
            b *= (float)E;
            z *= per;
            result[0] = fmaf(wb, b, wz * z);
            result[1] = b;
            result[2] = z;
            result[3] = (float)rows;
            result[4 + 2 * E] = 2.0f * wz * per;
        }
    }
}

// The result from the sums of a launch's B blocks, one cluster, each with its
// own in shared memory: the first block adds them in order and writes.  All
// threads of all blocks.
__device__ __forceinline__ void cluster_result(const float* P, const int* c, const float* z, const int* n, int B, int E,
                                               int k, float wb, float wz, float* result) {
    __shared__ float t_p[kLossMaxExperts];
    __shared__ int t_c[kLossMaxExperts];
    if (B > 1) op::cluster_sync();
    else __syncthreads();
    if (blockIdx.x == 0) {
        auto at = [&](const void* p, int b) { return op::ld_cluster_u32(op::mapa(op::smem_u32(p), (uint32_t)b)); };
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            uint32_t pv[kLossCluster], cv[kLossCluster];
#pragma unroll
            for (int b = 0; b < kLossCluster; ++b)
                if (b < B) pv[b] = at(P + e, b), cv[b] = at(c + e, b);
            float p = 0.f;
            int count = 0;
#pragma unroll
            for (int b = 0; b < kLossCluster; ++b)
                if (b < B) p += __uint_as_float(pv[b]), count += (int)cv[b];
            t_p[e] = p;
            t_c[e] = count;
        }
        uint32_t zv[kLossCluster], nv[kLossCluster];
#pragma unroll
        for (int b = 0; b < kLossCluster; ++b)
            if (b < B) zv[b] = at(z, b), nv[b] = at(n, b);
        float zs = 0.f;
        long long rows = 0;
#pragma unroll
        for (int b = 0; b < kLossCluster; ++b)
            if (b < B) zs += __uint_as_float(zv[b]), rows += (int)nv[b];
        __syncthreads();
        write_result(t_p, t_c, zs, rows, E, k, wb, wz, result);
    }
    if (B > 1) op::cluster_sync();  // the sums stay until the first block has read them
}

// Sums of each block's rows.  Up to kLossCluster blocks are one cluster whose
// first block adds the others' sums, over distributed shared memory, and
// writes the result; more blocks leave partials for the finishing kernel.
template <typename IT, int L, bool SIG>
__global__ void __launch_bounds__(kLossThreads, 2) router_loss_kernel(
    const IT* __restrict__ logits, long long ld, int T, int E, int k, int vec, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ idx, float wb, float wz, float* __restrict__ part, float* __restrict__ result) {
    op::pdl_enter();
    __shared__ float s_p[kLossWarps][kLossMaxExperts];
    __shared__ float s_z[kLossWarps];
    __shared__ int s_c[kLossMaxExperts];
    __shared__ int s_n[kLossWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int R = 32 / L;  // rows a warp takes at a time
    const int sub = lane & (L - 1), grp = lane / L;
    const int e0 = sub * kLossPer;
    for (int e = tid; e < E; e += kLossThreads) s_c[e] = 0;
    __syncthreads();
    float ps[kLossPer];
#pragma unroll
    for (int i = 0; i < kLossPer; ++i) ps[i] = 0.f;
    float zs = 0.f;
    int n = 0;
    const long long step = (long long)gridDim.x * kLossWarps * R;
    const long long first = ((long long)blockIdx.x * kLossWarps + warp) * R;
    Raw<IT> next;
    next.clear();
    if (first + grp < T) next.load(logits + (first + grp) * ld, e0, E, vec != 0);
    const bool full = E == L * kLossPer;
    for (long long t0 = first; t0 < T; t0 += step) {
        const long long t = t0 + grp;
        const bool kept = t < T && (!mask || mask[t] != 0);
        const Raw<IT> raw = next;
        next.clear();
        if (t + step < T) next.load(logits + (t + step) * ld, e0, E, vec != 0);  // the next row is on its way meanwhile
        float v[kLossPer];
        raw.widen(v, e0, E, full);
        RowStats<IT, L, SIG> st;
        bool clean, counted;
        if (idx) {
            counted = st.compute(v, kept, e0, E, clean);
            for (int j = sub; j < k; j += L) {
                const int e = counted ? idx[t * k + j] : -1;
                if (e >= 0 && e < E) atomicAdd(&s_c[e], 1);
            }
        } else if constexpr (sizeof(IT) == 4) {
            float u[kLossPer];
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) u[i] = v[i];
            counted = st.compute(v, kept, e0, E, clean);
            count_choices32<L>(u, e0, E, k, counted && sub == 0, s_c);
        } else {
            counted = st.compute(v, kept, e0, E, clean);
            if (!clean) raw.widen(v, e0, E, full);
            count_choices16<IT, L>(raw, v, clean, e0, E, k, counted && sub == 0, s_c);
        }
        const float w = counted ? st.iw : 0.0f;  // (a row that does not count has finite values)
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) ps[i] = fmaf(w, st.sg[i], ps[i]);
        if (sub == 0 && counted) {
            zs += st.lse * st.lse;
            ++n;
        }
    }
    // the groups of a warp, then the warps
#pragma unroll
    for (int o = 16; o >= L; o >>= 1) {
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) ps[i] += __shfl_xor_sync(0xffffffffu, ps[i], o);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        zs += __shfl_xor_sync(0xffffffffu, zs, o);
        n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if (grp == 0) {
#pragma unroll
        for (int i = 0; i < kLossPer; ++i)
            if (e0 + i < E) s_p[warp][e0 + i] = ps[i];
    }
    if (lane == 0) {
        s_z[warp] = zs;
        s_n[warp] = n;
    }
    __syncthreads();
    const bool alone = gridDim.x <= kLossCluster;  // one cluster is the whole launch
    float* mine = part + blockIdx.x * loss_partial_words(E);
    for (int e = tid; e < E; e += kLossThreads) {
        float p = 0.f;
#pragma unroll
        for (int w = 0; w < kLossWarps; ++w) p += s_p[w][e];
        if (alone) s_p[0][e] = p;  // read above by this thread alone
        else {
            mine[e] = p;
            mine[E + e] = __int_as_float(s_c[e]);
        }
    }
    if (tid == 0) {
        float z = 0.f;
        int c = 0;
#pragma unroll
        for (int w = 0; w < kLossWarps; ++w) {
            z += s_z[w];
            c += s_n[w];
        }
        if (alone) {
            s_z[0] = z;
            s_n[0] = c;
        } else {
            mine[2 * E] = z;
            mine[2 * E + 1] = __int_as_float(c);
        }
    }
    if (alone) cluster_result(s_p[0], s_c, s_z, s_n, gridDim.x, E, k, wb, wz, result);
}

// Adds the blocks' partials: one cluster of kLossCluster blocks of 1024
// threads, each expert's partials dealt out to the threads that share it,
// their sums added in a fixed order.
__global__ void __launch_bounds__(1024) router_loss_finish_kernel(const float* __restrict__ part, int blocks, int E,
                                                                  int lg, int k, float wb, float wz,
                                                                  float* __restrict__ result) {
    op::pdl_enter();
    __shared__ float s_p[1024], s_z[32];
    __shared__ int s_c[1024], s_n[32];
    const int tid = threadIdx.x, lane = tid & 31;
    const size_t W = loss_partial_words(E);
    const int e = tid & ((1 << lg) - 1), share = tid >> lg, shares = 1024 >> lg;  // 2^lg >= E columns
    float p = 0.f, z = 0.f;
    int c = 0, n = 0;
    const int mine = blockIdx.x + tid * kLossCluster;  // this thread's partial for z and n (at most 1024 in all)
    if (mine < blocks) {
        z = __ldcg(part + mine * W + 2 * E);
        n = __float_as_int(__ldcg(part + mine * W + 2 * E + 1));
    }
    if (e < E) {
#pragma unroll 8
        for (int b = blockIdx.x * shares + share; b < blocks; b += kLossCluster * shares) {
            p += __ldcg(part + b * W + e);
            c += __float_as_int(__ldcg(part + b * W + E + e));
        }
    }
    s_p[tid] = p;
    s_c[tid] = c;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
        n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if (lane == 0) {
        s_z[tid >> 5] = z;
        s_n[tid >> 5] = n;
    }
    for (int q = shares >> 1; q > 0; q >>= 1) {  // halves of the shares in turn
        __syncthreads();
        if (share < q) {
            s_p[tid] += s_p[tid + (q << lg)];
            s_c[tid] += s_c[tid + (q << lg)];
        }
    }
    __syncthreads();
    if (tid < 32) {
        z = s_z[lane];
        n = s_n[lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            z += __shfl_xor_sync(0xffffffffu, z, o);
            n += __shfl_xor_sync(0xffffffffu, n, o);
        }
        __syncwarp();
        if (lane == 0) {
            s_z[0] = z;
            s_n[0] = n;
        }
    }
    cluster_result(s_p, s_c, s_z, s_n, kLossCluster, E, k, wb, wz, result);
}

// The gradient of the logits (the rows' statistics are computed again: they
// cost less than a second pass over saved ones would).
template <typename IT, int L, bool SIG>
__global__ void __launch_bounds__(kGradThreads) router_loss_grad_kernel(
    const IT* __restrict__ logits, long long ld, int T, int E, int vec, const uint8_t* __restrict__ mask,
    const float* __restrict__ result, const float* __restrict__ upstream, IT* __restrict__ dl, long long ldd) {
    op::pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int R = 32 / L;
    const int sub = lane & (L - 1), grp = lane / L;
    const int e0 = sub * kLossPer;
    const float u = upstream ? *upstream : 1.0f;
    const float zc = u * result[4 + 2 * E];
    float a[kLossPer];
#pragma unroll
    for (int i = 0; i < kLossPer; ++i) a[i] = e0 + i < E ? u * result[4 + E + e0 + i] : 0.f;
    const long long step = (long long)gridDim.x * (kGradThreads / 32) * R;
    const long long first = ((long long)blockIdx.x * (kGradThreads / 32) + warp) * R;
    Raw<IT> next;
    next.clear();
    if (first + grp < T) next.load(logits + (first + grp) * ld, e0, E, vec != 0);
    const bool full = E == L * kLossPer;
    for (long long t0 = first; t0 < T; t0 += step) {
        const long long t = t0 + grp;
        const bool in = t < T;
        const bool kept = in && (!mask || mask[t] != 0);
        float v[kLossPer];
        next.widen(v, e0, E, full);
        next.clear();
        if (t + step < T) next.load(logits + (t + step) * ld, e0, E, vec != 0);  // the next row is on its way meanwhile
        RowStats<IT, L, SIG> st;
        bool clean;
        const bool counted = st.compute(v, kept, e0, E, clean);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) dot = fmaf(a[i], st.sg[i], dot);
        dot = row_sum<L>(dot) * st.iw;
        const float zl = zc * st.lse * st.inv;
        float g[kLossPer];
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) {
            float w = st.sg[i] * (st.iw * (a[i] - dot));
            if constexpr (SIG) w *= st.q[i];
            g[i] = fmaf(zl, st.ex[i], w);
        }
        if (!counted) {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) g[i] = 0.f;
        }
        if (!in) continue;
        IT* row = dl + t * ldd;
        if (vec) {
            if (e0 < E) {
                constexpr int V = 16 / (int)sizeof(IT);
#pragma unroll
                for (int q = 0; q < kLossPer / V; ++q) {
                    IT tmp[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) loss_store(tmp + i, g[q * V + i]);
                    reinterpret_cast<uint4*>(row + e0)[q] = *reinterpret_cast<const uint4*>(tmp);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i)
                if (e0 + i < E) loss_store(row + e0 + i, g[i]);
        }
    }
}

}  // namespace l4moe
