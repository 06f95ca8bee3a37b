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
// log2 L shuffles and small rows share a warp.  Sums are fp32 in a lane and a
// block, 64-bit across blocks, always in the same order.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

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

__device__ __forceinline__ float loss_to_f32(float v) { return v; }
__device__ __forceinline__ float loss_to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float loss_to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void loss_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void loss_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void loss_store(__half* p, float v) { *p = __float2half_rn(v); }

// exp for logits of type IT: the fast one (off by 2 + 1.2 |x| ulp) where the
// logits and their gradient are 16-bit values.
template <typename IT>
__device__ __forceinline__ float loss_exp(float x) {
    if constexpr (sizeof(IT) == 2) return __expf(x);
    else return expf(x);
}

// This lane's kLossPer logits of a row, -inf past the row's end.
template <typename IT>
__device__ __forceinline__ void loss_load(const IT* row, int e0, int E, bool vec, float (&v)[kLossPer]) {
    constexpr int V = 16 / (int)sizeof(IT);
    if (vec) {  // E % 8 == 0 and aligned rows: a lane's experts are all there or none is
        if (e0 < E) {
#pragma unroll
            for (int q = 0; q < kLossPer / V; ++q) {
                IT tmp[V];
                *reinterpret_cast<uint4*>(tmp) = __ldg(reinterpret_cast<const uint4*>(row + e0) + q);
#pragma unroll
                for (int i = 0; i < V; ++i) v[q * V + i] = loss_to_f32(tmp[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) v[i] = -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) v[i] = e0 + i < E ? loss_to_f32(row[e0 + i]) : -INFINITY;
    }
}

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

// One row's statistics: p (the score's share of each expert), slope (its
// factor 1 - sigma), soft (softmax), lse.
template <typename IT, int L, bool SIG>
struct RowStats {
    float soft[kLossPer], p[kLossPer], slope[kLossPer], lse;

    // The usual rows: no logit above 40 and a sum of exponentials that is not
    // tiny in any of the warp's rows, so nothing need be subtracted first and
    // sigma(l) = e^l / (1 + e^l) takes one exponential.  False (for the whole
    // warp): take general().
    __device__ __forceinline__ bool usual(const float (&v)[kLossPer]) {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < kLossPer; ++i) m = fmaxf(m, v[i]);
        if (__any_sync(0xffffffffu, m > 40.f)) return false;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) {
            soft[i] = loss_exp<IT>(v[i]);
            s += soft[i];
        }
        s = row_sum<L>(s);
        if (__any_sync(0xffffffffu, !(s > 1e-12f))) return false;  // (a NaN too)
        if constexpr (SIG) {
            float w = 0.f;
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) {
                slope[i] = __fdividef(1.0f, 1.0f + soft[i]);
                p[i] = soft[i] * slope[i];
                w += p[i];
            }
            w = row_sum<L>(w);
            const float iw = __fdividef(1.0f, w);
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) p[i] *= iw;
        }
        lse = __logf(s);
        const float inv = __fdividef(1.0f, s);
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) {
            soft[i] *= inv;
            if constexpr (!SIG) p[i] = soft[i];
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
            soft[i] = expf(v[i] - m);
            s += soft[i];
        }
        s = row_sum<L>(s);
        lse = m + logf(s);
        const float inv = 1.0f / s;
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) soft[i] *= inv;
        if constexpr (SIG) {
            float w = 0.f;
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) {
                const float t = expf(-fabsf(v[i])), r = 1.0f / (1.0f + t);
                p[i] = v[i] >= 0.f ? r : t * r;
                slope[i] = v[i] >= 0.f ? t * r : r;
                if (v[i] != v[i]) p[i] = slope[i] = v[i];
                w += p[i];
            }
            w = row_sum<L>(w);
            // logits all below -30: sigma(l) = e^l to 2^-43, so the shares are
            // the softmax's (the sum of the sigmas may underflow there)
            const bool deep = m < -30.f;
            const float iw = 1.0f / w;
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) p[i] = deep ? soft[i] : p[i] * iw;
        } else {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) p[i] = soft[i];
        }
    }

    // v: a row's logits (-inf past its end); a row that does not count is
    // replaced by zeros first, so that what it holds cannot matter.
    __device__ __forceinline__ void compute(float (&v)[kLossPer], bool counted, int e0, int E) {
        if (!counted) {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) v[i] = e0 + i < E ? 0.f : -INFINITY;
        }
        if (!usual(v)) general(v);
    }
};

// Whether a row holds a logit other than -inf.
template <int L>
__device__ __forceinline__ bool row_any(const float (&v)[kLossPer]) {
    bool some = false;
#pragma unroll
    for (int i = 0; i < kLossPer; ++i) some |= v[i] != -INFINITY;
    return (__ballot_sync(0xffffffffu, some) & row_lanes<L>()) != 0u;
}

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

// Counts the k choices of a row (its first lane adds to `counts` when the row
// is counted).  16-bit logits: value and index fit one 32-bit key (the value
// decides, then the lower index), so that a choice is one maximum; fp32: the
// largest value, then the lowest index that holds it.
template <typename IT, int L>
__device__ __forceinline__ void count_choices(const float (&v)[kLossPer], int e0, int E, int k, bool adds, int* counts) {
    uint32_t key[kLossPer];
#pragma unroll
    for (int i = 0; i < kLossPer; ++i) {
        key[i] = e0 + i < E ? choice_key(v[i]) : 0u;
        if constexpr (sizeof(IT) == 2) {
            // the lower 13 bits (f16) or 16 (bf16) of a widened value carry
            // nothing: ones for a negative one's key, zeros otherwise; 10 bits
            // are enough for the index
            if (e0 + i < E) key[i] = (key[i] & ~1023u) | (uint32_t)(1023 - (e0 + i));
        }
    }
    for (int j = 0; j < k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < kLossPer; ++i) best = max(best, key[i]);
        best = row_umax<L>(best);
        int e;
        if constexpr (sizeof(IT) == 2) {
            e = 1023 - (int)(best & 1023u);
        } else {
            uint32_t at = 0u;  // kLossMaxExperts - index: the largest is the lowest index
#pragma unroll
            for (int i = kLossPer - 1; i >= 0; --i)
                if (key[i] == best) at = (uint32_t)(kLossMaxExperts - (e0 + i));
            e = kLossMaxExperts - (int)row_umax<L>(at);
        }
#pragma unroll
        for (int i = 0; i < kLossPer; ++i)
            if (e0 + i == e) key[i] = 0u;
        if (adds && e < E) atomicAdd(counts + e, 1);
    }
}

// The result from the totals P [E], c [E], z and n (shared memory).  All
// threads of a block; at most 1024.
__device__ __forceinline__ void write_result(const double* P, const int* c, double z, long long rows, int E, int k,
                                             float wb, float wz, float* result) {
    __shared__ double s_red[32];
    const int tid = threadIdx.x;
    const double n = rows > 0 ? (double)rows : 1.0;
    double bal = 0.0;
    for (int e = tid; e < E; e += blockDim.x) {
        const double f = (double)c[e] / ((double)k * n);
        bal += f * P[e];
        reinterpret_cast<int*>(result)[4 + e] = c[e];
        result[4 + E + e] = (float)((double)wb * E * f / n);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bal += __shfl_xor_sync(0xffffffffu, bal, o);
    if ((tid & 31) == 0) s_red[tid >> 5] = bal;
    __syncthreads();
    if (tid == 0) {
        double b = 0.0;
        for (int w = 0; w < (int)(blockDim.x + 31) / 32; ++w) b += s_red[w];
        b *= (double)E / n;
        z /= n;
        result[0] = (float)((double)wb * b + (double)wz * z);
        result[1] = (float)b;
        result[2] = (float)z;
        result[3] = (float)rows;
        result[4 + 2 * E] = (float)(2.0 * (double)wz / n);
    }
}

// Sums of each block's rows.  Up to kLossCluster blocks are one cluster whose
// first block adds the others' sums, over distributed shared memory, and
// writes the result; more blocks leave partials for the finishing kernel.
template <typename IT, int L, bool SIG>
__global__ void __launch_bounds__(kLossThreads) router_loss_kernel(
    const IT* __restrict__ logits, long long ld, int T, int E, int k, int vec, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ idx, float wb, float wz, float* __restrict__ part, float* __restrict__ result) {
    op::pdl_enter();
    __shared__ float s_p[kLossWarps][kLossMaxExperts];
    __shared__ float s_z[kLossWarps];
    __shared__ int s_c[kLossMaxExperts];
    __shared__ int s_n[kLossWarps];
    __shared__ double t_p[kLossMaxExperts];
    __shared__ int t_c[kLossMaxExperts];
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
    for (long long t0 = ((long long)blockIdx.x * kLossWarps + warp) * R; t0 < T; t0 += step) {
        const long long t = t0 + grp;
        const bool in = t < T;
        const bool kept = in && (!mask || mask[t] != 0);
        float v[kLossPer];
        if (in) loss_load(logits + t * ld, e0, E, vec != 0, v);
        else {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) v[i] = -INFINITY;
        }
        const bool counted = row_any<L>(v) && kept;
        if (idx) {
            for (int j = sub; j < k; j += L) {
                const int e = counted ? idx[t * k + j] : -1;
                if (e >= 0 && e < E) atomicAdd(&s_c[e], 1);
            }
        } else {
            count_choices<IT, L>(v, e0, E, k, counted && sub == 0, s_c);
        }
        RowStats<IT, L, SIG> st;
        st.compute(v, counted, e0, E);
        const float w = counted ? 1.0f : 0.0f;  // (a row that does not count has finite values)
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) ps[i] = fmaf(w, st.p[i], ps[i]);
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
    if (!alone) return;
    const int B = gridDim.x;
    if (B > 1) op::cluster_sync();
    else __syncthreads();
    if (blockIdx.x == 0) {
        auto at = [&](const void* p, int b) { return op::ld_cluster_u32(op::mapa(op::smem_u32(p), (uint32_t)b)); };
        for (int e = tid; e < E; e += kLossThreads) {
            uint32_t pv[kLossCluster], cv[kLossCluster];
#pragma unroll
            for (int b = 0; b < kLossCluster; ++b)
                if (b < B) pv[b] = at(&s_p[0][e], b), cv[b] = at(&s_c[e], b);
            double p = 0.0;
            int c = 0;
#pragma unroll
            for (int b = 0; b < kLossCluster; ++b)
                if (b < B) p += (double)__uint_as_float(pv[b]), c += (int)cv[b];
            t_p[e] = p;
            t_c[e] = c;
        }
        double z = 0.0;
        long long rows = 0;
        for (int b = 0; b < B; ++b) {
            z += (double)__uint_as_float(at(&s_z[0], b));
            rows += (int)at(&s_n[0], b);
        }
        __syncthreads();
        write_result(t_p, t_c, z, rows, E, k, wb, wz, result);
    }
    if (B > 1) op::cluster_sync();  // the sums stay until the first block has read them
}

// Adds the blocks' partials: 1024 threads, each expert's blocks dealt out to
// the 1024 / 2^k threads that share it, their sums added in order.
__global__ void __launch_bounds__(1024) router_loss_finish_kernel(const float* __restrict__ part, int blocks, int E,
                                                                  int k, float wb, float wz,
                                                                  float* __restrict__ result) {
    op::pdl_enter();
    __shared__ double s_p[1024];
    __shared__ int s_c[1024];
    __shared__ double s_z[32];
    __shared__ long long s_n[32];
    const int tid = threadIdx.x;
    const size_t W = loss_partial_words(E);
    int lg = 0;  // columns: E rounded up to a power of two
    while ((1 << lg) < E) ++lg;
    const int e = tid & ((1 << lg) - 1), share = tid >> lg, shares = 1024 >> lg;
    double p = 0.0;
    int c = 0;
    if (e < E) {
#pragma unroll 8
        for (int b = share; b < blocks; b += shares) {
            p += (double)__ldcg(part + b * W + e);
            c += __float_as_int(__ldcg(part + b * W + E + e));
        }
    }
    s_p[tid] = p;
    s_c[tid] = c;
    double z = 0.0;
    long long rows = 0;
    if (tid < blocks) {  // at most 1024
        z = (double)__ldcg(part + tid * W + 2 * E);
        rows = __float_as_int(__ldcg(part + tid * W + 2 * E + 1));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
        rows += __shfl_xor_sync(0xffffffffu, rows, o);
    }
    if ((tid & 31) == 0) {
        s_z[tid >> 5] = z;
        s_n[tid >> 5] = rows;
    }
    __syncthreads();
    if (tid < E) {
        p = s_p[tid];
        c = s_c[tid];
        for (int q = 1; q < shares; ++q) {
            p += s_p[(q << lg) + tid];
            c += s_c[(q << lg) + tid];
        }
    }
    z = 0.0;
    rows = 0;
    for (int w = 0; w < 32; ++w) {
        z += s_z[w];
        rows += s_n[w];
    }
    __syncthreads();
    if (tid < E) {
        s_p[tid] = p;
        s_c[tid] = c;
    }
    __syncthreads();
    write_result(s_p, s_c, z, rows, E, k, wb, wz, result);
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
    for (long long t0 = ((long long)blockIdx.x * (kGradThreads / 32) + warp) * R; t0 < T; t0 += step) {
        const long long t = t0 + grp;
        const bool in = t < T;
        const bool kept = in && (!mask || mask[t] != 0);
        float v[kLossPer];
        if (in) loss_load(logits + t * ld, e0, E, vec != 0, v);
        else {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) v[i] = -INFINITY;
        }
        const bool counted = row_any<L>(v) && kept;
        RowStats<IT, L, SIG> st;
        st.compute(v, counted, e0, E);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) dot = fmaf(a[i], st.p[i], dot);
        dot = row_sum<L>(dot);
        const float zl = zc * st.lse;
        float g[kLossPer];
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) {
            float w = st.p[i] * (a[i] - dot);
            if constexpr (SIG) w *= st.slope[i];
            g[i] = counted ? fmaf(zl, st.soft[i], w) : 0.f;
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
