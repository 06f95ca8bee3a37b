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
// 16-byte load of a 16-bit row), so its maximum, sums and choices are
// butterflies of log2 L shuffles and small rows share a warp.  Sums are
// fp32 in a lane and a block, 64-bit across blocks, always in the same order.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "sm.cuh"

namespace l4moe {

constexpr int kLossThreads = 256;
constexpr int kLossWarps = kLossThreads / 32;
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

// exp and log for logits of type IT: the fast exp (2 ulp and the rounding of
// its scaled argument, below 2^-18 for |x| < 30) where the logits and their
// gradient are 16-bit values, the accurate one for fp32.
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

// One row's statistics: p (the score's share of each expert), slope (its
// factor 1 - sigma), soft (softmax), lse.
template <typename IT, int L, bool SIG>
struct RowStats {
    float soft[kLossPer], p[kLossPer], slope[kLossPer], lse;
    bool any;  // some logit is not -inf

    __device__ __forceinline__ void compute(const float (&v)[kLossPer]) {
        float m = -INFINITY;
        bool some = false;
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) {
            m = fmaxf(m, v[i]);  // NaN is passed over here and comes back through the sum
            some |= v[i] != -INFINITY;
        }
        m = row_max<L>(m);
        unsigned who = __ballot_sync(0xffffffffu, some);
        const unsigned lane = threadIdx.x & 31u;
        const unsigned mine = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1u) << (lane & ~(unsigned)(L - 1));
        any = (who & mine) != 0u;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) {
            soft[i] = loss_exp<IT>(v[i] - m);
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
                const float t = loss_exp<IT>(-fabsf(v[i])), r = 1.0f / (1.0f + t);
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
};

// A logit as an unsigned number in the order of the choice: numbers by value
// (-0 as +0), then NaN; 0 is kept for "taken" and for lanes past the row.
__device__ __forceinline__ uint32_t choice_key(float v) {
    if (v != v) return 1u;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sums the blocks' partials (in block order, 64-bit) and writes the result.
// Called by all threads of one block, at most 1024 of them.
__device__ __forceinline__ void loss_finish(const float* part, int blocks, int E, int k, float wb, float wz,
                                            float* result) {
    __shared__ double s_p[kLossMaxExperts], s_red[32];
    __shared__ int s_c[kLossMaxExperts];
    __shared__ double s_z;
    __shared__ long long s_n;
    const int tid = threadIdx.x;
    const size_t W = loss_partial_words(E);
    for (int e = tid; e < E; e += blockDim.x) {
        double p = 0.0;
        int c = 0;
        for (int b = 0; b < blocks; ++b) {
            p += (double)__ldcg(part + b * W + e);
            c += __float_as_int(__ldcg(part + b * W + E + e));
        }
        s_p[e] = p;
        s_c[e] = c;
    }
    if (tid < 32) {
        double z = 0.0;
        long long n = 0;
        for (int b = tid; b < blocks; b += 32) {
            z += (double)__ldcg(part + b * W + 2 * E);
            n += __float_as_int(__ldcg(part + b * W + 2 * E + 1));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            z += __shfl_xor_sync(0xffffffffu, z, o);
            n += __shfl_xor_sync(0xffffffffu, n, o);
        }
        if (tid == 0) {
            s_z = z;
            s_n = n;
        }
    }
    __syncthreads();
    const double n = s_n > 0 ? (double)s_n : 1.0;
    double bal = 0.0;
    for (int e = tid; e < E; e += blockDim.x) {
        const double f = (double)s_c[e] / ((double)k * n);
        bal += f * s_p[e];
        reinterpret_cast<int*>(result)[4 + e] = s_c[e];
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
        const double z = s_z / n;
        result[0] = (float)((double)wb * b + (double)wz * z);
        result[1] = (float)b;
        result[2] = (float)z;
        result[3] = (float)s_n;
        result[4 + 2 * E] = (float)(2.0 * (double)wz / n);
    }
}

// Partial sums of each block's rows; with one block, the result too.
template <typename IT, int L, bool SIG>
__global__ void __launch_bounds__(kLossThreads) router_loss_kernel(
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
    for (long long t0 = ((long long)blockIdx.x * kLossWarps + warp) * R; t0 < T; t0 += step) {
        const long long t = t0 + grp;
        const bool in = t < T;
        float v[kLossPer];
        if (in) loss_load(logits + t * ld, e0, E, vec != 0, v);
        else {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) v[i] = -INFINITY;
        }
        RowStats<IT, L, SIG> st;
        st.compute(v);
        const bool counted = in && st.any && (!mask || mask[t] != 0);
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) ps[i] += counted ? st.p[i] : 0.f;
        if (sub == 0 && counted) {
            zs += st.lse * st.lse;
            ++n;
        }
        if (idx) {
            for (int j = sub; j < k; j += L) {
                const int e = counted ? idx[t * k + j] : -1;
                if (e >= 0 && e < E) atomicAdd(&s_c[e], 1);
            }
        } else {
            uint32_t key[kLossPer];
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) key[i] = e0 + i < E ? choice_key(v[i]) : 0u;
            for (int j = 0; j < k; ++j) {
                uint32_t best = 0u;
                int at = 0;
#pragma unroll
                for (int i = 0; i < kLossPer; ++i)
                    if (key[i] > best) {
                        best = key[i];
                        at = i;
                    }
                int e = e0 + at;
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) {
                    const uint32_t ob = __shfl_xor_sync(0xffffffffu, best, o);
                    const int oe = __shfl_xor_sync(0xffffffffu, e, o);
                    if (ob > best || (ob == best && oe < e)) {
                        best = ob;
                        e = oe;
                    }
                }
#pragma unroll
                for (int i = 0; i < kLossPer; ++i)
                    if (e0 + i == e) key[i] = 0u;
                if (sub == 0 && counted && e < E) atomicAdd(&s_c[e], 1);
            }
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
    float* mine = part + blockIdx.x * loss_partial_words(E);
    for (int e = tid; e < E; e += kLossThreads) {
        float p = 0.f;
#pragma unroll
        for (int w = 0; w < kLossWarps; ++w) p += s_p[w][e];
        mine[e] = p;
        mine[E + e] = __int_as_float(s_c[e]);
    }
    if (tid == 0) {
        float z = 0.f;
        int c = 0;
#pragma unroll
        for (int w = 0; w < kLossWarps; ++w) {
            z += s_z[w];
            c += s_n[w];
        }
        mine[2 * E] = z;
        mine[2 * E + 1] = __int_as_float(c);
    }
    if (gridDim.x == 1) {
        __threadfence_block();
        __syncthreads();
        loss_finish(part, 1, E, k, wb, wz, result);
    }
}

__global__ void __launch_bounds__(1024) router_loss_finish_kernel(const float* __restrict__ part, int blocks, int E,
                                                                  int k, float wb, float wz,
                                                                  float* __restrict__ result) {
    op::pdl_enter();
    loss_finish(part, blocks, E, k, wb, wz, result);
}

// The gradient of the logits (the rows' statistics are computed again: they
// cost less than a second pass over saved ones would).
template <typename IT, int L, bool SIG>
__global__ void __launch_bounds__(kLossThreads) router_loss_grad_kernel(
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
    const long long step = (long long)gridDim.x * kLossWarps * R;
    for (long long t0 = ((long long)blockIdx.x * kLossWarps + warp) * R; t0 < T; t0 += step) {
        const long long t = t0 + grp;
        const bool in = t < T;
        float v[kLossPer];
        if (in) loss_load(logits + t * ld, e0, E, vec != 0, v);
        else {
#pragma unroll
            for (int i = 0; i < kLossPer; ++i) v[i] = -INFINITY;
        }
        RowStats<IT, L, SIG> st;
        st.compute(v);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) dot += a[i] * st.p[i];
        dot = row_sum<L>(dot);
        const bool counted = in && st.any && (!mask || mask[t] != 0);
        float g[kLossPer];
#pragma unroll
        for (int i = 0; i < kLossPer; ++i) {
            float w = st.p[i] * (a[i] - dot);
            if constexpr (SIG) w *= st.slope[i];
            g[i] = counted ? w + zc * st.lse * st.soft[i] : 0.f;
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
