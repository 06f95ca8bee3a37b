// router_loss.cu -- host side of l4moe_router_loss and l4moe_router_loss_grad
// (include/l4moe.h): argument checks and launches.
#include <algorithm>
#include <cstdio>

#include "l4moe.h"
#include "launch.cuh"
#include "router_loss.cuh"

using namespace l4moe;

namespace {

// Lanes per row: 8 experts to a lane, a power of two.
int lanes_of(int E) {
    int L = 1;
    while (L * kLossPer < E) L *= 2;
    return L;
}

int device_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

// Blocks of the sums: every warp has a row group to take; up to two passes of
// a cluster's blocks stay one cluster (one launch: a second costs about as
// much as a pass), more are two blocks per SM, whose partials the finishing
// cluster adds (clusters of 8 would leave SMs idle: 45 us for 65536 x 256 became 56).
int loss_blocks(int T, int E, int sms) {
    const long long rows = (long long)kLossWarps * (32 / lanes_of(E));  // per block and pass
    const long long need = std::max(1LL, (T + rows - 1) / rows);
    if (need <= 2 * kLossCluster) return (int)std::min<long long>(need, kLossCluster);
    return (int)std::min<long long>({need, 2LL * sms, 1024LL});
}

l4moe_status cuda_error(cudaError_t e, const char* what) {
    char msg[200];
    snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
    return op_fail(L4MOE_ERR_CUDA, msg);
}

size_t elem_bytes(l4moe_elem t) { return t == L4MOE_ELEM_F32 ? 4 : 2; }

// Whether rows of E elements at p (ld apart) and q (ldd apart) may share
// memory: their ranges do, unless both are columns of one matrix that lie
// side by side.
bool rows_overlap(int T, int E, const void* p, long long ld, const void* q, long long ldd, size_t size) {
    const size_t n = (size_t)E * size, a = (size_t)(T - 1) * ld * size, b = (size_t)(T - 1) * ldd * size;
    if (!overlap(p, a + n, q, b + n)) return false;
    if (ld != ldd) return true;
    const uintptr_t u = reinterpret_cast<uintptr_t>(p), v = reinterpret_cast<uintptr_t>(q);
    const size_t pitch = (size_t)ld * size, at = (u > v ? u - v : v - u) % pitch;
    return at < n || at > pitch - n;
}

// What both entry points ask of the logits.
l4moe_status check_logits(const char* fn, int T, int E, const void* logits, l4moe_elem type, long long ld,
                          l4moe_score score) {
    char msg[160];
    const char* bad = nullptr;
    l4moe_status s = L4MOE_ERR_ARG;
    if (T < 0 || E < 1 || E > kLossMaxExperts) bad = "needs T >= 0 and 1 <= E <= 256";
    else if (type != L4MOE_ELEM_F32 && type != L4MOE_ELEM_BF16 && type != L4MOE_ELEM_F16)
        bad = "unknown element type", s = L4MOE_ERR_DTYPE;
    else if (score != L4MOE_SCORE_SOFTMAX && score != L4MOE_SCORE_SIGMOID) bad = "unknown score";
    else if (T > 0 && !logits) bad = "null logits";
    else if (ld < E) bad = "row stride smaller than E";
    else if (reinterpret_cast<uintptr_t>(logits) % elem_bytes(type)) bad = "misaligned logits", s = L4MOE_ERR_ALIGN;
    if (!bad) return L4MOE_OK;
    snprintf(msg, sizeof msg, "%s: %s", fn, bad);
    return op_fail(s, msg);
}

// 16-byte loads of 8 experts: whole lanes only, every row aligned.
bool vectors(int E, const void* p, long long ld, l4moe_elem type) {
    return E % kLossPer == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 &&
           (unsigned long long)ld * elem_bytes(type) % 16 == 0;
}

struct LossArgs {
    const void* logits;
    long long ld;
    int T, E, k;
    const uint8_t* mask;
    const int32_t* idx;
    float wb, wz;
    float *part, *result;
    int blocks;
    bool vec;
};

template <typename IT, int L, bool SIG>
void launch_loss(const LossArgs& a, cudaStream_t st) {
    const bool alone = a.blocks <= kLossCluster;
    launch_cluster_x(router_loss_kernel<IT, L, SIG>, dim3(a.blocks), dim3(kLossThreads), 0, st,
                     alone && a.blocks > 1 ? (unsigned)a.blocks : 0u, static_cast<const IT*>(a.logits), a.ld, a.T, a.E,
                     a.k, a.vec ? 1 : 0, a.mask, a.idx, a.wb, a.wz, a.part, a.result);
    if (!alone) {
        int lg = 0;
        while ((1 << lg) < a.E) ++lg;
        launch_cluster_x(router_loss_finish_kernel, dim3(kLossCluster), dim3(1024), 0, st, (unsigned)kLossCluster,
                         (const float*)a.part, a.blocks, a.E, lg, a.k, a.wb, a.wz, a.result);
    }
}

struct GradArgs {
    const void* logits;
    long long ld;
    int T, E;
    const uint8_t* mask;
    const float *result, *upstream;
    void* dl;
    long long ldd;
    int blocks;
    bool vec;
};

template <typename IT, int L, bool SIG>
void launch_grad(const GradArgs& a, cudaStream_t st) {
    launch_k(router_loss_grad_kernel<IT, L, SIG>, dim3(a.blocks), dim3(kGradThreads), 0, st,
             static_cast<const IT*>(a.logits), a.ld, a.T, a.E, a.vec ? 1 : 0, a.mask, a.result, a.upstream,
             static_cast<IT*>(a.dl), a.ldd);
}

// f.template operator()<IT, L, SIG>() for the runtime type, width and score.
template <typename IT, bool SIG, typename F>
void with_lanes(int E, F&& f) {
    switch (lanes_of(E)) {
    case 1: f.template run<IT, 1, SIG>(); break;
    case 2: f.template run<IT, 2, SIG>(); break;
    case 4: f.template run<IT, 4, SIG>(); break;
    case 8: f.template run<IT, 8, SIG>(); break;
    case 16: f.template run<IT, 16, SIG>(); break;
    default: f.template run<IT, 32, SIG>(); break;
    }
}

template <typename F>
void dispatch(l4moe_elem type, l4moe_score score, int E, F&& f) {
    const bool sig = score == L4MOE_SCORE_SIGMOID;
    if (type == L4MOE_ELEM_F32) sig ? with_lanes<float, true>(E, f) : with_lanes<float, false>(E, f);
    else if (type == L4MOE_ELEM_BF16)
        sig ? with_lanes<__nv_bfloat16, true>(E, f) : with_lanes<__nv_bfloat16, false>(E, f);
    else sig ? with_lanes<__half, true>(E, f) : with_lanes<__half, false>(E, f);
}

struct RunLoss {
    const LossArgs& a;
    cudaStream_t st;
    template <typename IT, int L, bool SIG>
    void run() const { launch_loss<IT, L, SIG>(a, st); }
};
struct RunGrad {
    const GradArgs& a;
    cudaStream_t st;
    template <typename IT, int L, bool SIG>
    void run() const { launch_grad<IT, L, SIG>(a, st); }
};

}  // namespace

extern "C" {

size_t l4moe_router_loss_workspace(int T, int E) {
    if (T < 0 || E < 1 || E > kLossMaxExperts) return 0;
    const int sms = device_sms();
    if (sms < 1) return 0;
    return sizeof(float) * loss_partial_words(E) * (size_t)loss_blocks(T, E, sms);
}

l4moe_status l4moe_router_loss(int T, int E, int k, const void* logits, l4moe_elem type, long long ld,
                               const uint8_t* mask, const int32_t* idx, l4moe_score score, float balance_weight,
                               float z_weight, float* result, void* workspace, size_t ws_bytes, void* stream) {
    l4moe_status s = check_logits("l4moe_router_loss", T, E, logits, type, ld, score);
    if (s != L4MOE_OK) return s;
    if (k < 1 || k > kLossMaxK || k > E) return op_fail(L4MOE_ERR_ARG, "l4moe_router_loss: k must be in [1, min(4, E)]");
    if ((long long)T * k > INT32_MAX) return op_fail(L4MOE_ERR_ARG, "l4moe_router_loss: T k above 2^31 - 1 (32-bit counts)");
    if (!result || !workspace) return op_fail(L4MOE_ERR_ARG, "l4moe_router_loss: null result or workspace");
    if ((reinterpret_cast<uintptr_t>(result) | reinterpret_cast<uintptr_t>(workspace) |
         reinterpret_cast<uintptr_t>(idx)) & 3u)
        return op_fail(L4MOE_ERR_ALIGN, "l4moe_router_loss: result, workspace and idx must be 4-byte aligned");
    const int sms = device_sms();
    if (sms < 1) return op_fail(L4MOE_ERR_CUDA, "l4moe_router_loss: no CUDA device");
    LossArgs a{logits, ld, T, E, k, mask, idx, balance_weight, z_weight, static_cast<float*>(workspace), result,
               loss_blocks(T, E, sms), vectors(E, logits, ld, type)};
    if (ws_bytes < sizeof(float) * loss_partial_words(E) * (size_t)a.blocks)
        return op_fail(L4MOE_ERR_WORKSPACE, "l4moe_router_loss: workspace smaller than l4moe_router_loss_workspace");
    dispatch(type, score, E, RunLoss{a, static_cast<cudaStream_t>(stream)});
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? L4MOE_OK : cuda_error(e, "l4moe_router_loss launch");
}

l4moe_status l4moe_router_loss_grad(int T, int E, const void* logits, l4moe_elem type, long long ld,
                                    const uint8_t* mask, l4moe_score score, const float* result, const float* upstream,
                                    void* dlogits, long long ldd, void* stream) {
    l4moe_status s = check_logits("l4moe_router_loss_grad", T, E, logits, type, ld, score);
    if (s != L4MOE_OK) return s;
    if (!result || (T > 0 && !dlogits) || ldd < E)
        return op_fail(L4MOE_ERR_ARG, "l4moe_router_loss_grad: null result or gradient, or its row stride below E");
    if (reinterpret_cast<uintptr_t>(dlogits) % elem_bytes(type) ||
        ((reinterpret_cast<uintptr_t>(result) | reinterpret_cast<uintptr_t>(upstream)) & 3u))
        return op_fail(L4MOE_ERR_ALIGN, "l4moe_router_loss_grad: misaligned pointer");
    if (T == 0) return L4MOE_OK;
    if (rows_overlap(T, E, logits, ld, dlogits, ldd, elem_bytes(type)))
        return op_fail(L4MOE_ERR_ARG, "l4moe_router_loss_grad: dlogits overlaps the logits");
    const int sms = device_sms();
    if (sms < 1) return op_fail(L4MOE_ERR_CUDA, "l4moe_router_loss_grad: no CUDA device");
    const long long rows = (long long)(kGradThreads / 32) * (32 / lanes_of(E));
    const int blocks = (int)std::min<long long>((T + rows - 1) / rows, 8LL * sms);
    GradArgs a{logits, ld, T, E, mask, result, upstream, dlogits, ldd, blocks,
               vectors(E, logits, ld, type) && vectors(E, dlogits, ldd, type)};
    dispatch(type, score, E, RunGrad{a, static_cast<cudaStream_t>(stream)});
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? L4MOE_OK : cuda_error(e, "l4moe_router_loss_grad launch");
}

}  // extern "C"
