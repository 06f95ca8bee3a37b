// int4.cu -- host side of l4moe_int4_matvec (include/l4moe.h): argument
// checks and launch.
#include <algorithm>
#include <cstdio>

#include "int4_mv.cuh"
#include "l4moe.h"
#include "launch.cuh"

using namespace l4moe;

namespace {

struct Call {
    int T, K, N, group, sms;
    const void *x, *s;
    const uint8_t* w;
    void* y;
    cudaStream_t st;
    bool vec;
};

template <int NT8, typename XT, typename ST, bool VEC>
cudaError_t launch(const Call& c) {
    constexpr size_t smem = mv::Cfg<NT8, ST>::SMEM;
    static std::atomic<uint64_t> attr_done{0};
    ensure_smem_attr(attr_done, mv::int4_matvec_kernel<NT8, XT, ST, VEC>, smem);
    const int tiles = (c.N + mv::kCols - 1) / mv::kCols, tt = (c.T + NT8 * 8 - 1) / (NT8 * 8);
    const int S = mv::slices((long long)tiles * tt, c.K, c.sms, mv::Cfg<NT8, ST>::PER_SM);
    const mv::Weight<ST> W{c.w, static_cast<const ST*>(c.s), c.N / 2, c.N, c.K, c.group};
    launch_kc(mv::int4_matvec_kernel<NT8, XT, ST, VEC>, dim3(tiles, tt, S), dim3(mv::kThreads), smem, c.st,
              S > 1 ? (unsigned)S : 0u, static_cast<const XT*>(c.x), c.T, W, static_cast<XT*>(c.y));
    return cudaGetLastError();
}

template <typename XT, typename ST>
cudaError_t launch_x(const Call& c) {
    if (c.T <= 8) return c.vec ? launch<1, XT, ST, true>(c) : launch<1, XT, ST, false>(c);
    return c.vec ? launch<2, XT, ST, true>(c) : launch<2, XT, ST, false>(c);
}

template <typename XT>
cudaError_t launch_s(const Call& c, l4moe_elem s_type) {
    if (s_type == L4MOE_ELEM_F32) return launch_x<XT, float>(c);
    if (s_type == L4MOE_ELEM_BF16) return launch_x<XT, __nv_bfloat16>(c);
    return launch_x<XT, __half>(c);
}

}  // namespace

extern "C" l4moe_status l4moe_int4_matvec(int T, int K, int N, int group, const void* x, l4moe_elem x_type,
                                          const void* w, const void* scales, l4moe_elem s_type, void* y,
                                          void* stream) {
    if (T < 0 || K < 1 || N < 2 || N % 2)
        return op_fail(L4MOE_ERR_ARG, "l4moe_int4_matvec: needs T >= 0, K >= 1 and an even N >= 2");
    if (K > 1 << 30 || N > 1 << 30) return op_fail(L4MOE_ERR_ARG, "l4moe_int4_matvec: K or N above 2^30");
    if (T > L4MOE_INT4_MAX_TOKENS)
        return op_fail(L4MOE_ERR_ARG, "l4moe_int4_matvec: more than L4MOE_INT4_MAX_TOKENS tokens");
    if (group < 32 || group % 32) return op_fail(L4MOE_ERR_ARG, "l4moe_int4_matvec: group must be a multiple of 32");
    if (x_type != L4MOE_ELEM_BF16 && x_type != L4MOE_ELEM_F16)
        return op_fail(L4MOE_ERR_DTYPE, "l4moe_int4_matvec: x must be bf16 or f16");
    if (s_type != L4MOE_ELEM_F32 && s_type != L4MOE_ELEM_BF16 && s_type != L4MOE_ELEM_F16)
        return op_fail(L4MOE_ERR_DTYPE, "l4moe_int4_matvec: unknown scale type");
    if (T == 0) return L4MOE_OK;
    if (!x || !w || !scales || !y) return op_fail(L4MOE_ERR_ARG, "l4moe_int4_matvec: null tensor pointer");
    if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(scales) |
         reinterpret_cast<uintptr_t>(y)) & 15u)
        return op_fail(L4MOE_ERR_ALIGN, "l4moe_int4_matvec: tensor pointer not 16-byte aligned");
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return op_fail(L4MOE_ERR_CUDA, "l4moe_int4_matvec: no CUDA device");
    // 16-byte copies when every row starts on 16 bytes
    const Call c{T, K, N, group, sms, x, scales, static_cast<const uint8_t*>(w), y,
                 static_cast<cudaStream_t>(stream), N % 32 == 0};
    const cudaError_t e =
        x_type == L4MOE_ELEM_BF16 ? launch_s<__nv_bfloat16>(c, s_type) : launch_s<__half>(c, s_type);
    if (e == cudaSuccess) return L4MOE_OK;
    char msg[200];
    snprintf(msg, sizeof msg, "l4moe_int4_matvec launch: %s", cudaGetErrorString(e));
    return op_fail(L4MOE_ERR_CUDA, msg);
}
