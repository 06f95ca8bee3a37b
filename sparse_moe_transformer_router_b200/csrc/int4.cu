// int4.cu -- host side of l4moe_int4_matvec (include/l4moe.h): argument
// checks and launch.
#include <algorithm>
#include <cstdio>

#include "int4_mv.cuh"
#include "l4moe.h"
#include "launch.cuh"
#include "tensor_map.cuh"

using namespace l4moe;

namespace {

struct Call {
    int T, K, N, group, sms;
    const void *x, *s;
    const uint8_t* w;
    void* y;
    cudaStream_t st;
    bool tma;
};

template <typename T>
constexpr CUtensorMapDataType map_type() {
    return std::is_same<T, float>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
           : std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

template <int NT8, typename XT, typename ST, bool TMA>
cudaError_t launch(const Call& c) {
    using Cf = mv::Cfg<NT8, ST>;
    static std::atomic<uint64_t> attr_done{0};
    ensure_smem_attr(attr_done, mv::int4_matvec_kernel<NT8, XT, ST, TMA>, Cf::SMEM);
    const int tiles = (c.N + mv::kCols - 1) / mv::kCols, tt = (c.T + NT8 * 8 - 1) / (NT8 * 8);
    const int S = mv::slices((long long)tiles * tt, c.K, c.sms, Cf::PER_SM);
    CUtensorMap qm{}, sm{}, xm{};
    if (TMA && (!encode_2d(&qm, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.w, (uint64_t)c.N / 2, (uint64_t)c.K,
                           (uint64_t)c.N / 2, 64, mv::kRows, CU_TENSOR_MAP_SWIZZLE_64B) ||
                !encode_2d(&sm, map_type<ST>(), c.s, (uint64_t)c.N, ((uint64_t)c.K + c.group - 1) / c.group,
                           (uint64_t)c.N * sizeof(ST), mv::kCols, 1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
                !encode_2d(&xm, map_type<XT>(), c.x, (uint64_t)c.K, (uint64_t)c.T, (uint64_t)c.K * 2, mv::kRows, 1)))
        return cudaErrorInvalidValue;
    const mv::Weight<ST> W{nullptr, nullptr, c.w, static_cast<const ST*>(c.s), c.N, c.K, c.group};
    launch_kc(mv::int4_matvec_kernel<NT8, XT, ST, TMA>, dim3(tiles, tt, S), dim3(mv::kThreads), Cf::SMEM, c.st,
              S > 1 ? (unsigned)S : 0u, qm, sm, xm, static_cast<const XT*>(c.x), c.T, W, static_cast<XT*>(c.y));
    return cudaGetLastError();
}

template <typename XT, typename ST>
cudaError_t launch_x(const Call& c) {
    if (c.T <= 8) return c.tma ? launch<1, XT, ST, true>(c) : launch<1, XT, ST, false>(c);
    return c.tma ? launch<2, XT, ST, true>(c) : launch<2, XT, ST, false>(c);
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
    // the output is written while other CTAs still read the inputs
    const size_t xb = (size_t)T * K * 2, wb = (size_t)K * (N / 2), yb = (size_t)T * N * 2;
    const size_t sb = ((size_t)K + group - 1) / group * N * (s_type == L4MOE_ELEM_F32 ? 4 : 2);
    if (overlap(y, yb, x, xb) || overlap(y, yb, w, wb) || overlap(y, yb, scales, sb))
        return op_fail(L4MOE_ERR_ARG, "l4moe_int4_matvec: y overlaps an input");
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return op_fail(L4MOE_ERR_CUDA, "l4moe_int4_matvec: no CUDA device");
    // tensor maps want rows that start on 16 bytes
    const Call c{T, K, N, group, sms, x, scales, static_cast<const uint8_t*>(w), y,
                 static_cast<cudaStream_t>(stream), N % 32 == 0 && K % 8 == 0};
    const cudaError_t e =
        x_type == L4MOE_ELEM_BF16 ? launch_s<__nv_bfloat16>(c, s_type) : launch_s<__half>(c, s_type);
    if (e == cudaSuccess) return L4MOE_OK;
    char msg[200];
    snprintf(msg, sizeof msg, "l4moe_int4_matvec launch: %s", cudaGetErrorString(e));
    return op_fail(L4MOE_ERR_CUDA, msg);
}
