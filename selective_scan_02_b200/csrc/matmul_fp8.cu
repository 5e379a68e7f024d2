// matmul_fp8.cu -- e4m3 matrix product with a scale for each block of 128 (ss2d_matmul_fp8).
//
//   c[m, n] = sum_kb a_scales[m, kb] w_scales[n / 128, kb] sum_{k in kb} a[m, k] w[n, k] (+ bias[n])
//
// with kb the blocks of 128 columns of a and w, all sums in fp32.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stddef.h>
#include <stdint.h>

#include "api_internal.h"
#include "op_check.h"
#include "ss2d.h"

namespace ss2d {
namespace {

constexpr int kFmBlock = 128;

struct Fp8Args {
    const uint8_t *a, *w;
    const float *a_scales, *w_scales, *bias;
    void *c;
    int *err;
    int M, N, K, KB, c_bf16;
};

__device__ __forceinline__ float fm_value(uint8_t v)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
}

__global__ void __launch_bounds__(256) matmul_fp8_kernel(const Fp8Args p)
{
    const int m = blockIdx.y * 16 + threadIdx.y, n = blockIdx.x * 16 + threadIdx.x;
    if (m == 0 && n == 0)
        *p.err = 0;  // no wait to run out here
    if (m >= p.M || n >= p.N)
        return;
    float acc = 0.0f;
    for (int kb = 0; kb < p.KB; ++kb) {
        float part = 0.0f;
        const int end = min(p.K, (kb + 1) * kFmBlock);
        for (int k = kb * kFmBlock; k < end; ++k)
            part = fmaf(fm_value(p.a[(size_t)m * p.K + k]), fm_value(p.w[(size_t)n * p.K + k]), part);
        acc = fmaf(part, p.a_scales[(size_t)m * p.KB + kb] * p.w_scales[(size_t)(n / kFmBlock) * p.KB + kb], acc);
    }
    if (p.bias)
        acc += p.bias[n];
    const size_t at = (size_t)m * p.N + n;
    if (p.c_bf16)
        static_cast<__nv_bfloat16 *>(p.c)[at] = __float2bfloat16_rn(acc);
    else
        static_cast<float *>(p.c)[at] = acc;
}

constexpr size_t kFmWorkspace = 256;  // the error word of the bounded waits

int fm_check(const char *call, const ss2d_matmul_fp8_args *a)
{
    if (!a || a->struct_size != sizeof(ss2d_matmul_fp8_args))
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: args is null or its struct_size is wrong", call);
    if (a->M <= 0 || a->N <= 0 || a->K <= 0)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: sizes must be positive (M=%d N=%d K=%d)", call, a->M, a->N, a->K);
    if (a->K % 16 != 0)
        return op_fail(SS2D_ERR_UNSUPPORTED, "%s: K=%d is not a multiple of 16", call, a->K);
    if (a->c_dtype != SS2D_F32 && a->c_dtype != SS2D_BF16)
        return op_fail(SS2D_ERR_UNSUPPORTED, "%s: dtype code %d of c must be SS2D_F32 or SS2D_BF16", call, a->c_dtype);
    return SS2D_OK;
}

}  // namespace
}  // namespace ss2d

extern "C" size_t ss2d_matmul_fp8_workspace(const ss2d_matmul_fp8_args *args)
{
    using namespace ss2d;
    set_last_error(SS2D_OK, "");
    return fm_check("ss2d_matmul_fp8_workspace", args) == SS2D_OK ? kFmWorkspace : (size_t)-1;
}

extern "C" int ss2d_matmul_fp8(const ss2d_matmul_fp8_args *args, void *workspace, size_t workspace_bytes, void *stream)
{
    using namespace ss2d;
    static const char *call = "ss2d_matmul_fp8";
    set_last_error(SS2D_OK, "");
    int st = fm_check(call, args);
    if (st != SS2D_OK)
        return st;
    if (!args->a || !args->a_scales || !args->w || !args->w_scales || !args->c)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: a, a_scales, w, w_scales and c must be non-null", call);
    const size_t M = args->M, N = args->N, K = args->K, KB = (K + kFmBlock - 1) / kFmBlock;
    if (!workspace || workspace_bytes < kFmWorkspace)
        return op_fail(SS2D_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", call, kFmWorkspace,
                       workspace_bytes);
    const OpSpan in[] = {{"a", args->a, M * K},
                         {"a_scales", args->a_scales, M * KB * 4},
                         {"w", args->w, N * K},
                         {"w_scales", args->w_scales, (N + kFmBlock - 1) / kFmBlock * KB * 4},
                         {"bias", args->bias, N * 4}};
    const OpSpan out[] = {{"c", args->c, M * N * (args->c_dtype == SS2D_BF16 ? 2 : 4)},
                          {"workspace", workspace, kFmWorkspace}};
    st = op_check_tensors(call, in, 5, out, 2);
    if (st != SS2D_OK)
        return st;
    Fp8Args p{};
    p.a = static_cast<const uint8_t *>(args->a);
    p.w = static_cast<const uint8_t *>(args->w);
    p.a_scales = args->a_scales;
    p.w_scales = args->w_scales;
    p.bias = args->bias;
    p.c = args->c;
    p.err = static_cast<int *>(workspace);
    p.M = args->M;
    p.N = args->N;
    p.K = args->K;
    p.KB = (int)KB;
    p.c_bf16 = args->c_dtype == SS2D_BF16;
    const dim3 grid((unsigned)((N + 15) / 16), (unsigned)((M + 15) / 16));
    matmul_fp8_kernel<<<grid, dim3(16, 16), 0, static_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SS2D_OK : op_cuda_fail(e, "ss2d_matmul_fp8 launch");
}
