// rms_norm.cu -- root-mean-square norm with the residual's addition (ss2d_rms_norm).
//
//   r = x + residual                              fp32
//   y = r / sqrt(mean(r^2) + eps) * weight        fp32, stored as fp32, bf16, or e4m3 with
//   s_g = max(max_g |y| / 448, 2^-100)            a scale for each group of 128 columns,
//   q = e4m3(y / s_g)
//   residual_out = r                              rounded to the residual's type
//
// A row stays in registers between the reduction of its squares and the output, so each
// tensor is read or written once: the kernel is bounded by device memory.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stddef.h>
#include <stdint.h>

#include "api_internal.h"
#include "op_check.h"
#include "ss2d.h"

namespace ss2d {
namespace {

constexpr int kRnGroup = 128;          // columns of one e4m3 scale
constexpr float kRnE4m3Max = 448.0f;   // largest finite e4m3 value
constexpr float kRnScaleMin = 7.888609052210118e-31f;  // 2^-100: keeps y / s finite where a group is zero
constexpr int kRnThreads = 256;        // threads of a CTA that holds several rows

struct RmsArgs {
    const void *x, *residual;
    const float *weight;
    void *y, *residual_out;
    float *scales;
    long long rows;
    int D, groups;
    int x_bf16, res_bf16, y_dtype;
    float eps;
};

__device__ __forceinline__ float rn_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float rn_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Eight consecutive elements from column c on as fp32; columns past D are zero.  VEC: D % 8 == 0,
// so the eight are in range together and 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ void rn_load8(const void *base, bool bf16, long long row, int D, int c, float (&f)[8])
{
    if (VEC) {
        if (bf16) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + row * D + c));
            f[0] = rn_lo(v.x), f[1] = rn_hi(v.x), f[2] = rn_lo(v.y), f[3] = rn_hi(v.y);
            f[4] = rn_lo(v.z), f[5] = rn_hi(v.z), f[6] = rn_lo(v.w), f[7] = rn_hi(v.w);
        } else {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + row * D + c);
            const float4 a = __ldg(p), b = __ldg(p + 1);
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
            f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const long long at = row * D + c + i;
            f[i] = c + i >= D ? 0.0f
                   : bf16     ? __bfloat162float(static_cast<const __nv_bfloat16 *>(base)[at])
                              : static_cast<const float *>(base)[at];
        }
    }
}

__device__ __forceinline__ uint32_t rn_pack(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <bool VEC>
__device__ __forceinline__ void rn_store8(void *base, int dtype, long long row, int D, int c, const float (&f)[8])
{
    if (VEC) {
        if (dtype == SS2D_BF16) {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(base) + row * D + c) =
                make_uint4(rn_pack(f[0], f[1]), rn_pack(f[2], f[3]), rn_pack(f[4], f[5]), rn_pack(f[6], f[7]));
        } else if (dtype == SS2D_F32) {
            float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + row * D + c);
            p[0] = make_float4(f[0], f[1], f[2], f[3]);
            p[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            uint32_t w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[h] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f[4 * h], f[4 * h + 1]), __NV_SATFINITE, __NV_E4M3) |
                       (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f[4 * h + 2], f[4 * h + 3]), __NV_SATFINITE,
                                                          __NV_E4M3)
                           << 16;
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(base) + row * D + c) = make_uint2(w[0], w[1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c + i >= D)
                break;
            const long long at = row * D + c + i;
            if (dtype == SS2D_BF16)
                static_cast<__nv_bfloat16 *>(base)[at] = __float2bfloat16_rn(f[i]);
            else if (dtype == SS2D_F32)
                static_cast<float *>(base)[at] = f[i];
            else
                static_cast<uint8_t *>(base)[at] = __nv_cvt_float_to_fp8(f[i], __NV_SATFINITE, __NV_E4M3);
        }
    }
}

// TPR threads hold a row, each NV runs of 8 columns: run t + i * TPR of thread t.  A group of
// 128 columns is then 16 neighbouring lanes of one run index.
template <int TPR, int NV, bool VEC>
__global__ void __launch_bounds__(TPR > kRnThreads ? TPR : kRnThreads) rms_norm_kernel(const RmsArgs a)
{
    constexpr int kThreads = TPR > kRnThreads ? TPR : kRnThreads;
    constexpr int kRows = kThreads / TPR;
    const int t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool live = row < a.rows;
    float r[NV][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * TPR) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r[i][j] = 0.0f;
        if (live && c < a.D) {
            rn_load8<VEC>(a.x, a.x_bf16, row, a.D, c, r[i]);
            if (a.residual) {
                float e[8];
                rn_load8<VEC>(a.residual, a.res_bf16, row, a.D, c, e);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    r[i][j] += e[j];
                rn_store8<VEC>(a.residual_out, a.res_bf16 ? SS2D_BF16 : SS2D_F32, row, a.D, c, r[i]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum = fmaf(r[i][j], r[i][j], sum);
    }
#pragma unroll
    for (int d = (TPR < 32 ? TPR : 32) / 2; d > 0; d /= 2)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (TPR > 32) {
        constexpr int kWarps = TPR / 32;  // warps of a row
        __shared__ float part[kThreads / 32];
        if (threadIdx.x % 32 == 0)
            part[threadIdx.x / 32] = sum;
        __syncthreads();
        const int first = threadIdx.x / TPR * kWarps;
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i)
            sum += part[first + i];
    }
    const float rstd = rsqrtf(sum / (float)a.D + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * TPR) * 8;
        const bool in = live && c < a.D;
        float w[8];
        if (in)
            rn_load8<VEC>(a.weight, false, 0, a.D, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r[i][j] = in ? r[i][j] * rstd * w[j] : 0.0f;
        if (a.y_dtype == SS2D_E4M3) {
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                amax = fmaxf(amax, fabsf(r[i][j]));
#pragma unroll
            for (int d = 8; d > 0; d /= 2)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
            const float s = fmaxf(amax / kRnE4m3Max, kRnScaleMin);
            if (in && c % kRnGroup == 0)
                a.scales[row * a.groups + c / kRnGroup] = s;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                r[i][j] /= s;
        }
        if (in)
            rn_store8<VEC>(a.y, a.y_dtype, row, a.D, c, r[i]);
    }
}

template <int TPR, int NV>
cudaError_t rms_launch(const RmsArgs &a, cudaStream_t s)
{
    constexpr int kThreads = TPR > kRnThreads ? TPR : kRnThreads;
    const long long grid = (a.rows + kThreads / TPR - 1) / (kThreads / TPR);
    if (a.D % 8 == 0)
        rms_norm_kernel<TPR, NV, true><<<(unsigned)grid, kThreads, 0, s>>>(a);
    else
        rms_norm_kernel<TPR, NV, false><<<(unsigned)grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

size_t rms_esize(int dtype) { return dtype == SS2D_F32 ? 4 : dtype == SS2D_BF16 ? 2 : 1; }

}  // namespace
}  // namespace ss2d

extern "C" int ss2d_rms_norm(const void *x, int x_dtype, const void *residual, int residual_dtype,
                             const float *weight, float eps, void *y, int y_dtype, float *scales, void *residual_out,
                             long long rows, int D, void *stream)
{
    using namespace ss2d;
    static const char *call = "ss2d_rms_norm";
    set_last_error(SS2D_OK, "");
    if (!x || !weight || !y)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: x, weight and y must be non-null", call);
    if ((residual == nullptr) != (residual_out == nullptr))
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: residual and residual_out are given together", call);
    if ((y_dtype == SS2D_E4M3) != (scales != nullptr))
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: scales is given with an e4m3 y, and only then", call);
    if (rows <= 0 || D <= 0)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: sizes must be positive (rows=%lld D=%d)", call, rows, D);
    if (!(eps >= 0.0f) || eps > 1.0f)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: eps=%g is not within 0 and 1", call, (double)eps);
    if ((x_dtype != SS2D_F32 && x_dtype != SS2D_BF16) ||
        (residual && residual_dtype != SS2D_F32 && residual_dtype != SS2D_BF16))
        return op_fail(SS2D_ERR_UNSUPPORTED, "%s: dtype codes (%d, %d) of x and residual must be SS2D_F32 or SS2D_BF16",
                       call, x_dtype, residual_dtype);
    if (y_dtype != SS2D_F32 && y_dtype != SS2D_BF16 && y_dtype != SS2D_E4M3)
        return op_fail(SS2D_ERR_UNSUPPORTED, "%s: dtype code %d of y must be SS2D_F32, SS2D_BF16 or SS2D_E4M3", call,
                       y_dtype);
    if (D > 32768)
        return op_fail(SS2D_ERR_UNSUPPORTED, "%s: D=%d is above 32768", call, D);
    if (rows > 0x7fffffffLL)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: problem too large", call);
    const size_t n = (size_t)rows * D;
    const int groups = (D + kRnGroup - 1) / kRnGroup;
    const OpSpan in[] = {{"x", x, n * rms_esize(x_dtype)},
                         {"weight", weight, (size_t)D * 4},
                         // the residual may be updated in place: it is read and written by the same thread
                         {"residual", residual, residual == residual_out ? 0 : n * rms_esize(residual_dtype)}};
    const OpSpan out[] = {{"y", y, n * rms_esize(y_dtype)},
                          {"scales", scales, (size_t)rows * groups * 4},
                          {"residual_out", residual_out, n * rms_esize(residual_dtype)}};
    const int st = op_check_tensors(call, in, 3, out, 3);
    if (st != SS2D_OK)
        return st;
    RmsArgs a{};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.y = y;
    a.residual_out = residual_out;
    a.scales = scales;
    a.rows = rows;
    a.D = D;
    a.groups = groups;
    a.x_bf16 = x_dtype == SS2D_BF16;
    a.res_bf16 = residual_dtype == SS2D_BF16;
    a.y_dtype = y_dtype;
    a.eps = eps;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (D <= 128)
        e = rms_launch<16, 1>(a, s);
    else if (D <= 256)
        e = rms_launch<32, 1>(a, s);
    else if (D <= 1024)
        e = rms_launch<128, 1>(a, s);
    else if (D <= 2048)
        e = rms_launch<256, 1>(a, s);
    else if (D <= 4096)
        e = rms_launch<512, 1>(a, s);
    else if (D <= 8192)
        e = rms_launch<1024, 1>(a, s);
    else if (D <= 16384)
        e = rms_launch<1024, 2>(a, s);
    else
        e = rms_launch<1024, 4>(a, s);
    return e == cudaSuccess ? SS2D_OK : op_cuda_fail(e, "ss2d_rms_norm launch");
}
