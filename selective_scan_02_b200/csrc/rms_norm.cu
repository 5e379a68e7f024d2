// rms_norm.cu -- root-mean-square norm with the residual's addition (ss2d_rms_norm).
//
//   r = x + residual                              fp32
//   y = r / sqrt(mean(r^2) + eps) * weight        fp32, stored as fp32, bf16, or e4m3 with
//   s_g = max(max_g |y| / 448, 2^-100)            a scale for each group of 128 columns,
//   q = e4m3(y / s_g)
//   residual_out = r                              rounded to the residual's type
//
// A row stays in registers between the reduction of its squares and the output, so each
// tensor is read or written once: the kernel is bounded by device memory, and what matters is to keep
// enough loads in flight and the instructions few.  16384 rows of 4096 columns (bf16 with a bf16 residual,
// e4m3 out): 79.5 us a call on rows that change, 5.9 TB/s, 71 in a graph on the same ones (a part of them stays in L2);
// 100352 rows of 96 (fp32 in, bf16 out): 21.4 and 19.4 us, 6.3 TB/s.  Eight rows are 2.9 us on the GPU, most of it the
// launch.  Rows of single columns, whose accesses are of an element each, take up to 1.9 times as long (333 columns 70
// us, 37 at 384).  CTAs that stay and walk the rows, with or without an asynchronous ring of loads, took longer: other
// rows' CTAs hide one row's reduction better.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stddef.h>
#include <stdint.h>

#include "api_internal.h"
#include "launch_util.h"
#include "op_check.h"
#include "ss2d.h"

namespace ss2d {
namespace {

constexpr int kRnGroup = 128;          // columns of one e4m3 scale
constexpr float kRnE4m3Max = 448.0f;   // largest finite e4m3 value
constexpr float kRnScaleMin = 7.888609052210118e-31f;  // 2^-100: keeps 1 / s finite where a group is zero
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

// Eight consecutive elements, 16-byte aligned, as they lie in memory.
template <bool BF16>
struct Raw8 {
    static constexpr int kPieces = BF16 ? 1 : 2;
    uint4 v[kPieces];

    __device__ __forceinline__ void load(const void *base, long long i)
    {
        const uint4 *p = BF16 ? reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + i)
                              : reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + i);
#pragma unroll
        for (int x = 0; x < kPieces; ++x)
            v[x] = p[x];
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int x = 0; x < kPieces; ++x)
            v[x] = make_uint4(0, 0, 0, 0);
    }
    // elements 2 i and 2 i + 1
    __device__ __forceinline__ float2 pair(int i) const
    {
        const uint4 hi = v[kPieces - 1];
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, hi.x, hi.y, hi.z, hi.w};
        return BF16 ? make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u))
                    : make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
};

__device__ __forceinline__ uint32_t rn_pack(float2 f)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint32_t rn_pack_e4m3(float2 lo, float2 hi)
{
    return (uint32_t)__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3) << 16;
}

__device__ __forceinline__ void rn_store8(void *base, int dtype, long long at, const float2 (&f)[4])
{
    if (dtype == SS2D_BF16) {
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(base) + at) =
            make_uint4(rn_pack(f[0]), rn_pack(f[1]), rn_pack(f[2]), rn_pack(f[3]));
    } else if (dtype == SS2D_F32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
        p[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        p[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    } else {
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(base) + at) =
            make_uint2(rn_pack_e4m3(f[0], f[1]), rn_pack_e4m3(f[2], f[3]));
    }
}

template <bool BF16>
__device__ __forceinline__ float rn_load(const void *base, long long at)
{
    return BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(base)[at]) : static_cast<const float *>(base)[at];
}

__device__ __forceinline__ void rn_store(void *base, int dtype, long long at, float f)
{
    if (dtype == SS2D_BF16)
        static_cast<__nv_bfloat16 *>(base)[at] = __float2bfloat16_rn(f);
    else if (dtype == SS2D_F32)
        static_cast<float *>(base)[at] = f;
    else
        static_cast<uint8_t *>(base)[at] = __nv_cvt_float_to_fp8(f, __NV_SATFINITE, __NV_E4M3);
}

// The scale of a group, from the maximum over LANES neighbouring lanes: max / 448, rounded once.  (The product with the
// rounded reciprocal, corrected by what it leaves, which is exact in an fma: Markstein's division.  An ordinary
// one takes 2^25 elements in rows of 4100 columns from 90 to 103 us.)
template <int LANES>
__device__ __forceinline__ float rn_scale(float amax)
{
#pragma unroll
    for (int d = LANES / 2; d > 0; d /= 2)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    const float inverse = 1.0f / kRnE4m3Max, near = amax * inverse;
    const float left = fmaf(-kRnE4m3Max, near, amax);
    return fmaxf(amax < INFINITY ? fmaf(left, inverse, near) : amax, kRnScaleMin);
}

// TPR threads hold a row, each 8 NV of its columns.
//   VEC (D % 8 == 0, rows 16-byte aligned): NV runs of 8 neighbouring columns, run t + i * TPR of thread
//   t; a group of 128 columns is one run of 16 neighbouring lanes (or all of fewer).
//   else: single columns, a warp's 256 NV (or the row's) next to one another and 32 of them (or TPR) in the
//   lanes, so that accesses of rows of any alignment stay together; a group is four of a warp's 32, or eight of 16.
// The types of x and the residual are the template's, so that all of a thread's loads are issued before
// the first is used.  y is (r rstd) weight, and q is y (1 / s): every product stays finite where y and y / s are, s being
// at least 2^-100.  With the arithmetic in pairs (f32x2) a column takes about eight instructions, which the loads hide.
enum { kRnNone, kRnF32, kRnBf16 };

// Several single columns keep many addresses: 64 registers are the most, or too few rows share an SM (8184 rows of 4100:
// 128 us with the 89 that the compiler takes by itself, 87 so).
constexpr int rn_threads(int tpr) { return tpr > kRnThreads ? tpr : kRnThreads; }

template <int TPR, int NV, bool VEC, bool XBF16, int RES>
__global__ void __launch_bounds__(rn_threads(TPR), VEC || NV == 1 ? 0 : 1024 / rn_threads(TPR)) rms_norm_kernel(const RmsArgs a)
{
    constexpr int kThreads = rn_threads(TPR);
    constexpr int kRows = kThreads / TPR;
    constexpr bool kResBf16 = RES == kRnBf16;
    constexpr int kResType = kResBf16 ? SS2D_BF16 : SS2D_F32;
    const int t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool live = row < a.rows;
    const long long at = row * a.D;
    constexpr int kStep = TPR < 32 ? TPR : 32;             // single columns: in the lanes,
    constexpr int kPer = kStep == 32 ? 4 : 8;              // and of a group in one of them
    const int first = t / 32 * (256 * NV) + t % kStep;
    const bool e4m3 = a.y_dtype == SS2D_E4M3;
    grid_wait();
    grid_next();
    float2 r[NV][4];
    // the weights of one of the thread's NV parts: the next one's are loaded as soon as these are used, ahead of the stores
    // that they would otherwise stand behind
    float2 w[4];
    auto weigh = [&](int i) {
        if (VEC) {
            Raw8<false> v;
            v.clear();
            if ((t + i * TPR) * 8 < a.D)
                v.load(a.weight, (t + i * TPR) * 8);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = v.pair(j);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = first + (8 * i + 2 * j) * kStep;
                w[j] = make_float2(c < a.D ? a.weight[c] : 0.0f, c + kStep < a.D ? a.weight[c + kStep] : 0.0f);
            }
        }
    };
    if (VEC) {
        Raw8<XBF16> x[NV];
        Raw8<kResBf16> e[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i].clear();
            e[i].clear();
            if (live && (t + i * TPR) * 8 < a.D) {
                x[i].load(a.x, at + (t + i * TPR) * 8);
                if (RES)
                    e[i].load(a.residual, at + (t + i * TPR) * 8);
            }
        }
        if (NV <= 2)
            weigh(0);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r[i][j] = x[i].pair(j);
                if (RES)
                    r[i][j] = __fadd2_rn(r[i][j], e[i].pair(j));
            }
            if (RES && live && (t + i * TPR) * 8 < a.D)
                rn_store8(a.residual_out, kResType, at + (t + i * TPR) * 8, r[i]);
        }
    } else {
        float f[NV][8], e[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = first + (8 * i + j) * kStep;
                const bool in = live && c < a.D;
                f[i][j] = in ? rn_load<XBF16>(a.x, at + c) : 0.0f;
                if (RES)
                    e[i][j] = in ? rn_load<kResBf16>(a.residual, at + c) : 0.0f;
            }
        weigh(0);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (RES)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = first + (8 * i + j) * kStep;
                    f[i][j] += e[i][j];
                    if (live && c < a.D)
                        rn_store(a.residual_out, kResType, at + c, f[i][j]);
                }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r[i][j] = make_float2(f[i][2 * j], f[i][2 * j + 1]);
        }
    }
    if (VEC && NV > 2)
        weigh(0);
    float2 squares = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            squares = __ffma2_rn(r[i][j], r[i][j], squares);
    float sum = squares.x + squares.y;
#pragma unroll
    for (int d = (TPR < 32 ? TPR : 32) / 2; d > 0; d /= 2)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (TPR > 32) {
        constexpr int kWarps = TPR / 32;  // warps of a row
        __shared__ float part[kThreads / 32];
        if (threadIdx.x % 32 == 0)
            part[threadIdx.x / 32] = sum;
        __syncthreads();
        const int from = threadIdx.x / TPR * kWarps;
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i)
            sum += part[from + i];
    }
    const float rstd = rsqrtf(sum / (float)a.D + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r[i][j] = __fmul2_rn(__fmul2_rn(r[i][j], make_float2(rstd, rstd)), w[j]);
        if (i + 1 < NV)
            weigh(i + 1);
        if (VEC) {
            const int c = (t + i * TPR) * 8;
            const bool in = live && c < a.D;
            if (e4m3) {
                float amax = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    amax = fmaxf(amax, fmaxf(fabsf(r[i][j].x), fabsf(r[i][j].y)));
                const float s = rn_scale<TPR < 16 ? TPR : 16>(amax);
                const float k = 1.0f / s;
                if (in && c % kRnGroup == 0)
                    a.scales[row * a.groups + c / kRnGroup] = s;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    r[i][j] = __fmul2_rn(r[i][j], make_float2(k, k));
            }
            if (in)
                rn_store8(a.y, a.y_dtype, at + c, r[i]);
        } else {
#pragma unroll
            for (int h = 0; h < 8; h += kPer) {
                const int c = first + (8 * i + h) * kStep;  // this lane's first column in the group
                float f[kPer];
                float amax = 0.0f;
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const float2 pair = r[i][(h + j) / 2];
                    f[j] = j % 2 ? pair.y : pair.x;
                    amax = fmaxf(amax, fabsf(f[j]));
                }
                float k = 1.0f;
                if (e4m3) {
                    const float s = rn_scale<kStep>(amax);
                    k = 1.0f / s;
                    if (live && t % kStep == 0 && c < a.D)
                        a.scales[row * a.groups + c / kRnGroup] = s;
                }
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (live && c + j * kStep < a.D)
                        rn_store(a.y, a.y_dtype, at + c + j * kStep, f[j] * k);
            }
        }
    }
}

template <int TPR, int NV, bool VEC, bool XBF16>
cudaError_t rms_launch_types(const RmsArgs &a, cudaStream_t s)
{
    constexpr int kThreads = rn_threads(TPR);
    const unsigned grid = (unsigned)((a.rows + kThreads / TPR - 1) / (kThreads / TPR));
    if (!a.residual)
        return launch_early(rms_norm_kernel<TPR, NV, VEC, XBF16, kRnNone>, grid, kThreads, 0, s, 1, a);
    return a.res_bf16 ? launch_early(rms_norm_kernel<TPR, NV, VEC, XBF16, kRnBf16>, grid, kThreads, 0, s, 1, a)
                      : launch_early(rms_norm_kernel<TPR, NV, VEC, XBF16, kRnF32>, grid, kThreads, 0, s, 1, a);
}

template <int TPR, int NV>
cudaError_t rms_launch(const RmsArgs &a, cudaStream_t s)
{
    if (a.D % 8 == 0)
        return a.x_bf16 ? rms_launch_types<TPR, NV, true, true>(a, s) : rms_launch_types<TPR, NV, true, false>(a, s);
    return a.x_bf16 ? rms_launch_types<TPR, NV, false, true>(a, s) : rms_launch_types<TPR, NV, false, false>(a, s);
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
                          {"scales", scales, (size_t)rows * groups * 4, 4},
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
    // Many rows: 16 or 24 columns a thread, whichever fits the row better, so that each has several loads in flight, a
    // row needs few warps and few threads have no column.  (2^25 elements, bf16 with a bf16 residual to e4m3: 333 columns
    // 70 us in 16 threads of 24, 85 in 32 of 16;  5120 columns 41 us in 256 of 24, 59 in 512 of 16;  24576 columns 50 us in
    // 1024 of 24, 51 in 1024 of 32.)  Few rows (less than two for each of the B200's 148 SMs): 8 columns a thread, the
    // shortest way through a row.  Narrow rows: as many lanes as they need (100352 rows of 7, 33, 100 columns: 38 to 40 us
    // with a warp for each row, 4.5, 9.7, 18 so).
    const bool many = rows > 2 * 148;
    cudaError_t e;
    if (D <= 8)
        e = rms_launch<1, 1>(a, s);
    else if (D <= 16)
        e = rms_launch<2, 1>(a, s);
    else if (D <= 32)
        e = rms_launch<4, 1>(a, s);
    else if (D <= 64)
        e = rms_launch<8, 1>(a, s);
    else if (D <= 128)
        e = rms_launch<16, 1>(a, s);
    else if (D <= 256)
        e = rms_launch<32, 1>(a, s);
    else if (!many && D <= 2048)
        e = rms_launch<256, 1>(a, s);
    else if (!many && D <= 8192)
        e = rms_launch<1024, 1>(a, s);
    else if (D <= 16 * 24)
        e = rms_launch<16, 3>(a, s);
    else if (D <= 32 * 16)
        e = rms_launch<32, 2>(a, s);
    else if (D <= 32 * 24)
        e = rms_launch<32, 3>(a, s);
    else if (D <= 64 * 16)
        e = rms_launch<64, 2>(a, s);
    else if (D <= 64 * 24)
        e = rms_launch<64, 3>(a, s);
    else if (D <= 128 * 16)
        e = rms_launch<128, 2>(a, s);
    else if (D <= 128 * 24)
        e = rms_launch<128, 3>(a, s);
    else if (D <= 256 * 16)
        e = rms_launch<256, 2>(a, s);
    else if (D <= 256 * 24)
        e = rms_launch<256, 3>(a, s);
    else if (D <= 512 * 16)
        e = rms_launch<512, 2>(a, s);
    else if (D <= 512 * 24)
        e = rms_launch<512, 3>(a, s);
    else if (D <= 1024 * 16)
        e = rms_launch<1024, 2>(a, s);
    else if (D <= 1024 * 24)
        e = rms_launch<1024, 3>(a, s);
    else
        e = rms_launch<1024, 4>(a, s);
    return e == cudaSuccess ? SS2D_OK : op_cuda_fail(e, "ss2d_rms_norm launch");
}
