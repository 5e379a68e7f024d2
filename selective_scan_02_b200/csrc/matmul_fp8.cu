// matmul_fp8.cu -- e4m3 matrix product with a scale for each block of 128 (ss2d_matmul_fp8).
//
//   c[m, n] = sum_kb a_scales[m, kb] w_scales[n / 128, kb] P_kb[m, n] (+ bias[n])
//   P_kb[m, n] = sum_{k in block kb} a[m, k] w[n, k]
//
// The scales change from block to block of K, so a block's partial product P_kb cannot stay in the
// tensor cores' accumulator: tcgen05.mma (kind::f8f6f4, K = 32, four for a block) writes each P_kb
// into a fresh buffer of tensor memory, and warps of the CTA read it back, scale it and add it
// to fp32 sums in their registers while the next block's MMAs fill the next buffer.  TMA brings
// 128 x 128-byte tiles (one block of K) through a ring of stages.
//
// Two kernels, by which side of the MMA the tokens are on:
//   wide_kernel   tokens along the 128 lanes, BN weight rows along the columns.  A thread's row has one
//                 activation scale and its columns one weight scale for a block, so a partial product
//                 costs one multiply-add.  Persistent CTAs walk the tiles; where the tiles are too few
//                 for the GPU, K is split over the CTAs of a cluster instead.
//   narrow_kernel weight rows along the 128 lanes, few tokens along the columns, and K split over
//                 the CTAs of a cluster, which add up in distributed shared memory: the weights' bytes
//                 bound a product with few tokens, and this spreads their reading over all SMs.
//
// 8192 x 6144 x 4096: 190 to 233 us by what the power limit leaves of the clock, 1.8 to 2.1 PFLOP/s.  A block
// of K of a 128 x 256 tile takes 866 cycles; its 48 KB pass through shared memory twice (written by TMA, read by
// the MMAs), 768 cycles at 128 bytes a cycle, and that bounds the kernel; the tensor cores are busy 53 %.  A pair of
// CTAs on one 256 x 256 tile reads less, but has room for two buffers of partial products only, and waiting
// across the pair for them took 414 us.  4 tokens x 6144 x 2048: 4.9 us (13 MB of weights, 1.9 us at the copy's
// rate); 333 x 1000 x 1104: 10.3 us in a graph, the latency of a launch and nine blocks in 24 CTAs.
#include <cuda_bf16.h>
#include <stddef.h>
#include <stdint.h>

#include "api_internal.h"
#include "launch_util.h"
#include "op_check.h"
#include "ss2d.h"
#include "tma.cuh"
#include "wait_status.cuh"

namespace ss2d {
namespace {

constexpr int kFmBlock = 128;            // K (in bytes) of a block, a stage and a swizzled row
constexpr int kFmRows = 128;             // lanes of an MMA
constexpr uint32_t kFmTile = kFmRows * kFmBlock;  // bytes of a 128-row tile of a stage
constexpr size_t kFmWorkspace = 256;     // the error word of the bounded waits
constexpr int kFmMaxSplit = 8;           // CTAs of a cluster of the narrow kernel
constexpr int kFmMaxWideSplit = 4;       // of the wide one: eight, alone on their SMs, are slow to start (5 us more)

struct Fp8Args {
    const float *a_scales, *w_scales, *bias;
    void *c;
    int *err;
    int M, N, KB;
    int c_bf16;
    int vec;      // wide: bytes that rows of c and their tiles are aligned to: 32, 16 or 0
    int mtiles;   // wide: tiles along M;  narrow: tiles along the tokens
    int tiles;    // of the whole product
    int split;    // CTAs of a cluster, each with its part of K
};

// kind::f8f6f4: fp32 accumulate, e4m3 A and B, both K-major
__host__ __device__ constexpr uint32_t fm_idesc(int n)
{
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kFmRows >> 4) << 24);
}

__device__ __forceinline__ uint32_t fm_pack(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ void fm_store32(void *p, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// The block of K that `it` counts, over a ring of n slots: its slot, and the parity of its round.
struct Ring {
    uint32_t slot, round;
    __device__ __forceinline__ Ring(uint32_t it, uint32_t n) : slot(it % n), round((it / n) & 1u) {}
};

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// The address of this CTA's shared memory at `addr` in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_at(uint32_t addr, uint32_t rank)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(remote) : "r"(addr), "r"(rank));
    return remote;
}

__device__ __forceinline__ float cluster_ld(uint32_t remote)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

__device__ __forceinline__ float4 cluster_ld4(uint32_t remote)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(remote)
                 : "memory");
    return v;
}

// One block's MMAs, of one thread: A 128 rows, B n rows, 128 bytes of K.
__device__ __forceinline__ void fm_mma_block(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc)
{
#pragma unroll
    for (uint32_t k = 0; k < kFmBlock / 32; ++k)
        tc::mma_e4m3(tmem, a + 2 * k, b + 2 * k, idesc, k > 0);  // addresses in units of 16 bytes
}

// ---- wide ----------------------------------------------------------------------------------

constexpr int kWideThreads = 320;  // copy warp, MMA warp, eight warps that scale and add
constexpr int kWideSumWarps = 8;

template <int BN>
struct Wide {
    static constexpr int kStages = BN == 256 ? 4 : 6;
    static constexpr int kBuffers = 512 / BN;                 // of tensor memory
    static constexpr uint32_t kStage = kFmTile + BN * kFmBlock;
    static constexpr int kCols = BN / 2;                      // columns of one summing thread
    static constexpr uint32_t kPitch = BN * 4 + 16;           // bytes between rows of a split tile's sums
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + (2 * kStages + 2 * kBuffers) * 8 + 16;
    static_assert(kFmRows * kPitch <= kStages * kStage, "the sums reuse the stages");
    // CTAs of a cluster wait for one another, so none may wait for tensor memory that a CTA of another
    // cluster holds: no two CTAs that wait so fit an SM together (the narrow kernel's need 57 KB or more)
    static_assert(kSmem > 171 * 1024, "alone on its SM among those that wait for a cluster");
};

// Stores `n` (a multiple of 4 where vec, at least 1) neighbouring sums of a row.
template <int N>
__device__ __forceinline__ void fm_store(const Fp8Args &p, size_t at, const float2 (&acc)[N / 2], int n)
{
    if (p.c_bf16) {
        __nv_bfloat16 *c = static_cast<__nv_bfloat16 *>(p.c) + at;
#pragma unroll
        for (int i = 0; i < N / 16; ++i) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = fm_pack(acc[8 * i + j].x, acc[8 * i + j].y);
            if (p.vec == 32 && 16 * i + 16 <= n)
                fm_store32(c + 16 * i, w);
            else if (p.vec && 16 * i + 8 <= n) {
                *reinterpret_cast<uint4 *>(c + 16 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                if (16 * i + 16 <= n)
                    *reinterpret_cast<uint4 *>(c + 16 * i + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (16 * i + 2 * j < n)
                        c[16 * i + 2 * j] = __float2bfloat16_rn(acc[8 * i + j].x);
                    if (16 * i + 2 * j + 1 < n)
                        c[16 * i + 2 * j + 1] = __float2bfloat16_rn(acc[8 * i + j].y);
                }
            }
        }
    } else {
        float *c = static_cast<float *>(p.c) + at;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            if (p.vec && 4 * i + 4 <= n)
                *reinterpret_cast<float4 *>(c + 4 * i) =
                    make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
            else {
                const float f[4] = {acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (4 * i + j < n)
                        c[4 * i + j] = f[j];
            }
        }
    }
}

// SPLIT: one tile for each cluster, the CTA's part of K, and the parts added in distributed shared memory.
template <int BN, bool SPLIT>
__global__ void __launch_bounds__(kWideThreads, 1)
    matmul_fp8_wide_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w, const Fp8Args p)
{
    using W = Wide<BN>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t bars = base + W::kStages * W::kStage;
    auto full = [&](uint32_t s) { return bars + 8 * s; };
    auto empty = [&](uint32_t s) { return bars + 8 * (W::kStages + s); };
    auto done = [&](uint32_t b) { return bars + 8 * (2 * W::kStages + b); };
    auto taken = [&](uint32_t b) { return bars + 8 * (2 * W::kStages + W::kBuffers + b); };
    __shared__ uint32_t tmem_slot;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int s = 0; s < W::kStages; ++s) {
            tc::mbar_init(full(s), 1);
            tc::mbar_init(empty(s), 1);
        }
        for (int b = 0; b < W::kBuffers; ++b) {
            tc::mbar_init(done(b), 1);
            tc::mbar_init(taken(b), kWideSumWarps);
        }
        tc::mbar_init_fence();
    }
    if (warp == 0 && tc::elect_one()) {
        tc::tma_prefetch_map(&map_a);
        tc::tma_prefetch_map(&map_w);
    }
    if (warp == 1)
        tc::tmem_alloc(&tmem_slot, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    grid_wait();
    grid_next();
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *p.err = 0;  // long before any wait of this call can run out
    const uint32_t tmem = tmem_slot;
    bool good = true;
    const int rank = SPLIT ? (int)(blockIdx.x % p.split) : 0;
    const int first = SPLIT ? (int)(blockIdx.x / p.split) : (int)blockIdx.x;
    const int next = SPLIT ? p.tiles : (int)gridDim.x;
    const int kb0 = SPLIT ? (int)((long long)p.KB * rank / p.split) : 0;
    const int kb1 = SPLIT ? (int)((long long)p.KB * (rank + 1) / p.split) : p.KB;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            for (int tile = first; tile < p.tiles && good; tile += next) {
                const int m0 = tile % p.mtiles * kFmRows, n0 = tile / p.mtiles * BN;
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const Ring r(it, W::kStages);
                    good = tc::mbar_wait(empty(r.slot), r.round ^ 1u);
                    if (!good)
                        break;
                    const uint32_t a = base + r.slot * W::kStage;
                    tc::mbar_expect(full(r.slot), W::kStage);
                    tc::tma_load_2d(a, &map_a, full(r.slot), kb * kFmBlock, m0);
                    tc::tma_load_2d(a + kFmTile, &map_w, full(r.slot), kb * kFmBlock, n0);
                }
            }
            // copies must have landed before the CTA's shared memory goes
            for (uint32_t i = it > W::kStages ? it - W::kStages : 0; i < it; ++i)
                tc::mbar_wait(full(Ring(i, W::kStages).slot), Ring(i, W::kStages).round);
        }
    } else if (warp == 1) {
        const uint64_t a_desc = tc::swizzled_desc(base, 16, 1024), w_desc = tc::swizzled_desc(base + kFmTile, 16, 1024);
        uint32_t it = 0;
        for (int tile = first; tile < p.tiles && good; tile += next)
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const Ring r(it, W::kStages), t(it, W::kBuffers);
                good = tc::mbar_wait_warp(taken(t.slot), t.round ^ 1u) && tc::mbar_wait_warp(full(r.slot), r.round);
                if (!good)
                    break;
                tc::fence_after();
                if (tc::elect_one()) {
                    fm_mma_block(tmem + t.slot * BN, a_desc + r.slot * (W::kStage / 16), w_desc + r.slot * (W::kStage / 16),
                                 fm_idesc(BN));
                    tc::commit(empty(r.slot));
                    tc::commit(done(t.slot));
                }
                __syncwarp();
            }
    } else {
        const int group = (warp - 2) / 4;  // half of the tile's columns
        const uint32_t lanes = (uint32_t)(warp % 4) * 32;
        const int row = (int)lanes + lane;
        uint32_t it = 0;
        for (int tile = first; tile < p.tiles && good; tile += next) {
            const int m = tile % p.mtiles * kFmRows + row, n0 = tile / p.mtiles * BN + group * W::kCols;
            const float *sa = p.a_scales + (size_t)min(m, p.M - 1) * p.KB;
            const float *sw = p.w_scales + (size_t)(min(n0, p.N - 1) / kFmBlock) * p.KB;
            float2 acc[W::kCols / 2];
#pragma unroll
            for (int i = 0; i < W::kCols / 2; ++i)
                acc[i] = make_float2(0.0f, 0.0f);
            float s_a = kb0 < kb1 ? sa[kb0] : 0.0f, s_w = kb0 < kb1 ? sw[kb0] : 0.0f;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const Ring t(it, W::kBuffers);
                const float s = s_a * s_w;
                if (kb + 1 < kb1) {  // the next block's scales, on their way meanwhile
                    s_a = sa[kb + 1];
                    s_w = sw[kb + 1];
                }
                good = tc::mbar_wait_warp(done(t.slot), t.round);
                if (!good)
                    break;
                tc::fence_after();
                const uint32_t from = tmem + (lanes << 16) + t.slot * BN + group * W::kCols;
                const float2 s2 = make_float2(s, s);
                uint32_t v[2][16];
                tc::tmem_ld16(from, v[0]);
#pragma unroll
                for (int c = 0; c < W::kCols / 16; ++c) {
                    tc::tmem_wait16(v[c & 1]);
                    if (c + 1 < W::kCols / 16)
                        tc::tmem_ld16(from + 16 * (c + 1), v[(c + 1) & 1]);
                    else {
                        // all of the buffer is in registers
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0)
                            tc::mbar_arrive(taken(t.slot));
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        acc[c * 8 + i] = __ffma2_rn(
                            make_float2(__uint_as_float(v[c & 1][2 * i]), __uint_as_float(v[c & 1][2 * i + 1])), s2,
                            acc[c * 8 + i]);
                }
            }
            if (!good)
                break;
            if (SPLIT) {
                // the last block's MMAs are done and have read their stages: all of them are free
                float *const sums = reinterpret_cast<float *>(smem_raw + (base - tc::smem_u32(smem_raw)));
#pragma unroll
                for (int i = 0; i < W::kCols / 4; ++i)
                    *reinterpret_cast<float4 *>(sums + row * (W::kPitch / 4) + group * W::kCols + 4 * i) =
                        make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
            } else if (m < p.M && n0 < p.N) {
                const int cols = min(W::kCols, p.N - n0);
                if (p.bias)
#pragma unroll
                    for (int i = 0; i < W::kCols / 2; ++i) {
                        if (2 * i < cols)
                            acc[i].x += p.bias[n0 + 2 * i];
                        if (2 * i + 1 < cols)
                            acc[i].y += p.bias[n0 + 2 * i + 1];
                    }
                fm_store<W::kCols>(p, (size_t)m * p.N + n0, acc, cols);
            }
        }
    }
    if (!good && lane == 0)
        wait_ran_out(p.err);
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 1)
        tc::tmem_free(tmem, 512);
    if (SPLIT) {
        // The cluster's CTAs add their parts of K in rank order, each for its share of the tile's rows.
        cluster_sync();
        if (warp >= 2) {
            const int per = kFmRows / p.split, t = threadIdx.x - 64;
            const int m0 = first % p.mtiles * kFmRows, n0 = first / p.mtiles * BN;
            for (int x = t; x < per * (BN / 4); x += kWideSumWarps * 32) {
                const int r = rank * per + x / (BN / 4), c = x % (BN / 4) * 4;
                const int m = m0 + r, n = n0 + c;
                if (m >= p.M || n >= p.N)
                    continue;
                const uint32_t at = base + r * W::kPitch + c * 4;
                float4 part[kFmMaxWideSplit];
#pragma unroll
                for (int i = 0; i < kFmMaxWideSplit; ++i)
                    if (i < p.split)
                        part[i] = cluster_ld4(cluster_at(at, i));
                float y[4] = {part[0].x, part[0].y, part[0].z, part[0].w};
#pragma unroll
                for (int i = 1; i < kFmMaxWideSplit; ++i)
                    if (i < p.split)
                        y[0] += part[i].x, y[1] += part[i].y, y[2] += part[i].z, y[3] += part[i].w;
                const int left = min(4, p.N - n);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (p.bias && j < left)
                        y[j] += p.bias[n + j];
                const size_t to = (size_t)m * p.N + n;
                if (p.c_bf16) {
                    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.c) + to;
                    if (p.vec)
                        *reinterpret_cast<uint2 *>(o) = make_uint2(fm_pack(y[0], y[1]), fm_pack(y[2], y[3]));
                    else
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < left)
                                o[j] = __float2bfloat16_rn(y[j]);
                } else {
                    float *o = static_cast<float *>(p.c) + to;
                    if (p.vec)
                        *reinterpret_cast<float4 *>(o) = make_float4(y[0], y[1], y[2], y[3]);
                    else
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < left)
                                o[j] = y[j];
                }
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while another reads its sums
    }
}

// ---- narrow --------------------------------------------------------------------------------

constexpr int kNarrowThreads = 192;  // copy warp, MMA warp, four warps that scale and add
constexpr int kNarrowStages = 4;
// 128 columns of tensor memory for a CTA and more than a quarter of an SM's shared memory, so that all
// CTAs that fit an SM can hold their columns at once: the CTAs of a cluster wait for one another, and
// none may wait for columns that a CTA of another cluster holds.
constexpr int kNarrowCols = 128;

template <int BT>
struct Narrow {
    static constexpr int kBuffers = kNarrowCols / BT;
    static constexpr uint32_t kStage = kFmTile + BT * kFmBlock;
    static constexpr size_t kSmem = 1024 + (size_t)kNarrowStages * kStage + 2 * 4 * BT * 4 +
                                    (2 * kNarrowStages + 2 * kBuffers) * 8 + 16;
    static_assert(kSmem > 57 * 1024, "more than a quarter of an SM's shared memory");
    static_assert((size_t)kNarrowStages * kStage >= (size_t)BT * kFmRows * 4, "the sums reuse the stages");
};

template <int BT>
__global__ void __launch_bounds__(kNarrowThreads)
    matmul_fp8_narrow_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w, const Fp8Args p)
{
    using W = Narrow<BT>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    float *const sums = reinterpret_cast<float *>(smem_raw + (base - tc::smem_u32(smem_raw)));  // [BT][128]
    float *const scales = sums + kNarrowStages * W::kStage / 4;  // [warp][2][BT]
    const uint32_t bars = base + kNarrowStages * W::kStage + 2 * 4 * BT * 4;
    auto full = [&](uint32_t s) { return bars + 8 * s; };
    auto empty = [&](uint32_t s) { return bars + 8 * (kNarrowStages + s); };
    auto done = [&](uint32_t b) { return bars + 8 * (2 * kNarrowStages + b); };
    auto taken = [&](uint32_t b) { return bars + 8 * (2 * kNarrowStages + W::kBuffers + b); };
    __shared__ uint32_t tmem_slot;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int rank = (int)(blockIdx.x % p.split);
    const int tile = (int)(blockIdx.x / p.split);
    const int t0 = tile % p.mtiles * BT, n0 = tile / p.mtiles * kFmRows;
    const int kb0 = (int)((long long)p.KB * rank / p.split), kb1 = (int)((long long)p.KB * (rank + 1) / p.split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kNarrowStages; ++s) {
            tc::mbar_init(full(s), 1);
            tc::mbar_init(empty(s), 1);
        }
        for (int b = 0; b < W::kBuffers; ++b) {
            tc::mbar_init(done(b), 1);
            tc::mbar_init(taken(b), 4);
        }
        tc::mbar_init_fence();
        tc::tma_prefetch_map(&map_a);
        tc::tma_prefetch_map(&map_w);
    }
    if (warp == 1)
        tc::tmem_alloc(&tmem_slot, kNarrowCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    grid_wait();
    grid_next();
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *p.err = 0;
    const uint32_t tmem = tmem_slot;
    bool good = true;
    float2 acc[BT / 2];

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const Ring r(it, kNarrowStages);
                good = tc::mbar_wait(empty(r.slot), r.round ^ 1u);
                if (!good)
                    break;
                const uint32_t w = base + r.slot * W::kStage;
                tc::mbar_expect(full(r.slot), W::kStage);
                tc::tma_load_2d(w, &map_w, full(r.slot), kb * kFmBlock, n0);
                tc::tma_load_2d(w + kFmTile, &map_a, full(r.slot), kb * kFmBlock, t0);
            }
            // copies must have landed before the CTA's shared memory goes
            for (uint32_t i = it > kNarrowStages ? it - kNarrowStages : 0; i < it; ++i)
                tc::mbar_wait(full(Ring(i, kNarrowStages).slot), Ring(i, kNarrowStages).round);
        }
    } else if (warp == 1) {
        const uint64_t w_desc = tc::swizzled_desc(base, 16, 1024), a_desc = tc::swizzled_desc(base + kFmTile, 16, 1024);
        uint32_t it = 0;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const Ring r(it, kNarrowStages), t(it, W::kBuffers);
            good = tc::mbar_wait_warp(taken(t.slot), t.round ^ 1u) && tc::mbar_wait_warp(full(r.slot), r.round);
            if (!good)
                break;
            tc::fence_after();
            if (tc::elect_one()) {
                fm_mma_block(tmem + t.slot * BT, w_desc + r.slot * (W::kStage / 16), a_desc + r.slot * (W::kStage / 16),
                             fm_idesc(BT));
                tc::commit(empty(r.slot));
                tc::commit(done(t.slot));
            }
            __syncwarp();
        }
    } else {
        // Each warp keeps its own copy of a block's BT scales, two blocks deep.
        const uint32_t lanes = (uint32_t)(warp % 4) * 32;
        float *const mine = scales + (warp - 2) * 2 * BT;
        const float *sw = p.w_scales + (size_t)(n0 / kFmBlock) * p.KB;
        constexpr int kPer = (BT + 31) / 32;
        float next[kPer];
        auto fetch = [&](int kb) {
            const float w = sw[kb];
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                next[i] = lane + 32 * i < BT && t0 + lane + 32 * i < p.M
                              ? w * p.a_scales[(size_t)(t0 + lane + 32 * i) * p.KB + kb]
                              : 0.0f;
        };
#pragma unroll
        for (int i = 0; i < BT / 2; ++i)
            acc[i] = make_float2(0.0f, 0.0f);
        if (kb0 < kb1)
            fetch(kb0);
        uint32_t it = 0;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const Ring t(it, W::kBuffers);
            float *const s = mine + (it & 1) * BT;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (lane + 32 * i < BT)
                    s[lane + 32 * i] = next[i];
            if (kb + 1 < kb1)
                fetch(kb + 1);
            __syncwarp();
            good = tc::mbar_wait_warp(done(t.slot), t.round);
            if (!good)
                break;
            tc::fence_after();
            const uint32_t from = tmem + (lanes << 16) + t.slot * BT;
#pragma unroll
            for (int c = 0; c < BT / 16; ++c) {
                uint32_t v[16];
                tc::tmem_ld16(from + 16 * c, v);
                tc::tmem_wait16(v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 f = *reinterpret_cast<const float4 *>(s + 16 * c + 4 * i);
                    acc[c * 8 + 2 * i] = __ffma2_rn(
                        make_float2(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])), make_float2(f.x, f.y),
                        acc[c * 8 + 2 * i]);
                    acc[c * 8 + 2 * i + 1] = __ffma2_rn(
                        make_float2(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])), make_float2(f.z, f.w),
                        acc[c * 8 + 2 * i + 1]);
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive(taken(t.slot));
        }
    }
    if (!good && lane == 0)
        wait_ran_out(p.err);
    __syncwarp();
    tc::fence_before();
    __syncthreads();  // every MMA and copy of this CTA is done: its stages are free
    if (warp == 1)
        tc::tmem_free(tmem, kNarrowCols);
    if (warp >= 2) {
        const int row = (warp % 4) * 32 + lane;
#pragma unroll
        for (int i = 0; i < BT / 2; ++i) {
            sums[(2 * i) * kFmRows + row] = acc[i].x;
            sums[(2 * i + 1) * kFmRows + row] = acc[i].y;
        }
    }
    // The cluster's CTAs add their parts of K in rank order, each for its share of the tokens.
    if (p.split > 1)
        cluster_sync();
    else
        __syncthreads();
    if (warp >= 2) {
        const int row = (warp % 4) * 32 + lane, n = n0 + row;
        const float bias = p.bias && n < p.N ? p.bias[n] : 0.0f;
        const uint32_t from = base + (uint32_t)row * 4;
        for (int t = rank; t < BT && t0 + t < p.M; t += p.split) {
            float y;
            if (p.split > 1) {
                float part[kFmMaxSplit];
#pragma unroll
                for (int r = 0; r < kFmMaxSplit; ++r)
                    if (r < p.split)
                        part[r] = cluster_ld(cluster_at(from + (uint32_t)t * kFmRows * 4, (uint32_t)r));
                y = part[0];
#pragma unroll
                for (int r = 1; r < kFmMaxSplit; ++r)
                    if (r < p.split)
                        y += part[r];
            } else {
                y = sums[t * kFmRows + row];
            }
            y += bias;
            if (n < p.N) {
                const size_t at = (size_t)(t0 + t) * p.N + n;
                if (p.c_bf16)
                    static_cast<__nv_bfloat16 *>(p.c)[at] = __float2bfloat16_rn(y);
                else
                    static_cast<float *>(p.c)[at] = y;
            }
        }
    }
    __syncwarp();
    if (p.split > 1)
        cluster_sync();  // no CTA leaves while another reads its sums
}

// ---- host ----------------------------------------------------------------------------------

cudaError_t fm_map(CUtensorMap *map, const void *base, int rows, int K, int box_rows)
{
    const cuuint64_t sizes[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)K};
    const cuuint32_t box[2] = {kFmBlock, (cuuint32_t)box_rows};
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, sizes, strides, box);
}

template <int BN, bool SPLIT>
cudaError_t launch_wide(const ss2d_matmul_fp8_args &g, Fp8Args p, int split, int sms, cudaStream_t s)
{
    static int configured[kMaxDevices];
    CUtensorMap a, w;
    cudaError_t e = fm_map(&a, g.a, g.M, g.K, kFmRows);
    if (e == cudaSuccess)
        e = fm_map(&w, g.w, g.N, g.K, BN);
    if (e == cudaSuccess)
        e = configure_smem(matmul_fp8_wide_kernel<BN, SPLIT>, (int)Wide<BN>::kSmem, configured);
    if (e != cudaSuccess)
        return e;
    p.mtiles = (g.M + kFmRows - 1) / kFmRows;
    const long long tiles = (long long)p.mtiles * ((g.N + BN - 1) / BN);
    if (tiles > 0x7fffffff - sms)
        return cudaErrorInvalidConfiguration;
    p.tiles = (int)tiles;
    p.split = split;
    return launch_early(matmul_fp8_wide_kernel<BN, SPLIT>, (unsigned)(SPLIT ? p.tiles * split : min(p.tiles, sms)),
                        kWideThreads, Wide<BN>::kSmem, s, split, a, w, p);
}

template <int BT>
cudaError_t launch_narrow(const ss2d_matmul_fp8_args &g, Fp8Args p, int split, cudaStream_t s)
{
    static int configured[kMaxDevices];
    CUtensorMap a, w;
    cudaError_t e = fm_map(&a, g.a, g.M, g.K, BT);
    if (e == cudaSuccess)
        e = fm_map(&w, g.w, g.N, g.K, kFmRows);
    if (e == cudaSuccess)
        e = configure_smem(matmul_fp8_narrow_kernel<BT>, (int)Narrow<BT>::kSmem, configured);
    if (e != cudaSuccess)
        return e;
    p.mtiles = (g.M + BT - 1) / BT;
    p.tiles = p.mtiles * ((g.N + kFmRows - 1) / kFmRows);
    p.split = split;
    return launch_early(matmul_fp8_narrow_kernel<BT>, (unsigned)(p.tiles * split), kNarrowThreads, Narrow<BT>::kSmem, s,
                        split, a, w, p);
}

cudaError_t launch_matmul_fp8(const ss2d_matmul_fp8_args &g, const Fp8Args &p, cudaStream_t s)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    const long long wrows = (g.N + kFmRows - 1) / kFmRows, mtiles = (g.M + kFmRows - 1) / kFmRows;
    if (g.M <= 32) {
        // The weights' bytes count: as many CTAs as two for each SM, of two blocks of K or more.  (6144 x 2048,
        // 4 tokens: split 1, 2, 4, 8: 8.0, 6.3, 6.0, 7.2 us;  4096 x 8192: 16.9, 13.0, 10.6, 10.1 us.)
        int split = 1;
        while (split < kFmMaxSplit && wrows * split * 2 <= 2 * sms && split * 4 <= p.KB)
            split *= 2;
        return g.M <= 16 ? launch_narrow<16>(g, p, split, s) : launch_narrow<32>(g, p, split, s);
    }
    // In blocks of 128 columns: a 128 x 256 tile takes 1.5 times what a 128 x 128 one takes, and adding the parts
    // of a split about 9 blocks (128 tokens, 4096 x 8192: 27.4, 19.5, 14.7 us for split 1, 2, 4;  512 tokens,
    // 6144 x 2048: 15.4 us in 192 tiles of 128 columns, 12.3 us in 96 of 256).
    auto waves = [&](long long tiles) { return (tiles + sms - 1) / sms; };
    const long long t128 = mtiles * wrows, t256 = mtiles * ((g.N + 255) / 256);
    long long best = 2 * waves(t128) * p.KB;
    int split = 1;
    for (int x = 2; x <= kFmMaxWideSplit && t128 * x <= sms && x <= p.KB; x *= 2)
        if (2 * ((p.KB + x - 1) / x + 9) < best) {
            best = 2 * ((p.KB + x - 1) / x + 9);
            split = x;
        }
    return 3 * waves(t256) * p.KB < best ? launch_wide<256, false>(g, p, 1, sms, s)
           : split > 1                   ? launch_wide<128, true>(g, p, split, sms, s)
                                         : launch_wide<128, false>(g, p, 1, sms, s);
}

int fm_check(const char *call, const ss2d_matmul_fp8_args *a)
{
    if (!a || a->struct_size != sizeof(ss2d_matmul_fp8_args))
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: args is null or its struct_size is wrong", call);
    if (a->M <= 0 || a->N <= 0 || a->K <= 0)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: sizes must be positive (M=%d N=%d K=%d)", call, a->M, a->N, a->K);
    if (a->K % 16 != 0)
        return op_fail(SS2D_ERR_UNSUPPORTED, "%s: K=%d is not a multiple of 16", call, a->K);
    if (a->M > (1 << 30) || a->N > (1 << 30) || a->K > (1 << 30))
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: problem too large", call);
    if (a->c_dtype != SS2D_F32 && a->c_dtype != SS2D_BF16)
        return op_fail(SS2D_ERR_UNSUPPORTED, "%s: dtype code %d of c must be SS2D_F32 or SS2D_BF16", call, a->c_dtype);
    return SS2D_OK;
}

}  // namespace

cudaError_t matmul_fp8_wait_ran_out(bool *out, cudaStream_t s) { return take_wait_ran_out(out, s); }

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
                         {"a_scales", args->a_scales, M * KB * 4, 4},
                         {"w", args->w, N * K},
                         {"w_scales", args->w_scales, (N + kFmBlock - 1) / kFmBlock * KB * 4, 4},
                         {"bias", args->bias, N * 4, 4}};
    const size_t esize = args->c_dtype == SS2D_BF16 ? 2 : 4;
    const OpSpan out[] = {{"c", args->c, M * N * esize}, {"workspace", workspace, kFmWorkspace}};
    st = op_check_tensors(call, in, 5, out, 2);
    if (st != SS2D_OK)
        return st;
    Fp8Args p{};
    p.a_scales = args->a_scales;
    p.w_scales = args->w_scales;
    p.bias = args->bias;
    p.c = args->c;
    p.err = static_cast<int *>(workspace);
    p.M = args->M;
    p.N = args->N;
    p.KB = (int)KB;
    p.c_bf16 = args->c_dtype == SS2D_BF16;
    const uintptr_t along = reinterpret_cast<uintptr_t>(args->c) | (N * esize);
    p.vec = along % 32 == 0 ? 32 : along % 16 == 0 ? 16 : 0;
    const cudaError_t e = launch_matmul_fp8(*args, p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SS2D_OK : op_cuda_fail(e, "ss2d_matmul_fp8 launch");
}
