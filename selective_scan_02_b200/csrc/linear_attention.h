// linear_attention.h -- shared by the linear-attention kernels and their C entry points (internal).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ss2d {

// Head widths: multiples of 8 (16-byte rows of bf16) up to kLaMaxDim.
constexpr int kLaMaxDim = 128;

// Smallest log decay that the kernels tell apart from a decay of zero: exp(-128) is below
// the smallest fp32 number, and the clamp keeps sums of log decays finite.
constexpr float kLaMinLogDecay = -128.0f;

// NaN stays NaN.
__host__ __device__ inline float la_clamp(float g) { return g < kLaMinLogDecay ? kLaMinLogDecay : g; }

// One call over whole sequences (L tokens of B sequences) or, with slots or pool set, over one
// token of each of B rows (L = 1, states in a pool).
struct LinAttnArgs {
    const __nv_bfloat16 *q, *k, *v;
    long long q_batch, q_token, q_head;  // strides in elements
    long long k_batch, k_token, k_head;
    long long v_batch, v_token, v_head;
    const float *log_decay;  // (H), or (B, L, H) with per_token
    const int *lengths;      // (B) or null
    const int *slots;        // (B) or null (step only)
    const float *h0;         // (B, H, Dk, Dv) or null; the pool (step)
    float *h_last;           // (B, H, Dk, Dv) or null; the pool (step)
    __nv_bfloat16 *out;      // (B, L, H, Dv)
    int *err;                // the workspace's error word (null: step)
    float scale;
    int per_token;
    int B, L, G, H, Dk, Dv, pool;
};

// Token by token.
cudaError_t launch_linear_recurrent(const LinAttnArgs &a, bool step, cudaStream_t s);
// In chunks of 128 tokens, with linear_chunked_workspace (of the sizes alone) bytes of workspace.
size_t linear_chunked_workspace(const LinAttnArgs &a);
cudaError_t launch_linear_chunked(const LinAttnArgs &a, void *workspace, cudaStream_t s);

}  // namespace ss2d
