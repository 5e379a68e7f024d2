// linear_recurrent.cu -- linear attention token by token (ss2d_linear_attention_step, and short
// prompts of ss2d_linear_attention).
//
//   S <- exp(g) S + k v^T          S (Dk, Dv) fp32 for each sequence and head
//   o  = scale * S^T q             rounded to bf16
//
// One token reads and writes the whole state and does two multiply-adds for each of its
// elements, so the kernel is bounded by the state's bytes.  A CTA holds 32 columns of one
// head's state in registers: 8 lanes of 4 columns (16-byte accesses, a 128-byte run for each
// row of the state) by 16 rows at a time, so that even one sequence of few heads spreads over
// many SMs, and all of the state's loads are in flight at once.  Columns of the state do not
// meet: o's column j needs column j of S alone.  The state is not
// wanted again before the other layers' states have passed, so its accesses are marked as streaming: 64 rows of 32
// heads of 128 x 128 (270 MB) 46.4 -> 43.0 us, 6.3 TB/s, and no slower where it all fits L2 (24 heads of 64 x 96,
// 33 rows: 9.1 us both).  One row of 16 heads: 3.4 us a call, what launching it takes.  64 columns a CTA: 48.7 us.
#include "launch_util.h"
#include "linear_attention.h"

namespace ss2d {
namespace {

constexpr int kLrThreads = 128;
constexpr int kLrCols = 32;                       // columns of the state in one CTA
constexpr int kLrGroups = kLrThreads / (kLrCols / 4);  // rows of the state held by the CTA at a time

// STEP: the tokens of this CTA are the rows of the batch that name its slot, in their order (one,
// where no slot is named twice; the CTAs of the later ones have nothing to do).  Otherwise they
// are the tokens of sequence b.
//
// ROWS: of the state held by one thread; Dk at most kLrGroups times as many.  (128 rows of 32 heads of 64 x 64: 19.5 us
// with four, 24.5 with the eight that Dk = 128 needs.)
template <bool STEP, int ROWS>
__global__ void __launch_bounds__(kLrThreads) linear_recurrent_kernel(const LinAttnArgs a)
{
    __shared__ float sq[kLaMaxDim], sk[kLaMaxDim];
    __shared__ float part[kLrThreads / 32][kLrCols];
    __shared__ int next_row;
    const int tid = threadIdx.x, lane = tid % 32;
    const int slices = (a.Dv + kLrCols - 1) / kLrCols;
    const int slice = (int)(blockIdx.x % slices);
    const long long bh = blockIdx.x / slices;
    const int h = (int)(bh % a.H), b = (int)(bh / a.H);
    const int group = h / (a.H / a.G);
    const int c = slice * kLrCols + (tid % (kLrCols / 4)) * 4;  // this thread's first column
    const int r0 = tid / (kLrCols / 4);                         // and first row
    const bool cols = c < a.Dv;

    grid_wait();
    grid_next();
    if (!STEP && blockIdx.x == 0 && tid == 0)
        *a.err = 0;  // nothing here waits

    // one token's q, k, v and log decay: loads that are on their way before they are needed
    float q_in = 0.0f, k_in = 0.0f, g = 0.0f;
    uint2 v_in = make_uint2(0, 0);
    auto fetch = [&](long long rb, long long rt) {
        if (tid < a.Dk) {
            q_in = __bfloat162float(a.q[rb * a.q_batch + rt * a.q_token + group * a.q_head + tid]);
            k_in = __bfloat162float(a.k[rb * a.k_batch + rt * a.k_token + group * a.k_head + tid]);
        }
        if (cols)
            v_in = *reinterpret_cast<const uint2 *>(a.v + rb * a.v_batch + rt * a.v_token + h * a.v_head + c);
        g = a.log_decay[a.per_token ? (rb * (STEP ? 1 : a.L) + rt) * a.H + h : h];
    };
    if (STEP)
        fetch(b, 0);
    long long slot = b;
    int count = a.L;
    if (STEP && a.slots) {
        slot = a.slots[b];
        if (slot < 0 || slot >= a.pool)
            return;
    } else if (!STEP && a.lengths) {
        count = min(max(a.lengths[b], 0), a.L);
    }

    const size_t at = ((size_t)slot * a.H + h) * (size_t)a.Dk * a.Dv;
    float4 s[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = r0 + i * kLrGroups;
        s[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (a.h0 && cols && r < a.Dk)
            s[i] = __ldcs(reinterpret_cast<const float4 *>(a.h0 + at + (size_t)r * a.Dv + c));
    }

    // the first row of this slot after `from`; a.B if there is none
    auto find_next = [&](int from) {
        for (int i = from + 1 + tid; i < a.B; i += kLrThreads)
            if (a.slots[i] == (int)slot) {
                atomicMin(&next_row, i);
                break;
            }
    };
    if (STEP && a.slots) {
        // (while the state is on its way)
        if (tid == 0)
            next_row = a.B;
        __syncthreads();
        find_next(b);
        bool earlier = false;
        for (int i = tid; i < b; i += kLrThreads)
            earlier |= a.slots[i] == (int)slot;
        if (__syncthreads_or(earlier))
            return;
    }

    if (!STEP && count > 0)
        fetch(b, 0);
    int row = STEP ? b : 0;
    while (STEP || row < count) {
        const long long rb = STEP ? row : b, rt = STEP ? 0 : row;
        if (tid < a.Dk) {
            sq[tid] = q_in * a.scale;
            sk[tid] = k_in;
        }
        const float4 v = make_float4(__uint_as_float(v_in.x << 16), __uint_as_float(v_in.x & 0xffff0000u),
                                     __uint_as_float(v_in.y << 16), __uint_as_float(v_in.y & 0xffff0000u));
        // exp(g) = keep + grow: 1 and a small number for slow decays, whose rounding to fp32 would otherwise add up
        // over the tokens, else 0 and the decay itself
        const bool slow = g > -0.5f;
        const float keep = slow ? 1.0f : 0.0f, grow = slow ? expm1f(g) : expf(la_clamp(g));
        if (!STEP && row + 1 < count)
            fetch(b, row + 1);
        __syncthreads();
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int r = r0 + i * kLrGroups;
            if (r < a.Dk) {
                const float kr = sk[r], qr = sq[r];
                s[i].x = fmaf(s[i].x, keep, fmaf(s[i].x, grow, kr * v.x));
                s[i].y = fmaf(s[i].y, keep, fmaf(s[i].y, grow, kr * v.y));
                s[i].z = fmaf(s[i].z, keep, fmaf(s[i].z, grow, kr * v.z));
                s[i].w = fmaf(s[i].w, keep, fmaf(s[i].w, grow, kr * v.w));
                o.x = fmaf(qr, s[i].x, o.x);
                o.y = fmaf(qr, s[i].y, o.y);
                o.z = fmaf(qr, s[i].z, o.z);
                o.w = fmaf(qr, s[i].w, o.w);
            }
        }
        // the four rows of a warp, then the warps
#pragma unroll
        for (int d = 8; d < 32; d *= 2) {
            o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
            o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
            o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
            o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
        }
        if (lane < kLrCols / 4)
            *reinterpret_cast<float4 *>(&part[tid / 32][lane * 4]) = o;
        __syncthreads();
        if (tid < kLrCols && slice * kLrCols + tid < a.Dv) {
            float y = 0.0f;
#pragma unroll
            for (int w = 0; w < kLrThreads / 32; ++w)
                y += part[w][tid];
            a.out[((rb * (STEP ? 1 : a.L) + rt) * a.H + h) * a.Dv + slice * kLrCols + tid] = __float2bfloat16_rn(y);
        }
        if (STEP) {
            if (!a.slots || next_row >= a.B)
                break;
            row = next_row;
            fetch(row, 0);
            __syncthreads();
            if (tid == 0)
                next_row = a.B;
            __syncthreads();
            find_next(row);  // (the loop's next barrier stands before it is read)
        } else {
            ++row;
        }
    }
    if (a.h_last && cols) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int r = r0 + i * kLrGroups;
            if (r < a.Dk)
                __stcs(reinterpret_cast<float4 *>(a.h_last + at + (size_t)r * a.Dv + c), s[i]);
        }
    }
}

template <bool STEP>
cudaError_t launch_rows(const LinAttnArgs &a, int rows, unsigned grid, cudaStream_t s)
{
    return rows <= 2   ? launch_early(linear_recurrent_kernel<STEP, 2>, grid, kLrThreads, 0, s, 1, a)
           : rows <= 4 ? launch_early(linear_recurrent_kernel<STEP, 4>, grid, kLrThreads, 0, s, 1, a)
                       : launch_early(linear_recurrent_kernel<STEP, kLaMaxDim / kLrGroups>, grid, kLrThreads, 0, s, 1, a);
}

}  // namespace

cudaError_t launch_linear_recurrent(const LinAttnArgs &a, bool step, cudaStream_t s)
{
    const long long grid = (long long)a.B * a.H * ((a.Dv + kLrCols - 1) / kLrCols);
    if (grid > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    const int rows = (a.Dk + kLrGroups - 1) / kLrGroups;
    return step ? launch_rows<true>(a, rows, (unsigned)grid, s) : launch_rows<false>(a, rows, (unsigned)grid, s);
}

}  // namespace ss2d
