// linear_chunked.cu -- linear attention over whole sequences, in chunks of 128 tokens, on the tensor
// cores (ss2d_linear_attention).
//
// With c_i the sum of the log decays of tokens 0 .. i of a chunk, S the state before the chunk:
//
//   o_i = scale * sum_{j <= i} exp(c_i - c_j) (q_i . k_j) v_j  +  scale * exp(c_i) S^T q_i
//   S'  = exp(c_last) S + sum_j exp(c_last - c_j) k_j v_j^T
//
// so a chunk is four products of 128 tokens:  Q K^T,  P V with P the masked and decayed scores,
// Q S, and K^T (w V) with w_j = exp(c_last - c_j).  A CTA walks the chunks of one head of one
// sequence (or of one segment of it) with the state in registers:
//   copy warp    TMA: Q, K and V tiles, each in a ring of two slots
//   MMA warp     one thread issues tcgen05.mma
//   decay warp   c in 64 bits, and from it every factor that the others need in 32
//   8 warps      scores -> P (bf16, into tensor memory as the A operand of P V);
//                V -> w V (two bf16 parts, likewise, transposed: the A operand of (w V)^T K);
//                the state's update, and its bf16 copy in shared memory for the next Q S;
//                the output
//
// Roundings to bf16, all for an MMA's operands: P and the copy of S once (what they enter, o, is
// itself rounded to bf16), w V in two parts that together keep 16 bits, because the state is an fp32
// result and is summed over the whole sequence.  Sums, states and decays are fp32 or wider.
//
// The decays within a chunk: columns are cut in blocks of 32, m_b = c at the end of block b.  A score
// below the diagonal blocks takes exp(c_i - m_b) exp(m_b - c_j), a product of a row's and a column's
// factor, both at most 1; only the diagonal blocks need an exponential for each element.
//
// Where the heads of all sequences are too few for the GPU, a sequence is cut into segments: a first
// pass sums each segment's own state (K and V only), a small kernel carries the states from segment to
// segment, and the pass above then starts each segment from its own.
#include "api_internal.h"
#include "launch_util.h"
#include "linear_attention.h"
#include "tma.cuh"

namespace ss2d {
namespace {

constexpr int kLcChunk = 128;
constexpr int kLcThreads = 384;       // copy, MMA, decay and an idle warp, then eight computing ones
constexpr int kLcCompute = 4;         // the first of them
constexpr int kLcComputeWarps = 8;
constexpr uint32_t kLcBlock = kLcChunk * 128;  // bytes of 128 tokens by 64 columns of bf16
constexpr int kLcSms = 148;

// Factors of one chunk's decays, all from 64-bit sums; logarithms to base 2.
struct alignas(16) ChunkDecay {
    float cb[kLcChunk];  // c_j - m_b of j's block
    float f[kLcChunk];   // exp(m_b - c_j)
    float m[4];          // m_b
    float dm[4][4];      // m_q - m_b
    float e[4];          // exp(c_last - m_b)
    float total;         // exp(c_last)
};

struct ChunkedArgs {
    LinAttnArgs a;
    float *states;       // (B * H, nseg, Dk, Dv): the segments' own states, then those before them
    float *decays;       // (B * H, nseg): the segments' decays
    int nseg, seg_chunks;
};

template <int DK, int DV>
struct Lc {
    static constexpr uint32_t kQK = DK / 64 * kLcBlock;  // bytes of a tile of Q or K
    static constexpr uint32_t kV = DV / 64 * kLcBlock;
    static constexpr uint32_t kS = DK / 64 * DV * 128;   // the bf16 state: DV rows of DK, blocks of 64
    static constexpr uint32_t kTiles = 2 * (2 * kQK + kV) + kS;
    static constexpr uint32_t kDecayAt = kTiles;
    static constexpr uint32_t kBarsAt = kDecayAt + 2 * (uint32_t)sizeof(ChunkDecay);
    static constexpr size_t kSmem = kBarsAt + 24 * 8;
    static_assert(kSmem <= 232448, "shared memory of an SM");
    // tensor memory: scores (P in place), output, Q S and then (w V)^T K, the two parts of w V
    static constexpr uint32_t kScores = 0, kOut = 128, kInter = 256, kHi = 384, kLo = 448;
};

// kind::f16, fp32 accumulate, bf16 operands, 128 rows
__host__ __device__ constexpr uint32_t lc_idesc(int n, bool b_mn_major)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ uint32_t lc_pack(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float lc_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void lc_store32(void *p, const uint32_t *w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// STATES: the first pass over segments, which sums their own states alone.
template <int DK, int DV, bool STATES>
__global__ void __launch_bounds__(kLcThreads, 1)
    linear_chunked_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const ChunkedArgs p)
{
    using C = Lc<DK, DV>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const LinAttnArgs &a = p.a;
    const uint32_t base = tc::smem_u32(smem);
    const uint32_t sQ = base, sK = sQ + 2 * C::kQK, sV = sK + 2 * C::kQK, sS = sV + 2 * C::kV;
    ChunkDecay *const decay = reinterpret_cast<ChunkDecay *>(smem + C::kDecayAt);
    const uint32_t bars = base + C::kBarsAt;
    const uint32_t q_full = bars, k_full = bars + 16, v_full = bars + 32, q_free = bars + 48, k_free = bars + 64,
                   v_free = bars + 80, dec_full = bars + 96, dec_free = bars + 112, scores_done = bars + 128,
                   inter_done = bars + 136, operands = bars + 144, delta_done = bars + 152, out_done = bars + 160,
                   state_ready = bars + 168;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kBarsAt + 184);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    const int segs = STATES ? p.nseg - 1 : p.nseg;  // the last segment's own state is not carried on
    const int seg = (int)(blockIdx.x % segs);
    const long long bh = blockIdx.x / segs;
    const int h = (int)(bh % a.H), b = (int)(bh / a.H);
    const int group = h / (a.H / a.G);
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;
    const int t_first = seg * p.seg_chunks * kLcChunk;
    const int t_end = min(len, t_first + p.seg_chunks * kLcChunk);
    if ((STATES || p.nseg == 1) && blockIdx.x == 0 && threadIdx.x == 0)
        *a.err = 0;  // the call's first kernel, long before any wait of it can run out
    if (t_first >= len && !(len == 0 && seg == 0 && !STATES))
        return;
    const int chunks = (t_end - t_first + kLcChunk - 1) / kLcChunk;  // 0 for an empty sequence: its state is kept

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            for (uint32_t bar : {q_full, k_full, v_full, q_free, k_free, v_free, dec_full})
                tc::mbar_init(bar + 8 * i, 1);
            tc::mbar_init(dec_free + 8 * i, kLcComputeWarps);
        }
        for (uint32_t bar : {scores_done, inter_done, delta_done, out_done})
            tc::mbar_init(bar, 1);
        tc::mbar_init(operands, kLcComputeWarps);
        tc::mbar_init(state_ready, kLcComputeWarps);
        tc::mbar_init_fence();
    }
    if (warp == 1)
        tc::tmem_alloc(tmem_slot, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    bool good = true;

    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (int c = 0; c < chunks && good; ++c, ++issued) {
                const uint32_t i = c & 1, round = (c >> 1) & 1;
                const int t0 = t_first + c * kLcChunk;
                auto load = [&](uint32_t tile, const CUtensorMap &map, uint32_t full, uint32_t free, int bytes, int head) {
                    if (!tc::mbar_wait(free + 8 * i, round ^ 1u))
                        return false;
                    tc::mbar_expect(full + 8 * i, bytes);
                    for (int x = 0; x < bytes / (int)kLcBlock; ++x)
                        tc::tma_load_4d(tile + i * bytes + x * kLcBlock, &map, full + 8 * i, 64 * x, head, t0, b);
                    return true;
                };
                good = load(sK, map_k, k_full, k_free, C::kQK, group);
                if (good && !STATES)
                    good = load(sQ, map_q, q_full, q_free, C::kQK, group);
                if (good)
                    good = load(sV, map_v, v_full, v_free, C::kV, h);
            }
            // copies must have landed before the CTA's shared memory goes
            for (int c = max(0, issued - 2); c < issued; ++c)
                for (uint32_t full : {k_full, q_full, v_full})
                    if (!STATES || full != q_full)
                        tc::mbar_wait(full + 8 * (c & 1), (c >> 1) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int c = 0; c < chunks && good; ++c) {
                const uint32_t i = c & 1, round = (c >> 1) & 1, turn = c & 1;
                const uint32_t tQ = sQ + i * C::kQK, tK = sK + i * C::kQK, tV = sV + i * C::kV;
                good = tc::mbar_wait(k_full + 8 * i, round) && (STATES || tc::mbar_wait(q_full + 8 * i, round));
                if (!good)
                    break;
                if (!STATES) {
                    // scores = Q K^T; the P V of the chunk before, which reads P in its place, was issued before
                    tc::fence_after();
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k) {
                        const uint32_t off = k / 4 * kLcBlock + k % 4 * 32;
                        tc::mma_bf16(tmem + C::kScores, tc::swizzled_desc(tQ + off, 16, 1024),
                                     tc::swizzled_desc(tK + off, 16, 1024), lc_idesc(128, false), k > 0);
                    }
                    tc::commit(scores_done);
                    // Q S
                    good = tc::mbar_wait(state_ready, turn);
                    if (!good)
                        break;
                    tc::fence_after();
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k)
                        tc::mma_bf16(tmem + C::kInter, tc::swizzled_desc(tQ + k / 4 * kLcBlock + k % 4 * 32, 16, 1024),
                                     tc::swizzled_desc(sS + k / 4 * (DV * 128) + k % 4 * 32, 16, 1024),
                                     lc_idesc(DV, false), k > 0);
                    tc::commit(inter_done);
                    tc::commit(q_free + 8 * i);
                }
                good = tc::mbar_wait(v_full + 8 * i, round) && tc::mbar_wait(operands, turn);
                if (!good)
                    break;
                tc::fence_after();
                // (w V)^T K, the two parts of w V after one another
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int k = 0; k < kLcChunk / 16; ++k)
                        tc::mma_bf16_ta(tmem + C::kInter, tmem + (part ? C::kLo : C::kHi) + 8 * k,
                                        tc::swizzled_desc(tK + 2048 * k, kLcBlock, 1024), lc_idesc(DK, true),
                                        part > 0 || k > 0);
                tc::commit(delta_done);
                tc::commit(k_free + 8 * i);
                if (!STATES) {
                    // out += P V; P of tokens 32 b .. lies in the first 16 columns of block b of the scores
#pragma unroll
                    for (int k = 0; k < kLcChunk / 16; ++k)
                        tc::mma_bf16_ta(tmem + C::kOut, tmem + C::kScores + k / 2 * 32 + k % 2 * 8,
                                        tc::swizzled_desc(tV + 2048 * k, kLcBlock, 1024), lc_idesc(DV, true), 1);
                    tc::commit(out_done);
                }
                tc::commit(v_free + 8 * i);
            }
        }
    } else if (warp == 2) {
        // Four tokens of each lane, eight lanes of each block.
        const float fixed = a.per_token ? 0.0f : a.log_decay[h];
        const float *gates = a.log_decay + (a.per_token ? ((long long)b * a.L) * a.H + h : 0);
        float g[4];
        auto fetch = [&](int c) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = t_first + c * kLcChunk + lane * 4 + j;
                g[j] = t >= t_end ? 0.0f : la_clamp(a.per_token ? gates[(long long)t * a.H] : fixed);
            }
        };
        double whole = 0.0;
        if (chunks > 0)
            fetch(0);
        for (int c = 0; c < chunks && good; ++c) {
            const uint32_t i = c & 1, round = (c >> 1) & 1;
            double s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[j] = (j ? s[j - 1] : 0.0) + (double)g[j] * 1.4426950408889634;
            if (c + 1 < chunks)
                fetch(c + 1);
            double before = s[3];
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const double v = __shfl_up_sync(0xffffffffu, before, d);
                if (lane >= d)
                    before += v;
            }
            before -= s[3];
            // an exact zero before the first token, whatever the rounding of the two sums
            if (lane == 0)
                before = 0.0;
            const double end = before + s[3];
            double m[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                m[q] = __shfl_sync(0xffffffffu, end, 8 * q + 7);
            good = __all_sync(0xffffffffu, tc::mbar_wait(dec_free + 8 * i, round ^ 1u));
            if (!good)
                break;
            ChunkDecay &out = decay[i];
            const double mine = lane < 8 ? m[0] : lane < 16 ? m[1] : lane < 24 ? m[2] : m[3];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float cb = (float)(before + s[j] - mine);
                out.cb[lane * 4 + j] = cb;
                out.f[lane * 4 + j] = exp2f(-cb);
            }
            if (lane < 4) {
                const double own = lane == 0 ? m[0] : lane == 1 ? m[1] : lane == 2 ? m[2] : m[3];
                out.m[lane] = (float)own;
                out.e[lane] = exp2f((float)(m[3] - own));
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    out.dm[q][lane] = (float)(m[q] - own);
                if (lane == 0)
                    out.total = exp2f((float)m[3]);
            }
            whole += m[3];
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive(dec_full + 8 * i);
        }
        if (STATES && lane == 0 && good)
            p.decays[bh * p.nseg + seg] = exp2f((float)whole);
    } else if (warp >= kLcCompute) {
        const int quarter = warp % 4, half = (warp - kLcCompute) / 4;
        const uint32_t lanes = tmem + ((uint32_t)quarter << 21);  // this warp's 32 lanes of tensor memory
        const int row = quarter * 32 + lane;  // token of the scores and of the output; column of V and of S
        const bool mine = row < DV && row < a.Dv;
        constexpr int SK = DK / 2;            // rows of S in this thread
        float s[SK];
        const float *from = STATES ? nullptr
                            : p.nseg > 1 ? p.states + (bh * p.nseg + seg) * (long long)a.Dk * a.Dv
                            : a.h0       ? a.h0 + bh * (long long)a.Dk * a.Dv
                                         : nullptr;
#pragma unroll
        for (int i = 0; i < SK; ++i) {
            const int r = half * SK + i;
            s[i] = from && mine && r < a.Dk ? from[(long long)r * a.Dv + row] : 0.0f;
        }
        // the bf16 copy of S: row `row` of 64-column blocks, 16-byte pieces swizzled as TMA would
        auto publish = [&] {
            if (row < DV) {
#pragma unroll
                for (int x = 0; x < SK / 8; ++x) {
                    const int r = half * SK + 8 * x;
                    const uint32_t at = r / 64 * (DV * 128) + row * 128 + (((r % 64 / 8) ^ (row & 7)) << 4);
                    *reinterpret_cast<uint4 *>(smem + (sS - base) + at) =
                        make_uint4(lc_pack(s[8 * x], s[8 * x + 1]), lc_pack(s[8 * x + 2], s[8 * x + 3]),
                                   lc_pack(s[8 * x + 4], s[8 * x + 5]), lc_pack(s[8 * x + 6], s[8 * x + 7]));
                }
            }
            tc::fence_async_proxy();
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive(state_ready);
        };
        if (!STATES)
            publish();
        auto wait = [&](uint32_t bar, uint32_t parity) {
            good = __all_sync(0xffffffffu, tc::mbar_wait(bar, parity));
            tc::fence_after();
            return good;
        };
        for (int c = 0; c < chunks; ++c) {
            const uint32_t i = c & 1, round = (c >> 1) & 1, turn = c & 1;
            const int t0 = t_first + c * kLcChunk;
            const int n = min(kLcChunk, t_end - t0);
            const ChunkDecay &d = decay[i];
            unsigned char *const tileV = smem + (sV - base) + i * C::kV;
            if (!wait(dec_full + 8 * i, round) || !wait(v_full + 8 * i, round))
                break;
            // w V, transposed: lane = column of V, tokens in pairs along the columns of tensor memory
            if (quarter * 32 < DV) {
                const unsigned char *const col = tileV + row / 64 * kLcBlock + row % 8 * 2;
                const uint32_t piece = row % 64 / 8;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float e = d.e[half * 2 + x];
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const int t = half * 64 + x * 32 + y * 4;
                        const float4 f = *reinterpret_cast<const float4 *>(&d.f[t]);
                        float w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const __nv_bfloat16 v = *reinterpret_cast<const __nv_bfloat16 *>(
                                col + (t + z) * 128 + ((piece ^ ((t + z) & 7)) << 4));
                            w[z] = t + z < n ? __bfloat162float(v) * (w[z] * e) : 0.0f;
                        }
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t h2 = lc_pack(w[2 * z], w[2 * z + 1]);
                            hi[2 * y + z] = h2;
                            lo[2 * y + z] = lc_pack(w[2 * z] - __uint_as_float(h2 << 16),
                                                    w[2 * z + 1] - __uint_as_float(h2 & 0xffff0000u));
                        }
                    }
                    tc::tmem_st16(lanes + C::kHi + half * 32 + x * 16, hi);
                    tc::tmem_st16(lanes + C::kLo + half * 32 + x * 16, lo);
                }
            }
            if (!STATES) {
                const float cb = d.cb[row];
                // P: blocks of 32 columns, every other one
                if (!wait(scores_done, turn))
                    break;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int blk = 2 * x + half;
                    uint32_t w[16];
                    if (blk <= quarter) {
                        uint32_t v[2][16];
                        tc::tmem_ld16(lanes + C::kScores + blk * 32, v[0]);
                        tc::tmem_ld16(lanes + C::kScores + blk * 32 + 16, v[1]);
                        tc::tmem_wait16(v[0]);
                        tc::tmem_wait16(v[1]);
                        if (blk < quarter) {
                            const float r = a.scale * lc_ex2(cb + d.dm[quarter][blk]);
#pragma unroll
                            for (int y = 0; y < 8; ++y) {
                                const float4 f = *reinterpret_cast<const float4 *>(&d.f[blk * 32 + 4 * y]);
                                const uint32_t *u = &v[y / 4][y % 4 * 4];
                                w[2 * y] = lc_pack(__uint_as_float(u[0]) * (f.x * r), __uint_as_float(u[1]) * (f.y * r));
                                w[2 * y + 1] = lc_pack(__uint_as_float(u[2]) * (f.z * r), __uint_as_float(u[3]) * (f.w * r));
                            }
                        } else {
#pragma unroll
                            for (int y = 0; y < 8; ++y) {
                                const float4 f = *reinterpret_cast<const float4 *>(&d.cb[blk * 32 + 4 * y]);
                                const uint32_t *u = &v[y / 4][y % 4 * 4];
                                const float g[4] = {f.x, f.y, f.z, f.w};
                                float r[4];
#pragma unroll
                                for (int z = 0; z < 4; ++z)
                                    r[z] = 4 * y + z <= lane ? __uint_as_float(u[z]) * (a.scale * lc_ex2(cb - g[z])) : 0.0f;
                                w[2 * y] = lc_pack(r[0], r[1]);
                                w[2 * y + 1] = lc_pack(r[2], r[3]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < 16; ++y)
                            w[y] = 0;
                    }
                    tc::tmem_st16(lanes + C::kScores + blk * 32, w);
                }
                // what the state gives: the start of the output's sum
                if (!wait(inter_done, turn))
                    break;
                const float r = a.scale * lc_ex2(cb + d.m[quarter]);
#pragma unroll
                for (int x = 0; x < DV / 32; ++x) {
                    uint32_t v[16];
                    tc::tmem_ld16(lanes + C::kInter + half * (DV / 2) + 16 * x, v);
                    tc::tmem_wait16(v);
#pragma unroll
                    for (int y = 0; y < 16; ++y)
                        v[y] = __float_as_uint(__uint_as_float(v[y]) * r);
                    tc::tmem_st16(lanes + C::kOut + half * (DV / 2) + 16 * x, v);
                }
            }
            const float total = d.total;
            // rows of K and V behind the last token: zero, whatever the tensors hold there, since a factor of
            // zero would not hide a NaN.  Other warps, and the MMAs of the scores, may still read these rows
            // as they were: nothing of that reaches a row of the output or the state.
            if (n < kLcChunk) {
                if (!wait(k_full + 8 * i, round))
                    break;
                const int t = threadIdx.x - kLcCompute * 32;
                auto clear = [&](unsigned char *tile, int blocks) {
                    for (int x = t; x < blocks * (kLcChunk - n) * 8; x += kLcComputeWarps * 32) {
                        const int blk = x / ((kLcChunk - n) * 8), at = x % ((kLcChunk - n) * 8);
                        *reinterpret_cast<uint4 *>(tile + blk * kLcBlock + n * 128 + at * 16) = make_uint4(0, 0, 0, 0);
                    }
                };
                clear(smem + (sK - base) + i * C::kQK, DK / 64);
                clear(tileV, DV / 64);
                tc::fence_async_proxy();
            }
            tc::tmem_wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(operands);
                tc::mbar_arrive(dec_free + 8 * i);
            }
            if (!wait(delta_done, turn))
                break;
#pragma unroll
            for (int x = 0; x < SK / 16; ++x) {
                uint32_t v[16];
                tc::tmem_ld16(lanes + C::kInter + half * SK + 16 * x, v);
                tc::tmem_wait16(v);
#pragma unroll
                for (int y = 0; y < 16; ++y)
                    s[16 * x + y] = fmaf(s[16 * x + y], total, __uint_as_float(v[y]));
            }
            if (!STATES) {
                publish();
                if (!wait(out_done, turn))
                    break;
                const int t = t0 + row;
                __nv_bfloat16 *const o = a.out + (((long long)b * a.L + t) * a.H + h) * a.Dv + half * (DV / 2);
                const bool wide = a.Dv % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
#pragma unroll
                for (int x = 0; x < DV / 32; ++x) {
                    uint32_t v[16], w[8];
                    tc::tmem_ld16(lanes + C::kOut + half * (DV / 2) + 16 * x, v);
                    tc::tmem_wait16(v);
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        w[y] = lc_pack(__uint_as_float(v[2 * y]), __uint_as_float(v[2 * y + 1]));
                    const int left = a.Dv - half * (DV / 2) - 16 * x;  // columns from here on
                    if (t < t_end && left > 0) {
                        if (wide) {
                            lc_store32(o + 16 * x, w);
                        } else {
                            *reinterpret_cast<uint4 *>(o + 16 * x) = make_uint4(w[0], w[1], w[2], w[3]);
                            if (left > 8)
                                *reinterpret_cast<uint4 *>(o + 16 * x + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                }
            }
        }
        float *const to = STATES                       ? p.states + (bh * p.nseg + seg) * (long long)a.Dk * a.Dv
                          : a.h_last && t_end == len ? a.h_last + bh * (long long)a.Dk * a.Dv
                                                       : nullptr;
        if (good && to && mine)
#pragma unroll
            for (int i = 0; i < SK; ++i)
                if (half * SK + i < a.Dk)
                    to[(long long)(half * SK + i) * a.Dv + row] = s[i];
    }
    if (!good && lane == 0)
        atomicExch(a.err, 1);
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 1)
        tc::tmem_free(tmem, 512);
}

// The state before each segment, from the segments' own states: thread = one element of a head's state.
__global__ void __launch_bounds__(256) linear_carry_kernel(const ChunkedArgs p)
{
    const LinAttnArgs &a = p.a;
    const int size = a.Dk * a.Dv;
    const int per = (size + 255) / 256;
    const long long bh = blockIdx.x / per;
    const int at = (int)(blockIdx.x % per) * 256 + threadIdx.x;
    if (at >= size)
        return;
    const int b = (int)(bh / a.H);
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;
    const int tokens = p.seg_chunks * kLcChunk;
    const int segs = max(1, (len + tokens - 1) / tokens);  // with tokens
    float *s = p.states + bh * p.nseg * size + at;
    const float *decays = p.decays + bh * p.nseg;
    float carry = a.h0 ? a.h0[bh * size + at] : 0.0f;
    constexpr int kAhead = 8;
    for (int i = 0; i < segs; i += kAhead) {
        float own[kAhead], decay[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const bool in = i + j + 1 < segs;  // the last segment's own state is not summed
            own[j] = in ? s[(long long)(i + j) * size] : 0.0f;
            decay[j] = in ? decays[i + j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i + j < segs) {
                s[(long long)(i + j) * size] = carry;
                carry = fmaf(carry, decay[j], own[j]);
            }
    }
}

// Tensor map over (batch, token, head, column), boxes of 128 tokens by 64 columns of one head.
cudaError_t lc_map(CUtensorMap *map, const __nv_bfloat16 *base, int B, int L, int heads, int D, long long batch,
                   long long token, long long head)
{
    const cuuint64_t sizes[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)L, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)head * 2, (cuuint64_t)token * 2, (cuuint64_t)batch * 2};
    const cuuint32_t box[4] = {64, 1, kLcChunk, 1};
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, sizes, strides, box);
}

template <int DK, int DV>
cudaError_t launch_dims(const ChunkedArgs &p, cudaStream_t s)
{
    static int configured[2][kMaxDevices];
    const LinAttnArgs &a = p.a;
    CUtensorMap q, k, v;
    cudaError_t e = lc_map(&q, a.q, a.B, a.L, a.G, a.Dk, a.q_batch, a.q_token, a.q_head);
    if (e == cudaSuccess)
        e = lc_map(&k, a.k, a.B, a.L, a.G, a.Dk, a.k_batch, a.k_token, a.k_head);
    if (e == cudaSuccess)
        e = lc_map(&v, a.v, a.B, a.L, a.H, a.Dv, a.v_batch, a.v_token, a.v_head);
    if (e == cudaSuccess)
        e = configure_smem(linear_chunked_kernel<DK, DV, false>, (int)Lc<DK, DV>::kSmem, configured[0]);
    if (e != cudaSuccess)
        return e;
    const long long heads = (long long)a.B * a.H;
    if (p.nseg > 1) {
        e = configure_smem(linear_chunked_kernel<DK, DV, true>, (int)Lc<DK, DV>::kSmem, configured[1]);
        if (e != cudaSuccess)
            return e;
        linear_chunked_kernel<DK, DV, true>
            <<<(unsigned)(heads * (p.nseg - 1)), kLcThreads, Lc<DK, DV>::kSmem, s>>>(q, k, v, p);
        const long long per = ((long long)a.Dk * a.Dv + 255) / 256;
        linear_carry_kernel<<<(unsigned)(heads * per), 256, 0, s>>>(p);
    }
    linear_chunked_kernel<DK, DV, false><<<(unsigned)(heads * p.nseg), kLcThreads, Lc<DK, DV>::kSmem, s>>>(q, k, v, p);
    return cudaGetLastError();
}

// Segments of a sequence: as many as fill the GPU once, of at least four chunks each.
void lc_plan(const LinAttnArgs &a, int *nseg, int *seg_chunks)
{
    const long long heads = (long long)a.B * a.H;
    const int chunks = (a.L + kLcChunk - 1) / kLcChunk;
    long long n = kLcSms / heads;
    n = n < 1 ? 1 : n > chunks / 4 ? (chunks / 4 > 0 ? chunks / 4 : 1) : n;
    *seg_chunks = (int)((chunks + n - 1) / n);
    *nseg = (chunks + *seg_chunks - 1) / *seg_chunks;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t linear_chunked_workspace(const LinAttnArgs &a)
{
    int nseg, seg_chunks;
    lc_plan(a, &nseg, &seg_chunks);
    if (nseg == 1)
        return 0;
    const size_t heads = (size_t)a.B * a.H;
    return round256(heads * nseg * 4) + heads * nseg * a.Dk * a.Dv * 4;
}

cudaError_t launch_linear_chunked(const LinAttnArgs &a, void *workspace, cudaStream_t s)
{
    ChunkedArgs p{};
    p.a = a;
    lc_plan(a, &p.nseg, &p.seg_chunks);
    const long long heads = (long long)a.B * a.H;
    if (heads * p.nseg > 0x7fffffffLL || heads * 64 > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    if (p.nseg > 1) {
        p.decays = static_cast<float *>(workspace);
        p.states = reinterpret_cast<float *>(static_cast<char *>(workspace) + round256((size_t)heads * p.nseg * 4));
    }
    if (a.Dk <= 64)
        return a.Dv <= 64 ? launch_dims<64, 64>(p, s) : launch_dims<64, 128>(p, s);
    return a.Dv <= 64 ? launch_dims<128, 64>(p, s) : launch_dims<128, 128>(p, s);
}

}  // namespace ss2d
