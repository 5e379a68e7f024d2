// linear_chunked.cu -- linear attention over whole sequences, in chunks of 128 tokens, on the tensor
// cores (ss2d_linear_attention).
//
// With c_i the sum of the log decays of tokens 0 .. i of a chunk, S the state before the chunk:
//
//   o_i = scale * sum_{j <= i} exp(c_i - c_j) (q_i . k_j) v_j  +  scale * exp(c_i) S^T q_i
//   S'  = exp(c_last) S + sum_j exp(c_last - c_j) k_j v_j^T
//
// so a chunk is four products of 128 tokens:  Q K^T,  P V with P the masked and decayed scores,
// Q S, and K^T (w V) with w_j = exp(c_last - c_j).  A CTA walks the chunks of DV columns of one
// head's state (the columns of v, o and S do not meet) over one sequence or one segment of it.  Only
// S' = exp(c_last) S + ... is a chain from chunk to chunk, so every step has warps of its own and
// works on the chunk that is ready for it:
//   copy warp    TMA: Q, K and V tiles, each in a ring of slots
//   MMA warps    one thread of one issues the MMAs of the scores and of P V, one thread of the other
//                those of the state and of Q S
//   decay warp   sums of log decays, and from them every factor that the others need
//   weight warps V -> w V in three bf16 parts, in shared memory
//   score warps  scores -> P (bf16, in place in tensor memory: the A operand of P V)
//   state warps  the state, in registers, and its bf16 copy in shared memory for the next Q S
//   output warps P V and Q S -> o
//
// Roundings to bf16, all for an MMA's operands: P and the copy of S once (what they enter, o, is
// itself rounded to bf16); w V in three parts that together keep 24 bits, because the state is an
// fp32 result and is summed over the whole sequence.  Sums, states and decays are fp32 or wider.
//
// The decays within a chunk: columns are cut in blocks of 32, m_b = c at the end of block b.  A score
// below the diagonal blocks takes exp(c_i - m_b) exp(m_b - c_j), a product of a row's and a column's
// factor, both at most 1; only the diagonal blocks need an exponential for each element.
//
// Where the heads of all sequences are too few for the GPU, a sequence is cut into segments: a first
// pass sums each segment's own state (K and V only), a small kernel adds them up along the sequence, each decayed by
// what lies between, and the pass above starts each segment from the state before it.  The first segment needs no first
// pass: it goes beside the others' ones, in the same launch.
//
// What bounds it: a chunk of 128 x 64 columns takes about 4000 cycles.  Shared memory passes 3200 cycles' worth of bytes
// in them (tiles in, w V out, and the MMAs' operands: 64 columns read all of Q and K, and a product for each part of w V
// reads K three times), the warps issue 0.55 instructions a cycle and scheduler, the tensor cores are busy 42 %, and
// hand-overs between the warps (load, scores, P, P V, output; K^T w V, state, Q S) fill the rest.  32768 tokens of 16
// heads of 128 x 128: 217 to 280 us by what the power limit leaves of the clock, of which the first pass is a third
// (floor 82 us, bytes); 32 x 3136 tokens of 6 heads of 64 x 32: 61 to 67 us (floor 16).
#include "api_internal.h"
#include "launch_util.h"
#include "linear_attention.h"
#include "tma.cuh"
#include "wait_status.cuh"

namespace ss2d {
namespace {

constexpr int kLcChunk = 128;
constexpr int kLcThreads = 1024;      // copy warp, MMA warp, decay warp, the state's MMA warp, then the groups:
constexpr int kLcWeight = 4, kLcScore = 12, kLcState = 20, kLcOutput = 28;  // their first warps (8, 8, 8 and 4)
constexpr uint32_t kLcBlock = kLcChunk * 128;  // bytes of 128 tokens by 64 columns of bf16
constexpr int kLcParts = 3;           // of w V
constexpr int kLcAhead = 3;           // chunks that a tile is asked for in L2 before its load
constexpr int kLcIdlePolls = 1 << 24;  // of the copy warp and of a second piece, at 120 ns or more: about 2 s
constexpr int kLcStateWarps = 8;
constexpr int kLcSms = 148;  // of a B200; the plan, and the workspace with it, follow from the sizes alone, without a device
constexpr int kLcMaxSegments = 149;  // one CTA for each SM in either pass

constexpr float kLcLog2e = 1.4426950408889634f, kLcLn2 = 0.6931471805599453f;

// Factors of one chunk's decays; logarithms to base 2.
struct alignas(16) ChunkDecay {
    float cb[kLcChunk];  // c_j - m_b of j's block
    float f[kLcChunk];   // exp(m_b - c_j)
    float m[4];          // m_b
    float dm[4][4];      // m_q - m_b
    float e[4];          // exp(c_last - m_b)
    float keep, grow;    // exp(c_last) = keep + grow: 1 and a small number for slow decays, else 0 and itself
};

struct ChunkedArgs {
    LinAttnArgs a;
    // For every segment but the last: (B * H, nseg - 1, Dk, Dv) its own state, then that of the sequence behind it, and
    // (B * H, nseg - 1) its decay, or, with the sign set, a slow one less 1
    float *states, *decays;
    int nseg, first_chunks, seg_chunks;  // chunks of the first segment, and of the others
    int units;                           // of one segment: a CTA's columns of one head of one sequence
    // Cut units: the last `cut` ones are in two pieces, the first of which leaves its state in `states`.  CTAs take the
    // first pieces, the whole units, then the second pieces, by tickets: a CTA that has a second piece knows that a CTA
    // which runs, or has run, has the first.
    int cut, cut_chunks;
    int *tickets;        // those taken; then, of each cut unit, the warps that have stored the first piece's state
};

// STATES: the first pass over segments, which has the state's products alone in tensor memory.
template <int DK, int DV, bool STATES = false>
struct Lc {
    static constexpr int kSlots = DK == 64 ? 3 : 2;      // of the rings of tiles: chunks in flight
    static constexpr int kDecays = DK == 64 ? 4 : 2;     // of the ring of decays
    static constexpr uint32_t kQK = DK / 64 * kLcBlock;  // bytes of a tile of Q or K
    static constexpr uint32_t kW = (kLcParts * DV + 63) / 64 * kLcBlock;  // the parts of w V, next to one another
    static constexpr uint32_t kS = DK * 128;             // the bf16 state: DK rows of up to 64 columns
    static constexpr uint32_t kQAt = 0, kKAt = kQAt + kSlots * kQK, kVAt = kKAt + kSlots * kQK,
                              kWAt = kVAt + kSlots * kLcBlock, kSAt = kWAt + kW, kDecayAt = kSAt + kS,
                              kBarsAt = kDecayAt + kDecays * (uint32_t)sizeof(ChunkDecay);
    // Columns of tensor memory: scores (two buffers; P in place), P V, Q S, and K^T (w V), in as many buffers as
    // there is room for.  Of w V, all three parts in blocks of their own where they fit (one product), else the
    // first two, and the third is added to the second's (a product for each).
    static constexpr uint32_t kScoresAt = 0, kOutAt = 256, kInterAt = kOutAt + DV, kDeltaAt = STATES ? 0 : kInterAt + DV;
    static constexpr int kBlocks = kDeltaAt + kLcParts * DV <= 512 ? kLcParts : kLcParts - 1;
    static constexpr int kDelta = kBlocks * DV, kDeltas = (int)kDeltaAt + 2 * kDelta <= 512 ? 2 : 1;
    static_assert(kDeltaAt + kDeltas * kDelta <= 512, "tensor memory");
    // mbarriers: rings of kSlots, kDecays and kDeltas, then pairs, then single ones
    static constexpr int kQFull = 0, kKFull = kQFull + kSlots, kVFull = kKFull + kSlots, kQFree = kVFull + kSlots,
                         kKFree = kQFree + kSlots, kVFree = kKFree + kSlots, kDecFull = kVFree + kSlots,
                         kDecFree = kDecFull + kDecays, kDeltaDone = kDecFree + kDecays, kDeltaFree = kDeltaDone + kDeltas,
                         kScoresDone = kDeltaFree + kDeltas, kProbsReady = kScoresDone + 2, kWeightsReady = kProbsReady + 2,
                         kWeightsFree = kWeightsReady + 2, kStateReady = kWeightsFree + 2, kInterDone = kStateReady + 1,
                         kInterFree = kInterDone + 1, kOutDone = kInterFree + 1, kOutFree = kOutDone + 1,
                         kVChecked = kOutFree + 1, kBars = kVChecked + kSlots;
    // then the place of tensor memory, and marks of chunks whose V is not finite.  A slot of V is taken after
    // its last chunk's P V, which comes after the output of the chunk before that one.
    static constexpr int kMarks = kSlots + 1;
    static constexpr size_t kSmem = kBarsAt + kBars * 8 + 8 + kMarks * 4;
    static_assert(kSmem <= 232448, "shared memory of an SM");
};

// A chunk's place in a ring of N slots, and the parity of its round; no division as the chunks go by.
template <int N>
struct LcRing {
    uint32_t slot = 0, round = 0;
    __device__ __forceinline__ void operator++()
    {
        if (N == 1 || ++slot == N) {
            slot = 0;
            round ^= 1u;
        }
    }
};

// kind::f16, fp32 accumulate, bf16 operands, 128 rows
__host__ __device__ constexpr uint32_t lc_idesc(int n, bool a_mn_major, bool b_mn_major)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn_major ? 1u << 15 : 0u) | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
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

// What a warp's lanes wrote to global memory before the __syncwarp ahead of the one's lc_release_add is seen by those that
// read it behind the __syncwarp that follows the other's lc_acquire.
__device__ __forceinline__ void lc_release_add(int *p)
{
    asm volatile("red.release.gpu.global.add.s32 [%0], 1;\n" ::"l"(p) : "memory");
}

__device__ __forceinline__ int lc_acquire(const int *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// What a CTA does: all of it; the first pass over segments, which sums their own states alone; all of it with cut
// units; or all of it with the longest sequences first.  The last two are kernels of their own because the few values
// more that they hold cost the others 3 % of their time (registers).
enum { kLcAll, kLcStates, kLcCut, kLcSorted };

// `index`: the CTA's place among those of segments seg_from .. seg_from + segs - 1.
template <int DK, int DV, int PASS>
__device__ __forceinline__ void linear_chunked(const CUtensorMap &map_q, const CUtensorMap &map_k, const CUtensorMap &map_v,
                                               const ChunkedArgs &p, int index, int seg_from, int segs)
{
    constexpr bool STATES = PASS == kLcStates, CUT = PASS == kLcCut;
    using C = Lc<DK, DV, STATES>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const LinAttnArgs &a = p.a;
    const uint32_t base = tc::smem_u32(smem);
    ChunkDecay *const decay = reinterpret_cast<ChunkDecay *>(smem + C::kDecayAt);
    auto bar = [&](int which) { return base + C::kBarsAt + 8 * (uint32_t)which; };
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kBarsAt + C::kBars * 8);
    int *const marks = reinterpret_cast<int *>(tmem_slot + 2);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;

    const int slices = (a.Dv + DV - 1) / DV;
    grid_wait();
    int place = index;
    if (CUT) {
        int *const ticket = reinterpret_cast<int *>(tmem_slot + 1);
        if (threadIdx.x == 0)
            *ticket = atomicAdd(p.tickets, 1);
        __syncthreads();
        place = *ticket;
    }
    const int units = p.units;
    const bool piece0 = CUT && place < p.cut, piece1 = CUT && place >= units;
    const int unit = !CUT ? place : piece0 ? units - p.cut + place : place - p.cut;  // with cut units: one segment
    const int slice = unit % slices;
    const int seg = seg_from + unit / slices % segs;
    long long bh = unit / slices / segs;
    const int h = (int)(bh % a.H);
    int b = (int)(bh / a.H);
    const int group = h / (a.H / a.G);
    const int c0 = slice * DV;              // this CTA's columns of v, o and S
    const int cols = min(DV, a.Dv - c0);    // a multiple of 8
    if (PASS == kLcSorted) {
        // the sequence that b other ones go before
        const int mine = lane < a.B ? min(max(a.lengths[lane], 0), a.L) : -1;
        int before = 0;
        for (int x = 0; x < a.B; ++x) {
            const int other = __shfl_sync(0xffffffffu, mine, x);
            before += other > mine || (other == mine && x < lane);
        }
        b = __ffs(__ballot_sync(0xffffffffu, before == b)) - 1;
        bh = (long long)b * a.H + h;
    }
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;
    const int t_first = (piece1 ? p.cut_chunks : seg == 0 ? 0 : p.first_chunks + (seg - 1) * p.seg_chunks) * kLcChunk;
    const int t_end = min(len, t_first + (piece0 ? p.cut_chunks : seg == 0 ? p.first_chunks : p.seg_chunks) * kLcChunk);
    if (!STATES && seg_from == 0 && place == 0 && threadIdx.x == 0)
        *a.err = 0;  // the call's first kernel, long before any wait of it can run out
    if (t_first >= len && !(len == 0 && seg == 0 && !piece1))
        return;
    const int chunks = (t_end - t_first + kLcChunk - 1) / kLcChunk;  // 0 for an empty sequence: its state is kept

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            tc::mbar_init(bar(C::kQFull + i), 1);
            tc::mbar_init(bar(C::kKFull + i), 1);
            tc::mbar_init(bar(C::kVFull + i), 1);
            tc::mbar_init(bar(C::kQFree + i), 2);               // the scores and Q S
            tc::mbar_init(bar(C::kKFree + i), STATES ? 1 : 2);  // the scores and the state
            tc::mbar_init(bar(C::kVFree + i), STATES ? 16 : 9);  // the weight warps and P V
            tc::mbar_init(bar(C::kVChecked + i), 8);
        }
        for (int i = 0; i < C::kMarks; ++i)
            marks[i] = 0;
        for (int i = 0; i < C::kDecays; ++i) {
            tc::mbar_init(bar(C::kDecFull + i), 1);
            tc::mbar_init(bar(C::kDecFree + i), STATES ? 24 : 28);  // every warp of the groups
        }
        for (int i = 0; i < C::kDeltas; ++i) {
            tc::mbar_init(bar(C::kDeltaDone + i), 1);
            tc::mbar_init(bar(C::kDeltaFree + i), 8);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar(C::kScoresDone + i), 1);
            tc::mbar_init(bar(C::kProbsReady + i), 8);
            tc::mbar_init(bar(C::kWeightsReady + i), 8);
            tc::mbar_init(bar(C::kWeightsFree + i), 1);
        }
        tc::mbar_init(bar(C::kStateReady), 8);
        tc::mbar_init(bar(C::kInterDone), 1);
        tc::mbar_init(bar(C::kInterFree), 4);
        tc::mbar_init(bar(C::kOutDone), 1);
        tc::mbar_init(bar(C::kOutFree), 4);
        tc::mbar_init_fence();
    }
    if (warp == 1)
        tc::tmem_alloc(tmem_slot, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    grid_next();
    const uint32_t tmem = *tmem_slot;
    bool good = true;
    // a warp of a group: waits together
    auto wait = [&](int which, uint32_t parity) {
        good = tc::mbar_wait_warp(bar(which), parity);
        tc::fence_after();
        return good;
    };
    // the same, without waiting
    auto ready = [&](int which, uint32_t parity) {
        const bool yes = tc::mbar_test_warp(bar(which), parity);
        tc::fence_after();
        return yes;
    };
    auto arrive = [&](int which) {
        if (lane == 0)
            tc::mbar_arrive(bar(which));
    };
    const int quarter = warp % 4;                // of the 128 lanes of tensor memory
    const uint32_t lanes = tmem + ((uint32_t)quarter << 21);
    const int row = quarter * 32 + lane;

    if (warp == 0) {
        if (lane == 0) {
            // A slot of V is free again when its P V is done, one of K after the state's product, one of Q after Q S:
            // whichever is free next is filled next.
            const CUtensorMap *const maps[3] = {&map_k, &map_v, &map_q};
            int next[3] = {0, 0, STATES ? chunks : 0};
            for (int polls = 0; min(min(next[0], next[1]), next[2]) < chunks;) {
                bool idle = true;
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    const int c = next[x], i = c % C::kSlots;
                    const int free = x == 0 ? C::kKFree : x == 1 ? C::kVFree : C::kQFree;
                    const int full = x == 0 ? C::kKFull : x == 1 ? C::kVFull : C::kQFull;
                    if (c >= chunks || !tc::mbar_test(bar(free + i), ((c / C::kSlots) & 1) ^ 1u))
                        continue;
                    const uint32_t bytes = x == 1 ? kLcBlock : C::kQK;
                    const uint32_t at = base + (x == 0 ? C::kKAt : x == 1 ? C::kVAt : C::kQAt) + i * bytes;
                    tc::mbar_expect(bar(full + i), bytes);
#pragma unroll
                    for (int y = 0; y < (x == 1 ? 1 : DK / 64); ++y)
                        tc::tma_load_4d(at + y * kLcBlock, maps[x], bar(full + i), (x == 1 ? c0 : 0) + 64 * y,
                                        x == 1 ? h : group, t_first + c * kLcChunk, b);
                    // a slot fills from L2 in half the time that it takes from device memory
                    if (c + kLcAhead < chunks && (x == 1 || slice == 0))
#pragma unroll
                        for (int y = 0; y < (x == 1 ? 1 : DK / 64); ++y)
                            tc::tma_prefetch_4d(maps[x], (x == 1 ? c0 : 0) + 64 * y, x == 1 ? h : group,
                                                t_first + (c + kLcAhead) * kLcChunk, b);
                    next[x] = c + 1;
                    idle = false;
                }
                polls = idle ? polls + 1 : 0;
                if (polls > kLcIdlePolls) {
                    good = false;
                    break;
                }
                if (idle)
                    __nanosleep(64);
            }
            // copies must have landed before the CTA's shared memory goes
#pragma unroll
            for (int x = 0; x < (STATES ? 2 : 3); ++x)
                for (int c = max(0, next[x] - C::kSlots); c < next[x]; ++c)
                    tc::mbar_wait(bar((x == 0 ? C::kKFull : x == 1 ? C::kVFull : C::kQFull) + c % C::kSlots),
                                  (c / C::kSlots) & 1);
        }
    } else if (warp == 1 && !STATES) {
        // descriptors of the first slot's tiles; an address enters them in units of 16 bytes
        const uint64_t q_k = tc::swizzled_desc(base + C::kQAt, 16, 1024);         // K-major
        const uint64_t k_k = tc::swizzled_desc(base + C::kKAt, 16, 1024);
        const uint64_t v_mn = tc::swizzled_desc(base + C::kVAt, kLcBlock, 1024);  // MN-major
        LcRing<C::kSlots> tiles, ahead_of;  // of P V, and of the scores
        auto scores = [&](int c) {
            // (the buffer is free: the P V of two chunks before, which reads P in its place, is done)
            const uint32_t i = ahead_of.slot, round = ahead_of.round, two = c & 1;
            ++ahead_of;
            if (!wait(C::kKFull + i, round) || !wait(C::kQFull + i, round))
                return;
            const uint64_t q = q_k + i * (C::kQK / 16), k = k_k + i * (C::kQK / 16);
            if (tc::elect_one()) {
#pragma unroll
                for (int j = 0; j < DK / 16; ++j) {
                    const uint32_t off = (j / 4 * kLcBlock + j % 4 * 32) / 16;
                    tc::mma_bf16(tmem + C::kScoresAt + two * 128, q + off, k + off, lc_idesc(128, false, false), j > 0);
                }
                tc::commit(bar(C::kScoresDone + two));
                tc::commit(bar(C::kQFree + i));
                tc::commit(bar(C::kKFree + i));
            }
            __syncwarp();
        };
        if (chunks > 0)
            scores(0);
        for (int c = 0; c < chunks && good; ++c, ++tiles) {
            const uint32_t i = tiles.slot, round = tiles.round, two = c & 1, turn = (c >> 1) & 1;
            // the next chunk's scores first, unless its tiles are still on their way
            const int next = c + 1;
            const bool ahead = next < chunks && ready(C::kKFull + ahead_of.slot, ahead_of.round) &&
                               ready(C::kQFull + ahead_of.slot, ahead_of.round);
            // their buffer holds the P of the chunk before this one until its P V is done
            if (ahead) {
                if (!wait(C::kOutDone, two ^ 1u))
                    break;
                scores(next);
            }
            // P V; P of 16 tokens lies in the first 8 of their 16 columns of the scores
            if (!wait(C::kVFull + i, round) || !wait(C::kVChecked + i, round) || !wait(C::kProbsReady + two, turn) ||
                !wait(C::kOutFree, two ^ 1u))
                break;
            const uint64_t v = v_mn + i * (kLcBlock / 16);
            if (tc::elect_one()) {
#pragma unroll
                for (int j = 0; j < kLcChunk / 16; ++j)
                    tc::mma_bf16_ta(tmem + C::kOutAt, tmem + C::kScoresAt + two * 128 + j * 16, v + j * (2048 / 16),
                                    lc_idesc(DV, false, true), j > 0);
                tc::commit(bar(C::kOutDone));
                tc::commit(bar(C::kVFree + i));
            }
            __syncwarp();
            if (!ahead && next < chunks)
                scores(next);  // (kOutFree meant that the P V before this one was done)
        }
    } else if (warp == 3) {
        const uint64_t q_k = tc::swizzled_desc(base + C::kQAt, 16, 1024);         // K-major
        const uint64_t k_mn = tc::swizzled_desc(base + C::kKAt, kLcBlock, 1024);  // MN-major
        const uint64_t w_mn = tc::swizzled_desc(base + C::kWAt, kLcBlock, 1024);
        const uint64_t s_mn = tc::swizzled_desc(base + C::kSAt, kLcBlock, 1024);
        constexpr uint32_t kStep = 2048 / 16;  // 16 tokens (or rows of S) of an MN-major tile
        LcRing<C::kSlots> tiles;
        LcRing<C::kDeltas> deltas;
        for (int c = 0; c < chunks && good; ++c, ++tiles, ++deltas) {
            const uint32_t i = tiles.slot, turn = c & 1, buf = deltas.slot;
            // K^T (w V): lanes are rows of S.  With DK = 64 the upper 64 lanes read what lies behind the tile and give
            // rows that nobody reads.
            if (!wait(C::kKFull + i, tiles.round) || !wait(C::kDeltaFree + buf, deltas.round ^ 1u))
                break;
            const uint64_t kt = k_mn + i * (C::kQK / 16);
            const uint32_t to = tmem + C::kDeltaAt + buf * C::kDelta;
            for (int half = 0; half < 2 && wait(C::kWeightsReady + half, turn); ++half) {
                if (tc::elect_one()) {
#pragma unroll
                    for (int x = 0; x < kLcChunk / 32; ++x) {
                        const uint32_t j = half * 4 + x;
                        if (C::kBlocks == kLcParts) {
                            tc::mma_bf16(to, kt + j * kStep, w_mn + j * kStep, lc_idesc(C::kDelta, true, true), half > 0 || x > 0);
                            continue;
                        }
                        // A product for each part: MMAs are ordered where their accumulators and shapes are the same, so
                        // what the third adds to the second's columns has the second's shape.
#pragma unroll
                        for (int z = 0; z < kLcParts; ++z) {
                            const int block = min(z, C::kBlocks - 1);
                            tc::mma_bf16(to + block * DV, kt + j * kStep, w_mn + z * DV / 64 * (kLcBlock / 16) + j * kStep,
                                         lc_idesc(DV, true, true), half > 0 || x > 0 || z > block);
                        }
                    }
                    tc::commit(bar(C::kWeightsFree + half));
                    if (half) {
                        tc::commit(bar(C::kDeltaDone + buf));
                        tc::commit(bar(C::kKFree + i));
                    }
                }
                __syncwarp();
            }
            if (!good)
                break;
            if (STATES)
                continue;
            // Q S
            if (!wait(C::kQFull + i, tiles.round) || !wait(C::kStateReady, turn) || !wait(C::kInterFree, turn ^ 1u))
                break;
            const uint64_t q = q_k + i * (C::kQK / 16);
            if (tc::elect_one()) {
#pragma unroll
                for (int j = 0; j < DK / 16; ++j)
                    tc::mma_bf16(tmem + C::kInterAt, q + (j / 4 * kLcBlock + j % 4 * 32) / 16, s_mn + j * kStep,
                                 lc_idesc(DV, false, true), j > 0);
                tc::commit(bar(C::kInterDone));
                tc::commit(bar(C::kQFree + i));
            }
            __syncwarp();
        }
    } else if (warp == 2) {
        // Four tokens of each lane, eight lanes of each block.
        const float fixed = a.per_token ? 0.0f : a.log_decay[h];
        const float *gates = a.log_decay + (a.per_token ? ((long long)b * a.L) * a.H + h : 0);
        float g[4];  // of the next chunk, on their way while this one's are summed
        auto fetch = [&](int c) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = t_first + c * kLcChunk + lane * 4 + j;
                g[j] = t >= t_end ? 0.0f : a.per_token ? gates[(long long)t * a.H] : fixed;
            }
        };
        double whole = 0.0;
        if (chunks > 0)
            fetch(0);
        LcRing<C::kDecays> dec;
        for (int c = 0; c < chunks; ++c, ++dec) {
            // A NaN enters no sum, or it would reach the tokens before it: cb is one from its token on, and the weights and
            // rows that follow from cb carry it to the outputs and the state.
            int nan_at = 4;
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                if (g[j] != g[j])
                    nan_at = j;
                g[j] = fmaxf(g[j], kLaMinLogDecay);
            }
            const unsigned bad = __ballot_sync(0xffffffffu, nan_at < 4);
            // cb_j, the sum from a block's end back to j, added from the end: where a weight exp(-cb) counts, cb is
            // small, and so is its rounding.  The same for the blocks within the chunk.
            float after[4];  // of the lane's tokens: the lane's later ones
            after[3] = 0.0f;
#pragma unroll
            for (int j = 2; j >= 0; --j)
                after[j] = after[j + 1] + g[j + 1] * kLcLog2e;
            const float own = after[0] + g[0] * kLcLog2e;
            if (c + 1 < chunks)
                fetch(c + 1);
            float sum = own;  // of this lane and the block's later ones
#pragma unroll
            for (int d = 1; d < 8; d *= 2) {
                const float v = __shfl_down_sync(0xffffffffu, sum, d, 8);
                if (lane % 8 + d < 8)
                    sum += v;
            }
            float later = __shfl_down_sync(0xffffffffu, sum, 1, 8);
            if (lane % 8 == 7)
                later = 0.0f;
            float blocks[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                blocks[q] = __shfl_sync(0xffffffffu, sum, 8 * q);
            if (!wait(C::kDecFree + dec.slot, dec.round ^ 1u))
                break;
            ChunkDecay &out = decay[dec.slot];
            float cb[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                cb[j] = -(later + after[j]);
            if (bad) {
                const int first = __ffs(bad) - 1;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (lane > first || (lane == first && j >= nan_at))
                        cb[j] = __int_as_float(0x7fffffff);
            }
            *reinterpret_cast<float4 *>(&out.cb[lane * 4]) = make_float4(cb[0], cb[1], cb[2], cb[3]);
            *reinterpret_cast<float4 *>(&out.f[lane * 4]) =
                make_float4(exp2f(-cb[0]), exp2f(-cb[1]), exp2f(-cb[2]), exp2f(-cb[3]));
            const float all = ((blocks[3] + blocks[2]) + blocks[1]) + blocks[0];
            if (lane < 4) {
                float to_end = 0.0f, to_here = 0.0f;
#pragma unroll
                for (int q = 3; q >= 0; --q)
                    to_end += q > lane ? blocks[q] : 0.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    to_here += q <= lane ? blocks[q] : 0.0f;
                out.m[lane] = to_here;
                out.e[lane] = exp2f(to_end);
                float between = 0.0f;  // of blocks lane + 1 .. q
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    between += q > lane ? blocks[q] : 0.0f;
                    out.dm[q][lane] = between;
                }
                if (lane == 0) {
                    const bool slow = all > -0.5f;
                    out.keep = slow ? 1.0f : 0.0f;
                    out.grow = slow ? expm1f(all * kLcLn2) : exp2f(all);
                }
            }
            whole += all;
            __syncwarp();
            arrive(C::kDecFull + dec.slot);
        }
        if (STATES && lane == 0 && good)
            p.decays[bh * (p.nseg - 1) + seg] =
                whole > -0.5 ? copysignf(expm1f((float)(whole * (double)kLcLn2)), -1.0f) : exp2f((float)whole);
    } else if (warp >= kLcWeight && warp < (STATES ? kLcState : kLcScore)) {
        // V -> w V, 16 bytes at a time.  A part is the upper 16 bits of what the
        // parts before it leave, so the subtractions are exact and three parts hold all 24 bits.
        // In the first pass the score warps, which have nothing to do there, take the second half of the tokens.
        const int t = (threadIdx.x - kLcWeight * 32) % 256;
        constexpr int kHalves = STATES ? 1 : 2;
        const int first = STATES ? (warp - kLcWeight) / 8 : 0;
        LcRing<C::kSlots> tiles;
        LcRing<C::kDecays> dec;
        LcRing<C::kMarks> mark;
        for (int c = 0; c < chunks && good; ++c, ++tiles, ++dec, ++mark) {
            const uint32_t i = tiles.slot, round = tiles.round, turn = c & 1;
            const int n = min(kLcChunk, t_end - t_first - c * kLcChunk);
            const ChunkDecay &d = decay[dec.slot];
            unsigned char *const tileV = smem + C::kVAt + i * kLcBlock;
            unsigned char *const tileW = smem + C::kWAt;
            if (!wait(C::kVFull + i, round) || (n < kLcChunk && !wait(C::kKFull + i, round)))
                break;
            constexpr int kPieces = DV / 8, kEach = kPieces / 4;  // of a token, and of a thread's half
            const int piece = t % kPieces;
            uint4 v[kHalves][kEach];
            __nv_bfloat162 odd = __floats2bfloat162_rn(0.0f, 0.0f);  // 0, or a NaN where an element is not finite
#pragma unroll
            for (int x = 0; x < kHalves * kEach; ++x) {
                const int token = first * 64 + (x * 256 + t) / kPieces;
                uint4 &in = v[x / kEach][x % kEach];
                in = *reinterpret_cast<const uint4 *>(tileV + token * 128 + ((piece ^ (token & 7)) << 4));
                // a token behind the last: zero, whatever V holds there
                if (token >= n)
                    in = make_uint4(0, 0, 0, 0);
                if (!STATES)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        odd = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&(&in.x)[y]), __floats2bfloat162_rn(0.0f, 0.0f), odd);
            }
            // A factor of zero does not hide an infinity or a NaN.  So rows of K and V behind the last token are zero,
            // whatever the tensors hold there (other warps, and the MMAs of the scores, may still read these rows as
            // they were: nothing of that reaches a row of the output or the state), and P V takes zero for such an element,
            // which the outputs of the tokens before must not see; the output warps put a NaN in the others.
            const bool found = !STATES && (__isnan(__low2float(odd)) || __isnan(__high2float(odd)));
            if (found) {
                marks[mark.slot] = c + 1;
#pragma unroll 1
                for (int x = 0; x < 2 * kEach * 8; ++x) {
                    const int token = (x / 8 * 256 + t) / kPieces;
                    unsigned short *const e = reinterpret_cast<unsigned short *>(
                        tileV + token * 128 + ((piece ^ (token & 7)) << 4) + x % 8 * 2);
                    if ((*e & 0x7f80) == 0x7f80)
                        *e = 0;
                }
            }
            if (n < kLcChunk)
                for (int blk = 0; blk < (STATES ? 0 : 1) + DK / 64; ++blk) {
                    unsigned char *const tile = blk < DK / 64 ? smem + C::kKAt + i * C::kQK + blk * kLcBlock : tileV;
                    for (int x = max(n, first * 64) * 8 + t; x < (first + kHalves) * 64 * 8; x += 256)
                        *reinterpret_cast<uint4 *>(tile + x * 16) = make_uint4(0, 0, 0, 0);
                }
            if (!STATES) {
                if (found || n < kLcChunk)
                    tc::fence_async_proxy();
                __syncwarp();
                arrive(C::kVChecked + i);
            }
            if (!wait(C::kDecFull + dec.slot, dec.round))
                break;
#pragma unroll
            for (int y = 0; y < kHalves; ++y) {
                const int half = first + y;
                float w[kEach];
#pragma unroll
                for (int x = 0; x < kEach; ++x) {
                    const int token = half * 64 + (x * 256 + t) / kPieces;
                    w[x] = d.f[token] * d.e[token / 32];
                }
                if (!wait(C::kWeightsFree + half, turn ^ 1u))
                    break;
#pragma unroll
                for (int x = 0; x < kEach; ++x) {
                    const int token = half * 64 + (x * 256 + t) / kPieces;
                    const uint32_t in[4] = {v[y][x].x, v[y][x].y, v[y][x].z, v[y][x].w};
                    uint32_t part[kLcParts][4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        float2 r = __fmul2_rn(make_float2(__uint_as_float(in[u] << 16), __uint_as_float(in[u] & 0xffff0000u)),
                                              make_float2(w[x], w[x]));
#pragma unroll
                        for (int z = 0; z < kLcParts; ++z) {
                            const uint32_t lo = __float_as_uint(r.x), hi = __float_as_uint(r.y);
                            part[z][u] = __byte_perm(lo, hi, 0x7632);
                            r = __fadd2_rn(r, make_float2(__uint_as_float((lo & 0xffff0000u) ^ 0x80000000u),
                                                          __uint_as_float((hi & 0xffff0000u) ^ 0x80000000u)));
                        }
                    }
#pragma unroll
                    for (int z = 0; z < kLcParts; ++z) {
                        const int col = z * kPieces + piece;  // in pieces, eight to a block
                        *reinterpret_cast<uint4 *>(tileW + col / 8 * kLcBlock + token * 128 + ((col % 8 ^ (token & 7)) << 4)) =
                            make_uint4(part[z][0], part[z][1], part[z][2], part[z][3]);
                    }
                }
                tc::fence_async_proxy();
                __syncwarp();
                arrive(C::kWeightsReady + half);
            }
            arrive(C::kVFree + i);
            arrive(C::kDecFree + dec.slot);
        }
    } else if (warp >= kLcScore && warp < kLcState && !STATES) {
        const int half = (warp - kLcScore) / 4;  // 16 of a block's 32 columns
        LcRing<C::kDecays> dec;
        for (int c = 0; c < chunks; ++c, ++dec) {
            const uint32_t two = c & 1, turn2 = (c >> 1) & 1;  // of the scores' two buffers
            const ChunkDecay &d = decay[dec.slot];
            if (!wait(C::kDecFull + dec.slot, dec.round) || !wait(C::kScoresDone + two, turn2))
                break;
            const float cb = d.cb[row];
            const uint32_t at = lanes + C::kScoresAt + two * 128 + half * 16;
            auto factors = [&](const float *from, float2 (&f)[8]) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float4 v = reinterpret_cast<const float4 *>(from + half * 16)[y];
                    f[2 * y] = make_float2(v.x, v.y), f[2 * y + 1] = make_float2(v.z, v.w);
                }
            };
            auto probs = [&](uint32_t (&v)[16], const float2 (&f)[8], uint32_t (&w)[8]) {
                tc::tmem_wait16(v);
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const float2 r = __fmul2_rn(f[y], make_float2(__uint_as_float(v[2 * y]), __uint_as_float(v[2 * y + 1])));
                    w[y] = lc_pack(r.x, r.y);
                }
            };
            uint32_t v[16], w[8];
            float2 f[8];
#pragma unroll 1
            for (int blk = 0; blk < quarter; ++blk) {
                tc::tmem_ld16(at + blk * 32, v);
                const float r = a.scale * lc_ex2(cb + d.dm[quarter][blk]);
                factors(d.f + blk * 32, f);
#pragma unroll
                for (int y = 0; y < 8; ++y)
                    f[y] = __fmul2_rn(f[y], make_float2(r, r));
                probs(v, f, w);
                tc::tmem_st8(at + blk * 32, w);
            }
            tc::tmem_ld16(at + quarter * 32, v);
            factors(d.cb + quarter * 32, f);
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const float2 e = __fadd2_rn(make_float2(cb, cb), make_float2(-f[y].x, -f[y].y));
                f[y] = __fmul2_rn(make_float2(a.scale, a.scale), make_float2(lc_ex2(e.x), lc_ex2(e.y)));
            }
            probs(v, f, w);
            // columns behind the row's own token: none
            const int last = lane - half * 16;
#pragma unroll
            for (int y = 0; y < 8; ++y)
                w[y] &= (2 * y <= last ? 0xffffu : 0u) | (2 * y + 1 <= last ? 0xffff0000u : 0u);
            tc::tmem_st8(at + quarter * 32, w);
#pragma unroll
            for (int y = 0; y < 8; ++y)
                w[y] = 0;
#pragma unroll 1
            for (int blk = quarter + 1; blk < 4; ++blk)
                tc::tmem_st8(at + blk * 32, w);
            tc::tmem_wait_st();
            tc::fence_before();
            __syncwarp();
            arrive(C::kProbsReady + two);
            arrive(C::kDecFree + dec.slot);
        }
    } else if (warp >= kLcState && warp < kLcOutput) {
        const int half = (warp - kLcState) / 4;  // of the columns
        constexpr int kMine = DV / 2;
        const bool mine = row < a.Dk;  // row of S
        const int left = cols - half * kMine;  // columns in this thread, where above 0
        const long long size = (long long)a.Dk * a.Dv, in_head = (long long)row * a.Dv + c0 + half * kMine;
        float *const at_cut = p.states + ((long long)(unit - (units - p.cut)) * a.Dk + row) * DV + half * kMine;
        int *const stored = p.tickets + 1 + (unit - (units - p.cut));
        if (piece1) {
            // the first piece's warps, which run or are done, have all stored their rows
            int polls = 0;
            while (lane == 0 && lc_acquire(stored) < kLcStateWarps && polls < kLcIdlePolls) {
                ++polls;
                __nanosleep(64);
            }
            good = __shfl_sync(0xffffffffu, polls, 0) < kLcIdlePolls;
        }
        float2 s[kMine / 2];
        auto load = [&](const float *from, float2 (&v)[kMine / 2]) {
#pragma unroll
            for (int x = 0; x < kMine; x += 4) {
                float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (from && mine && x < left)
                    f = *reinterpret_cast<const float4 *>(from + x);
                v[x / 2] = make_float2(f.x, f.y), v[x / 2 + 1] = make_float2(f.z, f.w);
            }
        };
        load(piece1    ? at_cut
             : seg > 0 ? (STATES ? nullptr : p.states + (bh * (p.nseg - 1) + seg - 1) * size + in_head)
             : a.h0    ? a.h0 + bh * size + in_head
                       : nullptr,
             s);
        // the bf16 copy of S, its 16-byte pieces swizzled as TMA would
        auto publish = [&] {
            if (row < DK) {
#pragma unroll
                for (int x = 0; x < kMine / 8; ++x)
                    *reinterpret_cast<uint4 *>(smem + C::kSAt + row * 128 + (((half * (kMine / 8) + x) ^ (row & 7)) << 4)) =
                        make_uint4(lc_pack(s[4 * x].x, s[4 * x].y), lc_pack(s[4 * x + 1].x, s[4 * x + 1].y),
                                   lc_pack(s[4 * x + 2].x, s[4 * x + 2].y), lc_pack(s[4 * x + 3].x, s[4 * x + 3].y));
            }
            tc::fence_async_proxy();
            __syncwarp();
            arrive(C::kStateReady);
        };
        if (!STATES)
            publish();
        LcRing<C::kDecays> dec;
        LcRing<C::kDeltas> deltas;
        for (int c = 0; c < chunks && good; ++c, ++dec, ++deltas) {
            const uint32_t turn = c & 1;
            if (!wait(C::kDecFull + dec.slot, dec.round))
                break;
            const float2 grow = make_float2(decay[dec.slot].grow, decay[dec.slot].grow);
            const float2 keep = make_float2(decay[dec.slot].keep, decay[dec.slot].keep);
            __syncwarp();
            arrive(C::kDecFree + dec.slot);
            const uint32_t buf = deltas.slot;
            if (!wait(C::kDeltaDone + buf, deltas.round))
                break;
#pragma unroll
            for (int x = 0; x < kMine / 16; ++x) {
                const uint32_t at = lanes + C::kDeltaAt + buf * C::kDelta + half * kMine + 16 * x;
                uint32_t v[16];
                tc::tmem_ld16(at, v);
                tc::tmem_wait16(v);
#pragma unroll
                for (int y = 0; y < 8; ++y)
                    s[8 * x + y] = __ffma2_rn(s[8 * x + y], keep,
                                              __ffma2_rn(s[8 * x + y], grow, make_float2(__uint_as_float(v[2 * y]),
                                                                                         __uint_as_float(v[2 * y + 1]))));
                // the smaller parts
#pragma unroll
                for (int z = 1; z < C::kBlocks; ++z) {
                    tc::tmem_ld16(at + z * DV, v);
                    tc::tmem_wait16(v);
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        s[8 * x + y] = __fadd2_rn(s[8 * x + y], make_float2(__uint_as_float(v[2 * y]), __uint_as_float(v[2 * y + 1])));
                }
            }
            tc::fence_before();
            __syncwarp();
            arrive(C::kDeltaFree + buf);
            if (!STATES) {
                // Q S has read the copy that is replaced now
                if (!wait(C::kInterDone, turn))
                    break;
                publish();
            }
        }
        if (good && piece0 && t_end < len) {
            if (mine)
#pragma unroll
                for (int x = 0; x < kMine; x += 4)
                    *reinterpret_cast<float4 *>(at_cut + x) = make_float4(s[x / 2].x, s[x / 2].y, s[x / 2 + 1].x, s[x / 2 + 1].y);
            __syncwarp();
            if (lane == 0)
                lc_release_add(stored);
        }
        float *const to = !STATES && t_end == len       ? (a.h_last ? a.h_last + bh * size + in_head : nullptr)
                          : STATES || (seg == 0 && p.nseg > 1) ? p.states + (bh * (p.nseg - 1) + seg) * size + in_head
                                                                 : nullptr;
        if (good && to && mine)
#pragma unroll
            for (int x = 0; x < kMine; x += 4)
                if (x < left)
                    *reinterpret_cast<float4 *>(to + x) = make_float4(s[x / 2].x, s[x / 2].y, s[x / 2 + 1].x, s[x / 2 + 1].y);
    } else if (warp >= kLcOutput && !STATES) {
        const bool wide = a.Dv % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
        LcRing<C::kDecays> dec;
        LcRing<C::kMarks> mark;
        for (int c = 0; c < chunks; ++c, ++dec, ++mark) {
            const uint32_t turn = c & 1;
            const int t = t_first + c * kLcChunk + row;
            if (!wait(C::kDecFull + dec.slot, dec.round))
                break;
            const float r = a.scale * lc_ex2(decay[dec.slot].cb[row] + decay[dec.slot].m[quarter]);
            __syncwarp();
            arrive(C::kDecFree + dec.slot);
            if (!wait(C::kInterDone, turn) || !wait(C::kOutDone, turn))
                break;
            const bool marked = marks[mark.slot] == c + 1;
            __nv_bfloat16 *const o = a.out + (((long long)b * a.L + t) * a.H + h) * a.Dv + c0;
#pragma unroll 1
            for (int x = 0; x < DV / 16; ++x) {
                uint32_t u[16], v[16], w[8];
                tc::tmem_ld16(lanes + C::kInterAt + 16 * x, u);
                tc::tmem_ld16(lanes + C::kOutAt + 16 * x, v);
                tc::tmem_wait16(u);
                tc::tmem_wait16(v);
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const float2 z = __ffma2_rn(make_float2(r, r), make_float2(__uint_as_float(u[2 * y]), __uint_as_float(u[2 * y + 1])),
                                                make_float2(__uint_as_float(v[2 * y]), __uint_as_float(v[2 * y + 1])));
                    w[y] = lc_pack(z.x, z.y);
                }
                if (marked) {
                    // a NaN in every column whose v, at this row's token or before it in the chunk, is not finite
                    const __nv_bfloat16 *const from = a.v + b * a.v_batch + (t - row) * a.v_token + h * a.v_head + c0 + 16 * x;
                    for (int j = 0; j <= row && t - row + j < t_end; ++j)
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            if (16 * x + 2 * y < cols) {
                                const uint32_t e = *reinterpret_cast<const uint32_t *>(from + j * a.v_token + 2 * y);
                                w[y] |= ((e & 0x7f80u) == 0x7f80u ? 0x7fffu : 0u) |
                                        ((e & 0x7f800000u) == 0x7f800000u ? 0x7fff0000u : 0u);
                            }
                }
                if (t < t_end && 16 * x < cols) {
                    if (wide) {
                        lc_store32(o + 16 * x, w);
                    } else {
                        *reinterpret_cast<uint4 *>(o + 16 * x) = make_uint4(w[0], w[1], w[2], w[3]);
                        if (16 * x + 8 < cols)
                            *reinterpret_cast<uint4 *>(o + 16 * x + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
            }
            tc::fence_before();
            __syncwarp();
            arrive(C::kInterFree);
            arrive(C::kOutFree);
        }
    }
    if (!good && lane == 0)
        wait_ran_out(a.err);
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 1)
        tc::tmem_free(tmem, 512);
}

template <int DK, int DV, int PASS>
__global__ void __launch_bounds__(kLcThreads, 1)
    linear_chunked_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const ChunkedArgs p, int seg_from, int segs)
{
    linear_chunked<DK, DV, PASS>(map_q, map_k, map_v, p, (int)blockIdx.x, seg_from, segs);
}

// All of the first segments, and beside them the first pass over the others but the last ones.
template <int DK, int DV>
__global__ void __launch_bounds__(kLcThreads, 1)
    linear_first_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const ChunkedArgs p)
{
    if ((int)blockIdx.x < p.units)
        linear_chunked<DK, DV, kLcAll>(map_q, map_k, map_v, p, (int)blockIdx.x, 0, 1);
    else
        linear_chunked<DK, DV, kLcStates>(map_q, map_k, map_v, p, (int)blockIdx.x - p.units, 1, p.nseg - 2);
}

// No ticket taken, nothing stored: ahead of a kernel with cut units.
constexpr int kLcTicketThreads = 96;

__global__ void __launch_bounds__(kLcTicketThreads) linear_tickets_kernel(int *tickets, int n)
{
    grid_next();
    grid_wait();
    for (int i = threadIdx.x; i < n; i += kLcTicketThreads)
        tickets[i] = 0;
}

// The segments' own states -> the state behind each: one thread for four elements of a head's state, with the
// loads of kLcCarry segments on their way at once.  A slow decay comes less 1, for over a hundred segments would add up
// what its rounding to fp32 loses (4e-6 of the state, 3e-7 so).
constexpr int kLcCarry = 8, kLcCarryThreads = 128;

__global__ void __launch_bounds__(kLcCarryThreads) linear_carry_kernel(float *states, const float *decays, int segs, int size4,
                                                                       long long total)
{
    grid_next();
    grid_wait();
    const long long e = (long long)blockIdx.x * kLcCarryThreads + threadIdx.x;
    if (e >= total)
        return;
    const long long head = e / size4;
    float4 *const at = reinterpret_cast<float4 *>(states) + head * segs * size4 + e % size4;
    const float *const d = decays + head * segs;
    float4 s = at[0];
    for (int i0 = 1; i0 < segs; i0 += kLcCarry) {
        float4 own[kLcCarry];
        float by[kLcCarry];
#pragma unroll
        for (int i = 0; i < kLcCarry; ++i)
            if (i0 + i < segs)
                own[i] = at[(long long)(i0 + i) * size4], by[i] = d[i0 + i];
#pragma unroll
        for (int i = 0; i < kLcCarry; ++i)
            if (i0 + i < segs) {
                const float keep = __float_as_uint(by[i]) >> 31 ? 1.0f : 0.0f;
                s = make_float4(fmaf(s.x, keep, fmaf(s.x, by[i], own[i].x)), fmaf(s.y, keep, fmaf(s.y, by[i], own[i].y)),
                                fmaf(s.z, keep, fmaf(s.z, by[i], own[i].z)), fmaf(s.w, keep, fmaf(s.w, by[i], own[i].w)));
                at[(long long)(i0 + i) * size4] = s;
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
cudaError_t launch_width(const ChunkedArgs &p, cudaStream_t s)
{
    static int configured[4][kMaxDevices];
    const LinAttnArgs &a = p.a;
    CUtensorMap q, k, v;
    cudaError_t e = lc_map(&q, a.q, a.B, a.L, a.G, a.Dk, a.q_batch, a.q_token, a.q_head);
    if (e == cudaSuccess)
        e = lc_map(&k, a.k, a.B, a.L, a.G, a.Dk, a.k_batch, a.k_token, a.k_head);
    if (e == cudaSuccess)
        e = lc_map(&v, a.v, a.B, a.L, a.H, a.Dv, a.v_batch, a.v_token, a.v_head);
    ChunkedArgs part = p;
    part.units = (int)((long long)a.B * a.H * ((a.Dv + DV - 1) / DV));
    const unsigned units = (unsigned)part.units;
    // The longest sequences first, so that the last CTAs to end have little to do, where there is more than one CTA for
    // an SM and a warp can sort them.  (Seven of up to 1531 tokens, 32 heads of 128 x 64: 45.3 us as they come, 38.6 so.)
    const bool sorted = a.lengths && a.B > 1 && a.B <= 32 && p.nseg == 1 && units > (unsigned)kLcSms;
    const auto whole = sorted ? linear_chunked_kernel<DK, DV, kLcSorted> : linear_chunked_kernel<DK, DV, kLcAll>;
    const bool cut = p.cut && !sorted;
    if (e == cudaSuccess)
        e = cut ? configure_smem(linear_chunked_kernel<DK, DV, kLcCut>, (int)Lc<DK, DV>::kSmem, configured[2])
                : configure_smem(whole, (int)Lc<DK, DV>::kSmem, configured[sorted ? 3 : 0]);
    constexpr size_t kAllSmem = Lc<DK, DV>::kSmem, kPassSmem = Lc<DK, DV, true>::kSmem;
    constexpr size_t kFirstSmem = kAllSmem > kPassSmem ? kAllSmem : kPassSmem;
    if (e == cudaSuccess && p.nseg > 1)
        e = configure_smem(linear_first_kernel<DK, DV>, (int)kFirstSmem, configured[1]);
    if (e != cudaSuccess)
        return e;
    if (cut) {
        e = launch_early(linear_tickets_kernel, 1, kLcTicketThreads, 0, s, 1, p.tickets, p.cut + 1);
        return e != cudaSuccess ? e
                                : launch_early(linear_chunked_kernel<DK, DV, kLcCut>, units + (unsigned)p.cut, kLcThreads,
                                               Lc<DK, DV>::kSmem, s, 1, q, k, v, part, 0, 1);
    }
    if (p.nseg == 1)
        return launch_early(whole, units, kLcThreads, Lc<DK, DV>::kSmem, s, 1, q, k, v, part, 0, 1);
    e = launch_early(linear_first_kernel<DK, DV>, units * (unsigned)(p.nseg - 1), kLcThreads, kFirstSmem, s, 1, q, k, v, part);
    const long long elements = (long long)a.B * a.H * a.Dk * a.Dv / 4;
    if (e == cudaSuccess)
        e = launch_early(linear_carry_kernel, (unsigned)((elements + kLcCarryThreads - 1) / kLcCarryThreads), kLcCarryThreads, 0, s,
                         1, p.states, (const float *)p.decays, p.nseg - 1, a.Dk * a.Dv / 4, elements);
    if (e == cudaSuccess)
        e = launch_early(linear_chunked_kernel<DK, DV, kLcAll>, units * (unsigned)(p.nseg - 1), kLcThreads, Lc<DK, DV>::kSmem, s, 1,
                         q, k, v, part, 1, p.nseg - 1);
    return e;
}

// Columns of the state in one CTA.
int lc_cols(const LinAttnArgs &a) { return a.Dv <= 32 ? 32 : 64; }

// Segments of a sequence, and cut units, by the time that they take in tenths of a chunk's: whole waves of CTAs, two
// or three chunks to fill and drain a CTA, 0.55 of a chunk's time for one of the first pass (the first segment, which
// needs no such pass, is shorter than the others so as to end with theirs), and what the launches and the sums between
// the passes take.  (us for 16 heads of 128 x 128: 2048 tokens, 1, 3, 4, 5 segments: 40, 39, 36, 40;  32768 tokens, 4,
// 5, 9, 10: 286, 227, 232, 226.  One head of 128 x 64, 65536 tokens, 24, 103: 82, 40.)
//
// Where the units fill the last of several waves by half or less, those of that wave are cut in two instead: the first
// pieces go first, the second ones behind the whole units, when what they start from is long there (they wait for it all
// the same), and both together fill the SMs: 32 x 3136 tokens of 6 heads of 64 x 32, 75 us uncut, 62 so.  (Up to 32
// sequences with lengths are sorted instead, which evens out more.)
void lc_plan(const LinAttnArgs &a, ChunkedArgs *p)
{
    const long long units = (long long)a.B * a.H * ((a.Dv + lc_cols(a) - 1) / lc_cols(a));
    const int chunks = (a.L + kLcChunk - 1) / kLcChunk;
    long long best = 10 * ((units + kLcSms - 1) / kLcSms) * (chunks + 2);
    p->nseg = 1, p->cut = 0;
    p->first_chunks = p->seg_chunks = chunks;
    for (int n = 3; n <= kLcMaxSegments && n <= chunks; ++n) {
        const int each = (int)((100LL * chunks + 100 * n - 46) / (100 * n - 45));  // of n - 1 segments and 0.55 of one
        const int rest = (chunks - 1) / each, first = chunks - rest * each;       // at least one chunk
        const long long waves = (units * rest + kLcSms - 1) / kLcSms;
        const long long cost = waves * (5 * max(each, 2 * first) + 10 * each + 45) + 30 + n / 2;
        if (rest > 1 && cost < best) {
            best = cost;
            p->nseg = rest + 1;
            p->first_chunks = first;
            p->seg_chunks = each;
        }
    }
    const int over = (int)(units % kLcSms), half = (chunks + 1) / 2;
    if (units > kLcSms && over > 0 && over <= kLcSms / 2 && chunks > 1 &&
        10 * (units / kLcSms * (chunks + 2) + half + 2) + 20 < best) {
        p->nseg = 1;
        p->cut = over;
        p->cut_chunks = half;
        p->first_chunks = p->seg_chunks = chunks;
    }
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

cudaError_t linear_chunked_wait_ran_out(bool *out, cudaStream_t s) { return take_wait_ran_out(out, s); }

size_t linear_chunked_workspace(const LinAttnArgs &a)
{
    ChunkedArgs p{};
    lc_plan(a, &p);
    if (p.nseg == 1)
        return p.cut ? round256((size_t)(p.cut + 1) * 4) + (size_t)p.cut * a.Dk * lc_cols(a) * 4 : 0;
    const size_t heads = (size_t)a.B * a.H;
    return round256(heads * (p.nseg - 1) * 4) + heads * (p.nseg - 1) * a.Dk * a.Dv * 4;
}

cudaError_t launch_linear_chunked(const LinAttnArgs &a, void *workspace, cudaStream_t s)
{
    ChunkedArgs p{};
    p.a = a;
    lc_plan(a, &p);
    const long long heads = (long long)a.B * a.H;
    if (heads * p.nseg * 2 > 0x7fffffffLL || heads * 64 > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    if (p.nseg > 1) {
        p.decays = static_cast<float *>(workspace);
        p.states = reinterpret_cast<float *>(static_cast<char *>(workspace) + round256((size_t)heads * (p.nseg - 1) * 4));
    } else if (p.cut) {
        p.tickets = static_cast<int *>(workspace);
        p.states = reinterpret_cast<float *>(static_cast<char *>(workspace) + round256((size_t)(p.cut + 1) * 4));
    }
    if (lc_cols(a) == 32)
        return a.Dk <= 64 ? launch_width<64, 32>(p, s) : launch_width<128, 32>(p, s);
    return a.Dk <= 64 ? launch_width<64, 64>(p, s) : launch_width<128, 64>(p, s);
}

}  // namespace ss2d
