// Runs the two MMA-issuing branches of linear_chunked.cu's kernel on the host, one thread each, and prints what they
// issue, in order: MMAs (columns of tensor memory written and read, whether they accumulate), commits and waits.
// tests/test_chunked_mma_order.py puts the branches in and checks the order.  Nothing is computed; every wait succeeds.
// Arguments: DK DV states chunks ready, ready being what the polls answer: 0 no, 1 yes, 2 in turn.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#define __device__
#define __host__
#define __forceinline__ inline
using std::max;
using std::min;
inline void __syncwarp() {}
namespace tc {
inline uint64_t swizzled_desc(uint32_t addr, uint32_t, uint32_t) { return addr >> 4; }
inline bool elect_one() { return true; }
inline int cols_of(uint32_t idesc) { return (int)(idesc >> 17 & 63u) << 3; }
inline void mma(uint32_t d, int a, int an, uint32_t idesc, uint32_t acc)
{
    printf("mma %u %d %d %d %u %u\n", d, cols_of(idesc), a, an, acc, idesc);
}
inline void mma_bf16(uint32_t d, uint64_t, uint64_t, uint32_t idesc, uint32_t acc) { mma(d, 0, 0, idesc, acc); }
// A: 128 rows of 16 columns of K in bf16, two to a column
inline void mma_bf16_ta(uint32_t d, uint32_t a, uint64_t, uint32_t idesc, uint32_t acc) { mma(d, (int)a, 8, idesc, acc); }
inline void commit(uint32_t bar) { printf("commit %u\n", bar); }
}  // namespace tc
#include "kernel_emu.h"
using namespace ss2d;
static int g_ready, g_polls;
template <int DK, int DV, bool STATES>
void run(int warp, int chunks)
{
    using C = Lc<DK, DV, STATES>;
    const uint32_t base = 0, tmem = 0;
    bool good = true;
    auto bar = [](int which) { return (uint32_t)which; };
    auto wait = [](int which, uint32_t parity) { printf("wait %d %u\n", which, parity); return true; };
    auto ready = [](int, uint32_t) { return g_ready == 2 ? g_polls++ % 3 != 0 : g_ready != 0; };
    (void)base;
#define S(name) printf("bar %s %d\n", #name, (int)C::name)
    S(kScoresDone), S(kProbsReady), S(kWeightsReady), S(kWeightsFree), S(kStateReady), S(kInterDone), S(kInterFree), S(kOutDone),
        S(kOutFree), S(kDeltaDone), S(kDeltaFree), S(kKFree), S(kQFree), S(kVFree), S(kKFull), S(kQFull), S(kVFull), S(kVChecked);
    printf("rings %d %d\n", C::kSlots, C::kDeltas);
    if (warp == 1 && !STATES) {
        ISSUE_SCORES
    } else if (warp == 3) {
        ISSUE_STATE
    }
}
template <int DK, int DV>
void pick(int warp, int states, int chunks)
{
    if (states) run<DK, DV, true>(warp, chunks);
    else run<DK, DV, false>(warp, chunks);
}
int main(int argc, char **argv)
{
    if (argc != 7) return 1;
    const int dk = atoi(argv[1]), dv = atoi(argv[2]), states = atoi(argv[3]), chunks = atoi(argv[4]), warp = atoi(argv[6]);
    g_ready = atoi(argv[5]);
    if (dk == 64) dv == 32 ? pick<64, 32>(warp, states, chunks) : pick<64, 64>(warp, states, chunks);
    else dv == 32 ? pick<128, 32>(warp, states, chunks) : pick<128, 64>(warp, states, chunks);
    return 0;
}
