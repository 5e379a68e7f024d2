// Runs the decay warp of linear_chunked.cu's kernel on the host, a std::thread for each lane, and writes every chunk's
// factors; put together by tests/test_chunked_decay_emulation.py.  Waits and arrivals do nothing: the ring of decays is
// read out as each chunk is announced.
// Arguments: dir tokens first end states; dir/gates: (tokens) fp32.  Writes dir/decay: a ChunkDecay for each chunk.
#include <string>
#include "kernel_emu.h"
using namespace ss2d;
static std::vector<float> g_gates;
static std::vector<ChunkDecay> g_out;
static float g_decays[1] = {-1.0f};
struct Args { int per_token = 1, H = 1, L = 0; const float *log_decay; };
struct Params { Args a; float *decays = g_decays; int nseg = 2; };
template <bool STATES>
void warp2(const Params &p, int t_first, int t_end)
{
    using C = Lc<128, 64, STATES>;
    static ChunkDecay decay[C::kDecays];
    const Args &a = p.a;
    const int lane = g_lane, h = 0, b = 0, seg = 0;
    const long long bh = 0;
    bool good = true;
    const int chunks = (t_end - t_first + kLcChunk - 1) / kLcChunk;
    int announced = 0;
    auto wait = [](int, uint32_t) { return true; };
    auto arrive = [&](int) {
        if (lane == 0) g_out.push_back(decay[announced % C::kDecays]);
        ++announced;
        __syncwarp();
    };
    (void)b, (void)bh, (void)seg, (void)h;
    DECAY_WARP
}
int main(int argc, char **argv)
{
    if (argc != 6) return 1;
    const std::string dir = argv[1];
    const int n = atoi(argv[2]), first = atoi(argv[3]), end = atoi(argv[4]), states = atoi(argv[5]);
    g_gates.resize(n);
    FILE *f = fopen((dir + "/gates").c_str(), "rb");
    if (!f || fread(g_gates.data(), 4, n, f) != (size_t)n) return 2;
    fclose(f);
    Params p;
    p.a.L = n, p.a.log_decay = g_gates.data();
    emu_grid(1, 1, 32, 16, [&] { states ? warp2<true>(p, first, end) : warp2<false>(p, first, end); });
    f = fopen((dir + "/decay").c_str(), "wb");
    fwrite(g_out.data(), sizeof(ChunkDecay), g_out.size(), f);
    fwrite(g_decays, 4, 1, f);
    fclose(f);
    return 0;
}
