// Runs linear_recurrent.cu's kernel (linear attention token by token) and linear_chunked.cu's
// linear_carry_kernel on the host: one std::thread per thread of each CTA, __syncthreads on a per-CTA
// barrier, each CTA's shared memory in its own buffer; built with AddressSanitizer and UBSan by
// tests/test_recurrent_kernel_emulation.py.  The grids are the launchers'.
// Arguments: dir mode B L G H Dk Dv per_token pool
//   mode 0 / 1: a prompt of L tokens, 1 with dir/lengths ((B) int32)
//   mode 2 / 3: a step of B rows, 3 with dir/slots ((B) int32)
//     dir/q, dir/k ((B, L, G, Dk) bf16), dir/v ((B, L, H, Dv) bf16), dir/gates, dir/state ((B or pool, H, Dk, Dv),
//     replaced), dir/out ((B, L, H, Dv) bf16, rows that are not written stay)
//   mode 4: dir/state ((B, L, Dk, Dv): the states of L segments of B heads, replaced) with dir/gates ((B, L) decays)
#include <string>
#include "kernel_emu.h"
using namespace ss2d;
template <class T>
std::vector<T> rd(const std::string &f, size_t n)
{
    std::vector<T> v(n);
    FILE *fp = fopen(f.c_str(), "rb");
    if (!fp || fread(v.data(), sizeof(T), n, fp) != n) { fprintf(stderr, "read %s\n", f.c_str()); exit(2); }
    fclose(fp);
    return v;
}
template <class T>
void wr(const std::string &f, const std::vector<T> &v)
{
    FILE *fo = fopen(f.c_str(), "wb");
    fwrite(v.data(), sizeof(T), v.size(), fo);
    fclose(fo);
}
template <bool STEP>
void run(const LinAttnArgs &a, unsigned grid)
{
    const int rows = (a.Dk + kLrGroups - 1) / kLrGroups;
    emu_grid(grid, 1, kLrThreads, kEmuShared, [&] {
        if (rows <= 2) linear_recurrent_kernel<STEP, 2>(a);
        else if (rows <= 4) linear_recurrent_kernel<STEP, 4>(a);
        else linear_recurrent_kernel<STEP, kLaMaxDim / kLrGroups>(a);
    });
}
int main(int argc, char **argv)
{
    if (argc < 11) return 1;
    const std::string dir = argv[1];
    int n[9];
    for (int i = 0; i < 9; ++i) n[i] = atoi(argv[2 + i]);
    const int mode = n[0], B = n[1], L = n[2], G = n[3], H = n[4], Dk = n[5], Dv = n[6], per_token = n[7], pool = n[8];
    if (mode == 4) {
        auto states = rd<float>(dir + "/state", (size_t)B * L * Dk * Dv);
        auto decays = rd<float>(dir + "/gates", (size_t)B * L);
        const long long elements = (long long)B * Dk * Dv / 4;
        emu_grid((unsigned)((elements + kLcCarryThreads - 1) / kLcCarryThreads), 1, kLcCarryThreads, 0,
                 [&] { linear_carry_kernel(states.data(), decays.data(), L, Dk * Dv / 4, elements); });
        wr(dir + "/state", states);
        return 0;
    }
    auto q = rd<__nv_bfloat16>(dir + "/q", (size_t)B * L * G * Dk), k = rd<__nv_bfloat16>(dir + "/k", (size_t)B * L * G * Dk);
    auto v = rd<__nv_bfloat16>(dir + "/v", (size_t)B * L * H * Dv), out = rd<__nv_bfloat16>(dir + "/out", (size_t)B * L * H * Dv);
    auto gates = rd<float>(dir + "/gates", per_token ? (size_t)B * L * H : H);
    auto state = rd<float>(dir + "/state", (size_t)(mode < 2 ? B : pool) * H * Dk * Dv);
    std::vector<int> rows;
    if (mode == 1) rows = rd<int>(dir + "/lengths", B);
    if (mode == 3) rows = rd<int>(dir + "/slots", B);
    int err = 5;
    LinAttnArgs a{};
    a.q = q.data(), a.k = k.data(), a.v = v.data(), a.log_decay = gates.data(), a.out = out.data();
    a.q_batch = a.k_batch = (long long)L * G * Dk, a.q_token = a.k_token = (long long)G * Dk, a.q_head = a.k_head = Dk;
    a.v_batch = (long long)L * H * Dv, a.v_token = (long long)H * Dv, a.v_head = Dv;
    a.h0 = a.h_last = state.data();
    a.scale = 0.5f, a.per_token = per_token;
    a.B = B, a.L = L, a.G = G, a.H = H, a.Dk = Dk, a.Dv = Dv, a.pool = pool;
    const unsigned grid = (unsigned)(B * H * ((Dv + kLrCols - 1) / kLrCols));
    if (mode < 2) {
        a.lengths = mode == 1 ? rows.data() : nullptr;
        a.err = &err;
        run<false>(a, grid);
        if (err != 0) { fprintf(stderr, "error word %d\n", err); return 3; }
    } else {
        a.slots = mode == 3 ? rows.data() : nullptr;
        run<true>(a, grid);
    }
    wr(dir + "/out", out);
    wr(dir + "/state", state);
    return 0;
}
