// Runs rms_norm.cu's kernel on the host: one std::thread per thread of each CTA, __syncthreads on a per-CTA barrier; built
// with AddressSanitizer and UBSan by tests/test_norm_kernel_emulation.py.  The instance is the one that ss2d_rms_norm's own
// rule takes, and the grid is its launcher's.
// Arguments: dir rows D x_bf16 residual (0 none, 1 fp32, 2 bf16) y_dtype eps many
//   dir/x, dir/residual, dir/weight; writes dir/y, dir/scales (e4m3), dir/residual_out.  `many`: as if there were more rows.
#include <string>
#include "kernel_emu.h"
using namespace ss2d;
static std::vector<unsigned char> rd(const std::string &f, size_t n)
{
    std::vector<unsigned char> v(n);
    FILE *fp = fopen(f.c_str(), "rb");
    if (!fp || fread(v.data(), 1, n, fp) != n) { fprintf(stderr, "read %s\n", f.c_str()); exit(2); }
    fclose(fp);
    return v;
}
static void wr(const std::string &f, const std::vector<unsigned char> &v)
{
    FILE *fo = fopen(f.c_str(), "wb");
    fwrite(v.data(), 1, v.size(), fo);
    fclose(fo);
}
// 16-byte aligned, of exactly n bytes, so that the sanitizer sees an access behind it
struct Buffer {
    unsigned char *p;
    size_t n;
    explicit Buffer(size_t n) : p((unsigned char *)aligned_alloc(16, (n + 15) / 16 * 16)), n(n) { memset(p, 0xAB, n); }
    explicit Buffer(const std::vector<unsigned char> &v) : Buffer(v.size()) { memcpy(p, v.data(), n); }
    Buffer(const Buffer &) = delete;
    ~Buffer() { free(p); }
    std::vector<unsigned char> bytes() const { return {p, p + n}; }
};
int main(int argc, char **argv)
{
    if (argc != 9) return 1;
    const std::string dir = argv[1];
    const long long rows = atoll(argv[2]);
    const int D = atoi(argv[3]), x_bf16 = atoi(argv[4]), res = atoi(argv[5]), y_dtype = atoi(argv[6]);
    const int groups = (D + 127) / 128;
    const size_t n = (size_t)rows * D;
    Buffer x(rd(dir + "/x", n * (x_bf16 ? 2 : 4))), weight(rd(dir + "/weight", (size_t)D * 4));
    Buffer residual(res ? rd(dir + "/residual", n * (res == 2 ? 2 : 4)) : std::vector<unsigned char>(16));
    Buffer out(residual.n), y(n * (y_dtype == SS2D_F32 ? 4 : y_dtype == SS2D_BF16 ? 2 : 1)), scales((size_t)rows * groups * 4);
    RmsArgs a{};
    a.x = x.p, a.weight = (const float *)weight.p, a.y = y.p, a.scales = y_dtype == SS2D_E4M3 ? (float *)scales.p : nullptr;
    if (res) a.residual = residual.p, a.residual_out = out.p;
    a.rows = rows, a.D = D, a.groups = groups;
    a.x_bf16 = x_bf16, a.res_bf16 = res == 2, a.y_dtype = y_dtype, a.eps = (float)atof(argv[7]);
    const bool many = atoi(argv[8]) != 0;
    int e = 0, s = 0;
    (void)s;
    DISPATCH
    if (e) return 3;
    wr(dir + "/y", y.bytes());
    wr(dir + "/scales", scales.bytes());
    wr(dir + "/residual_out", out.bytes());
    return 0;
}
