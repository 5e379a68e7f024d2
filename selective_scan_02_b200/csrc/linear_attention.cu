// linear_attention.cu -- the C entry points of linear attention with a decay for each head
// (ss2d_linear_attention, ss2d_linear_attention_step) and of the operators' device status.
#include "linear_attention.h"

#include "op_check.h"
#include "ss2d.h"
#include "wait_words.h"

namespace ss2d {
namespace {

constexpr int kLaMaxSlotRows = 65536;   // of a step that names their states
constexpr size_t kLaStatusBytes = 256;  // the error word of the bounded waits

// The stride of a dimension, or a valid one where it has one element and its stride says nothing.
long long la_stride(long long stride, long long size) { return size > 1 ? stride : 8; }

// Bytes from a tensor's first element to behind its last (strides of 0 or below count as none).
size_t la_span(long long n0, long long s0, long long n1, long long s1, long long n2, long long s2, long long width)
{
    long long last = width;
    if (n0 > 1) last += (n0 - 1) * s0;
    if (n1 > 1) last += (n1 - 1) * s1;
    if (n2 > 1) last += (n2 - 1) * s2;
    return (size_t)last * 2;
}

int la_check_sizes(const char *call, long long B, long long L, long long G, long long H, long long Dk, long long Dv)
{
    if (B <= 0 || L <= 0 || G <= 0 || H <= 0 || Dk <= 0 || Dv <= 0)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: sizes must be positive (B=%lld L=%lld G=%lld H=%lld Dk=%lld Dv=%lld)",
                       call, B, L, G, H, Dk, Dv);
    if (H % G != 0)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: H=%lld is not a multiple of G=%lld", call, H, G);
    if (Dk % 8 != 0 || Dv % 8 != 0 || Dk > kLaMaxDim || Dv > kLaMaxDim)
        return op_fail(SS2D_ERR_UNSUPPORTED, "%s: Dk=%lld and Dv=%lld must be multiples of 8 up to %d", call, Dk, Dv,
                       kLaMaxDim);
    if (L > (1LL << 24) || B * H > (1LL << 24) || B * L > 0x7fffffffLL)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: problem too large", call);
    return SS2D_OK;
}

// Strides are in elements; those of dimensions with more than one element must keep 16-byte rows.
int la_check_stride(const char *call, const char *name, long long size, long long stride)
{
    if (size > 1 && (stride < 8 || stride % 8 != 0 || stride >= (1LL << 38)))
        return op_fail(SS2D_ERR_UNSUPPORTED, "%s: strides of %s must be positive multiples of 8 elements (got %lld)",
                       call, name, stride);
    return SS2D_OK;
}

// Sequences that run token by token: with few tokens a chunk of 128 is mostly padding.  (Token by token and in
// chunks, 16 heads of 128 x 128: one sequence of 4, 8, 16 tokens 5.4, 8.9, 15.7 and 8.9 us throughout; 64
// sequences of 8 and 16 tokens 57 and 103, in chunks 118 both.)
constexpr int kLaRecurrentTokens = 8;

size_t la_workspace(const ss2d_linear_attention_args &a)
{
    if (a.L <= kLaRecurrentTokens)
        return kLaStatusBytes;
    LinAttnArgs p{};
    p.B = a.B, p.L = a.L, p.G = a.G, p.H = a.H, p.Dk = a.Dk, p.Dv = a.Dv;
    return kLaStatusBytes + linear_chunked_workspace(p);
}

int la_check(const char *call, const ss2d_linear_attention_args *a)
{
    if (!a || a->struct_size != sizeof(ss2d_linear_attention_args))
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: args is null or its struct_size is wrong", call);
    return la_check_sizes(call, a->B, a->L, a->G, a->H, a->Dk, a->Dv);
}

}  // namespace
}  // namespace ss2d

extern "C" size_t ss2d_linear_attention_workspace(const ss2d_linear_attention_args *args)
{
    using namespace ss2d;
    set_last_error(SS2D_OK, "");
    if (la_check("ss2d_linear_attention_workspace", args) != SS2D_OK)
        return (size_t)-1;
    return la_workspace(*args);
}

extern "C" int ss2d_linear_attention(const ss2d_linear_attention_args *args, void *workspace, size_t workspace_bytes,
                                     void *stream)
{
    using namespace ss2d;
    static const char *call = "ss2d_linear_attention";
    set_last_error(SS2D_OK, "");
    int st = la_check(call, args);
    if (st != SS2D_OK)
        return st;
    const ss2d_linear_attention_args &a = *args;
    if (!a.q || !a.k || !a.v || !a.log_decay || !a.out)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: q, k, v, log_decay and out must be non-null", call);
    const struct { const char *name; long long heads; const long long *s; } strided[] = {
        {"q", a.G, a.q_stride}, {"k", a.G, a.k_stride}, {"v", a.H, a.v_stride}};
    for (const auto &t : strided)
        if ((st = la_check_stride(call, t.name, a.B, t.s[0])) != SS2D_OK ||
            (st = la_check_stride(call, t.name, a.L, t.s[1])) != SS2D_OK ||
            (st = la_check_stride(call, t.name, t.heads, t.s[2])) != SS2D_OK)
            return st;
    const size_t need = la_workspace(a);
    if (!workspace || workspace_bytes < need)
        return op_fail(SS2D_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", call, need, workspace_bytes);
    const size_t BH = (size_t)a.B * a.H, state = BH * a.Dk * a.Dv * 4;
    const OpSpan in[] = {
        {"q", a.q, la_span(a.B, a.q_stride[0], a.L, a.q_stride[1], a.G, a.q_stride[2], a.Dk)},
        {"k", a.k, la_span(a.B, a.k_stride[0], a.L, a.k_stride[1], a.G, a.k_stride[2], a.Dk)},
        {"v", a.v, la_span(a.B, a.v_stride[0], a.L, a.v_stride[1], a.H, a.v_stride[2], a.Dv)},
        {"log_decay", a.log_decay, (a.decay_per_token ? BH * a.L : (size_t)a.H) * 4},
        {"lengths", a.lengths, (size_t)a.B * 4, 4},
        // a state may be replaced in place: each element is read and then written by the same thread
        {"h0", a.h0, a.h0 == a.h_last ? 0 : state}};
    const OpSpan out[] = {{"out", a.out, BH * a.L * a.Dv * 2}, {"h_last", a.h_last, state}, {"workspace", workspace, need}};
    st = op_check_tensors(call, in, 6, out, 3);
    if (st != SS2D_OK)
        return st;
    LinAttnArgs p{};
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.k = static_cast<const __nv_bfloat16 *>(a.k);
    p.v = static_cast<const __nv_bfloat16 *>(a.v);
    p.q_batch = la_stride(a.q_stride[0], a.B), p.q_token = la_stride(a.q_stride[1], a.L), p.q_head = la_stride(a.q_stride[2], a.G);
    p.k_batch = la_stride(a.k_stride[0], a.B), p.k_token = la_stride(a.k_stride[1], a.L), p.k_head = la_stride(a.k_stride[2], a.G);
    p.v_batch = la_stride(a.v_stride[0], a.B), p.v_token = la_stride(a.v_stride[1], a.L), p.v_head = la_stride(a.v_stride[2], a.H);
    p.log_decay = a.log_decay;
    p.per_token = a.decay_per_token != 0;
    p.lengths = a.lengths;
    p.h0 = a.h0;
    p.h_last = a.h_last;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.err = static_cast<int *>(workspace);
    p.scale = a.scale;
    p.B = a.B, p.L = a.L, p.G = a.G, p.H = a.H, p.Dk = a.Dk, p.Dv = a.Dv;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a.L <= kLaRecurrentTokens
                              ? launch_linear_recurrent(p, false, s)
                              : launch_linear_chunked(p, static_cast<char *>(workspace) + kLaStatusBytes, s);
    return e == cudaSuccess ? SS2D_OK : op_cuda_fail(e, "ss2d_linear_attention launch");
}

extern "C" int ss2d_linear_attention_step(const ss2d_linear_attention_step_args *args, void *stream)
{
    using namespace ss2d;
    static const char *call = "ss2d_linear_attention_step";
    set_last_error(SS2D_OK, "");
    if (!args || args->struct_size != sizeof(ss2d_linear_attention_step_args))
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: args is null or its struct_size is wrong", call);
    const ss2d_linear_attention_step_args &a = *args;
    int st = la_check_sizes(call, a.B, 1, a.G, a.H, a.Dk, a.Dv);
    if (st != SS2D_OK)
        return st;
    if (a.pool <= 0 || (long long)a.pool * a.H > (1LL << 24))
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: pool=%d must be positive, and pool * H at most 2^24", call, a.pool);
    if (!a.slots && a.pool < a.B)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: without slots the pool's %d states must hold the batch of %d", call,
                       a.pool, a.B);
    // Every CTA compares its row's slot with all others: 2048 rows of 2 heads take 3 us by it, 32768 0.6 ms, and a million
    // would take seconds.
    if (a.slots && a.B > kLaMaxSlotRows)
        return op_fail(SS2D_ERR_UNSUPPORTED, "%s: with slots, B=%d is above %d", call, a.B, kLaMaxSlotRows);
    if (!a.q || !a.k || !a.v || !a.log_decay || !a.state || !a.out)
        return op_fail(SS2D_ERR_INVALID_ARG, "%s: q, k, v, log_decay, state and out must be non-null", call);
    const struct { const char *name; long long heads; const long long *s; } strided[] = {
        {"q", a.G, a.q_stride}, {"k", a.G, a.k_stride}, {"v", a.H, a.v_stride}};
    for (const auto &t : strided)
        if ((st = la_check_stride(call, t.name, a.B, t.s[0])) != SS2D_OK ||
            (st = la_check_stride(call, t.name, t.heads, t.s[1])) != SS2D_OK)
            return st;
    const size_t BH = (size_t)a.B * a.H;
    const OpSpan in[] = {{"q", a.q, la_span(a.B, a.q_stride[0], 1, 0, a.G, a.q_stride[1], a.Dk)},
                         {"k", a.k, la_span(a.B, a.k_stride[0], 1, 0, a.G, a.k_stride[1], a.Dk)},
                         {"v", a.v, la_span(a.B, a.v_stride[0], 1, 0, a.H, a.v_stride[1], a.Dv)},
                         {"log_decay", a.log_decay, (a.decay_per_token ? BH : (size_t)a.H) * 4},
                         {"slots", a.slots, (size_t)a.B * 4, 4}};
    const OpSpan out[] = {{"out", a.out, BH * a.Dv * 2}, {"state", a.state, (size_t)a.pool * a.H * a.Dk * a.Dv * 4}};
    st = op_check_tensors(call, in, 5, out, 2);
    if (st != SS2D_OK)
        return st;
    LinAttnArgs p{};
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.k = static_cast<const __nv_bfloat16 *>(a.k);
    p.v = static_cast<const __nv_bfloat16 *>(a.v);
    p.q_batch = la_stride(a.q_stride[0], a.B), p.q_head = la_stride(a.q_stride[1], a.G);
    p.k_batch = la_stride(a.k_stride[0], a.B), p.k_head = la_stride(a.k_stride[1], a.G);
    p.v_batch = la_stride(a.v_stride[0], a.B), p.v_head = la_stride(a.v_stride[1], a.H);
    p.log_decay = a.log_decay;
    p.per_token = a.decay_per_token != 0;
    p.slots = a.slots;
    p.h0 = a.state;
    p.h_last = a.state;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.scale = a.scale;
    p.B = a.B, p.L = 1, p.G = a.G, p.H = a.H, p.Dk = a.Dk, p.Dv = a.Dv, p.pool = a.pool;
    const cudaError_t e = launch_linear_recurrent(p, true, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SS2D_OK : op_cuda_fail(e, "ss2d_linear_attention_step launch");
}

extern "C" int ss2d_workspace_status(const void *workspace, void *stream)
{
    using namespace ss2d;
    static const char *call = "ss2d_workspace_status";
    set_last_error(SS2D_OK, "");
    if (!workspace)
        return op_fail(SS2D_ERR_WORKSPACE, "%s: the call's workspace is required", call);
    if (reinterpret_cast<uintptr_t>(workspace) & 15u)
        return op_fail(SS2D_ERR_MISALIGNED, "%s: workspace must be 16-byte aligned", call);
    int flag = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(&flag, workspace, sizeof(flag), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(s);
    if (e != cudaSuccess)
        return op_cuda_fail(e, "ss2d_workspace_status read");
    if (flag != 0)
        return op_fail(SS2D_ERR_DEVICE, "%s: a tensor-core kernel's bounded wait ran out; that call's outputs are not valid",
                       call);
    return SS2D_OK;
}

extern "C" int ss2d_wait_status(void *stream)
{
    using namespace ss2d;
    static const char *call = "ss2d_wait_status";
    set_last_error(SS2D_OK, "");
    bool out = false;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = matmul_fp8_wait_ran_out(&out, s);
    if (e == cudaSuccess)
        e = linear_chunked_wait_ran_out(&out, s);
    if (e == cudaSuccess)
        e = diag_wait_ran_out(&out, s);
    if (e != cudaSuccess)
        return op_cuda_fail(e, "ss2d_wait_status read");
    if (out)
        return op_fail(SS2D_ERR_DEVICE, "%s: a tensor-core kernel's bounded wait ran out on this device; the outputs of some call "
                                        "since the last ss2d_wait_status are not valid", call);
    return SS2D_OK;
}
