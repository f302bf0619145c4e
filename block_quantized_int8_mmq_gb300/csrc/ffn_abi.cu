// C entry points of the feed-forward operators: argument checks, then the launcher.  The error
// protocol is that of the whole library: a refused call launches nothing, writes nothing and prints
// one line.
#include "ffn.cuh"

namespace mmq {
namespace {

using namespace ffn;

constexpr int64_t LIMIT = (int64_t)1 << 40;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int refuse(const char* fn, int status, const char* why) {
    report(fn, status, why);
    return status;
}

// Sizes, types and weights, common to all four calls.
int check(const char* fn, int fmt, int dtype, int act, int64_t M, int64_t N, int64_t K, const void* w0, const void* w1,
          int mats, Call& c) {
    if (fmt < FMT_Q8_0 || fmt > FMT_Q6_K) return refuse(fn, MMQ_ERR_ARG, "fmt must be 0 (Q8_0), 1 (Q4_K), 2 (Q5_K) or 3 (Q6_K)");
    if (dtype != MMQ_F32 && dtype != MMQ_BF16 && dtype != MMQ_F16)
        return refuse(fn, MMQ_ERR_ARG, "dtype must be MMQ_F32, MMQ_BF16 or MMQ_F16");
    if (act < MMQ_ACT_NONE || act > MMQ_ACT_RELU) return refuse(fn, MMQ_ERR_ARG, "act must be one of the MMQ_ACT_ values");
    if (M < 0 || N < 1 || K < 1) return refuse(fn, MMQ_ERR_SHAPE, "M must be >= 0, N and K >= 1");
    const int64_t unit = is_superblock(fmt) ? QK_K : QK;
    if (K % unit != 0) return refuse(fn, MMQ_ERR_K_MULTIPLE, unit == QK_K ? "K % 256 != 0" : "K % 32 != 0");
    // rows, columns and 64-value steps are counted in 32 bits, with what rounding up adds
    if (M > 1 << 30 || N > 1 << 30 || K > 1 << 30 || M > LIMIT / K || N > LIMIT / K || M > LIMIT / N)
        return refuse(fn, MMQ_ERR_SHAPE, "a size above 2^30 or a product of two above 2^40");
    if (!w0 || (mats == 2 && !w1)) return refuse(fn, MMQ_ERR_NULL, "the weights must be non-NULL");
    if (!aligned(w0, 16) || !aligned(w1, 16)) return refuse(fn, MMQ_ERR_ALIGN, "the weights must be 16-byte aligned");
    c = Call{};
    c.fn = fn;
    c.fmt = fmt;
    c.dtype = dtype;
    c.act = act;
    c.mats = mats;
    c.M = M;
    c.N = N;
    c.K = K;
    c.w[0] = w0;
    c.w[1] = w1;
    return MMQ_OK;
}

// An array of M rows (contiguous: stride == width) of the call's element type.
int check_rows(const Call& c, const void* p, int64_t stride, int64_t width, const char* null_why) {
    if (!p && c.M > 0) return refuse(c.fn, MMQ_ERR_NULL, null_why);
    if (!aligned(p, c.dtype == MMQ_F32 ? 4 : 2)) return refuse(c.fn, MMQ_ERR_ALIGN, "arrays must be aligned to their elements");
    if (stride < width || stride > LIMIT) return refuse(c.fn, MMQ_ERR_SHAPE, "a row stride must be at least the row's width and at most 2^40");
    return MMQ_OK;
}

int check_x(const Call& c, const void* x, int64_t stride) {
    if (const int st = check_rows(c, x, stride, c.K, "x must be non-NULL")) return st;
    if (!aligned(x, 16) || (c.M > 1 && stride % (c.dtype == MMQ_F32 ? 4 : 8) != 0))
        return refuse(c.fn, MMQ_ERR_ALIGN, "every row of x must be 16-byte aligned (base and stride)");
    return MMQ_OK;
}

int check_bias(const Call& c, const float* b) {
    return aligned(b, 4) ? MMQ_OK : refuse(c.fn, MMQ_ERR_ALIGN, "a bias must be 4-byte aligned");
}

}  // namespace
}  // namespace mmq

using namespace mmq;
using namespace mmq::ffn;

extern "C" {

int mmq_project(int fmt, int dtype, const void* x, int64_t x_stride, int64_t M, const void* wq, int64_t N, int64_t K,
                const float* bias, int act, const void* residual, int64_t residual_stride, void* pre, void* out,
                void* stream) {
    const char* fn = "mmq_project";
    Call c;
    int st = check(fn, fmt, dtype, act, M, N, K, wq, nullptr, 1, c);
    if (!st) st = check_x(c, x, x_stride);
    if (!st) st = check_bias(c, bias);
    if (!st && residual) st = check_rows(c, residual, residual_stride, N, "");
    if (!st && pre) st = check_rows(c, pre, N, N, "");
    if (!st) st = check_rows(c, out, N, N, "out must be non-NULL");
    if (st || M == 0) return st;
    c.x = x;
    c.x_stride = x_stride;
    c.bias[0] = bias;
    c.residual = residual;
    c.residual_stride = residual_stride;
    c.pre[0] = pre;
    c.out = out;
    return ffn_launch(c, static_cast<cudaStream_t>(stream));
}

int mmq_gated(int fmt, int dtype, const void* x, int64_t x_stride, int64_t M, const void* w_gate, const void* w_up,
              int64_t N, int64_t K, const float* bias_gate, const float* bias_up, int act, void* gate, void* up, void* out,
              void* stream) {
    const char* fn = "mmq_gated";
    Call c;
    int st = check(fn, fmt, dtype, act, M, N, K, w_gate, w_up, 2, c);
    if (!st) st = check_x(c, x, x_stride);
    if (!st) st = check_bias(c, bias_gate);
    if (!st) st = check_bias(c, bias_up);
    if (!st && gate) st = check_rows(c, gate, N, N, "");
    if (!st && up) st = check_rows(c, up, N, N, "");
    if (!st) st = check_rows(c, out, N, N, "out must be non-NULL");
    if (st || M == 0) return st;
    c.x = x;
    c.x_stride = x_stride;
    c.bias[0] = bias_gate;
    c.bias[1] = bias_up;
    c.pre[0] = gate;
    c.pre[1] = up;
    c.out = out;
    return ffn_launch(c, static_cast<cudaStream_t>(stream));
}

int mmq_project_backward(int fmt, int dtype, const void* dy, int64_t dy_stride, int64_t M, const void* wq, int64_t N,
                         int64_t K, int act, const void* pre, void* dz, void* dx, void* stream) {
    const char* fn = "mmq_project_backward";
    Call c;
    int st = check(fn, fmt, dtype, act, M, N, K, wq, nullptr, 1, c);
    if (!st) st = check_rows(c, dy, dy_stride, N, "dy must be non-NULL");
    if (!st && act != MMQ_ACT_NONE) st = check_rows(c, pre, N, N, "pre must be non-NULL where act is not MMQ_ACT_NONE");
    if (!st && dz) st = check_rows(c, dz, N, N, "");
    if (!st) st = check_rows(c, dx, K, K, "dx must be non-NULL");
    if (st || M == 0) return st;
    c.backward = true;
    c.x = dy;
    c.x_stride = dy_stride;
    c.pre[0] = act != MMQ_ACT_NONE ? const_cast<void*>(pre) : nullptr;
    c.dz[0] = dz;
    c.out = dx;
    return ffn_launch(c, static_cast<cudaStream_t>(stream));
}

int mmq_gated_backward(int fmt, int dtype, const void* dh, int64_t dh_stride, int64_t M, const void* w_gate,
                       const void* w_up, int64_t N, int64_t K, int act, const void* gate, const void* up, void* dgate,
                       void* dup, void* dx, void* stream) {
    const char* fn = "mmq_gated_backward";
    Call c;
    int st = check(fn, fmt, dtype, act, M, N, K, w_gate, w_up, 2, c);
    if (!st) st = check_rows(c, dh, dh_stride, N, "dh must be non-NULL");
    if (!st) st = check_rows(c, gate, N, N, "gate must be non-NULL");
    if (!st) st = check_rows(c, up, N, N, "up must be non-NULL");
    if (!st && dgate) st = check_rows(c, dgate, N, N, "");
    if (!st && dup) st = check_rows(c, dup, N, N, "");
    if (!st) st = check_rows(c, dx, K, K, "dx must be non-NULL");
    if (st || M == 0) return st;
    c.backward = true;
    c.x = dh;
    c.x_stride = dh_stride;
    c.pre[0] = const_cast<void*>(gate);
    c.pre[1] = const_cast<void*>(up);
    c.dz[0] = dgate;
    c.dz[1] = dup;
    c.out = dx;
    return ffn_launch(c, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
