// Entry points of the operators around the module: argument checks on the host, then
// the launches (include/diffuser.h describes each).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "layer_ops.h"
#include "spans.h"
#include "turns.h"

namespace dfs {
namespace {

constexpr int64_t kMaxWidth = 1 << 16;
constexpr int64_t kMaxRows = 1 << 30;        // tile coordinates stay within 32 bits
// ---- norms and rotation ----------------------------------------------------------
int check_qk(int32_t dtype, int64_t B, int64_t Hq, int64_t Hk, int64_t n, int32_t d, float eps, double theta,
             int32_t rotary_dim) {
    if (B < 0 || n < 0 || Hq < 1 || Hk < 1 || B > INT32_MAX || n > INT32_MAX || Hq > 4096 || Hk > 4096)
        return fail(DIFFUSER_ERR_INVALID_ARG, "B, Hq, Hk or n out of range");
    if (d != kHeadDim) return fail(DIFFUSER_ERR_UNSUPPORTED, "head width d must be 64");
    if (dtype != DIFFUSER_DTYPE_FP32 && dtype != DIFFUSER_DTYPE_BF16)
        return fail(DIFFUSER_ERR_UNSUPPORTED, "dtype must be FP32 or BF16");
    if (n > 0 && B > (int64_t(1) << 40) / n) return fail(DIFFUSER_ERR_OVERFLOW, "too many tokens");
    if (!(eps > 0.f) || std::isinf(eps)) return fail(DIFFUSER_ERR_INVALID_ARG, "eps must be positive and finite");
    if (!(theta >= 1.0) || std::isinf(theta)) return fail(DIFFUSER_ERR_INVALID_ARG, "theta must be finite and at least 1");
    if (rotary_dim < 0 || rotary_dim > kHeadDim) return fail(DIFFUSER_ERR_INVALID_ARG, "rotary_dim must lie in [0, d]");
    if (rotary_dim % 16) return fail(DIFFUSER_ERR_UNSUPPORTED, "rotary_dim must be a multiple of 16");
    return DIFFUSER_OK;
}

QkArgs qk_args(const void* Q, const void* K, int64_t B, int64_t Hq, int64_t Hk, int64_t n, const void* wq, const void* wk,
               float eps, double theta, int32_t rot, const int64_t* pos, int64_t pos0) {
    QkArgs a{};
    a.q = Q;
    a.k = K;
    a.wq = wq;
    a.wk = wk;
    a.pos = pos;
    a.pos0 = pos0;
    a.tokens = B * n;
    a.n = n;
    a.Hq = (int32_t)Hq;
    a.Hk = (int32_t)Hk;
    a.rot = rot;
    a.eps = eps;
    if (rot) turns::fill(a.freq, a.freq_low, theta, rot);
    return a;
}

size_t qk_partial_bytes(int64_t tokens, int64_t Hq, int64_t Hk) {
    return tokens ? align256((size_t)qk_backward_blocks(tokens, Hq, Hk) * kHeadDim * sizeof(float)) : 256;
}

// ---- dense products ---------------------------------------------------------------
int check_dense(int64_t T, int64_t D, int64_t F, int32_t act) {
    if (T < 0 || D < 1 || F < 1 || T > kMaxRows) return fail(DIFFUSER_ERR_INVALID_ARG, "T, D or F out of range");
    if (D % 8 || F % 8 || D > kMaxWidth || F > kMaxWidth)
        return fail(DIFFUSER_ERR_UNSUPPORTED, "D and F must be multiples of 8, at most 65536");
    if (act < DIFFUSER_ACT_NONE || act > DIFFUSER_ACT_SILU) return fail(DIFFUSER_ERR_UNSUPPORTED, "unknown activation");
    return DIFFUSER_OK;
}

int zero(void* p, size_t bytes, cudaStream_t stream) {
    if (!p) return DIFFUSER_OK;
    const cudaError_t err = cudaMemsetAsync(p, 0, bytes, stream);
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "zeroing a gradient");
}

// workspace of the dense backward: dP (bf16), then the bias gradient's partial sums
struct DenseBwd {
    size_t dp, partial, total;
};
DenseBwd plan_dense_backward(int64_t T, int64_t F, int32_t act) {
    DenseBwd L{};
    if (T <= kFewBackward) return L;
    const size_t dp = act == DIFFUSER_ACT_NONE ? 0 : align256((size_t)T * F * 2);
    L.partial = dp;
    L.total = dp + align256((size_t)act_chunks(T, (int32_t)F) * F * sizeof(float));
    return L;
}
size_t gated_backward_bytes(int64_t T, int64_t F) { return T <= kFewBackward ? 0 : align256((size_t)T * F * 4); }

// a workspace that may be left out where none is needed
int check_backward_workspace(size_t need, void* ws, size_t ws_bytes) {
    return need ? check_workspace_bytes(need, ws, ws_bytes) : DIFFUSER_OK;
}

// dX = dP W and dW = dP^T X, a (dP, sizes, status) filled in, and what is left of the bias
// gradient; a null result is left out
int launch_both(const DenseArgs& a, const void* W, void* dX, const void* X, void* dW, const BiasSums& bias,
                cudaStream_t stream) {
    DenseArgs x = a, w = a;
    x.b = W;
    x.out = dX;
    w.b = X;
    w.out = dW;
    if (dX && dW) return launch_gradients(x, w, bias, stream);
    if (bias.out)
        if (const int st = launch_colsum(bias, stream)) return st;
    if (dX) return launch_dense(kInputGrad, x, stream);
    if (dW) return launch_dense(kWeightGrad, w, stream);
    return DIFFUSER_OK;
}

}  // namespace

int ready_status(int** word) {
    ProjStatus ps;
    const int st = projection_status(&ps);
    if (st) return st;
    if (*reinterpret_cast<volatile int*>(ps.h) != 0)
        return fail(DIFFUSER_ERR_DEVICE, "a projection or dense product kernel reported a failure (see diffuser_projection_status)");
    *word = ps.d;
    return DIFFUSER_OK;
}

}  // namespace dfs

using namespace dfs;

extern "C" {

int diffuser_qk_norm_rope(const void* Q, const void* K, int32_t dtype, int64_t B, int64_t Hq, int64_t Hk, int64_t n,
                          int32_t d, const void* q_weight, const void* k_weight, float eps, double theta,
                          int32_t rotary_dim, int32_t interleaved, const int64_t* positions, int64_t position_offset,
                          void* Qo, void* Ko, diffuser_stream stream) try {
    int st = check_qk(dtype, B, Hq, Hk, n, d, eps, theta, rotary_dim);
    if (st) return st;
    const size_t e = dtype == DIFFUSER_DTYPE_BF16 ? 2 : 4, row = kHeadDim * e;
    const size_t qb = (size_t)B * Hq * n * row, kb = (size_t)B * Hk * n * row;
    const Span in[5] = {{Q, qb}, {K, kb}, {q_weight, q_weight ? row : 0}, {k_weight, k_weight ? row : 0},
                        {positions, positions ? (size_t)B * n * 8 : 0}};
    const Span out[2] = {{Qo, qb}, {Ko, kb}};
    const int in_place[2] = {0, 1};
    if ((st = check_span(in[0], "Q")) || (st = check_span(in[1], "K")) || (st = check_span(in[2], "q_weight")) ||
        (st = check_span(in[3], "k_weight")) || (st = check_span(in[4], "positions", 8)) ||
        (st = check_span(out[0], "Qo")) || (st = check_span(out[1], "Ko")) ||
        (st = check_overlaps(in, 5, out, 2, in_place)))
        return st;
    if (B * n == 0) return DIFFUSER_OK;
    QkArgs a = qk_args(Q, K, B, Hq, Hk, n, q_weight, k_weight, eps, theta, rotary_dim, positions, position_offset);
    a.qo = Qo;
    a.ko = Ko;
    return launch_qk_norm_rope(a, dtype, interleaved != 0, static_cast<cudaStream_t>(stream));
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_qk_norm_rope_backward_workspace_size(int64_t B, int64_t Hq, int64_t Hk, int64_t n, int32_t d,
                                                  size_t* bytes) try {
    if (!bytes) return fail(DIFFUSER_ERR_INVALID_ARG, "NULL argument");
    const int st = check_qk(DIFFUSER_DTYPE_FP32, B, Hq, Hk, n, d, 1.f, 1.0, 0);
    if (st) return st;
    *bytes = qk_partial_bytes(B * n, Hq, Hk);
    return DIFFUSER_OK;
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_qk_norm_rope_backward(const void* Q, const void* K, const void* dQo, const void* dKo, int32_t dtype,
                                   int64_t B, int64_t Hq, int64_t Hk, int64_t n, int32_t d, const void* q_weight,
                                   const void* k_weight, float eps, double theta, int32_t rotary_dim,
                                   int32_t interleaved, const int64_t* positions, int64_t position_offset, void* dQ,
                                   void* dK, void* dq_weight, void* dk_weight, void* workspace, size_t workspace_bytes,
                                   diffuser_stream stream) try {
    int st = check_qk(dtype, B, Hq, Hk, n, d, eps, theta, rotary_dim);
    if (st) return st;
    const size_t e = dtype == DIFFUSER_DTYPE_BF16 ? 2 : 4, row = kHeadDim * e;
    const size_t qb = (size_t)B * Hq * n * row, kb = (size_t)B * Hk * n * row;
    if ((dq_weight && !q_weight) || (dk_weight && !k_weight))
        return fail(DIFFUSER_ERR_INVALID_ARG, "a weight gradient is asked for without its weight");
    const Span in[7] = {{Q, qb}, {K, kb}, {dQo, qb}, {dKo, kb}, {q_weight, q_weight ? row : 0},
                        {k_weight, k_weight ? row : 0}, {positions, positions ? (size_t)B * n * 8 : 0}};
    const Span out[5] = {{dQ, qb}, {dK, kb}, {dq_weight, dq_weight ? row : 0}, {dk_weight, dk_weight ? row : 0},
                         {workspace, workspace_bytes}};
    const char* names[4] = {"Q", "K", "dQo", "dKo"};
    for (int x = 0; x < 4; ++x)
        if ((st = check_span(in[x], names[x]))) return st;
    if ((st = check_span(in[4], "q_weight")) || (st = check_span(in[5], "k_weight")) ||
        (st = check_span(in[6], "positions", 8)) || (st = check_span(out[0], "dQ")) || (st = check_span(out[1], "dK")) ||
        (st = check_span(out[2], "dq_weight")) || (st = check_span(out[3], "dk_weight")) ||
        (st = check_workspace_bytes(qk_partial_bytes(B * n, Hq, Hk), workspace, workspace_bytes)) ||
        (st = check_overlaps(in, 7, out, 5)))
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B * n == 0) {
        if ((st = zero(dq_weight, row, s))) return st;
        return zero(dk_weight, row, s);
    }
    QkArgs a = qk_args(Q, K, B, Hq, Hk, n, q_weight, k_weight, eps, theta, rotary_dim, positions, position_offset);
    a.dqo = dQo;
    a.dko = dKo;
    a.qo = dQ;
    a.ko = dK;
    a.partial = dq_weight || dk_weight ? static_cast<float*>(workspace) : nullptr;
    return launch_qk_norm_rope_backward(a, dtype, interleaved != 0, dq_weight, dk_weight, s);
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_linear(const void* X, const void* W, const void* bias, const void* residual, int64_t T, int32_t D,
                    int32_t F, int32_t activation, void* Y, void* pre, diffuser_stream stream) try {
    int st = check_dense(T, D, F, activation);
    if (st) return st;
    const size_t yb = (size_t)T * F * 2;
    const Span in[4] = {{X, (size_t)T * D * 2}, {W, (size_t)F * D * 2}, {bias, bias ? (size_t)F * 2 : 0},
                        {residual, residual ? yb : 0}};
    const Span out[2] = {{Y, yb}, {pre, pre ? yb : 0}};
    const int in_place[2] = {3, -1};
    if ((st = check_span(in[0], "X")) || (st = check_span(in[1], "W")) || (st = check_span(in[2], "bias")) ||
        (st = check_span(in[3], "residual")) || (st = check_span(out[0], "Y")) || (st = check_span(out[1], "pre")) ||
        (st = check_overlaps(in, 4, out, 2, in_place)))
        return st;
    if (T == 0) return DIFFUSER_OK;
    DenseArgs a{};
    if ((st = ready_status(&a.status))) return st;
    a.a = X;
    a.b = W;
    a.rows = T;
    a.inner = D;
    a.cols = F;
    a.out = Y;
    a.pre = pre;
    a.bias = bias;
    a.residual = residual;
    a.act = activation;
    return launch_dense(kForward, a, static_cast<cudaStream_t>(stream));
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_linear_backward_workspace_size(int64_t T, int32_t D, int32_t F, int32_t activation,
                                            size_t* bytes) try {
    if (!bytes) return fail(DIFFUSER_ERR_INVALID_ARG, "NULL argument");
    const int st = check_dense(T, D, F, activation);
    if (st) return st;
    *bytes = plan_dense_backward(T, F, activation).total;
    return DIFFUSER_OK;
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_linear_backward(const void* X, const void* W, const void* dY, const void* pre, int64_t T, int32_t D,
                             int32_t F, int32_t activation, void* dX, void* dW, void* dbias, void* workspace,
                             size_t workspace_bytes, diffuser_stream stream) try {
    int st = check_dense(T, D, F, activation);
    if (st) return st;
    const bool has_act = activation != DIFFUSER_ACT_NONE;
    const size_t xb = (size_t)T * D * 2, wb = (size_t)F * D * 2, yb = (size_t)T * F * 2;
    const Span in[4] = {{X, xb}, {W, wb}, {dY, yb}, {pre, has_act ? yb : 0}};
    const Span out[4] = {{dX, dX ? xb : 0}, {dW, dW ? wb : 0}, {dbias, dbias ? (size_t)F * 2 : 0},
                         {workspace, workspace_bytes}};
    const DenseBwd L = plan_dense_backward(T, F, activation);
    if ((st = check_span(in[0], "X")) || (st = check_span(in[1], "W")) || (st = check_span(in[2], "dY")) ||
        (st = check_span(in[3], "pre")) || (st = check_span(out[0], "dX")) || (st = check_span(out[1], "dW")) ||
        (st = check_span(out[2], "dbias")) || (st = check_backward_workspace(L.total, workspace, workspace_bytes)) ||
        (st = check_overlaps(in, 4, out, 4)))
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if ((st = zero(dW, wb, s))) return st;
        return zero(dbias, (size_t)F * 2, s);
    }
    if (!dX && !dW && !dbias) return DIFFUSER_OK;
    DenseArgs a{};
    if ((st = ready_status(&a.status))) return st;
    if (T <= kFewBackward) return launch_few_backward(X, W, dY, pre, T, D, F, activation, false, dX, dW, dbias, s);
    char* ws = static_cast<char*>(workspace);
    const void* dP = has_act ? ws + L.dp : dY;
    BiasSums bias{};
    if (dbias || (has_act && (dX || dW)))
        if ((st = launch_act_backward(dY, pre, T, F, activation, has_act ? ws + L.dp : nullptr, dbias,
                                      reinterpret_cast<float*>(ws + L.partial), &bias, s)))
            return st;
    a.a = dP;
    a.rows = T;
    a.inner = D;
    a.cols = F;
    return launch_both(a, W, dX, X, dW, bias, s);
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_gated_linear(const void* X, const void* Wgu, int64_t T, int32_t D, int32_t F, int32_t activation, void* H,
                          void* pre, diffuser_stream stream) try {
    int st = check_dense(T, D, F, activation);
    if (st) return st;
    const size_t hb = (size_t)T * F * 2;
    const Span in[2] = {{X, (size_t)T * D * 2}, {Wgu, (size_t)2 * F * D * 2}};
    const Span out[2] = {{H, hb}, {pre, pre ? 2 * hb : 0}};
    if ((st = check_span(in[0], "X")) || (st = check_span(in[1], "Wgu")) || (st = check_span(out[0], "H")) ||
        (st = check_span(out[1], "pre")) || (st = check_overlaps(in, 2, out, 2)))
        return st;
    if (T == 0) return DIFFUSER_OK;
    DenseArgs a{};
    if ((st = ready_status(&a.status))) return st;
    a.a = X;
    a.b = Wgu;
    a.rows = T;
    a.inner = D;
    a.cols = 2 * F;
    a.out = H;
    a.pre = pre;
    a.act = activation;
    a.gated = true;
    return launch_dense(kForward, a, static_cast<cudaStream_t>(stream));
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_gated_linear_backward_workspace_size(int64_t T, int32_t D, int32_t F, size_t* bytes) try {
    if (!bytes) return fail(DIFFUSER_ERR_INVALID_ARG, "NULL argument");
    const int st = check_dense(T, D, F, DIFFUSER_ACT_NONE);
    if (st) return st;
    *bytes = gated_backward_bytes(T, F);
    return DIFFUSER_OK;
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_gated_linear_backward(const void* X, const void* Wgu, const void* dH, const void* pre, int64_t T,
                                   int32_t D, int32_t F, int32_t activation, void* dX, void* dWgu, void* workspace,
                                   size_t workspace_bytes, diffuser_stream stream) try {
    int st = check_dense(T, D, F, activation);
    if (st) return st;
    const size_t xb = (size_t)T * D * 2, wb = (size_t)2 * F * D * 2, hb = (size_t)T * F * 2;
    const Span in[4] = {{X, xb}, {Wgu, wb}, {dH, hb}, {pre, 2 * hb}};
    const Span out[3] = {{dX, dX ? xb : 0}, {dWgu, dWgu ? wb : 0}, {workspace, workspace_bytes}};
    if ((st = check_span(in[0], "X")) || (st = check_span(in[1], "Wgu")) || (st = check_span(in[2], "dH")) ||
        (st = check_span(in[3], "pre")) || (st = check_span(out[0], "dX")) || (st = check_span(out[1], "dWgu")) ||
        (st = check_backward_workspace(gated_backward_bytes(T, F), workspace, workspace_bytes)) || (st = check_overlaps(in, 4, out, 3)))
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return zero(dWgu, wb, s);
    if (!dX && !dWgu) return DIFFUSER_OK;
    DenseArgs a{};
    if ((st = ready_status(&a.status))) return st;
    if (T <= kFewBackward) return launch_few_backward(X, Wgu, dH, pre, T, D, F, activation, true, dX, dWgu, nullptr, s);
    if ((st = launch_gated_backward(dH, pre, T, F, activation, workspace, s))) return st;
    a.a = workspace;
    a.rows = T;
    a.inner = D;
    a.cols = 2 * F;
    return launch_both(a, Wgu, dX, X, dWgu, BiasSums{}, s);
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

}  // extern "C"
