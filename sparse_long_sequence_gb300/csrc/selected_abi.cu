// Entry points of the rotation alone and of the attention over chosen key blocks: argument checks
// on the host, then the launches (include/diffuser.h describes each).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "layer_ops.h"
#include "selected.h"
#include "spans.h"
#include "turns.h"

namespace dfs {
namespace {

// ---- the rotation alone -------------------------------------------------------------
int check_rope(int32_t dtype, int64_t B, int64_t Hq, int64_t Hk, int64_t n, int32_t d, const double* frequencies,
               int32_t rotary_dim, float magnitude) {
    if (B < 0 || n < 0 || Hq < 1 || Hk < 1 || B > INT32_MAX || n > INT32_MAX || Hq > 4096 || Hk > 4096)
        return fail(DIFFUSER_ERR_INVALID_ARG, "B, Hq, Hk or n out of range");
    if (d != kHeadDim) return fail(DIFFUSER_ERR_UNSUPPORTED, "head width d must be 64");
    if (dtype != DIFFUSER_DTYPE_FP32 && dtype != DIFFUSER_DTYPE_BF16)
        return fail(DIFFUSER_ERR_UNSUPPORTED, "dtype must be FP32 or BF16");
    if (n > 0 && B > (int64_t(1) << 40) / n) return fail(DIFFUSER_ERR_OVERFLOW, "too many tokens");
    if (rotary_dim < 1 || rotary_dim > kHeadDim) return fail(DIFFUSER_ERR_INVALID_ARG, "rotary_dim must lie in [1, d]");
    if (rotary_dim % 16) return fail(DIFFUSER_ERR_UNSUPPORTED, "rotary_dim must be a multiple of 16");
    if (!frequencies) return fail(DIFFUSER_ERR_INVALID_ARG, "frequencies is NULL");
    for (int i = 0; i < rotary_dim / 2; ++i)
        if (!(frequencies[i] >= 0.0 && frequencies[i] <= 4.0))
            return fail(DIFFUSER_ERR_INVALID_ARG, "a frequency lies outside [0, 4]");
    if (!(magnitude > 0.f) || std::isinf(magnitude))
        return fail(DIFFUSER_ERR_INVALID_ARG, "magnitude must be positive and finite");
    return DIFFUSER_OK;
}

int rope(const char* const (&names)[4], const void* Q, const void* K, int32_t dtype, int64_t B, int64_t Hq, int64_t Hk,
         int64_t n, int32_t d, const double* frequencies, int32_t rotary_dim, int32_t interleaved, float magnitude,
         const int64_t* positions, int64_t position_offset, bool back, void* Qo, void* Ko, diffuser_stream stream) {
    int st = check_rope(dtype, B, Hq, Hk, n, d, frequencies, rotary_dim, magnitude);
    if (st) return st;
    const size_t row = kHeadDim * (dtype == DIFFUSER_DTYPE_BF16 ? 2 : 4);
    const size_t qb = (size_t)B * Hq * n * row, kb = (size_t)B * Hk * n * row;
    const Span in[3] = {{Q, qb}, {K, kb}, {positions, positions ? (size_t)B * n * 8 : 0}};
    const Span out[2] = {{Qo, qb}, {Ko, kb}};
    const int in_place[2] = {0, 1};
    if ((st = check_span(in[0], names[0])) || (st = check_span(in[1], names[1])) ||
        (st = check_span(in[2], "positions", 8)) || (st = check_span(out[0], names[2])) ||
        (st = check_span(out[1], names[3])) || (st = check_overlaps(in, 3, out, 2, in_place)))
        return st;
    if (B * n == 0) return DIFFUSER_OK;
    QkArgs a{};
    a.q = Q;
    a.k = K;
    a.qo = Qo;
    a.ko = Ko;
    a.pos = positions;
    a.pos0 = position_offset;
    a.tokens = B * n;
    a.n = n;
    a.Hq = (int32_t)Hq;
    a.Hk = (int32_t)Hk;
    a.rot = rotary_dim;
    a.magnitude = magnitude;
    turns::fill_given(a.freq, a.freq_low, frequencies, rotary_dim / 2);
    return launch_rope(a, dtype, interleaved != 0, back, static_cast<cudaStream_t>(stream));
}

// ---- attention over chosen blocks -----------------------------------------------------
// Sizes that the calls share, into *s (lengths, starts and causal are the caller's to add).
int check_selected(int64_t B, int64_t Hq, int64_t Hk, int64_t n, int64_t m, int32_t d, int64_t top, SelectShape* s) {
    if (B < 0 || n < 0 || m < 0 || Hq < 1 || Hk < 1 || B > INT32_MAX || Hq > 4096)
        return fail(DIFFUSER_ERR_INVALID_ARG, "B, Hq, Hk, n or m out of range");
    if (Hq % Hk) return fail(DIFFUSER_ERR_INVALID_ARG, "Hq must be a multiple of Hk");
    if (d != kHeadDim) return fail(DIFFUSER_ERR_UNSUPPORTED, "head width d must be 64");
    if (top < 1 || top > kMaxTop) return fail(DIFFUSER_ERR_UNSUPPORTED, "top_k must lie in [1, 64]");
    if (m > kMaxKeys || n > kMaxKeys) return fail(DIFFUSER_ERR_UNSUPPORTED, "more than 2^20 queries or keys");
    if (n && B * Hq > (int64_t(1) << 40) / (n * top)) return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
    if (m && B * Hk > (int64_t(1) << 40) / m) return fail(DIFFUSER_ERR_OVERFLOW, "too many keys");
    if (n * (Hq / Hk) * top > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many queries of a key head");
    *s = SelectShape{};
    s->B = B;
    s->n = n;
    s->m = m;
    s->Hq = (int32_t)Hq;
    s->Hk = (int32_t)Hk;
    s->G = (int32_t)(Hq / Hk);
    s->top = (int32_t)top;
    s->nb = (int32_t)((m + kBlockKeys - 1) / kBlockKeys);
    return DIFFUSER_OK;
}

size_t rows_bytes(const SelectShape& s) { return (size_t)s.B * s.Hq * s.n * kHeadDim * 2; }
size_t keys_bytes(const SelectShape& s) { return (size_t)s.B * s.Hk * s.m * kHeadDim * 2; }
size_t list_bytes(const SelectShape& s) { return (size_t)s.B * s.Hk * s.n * s.top * 4; }
Span per_sequence(const int32_t* p, int64_t B) { return {p, p ? (size_t)B * 4 : 0}; }

}  // namespace
}  // namespace dfs

using namespace dfs;

extern "C" {

int diffuser_rope_frequencies(int32_t scaling, double theta, int32_t rotary_dim, double factor, double original_length,
                              double* frequencies, double* magnitude) try {
    if (!frequencies || !magnitude) return fail(DIFFUSER_ERR_INVALID_ARG, "NULL argument");
    if (scaling < DIFFUSER_ROPE_NONE || scaling > DIFFUSER_ROPE_YARN)
        return fail(DIFFUSER_ERR_UNSUPPORTED, "unknown scaling");
    if (!(theta >= 1.0) || std::isinf(theta)) return fail(DIFFUSER_ERR_INVALID_ARG, "theta must be finite and at least 1");
    if (rotary_dim < 1 || rotary_dim > kHeadDim) return fail(DIFFUSER_ERR_INVALID_ARG, "rotary_dim must lie in [1, d]");
    if (rotary_dim % 16) return fail(DIFFUSER_ERR_UNSUPPORTED, "rotary_dim must be a multiple of 16");
    if (scaling != DIFFUSER_ROPE_NONE && (!(factor >= 1.0) || std::isinf(factor)))
        return fail(DIFFUSER_ERR_INVALID_ARG, "factor must be finite and at least 1");
    if (scaling == DIFFUSER_ROPE_YARN && (!(original_length > 0.0) || std::isinf(original_length)))
        return fail(DIFFUSER_ERR_INVALID_ARG, "original_length must be positive and finite");
    const double r = rotary_dim;
    const double base = scaling == DIFFUSER_ROPE_NTK ? theta * std::pow(factor, r / (r - 2)) : theta;
    if (std::isinf(base)) return fail(DIFFUSER_ERR_INVALID_ARG, "theta and factor are too large");
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / r);
        if (scaling == DIFFUSER_ROPE_LINEAR) f /= factor;
        if (scaling == DIFFUSER_ROPE_YARN) {
            constexpr double kTurn = 6.283185307179586, kSlow = 1.0, kFast = 32.0;
            double keep = (original_length * f / kTurn - kSlow) / (kFast - kSlow);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f *= keep + (1.0 - keep) / factor;
        }
        frequencies[i] = f;
    }
    *magnitude = scaling == DIFFUSER_ROPE_YARN ? 1.0 + 0.1 * std::log(factor) : 1.0;
    return DIFFUSER_OK;
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_rope(const void* Q, const void* K, int32_t dtype, int64_t B, int64_t Hq, int64_t Hk, int64_t n, int32_t d,
                  const double* frequencies, int32_t rotary_dim, int32_t interleaved, float magnitude,
                  const int64_t* positions, int64_t position_offset, void* Qo, void* Ko, diffuser_stream stream) try {
    return rope({"Q", "K", "Qo", "Ko"}, Q, K, dtype, B, Hq, Hk, n, d, frequencies, rotary_dim, interleaved, magnitude,
                positions, position_offset, false, Qo, Ko, stream);
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_rope_backward(const void* dQo, const void* dKo, int32_t dtype, int64_t B, int64_t Hq, int64_t Hk,
                           int64_t n, int32_t d, const double* frequencies, int32_t rotary_dim, int32_t interleaved,
                           float magnitude, const int64_t* positions, int64_t position_offset, void* dQ, void* dK,
                           diffuser_stream stream) try {
    return rope({"dQo", "dKo", "dQ", "dK"}, dQo, dKo, dtype, B, Hq, Hk, n, d, frequencies, rotary_dim, interleaved,
                magnitude, positions, position_offset, true, dQ, dK, stream);
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_block_means(const void* K, int64_t B, int64_t Hk, int64_t m, int32_t d, const int32_t* lengths,
                         int64_t recent, void* means, diffuser_stream stream) try {
    SelectShape s;
    int st = check_selected(B, Hk, Hk, 0, m, d, 1, &s);
    if (st) return st;
    if (recent < 0) return fail(DIFFUSER_ERR_INVALID_ARG, "recent must not be negative");
    const Span in[2] = {{K, keys_bytes(s)}, per_sequence(lengths, B)};
    const Span out[1] = {{means, (size_t)B * Hk * s.nb * kHeadDim * 2}};
    if ((st = check_span(in[0], "K")) || (st = check_span(in[1], "lengths", 4)) || (st = check_span(out[0], "means")) ||
        (st = check_overlaps(in, 2, out, 1)))
        return st;
    if (B * m == 0) return DIFFUSER_OK;
    return launch_block_means(K, B, Hk, m, lengths, recent < m ? recent : m, means, static_cast<cudaStream_t>(stream));
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_select_blocks(const void* Q, const void* means, int64_t B, int64_t Hq, int64_t Hk, int64_t n, int64_t m,
                           int32_t d, int32_t top_k, int32_t sink_blocks, int32_t local_blocks, int32_t causal,
                           const int32_t* lengths, const int32_t* starts, int32_t* blocks, diffuser_stream stream) try {
    SelectShape s;
    int st = check_selected(B, Hq, Hk, n, m, d, top_k, &s);
    if (st) return st;
    if (sink_blocks < 0 || local_blocks < 0)
        return fail(DIFFUSER_ERR_INVALID_ARG, "sink_blocks and local_blocks must not be negative");
    const int64_t near = causal || !local_blocks ? local_blocks : 2 * (int64_t)local_blocks - 1;
    if (sink_blocks + near > top_k) return fail(DIFFUSER_ERR_INVALID_ARG, "more forced blocks than top_k");
    s.causal = causal != 0;
    s.lengths = lengths;
    s.starts = starts;
    const Span in[4] = {{Q, rows_bytes(s)}, {means, (size_t)B * Hk * s.nb * kHeadDim * 2}, per_sequence(lengths, B),
                        per_sequence(starts, B)};
    const Span out[1] = {{blocks, list_bytes(s)}};
    if ((st = check_span(in[0], "Q")) || (st = check_span(in[1], "means")) || (st = check_span(in[2], "lengths", 4)) ||
        (st = check_span(in[3], "starts", 4)) || (st = check_span(out[0], "blocks")) || (st = check_overlaps(in, 4, out, 1)))
        return st;
    if (B * n == 0) return DIFFUSER_OK;
    return launch_select_blocks(s, Q, means, sink_blocks, local_blocks, blocks, static_cast<cudaStream_t>(stream));
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_selected_attention_workspace_size(int64_t B, int64_t Hq, int64_t Hk, int64_t n, int64_t m, int32_t d,
                                               int32_t top_k, size_t* bytes) try {
    if (!bytes) return fail(DIFFUSER_ERR_INVALID_ARG, "NULL argument");
    SelectShape s;
    const int st = check_selected(B, Hq, Hk, n, m, d, top_k, &s);
    if (st) return st;
    *bytes = selected_workspace(s);
    return DIFFUSER_OK;
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_selected_attention(const void* Q, const void* K, const void* V, const int32_t* blocks, int64_t B,
                                int64_t Hq, int64_t Hk, int64_t n, int64_t m, int32_t d, int32_t top_k, int32_t causal,
                                const int32_t* lengths, const int32_t* starts, void* out, float* lse, void* workspace,
                                size_t workspace_bytes, diffuser_stream stream) try {
    SelectedArgs a{};
    int st = check_selected(B, Hq, Hk, n, m, d, top_k, &a.s);
    if (st) return st;
    const SelectShape& s = a.s;
    a.s.causal = causal != 0;
    a.s.lengths = lengths;
    a.s.starts = starts;
    const size_t qb = rows_bytes(s), need = selected_workspace(s);
    const Span in[6] = {{Q, qb}, {K, keys_bytes(s)}, {V, keys_bytes(s)}, {blocks, list_bytes(s)}, per_sequence(lengths, B),
                        per_sequence(starts, B)};
    const Span outs[3] = {{out, qb}, {lse, lse ? qb / 32 : 0}, {workspace, workspace_bytes}};
    if ((st = check_span(in[0], "Q")) || (st = check_span(in[1], "K")) || (st = check_span(in[2], "V")) ||
        (st = check_span(in[3], "blocks")) || (st = check_span(in[4], "lengths", 4)) ||
        (st = check_span(in[5], "starts", 4)) || (st = check_span(outs[0], "out")) || (st = check_span(outs[1], "lse")) ||
        (need && (st = check_workspace_bytes(need, workspace, workspace_bytes))) || (st = check_overlaps(in, 6, outs, 3)))
        return st;
    if (B * n == 0) return DIFFUSER_OK;
    a.q = static_cast<const __nv_bfloat16*>(Q);
    a.k = static_cast<const __nv_bfloat16*>(K);
    a.v = static_cast<const __nv_bfloat16*>(V);
    a.blocks = blocks;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    return launch_selected(a, static_cast<char*>(workspace), static_cast<cudaStream_t>(stream));
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_selected_attention_backward_workspace_size(int64_t B, int64_t Hq, int64_t Hk, int64_t n, int64_t m,
                                                        int32_t d, int32_t top_k, size_t* bytes) try {
    if (!bytes) return fail(DIFFUSER_ERR_INVALID_ARG, "NULL argument");
    SelectShape s;
    const int st = check_selected(B, Hq, Hk, n, m, d, top_k, &s);
    if (st) return st;
    *bytes = selected_backward_workspace(s);
    return DIFFUSER_OK;
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

int diffuser_selected_attention_backward(const void* Q, const void* K, const void* V, const int32_t* blocks,
                                         const void* out, const float* lse, const void* dOut, int64_t B, int64_t Hq,
                                         int64_t Hk, int64_t n, int64_t m, int32_t d, int32_t top_k, int32_t causal,
                                         const int32_t* lengths, const int32_t* starts, void* dQ, void* dK, void* dV,
                                         void* workspace, size_t workspace_bytes, diffuser_stream stream) try {
    SelectedArgs a{};
    int st = check_selected(B, Hq, Hk, n, m, d, top_k, &a.s);
    if (st) return st;
    const SelectShape& s = a.s;
    a.s.causal = causal != 0;
    a.s.lengths = lengths;
    a.s.starts = starts;
    const size_t qb = rows_bytes(s), kb = keys_bytes(s), need = selected_backward_workspace(s);
    const Span in[9] = {{Q, qb}, {K, kb}, {V, kb}, {blocks, list_bytes(s)}, {out, qb}, {lse, qb / 32}, {dOut, qb},
                        per_sequence(lengths, B), per_sequence(starts, B)};
    const Span outs[4] = {{dQ, qb}, {dK, kb}, {dV, kb}, {workspace, workspace_bytes}};
    const char* names[7] = {"Q", "K", "V", "blocks", "out", "lse", "dOut"};
    for (int x = 0; x < 7; ++x)
        if ((st = check_span(in[x], names[x]))) return st;
    if ((st = check_span(in[7], "lengths", 4)) || (st = check_span(in[8], "starts", 4)) ||
        (st = check_span(outs[0], "dQ")) || (st = check_span(outs[1], "dK")) || (st = check_span(outs[2], "dV")) ||
        (need && (st = check_workspace_bytes(need, workspace, workspace_bytes))) || (st = check_overlaps(in, 9, outs, 4)))
        return st;
    const cudaStream_t stream_ = static_cast<cudaStream_t>(stream);
    if (qb == 0 || kb == 0) {                // no query lists a key
        for (const Span& g : {outs[0], outs[1], outs[2]})
            if (g.bytes) {
                const cudaError_t err = cudaMemsetAsync(const_cast<void*>(g.p), 0, g.bytes, stream_);
                if (err != cudaSuccess) return cuda_fail(err, "zeroing a gradient");
            }
        return DIFFUSER_OK;
    }
    a.q = static_cast<const __nv_bfloat16*>(Q);
    a.k = static_cast<const __nv_bfloat16*>(K);
    a.v = static_cast<const __nv_bfloat16*>(V);
    a.blocks = blocks;
    a.out = static_cast<__nv_bfloat16*>(const_cast<void*>(out));
    a.lse = const_cast<float*>(lse);
    a.dout = static_cast<const __nv_bfloat16*>(dOut);
    a.dq = static_cast<__nv_bfloat16*>(dQ);
    a.dk = static_cast<__nv_bfloat16*>(dK);
    a.dv = static_cast<__nv_bfloat16*>(dV);
    return launch_selected_backward(a, static_cast<char*>(workspace), stream_);
} catch (...) {
    return fail(DIFFUSER_ERR_ALLOC, "unexpected exception");
}

}  // extern "C"
