// api.cu -- the extern "C" boundary declared in include/qlora_nf4.h: argument checks,
// size queries, path selection (few-token decode kernels or the tcgen05 GEMM) and launches.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <string>

#include "../../include/qlora_nf4.h"
#include "act8.h"
#include "int4.h"
#include "kernels.h"

namespace qn {

thread_local uint64_t g_launches = 0;
thread_local std::string g_err;

void count_launch(int n) { g_launches += static_cast<uint64_t>(n); }

namespace {

qn_status fail(qn_status s, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_err = buf;
    return s;
}

qn_status cuda_status(cudaError_t e, const char *what) {
    if (e == cudaSuccess) {
        g_err.clear();
        return QN_OK;
    }
    return fail(QN_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

qn_status check_shape(int64_t n, int64_t k) {
    if (n < 0 || k < 0) return fail(QN_EINVAL, "negative size n_out=%lld k_in=%lld", (long long)n, (long long)k);
    if (k % QN_BLOCK != 0) return fail(QN_ESHAPE, "k_in=%lld is not a multiple of %d", (long long)k, QN_BLOCK);
    if (n > kMaxDim || k > kMaxDim) return fail(QN_ESHAPE, "n_out or k_in above 2^31-1");
    if (n > 0 && k > 0 && (n * k) / QN_BLOCK >= (int64_t(1) << 40))
        return fail(QN_ESHAPE, "more than 2^40 blocks");
    return QN_OK;
}

qn_status check_weight(const qn_nf4_weight *w) {
    if (!w) return fail(QN_EINVAL, "null weight struct");
    qn_status s = check_shape(w->n_out, w->k_in);
    if (s != QN_OK) return s;
    if (w->quant_type != QN_QUANT_NF4 && w->quant_type != QN_QUANT_FP4)
        return fail(QN_EINVAL, "unknown quant_type %d", w->quant_type);
    if (w->const_format != QN_CONST_DQ && w->const_format != QN_CONST_F32)
        return fail(QN_EINVAL, "unknown const_format %d", w->const_format);
    if (w->n_out == 0 || w->k_in == 0) return QN_OK;
    if (w->const_format == QN_CONST_F32) {
        if (!w->codes || !w->absmax) return fail(QN_EINVAL, "null pointer in the quantised weight");
        if (!aligned16(w->codes) || !aligned16(w->absmax)) return fail(QN_EALIGN, "codes or absmax not 16-byte aligned");
        return QN_OK;
    }
    if (!w->codes || !w->absmax_q || !w->group_scale || !w->absmax_mean)
        return fail(QN_EINVAL, "null pointer in the quantised weight");
    if (!aligned16(w->codes) || !aligned16(w->absmax_q) || !aligned16(w->group_scale))
        return fail(QN_EALIGN, "codes, absmax_q or group_scale not 16-byte aligned");
    return QN_OK;
}

WeightView view(const qn_nf4_weight *w) {
    const bool f32 = w->const_format == QN_CONST_F32;
    return WeightView{w->n_out,
                      w->k_in,
                      w->codes,
                      f32 ? nullptr : w->absmax_q,
                      f32 ? nullptr : w->group_scale,
                      f32 ? nullptr : w->absmax_mean,
                      w->quant_type == QN_QUANT_FP4 ? 1 : 0,
                      f32 ? w->absmax : nullptr};
}

qn_status launch_quantize_into(const void *W, const qn_nf4_weight *out, void *ws, cudaStream_t st) {
    const bool f32 = out->const_format == QN_CONST_F32;
    return cuda_status(launch_quantize(static_cast<const uint16_t *>(W), out->n_out, out->k_in,
                                       out->quant_type == QN_QUANT_FP4 ? 1 : 0, out->codes,
                                       f32 ? nullptr : out->absmax_q, f32 ? nullptr : out->group_scale,
                                       f32 ? nullptr : out->absmax_mean, f32 ? out->absmax : nullptr, ws, st),
                       "nf4_quantize");
}

qn_status check_lora(const void *A, const void *B, int r, float alpha) {
    if (r < 0 || r > QN_MAX_RANK) return fail(QN_EINVAL, "rank r=%d outside [0, %d]", r, QN_MAX_RANK);
    if (r == 0) {
        if (A || B) return fail(QN_EINVAL, "r == 0 requires A == B == NULL");
        return QN_OK;
    }
    if (!A || !B) return fail(QN_EINVAL, "null adapter pointer with r=%d", r);
    if (!aligned16(A) || !aligned16(B)) return fail(QN_EALIGN, "A or B not 16-byte aligned");
    if (!(alpha == alpha) || alpha - alpha != 0.0f) return fail(QN_EINVAL, "alpha is not finite");
    return QN_OK;
}

// The kernels' mask parameters and the adapter scale under dropout (s / (1 - p)); off when d is
// null, p == 0 or there is no adapter.
qn_status resolve_dropout(const qn_lora_dropout *d, int r, float sc, DropoutArgs *drop, float *sc_eff) {
    *drop = DropoutArgs{0, 0, 0};
    *sc_eff = sc;
    if (!d || d->p == 0.0f || r == 0) return QN_OK;
    if (!(d->p > 0.0f && d->p < 1.0f)) return fail(QN_EINVAL, "dropout rate p=%g outside [0, 1)", (double)d->p);
    const double thr = floor(static_cast<double>(d->p) * 4294967296.0);
    *drop = DropoutArgs{d->seed, d->offset, static_cast<uint32_t>(thr)};
    *sc_eff = static_cast<float>(static_cast<double>(sc) / (1.0 - static_cast<double>(d->p)));
    return QN_OK;
}

bool aligned2(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

// A buffer of an entry point and whether the call writes it.
struct Span {
    const void *p;
    size_t bytes;
    bool written;
};

// Whether a written buffer shares a byte with any other.
template <int N>
bool overlap(const Span (&s)[N]) {
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j) {
            if (i == j || !s[i].written || !s[i].p || !s[j].p || s[i].bytes == 0 || s[j].bytes == 0) continue;
            const uintptr_t a = reinterpret_cast<uintptr_t>(s[i].p), b = reinterpret_cast<uintptr_t>(s[j].p);
            if (a < b + s[j].bytes && b < a + s[i].bytes) return true;
        }
    return false;
}

// rows x cols of an activation: both in range, cols a multiple of 64.
qn_status check_act8_shape(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return fail(QN_EINVAL, "negative size rows=%lld cols=%lld", (long long)rows, (long long)cols);
    if (cols % QN_BLOCK != 0) return fail(QN_ESHAPE, "cols=%lld is not a multiple of %d", (long long)cols, QN_BLOCK);
    if (rows > kMaxDim || cols > kMaxDim) return fail(QN_ESHAPE, "rows or cols above 2^31-1");
    if (rows > 0 && cols > 0 && rows * cols >= (int64_t(1) << 42)) return fail(QN_ESHAPE, "more than 2^42 values");
    return QN_OK;
}

qn_status check_act8(const qn_act8 *a, const char *name) {
    if (!a) return fail(QN_EINVAL, "null %s", name);
    qn_status s = check_act8_shape(a->rows, a->cols);
    if (s != QN_OK || a->rows == 0 || a->cols == 0) return s;
    if (!a->codes || !a->absmax) return fail(QN_EINVAL, "null buffer in %s", name);
    if (!aligned16(a->codes) || !aligned2(a->absmax))
        return fail(QN_EALIGN, "%s: codes not 16-byte or absmax not 2-byte aligned", name);
    return QN_OK;
}

size_t act8_values(const qn_act8 *a) { return static_cast<size_t>(a->rows) * static_cast<size_t>(a->cols); }
size_t act8_blocks(const qn_act8 *a) { return act8_values(a) / QN_BLOCK; }

qn_status check_int4_shape(int64_t n, int64_t k, int group) {
    if (group != 32 && group != 64 && group != 128) return fail(QN_EINVAL, "group=%d is not 32, 64 or 128", group);
    qn_status s = check_shape(n, k);
    if (s != QN_OK) return s;
    if (k % group != 0) return fail(QN_ESHAPE, "k_in=%lld is not a multiple of group=%d", (long long)k, group);
    if (n > 0 && k > 0 && n * k >= (int64_t(1) << 42)) return fail(QN_ESHAPE, "more than 2^42 weights");
    return QN_OK;
}

qn_status check_int4(const qn_int4_weight *w) {
    if (!w) return fail(QN_EINVAL, "null weight struct");
    qn_status s = check_int4_shape(w->n_out, w->k_in, w->group);
    if (s != QN_OK || w->n_out == 0 || w->k_in == 0) return s;
    if (!w->codes || !w->scale) return fail(QN_EINVAL, "null pointer in the quantised weight");
    if (!aligned16(w->codes) || !aligned2(w->scale))
        return fail(QN_EALIGN, "codes not 16-byte or scale not 2-byte aligned");
    return QN_OK;
}

Int4View view(const qn_int4_weight *w) {
    return Int4View{w->n_out, w->k_in, w->group, w->codes, w->scale, w->zero_point};
}

}  // namespace
}  // namespace qn

using namespace qn;

extern "C" {

const char *qn_status_string(qn_status s) {
    switch (s) {
        case QN_OK: return "ok";
        case QN_EINVAL: return "invalid argument";
        case QN_ESHAPE: return "unsupported shape";
        case QN_EALIGN: return "misaligned pointer";
        case QN_ECUDA: return "CUDA error";
        case QN_EWORKSPACE: return "workspace missing or too small";
        case QN_ETIMEOUT: return "a kernel gave up a bounded wait";
    }
    return "unknown status";
}

const char *qn_last_error(void) { return g_err.c_str(); }

uint64_t qn_launch_count(int reset) {
    const uint64_t v = g_launches;
    if (reset) g_launches = 0;
    return v;
}

qn_status qn_nf4_sizes(int64_t n_out, int64_t k_in, size_t *codes_bytes, size_t *absmax_bytes, size_t *scale_bytes,
                       size_t *mean_bytes) {
    if (!codes_bytes || !absmax_bytes || !scale_bytes || !mean_bytes) return fail(QN_EINVAL, "null output pointer");
    qn_status s = check_shape(n_out, k_in);
    if (s != QN_OK) return s;
    const int64_t nb = n_out * k_in / QN_BLOCK;
    *codes_bytes = static_cast<size_t>(n_out * k_in / 2);
    *absmax_bytes = static_cast<size_t>(nb);
    *scale_bytes = sizeof(float) * static_cast<size_t>((nb + QN_GROUP - 1) / QN_GROUP);
    *mean_bytes = sizeof(float);
    g_err.clear();
    return QN_OK;
}

qn_status qn_weight_sizes(int64_t n_out, int64_t k_in, int const_format, size_t *codes_bytes, size_t *absmax_bytes,
                          size_t *scale_bytes, size_t *mean_bytes, size_t *absmax_f32_bytes) {
    if (!absmax_f32_bytes) return fail(QN_EINVAL, "null output pointer");
    if (const_format != QN_CONST_DQ && const_format != QN_CONST_F32)
        return fail(QN_EINVAL, "unknown const_format %d", const_format);
    qn_status s = qn_nf4_sizes(n_out, k_in, codes_bytes, absmax_bytes, scale_bytes, mean_bytes);
    if (s != QN_OK) return s;
    *absmax_f32_bytes = 0;
    if (const_format == QN_CONST_F32) {
        *absmax_f32_bytes = sizeof(float) * *absmax_bytes;
        *absmax_bytes = *scale_bytes = *mean_bytes = 0;
    }
    return QN_OK;
}

qn_status qn_quantize_workspace_size(int64_t n_out, int64_t k_in, size_t *ws_bytes) {
    if (!ws_bytes) return fail(QN_EINVAL, "null output pointer");
    qn_status s = check_shape(n_out, k_in);
    if (s != QN_OK) return s;
    *ws_bytes = quantize_workspace_bytes(n_out, k_in);
    g_err.clear();
    return QN_OK;
}

qn_status nf4_quantize(const void *W, const qn_nf4_weight *out, void *ws, size_t ws_bytes, void *stream) {
    qn_status s = check_weight(out);
    if (s != QN_OK) return s;
    if (out->n_out == 0 || out->k_in == 0) return QN_OK;
    if (!W) return fail(QN_EINVAL, "null W");
    if (!aligned16(W)) return fail(QN_EALIGN, "W not 16-byte aligned");
    const size_t need = quantize_workspace_bytes(out->n_out, out->k_in);
    if (!ws || ws_bytes < need) return fail(QN_EWORKSPACE, "quantize workspace needs %zu bytes", need);
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return fail(QN_EALIGN, "workspace not 256-byte aligned");
    return launch_quantize_into(W, out, ws, static_cast<cudaStream_t>(stream));
}

qn_status nf4_quantize_static_ws(const void *W, const qn_nf4_weight *out, void *stream) {
    qn_status s = check_weight(out);
    if (s != QN_OK) return s;
    if (out->n_out == 0 || out->k_in == 0) return QN_OK;
    const size_t need = quantize_workspace_bytes(out->n_out, out->k_in);
    if (need > static_scratch_bytes())
        return fail(QN_EWORKSPACE,
                    "nf4_quantize_static_ws: a %lld x %lld weight needs %zu bytes of scratch, the static scratch holds "
                    "%zu (at most %lld weights); use nf4_quantize with a caller workspace",
                    (long long)out->n_out, (long long)out->k_in, need, static_scratch_bytes(),
                    (long long)((static_scratch_bytes() - 2304) / 4 * QN_BLOCK));
    if (!W) return fail(QN_EINVAL, "null W");
    if (!aligned16(W)) return fail(QN_EALIGN, "W not 16-byte aligned");
    void *ws = nullptr;
    cudaError_t e = static_scratch_address(&ws);
    if (e != cudaSuccess) return cuda_status(e, "nf4_quantize_static_ws: cudaGetSymbolAddress");
    return launch_quantize_into(W, out, ws, static_cast<cudaStream_t>(stream));
}

qn_status nf4_dequantize(const qn_nf4_weight *w, void *W_out, void *stream) {
    qn_status s = check_weight(w);
    if (s != QN_OK) return s;
    if (w->n_out == 0 || w->k_in == 0) return QN_OK;
    if (!W_out) return fail(QN_EINVAL, "null W_out");
    if (!aligned16(W_out)) return fail(QN_EALIGN, "W_out not 16-byte aligned");
    return cuda_status(launch_dequant(view(w), static_cast<uint16_t *>(W_out), static_cast<cudaStream_t>(stream)),
                       "nf4_dequantize");
}

qn_status qlora_merge_bf16(const qn_nf4_weight *w, const void *A, const void *B, int r, float alpha, void *W_out,
                           void *stream) {
    qn_status s = check_weight(w);
    if (s != QN_OK) return s;
    s = check_lora(A, B, r, alpha);
    if (s != QN_OK) return s;
    if (w->n_out == 0 || w->k_in == 0) return QN_OK;
    if (!W_out) return fail(QN_EINVAL, "null W_out");
    if (!aligned16(W_out)) return fail(QN_EALIGN, "W_out not 16-byte aligned");
    if (W_out == A || W_out == B) return fail(QN_EINVAL, "W_out aliases an adapter factor");
    const float sc = r > 0 ? alpha / static_cast<float>(r) : 0.0f;
    return cuda_status(launch_merge(view(w), static_cast<const uint16_t *>(A), static_cast<const uint16_t *>(B), r, sc,
                                    static_cast<uint16_t *>(W_out), static_cast<cudaStream_t>(stream)),
                       "qlora_merge_bf16");
}

qn_status qlora_lora_grads_workspace_size(int64_t M, int r, size_t *ws_bytes) {
    if (!ws_bytes) return fail(QN_EINVAL, "null output pointer");
    if (M < 0 || M > kMaxDim) return fail(QN_EINVAL, "M=%lld out of range", (long long)M);
    if (r < 1 || r > QN_MAX_RANK) return fail(QN_EINVAL, "rank r=%d outside [1, %d]", r, QN_MAX_RANK);
    *ws_bytes = lora_grads_workspace_bytes(M, r);
    g_err.clear();
    return QN_OK;
}

qn_status qlora_lora_grads(const void *x, const void *grad_h, int64_t M, int64_t n_out, int64_t k_in, const void *A,
                           const void *B, int r, float alpha, float *grad_A, float *grad_B, void *ws, size_t ws_bytes,
                           void *stream) {
    return qlora_lora_grads_dropout(x, grad_h, M, n_out, k_in, A, B, r, alpha, nullptr, grad_A, grad_B, ws, ws_bytes,
                                    stream);
}

qn_status qlora_lora_grads_dropout(const void *x, const void *grad_h, int64_t M, int64_t n_out, int64_t k_in,
                                   const void *A, const void *B, int r, float alpha, const qn_lora_dropout *dropout,
                                   float *grad_A, float *grad_B, void *ws, size_t ws_bytes, void *stream) {
    qn_status s = check_shape(n_out, k_in);
    if (s != QN_OK) return s;
    if (M < 0 || M > kMaxDim) return fail(QN_EINVAL, "M=%lld out of range", (long long)M);
    if (r < 1 || r > QN_MAX_RANK) return fail(QN_EINVAL, "rank r=%d outside [1, %d]", r, QN_MAX_RANK);
    s = check_lora(A, B, r, alpha);
    if (s != QN_OK) return s;
    if (!grad_A || !grad_B) return fail(QN_EINVAL, "null gradient output");
    if (n_out == 0 || k_in == 0) return QN_OK;
    if (M > 0 && (!x || !grad_h)) return fail(QN_EINVAL, "null activation pointer");
    if (M > 0 && (!aligned16(x) || !aligned16(grad_h))) return fail(QN_EALIGN, "x or grad_h not 16-byte aligned");
    const size_t need = lora_grads_workspace_bytes(M, r);
    if (!ws || ws_bytes < need) return fail(QN_EWORKSPACE, "adapter-gradient workspace needs %zu bytes", need);
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return fail(QN_EALIGN, "workspace not 256-byte aligned");
    DropoutArgs drop;
    float sc = alpha / static_cast<float>(r);
    s = resolve_dropout(dropout, r, sc, &drop, &sc);
    if (s != QN_OK) return s;
    return cuda_status(launch_lora_grads(static_cast<const uint16_t *>(x), static_cast<const uint16_t *>(grad_h), M,
                                         n_out, k_in, static_cast<const uint16_t *>(A),
                                         static_cast<const uint16_t *>(B), r, sc, drop, grad_A, grad_B, ws,
                                         static_cast<cudaStream_t>(stream)),
                       "qlora_lora_grads");
}

qn_status qlora_workspace_size(int64_t M, int64_t n_out, int64_t k_in, int r, size_t *ws_bytes) {
    if (!ws_bytes) return fail(QN_EINVAL, "null output pointer");
    qn_status s = check_shape(n_out, k_in);
    if (s != QN_OK) return s;
    if (M < 0 || M > kMaxDim) return fail(QN_EINVAL, "M=%lld out of range", (long long)M);
    if (r < 0 || r > QN_MAX_RANK) return fail(QN_EINVAL, "rank r=%d outside [0, %d]", r, QN_MAX_RANK);
    // The few-token kernels keep the error word, the adapter product and its ready flag there
    // (4 KB); the tensor-core path and the paths that add a dropout-masked adapter term after a
    // base-only pass the error word and the M x roundup(r, 64) adapter operand.
    const size_t few = decode_fwd_workspace_bytes() > 4096 ? decode_fwd_workspace_bytes() : 4096;
    const size_t op = gemm_workspace_bytes(M, r);
    *ws_bytes = op > few ? op : few;
    g_err.clear();
    return QN_OK;
}

static qn_status check_linear(const qn_nf4_weight *w, const void *in, int64_t M, const void *A, const void *B, int r,
                              float alpha, const void *out, void *ws, size_t ws_bytes) {
    qn_status s = check_weight(w);
    if (s != QN_OK) return s;
    if (M < 0 || M > kMaxDim) return fail(QN_EINVAL, "M=%lld out of range", (long long)M);
    s = check_lora(A, B, r, alpha);
    if (s != QN_OK) return s;
    if (M == 0 || w->n_out == 0 || w->k_in == 0) return QN_OK;
    if (!in || !out) return fail(QN_EINVAL, "null activation or output pointer");
    if (!aligned16(in) || !aligned16(out)) return fail(QN_EALIGN, "activation or output not 16-byte aligned");
    if (in == out) return fail(QN_EINVAL, "output aliases the input");
    size_t need = 0;
    qlora_workspace_size(M, w->n_out, w->k_in, r, &need);
    if (!ws || ws_bytes < need) return fail(QN_EWORKSPACE, "linear workspace needs %zu bytes", need);
    return QN_OK;
}

qn_status qlora_workspace_check(void *ws, void *stream) {
    if (!ws) return fail(QN_EINVAL, "null workspace");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int word = 0;
    cudaError_t e = cudaMemcpyAsync(&word, ws, sizeof(int), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_status(e, "qlora_workspace_check");
    if (word == 0) return cuda_status(cudaSuccess, "");
    e = cudaMemsetAsync(ws, 0, sizeof(int), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_status(e, "qlora_workspace_check");
    return fail(QN_ETIMEOUT,
                "a kernel that used this workspace stopped early (error word %d: %s); its output is incomplete", word,
                word == 2 ? "dynamic shared memory not 1024-byte aligned" : "a bounded wait ran out");
}

qn_status qn_selftest_wait_timeout(void *ws, size_t ws_bytes, void *stream) {
    if (!ws || ws_bytes < 256) return fail(QN_EWORKSPACE, "the self-test needs a zeroed workspace of 256 bytes");
    return cuda_status(launch_wait_timeout_selftest(ws, static_cast<cudaStream_t>(stream)), "qn_selftest_wait_timeout");
}

qn_status qlora_linear_fwd(const qn_nf4_weight *w, const void *x, int64_t M, const void *A, const void *B, int r,
                           float alpha, void *h, void *ws, size_t ws_bytes, void *stream) {
    return qlora_linear_fwd_dropout(w, x, M, A, B, r, alpha, nullptr, h, ws, ws_bytes, stream);
}

qn_status qlora_linear_fwd_dropout(const qn_nf4_weight *w, const void *x, int64_t M, const void *A, const void *B,
                                   int r, float alpha, const qn_lora_dropout *dropout, void *h, void *ws,
                                   size_t ws_bytes, void *stream) {
    qn_status s = check_linear(w, x, M, A, B, r, alpha, h, ws, ws_bytes);
    if (s != QN_OK) return s;
    DropoutArgs drop;
    float sc = r > 0 ? alpha / static_cast<float>(r) : 0.0f;
    s = resolve_dropout(dropout, r, sc, &drop, &sc);
    if (s != QN_OK) return s;
    if (M == 0 || w->n_out == 0) return QN_OK;
    const WeightView wv = view(w);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const uint16_t *xp = static_cast<const uint16_t *>(x);
    uint16_t *hp = static_cast<uint16_t *>(h);
    const uint16_t *Ap = static_cast<const uint16_t *>(A), *Bp = static_cast<const uint16_t *>(B);
    // few tokens and adapters of rank <= 64: the streamed kernel, 16 tokens per launch;
    // otherwise the tensor-core GEMM (any token count; the forward operand always suits TMA)
    if (M <= kDecodeMaxM && r <= kDecodeMaxRank) {
        int *err = static_cast<int *>(ws);
        for (int64_t m0 = 0; m0 < M; m0 += kDecodeTokens) {
            const int mc = static_cast<int>(M - m0 < kDecodeTokens ? M - m0 : kDecodeTokens);
            DropoutArgs dc = drop;
            dc.offset += static_cast<uint64_t>(m0 * w->k_in);  // element index of token m0
            cudaError_t e =
                launch_decode_fwd(wv, xp + m0 * w->k_in, mc, Ap, Bp, r, sc, dc, hp + m0 * w->n_out, err, st);
            if (e != cudaSuccess) return cuda_status(e, "qlora_linear_fwd");
        }
        return cuda_status(cudaSuccess, "");
    }
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return fail(QN_EALIGN, "workspace not 256-byte aligned");
    return cuda_status(launch_gemm_fwd(wv, xp, M, Ap, Bp, r, sc, hp, ws, st, &drop), "qlora_linear_fwd");
}

qn_status qlora_linear_bwd_x(const qn_nf4_weight *w, const void *grad_h, int64_t M, const void *A, const void *B,
                             int r, float alpha, void *grad_x, void *ws, size_t ws_bytes, void *stream) {
    return qlora_linear_bwd_x_dropout(w, grad_h, M, A, B, r, alpha, nullptr, grad_x, ws, ws_bytes, stream);
}

qn_status qlora_linear_bwd_x_dropout(const qn_nf4_weight *w, const void *grad_h, int64_t M, const void *A,
                                     const void *B, int r, float alpha, const qn_lora_dropout *dropout, void *grad_x,
                                     void *ws, size_t ws_bytes, void *stream) {
    qn_status s = check_linear(w, grad_h, M, A, B, r, alpha, grad_x, ws, ws_bytes);
    if (s != QN_OK) return s;
    DropoutArgs drop;
    float sc = r > 0 ? alpha / static_cast<float>(r) : 0.0f;
    s = resolve_dropout(dropout, r, sc, &drop, &sc);
    if (s != QN_OK) return s;
    if (M == 0 || w->k_in == 0) return QN_OK;
    const WeightView wv = view(w);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const uint16_t *gp = static_cast<const uint16_t *>(grad_h);
    uint16_t *xp = static_cast<uint16_t *>(grad_x);
    const uint16_t *Ap = static_cast<const uint16_t *>(A), *Bp = static_cast<const uint16_t *>(B);
    // few tokens, adapters of rank <= 64 and TMA-friendly rows: the streamed kernel, 16 tokens per
    // launch
    if (M <= kDecodeMaxM && r <= kDecodeMaxRank && decode_bwd_stream_supported(w->n_out, w->k_in, r)) {
        int *err = static_cast<int *>(ws);
        for (int64_t m0 = 0; m0 < M; m0 += kDecodeTokens) {
            const int mc = static_cast<int>(M - m0 < kDecodeTokens ? M - m0 : kDecodeTokens);
            DropoutArgs dc = drop;
            dc.offset += static_cast<uint64_t>(m0 * w->k_in);  // element index of token m0
            cudaError_t e =
                launch_decode_bwd_stream(wv, gp + m0 * w->n_out, mc, Ap, Bp, r, sc, dc, xp + m0 * w->k_in, err, st);
            if (e != cudaSuccess) return cuda_status(e, "qlora_linear_bwd_x");
        }
        return cuda_status(cudaSuccess, "");
    }
    // Under dropout the other paths run base-only and the masked adapter term is added after them
    // (u = s B^T grad_h into the workspace, then grad_x += mask * u A).
    const bool masked = drop.thr != 0u;
    const int ra = masked ? 0 : r;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return fail(QN_EALIGN, "workspace not 256-byte aligned");
    if (M > kDecodeMaxM && gemm_supported(w->n_out, w->k_in, M, true)) {
        cudaError_t e = launch_gemm_bwd(wv, gp, M, Ap, Bp, ra, sc, xp, ws, st);
        if (e != cudaSuccess) return cuda_status(e, "qlora_linear_bwd_x");
    } else {
        // many tokens with n_out % 8 != 0 (the GEMM's TMA row-stride rule), or few tokens with a
        // rank above 64 or rows the streamed kernel's boxes cannot read: the register-streaming
        // few-token kernel in chunks of 32 tokens
        constexpr int kChunk = 32;
        for (int64_t m0 = 0; m0 < M; m0 += kChunk) {
            const int mc = static_cast<int>(M - m0 < kChunk ? M - m0 : kChunk);
            cudaError_t e = launch_decode_bwd(wv, gp + m0 * w->n_out, mc, Ap, Bp, ra, sc, xp + m0 * w->k_in, st);
            if (e != cudaSuccess) return cuda_status(e, "qlora_linear_bwd_x");
        }
    }
    if (masked) {
        const int RT = (r + 63) / 64 * 64;
        uint16_t *u = reinterpret_cast<uint16_t *>(static_cast<char *>(ws) + 256);
        cudaError_t e = launch_lora_down(gp, M, w->n_out, Bp, 1, r, r, sc, u, RT, st);
        if (e == cudaSuccess) e = launch_adapter_up_masked(u, M, RT, Ap, r, w->k_in, drop, xp, st);
        if (e != cudaSuccess) return cuda_status(e, "qlora_linear_bwd_x");
    }
    return cuda_status(cudaSuccess, "");
}

// ------------------------------------------------------------- 8-bit activations

qn_status qn_act8_sizes(int64_t rows, int64_t cols, size_t *codes_bytes, size_t *absmax_bytes) {
    if (!codes_bytes || !absmax_bytes) return fail(QN_EINVAL, "null output pointer");
    qn_status s = check_act8_shape(rows, cols);
    if (s != QN_OK) return s;
    *codes_bytes = static_cast<size_t>(rows * cols);
    *absmax_bytes = 2 * static_cast<size_t>(rows * cols / QN_BLOCK);
    g_err.clear();
    return QN_OK;
}

// x <-> a: the checks of both directions.
static qn_status check_act8_pair(const qn_act8 *a, const void *x, bool write_x) {
    qn_status s = check_act8(a, "the 8-bit activation");
    if (s != QN_OK || a->rows == 0 || a->cols == 0) return s;
    if (!x) return fail(QN_EINVAL, "null activation pointer");
    if (!aligned16(x)) return fail(QN_EALIGN, "activation not 16-byte aligned");
    const Span sp[] = {{x, 2 * act8_values(a), write_x},
                       {a->codes, act8_values(a), !write_x},
                       {a->absmax, 2 * act8_blocks(a), !write_x}};
    if (overlap(sp)) return fail(QN_EINVAL, "an output overlaps another buffer");
    return QN_OK;
}

qn_status act8_quantize(const void *x, const qn_act8 *out, void *stream) {
    qn_status s = check_act8_pair(out, x, false);
    if (s != QN_OK) return s;
    if (out->rows == 0 || out->cols == 0) return QN_OK;
    return cuda_status(launch_act8_quantize(static_cast<const uint16_t *>(x), out->rows * out->cols, out->codes,
                                            out->absmax, static_cast<cudaStream_t>(stream)),
                       "act8_quantize");
}

qn_status act8_dequantize(const qn_act8 *a, void *x_out, void *stream) {
    qn_status s = check_act8_pair(a, x_out, true);
    if (s != QN_OK) return s;
    if (a->rows == 0 || a->cols == 0) return QN_OK;
    return cuda_status(launch_act8_dequantize(a->codes, a->absmax, a->rows * a->cols, static_cast<uint16_t *>(x_out),
                                              static_cast<cudaStream_t>(stream)),
                       "act8_dequantize");
}

static qn_status check_swiglu(const qn_act8 *gate8, const qn_act8 *up8, const qn_act8 *y8) {
    qn_status s = check_act8(gate8, "gate8");
    if (s != QN_OK) return s;
    s = check_act8(up8, "up8");
    if (s != QN_OK) return s;
    if (up8->rows != gate8->rows || up8->cols != gate8->cols) return fail(QN_ESHAPE, "gate8 and up8 differ in shape");
    if (!y8) return QN_OK;
    s = check_act8(y8, "y8");
    if (s != QN_OK) return s;
    if (y8->rows != gate8->rows || y8->cols != gate8->cols) return fail(QN_ESHAPE, "y8 and gate8 differ in shape");
    return QN_OK;
}

qn_status swiglu_act8_fwd(const void *gate, const void *up, void *y, const qn_act8 *gate8, const qn_act8 *up8,
                          void *stream) {
    qn_status s = check_swiglu(gate8, up8, nullptr);
    if (s != QN_OK) return s;
    if (gate8->rows == 0 || gate8->cols == 0) return QN_OK;
    if (!gate || !up || !y) return fail(QN_EINVAL, "null activation pointer");
    if (!aligned16(gate) || !aligned16(up) || !aligned16(y)) return fail(QN_EALIGN, "gate, up or y not 16-byte aligned");
    const size_t v = act8_values(gate8), b = act8_blocks(gate8);
    const Span sp[] = {{gate, 2 * v, false},       {up, 2 * v, false},         {y, 2 * v, true},
                       {gate8->codes, v, true},    {gate8->absmax, 2 * b, true}, {up8->codes, v, true},
                       {up8->absmax, 2 * b, true}};
    if (overlap(sp)) return fail(QN_EINVAL, "an output overlaps another buffer");
    return cuda_status(launch_swiglu_act8_fwd(static_cast<const uint16_t *>(gate), static_cast<const uint16_t *>(up),
                                              gate8->rows * gate8->cols, static_cast<uint16_t *>(y), gate8->codes,
                                              gate8->absmax, up8->codes, up8->absmax,
                                              static_cast<cudaStream_t>(stream)),
                       "swiglu_act8_fwd");
}

qn_status swiglu_act8_bwd(const qn_act8 *gate8, const qn_act8 *up8, const void *grad_y, void *grad_gate,
                          void *grad_up, const qn_act8 *y8, void *stream) {
    qn_status s = check_swiglu(gate8, up8, y8);
    if (s != QN_OK) return s;
    if (gate8->rows == 0 || gate8->cols == 0) return QN_OK;
    if (!grad_y || !grad_gate || !grad_up) return fail(QN_EINVAL, "null gradient pointer");
    if (!aligned16(grad_y) || !aligned16(grad_gate) || !aligned16(grad_up))
        return fail(QN_EALIGN, "grad_y, grad_gate or grad_up not 16-byte aligned");
    const size_t v = act8_values(gate8), b = act8_blocks(gate8);
    const Span sp[] = {{gate8->codes, v, false},
                       {gate8->absmax, 2 * b, false},
                       {up8->codes, v, false},
                       {up8->absmax, 2 * b, false},
                       {grad_y, 2 * v, false},
                       {grad_gate, 2 * v, true},
                       {grad_up, 2 * v, true},
                       {y8 ? y8->codes : nullptr, v, true},
                       {y8 ? y8->absmax : nullptr, 2 * b, true}};
    if (overlap(sp)) return fail(QN_EINVAL, "an output overlaps another buffer");
    return cuda_status(launch_swiglu_act8_bwd(gate8->codes, gate8->absmax, up8->codes, up8->absmax,
                                              static_cast<const uint16_t *>(grad_y), gate8->rows * gate8->cols,
                                              static_cast<uint16_t *>(grad_gate), static_cast<uint16_t *>(grad_up),
                                              y8 ? y8->codes : nullptr, y8 ? y8->absmax : nullptr,
                                              static_cast<cudaStream_t>(stream)),
                       "swiglu_act8_bwd");
}

qn_status qlora_lora_grads_act8_workspace_size(int64_t M, int64_t n_out, int r, size_t *ws_bytes) {
    if (!ws_bytes) return fail(QN_EINVAL, "null output pointer");
    if (M < 0 || M > kMaxDim) return fail(QN_EINVAL, "M=%lld out of range", (long long)M);
    if (n_out < 0 || n_out > kMaxDim) return fail(QN_EINVAL, "n_out=%lld out of range", (long long)n_out);
    if (r < 1 || r > QN_MAX_RANK) return fail(QN_EINVAL, "rank r=%d outside [1, %d]", r, QN_MAX_RANK);
    *ws_bytes = act8_grads_workspace_bytes(M, n_out, r);
    g_err.clear();
    return QN_OK;
}

// give_up: the self-test's call.
static qn_status grads_act8(const qn_act8 *x, const void *grad_h, int64_t n_out, const void *A, const void *B, int r,
                            float alpha, const qn_lora_dropout *dropout, float *grad_A, float *grad_B, void *ws,
                            size_t ws_bytes, void *stream, bool give_up) {
    qn_status s = check_act8(x, "x");
    if (s != QN_OK) return s;
    const int64_t M = x->rows, k = x->cols;
    s = check_shape(n_out, k);
    if (s != QN_OK) return s;
    if (r < 1 || r > QN_MAX_RANK) return fail(QN_EINVAL, "rank r=%d outside [1, %d]", r, QN_MAX_RANK);
    DropoutArgs drop;
    float sc = alpha / static_cast<float>(r);
    s = resolve_dropout(dropout, r, sc, &drop, &sc);
    if (s != QN_OK) return s;
    if (!(alpha - alpha == 0.0f)) return fail(QN_EINVAL, "alpha is not finite");
    const size_t a_bytes = static_cast<size_t>(r) * static_cast<size_t>(k), b_bytes = static_cast<size_t>(r) * static_cast<size_t>(n_out);
    if ((a_bytes && !grad_A) || (b_bytes && !grad_B)) return fail(QN_EINVAL, "null gradient output");
    if ((reinterpret_cast<uintptr_t>(grad_A) & 3u) != 0 || (reinterpret_cast<uintptr_t>(grad_B) & 3u) != 0)
        return fail(QN_EALIGN, "grad_A or grad_B not 4-byte aligned");
    const bool empty = M == 0 || k == 0 || n_out == 0;
    const size_t need = act8_grads_workspace_bytes(M, n_out, r);
    if (!empty) {
        if (!A || !B) return fail(QN_EINVAL, "null adapter pointer with r=%d", r);
        if (!grad_h) return fail(QN_EINVAL, "null activation pointer");
        if (!aligned16(A) || !aligned16(B) || !aligned16(grad_h)) return fail(QN_EALIGN, "A, B or grad_h not 16-byte aligned");
        if (!ws || ws_bytes < need) return fail(QN_EWORKSPACE, "adapter-gradient workspace needs %zu bytes", need);
        if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return fail(QN_EALIGN, "workspace not 256-byte aligned");
    }
    const Span sp[] = {{x->codes, act8_values(x), false},
                       {x->absmax, 2 * act8_blocks(x), false},
                       {grad_h, 2 * static_cast<size_t>(M) * static_cast<size_t>(n_out), false},
                       {A, 2 * a_bytes, false},
                       {B, 2 * b_bytes, false},
                       {grad_A, 4 * a_bytes, true},
                       {grad_B, 4 * b_bytes, true},
                       {empty ? nullptr : ws, need, true}};
    if (overlap(sp)) return fail(QN_EINVAL, "an output overlaps another buffer");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (empty) {  // no token, or one side without features: what gradients there are, are zero
        cudaError_t e = a_bytes ? cudaMemsetAsync(grad_A, 0, 4 * a_bytes, st) : cudaSuccess;
        if (e == cudaSuccess && b_bytes) e = cudaMemsetAsync(grad_B, 0, 4 * b_bytes, st);
        return cuda_status(e, "qlora_lora_grads_act8");
    }
    if (give_up)
        return cuda_status(launch_act8_grads_tc(x->codes, x->absmax, static_cast<const uint16_t *>(grad_h), M, n_out, k,
                                                static_cast<const uint16_t *>(A), static_cast<const uint16_t *>(B), r, sc,
                                                drop, grad_A, grad_B, ws, st, true),
                           "qn_selftest_grads_give_up");
    return cuda_status(launch_act8_grads(x->codes, x->absmax, static_cast<const uint16_t *>(grad_h), M, n_out, k,
                                         static_cast<const uint16_t *>(A), static_cast<const uint16_t *>(B), r, sc,
                                         drop, grad_A, grad_B, ws, st),
                       "qlora_lora_grads_act8");
}

qn_status qlora_lora_grads_act8(const qn_act8 *x, const void *grad_h, int64_t n_out, const void *A, const void *B,
                                int r, float alpha, const qn_lora_dropout *dropout, float *grad_A, float *grad_B,
                                void *ws, size_t ws_bytes, void *stream) {
    return grads_act8(x, grad_h, n_out, A, B, r, alpha, dropout, grad_A, grad_B, ws, ws_bytes, stream, false);
}

qn_status qn_selftest_grads_give_up(const qn_act8 *x, const void *grad_h, int64_t n_out, const void *A, const void *B,
                                    int r, float alpha, const qn_lora_dropout *dropout, float *grad_A, float *grad_B,
                                    void *ws, size_t ws_bytes, void *stream) {
    if (x && x->rows <= 1024) return fail(QN_ESHAPE, "the self-test wants more than 1024 tokens, has %lld", (long long)x->rows);
    if (!dropout || !(dropout->p > 0.0f)) return fail(QN_EINVAL, "the self-test wants a dropout");
    return grads_act8(x, grad_h, n_out, A, B, r, alpha, dropout, grad_A, grad_B, ws, ws_bytes, stream, true);
}

// ------------------------------------------------- 4-bit integers with group scales

qn_status qn_int4_sizes(int64_t n_out, int64_t k_in, int group, size_t *codes_bytes, size_t *scale_bytes,
                        size_t *zero_bytes) {
    if (!codes_bytes || !scale_bytes || !zero_bytes) return fail(QN_EINVAL, "null output pointer");
    qn_status s = check_int4_shape(n_out, k_in, group);
    if (s != QN_OK) return s;
    *codes_bytes = static_cast<size_t>(n_out * k_in / 2);
    *zero_bytes = static_cast<size_t>(n_out * (k_in / group));
    *scale_bytes = 2 * *zero_bytes;
    g_err.clear();
    return QN_OK;
}

// W <-> w: the checks of both directions.
static qn_status check_int4_pair(const qn_int4_weight *w, const void *W, bool write_W) {
    qn_status s = check_int4(w);
    if (s != QN_OK || w->n_out == 0 || w->k_in == 0) return s;
    if (!W) return fail(QN_EINVAL, "null matrix pointer");
    if (!aligned16(W)) return fail(QN_EALIGN, "matrix not 16-byte aligned");
    const size_t v = static_cast<size_t>(w->n_out * w->k_in), gr = v / static_cast<size_t>(w->group);
    const Span sp[] = {{W, 2 * v, write_W},
                       {w->codes, v / 2, !write_W},
                       {w->scale, 2 * gr, !write_W},
                       {w->zero_point, gr, !write_W}};
    if (overlap(sp)) return fail(QN_EINVAL, "an output overlaps another buffer");
    return QN_OK;
}

qn_status int4_quantize(const void *W, const qn_int4_weight *out, void *stream) {
    qn_status s = check_int4_pair(out, W, false);
    if (s != QN_OK) return s;
    if (out->n_out == 0 || out->k_in == 0) return QN_OK;
    return cuda_status(launch_int4_quantize(static_cast<const uint16_t *>(W), view(out),
                                            static_cast<cudaStream_t>(stream)),
                       "int4_quantize");
}

qn_status int4_dequantize(const qn_int4_weight *w, void *W_out, void *stream) {
    qn_status s = check_int4_pair(w, W_out, true);
    if (s != QN_OK) return s;
    if (w->n_out == 0 || w->k_in == 0) return QN_OK;
    return cuda_status(launch_int4_dequantize(view(w), static_cast<uint16_t *>(W_out),
                                              static_cast<cudaStream_t>(stream)),
                       "int4_dequantize");
}

qn_status int4_linear_fwd(const qn_int4_weight *w, const void *x, int64_t M, void *h, void *stream) {
    qn_status s = check_int4(w);
    if (s != QN_OK) return s;
    if (M < 0) return fail(QN_EINVAL, "M=%lld out of range", (long long)M);
    if (M > kDecodeMaxM) return fail(QN_ESHAPE, "M=%lld is above %d tokens", (long long)M, kDecodeMaxM);
    if (w->k_in > kInt4LinearMaxK)
        return fail(QN_ESHAPE, "k_in=%lld is above %lld", (long long)w->k_in, (long long)kInt4LinearMaxK);
    if (M == 0 || w->n_out == 0) return QN_OK;
    if (!h) return fail(QN_EINVAL, "null output pointer");
    if (!aligned16(h)) return fail(QN_EALIGN, "output not 16-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (w->k_in == 0)
        return cuda_status(cudaMemsetAsync(h, 0, 2 * static_cast<size_t>(M * w->n_out), st), "int4_linear_fwd");
    if (!x) return fail(QN_EINVAL, "null activation pointer");
    if (!aligned16(x)) return fail(QN_EALIGN, "activation not 16-byte aligned");
    const size_t v = static_cast<size_t>(w->n_out * w->k_in), gr = v / static_cast<size_t>(w->group);
    const Span sp[] = {{h, 2 * static_cast<size_t>(M * w->n_out), true},
                       {x, 2 * static_cast<size_t>(M * w->k_in), false},
                       {w->codes, v / 2, false},
                       {w->scale, 2 * gr, false},
                       {w->zero_point, gr, false}};
    if (overlap(sp)) return fail(QN_EINVAL, "h overlaps another buffer");
    return cuda_status(launch_int4_linear(view(w), static_cast<const uint16_t *>(x), static_cast<int>(M),
                                          static_cast<uint16_t *>(h), st),
                       "int4_linear_fwd");
}

}  // extern "C"
