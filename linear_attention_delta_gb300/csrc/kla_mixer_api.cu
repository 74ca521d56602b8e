// C entry points of the operators around the recurrence (layer norm, gated
// linear recurrence): argument validation and dispatch.  Every check runs on
// the host before any launch; see include/kla.h for each contract.
#include <cmath>
#include <cstdint>

#include "api_checks.cuh"
#include "kla_internal.cuh"

using namespace kla::api;

extern "C" kla_status kla_layernorm_fwd(
    const void* x, long long x_stride, const void* residual,
    long long residual_stride, const void* weight, const void* bias,
    float eps, void* y, void* sum, float* mean, float* rstd, int rows, int D,
    kla_dtype dtype, kla_dtype wdtype, kla_stream_t stream) {
    if (rows < 0 || D < 1 || x_stride < 0 || residual_stride < 0 ||
        !valid(dtype) || !valid(wdtype) || !(eps >= 0.f) ||
        !std::isfinite(eps) || (sum && !residual))
        return KLA_ERR_INVALID_ARG;
    if (D > kMaxCount) return KLA_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return KLA_OK;
    const size_t e = size_of(dtype), we = size_of(wdtype);
    if (!given(x, e) || !given(y, e) || !ok_or_null(residual, e) ||
        !ok_or_null(sum, e) || !ok_or_null(weight, we) ||
        !ok_or_null(bias, we) || !ok_or_null(mean, 4) || !ok_or_null(rstd, 4))
        return KLA_ERR_INVALID_ARG;
    const size_t out = (size_t)rows * D * e;
    const Span ins[] = {span(x, row_bytes(rows, D, x_stride, e)),
                        span(residual, row_bytes(rows, D, residual_stride, e)),
                        span(weight, D * we), span(bias, D * we)};
    const Span outs[] = {span(y, out), span(sum, out),
                         span(mean, (size_t)rows * 4),
                         span(rstd, (size_t)rows * 4)};
    if (any_overlap(ins, outs)) return KLA_ERR_INVALID_ARG;
    const kla::LayerNormArgs a{x, x_stride, residual, residual_stride, weight,
                               bias, eps, y, sum, mean, rstd, rows, D, dtype,
                               wdtype};
    return from_cuda(kla::launch_layernorm(
        a, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" kla_status kla_layernorm_bwd_workspace_size(int rows, int D,
                                                       kla_dtype dtype,
                                                       size_t* bytes) {
    if (!bytes || rows < 0 || D < 1 || !valid(dtype))
        return KLA_ERR_INVALID_ARG;
    if (D > kMaxCount) return KLA_ERR_UNSUPPORTED_SHAPE;
    *bytes = kla::layernorm_bwd_workspace_bytes(rows, D, dtype);
    return KLA_OK;
}

extern "C" kla_status kla_layernorm_bwd(
    const void* y_grad, long long y_grad_stride, const void* x,
    long long x_stride, const void* weight, const float* mean,
    const float* rstd, const void* sum_grad, long long sum_grad_stride,
    void* x_grad, void* weight_grad, void* bias_grad, int rows, int D,
    kla_dtype dtype, kla_dtype wdtype, void* workspace,
    size_t workspace_bytes, kla_stream_t stream) {
    if (rows < 0 || D < 1 || y_grad_stride < 0 || x_stride < 0 ||
        sum_grad_stride < 0 || !valid(dtype) || !valid(wdtype))
        return KLA_ERR_INVALID_ARG;
    if (D > kMaxCount) return KLA_ERR_UNSUPPORTED_SHAPE;
    const size_t e = size_of(dtype), we = size_of(wdtype);
    if (!ok_or_null(weight_grad, we) || !ok_or_null(bias_grad, we) ||
        !ok_or_null(weight, we) || !ok_or_null(sum_grad, e))
        return KLA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        for (void* g : {weight_grad, bias_grad})
            if (g && cudaMemsetAsync(g, 0, D * we, s) != cudaSuccess)
                return KLA_ERR_CUDA;
        return KLA_OK;
    }
    if (!given(y_grad, e) || !given(x, e) || !given(x_grad, e) ||
        !given(mean, 4) || !given(rstd, 4))
        return KLA_ERR_INVALID_ARG;
    const bool want = weight_grad || bias_grad;
    const size_t need =
        want ? kla::layernorm_bwd_workspace_bytes(rows, D, dtype) : 0;
    if (need && (!given(workspace, 16) || workspace_bytes < need))
        return KLA_ERR_INVALID_ARG;
    const Span ins[] = {span(y_grad, row_bytes(rows, D, y_grad_stride, e)),
                        span(x, row_bytes(rows, D, x_stride, e)),
                        span(sum_grad, row_bytes(rows, D, sum_grad_stride, e)),
                        span(weight, D * we), span(mean, (size_t)rows * 4),
                        span(rstd, (size_t)rows * 4)};
    const Span outs[] = {span(x_grad, (size_t)rows * D * e),
                         span(weight_grad, D * we), span(bias_grad, D * we),
                         span(workspace, need)};
    if (any_overlap(ins, outs)) return KLA_ERR_INVALID_ARG;
    const kla::LayerNormBwdArgs a{y_grad, y_grad_stride, x, x_stride, weight,
                                  mean, rstd, sum_grad, sum_grad_stride,
                                  x_grad, weight_grad, bias_grad, rows, D,
                                  dtype, wdtype};
    return from_cuda(kla::launch_layernorm_bwd(a, workspace, s));
}

namespace {

// Bytes spanned by a strided [B, T, D] input of the recurrence.
size_t span_bytes(const kla::GlrArgs& a, const kla::Strided& x, size_t elt) {
    const long long t = a.T ? (long long)(a.T - 1) * x.st : 0;
    const long long b = a.cu ? 0 : (long long)(a.B - 1) * x.sb;
    return a.T ? (size_t)(b + t + a.D) * elt : 0;
}

kla_status glr_impl(const kla::GlrArgs& a, bool bwd, kla_stream_t stream) {
    if (a.B < 0 || a.T < 0 || a.D < 1 || a.x.sb < 0 || a.x.st < 0 ||
        a.la.sb < 0 || a.la.st < 0 || a.g.sb < 0 || a.g.st < 0 ||
        !valid(a.dtype) || !valid(a.gdtype))
        return KLA_ERR_INVALID_ARG;
    if (!ok_or_null(a.h0, 4) || !ok_or_null(a.dhT, 4) ||
        !ok_or_null(a.hT, 4) || !ok_or_null(a.cu, 4))
        return KLA_ERR_INVALID_ARG;
    if (a.T > kMaxCount || a.D > kMaxCount || (a.cu && a.B > kMaxCount))
        return KLA_ERR_UNSUPPORTED_SHAPE;
    // packed tokens belong to some sequence
    if (a.B == 0) return a.cu && a.T > 0 ? KLA_ERR_INVALID_ARG : KLA_OK;
    const size_t e = size_of(a.dtype), ge = size_of(a.gdtype);
    if (a.T > 0 &&
        (!given(a.x.p, e) || !given(a.la.p, ge) || !given(a.o, e) ||
         (bwd && (!given(a.g.p, e) || !given(a.dla, ge)))))
        return KLA_ERR_INVALID_ARG;
    const size_t n = (size_t)a.T * (a.cu ? 1 : a.B) * a.D;
    const size_t st = (size_t)a.B * a.D * 4;
    // hT in the place of h0 is allowed in the forward: each state is read
    // before the one that replaces it is written
    const bool in_place = !bwd && a.hT == a.h0;
    const Span ins[] = {span(a.x.p, span_bytes(a, a.x, e)),
                        span(a.la.p, span_bytes(a, a.la, ge)),
                        span(a.g.p, span_bytes(a, a.g, e)),
                        span(in_place ? nullptr : a.h0, st),
                        span(a.dhT, st),
                        span(a.cu, ((size_t)a.B + 1) * 4)};
    const Span outs[] = {span(a.o, n * e), span(a.dla, n * ge),
                         span(a.hT, st)};
    if (any_overlap(ins, outs)) return KLA_ERR_INVALID_ARG;
    return from_cuda(
        kla::launch_glr(a, bwd, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" kla_status kla_glr_fwd(
    const void* x, long long x_sb, long long x_st, const void* log_alpha,
    long long a_sb, long long a_st, const float* h0, void* o, float* hT,
    const int* cu_seqlens, int B, int T, int D, kla_dtype dtype,
    kla_dtype gate_dtype, kla_stream_t stream) {
    const kla::GlrArgs a{{x, x_sb, x_st}, {log_alpha, a_sb, a_st},
                         {nullptr, 0, 0}, h0, nullptr, o, nullptr, hT,
                         cu_seqlens, B, T, D, dtype, gate_dtype};
    return glr_impl(a, false, stream);
}

extern "C" kla_status kla_glr_bwd(
    const void* o, long long o_sb, long long o_st, const void* log_alpha,
    long long a_sb, long long a_st, const float* h0, const void* o_grad,
    long long g_sb, long long g_st, const float* hT_grad, void* x_grad,
    void* log_alpha_grad, float* h0_grad, const int* cu_seqlens, int B, int T,
    int D, kla_dtype dtype, kla_dtype gate_dtype, kla_stream_t stream) {
    const kla::GlrArgs a{{o, o_sb, o_st}, {log_alpha, a_sb, a_st},
                         {o_grad, g_sb, g_st}, h0, hT_grad, x_grad,
                         log_alpha_grad, h0_grad, cu_seqlens, B, T, D, dtype,
                         gate_dtype};
    return glr_impl(a, true, stream);
}

extern "C" kla_status kla_glr_step(const void* x, long long x_stride,
                                   const void* log_alpha, long long a_stride,
                                   float* S, void* o, int N, int D,
                                   kla_dtype dtype, kla_dtype gate_dtype,
                                   kla_stream_t stream) {
    if (N < 0 || D < 1 || x_stride < 0 || a_stride < 0 || !valid(dtype) ||
        !valid(gate_dtype))
        return KLA_ERR_INVALID_ARG;
    if (D > kMaxCount) return KLA_ERR_UNSUPPORTED_SHAPE;
    if (N == 0) return KLA_OK;
    const size_t e = size_of(dtype), ge = size_of(gate_dtype);
    if (!given(x, e) || !given(log_alpha, ge) || !given(S, 4) || !given(o, e))
        return KLA_ERR_INVALID_ARG;
    const size_t n = (size_t)N * D;
    const Span ins[] = {span(x, row_bytes(N, D, x_stride, e)),
                        span(log_alpha, row_bytes(N, D, a_stride, ge))};
    const Span outs[] = {span(S, n * 4), span(o, n * e)};
    if (any_overlap(ins, outs)) return KLA_ERR_INVALID_ARG;
    return from_cuda(kla::launch_glr_step(
        x, x_stride, log_alpha, a_stride, S, o, N, D, dtype, gate_dtype,
        reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" kla_status kla_selftest_glr_timeout(kla_stream_t stream) {
    return from_cuda(kla::launch_glr_selftest(
        reinterpret_cast<cudaStream_t>(stream)));
}
