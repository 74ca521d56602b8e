// C entry points of linear attention with a decay for each head and of the
// log probabilities of given tokens: argument validation and dispatch.  Every
// check runs on the host before any launch; see include/kla.h for each
// contract.
#include <cmath>
#include <cstdint>

#include "api_checks.cuh"
#include "kla_internal.cuh"

using namespace kla::api;
using kla::Heads;

namespace {

constexpr long long kMaxHeads = 1ll << 24;   // B H: bounds the grids

bool strides_ok(const Heads& x) { return x.sb >= 0 && x.st >= 0 && x.sh >= 0; }

// Bytes from the first to the last element of a [B, T, H, d] tensor.
size_t heads_bytes(const Heads& x, int B, int T, int H, int d, size_t elt) {
    if (!B || !T || !H) return 0;
    return ((size_t)(B - 1) * (size_t)x.sb + (size_t)(T - 1) * (size_t)x.st +
            (size_t)(H - 1) * (size_t)x.sh + d) * elt;
}

kla_status sizes(int B, int T, int H, int dk, int dv, kla_dtype dtype) {
    if (B < 0 || T < 0 || H < 0 || dk < 1 || dv < 1 || !valid(dtype))
        return KLA_ERR_INVALID_ARG;
    if (dk > kla::kLinAttnMaxWidth || dv > kla::kLinAttnMaxWidth ||
        T > kMaxCount || (long long)B * H > kMaxHeads)
        return KLA_ERR_UNSUPPORTED_SHAPE;
    return KLA_OK;
}

// The passes of a call: the forward is one, the backward three.
kla::LinAttnArgs forward(const Heads& q, const Heads& k, const Heads& v,
                         const float* log_decay, const float* h0, void* o,
                         float* hT, int B, int T, int H, int dk, int dv,
                         kla_dtype dtype) {
    kla::LinAttnArgs a{};
    a.job[0] = {q, k, v, o, h0, hT, dv, 1, dk, dv, false};
    a.jobs = 1;
    a.log_decay = log_decay;
    a.B = B, a.T = T, a.H = H, a.dtype = dtype;
    return a;
}

kla::LinAttnArgs backward(const Heads& q, const Heads& k, const Heads& v,
                          const Heads& g, const float* log_decay,
                          const float* h0, const float* dhT, void* dq,
                          void* dkey, void* dval, float* dh0, int B, int T,
                          int H, int dk, int dv, kla_dtype dtype) {
    kla::LinAttnArgs a{};
    // q_grad_t = S_t g_t: the forward with (g, v, k) and transposed states
    a.job[0] = {g, v, k, dq, h0, nullptr, 1, dv, dv, dk, false};
    // k_grad_t = D_t v_t and v_grad_t = D_t^T k_t, from the last token on
    a.job[1] = {v, g, q, dkey, dhT, nullptr, 1, dv, dv, dk, true};
    a.job[2] = {k, q, g, dval, dhT, dh0, dv, 1, dk, dv, true};
    a.jobs = 3;
    a.log_decay = log_decay;
    a.B = B, a.T = T, a.H = H, a.dtype = dtype;
    return a;
}

// dst = src or zeros; nothing when dst is null or src itself.
kla_status copy_state(float* dst, const float* src, size_t bytes,
                      cudaStream_t s) {
    if (!dst || dst == src || !bytes) return KLA_OK;
    return from_cuda(src ? cudaMemcpyAsync(dst, src, bytes,
                                           cudaMemcpyDeviceToDevice, s)
                         : cudaMemsetAsync(dst, 0, bytes, s));
}

}  // namespace

extern "C" kla_status kla_linattn_workspace_size(int B, int T, int H, int dk,
                                                 int dv, kla_dtype dtype,
                                                 int backward_pass,
                                                 size_t* bytes) {
    if (!bytes) return KLA_ERR_INVALID_ARG;
    const kla_status st = sizes(B, T, H, dk, dv, dtype);
    if (st != KLA_OK) return st;
    const Heads x{};
    *bytes = B && H && T ? kla::linattn_workspace_bytes(
        backward_pass
            ? backward(x, x, x, x, nullptr, nullptr, nullptr, nullptr,
                       nullptr, nullptr, nullptr, B, T, H, dk, dv, dtype)
            : forward(x, x, x, nullptr, nullptr, nullptr, nullptr, B, T, H,
                      dk, dv, dtype)) : 0;
    return KLA_OK;
}

extern "C" kla_status kla_linattn_fwd(
    const void* q, long long q_sb, long long q_st, long long q_sh,
    const void* k, long long k_sb, long long k_st, long long k_sh,
    const void* v, long long v_sb, long long v_st, long long v_sh,
    const float* log_decay, const float* h0, void* o, float* hT, int B, int T,
    int H, int dk, int dv, kla_dtype dtype, void* workspace,
    size_t workspace_bytes, kla_stream_t stream) {
    const Heads hq{q, q_sb, q_st, q_sh}, hk{k, k_sb, k_st, k_sh},
        hv{v, v_sb, v_st, v_sh};
    if (!strides_ok(hq) || !strides_ok(hk) || !strides_ok(hv))
        return KLA_ERR_INVALID_ARG;
    const kla_status ok = sizes(B, T, H, dk, dv, dtype);
    if (ok != KLA_OK) return ok;
    if (!ok_or_null(h0, 4) || !ok_or_null(hT, 4)) return KLA_ERR_INVALID_ARG;
    if (!B || !H) return KLA_OK;
    const size_t e = size_of(dtype), st = (size_t)B * H * dk * dv * 4;
    if (T > 0 && (!given(q, e) || !given(k, e) || !given(v, e) ||
                  !given(o, e) || !given(log_decay, 4)))
        return KLA_ERR_INVALID_ARG;
    const kla::LinAttnArgs a = forward(hq, hk, hv, log_decay, h0, o, hT, B, T,
                                       H, dk, dv, dtype);
    const size_t need = T ? kla::linattn_workspace_bytes(a) : 0;
    if (need && (!given(workspace, 16) || workspace_bytes < need))
        return KLA_ERR_INVALID_ARG;
    const Span ins[] = {span(q, heads_bytes(hq, B, T, H, dk, e)),
                        span(k, heads_bytes(hk, B, T, H, dk, e)),
                        span(v, heads_bytes(hv, B, T, H, dv, e)),
                        span(log_decay, T ? (size_t)H * 4 : 0),
                        span(hT == h0 ? nullptr : h0, st)};
    const Span outs[] = {span(o, (size_t)B * T * H * dv * e), span(hT, st),
                         span(workspace, need)};
    if (any_overlap(ins, outs)) return KLA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) return copy_state(hT, h0, st, s);
    return from_cuda(kla::launch_linattn(a, workspace, s));
}

extern "C" kla_status kla_linattn_bwd(
    const void* q, long long q_sb, long long q_st, long long q_sh,
    const void* k, long long k_sb, long long k_st, long long k_sh,
    const void* v, long long v_sb, long long v_st, long long v_sh,
    const float* log_decay, const float* h0, const void* o_grad,
    long long g_sb, long long g_st, long long g_sh, const float* hT_grad,
    void* q_grad, void* k_grad, void* v_grad, float* h0_grad, int B, int T,
    int H, int dk, int dv, kla_dtype dtype, void* workspace,
    size_t workspace_bytes, kla_stream_t stream) {
    const Heads hq{q, q_sb, q_st, q_sh}, hk{k, k_sb, k_st, k_sh},
        hv{v, v_sb, v_st, v_sh}, hg{o_grad, g_sb, g_st, g_sh};
    if (!strides_ok(hq) || !strides_ok(hk) || !strides_ok(hv) ||
        !strides_ok(hg))
        return KLA_ERR_INVALID_ARG;
    const kla_status ok = sizes(B, T, H, dk, dv, dtype);
    if (ok != KLA_OK) return ok;
    if (!ok_or_null(h0, 4) || !ok_or_null(hT_grad, 4) ||
        !ok_or_null(h0_grad, 4))
        return KLA_ERR_INVALID_ARG;
    if (!B || !H) return KLA_OK;
    const size_t e = size_of(dtype), st = (size_t)B * H * dk * dv * 4;
    if (T > 0 && (!given(q, e) || !given(k, e) || !given(v, e) ||
                  !given(o_grad, e) || !given(q_grad, e) ||
                  !given(k_grad, e) || !given(v_grad, e) ||
                  !given(log_decay, 4)))
        return KLA_ERR_INVALID_ARG;
    const kla::LinAttnArgs a =
        backward(hq, hk, hv, hg, log_decay, h0, hT_grad, q_grad, k_grad,
                 v_grad, h0_grad, B, T, H, dk, dv, dtype);
    const size_t need = T ? kla::linattn_workspace_bytes(a) : 0;
    if (need && (!given(workspace, 16) || workspace_bytes < need))
        return KLA_ERR_INVALID_ARG;
    const size_t n = (size_t)B * T * H * e;
    const Span ins[] = {span(q, heads_bytes(hq, B, T, H, dk, e)),
                        span(k, heads_bytes(hk, B, T, H, dk, e)),
                        span(v, heads_bytes(hv, B, T, H, dv, e)),
                        span(o_grad, heads_bytes(hg, B, T, H, dv, e)),
                        span(log_decay, T ? (size_t)H * 4 : 0), span(h0, st),
                        span(hT_grad, st)};
    const Span outs[] = {span(q_grad, n * dk), span(k_grad, n * dk),
                         span(v_grad, n * dv), span(h0_grad, st),
                         span(workspace, need)};
    if (any_overlap(ins, outs)) return KLA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) return copy_state(h0_grad, hT_grad, st, s);
    return from_cuda(kla::launch_linattn(a, workspace, s));
}

extern "C" kla_status kla_linattn_step(
    const void* q, long long q_sn, long long q_sh, const void* k,
    long long k_sn, long long k_sh, const void* v, long long v_sn,
    long long v_sh, const float* log_decay, float* S, void* o, int N, int H,
    int dk, int dv, kla_dtype dtype, kla_stream_t stream) {
    const Heads hq{q, q_sn, 0, q_sh}, hk{k, k_sn, 0, k_sh},
        hv{v, v_sn, 0, v_sh};
    if (!strides_ok(hq) || !strides_ok(hk) || !strides_ok(hv))
        return KLA_ERR_INVALID_ARG;
    const kla_status ok = sizes(N, 1, H, dk, dv, dtype);
    if (ok != KLA_OK) return ok;
    if (!N || !H) return KLA_OK;
    const size_t e = size_of(dtype);
    if (!given(q, e) || !given(k, e) || !given(v, e) || !given(o, e) ||
        !given(S, 4) || !given(log_decay, 4))
        return KLA_ERR_INVALID_ARG;
    const Span ins[] = {span(q, heads_bytes(hq, N, 1, H, dk, e)),
                        span(k, heads_bytes(hk, N, 1, H, dk, e)),
                        span(v, heads_bytes(hv, N, 1, H, dv, e)),
                        span(log_decay, (size_t)H * 4)};
    const Span outs[] = {span(S, (size_t)N * H * dk * dv * 4),
                         span(o, (size_t)N * H * dv * e)};
    if (any_overlap(ins, outs)) return KLA_ERR_INVALID_ARG;
    const kla::LinAttnStepArgs a{hq, hk, hv, log_decay, S, o, N, H, dk, dv,
                                 dtype};
    return from_cuda(kla::launch_linattn_step(
        a, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" kla_status kla_logprob_fwd(
    const void* logits, long long logits_stride, const long long* tokens,
    float scale, float* logp, float* entropy, float* lse, float* top_logp,
    long long* top_ids, int N, int V, int top, kla_dtype dtype,
    kla_stream_t stream) {
    if (N < 0 || V < 1 || top < 0 || top > V || logits_stride < 0 ||
        !valid(dtype) || !(scale > 0.f) || !std::isfinite(scale))
        return KLA_ERR_INVALID_ARG;
    if (top > kla::kLogprobMaxTop || V > kMaxCount)
        return KLA_ERR_UNSUPPORTED_SHAPE;
    if (N == 0) return KLA_OK;
    const size_t e = size_of(dtype), n = (size_t)N;
    if (!given(logits, e) || !given(tokens, 8) || !given(logp, 4) ||
        !ok_or_null(entropy, 4) || !ok_or_null(lse, 4) ||
        (top && (!given(top_logp, 4) || !given(top_ids, 8))))
        return KLA_ERR_INVALID_ARG;
    const Span ins[] = {span(logits, row_bytes(N, V, logits_stride, e)),
                        span(tokens, n * 8)};
    const Span outs[] = {span(logp, n * 4), span(entropy, n * 4),
                         span(lse, n * 4), span(top_logp, n * top * 4),
                         span(top_ids, n * top * 8)};
    if (any_overlap(ins, outs)) return KLA_ERR_INVALID_ARG;
    const kla::LogprobArgs a{logits, logits_stride, tokens, scale, logp,
                             entropy, lse, top_logp, top_ids, N, V, top,
                             dtype};
    return from_cuda(kla::launch_logprob(
        a, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" kla_status kla_logprob_bwd(
    const void* logits, long long logits_stride, const long long* tokens,
    float scale, const float* lse, const float* entropy,
    const float* logp_grad, const float* entropy_grad, void* logits_grad,
    int N, int V, kla_dtype dtype, kla_stream_t stream) {
    if (N < 0 || V < 1 || logits_stride < 0 || !valid(dtype) ||
        !(scale > 0.f) || !std::isfinite(scale))
        return KLA_ERR_INVALID_ARG;
    if (V > kMaxCount) return KLA_ERR_UNSUPPORTED_SHAPE;
    if (N == 0) return KLA_OK;
    const size_t e = size_of(dtype), n = (size_t)N;
    if (!given(logits, e) || !given(tokens, 8) || !given(lse, 4) ||
        !given(logits_grad, e) || !ok_or_null(entropy, 4) ||
        !ok_or_null(logp_grad, 4) || !ok_or_null(entropy_grad, 4) ||
        (entropy_grad && !entropy))
        return KLA_ERR_INVALID_ARG;
    // in place each element is read by the thread that writes it
    const bool in_place =
        logits_grad == logits && (logits_stride == V || N == 1);
    const Span ins[] = {span(in_place ? nullptr : logits,
                             row_bytes(N, V, logits_stride, e)),
                        span(tokens, n * 8), span(lse, n * 4),
                        span(entropy, n * 4), span(logp_grad, n * 4),
                        span(entropy_grad, n * 4)};
    const Span outs[] = {span(logits_grad, n * V * e)};
    if (any_overlap(ins, outs)) return KLA_ERR_INVALID_ARG;
    const kla::LogprobBwdArgs a{logits, logits_stride, tokens, scale, lse,
                                entropy, logp_grad, entropy_grad,
                                logits_grad, N, V, dtype};
    return from_cuda(kla::launch_logprob_bwd(
        a, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" kla_status kla_selftest_linattn_timeout(kla_stream_t stream) {
    return from_cuda(kla::launch_linattn_selftest(
        reinterpret_cast<cudaStream_t>(stream)));
}
