// Gated linear recurrence, per sequence and channel:
//
//   h_t = alpha_t h_{t-1} + x_t,  alpha_t = exp(log_alpha_t),  o_t = h_t
//
// and its reverse: g_t = do_t + alpha_{t+1} g_{t+1}, dx_t = g_t,
// dlog_alpha_t = alpha_t g_t h_{t-1}, dh0 = alpha_1 g_1.  Bound by HBM: three
// to five operations per element of each tensor it reads.
#include "kla_internal.cuh"

namespace kla {
namespace {

using bf16 = __nv_bfloat16;

// The tokens [first, last) of sequence n, row addresses base + t * st.
struct Seq {
    int first, last;
    __device__ Seq(const GlrArgs& a, int n) {
        first = a.cu ? min(max(a.cu[n], 0), a.T) : 0;
        last = a.cu ? min(max(a.cu[n + 1], 0), a.T) : a.T;
    }
};

template <typename T>
__device__ __forceinline__ const T* base(const GlrArgs& a, const Strided& x,
                                         int n) {
    return static_cast<const T*>(x.p) + (a.cu ? 0 : n * x.sb);
}

// One thread per (sequence, channel), token after token.
template <typename T, typename G>
__global__ void glr_fwd_seq_kernel(GlrArgs a) {
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= a.D) return;
    for (int n = blockIdx.y; n < a.B; n += gridDim.y) {
        const Seq q(a, n);
        const T* x = base<T>(a, a.x, n) + d;
        const G* la = base<G>(a, a.la, n) + d;
        T* o = static_cast<T*>(a.o) + (a.cu ? 0 : (size_t)n * a.T * a.D) + d;
        float h = a.h0 ? a.h0[(size_t)n * a.D + d] : 0.f;
        for (long long t = q.first; t < q.last; ++t) {
            h = fmaf(expf(to_f32(la[t * a.la.st])), h,
                     to_f32(x[t * a.x.st]));
            o[t * a.D] = from_f32<T>(h);
        }
        if (a.hT) a.hT[(size_t)n * a.D + d] = h;
    }
}

template <typename T, typename G>
__global__ void glr_bwd_seq_kernel(GlrArgs a) {
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= a.D) return;
    for (int n = blockIdx.y; n < a.B; n += gridDim.y) {
        const Seq q(a, n);
        const T* o = base<T>(a, a.x, n) + d;
        const G* la = base<G>(a, a.la, n) + d;
        const T* g = base<T>(a, a.g, n) + d;
        const size_t out = (a.cu ? 0 : (size_t)n * a.T * a.D) + d;
        T* dx = static_cast<T*>(a.o) + out;
        G* dla = static_cast<G*>(a.dla) + out;
        const size_t nd = (size_t)n * a.D + d;
        float c = a.dhT ? a.dhT[nd] : 0.f;      // alpha_{t+1} g_{t+1}
        for (long long t = (long long)q.last - 1; t >= q.first; --t) {
            const float gt = to_f32(g[t * a.g.st]) + c;
            c = expf(to_f32(la[t * a.la.st])) * gt;
            const float h = t > q.first ? to_f32(o[(t - 1) * a.x.st])
                            : a.h0      ? a.h0[nd]
                                        : 0.f;
            dx[t * a.D] = from_f32<T>(gt);
            dla[t * a.D] = from_f32<G>(c * h);
        }
        if (a.hT) a.hT[nd] = c;
    }
}

template <typename T, typename G>
__global__ void glr_step_kernel(const T* x, long long xs, const G* la,
                                long long ls, float* S, T* o, int N, int D) {
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= D) return;
    for (int n = blockIdx.y; n < N; n += gridDim.y) {
        const size_t i = (size_t)n * D + d;
        const float h =
            fmaf(expf(to_f32(la[n * ls + d])), S[i], to_f32(x[n * xs + d]));
        S[i] = h;
        o[i] = from_f32<T>(h);
    }
}

dim3 grid_of(int D, int N) {
    return dim3((D + 127) / 128, N < 65535 ? N : 65535);
}

// f<T, G>() for the pair of element types.
template <typename F>
cudaError_t by_type(kla_dtype t, kla_dtype g, F f) {
    if (t == KLA_BF16)
        return g == KLA_BF16 ? f(bf16(), bf16()) : f(bf16(), float());
    return g == KLA_BF16 ? f(float(), bf16()) : f(float(), float());
}

}  // namespace

size_t glr_workspace_bytes(int, int, int, bool, kla_dtype, kla_dtype) {
    return 0;
}

cudaError_t launch_glr(const GlrArgs& a, bool bwd, void*,
                       cudaStream_t stream) {
    return by_type(a.dtype, a.gdtype, [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        if (bwd)
            glr_bwd_seq_kernel<T, G><<<grid_of(a.D, a.B), 128, 0, stream>>>(a);
        else
            glr_fwd_seq_kernel<T, G><<<grid_of(a.D, a.B), 128, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_glr_step(const void* x, long long x_stride,
                            const void* la, long long la_stride, float* S,
                            void* o, int N, int D, kla_dtype dtype,
                            kla_dtype gdtype, cudaStream_t stream) {
    return by_type(dtype, gdtype, [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        glr_step_kernel<T, G><<<grid_of(D, N), 128, 0, stream>>>(
            static_cast<const T*>(x), x_stride, static_cast<const G*>(la),
            la_stride, S, static_cast<T*>(o), N, D);
        return cudaGetLastError();
    });
}

}  // namespace kla
