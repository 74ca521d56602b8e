// Log probabilities of given tokens, with entropy and the largest
// alternatives, and their gradient.
//
// Forward, one pass over a row with a running maximum m (z = scale x):
//   s = sum exp(z - m),  t = sum exp(z - m) (z - m)
//   lse = m + log s,     entropy = log s - t / s
// and where two partial results meet, with m' = max(m1, m2), c = exp(m - m'):
//   s' = sum c s,        t' = sum c (t + s (m - m')).
#include "kla_internal.cuh"

namespace kla {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kNT = 256;

// Order of logits as whole numbers: larger values first, NaN above all.
__device__ __forceinline__ unsigned order_of(float x) {
    if (x != x) return 0xffffffffu;
    const unsigned u = __float_as_uint(x + 0.f);     // -0 counts as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned u) {
    return u == 0xffffffffu ? __uint_as_float(0x7fc00000u)
           : __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
// One key a logit: its order above, then the lower id.  0 is none.
__device__ __forceinline__ unsigned long long key_of(float x, int id) {
    return (unsigned long long)order_of(x) << 32 | (0xffffffffu - id);
}

// The larger of two, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Sums {
    float m, s, t;
};
// exp(d) and d of a difference d <= 0 from the maximum; -200 in place of
// what is far below has exp = 0, and 0 * -200 is no NaN.
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
    const float m = max_nan(a.m, b.m);
    if (m == -INFINITY) return a;
    const float da = max_nan(a.m - m, -200.f), db = max_nan(b.m - m, -200.f);
    const float ca = expf(da), cb = expf(db);
    return {m, ca * a.s + cb * b.s,
            ca * fmaf(a.s, da, a.t) + cb * fmaf(b.s, db, b.t)};
}
__device__ __forceinline__ void add(Sums& x, float z) {
    x = join(x, Sums{z, 1.f, 0.f});
}

template <typename T>
__global__ void __launch_bounds__(kNT) logprob_fwd(LogprobArgs a) {
    __shared__ Sums part[kNT / 32];
    __shared__ unsigned long long keys[kNT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    Sums acc{-INFINITY, 0.f, 0.f};
    for (int i = tid; i < a.V; i += kNT) add(acc, to_f32(x[i]) * a.scale);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        acc = join(acc, Sums{__shfl_xor_sync(~0u, acc.m, o),
                             __shfl_xor_sync(~0u, acc.s, o),
                             __shfl_xor_sync(~0u, acc.t, o)});
    if (lane == 0) part[warp] = acc;
    __syncthreads();
    acc = part[0];
    for (int w = 1; w < kNT / 32; ++w) acc = join(acc, part[w]);
    const bool none = acc.m == -INFINITY;
    const float ls = logf(acc.s), lse = none ? -INFINITY : acc.m + ls;
    if (tid == 0) {
        const long long t = a.tokens[row];
        float lp = 0.f;
        if (t >= 0 && t < a.V)
            lp = none ? -INFINITY : to_f32(x[t]) * a.scale - lse;
        a.logp[row] = lp;
        if (a.entropy) a.entropy[row] = none ? 0.f : ls - acc.t / acc.s;
        if (a.lse) a.lse[row] = lse;
    }
    unsigned long long last = ~0ull;
    for (int n = 0; n < a.top; ++n) {
        unsigned long long best = 0;
        for (int i = tid; i < a.V; i += kNT) {
            const unsigned long long k = key_of(to_f32(x[i]), i);
            if (k < last && k > best) best = k;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const unsigned long long k = __shfl_xor_sync(~0u, best, o);
            best = k > best ? k : best;
        }
        __syncthreads();
        if (lane == 0) keys[warp] = best;
        __syncthreads();
        for (int w = 0; w < kNT / 32; ++w)
            best = keys[w] > best ? keys[w] : best;
        last = best;
        if (tid == 0) {
            const size_t at = row * a.top + n;
            const float z = value_of((unsigned)(best >> 32)) * a.scale;
            a.top_logp[at] = none ? -INFINITY : z - lse;
            a.top_ids[at] = 0xffffffffu - (unsigned)best;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kNT) logprob_bwd(LogprobBwdArgs a) {
    const size_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    T* y = static_cast<T*>(a.logits_grad) + row * a.V;
    const float lse = a.lse[row];
    const long long t = a.tokens[row];
    const bool some = t >= 0 && t < a.V && lse != -INFINITY;
    const float g = a.logp_grad && some ? a.logp_grad[row] : 0.f;
    const float ge = a.entropy_grad ? a.entropy_grad[row] : 0.f;
    const float H = a.entropy_grad ? a.entropy[row] : 0.f;
    for (int i = threadIdx.x; i < a.V; i += kNT) {
        // log p; -200 in place of what is far below (p = 0)
        const float lp = lse == -INFINITY ? -200.f
            : max_nan(fmaf(to_f32(x[i]), a.scale, -lse), -200.f);
        const float p = expf(lp);
        float d = -p * fmaf(ge, lp + H, g);
        if (i == t) d += g;
        y[i] = from_f32<T>(d * a.scale);
    }
}

}  // namespace

cudaError_t launch_logprob(const LogprobArgs& a, cudaStream_t stream) {
    if (a.dtype == KLA_BF16)
        logprob_fwd<bf16><<<a.N, kNT, 0, stream>>>(a);
    else
        logprob_fwd<float><<<a.N, kNT, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_logprob_bwd(const LogprobBwdArgs& a, cudaStream_t stream) {
    if (a.dtype == KLA_BF16)
        logprob_bwd<bf16><<<a.N, kNT, 0, stream>>>(a);
    else
        logprob_bwd<float><<<a.N, kNT, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kla
