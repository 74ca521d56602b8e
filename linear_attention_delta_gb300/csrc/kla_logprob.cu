// Log probabilities of given tokens, with entropy and the largest
// alternatives, and their gradient.
//
// Forward, one pass over a row x with its running maximum m, in powers of two:
//   e = scale log2(e) (x - m),  s = sum 2^e,  t = sum 2^e e
//   lse = scale m + log s,      entropy = log s - t log(2) / s,
//   logp = scale (x - m) - log s
// (with m the maximum both terms of the entropy are of one sign and nothing
// cancels: relative to a number up to 40 below it, entropies under 1 came out
// up to 1e-5 off and below 0; and a difference of logits has the digits that
// one of scaled logits has lost where rows are far from 0),
// and where two partial results meet, with m' = max(m1, m2) and e of m - m':
//   s' = sum 2^e s,             t' = sum 2^e (t + s e).
// A row is read once; it belongs to one block, or, when there are few long
// rows, to a cluster of up to 8 that join their sums on chip.  Bound by HBM
// where there are many rows (8192 x 32000 bf16: 82 us, 0.94 of it; gradient 166
// us, 0.93); few rows are bound by the launch and its ramp (256 x 131072: 20 us,
// of which the bytes take 10).
//
// The largest: each thread keeps its own maximum.  The top-th largest of the
// block's maxima is a lower bound of the row's top-th logit, and only the few
// threads whose maximum reaches it read their part of the row again (from L2)
// and hand in what is not below it (8 alternatives of 8192 x 32000: 111 us, 20
// of 256 x 131072: 30).  Where ties make that more than fits, the row is
// searched round by round instead.
#include <cooperative_groups.h>

#include <algorithm>

#include "f32x2.cuh"
#include "kla_internal.cuh"

namespace kla {
namespace {

namespace cg = cooperative_groups;
using bf16 = __nv_bfloat16;
using u64 = unsigned long long;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kCand = 1024;      // candidates a block can hold
constexpr int kMaxParts = 8;     // blocks of a cluster
static_assert(kMaxParts * kLogprobMaxTop <= kCand, "room for all parts");

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
// One key a logit: its order above, then the lower id.  0 is none, and ~0 is
// above all of them (NaN at id 0 too).
__device__ __forceinline__ u64 key_of(float x, int id) {
    return (u64)order_of(x) << 32 | (0xfffffffeu - id);
}
__device__ __forceinline__ unsigned id_of(u64 key) {
    return 0xfffffffeu - (unsigned)key;
}

// The larger of two, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct Sums {
    float m, s, t;
};
// -300 in place of an e far below: 2^e of both is 0, and 0 * -300 is no NaN
// where 0 * -inf is.  (k: scale log2(e))
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b, float k) {
    const float m = max_nan(a.m, b.m);
    if (m == -INFINITY) return a;
    const float ea = max_nan((a.m - m) * k, -300.f);
    const float eb = max_nan((b.m - m) * k, -300.f);
    const float ca = ex2(ea), cb = ex2(eb);
    return {m, ca * a.s + cb * b.s,
            ca * fmaf(a.s, ea, a.t) + cb * fmaf(b.s, eb, b.t)};
}

// Moves the sums to logits of which `top` is the largest, if it is the largest
// so far.
__device__ __forceinline__ void refer(Sums& a, float top, float k) {
    if (top <= a.m) return;                            // (NaN goes on)
    const float m = max_nan(a.m, top);
    const float e = max_nan((a.m - m) * k, -300.f), c = ex2(e);
    a.t = c * fmaf(a.s, e, a.t);
    a.s *= c;
    a.m = m;
}
// The sums of LANES adjacent lanes.
template <int LANES>
__device__ __forceinline__ Sums join_lanes(Sums a, float k) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1)
        a = join(a, Sums{__shfl_xor_sync(~0u, a.m, o),
                         __shfl_xor_sync(~0u, a.s, o),
                         __shfl_xor_sync(~0u, a.t, o)}, k);
    return a;
}
// N logits into a thread's sums.
template <int N>
__device__ __forceinline__ void add(Sums& a, const float (&v)[N], float k) {
    if (a.m == -INFINITY) return;                      // all masked so far
    float2 s = both(0.f), t = both(0.f);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 d =
            add2(make_float2(v[i], i + 1 < N ? v[i + 1] : -INFINITY),
                 both(-a.m));
        float2 e = mul2(d, both(k));
        e.x = max_nan(e.x, -300.f);
        e.y = max_nan(e.y, -300.f);
        const float2 p = make_float2(ex2(e.x), ex2(e.y));
        s = add2(s, p);
        t = fma2(p, e, t);
    }
    a.s += s.x + s.y;
    a.t += t.x + t.y;
}

// 16 bytes of logits: as loaded, as floats, and the largest of K such.
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    using Raw = float4;
    static __device__ __forceinline__ Raw none() {
        return make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
    static __device__ __forceinline__ void floats(const Raw& v,
                                                  float (&x)[4]) {
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    }
    template <int K>
    static __device__ __forceinline__ float largest(const Raw (&v)[K]) {
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < K; ++k)
            m = max_nan(m, max_nan(max_nan(v[k].x, v[k].y),
                                   max_nan(v[k].z, v[k].w)));
        return m;
    }
};
template <> struct Vec<bf16> {
    static constexpr int N = 8;
    using Raw = uint4;
    static __device__ __forceinline__ Raw none() {
        return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
    }
    static __device__ __forceinline__ void floats(const Raw& v,
                                                  float (&x)[8]) {
        const unsigned u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = from_bf16x2(u[i]);
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ unsigned two(unsigned a, unsigned b) {
        unsigned r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    template <int K>
    static __device__ __forceinline__ float largest(const Raw (&v)[K]) {
        unsigned m = 0xff80ff80u;
#pragma unroll
        for (int k = 0; k < K; ++k)
            m = two(m, two(two(v[k].x, v[k].y), two(v[k].z, v[k].w)));
        const float2 f = from_bf16x2(m);
        return max_nan(f.x, f.y);
    }
};
template <typename T>
__device__ __forceinline__ typename Vec<T>::Raw load(const T* x) {
    return *reinterpret_cast<const typename Vec<T>::Raw*>(x);
}

// Part of a row: [begin, end); its whole 16-byte pieces are [first, last).
struct Range {
    int begin, first, last, end;
};
template <typename T>
__device__ __forceinline__ Range range_of(const T* x, int begin, int end) {
    constexpr int N = Vec<T>::N;
    const int off = (int)((reinterpret_cast<uintptr_t>(x + begin) & 15) /
                          sizeof(T));
    const int first = min(end, off ? begin + N - off : begin);
    return {begin, first, first + (end - first) / N * N, end};
}

// piece(id, values) for each of this thread's pieces of the range, after
// ready(the pieces as loaded, up to four at a time); single(id, value) for what
// is before and behind them.  The same split whenever called.
template <typename T, int NT, typename R, typename F, typename G>
__device__ __forceinline__ void for_each(const T* x, const Range& r, R ready,
                                         F piece, G single) {
    constexpr int N = Vec<T>::N;
    using Raw = typename Vec<T>::Raw;
    const int tid = threadIdx.x;
    // (distances from r.last: an id past it may pass 2^31)
    int i = r.first + tid * N;
    for (; r.last - i > 3 * NT * N; i += 4 * NT * N) {
        Raw v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = load(x + i + k * NT * N);
        ready(v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float f[N];
            Vec<T>::floats(v[k], f);
            piece(i + k * NT * N, f);
        }
    }
    // the up to three pieces left, on their way together too
    if (r.last - i > 0) {
        Raw v[3];
        v[0] = load(x + i);
#pragma unroll
        for (int k = 1; k < 3; ++k)
            v[k] = r.last - i > k * NT * N ? load(x + i + k * NT * N)
                                           : Vec<T>::none();
        ready(v);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (r.last - i <= k * NT * N) break;
            float f[N];
            Vec<T>::floats(v[k], f);
            piece(i + k * NT * N, f);
        }
    }
    if (r.begin + tid < r.first)
        single(r.begin + tid, to_f32(x[r.begin + tid]));
    if (r.last + tid < r.end) single(r.last + tid, to_f32(x[r.last + tid]));
}
struct Nothing {
    template <typename V> __device__ void operator()(const V&) const {}
};

// This thread's sums over its share of a range.
template <typename T, int NT>
__device__ __forceinline__ Sums sums_of(const T* x, const Range& r, float k) {
    Sums acc{-INFINITY, 0.f, 0.f};
    for_each<T, NT>(
        x, r, [&](const auto& v) { refer(acc, Vec<T>::largest(v), k); },
        [&](int, const float (&v)[Vec<T>::N]) { add(acc, v, k); },
        [&](int, float v) {
            const float one[1] = {v};
            refer(acc, v, k);
            add(acc, one, k);
        });
    return acc;
}
__device__ __forceinline__ float in_twos(float scale) {
    return fminf(scale * kLog2e, 3.4e38f);      // (0 times it is no NaN)
}
// scale m + ls, not below scale m whatever is rounded.
__device__ __forceinline__ float lse_of(float scale, float m, float ls) {
    return max_nan(fmaf(scale, m, ls), __fmul_ru(scale, m));
}

template <int NT>
__device__ __forceinline__ u64 block_max(u64 k, u64* keys) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const u64 y = __shfl_xor_sync(~0u, k, o);
        k = y > k ? y : k;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) keys[threadIdx.x >> 5] = k;
    __syncthreads();
    k = keys[0];
    for (int w = 1; w < NT / 32; ++w) k = keys[w] > k ? keys[w] : k;
    return k;
}

template <int NT> struct Shared {
    Sums part[NT / 32];
    Sums whole;                  // of this block's part
    u64 keys[NT / 32];
    u64 top[kLogprobMaxTop];     // this block's largest, sorted
    u64 cand[kCand];
    alignas(16) unsigned maxima[NT];
    unsigned bound;
    int count;
};

// The `top` largest of this block's part into sh.top, sorted (0: none).
// own: the largest order among the thread's logits (-inf's if it has none).
template <typename T, int NT>
__device__ __forceinline__ void largest(Shared<NT>& sh, const T* x,
                                        const Range& r, int top,
                                        unsigned own) {
    const int tid = threadIdx.x, lane = tid & 31;
    // the maxima of groups of four threads do while there are far more of
    // them than `top`
    const int G = top <= NT / 8 ? 4 : 1, groups = NT / G;
    unsigned gm = own;
    if (G == 4) {
        gm = max(gm, __shfl_xor_sync(~0u, gm, 1));
        gm = max(gm, __shfl_xor_sync(~0u, gm, 2));
    }
    sh.maxima[tid / G] = gm;
    if (tid == 0) sh.count = 0, sh.bound = 0;
    __syncthreads();
    // the top-th largest: each thread of a group compares with its share
    {
        int above = 0, level = 0;
        const int share = groups / G, from = tid % G * share;
        for (int i = from; i < from + share; i += 4) {
            const uint4 m = *reinterpret_cast<const uint4*>(&sh.maxima[i]);
            above += (m.x > gm) + (m.y > gm) + (m.z > gm) + (m.w > gm);
            level += (m.x == gm) + (m.y == gm) + (m.z == gm) + (m.w == gm);
        }
        if (G == 4) {
#pragma unroll
            for (int o = 1; o < 4; o *= 2) {
                above += __shfl_xor_sync(~0u, above, o);
                level += __shfl_xor_sync(~0u, level, o);
            }
        }
        if (above < top && above + level >= top) sh.bound = gm;
    }
    __syncthreads();
    const unsigned bound = sh.bound;
    // a warp reads the pieces of each of its threads that reach the bound
    constexpr int N = Vec<T>::N;
    unsigned found = __ballot_sync(~0u, own >= bound);
    auto take = [&](int id, float v) {
        if (order_of(v) < bound) return;
        const int at = atomicAdd(&sh.count, 1);
        if (at < kCand) sh.cand[at] = key_of(v, id);
    };
    while (found) {
        // two at a time: both threads' pieces are on their way together
        const int t0 = (tid & ~31) + __ffs(found) - 1;
        found &= found - 1;
        const int t1 = found ? (tid & ~31) + __ffs(found) - 1 : -1;
        found &= found - 1;
        // (a piece's distance from r.first, in 64 bits)
        for (long long at = (long long)lane * NT * N; at < r.last - r.first;
             at += 32ll * NT * N) {
            const long long i0 = r.first + at + t0 * N;
            const long long i1 = r.first + at + t1 * N;
            const bool in0 = i0 < r.last, in1 = t1 >= 0 && i1 < r.last;
            typename Vec<T>::Raw w0 = Vec<T>::none(), w1 = w0;
            if (in0) w0 = load(x + i0);
            if (in1) w1 = load(x + i1);
            float v[N];
            if (in0) {
                Vec<T>::floats(w0, v);
#pragma unroll
                for (int k = 0; k < N; ++k) take((int)i0 + k, v[k]);
            }
            if (in1) {
                Vec<T>::floats(w1, v);
#pragma unroll
                for (int k = 0; k < N; ++k) take((int)i1 + k, v[k]);
            }
        }
        const int t = lane < 2 ? t0 : t1;
        if (t >= 0 && lane < 4) {
            const int i = lane & 1 ? r.last + t : r.begin + t;
            if (i < (lane & 1 ? r.end : r.first)) take(i, to_f32(x[i]));
        }
    }
    __syncthreads();
    const int n = sh.count;
    if (n <= kCand) {
        // its rank is the number of larger keys (no two are equal)
        for (int i = tid; i < n; i += NT) {
            const u64 k = sh.cand[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += sh.cand[j] > k;
            if (rank < top) sh.top[rank] = k;
        }
        for (int i = n + tid; i < top; i += NT) sh.top[i] = 0;
        __syncthreads();
        return;
    }
    u64 last = ~0ull;
    for (int i = 0; i < top; ++i) {
        u64 best = 0;
        auto look = [&](int id, float v) {
            const u64 k = key_of(v, id);
            if (k < last && k > best) best = k;
        };
        for_each<T, NT>(
            x, r, Nothing(),
            [&](int id, const float (&v)[Vec<T>::N]) {
#pragma unroll
                for (int k = 0; k < Vec<T>::N; ++k) look(id + k, v[k]);
            },
            look);
        last = block_max<NT>(best, sh.keys);
        if (tid == 0) sh.top[i] = last;
    }
    __syncthreads();
}

// grid: rows x parts (a cluster each where parts > 1).
template <typename T, int NT, bool TOP>
__global__ void __launch_bounds__(NT, 1536 / NT)
logprob_fwd(LogprobArgs a, int parts) {
    __shared__ Shared<NT> sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t row = blockIdx.x / parts;
    const int part = blockIdx.x % parts;
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    const int len = (a.V + parts - 1) / parts;
    const int begin = (int)min((long long)a.V, (long long)part * len);
    const Range r = range_of(x, begin, min(a.V, begin + len));
    await_grid_before();
    release_grid_after();
    const float k = in_twos(a.scale);
    Sums acc = sums_of<T, NT>(x, r, k);
    const float own = acc.m;     // the largest of this thread's
    acc = join_lanes<32>(acc, k);
    if (lane == 0) sh.part[warp] = acc;
    __syncthreads();
    if (warp == 0) {
        acc = lane < NT / 32 ? sh.part[lane] : Sums{-INFINITY, 0.f, 0.f};
        acc = join_lanes<NT / 32>(acc, k);
        if (lane == 0) sh.whole = acc;
    }
    if (TOP) largest<T, NT>(sh, x, r, a.top, order_of(own));
    else __syncthreads();

    // one block of the row writes; the others' sums and largest come over
    // the cluster's shared memory, in the order of the parts
    if (parts > 1) cg::this_cluster().sync();
    if (part == 0) {
        if (parts > 1) {
            if (warp == 0) {
                Sums all{-INFINITY, 0.f, 0.f};
                if (lane < parts)
                    all = *cg::this_cluster().map_shared_rank(&sh.whole, lane);
                all = join_lanes<kMaxParts>(all, k);
                if (lane == 0) sh.part[0] = all;
            }
            if (TOP) {
                for (int i = tid; i < parts * a.top; i += NT)
                    sh.cand[i] = cg::this_cluster().map_shared_rank(
                        sh.top, i / a.top)[i % a.top];
            }
            __syncthreads();
        }
        const Sums all = parts > 1 ? sh.part[0] : sh.whole;
        // the largest z; below the range of fp32 it is masked, above it NaN
        const float top = a.scale * all.m;
        const bool none = top == -INFINITY;
        const float ls =
            top == INFINITY ? __uint_as_float(0x7fc00000u) : logf(all.s);
        const float lse = none ? -INFINITY : lse_of(a.scale, all.m, ls);
        auto logp = [&](float v) {
            return none ? -INFINITY : fmaf(v - all.m, a.scale, -ls);
        };
        if (tid == 0) {
            const long long t = a.tokens[row];
            float lp = 0.f;
            if (t >= 0 && t < a.V)
                lp = logp(to_f32(x[t]));
            a.logp[row] = lp;
            if (a.entropy)
                a.entropy[row] = none ? 0.f : fmaf(-kLn2, all.t / all.s, ls);
            if (a.lse) a.lse[row] = lse;
        }
        if (TOP) {
            const u64* keys = parts > 1 ? sh.cand : sh.top;
            const int n = parts * a.top;
            for (int i = tid; i < n; i += NT) {
                const u64 k = keys[i];
                if (k == 0) continue;
                // its place: the number of larger keys
                int rank = parts > 1 ? 0 : i;
                if (parts > 1)
                    for (int j = 0; j < n; ++j) rank += keys[j] > k;
                if (rank >= a.top) continue;
                const size_t out = row * a.top + rank;
                const float v = value_of((unsigned)(k >> 32));
                a.top_logp[out] = logp(v);
                a.top_ids[out] = id_of(k);
            }
        }
    }
    if (parts > 1) cg::this_cluster().sync();    // its shared memory is read
}

// ---------------------------------------------------------------- gradient

// d_j = -p_j (g + ge (log p_j + H)), + g at the token, times scale.
//
// log p_j = z_j - lse has lost what lse was rounded by, 2^-24 |lse| at most and
// the same relative to p (in a row of the type's lowest value p would be 1
// throughout).  From |lse| = 1024 on (2^-14) m and log s are formed again, and
// take the place of lse where they round to it; of part of a vocabulary with the
// whole's lse they do not, and lse is taken as it is.  Each block of such a row
// reads all of it, or, in place, the first one has it to itself (us if all rows
// are such: 8192 x 32000 bf16 246 for 166, 256 x 131072 160 for 27).  In 32
// registers: unbound it takes 40 and 45, and other rows 186 us for 166.
constexpr float kFar = 1024.f;
template <typename T, int NT, bool IN_PLACE>
__global__ void __launch_bounds__(NT, 2048 / NT)
logprob_bwd(LogprobBwdArgs a, int parts) {
    constexpr int N = Vec<T>::N;
    const size_t row = blockIdx.x / parts;
    const int part = blockIdx.x % parts;
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    T* y = static_cast<T*>(a.logits_grad) + row * a.V;
    const int len = (a.V + parts - 1) / parts;
    int begin = (int)min((long long)a.V, (long long)part * len);
    int end = min(a.V, begin + len);
    await_grid_before();
    release_grid_after();
    const float lse = a.lse[row];
    float x0 = 0.f, z0 = lse;    // log p = scale (x - x0) - z0
    if (fabsf(lse) >= kFar && fabsf(lse) < INFINITY) {
        if (IN_PLACE) {
            if (part > 0) return;
            begin = 0, end = a.V;
        }
        __shared__ Sums of_warp[NT / 32];
        const float k = in_twos(a.scale);
        Sums all = join_lanes<32>(sums_of<T, NT>(x, range_of(x, 0, a.V), k), k);
        if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x >> 5] = all;
        __syncthreads();
        all = of_warp[0];
        for (int w = 1; w < NT / 32; ++w) all = join(all, of_warp[w], k);
        const float ls = logf(all.s);
        if (fabsf(lse_of(a.scale, all.m, ls) - lse) <= 0x1p-22f * fabsf(lse))
            x0 = all.m, z0 = ls;
    }
    const long long t = a.tokens[row];
    const bool some = t >= 0 && t < a.V && lse != -INFINITY;
    const float g = a.logp_grad && some ? a.logp_grad[row] : 0.f;
    const float ge = a.entropy_grad ? a.entropy_grad[row] : 0.f;
    const float H = a.entropy_grad ? a.entropy[row] : 0.f;
    const int at = g != 0.f ? (int)t : -1;
    // -200 in place of a log p far below: p is 0, and 0 * -200 is no NaN
    auto grad = [&](int id, float v) {
        const float lp = lse == -INFINITY
                             ? -200.f
                             : max_nan(fmaf(v - x0, a.scale, -z0), -200.f);
        const float p = expf(lp);
        float d = -p * fmaf(ge, lp + H, g);
        if (id == at) d += g;
        return d * a.scale;
    };
    const Range r = range_of(x, begin, end);
    if (((reinterpret_cast<uintptr_t>(x + r.first) |
          reinterpret_cast<uintptr_t>(y + r.first)) & 15) == 0) {
        auto piece = [&](int id, const float (&v)[N]) {
            float d[N];
#pragma unroll
            for (int k = 0; k < N; ++k) d[k] = grad(id + k, v[k]);
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4*>(y + id) =
                    make_float4(d[0], d[1], d[2], d[3]);
            } else {
                __nv_bfloat162 o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[k] = __floats2bfloat162_rn(d[2 * k], d[2 * k + 1]);
                *reinterpret_cast<uint4*>(y + id) =
                    *reinterpret_cast<const uint4*>(o);
            }
        };
        for_each<T, NT>(x, r, Nothing(), piece, [&](int id, float v) {
            y[id] = from_f32<T>(grad(id, v));
        });
    } else {
        // logits and gradient rows that do not line up
        int i = begin + threadIdx.x;
        for (; end - i > 3 * NT; i += 4 * NT) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = to_f32(x[i + k * NT]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                y[i + k * NT] = from_f32<T>(grad(i + k * NT, v[k]));
        }
        for (; i < end; i += NT) y[i] = from_f32<T>(grad(i, to_f32(x[i])));
    }
}

// ---------------------------------------------------------------- launch

template <typename... P, typename... A>
cudaError_t launch_rows(void (*kernel)(P...), long long rows, int parts,
                        int threads, bool cluster, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * parts));
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster && parts > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args..., parts);
}

template <typename T, int NT>
cudaError_t launch_fwd_of(const LogprobArgs& a, int parts, cudaStream_t s) {
    return a.top ? launch_rows(logprob_fwd<T, NT, true>, a.N, parts, NT, true,
                               s, a)
                 : launch_rows(logprob_fwd<T, NT, false>, a.N, parts, NT,
                               true, s, a);
}
// Blocks of a row: up to four for every SM, of at least 16384 logits
// (measured, us with a row in one block and over a cluster: 1 x 32000 with 8
// alternatives 7.3 and 8.1, 64 x 32000 with 20 11.4 and 12.8, 8 x 131072 10.7 and
// 4.4, 256 x 131072 20.1 and 20.2, with 20 alternatives 32.2 and 30.3).  128
// threads for short rows (4096 x 1000 8.1 and 12.1 with 256, with 8 alternatives
// 23.5 and 34.5) and for more rows than fit the SMs twice at that size: blocks
// then start and end more evenly (8192 x 32000 81 and 85; but 1023 x 50257 28 and
// 24).
template <typename T>
cudaError_t launch_fwd(const LogprobArgs& a, cudaStream_t s) {
    int parts = 1;
    while (parts < kMaxParts && (long long)a.N * parts * 2 <= 4 * kPlanSMs &&
           a.V / (parts * 2) >= 16384)
        parts *= 2;
    return a.V / parts <= 4096 || a.N >= 24 * kPlanSMs
               ? launch_fwd_of<T, 128>(a, parts, s)
               : launch_fwd_of<T, 256>(a, parts, s);
}

// Many small blocks: up to 32 an SM, of at least 4096 logits (measured, us:
// 8192 x 32000 in 1, 2 and 8 blocks a row 166, 173, 224; 256 x 131072 in 8, 16
// and, by this rule, 19 27.5, 25.9, 26.9; 512 x 32000 in 4 and 7 16.5, 14.9).
template <typename T>
cudaError_t launch_bwd(const LogprobBwdArgs& a, cudaStream_t s) {
    const int parts =
        std::max(1, std::min({32 * kPlanSMs / a.N, a.V / 4096, 64}));
    return launch_rows(a.logits == a.logits_grad ? logprob_bwd<T, 128, true>
                                                 : logprob_bwd<T, 128, false>,
                       a.N, parts, 128, false, s, a);
}

}  // namespace

cudaError_t launch_logprob(const LogprobArgs& a, cudaStream_t stream) {
    return a.dtype == KLA_BF16 ? launch_fwd<bf16>(a, stream)
                               : launch_fwd<float>(a, stream);
}

cudaError_t launch_logprob_bwd(const LogprobBwdArgs& a, cudaStream_t stream) {
    return a.dtype == KLA_BF16 ? launch_bwd<bf16>(a, stream)
                               : launch_bwd<float>(a, stream);
}

}  // namespace kla
