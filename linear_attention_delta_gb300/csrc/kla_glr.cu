// Gated linear recurrence, per sequence and channel:
//
//   h_t = alpha_t h_{t-1} + x_t,  alpha_t = exp(log_alpha_t),  o_t = h_t
//
// and its reverse: g_t = do_t + alpha_{t+1} g_{t+1}, dx_t = g_t,
// dlog_alpha_t = alpha_t g_t h_{t-1}, dh0 = alpha_1 g_1.  Bound by HBM: three
// to five operations per element of each tensor it reads.
#include "kla_internal.cuh"
#include "tc_primitives.cuh"

namespace kla {
namespace {

using bf16 = __nv_bfloat16;

// ---------------------------------------------------------------------------
// The scan.  A tile is L = W * S consecutive tokens (in scan order: backwards
// in the backward pass) of 32 * VEC channels; warp w of its block holds S of
// the tokens in registers, a lane VEC channels.  Tiles of one run of tokens
// and one group of channels form a chain.  A block
//   1. loads its tile (each input element is read once),
//   2. reduces each warp's S steps to the affine map c -> P c + H of the
//      state, and the warps' maps to the tile's,
//   3. publishes the map, and finds the state before the tile: it polls the W
//      tiles before it (a warp each) until one has published its last state
//      and all between that one and this have published their maps,
//   4. publishes its own last state, and runs its steps again from the
//      now known state, writing the outputs.
// The state before a tile is always formed as P_{k-1} c_{k-1} + H_{k-1} from
// left to right, wherever the nearest published state was found, so the
// result has the same bits on every run.  Blocks take their tile from a
// counter, in token order, so that a block only waits for blocks that run
// already.
//
// A state that a sequence starts from replaces c (it is not multiplied by
// zero), so nothing of one packed sequence, not even a NaN, reaches the next.

// Workspace of the scan: the tile counter, then per tile and channel the map
// (P, H) and the last state.  Everything starts as all ones, which no
// published value is (see `publishable`).
struct ScanPlan {
    int tiles, groups, chains;   // tiles of a chain; channel groups; chains
    unsigned int* counter;
    unsigned long long* map;
    unsigned int* last;
};

constexpr unsigned int kEmpty = 0xffffffffu;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ unsigned int g_fault_glr = 0;

// The bits of x; a NaN with all bits set becomes another NaN.
__device__ __forceinline__ unsigned int publishable(float x) {
    const unsigned int b = __float_as_uint(x);
    return b == kEmpty ? 0x7fffffffu : b;
}

__device__ __forceinline__ void st_relaxed(unsigned long long* p,
                                           unsigned long long v) {
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v)
                 : "memory");
}
__device__ __forceinline__ void st_relaxed(unsigned int* p, unsigned int v) {
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v)
                 : "memory");
}
__device__ __forceinline__ unsigned long long ld_relaxed(
    const unsigned long long* p) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];"
                 : "=l"(v)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ unsigned int ld_relaxed(const unsigned int* p) {
    unsigned int v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];"
                 : "=r"(v)
                 : "l"(p)
                 : "memory");
    return v;
}

// P c + H; a zero state stays zero however large P grew.
__device__ __forceinline__ float apply(float P, float H, float c) {
    return c == 0.f ? H : fmaf(P, c, H);
}

// VEC adjacent elements as they lie in memory.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

// Where sequences begin and end among S tokens of one warp, and which.  In
// scan order: bit i of `mask` says that a sequence begins at step i, which is
// also the end of the one before it, after step i - 1; n is the sequence of
// step 0.
struct Bounds {
    unsigned int mask;
    int n;
};

// Packed sequences: the boundaries among the S tokens from t on (upwards, or
// downwards with BACK).  A warp works together: a 32-way search for the
// sequence of t, then 32 offsets at a time.  Any content of cu gives
// 0 <= n < B.
template <int S, bool BACK>
__device__ __forceinline__ Bounds find_bounds(const int* cu, int B,
                                              long long t) {
    const int lane = threadIdx.x % 32;
    int lo = 0, len = B;
    while (len > 1) {
        const int step = (len + 31) / 32;
        const int i = lane * step;
        const bool le = i < len && cu[lo + i] <= t;
        const int cnt = max(1, __popc(__ballot_sync(0xffffffffu, le)));
        const int skip = (cnt - 1) * step;
        lo += skip;
        len = min(step, len - skip);
    }
    unsigned int mask = 0;
    for (int j0 = BACK ? lo + 1 : lo;;) {
        const int j = BACK ? j0 - lane : j0 + lane;
        long long pos = -1;          // step at which the boundary lies
        bool beyond = true;
        if (j >= 0 && j <= B) {
            pos = BACK ? t + 1 - cu[j] : cu[j] - t;
            beyond = pos > S;
        }
        mask |= __reduce_or_sync(0xffffffffu,
                                 pos >= 0 && pos <= S ? 1u << pos : 0u);
        if (__any_sync(0xffffffffu, beyond)) break;
        j0 += BACK ? -32 : 32;
    }
    return {mask, lo};
}

template <typename T, typename G, int VEC, int S, int W, bool BWD,
          bool PACKED>
__global__ void __launch_bounds__(32 * W)
glr_scan_kernel(GlrArgs a, ScanPlan plan) {
    constexpr int CH = 32 * VEC;
    using PT = Pack<T, VEC>;
    using PG = Pack<G, VEC>;
    __shared__ float sP[W][CH], sH[W][CH];     // the warps' maps
    __shared__ float vP[W][CH], vH[W][CH];     // the tiles before
    __shared__ unsigned int s_ticket, s_begins[W];
    __shared__ int s_seen[W];

    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    unsigned int ticket = blockIdx.x;
    if (plan.tiles > 1) {
        if (threadIdx.x == 0) s_ticket = atomicAdd(plan.counter, 1u) + 1u;
        __syncthreads();
        ticket = s_ticket;
    }
    const int k = ticket / plan.chains;        // tile of the chain
    const int chain = ticket % plan.chains;
    const int group = chain % plan.groups;
    const int b = chain / plan.groups;         // 0 when packed
    const int d = group * CH + lane * VEC;
    const bool live = d < a.D;

    // scan position p <-> token t
    const long long p0 = (long long)k * (W * S) + w * S;
    const long long t0 = BWD ? a.T - 1 - p0 : p0;
    const int steps = (int)max(0ll, min((long long)S, a.T - p0));
    constexpr int DT = BWD ? -1 : 1;

    const T* xp = static_cast<const T*>(a.x.p) + b * a.x.sb + d;
    const G* lp = static_cast<const G*>(a.la.p) + b * a.la.sb + d;
    const T* gp = static_cast<const T*>(a.g.p) + b * a.g.sb + d;
    PT rx[S];                    // forward: x; backward: o of the token before
    PT rg[BWD ? S : 1];          // backward: o_grad
    PG rl[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
        rl[i] = PG{};
        rx[i] = PT{};
        if (BWD) rg[BWD ? i : 0] = PT{};
        if (live && i < steps) {
            const long long t = t0 + i * DT;
            rl[i] = *reinterpret_cast<const PG*>(lp + t * a.la.st);
            if (BWD) {
                rg[BWD ? i : 0] =
                    *reinterpret_cast<const PT*>(gp + t * a.g.st);
                if (t > 0)
                    rx[i] =
                        *reinterpret_cast<const PT*>(xp + (t - 1) * a.x.st);
            } else {
                rx[i] = *reinterpret_cast<const PT*>(xp + t * a.x.st);
            }
        }
    }

    Bounds bd{0u, b};
    if (PACKED) {
        if (steps > 0) bd = find_bounds<S, BWD>(a.cu, a.B, t0);
    } else {
        if (p0 == 0) bd.mask = 1u;
        if (steps > 0 && a.T - p0 <= S) bd.mask |= 1u << (a.T - p0);
    }
    const unsigned int begins = bd.mask & ((1u << S) - 1);
    const float* init = BWD ? a.dhT : a.h0;

    // Moves n on to the sequence that begins at step i.
    auto next = [&](int i, int& n) {
        if (!PACKED || i == 0) return;
        const long long t = t0 + i * DT;
        if (BWD) {
            n = max(n - 1, 0);
            while (n > 0 && a.cu[n] > t) --n;
        } else {
            n = min(n + 1, a.B - 1);
            while (n < a.B - 1 && a.cu[n + 1] <= t) ++n;
        }
    };
    auto start_of = [&](int n, float (&c)[VEC]) {
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            c[v] = init && live ? init[(size_t)n * a.D + d + v] : 0.f;
    };

    float al[S][VEC];            // alpha
    float P[VEC], H[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        P[v] = 1.f;
        H[v] = 0.f;
    }
    int n = bd.n;
    // the start of the last sequence that begins here: whoever ends it may
    // write its last state in the place of this start (hT == h0) before the
    // second pass
    float kept[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) kept[v] = 0.f;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        if (begins >> i & 1) {
            next(i, n);
            start_of(n, kept);
#pragma unroll
            for (int v = 0; v < VEC; ++v) H[v] = kept[v];
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            al[i][v] = expf(to_f32(rl[i].v[v]));
            P[v] *= al[i][v];
            H[v] = BWD ? al[i][v] * (H[v] + to_f32(rg[BWD ? i : 0].v[v]))
                       : fmaf(al[i][v], H[v], to_f32(rx[i].v[v]));
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        sP[w][lane * VEC + v] = P[v];
        sH[w][lane * VEC + v] = H[v];
    }
    if (lane == 0) s_begins[w] = begins;
    __syncthreads();

    // the tile's map, and whether its last state is known already
    bool known = (s_begins[0] & 1) || k == 0;
    const bool wait = !known;
    const size_t at = ((size_t)chain * plan.tiles + k) * CH + lane * VEC;
    const bool share = plan.tiles > 1 && k + 1 < plan.tiles;
    if (w == 0 && plan.tiles > 1) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            P[v] = 1.f;
            H[v] = 0.f;
        }
        for (int u = 0; u < W; ++u) {
            const bool fresh = s_begins[u] != 0;
            known |= fresh;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float pu = sP[u][lane * VEC + v];
                const float hu = sH[u][lane * VEC + v];
                H[v] = fresh ? hu : apply(pu, hu, H[v]);
                P[v] *= pu;
            }
        }
        if (share) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (known)
                    st_relaxed(plan.last + at + v, publishable(H[v]));
                else
                    st_relaxed(plan.map + at + v,
                               (unsigned long long)publishable(H[v]) << 32 |
                                   publishable(P[v]));
            }
        }
    }

    // the state before the tile
    float c[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) c[v] = 0.f;
    if (wait) {                  // the same in all threads
        int seen = 0;            // 1: the map, 2: the last state
        const size_t from = at - (size_t)(w + 1) * CH;
        const uint64_t begun = tc::globaltimer_ns();
        int r;
        while (true) {
            if (k - 1 - w >= 0 && seen < 2) {
                bool got = true;
                float h[VEC], q[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const unsigned int x = ld_relaxed(plan.last + from + v);
                    h[v] = __uint_as_float(x);
                    q[v] = 0.f;
                    got &= x != kEmpty;
                }
                if (__all_sync(0xffffffffu, got)) {
                    seen = 2;
                } else if (seen == 0) {
                    got = true;
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        const unsigned long long x =
                            ld_relaxed(plan.map + from + v);
                        q[v] = __uint_as_float((unsigned int)x);
                        h[v] = __uint_as_float((unsigned int)(x >> 32));
                        got &= x != ~0ull;
                    }
                    if (__all_sync(0xffffffffu, got)) seen = 1;
                    else got = false;
                } else {
                    got = false;
                }
                if (__all_sync(0xffffffffu, got)) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        vP[w][lane * VEC + v] = q[v];
                        vH[w][lane * VEC + v] = h[v];
                    }
                }
            }
            if (lane == 0) s_seen[w] = seen;
            const bool late = tc::globaltimer_ns() - begun > kWaitLimitNs;
            if (__syncthreads_or(late)) {
                r = -1;
                break;
            }
            r = 0;
            while (r < W && s_seen[r] == 1) ++r;
            if (r < W && s_seen[r] == 2) break;
            __syncthreads();
        }
        if (r < 0) {             // gave up: the tiles after this one go on
            if (threadIdx.x == 0) atomicOr(&g_fault_glr, 1u);
#pragma unroll
            for (int v = 0; v < VEC; ++v) c[v] = __uint_as_float(0x7fffffffu);
        } else {
#pragma unroll
            for (int v = 0; v < VEC; ++v) c[v] = vH[r][lane * VEC + v];
            for (int u = r - 1; u >= 0; --u)
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    c[v] = apply(vP[u][lane * VEC + v],
                                 vH[u][lane * VEC + v], c[v]);
        }
        if (w == 0 && share && !known) {
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                st_relaxed(plan.last + at + v,
                           publishable(apply(P[v], H[v], c[v])));
        }
    }
    // and before this warp's tokens
    for (int u = 0; u < w; ++u) {
        const bool fresh = s_begins[u] != 0;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float hu = sH[u][lane * VEC + v];
            c[v] = fresh ? hu : apply(sP[u][lane * VEC + v], hu, c[v]);
        }
    }

    if (live && steps > 0) {
        const size_t out = (PACKED ? 0 : (size_t)b * a.T * a.D) + d;
        T* op = static_cast<T*>(a.o) + out;
        G* dp = static_cast<G*>(a.dla) + out;
        n = bd.n;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            if (i < steps) {
                const long long t = t0 + i * DT;
                if (begins >> i & 1) {
                    next(i, n);
                    if (begins >> (i + 1)) {
                        start_of(n, c);
                    } else {
#pragma unroll
                        for (int v = 0; v < VEC; ++v) c[v] = kept[v];
                    }
                }
                const bool ends = bd.mask >> (i + 1) & 1;
                PT ro;
                if (BWD) {
                    PG rd;
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        const float g =
                            to_f32(rg[BWD ? i : 0].v[v]) + c[v];
                        ro.v[v] = from_f32<T>(g);
                        c[v] = al[i][v] * g;
                        float h = to_f32(rx[i].v[v]);
                        if (ends)
                            h = a.h0 ? a.h0[(size_t)n * a.D + d + v] : 0.f;
                        rd.v[v] = from_f32<G>(c[v] * h);
                    }
                    *reinterpret_cast<PG*>(dp + t * a.D) = rd;
                } else {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        c[v] = fmaf(al[i][v], c[v], to_f32(rx[i].v[v]));
                        ro.v[v] = from_f32<T>(c[v]);
                    }
                }
                *reinterpret_cast<PT*>(op + t * a.D) = ro;
                if (ends && a.hT) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v)
                        a.hT[(size_t)n * a.D + d + v] = c[v];
                }
            }
        }
    }

    // empty sequences, shared out over the tiles
    if (PACKED && a.hT && a.hT != init && live) {
        for (long long e = (long long)k * W + w; e < a.B;
             e += (long long)plan.tiles * W)
            if (a.cu[e] == a.cu[e + 1])
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    a.hT[e * a.D + d + v] =
                        init ? init[e * a.D + d + v] : 0.f;
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

namespace {

// Steps of a warp and warps of a block, by the bytes of one step.
constexpr int kWarps = 8;
template <typename T, typename G>
constexpr int steps_of() {
    return 8;
}
constexpr int kTile = kWarps * 8;

template <int VEC>
ScanPlan plan_of(int B, int T, int D, bool packed, void* ws) {
    ScanPlan p;
    p.tiles = (T + kTile - 1) / kTile;
    p.groups = (D + 32 * VEC - 1) / (32 * VEC);
    p.chains = p.groups * (packed ? 1 : B);
    const size_t n = (size_t)p.tiles * p.chains * 32 * VEC;
    p.counter = static_cast<unsigned int*>(ws);
    p.map = reinterpret_cast<unsigned long long*>(p.counter + 4);
    p.last = reinterpret_cast<unsigned int*>(p.map + n);
    return p;
}

template <int VEC>
size_t plan_bytes(int B, int T, int D, bool packed) {
    const ScanPlan p = plan_of<VEC>(B, T, D, packed, nullptr);
    return p.tiles <= 1 ? 0
                        : 16 + (size_t)p.tiles * p.chains * 32 * VEC * 12;
}

// Whether VEC adjacent channels of a strided input can be read at once.
bool packs(const Strided& x, size_t elt, int vec, bool batched) {
    return reinterpret_cast<uintptr_t>(x.p) % (elt * vec) == 0 &&
           x.st % vec == 0 && (!batched || x.sb % vec == 0);
}
bool packs(const void* p, size_t elt, int vec) {
    return reinterpret_cast<uintptr_t>(p) % (elt * vec) == 0;
}

template <typename T, typename G, int VEC, bool BWD, bool PACKED>
cudaError_t launch_scan(const GlrArgs& a, void* ws, cudaStream_t s) {
    const ScanPlan p = plan_of<VEC>(a.B, a.T, a.D, PACKED, ws);
    const long long blocks = (long long)p.tiles * p.chains;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (p.tiles > 1) {
        const cudaError_t e = cudaMemsetAsync(
            ws, 0xff, plan_bytes<VEC>(a.B, a.T, a.D, PACKED), s);
        if (e != cudaSuccess) return e;
    }
    glr_scan_kernel<T, G, VEC, steps_of<T, G>(), kWarps, BWD, PACKED>
        <<<(unsigned)blocks, 32 * kWarps, 0, s>>>(a, p);
    return cudaGetLastError();
}

template <typename T, typename G, int VEC>
cudaError_t launch_vec(const GlrArgs& a, bool bwd, void* ws, cudaStream_t s) {
    if (a.cu)
        return bwd ? launch_scan<T, G, VEC, true, true>(a, ws, s)
                   : launch_scan<T, G, VEC, false, true>(a, ws, s);
    return bwd ? launch_scan<T, G, VEC, true, false>(a, ws, s)
               : launch_scan<T, G, VEC, false, false>(a, ws, s);
}

}  // namespace

size_t glr_workspace_bytes(int B, int T, int D, bool packed, kla_dtype,
                           kla_dtype) {
    if (B <= 0) return 0;
    const size_t n1 = plan_bytes<1>(B, T, D, packed);
    const size_t n2 = plan_bytes<2>(B, T, D, packed);
    return n1 > n2 ? n1 : n2;
}

cudaError_t launch_glr(const GlrArgs& a, bool bwd, void* workspace,
                       cudaStream_t stream) {
    if (a.T == 0) {              // every sequence is empty
        const float* init = bwd ? a.dhT : a.h0;
        const size_t n = sizeof(float) * (size_t)a.B * a.D;
        if (!a.hT || a.hT == init) return cudaSuccess;
        return init ? cudaMemcpyAsync(a.hT, init, n, cudaMemcpyDeviceToDevice,
                                      stream)
                    : cudaMemsetAsync(a.hT, 0, n, stream);
    }
    return by_type(a.dtype, a.gdtype, [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        const bool batched = !a.cu && a.B > 1;
        const bool two = a.D % 2 == 0 && packs(a.x, sizeof(T), 2, batched) &&
                         packs(a.la, sizeof(G), 2, batched) &&
                         packs(a.g, sizeof(T), 2, batched) &&
                         packs(a.o, sizeof(T), 2) && packs(a.dla, sizeof(G), 2);
        return two ? launch_vec<T, G, 2>(a, bwd, workspace, stream)
                   : launch_vec<T, G, 1>(a, bwd, workspace, stream);
    });
}

cudaError_t read_and_clear_fault_glr(unsigned int* word) {
    cudaError_t e = cudaMemcpyFromSymbol(word, g_fault_glr,
                                         sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_fault_glr, &zero, sizeof(unsigned int));
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
