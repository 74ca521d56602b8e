// Layer norm over the last axis, forward (with an optional residual add) and
// backward:
//
//   s = x + r,  m = mean(s),  rstd = 1 / sqrt(mean((s - m)^2) + eps)
//   y = (s - m) rstd w + b
//   dx = rstd (w dy - mean(w dy) - xh mean(w dy xh)) + dsum,  xh = (x - m) rstd
//   dw = sum_rows dy xh,  db = sum_rows dy
//
// Both are bound by HBM: about 8 to 16 operations per element of 2 to 4
// bytes.  Everything is held and summed in fp32; the variance is the mean of
// the squared differences from the row's mean (not E[s^2] - m^2, which loses
// every digit on rows with a large offset).
//
// A row is the work of a group of threads, a warp to a block, which read it
// once.  Where there are many rows, a group walks through some of them, with
// the copies of its next rows into shared memory on their way meanwhile (a
// ring of rows per group).  Where there are few, a block per row loads it
// straight into registers.  Rows wider than a block can hold take the loop
// kernels at the end, which read them again.
//
// Measured on 16384 x 2048 bf16: forward with a residual 46 us (268 MB, 86 %
// of the copy bandwidth), without 25 us (80 %); backward with the residual's
// gradient 47.5 us (268 MB, 84 %), without 41 us (72 %).  (With the next row
// in registers instead of rings: 92 us for the backward.)  What bounds them
// is issue and the latency of the sums across threads: 16 instructions per
// element forward (20 with a residual) and 22 backward, at 54 to 58 % of the
// issue slots; fp32, with half the elements per byte, reaches 89 and 90 %.
//
// All kernels launch as programmatic dependents: their blocks take their
// places while the kernel before them on the stream drains, and wait for its
// end before they touch memory (3 us of the 49 that the forward took).
#include <algorithm>
#include <atomic>

#include "f32x2.cuh"
#include "kla_internal.cuh"
#include "tc_primitives.cuh"

namespace kla {
namespace {

using bf16 = __nv_bfloat16;

// V adjacent elements as they lie in memory.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

__device__ __forceinline__ float load(const void* p, long long i, int dt) {
    return dt == KLA_BF16 ? to_f32(static_cast<const bf16*>(p)[i])
                          : static_cast<const float*>(p)[i];
}
// V adjacent elements of a weight or bias of either type from element i on.
template <int V>
__device__ __forceinline__ void load_v(const void* p, int i, int dt,
                                       float (&out)[V]) {
    if (dt == KLA_BF16) {
        const auto q = *reinterpret_cast<const Pack<bf16, V>*>(
            static_cast<const bf16*>(p) + i);
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = to_f32(q.v[v]);
    } else {
        constexpr int U = V < 4 ? V : 4;
#pragma unroll
        for (int u = 0; u < V; u += U) {
            const auto q = *reinterpret_cast<const Pack<float, U>*>(
                static_cast<const float*>(p) + i + u);
#pragma unroll
            for (int v = 0; v < U; ++v) out[u + v] = q.v[v];
        }
    }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// Sum over a group of TPR threads (a warp, or the TPR threads that share the
// named barrier `bar`); every thread gets it.  `red`: TPR / 32 places, free
// when the call begins and not written again until the next call but one.
template <int TPR>
__device__ __forceinline__ float group_sum(float a, float* red, int bar) {
    a = warp_sum(a);
    if constexpr (TPR == 32) {
        return a;
    } else {
        if (threadIdx.x % 32 == 0) red[threadIdx.x % TPR / 32] = a;
        tc::named_bar_sync(bar, TPR);
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) t += red[w];
        return t;
    }
}
// The same of two values, each in half of a warp's lanes after the first
// step.
template <int TPR>
__device__ __forceinline__ float2 group_sum(float2 a, float2* red, int bar) {
    const bool low = threadIdx.x % 32 < 16;
    float v = low ? a.x : a.y;
    v += __shfl_xor_sync(0xffffffffu, low ? a.y : a.x, 16);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    if constexpr (TPR == 32) {
        return make_float2(__shfl_sync(0xffffffffu, v, 0),
                           __shfl_sync(0xffffffffu, v, 16));
    } else {
        if (threadIdx.x % 16 == 0)
            reinterpret_cast<float*>(red)[threadIdx.x % TPR / 16] = v;
        tc::named_bar_sync(bar, TPR);
        float2 t = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) t = add2(t, red[w]);
        return t;
    }
}

// Forward, the row in registers (as a programmatic dependent of the kernel
// before it): TPR threads per row, N packs of V elements
// each; a block of max(TPR, 128) threads.
template <typename T, int V, int TPR, int N>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
ln_fwd_kernel(const __grid_constant__ LayerNormArgs a) {
    using P = Pack<T, V>;
    constexpr int ROWS = TPR < 128 ? 128 / TPR : 1;
    __shared__ float red[2][ROWS * TPR / 32];
    const int sub = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * ROWS + sub;
    await_grid_before();
    release_grid_after();
    if (row >= a.rows) return;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* r = a.residual
                     ? static_cast<const T*>(a.residual) +
                           row * a.residual_stride
                     : nullptr;
    P px[N], pr[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * TPR + t) * V;
        if (c < a.D) px[i] = *reinterpret_cast<const P*>(x + c);
        if (r && c < a.D) pr[i] = *reinterpret_cast<const P*>(r + c);
    }
    float s[N][V];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool in = (i * TPR + t) * V < a.D;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[i][v] = in ? to_f32(px[i].v[v]) +
                               (r ? to_f32(pr[i].v[v]) : 0.f)
                         : 0.f;
            sum += s[i][v];
        }
    }
    const float mean =
        group_sum<TPR>(sum, red[0] + sub * (TPR / 32), 1 + sub) / a.D;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool in = (i * TPR + t) * V < a.D;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float d = s[i][v] - mean;
            sq = in ? fmaf(d, d, sq) : sq;
        }
    }
    const float rstd = rsqrtf(
        group_sum<TPR>(sq, red[1] + sub * (TPR / 32), 1 + sub) / a.D +
        a.eps);
    T* y = static_cast<T*>(a.y) + row * a.D;
    T* so = a.sum ? static_cast<T*>(a.sum) + row * a.D : nullptr;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * TPR + t) * V;
        if (c >= a.D) break;
        float w[V], b[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            w[v] = 1.f;
            b[v] = 0.f;
        }
        if (a.weight) load_v<V>(a.weight, c, a.wdtype, w);
        if (a.bias) load_v<V>(a.bias, c, a.wdtype, b);
        P py, ps;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            py.v[v] =
                from_f32<T>(fmaf((s[i][v] - mean) * rstd, w[v], b[v]));
            ps.v[v] = from_f32<T>(s[i][v]);
        }
        *reinterpret_cast<P*>(y + c) = py;
        if (so) *reinterpret_cast<P*>(so + c) = ps;
    }
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// The rows of a group on their way into shared memory: IN inputs a row, K
// rows.  Rows that line up on 16 bytes (WIDE) are copied whole by one thread
// (bulk copies, an mbarrier per place); others by all threads with the
// 16-byte pieces that they touch, each row keeping its place within the first
// of them (read from the piece's start to the row's end only: the bytes that
// it may hold before the row belong to the same allocation, which starts on
// 16 bytes).
constexpr int kMaxDepth = 8;

template <bool WIDE, typename T, int TPR, int IN>
struct Ring {
    unsigned char* at;           // the group's place in shared memory
    uint64_t* full;              // its mbarriers
    int depth, pitch, bytes;     // rows; bytes between and in inputs
    int t, bar;                  // thread and barrier of the group
    const T* src[IN];
    long long stride[IN];
    long long rows, step;        // rows in all; between those of the group
    int in;                      // inputs that there are

    __device__ const T* place(int slot, int i) const {
        return reinterpret_cast<const T*>(at + (slot * in + i) * pitch);
    }
    // Input i of a row in a slot: its first element.
    __device__ const T* row_of(int slot, int i, long long row) const {
        const T* p = place(slot, i);
        if (WIDE) return p;
        return p + (reinterpret_cast<uintptr_t>(src[i] + row * stride[i]) &
                    15) / sizeof(T);
    }
    __device__ void fetch(int slot, long long row) const {
        if (WIDE) {
            if (t != 0 || row >= rows) return;
            tc::mbar_arrive_expect_tx(full + slot, in * bytes);
#pragma unroll
            for (int i = 0; i < IN; ++i)
                if (i < in)
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::"
                        "complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                            tc::smem_u32(place(slot, i))),
                        "l"(src[i] + row * stride[i]), "r"(bytes),
                        "r"(tc::smem_u32(full + slot))
                        : "memory");
        } else {
            if (row < rows) {
#pragma unroll
                for (int i = 0; i < IN; ++i) {
                    if (i >= in) break;
                    const uintptr_t p =
                        reinterpret_cast<uintptr_t>(src[i] + row * stride[i]);
                    const uintptr_t from = p & ~(uintptr_t)15;
                    const int len = (int)(p - from) + bytes;
                    const unsigned int to = tc::smem_u32(place(slot, i));
                    for (int c = t * 16; c < len; c += TPR * 16)
                        asm volatile(
                            "cp.async.cg.shared.global [%0], [%1], 16, %2;"
                            ::"r"(to + c), "l"(from + c),
                            "r"(min(16, len - c))
                            : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    // Until the copy of the turn-th row is there; false: it never came.
    __device__ bool wait(int slot, int phase) const {
        if (WIDE) return tc::mbar_wait(full + slot, phase);
        // the pieces on their way: those of the kDepth - 2 rows after it
        asm volatile("cp.async.wait_group %0;" ::"n"(kLooseDepth - 2)
                     : "memory");
        if (TPR == 32) __syncwarp();
        else tc::named_bar_sync(bar, TPR);
        return true;
    }
    static constexpr int kLooseDepth = 4;

    // After a copy that never came: waits (1 ms each) for those that may be
    // on their way yet.
    __device__ void give_up() const {
        if constexpr (WIDE) {
            for (int k = 0; t == 0 && k < depth; ++k)
                for (int p = 0; p < 2; ++p)
                    tc::mbar_wait(full + k, p, 1000000);
        }
    }
};

// Whether some thread of the group gave up waiting for this row: known to all
// of them after the group's next barrier.  `dead` has two places per group,
// used in turns, so that a thread that is ahead does not disturb the answer.
template <int TPR>
__device__ __forceinline__ bool group_dead(bool fault, volatile int* dead) {
    if constexpr (TPR == 32) return __any_sync(0xffffffffu, fault);
    else return *dead != 0;
}

__device__ unsigned int g_fault_ln = 0;

// A thread's part of a row: N runs of V adjacent elements, run i from column
// (i * TPR + t) * V on, as pairs of fp32 (adjacent elements, or elements of
// runs 2 i and 2 i + 1 where V = 1).
template <typename T, bool WIDE>
constexpr int kV = WIDE ? 16 / (int)sizeof(T) : 1;

__device__ __forceinline__ void load_words(unsigned int (&q)[4],
                                           const void* p) {
    const uint4 v = *static_cast<const uint4*>(p);
    q[0] = v.x;
    q[1] = v.y;
    q[2] = v.z;
    q[3] = v.w;
}
__device__ __forceinline__ void load_words(unsigned int (&q)[2],
                                           const void* p) {
    const uint2 v = *static_cast<const uint2*>(p);
    q[0] = v.x;
    q[1] = v.y;
}

template <typename T, int V, int TPR, int N>
struct Part {
    static constexpr int E = N * V / 2;          // pairs
    float2 v[E];

    // Whether column (i * TPR + t) * V + ... of run i is in a row of D; runs
    // that lie inside for all threads need no test.
    __device__ static int column(int i, int t) { return (i * TPR + t) * V; }
    __device__ static bool inside(int i, int t, int D) {
        // the launch takes the narrowest kernel, so that the first half of
        // the runs lies inside; not so in the narrowest of all
        constexpr int sure = N == 1 || (V == 1 && N == 4) ? 0 : N / 2;
        return i < sure || (i + 1) * TPR * V <= D || column(i, t) < D;
    }
    // f(pair index, both elements in the row, the first, run) for all pairs
    // of which some element is in the row.
    template <typename F>
    __device__ static void each(int t, int D, F f) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = V == 1 ? 2 * e : 2 * e / V;
            const bool a = inside(i, t, D);
            const bool b = V == 1 ? inside(i + 1, t, D) : a;
            f(e, a, b);
        }
    }
    // From a row in memory (any type); zeros outside.
    template <typename U>
    __device__ void read(const U* p, int t, int D, float fill = 0.f) {
        if constexpr (V == 1) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[e] = both(fill);
                if (inside(2 * e, t, D)) v[e].x = to_f32(p[column(2 * e, t)]);
                if (inside(2 * e + 1, t, D))
                    v[e].y = to_f32(p[column(2 * e + 1, t)]);
            }
        } else {
            constexpr int M = 16 / sizeof(U) < V ? 16 / sizeof(U) : V;
#pragma unroll
            for (int i = 0; i < N; ++i) {
#pragma unroll
                for (int u = 0; u < V; u += M) {
                    const bool in = inside(i, t, D);
                    unsigned int q[M * sizeof(U) / 4];
                    if (in)
                        load_words(q, p + column(i, t) + u);
#pragma unroll
                    for (int w = 0; w < M; w += 2) {
                        float2 x;
                        if constexpr (sizeof(U) == 2)
                            x = from_bf16x2(q[w / 2]);
                        else
                            x = make_float2(__uint_as_float(q[w]),
                                            __uint_as_float(q[w + 1]));
                        v[(i * V + u + w) / 2] = in ? x : both(fill);
                    }
                }
            }
        }
    }
    // To a row in memory, rounded to T.
    __device__ void write(T* p, int t, int D) const {
        if constexpr (V == 1) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (inside(2 * e, t, D))
                    p[column(2 * e, t)] = from_f32<T>(v[e].x);
                if (inside(2 * e + 1, t, D))
                    p[column(2 * e + 1, t)] = from_f32<T>(v[e].y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (!inside(i, t, D)) continue;
                if constexpr (sizeof(T) == 2) {
                    uint4 q;
                    q.x = bf16x2(v[i * 4]);
                    q.y = bf16x2(v[i * 4 + 1]);
                    q.z = bf16x2(v[i * 4 + 2]);
                    q.w = bf16x2(v[i * 4 + 3]);
                    *reinterpret_cast<uint4*>(p + column(i, t)) = q;
                } else {
                    *reinterpret_cast<float4*>(p + column(i, t)) =
                        make_float4(v[i * 2].x, v[i * 2].y, v[i * 2 + 1].x,
                                    v[i * 2 + 1].y);
                }
            }
        }
    }
    __device__ static unsigned int bf16x2(float2 x) {
        return tc::pack_bf16x2(x.x, x.y);
    }
    // A weight or bias of either type (null: `fill` everywhere).
    __device__ void read_weight(const void* p, int dt, int t, int D,
                                float fill) {
        if (!p) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = both(fill);
        } else if (dt == KLA_BF16) {
            read(static_cast<const bf16*>(p), t, D, 0.f);
        } else {
            read(static_cast<const float*>(p), t, D, 0.f);
        }
    }
    __device__ float sum() const {
        float2 s = v[0];
#pragma unroll
        for (int e = 1; e < E; ++e) s = add2(s, v[e]);
        return s.x + s.y;
    }
};

// Waits for the grid before this one and starts the first rows of this
// thread's group on their way.
template <bool WIDE, typename T, int TPR, int GROUPS, int IN>
__device__ __forceinline__ void open_ring(Ring<WIDE, T, TPR, IN>& ring,
                                          unsigned char* smem, uint64_t* full,
                                          int* dead, long long rows, int D,
                                          int depth) {
    const int g = threadIdx.x / TPR;
    await_grid_before();
    release_grid_after();
    if (threadIdx.x < 2 * GROUPS) dead[threadIdx.x] = 0;
    ring.t = threadIdx.x % TPR;
    ring.bar = 1 + g;
    ring.depth = depth;
    ring.bytes = D * (int)sizeof(T);
    ring.pitch = (ring.bytes + (WIDE ? 0 : 15) + 15) / 16 * 16;
    ring.at = smem + (size_t)g * depth * ring.in * ring.pitch;
    ring.full = full + g * kMaxDepth;
    ring.rows = rows;
    ring.step = (long long)gridDim.x * GROUPS;
    if (WIDE) {
        if (ring.t == 0) {
            for (int k = 0; k < depth; ++k) tc::mbar_init(ring.full + k, 1);
            tc::fence_mbar_init();
        }
    }
    __syncthreads();
    const long long row = (long long)blockIdx.x * GROUPS + g;
    for (int k = 0; k < depth - 1; ++k) ring.fetch(k, row + k * ring.step);
}

// Forward over many rows: a thread holds N runs of V elements of its row.
template <typename T, bool WIDE, int TPR, int N, int GROUPS>
__global__ void __launch_bounds__(TPR * GROUPS)
ln_fwd_ring_kernel(const __grid_constant__ LayerNormArgs a, int depth) {
    constexpr int V = kV<T, WIDE>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full[GROUPS * kMaxDepth];
    __shared__ int dead[2][GROUPS];
    __shared__ float red[2][GROUPS * TPR / 32];
    const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
    Ring<WIDE, T, TPR, 2> ring;
    ring.src[0] = static_cast<const T*>(a.x);
    ring.src[1] = static_cast<const T*>(a.residual);
    ring.stride[0] = a.x_stride;
    ring.stride[1] = a.residual_stride;
    ring.in = a.residual ? 2 : 1;
    open_ring<WIDE, T, TPR, GROUPS>(ring, smem, full, dead[0], a.rows, a.D,
                                      depth);

    using Row = Part<T, V, TPR, N>;
    Row w, b;
    w.read_weight(a.weight, a.wdtype, t, a.D, 1.f);
    b.read_weight(a.bias, a.wdtype, t, a.D, 0.f);
    const float over = 1.f / a.D;
    bool fault = false;
    int slot = 0, phase = 0, turn = 0;
    for (long long row = (long long)blockIdx.x * GROUPS + g; row < a.rows;
         row += ring.step, turn ^= 1) {
        if (!ring.wait(slot, phase)) fault = dead[turn][g] = true;
        Row s;
        s.read(ring.row_of(slot, 0, row), t, a.D);
        if (a.residual) {
            Row r;
            r.read(ring.row_of(slot, 1, row), t, a.D);
#pragma unroll
            for (int e = 0; e < Row::E; ++e) s.v[e] = add2(s.v[e], r.v[e]);
        }
        // The sum over D, as a division rounds it: a row of one value has that
        // mean exactly, where the sum is exact, and y = bias.  (1 / D rounded
        // alone left 6e-5 of 1000 at D = 1000, which eps = 1e-5 makes 0.02
        // in y.)
        const float sum =
            group_sum<TPR>(s.sum(), red[0] + g * (TPR / 32), 1 + g);
        const float first = sum * over, rest = fmaf(-first, (float)a.D, sum);
        const float mean = rest == rest ? fmaf(rest, over, first) : first;
        if (group_dead<TPR>(fault, &dead[turn][g])) {
            fault = true;
            break;
        }
        // all of the group are done with the row before: its place is free
        ring.fetch(slot == 0 ? depth - 1 : slot - 1,
                   row + (depth - 1) * ring.step);
        if (++slot == depth) {
            slot = 0;
            phase ^= 1;
        }
        if (a.sum)
            s.write(static_cast<T*>(a.sum) + row * a.D, t, a.D);
        float2 sq = both(0.f);
        Row::each(t, a.D, [&](int e, bool p, bool q) {
            s.v[e] = add2(s.v[e], both(-mean));
            if (!p) s.v[e].x = 0.f;
            if (!q) s.v[e].y = 0.f;
            sq = fma2(s.v[e], s.v[e], sq);
        });
        const float rstd = rsqrtf(
            group_sum<TPR>(sq.x + sq.y, red[1] + g * (TPR / 32), 1 + g) *
                over + a.eps);
#pragma unroll
        for (int e = 0; e < Row::E; ++e)
            s.v[e] = fma2(mul2(s.v[e], both(rstd)), w.v[e], b.v[e]);
        s.write(static_cast<T*>(a.y) + row * a.D, t, a.D);
        if (t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
    if (!WIDE) asm volatile("cp.async.wait_all;" ::: "memory");
    if (fault) {
        if (t == 0) atomicOr(&g_fault_ln, 1u);
        ring.give_up();
    }
}

// Backward over the rows of a group, a thread keeping its N * V columns,
// whose dw and db it adds up in registers.  At the end the block's groups are
// added up in shared memory, in order, and the block's partial sums go to
// part [gridDim.x][2][D].  HOLD: w, xh and w dy stay in registers from the
// sums to the result (else they are formed again: very wide rows).
template <typename T, bool WIDE, int TPR, int N, int GROUPS, bool HOLD>
__global__ void __launch_bounds__(TPR * GROUPS, TPR * GROUPS <= 256 ? 2 : 1)
ln_bwd_ring_kernel(const __grid_constant__ LayerNormBwdArgs a, int depth,
                   float* part) {
    constexpr int V = kV<T, WIDE>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full[GROUPS * kMaxDepth];
    __shared__ int dead[2][GROUPS];
    __shared__ float2 red[2][GROUPS * TPR / 32];
    const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
    Ring<WIDE, T, TPR, 3> ring;
    ring.src[0] = static_cast<const T*>(a.x);
    ring.src[1] = static_cast<const T*>(a.dy);
    ring.src[2] = static_cast<const T*>(a.dsum);
    ring.stride[0] = a.x_stride;
    ring.stride[1] = a.dy_stride;
    ring.stride[2] = a.dsum_stride;
    ring.in = a.dsum ? 3 : 2;
    open_ring<WIDE, T, TPR, GROUPS>(ring, smem, full, dead[0], a.rows, a.D,
                                      depth);

    using Row = Part<T, V, TPR, N>;
    Row dw, db, w;
#pragma unroll
    for (int e = 0; e < Row::E; ++e) dw.v[e] = db.v[e] = both(0.f);
    if (HOLD) w.read_weight(a.weight, a.wdtype, t, a.D, 1.f);
    const float over = 1.f / a.D;
    bool fault = false;
    int slot = 0, phase = 0, turn = 0;
    long long row = (long long)blockIdx.x * GROUPS + g;
    float mean = 0.f, rstd = 0.f;
    if (row < a.rows) {
        mean = a.mean[row];
        rstd = a.rstd[row];
    }
    for (; row < a.rows; row += ring.step, turn ^= 1) {
        if (!ring.wait(slot, phase)) fault = dead[turn][g] = true;
        const T* x = ring.row_of(slot, 0, row);
        const T* y = ring.row_of(slot, 1, row);
        const T* d = a.dsum ? ring.row_of(slot, 2, row) : nullptr;
        // xh and w dy (zeros outside the row); dw and db, too
        Row xh, wy;
        auto form = [&](bool add) {
            if (!HOLD) w.read_weight(a.weight, a.wdtype, t, a.D, 1.f);
            xh.read(x, t, a.D, mean);
            wy.read(y, t, a.D);
#pragma unroll
            for (int e = 0; e < Row::E; ++e) {
                xh.v[e] = mul2(add2(xh.v[e], both(-mean)), both(rstd));
                if (add) {
                    dw.v[e] = fma2(wy.v[e], xh.v[e], dw.v[e]);
                    db.v[e] = add2(db.v[e], wy.v[e]);
                }
                wy.v[e] = mul2(wy.v[e], w.v[e]);
            }
        };
        form(true);
        float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
        for (int e = 0; e < Row::E; ++e) {
            s1 = fma2(wy.v[e], xh.v[e], s1);
            s2 = add2(s2, wy.v[e]);
        }
        const float2 sum = make_float2(s1.x + s1.y, s2.x + s2.y);
        float next_mean = 0.f, next_rstd = 0.f;
        if (row + ring.step < a.rows) {
            next_mean = a.mean[row + ring.step];
            next_rstd = a.rstd[row + ring.step];
        }
        const float2 c =
            group_sum<TPR>(sum, red[turn] + g * (TPR / 32), 1 + g);
        if (group_dead<TPR>(fault, &dead[turn][g])) {
            fault = true;
            break;
        }
        // all of the group are done with the row before: its place is free
        ring.fetch(slot == 0 ? depth - 1 : slot - 1,
                   row + (depth - 1) * ring.step);
        if (++slot == depth) {
            slot = 0;
            phase ^= 1;
        }
        const float c1 = c.x * over, c2 = c.y * over;
        if (!HOLD) form(false);
#pragma unroll
        for (int e = 0; e < Row::E; ++e)
            wy.v[e] = add2(fma2(xh.v[e], both(-c1), wy.v[e]), both(-c2));
        if (d) {
            Row ds;
            ds.read(d, t, a.D);
#pragma unroll
            for (int e = 0; e < Row::E; ++e)
                wy.v[e] = fma2(wy.v[e], both(rstd), ds.v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < Row::E; ++e)
                wy.v[e] = mul2(wy.v[e], both(rstd));
        }
        wy.write(static_cast<T*>(a.dx) + row * a.D, t, a.D);
        mean = next_mean;
        rstd = next_rstd;
    }
    if (!WIDE) asm volatile("cp.async.wait_all;" ::: "memory");
    if (fault) {
        if (t == 0) atomicOr(&g_fault_ln, 1u);
        ring.give_up();
    }
    if (!part) return;
    // every copy has been waited for: the rings' place is free
    float2* total = reinterpret_cast<float2*>(smem);     // [N * V][TPR]
    for (int q = 0; q < GROUPS; ++q) {
        __syncthreads();
        if (g != q) continue;
#pragma unroll
        for (int e = 0; e < 2 * Row::E; ++e) {
            float2& s = total[e * TPR + t];
            const float2 old = q ? s : both(0.f);
            const float x = e % 2 ? dw.v[e / 2].y : dw.v[e / 2].x;
            const float y = e % 2 ? db.v[e / 2].y : db.v[e / 2].x;
            s = make_float2(old.x + x, old.y + y);
        }
    }
    __syncthreads();
    float* p = part + (size_t)blockIdx.x * 2 * a.D;
    for (int c = threadIdx.x; c < a.D; c += TPR * GROUPS) {
        // column c: run c / (V TPR), thread c / V % TPR, element c % V
        const float2 s =
            total[(c / (V * TPR) * V + c % V) * TPR + c / V % TPR];
        p[c] = s.x;
        p[a.D + c] = s.y;
    }
}

constexpr int kLoopThreads = 512;

// Sum over a block of kLoopThreads of two values at once.
__device__ __forceinline__ float2 block_sum(float a, float b, float2* red) {
    __syncthreads();             // red is free again
    return group_sum<kLoopThreads>(make_float2(a, b), red, 0);
}

// Any D, strides and alignment: one block per row, which it reads three
// times (from L1 or L2 after the first), element by element.  For the rows
// that no other kernel takes: 2048 x 8191 bf16 in 39 us (floor 9.9), in the
// backward below 64 (floor 14.9).
template <typename T>
__global__ void __launch_bounds__(kLoopThreads)
ln_fwd_loop_kernel(LayerNormArgs a) {
    __shared__ float2 red[kLoopThreads / 32];
    const long long row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* r = a.residual ? static_cast<const T*>(a.residual) +
                                  row * a.residual_stride
                            : nullptr;
    auto s = [&](int i) {
        return r ? to_f32(x[i]) + to_f32(r[i]) : to_f32(x[i]);
    };
    float t = 0.f;
    for (int i = threadIdx.x; i < a.D; i += kLoopThreads) t += s(i);
    const float mean = block_sum(t, 0.f, red).x / a.D;
    t = 0.f;
    for (int i = threadIdx.x; i < a.D; i += kLoopThreads) {
        const float d = s(i) - mean;
        t = fmaf(d, d, t);
    }
    const float rstd = rsqrtf(block_sum(t, 0.f, red).x / a.D + a.eps);
    T* y = static_cast<T*>(a.y) + row * a.D;
    T* sum = a.sum ? static_cast<T*>(a.sum) + row * a.D : nullptr;
    for (int i = threadIdx.x; i < a.D; i += kLoopThreads) {
        const float v = s(i);
        const float w = a.weight ? load(a.weight, i, a.wdtype) : 1.f;
        const float b = a.bias ? load(a.bias, i, a.wdtype) : 0.f;
        y[i] = from_f32<T>(fmaf((v - mean) * rstd, w, b));
        if (sum) sum[i] = from_f32<T>(v);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

// dx of any D: one block per row, two passes over x and dy.
template <typename T>
__global__ void __launch_bounds__(kLoopThreads)
ln_bwd_loop_kernel(LayerNormBwdArgs a) {
    __shared__ float2 red[kLoopThreads / 32];
    const long long row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float t1 = 0.f, t2 = 0.f;
    for (int i = threadIdx.x; i < a.D; i += kLoopThreads) {
        const float w = a.weight ? load(a.weight, i, a.wdtype) : 1.f;
        const float g = w * to_f32(dy[i]);
        t1 = fmaf(g, (to_f32(x[i]) - mean) * rstd, t1);
        t2 += g;
    }
    const float2 c = block_sum(t1, t2, red);
    const float c1 = c.x / a.D, c2 = c.y / a.D;
    const T* ds = a.dsum ? static_cast<const T*>(a.dsum) +
                               row * a.dsum_stride
                         : nullptr;
    T* dx = static_cast<T*>(a.dx) + row * a.D;
    for (int i = threadIdx.x; i < a.D; i += kLoopThreads) {
        const float w = a.weight ? load(a.weight, i, a.wdtype) : 1.f;
        const float g = w * to_f32(dy[i]);
        const float xh = (to_f32(x[i]) - mean) * rstd;
        const float v = rstd * (g - c2 - xh * c1);
        dx[i] = from_f32<T>(ds ? v + to_f32(ds[i]) : v);
    }
}

// Partial dw, db of a slice of rows: one thread per column, blockIdx.y the
// slice; part [slices][2][D].
template <typename T>
__global__ void ln_bwd_cols_kernel(LayerNormBwdArgs a, float* part) {
    const int col = blockIdx.x * blockDim.x + threadIdx.x;
    if (col >= a.D) return;
    float w = 0.f, b = 0.f;
    for (long long row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float x =
            to_f32(static_cast<const T*>(a.x)[row * a.x_stride + col]);
        const float dy =
            to_f32(static_cast<const T*>(a.dy)[row * a.dy_stride + col]);
        w = fmaf(dy, (x - a.mean[row]) * a.rstd[row], w);
        b += dy;
    }
    float* p = part + (size_t)blockIdx.y * 2 * a.D;
    p[col] = w;
    p[(size_t)a.D + col] = b;
}

// dw, db = the partial sums added up in a fixed order: a block takes 32
// columns, a warp every 32nd slice (304 slices of 2048 columns: 1.5 us less
// than with 8 warps), then the warps are added up.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps)
ln_bwd_join_kernel(const float* part, int slices, int D, void* dw, void* db,
                   int wdtype) {
    __shared__ float2 red[kJoinWarps][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int col = blockIdx.x * 32 + lane;
    await_grid_before();
    float w = 0.f, b = 0.f;
    if (col < D) {
#pragma unroll 4
        for (int i = warp; i < slices; i += kJoinWarps) {
            w += part[(size_t)i * 2 * D + col];
            b += part[((size_t)i * 2 + 1) * D + col];
        }
    }
    red[warp][lane] = make_float2(w, b);
    __syncthreads();
    if (warp != 0 || col >= D) return;
    for (int u = 1; u < kJoinWarps; ++u) {
        w += red[u][lane].x;
        b += red[u][lane].y;
    }
    auto put = [&](void* p, float v) {
        if (!p) return;
        if (wdtype == KLA_BF16)
            static_cast<bf16*>(p)[col] = from_f32<bf16>(v);
        else
            static_cast<float*>(p)[col] = v;
    };
    put(dw, w);
    put(db, b);
}

// Rows of partial sums that a backward call may write (its workspace), which
// is the number of blocks that it launches at most: four an SM of 152, one
// where a row takes 512 threads or more (their registers leave no room for a
// second).  Every block's sums are written and read again: blocks beyond 128
// have 4 rows a group at least (1024 x 2048 8.9 -> 7.9 us, 256 x 2048 and 4096
// x 2048 the same).
int most_slices(int rows, int groups, int D, size_t elt) {
    const int sms = (size_t)D * elt > 8192 ? 152 : 608;
    const long long four = ((long long)rows + 4 * groups - 1) / (4 * groups);
    return std::max(1, (int)std::min<long long>({sms, rows,
                                                 std::max(128ll, four)}));
}

bool lines_up(const void* p, size_t elt, long long stride, int vec) {
    return reinterpret_cast<uintptr_t>(p) % (elt * vec) == 0 &&
           stride % vec == 0;
}

// Blocks of a ring kernel, and its ring: as many rows as fit beside the other
// blocks that an SM's registers hold, at most kMaxDepth and 2 at least; 4 for
// rows copied in pieces (0 blocks: they do not fit).
struct RingPlan {
    int blocks, depth, bytes;
};
constexpr int kSmBytes = 228 * 1024, kBlockBytes = 1024 + 1024;  // own, fixed

template <auto K>
RingPlan ring_plan(int threads, int groups, bool wide, int in, int elt, int D,
                   int rows, int least) {
    // blocks that an SM's registers and threads allow (looked up once)
    static std::atomic<int> found[64];
    RingPlan p{0, 0, 0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return p;
    int per = found[dev].load(std::memory_order_relaxed);
    if (per == 0) {
        if (cudaFuncSetAttribute(K,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 220 * 1024) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                &per, K, threads, 0) != cudaSuccess || per < 1)
            return p;
        found[dev].store(per, std::memory_order_relaxed);
    }
    const int pitch = (D * elt + (wide ? 0 : 15) + 15) / 16 * 16;
    const int row = groups * in * pitch;         // of all groups of a block
    const int share = std::min(kSmBytes / per - kBlockBytes, 220 * 1024);
    p.depth = wide ? std::max(2, std::min(kMaxDepth, share / row)) : 4;
    p.bytes = std::max(p.depth * row, least);
    if (p.bytes > 220 * 1024) return p;
    per = std::min(per, kSmBytes / (p.bytes + kBlockBytes));
    p.blocks = (int)std::min<long long>(
        ((long long)rows + groups - 1) / groups,
        (long long)std::max(1, per) * device_sm_count());
    return p;
}

template <typename T, int V, int TPR, int N>
cudaError_t fwd_rows(const LayerNormArgs& a, cudaStream_t s) {
    constexpr int threads = TPR < 128 ? 128 : TPR, rows = threads / TPR;
    const long long blocks = ((long long)a.rows + rows - 1) / rows;
    return launch_dependent(ln_fwd_kernel<T, V, TPR, N>,
                            dim3((unsigned)blocks), threads, s, 0, a);
}

template <typename T, bool WIDE, int TPR, int N>
cudaError_t fwd_ring(const LayerNormArgs& a, cudaStream_t s) {
    constexpr int LEAST = WIDE ? 128 : 256;      // threads of a block
    constexpr int GROUPS = TPR < LEAST ? LEAST / TPR : 1;
    constexpr auto* kernel = ln_fwd_ring_kernel<T, WIDE, TPR, N, GROUPS>;
    const RingPlan p = ring_plan<kernel>(TPR * GROUPS, GROUPS, WIDE,
                                         a.residual ? 2 : 1, sizeof(T), a.D,
                                         a.rows, 0);
    if (p.blocks <= 0) return cudaErrorInvalidConfiguration;
    return launch_dependent(kernel, dim3(p.blocks), TPR * GROUPS, s, p.bytes, a,
                            p.depth);
}

template <typename T, int V>
cudaError_t fwd_width(const LayerNormArgs& a, cudaStream_t s) {
    constexpr bool WIDE = V > 1;
    constexpr int M = WIDE ? 1 : 4;              // runs are 1 element then
    const int packs = (a.D + V - 1) / V;
    // Rings pay where a group gets more than a row or so.  Measured (ring /
    // rows, us): bf16 4096 x 512 4.0 / 3.7, 8192 x 512 5.0 / 5.9; 512 x 2048
    // 3.6 / 3.1, 1024 x 2048 4.1 / 4.5, 16384 x 2048 25 / 46; 64 x 8192 3.6 /
    // 3.7, 256 x 8192 4.7 / 6.2; fp32 256 x 2048 2.9 / 2.8, 512 x 2048 3.5 /
    // 3.7; 256 x 1001 2.6 / 3.8, 16384 x 1001 26 / 139.
    if ((long long)a.rows * packs >= 196608) {
        if (packs <= 32 * M) return fwd_ring<T, WIDE, 32, M>(a, s);
        if (packs <= 64 * M) return fwd_ring<T, WIDE, 32, 2 * M>(a, s);
        if (packs <= 128 * M) return fwd_ring<T, WIDE, 64, 2 * M>(a, s);
        if (packs <= 256 * M) return fwd_ring<T, WIDE, 128, 2 * M>(a, s);
        if (packs <= 512 * M) return fwd_ring<T, WIDE, 256, 2 * M>(a, s);
        if (packs <= 1024 * M) return fwd_ring<T, WIDE, 512, 2 * M>(a, s);
        // (1024 threads leave 64 registers: 8192 x 8200 94 instead of 62 us,
        // 2048 x 16384 34 instead of 26)
        if constexpr (WIDE) {
            if (packs <= 1280) return fwd_ring<T, WIDE, 640, 2>(a, s);
            if (packs <= 2048) return fwd_ring<T, WIDE, 512, 4>(a, s);
        }
    }
    if (packs <= 32) return fwd_rows<T, V, 32, 1>(a, s);
    if (packs <= 64) return fwd_rows<T, V, 32, 2>(a, s);
    if (packs <= 128) return fwd_rows<T, V, 128, 1>(a, s);
    if (packs <= 256) return fwd_rows<T, V, 256, 1>(a, s);
    if (packs <= 512) return fwd_rows<T, V, 512, 1>(a, s);
    if (packs <= 1024) return fwd_rows<T, V, 1024, 1>(a, s);
    if (packs <= 4096) return fwd_rows<T, V, 1024, 4>(a, s);
    ln_fwd_loop_kernel<T><<<a.rows, kLoopThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_fwd(const LayerNormArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const size_t we = a.wdtype == KLA_BF16 ? 2 : 4;
    const int wv = std::min<int>(V, 16 / we);
    const bool wide = a.D % V == 0 && lines_up(a.x, sizeof(T), a.x_stride, V) &&
                      lines_up(a.residual, sizeof(T), a.residual_stride, V) &&
                      lines_up(a.y, sizeof(T), 0, V) &&
                      lines_up(a.sum, sizeof(T), 0, V) &&
                      lines_up(a.weight, we, 0, wv) &&
                      lines_up(a.bias, we, 0, wv);
    return wide ? fwd_width<T, V>(a, s) : fwd_width<T, 1>(a, s);
}

cudaError_t join(const LayerNormBwdArgs& a, const float* part, int slices,
                 cudaStream_t s) {
    return launch_dependent(ln_bwd_join_kernel, dim3((a.D + 31) / 32),
                            32 * kJoinWarps, s, 0, part, slices, a.D, a.dw, a.db,
                            (int)a.wdtype);
}

template <typename T, bool WIDE, int TPR, int N, bool HOLD = true>
cudaError_t bwd_ring(const LayerNormBwdArgs& a, float* part, cudaStream_t s) {
    constexpr int GROUPS = TPR < 256 ? 256 / TPR : 1;
    constexpr auto* kernel =
        ln_bwd_ring_kernel<T, WIDE, TPR, N, GROUPS, HOLD>;
    const bool grads = a.dw || a.db;
    RingPlan p = ring_plan<kernel>(
        TPR * GROUPS, GROUPS, WIDE, a.dsum ? 3 : 2, sizeof(T), a.D, a.rows,
        TPR * N * kV<T, WIDE> * (int)sizeof(float2));
    if (p.blocks <= 0) return cudaErrorInvalidConfiguration;
    p.blocks = std::min(p.blocks,
                        most_slices(a.rows, GROUPS, a.D, sizeof(T)));
    const cudaError_t e =
        launch_dependent(kernel, dim3(p.blocks), TPR * GROUPS, s, p.bytes, a,
                         p.depth, grads ? part : nullptr);
    return e != cudaSuccess || !grads ? e : join(a, part, p.blocks, s);
}

template <typename T>
cudaError_t bwd_loop(const LayerNormBwdArgs& a, float* part, cudaStream_t s) {
    ln_bwd_loop_kernel<T><<<a.rows, kLoopThreads, 0, s>>>(a);
    if (!a.dw && !a.db) return cudaGetLastError();
    const int slices = std::min(a.rows, 128);
    ln_bwd_cols_kernel<T><<<dim3((a.D + 127) / 128, slices), 128, 0, s>>>(
        a, part);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : join(a, part, slices, s);
}

template <typename T, int V>
cudaError_t bwd_width(const LayerNormBwdArgs& a, float* part,
                      cudaStream_t s) {
    constexpr bool WIDE = V > 1;
    constexpr int M = WIDE ? 1 : 4;              // runs are 1 element then
    const int packs = (a.D + V - 1) / V;
    if (packs <= 32 * M) return bwd_ring<T, WIDE, 32, M>(a, part, s);
    if (packs <= 64 * M) return bwd_ring<T, WIDE, 32, 2 * M>(a, part, s);
    if (packs <= 128 * M) return bwd_ring<T, WIDE, 64, 2 * M>(a, part, s);
    if (packs <= 256 * M) return bwd_ring<T, WIDE, 128, 2 * M>(a, part, s);
    if (packs <= 512 * M) return bwd_ring<T, WIDE, 256, 2 * M>(a, part, s);
    if (packs <= 1024 * M) return bwd_ring<T, WIDE, 512, 2 * M>(a, part, s);
    // (a thread has the registers for 2 runs up to about 640 threads; 4 runs
    // formed twice take 38 instead of 28 us on 1023 rows of 8200)
    if constexpr (WIDE) {
        if (packs <= 1280) return bwd_ring<T, WIDE, 640, 2>(a, part, s);
        if (packs <= 1536) return bwd_ring<T, WIDE, 768, 2>(a, part, s);
        if (packs <= 2048)
            return bwd_ring<T, WIDE, 512, 4, false>(a, part, s);
    }
    return bwd_loop<T>(a, part, s);
}

template <typename T>
cudaError_t launch_bwd(const LayerNormBwdArgs& a, float* part,
                       cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const size_t we = a.wdtype == KLA_BF16 ? 2 : 4;
    const bool wide = a.D % V == 0 && lines_up(a.x, sizeof(T), a.x_stride, V) &&
                      lines_up(a.dy, sizeof(T), a.dy_stride, V) &&
                      lines_up(a.dsum, sizeof(T), a.dsum_stride, V) &&
                      lines_up(a.dx, sizeof(T), 0, V) &&
                      lines_up(a.weight, we, 0, std::min<int>(V, 16 / we));
    return wide ? bwd_width<T, V>(a, part, s) : bwd_width<T, 1>(a, part, s);
}

}  // namespace

cudaError_t read_and_clear_fault_ln(unsigned int* word) {
    cudaError_t e = cudaMemcpyFromSymbol(word, g_fault_ln,
                                         sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_fault_ln, &zero, sizeof(unsigned int));
}

cudaError_t launch_layernorm(const LayerNormArgs& a, cudaStream_t stream) {
    return a.dtype == KLA_BF16 ? launch_fwd<bf16>(a, stream)
                               : launch_fwd<float>(a, stream);
}

size_t layernorm_bwd_workspace_bytes(int rows, int D, kla_dtype dtype) {
    return (size_t)most_slices(rows, 1, D, dtype == KLA_BF16 ? 2 : 4) * 2 * D *
           sizeof(float);
}

cudaError_t launch_layernorm_bwd(const LayerNormBwdArgs& a, void* workspace,
                                 cudaStream_t stream) {
    float* part = static_cast<float*>(workspace);
    return a.dtype == KLA_BF16 ? launch_bwd<bf16>(a, part, stream)
                               : launch_bwd<float>(a, part, stream);
}

}  // namespace kla
