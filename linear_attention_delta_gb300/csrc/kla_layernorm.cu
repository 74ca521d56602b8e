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
// A row is held in the registers of a group of threads, which read it once:
// a warp, or a block.  V elements of a thread lie side by side (16 bytes), or
// one (rows that do not line up on 16 bytes).  Rows wider than a block's
// registers take the loop kernels at the end, which read them again.
#include <algorithm>

#include "kla_internal.cuh"

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
// named barrier `bar`) of two values at once; every thread gets both.  `red`:
// TPR / 32 places, free when the call begins and not reused until the next
// but one.
template <int TPR>
__device__ __forceinline__ float2 group_sum(float a, float b, float2* red,
                                            int bar) {
    a = warp_sum(a);
    b = warp_sum(b);
    if constexpr (TPR == 32) {
        return make_float2(a, b);
    } else {
        constexpr int NW = TPR / 32;
        const int warp = threadIdx.x % TPR / 32;
        if (threadIdx.x % 32 == 0) red[warp] = make_float2(a, b);
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(TPR) : "memory");
        float2 t = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float2 r = red[w];
            t.x += r.x;
            t.y += r.y;
        }
        return t;
    }
}

// Forward, the row in registers: TPR threads per row, N packs of V elements
// each; a block of max(TPR, 128) threads.
template <typename T, int V, int TPR, int N>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
ln_fwd_kernel(const __grid_constant__ LayerNormArgs a) {
    using P = Pack<T, V>;
    constexpr int ROWS = TPR < 128 ? 128 / TPR : 1;
    __shared__ float2 red[2][ROWS * TPR / 32];
    const int sub = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * ROWS + sub;
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
        group_sum<TPR>(sum, 0.f, red[0] + sub * (TPR / 32), 1 + sub).x / a.D;
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
    const float rstd =
        1.f / sqrtf(group_sum<TPR>(sq, 0.f, red[1] + sub * (TPR / 32),
                                   1 + sub).x / a.D + a.eps);
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

// Backward, the row in registers: a block of GROUPS groups of TPR threads
// walks the rows group by group (rows g, g + all groups, ...), a thread
// keeping its N * V columns, whose dw and db it adds up in registers; the
// next row's loads are issued before the present row is reduced.  At the end
// the block's groups are added up in shared memory, in order, and the block's
// partial sums go to part [gridDim.x][2][D].
template <typename T, int V, int TPR, int N, int GROUPS>
__global__ void __launch_bounds__(TPR * GROUPS)
ln_bwd_kernel(const __grid_constant__ LayerNormBwdArgs a, float* part) {
    using P = Pack<T, V>;
    __shared__ float2 red[2][GROUPS * TPR / 32];
    extern __shared__ float2 total[];            // [TPR * N * V] (dw, db)
    const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
    float w[N][V], dw[N][V], db[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * TPR + t) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            w[i][v] = 1.f;
            dw[i][v] = db[i][v] = 0.f;
        }
        if (a.weight && c < a.D) load_v<V>(a.weight, c, a.wdtype, w[i]);
    }
    const long long step = (long long)gridDim.x * GROUPS;
    long long row = (long long)blockIdx.x * GROUPS + g;
    P nx[N], ny[N], nd[N];
    float nm = 0.f, nr = 0.f;
    auto fetch = [&](long long row) {
        if (row >= a.rows) return;
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        const T* y = static_cast<const T*>(a.dy) + row * a.dy_stride;
        const T* d = static_cast<const T*>(a.dsum) + row * a.dsum_stride;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * TPR + t) * V;
            if (c < a.D) {
                nx[i] = *reinterpret_cast<const P*>(x + c);
                ny[i] = *reinterpret_cast<const P*>(y + c);
                if (a.dsum) nd[i] = *reinterpret_cast<const P*>(d + c);
            }
        }
        nm = a.mean[row];
        nr = a.rstd[row];
    };
    fetch(row);
    for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
        P px[N], py[N], pd[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            px[i] = nx[i];
            py[i] = ny[i];
            pd[i] = nd[i];
        }
        const float mean = nm, rstd = nr;
        fetch(row + step);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if ((i * TPR + t) * V >= a.D) break;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float xh = (to_f32(px[i].v[v]) - mean) * rstd;
                const float dy = to_f32(py[i].v[v]);
                const float wy = w[i][v] * dy;
                s1 = fmaf(wy, xh, s1);
                s2 += wy;
                dw[i][v] = fmaf(dy, xh, dw[i][v]);
                db[i][v] += dy;
            }
        }
        const float2 c = group_sum<TPR>(s1, s2, red[turn] + g * (TPR / 32),
                                        1 + g);
        const float c1 = c.x / a.D, c2 = c.y / a.D;
        T* dx = static_cast<T*>(a.dx) + row * a.D;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int col = (i * TPR + t) * V;
            if (col >= a.D) break;
            P out;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float xh = (to_f32(px[i].v[v]) - mean) * rstd;
                const float wy = w[i][v] * to_f32(py[i].v[v]);
                const float d = rstd * (wy - c2 - xh * c1);
                out.v[v] = from_f32<T>(
                    a.dsum ? d + to_f32(pd[i].v[v]) : d);
            }
            *reinterpret_cast<P*>(dx + col) = out;
        }
    }
    if (!part) return;
    for (int q = 0; q < GROUPS; ++q) {
        if (g == q) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float2& s = total[(i * V + v) * TPR + t];
                    const float2 old =
                        q ? s : make_float2(0.f, 0.f);
                    s = make_float2(old.x + dw[i][v], old.y + db[i][v]);
                }
        }
        __syncthreads();
    }
    float* p = part + (size_t)blockIdx.x * 2 * a.D;
    for (int e = threadIdx.x; e < N * V * TPR; e += TPR * GROUPS) {
        // column e of the row: pack e / V, thread (e / V) % TPR
        const int i = e / (V * TPR), u = e / V % TPR, v = e % V;
        if (e < a.D) {
            const float2 s = total[(i * V + v) * TPR + u];
            p[e] = s.x;
            p[a.D + e] = s.y;
        }
    }
}

constexpr int kLoopThreads = 512;

// Sum over a block of kLoopThreads of two values at once.
__device__ __forceinline__ float2 block_sum(float a, float b, float2* red) {
    __syncthreads();             // red is free again
    return group_sum<kLoopThreads>(a, b, red, 0);
}

// Any D, strides and alignment: one block per row, which it reads three
// times (from L1 or L2 after the first).
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
    const float rstd = 1.f / sqrtf(block_sum(t, 0.f, red).x / a.D + a.eps);
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
    p[a.D + col] = b;
}

// dw, db = the partial sums added up in a fixed order: a block takes 32
// columns, a warp every 8th slice, then the warps are added up.
__global__ void __launch_bounds__(256)
ln_bwd_join_kernel(const float* part, int slices, int D, void* dw, void* db,
                   int wdtype) {
    __shared__ float2 red[8][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int col = blockIdx.x * 32 + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float w = 0.f, b = 0.f;
    if (col < D) {
#pragma unroll 4
        for (int i = warp; i < slices; i += 8) {
            w += part[(size_t)i * 2 * D + col];
            b += part[((size_t)i * 2 + 1) * D + col];
        }
    }
    red[warp][lane] = make_float2(w, b);
    __syncthreads();
    if (warp != 0 || col >= D) return;
    for (int u = 1; u < 8; ++u) {
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

// Row groups of partial sums that a backward call may write (its workspace);
// the number of blocks that it launches at most.
constexpr int kMaxSlices = 608;

bool lines_up(const void* p, size_t elt, long long stride, int vec) {
    return reinterpret_cast<uintptr_t>(p) % (elt * vec) == 0 &&
           stride % vec == 0;
}

template <typename T, int V, int TPR, int N>
cudaError_t fwd_rows(const LayerNormArgs& a, cudaStream_t s) {
    constexpr int threads = TPR < 128 ? 128 : TPR, rows = threads / TPR;
    const long long blocks = ((long long)a.rows + rows - 1) / rows;
    ln_fwd_kernel<T, V, TPR, N><<<(unsigned)blocks, threads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t fwd_width(const LayerNormArgs& a, cudaStream_t s) {
    const int packs = (a.D + V - 1) / V;
    // enough rows to fill the GPU with a warp per row
    const bool many = a.rows >= 16 * device_sm_count();
    if (packs <= 32) return fwd_rows<T, V, 32, 1>(a, s);
    if (packs <= 64) return fwd_rows<T, V, 32, 2>(a, s);
    if (packs <= 128 && many) return fwd_rows<T, V, 32, 4>(a, s);
    if (packs <= 256 && many) return fwd_rows<T, V, 32, 8>(a, s);
    if (packs <= 128) return fwd_rows<T, V, 128, 1>(a, s);
    if (packs <= 256) return fwd_rows<T, V, 256, 1>(a, s);
    if (packs <= 512 && many) return fwd_rows<T, V, 128, 4>(a, s);
    if (packs <= 512) return fwd_rows<T, V, 512, 1>(a, s);
    if (packs <= 1024) return fwd_rows<T, V, 256, 4>(a, s);
    if (packs <= 2048) return fwd_rows<T, V, 512, 4>(a, s);
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.D + 31) / 32);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ln_bwd_join_kernel, part, slices, a.D,
                              a.dw, a.db, (int)a.wdtype);
}

template <typename T, int V, int TPR, int N, int GROUPS>
cudaError_t bwd_rows(const LayerNormBwdArgs& a, float* part, cudaStream_t s) {
    auto* kernel = ln_bwd_kernel<T, V, TPR, N, GROUPS>;
    constexpr int bytes = TPR * N * V * (int)sizeof(float2);
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    int per = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
        &per, kernel, TPR * GROUPS, bytes);
    if (e != cudaSuccess) return e;
    const long long want = ((long long)a.rows + GROUPS - 1) / GROUPS;
    const int blocks = (int)std::min<long long>(
        want, std::min(std::max(per, 1) * device_sm_count(), kMaxSlices));
    const bool grads = a.dw || a.db;
    kernel<<<blocks, TPR * GROUPS, bytes, s>>>(a, grads ? part : nullptr);
    e = cudaGetLastError();
    return e != cudaSuccess || !grads ? e : join(a, part, blocks, s);
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
    const int packs = (a.D + V - 1) / V;
    if (packs <= 32) return bwd_rows<T, V, 32, 1, 8>(a, part, s);
    if (packs <= 64) return bwd_rows<T, V, 64, 1, 8>(a, part, s);
    if (packs <= 128) return bwd_rows<T, V, 128, 1, 4>(a, part, s);
    if (packs <= 256) return bwd_rows<T, V, 256, 1, 2>(a, part, s);
    if (packs <= 512) return bwd_rows<T, V, 512, 1, 1>(a, part, s);
    if (packs <= 1024) return bwd_rows<T, V, 512, 2, 1>(a, part, s);
    if (packs <= 2048) return bwd_rows<T, V, 1024, 2, 1>(a, part, s);
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

cudaError_t launch_layernorm(const LayerNormArgs& a, cudaStream_t stream) {
    return a.dtype == KLA_BF16 ? launch_fwd<bf16>(a, stream)
                               : launch_fwd<float>(a, stream);
}

size_t layernorm_bwd_workspace_bytes(int rows, int D, kla_dtype) {
    return (size_t)std::max(1, std::min(rows, kMaxSlices)) * 2 * D *
           sizeof(float);
}

cudaError_t launch_layernorm_bwd(const LayerNormBwdArgs& a, void* workspace,
                                 cudaStream_t stream) {
    float* part = static_cast<float*>(workspace);
    return a.dtype == KLA_BF16 ? launch_bwd<bf16>(a, part, stream)
                               : launch_bwd<float>(a, part, stream);
}

}  // namespace kla
