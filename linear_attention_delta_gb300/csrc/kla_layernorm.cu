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
#include "kla_internal.cuh"

namespace kla {
namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float load(const void* p, long long i, int dt) {
    return dt == KLA_BF16 ? to_f32(static_cast<const bf16*>(p)[i])
                          : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// Sum over the block of two values at once; every thread gets both.
__device__ __forceinline__ float2 block_sum(float a, float b, float2* red) {
    const int warp = threadIdx.x / 32, nw = blockDim.x / 32;
    a = warp_sum(a);
    b = warp_sum(b);
    __syncthreads();             // red is free again
    if (threadIdx.x % 32 == 0) red[warp] = make_float2(a, b);
    __syncthreads();
    float2 t = make_float2(0.f, 0.f);
    for (int w = 0; w < nw; ++w) {
        t.x += red[w].x;
        t.y += red[w].y;
    }
    return t;
}

constexpr int kLoopThreads = 512;

// Any D, strides and alignment: one block per row, which it reads three
// times (from L1 or L2 after the first).
template <typename T>
__global__ void __launch_bounds__(kLoopThreads)
ln_fwd_loop_kernel(LayerNormArgs a) {
    __shared__ float2 red[kLoopThreads / 32];
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
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
        const float rstd =
            1.f / sqrtf(block_sum(t, 0.f, red).x / a.D + a.eps);
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
}

// dx of any D: one block per row, two passes over x and dy.
template <typename T>
__global__ void __launch_bounds__(kLoopThreads)
ln_bwd_loop_kernel(LayerNormBwdArgs a) {
    __shared__ float2 red[kLoopThreads / 32];
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
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

// dw, db = the slices' partial sums added up in a fixed order.
__global__ void ln_bwd_join_kernel(const float* part, int slices, int D,
                                   void* dw, void* db, int wdtype) {
    const int col = blockIdx.x * blockDim.x + threadIdx.x;
    if (col >= D) return;
    float w = 0.f, b = 0.f;
    for (int i = 0; i < slices; ++i) {
        w += part[(size_t)i * 2 * D + col];
        b += part[((size_t)i * 2 + 1) * D + col];
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

int row_slices(int rows) { return rows < 128 ? (rows ? rows : 1) : 128; }

template <typename T>
cudaError_t launch_fwd(const LayerNormArgs& a, cudaStream_t s) {
    ln_fwd_loop_kernel<T><<<a.rows, kLoopThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(const LayerNormBwdArgs& a, float* part,
                       cudaStream_t s) {
    if (a.rows > 0) ln_bwd_loop_kernel<T><<<a.rows, kLoopThreads, 0, s>>>(a);
    if (!a.dw && !a.db) return cudaGetLastError();
    const int blocks = (a.D + 127) / 128, slices = row_slices(a.rows);
    ln_bwd_cols_kernel<T><<<dim3(blocks, slices), 128, 0, s>>>(a, part);
    ln_bwd_join_kernel<<<blocks, 128, 0, s>>>(part, slices, a.D, a.dw, a.db,
                                              a.wdtype);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layernorm(const LayerNormArgs& a, cudaStream_t stream) {
    return a.dtype == KLA_BF16 ? launch_fwd<bf16>(a, stream)
                               : launch_fwd<float>(a, stream);
}

size_t layernorm_bwd_workspace_bytes(int rows, int D, kla_dtype) {
    return (size_t)row_slices(rows) * 2 * D * sizeof(float);
}

cudaError_t launch_layernorm_bwd(const LayerNormBwdArgs& a, void* workspace,
                                 cudaStream_t stream) {
    float* part = static_cast<float*>(workspace);
    return a.dtype == KLA_BF16 ? launch_bwd<bf16>(a, part, stream)
                               : launch_bwd<float>(a, part, stream);
}

}  // namespace kla
