// Linear attention with a decay for each head: the chunked pass on the CUDA
// cores (any width up to 256, fp32 or bf16, any strides) and one token.
//
// A pass (see LinAttnJob) counts its tokens r from the first or, in reverse,
// from the last.  Over a chunk of C tokens, with S the state before it and
// w = exp(log_decay):
//   P_rs = w^(r - s) (q_r k_s)  for s <= r, else 0
//   o_r  = sum_s P_rs v_s + w^(r + e) S^T q_r
//   S   <- w^C S + sum_s w^(C - e - s) k_s v_s^T
// so that the work per token is 2 C (dk + dv) / 2 + 4 dk dv products instead
// of a state update per token, and the state leaves the chip never.
#include "kla_linattn.cuh"

namespace kla {
namespace {

using la::kNV;
using la::Part;
using la::Plan;
using la::power;
using bf16 = __nv_bfloat16;

// ------------------------------------------------------------ chunked pass

constexpr int kNT = 256;

template <int DKP>
struct Shape {
    static constexpr int C = DKP == 256 ? 32 : 64;   // tokens a chunk
    static constexpr int LD = DKP + 4;   // row of q or k: 16 rows that lie
                                         // 16 apart start in 8 bank groups
    static constexpr int LP = C + 4;
    static constexpr int FLOATS =
        2 * C * LD + C * kNV + C * LP + DKP * kNV + C + 4;
};

struct PassParams {
    Part part;
    Plan plan;
    const float* log_decay;
    int T, H;
};

// Rows r0 .. r0 + C - 1 (in the pass's order) of x into dst [C][ld], zeros
// beyond `rows` and `width`; columns c0 .. c0 + W - 1.
template <typename T, int C, int W>
__device__ __forceinline__ void load_rows(float* dst, int ld, const T* x,
                                          long long st, long long first,
                                          long long step, int rows, int c0,
                                          int width) {
    for (int i = threadIdx.x; i < C * W; i += kNT) {
        const int r = i / W, c = i % W;
        float v = 0.f;
        if (r < rows && c0 + c < width)
            v = to_f32(x[(first + step * r) * st + c0 + c]);
        dst[r * ld + c] = v;
    }
}

template <typename T, int DKP, bool STATE_ONLY>
__global__ void __launch_bounds__(kNT, 1) linattn_pass(PassParams p) {
    using Sh = Shape<DKP>;
    const LinAttnJob& j = p.part.j;
    constexpr int C = Sh::C, LD = Sh::LD, LP = Sh::LP;
    constexpr int RI = C / 16;       // rows, and columns of P, of a thread
    constexpr int RD = DKP / 16;     // rows of the state of a thread
    extern __shared__ __align__(16) float smem[];
    float* Qs = smem;
    float* Ks = Qs + C * LD;
    float* Vs = Ks + C * LD;
    float* Ps = Vs + C * kNV;
    float* S = Ps + C * LP;
    float* w = S + DKP * kNV;        // w^0 .. w^C
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int slice = blockIdx.x % p.part.slices, n0 = slice * kNV;
    const size_t bh = blockIdx.x / p.part.slices;
    const int b = bh / p.H, h = bh % p.H, part = blockIdx.y;
    const int dk = j.dk, dv = j.dv, e = j.reverse ? 0 : 1;
    const float a = p.log_decay[h];
    const T* q = static_cast<const T*>(j.q.p) + b * j.q.sb + h * j.q.sh;
    const T* k = static_cast<const T*>(j.k.p) + b * j.k.sb + h * j.k.sh;
    const T* v = static_cast<const T*>(j.v.p) + b * j.v.sb + h * j.v.sh;
    T* o = static_cast<T*>(j.o);
    const size_t sn = (size_t)dk * dv;

    if (tid <= C) w[tid] = power(a, tid);
    const float* before =
        STATE_ONLY ? nullptr : la::state_before(p.part, p.plan, part, bh);
    for (int i = tid; i < DKP * kNV; i += kNT) {
        const int r = i / kNV, c = n0 + i % kNV;
        float s = 0.f;
        if (r < dk && c < dv) {
            const size_t at = (size_t)r * j.s_r + (size_t)c * j.s_c;
            if (STATE_ONLY) {
                if (part == 0 && j.S0)
                    p.part.ws[bh * p.plan.parts * sn + at] =
                        j.S0[bh * sn + at];
            } else if (before) {
                s = before[at];
            }
        }
        S[i] = s;
    }

    const int first = part * p.plan.len;
    const int end = min(p.T, first + p.plan.len);
    const long long step = j.reverse ? -1 : 1;
    for (int r0 = first; r0 < end; r0 += C) {
        const int rows = min(C, end - r0);
        const long long t0 = j.reverse ? p.T - 1 - r0 : r0;
        if (!STATE_ONLY)
            load_rows<T, C, DKP>(Qs, LD, q, j.q.st, t0, step, rows, 0, dk);
        load_rows<T, C, DKP>(Ks, LD, k, j.k.st, t0, step, rows, 0, dk);
        load_rows<T, C, kNV>(Vs, kNV, v, j.v.st, t0, step, rows, n0, dv);
        __syncthreads();
        if (!STATE_ONLY) {
            float s[RI][RI] = {};
#pragma unroll 2
            for (int d = 0; d < DKP; d += 4) {
                float4 x[RI], y[RI];
#pragma unroll
                for (int i = 0; i < RI; ++i) {
                    x[i] = *reinterpret_cast<const float4*>(
                        &Qs[(ty + 16 * i) * LD + d]);
                    y[i] = *reinterpret_cast<const float4*>(
                        &Ks[(tx + 16 * i) * LD + d]);
                }
#pragma unroll
                for (int i = 0; i < RI; ++i)
#pragma unroll
                    for (int j = 0; j < RI; ++j)
                        s[i][j] = fmaf(x[i].w, y[j].w, fmaf(x[i].z, y[j].z,
                                  fmaf(x[i].y, y[j].y,
                                       fmaf(x[i].x, y[j].x, s[i][j]))));
            }
#pragma unroll
            for (int i = 0; i < RI; ++i)
#pragma unroll
                for (int j = 0; j < RI; ++j) {
                    const int r = ty + 16 * i, c = tx + 16 * j;
                    Ps[r * LP + c] = c <= r ? s[i][j] * w[r - c] : 0.f;
                }
            __syncthreads();

            float acc[RI][4] = {};
#pragma unroll 2
            for (int d = 0; d < DKP; d += 4) {
                float4 x[RI], y[4];
#pragma unroll
                for (int i = 0; i < RI; ++i)
                    x[i] = *reinterpret_cast<const float4*>(
                        &Qs[(ty + 16 * i) * LD + d]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    y[j] = *reinterpret_cast<const float4*>(
                        &S[(d + j) * kNV + 4 * tx]);
#pragma unroll
                for (int i = 0; i < RI; ++i) {
                    const float z[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[i][0] = fmaf(z[j], y[j].x, acc[i][0]);
                        acc[i][1] = fmaf(z[j], y[j].y, acc[i][1]);
                        acc[i][2] = fmaf(z[j], y[j].z, acc[i][2]);
                        acc[i][3] = fmaf(z[j], y[j].w, acc[i][3]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                const float u = w[ty + 16 * i + e];
#pragma unroll
                for (int n = 0; n < 4; ++n) acc[i][n] *= u;
            }
            // later rows are skipped, not multiplied by 0: what is not finite
            // in them may not reach this one
#pragma unroll 2
            for (int c = 0; c < C; ++c) {
                const float4 y =
                    *reinterpret_cast<const float4*>(&Vs[c * kNV + 4 * tx]);
#pragma unroll
                for (int i = 0; i < RI; ++i) {
                    const int r = ty + 16 * i;
                    if (c <= r) {
                        const float x = Ps[r * LP + c];
                        acc[i][0] = fmaf(x, y.x, acc[i][0]);
                        acc[i][1] = fmaf(x, y.y, acc[i][1]);
                        acc[i][2] = fmaf(x, y.z, acc[i][2]);
                        acc[i][3] = fmaf(x, y.w, acc[i][3]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                const int r = ty + 16 * i;
                if (r >= rows) continue;
                const size_t t = (size_t)(t0 + step * r);
                T* dst = o + (((size_t)b * p.T + t) * p.H + h) * dv;
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    if (n0 + 4 * tx + n < dv)
                        dst[n0 + 4 * tx + n] = from_f32<T>(acc[i][n]);
            }
            __syncthreads();
        }
        // w^n S as S + (w^n - 1) S: n * log_decay close to 0 keeps its digits
        const float grow = expm1f(a * (float)rows);
        float4 u[RD] = {};
        for (int c = 0; c < rows; ++c) {
            const float x = w[rows - e - c];
            float4 y = *reinterpret_cast<const float4*>(&Vs[c * kNV + 4 * tx]);
            y.x *= x, y.y *= x, y.z *= x, y.w *= x;
            const float* kr = &Ks[c * LD + ty * RD];
#pragma unroll
            for (int d = 0; d < RD; ++d) {
                u[d].x = fmaf(kr[d], y.x, u[d].x);
                u[d].y = fmaf(kr[d], y.y, u[d].y);
                u[d].z = fmaf(kr[d], y.z, u[d].z);
                u[d].w = fmaf(kr[d], y.w, u[d].w);
            }
        }
#pragma unroll
        for (int d = 0; d < RD; ++d) {
            float4* s = reinterpret_cast<float4*>(
                &S[(ty * RD + d) * kNV + 4 * tx]);
            float4 x = *s;
            x.x = fmaf(grow, x.x, x.x) + u[d].x;
            x.y = fmaf(grow, x.y, x.y) + u[d].y;
            x.z = fmaf(grow, x.z, x.z) + u[d].z;
            x.w = fmaf(grow, x.w, x.w) + u[d].w;
            *s = x;
        }
        __syncthreads();
    }

    if (!STATE_ONLY && (part + 1 < p.plan.parts || !j.ST)) return;
    float* dst = STATE_ONLY ? p.part.ws + (bh * p.plan.parts + part + 1) * sn
                            : j.ST + bh * sn;
    for (int i = tid; i < DKP * kNV; i += kNT) {
        const int r = i / kNV, c = n0 + i % kNV;
        if (r < dk && c < dv)
            dst[(size_t)r * j.s_r + (size_t)c * j.s_c] = S[i];
    }
}

// A thread has one element of the states of one sequence and head.
__global__ void __launch_bounds__(256)
linattn_join(float* ws, const float* log_decay, int parts, int len, int H,
             int n, int blocks, bool first) {
    const size_t bh = blockIdx.x / blocks;
    const int at = blockIdx.x % blocks * 256 + threadIdx.x;
    if (at >= n) return;
    const float f = power(log_decay[bh % H], len);
    float* x = ws + bh * parts * n + at;
    float s = first ? x[0] : 0.f;
    for (int i = 1; i < parts; i += 8) {     // eight on their way at a time
        float u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k < parts) u[k] = x[(size_t)(i + k) * n];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i + k >= parts) break;
            s = fmaf(f, s, u[k]);
            x[(size_t)(i + k) * n] = s;
        }
    }
}

// Parts of a sequence: enough for about two blocks an SM, at least 256
// tokens each.
Plan plan(long long blocks, int T) {
    constexpr int kSMs = 152, kLeast = 256;
    long long parts = 2 * kSMs / blocks;
    if (parts > T / kLeast) parts = T / kLeast;
    if (parts > 32) parts = 32;
    if (parts < 2) return {1, T};
    int len = (int)((T + parts - 1) / parts);
    len = (len + 63) / 64 * 64;
    return {(T + len - 1) / len, len};
}

template <typename T, int DKP, bool STATE_ONLY>
cudaError_t launch_pass(const PassParams& p, long long bh,
                        cudaStream_t stream) {
    constexpr int bytes = Shape<DKP>::FLOATS * 4;
    auto kern = linattn_pass<T, DKP, STATE_ONLY>;
    cudaError_t e = cudaFuncSetAttribute(
        kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(bh * p.part.slices),
                    p.plan.parts - (STATE_ONLY ? 1 : 0));
    kern<<<grid, kNT, bytes, stream>>>(p);
    return cudaGetLastError();
}

template <typename T, int DKP>
cudaError_t launch_job(const PassParams& p, long long bh,
                       cudaStream_t stream) {
    if (p.plan.parts > 1) {
        cudaError_t e = launch_pass<T, DKP, true>(p, bh, stream);
        if (e == cudaSuccess)
            e = la::join_parts(p.part, p.plan, p.log_decay, bh, p.H, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_pass<T, DKP, false>(p, bh, stream);
}

Plan plan_of(const LinAttnArgs& a, int job) {
    return plan((long long)a.B * a.H * la::slices_of(a.job[job]), a.T);
}

// Floats of the part states of a job.
size_t part_floats(const LinAttnArgs& a, int job, const Plan& pl) {
    const LinAttnJob& j = a.job[job];
    return pl.parts > 1 ? (size_t)a.B * a.H * pl.parts * j.dk * j.dv : 0;
}

template <typename T>
cudaError_t launch_all(const LinAttnArgs& a, float* ws, cudaStream_t stream) {
    const long long bh = (long long)a.B * a.H;
    for (int i = 0; i < a.jobs; ++i) {
        const LinAttnJob& j = a.job[i];
        const Plan pl = plan_of(a, i);
        const PassParams p{{j, ws, la::slices_of(j)}, pl, a.log_decay, a.T,
                           a.H};
        const cudaError_t e =
            j.dk <= 64    ? launch_job<T, 64>(p, bh, stream)
            : j.dk <= 128 ? launch_job<T, 128>(p, bh, stream)
                          : launch_job<T, 256>(p, bh, stream);
        if (e != cudaSuccess) return e;
        if (pl.parts > 1) ws += part_floats(a, i, pl);
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t la::join_parts(const Part& p, const Plan& pl,
                           const float* log_decay, long long bh, int H,
                           cudaStream_t stream) {
    const int n = p.j.dk * p.j.dv, blocks = (n + 255) / 256;
    linattn_join<<<(unsigned)(bh * blocks), 256, 0, stream>>>(
        p.ws, log_decay, pl.parts, pl.len, H, n, blocks, p.j.S0 != nullptr);
    return cudaGetLastError();
}

// By the sizes alone, whichever form the tensors' alignment allows.
size_t linattn_workspace_bytes(const LinAttnArgs& a) {
    size_t n = 0, tc = 0;
    for (int i = 0; i < a.jobs; ++i) {
        n += part_floats(a, i, plan_of(a, i));
        if (linattn_tc_sizes(a)) tc += part_floats(a, i, linattn_tc_plan(a));
    }
    return (n > tc ? n : tc) * sizeof(float);
}

cudaError_t launch_linattn(const LinAttnArgs& a, void* workspace,
                           cudaStream_t stream) {
    float* ws = static_cast<float*>(workspace);
    if (linattn_tc_eligible(a)) return launch_linattn_tc(a, ws, stream);
    return a.dtype == KLA_BF16 ? launch_all<bf16>(a, ws, stream)
                               : launch_all<float>(a, ws, stream);
}

// ---------------------------------------------------------------- one token

namespace {

// One block per head and tile of CG * VEC columns; a thread holds VEC
// adjacent columns of every RS-th row.  The state is read and written once:
// 8 dk dv bytes a head are all that matters here.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
linattn_step(LinAttnStepArgs a, int cg_log2, int tiles) {
    constexpr int NT = 256, BATCH = 8;
    const int CG = 1 << cg_log2, RS = NT >> cg_log2;
    const int tid = threadIdx.x, cg = tid & (CG - 1), rs = tid >> cg_log2;
    const size_t head = blockIdx.x / tiles;
    const int n = head / a.H, h = head % a.H;
    const int col = (blockIdx.x % tiles) * CG * VEC + cg * VEC;
    const bool in = col < a.dv;      // dv is a multiple of VEC
    __shared__ float qs[kLinAttnMaxWidth], ks[kLinAttnMaxWidth];
    __shared__ float red[NT * VEC];
    await_grid_before();
    release_grid_after();
    float* S = a.S + head * a.dk * a.dv + col;
    float s[BATCH][VEC];
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = r0 + rs + i * RS;
            if (!in || r >= a.dk) continue;
            if constexpr (VEC == 4) {
                const float4 x = __ldcs(
                    reinterpret_cast<const float4*>(S + (size_t)r * a.dv));
                s[i][0] = x.x, s[i][1] = x.y, s[i][2] = x.z, s[i][3] = x.w;
            } else {
                s[i][0] = __ldcs(S + (size_t)r * a.dv);
            }
        }
    };
    load(0);
    const T* q = static_cast<const T*>(a.q.p) + n * a.q.sb + h * a.q.sh;
    const T* k = static_cast<const T*>(a.k.p) + n * a.k.sb + h * a.k.sh;
    const T* v = static_cast<const T*>(a.v.p) + n * a.v.sb + h * a.v.sh;
    if (tid < a.dk) {                // dk <= 256 threads
        qs[tid] = to_f32(q[tid]);
        ks[tid] = to_f32(k[tid]);
    }
    float val[VEC], acc[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        val[c] = in ? to_f32(v[col + c]) : 0.f;
        acc[c] = 0.f;
    }
    const float decay = expf(a.log_decay[h]);
    __syncthreads();
    for (int r0 = 0; r0 < a.dk; r0 += BATCH * RS) {
        if (r0) load(r0);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = r0 + rs + i * RS;
            if (!in || r >= a.dk) continue;
            const float kr = ks[r], qr = qs[r];
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                s[i][c] = fmaf(decay, s[i][c], kr * val[c]);
                acc[c] = fmaf(qr, s[i][c], acc[c]);
            }
            if constexpr (VEC == 4)
                __stcs(reinterpret_cast<float4*>(S + (size_t)r * a.dv),
                       make_float4(s[i][0], s[i][1], s[i][2], s[i][3]));
            else
                __stcs(S + (size_t)r * a.dv, s[i][0]);
        }
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) red[(rs * CG + cg) * VEC + c] = acc[c];
    __syncthreads();
    // thread = column: the sums of all row slices in a fixed order
    const int c = (blockIdx.x % tiles) * CG * VEC + tid;
    if (tid < CG * VEC && c < a.dv) {
        float x = 0.f;
        for (int r = 0; r < RS; ++r) x += red[r * CG * VEC + tid];
        static_cast<T*>(a.o)[head * a.dv + c] = from_f32<T>(x);
    }
}

template <typename T>
cudaError_t launch_step(const LinAttnStepArgs& a, cudaStream_t stream) {
    const long long heads = (long long)a.N * a.H;
    const bool vec = a.dv % 4 == 0 &&
                     (reinterpret_cast<uintptr_t>(a.S) & 15) == 0;
    const int v = vec ? 4 : 1;
    // a row of a tile is at least a 128-byte line (32 fp32), at most 128
    // columns; narrower tiles where the heads alone do not fill the SMs
    int cg = vec ? (heads >= 304 ? 5 : 3) : 5;
    while (cg > 3 && (v << (cg - 1)) >= a.dv) --cg;
    const int tiles = (a.dv + (v << cg) - 1) / (v << cg);
    const dim3 grid((unsigned)(heads * tiles));
    return vec ? launch_dependent(linattn_step<T, 4>, grid, 256, stream, 0, a,
                                  cg, tiles)
               : launch_dependent(linattn_step<T, 1>, grid, 256, stream, 0, a,
                                  cg, tiles);
}

}  // namespace

cudaError_t launch_linattn_step(const LinAttnStepArgs& a,
                                cudaStream_t stream) {
    return a.dtype == KLA_BF16 ? launch_step<bf16>(a, stream)
                               : launch_step<float>(a, stream);
}

}  // namespace kla
