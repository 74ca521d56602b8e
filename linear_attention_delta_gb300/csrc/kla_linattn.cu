// Linear attention with a decay for each head: the chunked pass for fp32 and
// for what the bf16 form on tcgen05 does not take (wide or odd heads, rows off
// their 16 bytes), and one token.
//
// A pass (see LinAttnJob) counts its tokens r from the first or, in reverse,
// from the last.  Over a chunk of C tokens, with S the state before it and
// w = exp(log_decay):
//   P_rs = w^(r - s) (q_r k_s)  for s <= r, else 0
//   o_r  = sum_s P_rs v_s + w^(r + e) S^T q_r
//   S   <- w^C S + sum_s w^(C - e - s) k_s v_s^T
// so that the work per token is 2 C (dk + dv) / 2 + 4 dk dv products instead
// of a state update per token, and the state leaves the chip never.
//
// The products are warp-level ones of tf32 (mma.sync): a number of fp32 is two
// of tf32, x = hi + lo up to 2^-23, and x y = hi hi' + hi lo' + lo hi' up to
// 2^-22; bf16 inputs are one of tf32 and need no lo.  (tcgen05 adds up inside
// the instruction, which cuts off what it adds: with sums there, and not outside
// as here, outputs were 7 times as far from the exact ones.  And it takes its
// operands from shared memory, where two tiles in place of each would leave no
// room for a second stage of 128-wide heads.)  Chunks of 64 tokens by 64 columns of the state a block, 16
// warps, two stages: 640 us at B4 T4096 H16 d128 fp32 (HBM would take 79), 10 us
// a chunk.  The warp-level products bound it: at 750 us, without two of the three
// of a pair 275 less; without them and the fragments taken apart for them 530
// less (Q S and the scores 290, U 167, P V 62).  On the way: one stage 878 us; a
// loop of its own for the scores, fragments by single loads 808; a place's
// address and bounds formed anew for every copy, single elements of P, S and o
// 745; the lower triangle's work uneven among the schedulers 692.
#include "f32x2.cuh"
#include "kla_linattn.cuh"
#include "tc_primitives.cuh"

namespace kla {
namespace {

using la::kMaxJobs;
using la::kNV;
using la::Part;
using la::Plan;
using la::power;
using bf16 = __nv_bfloat16;

// ------------------------------------------------------------ chunked pass

constexpr int kNT = 512;

template <int DKP>
struct Shape {
    static constexpr int C = DKP == 256 ? 32 : 64;   // tokens a chunk
    // rows of q, k and P lie 4 banks apart, those of v and S 8: a warp's
    // fragments come from 32 different banks
    static constexpr int LD = DKP + 4;
    static constexpr int LP = C + 4;
    static constexpr int LV = kNV + 8;
    static constexpr int STAGE = 2 * C * LD + C * LV;   // q, k and v
    static constexpr int FLOATS =
        2 * STAGE + C * LP + DKP * LV + C + 4 + kNV;
    static_assert(FLOATS * 4 <= 232448, "shared memory");
};

// A number as one or two of tf32 (11 bits; the products look at no lower
// ones), the first rounded by adding half a step to its bits (the conversion
// instruction has a quarter of the rate), the second cut off: 2^-22 of x.
template <bool EXACT>
struct Split {
    uint32_t hi, lo;
    __device__ __forceinline__ explicit Split(float x) {
        hi = __float_as_uint(x);
        lo = 0;
        if (!EXACT) {
            hi = (hi + 0x1000u) & 0xffffe000u;
            // what is not finite: NaN here, whatever hi is
            lo = __float_as_uint(x - __uint_as_float(hi));
        }
    }
};
template <bool EXACT>
struct FragA {
    uint32_t hi[4], lo[4];
    // elements (row g or g + 8, step t or t + 4)
    __device__ __forceinline__ FragA(float x0, float x1, float x2, float x3) {
        const float x[4] = {x0, x1, x2, x3};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Split<EXACT> s(x[i]);
            hi[i] = s.hi, lo[i] = s.lo;
        }
    }
};
// d[n] += a b[n] (16 x 8 x 8, N tiles) to the precision above.  The sum over k
// is d's own, in fp32: the product instruction cuts off what it adds up, which
// over a row of 72 ended 4 times as far from the exact sum.  The tiles'
// products alternate: those of one tile wait for one another.
template <bool XA, bool XB, int N>
__device__ __forceinline__ void mma(float (&d)[N][4], const FragA<XA>& a,
                                    const float (&b)[N][2]) {
    float s[N][4] = {};
    uint32_t hi[N][2], lo[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const Split<XB> x(b[n][i]);
            hi[n][i] = x.hi, lo[n][i] = x.lo;
        }
    if (!XA)
#pragma unroll
        for (int n = 0; n < N; ++n)
            tc::mma_m16n8k8_tf32(s[n], a.lo, hi[n][0], hi[n][1]);
    if (!XB)
#pragma unroll
        for (int n = 0; n < N; ++n)
            tc::mma_m16n8k8_tf32(s[n], a.hi, lo[n][0], lo[n][1]);
#pragma unroll
    for (int n = 0; n < N; ++n)
        tc::mma_m16n8k8_tf32(s[n], a.hi, hi[n][0], hi[n][1]);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const float2 x = add2(make_float2(d[n][i], d[n][i + 1]),
                                  make_float2(s[n][i], s[n][i + 1]));
            d[n][i] = x.x, d[n][i + 1] = x.y;
        }
}
// 8 x 4 blocks of fp32 (rows of 16 bytes at the addresses of 8 lanes each);
// lane 4 g + t gets element (g, t) of each: fragments of the products, where
// rows lie along the sum's axis (written before the last block barrier).
__device__ __forceinline__ void load_blocks(float& a, float& b, float& c,
                                            float& d, const float* row) {
    asm volatile(
        "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
        : "=f"(a), "=f"(b), "=f"(c), "=f"(d)
        : "r"(tc::smem_u32(row)));
}
__device__ __forceinline__ void load_blocks(float (&x)[2][2],
                                            const float* row) {
    load_blocks(x[0][0], x[0][1], x[1][0], x[1][1], row);
}
__device__ __forceinline__ void load_blocks(float (&x)[1][2],
                                            const float* row) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];"
                 : "=f"(x[0][0]), "=f"(x[0][1])
                 : "r"(tc::smem_u32(row)));
}

__device__ __forceinline__ void store_two(float* p, float a, float b) {
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
}
__device__ __forceinline__ void store_two(bf16* p, float a, float b) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

struct PassParams {
    Part part[kMaxJobs];
    int first[kMaxJobs + 1];     // first block of each pass
    Plan plan;                   // the same for all passes
    const float* log_decay;
    int T, H;
};

// Rows r0 .. r0 + C - 1 (in the pass's order) of x into dst [C][ld], zeros
// beyond `rows` and `width`; columns c0 .. c0 + W - 1, the first `most` of
// them.
// Four adjacent elements at a time where they line up (`by4`): fp32 straight to
// shared memory (complete after wait_copies).
template <typename T, int C, int W>
__device__ __forceinline__ void load_rows(float* dst, int ld, const T* x,
                                          long long st, long long first,
                                          long long step, int rows, int c0,
                                          int width, int most, bool by4) {
    if (by4) {
        // a thread has one place of every RS-th row
        constexpr int RS = kNT / (W / 4);
        const int r0 = threadIdx.x / (W / 4), c = threadIdx.x % (W / 4) * 4;
        if (c >= most) return;
        const bool inside = c0 + c < width;
        const T* from = x + (first + step * r0) * st + c0 + c;
        const long long next = step * RS * st;
        float* to = &dst[r0 * ld + c];
#pragma unroll
        for (int r = 0; r < C; r += RS, to += RS * ld) {
            const bool in = inside && r0 + r < rows;
            if constexpr (sizeof(T) == 4) {
                // 16 bytes, or none of them (zeros)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::
                                 "r"(tc::smem_u32(to)),
                             "l"(in ? from : x), "r"(in ? 16 : 0)
                             : "memory");
            } else {
                const uint2 u = in ? *reinterpret_cast<const uint2*>(from)
                                   : make_uint2(0u, 0u);
                const float2 y = from_bf16x2(u.x), z = from_bf16x2(u.y);
                *reinterpret_cast<float4*>(to) =
                    make_float4(y.x, y.y, z.x, z.y);
            }
            from += next;
        }
        return;
    }
#pragma unroll 8
    for (int i = threadIdx.x; i < C * W; i += kNT) {
        const int r = i / W, c = i % W;
        if (c >= most) continue;
        float v = 0.f;
        if (r < rows && c0 + c < width)
            v = to_f32(x[(first + step * r) * st + c0 + c]);
        dst[r * ld + c] = v;
    }
}
__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" :::
                     "memory");
}

// Whether rows of x can be read four elements at a time.
template <typename T>
__device__ __forceinline__ bool in_fours(const T* x, long long st, int width) {
    return (reinterpret_cast<uintptr_t>(x) % (4 * sizeof(T))) == 0 &&
           st % 4 == 0 && width % 4 == 0;
}

template <typename T, int DKP, bool STATE_ONLY>
__global__ void __launch_bounds__(kNT, 1) linattn_pass(PassParams p) {
    using Sh = Shape<DKP>;
    constexpr int C = Sh::C, LD = Sh::LD, LP = Sh::LP, LV = Sh::LV;
    constexpr bool X = sizeof(T) == 2;      // inputs are one of tf32 each
    // 16 warps: tiles of 16 rows, NG groups of 8-column tiles
    constexpr int MT = C / 16, NG = 16 / MT, NO = kNV / 8 / NG;
    constexpr int UT = DKP / 16, UG = 16 / UT, NU = kNV / 8 / UG;
    int job = 0;
    while (job + 1 < kMaxJobs && (int)blockIdx.x >= p.first[job + 1]) ++job;
    const Part& pt = p.part[job];
    const LinAttnJob& j = pt.j;
    extern __shared__ __align__(16) float smem[];
    float* Ps = smem + 2 * Sh::STAGE;
    float* S = Ps + C * LP;
    float* w = S + DKP * LV;         // w^0 .. w^C
    int* bad = reinterpret_cast<int*>(w + C + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int parts = STATE_ONLY ? p.plan.parts - 1 : p.plan.parts;
    int item = blockIdx.x - p.first[job];
    const int n0 = item % pt.slices * kNV;
    item /= pt.slices;
    const int part = item % parts;
    const size_t bh = item / parts;
    const int b = bh / p.H, h = bh % p.H;
    const int dk = j.dk, dv = j.dv, e = j.reverse ? 0 : 1;
    // (with parts the join came before, which itself waited: what is not of the
    // workspace is there)
    if (STATE_ONLY || p.plan.parts == 1) await_grid_before();
    const float a = p.log_decay[h];
    const T* q = static_cast<const T*>(j.q.p) + b * j.q.sb + h * j.q.sh;
    const T* k = static_cast<const T*>(j.k.p) + b * j.k.sb + h * j.k.sh;
    const T* v = static_cast<const T*>(j.v.p) + b * j.v.sb + h * j.v.sh;
    T* o = static_cast<T*>(j.o);
    const size_t sn = (size_t)dk * dv;
    const int dk8 = (dk + 7) / 8 * 8;     // columns of q and k that are looked at

    if (tid <= C) w[tid] = power(a, tid);
    // the state's elements in the order in which they lie in memory
    const bool by_row = j.s_c == 1;
    auto r_of = [&](int i) { return by_row ? i / kNV : i % DKP; };
    auto n_of = [&](int i) { return by_row ? i % kNV : i / DKP; };
    // two outputs at a time
    const bool o2 = dv % 2 == 0 &&
                    reinterpret_cast<uintptr_t>(o) % (2 * sizeof(T)) == 0;
    const bool q4 = in_fours(q, j.q.st, dk), k4 = in_fours(k, j.k.st, dk);
    const bool v4 = in_fours(v, j.v.st, dv);
    const int first = part * p.plan.len;
    const int end = first + min(p.T - first, p.plan.len);
    const long long step = j.reverse ? -1 : 1;
    // chunks alternate between two stages: one is loaded while the other is
    // worked on
    auto load = [&](int r0) {
        float* Qs = smem + ((r0 - first) / C & 1) * Sh::STAGE;
        const int rows = min(C, end - r0);
        const long long t0 = j.reverse ? p.T - 1 - r0 : r0;
        if (!STATE_ONLY)
            load_rows<T, C, DKP>(Qs, LD, q, j.q.st, t0, step, rows, 0, dk, dk8,
                                 q4);
        load_rows<T, C, DKP>(Qs + C * LD, LD, k, j.k.st, t0, step, rows, 0, dk,
                             dk8, k4);
        load_rows<T, C, kNV>(Qs + 2 * C * LD, LV, v, j.v.st, t0, step, rows,
                             n0, dv, kNV, v4);
    };
    load(first);
    await_grid_before();
    const float* before =
        STATE_ONLY ? nullptr : la::state_before(pt, p.plan, part, bh);
#pragma unroll 4
    for (int i = tid; i < DKP * kNV; i += kNT) {
        const int r = r_of(i), n = n_of(i), c = n0 + n;
        float s = 0.f;
        if (r < dk && c < dv) {
            const size_t at = (size_t)r * j.s_r + (size_t)c * j.s_c;
            if (STATE_ONLY) {
                if (part == 0 && j.S0)
                    pt.ws[bh * p.plan.parts * sn + at] = j.S0[bh * sn + at];
            } else if (before) {
                s = before[at];
            }
        }
        S[r * LV + n] = s;
    }
    for (int r0 = first; r0 < end; r0 += C) {
        float* Qs = smem + ((r0 - first) / C & 1) * Sh::STAGE;
        float* Ks = Qs + C * LD;
        float* Vs = Ks + C * LD;
        const int rows = min(C, end - r0);
        const long long t0 = j.reverse ? p.T - 1 - r0 : r0;
        if (tid < kNV) bad[tid] = C;
        wait_copies();
        __syncthreads();
        if (end - r0 > C) load(r0 + C);
        // What is not finite in v is taken out, as in P v it would meet the
        // zeros of earlier rows; its column's later outputs and state get NaN.
        bool found = false;
#pragma unroll
        for (int i = tid; i < C * kNV / 4; i += kNT) {
            const int r = i / (kNV / 4), c = i % (kNV / 4) * 4;
            float* x = &Vs[r * LV + c];
            const float4 y = *reinterpret_cast<const float4*>(x);
            // x - x is 0 of a finite x, else NaN
            if ((y.x - y.x) + (y.y - y.y) + (y.z - y.z) + (y.w - y.w) == 0.f)
                continue;
            found = true;
            for (int k = 0; k < 4; ++k)
                if ((__float_as_uint(x[k]) & 0x7f800000u) == 0x7f800000u) {
                    x[k] = 0.f;
                    atomicMin(&bad[c + k], r);
                }
        }
        // (warps of one scheduler, those equal modulo 4, have different rows, and
        // with 4 x 4 tiles of scores two or three of the lower triangle's ten)
        const int m = (warp ^ warp >> 2) & (MT - 1), ng = warp / MT;
        float acc[NO][4];
        // this lane's row of the blocks of an A fragment (16 x 8)
        const int arow = 16 * m + (lane & 15), acol = (lane >> 4) * 4;
        if (!STATE_ONLY) {
            // scores and Q S together, 16 rows x NO 8-column tiles a warp
            float sc[NO][4];
#pragma unroll
            for (int n = 0; n < NO; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = sc[n][i] = 0.f;
            const int s0 = (MT == 4 ? (warp + 2 * ng) & 3 : ng) * NO * 8;
            // columns all above the diagonal stay 0
            const bool below = s0 < C && s0 <= 16 * m + 15;
            const float* x = &Qs[arow * LD + acol];
            // (NO tiles; the lanes beyond 8 NO rows repeat addresses in use)
            const float* y =
                &Ks[((below ? s0 : 0) + (lane & 7) + (NO > 1 ? lane >> 4 << 3 : 0)) *
                        LD + (lane >> 3 & 1) * 4];
            const float* z = &S[t * LV + ng * NO * 8 + g];
#pragma unroll 2
            for (int d = 0; d < dk8; d += 8) {
                float v[4];
                load_blocks(v[0], v[1], v[2], v[3], x + d);
                const FragA<X> f(v[0], v[1], v[2], v[3]);
                if (below) {
                    float u[NO][2];
                    load_blocks(u, y + d);
                    mma<X, X>(sc, f, u);
                }
                float u[NO][2];
#pragma unroll
                for (int n = 0; n < NO; ++n)
                    u[n][0] = z[d * LV + 8 * n], u[n][1] = z[(d + 4) * LV + 8 * n];
                mma<X, false>(acc, f, u);
            }
            if (s0 < C) {
#pragma unroll
                for (int n = 0; n < NO; ++n)
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const int r = 16 * m + g + i * 4;
                        const int c = s0 + 8 * n + 2 * t;
                        *reinterpret_cast<float2*>(&Ps[r * LP + c]) =
                            make_float2(
                                c <= r ? sc[n][i] * w[r - c] : 0.f,
                                c < r ? sc[n][i + 1] * w[r - c - 1] : 0.f);
                    }
            }
            // rows of Q S times w^(r + e)
            const float u0 = w[16 * m + g + e], u1 = w[16 * m + g + 8 + e];
#pragma unroll
            for (int n = 0; n < NO; ++n)
                acc[n][0] *= u0, acc[n][1] *= u0, acc[n][2] *= u1,
                    acc[n][3] *= u1;
        }
        // P in place; S read
        const bool any = __syncthreads_or(found);
        if (!STATE_ONLY) {
            const float* x = &Ps[arow * LP + acol];
            const float* y = &Vs[t * LV + ng * NO * 8 + g];
#pragma unroll 2
            for (int c = 0; c < 16 * m + 16; c += 8) {
                float v[4];
                load_blocks(v[0], v[1], v[2], v[3], x + c);
                const FragA<false> f(v[0], v[1], v[2], v[3]);
                float u[NO][2];
#pragma unroll
                for (int n = 0; n < NO; ++n)
                    u[n][0] = y[c * LV + 8 * n], u[n][1] = y[(c + 4) * LV + 8 * n];
                mma<false, X>(acc, f, u);
            }
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const int r = 16 * m + g + i * 4;
                if (r >= rows) continue;
                const size_t at = (size_t)(t0 + step * r);
                T* dst = o + (((size_t)b * p.T + at) * p.H + h) * dv + n0;
#pragma unroll
                for (int n = 0; n < NO; ++n) {
                    const int c = (ng * NO + n) * 8 + 2 * t;
                    float u0 = acc[n][i], u1 = acc[n][i + 1];
                    if (any) {
                        const float nan = __uint_as_float(0x7fc00000u);
                        if (r >= bad[c]) u0 = nan;
                        if (r >= bad[c + 1]) u1 = nan;
                    }
                    if (o2) {        // dv is even
                        if (n0 + c < dv) store_two(dst + c, u0, u1);
                    } else {
                        if (n0 + c < dv) dst[c] = from_f32<T>(u0);
                        if (n0 + c + 1 < dv) dst[c + 1] = from_f32<T>(u1);
                    }
                }
            }
        }
        // U: 16 rows of the state x NU 8-column tiles a warp
        const int ug = warp / UT, um = (warp + ug) % UT;
        if (16 * um < dk) {
            float u[NU][4];
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) u[n][i] = 0.f;
            const float* x = &Ks[t * LD + 16 * um + g];
            const float* y = &Vs[t * LV + ug * NU * 8 + g];
#pragma unroll 1
            for (int c = 0; c < rows; c += 8) {
                // rows beyond the sequence are zero: their weight is any
                const float w0 = w[max(0, rows - e - c - t)];
                const float w1 = w[max(0, rows - e - c - t - 4)];
                const FragA<false> f(w0 * x[c * LD], w0 * x[c * LD + 8],
                                     w1 * x[(c + 4) * LD],
                                     w1 * x[(c + 4) * LD + 8]);
                float v[NU][2];
#pragma unroll
                for (int n = 0; n < NU; ++n)
                    v[n][0] = y[c * LV + 8 * n], v[n][1] = y[(c + 4) * LV + 8 * n];
                mma<false, X>(u, f, v);
            }
            // w^n S as S + (w^n - 1) S: n * log_decay close to 0 keeps its
            // digits
            const float grow = expm1f(a * (float)rows);
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const int c = (ug * NU + n) * 8 + 2 * t;
                    float2* s = reinterpret_cast<float2*>(
                        &S[(16 * um + g + i * 4) * LV + c]);
                    float2 y = *s;
                    y = add2(fma2(both(grow), y, y),
                             make_float2(u[n][i], u[n][i + 1]));
                    if (any) {
                        const float nan = __uint_as_float(0x7fc00000u);
                        if (bad[c] < C) y.x = nan;
                        if (bad[c + 1] < C) y.y = nan;
                    }
                    *s = y;
                }
        }
        __syncthreads();
    }

    if (!STATE_ONLY && (part + 1 < p.plan.parts || !j.ST)) return;
    float* dst = STATE_ONLY
                     ? pt.ws + (bh * p.plan.parts + part + 1) * sn
                     : j.ST + bh * sn;
    for (int i = tid; i < DKP * kNV; i += kNT) {
        const int r = r_of(i), n = n_of(i), c = n0 + n;
        if (r < dk && c < dv)
            dst[(size_t)r * j.s_r + (size_t)c * j.s_c] = S[r * LV + n];
    }
}

struct JoinParams {
    Part part[kMaxJobs];
    int first[kMaxJobs + 1];     // first block of each pass
    Plan plan;
    const float* log_decay;
    int H;
};

constexpr int kJoin = 256;       // elements a block has

// A thread has one element of the states of one sequence and head.
__global__ void __launch_bounds__(kJoin) linattn_join(JoinParams p) {
    int job = 0;
    while (job + 1 < kMaxJobs && (int)blockIdx.x >= p.first[job + 1]) ++job;
    const Part& pt = p.part[job];
    const int n = pt.j.dk * pt.j.dv, blocks = (n + kJoin - 1) / kJoin;
    const int item = blockIdx.x - p.first[job], parts = p.plan.parts;
    const size_t bh = item / blocks;
    const int at = item % blocks * kJoin + threadIdx.x;
    // the passes read what came before the first of them at once: not before
    // it is all there
    await_grid_before();
    release_grid_after();
    if (at >= n) return;
    const float f = power(p.log_decay[bh % p.H], p.plan.len);
    float* x = pt.ws + bh * parts * n + at;
    float s = pt.j.S0 ? x[0] : 0.f;
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

// Parts of a sequence.  A launch takes as many turns as its blocks, one an
// SM, fill the SMs.  Counted in chunks: a block takes about half a chunk's time
// besides its own, a chunk of the pass that forms the state 0.35, and the two
// launches more about one (shares of an earlier step, whose chunks took a fifth
// longer; us on the GPU now, fp32, in one part and by this rule: B1 T20000 H4 d64
// 2008 and 98, B3 T1001 H5 d72 119 and 51, B1 T4096 H4 d256 1294 and 228, B1 T4096
// H16 d128 638 and 234).
Plan plan(long long blocks, int dk, int T) {
    const int C = dk > 128 ? 32 : 64, slots = kPlanSMs;
    const int chunks = (T + C - 1) / C;
    auto turns = [&](long long n) { return (double)((n + slots - 1) / slots); };
    Plan best{1, T};
    double least = turns(blocks) * (chunks + 0.5);
    for (int p = 2; p <= 32 && p <= chunks; ++p) {
        const int len = (chunks + p - 1) / p;
        const int parts = (chunks + len - 1) / len;
        const double t = turns(blocks * parts) * (len + 0.5) +
                         turns(blocks * (parts - 1)) * (0.35 * len + 0.5) + 1;
        if (t < 0.97 * least) {
            least = t;
            best = {parts, len * C};
        }
    }
    return best;
}

template <typename T, int DKP, bool STATE_ONLY>
cudaError_t launch_pass(PassParams& p, int jobs, long long bh,
                        cudaStream_t stream) {
    constexpr int bytes = Shape<DKP>::FLOATS * 4;
    const cudaError_t e = la::allow_smem<linattn_pass<T, DKP, STATE_ONLY>>(bytes);
    if (e != cudaSuccess) return e;
    const long long parts = p.plan.parts - (STATE_ONLY ? 1 : 0);
    long long n = 0;
    for (int i = 0; i <= kMaxJobs; ++i) {
        p.first[i] = (int)n;
        if (i < jobs) n += bh * parts * p.part[i].slices;
    }
    return launch_dependent(linattn_pass<T, DKP, STATE_ONLY>,
                            dim3((unsigned)n), kNT, stream, bytes, p);
}

Plan plan_of(const LinAttnArgs& a) {
    long long blocks = 0;
    for (int i = 0; i < a.jobs; ++i)
        blocks += (long long)a.B * a.H * la::slices_of(a.job[i]);
    return plan(blocks, la::widest_key(a), a.T);
}

// Floats of the part states of a job.
size_t part_floats(const LinAttnArgs& a, int job, const Plan& pl) {
    const LinAttnJob& j = a.job[job];
    return pl.parts > 1 ? (size_t)a.B * a.H * pl.parts * j.dk * j.dv : 0;
}

template <typename T, int DKP>
cudaError_t launch_passes(const LinAttnArgs& a, float* ws,
                          cudaStream_t stream) {
    const long long bh = (long long)a.B * a.H;
    PassParams p{};
    p.plan = plan_of(a);
    p.log_decay = a.log_decay;
    p.T = a.T, p.H = a.H;
    for (int i = 0; i < a.jobs; ++i) {
        p.part[i] = {a.job[i], ws, la::slices_of(a.job[i])};
        if (p.plan.parts > 1) ws += part_floats(a, i, p.plan);
    }
    if (p.plan.parts > 1) {
        cudaError_t e = launch_pass<T, DKP, true>(p, a.jobs, bh, stream);
        if (e == cudaSuccess)
            e = la::join_parts(p.part, a.jobs, p.plan, a.log_decay, bh, a.H,
                               stream);
        if (e != cudaSuccess) return e;
    }
    return launch_pass<T, DKP, false>(p, a.jobs, bh, stream);
}

template <typename T>
cudaError_t launch_all(const LinAttnArgs& a, float* ws, cudaStream_t stream) {
    const int dk = la::widest_key(a);
    return dk <= 64    ? launch_passes<T, 64>(a, ws, stream)
           : dk <= 128 ? launch_passes<T, 128>(a, ws, stream)
                       : launch_passes<T, 256>(a, ws, stream);
}

}  // namespace

cudaError_t la::join_parts(const Part* part, int jobs, const Plan& pl,
                           const float* log_decay, long long bh, int H,
                           cudaStream_t stream) {
    JoinParams p{};
    p.plan = pl;
    p.log_decay = log_decay;
    p.H = H;
    long long n = 0;
    for (int i = 0; i <= kMaxJobs; ++i) {
        p.first[i] = (int)n;
        if (i >= jobs) continue;
        p.part[i] = part[i];
        n += bh * ((part[i].j.dk * part[i].j.dv + kJoin - 1) / kJoin);
    }
    return launch_dependent(linattn_join, dim3((unsigned)n), kJoin, stream, 0,
                            p);
}

// By the sizes alone, whichever form the tensors' alignment allows.
size_t linattn_workspace_bytes(const LinAttnArgs& a) {
    size_t n = 0, tc = 0;
    for (int i = 0; i < a.jobs; ++i) {
        n += part_floats(a, i, plan_of(a));
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
// 8 dk dv bytes a head are all that matters here (256 sequences of 16 heads of
// 128 x 128: 81 us, 0.97 of HBM; few heads: the launch's own 2 us).
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
    // columns; the narrower where there are fewer heads than SMs (measured,
    // dk = dv = 128, us with tiles of 32 and of 128 columns: 16 heads 2.4 and
    // 3.3, 64 heads 4.1 and 5.4, 256 heads 9.3 and 8.4, 4096 heads 102 and 81)
    int cg = vec ? (heads >= 128 ? 5 : 3) : 5;
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
