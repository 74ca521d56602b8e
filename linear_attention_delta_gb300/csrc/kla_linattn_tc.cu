// Linear attention with a decay for each head on the tensor cores (tcgen05):
// bf16 inputs, q and k up to 128 wide, chunks of 128 tokens.
//
// A block owns 64 columns of the state of one (pass, sequence, head, part)
// and walks its chunks (S the state before a chunk, w = exp(log_decay)):
//   P  = Q K^T                         128 x 128   scores, fp32 in TMEM
//   P~ = P o w^(r - s), s <= r          in place    bf16, again in TMEM
//   O  = P~ V + diag(w^(r + e)) Q S    two accumulators, joined on the way out
//   U  = K^T diag(w^(n - e - s)) V     128 x 64
//   S <- w^n S + U                     fp32, in registers
// U does not depend on S, so the only chain from chunk to chunk is one
// multiply-add of the state, and everything else runs ahead of it.
//
// What is rounded to 16 bits: P~ and the copy of S that Q S reads (both are
// multiplied by 16-bit values and end in a 16-bit output; measured, the
// outputs are 1.4 times as far from the exact ones as those rounded once).
// The weighted V of U is split into three bf16 parts (24 bits), so that the
// state keeps the digits of fp32.
//
// Warps: 0 copies (TMA), 1 issues the products, 4-7 turn scores into P~
// (thread = row), 8-11 weight V and hold the state (thread = row of S), 12-15
// write the outputs (thread = row).  They hand over through mbarriers.
//
// In reverse the tiles lie in memory order all the same; r counts from the
// tile's last row, masks and weights are mirrored.
//
// A value of V that is not finite is taken out of the tile of P~ V, where it
// would meet the zeros of earlier rows, and what it makes of its own and the
// later rows (NaN) is put in when they are written.
//
// Every wait is bounded (2 s) and gives up when another warp has: the block
// then sets the fault word, lets its copies and products finish, frees TMEM
// and returns.
#include <atomic>

#include "kla_linattn.cuh"
#include "tc_primitives.cuh"

namespace kla {
namespace {

using la::kNV;
using la::Part;
using la::Plan;
using la::power;
using bf16 = __nv_bfloat16;

__device__ unsigned int g_fault_la = 0;

constexpr int kC = 128;          // tokens a chunk
constexpr int kThreads = 512;
constexpr int kBox = kC * 128;   // bytes of a TMA box: 128 rows of 64 bf16
constexpr int kMaxJobs = 3;

// Shared memory (bytes from a 1024-aligned base): the ring of stages (Q | K |
// V, in boxes of 64 columns; without Q in the pass that forms part states),
// the three parts of the weighted V, the bf16 copy of S, the weights.
template <int DK, bool STATE_ONLY>
struct Smem {
    static constexpr int HALVES = DK / 64;
    static constexpr int Q = 0;
    static constexpr int K = STATE_ONLY ? 0 : HALVES * kBox;
    static constexpr int V = K + HALVES * kBox;
    static constexpr int STAGE = V + kBox;
    static constexpr int NS = STATE_ONLY ? (DK == 64 ? 5 : 3)
                                         : (DK == 64 ? 3 : 2);
    static constexpr int VW = NS * STAGE;        // 3 boxes
    static constexpr int S = VW + 3 * kBox;      // DK rows of 128 bytes
    static constexpr int W = S + DK * 128;       // w^0 .. w^128
    static constexpr int BAD = W + 4 * 132;      // [2][4 warps][64]: see below
    static constexpr int FLAG = BAD + 2 * 4 * 64;   // [2][4 warps]
    static constexpr int BARS = FLAG + 2 * 4 * 4;
    static constexpr int NUM_BARS = 2 * NS + 11;
    static constexpr int MISC = BARS + 8 * NUM_BARS;   // abort, TMEM, issued
    static constexpr int BYTES = MISC + 16 + 1024;     // alignment
    static_assert(BYTES <= 232448, "shared memory");
    static_assert(BARS % 8 == 0 && W % 16 == 0, "alignment");
};

// mbarriers: a phase a chunk, or a phase every other chunk where there are two
template <int NS>
struct Bars {
    static constexpr int FULL = 0;               // NS: stage loaded
    static constexpr int EMPTY = NS;             // NS: stage read by all
    static constexpr int P_FULL = 2 * NS;        // 2: scores in TMEM
    static constexpr int P_READY = 2 * NS + 2;   // 2: P~ in TMEM
    static constexpr int V_READY = 2 * NS + 4;   // 2: weighted V in place, U
                                                 // of the chunk before read
    static constexpr int U_FULL = 2 * NS + 6;
    static constexpr int S_READY = 2 * NS + 7;   // copy of S in place
    static constexpr int S_FREE = 2 * NS + 8;    // Q S done
    static constexpr int O_FULL = 2 * NS + 9;
    static constexpr int O_FREE = 2 * NS + 10;   // outputs read
};

// TMEM columns
constexpr uint32_t kColP = 0;        // 2 x 128: scores, then P~ (64 of them)
constexpr uint32_t kColPV = 256;
constexpr uint32_t kColQS = 320;
constexpr uint32_t kColU = 384;
constexpr uint32_t kTmemCols = 512;

constexpr uint32_t kIdQK = tc::idesc_bf16(128, 128, false, false);
constexpr uint32_t kIdRow = tc::idesc_bf16(128, kNV, false, true);
constexpr uint32_t kIdU = tc::idesc_bf16(128, kNV, true, true);

struct Maps {
    CUtensorMap q[kMaxJobs], k[kMaxJobs], v[kMaxJobs];
};

struct TcParams {
    Part part[kMaxJobs];
    int first[kMaxJobs + 1];     // first block of each pass
    const float* log_decay;
    Plan plan;                   // the same for all passes
    int T, H;
    uint64_t limit_ns;
    bool selftest;               // copies nothing
};

__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
    return tc::sdesc_sw128(addr, 16, 1024);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t lbo) {
    return tc::sdesc_sw128(addr, lbo, 1024);
}

// As tc::mma_bf16 with A in TMEM (lane = row, two bf16 a column).
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem,
                                            uint64_t b_desc, uint32_t idesc,
                                            bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(
            d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

__device__ __forceinline__ void st_global_32(void* p, const uint32_t* u) {
    asm volatile(
        "st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
            reinterpret_cast<uint64_t>(p)),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]),
        "r"(u[6]), "r"(u[7])
        : "memory");
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Two floats less the two bf16 they were rounded to.
__device__ __forceinline__ float2 rest(float2 x, uint32_t b) {
    return make_float2(x.x - __uint_as_float(b << 16),
                       x.y - __uint_as_float(b & 0xffff0000u));
}

template <int DK, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 1)
linattn_tc(const __grid_constant__ Maps maps,
           const __grid_constant__ TcParams p) {
    using Sm = Smem<DK, STATE_ONLY>;
    using B = Bars<Sm::NS>;
    constexpr int NS = Sm::NS, HALVES = Sm::HALVES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = tc::smem_u32(sm);
    float* w = reinterpret_cast<float*>(sm + Sm::W);
    // for each of two chunks, output warp and column: the first row (counted
    // as r) whose V is not finite, 255: none
    uint8_t* bad = sm + Sm::BAD;
    volatile int* flag = reinterpret_cast<int*>(sm + Sm::FLAG);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sm::BARS);
    int* abort_flag = reinterpret_cast<int*>(sm + Sm::MISC);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Sm::MISC + 4);
    int* issued = reinterpret_cast<int*>(sm + Sm::MISC + 8);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int job = 0;
    while (job + 1 < kMaxJobs && (int)blockIdx.x >= p.first[job + 1]) ++job;
    const Part& pt = p.part[job];
    const int parts = STATE_ONLY ? p.plan.parts - 1 : p.plan.parts;
    int item = blockIdx.x - p.first[job];
    const int n0 = item % pt.slices * kNV;
    item /= pt.slices;
    const int part = item % parts;
    const size_t bh = item / parts;
    const int b = bh / p.H, h = bh % p.H;
    const bool rev = pt.j.reverse;
    const int e = rev ? 0 : 1;
    const float a = p.log_decay[h];
    const int first = part * p.plan.len;
    const int end = min(p.T, first + p.plan.len);
    const int nchunks = (end - first + kC - 1) / kC;

    if (warp == 0) {
        tc::tmem_alloc(tmem_slot, kTmemCols);
        tc::tmem_relinquish();
    }
    if (tid == 32) {
        for (int i = 0; i < Sm::NUM_BARS; ++i) {
            // the groups of four warps arrive once a warp
            const bool group = i == B::P_READY || i == B::P_READY + 1 ||
                               i == B::V_READY || i == B::V_READY + 1 ||
                               i == B::S_READY || i == B::O_FREE;
            tc::mbar_init(&bars[i], group ? 4 : 1);
        }
        tc::fence_mbar_init();
        *abort_flag = 0;
        *issued = 0;
    }
    if (tid >= 64 && tid < 64 + kC + 1) w[tid - 64] = power(a, tid - 64);
    for (int i = tid; i < 2 * 4 * 64; i += kThreads) bad[i] = 255;
    if (tid < 8) flag[tid] = 0;
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    auto wait = [&](int bar, int phase) {
        const bool ok = tc::mbar_wait_or_abort(&bars[bar], phase & 1,
                                               abort_flag, p.limit_ns);
        if (!ok) *reinterpret_cast<volatile int*>(abort_flag) = 1;
        return ok;
    };
    auto wait_warp = [&](int bar, int phase) {
        return __all_sync(~0u, wait(bar, phase));
    };
    // the first token (in memory) of chunk c's tile; may be negative in
    // reverse
    auto tile_token = [&](int c) {
        const int r0 = first + c * kC;
        return rev ? p.T - r0 - kC : r0;
    };
    auto rows_of = [&](int c) { return min(kC, end - (first + c * kC)); };

    int last_bar = -1, last_phase = 0;   // the issuer's last commit
    float S[kNV];                        // the state group's

    if (tid == 0 && !p.selftest) {
        // ------------------------------------------------------ copies
        tc::prefetch_tmap(&maps.k[job]);
        tc::prefetch_tmap(&maps.v[job]);
        if (!STATE_ONLY) tc::prefetch_tmap(&maps.q[job]);
        for (int c = 0; c < nchunks; ++c) {
            const int s = c % NS;
            if (c >= NS && !wait(B::EMPTY + s, c / NS - 1)) break;
            uint8_t* st = sm + s * Sm::STAGE;
            uint64_t* full = &bars[B::FULL + s];
            const int t = tile_token(c);
            tc::mbar_arrive_expect_tx(full, Sm::STAGE);
#pragma unroll
            for (int i = 0; i < HALVES; ++i)
                tc::tma_load_4d(st + Sm::K + i * kBox, &maps.k[job], full,
                                64 * i, h, t, b);
            if (!STATE_ONLY)
#pragma unroll
                for (int i = 0; i < HALVES; ++i)
                    tc::tma_load_4d(st + Sm::Q + i * kBox, &maps.q[job], full,
                                    64 * i, h, t, b);
            tc::tma_load_4d(st + Sm::V, &maps.v[job], full, n0, h, t, b);
            *reinterpret_cast<volatile int*>(issued) = c + 1;
        }
    } else if (tid == 32) {
        // ---------------------------------------------------- products
        auto scores = [&](int c) {
            const uint32_t st = sbase + c % NS * Sm::STAGE;
            if (!wait(B::FULL + c % NS, c / NS)) return false;
            tc::tc_fence_after();
            // P~ V of chunk c - 2, which read this buffer, is ahead of this
            // product in the queue
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks) {
                const uint32_t off = (ks >> 2) * kBox + (ks & 3) * 32;
                tc::mma_bf16(tmem + kColP + 128 * (c & 1),
                             desc_k(st + Sm::Q + off),
                             desc_k(st + Sm::K + off), kIdQK, ks > 0);
            }
            tc::mma_commit(&bars[B::P_FULL + (c & 1)]);
            last_bar = B::P_FULL + (c & 1), last_phase = c >> 1;
            return true;
        };
        int scored = 0;      // chunks whose scores are issued
        for (int c = 0; c < nchunks; ++c) {
            const uint32_t st = sbase + c % NS * Sm::STAGE;
            if (!STATE_ONLY && scored == c) {
                if (!scores(c)) break;
                scored = c + 1;
            }
            if (!wait(B::V_READY + (c & 1), c >> 1)) break;
            tc::tc_fence_after();
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int ks = 0; ks < kC / 16; ++ks)
                    tc::mma_bf16(
                        tmem + kColU,
                        // 64 wide: rows 64 .. 127 of U repeat, unread
                        desc_mn(st + Sm::K + ks * 2048, DK == 128 ? kBox : 0),
                        desc_mn(sbase + Sm::VW + i * kBox + ks * 2048, 0),
                        kIdU, i + ks > 0);
            tc::mma_commit(&bars[B::U_FULL]);
            last_bar = B::U_FULL, last_phase = c;
            const bool again = c + NS < nchunks;   // the stage is loaded again
            if (STATE_ONLY) {
                if (again) tc::mma_commit(&bars[B::EMPTY + c % NS]);
                continue;
            }
            if (!wait(B::S_READY, c)) break;
            if (c > 0 && !wait(B::O_FREE, c - 1)) break;
            tc::tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks)
                tc::mma_bf16(tmem + kColQS,
                             desc_k(st + Sm::Q + (ks >> 2) * kBox +
                                    (ks & 3) * 32),
                             desc_mn(sbase + Sm::S + ks * 2048, 0), kIdRow,
                             ks > 0);
            tc::mma_commit(&bars[B::S_FREE]);
            last_bar = B::S_FREE, last_phase = c;
            // the next scores, when their inputs are here: they are in the
            // works while this chunk's become P~
            if (scored == c + 1 && scored < nchunks &&
                mbar_test(&bars[B::FULL + scored % NS], scored / NS & 1)) {
                if (!scores(scored)) break;
                ++scored;
            }
            if (!wait(B::P_READY + (c & 1), c >> 1)) break;
            tc::tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < kC / 16; ++ks)
                mma_bf16_ts(tmem + kColPV,
                            tmem + kColP + 128 * (c & 1) + 8 * ks,
                            desc_mn(st + Sm::V + ks * 2048, 0), kIdRow,
                            ks > 0);
            tc::mma_commit(&bars[B::O_FULL]);
            last_bar = B::O_FULL, last_phase = c;
            if (again) tc::mma_commit(&bars[B::EMPTY + c % NS]);
        }
    } else if (warp >= 4 && warp < 8 && !STATE_ONLY) {
        // ------------------------------------------- scores to P~ (row i)
        const int q = warp - 4, i = 32 * q + lane;
        for (int c = 0; c < nchunks; ++c) {
            if (!wait_warp(B::P_FULL + (c & 1), c >> 1)) break;
            tc::tc_fence_after();
            const uint32_t col =
                tmem + ((uint32_t)(32 * q) << 16) + kColP + 128 * (c & 1);
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {      // 32 columns
                float u[16];
                uint32_t* pk = reinterpret_cast<uint32_t*>(u);
                if (rev ? j < q : j > q) {
#pragma unroll
                    for (int n = 0; n < 16; ++n) pk[n] = 0;
                } else {
                    float x[32];
                    tc::tmem_ld32(col + 32 * j, x);
                    tc::tmem_ld_wait();
                    if (j == q) {
                        // the diagonal: what is masked is not multiplied by 0
#pragma unroll
                        for (int n = 0; n < 32; ++n) {
                            const int d = rev ? n - lane : lane - n;
                            x[n] = d >= 0 ? x[n] * w[d < 0 ? 0 : d] : 0.f;
                        }
                    } else {
                        // w^(r - s) as a factor of the row and one of the
                        // column, neither exponent negative
                        const float f =
                            w[rev ? 32 * j - i : i - 32 * j - 31];
#pragma unroll
                        for (int n = 0; n < 32; n += 4) {
                            const float4 g = *reinterpret_cast<const float4*>(
                                &w[rev ? n : 28 - n]);
                            x[n] *= f * (rev ? g.x : g.w);
                            x[n + 1] *= f * (rev ? g.y : g.z);
                            x[n + 2] *= f * (rev ? g.z : g.y);
                            x[n + 3] *= f * (rev ? g.w : g.x);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 16; ++n)
                        pk[n] = tc::pack_bf16x2(x[2 * n], x[2 * n + 1]);
                }
                tc::tmem_st16(col + 16 * j, u);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[B::P_READY + (c & 1)]);
        }
    } else if (warp >= 8 && warp < 12) {
        // -------------------------------- weighted V, and the state (row d)
        const int gt = tid - 256, d = gt;
        const bool mine = d < pt.j.dk;
        const size_t row = (size_t)d * pt.j.s_r;
        const size_t sn = (size_t)pt.j.dk * pt.j.dv;
#pragma unroll
        for (int n = 0; n < kNV; ++n) {
            S[n] = 0.f;
            if (mine && n0 + n < pt.j.dv) {
                const size_t at = row + (size_t)(n0 + n) * pt.j.s_c;
                if (STATE_ONLY) {
                    if (part == 0 && pt.j.S0)
                        pt.ws[bh * p.plan.parts * sn + at] =
                            pt.j.S0[bh * sn + at];
                } else {
                    S[n] = la::state_before(pt, p.plan, part, bh, at, a);
                }
            }
        }
        auto store_S = [&]() {     // the bf16 copy that Q S reads
            if (d < DK) {
                uint8_t* dst = sm + Sm::S + d * 128;
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    uint4 x;
                    x.x = tc::pack_bf16x2(S[8 * n], S[8 * n + 1]);
                    x.y = tc::pack_bf16x2(S[8 * n + 2], S[8 * n + 3]);
                    x.z = tc::pack_bf16x2(S[8 * n + 4], S[8 * n + 5]);
                    x.w = tc::pack_bf16x2(S[8 * n + 6], S[8 * n + 7]);
                    *reinterpret_cast<uint4*>(dst + ((n ^ (d & 7)) << 4)) = x;
                }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[B::S_READY]);
        };
        if (!STATE_ONLY) store_S();
        const uint32_t ucol =
            tmem + ((uint32_t)(32 * (warp - 8)) << 16) + kColU;
        for (int c = 0; c < nchunks; ++c) {
            const int n = rows_of(c);
            if (!wait_warp(B::FULL + c % NS, c / NS)) break;
            uint8_t* v = sm + c % NS * Sm::STAGE + Sm::V;
            uint32_t seen = 0;
#pragma unroll 2
            for (int i = 0; i < 8; ++i) {      // 8 of 1024 16-byte pieces
                const int at = (gt + 128 * i) * 16, j = (gt >> 3) + 16 * i;
                // rows beyond the sequence are zero: their weight is any
                const float f = w[max(0, rev ? n - kC + 1 + j : n - 1 - j)];
                const uint4 x = *reinterpret_cast<const uint4*>(v + at);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                uint32_t o[3][4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    asm("fma.rn.bf16x2 %0, %1, %2, %0;"
                        : "+r"(seen) : "r"(xs[m]), "r"(0u));
                    float2 y = make_float2(
                        __uint_as_float(xs[m] << 16) * f,
                        __uint_as_float(xs[m] & 0xffff0000u) * f);
                    o[0][m] = tc::pack_bf16x2(y.x, y.y);
                    y = rest(y, o[0][m]);
                    o[1][m] = tc::pack_bf16x2(y.x, y.y);
                    y = rest(y, o[1][m]);
                    o[2][m] = tc::pack_bf16x2(y.x, y.y);
                }
#pragma unroll
                for (int m = 0; m < 3; ++m)
                    *reinterpret_cast<uint4*>(sm + Sm::VW + m * kBox + at) =
                        make_uint4(o[m][0], o[m][1], o[m][2], o[m][3]);
            }
            bool ok = true;
            if (!STATE_ONLY && (seen & 0x7fff7fffu)) {
                // the outputs of chunk c - 2 have been read (those of c - 3
                // had been before U of c - 1 was formed)
                ok = c < 2 || wait(B::O_FREE, c - 2);
                const int slot = c & 1;
                for (int i = 0; i < 8 && ok; ++i) {
                    const int piece = gt + 128 * i, j = piece >> 3;
                    uint16_t* x =
                        reinterpret_cast<uint16_t*>(v + piece * 16);
                    for (int m = 0; m < 8; ++m) {
                        if ((x[m] & 0x7f80) != 0x7f80) continue;
                        x[m] = 0;
                        const int col = ((piece & 7) ^ (j & 7)) * 8 + m;
                        const int r = rev ? kC - 1 - j : j;
                        for (int o = 0; o < 4; ++o) {
                            // bytes: a compare-and-swap on their word
                            uint32_t* word = reinterpret_cast<uint32_t*>(
                                bad + (slot * 4 + o) * 64 + (col & ~3));
                            const int sh = (col & 3) * 8;
                            uint32_t old =
                                *reinterpret_cast<volatile uint32_t*>(word);
                            uint32_t was;
                            do {
                                was = old;
                                if ((int)(was >> sh & 255) <= r) break;
                                old = atomicCAS(word, was,
                                                (was & ~(255u << sh)) |
                                                    (uint32_t)r << sh);
                            } while (old != was);
                            flag[slot * 4 + o] = 1;
                        }
                    }
                }
            }
            tc::fence_proxy_async_smem();
            if (!__all_sync(~0u, ok)) break;
            if (lane == 0) tc::mbar_arrive(&bars[B::V_READY + (c & 1)]);
            if (!wait_warp(B::U_FULL, c)) break;
            tc::tc_fence_after();
            // w^n S as S + (w^n - 1) S: a decay close to 1 keeps its digits
            const float grow = expm1f(a * (float)n);
#pragma unroll
            for (int m = 0; m < kNV; m += 32) {
                float u[32];
                tc::tmem_ld32(ucol + m, u);
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    S[m + k] = fmaf(grow, S[m + k], S[m + k]) + u[k];
            }
            tc::tc_fence_before();     // U may be written again
            if (!STATE_ONLY && c + 1 < nchunks) {
                if (!wait_warp(B::S_FREE, c)) break;
                store_S();
            }
        }
        const bool done = *reinterpret_cast<volatile int*>(abort_flag) == 0;
        float* dst = STATE_ONLY
            ? pt.ws + (bh * p.plan.parts + part + 1) * sn
            : part + 1 == parts && pt.j.ST ? pt.j.ST + bh * sn : nullptr;
        if (done && mine && dst) {
#pragma unroll
            for (int n = 0; n < kNV; ++n)
                if (n0 + n < pt.j.dv)
                    dst[row + (size_t)(n0 + n) * pt.j.s_c] = S[n];
        }
    } else if (warp >= 12 && !STATE_ONLY) {
        // ------------------------------------------------ outputs (row i)
        const int q = warp - 12, i = 32 * q + lane, r = rev ? kC - 1 - i : i;
        const float f = w[r + e];
        const int width = min(kNV, pt.j.dv - n0);
        const size_t dv = pt.j.dv;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
        bf16* out = static_cast<bf16*>(pt.j.o);
        const uintptr_t align = reinterpret_cast<uintptr_t>(out) | dv * 2;
        for (int c = 0; c < nchunks; ++c) {
            // (the flags are set before V_READY; its phase after the next
            // does not begin before these outputs are read)
            if (!wait_warp(B::O_FULL, c) ||
                !wait_warp(B::V_READY + (c & 1), c >> 1))
                break;
            tc::tc_fence_after();
            uint32_t pk[kNV / 2];
            const bool any = flag[(c & 1) * 4 + q] != 0;
            uint8_t* own = bad + ((c & 1) * 4 + q) * 64;
#pragma unroll
            for (int m = 0; m < kNV; m += 16) {
                float x[16], y[16];
                tc::tmem_ld16(lanes + kColPV + m, x);
                tc::tmem_ld16(lanes + kColQS + m, y);
                tc::tmem_ld_wait();
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                    x[n] = fmaf(f, y[n], x[n]);
                    if (any && r >= own[m + n])
                        x[n] = __uint_as_float(0x7fc00000u);
                }
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    pk[m / 2 + n] = tc::pack_bf16x2(x[2 * n], x[2 * n + 1]);
            }
            tc::tc_fence_before();
            __syncwarp();
            if (any) {
                own[lane] = own[lane + 32] = 255;
                if (lane == 0) flag[(c & 1) * 4 + q] = 0;
                __syncwarp();
            }
            if (lane == 0) tc::mbar_arrive(&bars[B::O_FREE]);
            if (r >= rows_of(c)) continue;
            const size_t t = (size_t)(tile_token(c) + i);
            bf16* dst = out + (((size_t)b * p.T + t) * p.H + h) * dv + n0;
            if (align % 32 == 0) {
#pragma unroll
                for (int n = 0; n < kNV; n += 16)
                    if (n < width) st_global_32(dst + n, pk + n / 2);
            } else if (align % 16 == 0) {
#pragma unroll
                for (int n = 0; n < kNV; n += 8)
                    if (n < width)
                        *reinterpret_cast<uint4*>(dst + n) =
                            make_uint4(pk[n / 2], pk[n / 2 + 1],
                                       pk[n / 2 + 2], pk[n / 2 + 3]);
            } else {
#pragma unroll
                for (int n = 0; n < kNV; ++n)
                    if (n < width)
                        reinterpret_cast<uint16_t*>(dst)[n] =
                            (uint16_t)(n & 1 ? pk[n / 2] >> 16 : pk[n / 2]);
            }
        }
    }

    __syncwarp();
    __syncthreads();
    if (*reinterpret_cast<volatile int*>(abort_flag)) {
        constexpr uint64_t kDrain = 100000000ull;
        if (tid == 32 && last_bar >= 0)
            tc::mbar_wait(&bars[last_bar], last_phase & 1, kDrain);
        if (tid == 0) {
            atomicOr(&g_fault_la, 1u);
            const int n = *reinterpret_cast<volatile int*>(issued);
            for (int c = n - NS < 0 ? 0 : n - NS; c < n; ++c)
                tc::mbar_wait(&bars[B::FULL + c % NS], (c / NS) & 1, kDrain);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------- host side

// A stride that a tensor map can hold: whole 16-byte units, less than 2^40
// bytes; 0 (a repeated axis) has no map.  The stride of an axis of one is
// never used.
bool map_stride(long long st, int n) {
    return n == 1 || (st > 0 && st % 8 == 0 && st < (1ll << 39));
}
bool map_ok(const Heads& x, int B, int T, int H) {
    return (reinterpret_cast<uintptr_t>(x.p) & 15) == 0 &&
           map_stride(x.sb, B) && map_stride(x.st, T) && map_stride(x.sh, H);
}

// [B, T, H, d] bf16, boxes of 64 columns x 1 head x 128 tokens x 1 sequence,
// zeros out of range.
bool make_heads_map(CUtensorMap* m, const Heads& x, int B, int T, int H,
                    int d) {
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T,
                          (cuuint64_t)B};
    cuuint64_t strides[3] = {(cuuint64_t)(H == 1 ? 16 : x.sh * 2),
                             (cuuint64_t)(T == 1 ? 16 : x.st * 2),
                             (cuuint64_t)(B == 1 ? 16 : x.sb * 2)};
    cuuint32_t box[4] = {64, 1, kC, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return tile_map_encoder()(
               m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void*>(x.p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, bool STATE_ONLY>
cudaError_t launch(const Maps& maps, TcParams& p, int jobs, long long bh,
                   cudaStream_t stream) {
    using Sm = Smem<DK, STATE_ONLY>;
    auto kern = linattn_tc<DK, STATE_ONLY>;
    // the shared-memory opt-in, once a device
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!bit || !(done.load() & bit)) {
        e = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sm::BYTES);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    const long long parts = p.plan.parts - (STATE_ONLY ? 1 : 0);
    long long n = 0;
    for (int i = 0; i <= kMaxJobs; ++i) {
        p.first[i] = (int)n;
        if (i < jobs) n += bh * parts * p.part[i].slices;
    }
    kern<<<(unsigned)n, kThreads, Sm::BYTES, stream>>>(maps, p);
    return cudaGetLastError();
}

int widest_key(const LinAttnArgs& a) {
    int n = 0;
    for (int i = 0; i < a.jobs; ++i) n = a.job[i].dk > n ? a.job[i].dk : n;
    return n;
}

}  // namespace

bool linattn_tc_sizes(const LinAttnArgs& a) {
    return a.dtype == KLA_BF16 && widest_key(a) <= 128;
}

bool linattn_tc_eligible(const LinAttnArgs& a) {
    if (!linattn_tc_sizes(a) || !get_encoder()) return false;
    for (int i = 0; i < a.jobs; ++i) {
        const LinAttnJob& j = a.job[i];
        if (!map_ok(j.q, a.B, a.T, a.H) || !map_ok(j.k, a.B, a.T, a.H) ||
            !map_ok(j.v, a.B, a.T, a.H))
            return false;
    }
    return true;
}

la::Plan linattn_tc_plan(const LinAttnArgs& a) {
    constexpr int kSMs = 152, kLeast = 512;
    long long blocks = 0;
    for (int i = 0; i < a.jobs; ++i)
        blocks += (long long)a.B * a.H * la::slices_of(a.job[i]);
    long long parts = kSMs / blocks;
    if (parts > a.T / kLeast) parts = a.T / kLeast;
    if (parts < 2) return {1, a.T};
    int len = (int)((a.T + parts - 1) / parts);
    len = (len + kC - 1) / kC * kC;
    return {(a.T + len - 1) / len, len};
}

cudaError_t launch_linattn_tc(const LinAttnArgs& a, float* ws,
                              cudaStream_t stream) {
    Maps maps{};
    TcParams p{};
    const long long bh = (long long)a.B * a.H;
    p.log_decay = a.log_decay;
    p.plan = linattn_tc_plan(a);
    p.T = a.T, p.H = a.H;
    p.limit_ns = 2000000000ull;
    for (int i = 0; i < a.jobs; ++i) {
        const LinAttnJob& j = a.job[i];
        if (!make_heads_map(&maps.q[i], j.q, a.B, a.T, a.H, j.dk) ||
            !make_heads_map(&maps.k[i], j.k, a.B, a.T, a.H, j.dk) ||
            !make_heads_map(&maps.v[i], j.v, a.B, a.T, a.H, j.dv))
            return cudaErrorInvalidValue;
        p.part[i] = {j, ws, la::slices_of(j)};
        if (p.plan.parts > 1) ws += (size_t)bh * p.plan.parts * j.dk * j.dv;
    }
    const bool narrow = widest_key(a) <= 64;
    if (p.plan.parts > 1) {
        const cudaError_t e =
            narrow ? launch<64, true>(maps, p, a.jobs, bh, stream)
                   : launch<128, true>(maps, p, a.jobs, bh, stream);
        if (e != cudaSuccess) return e;
    }
    return narrow ? launch<64, false>(maps, p, a.jobs, bh, stream)
                  : launch<128, false>(maps, p, a.jobs, bh, stream);
}

cudaError_t launch_linattn_selftest(cudaStream_t stream) {
    Maps maps{};
    TcParams p{};
    void* word = nullptr;          // a device address, for the decay
    const cudaError_t e = cudaGetSymbolAddress(&word, g_fault_la);
    if (e != cudaSuccess) return e;
    p.log_decay = static_cast<const float*>(word);
    p.part[0].j.dk = p.part[0].j.dv = kNV;
    p.part[0].j.s_r = kNV, p.part[0].j.s_c = 1;
    p.part[0].slices = 1;
    p.plan = {1, kC};
    p.T = kC, p.H = 1;
    p.limit_ns = 1000000ull;
    p.selftest = true;
    return launch<64, false>(maps, p, 1, 1, stream);
}

cudaError_t read_and_clear_fault_la(unsigned int* word) {
    const cudaError_t e =
        cudaMemcpyFromSymbol(word, g_fault_la, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_fault_la, &zero, sizeof(unsigned int));
}

}  // namespace kla
