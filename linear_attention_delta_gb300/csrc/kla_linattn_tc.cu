// Linear attention with a decay for each head on the tensor cores (tcgen05):
// bf16 inputs, q and k up to 128 wide, chunks of 128 tokens.
//
// A block owns 64 columns of the state of one (pass, sequence, head, part)
// and walks its chunks (S the state before a chunk, w = exp(log_decay)):
//   P  = Q K^T                         128 x 128   scores, fp32 in TMEM
//   P~ = P o w^(r - s), s <= r                      bf16, again in TMEM
//   O  = diag(w^(r + e)) Q S + P~ V    128 x 64    one accumulator
//   U  = K^T diag(w^(n - e - s)) V     128 x 64
//   S <- w^n S + U                     fp32, in registers
// For Q S and P~ V to share an accumulator, w^(r - 63) is taken out of a row
// and multiplied in as it is written: P~ has the factor w^(63 - s) of its
// column, and S that of w^(63 + e).  These factors stay within e^48, which
// leaves bf16 its digits for scores up to 4e17 and states down to 1e-17;
// stronger decays (64 |log_decay| > 48: a memory of a token or two) have their
// rows of Q S scaled in TMEM instead, and every score its own factor (if all
// heads are such: 69 us where the others take 66 at B4 T4096 H16 d128, 61 and 56
// with d64, 256 and 217 at B8 T8192 H32 d64).
// U does not depend on S, so the only chain from chunk to chunk is one
// multiply-add of the state, and everything else runs ahead of it.
//
// What is rounded to 16 bits: P~ and the copy of S that Q S reads (both are
// multiplied by 16-bit values and end in a 16-bit output; measured, the
// outputs are 1.4 times as far from the exact ones as those rounded once).
// The weighted V of U is split into three bf16 parts (24 bits), so that the
// state keeps the digits of fp32.
//
// Warps: 0-7 hold the state (thread = row of S and half of its columns), 8-15
// weight V, 16-23 turn scores into P~ (thread = row and half of the columns),
// 24-27 write the outputs (thread = row), 28 issues the products, 29 the
// copies (TMA).  They hand over through mbarriers.
//
// What bounds it, at B4 T4096 H16 d128 (66 us on the GPU, as all times here
// unless they are said to be of an earlier step; HBM would take 40): a chunk
// takes a block 2.0 us, about 4100 cycles, in which 368 KB pass through shared
// memory (2900 cycles) and some 10000 warp instructions are issued.  Captured at
// B4 T2048 H16 d128 (37 us) the SMs at work use 58 % of their issue slots, and
// the tensor cores are busy in 42 % of the cycles.  At an earlier step, at 72 us,
// the hand-overs and products without the element-wise work took 59 us, the
// hand-overs alone 44.  Hence many warps with few registers, short loops, and
// weights in registers.  Measured and left out: weighted V by halves 65 us (but
// 57.5 for 56 with d64), scores twice buffered with one accumulator of outputs
// and P~ in the scores' place 69 (57.6 with d64); at earlier steps, at 72 to 80
// us, 18 larger warps 87, a second issuing thread 81, scores twice buffered with
// separate products for the parts of V 78.
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
#include <type_traits>

#include "f32x2.cuh"
#include "kla_linattn.cuh"
#include "tc_primitives.cuh"

namespace kla {
namespace {

using la::kMaxJobs;
using la::kNV;
using la::Part;
using la::Plan;
using la::widest_key;
using bf16 = __nv_bfloat16;

__device__ unsigned int g_fault_la = 0;

// w^n of w = exp(a), out of line: the kernel's loops have to stay short for
// the instruction caches, which hold the code of six kinds of warps.
__device__ __noinline__ float power(float a, int n) { return la::power(a, n); }

constexpr int kC = 128;          // tokens a chunk
constexpr int kThreads = 960;    // 64 registers each
constexpr int kIssuer = 28, kCopier = 29;   // warps
constexpr int kBox = kC * 128;   // bytes of a TMA box: 128 rows of 64 bf16
constexpr int kLdS = kNV + 1;    // row of the state's tile in shared memory

// Shared memory (bytes from a 1024-aligned base): the rings of Q, K and V
// tiles (boxes of 64 columns; no Q in the pass that forms part states), the
// three parts of the weighted V, the bf16 copy of S.
template <int DK, bool STATE_ONLY>
struct Smem {
    static constexpr int HALVES = DK / 64;
    static constexpr int NS = DK == 64 ? 3 : 2;
    static constexpr int NVW = STATE_ONLY ? 2 : 1;   // weighted tiles
    static constexpr int TILE = HALVES * kBox;   // of Q or K
    static constexpr int Q = 0;
    static constexpr int K = Q + (STATE_ONLY ? 0 : NS * TILE);
    static constexpr int V = K + NS * TILE;
    static constexpr int VW = V + NS * kBox;     // NVW x 3 boxes
    static constexpr int S = VW + NVW * 3 * kBox;   // DK rows of 128 bytes
    static constexpr int BAD = S + DK * 128;     // [2][4 warps][64]: see below
    static constexpr int FLAG = BAD + 2 * 4 * 64;   // [2][4 warps]
    static constexpr int DONE = FLAG + 2 * 4 * 4;   // [4 warps]
    static constexpr int BARS = DONE + 4 * 4;
    static constexpr int NUM_BARS = 5 * NS + 15;
    static constexpr int MISC = BARS + 8 * NUM_BARS;   // abort, TMEM, issued
    static constexpr int BYTES = MISC + 16 + 1024;     // alignment
    static_assert(BYTES <= 232448, "shared memory");
    static_assert(BARS % 8 == 0, "alignment");
};

// mbarriers, a phase a chunk (of a ring: a phase a turn).  A wait tells a
// phase from the one before or after it only, so none may complete two phases
// ahead of one that waits; where nothing else rules that out there are two
// barriers, for even and odd chunks.
template <int NS>
struct Bars {
    static constexpr int FULL = 0;               // NS: Q and K loaded
    static constexpr int FULL_V = NS;            // NS
    static constexpr int EMPTY_Q = 2 * NS;       // NS: read by all
    static constexpr int EMPTY_K = 3 * NS;       // NS
    static constexpr int EMPTY_V = 4 * NS;       // NS
    static constexpr int SC_FULL = 5 * NS;       // scores in TMEM
    static constexpr int SC_FREE = 5 * NS + 1;   // read
    static constexpr int P_READY = 5 * NS + 2;   // P~ in TMEM
    static constexpr int V_READY = 5 * NS + 3;   // 2: weighted V in place
    static constexpr int U_FULL = 5 * NS + 5;    // 2: U in TMEM (V's parts read)
    static constexpr int U_FREE = 5 * NS + 7;    // 2: read
    static constexpr int S_READY = 5 * NS + 9;   // copy of S in place
    static constexpr int S_FREE = 5 * NS + 10;   // Q S done
    static constexpr int O_FULL = 5 * NS + 11;   // 2: outputs in TMEM (P~ read)
    static constexpr int O_FREE = 5 * NS + 13;   // 2: read
};

// TMEM columns: all 512
constexpr uint32_t kColSC = 0;       // 128: scores
constexpr uint32_t kColP = 128;      // 64: P~, two bf16 a column
constexpr uint32_t kColO = 192;      // 2 x 64: outputs of even and odd chunks
constexpr uint32_t kColU = 320;      // 3 x 64: U from each part of V (two of
                                     // them, from 128 on, where only the
                                     // state is formed)
constexpr uint32_t kTmemCols = 512;

constexpr uint32_t kIdQK = tc::idesc_bf16(128, 128, false, false);
constexpr uint32_t kIdRow = tc::idesc_bf16(128, kNV, false, true);
// the parts of V side by side: K is read once for all three (three products
// of 64 columns are bound by reading K from shared memory)
constexpr uint32_t kIdU = tc::idesc_bf16(128, 3 * kNV, true, true);

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

// 32 lanes x 8 consecutive 32-bit columns per warp.
__device__ __forceinline__ void tmem_st8(uint32_t taddr,
                                         const uint32_t (&u)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]),
        "r"(u[6]), "r"(u[7])
        : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// The slow half of wait_phase: false, with *abort set, when `limit_ns` have
// passed or another warp has given up.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity,
                                       volatile int* abort,
                                       uint64_t limit_ns) {
    uint64_t t0 = 0;
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (tc::mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        const uint64_t t = tc::globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > limit_ns) *abort = 1;
    }
}

// Waits for the phase with the given parity; false when it gave up.  (The
// clock is slow to read: not before some turns.)
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity,
                                           volatile int* abort,
                                           uint64_t limit_ns) {
    const uint32_t at = tc::smem_u32(bar);
    if (tc::mbar_try_wait(at, parity)) return true;
    return wait_long(at, parity, abort, limit_ns);
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

// The upper halves of two floats, as two bf16: their first 8 bits.  What is
// left has the other 16, so that three parts hold a float whole.
__device__ __forceinline__ uint32_t upper(float2 x) {
    return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}
__device__ __forceinline__ float2 rest(float2 x) {
    return fma2(make_float2(
                    __uint_as_float(__float_as_uint(x.x) & 0xffff0000u),
                    __uint_as_float(__float_as_uint(x.y) & 0xffff0000u)),
                both(-1.f), x);
}

// Zeros in place of the values of this thread's pieces of a V tile that are
// not finite, and for each output warp their columns' first such row in `bad`.
__device__ __noinline__ void take_out(uint8_t* v, uint8_t* bad,
                                      volatile int* flag, volatile int* done,
                                      int c, int gt, bool rev,
                                      volatile int* abort,
                                      uint64_t limit_ns) {
    // the output warps are done with what chunk c - 2 left there
    const uint64_t t0 = tc::globaltimer_ns();
    for (int o = 0; o < 4; ++o)
        while (done[o] < c - 1) {
            if (tc::globaltimer_ns() - t0 > limit_ns) *abort = 1;
            if (*abort) return;
        }
    __threadfence_block();
    for (int m = 0; m < 4; ++m) {
        const int piece = gt + 256 * m, j = piece >> 3;
        uint16_t* x = reinterpret_cast<uint16_t*>(v + piece * 16);
        for (int k = 0; k < 8; ++k) {
            if ((x[k] & 0x7f80) != 0x7f80) continue;
            x[k] = 0;
            const int col = ((piece & 7) ^ (j & 7)) * 8 + k;
            const int r = rev ? kC - 1 - j : j;
            for (int o = 0; o < 4; ++o) {
                // bytes: a compare-and-swap on their word
                uint32_t* word =
                    reinterpret_cast<uint32_t*>(bad + o * kNV + (col & ~3));
                const int sh = (col & 3) * 8;
                uint32_t old = *reinterpret_cast<volatile uint32_t*>(word);
                uint32_t was;
                do {
                    was = old;
                    if ((int)(was >> sh & 255) <= r) break;
                    old = atomicCAS(word, was, (was & ~(255u << sh)) |
                                                   (uint32_t)r << sh);
                } while (old != was);
                flag[o] = 1;
            }
        }
    }
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
    // for each of two chunks, output warp and column: the first row (counted
    // as r) whose V is not finite, 255: none
    uint8_t* bad = sm + Sm::BAD;
    volatile int* flag = reinterpret_cast<int*>(sm + Sm::FLAG);
    // chunks whose outputs each output warp has read
    volatile int* done = reinterpret_cast<int*>(sm + Sm::DONE);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sm::BARS);
    volatile int* abort = reinterpret_cast<int*>(sm + Sm::MISC);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Sm::MISC + 4);
    int* issued = reinterpret_cast<int*>(sm + Sm::MISC + 8);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(~0u, tid >> 5, 0);   // uniform
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
    // (with parts the join came before, which itself waited: what is not of the
    // workspace is there)
    if (STATE_ONLY || p.plan.parts == 1) await_grid_before();
    const float a = p.log_decay[h];
    const int first = part * p.plan.len;
    const int end = first + min(p.T - first, p.plan.len);
    const int nchunks = (end - first + kC - 1) / kC;

    if (warp == 0) {
        tc::tmem_alloc(tmem_slot, kTmemCols);
        tc::tmem_relinquish();
    }
    if (tid == 32) {
        for (int i = 0; i < Sm::NUM_BARS; ++i) {
            // groups arrive once a warp; O_FULL by the products' end and by
            // the thread that issued them
            const int count =
                i == B::SC_FREE || i == B::P_READY || i == B::V_READY ||
                        i == B::V_READY + 1 || i == B::U_FREE ||
                        i == B::U_FREE + 1 || i == B::S_READY
                    ? 8
                : i == B::O_FREE || i == B::O_FREE + 1 ? 4
                : i == B::O_FULL || i == B::O_FULL + 1 ? 2 : 1;
            tc::mbar_init(&bars[i], count);
        }
        tc::fence_mbar_init();
        *abort = 0;
        *issued = 0;
    }
    const bool gentle = fabsf(a) * 64.f <= 48.f;
    for (int i = tid; i < 2 * 4 * 64; i += kThreads) bad[i] = 255;
    if (tid < 8) flag[tid] = 0;
    if (tid < 4) done[tid] = 0;
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    auto wait = [&](int bar, int phase) {
        return wait_phase(&bars[bar], phase & 1, abort, p.limit_ns);
    };
    // For all lanes.  Where the wait gave up the warp goes on (with what is in
    // place, in bounds all the same) and leaves at the end of its chunk.
    auto wait_warp = [&](int bar, int phase) {
        wait(bar, phase);
        __syncwarp();
    };
    auto gave_up = [&] { return __any_sync(~0u, *abort != 0); };
    // one arrival of a warp whose lanes are done (each with its own fences)
    auto arrive = [&](int bar) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[bar]);
    };
    // the first token (in memory) of chunk c's tile; may be negative in
    // reverse
    auto tile_token = [&](int c) {
        const int r0 = first + c * kC;
        return rev ? p.T - r0 - kC : r0;
    };
    auto u_col = [](int c) -> uint32_t {
        return STATE_ONLY ? kColU - 3 * kNV * (c & 1) : kColU;
    };
    auto rows_of = [&](int c) { return min(kC, end - (first + c * kC)); };

    // The state's rows and columns of this block, one row kLdS floats, where
    // the parts of V will be; by the first 512 threads.
    float* tile = reinterpret_cast<float*>(sm + Sm::VW);
    const size_t sn = (size_t)pt.j.dk * pt.j.dv;
    float* slots = pt.ws ? pt.ws + bh * p.plan.parts * sn : nullptr;
    if (warp < 16) {
        // 16 elements a thread, along the axis whose elements are adjacent;
        // those of one state are on their way together
        constexpr int E = kC * kNV / 512;
        const bool rows = pt.j.s_c == 1;
        const int r = rows ? tid / kNV : tid % kC;
        const int n = rows ? tid % kNV : tid / kC;
        const int dr = rows ? 512 / kNV : 0, dn = rows ? 0 : 512 / kC;
        const size_t at = (size_t)r * pt.j.s_r + (size_t)(n0 + n) * pt.j.s_c;
        const size_t step = (size_t)dr * pt.j.s_r + (size_t)dn * pt.j.s_c;
        float x[E];
#pragma unroll
        for (int k = 0; k < E; ++k) x[k] = 0.f;
        auto in = [&](int k) {
            return r + k * dr < pt.j.dk && n0 + n + k * dn < pt.j.dv;
        };
        if (STATE_ONLY) {
            if (part == 0 && pt.j.S0)
                for (int k = 0; k < E; ++k)
                    if (in(k))
                        slots[at + k * step] =
                            pt.j.S0[bh * sn + at + k * step];
        } else {
            await_grid_before();
            const float* from = la::state_before(pt, p.plan, part, bh);
            if (from) {
#pragma unroll
                for (int k = 0; k < E; ++k)
                    if (in(k)) x[k] = from[at + k * step];
            }
        }
#pragma unroll
        for (int k = 0; k < E; ++k)
            tile[(r + k * dr) * kLdS + n + k * dn] = x[k];
        tc::named_bar_sync(1, 512);
    }

    int last_bar = -1, last_phase = 0;   // the issuer's last commit

    if (tid == 32 * kCopier) {
        // ------------------------------------------------------ copies
#pragma unroll 1
        for (int c = 0; c < nchunks && !p.selftest; ++c) {
            const int s = c % NS, turn = c / NS;
            uint64_t* full = &bars[B::FULL + s];
            const int t = tile_token(c);
            if (turn && !wait(B::EMPTY_K + s, turn - 1)) break;
            tc::mbar_arrive_expect_tx(full,
                                      (STATE_ONLY ? 1 : 2) * Sm::TILE);
#pragma unroll
            for (int i = 0; i < HALVES; ++i)
                tc::tma_load_4d(sm + Sm::K + s * Sm::TILE + i * kBox,
                                &maps.k[job], full, 64 * i, h, t, b);
            *reinterpret_cast<volatile int*>(issued) = c + 1;
            if (!STATE_ONLY) {
                if (turn && !wait(B::EMPTY_Q + s, turn - 1)) break;
#pragma unroll
                for (int i = 0; i < HALVES; ++i)
                    tc::tma_load_4d(sm + Sm::Q + s * Sm::TILE + i * kBox,
                                    &maps.q[job], full, 64 * i, h, t, b);
            }
            if (turn && !wait(B::EMPTY_V + s, turn - 1)) break;
            tc::mbar_arrive_expect_tx(&bars[B::FULL_V + s], kBox);
            tc::tma_load_4d(sm + Sm::V + s * kBox, &maps.v[job],
                            &bars[B::FULL_V + s], n0, h, t, b);
        }
    } else if (warp == kIssuer) {
        // ---------------------------------------------------- products
        // The whole warp walks the chunks, one lane issues; what the products
        // take is the same in all lanes, so it stays in uniform registers.
        const bool issuer = elect_one();
        // descriptors of the first stage's tiles; addresses count in 16 bytes
        const uint64_t dQ = desc_k(sbase + Sm::Q), dK = desc_k(sbase + Sm::K);
        const uint64_t dKt =       // 64 wide: rows 64 .. 127 of U repeat, unread
            desc_mn(sbase + Sm::K, DK == 128 ? kBox : 0);
        const uint64_t dVw = desc_mn(sbase + Sm::VW, kBox);
        const uint64_t dS = desc_mn(sbase + Sm::S, 0);
        const uint64_t dV = desc_mn(sbase + Sm::V, 0);
        auto step_k = [](int ks) { return (ks >> 2) * (kBox >> 4) + (ks & 3) * 2; };
        auto commit = [&](int bar, int phase) {
            tc::mma_commit(&bars[bar]);
            last_bar = bar, last_phase = phase;
        };
        auto scores = [&](int c) {
            const uint32_t at = c % NS * (Sm::TILE >> 4);
            wait_warp(B::FULL + c % NS, c / NS);
            if (c > 0) wait_warp(B::SC_FREE, c - 1);
            tc::tc_fence_after();
            if (issuer) {
#pragma unroll 2
                for (int ks = 0; ks < DK / 16; ++ks)
                    tc::mma_bf16(tmem + kColSC, dQ + at + step_k(ks),
                                 dK + at + step_k(ks), kIdQK, ks > 0);
                commit(B::SC_FULL, c);
            }
            __syncwarp();
        };
        int scored = 0;      // chunks whose scores are issued
#pragma unroll 1
        for (int c = 0; c < nchunks && !gave_up(); ++c) {
            const int s = c % NS;
            const uint32_t at = s * (Sm::TILE >> 4);
            const bool again = c + NS < nchunks;   // the stage is loaded again
            if (!STATE_ONLY && scored == c) {
                scores(c);
                scored = c + 1;
            }
            wait_warp(B::V_READY + (c & 1), c >> 1);
            if (STATE_ONLY) wait_warp(B::FULL + s, c / NS);
            if (c >= Sm::NVW)
                wait_warp(B::U_FREE + ((c - Sm::NVW) & 1), (c - Sm::NVW) >> 1);
            tc::tc_fence_after();
            if (issuer) {
#pragma unroll 2
                for (int ks = 0; ks < kC / 16; ++ks)
                    tc::mma_bf16(tmem + u_col(c), dKt + at + ks * 128,
                                 dVw + c % Sm::NVW * (3 * kBox >> 4) + ks * 128,
                                 kIdU, ks > 0);
                commit(B::U_FULL + (c & 1), c >> 1);
                if (again) tc::mma_commit(&bars[B::EMPTY_K + s]);
                if (STATE_ONLY && again)
                    tc::mma_commit(&bars[B::EMPTY_V + s]);
            }
            __syncwarp();
            if (STATE_ONLY) continue;
            const uint32_t acc = tmem + kColO + kNV * (c & 1);
            wait_warp(B::S_READY, c);
            if (c > 1) wait_warp(B::O_FREE + (c & 1), (c >> 1) - 1);
            tc::tc_fence_after();
            if (issuer) {
#pragma unroll 2
                for (int ks = 0; ks < DK / 16; ++ks)
                    tc::mma_bf16(acc, dQ + at + step_k(ks), dS + ks * 128,
                                 kIdRow, ks > 0);
                commit(B::S_FREE, c);
                if (again) tc::mma_commit(&bars[B::EMPTY_Q + s]);
            }
            __syncwarp();
            // the next scores, when their inputs are here: they are in the
            // works while this chunk's become P~
            if (scored == c + 1 && scored < nchunks &&
                __all_sync(~0u, mbar_test(&bars[B::FULL + scored % NS],
                                          scored / NS & 1)))
                scores(scored++);
            wait_warp(B::P_READY, c);
            tc::tc_fence_after();
            if (issuer) {
#pragma unroll 2
                for (int ks = 0; ks < kC / 16; ++ks)
                    mma_bf16_ts(acc, tmem + kColP + 8 * ks,
                                dV + s * (kBox >> 4) + ks * 128, kIdRow, true);
                commit(B::O_FULL + (c & 1), c >> 1);
                // hands on what it saw
                tc::mbar_arrive(&bars[B::O_FULL + (c & 1)]);
                if (again) tc::mma_commit(&bars[B::EMPTY_V + s]);
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        // ------------------------------ state (row d, columns c0 .. c0 + 31)
        constexpr int W = kNV / 2;
        const int d = tid & 127, c0 = (warp >> 2) * W;
        float2 S[W / 2];
#pragma unroll
        for (int n = 0; n < W / 2; ++n)
            S[n] = make_float2(tile[d * kLdS + c0 + 2 * n],
                               tile[d * kLdS + c0 + 2 * n + 1]);
        tc::named_bar_sync(2, 512);    // the tile may be written over
        const float2 fs = both(gentle ? power(a, 63 + e) : 1.f);
        auto copy_S = [&] {        // the bf16 copy that Q S reads
            if (d < DK) {
                uint8_t* dst = sm + Sm::S + d * 128;
#pragma unroll
                for (int n = 0; n < W / 8; ++n) {
                    uint32_t x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 y = mul2(fs, S[4 * n + k]);
                        x[k] = tc::pack_bf16x2(y.x, y.y);
                    }
                    const int at = (warp >> 2) * (W / 8) + n;   // of 8 in the row
                    *reinterpret_cast<uint4*>(dst + ((at ^ (d & 7)) << 4)) =
                        make_uint4(x[0], x[1], x[2], x[3]);
                }
            }
            tc::fence_proxy_async_smem();
            arrive(B::S_READY);
        };
        if (!STATE_ONLY) copy_S();
        const uint32_t ucol =
            tmem + ((uint32_t)(d & 96) << 16) + (warp >> 2) * W;
        // w^n S as S + (w^n - 1) S: a decay close to 1 keeps its digits
        float grow = expm1f(a * (float)kC);
#pragma unroll 1
        for (int c = 0; c < nchunks && !gave_up(); ++c) {
            if (c + 1 == nchunks) grow = expm1f(a * (float)rows_of(c));
            wait_warp(B::U_FULL + (c & 1), c >> 1);
            tc::tc_fence_after();
#pragma unroll
            for (int m = 0; m < W; m += 8) {
                float u[3][8];
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    tc::tmem_ld8(ucol + u_col(c) + kNV * k + m, u[k]);
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float2& x = S[m / 2 + k];
                    const float2 y =
                        add2(make_float2(u[0][2 * k], u[0][2 * k + 1]),
                             add2(make_float2(u[1][2 * k], u[1][2 * k + 1]),
                                  make_float2(u[2][2 * k], u[2][2 * k + 1])));
                    x = add2(fma2(both(grow), x, x), y);
                }
            }
            tc::tc_fence_before();
            if (c + 1 < nchunks) {
                arrive(B::U_FREE + (c & 1));
                if (!STATE_ONLY) {
                    wait_warp(B::S_FREE, c);
                    copy_S();
                }
            }
        }
        // (U of the last chunk is formed: nobody reads V's parts any more)
#pragma unroll
        for (int n = 0; n < W / 2; ++n) {
            tile[d * kLdS + c0 + 2 * n] = S[n].x;
            tile[d * kLdS + c0 + 2 * n + 1] = S[n].y;
        }
    } else if (warp < 16) {
        // ------------------------------------------------------ weighted V
        tc::named_bar_sync(2, 512);    // the state has been taken out of there
        const int gt = tid - 256;
        // weights of this thread's rows j0 + 32 m of a whole chunk (no table
        // in shared memory: its bandwidth is what the products are bound by)
        const int j0 = gt >> 3;
        float wt[4];
        auto weigh = [&](int n) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int j = j0 + 32 * m;
                // rows beyond the sequence are zero: their weight is any
                wt[m] = power(a, max(0, rev ? n - kC + 1 + j : n - 1 - j));
            }
        };
        weigh(kC);
#pragma unroll 1
        for (int c = 0; c < nchunks && !gave_up(); ++c) {
            if (c + 1 == nchunks) weigh(rows_of(c));
            wait_warp(B::FULL_V + c % NS, c / NS);
            // the parts' last tile here has been read
            if (c >= Sm::NVW)
                wait_warp(B::U_FULL + ((c - Sm::NVW) & 1), (c - Sm::NVW) >> 1);
            uint8_t* v = sm + Sm::V + c % NS * kBox;
            uint8_t* vw = sm + Sm::VW + c % Sm::NVW * (3 * kBox);
            uint32_t seen = 0;
#pragma unroll
            for (int m = 0; m < 4; ++m) {      // 4 of 1024 16-byte pieces
                const int at = (gt + 256 * m) * 16;
                const float f = wt[m];
                const uint4 x = *reinterpret_cast<const uint4*>(v + at);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                uint32_t o[3][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float2 y = mul2(from_bf16x2(xs[k]), both(f));
                    o[0][k] = upper(y);
                    y = rest(y);
                    o[1][k] = upper(y);
                    o[2][k] = upper(rest(y));
                    seen |= o[2][k];
                }
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    *reinterpret_cast<uint4*>(vw + k * kBox + at) =
                        make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
            }
            // the third part of what is not finite is NaN; those of others are
            // below 2 unless the value is above 2^16: the exponent's top bit
            // tells where to look
            if (!STATE_ONLY && (seen & 0x40004000u)) {
                take_out(v, bad + (c & 1) * 4 * kNV, flag + (c & 1) * 4, done,
                         c, gt, rev, abort, p.limit_ns);
            }
            tc::fence_proxy_async_smem();
            arrive(B::V_READY + (c & 1));
        }
    } else if (warp < 24 && !STATE_ONLY) {
        // ------------------------------------------- scores to P~ (row i)
        const int q = warp & 3, i = 32 * q + lane;
        const int j0 = (warp - 16) >> 2 << 1;   // its two blocks of 32 columns
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
        // (a decay of 0 stays out of 0 * inf)
        const float a2 = (a < -1e4f ? -1e4f : a) * 1.4426950408889634f;
        const float2 row = both(power(a, (rev ? kC - 1 - i : i) + e));
        // the factor w^(63 - s) of column at + m: that of column `at` times
        // w^-m (in reverse w^m); in registers, as the weights of V
        float2 cw[8];
#pragma unroll
        for (int m = 0; m < 8; ++m)
            cw[m] = make_float2(power(a, rev ? 2 * m : -2 * m),
                                power(a, rev ? 2 * m + 1 : -2 * m - 1));
        // (a loop for each kind and order, as short as it can be: one loop
        // with the cases inside took 252 us where these took 222, at B8 T8192
        // H32 d64)
        auto walk = [&](auto kind, auto order) {
            constexpr bool GENTLE = decltype(kind)::value;
            constexpr bool REV = decltype(order)::value;
#pragma unroll 1
            for (int c = 0; c < nchunks && !gave_up(); ++c) {
                wait_warp(B::SC_FULL, c);
                if (c > 0) wait_warp(B::O_FULL + ((c - 1) & 1), (c - 1) >> 1);
                tc::tc_fence_after();
#pragma unroll 1
                for (int at = 32 * j0; at < 32 * j0 + 64; at += 16) {
                    const int j = at >> 5;
                    uint32_t pk[8];
                    float x[16];
                    const bool none = REV ? j < q : j > q;
                    if (!none) {
                        tc::tmem_ld16(lanes + kColSC + at, x);
                        tc::tmem_ld_wait();
                    }
                    if (at == 32 * j0 + 48) {
                        tc::tc_fence_before();
                        arrive(B::SC_FREE);
                    }
                    if (none) {
#pragma unroll
                        for (int m = 0; m < 8; ++m) pk[m] = 0;
                    } else {
                        if (GENTLE) {
                            const float2 f = both(tc::ex2(
                                a2 * (float)(REV ? at - (kC - 64) : 63 - at)));
#pragma unroll
                            for (int m = 0; m < 8; ++m) {
                                const float2 y =
                                    mul2(make_float2(x[2 * m], x[2 * m + 1]),
                                         mul2(f, cw[m]));
                                x[2 * m] = y.x, x[2 * m + 1] = y.y;
                            }
                        } else {
                            const int d = REV ? at - i : i - at;
#pragma unroll
                            for (int m = 0; m < 16; ++m)
                                x[m] *= tc::ex2(a2 * (float)max(0, REV ? d + m
                                                                      : d - m));
                        }
                        if (j == q) {    // masked, not multiplied by 0
                            const int d = lane - (at & 16);
#pragma unroll
                            for (int m = 0; m < 16; ++m)
                                if (REV ? m < d : m > d) x[m] = 0.f;
                        }
#pragma unroll
                        for (int m = 0; m < 8; ++m)
                            pk[m] = tc::pack_bf16x2(x[2 * m], x[2 * m + 1]);
                    }
                    tmem_st8(lanes + kColP + at / 2, pk);
                }
                if (!GENTLE) {       // rows of Q S, this warp's half of the columns
                    const uint32_t acc = lanes + kColO + kNV * (c & 1) + 16 * j0;
                    wait_warp(B::S_FREE, c);
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int m = 0; m < kNV / 2; m += 8) {
                        float x[8];
                        uint32_t u[8];
                        tc::tmem_ld8(acc + m, x);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 8; k += 2) {
                            const float2 y = mul2(row, make_float2(x[k], x[k + 1]));
                            u[k] = __float_as_uint(y.x);
                            u[k + 1] = __float_as_uint(y.y);
                        }
                        tmem_st8(acc + m, u);
                    }
                }
                tc::tmem_st_wait();
                tc::tc_fence_before();
                arrive(B::P_READY);
            }
        };
        const std::true_type yes;
        const std::false_type no;
        if (gentle) rev ? walk(yes, yes) : walk(yes, no);
        else rev ? walk(no, yes) : walk(no, no);
    } else if (warp < 28 && !STATE_ONLY) {
        // ------------------------------------------------ outputs (row i)
        const int q = warp - 24, i = 32 * q + lane, r = rev ? kC - 1 - i : i;
        const float2 f = both(gentle ? power(a, r - 63) : 1.f);
        const int width = min(kNV, pt.j.dv - n0);
        const size_t dv = pt.j.dv;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
        bf16* out = static_cast<bf16*>(pt.j.o);
        const uintptr_t align = reinterpret_cast<uintptr_t>(out) | dv * 2;
#pragma unroll 1
        for (int c = 0; c < nchunks; ++c) {
            wait_warp(B::O_FULL + (c & 1), c >> 1);
            if (gave_up()) break;      // writes nothing
            tc::tc_fence_after();
            const bool any = flag[(c & 1) * 4 + q] != 0;
            uint8_t* own = bad + ((c & 1) * 4 + q) * 64;
            const bool some = r < rows_of(c);
            bf16* dst = out + n0 +
                (((size_t)b * p.T + (some ? tile_token(c) + i : 0)) * p.H +
                 h) * dv;
#pragma unroll 1
            for (int m = 0; m < kNV; m += 16) {
                float x[16];
                uint32_t pk[8];
                __syncwarp();        // (rows beyond the sequence store nothing)
                tc::tmem_ld16(lanes + kColO + kNV * (c & 1) + m, x);
                tc::tmem_ld_wait();
#pragma unroll
                for (int n = 0; n < 16; n += 2) {
                    const float2 y = mul2(f, make_float2(x[n], x[n + 1]));
                    x[n] = y.x, x[n + 1] = y.y;
                }
                if (any) {
#pragma unroll
                    for (int n = 0; n < 16; ++n)
                        if (r >= own[m + n]) x[n] = __uint_as_float(0x7fc00000u);
                }
                if (m + 16 == kNV) {
                    tc::tc_fence_before();
                    __syncwarp();
                    if (any) {
                        own[lane] = own[lane + 32] = 255;
                        if (lane == 0) flag[(c & 1) * 4 + q] = 0;
                        __threadfence_block();
                        __syncwarp();
                    }
                    if (lane == 0) done[q] = c + 1;
                    arrive(B::O_FREE + (c & 1));
                }
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    pk[n] = tc::pack_bf16x2(x[2 * n], x[2 * n + 1]);
                if (some && m < width) {
                    if (align % 32 == 0) {
                        st_global_32(dst + m, pk);
                    } else if (align % 16 == 0) {
                        *reinterpret_cast<uint4*>(dst + m) =
                            make_uint4(pk[0], pk[1], pk[2], pk[3]);
                        if (m + 8 < width)
                            *reinterpret_cast<uint4*>(dst + m + 8) =
                                make_uint4(pk[4], pk[5], pk[6], pk[7]);
                    } else {
#pragma unroll
                        for (int n = 0; n < 16; ++n)
                            if (m + n < width)
                                reinterpret_cast<uint16_t*>(dst)[m + n] =
                                    (uint16_t)(n & 1 ? pk[n / 2] >> 16
                                                     : pk[n / 2]);
                    }
                }
            }
        }
    }

    __syncwarp();
    __syncthreads();
    if (*abort) {
        constexpr uint64_t kDrain = 100000000ull;
        if (warp == kIssuer && last_bar >= 0)   // (the lane that issued)
            tc::mbar_wait(&bars[last_bar], last_phase & 1, kDrain);
        if (tid == 0) {
            atomicOr(&g_fault_la, 1u);
            // copies in flight: at most the last turn of each ring (a barrier
            // that a copy of the turn was never armed for runs out)
            const int n = *reinterpret_cast<volatile int*>(issued);
            for (int c = n - NS < 0 ? 0 : n - NS; c < n; ++c) {
                tc::mbar_wait(&bars[B::FULL + c % NS], (c / NS) & 1, kDrain);
                tc::mbar_wait(&bars[B::FULL_V + c % NS], (c / NS) & 1,
                              kDrain);
            }
        }
    }
    float* dst = STATE_ONLY ? slots + (part + 1) * sn
                 : part + 1 == parts && pt.j.ST ? pt.j.ST + bh * sn : nullptr;
    if (*abort == 0 && dst)
#pragma unroll 1
        for (int i = tid; i < kC * kNV; i += kThreads) {
            const int r = pt.j.s_c == 1 ? i / kNV : i % kC;
            const int n = pt.j.s_c == 1 ? i % kNV : i / kC;
            if (r < pt.j.dk && n0 + n < pt.j.dv)
                dst[(size_t)r * pt.j.s_r + (size_t)(n0 + n) * pt.j.s_c] =
                    tile[r * kLdS + n];
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
    const cudaError_t e = la::allow_smem<linattn_tc<DK, STATE_ONLY>>(Sm::BYTES);
    if (e != cudaSuccess) return e;
    const long long parts = p.plan.parts - (STATE_ONLY ? 1 : 0);
    long long n = 0;
    for (int i = 0; i <= kMaxJobs; ++i) {
        p.first[i] = (int)n;
        if (i < jobs) n += bh * parts * p.part[i].slices;
    }
    return launch_dependent(linattn_tc<DK, STATE_ONLY>, dim3((unsigned)n),
                            kThreads, stream, Sm::BYTES, maps, p);
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

// Parts of a sequence.  A block has an SM to itself, so a launch takes as many
// turns as its blocks fill the SMs; counted with 2.2 us for a chunk, 1.1 us where
// only the state is formed, and 4 us for a block besides (figures of an earlier
// step; a chunk takes 1.7 to 2.0 us now).  More parts fill the last turn better
// and cost a pass over k and v more (us on the GPU, in one part and by this rule:
// d128 B1 T65536 H16 895 and 387, B1 T8192 H16 118 and 67; d64 B1 T16384 H16 227
// and 55, B2 T2049 H12 33 and 22, B4 T4096 H16, in two parts, 57 and 57; B4 T4096
// H16 d128 stays in one).
la::Plan linattn_tc_plan(const LinAttnArgs& a) {
    constexpr int kMost = 32;
    long long blocks = 0;
    for (int i = 0; i < a.jobs; ++i)
        blocks += (long long)a.B * a.H * la::slices_of(a.job[i]);
    const int chunks = (a.T + kC - 1) / kC;
    Plan best{1, a.T};
    auto turns = [&](long long n) { return (n + kPlanSMs - 1) / kPlanSMs; };
    double least = turns(blocks) * (2.2 * chunks + 4.0);
    for (int p = 2; p <= kMost && p <= chunks; ++p) {
        const int len = (chunks + p - 1) / p;           // chunks
        const int parts = (chunks + len - 1) / len;
        const double t =
            turns(blocks * parts) * (2.2 * len + 4.0 + 0.4 * parts) +
            turns(blocks * (parts - 1)) * (1.1 * len + 4.0) + 3.0;
        if (t < 0.97 * least) {
            least = t;
            best = {parts, len * kC};
        }
    }
    return best;
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
        cudaError_t e =
            narrow ? launch<64, true>(maps, p, a.jobs, bh, stream)
                   : launch<128, true>(maps, p, a.jobs, bh, stream);
        if (e == cudaSuccess)
            e = la::join_parts(p.part, a.jobs, p.plan, a.log_decay, bh, a.H,
                               stream);
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
