// Gated linear recurrence, per sequence and channel:
//
//   h_t = alpha_t h_{t-1} + x_t,  alpha_t = exp(log_alpha_t),  o_t = h_t
//
// and its reverse: g_t = do_t + alpha_{t+1} g_{t+1}, dx_t = g_t,
// dlog_alpha_t = alpha_t g_t h_{t-1}, dh0 = alpha_1 g_1.  Bound by HBM: three
// to five operations per element of each tensor it reads.
//
// Measured (us, share of the copy bandwidth; bf16 with fp32 gates): 4 x 4096
// x 2048 forward 45 (89 %), backward 76.5 (91 %); 65536 x 2048, bf16 gates,
// forward 141 (85 %), where a step of a team of 12 blocks takes 2.5 us: 1.2 of
// work on its tile, the rest waiting for the slowest block's map and for the
// next tile; 16411 x 1024 in 24 packed sequences of random lengths, forward 30
// (50 %); 8191 x 1001 in 9, backward in fp32 47.5 (51 %): rows that line up on
// 4 bytes only, copied in pieces by all threads (4 x 4096 x 2047 with bf16
// gates, forward, 55 against 38.5 us for 2048 channels).
//
// The kernels launch as programmatic dependents: their blocks take their
// places while the kernel before them on the stream drains, and wait for its
// end before they touch memory.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "f32x2.cuh"
#include "kla_internal.cuh"
#include "tc_primitives.cuh"

namespace kla {
namespace {

using bf16 = __nv_bfloat16;

// ---------------------------------------------------------------------------
// The scan.  A tile is W * S consecutive tokens (in scan order:
// backwards in the backward pass) of CH = 64 channels; warp w of its block
// holds S of the tokens, a lane two of the channels.  All tiles of one run of
// tokens (a batch entry, or a part of the packed tokens) and one group of
// channels form a chain.  A chain is walked by a team of G blocks, a thread-block cluster,
// which take every G-th tile each, in order; a block
//   1. waits for its tile's inputs in shared memory, takes them into
//      registers, and starts the copy of its next tile,
//   2. reduces each warp's S steps to the affine map c -> R^2 c + H of the
//      state, and the warps' maps to the tile's map,
//   3. sends the tile's map to all blocks of the team (st.async into their
//      shared memory) and waits for the G maps of this step,
//   4. applies the maps before its own tokens to the state before the step's
//      first tile, and all G to carry that state on: every block of the team
//      carries it by itself, so that no state is handed from block to block
//      and a step costs one exchange, not G,
//   5. runs its steps again from the now known state and writes the outputs.
// Packed tokens are cut into parts of similar length between two sequences
// where that lets more blocks work; every block looks its part up in the
// offsets.
//
// Every input element is read from HBM once.  Maps are applied in token
// order, so the result has the same bits on every run.
//
// A state that a sequence starts from replaces c (it is not multiplied by
// zero), so nothing of one packed sequence, not even a NaN, reaches the next:
// a map that does not depend on the state before it has R = -0, which no
// root of decays is.

constexpr int W = 4;             // warps of a block
// Tokens of a warp, S, and blocks that an SM is to hold, which bounds a
// thread's registers (3: 168, 2: 255; the decays take 2 per token, each input
// 1 or 2).  More tokens mean fewer exchanges, more blocks hide them.  Measured
// against each other, before the launches became dependent ones (us; 65536 tokens x 2048 forward, 4 x 4096 x 2048 forward with fp32 gates):
// bf16 forward 24 and 3 blocks 145, 47.8; 16 and 4 158, 46.4; 28 and 3 140,
// 48.0; 12 and 5 220, 48.5.  bf16 backward (the second) 16 and 3 blocks 79;
// 20 and 3 87; 12 and 4 81.  fp32, 16384 x 1000 forward: 20 and 2 blocks 45;
// 16 and 3 48; backward, 8191 x 1001 packed: 51 and 61.
template <typename T, bool BWD>
constexpr int kSteps = sizeof(T) == 4 ? 20 : BWD ? 16 : 24;
template <typename T>
constexpr int kResident = sizeof(T) == 4 ? 2 : 3;
template <typename T, bool BWD>
constexpr int kTile = W * kSteps<T, BWD>;
constexpr int CH = 64;           // channels of a tile
constexpr int kThreads = 32 * W;
constexpr int kMaxKept = 512;    // offsets of sequences kept on chip
constexpr int kMaxTeam = 16;     // blocks of a team: the largest cluster

struct ScanPlan {
    int tiles, groups;           // tiles of a chain; channel groups
    int rounds;                  // chains that each block walks alone, then
    int rest, team;              // `rest` chains walked by a team each
    int parts;                   // of the packed tokens (1: no rounds else)
    unsigned int wait_ns;        // how long a block waits for maps at most
    bool mute;                   // send none (the self-test of that wait)
};

__device__ unsigned int g_fault_glr = 0;
__device__ float g_selftest_glr[3 * CH];         // the self-test's tensors

// exp of two log decays.  Near 0, where a state remembers 1 / -l tokens and
// a decay's error is multiplied by as much, 1 + l + l^2 / 2 + l^3 / 6 (|l| <=
// 1/64: the rest of the series is below 2^-28, so that the last addition
// rounds correctly nearly always).  Elsewhere 2^(l log2 e) by the hardware's
// approximation (about 2 units of 2^-24 up to l = -1, 8 at l = -8, |l| further
// out: the rounding of l log2 e).
__device__ __forceinline__ float2 decay(float2 l) {
    float2 p = fma2(l, both(1.f / 6), both(0.5f));
    p = fma2(l, p, both(1.f));
    p = fma2(l, p, both(1.f));
    const float2 t = mul2(l, both(1.44269504f));
    const float ex = tc::ex2(t.x), ey = tc::ex2(t.y);
    return make_float2(fabsf(l.x) <= 0x1p-6f ? p.x : ex,
                       fabsf(l.y) <= 0x1p-6f ? p.y : ey);
}

// The square root of a product of decays, from the sum L of their logs: as
// `decay` of L / 2, with more terms of the series (|L| <= 1/2: the rest is below
// 2^-31), since a warp's tokens multiply their logs by their number: with
// `decay` itself, states that remember some hundred tokens came out with more
// than twice the error (hT of 4 x 4096 x 2048: 6.2e-7 instead of 2.3e-7; with
// the product of the rounded decays 4.2e-7).
__device__ __forceinline__ float2 root_decay(float2 L) {
    const float2 l = mul2(L, both(0.5f));
    float2 p = fma2(l, both(1.f / 5040), both(1.f / 720));
    p = fma2(l, p, both(1.f / 120));
    p = fma2(l, p, both(1.f / 24));
    p = fma2(l, p, both(1.f / 6));
    p = fma2(l, p, both(0.5f));
    p = fma2(l, p, both(1.f));
    p = fma2(l, p, both(1.f));
    const float2 t = mul2(l, both(1.44269504f));
    const float ex = tc::ex2(t.x), ey = tc::ex2(t.y);
    return make_float2(fabsf(l.x) <= 0.25f ? p.x : ex,
                       fabsf(l.y) <= 0.25f ? p.y : ey);
}

// Maps c -> R R c + H of two channels as (R.x, R.y, H.x, H.y).  R is the square
// root of the decays' product: the product of up to 96 decays may be far out of
// the range of fp32 where it meets a state that it brings back into it, and R
// has twice the range (a product of 2^-252 or 2^254 takes any state but
// denormal ones out of range).  R is finite (see `bounded`), so that a zero
// state stays zero however large the product grew.
__device__ __forceinline__ float2 plain_apply(float4 m, float2 c) {
    const float2 R = make_float2(m.x, m.y);
    return fma2(mul2(c, R), R, make_float2(m.z, m.w));
}
// Whether a map does not depend on the state before it.  That goes by the
// tokens, so it is the same in all channels.
__device__ __forceinline__ bool fresh(float4 m) {
    return __float_as_uint(m.x) == 0x80000000u;
}
__device__ __forceinline__ float2 apply(float4 m, float2 c) {
    return fresh(m) ? make_float2(m.z, m.w) : plain_apply(m, c);
}
// An R past the range (decays above 1) or NaN (then H is, too) becomes the
// largest number; -0 stays.
__device__ __forceinline__ float bounded(float R) { return fminf(R, 3e38f); }

// A map to the same place in the shared memory of block `rank` of the
// cluster, counted by that block's mbarrier.
__device__ __forceinline__ void send(float4* to, uint64_t* bar, int rank,
                                     float4 m) {
    asm volatile(
        "{\n\t.reg .b32 a, b;\n\t"
        "mapa.shared::cluster.u32 a, %0, %2;\n\t"
        "mapa.shared::cluster.u32 b, %1, %2;\n\t"
        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 "
        "[a], {%3, %4, %5, %6}, [b];\n\t}" ::"r"(tc::smem_u32(to)),
        "r"(tc::smem_u32(bar)), "r"(rank), "r"(__float_as_uint(m.x)),
        "r"(__float_as_uint(m.y)), "r"(__float_as_uint(m.z)),
        "r"(__float_as_uint(m.w))
        : "memory");
}
// Waits, `limit` ns at most, until the maps of a step have arrived.
__device__ __forceinline__ bool wait_maps(uint64_t* bar, uint32_t parity,
                                          uint64_t limit) {
    uint64_t begun = 0;
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, "
            "[%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(tc::smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        const uint64_t now = tc::globaltimer_ns();
        if (begun == 0) begun = now;
        if (now - begun > limit) return false;
    }
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\t"
        "barrier.cluster.wait.acquire.aligned;" ::
            : "memory");
}

// How the inputs' rows line up: on 16 bytes, so that whole tiles can be
// copied (TMA); on pairs of channels; on elements only.  In the last two
// cases a row is copied with the 16-byte pieces that it touches, and rows lie
// in shared memory as far apart, modulo 16 bytes, as in global memory, so
// that pieces meet pieces (kPitch: elements between them at most).
enum Align { kWide, kPair, kElement };
template <Align A, typename T>
constexpr int kPitch = CH + (A == kWide ? 0 : 32 / (int)sizeof(T));

// Where the rows of a tile lie: element 0 of row r at first + r * pitch.
template <Align A, typename T>
struct Rows {
    int first, pitch;
    __device__ Rows(const T* src, long long stride, long long t) {
        if (A == kWide) {
            first = 0;
            pitch = CH;
        } else {
            first = (int)((reinterpret_cast<uintptr_t>(src + t * stride)) &
                          15) / (int)sizeof(T);
            pitch = CH + (16 + (int)(stride * (long long)sizeof(T) & 15)) /
                             (int)sizeof(T);
        }
    }
};

// The two channels of a lane: adjacent where pairs are aligned, else 32
// apart, so that a warp's single elements are adjacent.
template <Align A>
__device__ __forceinline__ int channel(int lane, int v) {
    return A == kElement ? lane + 32 * v : 2 * lane + v;
}

// Two channels as they lie in memory.
template <typename T>
struct Two {
    float2 b;
};
template <>
struct Two<bf16> {
    unsigned int b;
};
__device__ __forceinline__ float2 values(Two<float> t) { return t.b; }
__device__ __forceinline__ float2 values(Two<bf16> t) {
    return from_bf16x2(t.b);
}

template <Align A, typename T>
__device__ __forceinline__ Two<T> read2(const T* row, int lane) {
    if constexpr (A != kElement) {
        return reinterpret_cast<const Two<T>*>(row)[lane];
    } else if constexpr (sizeof(T) == 4) {
        return {make_float2(row[lane], row[lane + 32])};
    } else {
        const auto* r = reinterpret_cast<const unsigned short*>(row);
        return {r[lane] | (unsigned int)r[lane + 32] << 16};
    }
}

// To the lane's channels of an output row (`row`: the lane's own place).
template <Align A, typename T>
__device__ __forceinline__ void write2(T* row, bool l0, bool l1, float2 c) {
    if constexpr (A == kElement) {
        if (l0) row[0] = from_f32<T>(c.x);
        if (l1) row[32] = from_f32<T>(c.y);
    } else if (l0) {
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float2*>(row) = c;
        else
            *reinterpret_cast<unsigned int*>(row) =
                tc::pack_bf16x2(c.x, c.y);
    }
}

// Copies rows t .. t + ROWS - 1 (`stride` elements apart) of `room` channels
// to their places (`Rows`) in dst; rows outside 0 .. n - 1 become zero.  A
// piece of 16 aligned bytes is read from its start to the row's end only; the
// bytes that it may hold before the row belong to the same allocation, which
// starts on 16 bytes.
template <Align A, int ROWS, typename T>
__device__ __forceinline__ void copy_rows(T* dst, const T* src,
                                          long long stride, long long t,
                                          int n, int room) {
    constexpr int P = CH * sizeof(T) / 16 + 1;         // pieces of a row
    constexpr int R = kThreads / (P - 1);              // rows at a time
    static_assert(kThreads % (P - 1) == 0 && kThreads >= ROWS, "");
    const uintptr_t none =
        reinterpret_cast<uintptr_t>(src) & ~(uintptr_t)15;
    const int bytes = min(room, CH) * (int)sizeof(T);
    const int first = (int)max(0ll, -t), last = (int)min((long long)ROWS, n - t);
    const Rows<A, T> place(src, stride, t);
    const int pitch = place.pitch * (int)sizeof(T);
    const unsigned int base = tc::smem_u32(dst);
    auto piece = [&](int r, int p, uintptr_t row, int at) {
        const int left = (int)(row & 15) + bytes - p * 16;
        const bool in = r >= first && r < last && left > 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         base + (at & ~15) + p * 16),
                     "l"(in ? (row & ~(uintptr_t)15) + p * 16 : none),
                     "r"(in ? min(left, 16) : 0)
                     : "memory");
    };
    // all pieces but the last: a thread keeps its place in the row
    const int r0 = threadIdx.x / (P - 1), p0 = threadIdx.x % (P - 1);
    uintptr_t row = reinterpret_cast<uintptr_t>(src + (t + r0) * stride);
    int at = place.first * (int)sizeof(T) + r0 * pitch;
    const long long by = R * stride * (long long)sizeof(T);
    if (first == 0 && last == ROWS && room >= CH) {      // most tiles: whole
#pragma unroll
        for (int r = 0; r < ROWS / R * R; r += R) {
            asm volatile(
                "cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                    base + (at & ~15) + p0 * 16),
                "l"((row & ~(uintptr_t)15) + p0 * 16)
                : "memory");
            row += by;
            at += R * pitch;
        }
    } else {
#pragma unroll 1
        for (int r = 0; r < ROWS / R * R; r += R) {
            piece(r0 + r, p0, row, at);
            row += by;
            at += R * pitch;
        }
    }
    if (ROWS % R && r0 < ROWS % R) piece(r0 + ROWS / R * R, p0, row, at);
    if (threadIdx.x < ROWS)
        piece(threadIdx.x, P - 1,
              reinterpret_cast<uintptr_t>(src + (t + threadIdx.x) * stride),
              place.first * (int)sizeof(T) + (int)threadIdx.x * pitch);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map,
                                            uint64_t* bar, int c0, int c1,
                                            int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::"
        "complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)),
        "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Where sequences begin and end among S tokens of one warp, and which.  In
// scan order: bit i of `mask` says that a sequence begins at step i, which is
// also the end of the one before it, after step i - 1; n is the sequence of
// step 0, last the one that begins last (if any does).
struct Bounds {
    unsigned int mask;
    int n, last;
};

// Packed sequences: the boundaries among the S tokens from t on (upwards, or
// downwards with BACK), of which `steps` are there.  A warp works together: a
// 32-way search for the sequence of t, then 32 offsets at a time.  Any content
// of cu gives 0 <= n, last < B.  Upwards, seq [S]: the sequence that begins at
// step i (any number, where cu is not sorted).
template <int S, bool BACK>
__device__ __forceinline__ Bounds find_bounds(const int* cu, int B,
                                              long long t, int steps,
                                              int* seq) {
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
    int last = lo;               // of the outermost boundary that begins one
    for (int j0 = BACK ? lo + 1 : lo;;) {
        const int j = BACK ? j0 - lane : j0 + lane;
        long long pos = -1;          // step at which the boundary lies
        bool beyond = true;
        if (j >= 0 && j <= B) {
            pos = BACK ? t + 1 - cu[j] : cu[j] - t;
            beyond = pos > S;
        }
        const bool in = pos >= 0 && pos <= S;
        mask |= __reduce_or_sync(0xffffffffu, in ? 1u << pos : 0u);
        if (!BACK && in && pos < S && j < B && cu[j] < cu[j + 1])
            seq[pos] = j;
        // upwards the sequence from the last such offset on, downwards the
        // one up to the first
        const int at = in && pos < steps ? (BACK ? j - 1 : j) : last;
        last = BACK ? __reduce_min_sync(0xffffffffu, at)
                    : __reduce_max_sync(0xffffffffu, at);
        if (__any_sync(0xffffffffu, beyond)) break;
        j0 += BACK ? -32 : 32;
    }
    return {mask, lo, min(max(last, 0), B - 1)};
}

// Packed sequences: the boundary that lies nearest to token t, but not 0.  A
// warp works together; 1 to T, whatever cu holds, rising with t where cu does.
__device__ __forceinline__ int nearest_bound(const int* cu, int B, int T,
                                             int t) {
    const int lane = threadIdx.x % 32;
    int lo = 0, len = B;         // the last one up to t (cu[0] = 0 is)
    while (len > 1) {
        const int step = (len + 31) / 32;
        const int i = lane * step;
        const bool le = i < len && cu[lo + i] <= t;
        const int cnt = max(1, __popc(__ballot_sync(0xffffffffu, le)));
        const int skip = (cnt - 1) * step;
        lo += skip;
        len = min(step, len - skip);
    }
    const long long below = cu[lo], above = cu[lo + 1];
    const long long u = below > 0 && t - below < above - t ? below : above;
    return (int)min(max(u, 1ll), (long long)T);
}

// The tiles of a block, in its order: tile k of the run of tokens b, channels
// from d on.
struct Cursor {
    int round, b, d, k, step, member;            // member of the team
    bool more;
    __device__ Cursor(const ScanPlan& p) : round(-1) { open(p); }
    // Of the packed tokens: the part of this block's chain.
    static __device__ int part(const ScanPlan& p) {
        return blockIdx.x / p.team / p.groups;
    }
    __device__ void open(const ScanPlan& p) {    // the next chain
        ++round;
        int chain = round * (int)gridDim.x + blockIdx.x;
        more = round < p.rounds;
        member = 0;
        step = 1;
        if (round == p.rounds) {
            chain = round * (int)gridDim.x + blockIdx.x / p.team;
            more = blockIdx.x < p.rest * p.team;
            member = blockIdx.x % p.team;
            step = p.team;
        }
        k = member;
        b = p.parts > 1 ? 0 : chain / p.groups;
        d = chain % p.groups * CH;
    }
    __device__ void move(const ScanPlan& p, int tiles) {
        k += step;
        if (k >= tiles && more) open(p);
    }
};

template <typename T, typename G, Align A, bool BWD>
struct Stage {
    T x[kTile<T, BWD>][kPitch<A, T>];
    G la[kTile<T, BWD>][kPitch<A, G>];
};
template <typename T, typename G, Align A>
struct Stage<T, G, A, true> {
    T x[kTile<T, true>][kPitch<A, T>];           // o of the token before
    G la[kTile<T, true>][kPitch<A, G>];
    T g[kTile<T, true>][kPitch<A, T>];           // o_grad
};
template <typename T, typename G, Align A, bool BWD>
struct Shared {
    Stage<T, G, A, BWD> stage;
    // the maps of all warps but the last, of this tile and the next
    float4 own[2][W - 1][32];
    float2 start[32];            // the state before the tile
    int cu[kMaxKept];            // packed sequences: their offsets, if few
    int begin, end, tiles;       // the part's tokens; tiles that they fill
    // the sequences that begin in a warp's tokens, of this tile and the next
    int seq[2][W][kSteps<T, BWD>];
    uint64_t full, got[2];       // the tile is there; the step's maps are
};

// Shared memory of a block of a team.
template <typename T, typename G, Align A, bool BWD>
constexpr int shared_bytes(int team) {
    return (int)sizeof(Shared<T, G, A, BWD>) + 2 * team * 512;
}

template <typename T, typename G, Align A, bool BWD, bool PACKED>
__global__ void __launch_bounds__(kThreads, kResident<T>)
glr_scan_kernel(const __grid_constant__ GlrArgs a,
                const __grid_constant__ ScanPlan plan,
                const __grid_constant__ CUtensorMap map_x,
                const __grid_constant__ CUtensorMap map_la,
                const __grid_constant__ CUtensorMap map_g) {
    extern __shared__ __align__(128) unsigned char smem[];
    auto& sh = *reinterpret_cast<Shared<T, G, A, BWD>*>(smem);
    // the team's maps of this step and the next: [2][team][32]
    auto* maps = reinterpret_cast<float4(*)[32]>(&sh + 1);
    constexpr int DT = BWD ? -1 : 1;             // token step of the scan
    constexpr int S = kSteps<T, BWD>, TILE = kTile<T, BWD>;
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const float* init = BWD ? a.dhT : a.h0;

    if (threadIdx.x == 0) {
        for (uint64_t* bar : {&sh.full, &sh.got[0], &sh.got[1]})
            tc::mbar_init(bar, 1);
        tc::fence_mbar_init();
        sh.begin = 0;
        sh.end = a.T;
        sh.tiles = plan.tiles;
    }
    await_grid_before();
    release_grid_after();
    const int* cu = a.cu;
    if (PACKED && a.B < kMaxKept) {
        for (int i = threadIdx.x; i <= a.B; i += kThreads) sh.cu[i] = a.cu[i];
        cu = sh.cu;
    }
    if (plan.team > 1) cluster_sync();
    else __syncthreads();
    if (PACKED && plan.parts > 1) {
        const int q = Cursor::part(plan);
        auto bound = [&](int i) {
            return i == 0            ? 0
                   : i == plan.parts ? a.T
                                     : nearest_bound(
                                           cu, a.B, a.T,
                                           (int)((long long)a.T * i /
                                                 plan.parts));
        };
        if (w == 0) {
            const int u = bound(q), v = max(u, bound(q + 1));
            if (lane == 0) {
                sh.begin = u;
                sh.end = v;
                sh.tiles = (v - u + TILE - 1) / TILE;
            }
        }
        __syncthreads();
    }
    // The chain's tokens, and tiles that they fill.
    auto begin = [&] { return PACKED ? sh.begin : 0; };
    auto end = [&] { return PACKED ? sh.end : a.T; };
    auto tiles = [&] { return PACKED ? sh.tiles : plan.tiles; };
    // Starts the copy of a tile's inputs: row r is token lo + r, lo the tile's
    // lowest token.
    Stage<T, G, A, BWD>& st = sh.stage;
    auto fetch = [&](const Cursor& at) {
        // (the last warp has the tile's map to form meanwhile)
        if (at.more && (A != kWide || threadIdx.x == 0)) {
            const int b = at.b, d = at.d;
            const int p = at.k * TILE;
            const int lo = BWD ? end() - TILE - p : begin() + p;
            if constexpr (A == kWide) {
                tc::mbar_arrive_expect_tx(&sh.full, sizeof(st));
                tma_load_3d(&st.la[0][0], &map_la, &sh.full, d, lo, b);
                tma_load_3d(&st.x[0][0], &map_x, &sh.full, d,
                            BWD ? lo - 1 : lo, b);
                if constexpr (BWD)
                    tma_load_3d(&st.g[0][0], &map_g, &sh.full, d, lo, b);
            } else {
                const int room = a.D - d;
                copy_rows<A, TILE>(
                    &st.la[0][0],
                    static_cast<const G*>(a.la.p) + b * a.la.sb + d, a.la.st,
                    lo, a.T, room);
                copy_rows<A, TILE>(
                    &st.x[0][0],
                    static_cast<const T*>(a.x.p) + b * a.x.sb + d, a.x.st,
                    BWD ? lo - 1ll : lo, a.T, room);
                if constexpr (BWD)
                    copy_rows<A, TILE>(
                        &st.g[0][0],
                        static_cast<const T*>(a.g.p) + b * a.g.sb + d,
                        a.g.st, lo, a.T, room);
            }
        }
        if (A != kWide) asm volatile("cp.async.commit_group;" ::: "memory");
    };

    Cursor here(plan);
    if (PACKED) here.more &= here.k < tiles();
    fetch(here);
    // What a warp needs to know of its tokens: the boundaries; the start of
    // the sequence that begins last (whoever ends it may write its last state
    // in the place of this start, hT == h0, once the team has this tile's
    // map); backwards, the state before the sequence that ends first.  Looked
    // up a tile ahead, except that without packing most tiles have none.
    Bounds soon{0u, here.b, here.b};
    float2 soon_start = both(0.f), soon_prev = both(0.f);
    auto look = [&](const Cursor& at, unsigned int turn) {
        const int p = at.k * TILE + w * S;
        soon = Bounds{0u, at.b, at.b};
        if (PACKED) {
            const int all = end() - begin();
            if (!at.more || p >= all) return;
            soon = find_bounds<S, BWD>(cu, a.B,
                                       BWD ? end() - 1 - p : begin() + p,
                                       min(S, all - p), sh.seq[turn & 1][w]);
        } else {
            if (p > 0 && p < a.T - S || p >= a.T || !at.more) return;
            if (p == 0) soon.mask = 1u;
            if (a.T - p <= S) soon.mask |= 1u << (a.T - p);
        }
        const int da = at.d + channel<A>(lane, 0);
        const int db = at.d + channel<A>(lane, 1);
        if (init && (soon.mask & ((1u << S) - 1))) {
            const float* q = init + (size_t)soon.last * a.D;
            if (da < a.D) soon_start.x = q[da];
            if (db < a.D) soon_start.y = q[db];
        }
        if (BWD && a.h0 && soon.mask >> 1) {
            const float* q = a.h0 + (size_t)soon.n * a.D;
            if (da < a.D) soon_prev.x = q[da];
            if (db < a.D) soon_prev.y = q[db];
        }
    };
    look(here, 0);

    // blocks that walked chains alone meet before they work as a team: no map
    // may come while its buffer and barrier are in use otherwise
    bool apart = plan.rounds > 0 && plan.team > 1;
    float2 carry = both(0.f);        // the state before the team's tiles
    bool fault = false, late = false;    // late: the tile has not come
    unsigned int turn = 0;
    for (; here.more; ++turn) {
        if (apart && here.step > 1) {
            cluster_sync();
            apart = false;
        }
        const int h = turn & 1;
        const int b = here.b;
        const int da = here.d + channel<A>(lane, 0);
        const int db = here.d + channel<A>(lane, 1);
        const bool la = da < a.D, lb = db < a.D;
        // scan position p <-> token t
        const int p0 = here.k * TILE + w * S;
        const int t0 = BWD ? end() - 1 - p0 : begin() + p0;
        const int steps = max(0, min(S, end() - begin() - p0));
        if (here.k < here.step) carry = both(0.f);       // a chain begins

        const Bounds bd = soon;
        const float2 start = soon_start, prev = soon_prev;
        // whether some map of this step may start anew
        const bool anew = PACKED || here.k < here.step;
        const unsigned int begins = bd.mask & ((1u << steps) - 1);
        // nothing begins, ends or is missing here
        const bool plain = bd.mask == 0 && steps == S;

        auto state_of = [&](const float* p, int n) {
            float2 c = both(0.f);
            if (p && la) c.x = p[(size_t)n * a.D + da];
            if (p && lb) c.y = p[(size_t)n * a.D + db];
            return c;
        };
        auto keep_state = [&](int n, float2 c) {
            if (a.hT && la) a.hT[(size_t)n * a.D + da] = c.x;
            if (a.hT && lb) a.hT[(size_t)n * a.D + db] = c.y;
        };

        if (A == kWide) {
            late = !tc::mbar_wait(&sh.full, h);
            fault |= late;
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
        }

        float2 al[S];                // decays
        Two<T> x[S], g[BWD ? S : 1]; // x; backward: o of the token before, do
        float2 L[2] = {both(0.f), both(0.f)};    // sums of their logs
        float2 H = both(0.f);
        // where the rows of this warp lie (backwards: from its last)
        const int lo = BWD ? end() - TILE - here.k * TILE
                           : begin() + here.k * TILE;
        const Rows<A, G> rl(static_cast<const G*>(a.la.p) + b * a.la.sb +
                                here.d, a.la.st, lo);
        const Rows<A, T> rx(static_cast<const T*>(a.x.p) + b * a.x.sb +
                                here.d, a.x.st, BWD ? lo - 1ll : lo);
        const Rows<A, T> rg(static_cast<const T*>(a.g.p) + b * a.g.sb +
                                here.d, a.g.st, lo);
        const int r0 = BWD ? TILE - 1 - w * S : w * S;
        const G* at_l = &st.la[0][0] + rl.first + r0 * rl.pitch;
        const T* at_x = &st.x[0][0] + rx.first + r0 * rx.pitch;
        const T* at_g = nullptr;
        if constexpr (BWD) at_g = &st.g[0][0] + rg.first + r0 * rg.pitch;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const float2 l = values(read2<A>(at_l + DT * i * rl.pitch, lane));
            al[i] = decay(l);
            x[i] = read2<A>(at_x + DT * i * rx.pitch, lane);
            // (in two halves: smaller sums, smaller roundings)
            L[2 * i / S] = add2(L[2 * i / S], l);
            if constexpr (BWD) {
                g[i] = read2<A>(at_g + DT * i * rg.pitch, lane);
                H = mul2(al[i], add2(H, values(g[i])));
            } else {
                H = fma2(al[i], H, values(x[i]));
            }
        }
        float2 R = root_decay(add2(L[0], L[1]));
        if (begins) {                // only the last sequence matters
            const int from = 31 - __clz(begins);
            R = both(-0.f);
            H = start;
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (i >= from) {
                    if constexpr (BWD)
                        H = mul2(al[i], add2(H, values(g[i])));
                    else
                        H = fma2(al[i], H, values(x[i]));
                }
        }
        const float4 mine =
            make_float4(bounded(R.x), bounded(R.y), H.x, H.y);
        if (w < W - 1) sh.own[h][w][lane] = mine;
        // the tile's place is free, the maps are there
        if (__syncthreads_or(fault)) {
            fault = true;
            break;
        }
        Cursor then = here;
        then.move(plan, tiles());
        if (A == kWide) fetch(then);

        const int m = here.member;
        const int there = min(here.step, tiles() - (here.k - m));
        float4(*team)[32] = maps + h * here.step;
        if (w == W - 1) {            // the tile's map, to all of the team
            float4 t = sh.own[h][0][lane];
            bool cut = fresh(t);
#pragma unroll
            for (int u = 1; u < W; ++u) {
                const float4 q = u < W - 1 ? sh.own[h][u][lane] : mine;
                const float2 v = plain_apply(q, make_float2(t.z, t.w));
                const float2 r =
                    mul2(make_float2(t.x, t.y), make_float2(q.x, q.y));
                t = make_float4(bounded(r.x), bounded(r.y), v.x, v.y);
                if (anew && fresh(q)) {
                    t.z = q.z;
                    t.w = q.w;
                    cut = true;
                }
            }
            if (cut) t.x = t.y = -0.f;
            if (lane == 0)
                tc::mbar_arrive_expect_tx(&sh.got[h], there * 512);
            __syncwarp();
            // a block that walks alone is its own team of one
            const int first = here.step > 1 ? 0 : blockIdx.x % plan.team;
#pragma unroll 4
            for (int r = 0; r < there && !plan.mute; ++r)
                send(&team[m][lane], &sh.got[h], first + r, t);
        }
        // meanwhile
        if (A != kWide) fetch(then);
        look(then, turn + 1);
        if (w == 0) {                // the state before the tile, and after
            fault |= !wait_maps(&sh.got[h], turn >> 1 & 1, plan.wait_ns);
            if (anew) {
#pragma unroll 4
                for (int j = 0; j < m; ++j)
                    carry = apply(team[j][lane], carry);
                sh.start[lane] = carry;
#pragma unroll 4
                for (int j = m; j < there; ++j)
                    carry = apply(team[j][lane], carry);
            } else {
                int j = 0;
#pragma unroll 4
                for (; j < m; ++j) carry = plain_apply(team[j][lane], carry);
                sh.start[lane] = carry;
#pragma unroll 4
                for (; j < there; ++j)
                    carry = plain_apply(team[j][lane], carry);
            }
        }
        __syncthreads();
        float2 c = sh.start[lane];
        if (anew) {
            for (int u = 0; u < w; ++u) c = apply(sh.own[h][u][lane], c);
        } else {
#pragma unroll
            for (int u = 0; u < W - 1; ++u)
                if (u < w) c = plain_apply(sh.own[h][u][lane], c);
        }

        const size_t out = ((size_t)b * a.T + t0) * a.D + da;
        T* op = static_cast<T*>(a.o) + out;
        G* dp = static_cast<G*>(a.dla) + out;
        if (plain) {
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if constexpr (BWD) {
                    c = add2(c, values(g[i]));
                    write2<A>(op, la, lb, c);
                    c = mul2(al[i], c);
                    write2<A>(dp, la, lb, mul2(c, values(x[i])));
                    dp -= a.D;
                    op -= a.D;
                } else {
                    c = fma2(al[i], c, values(x[i]));
                    write2<A>(op, la, lb, c);
                    op += a.D;
                }
            }
        } else if (!PACKED || (steps > 0 && (begins & (begins - 1)) == 0)) {
            // At most one sequence begins here (at `turn_at`), where the one
            // before it ends; another end may be after the last step.  (Code
            // that warps with a boundary alone run costs them most by its
            // length: its instructions have to be fetched.)
            const int turn_at = begins ? __ffs(begins) - 1 : S;
            const bool last_ends = bd.mask >> steps & 1;
            float2 ended = both(0.f), before = prev, tail = both(0.f);
            if (BWD && last_ends && begins && turn_at > 0)
                before = state_of(a.h0, bd.last);
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (i == turn_at) {
                    ended = c;
                    c = start;
                }
                const long long at = (long long)(i * DT) * a.D;
                const bool l0 = la && i < steps, l1 = lb && i < steps;
                if constexpr (BWD) {
                    float2 h = values(x[i]);
                    if (i == turn_at - 1) h = prev;
                    if (last_ends && i == steps - 1) h = before;
                    c = add2(c, values(g[i]));
                    write2<A>(op + at, l0, l1, c);
                    c = mul2(al[i], c);
                    write2<A>(dp + at, l0, l1, mul2(c, h));
                } else {
                    c = fma2(al[i], c, values(x[i]));
                    write2<A>(op + at, l0, l1, c);
                }
                if (PACKED && i == steps - 1) tail = c;
            }
            if (begins > 1) keep_state(bd.n, ended);
            // (steps that are missing leave c as it is; those of the next
            // part do not)
            if (last_ends)
                keep_state(begins ? bd.last : bd.n, PACKED ? tail : c);
        } else if (steps > 0 && !BWD) {
            // Any number of sequences, the states of K steps on their way at
            // a time.  (One state after the other: 256 sequences of a token,
            // 1024 channels, 26 instead of 12 us.)
            constexpr int K = 4;
            static_assert(S % K == 0, "");
            auto begins_at = [&](int i) {
                return min(max(sh.seq[h][w][i], 0), a.B - 1);
            };
            int n = bd.n;
#pragma unroll
            for (int i0 = 0; i0 < S; i0 += K) {
                float2 from[K];
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    from[k] = start;
                    if (begins >> (i0 + k) & 1 && begins >> (i0 + k + 1))
                        from[k] = state_of(init, begins_at(i0 + k));
                }
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int i = i0 + k;
                    if (i >= steps) break;
                    if (begins >> i & 1) {
                        if (i > 0) keep_state(n, c);
                        n = begins_at(i);
                        c = from[k];
                    }
                    c = fma2(al[i], c, values(x[i]));
                    write2<A>(op + (long long)i * a.D, la, lb, c);
                }
            }
            if (bd.mask >> steps & 1) keep_state(n, c);
        } else if (steps > 0) {
            // Backwards one sequence after the other, steps from .. to - 1
            // each.  (As above, with the states before them on their way too,
            // this took 56 instead of 49 us on 90 sequences of 8191 x 1001 in
            // fp32, 22 instead of 23 on 256 of a token.)
            int from = 0, n = bd.n;
            if (begins & 1) c = begins == 1 ? start : state_of(init, n);
            while (true) {
                const unsigned int rest = bd.mask >> (from + 1);
                const int to = min(rest ? from + __ffs(rest) : S, steps);
                float2 before = both(0.f);
                if (rest) before = n == bd.n ? prev : state_of(a.h0, n);
#pragma unroll
                for (int i = 0; i < S; ++i) {
                    if (i < from || i >= to) continue;
                    const long long at = (long long)(i * DT) * a.D;
                    float2 hp = values(x[i]);
                    if (rest && i == to - 1) hp = before;
                    c = add2(c, values(g[BWD ? i : 0]));
                    write2<A>(op + at, la, lb, c);
                    c = mul2(al[i], c);
                    write2<A>(dp + at, la, lb, mul2(c, hp));
                }
                if (rest) keep_state(n, c);
                if (!rest || to >= steps) break;
                from = to;
                if (begins >> (from + 1)) {      // not the last that begins
                    const int t = t0 - from;
                    n = max(n - 1, 0);
                    while (n > 0 && cu[n] > t) --n;
                    c = state_of(init, n);
                } else {
                    n = bd.last;
                    c = start;
                }
            }
        }

        // empty sequences, shared out over the tiles (of the first part)
        if (PACKED && a.hT && a.hT != init && begin() == 0) {
            for (long long e = (long long)here.k * W + w; e < a.B;
                 e += (long long)tiles() * W)
                if (cu[e] == cu[e + 1])
                    keep_state((int)e, state_of(init, (int)e));
        }
        here = then;
    }
    if (A != kWide) asm volatile("cp.async.wait_all;" ::: "memory");
    if (fault && threadIdx.x == 0) {
        atomicOr(&g_fault_glr, 1u);
        // The late copy may be on its way yet.  (A block that gave up waiting
        // for maps has still waited for its next tile before it left.)
        if (A == kWide && late) tc::mbar_wait(&sh.full, turn & 1, 1000000);
    }
    if (apart) cluster_sync();
    if (plan.team > 1) cluster_sync();           // nobody sends here any more
    else if (fault) __syncthreads();
}

// ---------------------------------------------------------------------------
// One token, as a programmatic dependent of the kernel before it: each state
// is read and written once.  A thread takes 4 channels of a sequence, adjacent
// ones (V = 4) or, where they do not line up, single ones 128 apart (V = 1),
// so that their loads are on their way together (1024 x 8191: 17 us, with one
// channel a thread 44; 256 x 2048: 1.6 us in a graph).
template <typename T, typename G, int V>
__global__ void __launch_bounds__(128)
glr_step_kernel(const T* x, long long xs, const G* la, long long ls,
                float* S, T* o, int N, int D) {
    struct alignas(sizeof(T) * V) PT { T v[V]; };
    struct alignas(sizeof(G) * V) PG { G v[V]; };
    struct alignas(4 * V) PS { float v[V]; };
    constexpr int U = 4 / V;
    const int d0 = blockIdx.x * 512 + threadIdx.x * V;
    await_grid_before();
    release_grid_after();
    for (long long n = blockIdx.y; n < N; n += gridDim.y) {
        const size_t i = (size_t)n * D;
        PT px[U];
        PG pl[U];
        PS ps[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int d = d0 + u * 128;
            if (d >= D) continue;
            px[u] = *reinterpret_cast<const PT*>(x + n * xs + d);
            pl[u] = *reinterpret_cast<const PG*>(la + n * ls + d);
            ps[u] = *reinterpret_cast<const PS*>(S + i + d);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int d = d0 + u * 128;
            if (d >= D) continue;
            PT po;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                ps[u].v[v] = fmaf(expf(to_f32(pl[u].v[v])), ps[u].v[v],
                                  to_f32(px[u].v[v]));
                po.v[v] = from_f32<T>(ps[u].v[v]);
            }
            *reinterpret_cast<PS*>(S + i + d) = ps[u];
            *reinterpret_cast<PT*>(o + i + d) = po;
        }
    }
}

// f<T, G>() for the pair of element types.
template <typename F>
cudaError_t by_type(kla_dtype t, kla_dtype g, F f) {
    if (t == KLA_BF16)
        return g == KLA_BF16 ? f(bf16(), bf16()) : f(bf16(), float());
    return g == KLA_BF16 ? f(float(), bf16()) : f(float(), float());
}

template <typename T, typename G, Align A, bool BWD>
void team_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr,
                 int blocks, int team) {
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = shared_bytes<T, G, A, BWD>(team);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = team;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
}

// Blocks in teams of `team` that the current GPU holds at the same time (looked
// up once per device).
template <typename T, typename G, Align A, bool BWD, bool PACKED>
int capacity(int team) {
    static std::atomic<int> found[64][kMaxTeam + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = found[dev][team].load(std::memory_order_relaxed);
    if (n > 0) return n;
    auto* kernel = glr_scan_kernel<T, G, A, BWD, PACKED>;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    team_config<T, G, A, BWD>(cfg, attr, team, team);
    if (cudaFuncSetAttribute(kernel,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             shared_bytes<T, G, A, BWD>(kMaxTeam)) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kernel,
                             cudaFuncAttributeNonPortableClusterSizeAllowed,
                             1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess)
        return 0;
    n *= team;
    found[dev][team].store(n, std::memory_order_relaxed);
    return n;
}

// How `chains` chains of `tiles` tiles share the blocks that the GPU holds:
// whole rounds of a chain per block, then the rest by a team each.  A round
// counts as 1, a team of t as 1 / t.
//
// Packed tokens can be cut between two of the `sequences`, into as many parts
// as leave a team of the chosen size to each.  A part is longer than the
// average by what the lengths are, which the host does not know: half a
// sequence per doubling is expected, and, the less likely the more sequences
// there are, one with nearly all of the tokens, where only one team has work.
// A step costs a larger team more (1 + 0.03 t).  How likely one long sequence
// is, is an assumption, not a measurement.  Measured (GPU us, whole / in parts;
// four draws of random lengths, one in six sequences empty and one a token): 24
// sequences of 16411 tokens, 1024 channels, forward 37 to 41 / 28 to 30,
// backward 52 to 57 / 39 to 42; 4 of them, forward 33 / 25 to 31; 600 of 32768
// x 2048 162 to 174 / 151 to 163; 64 of 65536 x 64 101 to 108 / 13 to 15; 1000
// of 65536 x 256 200 to 211 / 47 to 51.  Even lengths: 24 of 16411 x 1024 34 /
// 25.  One long sequence and single tokens: 41 / 43, backward 68 / 68.
template <typename T, typename G, Align A, bool BWD, bool PACKED>
ScanPlan plan_of(long long chains, int tiles, int D, int sequences,
                 int* blocks) {
    ScanPlan best{tiles, (D + CH - 1) / CH, 0, 0, 1, 1, 2000000000u, false};
    *blocks = 0;
    double cost = 0;
    for (int team = 1; team <= std::min(kMaxTeam, tiles); ++team) {
        const int slots = capacity<T, G, A, BWD, PACKED>(team);
        if (slots <= 0) break;
        const int rounds = (int)(chains / slots), rest = (int)(chains % slots);
        if ((long long)rest * team > slots) continue;
        const double c = rounds + (rest ? 1.0 / team : 0.0);
        if (*blocks && c >= cost) continue;
        cost = c;
        best.rounds = rounds;
        best.rest = rest;
        best.team = team;
        *blocks = rounds ? slots : rest * team;
    }
    if (sequences < 2 || *blocks == 0 || best.rounds) return best;
    // the time of a team, in steps of one block
    auto steps = [&](int team, double share) {
        return (1 + 0.03 * team) * std::max(1.0, tiles * share / team);
    };
    double least = steps(best.team, 1) - 1;
    // how likely one sequence has nearly all tokens
    const double one = std::min(0.25, 6.0 / sequences);
    for (int team = (best.team + 1) / 2, most = std::min(kMaxTeam, tiles);
         team <= most; ++team) {
        const int slots = capacity<T, G, A, BWD, PACKED>(team);
        if (slots <= 0) break;
        const int parts =
            std::min(sequences, slots / (best.groups * team));
        if (parts < 2) continue;
        const double share =
            1.0 / parts + std::log2((double)parts) / 2 / sequences;
        const double time =
            (1 - one) * steps(team, share) + one * steps(team, 1);
        if (time >= least) continue;
        least = time;
        best.parts = parts;
        best.rest = best.groups * parts;
        best.team = team;
        *blocks = best.rest * team;
    }
    return best;
}

// The element's tensor map over [B, T, D] with boxes of `tokens` tokens x
// CH channels (zeros outside).
template <typename T>
bool make_tile_map(CUtensorMap* m, const Strided& x, const GlrArgs& a,
                   int tokens) {
    const bool packed = a.cu != nullptr;
    cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.T,
                          (cuuint64_t)(packed ? 1 : a.B)};
    // a stride that no row is taken with still has to be a valid one
    const cuuint64_t row = ((cuuint64_t)a.D * sizeof(T) + 15) / 16 * 16;
    cuuint64_t strides[2] = {
        a.T > 1 ? (cuuint64_t)x.st * sizeof(T) : row,
        !packed && a.B > 1 ? (cuuint64_t)x.sb * sizeof(T) : row * a.T};
    cuuint32_t box[3] = {CH, (cuuint32_t)tokens, 1}, es[3] = {1, 1, 1};
    return tile_map_encoder()(
               m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
               3, const_cast<void*>(x.p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, typename G, Align A, bool BWD, bool PACKED>
cudaError_t launch_scan(const GlrArgs& a, cudaStream_t s) {
    const long long chains =
        (long long)((a.D + CH - 1) / CH) * (a.cu ? 1 : a.B);
    if (chains > 0x7fffffffLL) return cudaErrorInvalidValue;
    constexpr int TILE = kTile<T, BWD>;
    auto* kernel = glr_scan_kernel<T, G, A, BWD, PACKED>;
    int blocks = 0;
    const ScanPlan p = plan_of<T, G, A, BWD, PACKED>(
        chains, (int)((a.T + (long long)TILE - 1) / TILE), a.D,
        a.cu ? a.B : 1, &blocks);
    if (blocks <= 0) return cudaErrorInvalidValue;
    CUtensorMap mx{}, ml{}, mg{};
    if (A == kWide &&
        (!make_tile_map<T>(&mx, a.x, a, TILE) ||
         !make_tile_map<G>(&ml, a.la, a, TILE) ||
         (BWD && !make_tile_map<T>(&mg, a.g, a, TILE))))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    team_config<T, G, A, BWD>(cfg, attr, blocks, p.team);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kernel, a, p, mx, ml, mg);
}

// Whether all rows of a strided input start on a multiple of `bytes`.
bool lines_up(const Strided& x, size_t elt, size_t bytes) {
    return reinterpret_cast<uintptr_t>(x.p) % bytes == 0 &&
           x.st * elt % bytes == 0 && x.sb * elt % bytes == 0;
}
// Whether a tensor map can describe it: no repeated rows.
bool maps(const Strided& x, const GlrArgs& a) {
    return (a.T == 1 || x.st > 0) && (a.cu || a.B == 1 || x.sb > 0);
}

template <typename T, typename G, Align A>
cudaError_t launch_way(const GlrArgs& a, bool bwd, cudaStream_t s) {
    if (a.cu)
        return bwd ? launch_scan<T, G, A, true, true>(a, s)
                   : launch_scan<T, G, A, false, true>(a, s);
    return bwd ? launch_scan<T, G, A, true, false>(a, s)
               : launch_scan<T, G, A, false, false>(a, s);
}

}  // namespace

cudaError_t launch_glr(const GlrArgs& args, bool bwd, cudaStream_t stream) {
    // A stride that no step is taken with may be any number: how rows line up,
    // in global and in shared memory, must not be derived from it.
    GlrArgs a = args;
    for (Strided* x : {&a.x, &a.la, &a.g}) {
        if (a.T <= 1) x->st = 0;
        if (a.cu || a.B <= 1) x->sb = 0;
    }
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
        auto in = [&](size_t tb, size_t gb) {
            return lines_up(a.x, sizeof(T), tb) &&
                   lines_up(a.la, sizeof(G), gb) &&
                   (!bwd || lines_up(a.g, sizeof(T), tb));
        };
        // pairs: the outputs' rows (of D) too
        const bool pairs =
            a.D % 2 == 0 && in(2 * sizeof(T), 2 * sizeof(G)) &&
            reinterpret_cast<uintptr_t>(a.o) % (2 * sizeof(T)) == 0 &&
            reinterpret_cast<uintptr_t>(a.dla) % (2 * sizeof(G)) == 0;
        const bool wide = pairs && in(16, 16) && maps(a.x, a) &&
                          maps(a.la, a) && (!bwd || maps(a.g, a)) &&
                          get_encoder();
        return wide    ? launch_way<T, G, kWide>(a, bwd, stream)
               : pairs ? launch_way<T, G, kPair>(a, bwd, stream)
                       : launch_way<T, G, kElement>(a, bwd, stream);
    });
}

cudaError_t launch_glr_selftest(cudaStream_t stream) {
    // one tile of one token and CH channels in memory of its own
    void* p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_selftest_glr);
    if (e != cudaSuccess) return e;
    float* m = static_cast<float*>(p);
    GlrArgs a{};
    a.x = {m, CH, CH};
    a.la = {m + CH, CH, CH};
    a.o = m + 2 * CH;
    a.B = a.T = 1;
    a.D = CH;
    if (capacity<float, float, kPair, false, false>(1) <= 0)
        return cudaErrorInvalidValue;
    const ScanPlan plan{1, 1, 0, 1, 1, 1, 1000000u, true};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    team_config<float, float, kPair, false>(cfg, attr, 1, 1);
    cfg.stream = stream;
    const CUtensorMap none{};
    return cudaLaunchKernelEx(&cfg, glr_scan_kernel<float, float, kPair, false,
                                              false>,
                              a, plan, none, none, none);
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
        auto aligned = [](const void* p, size_t n) {
            return reinterpret_cast<uintptr_t>(p) % n == 0;
        };
        const bool four = D % 4 == 0 && x_stride % 4 == 0 &&
                          la_stride % 4 == 0 && aligned(x, 4 * sizeof(T)) &&
                          aligned(la, 4 * sizeof(G)) && aligned(S, 16) &&
                          aligned(o, 4 * sizeof(T));
        const dim3 grid((D + 511) / 512, std::min(N, 65535));
        return launch_dependent(
            four ? glr_step_kernel<T, G, 4> : glr_step_kernel<T, G, 1>, grid,
            128, stream, 0, static_cast<const T*>(x), x_stride,
            static_cast<const G*>(la), la_stride, S, static_cast<T*>(o), N,
            D);
    });
}

}  // namespace kla
