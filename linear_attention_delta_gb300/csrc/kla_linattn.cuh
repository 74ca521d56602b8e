// What the two forms of the chunked pass of linear attention share.
#pragma once

#include <atomic>

#include "kla_internal.cuh"

namespace kla {
namespace la {

constexpr int kNV = 64;          // columns of v (and of the state) a block has
constexpr int kMaxJobs = 3;      // passes of a call, all in the same launches

// w^n of w = exp(a) (w^0 = 1, whatever w is).
__device__ __forceinline__ float power(float a, int n) {
    return n == 0 ? 1.f : expf(a * (float)n);
}

// Sequences in parts of `len` tokens (a multiple of the chunk; the last part
// the rest).  With parts > 1 a first launch writes, for each part but the
// last, the state that its own tokens leave (slot i + 1 of part i) and a copy
// of S0 (slot 0, if there is one; the main launch may replace S0).  A second
// turns them into the states before the parts,
//   slot_i = w^len slot_{i - 1} + slot_i,
// so that a block of the main launch reads one state, however many parts come
// before its own.
struct Plan {
    int parts, len;
};

struct Part {
    LinAttnJob j;
    float* ws;                   // [B H][parts][dk dv], null with one part
    int slices;                  // blocks along dv
};

// The state before part `part` of sequence and head bh; null: zeros.
__device__ __forceinline__ const float* state_before(const Part& p,
                                                     const Plan& pl, int part,
                                                     size_t bh) {
    const size_t n = (size_t)p.j.dk * p.j.dv;
    if (pl.parts == 1) return p.j.S0 ? p.j.S0 + bh * n : nullptr;
    return part || p.j.S0 ? p.ws + (bh * pl.parts + part) * n : nullptr;
}

// The opt-in to more shared memory, once a kernel and device.
template <auto KERNEL>
cudaError_t allow_smem(int bytes) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (bit && (done.load() & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(
        KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

inline int slices_of(const LinAttnJob& j) { return (j.dv + kNV - 1) / kNV; }

inline int widest_key(const LinAttnArgs& a) {
    int n = 0;
    for (int i = 0; i < a.jobs; ++i) n = a.job[i].dk > n ? a.job[i].dk : n;
    return n;
}

// The second launch above for the passes over B x H sequences and heads.
cudaError_t join_parts(const Part* p, int jobs, const Plan& pl,
                       const float* log_decay, long long bh, int H,
                       cudaStream_t stream);

}  // namespace la

// The tensor-core form: bf16, q and k up to 128 wide, tensors that TMA can
// describe.  linattn_tc_plan looks at sizes only.
bool linattn_tc_sizes(const LinAttnArgs& a);
bool linattn_tc_eligible(const LinAttnArgs& a);
la::Plan linattn_tc_plan(const LinAttnArgs& a);
cudaError_t launch_linattn_tc(const LinAttnArgs& a, float* ws,
                              cudaStream_t stream);

}  // namespace kla
