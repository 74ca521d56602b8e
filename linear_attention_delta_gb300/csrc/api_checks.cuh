// Argument checks shared by the C entry points (host only).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "kla.h"

namespace kla {
namespace api {

inline bool aligned(const void* p, size_t n) {
    return (reinterpret_cast<uintptr_t>(p) % n) == 0;
}

inline kla_status from_cuda(cudaError_t e) {
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

// A buffer of the call: start and length in bytes (null or empty: none).
struct Span {
    const void* p;
    size_t n;
};

// True when the byte ranges of a and b share at least one byte.
inline bool overlap(Span a, Span b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p);
    const uintptr_t b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

// True when any written span overlaps any read span, or two written spans
// overlap each other.
template <size_t NI, size_t NO>
bool any_overlap(const Span (&ins)[NI], const Span (&outs)[NO]) {
    for (size_t i = 0; i < NO; ++i) {
        for (size_t j = 0; j < NI; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (size_t j = i + 1; j < NO; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

inline bool valid(kla_dtype t) { return t == KLA_F32 || t == KLA_BF16; }
inline size_t size_of(kla_dtype t) { return t == KLA_BF16 ? 2 : 4; }

// A pointer that may be null, aligned to its element.
inline bool ok_or_null(const void* p, size_t n) { return !p || aligned(p, n); }
inline bool given(const void* p, size_t n) { return p && aligned(p, n); }

// Bytes from the first to the last element of `rows` rows of D, `stride`
// apart (in elements of `elt` bytes).
inline size_t row_bytes(int rows, int D, long long stride, size_t elt) {
    return rows ? ((size_t)(rows - 1) * (size_t)stride + D) * elt : 0;
}

inline Span span(const void* p, size_t n) { return {p, p ? n : 0}; }

// The kernels count columns, tokens and packed sequences in 32 bits; a thread
// may step past the last one by a block's or a tile's worth.
constexpr int kMaxCount = 0x7fffffff - 4096;

}  // namespace api
}  // namespace kla
