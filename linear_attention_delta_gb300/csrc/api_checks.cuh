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

}  // namespace api
}  // namespace kla
