// Host-side helpers shared by the C ABI's translation units (internal header).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "spl.h"

namespace spl {

// SPL_OK, or SPL_ERR_CUDA with the error remembered for spl_last_cuda_error().
spl_status cuda_status(cudaError_t e);

// CUDA memory type of a pointer (cudaMemoryTypeDevice, cudaMemoryTypeHost for pinned host
// memory, ...), or -1 when the runtime cannot tell (the error is cleared).
int memory_type(const void* p);

inline bool aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Byte ranges [p, p + n) and [q, q + m) share a byte.
inline bool overlap(const void* p, size_t n, const void* q, size_t m) {
    if (p == nullptr || q == nullptr || n == 0 || m == 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + m && b < a + n;
}

}  // namespace spl
