// api_checks.cuh -- the host-side argument checks that the entry points share.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
    const void* p;
    size_t bytes;
};

inline bool overlap(Range a, Range b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

inline size_t esize(gdn_dtype d) { return d == GDN_BF16 ? 2 : 4; }
inline bool dtype_ok(gdn_dtype d) { return d == GDN_F32 || d == GDN_BF16; }
inline bool head_dim_ok(int32_t d) { return d == 64 || d == 128; }

// GDN_OK, or GDN_ERR_CUDA with the code kept for gdn_last_cuda_error (gdn_api.cu).
gdn_status cuda_status(cudaError_t e);

}  // namespace gdn
