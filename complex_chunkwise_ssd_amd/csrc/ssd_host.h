// ssd_host.h -- host-side helpers that the C ABI sources share: pointer checks,
// the status of a launch and one-dimensional grids. Included after the device
// header, which brings the HIP host API.
#pragma once

#include "ssd.h"

#include <stddef.h>
#include <stdint.h>

namespace ssd {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline int launch_status()
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

inline unsigned grid_1d(int64_t n, int threads) { return (unsigned)((n + threads - 1) / threads); }

// Whether [p, p + np) and [q, q + nq) (bytes) share any; a null or empty range shares none.
inline bool overlap_bytes(const void *p, int64_t np, const void *q, int64_t nq)
{
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return p && q && np > 0 && nq > 0 && a < b + (uintptr_t)nq && b < a + (uintptr_t)np;
}

}  // namespace ssd
