// ssd_host.h -- host-side helpers that the C ABI sources share: pointer checks,
// the status of a launch, one-dimensional grids, element types and sizes. Included after the device
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

constexpr int64_t kMaxThreads = (1LL << 32) - 1;  // of one launch: HIP refuses 2^32 and more
constexpr int64_t kMaxElems = 1LL << 40;  // of one operand: products of sizes and strides stay in 64 bits

inline bool grid_ok(int64_t groups, int threads) { return groups <= kMaxThreads / threads; }

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

inline bool dtype_ok(int dtype) { return dtype == SSD_F32 || dtype == SSD_BF16; }
inline int elem_size(int dtype) { return dtype == SSD_BF16 ? 2 : 4; }

// Bytes from a strided matrix's first element to past its last.
inline int64_t span(int64_t rows, int64_t cols, int64_t stride, int elem)
{
    return rows > 0 && cols > 0 ? ((rows - 1) * stride + cols) * elem : 0;
}

// A buffer of a call, and whether any output of one shares bytes with an input or with another output.
struct Range {
    const void *p;
    int64_t bytes;
};
inline bool overlaps(const Range *out, int outs, const Range *in, int ins)
{
    for (int i = 0; i < outs; ++i) {
        for (int j = 0; j < ins; ++j)
            if (overlap_bytes(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
                return true;
        for (int j = 0; j < i; ++j)
            if (overlap_bytes(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return true;
    }
    return false;
}

}  // namespace ssd
