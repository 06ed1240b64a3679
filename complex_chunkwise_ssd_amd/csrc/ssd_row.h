// ssd_row.h -- rows in registers, as the norms hold them: how many lanes share one, the sum over them and
// the root of its mean.
#pragma once

#include <ssd_elem.h>

namespace ssd {

constexpr int kNormMaxF = 16384;

template <int LANES>
struct NormShape {
    static constexpr int waves = LANES <= 256 ? 4 : LANES / 64;   // waves of a workgroup
    static constexpr int threads = 64 * waves;
    static constexpr int rows = threads / LANES;                  // rows it holds at once
};

// Sum over the LANES lanes that hold a row, in every one of them. `red` is this row's slot; rows
// alternate between two of them, so one barrier per row is enough.
template <int LANES>
SSD_DEVICE float row_sum(float v, float *red)
{
    if (LANES == 16)
        return row16_sum(v);
    v = wave_sum(v);
    if (LANES == 64)
        return v;
    if ((thread_id() & 63) == 0)
        red[wave_id()] = v;
    block_sync();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < LANES / 64; ++i)
        t += red[i];
    return t;
}

// 1 / sqrt(v) to little more than half a unit, once per row: a Newton step on the hardware's, its
// residue 1 - v r^2 without rounding errors of the first order (left out where it is no number: v
// is 0, infinite or NaN). The hardware's takes a denormal for 0: small values are scaled by 2^100.
SSD_DEVICE float exact_rsq(float value)
{
    const bool small = value < 0x1p-100f;
    const float v = small ? value * 0x1p+100f : value;
    const float r = hw_rsq(v);
    const float h = v * r, low = __builtin_fmaf(v, r, -h);
    const float d = __builtin_fmaf(-h, r, 1.f) - low * r;
    const float root = d * d < 1.f ? __builtin_fmaf(0.5f * r, d, r) : r;
    return small ? root * 0x1p+50f : root;
}

}  // namespace ssd
