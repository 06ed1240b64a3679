// ssd_delta_device.h -- further gfx950 primitives that the delta rule's kernels are written against.
#pragma once

#include <ssd_ops_device.h>

// The value itself, of which the compiler knows nothing: what is computed from it inside a loop stays there. The
// walks go over a chunk's tokens and a state's rows in unrolled steps of some sixty offsets, which would
// otherwise all be formed before the loop and held in registers (or spilled) through it.
SSD_DEVICE uint32_t opaque(uint32_t lane_value)
{
    asm volatile("" : "+v"(lane_value));
    return lane_value;
}
SSD_DEVICE uint32_t opaque_uniform(uint32_t value)
{
    asm volatile("" : "+s"(value));
    return value;
}
// Neither value is used before both are there.
SSD_DEVICE void together(float &a, float &b) { asm volatile("" : "+v"(a), "+v"(b)); }
