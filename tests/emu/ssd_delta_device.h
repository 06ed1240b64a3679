// ssd_delta_device.h (host emulation) -- TEST INFRASTRUCTURE. The primitives of the gfx950 header of the same name.
#pragma once

#include <ssd_ops_device.h>

SSD_DEVICE uint32_t opaque(uint32_t v) { return v; }
SSD_DEVICE uint32_t opaque_uniform(uint32_t v) { return v; }
SSD_DEVICE void together(float &, float &) {}
