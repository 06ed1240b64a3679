// ssd_ops_device.h -- the further gfx950 primitives that the operators around the
// scan (norm, 8-bit quantisation and products, gated recurrence) are written
// against: bfloat16 and e4m3 conversion, wave reductions, the 8-bit MFMA tile
// and loads straight into shared memory.
#pragma once

#include <ssd_device.h>

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

SSD_DEVICE uint32_t f2u(float v) { return __builtin_bit_cast(uint32_t, v); }
SSD_DEVICE float u2f(uint32_t v) { return __builtin_bit_cast(float, v); }

// Reciprocal, square root and its reciprocal (v_rcp_f32, v_sqrt_f32, v_rsq_f32; about 1 ulp).
SSD_DEVICE float hw_rcp(float x) { return __builtin_amdgcn_rcpf(x); }
SSD_DEVICE float hw_sqrt(float x) { return __builtin_amdgcn_sqrtf(x); }
SSD_DEVICE float hw_rsq(float x) { return __builtin_amdgcn_rsqf(x); }

// Two floats rounded to e4m3 (nearest, ties to even; NaN stays NaN) in the low or the
// high half of `old`. The caller keeps |a|, |b| below 464, the border to overflow.
template <bool HI>
SSD_DEVICE uint32_t cvt_pk_e4m3(float a, float b, uint32_t old)
{
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HI);
}

// Two floats rounded to bfloat16 (nearest, ties to even), the first in the low half.
SSD_DEVICE uint32_t cvt_pk_bf16(float a, float b)
{
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    const v2bf r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
}
SSD_DEVICE uint16_t cvt_bf16(float a) { return __builtin_bit_cast(uint16_t, (__bf16)a); }

// The value of the lane that differs by x in its index, inside groups of 16 lanes
// (1 and 2: quad permutations; 7 and 15: the half row's and the row's mirror image).
template <int x>
SSD_DEVICE uint32_t row_xor(uint32_t v)
{
    static_assert(x == 1 || x == 2 || x == 7 || x == 15, "one of the four DPP exchanges");
    constexpr int ctrl = x == 1 ? 0xb1 : x == 2 ? 0x4e : x == 7 ? 0x141 : 0x140;
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, true);
}

// D(16x16) += A(16x128) * B(128x16) in e4m3, one wave64. The hardware aligns each group of
// eight products (a lane's consecutive bytes) to the group's largest and drops what lies
// below 2^-13 of it; the groups are added in float32. Lane L supplies 32 values of A's row L % 16 and the same 32 k of B's column L % 16 (those
// of quarter L / 16; which k they are does not matter as long as both agree); it
// receives D[4 * (L / 16) + r][L % 16] in component r.
SSD_DEVICE v4f mfma_e4m3_16x16x128(v8i a, v8i b, v4f c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Eight e4m3 values as bfloat16 (exact), in their order.
SSD_DEVICE v4u e4m3_to_bf16(uint32_t lo, uint32_t hi)
{
    return v4u{
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.f, true)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.f, true))};
}

// D(16x16) += A(16x32) * B(32x16) in bfloat16 with float32 sums: as above with eight
// values per lane.
SSD_DEVICE v4f mfma_bf16_16x16x32(v4u a, v4u b, v4f c)
{
    typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Each lane's 16 (or 4) bytes at byte offset `off` of the buffer go straight to
// shared memory at `lds` + 16 (4) * lane; `lds` is wave-uniform. Bytes at or past the
// buffer's end arrive as zeros. Complete once the wave has waited (async_wait).
SSD_DEVICE void async_load16(buf_t r, uint32_t off, void *lds)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16,
                                             (int)off, 0, 0, 0);
}
SSD_DEVICE void async_load4(buf_t r, uint32_t off, void *lds)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 4,
                                             (int)off, 0, 0, 0);
}
// Waits until at most `n` of this wave's vector memory operations are outstanding, and none
// of its shared-memory operations.
template <int n>
SSD_DEVICE void async_wait()
{
    static_assert(n >= 0 && n < 64, "the wait counter has six bits");
    // vmcnt in bits 3:0 and 15:14, expcnt (7: no wait) in 6:4, lgkmcnt (0) in 11:8
    __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4));
}
// A workgroup barrier that waits for nothing but the other waves.
SSD_DEVICE void bare_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A float that no kernel writes, at a wave-uniform index: a scalar load.
SSD_DEVICE float ld_uniform(const float *p, int64_t i)
{
    using cf = __attribute__((address_space(4))) const float;
    return ((cf *)p)[i];
}
