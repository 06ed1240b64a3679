// ssd_elem.h -- rows of float32 or bfloat16 in groups of eight elements, and the
// e4m3 quantisation of 128 neighbouring values, as the norm and the quantiser use
// them.
//
// A lane holds eight neighbouring elements, so that a bfloat16 group is one 16-byte
// load (a float32 group two) and 16 lanes hold the 128 values that share a scale.
// Groups are loaded at any alignment (the hardware takes it); only a group that
// the end of its row cuts is read element by element.
#pragma once

#include <ssd_ops_device.h>

namespace ssd {

enum { kF32 = 0, kBF16 = 1 };

constexpr float kE4m3Max = 448.f;
constexpr float kTinyScale = 1.17549435082228750797e-38f;  // 2^-126, the smallest normal float

template <int T>
struct ElemSize {
    static constexpr int value = T == kBF16 ? 2 : 4;
};

// Eight elements as they lie in memory.
template <int T>
struct Raw8 {
    v4u w[T == kBF16 ? 1 : 2];
};

// Elements 0 .. n-1 of the group at p, zeros from n on (n may be any number).
template <int T>
SSD_DEVICE Raw8<T> load8(const void *p, int n)
{
    Raw8<T> r;
    if (n >= 8) {
        __builtin_memcpy(&r, p, 8 * ElemSize<T>::value);
        return r;
    }
    uint32_t u[T == kBF16 ? 4 : 8] = {};
    if (n <= 0) {  // a lane past the row's end; kept apart so that whole rows skip what follows
        __builtin_memcpy(&r, u, sizeof(r));
        return r;
    }
    if (T == kBF16) {
        const uint16_t *s = (const uint16_t *)p;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = 2 * e < n ? s[2 * e] : 0u;
            const uint32_t hi = 2 * e + 1 < n ? s[2 * e + 1] : 0u;
            u[e] = lo | hi << 16;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            u[e] = 0u;
            if (e < n)
                __builtin_memcpy(&u[e], (const char *)p + 4 * e, 4);
        }
    }
    __builtin_memcpy(&r, u, sizeof(r));
    return r;
}

template <int T>
SSD_DEVICE void unpack8(const Raw8<T> &r, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (T == kBF16) {
            const uint32_t u = r.w[0][e >> 1];
            v[e] = u2f(e & 1 ? u & 0xffff0000u : u << 16);
        } else {
            v[e] = u2f(r.w[T == kBF16 ? 0 : e >> 2][e & 3]);
        }
    }
}

// v rounded once to T and stored, elements 0 .. n-1.
template <int T>
SSD_DEVICE void store8(void *p, int n, const float (&v)[8])
{
    if (T == kBF16) {
        const v4u u = {cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]), cvt_pk_bf16(v[4], v[5]),
                       cvt_pk_bf16(v[6], v[7])};
        if (n >= 8) {
            __builtin_memcpy(p, &u, 16);
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n)
                ((uint16_t *)p)[e] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
    } else {
        if (n >= 8) {
            const v4f a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
            __builtin_memcpy(p, &a, 16);
            __builtin_memcpy((char *)p + 16, &b, 16);
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n)
                ((float *)p)[e] = v[e];
    }
}

// Largest magnitude of eight values, as the bits of |v|: in unsigned order infinity
// lies above every number and a NaN above infinity, so that neither is lost.
SSD_DEVICE uint32_t amax8(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = f2u(v[e]) & 0x7fffffffu;
        m = m > b ? m : b;
    }
    return m;
}

SSD_DEVICE uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Maximum over the 16 lanes of a row, in every one of them.
SSD_DEVICE uint32_t row16_max(uint32_t v)
{
    v = max_u(v, row_xor<1>(v));
    v = max_u(v, row_xor<2>(v));
    v = max_u(v, row_xor<7>(v));
    return max_u(v, row_xor<15>(v));
}

// Sums over a row of 16 lanes and over the wave's 64 (a fixed order), in every lane.
SSD_DEVICE float row16_sum(float v)
{
    v += u2f(row_xor<1>(f2u(v)));
    v += u2f(row_xor<2>(f2u(v)));
    v += u2f(row_xor<7>(f2u(v)));
    return v + u2f(row_xor<15>(f2u(v)));
}
SSD_DEVICE float wave_sum(float v)
{
    v = row16_sum(v);
    return (lane_read(v, 0) + lane_read(v, 16)) + (lane_read(v, 32) + lane_read(v, 48));
}

// The scale of a block from its largest magnitude: amax / 448, at least 2^-126 so that
// the reciprocal is a number (a block of zeros gets that). With an infinity or a NaN
// in the block it is infinite or NaN, and the block's values come back as NaN.
SSD_DEVICE float e4m3_scale(uint32_t amax)
{
    const float s = u2f(amax) / kE4m3Max;
    return s < kTinyScale ? kTinyScale : s;
}

// v / scale with the rounding of a division, inv = 1 / scale: one correction of v * inv by its
// remainder. (The product alone is off by up to one and a half units, which moves a value next to a
// border of two e4m3 values across it.)
SSD_DEVICE float e4m3_over(float v, float scale, float inv)
{
    const float q = v * inv;
    return __builtin_fmaf(__builtin_fmaf(-q, scale, v), inv, q);
}

// Eight values over their scale, rounded to e4m3. The quotients stay within
// 448 (1 + 2^-23), which rounds to 448: nothing overflows.
SSD_DEVICE v2u e4m3_pack8(const float (&v)[8], float scale, float inv)
{
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        t[e] = e4m3_over(v[e], scale, inv);
    v2u r = {0u, 0u};
    r[0] = cvt_pk_e4m3<false>(t[0], t[1], r[0]);
    r[0] = cvt_pk_e4m3<true>(t[2], t[3], r[0]);
    r[1] = cvt_pk_e4m3<false>(t[4], t[5], r[1]);
    r[1] = cvt_pk_e4m3<true>(t[6], t[7], r[1]);
    return r;
}

// The first n bytes of a group of eight e4m3 values.
SSD_DEVICE void store_e4m3(uint8_t *p, int n, v2u r)
{
    if (n >= 8) {
        __builtin_memcpy(p, &r, 8);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n)
            p[e] = (uint8_t)(r[e >> 2] >> (8 * (e & 3)));
}

}  // namespace ssd
