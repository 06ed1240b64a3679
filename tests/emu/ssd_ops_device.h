// ssd_ops_device.h (host emulation) -- TEST INFRASTRUCTURE. The further primitives of the
// gfx950 header of the same name, on top of the emulator's wave collectives.
#pragma once

#include <ssd_device.h>

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

SSD_DEVICE uint32_t f2u(float v) { return __builtin_bit_cast(uint32_t, v); }
SSD_DEVICE float u2f(uint32_t v) { return __builtin_bit_cast(float, v); }

// The hardware's take a denormal argument for zero, and give zero for a denormal result.
SSD_DEVICE float emu_flushed(float x) { return fabsf(x) < 1.17549435e-38f ? copysignf(0.f, x) : x; }
SSD_DEVICE float hw_rcp(float x) { return emu_flushed(1.f / emu_flushed(x)); }
SSD_DEVICE float hw_sqrt(float x) { return sqrtf(emu_flushed(x)); }
SSD_DEVICE float hw_rsq(float x) { return 1.f / sqrtf(emu_flushed(x)); }

// e4m3: nearest, ties to even; NaN stays NaN; past the border to overflow NaN as well.
SSD_DEVICE uint32_t emu_e4m3(float v)
{
    const uint32_t sign = f2u(v) >> 31 << 7;
    const double x = fabs((double)v);
    if (!(x < 464.0))
        return sign | 0x7f;
    if (x == 0.0)
        return sign;
    int e;
    (void)frexp(x, &e);
    e = e - 1 < -6 ? -6 : e - 1;
    const double m = nearbyint(ldexp(x, 3 - e));  // in steps of 2^(e - 3)
    if (m < 8)
        return sign | (uint32_t)m;                // subnormal: e is -6
    return sign | (m >= 16 ? (uint32_t)(e + 8) << 3 : (uint32_t)(e + 7) << 3 | ((uint32_t)m - 8));
}
SSD_DEVICE float emu_e4m3_value(uint32_t b)
{
    const int e = b >> 3 & 15, m = b & 7;
    if (e == 15 && m == 7)
        return NAN;
    const float v = e ? ldexpf((float)(8 + m), e - 10) : ldexpf((float)m, -9);
    return b & 0x80 ? -v : v;
}
template <bool HI>
SSD_DEVICE uint32_t cvt_pk_e4m3(float a, float b, uint32_t old)
{
    const uint32_t w = emu_e4m3(a) | emu_e4m3(b) << 8;
    return HI ? (old & 0xffffu) | w << 16 : (old & 0xffff0000u) | w;
}

SSD_DEVICE uint16_t cvt_bf16(float a)
{
    const uint32_t u = f2u(a);
    if (a != a)
        return (uint16_t)(u >> 16 | 0x40);
    return (uint16_t)((u + 0x7fffu + (u >> 16 & 1)) >> 16);
}
SSD_DEVICE uint32_t cvt_pk_bf16(float a, float b) { return cvt_bf16(a) | (uint32_t)cvt_bf16(b) << 16; }

template <int x>
SSD_DEVICE uint32_t row_xor(uint32_t v)
{
    return f2u(lane_fetch(u2f(v), (thread_id() & 63) ^ x));
}

SSD_DEVICE v4f mfma_e4m3_16x16x128(v8i a, v8i b, v4f c)
{
    struct Operands {
        uint8_t a[64][32], b[64][32];
    };
    static Operands waves[16];
    Operands &o = waves[thread_id() >> 6];
    const int lane = thread_id() & 63;
    memcpy(o.a[lane], &a, 32);
    memcpy(o.b[lane], &b, 32);
    wave_lds_sync();
    v4f d = c;
    for (int r = 0; r < 4; ++r) {
        double acc = c[r];
        for (int q = 0; q < 4; ++q)
            for (int k = 0; k < 32; ++k)
                acc += (double)emu_e4m3_value(o.a[16 * q + 4 * (lane >> 4) + r][k]) *
                       emu_e4m3_value(o.b[16 * q + (lane & 15)][k]);
        d[r] = (float)acc;
    }
    wave_lds_sync();
    return d;
}

SSD_DEVICE v4u e4m3_to_bf16(uint32_t lo, uint32_t hi)
{
    v4u r;
    for (int e = 0; e < 4; ++e) {
        const uint32_t w = e < 2 ? lo : hi;
        const uint32_t b = w >> (16 * (e & 1));
        r[e] = f2u(emu_e4m3_value(b & 0xff)) >> 16 | (f2u(emu_e4m3_value(b >> 8 & 0xff)) & 0xffff0000u);
    }
    return r;
}

SSD_DEVICE v4f mfma_bf16_16x16x32(v4u a, v4u b, v4f c)
{
    struct Operands {
        v4u a[64], b[64];
    };
    static Operands waves[16];
    Operands &o = waves[thread_id() >> 6];
    const int lane = thread_id() & 63;
    o.a[lane] = a;
    o.b[lane] = b;
    wave_lds_sync();
    v4f d = c;
    for (int r = 0; r < 4; ++r) {
        double acc = c[r];
        for (int q = 0; q < 4; ++q)
            for (int k = 0; k < 8; ++k) {
                const uint32_t x = o.a[16 * q + 4 * (lane >> 4) + r][k >> 1];
                const uint32_t y = o.b[16 * q + (lane & 15)][k >> 1];
                acc += (double)u2f(k & 1 ? x & 0xffff0000u : x << 16) * u2f(k & 1 ? y & 0xffff0000u : y << 16);
            }
        d[r] = (float)acc;
    }
    wave_lds_sync();
    return d;
}

// Loads straight into shared memory. Each lane's bytes arrive when its wave waits for them and not
// before, so that a read without the wait finds what was there. With shuffled threads, and under
// ThreadSanitizer, some (all) arrive at once as well, as they may: a load into what another wave still
// reads then shows. A workgroup that ends with loads in flight ends the process.
struct EmuLoad {
    void *at;
    char data[16];
    int n;
};
struct EmuLoads {
    EmuLoad load[16];
    int count;
    int64_t block;
};
static EmuLoads emu_loads[1024];

SSD_DEVICE void emu_async(void *at, const void *data, int n)
{
    EmuLoads &l = emu_loads[thread_id()];
    if (l.count > 0 && l.block != block_id()) {
        fprintf(stderr, "emu: workgroup %lld ended with loads in flight\n", (long long)l.block);
        abort();
    }
    if (l.count == 16) {
        fprintf(stderr, "emu: more loads in flight than are emulated\n");
        abort();
    }
#ifdef EMU_TSAN
    const bool now = true;
#else
    const bool now = emu::g_shuffle & 1;
#endif
    if (now)
        memcpy(at, data, (size_t)n);
    l.block = block_id();
    EmuLoad &e = l.load[l.count++];
    e.at = at;
    e.n = n;
    memcpy(e.data, data, (size_t)n);
}
SSD_DEVICE void async_load16(buf_t r, uint32_t off, void *lds)
{
    const v4f v = buf_load4(r, off);
    emu_async((char *)lds + 16 * (thread_id() & 63), &v, 16);
}
SSD_DEVICE void async_load4(buf_t r, uint32_t off, void *lds)
{
    const uint32_t v = buf_load_u32(r, off);
    emu_async((char *)lds + 4 * (thread_id() & 63), &v, 4);
}
template <int n>
SSD_DEVICE void async_wait()
{
    static_assert(n == 0, "a wait for some of the loads is not emulated");
    EmuLoads &l = emu_loads[thread_id()];
    for (int i = 0; i < l.count; ++i)
        memcpy(l.load[i].at, l.load[i].data, (size_t)l.load[i].n);
    l.count = 0;
}
SSD_DEVICE void bare_barrier() { block_sync(); }

SSD_DEVICE float ld_uniform(const float *p, int64_t i) { return p[i]; }
