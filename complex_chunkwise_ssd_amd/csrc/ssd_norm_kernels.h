// ssd_norm_kernels.h -- the RMS norm with the residual's addition, its 8-bit output
// and its gradients. Per row of F values:
//     s = x + res,  rstd = (sum s^2 / F + eps)^-1/2,  y = s rstd w
//     q = e4m3(y / scale), one scale per 128 neighbouring values of a row
// and, for l = sum gy y + sum gs s (gs arrives through the residual stream),
//     gx = gs + rstd (w gy - s rstd^2 (sum w gy s) / F)      gw = sum over rows gy s rstd
// A row is read once: its values stay in registers between the sum and the output.
//
// LANES lanes hold a row, STEPS groups of eight elements each (8 LANES STEPS elements at most):
// 16 lanes a row of up to 128 values, a wave one of up to 1024, and four to sixteen waves a
// longer one, which meet once per row. The workgroups walk over the rows, so that the weights
// are loaded once per wave, and hold the next row's values in flight.
//
// Bound by memory. Measured in bfloat16 with the residual (a copy runs at 5160 GB/s): 65536 x 1024 to
// 8 bits 92 us (5.1 TB/s), its gradients 112 us (4.8 TB/s); 32768 x 4096 190 us (4.9 TB/s);
// 65536 x 64 8.6 us. Eight rows take 2.8 us, mostly the launch. The gradients of float32 rows above
// 8192 spill 144 bytes a lane and reach 49 to 68 % of the copy's rate (4096 x 9000: 235 us).
#pragma once

#include <ssd_elem.h>

namespace ssd {

constexpr int kNormMaxF = 16384;

struct NormParams {
    const void *x;
    const void *res;      // nullable
    const float *w;
    void *y;              // nullable
    void *res_out;        // nullable
    uint8_t *q;           // nullable
    float *scale;         // (ceil(F / 128), rows), with q
    float *rstd;          // nullable
    int64_t rows, x_stride, res_stride;
    int F;
    float eps;
};

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

template <int T, int LANES, int STEPS>
SSD_KERNEL(NormShape<LANES>::threads) void rms_norm_kernel(NormParams p)
{
    using Shape = NormShape<LANES>;
    SSD_LDS float red[2][LANES > 64 ? LANES / 64 : 1];
    const int lane = thread_id() % LANES;          // of those that hold the row
    const int64_t step = grid_blocks() * Shape::rows;
    int at[STEPS], n[STEPS];
    float w[STEPS][8];
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        at[k] = 8 * (k * LANES + lane);
        n[k] = p.F - at[k];
        unpack8<kF32>(load8<kF32>(p.w + (n[k] > 0 ? at[k] : 0), n[k]), w[k]);
    }
    const char *x = (const char *)p.x;
    const char *res = (const char *)p.res;
    constexpr int E = ElemSize<T>::value;
    Raw8<T> rx[STEPS], rr[STEPS];
    int64_t row = block_id() * Shape::rows + thread_id() / LANES;
    const int64_t end = (p.rows + Shape::rows - 1) / Shape::rows * Shape::rows;
    const int64_t last = p.rows - 1;
    auto fetch = [&](int64_t r) {
        // rows past the end are computed and not stored; the last row's residual is not read for
        // them, which may be in place and so be written by the row's own lanes
        const bool in = r <= last;
        r = in ? r : last;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            rx[k] = load8<T>(x + (r * p.x_stride + (n[k] > 0 ? at[k] : 0)) * E, n[k]);
            if (res)
                rr[k] = load8<T>(res + (r * p.res_stride + (n[k] > 0 ? at[k] : 0)) * E, in ? n[k] : 0);
        }
    };
    fetch(row);
    int parity = 0;
    for (; row < end; row += step, parity ^= 1) {
        const bool live = row <= last;
        float s[STEPS][8];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            unpack8<T>(rx[k], s[k]);
            if (res) {
                float t[8];
                unpack8<T>(rr[k], t);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[k][e] += t[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum += s[k][e] * s[k][e];
        }
        if (row + step < end)
            fetch(row + step);
        const float rstd = exact_rsq(row_sum<LANES>(sum, red[parity]) / (float)p.F + p.eps);
        if (live && p.rstd && lane == 0)
            p.rstd[row] = rstd;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[e] = s[k][e] * rstd * w[k][e];
            const bool in = live && n[k] > 0;
            if (p.res_out && in)
                store8<T>((char *)p.res_out + (row * p.F + at[k]) * E, n[k], s[k]);
            if (p.y && in)
                store8<T>((char *)p.y + (row * p.F + at[k]) * E, n[k], y);
            if (p.q) {
                const float scale = e4m3_scale(row16_max(amax8(y)));
                if (in) {
                    store_e4m3(p.q + row * p.F + at[k], n[k], e4m3_pack8(y, scale, 1.f / scale));
                    if ((lane & 15) == 0)
                        p.scale[(int64_t)(at[k] >> 7) * p.rows + row] = scale;
                }
            }
        }
    }
}

struct NormBwdParams {
    const void *s;
    const float *w;
    const float *rstd;
    const void *gy;
    const void *gs;       // nullable: the gradient of the residual stream
    void *gx;
    float *part;          // (workgroups, F): each workgroup's share of gw
    int64_t rows, s_stride, gy_stride, gs_stride;
    int F;
};

template <int T, int LANES, int STEPS>
SSD_KERNEL(NormShape<LANES>::threads) void rms_norm_bwd_kernel(NormBwdParams p)
{
    using Shape = NormShape<LANES>;
    SSD_LDS float red[2][LANES > 64 ? LANES / 64 : 1];
    SSD_LDS float total[Shape::rows > 1 ? 8 * LANES * STEPS : 1];
    const int lane = thread_id() % LANES;          // of those that hold the row
    const int64_t step = grid_blocks() * Shape::rows;
    // with 16 waves to a row there are 128 registers: the weights come from the caches each time
    constexpr bool KEEP = LANES < 1024;
    int at[STEPS], n[STEPS];
    float w[KEEP ? STEPS : 1][8], gw[STEPS][8];
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        at[k] = 8 * (k * LANES + lane);
        n[k] = p.F - at[k];
        if (KEEP)
            unpack8<kF32>(load8<kF32>(p.w + (n[k] > 0 ? at[k] : 0), n[k]), w[KEEP ? k : 0]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            gw[k][e] = 0.f;
    }
    constexpr int E = ElemSize<T>::value;
    Raw8<T> rs[STEPS], rg[STEPS], rr[STEPS] = {};  // rr stays zero without gs
    float next_rstd = 0.f;
    int64_t row = block_id() * Shape::rows + thread_id() / LANES;
    const int64_t end = (p.rows + Shape::rows - 1) / Shape::rows * Shape::rows;
    const int64_t last = p.rows - 1;
    auto fetch = [&](int64_t r) {
        r = r < last ? r : last;
        next_rstd = p.rstd[r];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const int a = n[k] > 0 ? at[k] : 0;
            rs[k] = load8<T>((const char *)p.s + (r * p.s_stride + a) * E, n[k]);
            rg[k] = load8<T>((const char *)p.gy + (r * p.gy_stride + a) * E, n[k]);
            if (p.gs)
                rr[k] = load8<T>((const char *)p.gs + (r * p.gs_stride + a) * E, n[k]);
        }
    };
    fetch(row);
    int parity = 0;
    for (; row < end; row += step, parity ^= 1) {
        const bool live = row <= last;
        const float rstd = next_rstd;
        float s[STEPS][8], g[STEPS][8];
        Raw8<T> cr[STEPS];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            unpack8<T>(rs[k], s[k]);
            unpack8<T>(rg[k], g[k]);
            cr[k] = rr[k];
            if (!KEEP)
                unpack8<kF32>(load8<kF32>(p.w + (n[k] > 0 ? at[k] : 0), n[k]), w[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[k][e] *= rstd;                       // the normalised value
                if (live)
                    gw[k][e] += g[k][e] * s[k][e];
                g[k][e] *= w[KEEP ? k : 0][e];
                sum += g[k][e] * s[k][e];
            }
        }
        if (row + step < end)
            fetch(row + step);
        const float mean = row_sum<LANES>(sum, red[parity]) / (float)p.F;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            float gx[8];
            unpack8<T>(cr[k], gx);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                gx[e] += rstd * (g[k][e] - s[k][e] * mean);
            if (live && n[k] > 0)
                store8<T>((char *)p.gx + (row * p.F + at[k]) * E, n[k], gx);
        }
    }
    // The workgroup's share of gw: the lanes that held different rows add theirs in turn.
    const int mine = thread_id() / LANES;
    if (Shape::rows > 1) {
        for (int i = 0; i < Shape::rows; ++i) {
            if (mine == i) {
#pragma unroll
                for (int k = 0; k < STEPS; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (i > 0)
                            gw[k][e] += total[at[k] + e];
                        total[at[k] + e] = gw[k][e];
                    }
            }
            block_sync();
        }
    }
    if (mine == Shape::rows - 1)
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
            if (n[k] > 0)
                store8<kF32>(p.part + block_id() * p.F + at[k], n[k], gw[k]);
}

// out[c] = sum over r of part[r * n + c] in a fixed order: 64 columns per workgroup, its
// 16 waves take every 16th row and their sums are added in wave order.
constexpr int kColumnSumWaves = 16;

SSD_KERNEL(64 * kColumnSumWaves) void column_sum_kernel(const float *part, int rows, int64_t n,
                                                        float *out)
{
    SSD_LDS float sums[kColumnSumWaves][64];
    const int lane = thread_id() & 63;
    const int wave = wave_id();
    const int64_t c = block_id() * 64 + lane;
    float acc = 0.f;
    if (c < n) {
#pragma unroll 8
        for (int r = wave; r < rows; r += kColumnSumWaves)
            acc += part[r * n + c];
    }
    sums[wave][lane] = acc;
    block_sync();
    if (wave == 0 && c < n) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kColumnSumWaves; ++i)
            t += sums[i][lane];
        out[c] = t;
    }
}

}  // namespace ssd
