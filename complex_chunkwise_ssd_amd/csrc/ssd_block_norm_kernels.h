// ssd_block_norm_kernels.h -- the norms around a block. The gated norm stands between the block's mixer and
// its last product: per head of D values, with z the gate,
//     r = (sum x^2 / D + eps)^-1/2     y = x r w silu(z)        q = e4m3(y / scale) by 128 neighbours
//     gw = sum gy silu(z) x r          gz = gy x r w sigmoid(z) (1 + z (1 - sigmoid(z)))
//     gx = r (b - x r mean(b x r))     with b = gy silu(z) w
// The block norm stands at its end, with the next block's norm: per row of F values
//     s = res + alpha x r1 w1          y = s r2 w2              q as above
// with r1 of x and r2 of s, and, for l = sum gy y + sum gs s,
//     g_res = gs + r2 (w2 gy - m mean(w2 gy m))                 with m = s r2
//     gx = alpha r1 (w1 g_res - n mean(w1 g_res n))             with n = x r1
//     gw1 = alpha sum g_res n          gw2 = sum gy m
//
// Rows lie in registers as in ssd_norm_kernels.h: every value is read once and written once. Heads of
// 8, 16, 32, 64 or 128 values are whole lanes of one row of 16 and are summed by lane exchange; other
// widths go through shared memory, where a lane leaves the sums of the two heads that its eight values
// may belong to.
//
// 65536 rows of 1024 in bfloat16: the gated norm to 8 bits 80 to 97 us (336 MB; bound by the gate's exponential and
// reciprocal, VALU 93 %; 75.5 with the hardware's reciprocal alone), its gradients 140 (671 MB, 4.8 TB/s); the block norm to
// 8 bits 94 (470 MB, 5.0 TB/s), its gradients with the residual's 159 (805 MB, 5.1 TB/s): all but the first near the
// rate of a copy, also in float32 (128, 253, 164 and 300 us) and for rows up to 8192. Above, 16 waves share a row and a lane has
// 128 registers: gradients spill (gated 148 to 220 bytes a lane, block 180 and 228; block_norm_kernel in float32 36), read
// their weights again and load no row ahead. 4096 rows of 12288, TB/s in bfloat16 / float32: gated 2.7 / 3.4,
// its gradients 2.2 / 3.6, block 4.1 / 4.1, its gradients 2.0 / 2.5.
#pragma once

#include <ssd_row.h>

namespace ssd {

struct GatedNormParams {
    const void *x, *gate;
    const float *w;       // (D)
    void *y;              // nullable
    uint8_t *q;           // nullable
    float *scale;         // (ceil(F / 128), rows), with q
    float *rstd;          // (rows, H), nullable forwards
    const void *gy;       // backwards
    void *gx, *gz;
    float *part;          // (workgroups, D): shares of gw
    int64_t rows, x_stride, gate_stride, gy_stride;
    int F, D, H;
    int log_lanes;        // lanes of a head are 2^log_lanes, or -1
    float eps;
};

// 1 / (1 + e^-z) to about a unit: the exponent's rounding is made up for (it would move a gated value across
// the border of two e4m3 values 16 times as often), and the reciprocal gets a Newton step where it is a number. Below
// 2^-126 (z < -87.3) it is 0.
SSD_DEVICE float exact_sigmoid(float z)
{
    const float log2e = 1.44269502f, rest = 1.92596303e-8f;  // their sum is log2 e to 2^-50
    const float t = -log2e * z;
    const float low = -__builtin_fmaf(log2e, z, t) - rest * z, e = hw_exp2(t);
    const float d = 1.f + (t > -126.f && t < 126.f ? __builtin_fmaf(e, 0.693147182f * low, e) : e);
    const float r = hw_rcp(d);
    return d < 0x1p+100f ? __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r) : r;
}

// Sum over 2^log neighbouring lanes (up to 16), in every one of them.
SSD_DEVICE float lanes_sum(float v, int log)
{
    if (log > 0)
        v += u2f(row_xor<1>(f2u(v)));
    if (log > 1)
        v += u2f(row_xor<2>(f2u(v)));
    if (log > 2)
        v += u2f(row_xor<7>(f2u(v)));
    if (log > 3)
        v += u2f(row_xor<15>(f2u(v)));
    return v;
}

// What the heads of a row share, for widths that are not whole lanes.
template <int LANES, int STEPS, bool WHOLE>
struct HeadSums {
    static constexpr int groups = WHOLE ? 1 : LANES * STEPS;
    float first[groups], second[groups];  // of a lane's values: those of its first head, the rest
    float sum[groups + 1];                // by head; a lane holds eight values, a head at least eight
};

// The sums of `t` over the heads that the lane's values belong to: those of its first values, and of
// those from `cut` on. All lanes of the workgroup arrive (two barriers where a head is not whole lanes).
template <int LANES, int STEPS, bool WHOLE>
SSD_DEVICE void head_sums(const float (&t)[STEPS][8], const int (&at)[STEPS], const int (&cut)[STEPS],
                          const int (&head)[STEPS], int lane, const GatedNormParams &p,
                          HeadSums<LANES, STEPS, WHOLE> &lds, float (&a)[STEPS], float (&b)[STEPS])
{
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        a[k] = b[k] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (WHOLE || e < cut[k])
                a[k] += t[k][e];
            else
                b[k] += t[k][e];
        }
        if (WHOLE)
            a[k] = lanes_sum(a[k], p.log_lanes);
    }
    if (WHOLE)
        return;
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        lds.first[WHOLE ? 0 : at[k] >> 3] = a[k];
        lds.second[WHOLE ? 0 : at[k] >> 3] = b[k];
    }
    block_sync();
    // sixteen lanes a head
    const int heads = p.H;
    for (int h0 = 0; h0 < heads; h0 += LANES / 16) {
        const int h = h0 + (lane >> 4), from = h * p.D, to = from + p.D;
        float s = 0.f;
        if (h < heads) {
            const int g0 = from >> 3, g1 = (to - 1) >> 3;
            for (int g = g0 + (lane & 15); g <= g1; g += 16)
                s += g * 8 < from ? lds.second[WHOLE ? 0 : g] : lds.first[WHOLE ? 0 : g];
        }
        s = row16_sum(s);
        if (h < heads && (lane & 15) == 0)
            lds.sum[WHOLE ? 0 : h] = s;
    }
    block_sync();
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const int h = head[k] < heads ? head[k] : heads - 1;
        a[k] = lds.sum[WHOLE ? 0 : h];
        b[k] = lds.sum[WHOLE ? 0 : h + 1 < heads ? h + 1 : h];
    }
}

template <int T, int LANES, int STEPS, bool WHOLE>
SSD_KERNEL(NormShape<LANES>::threads) void gated_norm_kernel(GatedNormParams p)
{
    using Shape = NormShape<LANES>;
    SSD_LDS HeadSums<LANES, STEPS, WHOLE> sums[Shape::rows];
    const int lane = thread_id() % LANES, mine = thread_id() / LANES;
    const int64_t step = grid_blocks() * Shape::rows;
    int at[STEPS], n[STEPS], cut[STEPS], head[STEPS];
    float w[STEPS][8];
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        at[k] = 8 * (k * LANES + lane);
        n[k] = p.F - at[k];
        head[k] = at[k] / p.D;
        cut[k] = (head[k] + 1) * p.D - at[k];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[k][e] = e < n[k] ? p.w[(at[k] + e) % p.D] : 0.f;
    }
    constexpr int E = ElemSize<T>::value;
    Raw8<T> rx[STEPS], rz[STEPS];
    int64_t row = block_id() * Shape::rows + mine;
    const int64_t end = (p.rows + Shape::rows - 1) / Shape::rows * Shape::rows;
    const int64_t last = p.rows - 1;
    auto fetch = [&](int64_t r) {
        r = r < last ? r : last;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const int i = n[k] > 0 ? at[k] : 0;
            rx[k] = load8<T>((const char *)p.x + (r * p.x_stride + i) * E, n[k]);
            rz[k] = load8<T>((const char *)p.gate + (r * p.gate_stride + i) * E, n[k]);
        }
    };
    fetch(row);
    const float over = 1.f / (float)p.D;
    for (; row < end; row += step) {
        const bool live = row <= last;
        float x[STEPS][8], z[STEPS][8], t[STEPS][8], a[STEPS], b[STEPS];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            unpack8<T>(rx[k], x[k]);
            unpack8<T>(rz[k], z[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[k][e] = x[k][e] * x[k][e];
        }
        if (row + step < end)
            fetch(row + step);
        head_sums<LANES, STEPS, WHOLE>(t, at, cut, head, lane, p, sums[mine], a, b);
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const float r0 = exact_rsq(a[k] * over + p.eps), r1 = WHOLE ? r0 : exact_rsq(b[k] * over + p.eps);
            const bool in = live && n[k] > 0;
            if (p.rstd && in) {  // by the lane that holds the head's first value
                if (at[k] == head[k] * p.D)
                    p.rstd[row * p.H + head[k]] = r0;
                else if (!WHOLE && cut[k] < 8 && cut[k] < n[k])
                    p.rstd[row * p.H + head[k] + 1] = r1;
            }
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[e] = x[k][e] * (WHOLE || e < cut[k] ? r0 : r1) * w[k][e] * (z[k][e] * exact_sigmoid(z[k][e]));
            if (p.y && in)
                store8<T>((char *)p.y + (row * p.F + at[k]) * E, n[k], y);
            if (p.q) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = e < n[k] ? y[e] : 0.f;
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

template <int T, int LANES, int STEPS, bool WHOLE>
SSD_KERNEL(NormShape<LANES>::threads) void gated_norm_bwd_kernel(GatedNormParams p)
{
    using Shape = NormShape<LANES>;
    SSD_LDS HeadSums<LANES, STEPS, WHOLE> sums[Shape::rows];
    SSD_LDS float total[8 * LANES * STEPS];
    const int lane = thread_id() % LANES, mine = thread_id() / LANES;
    const int64_t step = grid_blocks() * Shape::rows;
    int at[STEPS], n[STEPS], cut[STEPS], head[STEPS];
    float gw[STEPS][8];
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        at[k] = 8 * (k * LANES + lane);
        n[k] = p.F - at[k];
        head[k] = at[k] / p.D;
        cut[k] = (head[k] + 1) * p.D - at[k];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            gw[k][e] = 0.f;
    }
    constexpr int E = ElemSize<T>::value;
    constexpr bool AHEAD = LANES < 1024;  // with 16 waves to a row there are 128 registers
    float w[AHEAD ? STEPS : 1][8];
    auto weights = [&](int k) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[AHEAD ? k : 0][e] = e < n[k] ? p.w[(at[k] + e) % p.D] : 0.f;
    };
    if (AHEAD)
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
            weights(k);
    Raw8<T> rx[STEPS], rz[STEPS], rg[STEPS];
    float r0[STEPS], r1[STEPS];
    int64_t row = block_id() * Shape::rows + mine;
    const int64_t end = (p.rows + Shape::rows - 1) / Shape::rows * Shape::rows;
    const int64_t last = p.rows - 1;
    auto fetch = [&](int64_t r) {
        r = r < last ? r : last;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const int i = n[k] > 0 ? at[k] : 0;
            rx[k] = load8<T>((const char *)p.x + (r * p.x_stride + i) * E, n[k]);
            rz[k] = load8<T>((const char *)p.gate + (r * p.gate_stride + i) * E, n[k]);
            rg[k] = load8<T>((const char *)p.gy + (r * p.gy_stride + i) * E, n[k]);
            const int h = head[k] < p.H ? head[k] : p.H - 1;
            r0[k] = p.rstd[r * p.H + h];
            r1[k] = WHOLE ? r0[k] : p.rstd[r * p.H + (h + 1 < p.H ? h + 1 : h)];
        }
    };
    if (AHEAD)
        fetch(row);
    const float over = 1.f / (float)p.D;
    for (; row < end; row += step) {
        const bool live = row <= last;
        if (!AHEAD)
            fetch(row);
        float x[STEPS][8], b[STEPS][8], t[STEPS][8], s0[STEPS], s1[STEPS], q0[STEPS], q1[STEPS];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            float z[8], g[8];
            unpack8<T>(rx[k], x[k]);
            unpack8<T>(rz[k], z);
            unpack8<T>(rg[k], g);
            q0[k] = r0[k];
            q1[k] = r1[k];
            if (!AHEAD)
                weights(k);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float sig = exact_sigmoid(z[e]), wk = w[AHEAD ? k : 0][e];
                x[k][e] *= WHOLE || e < cut[k] ? q0[k] : q1[k];  // the normed value
                const float gn = g[e] * (z[e] * sig);
                if (live)
                    gw[k][e] += gn * x[k][e];
                z[e] = g[e] * x[k][e] * wk * (sig * (1.f + z[e] * (1.f - sig)));
                b[k][e] = gn * wk;
                t[k][e] = b[k][e] * x[k][e];
            }
            if (live && n[k] > 0)
                store8<T>((char *)p.gz + (row * p.F + at[k]) * E, n[k], z);
        }
        if (AHEAD && row + step < end)
            fetch(row + step);
        head_sums<LANES, STEPS, WHOLE>(t, at, cut, head, lane, p, sums[mine], s0, s1);
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            float gx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool one = WHOLE || e < cut[k];
                gx[e] = (one ? q0[k] : q1[k]) * (b[k][e] - x[k][e] * ((one ? s0[k] : s1[k]) * over));
            }
            if (live && n[k] > 0)
                store8<T>((char *)p.gx + (row * p.F + at[k]) * E, n[k], gx);
        }
    }
    // the workgroup's share of gw: the rows that it held at once add theirs in turn, then the heads
    for (int i = 0; i < Shape::rows; ++i) {
        if (mine == i) {
#pragma unroll
            for (int k = 0; k < STEPS; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    total[at[k] + e] = i > 0 ? total[at[k] + e] + gw[k][e] : gw[k][e];
        }
        block_sync();
    }
    for (int d = thread_id(); d < p.D; d += Shape::threads) {
        double s = 0.;
        for (int h = 0; h < p.H; ++h)
            s += total[h * p.D + d];
        p.part[block_id() * p.D + d] = (float)s;
    }
}

struct BlockNormParams {
    const void *x;
    const void *res;      // forwards the residual stream, backwards s
    const float *w1, *w2;
    void *y;              // nullable
    void *res_out;        // s
    uint8_t *q;           // nullable
    float *scale;         // (ceil(F / 128), rows), with q
    float *rstd1, *rstd2; // (rows), nullable forwards
    const void *gy;       // backwards
    const void *gs;       // nullable: the gradient of the residual stream
    void *gx, *gres;
    float *part;          // (workgroups, 2, F): shares of gw1 and of gw2
    int64_t rows, x_stride, res_stride, gy_stride, gs_stride;
    int F;
    float alpha, eps;
};

template <int T, int LANES, int STEPS>
SSD_KERNEL(NormShape<LANES>::threads) void block_norm_kernel(BlockNormParams p)
{
    using Shape = NormShape<LANES>;
    SSD_LDS float red[2][LANES > 64 ? LANES / 64 : 1];
    const int lane = thread_id() % LANES;
    const int64_t step = grid_blocks() * Shape::rows;
    int at[STEPS], n[STEPS];
    float w1[STEPS][8], w2[STEPS][8];
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        at[k] = 8 * (k * LANES + lane);
        n[k] = p.F - at[k];
        unpack8<kF32>(load8<kF32>(p.w1 + (n[k] > 0 ? at[k] : 0), n[k]), w1[k]);
        unpack8<kF32>(load8<kF32>(p.w2 + (n[k] > 0 ? at[k] : 0), n[k]), w2[k]);
    }
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
            const int i = n[k] > 0 ? at[k] : 0;
            rx[k] = load8<T>((const char *)p.x + (r * p.x_stride + i) * E, n[k]);
            rr[k] = load8<T>((const char *)p.res + (r * p.res_stride + i) * E, in ? n[k] : 0);
        }
    };
    fetch(row);
    for (; row < end; row += step) {
        const bool live = row <= last;
        float x[STEPS][8], s[STEPS][8];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            unpack8<T>(rx[k], x[k]);
            unpack8<T>(rr[k], s[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum += x[k][e] * x[k][e];
        }
        if (row + step < end)
            fetch(row + step);
        // a slot of its own for each of the two sums: one is read before the other's barrier
        const float r1 = exact_rsq(row_sum<LANES>(sum, red[0]) / (float)p.F + p.eps);
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[k][e] = __builtin_fmaf(p.alpha * w1[k][e], x[k][e] * r1, s[k][e]);
                sum += s[k][e] * s[k][e];
            }
        const float r2 = exact_rsq(row_sum<LANES>(sum, red[1]) / (float)p.F + p.eps);
        if (live && lane == 0) {
            if (p.rstd1)
                p.rstd1[row] = r1;
            if (p.rstd2)
                p.rstd2[row] = r2;
        }
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const bool in = live && n[k] > 0;
            if (in)
                store8<T>((char *)p.res_out + (row * p.F + at[k]) * E, n[k], s[k]);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[e] = s[k][e] * r2 * w2[k][e];
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

template <int T, int LANES, int STEPS>
SSD_KERNEL(NormShape<LANES>::threads) void block_norm_bwd_kernel(BlockNormParams p)
{
    using Shape = NormShape<LANES>;
    SSD_LDS float red[2][LANES > 64 ? LANES / 64 : 1];
    SSD_LDS float total[Shape::rows > 1 ? 16 * LANES * STEPS : 1];
    const int lane = thread_id() % LANES;
    const int64_t step = grid_blocks() * Shape::rows;
    // with 16 waves to a row there are 128 registers: the weights come from the caches each time, and
    // the next row is not loaded ahead
    constexpr bool AHEAD = LANES < 1024;
    int at[STEPS], n[STEPS];
    float w1[AHEAD ? STEPS : 1][8], w2[AHEAD ? STEPS : 1][8], gw1[STEPS][8], gw2[STEPS][8];
    auto weights = [&](float (&w)[8], const float *from, int k) {
        unpack8<kF32>(load8<kF32>(from + (n[k] > 0 ? at[k] : 0), n[k]), w);
    };
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        at[k] = 8 * (k * LANES + lane);
        n[k] = p.F - at[k];
        if (AHEAD) {
            weights(w1[AHEAD ? k : 0], p.w1, k);
            weights(w2[AHEAD ? k : 0], p.w2, k);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            gw1[k][e] = gw2[k][e] = 0.f;
    }
    constexpr int E = ElemSize<T>::value;
    Raw8<T> rx[STEPS], rs[STEPS], rg[STEPS], rr[STEPS] = {};  // rr stays zero without gs
    float next1 = 0.f, next2 = 0.f;
    int64_t row = block_id() * Shape::rows + thread_id() / LANES;
    const int64_t end = (p.rows + Shape::rows - 1) / Shape::rows * Shape::rows;
    const int64_t last = p.rows - 1;
    auto fetch = [&](int64_t r) {
        r = r < last ? r : last;
        next1 = p.rstd1[r];
        next2 = p.rstd2[r];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const int i = n[k] > 0 ? at[k] : 0;
            rx[k] = load8<T>((const char *)p.x + (r * p.x_stride + i) * E, n[k]);
            rs[k] = load8<T>((const char *)p.res + (r * p.res_stride + i) * E, n[k]);
            rg[k] = load8<T>((const char *)p.gy + (r * p.gy_stride + i) * E, n[k]);
            if (p.gs)
                rr[k] = load8<T>((const char *)p.gs + (r * p.gs_stride + i) * E, n[k]);
        }
    };
    if (AHEAD)
        fetch(row);
    for (; row < end; row += step) {
        if (!AHEAD)
            fetch(row);
        const bool live = row <= last;
        const float r1 = next1, r2 = next2;
        float m[STEPS][8], g[STEPS][8], x[STEPS][8], sum = 0.f;
        Raw8<T> cr[STEPS];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            unpack8<T>(rs[k], m[k]);
            unpack8<T>(rg[k], g[k]);
            unpack8<T>(rx[k], x[k]);
            cr[k] = rr[k];
            if (!AHEAD)
                weights(w2[0], p.w2, k);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                m[k][e] *= r2;
                x[k][e] *= r1;
                if (live)
                    gw2[k][e] += g[k][e] * m[k][e];
                g[k][e] *= w2[AHEAD ? k : 0][e];
                sum += g[k][e] * m[k][e];
            }
        }
        if (AHEAD && row + step < end)
            fetch(row + step);
        const float mean2 = row_sum<LANES>(sum, red[0]) / (float)p.F;
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            float gr[8];
            unpack8<T>(cr[k], gr);
            if (!AHEAD)
                weights(w1[0], p.w1, k);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                gr[e] += r2 * (g[k][e] - m[k][e] * mean2);
                const float ga = p.alpha * gr[e];
                if (live)
                    gw1[k][e] += ga * x[k][e];
                g[k][e] = ga * w1[AHEAD ? k : 0][e];
                sum += g[k][e] * x[k][e];
            }
            if (live && n[k] > 0)
                store8<T>((char *)p.gres + (row * p.F + at[k]) * E, n[k], gr);
        }
        const float mean1 = row_sum<LANES>(sum, red[1]) / (float)p.F;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            float gx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                gx[e] = r1 * (g[k][e] - x[k][e] * mean1);
            if (live && n[k] > 0)
                store8<T>((char *)p.gx + (row * p.F + at[k]) * E, n[k], gx);
        }
    }
    // the workgroup's shares: the rows that it held at once add theirs in turn
    const int mine = thread_id() / LANES;
    if (Shape::rows > 1) {
        for (int i = 0; i < Shape::rows; ++i) {
            if (mine == i) {
#pragma unroll
                for (int k = 0; k < STEPS; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int j = at[k] + e, h = 8 * LANES * STEPS + j;
                        if (i > 0) {
                            gw1[k][e] += total[Shape::rows > 1 ? j : 0];
                            gw2[k][e] += total[Shape::rows > 1 ? h : 0];
                        }
                        total[Shape::rows > 1 ? j : 0] = gw1[k][e];
                        total[Shape::rows > 1 ? h : 0] = gw2[k][e];
                    }
            }
            block_sync();
        }
    }
    if (mine == Shape::rows - 1)
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
            if (n[k] > 0) {
                store8<kF32>(p.part + (2 * block_id()) * p.F + at[k], n[k], gw1[k]);
                store8<kF32>(p.part + (2 * block_id() + 1) * p.F + at[k], n[k], gw2[k]);
            }
}

// Sums over the workgroups' shares part (rows, n), in a fixed order, the first `split` columns to out0
// and the others to out1: 64 columns per workgroup, its 16 waves take every 16th row and their sums are
// added in wave order, all in float64.
constexpr int kShareSumWaves = 16;

SSD_KERNEL(64 * kShareSumWaves) void share_sum_kernel(const float *part, int rows, int n, int split, float *out0,
                                                      float *out1)
{
    SSD_LDS double sums[kShareSumWaves][64];
    const int lane = thread_id() & 63, wave = wave_id();
    const int64_t c = block_id() * 64 + lane;
    double acc = 0.;
    if (c < n) {
#pragma unroll 8
        for (int r = wave; r < rows; r += kShareSumWaves)
            acc += part[(int64_t)r * n + c];
    }
    sums[wave][lane] = acc;
    block_sync();
    if (wave == 0 && c < n) {
        double t = 0.;
#pragma unroll
        for (int i = 0; i < kShareSumWaves; ++i)
            t += sums[i][lane];
        if (c < split)
            out0[c] = (float)t;
        else
            out1[c - split] = (float)t;
    }
}

SSD_KERNEL(256) void share_zero_kernel(float *out, int n)
{
    const int64_t i = block_id() * 256 + thread_id();
    if (i < n)
        out[i] = 0.f;
}

}  // namespace ssd
