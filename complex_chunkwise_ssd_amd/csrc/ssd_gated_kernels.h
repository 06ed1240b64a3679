// ssd_gated_kernels.h -- the gated linear recurrence: per sequence and channel, with i and r
// the sigmoids of the input gate and of the decay gate,
//     l_t = -k softplus(lam) r_t      a_t = exp(l_t)      m_t = sqrt(1 - a_t^2)
//     h_t = a_t h_{t-1} + m_t i_t x_t
// and its gradients, with g_t = gh_t + a_{t+1} g_{t+1} the adjoint of h_t:
//     gx = g m i     g_input = g m x i (1 - i)     E = g h_{t-1} a l - g i x a^2 (l / m)
//     g_decay = E (1 - r)     g_lam = sigmoid(lam) / softplus(lam) sum_t E
// (l / m and not 1 / m: as r goes to 0 so do l and m, and their ratio with them).
//
// Both are bound by memory in float32 and by the arithmetic of the gates in bfloat16 (three
// exponentials, two reciprocals, a root and some 25 other instructions a value, all on the vector unit).
// Measured, with a copy at 5160 GB/s: 4 x 2048 x 4096 float32, 4.74 TB/s forward and 4.63
// backward; 32 x 2048 x 1024 bfloat16 126 us (4.3 TB/s), gradients 214 us (4.4 TB/s); cut into
// segments, 3 x 16411 x 1000 float32, 273 us, with random lengths 228 us (91 of them the pass before).
//
// A composition of steps over a span is a pair (A, U):
// h -> A h + U. A workgroup walks over the tokens of one block of channels in tiles; its
// waves each take kGatedSteps neighbouring tokens of the tile, find their (A, U) with the
// gates in registers, meet once in shared memory, fold the pairs of the waves before them
// onto the state that entered the tile and put out their own tokens from there. So every
// value is read once, a row of a tile is one full line per wave, and the next tile's
// loads are in flight meanwhile. Where sequences and channels give too few workgroups, the
// tokens are cut into segments, and a pass over the gates finds each segment's (A, U)
// first; each segment then folds those before it.
#pragma once

#include <ssd_elem.h>

namespace ssd {

constexpr int kGatedChunk = 64;    // tokens between two stored states

struct GatedParams {
    const void *x, *gi, *gr;
    const float *lam;
    const float *init;        // nullable: (B, C)
    const int *lengths;       // nullable: (B)
    void *h;                  // (B, T, C)
    float *final_state;       // nullable: (B, C)
    float *states;            // nullable: (B, ceil(T / 64), C), the state entering each chunk
    float *seg;               // (B, segments, 2, C): A then U of each segment (see below)
    // backward
    const void *gh;           // (B, T, C)
    const float *gfinal;      // nullable: (B, C)
    const float *chunk_states;
    void *gx, *ggi, *ggr;     // (B, T, C)
    float *part;              // (B * segments, C): shares of sum E
    float *ginit;             // nullable: (B, C)
    int64_t x_stride, gi_stride, gr_stride;  // elements between tokens; a sequence is T of them
    int B, T, C;
    int blocks;               // channel blocks
    int segments, seg_tokens;
    int launched, seg_first;  // segments of this launch: seg_first .. seg_first + launched - 1
    float k;                  // decay scale
};

// Channels per lane: CH neighbouring channels, one load of CH elements.
template <int T, int CH>
struct GatedRaw {
    uint32_t w[T == kF32 ? CH : 1];
};

template <int T, int CH>
SSD_DEVICE GatedRaw<T, CH> gated_load(const void *p)
{
    GatedRaw<T, CH> r;
    if (T == kBF16 && CH == 1)
        r.w[0] = *(const uint16_t *)p;
    else
        __builtin_memcpy(&r, p, sizeof(r));
    return r;
}

template <int T, int CH>
SSD_DEVICE float gated_value(const GatedRaw<T, CH> &r, int c)
{
    if (T == kF32)
        return u2f(r.w[T == kF32 ? c : 0]);
    return u2f(c ? r.w[0] & 0xffff0000u : r.w[0] << 16);
}

template <int T, int CH>
SSD_DEVICE void gated_store(void *p, const float (&v)[CH])
{
    if (T == kF32) {
        __builtin_memcpy(p, v, 4 * CH);
    } else if (CH == 2) {
        const uint32_t u = cvt_pk_bf16(v[0], v[CH - 1]);
        __builtin_memcpy(p, &u, 4);
    } else {
        *(uint16_t *)p = cvt_bf16(v[0]);
    }
}

constexpr float kLog2e = 1.44269504088896340736f;

SSD_DEVICE float sigmoid(float v) { return hw_rcp(1.f + hw_exp2(-kLog2e * v)); }

SSD_DEVICE float softplus(float v)
{
    return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
}

// -k softplus(lam), l at an open gate: held to a finite number, so that l times a closed gate is 0, and
// so is l times a decay of 0 in the gradients.
SSD_DEVICE float decay_rate(float k, float lam)
{
    const float most = -3.402823466e38f, rate = -k * softplus(lam);
    return rate < most ? most : rate;
}

// a = exp(l), l <= 0, and 1 - a. Near a = 1 the recurrence remembers 1 / (1 - a) steps, and an error
// of the exponential would add up over them: with w = -l below 1/16, 1 - exp(-w) comes from its
// series (the first term left out is w^5 / 720 of it, 1e-9) and a is one minus that, right to half a
// unit; above, 1 - a loses at most four bits. Every kernel takes its decays from here, so that an
// adjoint passes over the same ones as the state.
struct Decay {
    float a, rest;
};
SSD_DEVICE Decay decay_of(float l)
{
    const float w = -l;
    float s = 1.f / 120.f;
    s = s * w - 1.f / 24.f;
    s = s * w + 1.f / 6.f;
    s = s * w - 0.5f;
    s = s * w + 1.f;
    s = s * w;
    const float e = hw_exp2(kLog2e * l);
    const bool near = w < 0.0625f;
    return {near ? 1.f - s : e, near ? s : 1.f - e};
}

// The gates of one value. nk: decay_rate; 1 - a^2 is (1 - a) (1 + a).
struct Gates {
    float i, r, l, a, m;
};
SSD_DEVICE Gates gates(float gi, float gr, float nk)
{
    Gates g;
    g.i = sigmoid(gi);
    g.r = sigmoid(gr);
    g.l = nk * g.r;
    const Decay d = decay_of(g.l);
    g.a = d.a;
    g.m = hw_sqrt(d.rest * (1.f + d.a));
    return g;
}

// Where a workgroup works: sequence, segment, and this lane's channels.
template <int CH>
struct GatedPlace {
    int64_t b;
    int seg, c0;              // first channel; a lane past the last channel reads channel 0
    bool live;                // whether the lane has channels: all CH of them (C is a multiple of CH)
    int t0, t1, lim;          // the segment's tokens; the first of them that is padding (or t1)
};
template <int CH>
SSD_DEVICE GatedPlace<CH> gated_place(const GatedParams &p)
{
    GatedPlace<CH> g;
    const int64_t id = block_id();
    const int64_t rest = id / p.blocks;
    const int blk = (int)(id - rest * p.blocks);
    g.b = rest / p.launched;
    g.seg = (int)(rest - g.b * p.launched) + p.seg_first;
    g.c0 = blk * 64 * CH + (thread_id() & 63) * CH;
    g.live = g.c0 < p.C;
    g.c0 = g.live ? g.c0 : 0;
    g.t0 = g.seg * p.seg_tokens;
    g.t1 = g.t0 + p.seg_tokens < p.T ? g.t0 + p.seg_tokens : p.T;
    g.lim = g.t1;
    if (p.lengths) {
        int len = uniform_i(p.lengths[g.b]);
        len = len > 0 ? len : 0;  // lim - 1 below has to be a number
        g.lim = len < g.t1 ? len : g.t1;
    }
    return g;
}

// One token's channels of this lane. A token that is padding or past the segment reads the last
// one that is not (the segment's first, if none is, padding itself): its values are replaced
// afterwards.
template <int T, int CH>
SSD_DEVICE GatedRaw<T, CH> gated_read(const void *p, int64_t stride, const GatedParams &q,
                                      const GatedPlace<CH> &g, int t)
{
    t = t < g.lim ? t : g.lim - 1;
    t = t > g.t0 ? t : g.t0;
    const char *row = (const char *)p + (g.b * q.T + t) * stride * ElemSize<T>::value;
    return gated_load<T, CH>(row + (uint32_t)g.c0 * ElemSize<T>::value);
}
template <int T, int CH>
SSD_DEVICE void gated_write(void *p, const GatedParams &q, const GatedPlace<CH> &g, int t,
                            const float (&v)[CH])
{
    char *row = (char *)p + (g.b * q.T + t) * q.C * ElemSize<T>::value;
    if (g.live)
        gated_store<T, CH>(row + (uint32_t)g.c0 * ElemSize<T>::value, v);
}

// Folds `count` segments' pairs (number first, first + step, ...) onto carry: every wave folds its
// share of them, then all fold the waves' pairs from shared memory. One wait for memory and not
// one per segment.
template <int CH, int WAVES, int PARTS>
SSD_DEVICE void gated_fold(const GatedParams &p, const GatedPlace<CH> &g, int first, int step, int count,
                           float (&slots)[WAVES][PARTS][64 * CH], float (&carry)[CH])
{
    const int lane = thread_id() & 63;
    const int wave = wave_id();
    const int share = (count + WAVES - 1) / WAVES;
    const int end = (wave + 1) * share < count ? (wave + 1) * share : count;
    float A[CH], U[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        A[c] = 1.f;
        U[c] = 0.f;
    }
#pragma unroll 4
    for (int i = wave * share; i < end; ++i) {
        const float *q = p.seg + ((g.b * p.segments + first + step * i) * 2) * (int64_t)p.C + g.c0;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const float a = q[c];
            A[c] *= a;
            U[c] = a * U[c] + q[p.C + c];
        }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        slots[wave][0][c * 64 + lane] = A[c];
        slots[wave][1][c * 64 + lane] = U[c];
    }
    block_sync();
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
#pragma unroll
        for (int c = 0; c < CH; ++c)
            carry[c] = slots[w][0][c * 64 + lane] * carry[c] + slots[w][1][c * 64 + lane];
}

// SUMMARY: only the segment's (A, U) is wanted, for all but the last segment. That pass walks
// over its tiles from the last to the first: what it read last, and the caches behind the
// compute units still hold, is what the pass after it reads first. The last segment's
// slot takes a copy of the entering state instead, so that final_state may be initial_state:
// the pass that writes it then reads the copy. Otherwise the outputs.
template <int T, int CH, int WAVES, int STEPS, bool SUMMARY>
SSD_KERNEL(64 * WAVES) void gated_scan_kernel(GatedParams p)
{
    constexpr int TILE = WAVES * STEPS;
    SSD_LDS float pairs[2][WAVES][2][64 * CH];
    const int lane = thread_id() & 63;
    const int wave = wave_id();
    const GatedPlace<CH> g = gated_place<CH>(p);
    float nk[CH], carry[CH], decay[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        nk[c] = g.live ? decay_rate(p.k, p.lam[g.c0 + c]) : 0.f;
        carry[c] = 0.f;
        decay[c] = 1.f;
        if (g.live) {
            float *copy = p.seg + (g.b * p.segments + p.segments - 1) * 2 * (int64_t)p.C + g.c0 + c;
            const float *from = p.init ? p.init + g.b * p.C + g.c0 + c : nullptr;
            if (SUMMARY) {
                if (g.seg == 0 && wave == 0)
                    *copy = from ? *from : 0.f;
            } else {
                carry[c] = p.segments > 1 ? *copy : from ? *from : 0.f;
            }
        }
    }
    if (!SUMMARY && g.seg > 0)  // the slots are the second tile's: its writes are a barrier away
        gated_fold<CH, WAVES>(p, g, 0, 1, g.seg, pairs[1], carry);
    GatedRaw<T, CH> rx[STEPS], ri[STEPS], rr[STEPS];
    auto fetch = [&](int t) {  // this wave's tokens from t on
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            rx[k] = gated_read<T, CH>(p.x, p.x_stride, p, g, t + k);
            ri[k] = gated_read<T, CH>(p.gi, p.gi_stride, p, g, t + k);
            rr[k] = gated_read<T, CH>(p.gr, p.gr_stride, p, g, t + k);
        }
    };
    const int tiles = (g.t1 - g.t0 + TILE - 1) / TILE;
    constexpr int NEXT = SUMMARY ? -TILE : TILE;
    int t = g.t0 + (SUMMARY ? (tiles - 1) * TILE : 0) + wave * STEPS;
    fetch(t);
    int parity = 0;
    for (int tile = 0; tile < tiles; ++tile, t += NEXT, parity ^= 1) {
        const bool whole = t + STEPS <= g.lim;
        float a[STEPS][CH], u[STEPS][CH], A[CH], U[CH];
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const Gates q = gates(gated_value<T, CH>(ri[k], c), gated_value<T, CH>(rr[k], c), nk[c]);
                a[k][c] = q.a;
                u[k][c] = q.m * q.i * gated_value<T, CH>(rx[k], c);
            }
        if (!whole) {  // padding and what lies past the segment: a step that changes nothing
#pragma unroll
            for (int k = 0; k < STEPS; ++k)
                if (t + k >= g.lim)
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        a[k][c] = 1.f;
                        u[k][c] = 0.f;
                    }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            A[c] = a[0][c];
            U[c] = u[0][c];
#pragma unroll
            for (int k = 1; k < STEPS; ++k) {
                A[c] *= a[k][c];
                U[c] = a[k][c] * U[c] + u[k][c];
            }
        }
        if (tile + 1 < tiles)
            fetch(t + NEXT);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            pairs[parity][wave][0][c * 64 + lane] = A[c];
            pairs[parity][wave][1][c * 64 + lane] = U[c];
        }
        block_sync();
        if (SUMMARY) {  // this tile comes before what is in (decay, carry)
#pragma unroll
            for (int w = WAVES - 1; w >= 0; --w)
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    carry[c] += decay[c] * pairs[parity][w][1][c * 64 + lane];
                    decay[c] *= pairs[parity][w][0][c * 64 + lane];
                }
        } else {
            float mine[CH];
#pragma unroll
            for (int w = 0; w < WAVES; ++w)
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    if (w == 0 || w == wave)
                        mine[c] = carry[c];
                    carry[c] = pairs[parity][w][0][c * 64 + lane] * carry[c] + pairs[parity][w][1][c * 64 + lane];
                }
            if (p.states && t % kGatedChunk == 0 && t < g.t1)
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    if (g.live)
                        p.states[(g.b * ((p.T + kGatedChunk - 1) / kGatedChunk) + t / kGatedChunk) * p.C + g.c0 + c] = mine[c];
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
                float out[CH];
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    mine[c] = a[k][c] * mine[c] + u[k][c];
                    out[c] = whole || t + k < g.lim ? mine[c] : 0.f;
                }
                if (whole || t + k < g.t1)
                    gated_write<T, CH>(p.h, p, g, t + k, out);
            }
        }
    }
    if (wave != 0)
        return;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (!g.live)
            continue;
        if (SUMMARY) {
            float *q = p.seg + ((g.b * p.segments + g.seg) * 2) * (int64_t)p.C + g.c0 + c;
            q[0] = decay[c];
            q[p.C] = carry[c];
        } else if (p.final_state && g.seg == p.segments - 1) {
            p.final_state[g.b * p.C + g.c0 + c] = carry[c];
        }
    }
}

// A few tokens per sequence: a lane per channel walks over them, nothing to fold. 64 sequences of
// one token, C = 1024 in bfloat16: 3.4 us, a launch and two trips to memory.
constexpr int kGatedWalk = 32;     // within the first chunk

template <int T>
SSD_KERNEL(64) void gated_step_kernel(GatedParams p)
{
    const GatedPlace<1> g = gated_place<1>(p);
    if (!g.live)
        return;
    const float nk = decay_rate(p.k, p.lam[g.c0]);
    float h = p.init ? p.init[g.b * p.C + g.c0] : 0.f;
    if (p.states)
        p.states[g.b * p.C + g.c0] = h;
    for (int t = 0; t < p.T; ++t) {
        const bool in = t < g.lim;
        if (in) {
            const Gates q = gates(gated_value<T, 1>(gated_read<T, 1>(p.gi, p.gi_stride, p, g, t), 0),
                                  gated_value<T, 1>(gated_read<T, 1>(p.gr, p.gr_stride, p, g, t), 0), nk);
            h = q.a * h + q.m * q.i * gated_value<T, 1>(gated_read<T, 1>(p.x, p.x_stride, p, g, t), 0);
        }
        const float out[1] = {in ? h : 0.f};
        gated_write<T, 1>(p.h, p, g, t, out);
    }
    if (p.final_state)
        p.final_state[g.b * p.C + g.c0] = h;
}

// The adjoint that enters a segment from its right, without the segments after it: each
// segment's (A, V), Q -> A Q + V, where Q_t = a_t g_t is what token t hands to the one
// before it. SUMMARY of the backward: reads the decay gate and gh only.
template <int T, int CH, int WAVES, int STEPS>
SSD_KERNEL(64 * WAVES) void gated_bwd_summary_kernel(GatedParams p)
{
    constexpr int TILE = WAVES * STEPS;
    SSD_LDS float pairs[2][WAVES][2][64 * CH];
    const int lane = thread_id() & 63;
    const int wave = wave_id();
    const GatedPlace<CH> g = gated_place<CH>(p);
    float nk[CH], carry[CH], decay[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        nk[c] = g.live ? decay_rate(p.k, p.lam[g.c0 + c]) : 0.f;
        carry[c] = 0.f;
        decay[c] = 1.f;
    }
    GatedRaw<T, CH> rr[STEPS], rh[STEPS];
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            rr[k] = gated_read<T, CH>(p.gr, p.gr_stride, p, g, t + k);
            rh[k] = gated_read<T, CH>(p.gh, p.C, p, g, t + k);
        }
    };
    const int tiles = (g.t1 - g.t0 + TILE - 1) / TILE;
    fetch(g.t0 + (tiles - 1) * TILE + wave * STEPS);
    int parity = 0;
    for (int i = tiles - 1; i >= 0; --i, parity ^= 1) {
        const int t = g.t0 + i * TILE + wave * STEPS;
        float A[CH], V[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            A[c] = 1.f;
            V[c] = 0.f;
        }
#pragma unroll
        for (int k = STEPS - 1; k >= 0; --k) {
            const bool in = t + k < g.lim;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const float a = in ? decay_of(nk[c] * sigmoid(gated_value<T, CH>(rr[k], c))).a : 1.f;
                A[c] *= a;
                V[c] = a * (V[c] + (in ? gated_value<T, CH>(rh[k], c) : 0.f));
            }
        }
        if (i > 0)
            fetch(t - TILE);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            pairs[parity][wave][0][c * 64 + lane] = A[c];
            pairs[parity][wave][1][c * 64 + lane] = V[c];
        }
        block_sync();
#pragma unroll
        for (int w = WAVES - 1; w >= 0; --w)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const float wa = pairs[parity][w][0][c * 64 + lane];
                carry[c] = wa * carry[c] + pairs[parity][w][1][c * 64 + lane];
                decay[c] *= wa;
            }
    }
    if (wave != 0)
        return;
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if (g.live) {
            float *q = p.seg + ((g.b * p.segments + g.seg) * 2) * (int64_t)p.C + g.c0 + c;
            q[0] = decay[c];
            q[p.C] = carry[c];
        }
}

// The gradients, tile by tile from the last to the first. In bfloat16 116 registers with two channels
// per lane, so that a compute unit holds one workgroup of 16 waves; workgroups of 8 waves, and
// loads issued earlier, gained nothing. A tile is one chunk (64 tokens):
// its entering state was stored, so the states inside it come from a fold to the right and
// the adjoints from a fold to the left, over the same products A.
template <int T, int CH, int WAVES>
SSD_KERNEL(64 * WAVES) void gated_scan_bwd_kernel(GatedParams p)
{
    constexpr int STEPS = kGatedChunk / WAVES;  // a tile is a chunk
    SSD_LDS float pairs[2][WAVES][3][64 * CH];
    const int lane = thread_id() & 63;
    const int wave = wave_id();
    const GatedPlace<CH> g = gated_place<CH>(p);
    const int64_t chunks = (p.T + kGatedChunk - 1) / kGatedChunk;
    float nk[CH], carry[CH], sum_e[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        nk[c] = g.live ? decay_rate(p.k, p.lam[g.c0 + c]) : 0.f;
        carry[c] = p.gfinal && g.live ? p.gfinal[g.b * p.C + g.c0 + c] : 0.f;
        sum_e[c] = 0.f;
    }
    if (g.seg < p.segments - 1)  // the slots are the second tile's: its writes are a barrier away
        gated_fold<CH, WAVES>(p, g, p.segments - 1, -1, p.segments - 1 - g.seg, pairs[1], carry);
    GatedRaw<T, CH> rx[STEPS], ri[STEPS], rr[STEPS], rh[STEPS];
    float enter[CH];
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            rx[k] = gated_read<T, CH>(p.x, p.x_stride, p, g, t + k);
            ri[k] = gated_read<T, CH>(p.gi, p.gi_stride, p, g, t + k);
            rr[k] = gated_read<T, CH>(p.gr, p.gr_stride, p, g, t + k);
            rh[k] = gated_read<T, CH>(p.gh, p.C, p, g, t + k);
        }
    };
    auto fetch_state = [&](int tile) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            enter[c] = g.live ? p.chunk_states[(g.b * chunks + tile / kGatedChunk) * p.C + g.c0 + c] : 0.f;
    };
    const int last = g.t0 + (g.t1 - g.t0 - 1) / kGatedChunk * kGatedChunk;
    fetch(last + wave * STEPS);
    fetch_state(last);
    int parity = 0;
    for (int tile = last; tile >= g.t0; tile -= kGatedChunk, parity ^= 1) {
        const int t = tile + wave * STEPS;
        // i, r, a, m of each value; x and gh stay as they were loaded, l is nk r again
        float vi[STEPS][CH], vr[STEPS][CH], va[STEPS][CH], vm[STEPS][CH];
        GatedRaw<T, CH> x[STEPS], gh[STEPS];
        float before[CH], A[CH], U[CH], V[CH];
        const bool whole = t + STEPS <= g.lim;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            x[k] = rx[k];
            gh[k] = rh[k];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const Gates q = gates(gated_value<T, CH>(ri[k], c), gated_value<T, CH>(rr[k], c), nk[c]);
                vi[k][c] = q.i;
                vr[k][c] = q.r;
                va[k][c] = q.a;
                vm[k][c] = q.m;
            }
        }
        if (!whole) {  // padding and what lies past the segment: nothing goes in, a = 1, l = m = 0
#pragma unroll
            for (int k = 0; k < STEPS; ++k)
                if (t + k >= g.lim) {
                    x[k] = GatedRaw<T, CH>{};
                    gh[k] = GatedRaw<T, CH>{};
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        vi[k][c] = vr[k][c] = vm[k][c] = 0.f;
                        va[k][c] = 1.f;
                    }
                }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            before[c] = enter[c];
            A[c] = va[0][c];
            U[c] = vm[0][c] * vi[0][c] * gated_value<T, CH>(x[0], c);
            V[c] = 0.f;
#pragma unroll
            for (int k = 1; k < STEPS; ++k) {
                A[c] *= va[k][c];
                U[c] = va[k][c] * U[c] + vm[k][c] * vi[k][c] * gated_value<T, CH>(x[k], c);
            }
#pragma unroll
            for (int k = STEPS - 1; k >= 0; --k)
                V[c] = va[k][c] * (V[c] + gated_value<T, CH>(gh[k], c));
        }
        if (tile - kGatedChunk >= g.t0) {
            fetch(t - kGatedChunk);
            fetch_state(tile - kGatedChunk);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            pairs[parity][wave][0][c * 64 + lane] = A[c];
            pairs[parity][wave][1][c * 64 + lane] = U[c];
            pairs[parity][wave][2][c * 64 + lane] = V[c];
        }
        block_sync();
        for (int w = 0; w < wave; ++w)
#pragma unroll
            for (int c = 0; c < CH; ++c)
                before[c] = pairs[parity][w][0][c * 64 + lane] * before[c] + pairs[parity][w][1][c * 64 + lane];
        float right[CH];  // a g of the token after this wave's last
#pragma unroll
        for (int w = WAVES - 1; w >= 0; --w)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (w == WAVES - 1 || w == wave)
                    right[c] = carry[c];
                carry[c] = pairs[parity][w][0][c * 64 + lane] * carry[c] + pairs[parity][w][2][c * 64 + lane];
            }
        float hb[STEPS][CH];
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                hb[k][c] = before[c];
                before[c] = va[k][c] * before[c] + vm[k][c] * vi[k][c] * gated_value<T, CH>(x[k], c);
            }
#pragma unroll
        for (int k = STEPS - 1; k >= 0; --k) {
            float gx[CH], ggi[CH], ggr[CH], e[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const float a = va[k][c], m = vm[k][c], i = vi[k][c], r = vr[k][c];
                const float l = nk[c] * r, xv = gated_value<T, CH>(x[k], c);
                const float gt = gated_value<T, CH>(gh[k], c) + right[c];
                right[c] = a * gt;
                const float ratio = m > 0.f ? l * hw_rcp(m) : 0.f;
                const float gi = gt * i;
                e[c] = right[c] * l * hb[k][c] - gi * xv * (a * a * ratio);  // a l first: it is bounded
                gx[c] = gi * m;
                ggi[c] = gx[c] * xv * (1.f - i);
                ggr[c] = e[c] * (1.f - r);
            }
            if (!whole) {
                if (t + k >= g.t1)
                    continue;
                if (t + k >= g.lim)  // padding, whatever adjoint passes over it
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        gx[c] = ggi[c] = ggr[c] = e[c] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < CH; ++c)
                sum_e[c] += e[c];
            gated_write<T, CH>(p.gx, p, g, t + k, gx);
            gated_write<T, CH>(p.ggi, p, g, t + k, ggi);
            gated_write<T, CH>(p.ggr, p, g, t + k, ggr);
        }
    }
    // sum over the waves, in wave order (the slot that the last tile did not use)
#pragma unroll
    for (int c = 0; c < CH; ++c)
        pairs[parity][wave][0][c * 64 + lane] = sum_e[c];
    block_sync();
    if (wave != 0)
        return;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (!g.live)
            continue;
        float e = 0.f;
        for (int w = 0; w < WAVES; ++w)
            e += pairs[parity][w][0][c * 64 + lane];
        p.part[(g.b * p.segments + g.seg) * p.C + g.c0 + c] = e;
        if (p.ginit && g.seg == 0)
            p.ginit[g.b * p.C + g.c0 + c] = carry[c];
    }
}

// g_lam = sigmoid(lam) / softplus(lam) * sum of the shares, in their order (the ratio goes to
// 1, and is 1 where lam is so low that both are 0). 64 channels per workgroup, 16 waves.
SSD_KERNEL(64 * 16) void gated_lam_kernel(const float *part, int rows, int C, const float *lam, float *out)
{
    SSD_LDS float sums[16][64];
    const int lane = thread_id() & 63;
    const int wave = wave_id();
    const int c = (int)block_id() * 64 + lane;
    float acc = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int r = wave; r < rows; r += 16)
            acc += part[(int64_t)r * C + c];
    }
    sums[wave][lane] = acc;
    block_sync();
    if (wave == 0 && c < C) {
        float t = 0.f;
        for (int i = 0; i < 16; ++i)
            t += sums[i][lane];
        const float v = lam[c];
        const float e = expf(-fabsf(v));  // of -|v|: exp(-v) would be infinite from lam = -89 down
        const float sp = softplus(v);
        out[c] = t * (sp > 0.f ? (v < 0.f ? e : 1.f) / (1.f + e) / sp : 1.f);
    }
}

// final = init (or zeros): T = 0.
SSD_KERNEL(256) void gated_copy_kernel(const float *init, float *out, int64_t n)
{
    const int64_t step = grid_blocks() * 256;
    for (int64_t e = block_id() * 256 + thread_id(); e < n; e += step)
        out[e] = init ? init[e] : 0.f;
}

}  // namespace ssd
