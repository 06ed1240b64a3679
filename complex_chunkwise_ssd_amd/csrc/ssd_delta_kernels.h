// ssd_delta_kernels.h -- the gated delta rule. Per sequence and value head, with the state S
// (Dk x Dv, float32) and a = exp(g),
//     u_t = beta_t (v_t - a_t S_{t-1}^T k_t)     S_t = a_t S_{t-1} + k_t u_t^T     o_t = scale S_t^T q_t
// For a chunk of 64 tokens with G the running sum of g in it, D_ij = exp(G_i - G_j) for i >= j and
// A_ij = beta_i D_ij k_i.k_j for i > j:
//     (I + A) U = R = beta (V - e^G K S)         O = scale (e^G Q S + (Q K^T o D) U)
//     S' = e^{G_C} S + (e^{G_C - G} K)^T U
// The columns of S, V, U and O (over Dv) do not meet, so a wave walks over the chunks with 16 columns
// of the state in its registers. The 64 x 64 system is solved in two blocks of 32 with their own
// inverses T_00 and T_11 (blocks of 16 by substitution, which is stable whatever the keys, the rest by
// products), which the walks and the gradients' kernel form chunk by chunk; only with few heads does a kernel
// before the walk make those of a whole range of chunks:
//     U_0 = T_00 R_0       U_1 = T_11 (R_1 - A_10 U_0)
//
// Backwards, for the gradients of O and of S':
//     dU = P^T dO + e^{G_C - G} K dS'      with P = scale Q K^T o D
//     dR_1 = T_11^T dU_1    dR_0 = T_00^T (dU_0 - A_10^T dR_1)
//     dS = e^{G_C} dS' + scale Q^T e^G dO - K^T beta e^G dR             (one walk, again by columns)
//     dV = beta dR    dP = scale (dO U^T) o D    E = -(dR U^T) o beta D below the diagonal
//     dQ = scale e^G dO S^T + dP K
//     reads  = E K - beta e^G dR S^T             what reaches k_i as the key that reads
//     writes = dP^T Q + E^T K + e^{G_C - G} U dS'^T          ... as the key that writes
//     dK = reads + writes    dbeta = dR . (V - e^G K S) - sum_j (dR U^T) o D o K K^T
//     dG_i = q_i.dq_i + k_i.(reads_i - writes_i), and <S', dS'> more at the chunk's last token,
//     dg_t = sum over i >= t of dG_i            (every chunk by itself, once dS' is known)
//
// G is summed in float64: D is the exponential of a difference, and float32 sums over a token that
// forgets (g = -300, say) would leave nothing of the decays behind it. g below -1000 counts as -1000,
// where exp is 0. Everything else is float32 (see ssd_split.h), rounded once as it is stored.
#pragma once

#include <ssd_delta_device.h>
#include <ssd_split.h>

namespace ssd {

constexpr int kDeltaChunk = 64;
constexpr int kDeltaFrags = 6;            // operand tiles of the solve: (span, tile, span of k)

struct DeltaParams {
    const void *q, *k, *v;                // (B, T, heads, D), tokens *_stride elements apart
    const float *g, *beta;                // (B, T, Hv)
    const float *init;                    // nullable: (B, Hv, Dk, Dv)
    const int *lengths;                   // nullable: (B)
    void *o;                              // (B, T, Hv, Dv)
    float *final_state;                   // nullable: (B, Hv, Dk, Dv)
    float *states;                        // nullable: (B, chunks, Hv, Dk, Dv), the state entering each chunk
    // backward
    const float *chunk_states;
    const void *go;                       // (B, T, Hv, Dv)
    const float *gfinal;                  // nullable: (B, Hv, Dk, Dv)
    void *gq, *gk, *gv;                   // as q, k, v, dense
    float *gg, *gbeta;                    // (B, T, Hv)
    float *ginit;                         // nullable: (B, Hv, Dk, Dv)
    float *wq, *wk;                       // (B, T, Hv, Dk): dQ and dK by value heads, where they share keys
    float *gs;                            // (B, Hv, chunks, Dk, Dv): dS' of each chunk
    float *gr;                            // (B, Hv, chunks, 64, Dv): dR
    int64_t q_stride, k_stride, v_stride;
    int B, T, Hk, Hv, Dk, Dv, chunks;
    int columns;                          // column blocks of a head
    // few heads
    v4u *pack;                            // (B, Hv, chunk_to - chunk_from) times what a chunk is packed into
    float *carry;                         // (B, Hv, Dk, Dv): the state between two ranges of chunks
    int chunk_from, chunk_to;
    float scale;
};

// ------------------------------------------------------------------ operands

template <int T>
struct DeltaElem;
template <>
struct DeltaElem<kBF16> {
    typedef uint16_t type;
    static constexpr int parts = 1, pad = 8;
};
template <>
struct DeltaElem<kF32> {
    typedef float type;
    static constexpr int parts = 3, pad = 4;
};
constexpr int kParts = 3;

// The lane's eight neighbours at p in shared memory.
SSD_DEVICE Parts<1> lds_operand(const uint16_t *p)
{
    Parts<1> r;
    r.p[0] = *(const v4u *)p;
    return r;
}
SSD_DEVICE Parts<3> lds_operand(const float *p)
{
    const v4f a = *(const v4f *)p, b = *(const v4f *)(p + 4);
    return split_tiles<3>(a, b);
}

template <int T>
SSD_DEVICE void lds_values(const typename DeltaElem<T>::type *p, float (&v)[8])
{
    Raw8<T> raw;
#pragma unroll
    for (int i = 0; i < (T == kBF16 ? 1 : 2); ++i)
        raw.w[i] = *(const v4u *)((const char *)p + 16 * i);
    unpack8<T>(raw, v);
}

// Which six operand tiles a lower (or upper) triangle of spans has: the first two and the last two are those of the
// blocks on the diagonal. The parts of a tile lie one after the other.
SSD_DEVICE int frag_of(int s, int h, int t) { return s == 0 ? h : 2 + 2 * t + h; }          // t <= s
SSD_DEVICE int frag_of_upper(int s, int h, int t) { return s == 1 ? 4 + h : 2 * t + h; }    // t >= s

// Running sums over a wave's lanes in float64.
template <int n>
SSD_DEVICE double row_shr_d(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)row_shr_i<n>((int)(uint32_t)u);
    const uint32_t hi = (uint32_t)row_shr_i<n>((int)(uint32_t)(u >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
SSD_DEVICE double lane_read_d(double v, int src)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)lane_read_i((int)(uint32_t)u, src);
    const uint32_t hi = (uint32_t)lane_read_i((int)(uint32_t)(u >> 32), src);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
SSD_DEVICE double wave_scan_d(double v)
{
    v += row_shr_d<1>(v);
    v += row_shr_d<2>(v);
    v += row_shr_d<4>(v);
    v += row_shr_d<8>(v);
    const int row = (thread_id() & 63) >> 4;
    const double a = lane_read_d(v, 15), b = lane_read_d(v, 31), c = lane_read_d(v, 47);
    return v + (row == 0 ? 0. : row == 1 ? a : row == 2 ? a + b : a + b + c);
}

// A token's log decay in powers of two.
SSD_DEVICE double delta_log2(float g) { return (g < -1000.f ? -1000. : (double)g) * 1.44269504088896340736; }
// To a unit or two: what the exponent's rounding to float32 takes off (22 units at 2^-125) is made up for.
SSD_DEVICE float delta_exp(double log2)
{
    const float t = (float)log2, low = (float)(log2 - (double)t), e = hw_exp2(t);
    return __builtin_fmaf(e, 0.693147182f * low, e);
}

// What a chunk's decays are, for each of its tokens; read by fours, also from the second of two side by side.
struct alignas(16) DeltaGates {
    double sum[64];      // G, in powers of two
    float since[64];     // e^G
    float left[64];      // e^(G_C - G)
    float beta[64];
    float whole;         // e^G_C
};

// By one wave, lane = token; tokens from n on leave the state as it is.
SSD_DEVICE void delta_gates_of(DeltaGates &s, float g, float beta, int n)
{
    const int t = thread_id() & 63;
    const double sum = wave_scan_d(t < n ? delta_log2(g) : 0.);
    const double last = lane_read_d(sum, 63);
    s.sum[t] = sum;
    s.since[t] = delta_exp(sum);
    s.left[t] = delta_exp(last - sum);
    s.beta[t] = t < n ? beta : 0.f;
    if (t == 0)
        s.whole = delta_exp(last);
}
SSD_DEVICE void delta_gates(DeltaGates &s, const float *g, const float *beta, int64_t at, int step, int n)
{
    const int t = (thread_id() & 63) < n ? thread_id() & 63 : n - 1;
    delta_gates_of(s, g[at + (int64_t)t * step], beta[at + (int64_t)t * step], n);
}

// Rows 0 .. 63 (tokens, zeros from n on; n > 0) by COLS columns (zeros from D on) of a matrix in memory, on
// their way into shared memory by NT threads: each takes blocks of 4 x 4. Loads are made without branches, at
// the nearest place that exists, and what lies outside is cleared afterwards: a branch around a load would make
// each wait for its own. Offsets within a chunk are 32 bits wide.
template <int T, int COLS, int NT>
struct Blocks {
    static constexpr int units = 4 * COLS / NT;
    static_assert(4 * COLS % NT == 0, "every thread has as many blocks");
    typename DeltaElem<T>::type v[units][4][4];
};
template <int COLS, int NT>
SSD_DEVICE int block_col(int thread, int i) { return 4 * ((thread + NT * i) % (COLS / 4)); }
template <int COLS, int NT>
SSD_DEVICE int block_row(int thread, int i) { return 4 * ((thread + NT * i) / (COLS / 4)); }

template <int T, int COLS, int NT>
SSD_DEVICE void blocks_load(Blocks<T, COLS, NT> &d, const void *src, int stride, int D, int n)
{
    typedef typename DeltaElem<T>::type E;
    const char *x = (const char *)src;
    const uint32_t step = opaque_uniform((uint32_t)stride * sizeof(E));
    const int thread = (int)opaque((uint32_t)thread_id());
#pragma unroll
    for (int i = 0; i < d.units; ++i) {
        const int f = block_col<COLS, NT>(thread, i), t = block_row<COLS, NT>(thread, i);
        if (D % 4 == 0 && n == 64) {
            const uint32_t off = (uint32_t)t * step + (uint32_t)(f < D ? f : 0) * sizeof(E);
#pragma unroll
            for (int a = 0; a < 4; ++a)
                __builtin_memcpy(d.v[i][a], x + (off + a * step), sizeof(d.v[i][a]));
        } else if (D % 4 == 0) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
                __builtin_memcpy(d.v[i][a], x + ((uint32_t)(t + a < n ? t + a : n - 1) * step +
                                                 (uint32_t)(f < D ? f : 0) * sizeof(E)), sizeof(d.v[i][a]));
        } else {
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    __builtin_memcpy(&d.v[i][a][b], x + ((uint32_t)(t + a < n ? t + a : n - 1) * step +
                                                         (uint32_t)(f + b < D ? f + b : D - 1) * sizeof(E)), sizeof(E));
        }
    }
}
// Into rows (RS apart) and / or their transpose.
template <int T, int COLS, int NT, bool ROWS, bool TURNED>
SSD_DEVICE void blocks_store(Blocks<T, COLS, NT> &d, int D, int n, typename DeltaElem<T>::type *rows,
                             typename DeltaElem<T>::type *turned)
{
    typedef typename DeltaElem<T>::type E;
    constexpr int pad = DeltaElem<T>::pad, RS = COLS + pad, TS = 64 + pad;
    const int thread = (int)opaque((uint32_t)thread_id());
#pragma unroll
    for (int i = 0; i < d.units; ++i) {
        const int f = block_col<COLS, NT>(thread, i), t = block_row<COLS, NT>(thread, i);
        E (&v)[4][4] = d.v[i];
        if (n < 64 || D < COLS) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    v[a][b] = t + a < n && f + b < D ? v[a][b] : (E)0;
        }
        if (ROWS)
#pragma unroll
            for (int a = 0; a < 4; ++a)
                __builtin_memcpy(__builtin_assume_aligned(rows + (t + a) * RS + f, sizeof(v[a])), v[a], sizeof(v[a]));
        if (TURNED)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const E w[4] = {v[0][b], v[1][b], v[2][b], v[3][b]};
                __builtin_memcpy(__builtin_assume_aligned(turned + (f + b) * TS + t, sizeof(w)), w, sizeof(w));
            }
    }
}

SSD_DEVICE int delta_valid(const DeltaParams &p, int b)  // tokens of a sequence
{
    if (!p.lengths)
        return p.T;
    const int n = p.lengths[b];
    return n < 0 ? 0 : n < p.T ? n : p.T;
}
SSD_DEVICE int delta_chunk_tokens(int length, int chunk)
{
    const int n = length - chunk * kDeltaChunk;
    return n < 0 ? 0 : n < kDeltaChunk ? n : kDeltaChunk;
}

// --------------------------------------------------------- a chunk's triangle

// Tile (tx, ty) of X Y^T: rows (lanes' components) of X, columns of Y, in tiles of 16 as they lie.
template <int T, int KP>
SSD_DEVICE v4f delta_tile(const typename DeltaElem<T>::type *x, int tx, const typename DeltaElem<T>::type *y, int ty)
{
    constexpr int RS = 32 * KP + DeltaElem<T>::pad;
    const int l = thread_id() & 15, q = (thread_id() & 63) >> 4;
    v4f c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KP; ++s)
        c = mm<kParts>(lds_operand(x + (16 * tx + l) * RS + 32 * s + 8 * q),
                       lds_operand(y + (16 * ty + l) * RS + 32 * s + 8 * q), c);
    return c;
}

template <int N>
SSD_DEVICE Parts<N> frag_operand(const v4u *frags, int f)
{
    Parts<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i)
        r.p[i] = frags[(f * N + i) * 64 + (thread_id() & 63)];
    return r;
}

// An element as it lies in memory, and its value: what is loaded ahead is kept as it is, since a conversion
// waits for it.
template <int T>
SSD_DEVICE uint32_t delta_raw(const typename DeltaElem<T>::type *p)
{
    if (T == kBF16) {
        uint16_t u;
        __builtin_memcpy(&u, p, 2);
        return u;
    }
    uint32_t u;
    __builtin_memcpy(&u, p, 4);
    return u;
}
template <int T>
SSD_DEVICE float delta_value(uint32_t raw) { return u2f(T == kBF16 ? raw << 16 : raw); }

template <int T>
SSD_DEVICE float delta_load(const typename DeltaElem<T>::type *p)
{
    if (T == kBF16) {
        uint16_t u;
        __builtin_memcpy(&u, p, 2);
        return u2f((uint32_t)u << 16);
    }
    float v;
    __builtin_memcpy(&v, p, 4);
    return v;
}
template <int T>
SSD_DEVICE void delta_store(typename DeltaElem<T>::type *p, float v)
{
    if (T == kBF16) {
        const uint16_t u = cvt_bf16(v);
        __builtin_memcpy(p, &u, 2);
    } else {
        __builtin_memcpy(p, &v, 4);
    }
}

// ------------------------------------------------------------- the walk over chunks

constexpr int kPairStride = 36;

// The block of 32 on the diagonal that becomes T_00 or T_11 (float32, transposed) stands where their operand tiles will.
SSD_DEVICE float *pair_block(v4u *tri, int pair) { return (float *)(tri + 4 * pair * kParts * 64); }
static_assert(32 * kPairStride * 4 <= 2 * kParts * 64 * 16, "a block fits where its tiles come to stand");

// Four neighbours (i, j .. j + 3) of a 64 x 64 matrix into its operand tiles, in N parts.
template <int N>
SSD_DEVICE void frag_store(v4u *frags, int f, int i, int j, v4f w)
{
    const float v[8] = {w[0], w[1], w[2], w[3], 0.f, 0.f, 0.f, 0.f};
    const Parts<N> parts = split8<N>(v);
    const int lane = 16 * (j >> 3 & 3) + 4 * (i >> 3 & 3) + (i & 3);
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const v2u half = {parts.p[e][0], parts.p[e][1]};
        *(v2u *)((char *)&frags[(f * N + e) * 64 + lane] + 2 * (j & 7)) = half;
    }
}

// A chunk's triangle and P, by all waves, in tiles of 16: A = beta D o K K^T below the diagonal and
// P = scale Q K^T o D. Of the two 32 x 32 blocks of I + A on the diagonal the inverses of their own blocks of 16 and
// A between them go where pair_block says; A_10 and P into operand tiles, or, with TURNED, A_10^T and P^T.
// Each of the first four waves has one tile on the diagonal, the others are dealt out so that the first two,
// which finish the inverses afterwards, have the fewest.
template <int T, int KP, int WAVES, bool TURNED>
SSD_DEVICE void delta_tiles(const typename DeltaElem<T>::type *k, const typename DeltaElem<T>::type *q,
                            const DeltaGates &gates, float scale, v4u *tri, v4u *pf)
{
    const int l = thread_id() & 15, quarter = (thread_id() & 63) >> 4, wave = wave_id();
    if (thread_id() < 128)  // above the diagonal of a block of 32 there are zeros
        *(v4f *)(pair_block(tri, wave) + (16 + (4 * quarter + (l >> 2))) * kPairStride + 4 * (l & 3)) = v4f{0.f, 0.f, 0.f, 0.f};
    // off the diagonal: (1,0) (3,2) (2,0) (2,1) (3,0) (3,1); of four waves 2 and 3 take two of them
    const int mine = WAVES == 4 ? (wave < 2 ? 4 + wave : 2 * wave - 4) : (wave < 4 ? 2 + wave : wave - 4);
    const int many = WAVES == 4 ? (wave < 2 ? 1 : 2) : (wave < 2 ? 0 : 1);
    constexpr int most = WAVES == 4 ? 3 : 2;
    int ti[most], tj[most];
    bool has[most];
    v4f kk[most], qk[most];
#pragma unroll
    for (int c = 0; c < most; ++c) {
        const int o = mine + c - 1;
        has[c] = c == 0 ? wave < 4 : c <= many;
        ti[c] = c == 0 ? wave : o == 0 ? 1 : o == 2 || o == 3 ? 2 : 3;
        tj[c] = c == 0 ? wave : o == 1 ? 2 : o == 3 || o == 5 ? 1 : 0;
        if (has[c]) {  // rows j, column i; or rows i, column j
            kk[c] = TURNED ? delta_tile<T, KP>(k, ti[c], k, tj[c]) : delta_tile<T, KP>(k, tj[c], k, ti[c]);
            if (pf)
                qk[c] = TURNED ? delta_tile<T, KP>(q, ti[c], k, tj[c]) : delta_tile<T, KP>(k, tj[c], q, ti[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < most; ++c) {
        if (!has[c])
            continue;
        const int row = 16 * (TURNED ? ti[c] : tj[c]) + 4 * quarter, col = 16 * (TURNED ? tj[c] : ti[c]) + l;
        float *const pair = pair_block(tri, col >> 5);
        const double sum = gates.sum[col];
        v4f a, w;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float d = delta_exp(TURNED ? gates.sum[row + r] - sum : sum - gates.sum[row + r]);
            const int below = TURNED ? row + r - col : col - row - r;  // i - j
            a[r] = c > 0 || below > 0 ? gates.beta[TURNED ? row + r : col] * d * kk[c][r] : 0.f;
            w[r] = pf && (c > 0 || below >= 0) ? scale * d * qk[c][r] : 0.f;
        }
        const int f = TURNED ? frag_of_upper(col >> 5, col >> 2 & 1, row >> 5) : frag_of(col >> 5, col >> 2 & 1, row >> 5);
        if (pf)
            frag_store<kParts>(pf, f, col, row, w);
        if (c == 0) {
            // column l of the block's inverse, in every quarter: each value is taken from all that follow it
            // as soon as it is known; the block's entries reach all lanes as scalars
            float x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
                x[e] = e == l ? 1.f : 0.f;
            v4f minus = -a;
#pragma unroll
            for (int e = 0; e < 15; ++e) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {  // no more scalars at a time than there are
                    float m = minus[r];
                    together(m, x[e]);
                    minus[r] = m;
                }
#pragma unroll
                for (int u = e + 1; u < 16; ++u)
                    x[u] = __builtin_fmaf(TURNED ? lane_read(minus[u & 3], 16 * (u >> 2) + e)
                                                 : lane_read(minus[e & 3], 16 * (e >> 2) + u), x[e], x[u]);
            }
            if (quarter == 0)
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *(v4f *)(pair + (col & 31) * kPairStride + (16 * wave & 16) + e) = v4f{x[e], x[e + 1], x[e + 2], x[e + 3]};
        } else if (ti[c] >> 1 == tj[c] >> 1) {
            if (TURNED)
                *(v4f *)(pair + (col & 31) * kPairStride + (row & 31)) = a;
            else
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    pair[((row & 31) + r) * kPairStride + (col & 31)] = a[r];
        } else {
            frag_store<kParts>(tri, f, col, row, a);
        }
    }
}

// The corner of the inverse of a block of 32 (held transposed), - T_1 A T_0, and the block (with TURNED its transpose)
// into operand tiles, by one wave.
template <bool TURNED>
SSD_DEVICE void delta_invert(int pair, v4u *tri)
{
    float *const block = pair_block(tri, pair);
    const int l = thread_id() & 15, quarter = (thread_id() & 63) >> 4;
    // the transpose's is - T_0^T (A^T T_1^T)
    float *corner = block + 16;  // A^T: rows of the first 16, columns of the second
    const v4f a = *(const v4f *)(corner + l * kPairStride + 4 * quarter);
    const v4f t0 = *(const v4f *)(block + l * kPairStride + 4 * quarter);
    v4f y = {0.f, 0.f, 0.f, 0.f}, z = y;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        y = mfma_16x16x4(a[r], corner[(16 + 4 * quarter + r) * kPairStride + l], y);
#pragma unroll
    for (int r = 0; r < 4; ++r)
        z = mfma_16x16x4(t0[r], -y[r], z);
    wave_lds_sync();
#pragma unroll
    for (int r = 0; r < 4; ++r)
        corner[(4 * quarter + r) * kPairStride + l] = z[r];
    wave_lds_sync();
    float x[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // row i of the operand is column i of what is held
        float (&v)[8] = x[h];
        if (TURNED) {
            const float *row = block + (tile_row(0, l) + 4 * h) * kPairStride + 8 * quarter;
            const v4f lo = *(const v4f *)row, hi = *(const v4f *)(row + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = e < 4 ? lo[e & 3] : hi[e & 3];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = block[8 * quarter * kPairStride + tile_row(0, l) + (e * kPairStride + 4 * h)];
        }
    }
    wave_lds_sync();  // all of the block has been read
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const Parts<kParts> parts = split8<kParts>(x[h]);
        const int f = TURNED ? frag_of_upper(pair, h, pair) : frag_of(pair, h, pair);
#pragma unroll
        for (int e = 0; e < kParts; ++e)
            tri[(f * kParts + e) * 64 + (thread_id() & 63)] = parts.p[e];
    }
}

// The feature that a lane holds in component r of tile i of its state, less 8 q.
SSD_DEVICE constexpr int state_at(int i, int r) { return 32 * (i >> 1) + 4 * (i & 1) + r; }

template <int KP>
SSD_DEVICE void state_store(const v4f (&S)[2 * KP], float *to, int Dk, int Dv)
{
    const uint32_t step = opaque_uniform((uint32_t)Dv * 4);
    const int q8 = (int)opaque(8 * (((uint32_t)thread_id() & 63) >> 4));
    const uint32_t off = (uint32_t)q8 * step;
    char *at = (char *)to;
    if (Dk == 32 * KP) {
#pragma unroll
        for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *(float *)(at + (off + (uint32_t)state_at(i, r) * step)) = S[i][r];
        return;
    }
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (q8 < Dk - state_at(i, r))
                *(float *)(at + (off + (uint32_t)state_at(i, r) * step)) = S[i][r];
}
template <int KP>
SSD_DEVICE void state_fetch(v4f (&S)[2 * KP], const float *from, int Dk, int Dv)
{
    const int q8 = 8 * ((thread_id() & 63) >> 4);
    if (Dk == 32 * KP) {
        const uint32_t step = opaque_uniform((uint32_t)Dv * 4), off = opaque((uint32_t)q8 * step);
#pragma unroll
        for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[i][r] = *(const float *)((const char *)from + (off + (uint32_t)state_at(i, r) * step));
        return;
    }
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[i][r] = from[(uint32_t)(q8 < Dk - state_at(i, r) ? q8 + state_at(i, r) : 0) * (uint32_t)Dv];
}
template <int KP>
SSD_DEVICE void state_mask(v4f (&S)[2 * KP], int Dk)
{
    if (Dk == 32 * KP)
        return;
    const int q8 = 8 * ((thread_id() & 63) >> 4);
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[i][r] = q8 < Dk - state_at(i, r) ? S[i][r] : 0.f;
}
template <int KP>
SSD_DEVICE void state_load(v4f (&S)[2 * KP], const float *from, int Dk, int Dv)
{
    state_fetch<KP>(S, from, Dk, Dv);
    state_mask<KP>(S, Dk);
}

// Waits for a state that is loaded before a walk. Without it the compiler, which counts loads in their order, would wait
// in every chunk as if the state were what was loaded last, and so for all that is on its way to the next one.
template <int N>
SSD_DEVICE void state_arrived(v4f (&S)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
            float a = S[i][r], b = S[i][r + 1];
            together(a, b);
            S[i][r] = a;
            S[i][r + 1] = b;
        }
}

// c += x, span f's share of K S. In float32 all forms of the forward walk sum it span by span, as the one that deals the
// spans out to waves has to: a sequence's results are the same bits in a large batch and alone.
SSD_DEVICE void span_add(v4f &c, v4f x, int f)
{
#pragma unroll
    for (int r = 0; r < 4; ++r)
        c[r] = f == 0 ? x[r] : c[r] + x[r];
}
template <int T, int N>
SSD_DEVICE void span_mm(v4f &c, const Parts<N> &a, const Parts<kParts> &b, int f)
{
    if (T == kF32)
        span_add(c, mm<kParts>(a, b, v4f{0.f, 0.f, 0.f, 0.f}), f);
    else
        c = mm<kParts>(a, b, c);
}

// A workgroup takes 16 WAVES columns of a value head, a wave 16 of them: lane l the column l, and of 2 KP tiles
// the features 32 s + 8 q + 4 h + r of the state. The chunk's triangle and P are made by all of them; while two
// waves solve the blocks of 32, the others go on with what the state gives. The next chunk's rows are in
// flight meanwhile. Outputs have all three parts too, whatever type they are stored in: with two, 16 bits, values within 2^-16
// of the middle of two bfloat16 numbers went to the wrong one, for 6 % less time.
// 32 x 2048 tokens on 16 heads of 64 in bfloat16, with states: 350 us (822 MB, 2.3 TB/s; 330 with two parts). No unit
// is full: VALU 49 % of all cycles, MFMA 20 %. With 237 registers and 76 KB of shared memory two waves run on a SIMD, and
// each waits 38 % of its time, for the four barriers of a chunk, shared memory and its own products. In float32 and
// with 128 features it is one wave, or two that spill (eight waves: 37 registers, 152 bytes a lane); 512 heads of 64
// 947 us, 256 heads of 128 997 (bfloat16 401). As two kernels, triangles first, it was 1199 us; with the blocks on the
// diagonal inverted through shared memory 379.
template <int T, int KP, int WAVES>
SSD_KERNEL_WAVES(64 * WAVES, (WAVES == 8 || (T == kBF16 && KP <= 2) ? 2 : 1)) void delta_scan_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    constexpr int NT = 64 * WAVES, COLS = 16 * WAVES;
    constexpr int pad = DeltaElem<T>::pad, RS = 32 * KP + pad, TS = 64 + pad;
    constexpr bool STAGE_V = T == kBF16;      // float32 rows leave no room
    SSD_LDS E k[64 * RS], q[64 * RS], kt[32 * KP * TS], vt[STAGE_V ? COLS * TS : 8];
    SSD_LDS v4u tri[kParts * kDeltaFrags * 64], pf[kParts * kDeltaFrags * 64];
    SSD_LDS DeltaGates both[2];
    const int64_t id = block_id();
    const int block = (int)(id % p.columns), hv = (int)(id / p.columns % p.Hv), b = (int)(id / p.columns / p.Hv);
    const int hk = hv / (p.Hv / p.Hk), wave = wave_id(), lane = thread_id() & 63;
    const int l = thread_id() & 15, quarter = lane >> 4, q8 = 8 * quarter;
    const int first = COLS * block, dv = first + 16 * wave + l;
    const bool live = dv < p.Dv;
    const int64_t head = ((int64_t)b * p.Hv + hv) * p.Dk * p.Dv;
    v4f S[2 * KP];
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i)
        S[i] = v4f{0.f, 0.f, 0.f, 0.f};
    if (p.init && live)
        state_load<KP>(S, p.init + head + dv, p.Dk, p.Dv);
    const int length = delta_valid(p, b);
    const int o_stride = p.Hv * p.Dv;
    const int64_t row = (int64_t)b * p.T;
    const E *qrow = (const E *)p.q + row * p.q_stride + hk * p.Dk, *krow = (const E *)p.k + row * p.k_stride + hk * p.Dk;
    const E *vrow = (const E *)p.v + row * p.v_stride + hv * p.Dv + first;
    const int vcols = p.Dv - first;

    Blocks<T, 32 * KP, NT> nk, nq;
    Blocks<T, COLS, NT> nv;
    float ng = 0.f, nbeta = 0.f;
    auto fetch = [&](int chunk, int n) {
        const int64_t t = (int64_t)chunk * kDeltaChunk;
        blocks_load<T, 32 * KP, NT>(nk, krow + t * p.k_stride, (int)p.k_stride, p.Dk, n);
        blocks_load<T, 32 * KP, NT>(nq, qrow + t * p.q_stride, (int)p.q_stride, p.Dk, n);
        if (STAGE_V)
            blocks_load<T, COLS, NT>(nv, vrow + t * p.v_stride, (int)p.v_stride, vcols, n);
        if (wave == WAVES - 1) {
            const int64_t at = (row + t + (lane < n ? lane : n - 1)) * p.Hv + hv;
            ng = p.g[at];
            nbeta = p.beta[at];
        }
    };
    const E *kl = k + tile_row(0, l) * RS + q8, *ql = q + tile_row(0, l) * RS + q8, *ktl = kt + tile_row(0, l) * TS + q8;
    const E *vl = vt + (STAGE_V ? (16 * wave + l) * TS + q8 : 0);
    int n = delta_chunk_tokens(length, 0);
    if (n > 0) {
        fetch(0, n);
        if (wave == WAVES - 1)
            delta_gates_of(both[0], ng, nbeta, n);
    }
    for (int i = thread_id(); i < kParts * kDeltaFrags * 64; i += NT)
        pf[i] = v4u{0u, 0u, 0u, 0u};  // above its diagonal P's tiles stay so
    for (int chunk = 0; chunk < p.chunks; ++chunk) {
        n = delta_chunk_tokens(length, chunk);
        const int rows = p.T - chunk * kDeltaChunk < 64 ? p.T - chunk * kDeltaChunk : 64;
        if (p.states && live)
            state_store<KP>(S, p.states + (((int64_t)b * p.chunks + chunk) * p.Hv + hv) * p.Dk * p.Dv + dv, p.Dk, p.Dv);
        E *o = (E *)p.o + (row + chunk * kDeltaChunk) * o_stride + hv * p.Dv + dv;
        if (n == 0) {  // padding
            if (live)
                for (int t = quarter; t < rows; t += 4)
                    delta_store<T>(o + (int64_t)t * o_stride, 0.f);
            continue;
        }
        const DeltaGates &gates = both[chunk & 1];
        block_sync();  // the last chunk's operands have been read
        blocks_store<T, 32 * KP, NT, true, true>(nk, p.Dk, n, k, kt);
        blocks_store<T, 32 * KP, NT, true, false>(nq, p.Dk, n, q, (E *)nullptr);
        if (STAGE_V)
            blocks_store<T, COLS, NT, false, true>(nv, vcols, n, (E *)nullptr, vt);
        block_sync();
        const int next = delta_chunk_tokens(length, chunk + 1);
        if (next > 0)
            fetch(chunk + 1, next);
        delta_tiles<T, KP, WAVES, false>(k, q, gates, p.scale, tri, pf);
        block_sync();
        if (wave < 2)
            delta_invert<false>(wave, tri);
        // R = beta (V - e^G K S), and e^G Q S
        Parts<kParts> Sp[KP];
#pragma unroll
        for (int s = 0; s < KP; ++s)
            Sp[s] = split_tiles<kParts>(S[2 * s], S[2 * s + 1]);
        float R[2][8], O[2][8];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float v[8];
            if (STAGE_V) {
                lds_values<T>(vl + 32 * s, v);
            } else {
                const E *at = vrow + (int64_t)chunk * kDeltaChunk * p.v_stride + (live ? 16 * wave + l : 0);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = delta_load<T>(at + (uint32_t)(q8 < n - (32 * s + e) ? q8 + (32 * s + e) : n - 1) * (uint32_t)p.v_stride);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = live && q8 < n - (32 * s + e) ? v[e] : 0.f;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4f ks = {0.f, 0.f, 0.f, 0.f}, qs = ks;
#pragma unroll
                for (int f = 0; f < KP; ++f) {
                    span_mm<T>(ks, lds_operand(kl + ((32 * s + 4 * h) * RS + 32 * f)), Sp[f], f);
                    qs = mm<kParts>(lds_operand(ql + ((32 * s + 4 * h) * RS + 32 * f)), Sp[f], qs);
                }
                const v4f since = *(const v4f *)(gates.since + q8 + (32 * s + 4 * h));
                const v4f beta = *(const v4f *)(gates.beta + q8 + (32 * s + 4 * h));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    R[s][4 * h + r] = beta[r] * (v[4 * h + r] - since[r] * ks[r]);
                    O[s][4 * h + r] = p.scale * since[r] * qs[r];
                }
            }
            sched_fence();
        }
        block_sync();  // the triangle is there
        // U, and O += P U
        const Parts<kParts> R0 = split8<kParts>(R[0]);
        v4f U[4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            U[h] = mm<kParts>(frag_operand<kParts>(tri, frag_of(0, h, 0)), R0, v4f{0.f, 0.f, 0.f, 0.f});
        const Parts<kParts> U0 = split_tiles<kParts>(U[0], U[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const v4f c = mm<kParts>(frag_operand<kParts>(tri, frag_of(1, h, 0)), U0, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r)
                R[1][4 * h + r] -= c[r];
        }
        const Parts<kParts> R1 = split8<kParts>(R[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            U[2 + h] = mm<kParts>(frag_operand<kParts>(tri, frag_of(1, h, 1)), R1, v4f{0.f, 0.f, 0.f, 0.f});
        const Parts<kParts> U1 = split_tiles<kParts>(U[2], U[3]);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4f c = {O[s][4 * h], O[s][4 * h + 1], O[s][4 * h + 2], O[s][4 * h + 3]};
                c = mm<kParts>(frag_operand<kParts>(pf, frag_of(s, h, 0)), U0, c);
                if (s == 1)
                    c = mm<kParts>(frag_operand<kParts>(pf, frag_of(1, h, 1)), U1, c);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    O[s][4 * h + r] = c[r];
            }
        if (live) {
            const uint32_t step = opaque_uniform((uint32_t)o_stride * sizeof(E)), off = opaque((uint32_t)q8 * step);
            if (n == 64) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        delta_store<T>((E *)((char *)o + (off + (32 * s + e) * step)), O[s][e]);
            } else {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (q8 < rows - (32 * s + e))
                            delta_store<T>((E *)((char *)o + (off + (32 * s + e) * step)),
                                           q8 < n - (32 * s + e) ? O[s][e] : 0.f);
            }
        }
        // the state
        Parts<kParts> W[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float w[8];
            const float *left = gates.left + q8 + 32 * s;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = left[e] * U[2 * s + (e >> 2)][e & 3];
            W[s] = split8<kParts>(w);
        }
        const float whole = gates.whole;
#pragma unroll
        for (int i = 0; i < 2 * KP; ++i) {
            v4f c;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                c[r] = whole * S[i][r];
#pragma unroll
            for (int s = 0; s < 2; ++s)
                c = mm<kParts>(lds_operand(ktl + (state_at(i, 0) * TS + 32 * s)), W[s], c);
            S[i] = c;
            if (i & 1)
                sched_fence();
        }
        if (next > 0 && wave == WAVES - 1)
            delta_gates_of(both[(chunk + 1) & 1], ng, nbeta, next);
    }
    if (p.final_state && live)
        state_store<KP>(S, p.final_state + head + dv, p.Dk, p.Dv);
}

// ------------------------------------------------------------- few heads, long sequences

// Where sequences and heads give too few workgroups, what a chunk has beside the state is made for a range of chunks at once
// (delta_pack_kernel) and laid out as the operands that the walk takes, and the walk has 16 columns a workgroup and no
// more to do than the state asks for: one wave passes the state on, a second one makes the outputs
// from what the first leaves in shared memory.

// What a chunk is packed into, in units of 16 bytes: operand tiles of 64 lanes each, and the gates.
template <int T, int KP>
struct DeltaPack {
    static constexpr int IN = DeltaElem<T>::parts;
    static constexpr int tri = 0, pf = tri + kParts * kDeltaFrags * 64, kr = pf + kParts * kDeltaFrags * 64;
    static constexpr int kt = kr + 4 * KP * IN * 64, q = kt + 4 * KP * IN * 64;  // Q by rows, backwards by features
    static constexpr int gates = q + 4 * KP * IN * 64, size = gates + 64;  // since, left, beta, and e^G_C in the last place
};

template <int T, int KP, bool BACKWARD>
SSD_KERNEL(256) void delta_pack_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    typedef DeltaPack<T, KP> Pack;
    constexpr int pad = DeltaElem<T>::pad, RS = 32 * KP + pad, TS = 64 + pad, IN = Pack::IN;
    SSD_LDS E k[64 * RS], q[BACKWARD && 32 * KP * TS > 64 * RS ? 32 * KP * TS : 64 * RS], kt[32 * KP * TS];
    E *const qt = q;  // by features once its rows have been used
    SSD_LDS v4u tri[kParts * kDeltaFrags * 64], pf[kParts * kDeltaFrags * 64];
    SSD_LDS DeltaGates gates;
    const int64_t id = block_id();
    const int range = p.chunk_to - p.chunk_from;
    const int at = (int)(id % range), chunk = p.chunk_from + at, hv = (int)(id / range % p.Hv), b = (int)(id / range / p.Hv);
    const int hk = hv / (p.Hv / p.Hk), wave = wave_id(), lane = thread_id() & 63, l = lane & 15, q8 = 8 * (lane >> 4);
    const int n = delta_chunk_tokens(delta_valid(p, b), chunk);
    if (n == 0)
        return;
    const int64_t token = (int64_t)b * p.T + chunk * kDeltaChunk;
    Blocks<T, 32 * KP, 256> nk, nq;
    blocks_load<T, 32 * KP, 256>(nk, (const E *)p.k + token * p.k_stride + hk * p.Dk, (int)p.k_stride, p.Dk, n);
    blocks_load<T, 32 * KP, 256>(nq, (const E *)p.q + token * p.q_stride + hk * p.Dk, (int)p.q_stride, p.Dk, n);
    if (wave == 3)
        delta_gates(gates, p.g, p.beta, token * p.Hv + hv, p.Hv, n);
    blocks_store<T, 32 * KP, 256, true, true>(nk, p.Dk, n, k, kt);
    blocks_store<T, 32 * KP, 256, true, false>(nq, p.Dk, n, q, (E *)nullptr);
    for (int i = thread_id(); i < kParts * kDeltaFrags * 64; i += 256)
        pf[i] = v4u{0u, 0u, 0u, 0u};
    block_sync();
    delta_tiles<T, KP, 4, BACKWARD>(k, q, gates, p.scale, tri, pf);
    block_sync();
    if (BACKWARD)
        blocks_store<T, 32 * KP, 256, false, true>(nq, p.Dk, n, (E *)nullptr, qt);
    if (wave < 2)
        delta_invert<BACKWARD>(wave, tri);
    block_sync();
    v4u *out = p.pack + (((int64_t)b * p.Hv + hv) * range + at) * Pack::size;
    const E *kl = k + tile_row(0, l) * RS + q8, *ql = q + tile_row(0, l) * RS + q8;
    const E *ktl = kt + tile_row(0, l) * TS + q8, *qtl = qt + tile_row(0, l) * TS + q8;
    auto put = [&](int to, int tile, const Parts<IN> &x) {
#pragma unroll
        for (int e = 0; e < IN; ++e)
            out[to + (tile * IN + e) * 64 + lane] = x.p[e];
    };
    for (int i = wave; i < 4 * KP; i += 4) {
        const int h = i / KP, f = i % KP, row = (32 * (h >> 1) + 4 * (h & 1)) * RS + 32 * f;   // rows: (tile, span)
        const int col = state_at(i >> 1, 0) * TS + 32 * (i & 1);                               // features: (tile, span)
        put(Pack::kr, i, lds_operand(kl + row));
        put(Pack::kt, i, lds_operand(ktl + col));
        put(Pack::q, i, BACKWARD ? lds_operand(qtl + col) : lds_operand(ql + row));
    }
    if (thread_id() < 64) {
        float *to = (float *)(out + Pack::gates);
        to[lane] = gates.since[lane];
        to[64 + lane] = gates.left[lane];
        to[128 + lane] = gates.beta[lane];
        to[192 + lane] = gates.whole;
    }
    for (int i = thread_id(); i < kParts * kDeltaFrags * 64; i += 256) {
        out[Pack::tri + i] = tri[i];
        out[Pack::pf + i] = pf[i];
    }
}

// The workgroup's head and columns: the columns of a head lie a multiple of eight workgroups apart, on the same
// die, whose cache then holds the head's operands for all of them.
SSD_DEVICE void long_place(const DeltaParams &p, int64_t &head, int &block)
{
    const int64_t id = block_id();
    head = id / (8 * (int64_t)p.columns) * 8 + id % 8;
    block = (int)(id / 8 % p.columns);
}

template <int N>
SSD_DEVICE void pack_load(Parts<N> &x, const v4u *from)
{
#pragma unroll
    for (int e = 0; e < N; ++e)
        x.p[e] = from[e * 64];
}
// Tiles of the triangle and of P.
SSD_DEVICE void pack_load_frag(Parts<kParts> &x, const v4u *from, int f) { pack_load(x, from + f * kParts * 64); }
// The values of the lane's 16 tokens.
SSD_DEVICE void pack_gate(v4f (&g)[4], const float *from, int q8)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        g[i] = *(const v4f *)(from + q8 + (32 * (i >> 1) + 4 * (i & 1)));
}

template <int T, int KP>
SSD_KERNEL(128) void delta_long_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    typedef DeltaPack<T, KP> Pack;
    constexpr int IN = Pack::IN;
    constexpr bool AHEAD = T == kBF16;  // K's rows of the next chunk; in float32 there are too many
    SSD_LDS v4u state[2][KP * kParts * 64], us[2][2 * kParts * 64];
    int64_t bh;
    int block;
    long_place(p, bh, block);
    if (bh >= (int64_t)p.B * p.Hv)
        return;
    const int hv = (int)(bh % p.Hv), b = (int)(bh / p.Hv);
    const int lane = thread_id() & 63, l = lane & 15, q8 = 8 * (lane >> 4);
    const int dv = 16 * block + l;
    const bool live = dv < p.Dv;
    const int length = delta_valid(p, b), range = p.chunk_to - p.chunk_from;
    const int64_t row = (int64_t)b * p.T;
    const v4u *pack = p.pack + bh * range * Pack::size + lane;
    const int last = (length + kDeltaChunk - 1) / kDeltaChunk;  // chunks with tokens
    const int to = last < p.chunk_to ? last : p.chunk_to;
    if (wave_id() == 0) {
        v4f S[2 * KP];
#pragma unroll
        for (int i = 0; i < 2 * KP; ++i)
            S[i] = v4f{0.f, 0.f, 0.f, 0.f};
        const float *init = p.chunk_from > 0 ? p.carry : p.init;
        if (init && live)
            state_load<KP>(S, init + bh * p.Dk * p.Dv + dv, p.Dk, p.Dv);
        state_arrived(S);
        const E *vrow = (const E *)p.v + row * p.v_stride + hv * p.Dv + (live ? dv : 0);
        uint32_t V[16];
        v4f since[4], beta[4], left[4];
        float whole = 0.f;
        Parts<IN> kr[AHEAD ? 4 * KP : 2 * KP];
        auto fetch = [&](int chunk) {
            const v4u *at = pack + (int64_t)(chunk - p.chunk_from) * Pack::size;
            const float *g = (const float *)(at - lane + Pack::gates);
            if (AHEAD)
#pragma unroll
                for (int i = 0; i < 4 * KP; ++i)
                    pack_load(kr[AHEAD ? i : i % KP], at + Pack::kr + i * IN * 64);
            pack_gate(since, g, q8);
            pack_gate(left, g + 64, q8);
            pack_gate(beta, g + 128, q8);
            whole = g[192];
            const int n = delta_chunk_tokens(length, chunk);
            const char *v = (const char *)(vrow + (int64_t)chunk * kDeltaChunk * p.v_stride);
            const uint32_t step = opaque_uniform((uint32_t)p.v_stride * sizeof(E)), first = opaque((uint32_t)q8 * step);
            if (n == 64) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    V[e] = delta_raw<T>((const E *)(v + (first + (uint32_t)(32 * (e >> 3) + (e & 7)) * step)));
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int t = 32 * (e >> 3) + (e & 7);
                    V[e] = delta_raw<T>((const E *)(v + (uint32_t)(q8 < n - t ? q8 + t : n - 1) * step));
                }
            }
        };
        if (p.chunk_from < to)
            fetch(p.chunk_from);
        for (int chunk = p.chunk_from; chunk < p.chunk_to; ++chunk) {
            if (p.states && live)
                state_store<KP>(S, p.states + (((int64_t)b * p.chunks + chunk) * p.Hv + hv) * p.Dk * p.Dv + dv, p.Dk, p.Dv);
            if (chunk >= to)
                continue;
            const v4u *at = pack + (int64_t)(chunk - p.chunk_from) * Pack::size;
            const int n = delta_chunk_tokens(length, chunk);
            Parts<kParts> tri[kDeltaFrags];
            Parts<IN> kt[4 * KP];
            if (!AHEAD)
#pragma unroll
                for (int f = 0; f < KP; ++f)
                    pack_load(kr[f], at + Pack::kr + f * IN * 64);
#pragma unroll
            for (int f = 0; f < kDeltaFrags; ++f)
                pack_load_frag(tri[f], at + Pack::tri, f);
            Parts<kParts> Sp[KP];
#pragma unroll
            for (int s = 0; s < KP; ++s) {
                Sp[s] = split_tiles<kParts>(S[2 * s], S[2 * s + 1]);
#pragma unroll
                for (int e = 0; e < kParts; ++e)
                    state[chunk & 1][(s * kParts + e) * 64 + lane] = Sp[s].p[e];
            }
            // R = beta (V - e^G K S)
            float R[2][8];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                v4f ks = {0.f, 0.f, 0.f, 0.f};
                if (!AHEAD && h < 3)
#pragma unroll
                    for (int f = 0; f < KP; ++f)
                        pack_load(kr[(h + 1) % 2 * KP + f], at + Pack::kr + ((h + 1) * KP + f) * IN * 64);
#pragma unroll
                for (int f = 0; f < KP; ++f)
                    span_mm<T>(ks, kr[AHEAD ? h * KP + f : h % 2 * KP + f], Sp[f], f);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int e = 4 * (h & 1) + r;
                    const float x = live && q8 < n - (32 * (h >> 1) + e) ? delta_value<T>(V[8 * (h >> 1) + e]) : 0.f;
                    R[h >> 1][e] = beta[h][r] * (x - since[h][r] * ks[r]);
                }
            }
            // U
#pragma unroll
            for (int i = 0; i < 4 * KP; ++i)
                pack_load(kt[i], at + Pack::kt + i * IN * 64);
            const Parts<kParts> R0 = split8<kParts>(R[0]);
            v4f U[4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                U[h] = mm<kParts>(tri[frag_of(0, h, 0)], R0, v4f{0.f, 0.f, 0.f, 0.f});
            const Parts<kParts> U0 = split_tiles<kParts>(U[0], U[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4f c = mm<kParts>(tri[frag_of(1, h, 0)], U0, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    R[1][4 * h + r] -= c[r];
            }
            const Parts<kParts> R1 = split8<kParts>(R[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                U[2 + h] = mm<kParts>(tri[frag_of(1, h, 1)], R1, v4f{0.f, 0.f, 0.f, 0.f});
            const Parts<kParts> U1 = split_tiles<kParts>(U[2], U[3]);
#pragma unroll
            for (int e = 0; e < kParts; ++e) {
                us[chunk & 1][e * 64 + lane] = U0.p[e];
                us[chunk & 1][(kParts + e) * 64 + lane] = U1.p[e];
            }
            // the state
            Parts<kParts> W[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e] = left[2 * s + (e >> 2)][e & 3] * U[2 * s + (e >> 2)][e & 3];
                W[s] = split8<kParts>(w);
            }
            const float hold = whole;
            if (chunk + 1 < to)
                fetch(chunk + 1);
#pragma unroll
            for (int i = 0; i < 2 * KP; ++i) {
                v4f c;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    c[r] = hold * S[i][r];
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    c = mm<kParts>(kt[2 * i + s], W[s], c);
                S[i] = c;
            }
            block_sync();  // what the outputs need is there, those of the chunk before are made
        }
        float *out = p.chunk_to < p.chunks ? p.carry : p.final_state;
        if (out && live)
            state_store<KP>(S, out + bh * p.Dk * p.Dv + dv, p.Dk, p.Dv);
    } else {
        const int o_stride = p.Hv * p.Dv;
        for (int chunk = p.chunk_from; chunk < p.chunk_to; ++chunk) {
            const int rows = p.T - chunk * kDeltaChunk < 64 ? p.T - chunk * kDeltaChunk : 64;
            E *o = (E *)p.o + (row + (int64_t)chunk * kDeltaChunk) * o_stride + hv * p.Dv + dv;
            if (chunk >= to) {  // padding
                if (live)
                    for (int t = q8 >> 3; t < rows; t += 4)
                        delta_store<T>(o + (int64_t)t * o_stride, 0.f);
                continue;
            }
            const v4u *at = pack + (int64_t)(chunk - p.chunk_from) * Pack::size;
            const int n = delta_chunk_tokens(length, chunk);
            Parts<IN> qr[4 * KP];
            Parts<kParts> pf[kDeltaFrags];
            v4f since[4];
#pragma unroll
            for (int i = 0; i < 4 * KP; ++i)
                pack_load(qr[i], at + Pack::q + i * IN * 64);
#pragma unroll
            for (int f = 0; f < kDeltaFrags; ++f)
                pack_load_frag(pf[f], at + Pack::pf, f);
            pack_gate(since, (const float *)(at - lane + Pack::gates), q8);
            block_sync();  // the state and U are there
            Parts<kParts> Sp[KP], U[2];
#pragma unroll
            for (int s = 0; s < KP; ++s)
                pack_load(Sp[s], &state[chunk & 1][s * kParts * 64 + lane]);
#pragma unroll
            for (int s = 0; s < 2; ++s)
                pack_load(U[s], &us[chunk & 1][s * kParts * 64 + lane]);
            const uint32_t step = opaque_uniform((uint32_t)o_stride * sizeof(E)), off = opaque((uint32_t)q8 * step);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                v4f c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int f = 0; f < KP; ++f)
                    c = mm<kParts>(qr[h * KP + f], Sp[f], c);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    c[r] *= p.scale * since[h][r];
                c = mm<kParts>(pf[frag_of(h >> 1, h & 1, 0)], U[0], c);
                if (h > 1)
                    c = mm<kParts>(pf[frag_of(1, h & 1, 1)], U[1], c);
                if (live)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = 32 * (h >> 1) + 4 * (h & 1) + r;
                        if (q8 < rows - t)
                            delta_store<T>((E *)((char *)o + (off + (uint32_t)t * step)), q8 < n - t ? c[r] : 0.f);
                    }
            }
        }
    }
}

// The same in float32, whose operands have three parts and whose products six terms: a wave for each span of 32
// features of the state, which sums its share of K S and updates its own rows; the shares meet in shared
// memory, every wave solves for U, and each makes some of the outputs' tiles. Operands are loaded a chunk
// ahead, into the registers that the last ones leave. A chunk is a chain of dependent products and their splitting
// into parts, some 3 us of it whatever the width; one wave with all features takes 4 to 6 (T 2048, us, this form / the
// other: 16 heads of 64 139 / 184, 96 heads 331 / 374, 32 heads of 128 249 / 364). With up to 64 features it is
// always taken; with more, its four waves have a compute unit to themselves, and where there are more workgroups
// than units the other form is as fast or faster (48 heads of 128: 459 / 449). In bfloat16, where K, and the products
// of K, have a third of the parts, it gains 7 % with 64 features and loses 18 % with 128: not taken (with 64 alone it would
// have the walk over many heads sum span by span as well, for the same bits, which costs that 3 %).
constexpr int kSpansMost = 256;  // workgroups

// Operands at a place that is the same for all lanes, so that its address is scalar work.
template <int N>
SSD_DEVICE void span_load(Parts<N> &x, const v4u *from)
{
    const uint32_t off = 16 * ((uint32_t)thread_id() & 63);
#pragma unroll
    for (int e = 0; e < N; ++e)
        x.p[e] = *(const v4u *)((const char *)(from + e * 64) + off);
}
SSD_DEVICE void span_load_frag(Parts<kParts> &x, const v4u *from, int f) { span_load(x, from + f * kParts * 64); }
SSD_DEVICE v4f span_gate(const float *from, int t)
{
    return *(const v4f *)((const char *)(from + t) + 32 * (((uint32_t)thread_id() & 63) >> 4));
}
SSD_DEVICE void span_gates(v4f (&g)[4], const float *from)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        g[i] = span_gate(from, 32 * (i >> 1) + 4 * (i & 1));
}

// A wave's first feature (or 0, if there is none), and how many it has.
SSD_DEVICE int span_first(int wave, int Dk) { return 32 * wave < Dk ? 32 * wave : 0; }
SSD_DEVICE int span_many(int wave, int Dk) { return Dk - 32 * wave < 32 ? Dk - 32 * wave : 32; }
// The shares of tile h, added in the spans' order.
template <int KP>
SSD_DEVICE v4f spans_sum(const v4f (&share)[KP][4][64], int h, int lane)
{
    v4f c;
#pragma unroll
    for (int w = 0; w < KP; ++w)
        span_add(c, share[w][h][lane], w);
    return c;
}

template <int T, int KP>
SSD_KERNEL(64 * KP) void delta_spans_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    typedef DeltaPack<T, KP> Pack;
    constexpr int IN = Pack::IN, OWN = 4 / KP;  // tiles of 16 tokens to a wave
    SSD_LDS v4f share[2][KP][4][64];
    SSD_LDS v4u state[2][KP * kParts * 64];
    int64_t bh;
    int block;
    long_place(p, bh, block);
    if (bh >= (int64_t)p.B * p.Hv)
        return;
    const int hv = (int)(bh % p.Hv), b = (int)(bh / p.Hv);
    const int lane = thread_id() & 63, l = lane & 15, q8 = 8 * (lane >> 4), wave = wave_id();
    const int dv = 16 * block + l;
    const bool live = dv < p.Dv;
    const int length = delta_valid(p, b), range = p.chunk_to - p.chunk_from, o_stride = p.Hv * p.Dv;
    const int64_t row = (int64_t)b * p.T;
    const v4u *pack = p.pack + bh * range * Pack::size;
    const int last = (length + kDeltaChunk - 1) / kDeltaChunk;  // chunks with tokens
    const int to = last < p.chunk_to ? last : p.chunk_to;
    const int first = span_first(wave, p.Dk), many = span_many(wave, p.Dk);
    const int tile = OWN * wave, span = tile >> 1;  // of the outputs
    const int64_t state_at0 = (int64_t)first * p.Dv + dv;
    v4f S[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    const float *init = p.chunk_from > 0 ? p.carry : p.init;
    if (init && live)
        state_load<1>(S, init + bh * p.Dk * p.Dv + state_at0, many, p.Dv);
    state_arrived(S);
    const E *vrow = (const E *)p.v + row * p.v_stride + hv * p.Dv + (live ? dv : 0);
    uint32_t V[16];
    v4f since[4], beta[4], left[4], mine[OWN];
    float whole = 0.f;
    Parts<IN> kr[4], kt[2][2], qr[OWN][KP];
    Parts<kParts> tri[kDeltaFrags];
    Parts<kParts> pf[OWN][2];
    auto place = [&](int chunk) { return pack + (int64_t)(chunk - p.chunk_from) * Pack::size; };
    auto fetch_rows = [&](const v4u *at) {
#pragma unroll
        for (int h = 0; h < 4; ++h)
            span_load(kr[h], at + Pack::kr + (h * KP + wave) * IN * 64);
    };
    auto fetch_solve = [&](const v4u *at, int chunk) {
        const float *g = (const float *)(at + Pack::gates);
#pragma unroll
        for (int f = 0; f < kDeltaFrags; ++f)
            span_load_frag(tri[f], at + Pack::tri, f);
        span_gates(since, g);
        span_gates(left, g + 64);
        span_gates(beta, g + 128);
        whole = g[192];
        const int n = delta_chunk_tokens(length, chunk);
        const char *v = (const char *)(vrow + (int64_t)chunk * kDeltaChunk * p.v_stride);
        const uint32_t step = opaque_uniform((uint32_t)p.v_stride * sizeof(E)), from = opaque((uint32_t)q8 * step);
        if (n == 64) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                V[e] = delta_raw<T>((const E *)(v + (from + (uint32_t)(32 * (e >> 3) + (e & 7)) * step)));
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int t = 32 * (e >> 3) + (e & 7);
                V[e] = delta_raw<T>((const E *)(v + (uint32_t)(q8 < n - t ? q8 + t : n - 1) * step));
            }
        }
    };
    auto fetch_features = [&](const v4u *at) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                span_load(kt[i][s], at + Pack::kt + (2 * (2 * wave + i) + s) * IN * 64);
    };
    auto fetch_outputs = [&](const v4u *at) {
        const float *g = (const float *)(at + Pack::gates);
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int h = (tile + i) & 1;
#pragma unroll
            for (int f = 0; f < KP; ++f)
                span_load(qr[i][f], at + Pack::q + ((tile + i) * KP + f) * IN * 64);
            span_load_frag(pf[i][0], at + Pack::pf, frag_of(span, h, 0));
            span_load_frag(pf[i][1], at + Pack::pf, frag_of(span, h, span));
            mine[i] = span_gate(g, 32 * span + 4 * h);
        }
    };
    if (p.chunk_from < to) {
        const v4u *at = place(p.chunk_from);
        fetch_rows(at);  // in the order of the loop: what is waited for is what was loaded before
        sched_fence();
        fetch_solve(at, p.chunk_from);
        fetch_features(at);
        sched_fence();
        fetch_outputs(at);
    }
    for (int chunk = p.chunk_from; chunk < p.chunk_to; ++chunk) {
        if (p.states && live)
            state_store<1>(S, p.states + (((int64_t)b * p.chunks + chunk) * p.Hv + hv) * p.Dk * p.Dv + state_at0, many, p.Dv);
        const int rows = p.T - chunk * kDeltaChunk < 64 ? p.T - chunk * kDeltaChunk : 64;
        E *o = (E *)p.o + (row + (int64_t)chunk * kDeltaChunk) * o_stride + hv * p.Dv + dv;
        if (chunk >= to) {  // padding
            if (live)
                for (int t = 4 * wave + (q8 >> 3); t < rows; t += 4 * KP)
                    delta_store<T>(o + (int64_t)t * o_stride, 0.f);
            continue;
        }
        const int n = delta_chunk_tokens(length, chunk);
        // after the last chunk its own operands once more: with branches around the loads the waits for
        // them would be as long as if each were the only one taken
        const int ahead = chunk + 1 < to ? chunk + 1 : chunk;
        const v4u *next = place(ahead);
        const Parts<kParts> Sp = split_tiles<kParts>(S[0], S[1]);
#pragma unroll
        for (int e = 0; e < kParts; ++e)
            state[chunk & 1][(wave * kParts + e) * 64 + lane] = Sp.p[e];
#pragma unroll
        for (int h = 0; h < 4; ++h)
            share[chunk & 1][wave][h][lane] = mm<kParts>(kr[h], Sp, v4f{0.f, 0.f, 0.f, 0.f});
        fetch_rows(next);
        sched_fence();
        block_sync();  // one a chunk: the two halves of what is shared take turns
        // R = beta (V - e^G K S)
        float R[2][8];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const v4f ks = spans_sum<KP>(share[chunk & 1], h, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int e = 4 * (h & 1) + r;
                const float x = live && q8 < n - (32 * (h >> 1) + e) ? delta_value<T>(V[8 * (h >> 1) + e]) : 0.f;
                R[h >> 1][e] = beta[h][r] * (x - since[h][r] * ks[r]);
            }
        }
        // U
        const Parts<kParts> R0 = split8<kParts>(R[0]);
        v4f U[4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            U[h] = mm<kParts>(tri[frag_of(0, h, 0)], R0, v4f{0.f, 0.f, 0.f, 0.f});
        const Parts<kParts> U0 = split_tiles<kParts>(U[0], U[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const v4f c = mm<kParts>(tri[frag_of(1, h, 0)], U0, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r)
                R[1][4 * h + r] -= c[r];
        }
        const Parts<kParts> R1 = split8<kParts>(R[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            U[2 + h] = mm<kParts>(tri[frag_of(1, h, 1)], R1, v4f{0.f, 0.f, 0.f, 0.f});
        // the state
        Parts<kParts> W[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = left[2 * s + (e >> 2)][e & 3] * U[2 * s + (e >> 2)][e & 3];
            W[s] = split8<kParts>(w);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v4f c;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                c[r] = whole * S[i][r];
#pragma unroll
            for (int s = 0; s < 2; ++s)
                c = mm<kParts>(kt[i][s], W[s], c);
            S[i] = c;
        }
        fetch_solve(next, ahead);
        fetch_features(next);
        sched_fence();
        // the outputs
        Parts<kParts> old[KP];
#pragma unroll
        for (int f = 0; f < KP; ++f)
            pack_load(old[f], &state[chunk & 1][f * kParts * 64 + lane]);
        const Parts<kParts> U1 = split_tiles<kParts>(U[2], U[3]);
        const uint32_t step = opaque_uniform((uint32_t)o_stride * sizeof(E)), off = opaque((uint32_t)q8 * step);
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            v4f c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int f = 0; f < KP; ++f)
                c = mm<kParts>(qr[i][f], old[f], c);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                c[r] *= p.scale * mine[i][r];
            c = mm<kParts>(pf[i][0], U0, c);
            if (span == 1)
                c = mm<kParts>(pf[i][1], U1, c);
            const int t0 = 32 * span + 4 * ((tile + i) & 1);
            if (live)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (q8 < rows - t0 - r)
                        delta_store<T>((E *)((char *)o + (off + (uint32_t)(t0 + r) * step)), q8 < n - t0 - r ? c[r] : 0.f);
        }
        fetch_outputs(next);
    }
    float *out = p.chunk_to < p.chunks ? p.carry : p.final_state;
    if (out && live)
        state_store<1>(S, out + bh * p.Dk * p.Dv + state_at0, many, p.Dv);
}

// ------------------------------------------------------------ a few tokens on the state

constexpr int kDeltaFew = 8;  // tokens that are walked one by one

// A wave holds 16 columns of the state: lane 16 c + r the rows r, r + 16, ... of the columns
// 4 c .. 4 c + 3. Sums over rows go over the 16 lanes. Bound by the state, in and out: 64 sequences' step on 16 heads
// of 64 moves 34 MB in 9.6 to 11.2 us; 16 x 5 tokens on 16 heads of 128 16.8 (25.2 without the next token's values ahead).
template <int T, int ROWS>
SSD_KERNEL(256) void delta_few_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    const int64_t id = block_id();
    const int block = (int)(id % p.columns), hv = (int)(id / p.columns % p.Hv), b = (int)(id / p.columns / p.Hv);
    const int hk = hv / (p.Hv / p.Hk);
    const int r = thread_id() & 15, dv = 64 * block + 16 * wave_id() + 4 * ((thread_id() & 63) >> 4);
    const int left = p.Dv - dv;
    const int length = delta_valid(p, b);
    const int64_t head = ((int64_t)b * p.Hv + hv) * p.Dk * p.Dv;
    float S[ROWS][4];
    auto store = [&](float *to) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (r + 16 * i < p.Dk) {
                float *at = to + (int64_t)(r + 16 * i) * p.Dv + dv;
                if (left >= 4) {
                    __builtin_memcpy(at, S[i], 16);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < left)
                            at[e] = S[i][e];
                }
            }
    };
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            S[i][e] = 0.f;
    if (p.init && left >= 4) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            __builtin_memcpy(S[i], p.init + head + (int64_t)(r + 16 * i < p.Dk ? r + 16 * i : 0) * p.Dv + dv, 16);
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[i][e] = r + 16 * i < p.Dk ? S[i][e] : 0.f;
    } else if (p.init && left > 0) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[i][e] = r + 16 * i < p.Dk && e < left ? p.init[head + (int64_t)(r + 16 * i) * p.Dv + dv + e] : 0.f;
    }
    if (p.states)  // one chunk
        store(p.states + head);
    // the next token's values are on their way while one is gone through; loads go to places that exist
    const int64_t o_stride = (int64_t)p.Hv * p.Dv;
    const int cols = left < 0 ? 0 : left < 4 ? left : 4;
    uint32_t nk[ROWS], nq[ROWS], nv[4];
    float ng, nbeta;
    auto fetch = [&](int t) {
        const int64_t token = (int64_t)b * p.T + t;
        const E *q = (const E *)p.q + token * p.q_stride + hk * p.Dk, *k = (const E *)p.k + token * p.k_stride + hk * p.Dk;
        const E *v = (const E *)p.v + token * p.v_stride + hv * p.Dv;
        ng = p.g[token * p.Hv + hv];
        nbeta = p.beta[token * p.Hv + hv];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int f = r + 16 * i < p.Dk ? r + 16 * i : p.Dk - 1;
            nk[i] = delta_raw<T>(k + f);
            nq[i] = delta_raw<T>(q + f);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            nv[e] = delta_raw<T>(v + (e < cols ? dv + e : 0));
    };
    if (length > 0)
        fetch(0);
    for (int t = 0; t < p.T; ++t) {
        E *o = (E *)p.o + ((int64_t)b * p.T + t) * o_stride + hv * p.Dv + dv;
        float out[4] = {0.f, 0.f, 0.f, 0.f};
        if (t < length) {
            float kr[ROWS], qr[ROWS], u[4];
            const float a = delta_exp(delta_log2(ng)), beta = nbeta;
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                kr[i] = r + 16 * i < p.Dk ? delta_value<T>(nk[i]) : 0.f;
                qr[i] = r + 16 * i < p.Dk ? delta_value<T>(nq[i]) : 0.f;
            }
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = e < cols ? delta_value<T>(nv[e]) : 0.f;
            if (t + 1 < length)
                fetch(t + 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u[e] = 0.f;
#pragma unroll
                for (int i = 0; i < ROWS; ++i) {
                    S[i][e] *= a;
                    u[e] = __builtin_fmaf(kr[i], S[i][e], u[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u[e] = beta * (x[e] - row16_sum(u[e]));
#pragma unroll
                for (int i = 0; i < ROWS; ++i) {
                    S[i][e] = __builtin_fmaf(kr[i], u[e], S[i][e]);
                    out[e] = __builtin_fmaf(qr[i], S[i][e], out[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                out[e] = p.scale * row16_sum(out[e]);
        }
        if (r == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < cols)
                    delta_store<T>(o + e, out[e]);
        }
    }
    if (p.final_state)
        store(p.final_state + head);
}

// ------------------------------------------------------------ gradients: the walk backwards

// As delta_scan_kernel, from the last chunk to the first, with the gradient of the state: dS' of every chunk and
// dR go to memory. K's rows make room for Q's columns once they have been used, Q's rows for those of dO, so that
// two workgroups fit a compute unit. 32 x 2048 tokens on 16 heads of 64 in bfloat16: 360 us; VALU 49 %, MFMA 17 %, and
// a wave, of two on a SIMD, waits 36 % of its time, as forwards.
template <int T, int KP, int WAVES>
SSD_KERNEL_WAVES(64 * WAVES, (WAVES == 8 || (T == kBF16 && KP <= 2) ? 2 : 1)) void delta_scan_bwd_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    constexpr int NT = 64 * WAVES, COLS = 16 * WAVES;
    constexpr int pad = DeltaElem<T>::pad, RS = 32 * KP + pad, TS = 64 + pad;
    constexpr int IN = DeltaElem<T>::parts;
    constexpr int K_ROOM = 64 * RS > 32 * KP * TS ? 64 * RS : 32 * KP * TS;
    constexpr int Q_ROOM = 64 * RS > COLS * TS ? 64 * RS : COLS * TS;
    SSD_LDS E k[K_ROOM], q[Q_ROOM], kt[32 * KP * TS];
    SSD_LDS v4u tri[kParts * kDeltaFrags * 64], pt[kParts * kDeltaFrags * 64];
    SSD_LDS DeltaGates gates;
    E *const qt = k, *const got = q;
    const int64_t id = block_id();
    const int block = (int)(id % p.columns), hv = (int)(id / p.columns % p.Hv), b = (int)(id / p.columns / p.Hv);
    const int hk = hv / (p.Hv / p.Hk), wave = wave_id(), lane = thread_id() & 63;
    const int l = thread_id() & 15, quarter = lane >> 4, q8 = 8 * quarter;
    const int first = COLS * block, dv = first + 16 * wave + l;
    const bool live = dv < p.Dv;
    const int64_t head = ((int64_t)b * p.Hv + hv) * p.Dk * p.Dv;
    v4f S[2 * KP];  // the gradient of the state after the chunk
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i)
        S[i] = v4f{0.f, 0.f, 0.f, 0.f};
    if (p.gfinal && live)
        state_load<KP>(S, p.gfinal + head + dv, p.Dk, p.Dv);
    const int length = delta_valid(p, b);
    const int o_stride = p.Hv * p.Dv;
    const int64_t row = (int64_t)b * p.T;
    const E *qrow = (const E *)p.q + row * p.q_stride + hk * p.Dk, *krow = (const E *)p.k + row * p.k_stride + hk * p.Dk;
    const E *orow = (const E *)p.go + row * o_stride + hv * p.Dv + first;
    const int vcols = p.Dv - first;
    const E *kl = k + tile_row(0, l) * RS + q8, *ktl = kt + tile_row(0, l) * TS + q8, *qtl = qt + tile_row(0, l) * TS + q8;
    const E *gl = got + (16 * wave + l) * TS + q8;

    Blocks<T, 32 * KP, NT> nk, nq;
    Blocks<T, COLS, NT> no;
    float ng = 0.f, nbeta = 0.f;
    auto fetch = [&](int chunk, int n) {
        const int64_t t = (int64_t)chunk * kDeltaChunk;
        blocks_load<T, 32 * KP, NT>(nk, krow + t * p.k_stride, (int)p.k_stride, p.Dk, n);
        blocks_load<T, 32 * KP, NT>(nq, qrow + t * p.q_stride, (int)p.q_stride, p.Dk, n);
        blocks_load<T, COLS, NT>(no, orow + t * o_stride, o_stride, vcols, n);
        if (wave == WAVES - 1) {
            const int64_t at = (row + t + (lane < n ? lane : n - 1)) * p.Hv + hv;
            ng = p.g[at];
            nbeta = p.beta[at];
        }
    };
    const int chunks = (length + kDeltaChunk - 1) / kDeltaChunk;  // those with tokens
    if (chunks > 0)
        fetch(chunks - 1, delta_chunk_tokens(length, chunks - 1));
    for (int i = thread_id(); i < kParts * kDeltaFrags * 64; i += NT)
        pt[i] = v4u{0u, 0u, 0u, 0u};
    for (int chunk = chunks - 1; chunk >= 0; --chunk) {
        const int n = delta_chunk_tokens(length, chunk);
        const int64_t at = ((int64_t)b * p.Hv + hv) * p.chunks + chunk;
        if (live)
            state_store<KP>(S, p.gs + at * p.Dk * p.Dv + dv, p.Dk, p.Dv);
        block_sync();  // the last chunk's operands have been read
        blocks_store<T, 32 * KP, NT, true, true>(nk, p.Dk, n, k, kt);
        blocks_store<T, 32 * KP, NT, true, false>(nq, p.Dk, n, q, (E *)nullptr);
        if (wave == WAVES - 1)
            delta_gates_of(gates, ng, nbeta, n);
        block_sync();
        delta_tiles<T, KP, WAVES, true>(k, q, gates, p.scale, tri, pt);
        block_sync();
        blocks_store<T, COLS, NT, false, true>(no, vcols, n, (E *)nullptr, got);
        if (wave < 2)
            delta_invert<true>(wave, tri);
        // e^(G_C - G) K dS'
        Parts<kParts> Sp[KP];
#pragma unroll
        for (int s = 0; s < KP; ++s)
            Sp[s] = split_tiles<kParts>(S[2 * s], S[2 * s + 1]);
        float dU[2][8];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4f ks = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int f = 0; f < KP; ++f)
                    ks = mm<kParts>(lds_operand(kl + ((32 * s + 4 * h) * RS + 32 * f)), Sp[f], ks);
                const v4f left = *(const v4f *)(gates.left + q8 + (32 * s + 4 * h));
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    dU[s][4 * h + r] = left[r] * ks[r];
            }
            sched_fence();
        }
        block_sync();  // the triangle and dO are there, K's rows have been read
        blocks_store<T, 32 * KP, NT, false, true>(nq, p.Dk, n, (E *)nullptr, qt);
        if (chunk > 0)
            fetch(chunk - 1, kDeltaChunk);
        Parts<IN> G[2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
            G[s] = lds_operand(gl + 32 * s);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4f c = {dU[s][4 * h], dU[s][4 * h + 1], dU[s][4 * h + 2], dU[s][4 * h + 3]};
#pragma unroll
                for (int t = s; t < 2; ++t)
                    c = mm<kParts>(frag_operand<kParts>(pt, frag_of_upper(s, h, t)), G[t], c);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    dU[s][4 * h + r] = c[r];
            }
        sched_fence();
        // dR
        v4f dR[4];
        const Parts<kParts> u1 = split8<kParts>(dU[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            dR[2 + h] = mm<kParts>(frag_operand<kParts>(tri, frag_of_upper(1, h, 1)), u1, v4f{0.f, 0.f, 0.f, 0.f});
        const Parts<kParts> r1 = split_tiles<kParts>(dR[2], dR[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const v4f c = mm<kParts>(frag_operand<kParts>(tri, frag_of_upper(0, h, 1)), r1, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r)
                dU[0][4 * h + r] -= c[r];
        }
        const Parts<kParts> u0 = split8<kParts>(dU[0]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            dR[h] = mm<kParts>(frag_operand<kParts>(tri, frag_of_upper(0, h, 0)), u0, v4f{0.f, 0.f, 0.f, 0.f});
        if (live) {
            const uint32_t step = opaque_uniform((uint32_t)p.Dv * 4), off = opaque((uint32_t)q8 * step);
            char *to = (char *)(p.gr + at * 64 * p.Dv + dv);
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    *(float *)(to + (off + (32 * s + e) * step)) = dR[2 * s + (e >> 2)][e & 3];
        }
        // the state's gradient before the chunk
        Parts<kParts> W[2], X[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float w[8], x[8];
            unpack8<kF32>(load8<kF32>(gates.since + q8 + 32 * s, 8), x);
            unpack8<kF32>(load8<kF32>(gates.beta + q8 + 32 * s, 8), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[e] = -x[e] * w[e] * dR[2 * s + (e >> 2)][e & 3];
                x[e] *= p.scale;
            }
            W[s] = split8<kParts>(w);
            lds_values<T>(gl + 32 * s, w);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] *= w[e];
            X[s] = split8<kParts>(x);
        }
        const float whole = gates.whole;
        block_sync();  // Q's columns are there
#pragma unroll
        for (int i = 0; i < 2 * KP; ++i) {
            v4f c;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                c[r] = whole * S[i][r];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                c = mm<kParts>(lds_operand(qtl + (state_at(i, 0) * TS + 32 * s)), X[s], c);
                c = mm<kParts>(lds_operand(ktl + (state_at(i, 0) * TS + 32 * s)), W[s], c);
            }
            S[i] = c;
            if (i & 1)
                sched_fence();
        }
    }
    if (p.ginit && live)
        state_store<KP>(S, p.ginit + head + dv, p.Dk, p.Dv);
}

// The same with few heads: by spans of features, as delta_spans_kernel, on what delta_pack_kernel made. Here the walk
// has twice the products, and one wave with all features was slower in both types (the gradients as a whole,
// T 2048, us, this form / that: 16 heads of 128 in bfloat16 275 / 342, in float32 389 / 685; 32 heads 438 / 526 and
// 639 / 1119).
template <int T, int KP>
SSD_KERNEL(64 * KP) void delta_spans_bwd_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    typedef DeltaPack<T, KP> Pack;
    constexpr int IN = Pack::IN, OWN = 4 / KP;  // tiles of 16 tokens to a wave
    SSD_LDS v4f share[2][KP][4][64];
    int64_t bh;
    int block;
    long_place(p, bh, block);
    if (bh >= (int64_t)p.B * p.Hv)
        return;
    const int hv = (int)(bh % p.Hv), b = (int)(bh / p.Hv);
    const int lane = thread_id() & 63, l = lane & 15, q8 = 8 * (lane >> 4), wave = wave_id();
    const int dv = 16 * block + l;
    const bool live = dv < p.Dv;
    const int length = delta_valid(p, b), range = p.chunk_to - p.chunk_from, o_stride = p.Hv * p.Dv;
    const v4u *pack = p.pack + bh * range * Pack::size;
    const int last = (length + kDeltaChunk - 1) / kDeltaChunk;  // chunks with tokens
    const int to = last < p.chunk_to ? last : p.chunk_to;
    const int first = span_first(wave, p.Dk), many = span_many(wave, p.Dk);
    const int tile = OWN * wave, span = tile >> 1;  // of P^T dO
    const int64_t state_at0 = (int64_t)first * p.Dv + dv;
    v4f S[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // the gradient of the state after the chunk
    const float *init = p.chunk_to < p.chunks ? p.carry : p.gfinal;
    if (init && live)
        state_load<1>(S, init + bh * p.Dk * p.Dv + state_at0, many, p.Dv);
    state_arrived(S);
    const E *orow = (const E *)p.go + (int64_t)b * p.T * o_stride + hv * p.Dv + (live ? dv : 0);
    uint32_t raw[16];
    v4f since[4], beta[4], left[4];
    float whole = 0.f;
    Parts<IN> kr[4], kt[2][2], qt[2][2];
    Parts<kParts> tri[kDeltaFrags], pt[OWN][2];
    auto place = [&](int chunk) { return pack + (int64_t)(chunk - p.chunk_from) * Pack::size; };
    auto fetch_first = [&](const v4u *at) {
#pragma unroll
        for (int h = 0; h < 4; ++h)
            span_load(kr[h], at + Pack::kr + (h * KP + wave) * IN * 64);
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int h = (tile + i) & 1;
            span_load_frag(pt[i][0], at + Pack::pf, frag_of_upper(span, h, span));
            span_load_frag(pt[i][1], at + Pack::pf, frag_of_upper(span, h, 1));
        }
    };
    auto fetch_queries = [&](const v4u *at) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                span_load(qt[i][s], at + Pack::q + (2 * (2 * wave + i) + s) * IN * 64);
    };
    auto fetch_rest = [&](const v4u *at, int chunk) {
        const float *g = (const float *)(at + Pack::gates);
        span_gates(since, g);
        span_gates(left, g + 64);
        span_gates(beta, g + 128);
        whole = g[192];
        const int n = delta_chunk_tokens(length, chunk);
        const char *o = (const char *)(orow + (int64_t)chunk * kDeltaChunk * o_stride);
        const uint32_t step = opaque_uniform((uint32_t)o_stride * sizeof(E)), from = opaque((uint32_t)q8 * step);
        if (n == 64) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                raw[e] = delta_raw<T>((const E *)(o + (from + (uint32_t)(32 * (e >> 3) + (e & 7)) * step)));
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int t = 32 * (e >> 3) + (e & 7);
                raw[e] = delta_raw<T>((const E *)(o + (uint32_t)(q8 < n - t ? q8 + t : n - 1) * step));
            }
        }
#pragma unroll
        for (int f = 0; f < kDeltaFrags; ++f)
            span_load_frag(tri[f], at + Pack::tri, f);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                span_load(kt[i][s], at + Pack::kt + (2 * (2 * wave + i) + s) * IN * 64);
    };
    if (p.chunk_from < to) {
        const v4u *at = place(to - 1);
        fetch_first(at);  // in the order of the loop: what is waited for is what was loaded before
        sched_fence();
        fetch_queries(at);
        sched_fence();
        fetch_rest(at, to - 1);
    }
    for (int chunk = to - 1; chunk >= p.chunk_from; --chunk) {
        const int n = delta_chunk_tokens(length, chunk);
        const int ahead = chunk > p.chunk_from ? chunk - 1 : chunk;
        const v4u *next = place(ahead);
        const int64_t at = bh * p.chunks + chunk;
        if (live)
            state_store<1>(S, p.gs + at * p.Dk * p.Dv + state_at0, many, p.Dv);
        const Parts<kParts> Sp = split_tiles<kParts>(S[0], S[1]);
        Parts<IN> go[2];
        float G[2][8];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                G[s][e] = live && q8 < n - (32 * s + e) ? delta_value<T>(raw[8 * s + e]) : 0.f;
            go[s] = split8<IN>(G[s]);
        }
        // the span's share of e^(G_C - G) K dS', and in some tiles all of P^T dO
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            v4f c = mm<kParts>(kr[h], Sp, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r)
                c[r] *= left[h][r];
            if (h / OWN == wave) {
                if (h < 2)
                    c = mm<kParts>(pt[h % OWN][0], go[0], c);
                c = mm<kParts>(pt[h % OWN][1], go[1], c);
            }
            share[chunk & 1][wave][h][lane] = c;
        }
        fetch_first(next);
        sched_fence();
        // what the state's gradient gets from the outputs
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                G[s][e] *= p.scale * since[2 * s + (e >> 2)][e & 3];
            const Parts<kParts> X = split8<kParts>(G[s]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (s == 0)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        S[i][r] *= whole;
                S[i] = mm<kParts>(qt[i][s], X, S[i]);
            }
        }
        fetch_queries(next);
        sched_fence();
        block_sync();  // one a chunk: the two halves of what is shared take turns
        float dU[2][8];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const v4f c = spans_sum<KP>(share[chunk & 1], h, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                dU[h >> 1][4 * (h & 1) + r] = c[r];
        }
        // dR
        v4f dR[4];
        const Parts<kParts> u1 = split8<kParts>(dU[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            dR[2 + h] = mm<kParts>(tri[frag_of_upper(1, h, 1)], u1, v4f{0.f, 0.f, 0.f, 0.f});
        const Parts<kParts> r1 = split_tiles<kParts>(dR[2], dR[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const v4f c = mm<kParts>(tri[frag_of_upper(0, h, 1)], r1, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r)
                dU[0][4 * h + r] -= c[r];
        }
        const Parts<kParts> u0 = split8<kParts>(dU[0]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            dR[h] = mm<kParts>(tri[frag_of_upper(0, h, 0)], u0, v4f{0.f, 0.f, 0.f, 0.f});
        if (live) {
            const uint32_t step = opaque_uniform((uint32_t)p.Dv * 4), off = opaque((uint32_t)q8 * step);
            char *out = (char *)(p.gr + at * 64 * p.Dv + dv);
#pragma unroll
            for (int h = 0; h < 4; ++h)
                if (h / OWN == wave)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        *(float *)(out + (off + (32 * (h >> 1) + 4 * (h & 1) + r) * step)) = dR[h][r];
        }
        // the state's gradient before the chunk
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int h = 2 * s + (e >> 2), r = e & 3;
                w[e] = -since[h][r] * beta[h][r] * dR[h][r];
            }
            const Parts<kParts> W = split8<kParts>(w);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                S[i] = mm<kParts>(kt[i][s], W, S[i]);
        }
        fetch_rest(next, ahead);
    }
    float *out = p.chunk_from > 0 ? p.carry : p.ginit;
    if (out && live)
        state_store<1>(S, out + bh * p.Dk * p.Dv + state_at0, many, p.Dv);
}

// -------------------------------------------------------- gradients: every chunk by itself

constexpr int kGradStride = 72;   // 64 columns and room against bank conflicts

// ROWS rows by 8 ACROSS columns of a float32 matrix in memory, on their way into shared memory in parts, row-major,
// by 256 threads: units of eight neighbours. Zeros from `in` rows and `cols` columns on.
template <int ROWS, int ACROSS>
struct GradBlocks {
    static constexpr int units = (ROWS * ACROSS + 255) / 256;
    float v[units][8];
};
template <int ROWS, int ACROSS>
SSD_DEVICE void grad_load(GradBlocks<ROWS, ACROSS> &d, const float *src, int stride, int in, int cols)
{
    const uint32_t step = opaque_uniform((uint32_t)stride * 4);
    const int thread = (int)opaque((uint32_t)thread_id());
    const char *x = (const char *)src;
#pragma unroll
    for (int i = 0; i < d.units; ++i) {
        const int unit = thread + 256 * i, r = unit / ACROSS, c = 8 * (unit % ACROSS);
        const uint32_t off = (uint32_t)(r < in ? r : in - 1) * step;
        if (cols % 4 == 0) {
            v4f lo, hi;  // at the alignment of an element: the stored states are the caller's
            __builtin_memcpy(&lo, x + (off + 4 * (uint32_t)(c < cols ? c : 0)), sizeof(lo));
            __builtin_memcpy(&hi, x + (off + 4 * (uint32_t)(c + 4 < cols ? c + 4 : 0)), sizeof(hi));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                d.v[i][e] = e < 4 ? lo[e & 3] : hi[e & 3];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                d.v[i][e] = *(const float *)(x + (off + 4 * (uint32_t)(c + e < cols ? c + e : 0)));
        }
    }
}
template <int ROWS, int ACROSS>
SSD_DEVICE void grad_clear(GradBlocks<ROWS, ACROSS> &d, int in, int cols)
{
    if (in >= ROWS && cols >= 8 * ACROSS)
        return;
#pragma unroll
    for (int i = 0; i < d.units; ++i) {
        const int unit = thread_id() + 256 * i, r = unit / ACROSS, c = 8 * (unit % ACROSS);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            d.v[i][e] = r < in && c + e < cols ? d.v[i][e] : 0.f;
    }
}
template <int ROWS, int ACROSS, int STRIDE>
SSD_DEVICE void grad_store(const GradBlocks<ROWS, ACROSS> &d, uint16_t *dst)
{
#pragma unroll
    for (int i = 0; i < d.units; ++i) {
        const int unit = thread_id() + 256 * i, r = unit / ACROSS, c = 8 * (unit % ACROSS);
        const Parts<kParts> parts = split8<kParts>(d.v[i]);
#pragma unroll
        for (int e = 0; e < kParts; ++e)
            *(v4u *)(dst + (e * ROWS + r) * STRIDE + c) = parts.p[e];
    }
}
template <int ROWS, int STRIDE>
SSD_DEVICE Parts<kParts> grad_operand(const uint16_t *at)
{
    Parts<kParts> r;
#pragma unroll
    for (int i = 0; i < kParts; ++i)
        r.p[i] = *(const v4u *)(at + i * ROWS * STRIDE);
    return r;
}

// Eight features of a token from `at` on, as they lie in memory; what lies past the D features, or belongs to no
// token, is cleared as the values are used.
template <int T>
SSD_DEVICE void row_load(Raw8<T> &raw, const typename DeltaElem<T>::type *p, int at, int D)
{
    if (D % 8 == 0) {
        __builtin_memcpy(&raw, p + (at < D ? at : 0), sizeof(raw));
    } else {
        typename DeltaElem<T>::type v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = p[at + e < D ? at + e : 0];
        __builtin_memcpy(&raw, v, sizeof(raw));
    }
}
// Whole: all lanes hold eight features of a token.
template <int T>
SSD_DEVICE void row_values(const Raw8<T> &raw, int at, int D, bool in, bool whole, float (&v)[8])
{
    unpack8<T>(raw, v);
    if (!whole)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = in && at + e < D ? v[e] : 0.f;
}
SSD_DEVICE Parts<1> row_parts(const Raw8<kBF16> &raw)
{
    Parts<1> r;
    r.p[0] = raw.w[0];
    return r;
}
SSD_DEVICE Parts<3> row_parts(const Raw8<kF32> &raw)
{
    float v[8];
    unpack8<kF32>(raw, v);
    return split8<3>(v);
}
template <int T>
SSD_DEVICE Parts<DeltaElem<T>::parts> row_operand(const Raw8<T> &raw, int at, int D, bool in, bool whole)
{
    if (whole)
        return row_parts(raw);
    float v[8];
    row_values<T>(raw, at, D, in, false, v);
    return split8<DeltaElem<T>::parts>(v);
}

// Sum over the four quarters of a wave, in every lane.
SSD_DEVICE float quarter_sum(float v)
{
    const int lane = thread_id() & 63;
    v += lane_fetch(v, lane ^ 16);
    return v + lane_fetch(v, lane ^ 32);
}

// Shared memory of the gradients' kernel. The columns are gone through 64 at a time: first U and dR stand in it (for the
// products over the tokens), then the state and its gradient, 32 of their columns at a time with wide keys; at the
// end K and Q by features. The triangle, from which U is made, lies where dR comes to stand, unless there are
// more columns.
template <int T, int KP, bool MANY>
struct GradLds {
    typedef typename DeltaElem<T>::type E;
    static constexpr int TS = 64 + DeltaElem<T>::pad, RS = 32 * KP + DeltaElem<T>::pad;
    static constexpr int SW = KP <= 2 ? 64 : 32, SS = SW + 8;  // columns of the state at a time
    static constexpr int u_size = kParts * 64 * kGradStride, s_size = kParts * 32 * KP * SS;
    static constexpr int tri_bytes = kParts * kDeltaFrags * 64 * 16;
    static_assert(tri_bytes <= u_size * 2, "the triangle fits where dR comes to stand");
    union {
        struct {
            uint16_t u[u_size], r[u_size];
        } a;
        struct {
            uint16_t s[s_size], gs[s_size];
        } b;
        struct {
            E qt[32 * KP * TS], kt[32 * KP * TS];
        } c;
    };
    static constexpr bool KEEP = T == kBF16;  // K by features has room of its own from the start
    char own_tri[MANY ? tri_bytes : 16];
    E k[64 * RS], own_kt[KEEP ? 32 * KP * TS : 8];
    DeltaGates gates;
    float beta[4][64];   // shares of dbeta
    float sums[64];      // dG
    float dots[4];       // shares of <S', dS'>
};

// dQ, dK, dV, dg and dbeta of a chunk and value head. A wave takes 16 tokens as columns of everything: lane l token
// 16 w + l, and as rows the features or the other tokens. Where value heads share a key head, their dQ and dK
// go to memory in float32 and are added afterwards. 32 x 2048 tokens on 16 heads of 64 in bfloat16: 800 us; VALU 54 %,
// MFMA 21 %, and a wave waits 41 % of its time: 230 registers let two run on a SIMD. Where it spilled there, the
// gradients as a whole took 1709 us, without 1308 (now 1160). With more features or columns one wave runs on a SIMD, and with both
// it spills: 121 registers (488 bytes a lane) in bfloat16, 128 (516) in float32; 256 heads of 128, the gradients as a
// whole, 2335 us (1.5 GB) and 3654.
template <int T, int KP, bool MANY>
SSD_KERNEL_WAVES(256, (KP <= 2 && !MANY ? 2 : 1)) void delta_grad_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    typedef GradLds<T, KP, MANY> Lds;
    constexpr int TS = Lds::TS, RS = Lds::RS, SS = Lds::SS, SW = Lds::SW, IN = DeltaElem<T>::parts;
    SSD_LDS Lds lds;
    const int64_t id = block_id();
    const int chunk = (int)(id % p.chunks), hv = (int)(id / p.chunks % p.Hv), b = (int)(id / p.chunks / p.Hv);
    const int share = p.Hv / p.Hk, hk = hv / share, wave = wave_id(), lane = thread_id() & 63;
    const int l = thread_id() & 15, quarter = lane >> 4, q8 = 8 * quarter, own = 16 * wave + l;
    const int n = delta_chunk_tokens(delta_valid(p, b), chunk);
    const int rows = p.T - chunk * kDeltaChunk < 64 ? p.T - chunk * kDeltaChunk : 64;
    const int64_t token = (int64_t)b * p.T + chunk * kDeltaChunk;
    const int o_stride = p.Hv * p.Dv;
    E *gv = (E *)p.gv + token * o_stride + hv * p.Dv;
    if (n == 0) {  // padding
        for (int i = thread_id(); i < rows; i += 256)
            p.gg[(token + i) * p.Hv + hv] = p.gbeta[(token + i) * p.Hv + hv] = 0.f;
        for (int i = thread_id(); i < rows * p.Dv; i += 256)
            delta_store<T>(gv + (int64_t)(i / p.Dv) * o_stride + i % p.Dv, 0.f);
        for (int i = thread_id(); i < rows * p.Dk; i += 256) {
            const int t = i / p.Dk, f = i % p.Dk;
            if (share > 1) {
                const int64_t to = ((token + t) * p.Hv + hv) * p.Dk + f;
                p.wq[to] = p.wk[to] = 0.f;
            } else {
                const int64_t to = ((token + t) * p.Hk + hk) * p.Dk + f;
                delta_store<T>((E *)p.gq + to, 0.f);
                delta_store<T>((E *)p.gk + to, 0.f);
            }
        }
        return;
    }
    const E *q = (const E *)p.q + token * p.q_stride + hk * p.Dk, *k = (const E *)p.k + token * p.k_stride + hk * p.Dk;
    const int64_t at = ((int64_t)b * p.Hv + hv) * p.chunks + chunk;
    const float *S = p.chunk_states + (((int64_t)b * p.chunks + chunk) * p.Hv + hv) * p.Dk * p.Dv;
    const float *gs = p.gs + at * p.Dk * p.Dv, *gr = p.gr + at * 64 * p.Dv;
    const E *v = (const E *)p.v + token * p.v_stride + hv * p.Dv, *go = (const E *)p.go + token * o_stride + hv * p.Dv;
    v4u *const tri = (v4u *)(MANY ? lds.own_tri : (char *)lds.a.r);
    v4f aq[2 * KP], reads[2 * KP], writes[2 * KP], m1t[4], m1[4], m2t[4], m2[4];
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i)
        aq[i] = reads[i] = writes[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m1t[i] = m1[i] = m2t[i] = m2[i] = v4f{0.f, 0.f, 0.f, 0.f};
    float dot = 0.f;
    // the first columns' values are on their way while the triangle is made
    v4f s[2 * KP];
    uint32_t vraw[2][8];
    float R[2][8], by[2][8];
    auto fetch_columns = [&](int col) {
        const int dv = col + 16 * wave + l;
        state_fetch<KP>(s, S + (dv < p.Dv ? dv : col), p.Dk, p.Dv);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int t = q8 < n - (32 * h + e) ? q8 + (32 * h + e) : n - 1;
                vraw[h][e] = delta_raw<T>(v + (uint32_t)t * (uint32_t)p.v_stride + (dv < p.Dv ? dv : col));
                by[h][e] = gr[(uint32_t)(q8 + (32 * h + e)) * (uint32_t)p.Dv + (dv < p.Dv ? dv : col)];
            }
    };
    Blocks<T, 32 * KP, 256> kb;
    blocks_load<T, 32 * KP, 256>(kb, k, (int)p.k_stride, p.Dk, n);
    float g0 = 0.f, beta0 = 0.f;
    if (wave == 3) {
        const int64_t from = (token + (lane < n ? lane : n - 1)) * p.Hv + hv;
        g0 = p.g[from];
        beta0 = p.beta[from];
    }
    fetch_columns(0);
    if (wave == 3)
        delta_gates_of(lds.gates, g0, beta0, n);
    E *const kt = Lds::KEEP ? lds.own_kt : lds.c.kt;
    blocks_store<T, 32 * KP, 256, true, Lds::KEEP>(kb, p.Dk, n, lds.k, kt);
    block_sync();
    const DeltaGates &gates = lds.gates;
    delta_tiles<T, KP, 4, false>(lds.k, nullptr, gates, 0.f, tri, nullptr);
    block_sync();
    if (wave < 2)
        delta_invert<false>(wave, tri);
    const E *kl = lds.k + tile_row(0, l) * RS + q8;
    const bool valid = own < n;
    for (int col = 0; MANY ? col < p.Dv : col == 0; col += 64) {
        const int cols = p.Dv - col;
        GradBlocks<64, 8> d;
        // U of 16 columns, as in the walk
        {
            const int dv = col + 16 * wave + l;
            const bool live = dv < p.Dv;
            if (MANY && col > 0)
                fetch_columns(col);
            state_mask<KP>(s, p.Dk);
            Parts<kParts> Sp[KP];
#pragma unroll
            for (int i = 0; i < KP; ++i)
                Sp[i] = split_tiles<kParts>(s[2 * i], s[2 * i + 1]);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                v4f ks = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int f = 0; f < KP; ++f)
                    ks = mm<kParts>(lds_operand(kl + ((32 * (h >> 1) + 4 * (h & 1)) * RS + 32 * f)), Sp[f], ks);
                const v4f since = *(const v4f *)(gates.since + q8 + (32 * (h >> 1) + 4 * (h & 1)));
                const v4f beta = *(const v4f *)(gates.beta + q8 + (32 * (h >> 1) + 4 * (h & 1)));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int e = 4 * (h & 1) + r;
                    const float x = live && q8 < n - (32 * (h >> 1) + e) ? delta_value<T>(vraw[h >> 1][e]) : 0.f;
                    const float read = x - since[r] * ks[r];
                    R[h >> 1][e] = live ? beta[r] * read : 0.f;
                    by[h >> 1][e] = live ? by[h >> 1][e] * read : 0.f;
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float sum = row16_sum(by[h][e]);
                    if (l == 0) {
                        float *to = &lds.beta[wave][q8 + (32 * h + e)];
                        *to = (MANY && col > 0 ? *to : 0.f) + sum;
                    }
                }
            grad_load<64, 8>(d, gr + col, p.Dv, 64, cols);
            block_sync();  // the triangle is there; with more columns the last ones have been read
            const Parts<kParts> R0 = split8<kParts>(R[0]);
            v4f U[2];
            uint16_t *to = lds.a.u + tile_row(0, l) * kGradStride + 16 * wave + 4 * quarter;
            auto put = [&](int s, int h, v4f x) {  // four columns of token 32 s + tile_row(h, l)
                const float w[8] = {x[0], x[1], x[2], x[3], 0.f, 0.f, 0.f, 0.f};
                const Parts<kParts> parts = split8<kParts>(w);
#pragma unroll
                for (int i = 0; i < kParts; ++i)
                    *(v2u *)(to + ((i * 64 + 32 * s + 4 * h) * kGradStride)) = v2u{parts.p[i][0], parts.p[i][1]};
            };
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const Parts<kParts> f = frag_operand<kParts>(tri, frag_of(0, h, 0));
                U[h] = mm<kParts>(f, R0, v4f{0.f, 0.f, 0.f, 0.f});
                put(0, h, mm<kParts>(R0, f, v4f{0.f, 0.f, 0.f, 0.f}));
            }
            const Parts<kParts> U0 = split_tiles<kParts>(U[0], U[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4f c = mm<kParts>(frag_operand<kParts>(tri, frag_of(1, h, 0)), U0, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    R[1][4 * h + r] -= c[r];
            }
            const Parts<kParts> R1 = split8<kParts>(R[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                put(1, h, mm<kParts>(R1, frag_operand<kParts>(tri, frag_of(1, h, 1)), v4f{0.f, 0.f, 0.f, 0.f}));
        }
        // dO of the own token and of those after, on its way
        const bool whole = n == 64 && cols >= 64;
        Raw8<T> oo[2], ao[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            row_load<T>(oo[t], go + (uint32_t)(valid ? own : 0) * (uint32_t)o_stride + col, 32 * t + q8, cols);
            if (Lds::KEEP)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((i >> 1) >= (wave >> 1)) {
                        const int row = 32 * (i >> 1) + tile_row(i & 1, l);
                        row_load<T>(ao[t][i], go + (uint32_t)(row < n ? row : 0) * (uint32_t)o_stride + col, 32 * t + q8, cols);
                    }
        }
        // dR, and dV = beta dR
        {
            if (!MANY)
                block_sync();  // the triangle has been read
            grad_clear<64, 8>(d, 64, cols);
            grad_store<64, 8, kGradStride>(d, lds.a.r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int unit = thread_id() + 256 * i, r = unit >> 3, c = 8 * (unit & 7);
                const float beta = gates.beta[r];  // zero in the padding
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = r < n ? beta * d.v[i][e] : 0.f;
                if (r < rows && c < cols)
                    store8<T>(gv + (uint32_t)r * (uint32_t)o_stride + col + c, cols - c, x);
            }
        }
        block_sync();
        // over the tokens; the state's first columns on their way
        GradBlocks<32 * KP, SW / 8> ds, dg;
        grad_load<32 * KP, SW / 8>(ds, S + col, p.Dv, p.Dk, cols);
        Parts<IN> op[2];
        Parts<kParts> ro[2], uo[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            op[t] = row_operand<T>(oo[t], 32 * t + q8, cols, valid, whole);
            ro[t] = grad_operand<64, kGradStride>(lds.a.r + own * kGradStride + q8 + 32 * t);
            uo[t] = grad_operand<64, kGradStride>(lds.a.u + own * kGradStride + q8 + 32 * t);
        }
        const uint16_t *ul = lds.a.u + tile_row(0, l) * kGradStride + q8, *rl = lds.a.r + tile_row(0, l) * kGradStride + q8;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at0 = (32 * (i >> 1) + 4 * (i & 1)) * kGradStride + 32 * t;
                if ((i >> 1) <= (wave >> 1)) {  // rows j up to the own token i
                    const Parts<kParts> u = grad_operand<64, kGradStride>(ul + at0);
                    m1t[i] = mm<kParts>(u, op[t], m1t[i]);
                    m2t[i] = mm<kParts>(u, ro[t], m2t[i]);
                }
                if ((i >> 1) >= (wave >> 1)) {  // rows i from the own token j on
                    const int row = 32 * (i >> 1) + tile_row(i & 1, l);
                    if (!Lds::KEEP)  // float32 rows would fill the registers
                        row_load<T>(ao[t][i], go + (uint32_t)(row < n ? row : 0) * (uint32_t)o_stride + col, 32 * t + q8, cols);
                    m1[i] = mm<kParts>(row_operand<T>(ao[t][i], 32 * t + q8, cols, row < n, whole), uo[t], m1[i]);
                    m2[i] = mm<kParts>(grad_operand<64, kGradStride>(rl + at0), uo[t], m2[i]);
                }
            }
        // over the state's columns
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += SW) {
            if (c0 >= cols)
                break;
            if (c0 > 0)
                grad_load<32 * KP, SW / 8>(ds, S + col + c0, p.Dv, p.Dk, cols - c0);
            grad_load<32 * KP, SW / 8>(dg, gs + col + c0, p.Dv, p.Dk, cols - c0);
            block_sync();  // U and dR, or the columns before, have been read
            grad_clear<32 * KP, SW / 8>(ds, p.Dk, cols - c0);
            grad_clear<32 * KP, SW / 8>(dg, p.Dk, cols - c0);
#pragma unroll
            for (int i = 0; i < ds.units; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dot = __builtin_fmaf(ds.v[i][e], dg.v[i][e], dot);
            grad_store<32 * KP, SW / 8, SS>(ds, lds.b.s);
            grad_store<32 * KP, SW / 8, SS>(dg, lds.b.gs);
            block_sync();
            const uint16_t *sl = lds.b.s + tile_row(0, l) * SS + q8, *gsl = lds.b.gs + tile_row(0, l) * SS + q8;
#pragma unroll
            for (int t = 0; t < SW / 32; ++t)
#pragma unroll
                for (int i = 0; i < 2 * KP; ++i) {
                    const int t0 = c0 / 32 + t, at0 = state_at(i, 0) * SS + 32 * t;
                    const Parts<kParts> s = grad_operand<32 * KP, SS>(sl + at0);
                    aq[i] = mm<kParts>(s, op[t0], aq[i]);
                    reads[i] = mm<kParts>(s, ro[t0], reads[i]);
                    writes[i] = mm<kParts>(grad_operand<32 * KP, SS>(gsl + at0), uo[t0], writes[i]);
                }
        }
        if (MANY)
            block_sync();  // before the next columns' U
    }
    dot = wave_sum(dot);
    Blocks<T, 32 * KP, 256> qb;
    blocks_load<T, 32 * KP, 256>(qb, q, (int)p.q_stride, p.Dk, n);
    Raw8<T> qo[KP];
#pragma unroll
    for (int s = 0; s < KP; ++s)
        row_load<T>(qo[s], q + (uint32_t)(valid ? own : 0) * (uint32_t)p.q_stride, 32 * s + q8, p.Dk);
    if (!Lds::KEEP)
        blocks_load<T, 32 * KP, 256>(kb, k, (int)p.k_stride, p.Dk, n);
    block_sync();
    if (!Lds::KEEP)
        blocks_store<T, 32 * KP, 256, false, true>(kb, p.Dk, n, (E *)nullptr, kt);
    blocks_store<T, 32 * KP, 256, false, true>(qb, p.Dk, n, (E *)nullptr, lds.c.qt);
    const double sum_own = gates.sum[own];
    const float since = gates.since[own], beta = gates.beta[own], hold = gates.left[own];
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            aq[i][r] *= p.scale * since;
            reads[i][r] *= -beta * since;
            writes[i][r] *= hold;
        }
    // the share of <S', dS'> that U brought: sum over tokens of k . (e^(G_C - G) U dS'^T)
    float held = 0.f, dots = 0.f;
    Parts<IN> ko[KP];
#pragma unroll
    for (int s = 0; s < KP; ++s) {
        float w[8];
        lds_values<T>(lds.k + own * RS + q8 + 32 * s, w);
        ko[s] = split8<IN>(w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            held = __builtin_fmaf(w[e], writes[2 * s + (e >> 2)][e & 3], held);
    }
    held = wave_sum(held);
    if (lane == 0)
        lds.dots[wave] = gates.whole * dot + held;
    block_sync();
    const E *ktl = kt + tile_row(0, l) * TS + q8, *qtl = lds.c.qt + tile_row(0, l) * TS + q8;
    float by_own = 0.f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (s <= (wave >> 1)) {  // token rows j at or before the own token i
            float d[8], e[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4f kk = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int f = 0; f < KP; ++f)
                    kk = mm<kParts>(lds_operand(kl + ((32 * s + 4 * h) * RS + 32 * f)), ko[f], kk);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 32 * s + 4 * h + r, behind = own - q8 - j;  // i - j
                    const float decay = behind >= 0 ? delta_exp(sum_own - gates.sum[q8 + j]) : 0.f;
                    const float x = behind > 0 ? -m2t[2 * s + h][r] * decay : 0.f;
                    d[4 * h + r] = behind >= 0 ? p.scale * decay * m1t[2 * s + h][r] : 0.f;
                    e[4 * h + r] = beta * x;
                    by_own = __builtin_fmaf(x, kk[r], by_own);
                }
            }
            const Parts<kParts> dp = split8<kParts>(d), ep = split8<kParts>(e);
#pragma unroll
            for (int i = 0; i < 2 * KP; ++i) {
                const auto a = lds_operand(ktl + (state_at(i, 0) * TS + 32 * s));
                aq[i] = mm<kParts>(a, dp, aq[i]);
                reads[i] = mm<kParts>(a, ep, reads[i]);
            }
        }
        if (s >= (wave >> 1)) {  // token rows i at or after the own token j
            float d[8], e[8];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = 32 * s + 4 * h + r, ahead = q8 + i - own;  // i - j
                    const float decay = ahead >= 0 ? delta_exp(gates.sum[q8 + i] - sum_own) : 0.f;
                    d[4 * h + r] = ahead >= 0 ? p.scale * decay * m1[2 * s + h][r] : 0.f;
                    e[4 * h + r] = ahead > 0 ? -gates.beta[q8 + i] * decay * m2[2 * s + h][r] : 0.f;
                }
            const Parts<kParts> dp = split8<kParts>(d), ep = split8<kParts>(e);
#pragma unroll
            for (int i = 0; i < 2 * KP; ++i) {
                writes[i] = mm<kParts>(lds_operand(qtl + (state_at(i, 0) * TS + 32 * s)), dp, writes[i]);
                writes[i] = mm<kParts>(lds_operand(ktl + (state_at(i, 0) * TS + 32 * s)), ep, writes[i]);
            }
        }
    }
    // q . dq + k . (reads - writes), and the results
#pragma unroll
    for (int s = 0; s < KP; ++s) {
        float x[8], y[8];
        const int f = 32 * s + q8;
        lds_values<T>(lds.k + own * RS + f, y);
        row_values<T>(qo[s], f, p.Dk, valid, n == 64 && p.Dk == 32 * KP, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = 2 * s + (e >> 2), r = e & 3;
            dots = __builtin_fmaf(x[e], aq[i][r], dots);
            dots = __builtin_fmaf(y[e], reads[i][r] - writes[i][r], dots);
            x[e] = aq[i][r];
            y[e] = reads[i][r] + writes[i][r];
        }
        if (own < rows && f < p.Dk) {
            if (share > 1) {
                const int64_t to = ((token + own) * p.Hv + hv) * p.Dk + f;
                store8<kF32>(p.wq + to, p.Dk - f, x);
                store8<kF32>(p.wk + to, p.Dk - f, y);
            } else {
                const int64_t to = ((token + own) * p.Hk + hk) * p.Dk + f;
                store8<T>((E *)p.gq + to, p.Dk - f, x);
                store8<T>((E *)p.gk + to, p.Dk - f, y);
            }
        }
    }
    dots = quarter_sum(dots);
    by_own = quarter_sum(by_own);
    if (quarter == 0) {
        lds.sums[own] = dots;
        lds.beta[0][own] = lds.beta[0][own] + lds.beta[1][own] + lds.beta[2][own] + lds.beta[3][own] + by_own;
    }
    block_sync();
    if (wave == 0) {
        // sums from the last token back: of everything less those before
        const double all = (double)lds.sums[lane] + (lane == n - 1 ? (double)lds.dots[0] + lds.dots[1] + lds.dots[2] + lds.dots[3] : 0.);
        const double before = wave_scan_d(all);
        const double total = lane_read_d(before, 63);
        if (lane < rows) {
            const int64_t to = (token + lane) * p.Hv + hv;
            p.gg[to] = lane < n ? (float)(total - before + all) : 0.f;
            p.gbeta[to] = lane < n ? lds.beta[0][lane] : 0.f;
        }
    }
}

// dQ and dK of key heads from those of the value heads that share them, in their order.
template <int T>
SSD_KERNEL(256) void delta_share_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    const int share = p.Hv / p.Hk;
    const int64_t total = (int64_t)p.B * p.T * p.Hk * p.Dk;
    for (int64_t i = block_id() * 256 + thread_id(); i < total; i += grid_blocks() * 256) {
        const int64_t from = i / p.Dk * share * p.Dk + i % p.Dk;
        float x = 0.f, y = 0.f;
        for (int s = 0; s < share; ++s) {
            x += p.wq[from + (int64_t)s * p.Dk];
            y += p.wk[from + (int64_t)s * p.Dk];
        }
        delta_store<T>((E *)p.gq + i, x);
        delta_store<T>((E *)p.gk + i, y);
    }
}

// out = from, or zeros.
SSD_KERNEL(256) void delta_copy_kernel(const float *from, float *out, int64_t n)
{
    for (int64_t i = block_id() * 256 + thread_id(); i < n; i += grid_blocks() * 256)
        out[i] = from ? from[i] : 0.f;
}

}  // namespace ssd
