// ssd_delta_kernels.h -- the gated delta rule. Per sequence and value head, with the state S
// (Dk x Dv, float32) and a = exp(g),
//     u_t = beta_t (v_t - a_t S_{t-1}^T k_t)     S_t = a_t S_{t-1} + k_t u_t^T     o_t = scale S_t^T q_t
// For a chunk of 64 tokens with G the running sum of g in it, D_ij = exp(G_i - G_j) for i >= j and
// A_ij = beta_i D_ij k_i.k_j for i > j:
//     (I + A) U = R = beta (V - e^G K S)         O = scale (e^G Q S + (Q K^T o D) U)
//     S' = e^{G_C} S + (e^{G_C - G} K)^T U
// The columns of S, V, U and O (over Dv) do not meet, so a wave walks over the chunks with 16 columns
// of the state in its registers. The 64 x 64 system is solved in two blocks of 32, whose own
// inverses T_00 and T_11 are formed beforehand for all chunks at once (rows of 16 by substitution,
// which is stable whatever the keys, the rest by products):
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
constexpr int kDeltaFragFloats = kDeltaFrags * 64 * 8;

struct DeltaParams {
    const void *q, *k, *v;                // (B, T, heads, D), tokens *_stride elements apart
    const float *g, *beta;                // (B, T, Hv)
    const float *init;                    // nullable: (B, Hv, Dk, Dv)
    const int *lengths;                   // nullable: (B)
    void *o;                              // (B, T, Hv, Dv)
    float *final_state;                   // nullable: (B, Hv, Dk, Dv)
    float *states;                        // nullable: (B, chunks, Hv, Dk, Dv), the state entering each chunk
    float *tri;                           // (B, Hv, chunks) times kDeltaFragFloats: T_00, A_10, T_11
    // backward
    const float *chunk_states;
    const void *go;                       // (B, T, Hv, Dv)
    const float *gfinal;                  // nullable: (B, Hv, Dk, Dv)
    void *gq, *gk, *gv;                   // as q, k, v, dense
    float *gg, *gbeta;                    // (B, T, Hv)
    float *ginit;                         // nullable: (B, Hv, Dk, Dv)
    float *tri_t, *pt;                    // as tri: the transposed ones, and P^T
    float *gs;                            // (B, Hv, chunks, Dk, Dv): dS' of each chunk
    float *gr;                            // (B, Hv, chunks, 64, Dv): dR
    int64_t q_stride, k_stride, v_stride;
    int B, T, Hk, Hv, Dk, Dv, chunks;
    int columns;                          // column blocks of a head
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

// Which six operand tiles a lower (or upper) triangle of spans has.
SSD_DEVICE int frag_of(int s, int h, int t) { return s == 0 ? h : 2 + 2 * h + t; }          // t <= s
SSD_DEVICE int frag_of_upper(int s, int h, int t) { return s == 1 ? 4 + h : 2 * h + t; }    // t >= s

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
SSD_DEVICE float delta_exp(double log2) { return hw_exp2((float)log2); }

// What a chunk's decays are, for each of its tokens.
struct DeltaGates {
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
    static constexpr int across = COLS / 4, units = (16 * across + NT - 1) / NT;
    static constexpr bool even = 16 * across % NT == 0;
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
        if (D % 4 == 0 && n == 64 && d.even) {
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
        if (!d.even && t >= 64)
            break;
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
template <int T, int KP, bool ROWS, bool TURNED>
SSD_DEVICE void delta_stage(const void *src, int64_t stride, int D, int n, typename DeltaElem<T>::type *rows,
                            typename DeltaElem<T>::type *turned)
{
    Blocks<T, 32 * KP, 256> blocks;
    blocks_load<T, 32 * KP, 256>(blocks, src, (int)stride, D, n);
    blocks_store<T, 32 * KP, 256, ROWS, TURNED>(blocks, D, n, rows, turned);
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

constexpr int kTriStride = 68;

// Tile (ti, tj) of X Y^T: rows (lanes' components) of X, columns of Y, in tiles of 16 as they lie.
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

// A (below the diagonal, zeros on it) of a chunk into tri[64][kTriStride], by four waves; the two tiles
// above the diagonal that the blocks of 32 hold become zeros.
template <int T, int KP>
SSD_DEVICE void delta_products(const typename DeltaElem<T>::type *k, const DeltaGates &gates, float *tri)
{
    const int l = thread_id() & 15, q = (thread_id() & 63) >> 4;
    for (int i = wave_id(); i < 10; i += 4) {  // (0,0) (1,0) (1,1) (2,0) ... (3,3)
        const int ti = i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3, tj = i - ti * (ti + 1) / 2;
        const v4f c = delta_tile<T, KP>(k, tj, k, ti);  // rows j, column i
        const int row = 16 * ti + l, col = 16 * tj + 4 * q;
        v4f w;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            w[r] = row > col + r ? gates.beta[row] * delta_exp(gates.sum[row] - gates.sum[col + r]) * c[r] : 0.f;
        *(v4f *)(tri + row * kTriStride + col) = w;
    }
    if (wave_id() < 2) {
        const v4f zero = {0.f, 0.f, 0.f, 0.f};
        *(v4f *)(tri + (32 * wave_id() + l) * kTriStride + 32 * wave_id() + 16 + 4 * q) = zero;
    }
}

// The blocks of 16 on the diagonal become (I + A)^-1, by one wave: lane 16 d + c finds column c of
// block d, one value after the other.
SSD_DEVICE void delta_diagonal(float *tri)
{
    const int c = thread_id() & 15, d = (thread_id() & 63) >> 4;
    float *block = tri + 16 * d * kTriStride + 16 * d;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float s = i == c ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < i; j += 4) {
            const v4f a = *(const v4f *)(block + i * kTriStride + j);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < i)
                    s = __builtin_fmaf(-a[e], x[j + e], s);
        }
        x[i] = s;
    }
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < 16; ++i)
        block[i * kTriStride + c] = x[i];
    wave_lds_sync();
}

// ... and the block of 32 around two of them: - T_1 A T_0 in its lower left, by one wave.
SSD_DEVICE void delta_corner(float *tri, int pair)
{
    const int l = thread_id() & 15, q = (thread_id() & 63) >> 4;
    float *t0 = tri + 32 * pair * kTriStride + 32 * pair, *a = t0 + 16 * kTriStride, *t1 = a + 16;
    const v4f ra = *(const v4f *)(a + l * kTriStride + 4 * q), r1 = *(const v4f *)(t1 + l * kTriStride + 4 * q);
    v4f y = {0.f, 0.f, 0.f, 0.f}, z = y;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        y = mfma_16x16x4(ra[r], t0[(4 * q + r) * kTriStride + l], y);
#pragma unroll
    for (int r = 0; r < 4; ++r)
        z = mfma_16x16x4(r1[r], -y[r], z);
    wave_lds_sync();
#pragma unroll
    for (int r = 0; r < 4; ++r)
        a[(4 * q + r) * kTriStride + l] = z[r];
}

// The triangles of every chunk (and, for the backward pass, their transposes and P^T), in the order in
// which the walks read them as operands: tile, lane, eight values.
template <int T, int KP, bool BACKWARD>
SSD_KERNEL(256) void delta_prepare_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    constexpr int RS = 32 * KP + DeltaElem<T>::pad;
    SSD_LDS E k[64 * RS], q[BACKWARD ? 64 * RS : 8];
    SSD_LDS float tri[64 * kTriStride], pp[BACKWARD ? 64 * kTriStride : 4];
    SSD_LDS DeltaGates gates;
    const int64_t id = block_id();
    const int chunk = (int)(id % p.chunks), hv = (int)(id / p.chunks % p.Hv), b = (int)(id / p.chunks / p.Hv);
    const int hk = hv / (p.Hv / p.Hk);
    const int n = delta_chunk_tokens(delta_valid(p, b), chunk);
    if (n == 0)
        return;
    const int64_t token = (int64_t)b * p.T + chunk * kDeltaChunk;
    delta_stage<T, KP, true, false>((const E *)p.k + token * p.k_stride + hk * p.Dk, p.k_stride, p.Dk, n, k, nullptr);
    if (BACKWARD)
        delta_stage<T, KP, true, false>((const E *)p.q + token * p.q_stride + hk * p.Dk, p.q_stride, p.Dk, n, q, nullptr);
    if (wave_id() == 0)
        delta_gates(gates, p.g, p.beta, token * p.Hv + hv, p.Hv, n);
    block_sync();
    delta_products<T, KP>(k, gates, tri);
    const int l = thread_id() & 15, quarter = (thread_id() & 63) >> 4;
    if (BACKWARD) {
        for (int i = wave_id(); i < 10; i += 4) {
            const int ti = i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3, tj = i - ti * (ti + 1) / 2;
            const v4f c = delta_tile<T, KP>(q, ti, k, tj);  // rows i, column j
            const int row = 16 * ti + 4 * quarter, col = 16 * tj + l;
            v4f w;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                w[r] = row + r >= col ? p.scale * delta_exp(gates.sum[row + r] - gates.sum[col]) * c[r] : 0.f;
            *(v4f *)(pp + col * kTriStride + row) = w;  // P^T: row j, column i
        }
        if (wave_id() < 2) {  // what lies below its diagonal in the blocks of 32
            const v4f zero = {0.f, 0.f, 0.f, 0.f};
            *(v4f *)(pp + (32 * wave_id() + 16 + l) * kTriStride + 32 * wave_id() + 4 * quarter) = zero;
        }
    }
    block_sync();
    if (wave_id() == 0)
        delta_diagonal(tri);
    block_sync();
    if (wave_id() < 2)
        delta_corner(tri, wave_id());
    block_sync();
    const int64_t out = id * kDeltaFragFloats;
    for (int unit = thread_id(); unit < kDeltaFrags * 64; unit += 256) {
        const int f = unit >> 6, m = unit & 15, k8 = 8 * ((unit & 63) >> 4);
        {
            const int s = f >= 2, h = s ? (f - 2) >> 1 : f, t = s ? (f - 2) & 1 : 0;
            const float *row = tri + (32 * s + tile_row(h, m)) * kTriStride + 32 * t + k8;
            *(v4f *)(p.tri + out + 8 * unit) = *(const v4f *)row;
            *(v4f *)(p.tri + out + 8 * unit + 4) = *(const v4f *)(row + 4);
        }
        if (BACKWARD) {
            const int s = f >= 4, h = s ? f - 4 : f >> 1, t = s ? 1 : f & 1;
            const int j = 32 * s + tile_row(h, m);
            const float *row = pp + j * kTriStride + 32 * t + k8;
            *(v4f *)(p.pt + out + 8 * unit) = *(const v4f *)row;
            *(v4f *)(p.pt + out + 8 * unit + 4) = *(const v4f *)(row + 4);
            v4f a, c;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = tri[(32 * t + k8 + e) * kTriStride + j];
                c[e] = tri[(32 * t + k8 + 4 + e) * kTriStride + j];
            }
            *(v4f *)(p.tri_t + out + 8 * unit) = a;
            *(v4f *)(p.tri_t + out + 8 * unit + 4) = c;
        }
    }
}

// Operand tiles from memory (as delta_prepare_kernel leaves them) into shared memory in parts.
template <int N>
SSD_DEVICE void delta_stage_frags(const float *src, v4u *dst, int threads)
{
    for (int unit = thread_id(); unit < kDeltaFrags * 64; unit += threads) {
        const Parts<N> r = split_tiles<N>(*(const v4f *)(src + 8 * unit), *(const v4f *)(src + 8 * unit + 4));
#pragma unroll
        for (int i = 0; i < N; ++i)
            dst[(i * kDeltaFrags + (unit >> 6)) * 64 + (unit & 63)] = r.p[i];
    }
}
template <int N>
SSD_DEVICE Parts<N> frag_operand(const v4u *frags, int f)
{
    Parts<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i)
        r.p[i] = frags[(i * kDeltaFrags + f) * 64 + (thread_id() & 63)];
    return r;
}

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
        *(v2u *)((char *)&frags[(e * kDeltaFrags + f) * 64 + lane] + 2 * (j & 7)) = half;
    }
}

// A chunk's triangle and P, by all waves, in tiles of 16: A = beta D o K K^T below the diagonal and
// P = scale Q K^T o D. Of the two 32 x 32 blocks of I + A on the diagonal the inverses of their own blocks of 16 and
// A between them go into `pairs` (float32, transposed); A_10 and P into operand tiles. Each of the first four
// waves has one tile on the diagonal, the others are dealt out so that the first two, which finish the
// inverses afterwards, have the fewest.
template <int T, int KP, int OUT, int WAVES>
SSD_DEVICE void delta_tiles(const typename DeltaElem<T>::type *k, const typename DeltaElem<T>::type *q,
                            const DeltaGates &gates, float scale, float *pairs, v4u *tri, v4u *pf)
{
    const int l = thread_id() & 15, quarter = (thread_id() & 63) >> 4, wave = wave_id();
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
        if (has[c]) {
            kk[c] = delta_tile<T, KP>(k, tj[c], k, ti[c]);  // rows j, column i
            qk[c] = delta_tile<T, KP>(k, tj[c], q, ti[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < most; ++c) {
        if (!has[c])
            continue;
        const int i = 16 * ti[c] + l, j = 16 * tj[c] + 4 * quarter;
        const double sum = gates.sum[i];
        const float beta = gates.beta[i];
        v4f a, w;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float d = delta_exp(sum - gates.sum[j + r]);
            a[r] = c > 0 || i > j + r ? beta * d * kk[c][r] : 0.f;
            w[r] = c > 0 || i >= j + r ? scale * d * qk[c][r] : 0.f;
        }
        const int f = frag_of(i >> 5, i >> 2 & 1, j >> 5);
        frag_store<OUT>(pf, f, i, j, w);
        if (c == 0) {
            // column l of the block's inverse, in every quarter: each value is taken from all that follow it
            // as soon as it is known; the block's entries reach all lanes as scalars
            float x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
                x[e] = e == l ? 1.f : 0.f;
            const v4f minus = -a;
#pragma unroll
            for (int e = 0; e < 15; ++e)
#pragma unroll
                for (int u = e + 1; u < 16; ++u)
                    x[u] = __builtin_fmaf(lane_read(minus[e & 3], 16 * (e >> 2) + u), x[e], x[u]);
            if (quarter == 0)
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *(v4f *)(pairs + i * kPairStride + (16 * wave & 16) + e) = v4f{x[e], x[e + 1], x[e + 2], x[e + 3]};
        } else if (ti[c] >> 1 == tj[c] >> 1) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                pairs[(j + r) * kPairStride + (i & 31)] = a[r];
        } else {
            frag_store<kParts>(tri, f, i, j, a);
        }
    }
}

// The corner of the inverse of a block of 32 (held transposed), - T_1 A T_0, and the block into operand tiles, by
// one wave.
SSD_DEVICE void delta_invert(float *block, int pair, v4u *tri)
{
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
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // row i of the operand is column i of what is held
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = block[8 * quarter * kPairStride + tile_row(0, l) + (e * kPairStride + 4 * h)];
        const Parts<kParts> parts = split8<kParts>(v);
#pragma unroll
        for (int e = 0; e < kParts; ++e)
            tri[(e * kDeltaFrags + frag_of(pair, h, pair)) * 64 + (thread_id() & 63)] = parts.p[e];
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
SSD_DEVICE void state_load(v4f (&S)[2 * KP], const float *from, int Dk, int Dv)
{
    const int q8 = 8 * ((thread_id() & 63) >> 4);
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[i][r] = from[(uint32_t)(q8 < Dk - state_at(i, r) ? q8 + state_at(i, r) : 0) * (uint32_t)Dv];
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[i][r] = q8 < Dk - state_at(i, r) ? S[i][r] : 0.f;
}

// A workgroup takes 16 WAVES columns of a value head, a wave 16 of them: lane l the column l, and of 2 KP tiles
// the features 32 s + 8 q + 4 h + r of the state. The chunk's triangle and P are made by all of them; while two
// waves solve the blocks of 32, the others go on with what the state gives. The next chunk's rows are in
// flight meanwhile.
template <int T, int KP, int WAVES>
SSD_KERNEL_WAVES(64 * WAVES, 2) void delta_scan_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    constexpr int NT = 64 * WAVES, COLS = 16 * WAVES;
    constexpr int pad = DeltaElem<T>::pad, RS = 32 * KP + pad, TS = 64 + pad;
    constexpr int OUT = T == kBF16 ? 2 : 3;  // parts of what only reaches o
    constexpr bool STAGE_V = T == kBF16;      // float32 rows leave no room
    SSD_LDS E k[64 * RS], q[64 * RS], kt[32 * KP * TS], vt[STAGE_V ? COLS * TS : 8];
    SSD_LDS float pairs[64 * kPairStride];
    SSD_LDS v4u tri[kParts * kDeltaFrags * 64], pf[OUT * kDeltaFrags * 64];
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
    // above the diagonal the blocks (held transposed) and tiles stay zero
    for (int i = thread_id(); i < 16 * 16; i += NT)
        pairs[(16 + (i >> 4)) * kPairStride + (i & 15)] = pairs[(48 + (i >> 4)) * kPairStride + (i & 15)] = 0.f;
    for (int i = thread_id(); i < OUT * kDeltaFrags * 64; i += NT)
        pf[i] = v4u{0u, 0u, 0u, 0u};
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
        delta_tiles<T, KP, OUT, WAVES>(k, q, gates, p.scale, pairs, tri, pf);
        block_sync();
        if (wave < 2)
            delta_invert(pairs + 32 * wave * kPairStride, wave, tri);
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
                Raw8<T> raw;
                raw.w[0] = *(const v4u *)(vl + 32 * s);
                unpack8<T>(raw, v);
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
                    ks = mm<kParts>(lds_operand(kl + ((32 * s + 4 * h) * RS + 32 * f)), Sp[f], ks);
                    qs = mm<OUT>(lds_operand(ql + ((32 * s + 4 * h) * RS + 32 * f)), Sp[f], qs);
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
                c = mm<OUT>(frag_operand<OUT>(pf, frag_of(s, h, 0)), U0, c);
                if (s == 1)
                    c = mm<OUT>(frag_operand<OUT>(pf, frag_of(1, h, 1)), U1, c);
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

// ------------------------------------------------------------ a few tokens on the state

constexpr int kDeltaFew = 8;  // tokens that are walked one by one

// A wave holds 16 columns of the state: lane 16 c + r the rows r, r + 16, ... of the columns
// 4 c .. 4 c + 3. Sums over rows go over the 16 lanes.
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
    for (int i = 0; i < ROWS; ++i) {
        const float *at = p.init + head + (int64_t)(r + 16 * i) * p.Dv + dv;
        const bool in = p.init && r + 16 * i < p.Dk;
        if (in && left >= 4) {
            __builtin_memcpy(S[i], at, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[i][e] = in && e < left ? at[e] : 0.f;
        }
    }
    if (p.states)  // one chunk
        store(p.states + head);
    const int64_t o_stride = (int64_t)p.Hv * p.Dv;
    for (int t = 0; t < p.T; ++t) {
        const int64_t token = (int64_t)b * p.T + t;
        E *o = (E *)p.o + token * o_stride + hv * p.Dv + dv;
        float out[4] = {0.f, 0.f, 0.f, 0.f};
        if (t < length) {
            const E *q = (const E *)p.q + token * p.q_stride + hk * p.Dk;
            const E *k = (const E *)p.k + token * p.k_stride + hk * p.Dk;
            const E *v = (const E *)p.v + token * p.v_stride + hv * p.Dv + dv;
            const float a = delta_exp(delta_log2(p.g[token * p.Hv + hv])), beta = p.beta[token * p.Hv + hv];
            float kr[ROWS], qr[ROWS], u[4];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const bool in = r + 16 * i < p.Dk;
                kr[i] = in ? delta_load<T>(k + r + 16 * i) : 0.f;
                qr[i] = in ? delta_load<T>(q + r + 16 * i) : 0.f;
            }
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
                const float x = e < left ? delta_load<T>(v + e) : 0.f;
                u[e] = beta * (x - row16_sum(u[e]));
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
        if (r == 0)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left)
                    delta_store<T>(o + e, out[e]);
    }
    if (p.final_state)
        store(p.final_state + head);
}

// ------------------------------------------------------------ gradients: the walk backwards

// Eight tokens of one column as an operand: tokens at p and every `stride` after it, `n` of them.
template <int T>
SSD_DEVICE Parts<DeltaElem<T>::parts> column_operand(const typename DeltaElem<T>::type *p, int64_t stride, int n)
{
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = e < n ? delta_load<T>(p + e * stride) : 0.f;
    return split8<DeltaElem<T>::parts>(v);
}

// As delta_scan_kernel, from the last chunk to the first, with the gradient of the state.
template <int T, int KP>
SSD_KERNEL(256) void delta_scan_bwd_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    constexpr int pad = DeltaElem<T>::pad, RS = 32 * KP + pad, TS = 64 + pad;
    constexpr int IN = DeltaElem<T>::parts;
    SSD_LDS E k[64 * RS], kt[32 * KP * TS], qt[32 * KP * TS];
    SSD_LDS v4u tri[kParts * kDeltaFrags * 64], pt[kParts * kDeltaFrags * 64];
    SSD_LDS DeltaGates gates;
    const int64_t id = block_id();
    const int block = (int)(id % p.columns), hv = (int)(id / p.columns % p.Hv), b = (int)(id / p.columns / p.Hv);
    const int hk = hv / (p.Hv / p.Hk);
    const int l = thread_id() & 15, quarter = (thread_id() & 63) >> 4;
    const int dv = 64 * block + 16 * wave_id() + l;
    const bool live = dv < p.Dv;
    const int64_t head = ((int64_t)b * p.Hv + hv) * p.Dk * p.Dv;
    v4f S[2 * KP];  // the gradient of the state after the chunk
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int f = 32 * (i >> 1) + 8 * quarter + 4 * (i & 1) + r;
            S[i][r] = p.gfinal && live && f < p.Dk ? p.gfinal[head + (int64_t)f * p.Dv + dv] : 0.f;
        }
    const int length = delta_valid(p, b);
    const int row_dv = hv * p.Dv + dv;
    const int64_t o_stride = (int64_t)p.Hv * p.Dv;
    for (int chunk = p.chunks - 1; chunk >= 0; --chunk) {
        const int n = delta_chunk_tokens(length, chunk);
        const int64_t token = (int64_t)b * p.T + chunk * kDeltaChunk;
        const int rows = p.T - chunk * kDeltaChunk < 64 ? p.T - chunk * kDeltaChunk : 64;
        E *gv = (E *)p.gv + token * o_stride + row_dv;
        if (n == 0) {  // padding
            if (live)
                for (int t = quarter; t < rows; t += 4)
                    delta_store<T>(gv + t * o_stride, 0.f);
            continue;
        }
        const int64_t at = ((int64_t)b * p.Hv + hv) * p.chunks + chunk;
        block_sync();  // the last chunk's operands have been read
        delta_stage<T, KP, true, true>((const E *)p.k + token * p.k_stride + hk * p.Dk, p.k_stride, p.Dk, n, k, kt);
        delta_stage<T, KP, false, true>((const E *)p.q + token * p.q_stride + hk * p.Dk, p.q_stride, p.Dk, n, nullptr, qt);
        delta_stage_frags<kParts>(p.tri_t + at * kDeltaFragFloats, tri, 256);
        delta_stage_frags<kParts>(p.pt + at * kDeltaFragFloats, pt, 256);
        if (wave_id() == 0)
            delta_gates(gates, p.g, p.beta, token * p.Hv + hv, p.Hv, n);
        if (live) {
            float *to = p.gs + at * p.Dk * p.Dv + dv;
#pragma unroll
            for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int f = 32 * (i >> 1) + 8 * quarter + 4 * (i & 1) + r;
                    if (f < p.Dk)
                        to[(int64_t)f * p.Dv] = S[i][r];
                }
        }
        block_sync();
        // dU = P^T dO + e^(G_C - G) K dS'
        Parts<kParts> Sp[KP];
#pragma unroll
        for (int s = 0; s < KP; ++s)
            Sp[s] = split_tiles<kParts>(S[2 * s], S[2 * s + 1]);
        const E *go = (const E *)p.go + token * o_stride + (live ? row_dv : 0);
        Parts<IN> G[2];
        float raw[2][8];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int t = 32 * s + 8 * quarter;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                raw[s][e] = delta_load<T>(go + (t + e < n ? t + e : n - 1) * o_stride);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                raw[s][e] = live && t + e < n ? raw[s][e] : 0.f;
            G[s] = split8<IN>(raw[s]);
        }
        float dU[2][8], dR[2][8];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4f c = {0.f, 0.f, 0.f, 0.f}, ks = c;
                const int row = (32 * s + tile_row(h, l)) * RS + 8 * quarter;
#pragma unroll
                for (int f = 0; f < KP; ++f)
                    ks = mm<kParts>(lds_operand(k + row + 32 * f), Sp[f], ks);
#pragma unroll
                for (int t = s; t < 2; ++t)
                    c = mm<kParts>(frag_operand<kParts>(pt, frag_of_upper(s, h, t)), G[t], c);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    dU[s][4 * h + r] = c[r] + gates.left[32 * s + 8 * quarter + 4 * h + r] * ks[r];
            }
        // dR
        const Parts<kParts> u1 = split8<kParts>(dU[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const v4f c = mm<kParts>(frag_operand<kParts>(tri, frag_of_upper(1, h, 1)), u1, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r)
                dR[1][4 * h + r] = c[r];
        }
        const Parts<kParts> r1 = split8<kParts>(dR[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const v4f c = mm<kParts>(frag_operand<kParts>(tri, frag_of_upper(0, h, 1)), r1, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r)
                dU[0][4 * h + r] -= c[r];
        }
        const Parts<kParts> u0 = split8<kParts>(dU[0]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const v4f c = mm<kParts>(frag_operand<kParts>(tri, frag_of_upper(0, h, 0)), u0, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r)
                dR[0][4 * h + r] = c[r];
        }
        // dR and dV out, and the state's gradient before the chunk
        Parts<kParts> W[2], X[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float w[8], x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int t = 32 * s + 8 * quarter + e;
                const float by = gates.beta[t] * dR[s][e];
                if (live) {
                    p.gr[(at * 64 + t) * p.Dv + dv] = dR[s][e];
                    if (t < rows)
                        delta_store<T>(gv + t * o_stride, t < n ? by : 0.f);
                }
                w[e] = -gates.since[t] * by;
                x[e] = p.scale * gates.since[t] * raw[s][e];
            }
            W[s] = split8<kParts>(w);
            X[s] = split8<kParts>(x);
        }
        const float whole = gates.whole;
#pragma unroll
        for (int i = 0; i < 2 * KP; ++i) {
            v4f c;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                c[r] = whole * S[i][r];
            const int row = (32 * (i >> 1) + tile_row(i & 1, l)) * TS + 8 * quarter;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                c = mm<kParts>(lds_operand(qt + row + 32 * s), X[s], c);
                c = mm<kParts>(lds_operand(kt + row + 32 * s), W[s], c);
            }
            S[i] = c;
        }
    }
    if (p.ginit && live)
#pragma unroll
        for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int f = 32 * (i >> 1) + 8 * quarter + 4 * (i & 1) + r;
                if (f < p.Dk)
                    p.ginit[head + (int64_t)f * p.Dv + dv] = S[i][r];
            }
}

// -------------------------------------------------------- gradients: every chunk by itself

constexpr int kGradCols = 32;            // columns (over Dv) held at a time
constexpr int kGradStride = kGradCols + 8;

// Rows by kGradCols columns of a matrix in memory into shared memory in N parts, row-major; zeros from
// `rows_in` and from `cols` on.
template <int T, int N>
SSD_DEVICE void grad_stage(const typename DeltaElem<T>::type *src, int64_t stride, int rows, int rows_in, int cols,
                           uint16_t *dst, int thread, int threads)
{
    for (int unit = thread; unit < rows * (kGradCols / 8); unit += threads) {
        const int row = unit / (kGradCols / 8), col = 8 * (unit % (kGradCols / 8));
        float v[8];
        unpack8<T>(load8<T>(src + (row < rows_in ? row * stride : 0) + (cols > col ? col : 0),
                            row < rows_in ? cols - col : 0), v);
        const Parts<N> r = split8<N>(v);
#pragma unroll
        for (int i = 0; i < N; ++i)
            *(v4u *)(dst + (i * rows + row) * kGradStride + col) = r.p[i];
    }
}
template <int N>
SSD_DEVICE Parts<N> grad_operand(const uint16_t *src, int rows, int row)
{
    Parts<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i)
        r.p[i] = *(const v4u *)(src + (i * rows + row) * kGradStride + 8 * ((thread_id() & 63) >> 4));
    return r;
}

// Eight features of a token as an operand, from memory.
template <int T>
SSD_DEVICE Parts<DeltaElem<T>::parts> row_operand(const typename DeltaElem<T>::type *p, int at, int n)
{
    float v[8];
    unpack8<T>(load8<T>(p + (n > at ? at : 0), n - at), v);
    return split8<DeltaElem<T>::parts>(v);
}

template <int T, int KP>
struct GradLds {
    typedef typename DeltaElem<T>::type E;
    static constexpr int TS = 64 + DeltaElem<T>::pad, IN = DeltaElem<T>::parts;
    union {
        struct {  // while the columns are gone through
            uint16_t u[kParts * 64 * kGradStride], r[kParts * 64 * kGradStride], o[IN * 64 * kGradStride];
            uint16_t s[kParts * 32 * KP * kGradStride], gs[kParts * 32 * KP * kGradStride];
        } a;
        struct {  // after
            E kt[32 * KP * TS], qt[32 * KP * TS];
        } b;
    };
    DeltaGates gates;
    float beta[2][64];   // shares of dbeta
    float sums[64];      // dG
    float dots[4];       // shares of <S, dS'>
};

// Sum over the four quarters of a wave, in every lane.
SSD_DEVICE float quarter_sum(float v)
{
    const int lane = thread_id() & 63;
    v += lane_fetch(v, lane ^ 16);
    return v + lane_fetch(v, lane ^ 32);
}

// dQ, dK, dg and dbeta of a chunk, of one key head: its value heads one after the other. A wave takes 16
// tokens as columns of everything: lane l token 16 w + l, and as rows the features or the other tokens.
template <int T, int KP>
SSD_KERNEL(256) void delta_grad_kernel(DeltaParams p)
{
    typedef typename DeltaElem<T>::type E;
    constexpr int TS = 64 + DeltaElem<T>::pad, IN = DeltaElem<T>::parts;
    SSD_LDS GradLds<T, KP> lds;
    const int64_t id = block_id();
    const int chunk = (int)(id % p.chunks), hk = (int)(id / p.chunks % p.Hk), b = (int)(id / p.chunks / p.Hk);
    const int share = p.Hv / p.Hk, wave = wave_id();
    const int l = thread_id() & 15, quarter = (thread_id() & 63) >> 4, own = 16 * wave + l, lane = thread_id() & 63;
    const int n = delta_chunk_tokens(delta_valid(p, b), chunk);
    const int rows = p.T - chunk * kDeltaChunk < 64 ? p.T - chunk * kDeltaChunk : 64;
    const int64_t token = (int64_t)b * p.T + chunk * kDeltaChunk;
    const int64_t dense = (int64_t)p.Hk * p.Dk, o_stride = (int64_t)p.Hv * p.Dv;
    E *gq = (E *)p.gq + (token + own) * dense + hk * p.Dk, *gk = (E *)p.gk + (token + own) * dense + hk * p.Dk;
    const E *q = (const E *)p.q + token * p.q_stride + hk * p.Dk, *k = (const E *)p.k + token * p.k_stride + hk * p.Dk;
    v4f tq[2 * KP], tk[2 * KP];
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i)
        tq[i] = tk[i] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int hv = hk * share; hv < (hk + 1) * share; ++hv) {
        if (n == 0) {  // padding
            if (thread_id() < rows)
                p.gg[(token + thread_id()) * p.Hv + hv] = p.gbeta[(token + thread_id()) * p.Hv + hv] = 0.f;
            continue;
        }
        const int64_t at = ((int64_t)b * p.Hv + hv) * p.chunks + chunk;
        const float *S = p.chunk_states + (((int64_t)b * p.chunks + chunk) * p.Hv + hv) * p.Dk * p.Dv;
        const float *gs = p.gs + at * p.Dk * p.Dv, *gr = p.gr + at * 64 * p.Dv;
        const E *v = (const E *)p.v + token * p.v_stride + hv * p.Dv, *go = (const E *)p.go + token * o_stride + hv * p.Dv;
        v4f aq[2 * KP], reads[2 * KP], writes[2 * KP], m1t[4], m1[4], m2t[4], m2[4];
#pragma unroll
        for (int i = 0; i < 2 * KP; ++i)
            aq[i] = reads[i] = writes[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m1t[i] = m1[i] = m2t[i] = m2[i] = v4f{0.f, 0.f, 0.f, 0.f};
        float by_beta[2][8] = {}, dot = 0.f;
        block_sync();  // the last head's operands have been read
        if (wave == 0)
            delta_gates(lds.gates, p.g, p.beta, token * p.Hv + hv, p.Hv, n);
        block_sync();
        for (int col = 0; col < p.Dv; col += kGradCols) {
            if (wave < 2) {  // U of 16 columns, as in the walk
                const int dv = col + 16 * wave + l;
                const bool live = dv < p.Dv;
                Parts<kParts> Sp[KP];
#pragma unroll
                for (int s = 0; s < KP; ++s) {
                    float w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int f = 32 * s + 8 * quarter + e;
                        w[e] = S[(int64_t)(f < p.Dk ? f : 0) * p.Dv + (live ? dv : 0)];
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[e] = live && 32 * s + 8 * quarter + e < p.Dk ? w[e] : 0.f;
                    Sp[s] = split8<kParts>(w);
                }
                float R[2][8];
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        v4f ks = {0.f, 0.f, 0.f, 0.f};
                        const int row = 32 * s + tile_row(h, l);
#pragma unroll
                        for (int f = 0; f < KP; ++f)
                            ks = mm<kParts>(row_operand<T>(k + (row < n ? row : 0) * p.k_stride, 32 * f + 8 * quarter,
                                                           row < n ? p.Dk : 0), Sp[f], ks);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int t = 32 * s + 8 * quarter + 4 * h + r;
                            const float x = delta_load<T>(v + (t < n ? t : n - 1) * p.v_stride + (live ? dv : 0));
                            const float read = (live && t < n ? x : 0.f) - lds.gates.since[t] * ks[r];
                            const float by = gr[(int64_t)t * p.Dv + (live ? dv : 0)];
                            R[s][4 * h + r] = lds.gates.beta[t] * read;
                            by_beta[s][4 * h + r] += live ? read * by : 0.f;
                        }
                    }
                const float *tri = p.tri + at * kDeltaFragFloats + 8 * lane;
                auto frag = [&](int f) {
                    return split_tiles<kParts>(*(const v4f *)(tri + 512 * f), *(const v4f *)(tri + 512 * f + 4));
                };
                const Parts<kParts> R0 = split8<kParts>(R[0]);
                v4f U[4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    U[h] = mm<kParts>(frag(frag_of(0, h, 0)), R0, v4f{0.f, 0.f, 0.f, 0.f});
                const Parts<kParts> U0 = split_tiles<kParts>(U[0], U[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const v4f c = mm<kParts>(frag(frag_of(1, h, 0)), U0, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        R[1][4 * h + r] -= c[r];
                }
                const Parts<kParts> R1 = split8<kParts>(R[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    U[2 + h] = mm<kParts>(frag(frag_of(1, h, 1)), R1, v4f{0.f, 0.f, 0.f, 0.f});
                const Parts<kParts> up[2] = {U0, split_tiles<kParts>(U[2], U[3])};
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < kParts; ++i)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            lds.a.u[(i * 64 + 32 * s + 8 * quarter + e) * kGradStride + 16 * wave + l] =
                                (uint16_t)(up[s].p[i][e >> 1] >> (16 * (e & 1)));
            } else {
                const int thread = thread_id() - 128, cols = p.Dv - col;
                grad_stage<kF32, kParts>(gr + col, p.Dv, 64, 64, cols, lds.a.r, thread, 128);
                grad_stage<T, IN>(go + col, o_stride, 64, n, cols, lds.a.o, thread, 128);
                grad_stage<kF32, kParts>(S + col, p.Dv, 32 * KP, p.Dk, cols, lds.a.s, thread, 128);
                grad_stage<kF32, kParts>(gs + col, p.Dv, 32 * KP, p.Dk, cols, lds.a.gs, thread, 128);
            }
            block_sync();
            const Parts<IN> oo = grad_operand<IN>(lds.a.o, 64, own);
            const Parts<kParts> ro = grad_operand<kParts>(lds.a.r, 64, own), uo = grad_operand<kParts>(lds.a.u, 64, own);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 32 * (i >> 1) + tile_row(i & 1, l);
                if ((i >> 1) <= (wave >> 1)) {  // rows j up to the own token i
                    const Parts<kParts> u = grad_operand<kParts>(lds.a.u, 64, row);
                    m1t[i] = mm<kParts>(u, oo, m1t[i]);
                    m2t[i] = mm<kParts>(u, ro, m2t[i]);
                }
                if ((i >> 1) >= (wave >> 1)) {  // rows i from the own token j on
                    m1[i] = mm<kParts>(grad_operand<IN>(lds.a.o, 64, row), uo, m1[i]);
                    m2[i] = mm<kParts>(grad_operand<kParts>(lds.a.r, 64, row), uo, m2[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2 * KP; ++i) {
                const int row = 32 * (i >> 1) + tile_row(i & 1, l);
                const Parts<kParts> s = grad_operand<kParts>(lds.a.s, 32 * KP, row);
                aq[i] = mm<kParts>(s, oo, aq[i]);
                reads[i] = mm<kParts>(s, ro, reads[i]);
                writes[i] = mm<kParts>(grad_operand<kParts>(lds.a.gs, 32 * KP, row), uo, writes[i]);
            }
            block_sync();
        }
        // <S, dS'>
        for (int i = thread_id(); i < p.Dk * p.Dv; i += 256)
            dot = __builtin_fmaf(S[i], gs[i], dot);
        dot = wave_sum(dot);
        if (lane == 0)
            lds.dots[wave] = dot;
        if (wave < 2)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float sum = row16_sum(by_beta[s][e]);
                    if (l == 0)
                        lds.beta[wave][32 * s + 8 * quarter + e] = sum;
                }
        delta_stage<T, KP, false, true>(k, p.k_stride, p.Dk, n, nullptr, lds.b.kt);
        delta_stage<T, KP, false, true>(q, p.q_stride, p.Dk, n, nullptr, lds.b.qt);
        block_sync();
        const DeltaGates &gates = lds.gates;
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
        const bool valid = own < n;
#pragma unroll
        for (int s = 0; s < KP; ++s) {
            float w[8];
            const int f = 32 * s + 8 * quarter;
            unpack8<T>(load8<T>(k + (valid ? own * p.k_stride : 0) + (p.Dk > f ? f : 0), valid ? p.Dk - f : 0), w);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                held = __builtin_fmaf(w[e], writes[2 * s + (e >> 2)][e & 3], held);
        }
        held = wave_sum(held);
        Parts<IN> ko[KP];
#pragma unroll
        for (int s = 0; s < KP; ++s)
            ko[s] = row_operand<T>(k + (valid ? own * p.k_stride : 0), 32 * s + 8 * quarter, valid ? p.Dk : 0);
        float by_own = 0.f;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (s <= (wave >> 1)) {  // token rows j at or before the own token i
                float d[8], e[8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v4f kk = {0.f, 0.f, 0.f, 0.f};
                    const int row = 32 * s + tile_row(h, l);
#pragma unroll
                    for (int f = 0; f < KP; ++f)
                        kk = mm<kParts>(row_operand<T>(k + (row < n ? row : 0) * p.k_stride, 32 * f + 8 * quarter,
                                                       row < n ? p.Dk : 0), ko[f], kk);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = 32 * s + 8 * quarter + 4 * h + r;
                        const float decay = j <= own ? delta_exp(sum_own - gates.sum[j]) : 0.f;
                        const float x = j < own ? -m2t[2 * s + h][r] * decay : 0.f;
                        d[4 * h + r] = j <= own ? p.scale * decay * m1t[2 * s + h][r] : 0.f;
                        e[4 * h + r] = beta * x;
                        by_own = __builtin_fmaf(x, kk[r], by_own);
                    }
                }
                const Parts<kParts> dp = split8<kParts>(d), ep = split8<kParts>(e);
#pragma unroll
                for (int i = 0; i < 2 * KP; ++i) {
                    const auto a = lds_operand(lds.b.kt + (32 * (i >> 1) + tile_row(i & 1, l)) * TS + 32 * s + 8 * quarter);
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
                        const int i = 32 * s + 8 * quarter + 4 * h + r;
                        const float decay = i >= own ? delta_exp(gates.sum[i] - sum_own) : 0.f;
                        d[4 * h + r] = i >= own ? p.scale * decay * m1[2 * s + h][r] : 0.f;
                        e[4 * h + r] = i > own ? -gates.beta[i] * decay * m2[2 * s + h][r] : 0.f;
                    }
                const Parts<kParts> dp = split8<kParts>(d), ep = split8<kParts>(e);
#pragma unroll
                for (int i = 0; i < 2 * KP; ++i) {
                    const int row = (32 * (i >> 1) + tile_row(i & 1, l)) * TS + 32 * s + 8 * quarter;
                    writes[i] = mm<kParts>(lds_operand(lds.b.qt + row), dp, writes[i]);
                    writes[i] = mm<kParts>(lds_operand(lds.b.kt + row), ep, writes[i]);
                }
            }
        }
        // q . dq + k . (reads - writes), and the sums over the value heads
#pragma unroll
        for (int s = 0; s < KP; ++s) {
            float x[8], y[8];
            const int f = 32 * s + 8 * quarter;
            unpack8<T>(load8<T>(q + (valid ? own * p.q_stride : 0) + (p.Dk > f ? f : 0), valid ? p.Dk - f : 0), x);
            unpack8<T>(load8<T>(k + (valid ? own * p.k_stride : 0) + (p.Dk > f ? f : 0), valid ? p.Dk - f : 0), y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = 2 * s + (e >> 2), r = e & 3;
                dots = __builtin_fmaf(x[e], aq[i][r], dots);
                dots = __builtin_fmaf(y[e], reads[i][r] - writes[i][r], dots);
                tq[i][r] += aq[i][r];
                tk[i][r] += reads[i][r] + writes[i][r];
            }
        }
        dots = quarter_sum(dots);
        by_own = quarter_sum(by_own);
        if (quarter == 0) {
            lds.sums[own] = dots;
            lds.beta[0][own] += lds.beta[1][own] + by_own;
        }
        block_sync();
        if (lane == 0)  // the dots of the state's gradient are read below; each wave adds its tokens' share
            lds.dots[wave] = gates.whole * lds.dots[wave] + held;
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
    if (own < rows)
#pragma unroll
        for (int s = 0; s < KP; ++s) {
            const int f = 32 * s + 8 * quarter;
            const float x[8] = {tq[2 * s][0], tq[2 * s][1], tq[2 * s][2], tq[2 * s][3],
                                tq[2 * s + 1][0], tq[2 * s + 1][1], tq[2 * s + 1][2], tq[2 * s + 1][3]};
            const float y[8] = {tk[2 * s][0], tk[2 * s][1], tk[2 * s][2], tk[2 * s][3],
                                tk[2 * s + 1][0], tk[2 * s + 1][1], tk[2 * s + 1][2], tk[2 * s + 1][3]};
            if (f < p.Dk) {
                store8<T>(gq + f, p.Dk - f, x);
                store8<T>(gk + f, p.Dk - f, y);
            }
        }
}

// out = from, or zeros.
SSD_KERNEL(256) void delta_copy_kernel(const float *from, float *out, int64_t n)
{
    for (int64_t i = block_id() * 256 + thread_id(); i < n; i += grid_blocks() * 256)
        out[i] = from ? from[i] : 0.f;
}

}  // namespace ssd
