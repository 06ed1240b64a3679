// ssd_fp8_kernels.h -- the product of two e4m3 matrices with a float32 scale per block of
// 128 values:
//     out[m, n] = sum over kb of sa[kb, m] sb[., .] * sum over k in block kb of a[m, k] b[n, k]
// sb is one value per 128 x 128 block of b (weights) or one per row of b and block (both
// operands activations or gradients).
//
// The inner sum of 128 products is exactly one 16x16x128 e4m3 MFMA, started from zero; its
// four results per lane are then multiplied by the two scales and added to the float32
// sums. That is four vector FMAs per MFMA (16 of its 32 cycles), which run beside the next
// MFMAs: a loop of MFMAs alone ran at 4.4e15 flop/s, with four FMAs each 3 % slower, with six 24 %.
// b's rows are the MFMA's rows and a's rows its columns, so that a lane holds one m:
// its a-scale is one register per 16 rows of a, and b's block scale is the wave's.
//
// Precision. The e4m3 MFMA holds its inner sums to 2^-13 of the largest of each eight products,
// measured 1.3e-5 of a result (rms, normally distributed operands): a 130th of what the
// rounding to bfloat16 makes, so bfloat16 results are formed that way. It is 50 times
// what float32 sums make, so float32 results (weight gradients, for the most part) are formed from the
// same values widened to bfloat16, which is exact, by the 16x16x32 bfloat16 MFMA, which adds in
// float32, at half the rate (measured 4.4e15 against 2.2e15 flop/s).
#pragma once

#include <ssd_elem.h>

namespace ssd {

struct Fp8Params {
    const uint8_t *a, *b;
    const float *sa;          // (KB, M)
    const float *sb;          // (ceil(N / 128), KB), or (KB, N)
    void *out;
    float *part;              // (splits, M, N) when the sum over k is split
    int64_t a_stride, b_stride, out_stride;
    int M, N, K;
    int tiles_m, tiles_n, splits, split_blocks;  // split_blocks: k blocks per split
};

// Bytes k .. k + 15 of a row, zeros from K on.
SSD_DEVICE v4u fp8_chunk(const uint8_t *row, int k, int K)
{
    v4u r = {0u, 0u, 0u, 0u};
    if (k + 16 <= K) {
        __builtin_memcpy(&r, row + k, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (k + e < K)
                r[e >> 2] |= (uint32_t)row[k + e] << (8 * (e & 3));
    }
    return r;
}

// The outputs n .. n + 7 of one row, rounded to OUT.
template <int OUT>
SSD_DEVICE void fp8_store(void *out, int64_t at, int n, int N, const float (&v)[8])
{
    if (n < N)
        store8<OUT>((char *)out + (at + n) * ElemSize<OUT>::value, N - n, v);
}

// One operand's 32 values of a lane, as its MFMA takes them.
template <bool WIDE>
struct Fp8Operand {
    v4u w[WIDE ? 4 : 2];
};
template <bool WIDE>
SSD_DEVICE Fp8Operand<WIDE> fp8_operand(v4u lo, v4u hi)
{
    Fp8Operand<WIDE> r;
    if (WIDE) {
        r.w[0] = e4m3_to_bf16(lo[0], lo[1]);
        r.w[1] = e4m3_to_bf16(lo[2], lo[3]);
        r.w[WIDE ? 2 : 0] = e4m3_to_bf16(hi[0], hi[1]);
        r.w[WIDE ? 3 : 0] = e4m3_to_bf16(hi[2], hi[3]);
    } else {
        r.w[0] = lo;
        r.w[1] = hi;
    }
    return r;
}
template <bool WIDE>
SSD_DEVICE v4f fp8_block(const Fp8Operand<WIDE> &a, const Fp8Operand<WIDE> &b)
{
    v4f d = {0.f, 0.f, 0.f, 0.f};
    if (WIDE) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            d = mfma_bf16_16x16x32(a.w[WIDE ? t : 0], b.w[WIDE ? t : 0], d);
        return d;
    }
    const v8i x = {(int)a.w[0][0], (int)a.w[0][1], (int)a.w[0][2], (int)a.w[0][3],
                   (int)a.w[1][0], (int)a.w[1][1], (int)a.w[1][2], (int)a.w[1][3]};
    const v8i y = {(int)b.w[0][0], (int)b.w[0][1], (int)b.w[0][2], (int)b.w[0][3],
                   (int)b.w[1][0], (int)b.w[1][1], (int)b.w[1][2], (int)b.w[1][3]};
    return mfma_e4m3_16x16x128(x, y, d);
}

// Two at a time, their steps in turn.
template <bool WIDE>
SSD_DEVICE void fp8_blocks(const Fp8Operand<WIDE> &a0, const Fp8Operand<WIDE> &a1,
                           const Fp8Operand<WIDE> &b, v4f &d0, v4f &d1)
{
    if (!WIDE) {
        d0 = fp8_block<WIDE>(a0, b);
        d1 = fp8_block<WIDE>(a1, b);
        return;
    }
    d0 = d1 = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        d0 = mfma_bf16_16x16x32(a0.w[WIDE ? t : 0], b.w[WIDE ? t : 0], d0);
        d1 = mfma_bf16_16x16x32(a1.w[WIDE ? t : 0], b.w[WIDE ? t : 0], d1);
    }
}

// The rows of an operand that do not start on 16 bytes, laid out anew so that they do, with zeros
// up to the next multiple of 16: what the large form reads. One 16-byte piece per thread.
SSD_KERNEL(256) void fp8_pack_kernel(const uint8_t *x, int64_t stride, int64_t rows, int K, uint8_t *out)
{
    const int pieces = (K + 15) >> 4;
    const int64_t n = rows * pieces, step = grid_blocks() * 256;
    for (int64_t e = block_id() * 256 + thread_id(); e < n; e += step) {
        const int64_t r = e / pieces;
        const int k = (int)(e - r * pieces) * 16;
        *(v4u *)(out + (r * pieces) * 16 + k) = fp8_chunk(x + r * stride, k, K);
    }
}

// The large form: a workgroup of 8 waves, 4 along b's rows and 2 along a's, each 64 rows of b by
// 16 MB rows of a: 256 x 32 MB results. The next block's rows go straight into the other of two
// stages of shared memory, in five parts between the MFMAs, so that a compute unit holds one
// workgroup and two waves per SIMD. A wave reads 24 16-byte pieces per 32 MFMAs (MB = 8; 8 of b, 16 of a),
// three quarters of the shared memory's rate, without bank conflicts.
//
// Measured: 8192 x 8192 x 8192 to bfloat16 475 us (2310 Tflop/s at 1.9 GHz, the MFMAs busy 53 % of the
// time), to float32 1020 us (1080); 65536 x 5136 x 1024 410 to 450 us (1690 to 1530), of
// which 100 are the stores of 673 MB: 8 blocks of k to a tile leave nothing for them to run beside.
// Tried and slower: b's rows straight from memory into registers (470 -> 552), loads two blocks
// ahead with two barriers a block (476 -> 496), two workgroups of one stage per compute unit
// (449 -> 482), 32 x 32 x 16 MFMAs for float32 (735 -> 782). Within 2 % either way: workgroups that go
// from tile to tile and load the next while they store (445 -> 440, small products 2 % slower),
// their starts spread over a tile's time, stores of whole 128-byte lines, one barrier in the
// middle of a block (float32 716 -> 697, bfloat16 445 -> 453).
constexpr int kBigN = 256;
constexpr uint32_t kBigOut = 0xfffffff0u;         // a byte offset past every buffer

// Where chunk c of staged row r lies in its row of eight: neighbouring lanes of a wave's read
// (rows r, r + 1, .. of a; rows 0-3, 8-11, 16-19, 24-27 of b) then meet different banks.
SSD_DEVICE int big_key_a(int r) { return r & 7; }
SSD_DEVICE int big_key_b(int r) { return (r & 3) | (r >> 1 & 4); }

// Which tile a workgroup takes. Workgroup i runs on XCD i % 8, each with an L2 of its own, so
// each XCD gets a contiguous part of an order in which four row tiles of a go over all
// column tiles: the 32 workgroups that it runs at a time share 4 tiles of a and 8 of b.
SSD_DEVICE void fp8_place(const Fp8Params &p, int64_t id, int &tm, int &tn)
{
    const int64_t all = (int64_t)p.tiles_m * p.tiles_n;
    const int64_t each = all >> 3, more = all & 7, x = id & 7;
    const int64_t at = x * each + (x < more ? x : more) + (id >> 3);
    const int64_t group = at / (4 * p.tiles_n);
    const int rest = (int)(at - group * (4 * p.tiles_n));
    const int in = p.tiles_m - 4 * group < 4 ? (int)(p.tiles_m - 4 * group) : 4;
    tn = rest / in;
    tm = (int)(4 * group) + rest - tn * in;
}

template <int MB, bool BROW, int OUT>
SSD_KERNEL_WAVES(512, 2) void fp8_matmul_big_kernel(Fp8Params p)
{
    constexpr bool WIDE = OUT == kF32;
    constexpr int NB = 4, TM = 32 * MB, STAGE = (kBigN + TM) * 128;
    static_assert(MB % 2 == 0 && MB <= 8, "whole loads of 64 rows, and at most 256 of them");
    // Two stages, each an array of its own: the compiler then knows that reading one need not wait
    // for the loads into the other. Scales: a's, then b's (BROW).
    SSD_LDS uint8_t tile0[STAGE];
    SSD_LDS uint8_t tile1[STAGE];
    SSD_LDS float scales0[512];
    SSD_LDS float scales1[512];
    const int tid = thread_id();
    const int lane = tid & 63, wave = wave_id();
    const int wn = wave & 3, wm = wave >> 2;
    const int i16 = lane & 15, q = lane >> 4;
    const int KB = (p.K + 127) >> 7;
    const int64_t all = (int64_t)p.tiles_m * p.tiles_n;
    const int split = (int)(block_id() / all);
    int tm, tn;
    fp8_place(p, block_id() - split * all, tm, tn);
    const int n0 = tn * kBigN, m0 = tm * TM;
    const int kb0 = split * p.split_blocks;
    const int kb1 = kb0 + p.split_blocks < KB ? kb0 + p.split_blocks : KB;
    const int rows_n = p.N - n0 < kBigN ? p.N - n0 : kBigN;
    const int rows_m = p.M - m0 < TM ? p.M - m0 : TM;
    // Staging: this lane's place in the 8 rows that its wave loads at once (64 rows further on for
    // each of the four loads of an operand; the keys do not depend on which).
    const int r8 = lane >> 3, c8 = lane & 7;
    const int ka = 16 * (c8 ^ big_key_a(r8)), kb_ = 16 * (c8 ^ big_key_b(wave * 8 + r8));
    uint32_t off_a[TM / 64], off_b[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        off_b[r] = (uint32_t)(64 * r + wave * 8 + r8) * (uint32_t)p.b_stride + (uint32_t)kb_;
        if (r < TM / 64)
            off_a[r % (TM / 64)] = (uint32_t)(64 * r + wave * 8 + r8) * (uint32_t)p.a_stride + (uint32_t)ka;
    }
    const uint8_t *first_a = p.a + m0 * p.a_stride, *first_b = p.b + n0 * p.b_stride;
    const uint32_t end_a = (uint32_t)(rows_m - 1) * (uint32_t)p.a_stride + (uint32_t)p.K;
    const uint32_t end_b = (uint32_t)(rows_n - 1) * (uint32_t)p.b_stride + (uint32_t)p.K;
    // One of the five parts of a block's loads. No branches in here: past the last block (and for
    // scales that there are not) the buffers are empty.
    auto fetch = [&](int part, int kb, uint8_t *tile, float *scales) {
        const int k = kb * 128;
        const bool any = kb < kb1;
        if (part < 4) {
            // 16 bytes from K on lie past the buffer's end, as rows past the matrix's do: zeros
            async_load16(make_buf(first_b + k, any ? end_b - (uint32_t)k : 0u), k + kb_ < p.K ? off_b[part % 4] : kBigOut,
                         &tile[(64 * part + wave * 8) * 128]);
            if (part < TM / 64)
                async_load16(make_buf(first_a + k, any ? end_a - (uint32_t)k : 0u),
                             k + ka < p.K ? off_a[part % (TM / 64)] : kBigOut,
                             &tile[kBigN * 128 + (64 * part + wave * 8) * 128]);
        } else {
            const bool isa = wave < 4;
            const float *from = isa || !BROW ? p.sa + (int64_t)kb * p.M + m0 : p.sb + (int64_t)kb * p.N + n0;
            const int many = !any ? 0 : isa ? rows_m : BROW ? rows_n : 0;
            async_load4(make_buf(from, (uint32_t)many * 4u), (uint32_t)(tid & 255) * 4u, &scales[wave * 64]);
        }
    };
    // Operands: row 8 (i16 / 4) + i16 % 4 + 4 (j % 2) + 32 (j / 2) of b's 64, row 16 i + i16 of a's
    // 16 MB; the keys do not depend on i and j, so that these are constant distances. A lane's
    // results of blocks 2 g and 2 g + 1 are then the eight n from 32 g + 8 q on, one 16-byte
    // store of bfloat16, and four lanes' stores are 64 neighbouring bytes.
    const int rb = wn * 64 + 8 * (i16 >> 2) + (i16 & 3), ra = wm * 16 * MB + i16;
    const int b_lo = rb * 128 + 16 * (q ^ big_key_b(rb)), b_hi = rb * 128 + 16 * ((q + 4) ^ big_key_b(rb));
    const int a_lo = kBigN * 128 + ra * 128 + 16 * (q ^ big_key_a(ra));
    const int a_hi = kBigN * 128 + ra * 128 + 16 * ((q + 4) ^ big_key_a(ra));

    v4f acc[NB][MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i)
            acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};
    const int nw = n0 + wn * 64, mw = m0 + wm * 16 * MB;
    const int nb128 = (nw < p.N ? nw : p.N - 1) >> 7;
    auto step = [&](int kb, uint8_t *tile, float *scales, uint8_t *next_tile, float *next_scales) {
        async_wait<0>();
        bare_barrier();
        Fp8Operand<WIDE> bf[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j)
            bf[j] = fp8_operand<WIDE>(*(const v4u *)&tile[b_lo + 512 * (j & 1) + 4096 * (j >> 1)],
                                      *(const v4u *)&tile[b_hi + 512 * (j & 1) + 4096 * (j >> 1)]);
        v4f sb4[BROW ? NB : 1];
        float sb = 1.f;
        if (BROW) {
#pragma unroll
            for (int j = 0; j < NB; ++j)
                sb4[BROW ? j : 0] = *(const v4f *)&scales[256 + wn * 64 + 8 * q + 4 * (j & 1) + 32 * (j >> 1)];
        } else {
            sb = ld_uniform(p.sb, (int64_t)nb128 * KB + kb);
        }
        // Two MFMAs behind, results are scaled and added while the next two run; the next rows of a
        // are on their way from shared memory.
        v4f d[2][2];
        float sa = 0.f, sa_before = 0.f;
        v4u lo = *(const v4u *)&tile[a_lo], hi = *(const v4u *)&tile[a_hi];
        float sa_next = scales[ra];
        Fp8Operand<WIDE> af = fp8_operand<WIDE>(lo, hi);
#pragma unroll
        for (int u = 0; u <= 2 * MB; ++u) {
            const int i = u >> 1, j = 2 * (u & 1);
            sched_fence();
            if (u < 5)
                fetch(u, kb + 1, next_tile, next_scales);
            if (u < 2 * MB) {
                if (j == 0) {
                    af = fp8_operand<WIDE>(lo, hi);
                    sa_before = sa;
                    sa = sa_next * sb;
                    if (i + 1 < MB) {
                        sa_next = scales[ra + 16 * (i + 1)];
                        lo = *(const v4u *)&tile[a_lo + 2048 * (i + 1)];
                        hi = *(const v4u *)&tile[a_hi + 2048 * (i + 1)];
                    }
                } else {
                    sa_before = sa;
                }
                fp8_blocks<WIDE>(bf[j], bf[j + 1], af, d[u & 1][0], d[u & 1][1]);
            } else {
                sa_before = sa;
            }
            sched_fence();
            if (u > 0) {
                const int pi = (u - 1) >> 1, pj = 2 * ((u - 1) & 1);
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float f = BROW ? sa_before * sb4[BROW ? pj + g : 0][e] : sa_before;
                        acc[pj + g][pi][e] += d[(u - 1) & 1][g][e] * f;
                    }
            }
        }
    };
#pragma unroll
    for (int part = 0; part < 5; ++part)
        fetch(part, kb0, tile0, scales0);
    int kb = kb0;
    for (; kb + 1 < kb1; kb += 2) {
        step(kb, tile0, scales0, tile1, scales1);
        step(kb + 1, tile1, scales1, tile0, scales0);
    }
    if (kb < kb1)
        step(kb, tile0, scales0, tile1, scales1);
    async_wait<0>();  // the loads past the last block, before the shared memory is given back
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int m = mw + 16 * i + i16;
        if (m >= p.M)
            continue;
#pragma unroll
        for (int g = 0; g < NB / 2; ++g) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = acc[2 * g + (e >> 2)][i][e & 3];
            if (p.splits > 1)
                fp8_store<kF32>(p.part, ((int64_t)split * p.M + m) * p.N, nw + 32 * g + 8 * q, p.N, v);
            else
                fp8_store<OUT>(p.out, m * p.out_stride, nw + 32 * g + 8 * q, p.N, v);
        }
    }
}

// Few rows of a (16 MB at most): bound by reading b once, and below some 10 MB of it by the time that a
// launch and one trip to memory take. Measured: 8 x 5136 x 1024 4.0 us, 64 x 5136 x 1024 7.7.
// A wave takes 16 rows of b and every
// WK-th k block, straight from memory into the MFMA's registers (four lanes cover a row's 128
// bytes), AHEAD blocks in flight; the workgroup's WK waves add up through shared memory in
// wave order. a comes from the caches.
template <int MB, int WK, bool BROW, int OUT>
SSD_KERNEL(64 * WK) void fp8_matmul_few_kernel(Fp8Params p)
{
    constexpr bool WIDE = OUT == kF32;
    constexpr int AHEAD = MB == 1 ? (WK == 4 ? 4 : 3) : MB == 2 ? 2 : (WK == 4 ? 2 : 1);  // what the registers hold
    SSD_LDS float sums[WK - 1][MB * 4][64];
    const int lane = thread_id() & 63, wave = wave_id();
    const int i16 = lane & 15, q = lane >> 4;
    const int n0 = (int)block_id() * 16;
    const int full = p.K >> 7, KB = (p.K + 127) >> 7;
    const int brow = n0 + i16 < p.N ? n0 + i16 : p.N - 1;   // rows past the end repeat the last; not stored
    const uint8_t *b = p.b + (int64_t)brow * p.b_stride + 32 * q;
    const uint8_t *a[MB];
    int arow[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        arow[i] = 16 * i + i16 < p.M ? 16 * i + i16 : p.M - 1;
        a[i] = p.a + (int64_t)arow[i] * p.a_stride + 32 * q;
    }
    v4f acc[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
        acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
    struct Block {
        v4u b[2], a[MB][2];
        float sa[MB], sb[BROW ? 4 : 1];
    };
    auto scales = [&](Block &h, int kb) {
#pragma unroll
        for (int i = 0; i < MB; ++i)
            h.sa[i] = p.sa[(int64_t)kb * p.M + arow[i]];
        if (BROW) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = n0 + 4 * q + e;
                h.sb[BROW ? e : 0] = p.sb[(int64_t)kb * p.N + (n < p.N ? n : p.N - 1)];
            }
        } else {
            h.sb[0] = ld_uniform(p.sb, (int64_t)(n0 >> 7) * KB + kb);
        }
    };
    auto add = [&](const Block &h) {
        const Fp8Operand<WIDE> bf = fp8_operand<WIDE>(h.b[0], h.b[1]);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const v4f d = fp8_block<WIDE>(bf, fp8_operand<WIDE>(h.a[i][0], h.a[i][1]));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][e] += d[e] * (h.sa[i] * h.sb[BROW ? e : 0]);
        }
    };
    for (int first = wave; first < full; first += WK * AHEAD) {
        Block h[AHEAD];
#pragma unroll
        for (int g = 0; g < AHEAD; ++g) {
            const int kb = first + WK * g;
            if (kb >= full)
                break;
            __builtin_memcpy(h[g].b, b + kb * 128, 32);
#pragma unroll
            for (int i = 0; i < MB; ++i)
                __builtin_memcpy(h[g].a[i], a[i] + kb * 128, 32);
            scales(h[g], kb);
        }
#pragma unroll
        for (int g = 0; g < AHEAD; ++g) {
            if (first + WK * g >= full)
                break;
            add(h[g]);
        }
    }
    if (full < KB && full % WK == wave) {  // the block that K cuts
        Block h;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int k = full * 128 + 16 * t;
            h.b[t] = fp8_chunk(b, k, p.K - 32 * q);
#pragma unroll
            for (int i = 0; i < MB; ++i)
                h.a[i][t] = fp8_chunk(a[i], k, p.K - 32 * q);
        }
        scales(h, full);
        add(h);
    }
    if (wave > 0) {
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sums[wave - 1][4 * i + e][lane] = acc[i][e];
    }
    block_sync();
    if (wave > 0)
        return;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            for (int w = 0; w < WK - 1; ++w)
                acc[i][e] += sums[w][4 * i + e][lane];
    const int left = p.N - n0 - 4 * q;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int m = 16 * i + i16;
        if (m >= p.M || left <= 0)
            continue;
        char *out = (char *)p.out + (m * p.out_stride + n0 + 4 * q) * ElemSize<OUT>::value;
        const v2u u = {cvt_pk_bf16(acc[i][0], acc[i][1]), cvt_pk_bf16(acc[i][2], acc[i][3])};
        if (left >= 4) {
            if (OUT == kBF16)
                __builtin_memcpy(out, &u, 8);
            else
                __builtin_memcpy(out, &acc[i], 16);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < left) {
                    if (OUT == kBF16)
                        ((uint16_t *)out)[e] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
                    else
                        ((float *)out)[e] = acc[i][e];
                }
        }
    }
}

// out[m, n] = the sum of the splits' parts in their order, rounded to OUT.
template <int OUT>
SSD_KERNEL(256) void fp8_split_sum_kernel(Fp8Params p)
{
    const int64_t n = (int64_t)p.M * p.N;
    const int64_t step = grid_blocks() * 256;
    for (int64_t e = block_id() * 256 + thread_id(); e < n; e += step) {
        float acc = 0.f;
        for (int s = 0; s < p.splits; ++s)
            acc += p.part[s * n + e];
        const int64_t m = e / p.N, at = m * p.out_stride + (e - m * p.N);
        if (OUT == kBF16)
            ((uint16_t *)p.out)[at] = cvt_bf16(acc);
        else
            ((float *)p.out)[at] = acc;
    }
}

// out = 0: K = 0 has no terms.
template <int OUT>
SSD_KERNEL(256) void fp8_zero_kernel(Fp8Params p)
{
    const int64_t n = (int64_t)p.M * p.N;
    const int64_t step = grid_blocks() * 256;
    for (int64_t e = block_id() * 256 + thread_id(); e < n; e += step) {
        const int64_t m = e / p.N, at = m * p.out_stride + (e - m * p.N);
        if (OUT == kBF16)
            ((uint16_t *)p.out)[at] = 0;
        else
            ((float *)p.out)[at] = 0.f;
    }
}

}  // namespace ssd
