// ssd_quant_kernels.h -- e4m3 quantisation with a scale per block of 128 values.
// For a block of values v: scale = max(max |v| / 448, 2^-126), q = e4m3(v / scale).
// Three forms of block: 1 x 128 along a row, 1 x 128 along a column (the matrix turned, for
// a product that sums over its rows) and 128 x 128 (weights), this one plain or turned.
// All are bound by memory: each value is read once (2 or 4 bytes) and written once (1 byte).
// Measured (a copy runs at 5160 GB/s): 65536 x 1024 bfloat16 along the rows 35 us (5.7 TB/s), turned
// 43 us (4.7 TB/s); 5136 x 1024 float32 in 128 x 128 blocks, turned, 5.2 us (5.1 TB/s).
#pragma once

#include <ssd_elem.h>

namespace ssd {

struct QuantParams {
    const void *x;
    uint8_t *q;
    float *scale;
    int64_t rows, cols, x_stride, q_stride;
};

// 1 x 128 blocks along the rows. 16 lanes hold a block; a workgroup's 256 threads hold
// kQuantUnroll x 16 neighbouring blocks of the row-major (row, block) order. Four in flight per
// thread: 65536 x 1024 bfloat16 35 us, with one 41, with eight 38 (float32: 65, 60, 67).
constexpr int kQuantUnroll = 4;

template <int T>
SSD_KERNEL(256) void quantise_rows_kernel(QuantParams p)
{
    const int64_t kb = (p.cols + 127) >> 7;
    const int64_t blocks = p.rows * kb;
    const int lane16 = thread_id() & 15;
    const int64_t first = block_id() * (16 * kQuantUnroll) + (thread_id() >> 4);
    Raw8<T> raw[kQuantUnroll];
    int64_t row[kQuantUnroll], col[kQuantUnroll];
    int n[kQuantUnroll];
#pragma unroll
    for (int k = 0; k < kQuantUnroll; ++k) {
        const int64_t b = first + 16 * k;
        const int64_t bb = b < blocks ? b : blocks - 1;
        row[k] = (uint64_t)bb >> 32 ? bb / kb : (int64_t)((uint32_t)bb / (uint32_t)kb);
        col[k] = (bb - row[k] * kb) * 128 + 8 * lane16;
        const int64_t left = p.cols - col[k];
        n[k] = b < blocks ? (int)(left < 8 ? left : 8) : 0;
        raw[k] = load8<T>((const char *)p.x +
                              (row[k] * p.x_stride + (n[k] > 0 ? col[k] : 0)) * ElemSize<T>::value,
                          n[k]);
    }
#pragma unroll
    for (int k = 0; k < kQuantUnroll; ++k) {
        float v[8];
        unpack8<T>(raw[k], v);
        const float scale = e4m3_scale(row16_max(amax8(v)));
        if (n[k] > 0) {
            store_e4m3(p.q + row[k] * p.q_stride + col[k], n[k], e4m3_pack8(v, scale, 1.f / scale));
            if (lane16 == 0)
                p.scale[(col[k] >> 7) * p.rows + row[k]] = scale;
        }
    }
}

// One 128 x 128 tile of x (rows r0.., columns c0..) per workgroup. Thread (rg, cg) =
// (tid / 16, tid % 16) holds rows 8 rg .. +7 of columns 8 cg .. +7, so a load covers 128
// columns of a row with 16 lanes, and eight rows of one column are eight bytes.
//   WHOLE: one scale for the tile, else one per column (the maximum over the 16 rg).
//   TURN: q is (cols, rows). The bytes cross shared memory: column 8 cg + e's 128 bytes lie at
//   row 16 e + cg of 136 bytes, which spreads a wave's eight-byte writes over the banks, and
//   leave as eight 16-byte pieces of a row of q.
constexpr int kTileLd = 136;

template <int T, bool WHOLE, bool TURN>
SSD_KERNEL(256) void quantise_tile_kernel(QuantParams p)
{
    SSD_LDS uint8_t tile[TURN ? 128 * kTileLd : 16];
    SSD_LDS uint32_t top[16 * 128];
    const int tid = thread_id();
    const int cg = tid & 15, rg = tid >> 4;
    const int64_t ctiles = (p.cols + 127) >> 7, rtiles = (p.rows + 127) >> 7;
    const int64_t rt = block_id() / ctiles, ct = block_id() % ctiles;
    const int64_t r0 = rt * 128 + 8 * rg, c0 = ct * 128 + 8 * cg;
    const int nc = (int)(p.cols - c0 < 8 ? p.cols - c0 : 8);
    const int nr = (int)(p.rows - r0 < 8 ? p.rows - r0 : 8);
    Raw8<T> raw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const bool in = j < nr && nc > 0;
        raw[j] = load8<T>((const char *)p.x +
                              (in ? (r0 + j) * p.x_stride + c0 : 0) * ElemSize<T>::value,
                          in ? nc : 0);
    }
    float v[8][8];
    uint32_t m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        m[e] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        unpack8<T>(raw[j], v[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            m[e] = max_u(m[e], f2u(v[j][e]) & 0x7fffffffu);
    }
    float by[8], inv[8];      // the scales and their reciprocals
    if (WHOLE) {
        uint32_t t = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            t = max_u(t, m[e]);
        top[tid] = row16_max(t);
        block_sync();
        t = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            t = max_u(t, top[16 * i]);
        const float scale = e4m3_scale(t);
        if (tid == 0)
            p.scale[TURN ? ct * rtiles + rt : rt * ctiles + ct] = scale;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            by[e] = scale;
            inv[e] = 1.f / scale;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top[rg * 128 + 16 * e + cg] = m[e];
        block_sync();
        if (tid < 128) {  // column 8 (tid % 16) + tid / 16
            uint32_t t = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                t = max_u(t, top[i * 128 + tid]);
            top[tid] = t;  // only this thread has read row 0's entry
        }
        block_sync();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float scale = e4m3_scale(top[16 * e + cg]);
            if (rg == 0 && e < nc)
                p.scale[rt * p.cols + c0 + e] = scale;
            by[e] = scale;
            inv[e] = 1.f / scale;
        }
    }
    if (!TURN) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < nr && nc > 0)
                store_e4m3(p.q + (r0 + j) * p.q_stride + c0, nc, e4m3_pack8(v[j], by[0], inv[0]));
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float col[8] = {v[0][e], v[1][e], v[2][e], v[3][e], v[4][e], v[5][e], v[6][e], v[7][e]};
        *(v2u *)&tile[(16 * e + cg) * kTileLd + 8 * rg] = e4m3_pack8(col, by[e], inv[e]);
    }
    block_sync();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = (tid >> 3) + 32 * k, piece = tid & 7;
        const int64_t out_row = ct * 128 + c, out_col = rt * 128 + 16 * piece;
        if (out_row >= p.cols || out_col >= p.rows)
            continue;
        const uint8_t *src = &tile[(16 * (c & 7) + (c >> 3)) * kTileLd + 16 * piece];
        const v2u lo = *(const v2u *)src, hi = *(const v2u *)(src + 8);
        uint8_t *dst = p.q + out_row * p.q_stride + out_col;
        if (out_col + 16 <= p.rows) {
            const v4u w = {lo[0], lo[1], hi[0], hi[1]};
            __builtin_memcpy(dst, &w, 16);
        } else {
            const int left = (int)(p.rows - out_col);
            store_e4m3(dst, left, lo);
            if (left > 8)
                store_e4m3(dst + 8, left - 8, hi);
        }
    }
}

}  // namespace ssd
