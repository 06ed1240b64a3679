// ssd_split.h -- float32 products on the bfloat16 matrix unit. A float32 value is the sum of three
// bfloat16 parts (8 + 8 + 8 bits of its 24), so a product of two is the sum of the parts' products,
// each exact in float32; those below 2^-24 of it are left out. A value that is a bfloat16
// already is one part. The bfloat16 MFMA does 16 times the float32 MFMA's products a cycle, so that
// six of them per product still leave 2.7 times its rate.
//
// An infinity has no parts (what is left of it is a NaN), nor has a value above 3.39e38, which
// rounds to one: such operands give NaN.
//
// Every operand is laid out in the same way. An index is cut into spans of 32; a lane of quarter
// q = lane / 16 holds the eight neighbours 8 q .. 8 q + 7 of a span as the product's summed index
// ("k"), and the two result tiles h = 0, 1 of a span hold in their row m the index
// 8 (m / 4) + 4 h + m % 4, so that component r of a lane is 8 q + 4 h + r: the two tiles of a result
// are the lane's eight neighbours again, and feed the next product as they are.
#pragma once

#include <ssd_elem.h>

namespace ssd {

// Eight values of a lane in N parts.
template <int N>
struct Parts {
    v4u p[N];
};

// The parts of eight values, the largest first.
template <int N>
SSD_DEVICE Parts<N> split8(const float (&v)[8])
{
    Parts<N> r;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float a = v[e], b = v[e + 1];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t u = cvt_pk_bf16(a, b);
            r.p[i][e >> 1] = u;
            if (i + 1 < N) {
                a -= u2f(u << 16);
                b -= u2f(u & 0xffff0000u);
            }
        }
    }
    return r;
}
template <int N>
SSD_DEVICE Parts<N> split_tiles(v4f lo, v4f hi)
{
    const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return split8<N>(v);
}

// c += a b over a span of 32, to P parts' precision, the smallest products first.
template <int P, int NA, int NB>
SSD_DEVICE v4f mm(const Parts<NA> &a, const Parts<NB> &b, v4f c)
{
#pragma unroll
    for (int s = P - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
                c = mfma_bf16_16x16x32(a.p[i], b.p[s - i < 0 || s - i >= NB ? 0 : s - i], c);
    return c;
}

// The index that row m of tile h of a span has in it.
SSD_DEVICE int tile_row(int h, int m) { return 8 * (m >> 2) + 4 * h + (m & 3); }

}  // namespace ssd
