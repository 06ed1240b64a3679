// ssd_ops_api.hip -- C ABI of the operators around the scan (declared in include/ssd.h): the
// gated recurrence, the RMS norm, 8-bit quantisation and products. Argument checks, work planning and
// kernel launches on the caller's stream; nothing is allocated.
#include "ssd.h"

#include <ssd_fp8_kernels.h>
#include <ssd_gated_kernels.h>
#include <ssd_norm_kernels.h>
#include <ssd_quant_kernels.h>
#include <ssd_host.h>

namespace {

using ssd::align256;
using ssd::aligned;
using ssd::dtype_ok;
using ssd::elem_size;
using ssd::grid_1d;
using ssd::grid_ok;
using ssd::kMaxElems;
using ssd::launch_status;
using ssd::overlap_bytes;
using ssd::span;

// ------------------------------------------------------------------ RMS norm

int check_norm(int dtype, int64_t rows, int64_t F)
{
    if (!dtype_ok(dtype) || rows < 0 || F < 1)
        return SSD_ERR_SHAPE;
    if (F > ssd::kNormMaxF || rows > (1LL << 31) - 1)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Workgroups that the norm kernels are launched with: they walk over the rows, so about as
// many as the GPU holds at once (256 compute units, several each).
int64_t norm_groups(int64_t rows, int rows_per_group, int64_t most)
{
    const int64_t need = (rows + rows_per_group - 1) / rows_per_group;
    return need < most ? need : most;
}
constexpr int64_t kNormGroups = 2048;

// Lanes per row, both norms: as few as hold it in the registers of 8 or 16 values each. Measured in us:
// 65536 x 64 with 16 lanes 8.6, with a wave 25; 32768 x 512 with a wave 19.9 (gradients 27), with four
// 34.8 (37); 32768 x 1024 with a wave 40.4 (54.6), with four 43.8 (51.5); 6553 x 5120, gradients: 53 with 8 waves, 113 with four.
template <int T, int LANES, int STEPS>
int launch_norm_as(const ssd::NormParams &p, hipStream_t s)
{
    using Shape = ssd::NormShape<LANES>;
    const int64_t groups = norm_groups(p.rows, Shape::rows, kNormGroups);
    hipLaunchKernelGGL((ssd::rms_norm_kernel<T, LANES, STEPS>), dim3((unsigned)groups),
                       dim3(Shape::threads), 0, s, p);
    return launch_status();
}

template <int T>
int launch_norm(const ssd::NormParams &p, hipStream_t s)
{
    if (p.F <= 128)
        return launch_norm_as<T, 16, 1>(p, s);
    if (p.F <= 512)
        return launch_norm_as<T, 64, 1>(p, s);
    if (p.F <= 1024)
        return launch_norm_as<T, 64, 2>(p, s);
    if (p.F <= 2048)
        return launch_norm_as<T, 256, 1>(p, s);
    if (p.F <= 4096)
        return launch_norm_as<T, 256, 2>(p, s);
    if (p.F <= 8192)
        return launch_norm_as<T, 512, 2>(p, s);
    return launch_norm_as<T, 1024, 2>(p, s);
}

// Workgroups of the gradients' kernel: each leaves a row of shares of grad_weight.
int64_t norm_bwd_groups(int64_t rows, int64_t F)
{
    const int held = F <= 128 ? 16 : F <= 1024 ? 4 : 1;
    return norm_groups(rows, held, F <= 4096 ? 1024 : 512);
}

template <int T, int LANES, int STEPS>
int launch_norm_bwd_as(const ssd::NormBwdParams &p, int64_t groups, hipStream_t s)
{
    hipLaunchKernelGGL((ssd::rms_norm_bwd_kernel<T, LANES, STEPS>), dim3((unsigned)groups),
                       dim3(ssd::NormShape<LANES>::threads), 0, s, p);
    return launch_status();
}

template <int T>
int launch_norm_bwd(const ssd::NormBwdParams &p, int64_t groups, hipStream_t s)
{
    if (p.F <= 128)
        return launch_norm_bwd_as<T, 16, 1>(p, groups, s);
    if (p.F <= 512)
        return launch_norm_bwd_as<T, 64, 1>(p, groups, s);
    if (p.F <= 1024)
        return launch_norm_bwd_as<T, 64, 2>(p, groups, s);
    if (p.F <= 2048)
        return launch_norm_bwd_as<T, 256, 1>(p, groups, s);
    if (p.F <= 4096)
        return launch_norm_bwd_as<T, 256, 2>(p, groups, s);
    if (p.F <= 8192)
        return launch_norm_bwd_as<T, 512, 2>(p, groups, s);
    return launch_norm_bwd_as<T, 1024, 2>(p, groups, s);
}

// -------------------------------------------------------------- 8-bit values

template <int T>
int launch_quantise(const ssd::QuantParams &p, bool whole, bool turn, hipStream_t s)
{
    if (!whole && !turn) {
        const int64_t blocks = p.rows * ((p.cols + 127) / 128);
        const int64_t grid = (blocks + 16 * ssd::kQuantUnroll - 1) / (16 * ssd::kQuantUnroll);
        if (!grid_ok(grid, 256))
            return SSD_ERR_UNSUPPORTED;
        hipLaunchKernelGGL((ssd::quantise_rows_kernel<T>), dim3((unsigned)grid), dim3(256), 0, s, p);
        return launch_status();
    }
    const int64_t tiles = ((p.rows + 127) / 128) * ((p.cols + 127) / 128);
    if (!grid_ok(tiles, 256))
        return SSD_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)tiles), block(256);
    if (whole && turn)
        hipLaunchKernelGGL((ssd::quantise_tile_kernel<T, true, true>), grid, block, 0, s, p);
    else if (whole)
        hipLaunchKernelGGL((ssd::quantise_tile_kernel<T, true, false>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((ssd::quantise_tile_kernel<T, false, true>), grid, block, 0, s, p);
    return launch_status();
}

// Which kernel a product takes, and how the sum over k is split.
struct Fp8Plan {
    bool few;
    int mb;                   // 16 mb rows of a per wave
    int waves;                // few: waves of a workgroup
    int tiles_m, tiles_n, splits, split_blocks;
    size_t part_bytes;        // partial sums
    size_t a_bytes, b_bytes;  // operands laid out anew (rows that do not start on 16 bytes)
    size_t bytes() const { return part_bytes + a_bytes + b_bytes; }
};

int check_fp8(int64_t M, int64_t N, int64_t K, int64_t b_block_rows, int out_dtype)
{
    if (M < 0 || N < 1 || K < 0 || (b_block_rows != 1 && b_block_rows != 128) || !dtype_ok(out_dtype))
        return SSD_ERR_SHAPE;
    if (M > (1LL << 30) || N > (1LL << 30) || K > (1LL << 24) - 16)
        return SSD_ERR_UNSUPPORTED;
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);  // a plan's numbers stay in 32 bits
    return tiles > 1LL << 25 ? SSD_ERR_UNSUPPORTED : SSD_OK;
}

// Time of a product in us by the large form: every compute unit takes tiles * splits / 256 of
// them, each its k blocks (per_block us) and a start and end (per_tile us); the parts of a split
// sum are written and read once more.
double fp8_cost(int64_t M, int64_t N, int64_t tiles, int64_t kb, int splits, double per_block,
                double per_tile)
{
    const double rounds = (double)((tiles * splits + 255) / 256);
    const double parts = splits > 1 ? 4 + 8e-6 / 4.5 * splits * (double)M * (double)N : 0.;
    return rounds * (per_block * (double)((kb + splits - 1) / splits) + per_tile) + parts;
}

// `aligned_rows`: rows of both operands start on 16 bytes and K is a multiple of 16.
Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t K, int out_dtype, bool aligned_rows)
{
    Fp8Plan p{};
    const bool wide = out_dtype == SSD_F32;
    const int64_t kb = (K + 127) / 128;
    double best = -1.;
    for (int mb = 4; mb <= (wide ? 4 : 8); mb += 4) {
        const int64_t tm = (M + 32 * mb - 1) / (32 * mb), tn = (N + 255) / 256;
        // Measured for 256 x 256 tiles of bfloat16 results, and for 256 x 128 of float32 and of
        // bfloat16. What the choice gives, in us: 512 x 5136 x 1024 11.8 with the smaller tile, 17.0
        // with the larger; 16384 x 1024 x 1024 26.1 and 23.1. Splits: 1024 x 1024 x 16384 37 to
        // bfloat16 and 56 to float32, unsplit 109 and 226.
        const double per_block = mb == 8 || wide ? 1.85 : 1.1;
        for (int s = 1; s <= 32 && (s == 1 || s * 2 <= kb); ++s) {
            const double cost = fp8_cost(M, N, tm * tn, kb, s, per_block, mb == 8 ? 6. : 3.);
            if (best < 0. || cost < best) {
                best = cost;
                p.mb = mb;
                p.tiles_m = (int)tm;
                p.tiles_n = (int)tn;
                p.split_blocks = (int)((kb + s - 1) / s);
            }
        }
    }
    p.splits = kb > 0 ? (int)((kb + p.split_blocks - 1) / p.split_blocks) : 1;
    if (M <= 64) {
        // The form for few rows: a wave's time per k block grows with the rows of a it holds, and
        // 16 rows of b are a workgroup's. 8 x 5136 x 1024 3.9 us against the large form's 7.6, 64 x 5136 x
        // 1024 7.7 against 11.4; with N small and K long the large form's splits win (64 x 512 x
        // 16384: 38 against 18).
        const int mb = M <= 16 ? 1 : M <= 32 ? 2 : 4;
        const int64_t groups = (N + 15) / 16;
        // with fewer workgroups than fill the chip, more waves share a workgroup's sum
        const int waves = groups < 512 && kb > 8 ? (mb == 1 ? 16 : 8) : 4;
        const double few = 3 + (double)((groups + 511) / 512) * (double)((kb + waves - 1) / waves) *
                                   (mb == 1 ? 1.2 : mb == 2 ? 1.4 : 2.2);
        // The large form's model leaves out some 6 us (10 where it lays rows out anew first) of what it
        // takes at these sizes. Over 240 products (M 1 to 64, N 64 to 16384, K 512 to 16384, both results),
        // each measured in both forms, the choice is 2.1 % slower than the better one on average
        // (without the 6 and 10: 3.7 %), at worst 64 x 5136 x 16384 to float32, 75 against 30.
        if (few < best + (aligned_rows ? 6. : 10.)) {
            p.few = true;
            p.mb = mb;
            p.waves = waves;
            p.splits = 1;
            return p;
        }
    }
    p.part_bytes = p.splits > 1 ? align256((size_t)p.splits * M * N * 4) : 0;
    if (!aligned_rows) {
        p.a_bytes = align256((size_t)M * ((K + 15) / 16) * 16);
        p.b_bytes = align256((size_t)N * ((K + 15) / 16) * 16);
    }
    return p;
}

template <int MB, bool BROW, int OUT>
int launch_fp8_few(const ssd::Fp8Params &p, int waves, hipStream_t s)
{
    const unsigned groups = (unsigned)((p.N + 15) / 16);
    constexpr int MANY = MB == 1 ? 16 : 8;
    if (waves == MANY)
        hipLaunchKernelGGL((ssd::fp8_matmul_few_kernel<MB, MANY, BROW, OUT>), dim3(groups), dim3(64 * MANY), 0, s, p);
    else
        hipLaunchKernelGGL((ssd::fp8_matmul_few_kernel<MB, 4, BROW, OUT>), dim3(groups), dim3(256), 0, s, p);
    return launch_status();
}

int launch_pack(const uint8_t *x, int64_t stride, int64_t rows, int K, uint8_t *out, hipStream_t s)
{
    const int64_t n = rows * ((K + 15) / 16);
    const int64_t blocks = (n + 255) / 256 < 16384 ? (n + 255) / 256 : 16384;
    hipLaunchKernelGGL(ssd::fp8_pack_kernel, dim3((unsigned)blocks), dim3(256), 0, s, x, stride, rows, K, out);
    return launch_status();
}

template <bool BROW, int OUT>
int launch_fp8(ssd::Fp8Params p, const Fp8Plan &plan, bool aligned_rows, char *workspace, hipStream_t s)
{
    const int64_t n = (int64_t)p.M * p.N;
    const unsigned flat = (unsigned)((n + 255) / 256 < 8192 ? (n + 255) / 256 : 8192);
    if (p.K == 0) {
        hipLaunchKernelGGL((ssd::fp8_zero_kernel<OUT>), dim3(flat), dim3(256), 0, s, p);
        return launch_status();
    }
    if (plan.few)
        return plan.mb == 1   ? launch_fp8_few<1, BROW, OUT>(p, plan.waves, s)
               : plan.mb == 2 ? launch_fp8_few<2, BROW, OUT>(p, plan.waves, s)
                              : launch_fp8_few<4, BROW, OUT>(p, plan.waves, s);
    if (!aligned_rows) {
        uint8_t *a = (uint8_t *)workspace + plan.part_bytes, *b = a + plan.a_bytes;
        if (int st = launch_pack(p.a, p.a_stride, p.M, p.K, a, s))
            return st;
        if (int st = launch_pack(p.b, p.b_stride, p.N, p.K, b, s))
            return st;
        p.a = a;
        p.b = b;
        p.K = (p.K + 15) / 16 * 16;  // the same k blocks
        p.a_stride = p.b_stride = p.K;
    }
    const dim3 grid((unsigned)((int64_t)p.tiles_m * p.tiles_n * p.splits));
    if (OUT == ssd::kBF16 && plan.mb == 8)
        hipLaunchKernelGGL((ssd::fp8_matmul_big_kernel<8, BROW, ssd::kBF16>), grid, dim3(512), 0, s, p);
    else
        hipLaunchKernelGGL((ssd::fp8_matmul_big_kernel<4, BROW, OUT>), grid, dim3(512), 0, s, p);
    if (int st = launch_status())
        return st;
    if (p.splits > 1) {
        hipLaunchKernelGGL((ssd::fp8_split_sum_kernel<OUT>), dim3(flat), dim3(256), 0, s, p);
        return launch_status();
    }
    return SSD_OK;
}

// ------------------------------------------------------------ gated recurrence

constexpr int kGatedWaves = 16, kGatedSteps = 8;  // backwards a wave takes 64 / kGatedWaves tokens

struct GatedPlan {
    int ch;                   // channels per lane
    int blocks;               // channel blocks
    int segments, seg_tokens;
    bool walk;                // a lane per channel walks over the tokens
    size_t seg_bytes;
};

int check_gated(int dtype, int64_t batch, int64_t T, int64_t C, int64_t s0, int64_t s1, int64_t s2)
{
    if (!dtype_ok(dtype) || batch < 0 || T < 0 || C < 1 || s0 < C || s1 < C || s2 < C)
        return SSD_ERR_SHAPE;
    if (T > (1LL << 30) || C > (1LL << 24) || batch > (1LL << 24))
        return SSD_ERR_UNSUPPORTED;
    const int64_t stride = s0 > s1 ? (s0 > s2 ? s0 : s2) : (s1 > s2 ? s1 : s2);
    const int64_t tokens = batch * T;
    if (tokens > 0 && stride > kMaxElems / tokens)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Segments that give about 256 workgroups (one per compute unit), each at least 256 tokens.
int64_t gated_segments(int64_t groups, int64_t T)
{
    const int64_t seg = 256 / groups < T / 256 ? 256 / groups : T / 256;
    return seg < 1 ? 1 : seg;
}

// How the work is cut. Measured in us, bfloat16 unless said:
//  - Channels per lane: two take 1.6 times as long as one, and a compute unit holds one workgroup
//    at a time (32 x 2048 x 1024: 135 with two, 165 with one; cut into segments either way,
//    8 x 4096 x 1024: 113 and 128). But one where only two would need segments, whose gates are
//    formed twice (16 x 2048 x 1024: 81 with one, 118 with two).
//  - Two segments are not worth their second pass in float32, whose forward is bound by memory with
//    128 workgroups already (8 x 4096 x 1024: 143 in one, 164 in two; 1 x 8192 x 5504: 236 and
//    239). In bfloat16, and backwards in either type, they are (8 x 4096 x 1023: 143 against
//    147; gradients of 8 x 4096 x 1024 in float32: 229 against 255). About 128 or 512 workgroups
//    instead of 256: 1 x 32768 x 1024 in float32 239 and 205 against 188.
//  - The walk: a round of the scan's workgroups costs 7 to 10 however few the tokens, the walk 0.2
//    a token (64 x 8 x 1024: 6 and 21; 64 x 32 x 1024: 11 and 20; in one round, 4 x 16 x 256, 7.5
//    and 6.7).
GatedPlan gated_plan(int64_t batch, int64_t T, int64_t C, int dtype, bool backward)
{
    GatedPlan p{};
    batch = batch > 0 ? batch : 1;
    const int64_t one = batch * ((C + 63) / 64), two = batch * ((C + 127) / 128);
    const bool pairs = dtype == SSD_BF16 && C % 2 == 0;
    p.ch = pairs && (gated_segments(two, T) == 1 || gated_segments(one, T) > 1) ? 2 : 1;
    const int64_t groups = p.ch == 2 ? two : one;
    p.blocks = (int)((C + 64 * p.ch - 1) / (64 * p.ch));
    p.walk = !backward && (T <= 8 || (T <= ssd::kGatedWalk && groups > 256));
    if (p.walk) {
        p.ch = p.segments = 1;
        p.blocks = (int)((C + 63) / 64);
        p.seg_tokens = (int)T;
        return p;
    }
    int64_t seg = gated_segments(groups, T);
    if (!backward && dtype == SSD_F32 && seg == 2)
        seg = 1;
    int64_t tokens = (T + seg - 1) / seg;
    tokens = (tokens + ssd::kGatedChunk - 1) / ssd::kGatedChunk * ssd::kGatedChunk;
    p.segments = T > 0 ? (int)((T + tokens - 1) / tokens) : 1;
    p.seg_tokens = (int)tokens;
    p.seg_bytes = p.segments > 1 ? align256((size_t)batch * p.segments * 2 * C * 4) : 0;
    return p;
}

bool gated_grid_ok(const GatedPlan &p, int64_t batch)
{
    return grid_ok(batch * p.blocks * p.segments, p.walk ? 64 : 64 * kGatedWaves);
}

template <int T, int CH>
int launch_gated(ssd::GatedParams p, hipStream_t s)
{
    const dim3 block(64 * kGatedWaves);
    if (p.segments > 1) {
        ssd::GatedParams q = p;
        q.launched = p.segments - 1;
        hipLaunchKernelGGL((ssd::gated_scan_kernel<T, CH, kGatedWaves, kGatedSteps, true>),
                           dim3((unsigned)((int64_t)p.B * p.blocks * q.launched)), block, 0, s, q);
        if (int st = launch_status())
            return st;
    }
    hipLaunchKernelGGL((ssd::gated_scan_kernel<T, CH, kGatedWaves, kGatedSteps, false>),
                       dim3((unsigned)((int64_t)p.B * p.blocks * p.segments)), block, 0, s, p);
    return launch_status();
}

template <int T, int CH>
int launch_gated_bwd(ssd::GatedParams p, float *grad_lam, hipStream_t s)
{
    if (p.segments > 1) {
        ssd::GatedParams q = p;
        q.launched = p.segments - 1;
        q.seg_first = 1;
        hipLaunchKernelGGL((ssd::gated_bwd_summary_kernel<T, CH, kGatedWaves, kGatedSteps>),
                           dim3((unsigned)((int64_t)p.B * p.blocks * q.launched)),
                           dim3(64 * kGatedWaves), 0, s, q);
        if (int st = launch_status())
            return st;
    }
    hipLaunchKernelGGL((ssd::gated_scan_bwd_kernel<T, CH, kGatedWaves>),
                       dim3((unsigned)((int64_t)p.B * p.blocks * p.segments)), dim3(64 * kGatedWaves), 0, s, p);
    if (int st = launch_status())
        return st;
    hipLaunchKernelGGL(ssd::gated_lam_kernel, dim3(grid_1d(p.C, 64)), dim3(1024), 0, s,
                       (const float *)p.part, p.B * p.segments, p.C, p.lam, grad_lam);
    return launch_status();
}

int launch_copy(const float *from, float *to, int64_t n, hipStream_t s)
{
    const int64_t blocks = (n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096;
    hipLaunchKernelGGL(ssd::gated_copy_kernel, dim3((unsigned)blocks), dim3(256), 0, s, from, to, n);
    return launch_status();
}

}  // namespace

extern "C" {

int ssd_rms_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                 const float *weight, int dtype, int64_t rows, int64_t F, float eps, void *y,
                 void *residual_out, uint8_t *q, float *scale, float *rstd, ssd_stream_t stream)
{
    if (int st = check_norm(dtype, rows, F))
        return st;
    if (x_stride < F || (residual && residual_stride < F) || !(eps >= 0.f))
        return SSD_ERR_SHAPE;
    if (rows == 0)
        return SSD_OK;
    if (x_stride > kMaxElems / rows || (residual && residual_stride > kMaxElems / rows))
        return SSD_ERR_UNSUPPORTED;
    if (!x || !weight || (!y && !q) || (q && !scale) || (residual_out && !residual))
        return SSD_ERR_NULL;
    const int e = elem_size(dtype);
    if (!aligned(x, e) || !aligned(residual, e) || !aligned(weight, 4) || !aligned(y, e) ||
        !aligned(residual_out, e) || !aligned(scale, 4) || !aligned(rstd, 4))
        return SSD_ERR_ALIGN;
    const int64_t n = rows * F;
    const struct { const void *p; int64_t bytes; } out[5] = {
        {y, n * e}, {residual_out, n * e}, {q, n}, {q ? scale : nullptr, (F + 127) / 128 * rows * 4},
        {rstd, rows * 4}};
    const int64_t xs = span(rows, F, x_stride, e), rs = span(rows, F, residual_stride, e);
    for (int i = 0; i < 5; ++i) {
        const bool in_place = i == 1 && residual_out == residual && residual_stride == F;
        if (overlap_bytes(out[i].p, out[i].bytes, x, xs) ||
            (!in_place && overlap_bytes(out[i].p, out[i].bytes, residual, rs)) ||
            overlap_bytes(out[i].p, out[i].bytes, weight, F * 4))
            return SSD_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap_bytes(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return SSD_ERR_ALIAS;
    }
    ssd::NormParams p{};
    p.x = x;
    p.res = residual;
    p.w = weight;
    p.y = y;
    p.res_out = residual_out;
    p.q = q;
    p.scale = scale;
    p.rstd = rstd;
    p.rows = rows;
    p.x_stride = x_stride;
    p.res_stride = residual_stride;
    p.F = (int)F;
    p.eps = eps;
    const hipStream_t s = (hipStream_t)stream;
    return dtype == SSD_BF16 ? launch_norm<ssd::kBF16>(p, s) : launch_norm<ssd::kF32>(p, s);
}

size_t ssd_rms_norm_backward_workspace_bytes(int64_t rows, int64_t F)
{
    if (check_norm(SSD_F32, rows, F) || rows == 0)
        return 0;
    return align256((size_t)(norm_bwd_groups(rows, F) * F) * 4);
}

int ssd_rms_norm_backward(const void *s, int64_t s_stride, const float *weight, const float *rstd,
                          const void *grad_y, int64_t grad_y_stride, const void *grad_residual,
                          int64_t grad_residual_stride, int dtype, int64_t rows, int64_t F,
                          void *grad_x, float *grad_weight, void *workspace,
                          size_t workspace_bytes, ssd_stream_t stream)
{
    if (int st = check_norm(dtype, rows, F))
        return st;
    if (s_stride < F || grad_y_stride < F || (grad_residual && grad_residual_stride < F))
        return SSD_ERR_SHAPE;
    const hipStream_t st_ = (hipStream_t)stream;
    if (!grad_weight)
        return SSD_ERR_NULL;
    if (!aligned(grad_weight, 4))
        return SSD_ERR_ALIGN;
    if (rows == 0)
        return launch_copy(nullptr, grad_weight, F, st_);
    if (s_stride > kMaxElems / rows || grad_y_stride > kMaxElems / rows ||
        (grad_residual && grad_residual_stride > kMaxElems / rows))
        return SSD_ERR_UNSUPPORTED;
    if (!s || !weight || !rstd || !grad_y || !grad_x)
        return SSD_ERR_NULL;
    const int e = elem_size(dtype);
    if (!aligned(s, e) || !aligned(weight, 4) || !aligned(rstd, 4) || !aligned(grad_y, e) ||
        !aligned(grad_residual, e) || !aligned(grad_x, e))
        return SSD_ERR_ALIGN;
    const size_t need = ssd_rms_norm_backward_workspace_bytes(rows, F);
    if (!workspace || workspace_bytes < need)
        return SSD_ERR_WORKSPACE;
    if (!aligned(workspace, 256))
        return SSD_ERR_ALIGN;
    const struct { const void *p; int64_t bytes; } in[5] = {
        {s, span(rows, F, s_stride, e)}, {weight, F * 4}, {rstd, rows * 4},
        {grad_y, span(rows, F, grad_y_stride, e)},
        {grad_residual, span(rows, F, grad_residual_stride, e)}};
    const struct { const void *p; int64_t bytes; } out[3] = {
        {grad_x, rows * F * e}, {grad_weight, F * 4}, {workspace, (int64_t)need}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 5; ++j)
            if (overlap_bytes(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
                return SSD_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap_bytes(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return SSD_ERR_ALIAS;
    }
    ssd::NormBwdParams p{};
    p.s = s;
    p.w = weight;
    p.rstd = rstd;
    p.gy = grad_y;
    p.gs = grad_residual;
    p.gx = grad_x;
    p.part = (float *)workspace;
    p.rows = rows;
    p.s_stride = s_stride;
    p.gy_stride = grad_y_stride;
    p.gs_stride = grad_residual_stride;
    p.F = (int)F;
    const int64_t groups = norm_bwd_groups(rows, F);
    if (int st = dtype == SSD_BF16 ? launch_norm_bwd<ssd::kBF16>(p, groups, st_)
                                   : launch_norm_bwd<ssd::kF32>(p, groups, st_))
        return st;
    hipLaunchKernelGGL(ssd::column_sum_kernel, dim3(grid_1d(F, 64)),
                       dim3(64 * ssd::kColumnSumWaves), 0, st_, (const float *)workspace,
                       (int)groups, F, grad_weight);
    return launch_status();
}

int ssd_fp8_quantise(const void *x, int64_t x_stride, int dtype, int64_t rows, int64_t cols,
                     int64_t block_rows, int transpose, uint8_t *q, int64_t q_stride, float *scale,
                     ssd_stream_t stream)
{
    if (!dtype_ok(dtype) || rows < 0 || cols < 1 || (block_rows != 1 && block_rows != 128) ||
        x_stride < cols || q_stride < (transpose ? rows : cols))
        return SSD_ERR_SHAPE;
    if (rows == 0)
        return SSD_OK;
    if (cols > (1LL << 31) || rows > (1LL << 31) || x_stride > kMaxElems / rows ||
        q_stride > kMaxElems / (transpose ? cols : rows))
        return SSD_ERR_UNSUPPORTED;
    if (!x || !q || !scale)
        return SSD_ERR_NULL;
    const int e = elem_size(dtype);
    if (!aligned(x, e) || !aligned(scale, 4))
        return SSD_ERR_ALIGN;
    const int64_t qr = transpose ? cols : rows, qc = transpose ? rows : cols;
    const int64_t scales = (qc + 127) / 128 * (block_rows == 1 ? qr : (qr + 127) / 128) * 4;
    const int64_t xs = span(rows, cols, x_stride, e), qs = span(qr, qc, q_stride, 1);
    if (overlap_bytes(q, qs, x, xs) || overlap_bytes(scale, scales, x, xs) ||
        overlap_bytes(q, qs, scale, scales))
        return SSD_ERR_ALIAS;
    ssd::QuantParams p{};
    p.x = x;
    p.q = q;
    p.scale = scale;
    p.rows = rows;
    p.cols = cols;
    p.x_stride = x_stride;
    p.q_stride = q_stride;
    const hipStream_t s = (hipStream_t)stream;
    const bool whole = block_rows == 128, turn = transpose != 0;
    return dtype == SSD_BF16 ? launch_quantise<ssd::kBF16>(p, whole, turn, s)
                             : launch_quantise<ssd::kF32>(p, whole, turn, s);
}

size_t ssd_fp8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t b_block_rows,
                                      int out_dtype, int rows_on_16)
{
    if (check_fp8(M, N, K, b_block_rows, out_dtype) || M == 0 || K == 0)
        return 0;
    return fp8_plan(M, N, K, out_dtype, rows_on_16 && K % 16 == 0).bytes();
}

int ssd_fp8_matmul(const uint8_t *a, int64_t a_stride, const float *a_scale, const uint8_t *b,
                   int64_t b_stride, const float *b_scale, int64_t M, int64_t N, int64_t K,
                   int64_t b_block_rows, int out_dtype, void *out, int64_t out_stride,
                   void *workspace, size_t workspace_bytes, ssd_stream_t stream)
{
    if (int st = check_fp8(M, N, K, b_block_rows, out_dtype))
        return st;
    if (a_stride < K || b_stride < K || out_stride < N)
        return SSD_ERR_SHAPE;
    if (M == 0)
        return SSD_OK;
    if (a_stride > kMaxElems / M || b_stride > kMaxElems / N || out_stride > kMaxElems / M)
        return SSD_ERR_UNSUPPORTED;
    if (!out || (K > 0 && (!a || !b || !a_scale || !b_scale)))
        return SSD_ERR_NULL;
    const int e = elem_size(out_dtype);
    if (!aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(out, e))
        return SSD_ERR_ALIGN;
    const bool rows16 = K % 16 == 0 && aligned(a, 16) && aligned(b, 16) && a_stride % 16 == 0 &&
                        b_stride % 16 == 0 && a_stride < (1 << 24) && b_stride < (1 << 24);
    const Fp8Plan plan = fp8_plan(M, N, K, out_dtype, rows16);
    if (K > 0 && !plan.few && !grid_ok((int64_t)plan.tiles_m * plan.tiles_n * plan.splits, 512))
        return SSD_ERR_UNSUPPORTED;
    const size_t need = K > 0 ? plan.bytes() : 0;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return SSD_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256))
        return SSD_ERR_ALIGN;
    const int64_t kb = (K + 127) / 128;
    const struct { const void *p; int64_t bytes; } in[4] = {
        {a, span(M, K, a_stride, 1)}, {b, span(N, K, b_stride, 1)}, {a_scale, kb * M * 4},
        {b_scale, kb * (b_block_rows == 1 ? N : (N + 127) / 128) * 4}};
    const int64_t os = span(M, N, out_stride, e);
    for (int j = 0; j < 4; ++j)
        if (overlap_bytes(out, os, in[j].p, in[j].bytes) ||
            (need && overlap_bytes(workspace, (int64_t)need, in[j].p, in[j].bytes)))
            return SSD_ERR_ALIAS;
    if (need && overlap_bytes(workspace, (int64_t)need, out, os))
        return SSD_ERR_ALIAS;
    ssd::Fp8Params p{};
    p.a = a;
    p.b = b;
    p.sa = a_scale;
    p.sb = b_scale;
    p.out = out;
    p.part = (float *)workspace;
    p.a_stride = a_stride;
    p.b_stride = b_stride;
    p.out_stride = out_stride;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.tiles_m = plan.tiles_m;
    p.tiles_n = plan.tiles_n;
    p.splits = plan.splits;
    p.split_blocks = plan.split_blocks;
    const hipStream_t s = (hipStream_t)stream;
    char *ws = (char *)workspace;
    if (b_block_rows == 1)
        return out_dtype == SSD_BF16 ? launch_fp8<true, ssd::kBF16>(p, plan, rows16, ws, s) : launch_fp8<true, ssd::kF32>(p, plan, rows16, ws, s);
    return out_dtype == SSD_BF16 ? launch_fp8<false, ssd::kBF16>(p, plan, rows16, ws, s) : launch_fp8<false, ssd::kF32>(p, plan, rows16, ws, s);
}

size_t ssd_gated_scan_workspace_bytes(int64_t batch, int64_t T, int64_t C, int dtype)
{
    if (check_gated(dtype, batch, T, C, C, C, C) || batch == 0 || T == 0)
        return 0;
    return gated_plan(batch, T, C, dtype, false).seg_bytes;
}

int ssd_gated_scan(const void *x, int64_t x_stride, const void *input_gate,
                   int64_t input_gate_stride, const void *decay_gate, int64_t decay_gate_stride,
                   const float *lam, float decay_scale, int dtype, int64_t batch, int64_t T,
                   int64_t C, const float *initial_state, const int32_t *lengths, void *h,
                   float *final_state, float *chunk_states, void *workspace,
                   size_t workspace_bytes, ssd_stream_t stream)
{
    if (int st = check_gated(dtype, batch, T, C, x_stride, input_gate_stride, decay_gate_stride))
        return st;
    if (!(decay_scale >= 0.f) || decay_scale > 1e30f)
        return SSD_ERR_SHAPE;
    if (batch == 0)
        return SSD_OK;
    const hipStream_t s = (hipStream_t)stream;
    const int e = elem_size(dtype);
    if (!aligned(initial_state, 4) || !aligned(final_state, 4) || !aligned(chunk_states, 4) ||
        !aligned(x, e) || !aligned(input_gate, e) || !aligned(decay_gate, e) || !aligned(lam, 4) ||
        !aligned(lengths, 4) || !aligned(h, e))
        return SSD_ERR_ALIGN;
    const int64_t bc = batch * C * 4;
    if (T == 0) {
        if (!final_state || final_state == initial_state)
            return SSD_OK;
        if (overlap_bytes(final_state, bc, initial_state, bc))
            return SSD_ERR_ALIAS;
        return launch_copy(initial_state, final_state, batch * C, s);
    }
    if (!x || !input_gate || !decay_gate || !lam || !h)
        return SSD_ERR_NULL;
    const GatedPlan plan = gated_plan(batch, T, C, dtype, false);
    if (!gated_grid_ok(plan, batch))
        return SSD_ERR_UNSUPPORTED;
    if (plan.seg_bytes > 0 && (!workspace || workspace_bytes < plan.seg_bytes))
        return SSD_ERR_WORKSPACE;
    if (plan.seg_bytes > 0 && !aligned(workspace, 256))
        return SSD_ERR_ALIGN;
    const int64_t tokens = batch * T;
    const struct { const void *p; int64_t bytes; } in[6] = {
        {x, span(tokens, C, x_stride, e)}, {input_gate, span(tokens, C, input_gate_stride, e)},
        {decay_gate, span(tokens, C, decay_gate_stride, e)}, {lam, C * 4}, {initial_state, bc},
        {lengths, batch * 4}};
    const struct { const void *p; int64_t bytes; } out[4] = {
        {h, tokens * C * e}, {final_state, bc},
        {chunk_states, batch * ((T + SSD_GATED_CHUNK - 1) / SSD_GATED_CHUNK) * C * 4},
        {plan.seg_bytes ? workspace : nullptr, (int64_t)plan.seg_bytes}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 6; ++j)
            if (!(i == 1 && j == 4 && final_state == initial_state) &&
                overlap_bytes(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
                return SSD_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap_bytes(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return SSD_ERR_ALIAS;
    }
    ssd::GatedParams p{};
    p.x = x;
    p.gi = input_gate;
    p.gr = decay_gate;
    p.lam = lam;
    p.init = initial_state;
    p.lengths = lengths;
    p.h = h;
    p.final_state = final_state;
    p.states = chunk_states;
    p.seg = (float *)workspace;
    p.x_stride = x_stride;
    p.gi_stride = input_gate_stride;
    p.gr_stride = decay_gate_stride;
    p.B = (int)batch;
    p.T = (int)T;
    p.C = (int)C;
    p.blocks = plan.blocks;
    p.segments = plan.segments;
    p.seg_tokens = plan.seg_tokens;
    p.launched = plan.segments;
    p.k = decay_scale;
    if (plan.walk) {
        const dim3 grid((unsigned)(batch * p.blocks));
        if (dtype == SSD_BF16)
            hipLaunchKernelGGL((ssd::gated_step_kernel<ssd::kBF16>), grid, dim3(64), 0, s, p);
        else
            hipLaunchKernelGGL((ssd::gated_step_kernel<ssd::kF32>), grid, dim3(64), 0, s, p);
        return launch_status();
    }
    return dtype == SSD_F32 ? launch_gated<ssd::kF32, 1>(p, s)
           : plan.ch == 2   ? launch_gated<ssd::kBF16, 2>(p, s)
                            : launch_gated<ssd::kBF16, 1>(p, s);
}

size_t ssd_gated_scan_backward_workspace_bytes(int64_t batch, int64_t T, int64_t C, int dtype)
{
    if (check_gated(dtype, batch, T, C, C, C, C) || batch == 0 || T == 0)
        return 0;
    const GatedPlan plan = gated_plan(batch, T, C, dtype, true);
    return plan.seg_bytes + align256((size_t)batch * plan.segments * C * 4);
}

int ssd_gated_scan_backward(const void *x, int64_t x_stride, const void *input_gate,
                            int64_t input_gate_stride, const void *decay_gate,
                            int64_t decay_gate_stride, const float *lam, float decay_scale,
                            int dtype, int64_t batch, int64_t T, int64_t C,
                            const float *chunk_states, const int32_t *lengths, const void *grad_h,
                            const float *grad_final_state, void *grad_x, void *grad_input_gate,
                            void *grad_decay_gate, float *grad_lam, float *grad_initial_state,
                            void *workspace, size_t workspace_bytes, ssd_stream_t stream)
{
    if (int st = check_gated(dtype, batch, T, C, x_stride, input_gate_stride, decay_gate_stride))
        return st;
    if (!(decay_scale >= 0.f) || decay_scale > 1e30f)
        return SSD_ERR_SHAPE;
    const hipStream_t s = (hipStream_t)stream;
    const int e = elem_size(dtype);
    if (!grad_lam)
        return SSD_ERR_NULL;
    if (!aligned(chunk_states, 4) || !aligned(grad_final_state, 4) || !aligned(grad_lam, 4) ||
        !aligned(grad_initial_state, 4) || !aligned(x, e) || !aligned(input_gate, e) ||
        !aligned(decay_gate, e) || !aligned(lam, 4) || !aligned(lengths, 4) || !aligned(grad_h, e) ||
        !aligned(grad_x, e) || !aligned(grad_input_gate, e) || !aligned(grad_decay_gate, e))
        return SSD_ERR_ALIGN;
    const int64_t bc = batch * C * 4, tokens = batch * T;
    if (tokens > 0 && (!x || !input_gate || !decay_gate || !lam || !chunk_states || !grad_h ||
                       !grad_x || !grad_input_gate || !grad_decay_gate))
        return SSD_ERR_NULL;
    const GatedPlan plan = gated_plan(batch, T, C, dtype, true);
    if (tokens > 0 && !gated_grid_ok(plan, batch))
        return SSD_ERR_UNSUPPORTED;
    const size_t need = ssd_gated_scan_backward_workspace_bytes(batch, T, C, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return SSD_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256))
        return SSD_ERR_ALIGN;
    const struct { const void *p; int64_t bytes; } in[8] = {
        {x, span(tokens, C, x_stride, e)}, {input_gate, span(tokens, C, input_gate_stride, e)},
        {decay_gate, span(tokens, C, decay_gate_stride, e)}, {lam, C * 4},
        {chunk_states, batch * ((T + SSD_GATED_CHUNK - 1) / SSD_GATED_CHUNK) * C * 4},
        {lengths, batch * 4}, {grad_h, tokens * C * e}, {grad_final_state, bc}};
    const struct { const void *p; int64_t bytes; } out[6] = {
        {grad_x, tokens * C * e}, {grad_input_gate, tokens * C * e},
        {grad_decay_gate, tokens * C * e}, {grad_lam, C * 4}, {grad_initial_state, bc},
        {need ? workspace : nullptr, (int64_t)need}};
    for (int i = 0; i < 6; ++i) {
        for (int j = 0; j < 8; ++j)
            if (overlap_bytes(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
                return SSD_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap_bytes(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return SSD_ERR_ALIAS;
    }
    if (tokens == 0) {
        if (int st = launch_copy(nullptr, grad_lam, C, s))
            return st;
        if (grad_initial_state && batch > 0)
            return launch_copy(grad_final_state, grad_initial_state, batch * C, s);
        return SSD_OK;
    }
    ssd::GatedParams p{};
    p.x = x;
    p.gi = input_gate;
    p.gr = decay_gate;
    p.lam = lam;
    p.lengths = lengths;
    p.seg = (float *)workspace;
    p.gh = grad_h;
    p.gfinal = grad_final_state;
    p.chunk_states = chunk_states;
    p.gx = grad_x;
    p.ggi = grad_input_gate;
    p.ggr = grad_decay_gate;
    p.part = (float *)((char *)workspace + plan.seg_bytes);
    p.ginit = grad_initial_state;
    p.x_stride = x_stride;
    p.gi_stride = input_gate_stride;
    p.gr_stride = decay_gate_stride;
    p.B = (int)batch;
    p.T = (int)T;
    p.C = (int)C;
    p.blocks = plan.blocks;
    p.segments = plan.segments;
    p.seg_tokens = plan.seg_tokens;
    p.launched = plan.segments;
    p.k = decay_scale;
    return dtype == SSD_F32 ? launch_gated_bwd<ssd::kF32, 1>(p, grad_lam, s)
           : plan.ch == 2   ? launch_gated_bwd<ssd::kBF16, 2>(p, grad_lam, s)
                            : launch_gated_bwd<ssd::kBF16, 1>(p, grad_lam, s);
}

}  // extern "C"
