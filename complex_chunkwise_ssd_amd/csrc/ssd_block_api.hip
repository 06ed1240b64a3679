// ssd_block_api.hip -- C ABI of the norms around a block (declared in include/ssd.h): argument checks, work
// planning and kernel launches on the caller's stream; nothing is allocated.
#include "ssd.h"

#include <ssd_block_norm_kernels.h>
#include <ssd_host.h>

namespace {

using ssd::align256;
using ssd::aligned;
using ssd::grid_1d;
using ssd::kMaxElems;
using ssd::launch_status;
using ssd::Range;
using ssd::span;

int check_rows(int dtype, int64_t rows, int64_t F)
{
    if (!ssd::dtype_ok(dtype) || rows < 0 || F < 1)
        return SSD_ERR_SHAPE;
    return F > ssd::kNormMaxF || rows > (1LL << 31) - 1 ? SSD_ERR_UNSUPPORTED : SSD_OK;
}

int check_heads(int64_t F, int64_t D)
{
    if (D < 1 || F % D != 0)
        return SSD_ERR_SHAPE;
    return D < 8 ? SSD_ERR_UNSUPPORTED : SSD_OK;
}

bool strides_long(int64_t rows, int64_t a, int64_t b, int64_t c = 0, int64_t d = 0)
{
    const int64_t most = kMaxElems / (rows > 0 ? rows : 1);
    return a > most || b > most || c > most || d > most;
}

// Workgroups: they walk over the rows.
int64_t row_groups(int64_t rows, int held, int64_t most)
{
    const int64_t need = (rows + held - 1) / held;
    return need < most ? need : most;
}
// Backwards a lane adds its rows' shares of the weights' gradients in float32: kChain of them at most, however many
// rows there are, and the workgroups' shares are added in float64.
constexpr int64_t kChain = 256;
int64_t bwd_groups(int64_t rows, int64_t F)
{
    const int held = F <= 128 ? 16 : F <= 1024 ? 4 : 1;
    const int64_t few = F <= 4096 ? 1024 : 512, chains = (rows + held * kChain - 1) / (held * kChain);
    const int64_t most = ssd::kMaxThreads / 1024;  // of one launch
    return row_groups(rows, held, chains < few ? few : chains < most ? chains : most);
}

// Lanes of a head, as a power of two, or -1 (see the kernels).
int head_lanes(int64_t D)
{
    for (int log = 0; log <= 4; ++log)
        if (D == 8LL << log)
            return log;
    return -1;
}

#define SSD_BY_WIDTH(F, CALL)                \
    ((F) <= 128    ? CALL(16, 1)             \
     : (F) <= 512  ? CALL(64, 1)             \
     : (F) <= 1024 ? CALL(64, 2)             \
     : (F) <= 2048 ? CALL(256, 1)            \
     : (F) <= 4096 ? CALL(256, 2)            \
     : (F) <= 8192 ? CALL(512, 2)            \
                   : CALL(1024, 2))

template <int T, int LANES, int STEPS, bool BACKWARD>
int launch_gated_as(const ssd::GatedNormParams &p, hipStream_t s)
{
    using Shape = ssd::NormShape<LANES>;
    const int64_t groups = BACKWARD ? bwd_groups(p.rows, p.F) : row_groups(p.rows, Shape::rows, 2048);
    const dim3 grid((unsigned)groups), block(Shape::threads);
    const bool whole = p.log_lanes >= 0;
    if (BACKWARD && whole)
        hipLaunchKernelGGL((ssd::gated_norm_bwd_kernel<T, LANES, STEPS, true>), grid, block, 0, s, p);
    else if (BACKWARD)
        hipLaunchKernelGGL((ssd::gated_norm_bwd_kernel<T, LANES, STEPS, false>), grid, block, 0, s, p);
    else if (whole)
        hipLaunchKernelGGL((ssd::gated_norm_kernel<T, LANES, STEPS, true>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((ssd::gated_norm_kernel<T, LANES, STEPS, false>), grid, block, 0, s, p);
    return launch_status();
}
template <int T, bool BACKWARD>
int launch_gated(const ssd::GatedNormParams &p, hipStream_t s)
{
#define CALL(LANES, STEPS) launch_gated_as<T, LANES, STEPS, BACKWARD>(p, s)
    return SSD_BY_WIDTH(p.F, CALL);
#undef CALL
}

template <int T, int LANES, int STEPS, bool BACKWARD>
int launch_block_as(const ssd::BlockNormParams &p, hipStream_t s)
{
    using Shape = ssd::NormShape<LANES>;
    const int64_t groups = BACKWARD ? bwd_groups(p.rows, p.F) : row_groups(p.rows, Shape::rows, 2048);
    const dim3 grid((unsigned)groups), block(Shape::threads);
    if (BACKWARD)
        hipLaunchKernelGGL((ssd::block_norm_bwd_kernel<T, LANES, STEPS>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((ssd::block_norm_kernel<T, LANES, STEPS>), grid, block, 0, s, p);
    return launch_status();
}
template <int T, bool BACKWARD>
int launch_block(const ssd::BlockNormParams &p, hipStream_t s)
{
#define CALL(LANES, STEPS) launch_block_as<T, LANES, STEPS, BACKWARD>(p, s)
    return SSD_BY_WIDTH(p.F, CALL);
#undef CALL
}

int launch_zero(float *out, int64_t n, hipStream_t s)
{
    hipLaunchKernelGGL(ssd::share_zero_kernel, dim3(grid_1d(n, 256)), dim3(256), 0, s, out, (int)n);
    return launch_status();
}

int launch_shares(const void *part, int64_t rows, int64_t n, int64_t split, float *out0, float *out1, hipStream_t s)
{
    hipLaunchKernelGGL(ssd::share_sum_kernel, dim3(grid_1d(n, 64)), dim3(64 * ssd::kShareSumWaves), 0, s,
                       (const float *)part, (int)rows, (int)n, (int)split, out0, out1);
    return launch_status();
}

}  // namespace

extern "C" {

int ssd_gated_norm(const void *x, int64_t x_stride, const void *gate, int64_t gate_stride, const float *weight,
                   int dtype, int64_t rows, int64_t F, int64_t D, float eps, void *y, uint8_t *q, float *scale,
                   float *rstd, ssd_stream_t stream)
{
    if (int st = check_rows(dtype, rows, F))
        return st;
    if (int st = check_heads(F, D))
        return st;
    if (x_stride < F || gate_stride < F || !(eps >= 0.f))
        return SSD_ERR_SHAPE;
    if (rows == 0)
        return SSD_OK;
    if (strides_long(rows, x_stride, gate_stride))
        return SSD_ERR_UNSUPPORTED;
    if (!x || !gate || !weight || (!y && !q) || (q && !scale))
        return SSD_ERR_NULL;
    const int e = ssd::elem_size(dtype);
    if (!aligned(x, e) || !aligned(gate, e) || !aligned(weight, 4) || !aligned(y, e) || !aligned(scale, 4) ||
        !aligned(rstd, 4))
        return SSD_ERR_ALIGN;
    const Range in[3] = {{x, span(rows, F, x_stride, e)}, {gate, span(rows, F, gate_stride, e)}, {weight, D * 4}};
    const Range out[4] = {{y, rows * F * e}, {q, rows * F}, {q ? scale : nullptr, (F + 127) / 128 * rows * 4},
                          {rstd, rows * (F / D) * 4}};
    if (ssd::overlaps(out, 4, in, 3))
        return SSD_ERR_ALIAS;
    ssd::GatedNormParams p{};
    p.x = x;
    p.gate = gate;
    p.w = weight;
    p.y = y;
    p.q = q;
    p.scale = scale;
    p.rstd = rstd;
    p.rows = rows;
    p.x_stride = x_stride;
    p.gate_stride = gate_stride;
    p.F = (int)F;
    p.D = (int)D;
    p.H = (int)(F / D);
    p.log_lanes = head_lanes(D);
    p.eps = eps;
    const hipStream_t s = (hipStream_t)stream;
    return dtype == SSD_BF16 ? launch_gated<ssd::kBF16, false>(p, s) : launch_gated<ssd::kF32, false>(p, s);
}

size_t ssd_gated_norm_backward_workspace_bytes(int64_t rows, int64_t F, int64_t D)
{
    if (check_rows(SSD_F32, rows, F) || check_heads(F, D) || rows == 0)
        return 0;
    return align256((size_t)(bwd_groups(rows, F) * D) * 4);
}

int ssd_gated_norm_backward(const void *x, int64_t x_stride, const void *gate, int64_t gate_stride, const float *weight,
                            const float *rstd, const void *grad_y, int64_t grad_y_stride, int dtype, int64_t rows,
                            int64_t F, int64_t D, void *grad_x, void *grad_gate, float *grad_weight, void *workspace,
                            size_t workspace_bytes, ssd_stream_t stream)
{
    if (int st = check_rows(dtype, rows, F))
        return st;
    if (int st = check_heads(F, D))
        return st;
    if (x_stride < F || gate_stride < F || grad_y_stride < F)
        return SSD_ERR_SHAPE;
    if (!grad_weight)
        return SSD_ERR_NULL;
    if (!aligned(grad_weight, 4))
        return SSD_ERR_ALIGN;
    const hipStream_t s = (hipStream_t)stream;
    if (rows == 0)
        return launch_zero(grad_weight, D, s);
    if (strides_long(rows, x_stride, gate_stride, grad_y_stride))
        return SSD_ERR_UNSUPPORTED;
    if (!x || !gate || !weight || !rstd || !grad_y || !grad_x || !grad_gate)
        return SSD_ERR_NULL;
    const int e = ssd::elem_size(dtype);
    if (!aligned(x, e) || !aligned(gate, e) || !aligned(weight, 4) || !aligned(rstd, 4) || !aligned(grad_y, e) ||
        !aligned(grad_x, e) || !aligned(grad_gate, e))
        return SSD_ERR_ALIGN;
    const size_t need = ssd_gated_norm_backward_workspace_bytes(rows, F, D);
    if (!workspace || workspace_bytes < need)
        return SSD_ERR_WORKSPACE;
    if (!aligned(workspace, 256))
        return SSD_ERR_ALIGN;
    const Range in[5] = {{x, span(rows, F, x_stride, e)}, {gate, span(rows, F, gate_stride, e)}, {weight, D * 4},
                         {rstd, rows * (F / D) * 4}, {grad_y, span(rows, F, grad_y_stride, e)}};
    const Range out[4] = {{grad_x, rows * F * e}, {grad_gate, rows * F * e}, {grad_weight, D * 4},
                          {workspace, (int64_t)need}};
    if (ssd::overlaps(out, 4, in, 5))
        return SSD_ERR_ALIAS;
    ssd::GatedNormParams p{};
    p.x = x;
    p.gate = gate;
    p.w = weight;
    p.rstd = (float *)rstd;
    p.gy = grad_y;
    p.gx = grad_x;
    p.gz = grad_gate;
    p.part = (float *)workspace;
    p.rows = rows;
    p.x_stride = x_stride;
    p.gate_stride = gate_stride;
    p.gy_stride = grad_y_stride;
    p.F = (int)F;
    p.D = (int)D;
    p.H = (int)(F / D);
    p.log_lanes = head_lanes(D);
    if (int st = dtype == SSD_BF16 ? launch_gated<ssd::kBF16, true>(p, s) : launch_gated<ssd::kF32, true>(p, s))
        return st;
    return launch_shares(workspace, bwd_groups(rows, F), D, D, grad_weight, nullptr, s);
}

int ssd_block_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                   const float *post_weight, const float *pre_weight, float residual_scale, int dtype, int64_t rows,
                   int64_t F, float eps, void *y, void *residual_out, uint8_t *q, float *scale, float *post_rstd,
                   float *pre_rstd, ssd_stream_t stream)
{
    if (int st = check_rows(dtype, rows, F))
        return st;
    if (x_stride < F || residual_stride < F || !(eps >= 0.f) || !(residual_scale >= -1e30f && residual_scale <= 1e30f))
        return SSD_ERR_SHAPE;
    if (rows == 0)
        return SSD_OK;
    if (strides_long(rows, x_stride, residual_stride))
        return SSD_ERR_UNSUPPORTED;
    if (!x || !residual || !post_weight || !pre_weight || !residual_out || (!y && !q) || (q && !scale))
        return SSD_ERR_NULL;
    const int e = ssd::elem_size(dtype);
    if (!aligned(x, e) || !aligned(residual, e) || !aligned(post_weight, 4) || !aligned(pre_weight, 4) ||
        !aligned(y, e) || !aligned(residual_out, e) || !aligned(scale, 4) || !aligned(post_rstd, 4) ||
        !aligned(pre_rstd, 4))
        return SSD_ERR_ALIGN;
    const bool in_place = residual_out == residual && residual_stride == F;
    const Range in[4] = {{x, span(rows, F, x_stride, e)}, {post_weight, F * 4}, {pre_weight, F * 4},
                         {in_place ? nullptr : residual, span(rows, F, residual_stride, e)}};
    const Range out[6] = {{y, rows * F * e}, {residual_out, rows * F * e}, {q, rows * F},
                          {q ? scale : nullptr, (F + 127) / 128 * rows * 4}, {post_rstd, rows * 4}, {pre_rstd, rows * 4}};
    if (ssd::overlaps(out, 6, in, 4))
        return SSD_ERR_ALIAS;
    ssd::BlockNormParams p{};
    p.x = x;
    p.res = residual;
    p.w1 = post_weight;
    p.w2 = pre_weight;
    p.y = y;
    p.res_out = residual_out;
    p.q = q;
    p.scale = scale;
    p.rstd1 = post_rstd;
    p.rstd2 = pre_rstd;
    p.rows = rows;
    p.x_stride = x_stride;
    p.res_stride = residual_stride;
    p.F = (int)F;
    p.alpha = residual_scale;
    p.eps = eps;
    const hipStream_t s = (hipStream_t)stream;
    return dtype == SSD_BF16 ? launch_block<ssd::kBF16, false>(p, s) : launch_block<ssd::kF32, false>(p, s);
}

size_t ssd_block_norm_backward_workspace_bytes(int64_t rows, int64_t F)
{
    if (check_rows(SSD_F32, rows, F) || rows == 0)
        return 0;
    return align256((size_t)(bwd_groups(rows, F) * 2 * F) * 4);
}

int ssd_block_norm_backward(const void *x, int64_t x_stride, const void *s, int64_t s_stride, const float *post_weight,
                            const float *pre_weight, const float *post_rstd, const float *pre_rstd, float residual_scale,
                            const void *grad_y, int64_t grad_y_stride, const void *grad_residual,
                            int64_t grad_residual_stride, int dtype, int64_t rows, int64_t F, void *grad_x,
                            void *grad_residual_in, float *grad_post_weight, float *grad_pre_weight, void *workspace,
                            size_t workspace_bytes, ssd_stream_t stream)
{
    if (int st = check_rows(dtype, rows, F))
        return st;
    if (x_stride < F || s_stride < F || grad_y_stride < F || (grad_residual && grad_residual_stride < F) ||
        !(residual_scale >= -1e30f && residual_scale <= 1e30f))
        return SSD_ERR_SHAPE;
    if (!grad_post_weight || !grad_pre_weight)
        return SSD_ERR_NULL;
    if (!aligned(grad_post_weight, 4) || !aligned(grad_pre_weight, 4))
        return SSD_ERR_ALIGN;
    const hipStream_t st_ = (hipStream_t)stream;
    if (rows == 0) {
        if (ssd::overlap_bytes(grad_post_weight, F * 4, grad_pre_weight, F * 4))
            return SSD_ERR_ALIAS;
        if (int st = launch_zero(grad_post_weight, F, st_))
            return st;
        return launch_zero(grad_pre_weight, F, st_);
    }
    if (strides_long(rows, x_stride, s_stride, grad_y_stride, grad_residual ? grad_residual_stride : 0))
        return SSD_ERR_UNSUPPORTED;
    if (!x || !s || !post_weight || !pre_weight || !post_rstd || !pre_rstd || !grad_y || !grad_x || !grad_residual_in)
        return SSD_ERR_NULL;
    const int e = ssd::elem_size(dtype);
    if (!aligned(x, e) || !aligned(s, e) || !aligned(post_weight, 4) || !aligned(pre_weight, 4) ||
        !aligned(post_rstd, 4) || !aligned(pre_rstd, 4) || !aligned(grad_y, e) || !aligned(grad_residual, e) ||
        !aligned(grad_x, e) || !aligned(grad_residual_in, e))
        return SSD_ERR_ALIGN;
    const size_t need = ssd_block_norm_backward_workspace_bytes(rows, F);
    if (!workspace || workspace_bytes < need)
        return SSD_ERR_WORKSPACE;
    if (!aligned(workspace, 256))
        return SSD_ERR_ALIGN;
    const Range in[8] = {{x, span(rows, F, x_stride, e)}, {s, span(rows, F, s_stride, e)}, {post_weight, F * 4},
                         {pre_weight, F * 4}, {post_rstd, rows * 4}, {pre_rstd, rows * 4},
                         {grad_y, span(rows, F, grad_y_stride, e)},
                         {grad_residual, span(rows, F, grad_residual_stride, e)}};
    const Range out[5] = {{grad_x, rows * F * e}, {grad_residual_in, rows * F * e}, {grad_post_weight, F * 4},
                          {grad_pre_weight, F * 4}, {workspace, (int64_t)need}};
    if (ssd::overlaps(out, 5, in, 8))
        return SSD_ERR_ALIAS;
    ssd::BlockNormParams p{};
    p.x = x;
    p.res = s;
    p.w1 = post_weight;
    p.w2 = pre_weight;
    p.rstd1 = (float *)post_rstd;
    p.rstd2 = (float *)pre_rstd;
    p.gy = grad_y;
    p.gs = grad_residual;
    p.gx = grad_x;
    p.gres = grad_residual_in;
    p.part = (float *)workspace;
    p.rows = rows;
    p.x_stride = x_stride;
    p.res_stride = s_stride;
    p.gy_stride = grad_y_stride;
    p.gs_stride = grad_residual_stride;
    p.F = (int)F;
    p.alpha = residual_scale;
    if (int st = dtype == SSD_BF16 ? launch_block<ssd::kBF16, true>(p, st_) : launch_block<ssd::kF32, true>(p, st_))
        return st;
    return launch_shares(workspace, bwd_groups(rows, F), 2 * F, F, grad_post_weight, grad_pre_weight, st_);
}

}  // extern "C"
