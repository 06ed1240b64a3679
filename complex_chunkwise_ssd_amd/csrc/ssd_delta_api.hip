// ssd_delta_api.hip -- C ABI of the gated delta rule (declared in include/ssd.h): argument checks,
// work planning and kernel launches on the caller's stream; nothing is allocated.
#include "ssd.h"

#include <ssd_delta_kernels.h>
#include <ssd_host.h>

#include <math.h>

namespace {

using ssd::align256;
using ssd::aligned;
using ssd::grid_ok;
using ssd::kMaxElems;
using ssd::launch_status;

struct DeltaSizes {
    int64_t B, T, Hk, Hv, Dk, Dv;
    int64_t chunks() const { return (T + ssd::kDeltaChunk - 1) / ssd::kDeltaChunk; }
    int64_t states() const { return B * Hv * Dk * Dv * 4; }  // bytes
    bool empty() const { return B == 0 || T == 0; }
};

int check_delta(const DeltaSizes &z, int dtype, float scale)
{
    if (!ssd::dtype_ok(dtype) || z.B < 0 || z.T < 0 || z.Hk < 1 || z.Hv < 1 || z.Dk < 1 || z.Dv < 1 ||
        !(fabsf(scale) <= 1e30f))
        return SSD_ERR_SHAPE;
    if (z.Dk > 128 || z.Dv > 256)
        return SSD_ERR_BLOCK_DIMS;
    if (z.B > (1LL << 24) || z.T > (1LL << 30) || z.Hk > (1LL << 16) || z.Hv > (1LL << 16))
        return SSD_ERR_UNSUPPORTED;
    if (z.Hv % z.Hk != 0)
        return SSD_ERR_SHAPE;
    const int64_t column_blocks = z.Dv <= 64 ? 1 : (z.Dv + 127) / 128 * 2;  // of 256 threads: the walks take up to 512
    const int64_t most = column_blocks > z.chunks() ? column_blocks : z.chunks();
    // a batch has 2^40 heads at most, whose chunks pass 2^63
    return z.B * z.Hv <= ssd::kMaxThreads && grid_ok(z.B * z.Hv * most, 256) ? SSD_OK : SSD_ERR_UNSUPPORTED;
}

int check_delta_strides(const DeltaSizes &z, int64_t q, int64_t k, int64_t v)
{
    if (q < z.Hk * z.Dk || k < z.Hk * z.Dk || v < z.Hv * z.Dv)
        return SSD_ERR_SHAPE;
    const int64_t most = q > k ? (q > v ? q : v) : (k > v ? k : v);
    // offsets within a chunk of 64 tokens have 32 bits
    if (most > (1LL << 23) || z.Hv * z.Dv > (1LL << 23) || (!z.empty() && most > kMaxElems / (z.B * z.T)))
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

bool delta_few(const DeltaSizes &z) { return z.T <= ssd::kDeltaFew; }

// Whether a call's heads are too few for a walk of their own to fill the chip, in blocks of 64 columns. A packed walk's time
// grows with the blocks, the other's hardly does up to a workgroup (or two) for each compute unit. Both
// measured from 32 to 768 blocks with heads of 64 and of 128; at one side and the other of each bound (2048 tokens, us, packed /
// not; at 200 and at 8192 tokens they cross at the same place):
//   bfloat16          64 x 64     96 blocks 223 / 252   128 blocks 274 / 253     64 x 128   128: 188 / 254   192: 274 / 257
//                     128 x 64    96        288 / 327   128        338 / 336    128 x 128   128: 257 / 349   192: 428 / 355
//   its gradients     64 x 64     96        361 / 393   160        609 / 499     64 x 128   128: 456 / 516   192: 725 / 655
//   with 128 features 128 x 64    64        484 / 556    96        784 / 688    128 x 128    96: 702 / 712   128: 859 / 835
//   float32           64 x 64    128        412 / 463   160        585 / 466     64 x 128   128: 290 / 446   192: 479 / 467
//                     128 x 64   128        676 / 745   160        948 / 750    128 x 128   128: 524 / 872   192: 940 / 896
//   its gradients     64 x 64    128        767 / 793   160       1032 / 879     64 x 128   128: 691 / 842   192: 1076 / 1038
//                     128 x 64    96       1248 / 1326  160       2015 / 1731   128 x 128   128: 1241 / 1571 256: 2484 / 2268
//   float32           128 x 256  192        756 / 877   256        912 / 919   (gradients 1530 / 1729, 2045 / 2016)
bool delta_long(const DeltaSizes &z, int dtype, bool backward)
{
    const bool wide = z.Dv > 64;
    const int64_t most = dtype == SSD_F32         ? (z.Dk > 64 && z.Dv > 128 ? 240 : wide ? 176 : 128)
                         : backward && z.Dk > 64 ? (wide ? 112 : 80)
                                                 : (wide ? 160 : 112);
    return z.B * z.Hv * ((z.Dv + 63) / 64) <= most;
}

template <int T, int KP>
constexpr size_t pack_bytes() { return 16 * (size_t)ssd::DeltaPack<T, KP>::size; }

// Bytes that a chunk of a head is packed into; chunks that are packed at a time (some 192 MB, which the caches of the
// memory side hold until they are read).
struct DeltaRange {
    int64_t chunks;
    size_t pack, carry;
    size_t bytes() const { return pack + carry; }
};
DeltaRange delta_range(const DeltaSizes &z, int dtype, bool backward)
{
    if (!delta_long(z, dtype, backward))
        return {0, 0, 0};
    const size_t one = dtype == SSD_BF16 ? (z.Dk <= 64 ? pack_bytes<ssd::kBF16, 2>() : pack_bytes<ssd::kBF16, 4>())
                                         : (z.Dk <= 64 ? pack_bytes<ssd::kF32, 2>() : pack_bytes<ssd::kF32, 4>());
    const size_t heads = one * (size_t)(z.B * z.Hv);
    int64_t chunks = (int64_t)((size_t)192 * 1024 * 1024 / heads);
    chunks = chunks < 1 ? 1 : chunks < z.chunks() ? chunks : z.chunks();
    return {chunks, align256(heads * (size_t)chunks), align256((size_t)z.states())};
}

// Workspace of the gradients: dS' and dR of every chunk, and dQ and dK by value heads where they share keys.
struct DeltaSpace {
    size_t gs, gr, w;
    size_t bytes() const { return gs + gr + 2 * w; }
};
DeltaSpace delta_space(const DeltaSizes &z)
{
    const size_t each = (size_t)(z.B * z.Hv * z.chunks());
    return {align256(each * z.Dk * z.Dv * 4), align256(each * 64 * z.Dv * 4),
            z.Hv > z.Hk ? align256((size_t)(z.B * z.T * z.Hv) * z.Dk * 4) : 0};
}

ssd::DeltaParams delta_params(const DeltaSizes &z, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                              const void *v, int64_t v_stride, const float *g, const float *beta, float scale,
                              const int32_t *lengths)
{
    ssd::DeltaParams p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.g = g;
    p.beta = beta;
    p.lengths = lengths;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.B = (int)z.B;
    p.T = (int)z.T;
    p.Hk = (int)z.Hk;
    p.Hv = (int)z.Hv;
    p.Dk = (int)z.Dk;
    p.Dv = (int)z.Dv;
    p.chunks = (int)z.chunks();
    p.columns = (int)((z.Dv + 63) / 64);
    p.scale = scale;
    return p;
}

template <int T>
int launch_delta_few(const ssd::DeltaParams &p, hipStream_t s)
{
    const dim3 grid((unsigned)((int64_t)p.B * p.Hv * p.columns)), block(256);
    if (p.Dk <= 64)
        hipLaunchKernelGGL((ssd::delta_few_kernel<T, 4>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((ssd::delta_few_kernel<T, 8>), grid, block, 0, s, p);
    return launch_status();
}

template <int T, int KP, int WAVES>
int launch_delta_as(ssd::DeltaParams p, hipStream_t s)
{
    p.columns = (p.Dv + 16 * WAVES - 1) / (16 * WAVES);
    hipLaunchKernelGGL((ssd::delta_scan_kernel<T, KP, WAVES>), dim3((unsigned)((int64_t)p.B * p.Hv * p.columns)),
                       dim3(64 * WAVES), 0, s, p);
    return launch_status();
}
// Range after range of chunks, packed and walked over.
template <int T, int KP, bool BACKWARD>
int launch_delta_long(ssd::DeltaParams p, const DeltaRange &range, char *workspace, hipStream_t s)
{
    p.pack = (v4u *)workspace;
    p.carry = (float *)(workspace + range.pack);
    p.columns = (p.Dv + 15) / 16;
    const int64_t heads = (int64_t)p.B * p.Hv;
    const int ranges = (int)((p.chunks + range.chunks - 1) / range.chunks);
    for (int i = 0; i < ranges; ++i) {
        p.chunk_from = (int)range.chunks * (BACKWARD ? ranges - 1 - i : i);
        p.chunk_to = p.chunk_from + (int)range.chunks < p.chunks ? p.chunk_from + (int)range.chunks : p.chunks;
        hipLaunchKernelGGL((ssd::delta_pack_kernel<T, KP, BACKWARD>), dim3((unsigned)(heads * (p.chunk_to - p.chunk_from))),
                           dim3(256), 0, s, p);
        if (int st = launch_status())
            return st;
        const dim3 grid((unsigned)((heads + 7) / 8 * 8 * p.columns));
        if constexpr (BACKWARD) {
            hipLaunchKernelGGL((ssd::delta_spans_bwd_kernel<T, KP>), grid, dim3(64 * KP), 0, s, p);
        } else if constexpr (T == ssd::kBF16) {
            hipLaunchKernelGGL((ssd::delta_long_kernel<T, KP>), grid, dim3(128), 0, s, p);
        } else if (KP == 2 || heads * p.columns <= ssd::kSpansMost) {
            hipLaunchKernelGGL((ssd::delta_spans_kernel<T, KP>), grid, dim3(64 * KP), 0, s, p);
        } else {
            hipLaunchKernelGGL((ssd::delta_long_kernel<T, 4>), grid, dim3(128), 0, s, p);
        }
        if (int st = launch_status())
            return st;
    }
    return SSD_OK;
}

template <int T, int KP>
int launch_delta(const ssd::DeltaParams &p, const DeltaRange &range, char *workspace, hipStream_t s)
{
    if (range.chunks > 0)
        return launch_delta_long<T, KP, false>(p, range, workspace, s);
    if constexpr (KP == 4)
        if (p.Dv > 64)
            return launch_delta_as<T, KP, 8>(p, s);
    return launch_delta_as<T, KP, 4>(p, s);
}

template <int T, int KP, int WAVES>
int launch_delta_scan_bwd(ssd::DeltaParams p, hipStream_t s)
{
    p.columns = (p.Dv + 16 * WAVES - 1) / (16 * WAVES);
    hipLaunchKernelGGL((ssd::delta_scan_bwd_kernel<T, KP, WAVES>), dim3((unsigned)((int64_t)p.B * p.Hv * p.columns)),
                       dim3(64 * WAVES), 0, s, p);
    return launch_status();
}
template <int T, int KP>
int launch_delta_walk_bwd(const ssd::DeltaParams &p, const DeltaRange &range, char *workspace, hipStream_t s)
{
    if (range.chunks > 0)
        return launch_delta_long<T, KP, true>(p, range, workspace, s);
    if constexpr (KP == 4)
        if (p.Dv > 64)
            return launch_delta_scan_bwd<T, KP, 8>(p, s);
    return launch_delta_scan_bwd<T, KP, 4>(p, s);
}
template <int T, int KP>
int launch_delta_bwd(const ssd::DeltaParams &p, const DeltaRange &range, char *workspace, hipStream_t s)
{
    if (int st = launch_delta_walk_bwd<T, KP>(p, range, workspace, s))
        return st;
    const dim3 grid((unsigned)((int64_t)p.B * p.Hv * p.chunks)), block(256);
    if (p.Dv > 64)
        hipLaunchKernelGGL((ssd::delta_grad_kernel<T, KP, true>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((ssd::delta_grad_kernel<T, KP, false>), grid, block, 0, s, p);
    if (int st = launch_status())
        return st;
    if (p.Hv > p.Hk) {
        const int64_t blocks = ((int64_t)p.B * p.T * p.Hk * p.Dk + 255) / 256;
        hipLaunchKernelGGL((ssd::delta_share_kernel<T>), dim3((unsigned)(blocks < 8192 ? blocks : 8192)), block, 0, s, p);
        return launch_status();
    }
    return SSD_OK;
}

int launch_delta_copy(const float *from, float *to, int64_t n, hipStream_t s)
{
    const int64_t blocks = (n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096;
    if (!to || n == 0 || from == to)
        return SSD_OK;
    hipLaunchKernelGGL(ssd::delta_copy_kernel, dim3((unsigned)blocks), dim3(256), 0, s, from, to, n);
    return launch_status();
}

}  // namespace

extern "C" {

size_t ssd_gated_delta_workspace_bytes(int64_t batch, int64_t T, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv,
                                       int dtype)
{
    const DeltaSizes z{batch, T, Hk, Hv, Dk, Dv};
    if (check_delta(z, dtype, 1.f) || z.empty() || delta_few(z))
        return 0;
    return delta_range(z, dtype, false).bytes();
}

int ssd_gated_delta(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                    const float *g, const float *beta, float scale, int dtype, int64_t batch, int64_t T, int64_t Hk,
                    int64_t Hv, int64_t Dk, int64_t Dv, const float *initial_state, const int32_t *lengths, void *o,
                    float *final_state, float *chunk_states, void *workspace, size_t workspace_bytes,
                    ssd_stream_t stream)
{
    const DeltaSizes z{batch, T, Hk, Hv, Dk, Dv};
    if (int st = check_delta(z, dtype, scale))
        return st;
    if (int st = check_delta_strides(z, q_stride, k_stride, v_stride))
        return st;
    const int e = ssd::elem_size(dtype);
    if (!aligned(initial_state, 4) || !aligned(final_state, 4))
        return SSD_ERR_ALIGN;
    const int64_t tokens = batch * T, heads = tokens * Hv * 4;
    const size_t need = ssd_gated_delta_workspace_bytes(batch, T, Hk, Hv, Dk, Dv, dtype);
    const bool in_place = final_state == initial_state;
    const ssd::Range in[7] = {{q, ssd::span(tokens, Hk * Dk, q_stride, e)}, {k, ssd::span(tokens, Hk * Dk, k_stride, e)},
                              {v, ssd::span(tokens, Hv * Dv, v_stride, e)}, {g, heads}, {beta, heads},
                              {lengths, batch * 4}, {in_place ? nullptr : initial_state, z.states()}};
    const ssd::Range out[4] = {{o, tokens * Hv * Dv * e}, {final_state, z.states()},
                               {chunk_states, z.states() * z.chunks()}, {workspace, (int64_t)need}};
    const hipStream_t s = (hipStream_t)stream;
    if (z.empty()) {
        if (ssd::overlaps(out + 1, 1, in + 6, 1))
            return SSD_ERR_ALIAS;
        return launch_delta_copy(initial_state, final_state, batch * Hv * Dk * Dv, s);
    }
    if (!q || !k || !v || !g || !beta || !o)
        return SSD_ERR_NULL;
    if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(o, e) || !aligned(g, 4) || !aligned(beta, 4) ||
        !aligned(lengths, 4) || !aligned(chunk_states, 4))
        return SSD_ERR_ALIGN;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return SSD_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256))
        return SSD_ERR_ALIGN;
    // the state in place is its own input, and no other output may reach into it
    if (ssd::overlaps(out, 4, in, 7))
        return SSD_ERR_ALIAS;
    ssd::DeltaParams p = delta_params(z, q, q_stride, k, k_stride, v, v_stride, g, beta, scale, lengths);
    p.init = initial_state;
    p.o = o;
    p.final_state = final_state;
    p.states = chunk_states;
    if (delta_few(z))
        return dtype == SSD_BF16 ? launch_delta_few<ssd::kBF16>(p, s) : launch_delta_few<ssd::kF32>(p, s);
    const DeltaRange range = delta_range(z, dtype, false);
    char *at = (char *)workspace;
    if (dtype == SSD_BF16)
        return Dk <= 64 ? launch_delta<ssd::kBF16, 2>(p, range, at, s) : launch_delta<ssd::kBF16, 4>(p, range, at, s);
    return Dk <= 64 ? launch_delta<ssd::kF32, 2>(p, range, at, s) : launch_delta<ssd::kF32, 4>(p, range, at, s);
}

size_t ssd_gated_delta_backward_workspace_bytes(int64_t batch, int64_t T, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv,
                                                int dtype)
{
    const DeltaSizes z{batch, T, Hk, Hv, Dk, Dv};
    if (check_delta(z, dtype, 1.f) || z.empty())
        return 0;
    return delta_space(z).bytes() + delta_range(z, dtype, true).bytes();
}

int ssd_gated_delta_backward(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, const float *g, const float *beta, float scale, int dtype, int64_t batch,
                             int64_t T, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, const float *chunk_states,
                             const int32_t *lengths, const void *grad_o, const float *grad_final_state, void *grad_q,
                             void *grad_k, void *grad_v, float *grad_g, float *grad_beta, float *grad_initial_state,
                             void *workspace, size_t workspace_bytes, ssd_stream_t stream)
{
    const DeltaSizes z{batch, T, Hk, Hv, Dk, Dv};
    if (int st = check_delta(z, dtype, scale))
        return st;
    if (int st = check_delta_strides(z, q_stride, k_stride, v_stride))
        return st;
    const int e = ssd::elem_size(dtype);
    if (!aligned(grad_final_state, 4) || !aligned(grad_initial_state, 4))
        return SSD_ERR_ALIGN;
    const int64_t tokens = batch * T, heads = tokens * Hv * 4;
    const size_t need = ssd_gated_delta_backward_workspace_bytes(batch, T, Hk, Hv, Dk, Dv, dtype);
    const ssd::Range in[9] = {{q, ssd::span(tokens, Hk * Dk, q_stride, e)}, {k, ssd::span(tokens, Hk * Dk, k_stride, e)},
                              {v, ssd::span(tokens, Hv * Dv, v_stride, e)}, {g, heads}, {beta, heads},
                              {lengths, batch * 4}, {chunk_states, z.states() * z.chunks()},
                              {grad_o, tokens * Hv * Dv * e}, {grad_final_state, z.states()}};
    const ssd::Range out[7] = {{grad_q, tokens * Hk * Dk * e}, {grad_k, tokens * Hk * Dk * e},
                               {grad_v, tokens * Hv * Dv * e}, {grad_g, heads}, {grad_beta, heads},
                               {grad_initial_state, z.states()}, {workspace, (int64_t)need}};
    const hipStream_t s = (hipStream_t)stream;
    if (z.empty()) {
        if (ssd::overlaps(out + 5, 1, in + 8, 1))
            return SSD_ERR_ALIAS;
        return launch_delta_copy(grad_final_state, grad_initial_state, batch * Hv * Dk * Dv, s);
    }
    if (!q || !k || !v || !g || !beta || !chunk_states || !grad_o || !grad_q || !grad_k || !grad_v || !grad_g ||
        !grad_beta)
        return SSD_ERR_NULL;
    if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(grad_o, e) || !aligned(grad_q, e) ||
        !aligned(grad_k, e) || !aligned(grad_v, e) || !aligned(g, 4) || !aligned(beta, 4) || !aligned(lengths, 4) ||
        !aligned(chunk_states, 4) || !aligned(grad_g, 4) || !aligned(grad_beta, 4))
        return SSD_ERR_ALIGN;
    if (!workspace || workspace_bytes < need)
        return SSD_ERR_WORKSPACE;
    if (!aligned(workspace, 256))
        return SSD_ERR_ALIGN;
    if (ssd::overlaps(out, 7, in, 9))
        return SSD_ERR_ALIAS;
    ssd::DeltaParams p = delta_params(z, q, q_stride, k, k_stride, v, v_stride, g, beta, scale, lengths);
    p.chunk_states = chunk_states;
    p.go = grad_o;
    p.gfinal = grad_final_state;
    p.gq = grad_q;
    p.gk = grad_k;
    p.gv = grad_v;
    p.gg = grad_g;
    p.gbeta = grad_beta;
    p.ginit = grad_initial_state;
    const DeltaSpace space = delta_space(z);
    char *at = (char *)workspace;
    p.gs = (float *)at;
    p.gr = (float *)(at + space.gs);
    p.wq = (float *)(at + space.gs + space.gr);
    p.wk = (float *)(at + space.gs + space.gr + space.w);
    const DeltaRange range = delta_range(z, dtype, true);
    at += space.bytes();
    if (dtype == SSD_BF16)
        return Dk <= 64 ? launch_delta_bwd<ssd::kBF16, 2>(p, range, at, s) : launch_delta_bwd<ssd::kBF16, 4>(p, range, at, s);
    return Dk <= 64 ? launch_delta_bwd<ssd::kF32, 2>(p, range, at, s) : launch_delta_bwd<ssd::kF32, 4>(p, range, at, s);
}

}  // extern "C"
