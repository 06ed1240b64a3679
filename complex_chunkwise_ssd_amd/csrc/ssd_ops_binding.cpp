// ssd_ops_binding.cpp -- the Python binding of the operators around the scan: checks of the
// tensors, outputs and workspaces from torch's allocator, and one call of the C ABI on the
// current stream of the tensors' device. Compiled, because at the sizes of generation the same
// steps in Python took longer than the kernels (12 us a call against 3 us).
#include "ssd_binding.h"

namespace {

// The entry points of the library that the package loaded, by address: the loader would take the
// first library of that name in the process, whichever file it came from.
#define SSD_OPERATORS(F)                                                              \
    F(ssd_gated_scan_workspace_bytes) F(ssd_gated_scan)                               \
    F(ssd_gated_scan_backward_workspace_bytes) F(ssd_gated_scan_backward)             \
    F(ssd_rms_norm) F(ssd_rms_norm_backward_workspace_bytes) F(ssd_rms_norm_backward) \
    F(ssd_fp8_quantise) F(ssd_fp8_matmul_workspace_bytes) F(ssd_fp8_matmul)
struct Library {
#define F(name) decltype(&::name) name = nullptr;
    SSD_OPERATORS(F)
#undef F
} library;

void bind(const std::function<uintptr_t(const char *)> &address)
{
    Library found;
#define F(name) found.name = (decltype(found.name))address(#name);
    SSD_OPERATORS(F)
#undef F
    library = found;
}

std::map<std::string, uintptr_t> bound()
{
    std::map<std::string, uintptr_t> r;
#define F(name) r[#name] = (uintptr_t)library.name;
    SSD_OPERATORS(F)
#undef F
    return r;
}

void need_gpu(const Tensor &t)
{
    if (!library.ssd_fp8_matmul)
        throw std::runtime_error("the binding has no library yet (complex_chunkwise_ssd_amd.ops gives it one)");
    if (!t.device().is_cuda())
        bad("tensors must be on a GPU device, got " + t.device().str());
}

struct Gated {
    at::Device dev;
    int dtype;
    int64_t B, T, C, sx, si, sr, chunks;
    at::ScalarType type;
};
Gated gated_inputs(const Tensor &x, const Tensor &gi, const Tensor &gr, const Tensor &lam,
                   const optional<Tensor> &lengths)
{
    need_gpu(x);
    if (x.dim() != 3)
        bad("x must be a (B, T, C) tensor");
    Gated g{x.device(), dtype_of(x, "x"), x.size(0), x.size(1), x.size(2), 0, 0, 0, 0, x.scalar_type()};
    g.sx = row_stride(x, "x");
    g.si = strided(gi, "input_gate", g.type, x.sizes(), g.dev);
    g.sr = strided(gr, "decay_gate", g.type, x.sizes(), g.dev);
    check(lam, "lam", at::kFloat, {g.C}, g.dev);
    if (lengths)
        check(*lengths, "lengths", at::kInt, {g.B}, g.dev);
    g.chunks = (g.T + SSD_GATED_CHUNK - 1) / SSD_GATED_CHUNK;
    return g;
}

std::tuple<Tensor, optional<Tensor>, optional<Tensor>>
gated_scan(const Tensor &x, const Tensor &gi, const Tensor &gr, const Tensor &lam, double k,
           const optional<Tensor> &init, const optional<Tensor> &lengths, bool want_final,
           bool want_states, const optional<Tensor> &h_, const optional<Tensor> &final_,
           const optional<Tensor> &states_, const optional<Tensor> &ws_)
{
    const Gated g = gated_inputs(x, gi, gr, lam, lengths);
    if (init)
        check(*init, "initial_state", at::kFloat, {g.B, g.C}, g.dev);
    const c10::DeviceGuard guard(g.dev);
    const Tensor h = output(h_, "h", g.type, x.sizes(), g.dev);
    const auto fin = maybe_output(final_, "final_state", at::kFloat, {g.B, g.C}, g.dev, want_final);
    const auto cs = maybe_output(states_, "chunk_states", at::kFloat, {g.B, g.chunks, g.C}, g.dev, want_states);
    const Workspace ws = workspace_of(ws_, library.ssd_gated_scan_workspace_bytes(g.B, g.T, g.C, g.dtype), g.dev);
    check_status(library.ssd_gated_scan(at_of(x), g.sx, at_of(gi), g.si, at_of(gr), g.sr, at_of<float>(lam), (float)k,
                                g.dtype, g.B, g.T, g.C, at_of<float>(init), at_of<int32_t>(lengths), at_of(h),
                                at_of<float>(fin), at_of<float>(cs), ws.at, ws.bytes, stream_of(g.dev)),
                 "ssd_gated_scan");
    return {h, fin, cs};
}

std::tuple<Tensor, Tensor, Tensor, Tensor, optional<Tensor>>
gated_scan_backward(const Tensor &x, const Tensor &gi, const Tensor &gr, const Tensor &lam,
                    const Tensor &states, const Tensor &grad_h, const optional<Tensor> &grad_final,
                    double k, const optional<Tensor> &lengths, bool want_init,
                    const optional<Tensor> &gx_, const optional<Tensor> &ggi_, const optional<Tensor> &ggr_,
                    const optional<Tensor> &glam_, const optional<Tensor> &ginit_,
                    const optional<Tensor> &ws_)
{
    const Gated g = gated_inputs(x, gi, gr, lam, lengths);
    check(states, "chunk_states", at::kFloat, {g.B, g.chunks, g.C}, g.dev);
    check(grad_h, "grad_h", g.type, x.sizes(), g.dev);
    if (grad_final)
        check(*grad_final, "grad_final_state", at::kFloat, {g.B, g.C}, g.dev);
    const c10::DeviceGuard guard(g.dev);
    const Tensor gx = output(gx_, "grad x", g.type, x.sizes(), g.dev);
    const Tensor ggi = output(ggi_, "grad input_gate", g.type, x.sizes(), g.dev);
    const Tensor ggr = output(ggr_, "grad decay_gate", g.type, x.sizes(), g.dev);
    const Tensor glam = output(glam_, "grad lam", at::kFloat, {g.C}, g.dev);
    const auto ginit = maybe_output(ginit_, "grad initial_state", at::kFloat, {g.B, g.C}, g.dev, want_init);
    const Workspace ws =
        workspace_of(ws_, library.ssd_gated_scan_backward_workspace_bytes(g.B, g.T, g.C, g.dtype), g.dev);
    check_status(library.ssd_gated_scan_backward(at_of(x), g.sx, at_of(gi), g.si, at_of(gr), g.sr, at_of<float>(lam),
                                         (float)k, g.dtype, g.B, g.T, g.C, at_of<float>(states),
                                         at_of<int32_t>(lengths), at_of(grad_h), at_of<float>(grad_final),
                                         at_of(gx), at_of(ggi), at_of(ggr), at_of<float>(glam),
                                         at_of<float>(ginit), ws.at, ws.bytes, stream_of(g.dev)),
                 "ssd_gated_scan_backward");
    return {gx, ggi, ggr, glam, ginit};
}

std::tuple<optional<Tensor>, optional<Tensor>, optional<Tensor>, optional<Tensor>, optional<Tensor>>
rms_norm(const Tensor &x, const Tensor &weight, const optional<Tensor> &residual, double eps, bool want_y,
         bool fp8, bool want_rstd, const optional<Tensor> &y_, const optional<Tensor> &residual_out_,
         const optional<Tensor> &q_, const optional<Tensor> &scale_, const optional<Tensor> &rstd_)
{
    need_gpu(x);
    const int dtype = dtype_of(x, "x");
    if (x.dim() < 1)
        bad("x must have a last dimension");
    const at::Device dev = x.device();
    const at::ScalarType type = x.scalar_type();
    const int64_t F = x.size(-1), rows = rows_of(x);
    const int64_t sx = row_stride(x, "x");
    const int64_t sr = residual ? strided(*residual, "residual", type, x.sizes(), dev) : 0;
    check(weight, "weight", at::kFloat, {F}, dev);
    if (!residual && residual_out_)
        bad("residual_out without a residual");
    const c10::DeviceGuard guard(dev);
    const auto y = maybe_output(y_, "y", type, x.sizes(), dev, want_y);
    const auto s = maybe_output(residual_out_, "residual_out", type, x.sizes(), dev, residual.has_value());
    const auto q = maybe_output(q_, "q", at::kFloat8_e4m3fn, x.sizes(), dev, fp8);
    const auto scale = maybe_output(scale_, "scale", at::kFloat, {(F + 127) / 128, rows}, dev, q.has_value());
    const auto rstd = maybe_output(rstd_, "rstd", at::kFloat, {rows}, dev, want_rstd);
    check_status(library.ssd_rms_norm(at_of(x), sx, at_of(residual), sr, at_of<float>(weight), dtype, rows, F,
                              (float)eps, at_of(y), at_of(s), at_of<uint8_t>(q), at_of<float>(scale),
                              at_of<float>(rstd), stream_of(dev)),
                 "ssd_rms_norm");
    return {y, s, q, scale, rstd};
}

std::tuple<Tensor, Tensor> rms_norm_backward(const Tensor &s, const Tensor &weight, const Tensor &rstd,
                                             const Tensor &grad_y, const optional<Tensor> &grad_residual,
                                             const optional<Tensor> &gx_, const optional<Tensor> &gw_,
                                             const optional<Tensor> &ws_)
{
    need_gpu(s);
    const int dtype = dtype_of(s, "s");
    if (s.dim() < 1)
        bad("s must have a last dimension");
    const at::Device dev = s.device();
    const at::ScalarType type = s.scalar_type();
    const int64_t F = s.size(-1), rows = rows_of(s);
    const int64_t ss = row_stride(s, "s");
    const int64_t sg = strided(grad_y, "grad_y", type, s.sizes(), dev);
    const int64_t sr = grad_residual ? strided(*grad_residual, "grad_residual", type, s.sizes(), dev) : 0;
    check(weight, "weight", at::kFloat, {F}, dev);
    check(rstd, "rstd", at::kFloat, {rows}, dev);
    const c10::DeviceGuard guard(dev);
    const Tensor gx = output(gx_, "grad_x", type, s.sizes(), dev);
    const Tensor gw = output(gw_, "grad_weight", at::kFloat, {F}, dev);
    const Workspace ws = workspace_of(ws_, library.ssd_rms_norm_backward_workspace_bytes(rows, F), dev);
    check_status(library.ssd_rms_norm_backward(at_of(s), ss, at_of<float>(weight), at_of<float>(rstd), at_of(grad_y),
                                       sg, at_of(grad_residual), sr, dtype, rows, F, at_of(gx),
                                       at_of<float>(gw), ws.at, ws.bytes, stream_of(dev)),
                 "ssd_rms_norm_backward");
    return {gx, gw};
}

std::tuple<Tensor, Tensor> fp8_quantise(const Tensor &x, int64_t block_rows, bool transpose,
                                        const optional<Tensor> &q_, const optional<Tensor> &scale_)
{
    need_gpu(x);
    const int dtype = dtype_of(x, "x");
    if (x.dim() < 1)
        bad("x must have a last dimension");
    const at::Device dev = x.device();
    const int64_t cols = x.size(-1), rows = rows_of(x);
    const int64_t sx = row_stride(x, "x");
    const int64_t R = transpose ? cols : rows, K = transpose ? rows : cols;
    std::vector<int64_t> shape = transpose ? std::vector<int64_t>{cols, rows} : x.sizes().vec();
    const c10::DeviceGuard guard(dev);
    Tensor q;
    if (q_) {
        q = *q_;
    } else {  // rows that start on 16 bytes
        shape.back() = (K + 15) / 16 * 16;
        q = fresh(shape, at::kFloat8_e4m3fn, dev);
        if (shape.back() != K)
            q = q.narrow(-1, 0, K);
        shape.back() = K;
    }
    const int64_t sq = strided(q, "q", at::kFloat8_e4m3fn, shape, dev);
    const Tensor scale = block_rows == 1
                             ? output(scale_, "scale", at::kFloat, {(K + 127) / 128, R}, dev)
                             : output(scale_, "scale", at::kFloat, {(R + 127) / 128, (K + 127) / 128}, dev);
    check_status(library.ssd_fp8_quantise(at_of(x), sx, dtype, rows, cols, block_rows, transpose, at_of<uint8_t>(q), sq,
                                  at_of<float>(scale), stream_of(dev)),
                 "ssd_fp8_quantise");
    return {q, scale};
}

Tensor fp8_matmul(const Tensor &a, const Tensor &a_scale, const Tensor &b, const Tensor &b_scale,
                  int64_t block_rows, at::ScalarType out_dtype, const optional<Tensor> &out_,
                  const optional<Tensor> &ws_)
{
    need_gpu(a);
    if (out_dtype != at::kFloat && out_dtype != at::kBFloat16)
        bad(std::string("out_dtype must be float32 or bfloat16, got ") + at::toString(out_dtype));
    if (a.dim() < 1 || b.dim() != 2)
        bad("a must be (..., K) and b (N, K)");
    const at::Device dev = a.device();
    const int64_t K = a.size(-1), N = b.size(0), M = rows_of(a), kb = (K + 127) / 128;
    const int64_t sa = strided(a, "a", at::kFloat8_e4m3fn, a.sizes(), dev);
    const int64_t sb = strided(b, "b", at::kFloat8_e4m3fn, {N, K}, dev);
    check(a_scale, "a_scale", at::kFloat, {kb, M}, dev);
    if (block_rows == 1)
        check(b_scale, "b_scale", at::kFloat, {kb, N}, dev);
    else
        check(b_scale, "b_scale", at::kFloat, {(N + 127) / 128, kb}, dev);
    std::vector<int64_t> shape = a.sizes().vec();
    shape.back() = N;
    const c10::DeviceGuard guard(dev);
    const Tensor out = out_ ? *out_ : fresh(shape, out_dtype, dev);
    const int64_t so = strided(out, "out", out_dtype, shape, dev);
    const int dt = out_dtype == at::kBFloat16 ? SSD_BF16 : SSD_F32;
    const uintptr_t bits = (uintptr_t)a.data_ptr() | (uintptr_t)b.data_ptr() | (uintptr_t)sa | (uintptr_t)sb;
    const int on16 = bits % 16 == 0 && sa < (1 << 24) && sb < (1 << 24);
    const Workspace ws = workspace_of(ws_, library.ssd_fp8_matmul_workspace_bytes(M, N, K, block_rows, dt, on16), dev);
    check_status(library.ssd_fp8_matmul(at_of<uint8_t>(a), sa, at_of<float>(a_scale), at_of<uint8_t>(b), sb,
                                at_of<float>(b_scale), M, N, K, block_rows, dt, at_of(out), so, ws.at, ws.bytes,
                                stream_of(dev)),
                 "ssd_fp8_matmul");
    return out;
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m)
{
    m.def("bind", &bind);
    m.def("bound", &bound);
    m.def("row_stride", [](const Tensor &t) { return row_stride(t, "t"); });
    m.def("gated_scan", &gated_scan);
    m.def("gated_scan_backward", &gated_scan_backward);
    m.def("rms_norm", &rms_norm);
    m.def("rms_norm_backward", &rms_norm_backward);
    m.def("fp8_quantise", &fp8_quantise);
    m.def("fp8_matmul", [](const Tensor &a, const Tensor &a_scale, const Tensor &b, const Tensor &b_scale,
                           int64_t block_rows, const py::object &out_dtype, const optional<Tensor> &out,
                           const optional<Tensor> &ws) {
        return fp8_matmul(a, a_scale, b, b_scale, block_rows,
                          torch::python::detail::py_object_to_dtype(out_dtype), out, ws);
    });
}
