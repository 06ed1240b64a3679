// ssd_block_binding.cpp -- the Python binding of the gated delta rule and of the norms around a block,
// made as that of the other operators (ssd_ops_binding.cpp).
#include "ssd_binding.h"

namespace {

#define SSD_OPERATORS(F)                                     \
    F(ssd_gated_delta_workspace_bytes) F(ssd_gated_delta)    \
    F(ssd_gated_delta_backward_workspace_bytes) F(ssd_gated_delta_backward) \
    F(ssd_gated_norm) F(ssd_gated_norm_backward_workspace_bytes) F(ssd_gated_norm_backward) \
    F(ssd_block_norm) F(ssd_block_norm_backward_workspace_bytes) F(ssd_block_norm_backward)
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
    if (!library.ssd_gated_delta)
        throw std::runtime_error("the binding has no library yet (complex_chunkwise_ssd_amd.block gives it one)");
    if (!t.device().is_cuda())
        bad("tensors must be on a GPU device, got " + t.device().str());
}

// Elements between the tokens of t (B, T, H, D): a token's heads and features dense, the tokens evenly
// spaced over the whole batch.
int64_t token_stride(const Tensor &t, const char *name)
{
    const int64_t B = t.size(0), T = t.size(1), H = t.size(2), D = t.size(3);
    if (t.is_neg())
        bad(std::string(name) + " must not be a lazily negated view");
    if (t.is_contiguous() || t.numel() == 0)
        return H * D;
    const int64_t step = T > 1 ? t.stride(1) : B > 1 ? t.stride(0) : H * D;
    if ((D > 1 && t.stride(3) != 1) || (H > 1 && t.stride(2) != D) || (B > 1 && t.stride(0) != T * step) || step < H * D)
        bad(std::string(name) + " must have dense heads and features and evenly spaced tokens, got strides " +
            text(t.strides()));
    return step;
}

struct Delta {
    at::Device dev;
    int dtype;
    at::ScalarType type;
    int64_t B, T, Hk, Hv, Dk, Dv, chunks, sq, sk, sv;
};
Delta delta_inputs(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &g, const Tensor &beta,
                   const optional<Tensor> &lengths)
{
    need_gpu(q);
    if (q.dim() != 4 || v.dim() != 4)
        bad("q must be a (B, T, Hk, Dk) and v a (B, T, Hv, Dv) tensor");
    Delta d{q.device(), dtype_of(q, "q"), q.scalar_type(), q.size(0), q.size(1), q.size(2), v.size(2),
            q.size(3), v.size(3), 0, 0, 0, 0};
    check_like(k, "k", d.type, q.sizes(), d.dev);
    check_like(v, "v", d.type, {d.B, d.T, d.Hv, d.Dv}, d.dev);
    d.sq = token_stride(q, "q");
    d.sk = token_stride(k, "k");
    d.sv = token_stride(v, "v");
    check(g, "g", at::kFloat, {d.B, d.T, d.Hv}, d.dev);
    check(beta, "beta", at::kFloat, {d.B, d.T, d.Hv}, d.dev);
    if (lengths)
        check(*lengths, "lengths", at::kInt, {d.B}, d.dev);
    d.chunks = (d.T + SSD_DELTA_CHUNK - 1) / SSD_DELTA_CHUNK;
    return d;
}

float delta_scale(const optional<double> &scale, const Delta &d)
{
    return scale ? (float)*scale : 1.f / std::sqrt((float)(d.Dk > 0 ? d.Dk : 1));
}

std::tuple<Tensor, optional<Tensor>, optional<Tensor>>
gated_delta(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &g, const Tensor &beta,
            const optional<double> &scale, const optional<Tensor> &init, const optional<Tensor> &lengths,
            bool want_final, bool want_states, const optional<Tensor> &o_, const optional<Tensor> &final_,
            const optional<Tensor> &states_, const optional<Tensor> &ws_)
{
    const Delta d = delta_inputs(q, k, v, g, beta, lengths);
    if (init)
        check(*init, "initial_state", at::kFloat, {d.B, d.Hv, d.Dk, d.Dv}, d.dev);
    const c10::DeviceGuard guard(d.dev);
    const Tensor o = output(o_, "o", d.type, v.sizes(), d.dev);
    const auto fin = maybe_output(final_, "final_state", at::kFloat, {d.B, d.Hv, d.Dk, d.Dv}, d.dev, want_final);
    const auto cs = maybe_output(states_, "chunk_states", at::kFloat, {d.B, d.chunks, d.Hv, d.Dk, d.Dv}, d.dev, want_states);
    const Workspace ws = workspace_of(
        ws_, library.ssd_gated_delta_workspace_bytes(d.B, d.T, d.Hk, d.Hv, d.Dk, d.Dv, d.dtype), d.dev);
    check_status(library.ssd_gated_delta(at_of(q), d.sq, at_of(k), d.sk, at_of(v), d.sv, at_of<float>(g),
                                         at_of<float>(beta), delta_scale(scale, d), d.dtype, d.B, d.T, d.Hk, d.Hv, d.Dk,
                                         d.Dv, at_of<float>(init), at_of<int32_t>(lengths), at_of(o), at_of<float>(fin),
                                         at_of<float>(cs), ws.at, ws.bytes, stream_of(d.dev)),
                 "ssd_gated_delta");
    return {o, fin, cs};
}

std::tuple<Tensor, Tensor, Tensor, Tensor, Tensor, optional<Tensor>>
gated_delta_backward(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &g, const Tensor &beta,
                     const Tensor &states, const Tensor &grad_o, const optional<Tensor> &grad_final,
                     const optional<double> &scale, const optional<Tensor> &lengths, bool want_init,
                     const optional<Tensor> &gq_, const optional<Tensor> &gk_, const optional<Tensor> &gv_,
                     const optional<Tensor> &gg_, const optional<Tensor> &gbeta_, const optional<Tensor> &ginit_,
                     const optional<Tensor> &ws_)
{
    const Delta d = delta_inputs(q, k, v, g, beta, lengths);
    const std::vector<int64_t> state = {d.B, d.Hv, d.Dk, d.Dv};
    check(states, "chunk_states", at::kFloat, {d.B, d.chunks, d.Hv, d.Dk, d.Dv}, d.dev);
    check(grad_o, "grad_o", d.type, v.sizes(), d.dev);
    if (grad_final)
        check(*grad_final, "grad_final_state", at::kFloat, state, d.dev);
    const c10::DeviceGuard guard(d.dev);
    const Tensor gq = output(gq_, "grad q", d.type, q.sizes(), d.dev);
    const Tensor gk = output(gk_, "grad k", d.type, q.sizes(), d.dev);
    const Tensor gv = output(gv_, "grad v", d.type, v.sizes(), d.dev);
    const Tensor gg = output(gg_, "grad g", at::kFloat, g.sizes(), d.dev);
    const Tensor gbeta = output(gbeta_, "grad beta", at::kFloat, g.sizes(), d.dev);
    const auto ginit = maybe_output(ginit_, "grad initial_state", at::kFloat, state, d.dev, want_init);
    const Workspace ws = workspace_of(
        ws_, library.ssd_gated_delta_backward_workspace_bytes(d.B, d.T, d.Hk, d.Hv, d.Dk, d.Dv, d.dtype), d.dev);
    check_status(library.ssd_gated_delta_backward(
                     at_of(q), d.sq, at_of(k), d.sk, at_of(v), d.sv, at_of<float>(g), at_of<float>(beta),
                     delta_scale(scale, d), d.dtype, d.B, d.T, d.Hk, d.Hv, d.Dk, d.Dv, at_of<float>(states),
                     at_of<int32_t>(lengths), at_of(grad_o), at_of<float>(grad_final), at_of(gq), at_of(gk), at_of(gv),
                     at_of<float>(gg), at_of<float>(gbeta), at_of<float>(ginit), ws.at, ws.bytes, stream_of(d.dev)),
                 "ssd_gated_delta_backward");
    return {gq, gk, gv, gg, gbeta, ginit};
}

struct Rows {
    at::Device dev;
    int dtype;
    at::ScalarType type;
    int64_t rows, F, stride;
};
Rows rows_input(const Tensor &x, const char *name)
{
    need_gpu(x);
    if (x.dim() < 1)
        bad(std::string(name) + " must have a last dimension");
    return {x.device(), dtype_of(x, name), x.scalar_type(), rows_of(x), x.size(-1), row_stride(x, name)};
}

using MaybeTensor = optional<Tensor>;

std::tuple<MaybeTensor, MaybeTensor, MaybeTensor, MaybeTensor>
gated_norm(const Tensor &x, const Tensor &gate, const Tensor &weight, double eps, bool want_y, bool fp8, bool want_rstd,
           const MaybeTensor &y_, const MaybeTensor &q_, const MaybeTensor &scale_, const MaybeTensor &rstd_)
{
    const Rows r = rows_input(x, "x");
    const int64_t sg = strided(gate, "gate", r.type, x.sizes(), r.dev);
    if (weight.dim() != 1 || weight.size(0) < 1 || r.F % weight.size(0) != 0)
        bad("weight must be a (D,) tensor, D a divisor of x's last dimension, got " + text(weight.sizes()));
    const int64_t D = weight.size(0);
    check(weight, "weight", at::kFloat, {D}, r.dev);
    const c10::DeviceGuard guard(r.dev);
    const auto y = maybe_output(y_, "y", r.type, x.sizes(), r.dev, want_y);
    const auto q = maybe_output(q_, "q", at::kFloat8_e4m3fn, x.sizes(), r.dev, fp8);
    const auto scale = maybe_output(scale_, "scale", at::kFloat, {(r.F + 127) / 128, r.rows}, r.dev, q.has_value());
    const auto rstd = maybe_output(rstd_, "rstd", at::kFloat, {r.rows, r.F / D}, r.dev, want_rstd);
    check_status(library.ssd_gated_norm(at_of(x), r.stride, at_of(gate), sg, at_of<float>(weight), r.dtype, r.rows, r.F,
                                        D, (float)eps, at_of(y), at_of<uint8_t>(q), at_of<float>(scale),
                                        at_of<float>(rstd), stream_of(r.dev)),
                 "ssd_gated_norm");
    return {y, q, scale, rstd};
}

std::tuple<Tensor, Tensor, Tensor> gated_norm_backward(const Tensor &x, const Tensor &gate, const Tensor &weight,
                                                       const Tensor &rstd, const Tensor &grad_y, const MaybeTensor &gx_,
                                                       const MaybeTensor &gz_, const MaybeTensor &gw_,
                                                       const MaybeTensor &ws_)
{
    const Rows r = rows_input(x, "x");
    const int64_t sz = strided(gate, "gate", r.type, x.sizes(), r.dev);
    const int64_t sg = strided(grad_y, "grad_y", r.type, x.sizes(), r.dev);
    if (weight.dim() != 1 || weight.size(0) < 1 || r.F % weight.size(0) != 0)
        bad("weight must be a (D,) tensor, D a divisor of x's last dimension, got " + text(weight.sizes()));
    const int64_t D = weight.size(0);
    check(weight, "weight", at::kFloat, {D}, r.dev);
    check(rstd, "rstd", at::kFloat, {r.rows, r.F / D}, r.dev);
    const c10::DeviceGuard guard(r.dev);
    const Tensor gx = output(gx_, "grad_x", r.type, x.sizes(), r.dev);
    const Tensor gz = output(gz_, "grad_gate", r.type, x.sizes(), r.dev);
    const Tensor gw = output(gw_, "grad_weight", at::kFloat, {D}, r.dev);
    const Workspace ws = workspace_of(ws_, library.ssd_gated_norm_backward_workspace_bytes(r.rows, r.F, D), r.dev);
    check_status(library.ssd_gated_norm_backward(at_of(x), r.stride, at_of(gate), sz, at_of<float>(weight),
                                                 at_of<float>(rstd), at_of(grad_y), sg, r.dtype, r.rows, r.F, D,
                                                 at_of(gx), at_of(gz), at_of<float>(gw), ws.at, ws.bytes,
                                                 stream_of(r.dev)),
                 "ssd_gated_norm_backward");
    return {gx, gz, gw};
}

std::tuple<MaybeTensor, Tensor, MaybeTensor, MaybeTensor, MaybeTensor, MaybeTensor>
block_norm(const Tensor &x, const Tensor &residual, const Tensor &post, const Tensor &pre, double alpha, double eps,
           bool want_y, bool fp8, bool want_rstd, const MaybeTensor &y_, const MaybeTensor &residual_out_,
           const MaybeTensor &q_, const MaybeTensor &scale_, const MaybeTensor &post_rstd_,
           const MaybeTensor &pre_rstd_)
{
    const Rows r = rows_input(x, "x");
    const int64_t sr = strided(residual, "residual", r.type, x.sizes(), r.dev);
    check(post, "post_weight", at::kFloat, {r.F}, r.dev);
    check(pre, "pre_weight", at::kFloat, {r.F}, r.dev);
    const c10::DeviceGuard guard(r.dev);
    const auto y = maybe_output(y_, "y", r.type, x.sizes(), r.dev, want_y);
    const Tensor s = output(residual_out_, "residual_out", r.type, x.sizes(), r.dev);
    const auto q = maybe_output(q_, "q", at::kFloat8_e4m3fn, x.sizes(), r.dev, fp8);
    const auto scale = maybe_output(scale_, "scale", at::kFloat, {(r.F + 127) / 128, r.rows}, r.dev, q.has_value());
    const auto rstd1 = maybe_output(post_rstd_, "post_rstd", at::kFloat, {r.rows}, r.dev, want_rstd);
    const auto rstd2 = maybe_output(pre_rstd_, "pre_rstd", at::kFloat, {r.rows}, r.dev, want_rstd);
    check_status(library.ssd_block_norm(at_of(x), r.stride, at_of(residual), sr, at_of<float>(post), at_of<float>(pre),
                                        (float)alpha, r.dtype, r.rows, r.F, (float)eps, at_of(y), at_of(s),
                                        at_of<uint8_t>(q), at_of<float>(scale), at_of<float>(rstd1),
                                        at_of<float>(rstd2), stream_of(r.dev)),
                 "ssd_block_norm");
    return {y, s, q, scale, rstd1, rstd2};
}

std::tuple<Tensor, Tensor, Tensor, Tensor>
block_norm_backward(const Tensor &x, const Tensor &s, const Tensor &post, const Tensor &pre, const Tensor &post_rstd,
                    const Tensor &pre_rstd, const Tensor &grad_y, const MaybeTensor &grad_residual, double alpha,
                    const MaybeTensor &gx_, const MaybeTensor &gr_, const MaybeTensor &gpost_, const MaybeTensor &gpre_,
                    const MaybeTensor &ws_)
{
    const Rows r = rows_input(x, "x");
    const int64_t ss = strided(s, "s", r.type, x.sizes(), r.dev);
    const int64_t sg = strided(grad_y, "grad_y", r.type, x.sizes(), r.dev);
    const int64_t sr = grad_residual ? strided(*grad_residual, "grad_residual", r.type, x.sizes(), r.dev) : 0;
    check(post, "post_weight", at::kFloat, {r.F}, r.dev);
    check(pre, "pre_weight", at::kFloat, {r.F}, r.dev);
    check(post_rstd, "post_rstd", at::kFloat, {r.rows}, r.dev);
    check(pre_rstd, "pre_rstd", at::kFloat, {r.rows}, r.dev);
    const c10::DeviceGuard guard(r.dev);
    const Tensor gx = output(gx_, "grad_x", r.type, x.sizes(), r.dev);
    const Tensor gr = output(gr_, "grad_residual_in", r.type, x.sizes(), r.dev);
    const Tensor gpost = output(gpost_, "grad_post_weight", at::kFloat, {r.F}, r.dev);
    const Tensor gpre = output(gpre_, "grad_pre_weight", at::kFloat, {r.F}, r.dev);
    const Workspace ws = workspace_of(ws_, library.ssd_block_norm_backward_workspace_bytes(r.rows, r.F), r.dev);
    check_status(library.ssd_block_norm_backward(at_of(x), r.stride, at_of(s), ss, at_of<float>(post), at_of<float>(pre),
                                                 at_of<float>(post_rstd), at_of<float>(pre_rstd), (float)alpha,
                                                 at_of(grad_y), sg, at_of(grad_residual), sr, r.dtype, r.rows, r.F,
                                                 at_of(gx), at_of(gr), at_of<float>(gpost), at_of<float>(gpre), ws.at,
                                                 ws.bytes, stream_of(r.dev)),
                 "ssd_block_norm_backward");
    return {gx, gr, gpost, gpre};
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m)
{
    m.def("bind", &bind);
    m.def("bound", &bound);
    m.def("token_stride", [](const Tensor &t) { return token_stride(t, "t"); });
    m.def("gated_delta", &gated_delta);
    m.def("gated_delta_backward", &gated_delta_backward);
    m.def("gated_norm", &gated_norm);
    m.def("gated_norm_backward", &gated_norm_backward);
    m.def("block_norm", &block_norm);
    m.def("block_norm_backward", &block_norm_backward);
}
