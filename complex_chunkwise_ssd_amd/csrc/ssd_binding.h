// ssd_binding.h -- what the parts of the Python binding share: checks of tensors, outputs and workspaces
// from torch's allocator, the current stream, and the error of a rejected call.
#pragma once

#include <torch/extension.h>

#include <pybind11/functional.h>
#include <pybind11/stl.h>

#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>

#include <functional>
#include <map>
#include <optional>
#include <string>
#include <tuple>

#include "ssd.h"

namespace {

using at::Tensor;
using std::optional;
namespace py = pybind11;

[[noreturn]] inline void bad(const std::string &what) { throw py::value_error(what); }

inline std::string text(at::IntArrayRef s)
{
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i)
        r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

inline int dtype_of(const Tensor &t, const char *name)
{
    if (t.scalar_type() == at::kBFloat16)
        return SSD_BF16;
    if (t.scalar_type() != at::kFloat)
        bad(std::string(name) + " must be float32 or bfloat16, got " + at::toString(t.scalar_type()));
    return SSD_F32;
}

inline void check_like(const Tensor &t, const char *name, at::ScalarType dtype, at::IntArrayRef shape,
                at::Device dev)
{
    if (t.scalar_type() != dtype || t.device() != dev || t.sizes() != shape)
        bad(std::string(name) + " must be " + at::toString(dtype) + " of shape " + text(shape) + " on " +
            dev.str() + ", got " + at::toString(t.scalar_type()) + " of shape " + text(t.sizes()) +
            " on " + t.device().str());
    if (t.is_neg())
        bad(std::string(name) + " must not be a lazily negated view");
}

// A dense tensor of this type, shape and device.
inline void check(const Tensor &t, const char *name, at::ScalarType dtype, at::IntArrayRef shape, at::Device dev)
{
    check_like(t, name, dtype, shape, dev);
    if (!t.is_contiguous())
        bad(std::string(name) + " must be contiguous");
}

// Elements between the rows of t (..., F): its last dimension dense, the rows evenly spaced (a
// contiguous tensor, or a column range of one).
inline int64_t row_stride(const Tensor &t, const char *name)
{
    const int64_t F = t.size(-1);
    if (t.is_neg())
        bad(std::string(name) + " must not be a lazily negated view");
    if (t.is_contiguous())
        return F;
    int64_t want = -1, step = 0;  // between neighbouring rows; that the next dimension out has to have
    for (int64_t d = t.dim() - 2; d >= 0 && want != 0; --d) {
        if (t.size(d) == 1)
            continue;
        if (want < 0)
            want = step = t.stride(d);
        if (t.stride(d) != step)
            want = 0;
        step *= t.size(d);
    }
    if (F > 1 && t.stride(-1) != 1)
        want = 0;
    if (want < 0)
        want = F;
    if (want < F)
        bad(std::string(name) + " must have a dense last dimension and evenly spaced rows, got strides " +
            text(t.strides()));
    return want;
}

inline int64_t strided(const Tensor &t, const char *name, at::ScalarType dtype, at::IntArrayRef shape, at::Device dev)
{
    check_like(t, name, dtype, shape, dev);
    return row_stride(t, name);
}

inline Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, at::Device dev)
{
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(dev));
}

// The output that was passed in, checked, or a new one.
inline Tensor output(const optional<Tensor> &given, const char *name, at::ScalarType dtype, at::IntArrayRef shape,
              at::Device dev)
{
    if (!given)
        return fresh(shape, dtype, dev);
    check(*given, name, dtype, shape, dev);
    return *given;
}
inline optional<Tensor> maybe_output(const optional<Tensor> &given, const char *name, at::ScalarType dtype,
                              at::IntArrayRef shape, at::Device dev, bool want)
{
    if (!given && !want)
        return std::nullopt;
    return output(given, name, dtype, shape, dev);
}

struct Workspace {
    Tensor held;
    void *at = nullptr;
    size_t bytes = 0;
};
inline Workspace workspace_of(const optional<Tensor> &given, size_t need, at::Device dev)
{
    Workspace w;
    if (given) {
        if (given->device() != dev || !given->is_contiguous())
            bad("workspace must be a contiguous tensor on " + dev.str());
        w.held = *given;
        w.bytes = given->nbytes();
    } else if (need > 0) {
        w.held = fresh({(int64_t)need}, at::kByte, dev);
        w.bytes = need;
    }
    w.at = w.held.defined() ? w.held.data_ptr() : nullptr;
    return w;
}

template <class T = void>
T *at_of(const optional<Tensor> &t) { return t ? (T *)t->data_ptr() : nullptr; }
template <class T = void>
T *at_of(const Tensor &t) { return (T *)t.data_ptr(); }

inline ssd_stream_t stream_of(at::Device dev)
{
    return (ssd_stream_t)c10::hip::getCurrentHIPStream(dev.index()).stream();
}

inline void check_status(int status, const char *where)
{
    if (status == SSD_OK)
        return;
    const py::object error = py::module_::import("complex_chunkwise_ssd_amd").attr("SSDError");
    PyErr_SetObject(error.ptr(), error(status, where).ptr());
    throw py::error_already_set();
}

inline int64_t rows_of(const Tensor &t)
{
    int64_t n = 1;
    for (int64_t d = 0; d + 1 < t.dim(); ++d)
        n *= t.size(d);
    return n;
}

}  // namespace
