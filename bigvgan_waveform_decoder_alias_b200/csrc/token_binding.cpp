// Tensor marshalling of the token operators (argument checks, new outputs, the
// current stream) in C++: these are called once a layer and token, where a
// marshalling in Python took longer than the kernels.  The computation is
// libbv's, reached through the addresses that bind() is given, so this module
// links no CUDA code of its own.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include "bv.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using Opt = std::optional<Tensor>;

struct Library {
  decltype(&bv_last_error) last_error = nullptr;
  decltype(&bv_rms_norm) rms_norm = nullptr;
  decltype(&bv_rms_norm_int8) rms_norm_int8 = nullptr;
  decltype(&bv_quantize_rows) quantize_rows = nullptr;
  decltype(&bv_int8_matmul) int8_matmul = nullptr;
  PyObject *error = nullptr;  // BVError(status, message); kept for the process
} lib;

[[noreturn]] void raise(int status, const std::string &message) {
  py::object e = py::reinterpret_borrow<py::object>(lib.error)(status, message);
  PyErr_SetObject(lib.error, e.ptr());
  throw py::error_already_set();
}
void check(bv_status st) {
  if (st != BV_OK) raise(st, lib.last_error());
}

// (No stream formatting here: a build compiler newer than the libstdc++ that the
// process has loaded can disagree with it on streams.)
std::string text(at::IntArrayRef sizes) {
  std::string s = "[";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
  return s + "]";
}

int dtype_of(at::ScalarType t, const char *name) {
  switch (t) {
    case at::kFloat: return BV_F32;
    case at::kBFloat16: return BV_BF16;
    case at::kHalf: return BV_F16;
    default: raise(BV_ERR_ARG, std::string(name) + " of type " + c10::toString(t));
  }
}

// A tensor as [rows, cols]: consecutive elements within a row, one stride
// between rows.
struct Rows {
  void *p;
  int64_t stride, rows, cols;
};
Rows rows_of(const Tensor &t, const char *name) {
  if (t.dim() == 0) raise(BV_ERR_SHAPE, std::string(name) + " needs a last dimension");
  Rows r;
  r.cols = t.size(-1);
  r.rows = 1;
  for (int64_t i = 0; i + 1 < t.dim(); ++i) r.rows *= t.size(i);
  r.p = t.data_ptr();
  r.stride = r.cols;
  if (t.is_contiguous()) return r;
  if (t.stride(-1) != 1 && r.cols > 1)
    raise(BV_ERR_ARG, std::string("the rows of ") + name + " must be contiguous");
  // the leading dimensions have to advance as one
  int64_t step = -1, next = 0;
  for (int64_t i = t.dim() - 2; i >= 0; --i) {
    if (t.size(i) == 1) continue;
    if (step < 0) step = t.stride(i);
    else if (t.stride(i) != next)
      raise(BV_ERR_ARG, std::string(name) + " has no single stride between its rows");
    next = t.stride(i) * t.size(i);
  }
  if (step >= 0 && r.rows > 1) r.stride = step;
  return r;
}

void on_device(const Tensor &t, const Tensor &x, const char *name) {
  if (t.device() != x.device())
    raise(BV_ERR_ARG, std::string(name) + " is on " + t.device().str() + ", not on " + x.device().str());
}
const float *vec(const Tensor &t, int64_t n, const Tensor &x, const char *name) {
  on_device(t, x, name);
  if (t.scalar_type() != at::kFloat || t.numel() != n || !t.is_contiguous())
    raise(BV_ERR_ARG, std::string(name) + " must be a contiguous float32 tensor of " +
                          std::to_string(n) + " values");
  return t.data_ptr<float>();
}
void shaped(const Tensor &t, at::IntArrayRef sizes, at::ScalarType dtype, const Tensor &x,
            const char *name) {
  if (t.sizes() != sizes || t.scalar_type() != dtype) {
    raise(BV_ERR_SHAPE, std::string(name) + " must be " + c10::toString(dtype) + " of shape " +
                            text(sizes));
  }
  on_device(t, x, name);
}

// Entered by every call: tensors on a GPU, that GPU current.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  void *stream;
  explicit On(const Tensor &x) {
    if (!x.is_cuda()) raise(BV_ERR_ARG, "tensors must be CUDA tensors");
    guard.set_device(x.device());
    stream = c10::cuda::getCurrentCUDAStream(x.device().index()).stream();
  }
};

Tensor new_rows(const Tensor &x, at::ScalarType dtype) {
  return at::empty(x.sizes(), x.options().dtype(dtype));
}

// int8 of x's shape whose rows start on 16 bytes, as bv_int8_matmul reads them
// fastest: where cols is no multiple of 16, the cols of each padded row (the
// padding holds nothing).
Tensor int8_rows(const Tensor &x) {
  if (x.dim() == 0) raise(BV_ERR_SHAPE, "x needs a last dimension");
  const int64_t cols = x.size(-1), padded = (cols + 15) / 16 * 16;
  if (cols == padded) return new_rows(x, at::kChar);
  auto sizes = x.sizes().vec();
  sizes.back() = padded;
  return at::empty(sizes, x.options().dtype(at::kChar)).narrow(-1, 0, cols);
}

struct NormIn {
  Rows x, r{nullptr, 0, 0, 0}, h{nullptr, 0, 0, 0};
  const void *gain = nullptr;
  int dtype, gain_dtype = 0;
};
// The operands that both norms share; h is made here where a residual asks
// for it.
NormIn norm_in(const Tensor &x, const Opt &gain, const Opt &residual, Opt &h) {
  NormIn a;
  a.dtype = dtype_of(x.scalar_type(), "x");
  a.x = rows_of(x, "x");
  if (residual) {
    shaped(*residual, x.sizes(), x.scalar_type(), x, "residual");
    a.r = rows_of(*residual, "residual");
    if (!h) h = new_rows(x, x.scalar_type());
  }
  if (h) {
    shaped(*h, x.sizes(), x.scalar_type(), x, "h");
    a.h = rows_of(*h, "h");
  }
  if (gain) {
    a.gain_dtype = dtype_of(gain->scalar_type(), "gain");
    on_device(*gain, x, "gain");
    if (gain->numel() != a.x.cols || !gain->is_contiguous())
      raise(BV_ERR_ARG, "gain must be " + std::to_string(a.x.cols) + " contiguous values");
    a.gain = gain->data_ptr();
  }
  if (a.x.cols > INT32_MAX) raise(BV_ERR_SHAPE, "rows of 2^31 values and more");
  return a;
}

struct Int8Out {
  Tensor q, scale;
  Rows rows;
  float *scale_p;
};
Int8Out int8_out(const Tensor &x, const Opt &q, const Opt &scale, int64_t rows) {
  Int8Out o;
  if (q) shaped(*q, x.sizes(), at::kChar, x, "q");
  o.q = q ? *q : int8_rows(x);
  o.scale = scale ? *scale
                  : at::empty(x.sizes().slice(0, x.dim() - 1), x.options().dtype(at::kFloat));
  o.rows = rows_of(o.q, "q");
  o.scale_p = const_cast<float *>(vec(o.scale, rows, x, "scale"));
  return o;
}

py::object rms_norm(const Tensor &x, const Opt &gain, double eps, const Opt &residual, Opt h,
                    const Opt &y) {
  const On on(x);
  const NormIn a = norm_in(x, gain, residual, h);
  if (y) shaped(*y, x.sizes(), x.scalar_type(), x, "y");
  const Tensor out = y ? *y : new_rows(x, x.scalar_type());
  const Rows o = rows_of(out, "y");
  check(lib.rms_norm(a.x.p, a.x.stride, a.r.p, a.r.stride, a.h.p, a.h.stride, a.gain, a.gain_dtype,
                     (float)eps, a.x.rows, (int)a.x.cols, a.dtype, o.p, o.stride, on.stream));
  if (residual) return py::make_tuple(out, *h);
  return py::cast(out);
}

py::tuple rms_norm_int8(const Tensor &x, const Opt &gain, double eps, const Opt &residual, Opt h,
                        const Opt &q, const Opt &scale) {
  const On on(x);
  const NormIn a = norm_in(x, gain, residual, h);
  const Int8Out o = int8_out(x, q, scale, a.x.rows);
  check(lib.rms_norm_int8(a.x.p, a.x.stride, a.r.p, a.r.stride, a.h.p, a.h.stride, a.gain,
                          a.gain_dtype, (float)eps, a.x.rows, (int)a.x.cols, a.dtype,
                          static_cast<int8_t *>(o.rows.p), o.rows.stride, o.scale_p, on.stream));
  if (residual) return py::make_tuple(o.q, o.scale, *h);
  return py::make_tuple(o.q, o.scale);
}

py::tuple quantize_rows(const Tensor &x, const Opt &q, const Opt &scale) {
  const On on(x);
  const int dtype = dtype_of(x.scalar_type(), "x");
  const Rows r = rows_of(x, "x");
  if (r.cols > INT32_MAX) raise(BV_ERR_SHAPE, "rows of 2^31 values and more");
  const Int8Out o = int8_out(x, q, scale, r.rows);
  check(lib.quantize_rows(r.p, r.stride, r.rows, (int)r.cols, dtype,
                          static_cast<int8_t *>(o.rows.p), o.rows.stride, o.scale_p, on.stream));
  return py::make_tuple(o.q, o.scale);
}

Tensor int8_matmul(const Tensor &a, const Tensor &a_scale, const Tensor &w, const Tensor &w_scale,
                   const Opt &bias, const Opt &residual, std::optional<at::ScalarType> out_dtype,
                   bool channels_first, const Opt &y) {
  const On on(a);
  if (a.scalar_type() != at::kChar || w.scalar_type() != at::kChar)
    raise(BV_ERR_ARG, "a and w must be int8");
  on_device(w, a, "w");
  const Rows ra = rows_of(a, "a"), rw = rows_of(w, "w");
  if (w.dim() != 2 || ra.cols != rw.cols) {
    raise(BV_ERR_SHAPE, "a [..., " + std::to_string(ra.cols) + "] times w " + text(w.sizes()));
  }
  if (ra.rows > INT32_MAX || rw.rows > INT32_MAX || ra.cols > INT32_MAX)
    raise(BV_ERR_SHAPE, "sizes of 2^31 and more");
  const at::ScalarType type = out_dtype  ? *out_dtype
                              : y        ? y->scalar_type()
                              : residual ? residual->scalar_type()
                                         : at::kFloat;
  const int dtype = dtype_of(type, "y");
  c10::SmallVector<int64_t, 5> sizes;
  if (channels_first) {
    sizes = {rw.rows, ra.rows};
  } else {
    sizes.append(a.sizes().begin(), a.sizes().end());
    sizes.back() = rw.rows;
  }
  if (y) shaped(*y, sizes, type, a, "y");
  const Tensor out = y ? *y : at::empty(sizes, a.options().dtype(type));
  const Rows ro = rows_of(out, "y");
  Rows rr{nullptr, 0, 0, 0};
  if (residual) {
    shaped(*residual, sizes, type, a, "residual");
    rr = rows_of(*residual, "residual");
  }
  check(lib.int8_matmul(static_cast<const int8_t *>(ra.p), ra.stride,
                        vec(a_scale, ra.rows, a, "a_scale"), static_cast<const int8_t *>(rw.p),
                        rw.stride, vec(w_scale, rw.rows, a, "w_scale"),
                        bias ? vec(*bias, rw.rows, a, "bias") : nullptr, (int)ra.rows,
                        (int)rw.rows, (int)ra.cols, rr.p, rr.stride, out.data_ptr(), ro.stride,
                        dtype, channels_first ? 1 : 0, on.stream));
  return out;
}

// Addresses of libbv's entries by name, and the exception that errors become.
void bind(const py::dict &at, const py::object &error) {
  auto get = [&](const char *name) { return at[name].cast<uintptr_t>(); };
  lib.last_error = reinterpret_cast<decltype(lib.last_error)>(get("bv_last_error"));
  lib.rms_norm = reinterpret_cast<decltype(lib.rms_norm)>(get("bv_rms_norm"));
  lib.rms_norm_int8 = reinterpret_cast<decltype(lib.rms_norm_int8)>(get("bv_rms_norm_int8"));
  lib.quantize_rows = reinterpret_cast<decltype(lib.quantize_rows)>(get("bv_quantize_rows"));
  lib.int8_matmul = reinterpret_cast<decltype(lib.int8_matmul)>(get("bv_int8_matmul"));
  lib.error = py::object(error).release().ptr();
}

}  // namespace

PYBIND11_MODULE(_tokens, m) {
  m.attr("built_for") = BUILT_FOR;  // the torch of the build, which the build script looks for
  m.def("bind", &bind);
  m.def("rms_norm", &rms_norm);
  m.def("rms_norm_int8", &rms_norm_int8);
  m.def("quantize_rows", &quantize_rows);
  m.def("int8_matmul", &int8_matmul);
}
