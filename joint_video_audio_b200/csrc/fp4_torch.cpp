// The 4-bit linear path and the sandwich norm for torch tensors: checks of the
// arguments, outputs and the calls of include/h3blk.h on the current stream, as
// a Python module. In C++ because these calls are short: a quantisation of a few
// rows is 2 us on the GPU, and the same marshalling over ctypes took the host 7 us.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "h3blk.h"

namespace {
using at::Tensor;

PyObject* g_error = nullptr;  // H3BlkError(name of the call, status)

struct Failed {
  const char* call;
  int status;
};
void check(const char* call, int status) {
  if (status != H3BLK_OK) throw Failed{call, status};
}

// Other Python threads run during allocations and launches, which may block.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};
// On a CUDA device, past the dispatcher: 0.3 us less an output.
Tensor empty(at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  const NoGil n;
  return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

// ------------------------------------------------------------------ arguments
bool given(PyObject* o) { return o != Py_None; }
const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, ": expected a torch.Tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int int32(PyObject* o) {
  const int64_t v = integer(o);
  TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, "an argument does not fit 32 bits: ", v);
  return (int)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}

// A 2-D CUDA tensor with unit column stride and its row stride.
struct Rows {
  int64_t rows, cols, ld;
};
Rows rows_of(const Tensor& t, const char* name, at::ScalarType type) {
  TORCH_CHECK_VALUE(t.is_cuda() && t.scalar_type() == type && t.dim() == 2, name, ": expected a 2-D ", type,
                    " CUDA tensor, got ", t.scalar_type(), " ", t.sizes(), " on ", t.device());
  const int64_t rows = t.size(0), cols = t.size(1), ld = t.stride(0);
  TORCH_CHECK_VALUE(t.stride(1) == 1 || cols <= 1, name, ": its rows are not contiguous");
  if (rows < 2) return {rows, cols, (cols + 7) / 8 * 8};
  TORCH_CHECK_VALUE(ld >= cols && ld % 8 == 0, name, ": row stride ", ld, " is not a multiple of 8 of at least ", cols);
  return {rows, cols, ld};
}
void want(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
  TORCH_CHECK_VALUE(t.scalar_type() == type && t.sizes() == shape && t.device() == dev && t.is_cuda() && t.is_contiguous(),
                    name, ": expected ", type, " ", shape, " contiguous on CUDA device ", dev, ", got ", t.scalar_type(),
                    " ", t.sizes(), " on ", t.device());
}

// The parts of a 4-bit matrix in its buffer: each on a 256-byte boundary.
struct Layout {
  size_t len[3], at[3], total;
};
Layout layout(int format, int64_t rows, int K) {
  Layout l;
  check("h3blk_fp4_bytes", h3blk_fp4_bytes(format, rows, K, &l.len[0], &l.len[1], &l.len[2]));
  size_t at = 0;
  for (int i = 0; i < 3; ++i) {
    l.at[i] = at;
    at += (l.len[i] + 255) / 256 * 256;
  }
  l.total = at < 256 ? 256 : at;
  return l;
}
h3blk_fp4 fp4(const Tensor& buffer, int format, int64_t rows, int K) {
  const Layout l = layout(format, rows, K);
  TORCH_CHECK_VALUE(buffer.scalar_type() == at::kByte && buffer.is_contiguous() && (size_t)buffer.numel() >= l.total,
                    "a 4-bit matrix's buffer does not fit its shape");
  uint8_t* p = static_cast<uint8_t*>(buffer.data_ptr());
  h3blk_fp4 q;
  q.format = format;
  q.K = K;
  q.rows = rows;
  q.codes = p;
  q.scales = p + l.at[1];
  q.row_scale = reinterpret_cast<float*>(p + l.at[2]);
  return q;
}
Tensor new_buffer(int format, int64_t rows, int K, c10::Device dev) {
  return empty({(int64_t)layout(format, rows, K).total}, at::kByte, dev);
}

// The output tensor, made here where none is given, and its row stride; one that
// is no multiple of 8 (columns that are not) is the library's to refuse.
Tensor output(PyObject* o, int64_t rows, int64_t cols, bool f32, c10::Device dev, int64_t* ld) {
  TORCH_CHECK_VALUE(dev.is_cuda(), "expected operands on a CUDA device, got ", dev);
  const at::ScalarType type = f32 ? at::kFloat : at::kBFloat16;
  if (!given(o)) {
    *ld = cols;
    return empty({rows, cols}, type, dev);
  }
  const Tensor& t = tensor(o, "out");
  const int64_t shape[2] = {rows, cols};
  TORCH_CHECK_VALUE(t.sizes() == at::IntArrayRef(shape, 2) && t.scalar_type() == type && t.device() == dev,
                    "out: expected ", type, " ", at::IntArrayRef(shape, 2), " on ", dev, ", got ", t.scalar_type(), " ",
                    t.sizes(), " on ", t.device());
  *ld = rows_of(t, "out", type).ld;
  return t;
}

// The device's current stream, with that device current, and no Python.
struct On {
  NoGil no_gil;
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit On(c10::Device dev) : guard(dev), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream()) {}
};

// ------------------------------------------------------------------ calls
// layout(format, rows, K) -> (lengths, offsets, total)
PyObject* py_layout(PyObject* const* a) {
  const Layout l = layout(int32(a[0]), integer(a[1]), int32(a[2]));
  return Py_BuildValue("((nnn)(nnn)n)", l.len[0], l.len[1], l.len[2], l.at[0], l.at[1], l.at[2], l.total);
}

// quantize(x, format, rotate, buffer or None) -> (shape, buffer)
PyObject* py_quantize(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Rows r = rows_of(x, "x", at::kBFloat16);
  const int format = int32(a[1]);
  TORCH_CHECK_VALUE(r.cols <= INT32_MAX, "x: too many columns");
  const Tensor buffer = given(a[3]) ? tensor(a[3], "out") : new_buffer(format, r.rows, (int)r.cols, x.device());
  TORCH_CHECK_VALUE(buffer.device() == x.device(), "out: expected a matrix on ", x.device(), ", got one on ", buffer.device());
  const h3blk_fp4 q = fp4(buffer, format, r.rows, (int)r.cols);
  const bool rotate = truth(a[2]);
  if (r.rows) {
    const On on(x.device());
    check("h3blk_quantize_fp4", h3blk_quantize_fp4(x.data_ptr(), r.ld, rotate, &q, on.stream));
  }
  return Py_BuildValue("((LL)N)", (long long)r.rows, (long long)r.cols, THPVariable_Wrap(buffer));
}

// dequantize(buffer, format, rows, K, f32, out or None) -> out
PyObject* py_dequantize(PyObject* const* a) {
  const Tensor& buffer = tensor(a[0], "q");
  const int64_t rows = integer(a[2]);
  const int K = int32(a[3]);
  const bool f32 = truth(a[4]);
  int64_t ld = 0;
  const Tensor out = output(a[5], rows, K, f32, buffer.device(), &ld);
  const h3blk_fp4 q = fp4(buffer, int32(a[1]), rows, K);
  if (rows) {
    const On on(buffer.device());
    check("h3blk_dequantize_fp4", h3blk_dequantize_fp4(&q, f32 ? H3BLK_F32 : H3BLK_BF16, out.data_ptr(), ld, on.stream));
  }
  return THPVariable_Wrap(out);
}

// gemm(buffer a, rows a, buffer b, rows b, format, K, swiglu, f32, out or None) -> out
PyObject* py_gemm(PyObject* const* a) {
  const Tensor &ba = tensor(a[0], "a"), &bb = tensor(a[2], "b");
  const int64_t rows = integer(a[1]), cols = integer(a[3]);
  const int format = int32(a[4]), K = int32(a[5]);
  const bool swiglu = truth(a[6]), f32 = truth(a[7]);
  TORCH_CHECK_VALUE(ba.device() == bb.device(), "operands do not match: one is on ", ba.device(), ", one on ", bb.device());
  int64_t ld = 0;
  const Tensor out = output(a[8], rows, swiglu ? cols / 2 : cols, f32, ba.device(), &ld);
  const h3blk_fp4 qa = fp4(ba, format, rows, K), qb = fp4(bb, format, cols, K);
  if (rows) {
    const On on(ba.device());
    check("h3blk_gemm_fp4", h3blk_gemm_fp4(&qa, &qb, swiglu ? H3BLK_FP4_SWIGLU : H3BLK_FP4_STORE,
                                           f32 ? H3BLK_F32 : H3BLK_BF16, out.data_ptr(), ld, on.stream));
  }
  return THPVariable_Wrap(out);
}

// sandwich(x, y, tag, tidx, table, branch, norm table or None, post_norm, gain or
// None, post_eps, norm_eps, branch_scale, h, rotate, x_out or None), h: -2 none,
// -1 bf16, else a 4-bit format -> (x_out, h: a tensor, a matrix's buffer or None)
PyObject* py_sandwich(PyObject* const* a) {
  const Tensor &x = tensor(a[0], "x"), &y = tensor(a[1], "y"), &tag = tensor(a[2], "tag"), &tidx = tensor(a[3], "tidx");
  const Tensor& table = tensor(a[4], "table");
  TORCH_CHECK_VALUE(x.dim() == 2 && table.dim() == 4, "expected x [rows, hidden] and table [n_tags, n_t, 6, hidden]");
  const c10::Device dev = x.device();
  const int64_t n = x.size(0), c = x.size(1), shape[2] = {n, c}, tab[4] = {table.size(0), table.size(1), 6, c};
  const at::IntArrayRef rows(shape, 2), row(shape, 1), chan(shape + 1, 1), tabs(tab, 4);
  const int h = int32(a[12]);
  h3blk_sandwich s{};
  want(x, "x", at::kBFloat16, rows, dev);
  want(y, "y", at::kBFloat16, rows, dev);
  want(tag, "tag", at::kInt, row, dev);
  want(tidx, "tidx", at::kInt, row, dev);
  want(table, "table", at::kFloat, tabs, dev);
  TORCH_CHECK_VALUE(c <= INT32_MAX && tab[0] <= INT32_MAX && tab[1] <= INT32_MAX, "a dimension does not fit 32 bits");
  if (given(a[6])) {
    const Tensor& t = tensor(a[6], "next_table");
    want(t, "next_table", at::kFloat, tabs, dev);
    s.norm_table = t.data_ptr<float>();
  }
  if (given(a[8])) {
    const Tensor& t = tensor(a[8], "post_gain");
    want(t, "post_gain", at::kBFloat16, chan, dev);
    s.post_gain = t.data_ptr();
  }
  const Tensor x_out = given(a[14]) ? tensor(a[14], "x_out") : empty(rows, at::kBFloat16, dev);
  want(x_out, "x_out", at::kBFloat16, rows, dev);
  Tensor out;
  h3blk_fp4 q;
  if (s.norm_table && h == -1) {
    out = empty(rows, at::kBFloat16, dev);
    s.h = out.data_ptr();
  } else if (s.norm_table) {
    out = new_buffer(h, n, (int)c, dev);
    q = fp4(out, h, n, (int)c);
    s.h_fp4 = &q;
  }
  s.n_rows = n;
  s.hidden = (int)c;
  s.n_tags = (int)tab[0];
  s.n_t = (int)tab[1];
  s.branch = int32(a[5]);
  s.post_norm = truth(a[7]);
  s.post_eps = real(a[9]);
  s.norm_eps = real(a[10]);
  s.branch_scale = real(a[11]);
  s.x = x.data_ptr();
  s.y = y.data_ptr();
  s.tag = tag.data_ptr<int32_t>();
  s.tidx = tidx.data_ptr<int32_t>();
  s.mod_table = table.data_ptr<float>();
  s.x_out = x_out.data_ptr();
  s.rotate = truth(a[13]);
  if (n) {
    const On on(dev);
    check("h3blk_sandwich_norm", h3blk_sandwich_norm(&s, on.stream));
  }
  if (!out.defined()) return Py_BuildValue("(NO)", THPVariable_Wrap(x_out), Py_None);
  return Py_BuildValue("(NN)", THPVariable_Wrap(x_out), THPVariable_Wrap(out));
}

PyObject* py_set_error(PyObject* const* a) {
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  Py_RETURN_NONE;
}

template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
    return nullptr;
  }
  try {
    return kCall(args);
  } catch (const Failed& f) {
    PyObject* e = PyObject_CallFunction(g_error ? g_error : PyExc_RuntimeError, "si", f.call, f.status);
    if (e) {
      PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
      Py_DECREF(e);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<kCall, kArgs>)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<py_layout, 3>("layout"), method<py_quantize, 4>("quantize"),
                           method<py_dequantize, 6>("dequantize"), method<py_gemm, 9>("gemm"),
                           method<py_sandwich, 15>("sandwich"), method<py_set_error, 1>("set_error"), {}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fp4_torch", nullptr, -1, g_methods};
}  // namespace

PyMODINIT_FUNC PyInit__fp4_torch() { return PyModule_Create(&g_module); }
