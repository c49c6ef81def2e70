// kl_python.cpp -- torch tensors <-> libklein.so's entry points of the
// projection path, as a CPython module (klein_torch).
//
// The small calls of that path run a few microseconds on the GPU, and making
// them from Python (checks, torch.empty, ctypes) took 12 to 22 of the CPU; the
// same steps here take 4 to 8.  Each function checks its tensors (ValueError),
// allocates its outputs and scratch on the current stream of the tensors'
// device, whichever device is current, and calls the C entry point; a status
// other than KL_OK becomes a KLError.  Nothing is kept between calls.
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include "../../include/klein.h"

namespace {

PyObject* g_error = nullptr;  // KLError(status, where)

const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, ": expected a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  // results carry no graph: with grad mode on, one would be cut without a word
  TORCH_CHECK_VALUE(!(t.requires_grad() && at::GradMode::is_enabled()), name,
                    ": requires a gradient, which this call does not record; pass it detached, or call under "
                    "torch.no_grad() or from a torch.autograd.Function");
  return t;
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// KL_BF16 / KL_F32 / KL_F16, or -1
int kind(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return KL_BF16;
    case at::kFloat: return KL_F32;
    case at::kHalf: return KL_F16;
    default: return -1;
  }
}
int need_float(const at::Tensor& t, const char* name) {
  const int k = kind(t);
  TORCH_CHECK_VALUE(t.is_cuda() && k >= 0, name, ": expected a CUDA tensor of bfloat16, float16 or float32");
  return k;
}
void need(const at::Tensor& t, const at::Device& dev, at::ScalarType type, const char* name) {
  TORCH_CHECK_VALUE(t.is_cuda() && t.scalar_type() == type, name, ": expected a CUDA tensor of ", type);
  TORCH_CHECK_VALUE(t.device() == dev, name, ": on ", t.device(), ", the call is on ", dev);
}

struct Rows {
  int64_t rows, cols, ld;
};
// t [..., cols] as a matrix whose rows lie at one stride (no copy is made)
Rows rows_of(const at::Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.dim() >= 1 && t.numel() > 0, name, ": expected a tensor [..., cols] that is not empty");
  const int64_t cols = t.size(-1);
  if (t.is_contiguous()) return {t.numel() / cols, cols, cols};
  TORCH_CHECK_VALUE(cols == 1 || t.stride(-1) == 1, name, ": the last dimension must be consecutive");
  int64_t rows = 1, ld = cols;
  for (int64_t d = t.dim() - 2; d >= 0; --d) {
    const int64_t n = t.size(d), st = t.stride(d);
    if (n == 1) continue;
    if (rows == 1)
      ld = st;
    else
      TORCH_CHECK_VALUE(st == rows * ld, name, ": rows must lie at one stride");
    rows *= n;
  }
  TORCH_CHECK_VALUE(ld >= cols, name, ": rows must not overlap");
  return {rows, cols, ld};
}

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const at::Device& dev) {
  return at::detail::empty_cuda(sizes, type, dev, std::nullopt);
}
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
PyObject* wrap(at::Tensor t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(t));
}
PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = wrap(t);
    if (!o) {
      Py_DECREF(r);
      throw python_error();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// A caller's tensor has been written: its version moves on, as for torch's own
// writes in place, so that autograd refuses to use values it saved from before.
// (Inference tensors have no version and are never saved.)
void written(const at::Tensor& t) {
  if (!t.is_inference()) torch::autograd::impl::bump_version(t);
}

// f(stream) with the tensors' device current
template <typename F>
void call(const at::Device& dev, const char* name, F f) {
  const c10::cuda::OptionalCUDAGuard guard(dev);
  const kl_status st = f((void*)c10::cuda::getCurrentCUDAStream(dev.index()).stream());
  if (st == KL_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, name);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

void arity(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK(n == want, "expected ", want, " arguments, got ", n); }

#define KL_METHOD(name) \
  PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n) { \
    HANDLE_TH_ERRORS
#define KL_METHOD_END \
  END_HANDLE_TH_ERRORS \
  }

// (x, name) -> (rows, cols, row stride)
KL_METHOD(py_rows)
arity(n, 2);
const char* name = PyUnicode_AsUTF8(a[1]);
if (!name) throw python_error();
const Rows r = rows_of(tensor(a[0], name), name);
return Py_BuildValue("LLL", (long long)r.rows, (long long)r.cols, (long long)r.ld);
KL_METHOD_END

// (x, flags) -> (codes, scales, rows, cols)
KL_METHOD(py_quantize)
arity(n, 2);
const at::Tensor& x = tensor(a[0], "x");
const int dtype = need_float(x, "x"), flags = (int)integer(a[1]);
const Rows r = rows_of(x, "x");
const bool tr = flags & KL_FP8_TRANSPOSE;
const int64_t rows = tr ? r.cols : r.rows, cols = tr ? r.rows : r.cols, ldc = (cols + 15) / 16 * 16;
const at::Device dev = x.device();
at::Tensor codes = empty({rows, ldc}, at::kByte, dev);
const int64_t blocks = (cols + 127) / 128, bytes = (int64_t)kl_fp8_scales_bytes(rows, cols, flags);
at::Tensor scales = flags & KL_SCALE_MMA ? empty({bytes}, at::kByte, dev)
                                         : empty({bytes / blocks, blocks}, at::kByte, dev);
call(dev, "kl_quantize_fp8_block", [&](void* s) {
  return kl_quantize_fp8_block(x.data_ptr(), dtype, r.rows, r.cols, r.ld, codes.data_ptr(), ldc, scales.data_ptr(),
                               flags, s);
});
return Py_BuildValue("NNLL", wrap(std::move(codes)), wrap(std::move(scales)), (long long)rows, (long long)cols);
KL_METHOD_END

kl_fp8_tensor operand(PyObject* codes_o, PyObject* scales_o, int64_t rows, int64_t cols, const at::Device& dev,
                      const char* name) {
  const at::Tensor &codes = tensor(codes_o, name), &scales = tensor(scales_o, name);
  need(codes, dev, at::kByte, name);
  need(scales, dev, at::kByte, name);
  TORCH_CHECK_VALUE(
      codes.dim() == 2 && codes.size(0) >= rows && codes.size(1) >= cols && (codes.size(1) == 1 || codes.stride(1) == 1),
      name, ".codes: expected [rows, >= cols] with consecutive columns");
  TORCH_CHECK_VALUE(scales.is_contiguous() && scales.numel() >= (rows + 127) / 128 * ((cols + 511) / 512) * 512, name,
                    ".scales: too small for [", rows, ", ", cols, "]");
  // (a single row may have any stride)
  return {codes.data_ptr(), scales.data_ptr(), codes.size(0) == 1 ? (codes.size(1) + 15) / 16 * 16 : codes.stride(0)};
}

// (A.codes, A.scales, M, W.codes, W.scales, N, K, out or None, out type, kernel) -> out
KL_METHOD(py_gemm)
arity(n, 10);
const at::Device dev = tensor(a[0], "A").device();
TORCH_CHECK_VALUE(dev.is_cuda(), "A: expected a CUDA tensor");
const int64_t M = integer(a[2]), N = integer(a[5]), K = integer(a[6]);
const kl_fp8_tensor A = operand(a[0], a[1], M, K, dev, "A"), W = operand(a[3], a[4], N, K, dev, "W");
int type = (int)integer(a[8]);
const int kernel = (int)integer(a[9]);
at::Tensor out;
int64_t ldo = N;
if (a[7] == Py_None) {
  TORCH_CHECK_VALUE(M > 0 && N > 0, "operands must not be empty");
  out = empty({M, N}, type == KL_F32 ? at::kFloat : at::kBFloat16, dev);
} else {
  out = tensor(a[7], "out");
  type = kind(out);
  TORCH_CHECK_VALUE(out.is_cuda() && (type == KL_F32 || type == KL_BF16) && out.device() == dev,
                    "out: expected a tensor of bfloat16 or float32 on ", dev);
  TORCH_CHECK_VALUE(out.dim() == 2 && out.size(0) == M && out.size(1) == N && (N == 1 || out.stride(1) == 1) &&
                        (M == 1 || out.stride(0) >= N),
                    "out: expected [", M, ", ", N, "] with consecutive columns");
  ldo = std::max(out.stride(0), N);
}
call(dev, "kl_gemm_fp8_block",
     [&](void* s) { return kl_gemm_fp8_block(&A, &W, M, N, K, out.data_ptr(), type, ldo, kernel, s); });
if (a[7] != Py_None) written(out);
return wrap(std::move(out));
KL_METHOD_END

// (x, pos, sections, theta, flags, out or None) -> out
KL_METHOD(py_rope)
arity(n, 6);
const at::Tensor &x = tensor(a[0], "x"), &p = tensor(a[1], "pos");
kl_rope_args r{};
r.dtype = need_float(x, "x");
const at::Device dev = x.device();
const auto pt = p.scalar_type();
TORCH_CHECK_VALUE(p.is_cuda() && (pt == at::kInt || pt == at::kLong || pt == at::kFloat),
                  "pos: expected a CUDA tensor of int32, int64 or float32");
TORCH_CHECK_VALUE(p.device() == dev, "pos: on ", p.device(), ", the call is on ", dev);
r.pos_type = pt == at::kInt ? KL_POS_I32 : pt == at::kLong ? KL_POS_I64 : KL_POS_F32;
const int64_t nd = x.dim();
TORCH_CHECK_VALUE((nd == 3 || nd == 4) && x.numel() > 0 && (x.size(-1) == 1 || x.stride(-1) == 1),
                  "x: expected [tokens, heads, dim] or [batch, tokens, heads, dim], dims consecutive");
r.batch = nd == 4 ? x.size(0) : 1;
r.tokens = x.size(-3);
r.heads = x.size(-2);
r.dim = x.size(-1);
const Py_ssize_t naxes = PySequence_Size(a[2]);
if (naxes < 0) throw python_error();
TORCH_CHECK_VALUE(naxes >= 1 && naxes <= KL_ROPE_MAX_AXES, "sections: expected 1 to 4 axes");
r.naxes = (int)naxes;
for (Py_ssize_t i = 0; i < naxes; ++i) {
  THPObjectPtr o(PySequence_GetItem(a[2], i));
  if (!o) throw python_error();
  r.sections[i] = integer(o.get());
}
const bool shared = p.dim() == 2 && p.size(0) == r.tokens && p.size(1) == naxes;
TORCH_CHECK_VALUE(shared || (nd == 4 && p.dim() == 3 && p.size(0) == r.batch && p.size(1) == r.tokens && p.size(2) == naxes),
                  "pos: expected [", r.tokens, ", ", naxes, "] or [", r.batch, ", ", r.tokens, ", ", naxes, "]");
r.pos_shared = shared;
r.theta = real(a[3]);
r.flags = (int)integer(a[4]);
at::Tensor out;
if (a[5] == Py_None) {
  out = empty(x.sizes(), x.scalar_type(), dev);
} else {
  out = tensor(a[5], "out");
  need(out, dev, x.scalar_type(), "out");
  bool ok = out.sizes() == x.sizes() && (r.dim == 1 || out.stride(-1) == 1);
  for (int64_t d = 0; ok && d < nd; ++d) ok = out.size(d) == 1 || out.stride(d) != 0;
  TORCH_CHECK_VALUE(ok, "out: expected x's shape, dims consecutive, no broadcast dimensions");
}
const c10::cuda::OptionalCUDAGuard guard(dev);  // (a copy of pos runs there too)
const at::Tensor pos = p.contiguous();
for (int64_t i = 0, d = nd - 4; i < 3; ++i, ++d) {  // batch, token, head
  r.x_stride[i] = d >= 0 ? x.stride(d) : 0;
  r.out_stride[i] = d >= 0 ? out.stride(d) : 0;
}
r.x = x.data_ptr();
r.out = out.data_ptr();
r.pos = pos.data_ptr();
call(dev, "kl_rope_axes", [&](void* s) { return kl_rope_axes(&r, s); });
if (a[5] != Py_None) written(out);
return wrap(std::move(out));
KL_METHOD_END

// gain and bias: [cols] or [groups, cols], of one type
struct Params {
  int64_t groups = -1;
  int type = -1;
  at::Tensor add(PyObject* o, int64_t cols, const at::Device& dev, const char* name) {
    if (o == Py_None) return at::Tensor();
    const at::Tensor& t = tensor(o, name);
    const int k = need_float(t, name);
    TORCH_CHECK_VALUE(t.device() == dev, name, ": on ", t.device(), ", the call is on ", dev);
    TORCH_CHECK_VALUE(t.is_contiguous() && (t.dim() == 1 || t.dim() == 2) && t.size(-1) == cols, name,
                      ": expected a contiguous [", cols, "] or [groups, ", cols, "] tensor");
    const int64_t g = t.dim() == 2 ? t.size(0) : 1;
    TORCH_CHECK_VALUE(groups < 0 || g == groups, name, ": ", g, " groups, expected ", groups);
    TORCH_CHECK_VALUE(type < 0 || k == type, "gain and bias must have one type");
    groups = g;
    type = k;
    return t;
  }
  void finish(int64_t rows) {
    if (groups < 0) groups = 1;
    if (type < 0) type = KL_F32;
    TORCH_CHECK_VALUE(groups >= 1 && rows % groups == 0, groups, " groups do not divide ", rows, " rows");
  }
};

// (x, gain, bias, modulate, eps) -> (y, mean, rstd)
KL_METHOD(py_ln_forward)
arity(n, 5);
const at::Tensor& x = tensor(a[0], "x");
const int dtype = need_float(x, "x");
const Rows r = rows_of(x, "x");
const at::Device dev = x.device();
Params p;
const at::Tensor gain = p.add(a[1], r.cols, dev, "gain"), bias = p.add(a[2], r.cols, dev, "bias");
p.finish(r.rows);
const int flags = truth(a[3]) ? KL_LN_MODULATE : 0;
const float eps = (float)real(a[4]);
at::Tensor y = empty(x.sizes(), x.scalar_type(), dev);
at::Tensor mean = empty({r.rows}, at::kFloat, dev), rstd = empty({r.rows}, at::kFloat, dev);
call(dev, "kl_layer_norm_forward", [&](void* s) {
  return kl_layer_norm_forward(x.data_ptr(), dtype, r.rows, r.cols, r.ld, ptr(gain), ptr(bias), p.type, p.groups, eps,
                               flags, y.data_ptr(), r.cols, (float*)mean.data_ptr(), (float*)rstd.data_ptr(), s);
});
return tuple({std::move(y), std::move(mean), std::move(rstd)});
KL_METHOD_END

// (dy, x, mean, rstd, gain, modulate, groups or None, param_grads) -> (dx, dgain, dbias)
KL_METHOD(py_ln_backward)
arity(n, 8);
const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x");
const at::Tensor &mean = tensor(a[2], "mean"), &rstd = tensor(a[3], "rstd");
const int dtype = need_float(x, "x");
const at::Device dev = x.device();
need(dy, dev, x.scalar_type(), "dy");
TORCH_CHECK_VALUE(dy.sizes() == x.sizes(), "dy and x must have one shape");
const Rows r = rows_of(x, "x");
const int64_t lddy = rows_of(dy, "dy").ld;
need(mean, dev, at::kFloat, "mean");
need(rstd, dev, at::kFloat, "rstd");
TORCH_CHECK_VALUE(mean.numel() == r.rows && mean.is_contiguous() && rstd.numel() == r.rows && rstd.is_contiguous(),
                  "mean, rstd: expected contiguous fp32 [", r.rows, "]");
Params p;
if (a[6] != Py_None) {
  p.groups = integer(a[6]);
  TORCH_CHECK_VALUE(p.groups >= 1, "groups: expected one or more");
}
const at::Tensor gain = p.add(a[4], r.cols, dev, "gain");
p.finish(r.rows);
const int flags = truth(a[5]) ? KL_LN_MODULATE : 0;
at::Tensor dx = empty(x.sizes(), x.scalar_type(), dev), dgain, dbias, ws;
size_t bytes = 0;
if (truth(a[7])) {
  dgain = empty({p.groups, r.cols}, at::kFloat, dev);
  dbias = empty({p.groups, r.cols}, at::kFloat, dev);
  bytes = kl_layer_norm_backward_workspace_size(dtype, r.rows, r.cols, p.groups);
  if (bytes) ws = empty({(int64_t)bytes}, at::kByte, dev);
}
call(dev, "kl_layer_norm_backward", [&](void* s) {
  return kl_layer_norm_backward(dy.data_ptr(), lddy, x.data_ptr(), r.ld, dtype, r.rows, r.cols,
                                (const float*)mean.data_ptr(), (const float*)rstd.data_ptr(), ptr(gain), p.type,
                                p.groups, flags, dx.data_ptr(), r.cols, (float*)ptr(dgain), (float*)ptr(dbias), ptr(ws),
                                bytes, s);
});
return tuple({std::move(dx), std::move(dgain), std::move(dbias)});
KL_METHOD_END

// (KLError,): the exception a status other than KL_OK raises
KL_METHOD(py_set_error)
arity(n, 1);
Py_INCREF(a[0]);
Py_XDECREF(g_error);
g_error = a[0];
Py_RETURN_NONE;
KL_METHOD_END

#define KL_ENTRY(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KL_ENTRY(rows),       KL_ENTRY(quantize),    KL_ENTRY(gemm),      KL_ENTRY(rope),
                         KL_ENTRY(ln_forward), KL_ENTRY(ln_backward), KL_ENTRY(set_error), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "klein_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit_klein_torch() { return PyModule_Create(&module); }
