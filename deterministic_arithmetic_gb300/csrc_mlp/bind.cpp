// bind.cpp -- the Python binding of include/lora_mlp.h: argument checks, outputs and workspaces as
// torch tensors, the call on the current stream. Argument marshalling only; the kernels do the work.
//
// A compiled module rather than ctypes, because the small calls of these operators are bound by the
// host: a layer norm of 8 rows takes the GPU 3.5 us, and its checks, three outputs and launch took 17 us
// through ctypes and take 5.5 us here. The calls keep the library's C ABI between them and the kernels.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <sstream>

#include "../../include/lora_mlp.h"

namespace {

using at::Tensor;
using Shape = std::vector<int64_t>;
constexpr auto BF16 = at::kBFloat16, F32 = at::kFloat, U8 = at::kByte, I8 = at::kChar;

PyObject *packed_type = nullptr, *error_type = nullptr;      // Packed8 and LoraDeltaError, given by setup()
PyObject *codes_name = nullptr, *scales_name = nullptr, *cols_name = nullptr;

struct Raised {};                                             // a Python error is set

[[noreturn]] void raise(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw Raised{};
}

// An owned reference.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* p) : p(p) {
    if (!p) throw Raised{};
  }
  Ref(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  PyObject* release() {
    PyObject* q = p;
    p = nullptr;
    return q;
  }
};

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

const char* dtype_name(at::ScalarType t) { return t == BF16 ? "torch.bfloat16" : t == F32 ? "torch.float32" : t == U8 ? "torch.uint8" : t == I8 ? "torch.int8" : c10::toString(t); }

[[noreturn]] void refuse(const Tensor& t, const char* name, const char* want, c10::IntArrayRef shape, int dev) {
  std::ostringstream s;
  s << name << ": expected contiguous " << want << " " << shape << " on ";
  if (dev < 0) s << "a CUDA device";
  else s << "cuda:" << dev;
  s << ", got " << dtype_name(t.scalar_type()) << " " << t.sizes() << " on " << t.device()
    << (t.is_contiguous() ? "" : ", not contiguous");
  raise(PyExc_ValueError, s.str());
}

// The address of t, a contiguous tensor of that type and shape on CUDA device dev.
void* check(const Tensor& t, const char* name, c10::IntArrayRef shape, at::ScalarType type, int dev) {
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
    refuse(t, name, dtype_name(type), shape, dev);
  return t.data_ptr();
}
void* check(PyObject* o, const char* name, c10::IntArrayRef shape, at::ScalarType type, int dev) {
  return check(tensor(o, name), name, shape, type, dev);
}
// The same for a bf16 or fp32 tensor; *code its LORA_BF16 or LORA_F32.
void* check_either(const Tensor& t, const char* name, c10::IntArrayRef shape, int dev, int* code) {
  if (t.scalar_type() != BF16 && t.scalar_type() != F32) refuse(t, name, "torch.bfloat16 or torch.float32", shape, dev);
  *code = t.scalar_type() == BF16 ? LORA_BF16 : LORA_F32;
  return check(t, name, shape, t.scalar_type(), dev);
}
// The device an operator runs on, that of its first tensor, and that tensor's two sizes. The library
// launches on the current device, where another device's addresses are not to be used: they are refused.
int first(const Tensor& t, const char* name, int64_t* rows, int64_t* cols) {
  if (t.dim() != 2 || !t.is_cuda()) refuse(t, name, "2-D tensor", t.sizes(), t.is_cuda() ? int(t.get_device()) : -1);
  const int dev = int(t.get_device());
  c10::DeviceIndex current = -1;
  if (c10::cuda::GetDevice(&current) != cudaSuccess || current != dev)
    raise(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(dev) + ", which is not the current device" +
                                (current < 0 ? "" : " (cuda:" + std::to_string(int(current)) + ")"));
  *rows = t.size(0);
  *cols = t.size(1);
  return dev;
}
Tensor empty(c10::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, c10::DeviceIndex(dev)), std::nullopt);
}
// An output: the caller's tensor, checked, or a new one.
Tensor out(PyObject* o, const char* name, c10::IntArrayRef shape, at::ScalarType type, int dev) {
  if (o == Py_None) return empty(shape, type, dev);
  const Tensor& t = tensor(o, name);
  check(t, name, shape, type, dev);
  return t;
}
// A workspace of at least `bytes` bytes: the caller's (its size is the library's to judge) or a new one.
Tensor scratch(PyObject* o, size_t bytes, int dev) {
  if (o == Py_None) return empty({int64_t(bytes)}, U8, dev);
  const Tensor& t = tensor(o, "workspace");
  if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous()) raise(PyExc_ValueError, "workspace: expected a contiguous tensor on cuda:" + std::to_string(dev));
  return t;
}
void* stream(int dev) { return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream(); }

void done(lora_status rc, const char* where) {
  if (rc == LORA_OK) return;
  Ref e(PyObject_CallFunction(error_type, "is", int(rc), where));
  PyErr_SetObject(error_type, e.p);
  throw Raised{};
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
template <class... T>
PyObject* tuple(T... item) {                                  // steals its items, also when it fails
  PyObject* all[] = {item...};
  PyObject* t = PyTuple_New(sizeof...(item));
  bool ok = t != nullptr;
  for (PyObject* o : all) ok = ok && o;
  for (size_t i = 0; i < sizeof...(item); ++i) {
    if (ok) PyTuple_SET_ITEM(t, i, all[i]);
    else Py_XDECREF(all[i]);
  }
  if (!ok) {
    Py_XDECREF(t);
    throw Raised{};
  }
  return t;
}
PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

int64_t groups(int64_t cols) { return (cols + 31) / 32; }
bool is_packed(PyObject* o) { return Py_TYPE(o) == reinterpret_cast<PyTypeObject*>(packed_type); }
// The codes and scales of a Packed8 of that size.
struct Packed {
  void *codes, *scales;
};
int64_t packed_cols(PyObject* o, const char* name) {
  if (!is_packed(o)) raise(PyExc_TypeError, std::string(name) + " must be a Packed8");
  Ref n(PyObject_GetAttr(o, cols_name));
  const int64_t v = PyLong_AsLongLong(n.p);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
Packed check_packed(PyObject* o, const char* name, int64_t rows, int64_t cols, int dev) {
  const int64_t have = packed_cols(o, name);
  if (have != cols) raise(PyExc_ValueError, std::string(name) + ": expected " + std::to_string(cols) + " columns, got " + std::to_string(have));
  Ref c(PyObject_GetAttr(o, codes_name)), s(PyObject_GetAttr(o, scales_name));
  const int64_t g = groups(cols);
  return {check(c.p, (std::string(name) + ".codes").c_str(), {rows, 32 * g}, I8, dev),
          check(s.p, (std::string(name) + ".scales").c_str(), {rows, g}, U8, dev)};
}
// A new Packed8; *p its parts.
PyObject* new_packed(int64_t rows, int64_t cols, int dev, Packed* p) {
  const int64_t g = groups(cols);
  const Tensor c = empty({rows, 32 * g}, I8, dev), s = empty({rows, g}, U8, dev);
  *p = {c.data_ptr(), s.data_ptr()};
  Ref a(wrap(c)), b(wrap(s)), n(PyLong_FromLongLong(cols));
  PyObject* args[] = {a.p, b.p, n.p};
  PyObject* made = PyObject_Vectorcall(packed_type, args, 3, nullptr);
  if (!made) throw Raised{};
  return made;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

// ------------------------------------------------------------- the operators
// Each takes its Python function's arguments in order, all given.

PyObject* layer_norm_fwd(PyObject* const* a) {                // x, weight, bias, eps, y, mean, rstd
  const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
  int64_t M, N;
  int xt, wt;
  const int dev = first(x, "x", &M, &N);
  const void* xp = check_either(x, "x", x.sizes(), dev, &xt);
  const void* wp = check_either(w, "weight", {N}, dev, &wt);
  const void* bp = a[2] == Py_None ? nullptr : check(a[2], "bias", {N}, w.scalar_type(), dev);
  const float eps = float(number(a[3]));
  const Tensor y = out(a[4], "y", x.sizes(), x.scalar_type(), dev);
  const Tensor mean = out(a[5], "mean", {M}, F32, dev), rstd = out(a[6], "rstd", {M}, F32, dev);
  done(lora_layer_norm_fwd(xp, xt, wp, bp, wt, eps, M, N, y.data_ptr(), mean.data_ptr<float>(), rstd.data_ptr<float>(),
                           stream(dev)), "lora_layer_norm_fwd");
  return tuple(wrap(y), wrap(mean), wrap(rstd));
}

PyObject* layer_norm_bwd(PyObject* const* a) {                // dy, x, weight, mean, rstd, bias_grad, dx, dw, db, workspace
  const Tensor &dy = tensor(a[0], "dy"), &w = tensor(a[2], "weight");
  int64_t M, N;
  int type, wt;
  const int dev = first(dy, "dy", &M, &N);
  const void* dyp = check_either(dy, "dy", dy.sizes(), dev, &type);
  Packed x{nullptr, nullptr};
  if (is_packed(a[1])) x = check_packed(a[1], "x", M, N, dev);
  else x.codes = check(a[1], "x", dy.sizes(), dy.scalar_type(), dev);
  const void* wp = check_either(w, "weight", {N}, dev, &wt);
  const float* mean = static_cast<const float*>(check(a[3], "mean", {M}, F32, dev));
  const float* rstd = static_cast<const float*>(check(a[4], "rstd", {M}, F32, dev));
  const int bias = PyObject_IsTrue(a[5]);
  if (bias < 0) throw Raised{};
  const Tensor dx = out(a[6], "dx", dy.sizes(), dy.scalar_type(), dev), dw = out(a[7], "dw", {N}, F32, dev);
  Tensor db;
  if (bias) db = out(a[8], "db", {N}, F32, dev);
  const Tensor ws = scratch(a[9], lora_layer_norm_bwd_workspace_size(M, N), dev);
  done(lora_layer_norm_bwd(dyp, type, x.codes, x.scales, wp, wt, mean, rstd, M, N, dx.data_ptr(), dw.data_ptr<float>(),
                           bias ? db.data_ptr<float>() : nullptr, ws.data_ptr(), ws.nbytes(), stream(dev)),
       "lora_layer_norm_bwd");
  return tuple(wrap(dx), wrap(dw), bias ? wrap(db) : none());
}

PyObject* pack8(PyObject* const* a) {                         // x, out
  const Tensor& x = tensor(a[0], "x");
  int64_t M, K;
  int xt;
  const int dev = first(x, "x", &M, &K);
  const void* xp = check_either(x, "x", x.sizes(), dev, &xt);
  Packed p;
  if (a[1] != Py_None) p = check_packed(a[1], "out", M, K, dev), Py_INCREF(a[1]);
  Ref o(a[1] == Py_None ? new_packed(M, K, dev, &p) : a[1]);
  done(lora_pack8(xp, xt, M, K, p.codes, p.scales, stream(dev)), "lora_pack8");
  return o.release();
}

PyObject* unpack8(PyObject* const* a) {                       // p, dtype code, out
  const int64_t K = packed_cols(a[0], "p");
  int64_t M, ld;
  int dev;
  {
    Ref c(PyObject_GetAttr(a[0], codes_name));
    dev = first(tensor(c.p, "p.codes"), "p.codes", &M, &ld);
  }
  const Packed p = check_packed(a[0], "p", M, K, dev);
  int code = int(integer(a[1]));
  Tensor o;
  if (a[2] == Py_None) {
    o = empty({M, K}, code == LORA_BF16 ? BF16 : F32, dev);
  } else {
    o = tensor(a[2], "out");
    check_either(o, "out", {M, K}, dev, &code);
  }
  done(lora_unpack8(p.codes, p.scales, M, K, o.data_ptr(), code, stream(dev)), "lora_unpack8");
  return wrap(o);
}

PyObject* pack8_da(PyObject* const* a) {                      // du, p, da, workspace
  const Tensor& du = tensor(a[0], "du");
  int64_t M, R;
  const int dev = first(du, "du", &M, &R);
  const void* dup = check(du, "du", du.sizes(), BF16, dev);
  const int64_t K = packed_cols(a[1], "p");
  const Packed p = check_packed(a[1], "p", M, K, dev);
  const Tensor da = out(a[2], "da", {R, K}, F32, dev);
  const Tensor ws = scratch(a[3], lora_pack8_da_workspace_size(M, K, R), dev);
  done(lora_pack8_da(dup, p.codes, p.scales, M, K, R, da.data_ptr<float>(), ws.data_ptr(), ws.nbytes(), stream(dev)),
       "lora_pack8_da");
  return wrap(da);
}

PyObject* lora_delta_bwd_packed8(PyObject* const* v) {        // dy, p, a, b, u, alpha, dx, da, db, du, workspace
  const Tensor &dy = tensor(v[0], "dy"), &a = tensor(v[2], "a");
  int64_t M, N;
  const int dev = first(dy, "dy", &M, &N);
  const int64_t K = packed_cols(v[1], "p"), R = a.dim() ? a.size(0) : 0;
  const void* dyp = check(dy, "dy", dy.sizes(), BF16, dev);
  const Packed p = check_packed(v[1], "p", M, K, dev);
  const void *ap = check(a, "a", {R, K}, BF16, dev), *bp = check(v[3], "b", {N, R}, BF16, dev), *up = check(v[4], "u", {M, R}, BF16, dev);
  const float alpha = float(number(v[5]));
  const Tensor dx = out(v[6], "dx", {M, K}, F32, dev), da = out(v[7], "da", {R, K}, F32, dev);
  const Tensor db = out(v[8], "db", {N, R}, F32, dev), du = out(v[9], "du", {M, R}, BF16, dev);
  const size_t need = lora_delta_bwd_packed8_workspace_size(M, K, N, R);
  // a new one is zeroed: it starts with the delta's control block
  const Tensor ws = v[10] == Py_None ? at::zeros({int64_t(need)}, at::TensorOptions().dtype(U8).device(c10::kCUDA, c10::DeviceIndex(dev)))
                                     : scratch(v[10], need, dev);
  done(::lora_delta_bwd_packed8(dyp, p.codes, p.scales, ap, bp, up, alpha, M, K, N, R, dx.data_ptr<float>(),
                              da.data_ptr<float>(), db.data_ptr<float>(), du.data_ptr(), ws.data_ptr(), ws.nbytes(),
                              stream(dev)), "lora_delta_bwd_packed8");
  return tuple(wrap(dx), wrap(da), wrap(db), wrap(du));
}

// One kept gate or up: bf16, or packed.
Packed kept(PyObject* o, const char* name, int64_t M, int64_t F, int dev) {
  if (is_packed(o)) return check_packed(o, name, M, F, dev);
  return {check(o, name, {M, F}, BF16, dev), nullptr};
}

PyObject* gated_ffn_fwd(PyObject* const* a) {  // x, w_gate, w_up, activation code, delta_gate, delta_up, keep code, h, gate, up
  const Tensor &x = tensor(a[0], "x"), &wg = tensor(a[1], "w_gate");
  int64_t M, K;
  const int dev = first(x, "x", &M, &K);
  const int64_t F = wg.dim() ? wg.size(0) : 0;
  const void* xp = check(x, "x", x.sizes(), BF16, dev);
  const void *wgp = check(wg, "w_gate", {F, K}, BF16, dev), *wup = check(a[2], "w_up", {F, K}, BF16, dev);
  const int act = int(integer(a[3])), keep = int(integer(a[6]));
  const float *dg = nullptr, *du = nullptr;
  if (a[4] != Py_None || a[5] != Py_None) {                   // both or neither
    dg = static_cast<const float*>(check(a[4], "delta_gate", {M, F}, F32, dev));
    du = static_cast<const float*>(check(a[5], "delta_up", {M, F}, F32, dev));
  }
  const Tensor h = out(a[7], "h", {M, F}, BF16, dev);
  PyObject* made[2] = {none(), none()};
  Packed p[2] = {{nullptr, nullptr}, {nullptr, nullptr}};
  const char* name[2] = {"gate", "up"};
  try {
    for (int i = 0; i < 2 && keep != LORA_KEEP_NONE; ++i) {
      PyObject* given = a[8 + i];
      PyObject* o;
      if (given == Py_None && keep == LORA_KEEP_PACKED8) {
        o = new_packed(M, F, dev, &p[i]);
      } else if (given == Py_None) {
        const Tensor t = empty({M, F}, BF16, dev);
        p[i].codes = t.data_ptr();
        o = wrap(t);
        if (!o) throw Raised{};
      } else {
        if (is_packed(given) != (keep == LORA_KEEP_PACKED8))
          raise(PyExc_ValueError, std::string(name[i]) + (keep == LORA_KEEP_PACKED8 ? ": expected a Packed8" : ": expected a bf16 tensor") + " for this save");
        p[i] = kept(given, name[i], M, F, dev);
        Py_INCREF(given);
        o = given;
      }
      Py_DECREF(made[i]);
      made[i] = o;
    }
    done(lora_gated_ffn_fwd(xp, wgp, wup, dg, du, act, M, K, F, h.data_ptr(), keep, p[0].codes, p[1].codes, p[0].scales,
                            p[1].scales, stream(dev)), "lora_gated_ffn_fwd");
  } catch (...) {
    Py_DECREF(made[0]);
    Py_DECREF(made[1]);
    throw;
  }
  return tuple(wrap(h), made[0], made[1]);
}

// dh, x, w_gate, w_up, gate, up, activation code, weight_grads, dx, dgate, dup, dw_gate, dw_up
PyObject* gated_ffn_bwd(PyObject* const* a) {
  const Tensor &dh = tensor(a[0], "dh"), &wg = tensor(a[2], "w_gate");
  int64_t M, F;
  const int dev = first(dh, "dh", &M, &F);
  const int64_t K = wg.dim() == 2 ? wg.size(1) : 0;
  const void* dhp = check(dh, "dh", dh.sizes(), BF16, dev);
  const int act = int(integer(a[6])), grads = PyObject_IsTrue(a[7]);
  if (grads < 0) throw Raised{};
  const void* xp = grads || a[1] != Py_None ? check(a[1], "x", {M, K}, BF16, dev) : nullptr;
  const void *wgp = check(wg, "w_gate", {F, K}, BF16, dev), *wup = check(a[3], "w_up", {F, K}, BF16, dev);
  if (is_packed(a[4]) != is_packed(a[5])) raise(PyExc_ValueError, "gate, up: both bf16 tensors or both Packed8");
  const Packed g = kept(a[4], "gate", M, F, dev), u = kept(a[5], "up", M, F, dev);
  const Tensor dx = out(a[8], "dx", {M, K}, BF16, dev);
  const Tensor dg = out(a[9], "dgate", {M, F}, BF16, dev), du = out(a[10], "dup", {M, F}, BF16, dev);
  Tensor dwg, dwu;
  if (grads) dwg = out(a[11], "dw_gate", {F, K}, BF16, dev), dwu = out(a[12], "dw_up", {F, K}, BF16, dev);
  done(lora_gated_ffn_bwd(dhp, xp, wgp, wup, g.scales ? LORA_KEEP_PACKED8 : LORA_KEEP_BF16, g.codes, u.codes, g.scales,
                          u.scales, act, M, K, F, dx.data_ptr(), dg.data_ptr(), du.data_ptr(),
                          grads ? dwg.data_ptr() : nullptr, grads ? dwu.data_ptr() : nullptr, stream(dev)),
       "lora_gated_ffn_bwd");
  return tuple(wrap(dx), wrap(dg), wrap(du), grads ? wrap(dwg) : none(), grads ? wrap(dwu) : none());
}

// setup(Packed8, LoraDeltaError)
PyObject* setup(PyObject* const* a) {
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  Py_XSETREF(packed_type, a[0]);
  Py_XSETREF(error_type, a[1]);
  return none();
}

// An operator as a module function of n arguments. No C++ exception leaves it.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<layer_norm_fwd, 7>("layer_norm_fwd"), method<layer_norm_bwd, 10>("layer_norm_bwd"), method<pack8, 2>("pack8"),
    method<unpack8, 3>("unpack8"), method<pack8_da, 4>("pack8_da"), method<lora_delta_bwd_packed8, 11>("lora_delta_bwd_packed8"),
    method<gated_ffn_fwd, 10>("gated_ffn_fwd"), method<gated_ffn_bwd, 13>("gated_ffn_bwd"), method<setup, 2>("setup"),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mlp", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mlp() {
  codes_name = PyUnicode_InternFromString("codes");
  scales_name = PyUnicode_InternFromString("scales");
  cols_name = PyUnicode_InternFromString("cols");
  return codes_name && scales_name && cols_name ? PyModule_Create(&module) : nullptr;
}
