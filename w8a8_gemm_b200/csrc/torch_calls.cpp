// torch_calls.cpp -- the short way from torch tensors to the C ABI's operators
// around the quantized linear: a CPython module (_sqtorch) that checks the
// tensors, makes the outputs and the workspace, and calls the library.  These
// operators take a few microseconds on the GPU for a decoding step; through
// ctypes the host needed 19 us for such a call of the adapters, 10 of them
// outside the library (checks 4, three allocations 6), here 3.
//
// Each function returns its outputs as a tuple, the library's status as an int
// where it refused the call, or None where an argument does not fit; binding.py
// then looks for the reason.  The library is the one that binding.py has loaded:
// init() takes its handle.  It touches the host only; no C++ exception leaves it.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "segquant.h"

namespace {

using at::ScalarType;
using at::Tensor;
constexpr ScalarType BF16 = at::kBFloat16, F32 = at::kFloat, I32 = at::kInt, I8 = at::kChar;

struct Library {
  decltype(&sq_lora_plan_bytes) lora_plan_bytes;
  decltype(&sq_lora_workspace_bytes) lora_workspace_bytes;
  decltype(&sq_lora_forward) lora_forward;
  decltype(&sq_lora_backward) lora_backward;
  decltype(&sq_rope_forward) rope_forward;
  decltype(&sq_rope_backward) rope_backward;
  decltype(&sq_group_norm_workspace_bytes) gn_workspace_bytes;
  decltype(&sq_group_norm_forward) gn_forward;
  decltype(&sq_group_norm_backward) gn_backward;
  decltype(&sq_input_grad_workspace_bytes) input_grad_workspace_bytes;
  decltype(&sq_dualscale_seglinear_input_grad) input_grad;
} lib;

// An argument that does not fit: the function returns None.
struct Misfit {};
void need(bool ok) {
  if (!ok) throw Misfit();
}

const Tensor *optional_tensor(PyObject *o) {
  if (o == Py_None) return nullptr;
  need(THPVariable_Check(o));
  return &THPVariable_Unpack(o);
}
const Tensor &tensor(PyObject *o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Misfit();
  }
  return v;
}
float real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Misfit();
  }
  return static_cast<float>(v);
}
int32_t int32_of(PyObject *o) {
  const int64_t v = integer(o);
  need(v >= INT32_MIN && v <= INT32_MAX);
  return static_cast<int32_t>(v);
}
bool truth(PyObject *o) { return PyObject_IsTrue(o) == 1; }

bool plain(const Tensor &t, ScalarType type, int dev) {
  return t.is_cuda() && t.layout() == at::kStrided && t.scalar_type() == type &&
         t.get_device() == dev;
}
// For each tensor that a call will write (absent ones left out), before any
// address is taken: a tensor that shares its storage until the first write (copy
// on write) gets its own now.  Addresses can then be taken as for reading, which
// leaves such inputs shared.
void will_write(std::initializer_list<PyObject *> out) {
  for (PyObject *o : out)
    if (const Tensor *t = optional_tensor(o))
      if (t->is_cuda() && t->layout() == at::kStrided) t->mutable_data_ptr();
}
// The device of the tensor that gives a call its sizes: the current one.
int device_of(const Tensor &t) {
  need(t.is_cuda() && t.get_device() == c10::cuda::current_device());
  return t.get_device();
}
// Address of a contiguous tensor of this type and shape.
void *whole(const Tensor &t, ScalarType type, at::IntArrayRef shape, int dev) {
  need(plain(t, type, dev) && t.sizes() == shape && t.is_contiguous());
  return const_cast<void *>(t.const_data_ptr());
}
// Rows with unit column stride; a single row's stride says nothing.
struct Rows {
  void *p = nullptr;
  int64_t ld = 0;
};
Rows rows_of(const Tensor &t, ScalarType type, int64_t rows, int64_t cols, int dev) {
  need(plain(t, type, dev) && t.dim() == 2 && t.size(0) == rows && t.size(1) == cols);
  need(t.stride(1) == 1 || cols <= 1 || rows == 0);
  const int64_t ld = rows <= 1 ? (cols + 7) / 8 * 8 : t.stride(0);
  return {const_cast<void *>(t.const_data_ptr()), ld};
}
// [B][S][C] whose samples and rows lie at one row stride.
Rows samples_of(const Tensor &t, int64_t B, int64_t S, int64_t C, int dev) {
  need(plain(t, BF16, dev) && t.dim() == 3 && t.size(0) == B && t.size(1) == S && t.size(2) == C);
  void *p = const_cast<void *>(t.const_data_ptr());
  if (B * S <= 1) return {p, (C + 7) / 8 * 8};
  const int64_t ld = S > 1 ? t.stride(1) : t.stride(0);
  need((t.stride(2) == 1 || C == 1) && (B == 1 || S == 1 || t.stride(0) == S * ld));
  return {p, ld};
}
int out_kind(ScalarType type) {
  need(type == BF16 || type == F32);
  return type == BF16 ? SQ_OUT_BF16 : SQ_OUT_F32;
}

Tensor empty(at::IntArrayRef shape, ScalarType type, int dev) {
  return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, dev), c10::nullopt);
}

// The caller's workspace, or memory that is free again when the call returns
// (torch hands it out to later work of the same stream only).
struct Workspace {
  c10::DataPtr own;
  void *p = nullptr;
  size_t n = 0;
  template <typename Size>
  Workspace(PyObject *o, int dev, Size &&size) {
    if (const Tensor *t = optional_tensor(o)) {
      need(plain(*t, at::kByte, dev) && t->is_contiguous());
      p = const_cast<void *>(t->const_data_ptr());
      n = t->numel();
    } else {
      n = size();
      own = c10::cuda::CUDACachingAllocator::get()->allocate(n);
      p = own.get();
    }
  }
};

sq_stream_t stream_on(int dev) {
  return reinterpret_cast<sq_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
}

template <typename F>
sq_status unlocked(F &&f) {
  PyThreadState *state = PyEval_SaveThread();
  const sq_status s = f();
  PyEval_RestoreThread(state);
  return s;
}

PyObject *wrap(const Tensor &t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
PyObject *results(sq_status s, std::initializer_list<Tensor> out) {
  if (s != SQ_OK) return PyLong_FromLong(s);
  PyObject *r = PyTuple_New(static_cast<Py_ssize_t>(out.size()));
  Py_ssize_t i = 0;
  if (r != nullptr)
    for (const Tensor &t : out) {
      PyObject *o = wrap(t);
      if (o == nullptr) {
        Py_DECREF(r);
        return nullptr;
      }
      PyTuple_SET_ITEM(r, i++, o);
    }
  return r;
}

// x, A, B, scale, plan, base, y, t, workspace -> (y, t)
PyObject *lora_forward(PyObject *const *a) {
  will_write({a[6], a[7], a[8]});
  const Tensor &x = tensor(a[0]), &A = tensor(a[1]), &B = tensor(a[2]);
  const Tensor *base = optional_tensor(a[5]), *y_in = optional_tensor(a[6]),
               *t_in = optional_tensor(a[7]);
  const int dev = device_of(x);
  need(x.dim() == 2 && A.dim() == 3 && B.dim() == 3);
  const int64_t M = x.size(0), K = x.size(1), L = A.size(0), R = A.size(1), N = B.size(1);
  need(L <= INT32_MAX && R <= INT32_MAX);
  const ScalarType type = y_in ? y_in->scalar_type() : base ? base->scalar_type() : BF16;
  const sq_out_dtype kind = static_cast<sq_out_dtype>(out_kind(type));
  const Rows px = rows_of(x, BF16, M, K, dev);
  const Rows pb = base ? rows_of(*base, type, M, N, dev) : Rows();
  const void *pA = whole(A, BF16, {L, R, K}, dev), *pB = whole(B, BF16, {L, N, R}, dev);
  const float *scale = static_cast<float *>(whole(tensor(a[3]), F32, {L}, dev));
  const int64_t words = lib.lora_plan_bytes(M, static_cast<int32_t>(L)) / 4;
  const int32_t *plan = static_cast<int32_t *>(whole(tensor(a[4]), I32, {words}, dev));
  const Tensor y = y_in ? *y_in : empty({M, N}, type, dev);
  const Tensor t = t_in ? *t_in : empty({M, R}, F32, dev);
  const Rows py = rows_of(y, type, M, N, dev);
  float *pt = static_cast<float *>(whole(t, F32, {M, R}, dev));
  const int32_t R32 = static_cast<int32_t>(R), L32 = static_cast<int32_t>(L);
  const Workspace ws(a[8], dev, [&] { return lib.lora_workspace_bytes(M, R32, L32, kind); });
  const sq_stream_t stream = stream_on(dev);
  return results(unlocked([&] {
                   return lib.lora_forward(px.p, px.ld, pA, pB, scale, plan, pb.p, pb.ld, py.p,
                                           py.ld, kind, pt, ws.p, ws.n, M, N, K, R32, L32, stream);
                 }),
                 {y, t});
}

// dy, x, t, A, B, scale, plan, dx_base, dx, dA, dB, fp32 gradients, workspace,
// need_dx, need_weights -> (dA, dB, dx)
PyObject *lora_backward(PyObject *const *a) {
  will_write({a[8], a[9], a[10], a[12]});
  const Tensor &dy = tensor(a[0]), &x = tensor(a[1]), &A = tensor(a[3]), &B = tensor(a[4]);
  const Tensor *base = optional_tensor(a[7]), *dx_in = optional_tensor(a[8]),
               *dA_in = optional_tensor(a[9]), *dB_in = optional_tensor(a[10]);
  const bool need_dx = truth(a[13]), need_weights = truth(a[14]);
  need(need_dx || (base == nullptr && dx_in == nullptr));
  need(need_weights || (dA_in == nullptr && dB_in == nullptr));
  const int dev = device_of(dy);
  need(dy.dim() == 2 && A.dim() == 3 && B.dim() == 3);
  const int64_t M = dy.size(0), N = dy.size(1), L = A.size(0), R = A.size(1), K = A.size(2);
  need(L <= INT32_MAX && R <= INT32_MAX);
  const ScalarType type = truth(a[11]) ? F32 : BF16;
  const sq_out_dtype kind = static_cast<sq_out_dtype>(out_kind(type));
  const Rows pdy = rows_of(dy, BF16, M, N, dev), px = rows_of(x, BF16, M, K, dev);
  const Rows pb = base ? rows_of(*base, BF16, M, K, dev) : Rows();
  const void *pA = whole(A, BF16, {L, R, K}, dev), *pB = whole(B, BF16, {L, N, R}, dev);
  const float *pt = static_cast<float *>(whole(tensor(a[2]), F32, {M, R}, dev));
  const float *scale = static_cast<float *>(whole(tensor(a[5]), F32, {L}, dev));
  const int64_t words = lib.lora_plan_bytes(M, static_cast<int32_t>(L)) / 4;
  const int32_t *plan = static_cast<int32_t *>(whole(tensor(a[6]), I32, {words}, dev));
  Tensor dx, dA, dB;
  Rows pdx;
  void *pdA = nullptr, *pdB = nullptr;
  if (need_dx) {
    dx = dx_in ? *dx_in : empty({M, K}, BF16, dev);
    pdx = rows_of(dx, BF16, M, K, dev);
  }
  if (need_weights) {
    dA = dA_in ? *dA_in : empty({L, R, K}, type, dev);
    dB = dB_in ? *dB_in : empty({L, N, R}, type, dev);
    pdA = whole(dA, type, {L, R, K}, dev);
    pdB = whole(dB, type, {L, N, R}, dev);
  }
  const int32_t R32 = static_cast<int32_t>(R), L32 = static_cast<int32_t>(L);
  const Workspace ws(a[12], dev, [&] { return lib.lora_workspace_bytes(M, R32, L32, kind); });
  const sq_stream_t stream = stream_on(dev);
  return results(unlocked([&] {
                   return lib.lora_backward(pdy.p, pdy.ld, px.p, px.ld, pt, pA, pB, scale, plan,
                                            pb.p, pb.ld, pdx.p, pdx.ld, pdA, pdB, kind, ws.p, ws.n,
                                            M, N, K, R32, L32, stream);
                 }),
                 {dA, dB, dx});
}

// backward, x, positions, inv_freq, head_dim, out, layout, axis_pairs, factor -> (out,)
PyObject *rope(PyObject *const *a) {
  will_write({a[5]});
  const Tensor &x = tensor(a[1]), &pos = tensor(a[2]), &inv_freq = tensor(a[3]);
  const Tensor *out_in = optional_tensor(a[5]);
  const int dev = device_of(x);
  need(x.dim() == 2 && inv_freq.dim() == 1);
  const ScalarType type = x.scalar_type();
  const sq_out_dtype kind = static_cast<sq_out_dtype>(out_kind(type));
  const int64_t M = x.size(0), cols = x.size(1), D = integer(a[4]), pairs = inv_freq.size(0);
  need(D >= 1 && cols % D == 0 && D <= INT32_MAX && cols / D <= INT32_MAX && pairs <= 1 << 24);
  int32_t axis_pairs[SQ_ROPE_MAX_AXES], axes = 1;
  const bool split = a[7] != Py_None;
  if (split) {
    need(PyTuple_Check(a[7]) || PyList_Check(a[7]));
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(a[7]);
    need(n >= 1 && n <= SQ_ROPE_MAX_AXES);
    axes = static_cast<int32_t>(n);
    for (Py_ssize_t i = 0; i < n; ++i)
      axis_pairs[i] = int32_of(PySequence_Fast_GET_ITEM(a[7], i));
  }
  const Rows px = rows_of(x, type, M, cols, dev);
  const int32_t *positions = static_cast<int32_t *>(
      pos.dim() == 1 && axes == 1 ? whole(pos, I32, {M}, dev) : whole(pos, I32, {M, axes}, dev));
  const float *freq = static_cast<float *>(whole(inv_freq, F32, {pairs}, dev));
  const sq_rope_layout layout = static_cast<sq_rope_layout>(int32_of(a[6]));
  const float factor = real(a[8]);
  const Tensor out = out_in ? *out_in : empty({M, cols}, type, dev);
  const Rows po = rows_of(out, type, M, cols, dev);
  const auto call = truth(a[0]) ? lib.rope_backward : lib.rope_forward;
  const sq_stream_t stream = stream_on(dev);
  return results(unlocked([&] {
                   return call(px.p, px.ld, po.p, po.ld, kind, positions, freq,
                               split ? axis_pairs : nullptr, axes, factor, M,
                               static_cast<int32_t>(cols / D), static_cast<int32_t>(D),
                               static_cast<int32_t>(2 * pairs), layout, stream);
                 }),
                 {out});
}

// x, groups, gamma, beta, eps, act, y, workspace -> (y, mean, rstd)
PyObject *group_norm_forward(PyObject *const *a) {
  will_write({a[6], a[7]});
  const Tensor &x = tensor(a[0]);
  const Tensor *gamma = optional_tensor(a[2]), *beta = optional_tensor(a[3]),
               *y_in = optional_tensor(a[6]);
  const int dev = device_of(x);
  need(x.dim() == 3);
  const int64_t B = x.size(0), S = x.size(1), C = x.size(2), G = integer(a[1]);
  need(G >= 0 && G <= C);
  const Rows px = samples_of(x, B, S, C, dev);
  const void *pg = gamma ? whole(*gamma, BF16, {C}, dev) : nullptr;
  const void *pb = beta ? whole(*beta, BF16, {C}, dev) : nullptr;
  const float eps = real(a[4]);
  const sq_activation act = static_cast<sq_activation>(int32_of(a[5]));
  const Tensor y = y_in ? *y_in : empty({B, S, C}, BF16, dev);
  const Rows py = samples_of(y, B, S, C, dev);
  const Tensor mean = empty({B, G}, F32, dev), rstd = empty({B, G}, F32, dev);
  const Workspace ws(a[7], dev, [&] { return lib.gn_workspace_bytes(B, S, C, G); });
  float *pm = static_cast<float *>(mean.data_ptr()), *pr = static_cast<float *>(rstd.data_ptr());
  const sq_stream_t stream = stream_on(dev);
  return results(unlocked([&] {
                   return lib.gn_forward(px.p, px.ld, B, S, C, G, pg, pb, eps, act, py.p, py.ld, pm,
                                         pr, ws.p, ws.n, stream);
                 }),
                 {y, mean, rstd});
}

// dy, x, groups, gamma, beta, mean, rstd, act, dx, fp32 gradients, workspace,
// need_dx -> (dx, dgamma, dbeta)
PyObject *group_norm_backward(PyObject *const *a) {
  will_write({a[8], a[10]});
  const Tensor &dy = tensor(a[0]), &x = tensor(a[1]);
  const Tensor *gamma = optional_tensor(a[3]), *beta = optional_tensor(a[4]),
               *dx_in = optional_tensor(a[8]);
  const bool need_dx = truth(a[11]);
  need(need_dx || dx_in == nullptr);
  const int dev = device_of(x);
  need(x.dim() == 3);
  const int64_t B = x.size(0), S = x.size(1), C = x.size(2), G = integer(a[2]);
  const ScalarType type = truth(a[9]) ? F32 : BF16;
  const sq_out_dtype kind = static_cast<sq_out_dtype>(out_kind(type));
  const Rows pdy = samples_of(dy, B, S, C, dev), px = samples_of(x, B, S, C, dev);
  const void *pg = gamma ? whole(*gamma, BF16, {C}, dev) : nullptr;
  const void *pb = beta ? whole(*beta, BF16, {C}, dev) : nullptr;
  const float *mean = static_cast<float *>(whole(tensor(a[5]), F32, {B, G}, dev));
  const float *rstd = static_cast<float *>(whole(tensor(a[6]), F32, {B, G}, dev));
  const sq_activation act = static_cast<sq_activation>(int32_of(a[7]));
  Tensor dx, dgamma, dbeta;
  Rows pdx;
  if (need_dx) {
    dx = dx_in ? *dx_in : empty({B, S, C}, BF16, dev);
    pdx = samples_of(dx, B, S, C, dev);
  }
  if (gamma) dgamma = empty({C}, type, dev);
  if (beta) dbeta = empty({C}, type, dev);
  const Workspace ws(a[10], dev, [&] { return lib.gn_workspace_bytes(B, S, C, G); });
  void *pdg = gamma ? dgamma.data_ptr() : nullptr, *pdb = beta ? dbeta.data_ptr() : nullptr;
  const sq_stream_t stream = stream_on(dev);
  return results(unlocked([&] {
                   return lib.gn_backward(pdy.p, pdy.ld, px.p, px.ld, B, S, C, G, pg, pb, mean,
                                          rstd, act, pdx.p, pdx.ld, pdg, pdb, kind, ws.p, ws.n,
                                          stream);
                 }),
                 {dx, dgamma, dbeta});
}

// dy, wq, s_w, d, address of the segment table, its groups, its rows of steps, dx,
// workspace -> (dx,)
PyObject *input_grad(PyObject *const *a) {
  will_write({a[7], a[8]});
  const Tensor &dy = tensor(a[0]), &wq = tensor(a[1]);
  const Tensor *d = optional_tensor(a[3]), *dx_in = optional_tensor(a[7]);
  const int dev = device_of(dy);
  need(dy.dim() == 2 && wq.dim() == 2);
  const int64_t M = dy.size(0), N = dy.size(1), K = wq.size(1);
  const sq_segments *seg = static_cast<sq_segments *>(PyLong_AsVoidPtr(a[4]));
  const int64_t G = integer(a[5]), S = integer(a[6]);
  const Rows pdy = rows_of(dy, BF16, M, N, dev);
  const int8_t *pw = static_cast<int8_t *>(whole(wq, I8, {N, K}, dev));
  const float *s_w = static_cast<float *>(whole(tensor(a[2]), F32, {S, N}, dev));
  const float *pd = d ? static_cast<float *>(whole(*d, F32, {G, K}, dev)) : nullptr;
  const Tensor dx = dx_in ? *dx_in : empty({M, K}, BF16, dev);
  const Rows pdx = rows_of(dx, BF16, M, K, dev);
  const Workspace ws(a[8], dev, [&] { return lib.input_grad_workspace_bytes(N, K); });
  const sq_stream_t stream = stream_on(dev);
  return results(unlocked([&] {
                   return lib.input_grad(pdy.p, pdy.ld, pw, s_w, pd, seg, pdx.p, pdx.ld, M, N, K,
                                         ws.p, ws.n, stream);
                 }),
                 {dx});
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N || lib.input_grad == nullptr) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or no library");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Misfit &) {
    Py_RETURN_NONE;
  }
  END_HANDLE_TH_ERRORS
}

template <typename T>
bool find(void *handle, const char *name, T &to) {
  to = reinterpret_cast<T>(dlsym(handle, name));
  if (to == nullptr) PyErr_Format(PyExc_RuntimeError, "the library has no %s", name);
  return to != nullptr;
}

PyObject *init(PyObject *, PyObject *handle) {
  void *h = PyLong_AsVoidPtr(handle);
  if (h == nullptr && PyErr_Occurred()) return nullptr;
  if (find(h, "sq_lora_plan_bytes", lib.lora_plan_bytes) &&
      find(h, "sq_lora_workspace_bytes", lib.lora_workspace_bytes) &&
      find(h, "sq_lora_forward", lib.lora_forward) &&
      find(h, "sq_lora_backward", lib.lora_backward) &&
      find(h, "sq_rope_forward", lib.rope_forward) &&
      find(h, "sq_rope_backward", lib.rope_backward) &&
      find(h, "sq_group_norm_workspace_bytes", lib.gn_workspace_bytes) &&
      find(h, "sq_group_norm_forward", lib.gn_forward) &&
      find(h, "sq_group_norm_backward", lib.gn_backward) &&
      find(h, "sq_input_grad_workspace_bytes", lib.input_grad_workspace_bytes) &&
      find(h, "sq_dualscale_seglinear_input_grad", lib.input_grad))
    Py_RETURN_NONE;
  return nullptr;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<F, N>)), METH_FASTCALL,
          nullptr};
}

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_sqtorch", nullptr, -1, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sqtorch() {
  static PyMethodDef methods[] = {
      {"init", init, METH_O, nullptr},
      method<lora_forward, 9>("lora_forward"),
      method<lora_backward, 15>("lora_backward"),
      method<rope, 9>("rope"),
      method<group_norm_forward, 8>("group_norm_forward"),
      method<group_norm_backward, 12>("group_norm_backward"),
      method<input_grad, 9>("input_grad"),
      {nullptr, nullptr, 0, nullptr}};
  module_def.m_methods = methods;
  return PyModule_Create(&module_def);
}
