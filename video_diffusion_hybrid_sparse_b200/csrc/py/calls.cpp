// calls.cpp - the binding's calls of the causal linear memory and of the
// residual RMSNorm, from tensor objects to the C ABI in one step.
//
// The smallest of these calls run for 4 us on the device; reading shapes,
// strides and pointers of eight tensors in Python and filling the config takes
// longer than that.  A call is made here only where nothing is out of the
// ordinary: plain CUDA tensors of the current device with the expected shapes
// and types, on the current stream.  Everything else returns None, and the
// binding's Python does the checks, with their messages, and the call.
//
// Results: the output (or a tuple of outputs); an int, a status code other than
// VDN_OK of the C ABI; or None (not made here).
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "vdnattn.h"

namespace {

using at::Tensor;

// A positional argument that is a tensor, or None where `optional`.
struct Arg {
  bool ok = false;          // as expected so far
  const Tensor* t = nullptr;  // null: None
  Arg(PyObject* o, bool optional) {
    if (o == Py_None) {
      ok = optional;
    } else if (THPVariable_CheckExact(o)) {
      t = &THPVariable_Unpack(o);
      ok = t->is_cuda() && t->layout() == at::kStrided && !t->is_conj() && !t->is_neg();
    }
  }
  void* ptr() const { return t ? t->data_ptr() : nullptr; }
};

bool alike(const Tensor& a, const Tensor& like) {
  return a.sizes() == like.sizes() && a.scalar_type() == like.scalar_type() && a.device() == like.device();
}

int dtype_of(const Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? VDN_BF16 : t.scalar_type() == at::kFloat ? VDN_FP32 : -1;
}

// The tensors' device is the current one.
bool here(const Tensor& t) { return t.device().index() == c10::cuda::current_device(); }
void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

bool vector(const Arg& a, int64_t n, at::ScalarType type, const Tensor& like) {
  return a.ok && (!a.t || (a.t->dim() == 1 && a.t->size(0) == n && a.t->scalar_type() == type &&
                           a.t->device() == like.device() && a.t->is_contiguous()));
}

// [B, N, H, d] or (a step's) [B, H, d] like `like`, with contiguous rows
bool view(const Arg& a, const Tensor& like, vdn_view* v) {
  if (!a.ok || !a.t || !alike(*a.t, like)) return false;
  const auto s = a.t->strides();
  const size_t n = s.size();
  if (s[n - 1] != 1) return false;
  *v = n == 4 ? vdn_view{a.t->data_ptr(), s[0], s[1], s[2]} : vdn_view{a.t->data_ptr(), s[0], 0, s[1]};
  return true;
}

// [n, H, d, d] fp32 states, each contiguous and none on another
bool states(const Arg& a, int64_t n, int64_t H, int64_t d, const Tensor& like, float** p, int64_t* stride) {
  *p = nullptr;
  *stride = 0;
  if (!a.ok) return false;
  if (!a.t) return true;
  const Tensor& t = *a.t;
  if (t.dim() != 4 || t.size(0) != n || t.size(1) != H || t.size(2) != d || t.size(3) != d ||
      t.scalar_type() != at::kFloat || t.device() != like.device())
    return false;
  if (t.stride(3) != 1 || t.stride(2) != d || (H > 1 && t.stride(1) != d * d)) return false;
  if (n > 1 && t.stride(0) < H * d * d) return false;
  *p = static_cast<float*>(t.data_ptr());
  *stride = n > 1 ? t.stride(0) : 0;
  return true;
}

Tensor new_like(const Tensor& t) { return at::empty_like(t, t.options(), at::MemoryFormat::Contiguous); }
Tensor scratch(size_t n, const Tensor& like) { return at::empty({(int64_t)n}, like.options().dtype(at::kByte)); }

// [B, N, H, d] (dims 4) or [B, H, d] into cfg
bool sizes(const Arg& q, int dims, vdn_linear_cfg* c) {
  if (!q.ok || !q.t || q.t->dim() != dims || !here(*q.t)) return false;
  c->dtype = dtype_of(*q.t);
  const auto s = q.t->sizes();
  for (int i = 0; i < dims; ++i)
    if (s[i] > INT32_MAX) return false;
  c->batch = (int32_t)s[0];
  c->tokens = dims == 4 ? (int32_t)s[1] : 0;
  c->heads = (int32_t)s[dims - 2];
  c->head_dim = (int32_t)s[dims - 1];
  return c->dtype >= 0 && q.t->numel() > 0;
}

PyObject* none() { Py_RETURN_NONE; }

// Other Python threads go on while this one allocates and launches (a full launch queue makes it wait for the device).
class Released {
 public:
  Released() : state_(PyEval_SaveThread()) {}
  ~Released() { PyEval_RestoreThread(state_); }
  Released(const Released&) = delete;
  Released& operator=(const Released&) = delete;

 private:
  PyThreadState* state_;
};

// q, k, v, log_decay, scale, state_in, state_out, lengths, out, status, debug_flags
PyObject* linear_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 11) return none();
  const Arg q(a[0], false), k(a[1], false), v(a[2], false), ld(a[3], false), s_in(a[5], true), s_out(a[6], true),
      lengths(a[7], true), status(a[9], true);
  vdn_linear_cfg c = {};
  vdn_view x[4];
  if (!sizes(q, 4, &c) || !view(q, *q.t, &x[0]) || !view(k, *q.t, &x[1]) || !view(v, *q.t, &x[2])) return none();
  const Arg out(a[8], true);
  if (!out.ok || (out.t && !view(out, *q.t, &x[3]))) return none();
  if (!vector(ld, c.heads, at::kFloat, *q.t) || !vector(lengths, c.batch, at::kInt, *q.t) || !vector(status, 1, at::kInt, *q.t) ||
      !states(s_in, c.batch, c.heads, c.head_dim, *q.t, const_cast<float**>(&c.state_in), &c.state_in_stride) ||
      !states(s_out, c.batch, c.heads, c.head_dim, *q.t, &c.state_out, &c.state_out_stride))
    return none();
  c.scale = (float)PyFloat_AsDouble(a[4]);
  c.debug_flags = (int32_t)PyLong_AsLong(a[10]);
  if (PyErr_Occurred()) return nullptr;
  c.log_decay = static_cast<const float*>(ld.ptr());
  c.lengths = static_cast<const int32_t*>(lengths.ptr());
  c.status_word = static_cast<int32_t*>(status.ptr());
  c.workspace_bytes = vdn_linear_workspace_bytes(&c, 0);
  if (c.workspace_bytes == 0) return none();
  Tensor made;
  vdn_status r;
  {
    Released others;
    const Tensor ws = scratch(c.workspace_bytes, *q.t);
    made = out.t ? *out.t : new_like(*q.t);
    c.workspace = ws.data_ptr();
    if (!out.t) x[3] = vdn_view{made.data_ptr(), made.stride(0), made.stride(1), made.stride(2)};
    r = vdn_linear_attn_fwd(&x[0], &x[1], &x[2], &x[3], &c, stream_of(*q.t));
  }
  return r == VDN_OK ? THPVariable_Wrap(made) : PyLong_FromLong(r);
  END_HANDLE_TH_ERRORS
}

// q, k, v, log_decay, d_out, scale, state_in, d_state_out, d_state_in, lengths, dq, dk, dv, status, debug_flags
PyObject* linear_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 15) return none();
  const Arg q(a[0], false), k(a[1], false), v(a[2], false), ld(a[3], false), d_out(a[4], false), s_in(a[6], true),
      ds_out(a[7], true), ds_in(a[8], true), lengths(a[9], true), status(a[13], true);
  const Arg g[3] = {Arg(a[10], true), Arg(a[11], true), Arg(a[12], true)};
  vdn_linear_cfg c = {};
  vdn_view x[7];
  if (!sizes(q, 4, &c) || !view(q, *q.t, &x[0]) || !view(k, *q.t, &x[1]) || !view(v, *q.t, &x[2]) || !view(d_out, *q.t, &x[3]))
    return none();
  for (int i = 0; i < 3; ++i)
    if (!g[i].ok || (g[i].t && !view(g[i], *q.t, &x[4 + i]))) return none();
  if (!vector(ld, c.heads, at::kFloat, *q.t) || !vector(lengths, c.batch, at::kInt, *q.t) || !vector(status, 1, at::kInt, *q.t) ||
      !states(s_in, c.batch, c.heads, c.head_dim, *q.t, const_cast<float**>(&c.state_in), &c.state_in_stride) ||
      !states(ds_out, c.batch, c.heads, c.head_dim, *q.t, const_cast<float**>(&c.d_state_out), &c.d_state_out_stride) ||
      !states(ds_in, c.batch, c.heads, c.head_dim, *q.t, &c.d_state_in, &c.d_state_in_stride))
    return none();
  c.scale = (float)PyFloat_AsDouble(a[5]);
  c.debug_flags = (int32_t)PyLong_AsLong(a[14]);
  if (PyErr_Occurred()) return nullptr;
  c.log_decay = static_cast<const float*>(ld.ptr());
  c.lengths = static_cast<const int32_t*>(lengths.ptr());
  c.status_word = static_cast<int32_t*>(status.ptr());
  c.workspace_bytes = vdn_linear_workspace_bytes(&c, 1);
  if (c.workspace_bytes == 0) return none();
  Tensor made[3];
  vdn_status r;
  {
    Released others;
    const Tensor ws = scratch(c.workspace_bytes, *q.t);
    c.workspace = ws.data_ptr();
    for (int i = 0; i < 3; ++i) {
      made[i] = g[i].t ? *g[i].t : new_like(*q.t);
      if (!g[i].t) x[4 + i] = vdn_view{made[i].data_ptr(), made[i].stride(0), made[i].stride(1), made[i].stride(2)};
    }
    r = vdn_linear_attn_bwd(&x[0], &x[1], &x[2], &x[3], &x[4], &x[5], &x[6], &c, stream_of(*q.t));
  }
  if (r != VDN_OK) return PyLong_FromLong(r);
  return Py_BuildValue("(NNN)", THPVariable_Wrap(made[0]), THPVariable_Wrap(made[1]), THPVariable_Wrap(made[2]));
  END_HANDLE_TH_ERRORS
}

// q, k, v, log_decay, state, slots, scale, out, status
PyObject* linear_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) return none();
  const Arg q(a[0], false), k(a[1], false), v(a[2], false), ld(a[3], false), pool(a[4], false), slots(a[5], true),
      out(a[7], true), status(a[8], true);
  vdn_linear_cfg c = {};
  vdn_view x[4];
  if (!sizes(q, 3, &c) || !view(q, *q.t, &x[0]) || !view(k, *q.t, &x[1]) || !view(v, *q.t, &x[2])) return none();
  if (!out.ok || (out.t && !view(out, *q.t, &x[3]))) return none();
  if (!pool.ok || pool.t->dim() != 4 || pool.t->size(0) > INT32_MAX ||
      !states(pool, pool.t->size(0), c.heads, c.head_dim, *q.t, &c.state_out, &c.state_out_stride) ||
      !vector(ld, c.heads, at::kFloat, *q.t) || !vector(slots, c.batch, at::kInt, *q.t) || !vector(status, 1, at::kInt, *q.t))
    return none();
  c.scale = (float)PyFloat_AsDouble(a[6]);
  if (PyErr_Occurred()) return nullptr;
  c.log_decay = static_cast<const float*>(ld.ptr());
  c.slots = static_cast<const int32_t*>(slots.ptr());
  c.n_slots = (int32_t)pool.t->size(0);
  c.status_word = static_cast<int32_t*>(status.ptr());
  Tensor made;
  vdn_status r;
  {
    Released others;
    made = out.t ? *out.t : new_like(*q.t);
    if (!out.t) x[3] = vdn_view{made.data_ptr(), made.stride(0), 0, made.stride(1)};
    r = vdn_linear_attn_step(&x[0], &x[1], &x[2], &x[3], &c, stream_of(*q.t));
  }
  return r == VDN_OK ? THPVariable_Wrap(made) : PyLong_FromLong(r);
  END_HANDLE_TH_ERRORS
}

// a [rows, W] tensor of `type` like x; its row stride (0 where there is one row)
bool matrix(const Arg& a, const Tensor& x, at::ScalarType type, int64_t* stride) {
  *stride = 0;
  if (!a.ok) return false;
  if (!a.t) return true;
  const Tensor& t = *a.t;
  if (t.sizes() != x.sizes() || t.scalar_type() != type || t.device() != x.device()) return false;
  if (t.stride(1) != 1 && t.size(1) != 1) return false;
  if (t.size(0) > 1) {
    if (t.stride(0) < t.size(1)) return false;
    *stride = t.stride(0);
  }
  return true;
}

bool norm_sizes(const Arg& x, const Arg& weight, PyObject* eps, vdn_norm_cfg* c) {
  if (!x.ok || !x.t || x.t->dim() != 2 || x.t->numel() == 0 || x.t->size(1) > INT32_MAX || !here(*x.t)) return false;
  c->dtype = dtype_of(*x.t);
  c->rows = x.t->size(0);
  c->width = (int32_t)x.t->size(1);
  c->eps = (float)PyFloat_AsDouble(eps);
  c->weight = static_cast<const float*>(weight.ptr());
  return c->dtype >= 0 && vector(weight, c->width, at::kFloat, *x.t);
}

// x, weight, residual, residual_out, eps, out_mode, out, scales
PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) return none();
  const Arg x(a[0], false), weight(a[1], true), res(a[2], true), res_out(a[3], true), out(a[6], true), scales(a[7], true);
  vdn_norm_cfg c = {};
  c.output = (int32_t)PyLong_AsLong(a[5]);
  const bool fits = norm_sizes(x, weight, a[4], &c);
  if (PyErr_Occurred()) return nullptr;
  if (!fits || c.output < VDN_NORM_TENSOR || c.output > VDN_NORM_E4M3_GROUP) return none();
  const bool quant = c.output != VDN_NORM_TENSOR;
  const at::ScalarType kind = quant ? at::kFloat8_e4m3fn : x.t->scalar_type();
  if (!matrix(x, *x.t, x.t->scalar_type(), &c.x_stride) || !matrix(res, *x.t, x.t->scalar_type(), &c.residual_stride) ||
      !matrix(res_out, *x.t, x.t->scalar_type(), &c.residual_out_stride) || !matrix(out, *x.t, kind, &c.out_stride))
    return none();
  Tensor s, made;
  int64_t groups = 0;
  if (quant) {
    groups = c.output == VDN_NORM_E4M3_ROW ? 1 : (c.width + 127) / 128;
    if (!scales.ok) return none();
    if (scales.t) {
      s = *scales.t;
      if (s.dim() != 2 || s.size(0) != c.rows || s.size(1) != groups || s.scalar_type() != at::kFloat ||
          s.device() != x.t->device() || !s.is_contiguous())
        return none();
    }
  }
  vdn_status r;
  {
    Released others;
    if (quant && !scales.t) s = at::empty({c.rows, groups}, x.t->options().dtype(at::kFloat));
    made = out.t ? *out.t : at::empty(x.t->sizes(), x.t->options().dtype(kind));
    r = vdn_add_rmsnorm_fwd(x.ptr(), res.ptr(), res_out.ptr(), made.data_ptr(),
                            quant ? static_cast<float*>(s.data_ptr()) : nullptr, &c, stream_of(*x.t));
  }
  if (r != VDN_OK) return PyLong_FromLong(r);
  return quant ? Py_BuildValue("(NN)", THPVariable_Wrap(made), THPVariable_Wrap(s)) : THPVariable_Wrap(made);
  END_HANDLE_TH_ERRORS
}

// h, weight, dy, dh, eps, dx, dweight, want_dweight
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) return none();
  const Arg h(a[0], false), weight(a[1], true), dy(a[2], false), dh(a[3], true), dx(a[5], true), dweight(a[6], true);
  vdn_norm_cfg c = {};
  const bool fits = norm_sizes(h, weight, a[4], &c);
  const int want = PyObject_IsTrue(a[7]);
  if (PyErr_Occurred()) return nullptr;
  if (!fits) return none();
  const at::ScalarType type = h.t->scalar_type();
  if (!matrix(h, *h.t, type, &c.x_stride) || !matrix(dy, *h.t, type, &c.dy_stride) || !matrix(dh, *h.t, type, &c.dh_stride) ||
      !matrix(dx, *h.t, type, &c.dx_stride) || !vector(dweight, c.width, at::kFloat, *h.t))
    return none();
  if (want && (c.workspace_bytes = vdn_norm_workspace_bytes(&c)) == 0) return none();
  Tensor made, w;
  vdn_status r;
  {
    Released others;
    Tensor ws;
    if (want) {
      ws = scratch(c.workspace_bytes, *h.t);
      c.workspace = ws.data_ptr();
      w = dweight.t ? *dweight.t : at::empty({c.width}, h.t->options().dtype(at::kFloat));
    }
    made = dx.t ? *dx.t : new_like(*h.t);
    r = vdn_add_rmsnorm_bwd(h.ptr(), dy.ptr(), dh.ptr(), made.data_ptr(), want ? static_cast<float*>(w.data_ptr()) : nullptr,
                            &c, stream_of(*h.t));
  }
  if (r != VDN_OK) return PyLong_FromLong(r);
  if (want) return Py_BuildValue("(NN)", THPVariable_Wrap(made), THPVariable_Wrap(w));
  return Py_BuildValue("(NO)", THPVariable_Wrap(made), Py_None);
  END_HANDLE_TH_ERRORS
}

#define VDN_CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {VDN_CALL(linear_fwd), VDN_CALL(linear_bwd), VDN_CALL(linear_step), VDN_CALL(norm_fwd),
                         VDN_CALL(norm_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  // the torch it was built with, which the binding compares
  if (m && PyModule_AddStringConstant(m, "torch_version", VDN_TORCH) != 0) Py_CLEAR(m);
  return m;
}
