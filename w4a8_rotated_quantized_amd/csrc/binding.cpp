// CPython side of the microscaled 4-bit linear, of layer norm and of the
// optimizer step: checks of tensor arguments, allocation of outputs, and the call
// into the C ABI. The Python functions in __init__.py wrap these with their
// signatures; here arguments are positional. A call that the library refuses returns its
// status as an int; wrong tensors raise ValueError. The last argument is the stream's
// handle, or None for the current stream of the tensors' GPU; NotImplemented comes back
// where that GPU is not the current one.
//
// Why native: the small sizes of these operators are bound by the host. Checking and
// allocating in Python through ctypes took 12.4 us for a layer norm of 77 rows,
// 3 us of it the launch, while the kernel takes 4.
#include <Python.h>
#include <unistd.h>

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <c10/util/SmallVector.h>

#include <cstdio>
#include <cstring>
#include <vector>

#include "../../include/convrot.h"

namespace {

using at::ScalarType;
using at::Tensor;

// What a check throws; turned into ValueError.
struct Wrong {
  char text[240];
};
template <typename... A>
[[noreturn]] void wrong(const char* format, A... a) {
  Wrong w;
  std::snprintf(w.text, sizeof w.text, format, a...);
  throw w;
}
[[noreturn]] void wrong(const char* text) { wrong("%s", text); }

const char* type_name(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Byte: return "torch.uint8";
    default: return "torch.int8";
  }
}

const Tensor* tensor_or_none(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) wrong("%s must be a tensor", what);
  return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* what) {
  const Tensor* t = tensor_or_none(o, what);
  if (!t) wrong("%s must be a tensor", what);
  return *t;
}

int gpu_of(const Tensor& t, const char* what) {
  if (!t.is_cuda()) wrong("%s must be on the GPU", what);
  return (int)t.get_device();
}

bool on(const Tensor& t, int index) { return t.is_cuda() && (int)t.get_device() == index; }

// A dense tensor of the given type and sizes: its address.
void* dense(const Tensor& t, const char* what, ScalarType type, int index, at::IntArrayRef sizes) {
  if (t.scalar_type() != type || !on(t, index) || t.sizes() != sizes || !t.is_contiguous()) {
    char shape[80] = "";
    int at = 0;
    for (int64_t s : sizes) at += std::snprintf(shape + at, sizeof shape - (size_t)at, at ? ", %lld" : "%lld", (long long)s);
    wrong("%s must be a contiguous %s tensor of shape (%s) on GPU %d", what, type_name(type), shape, index);
  }
  return t.data_ptr();
}
void* dense_or_null(const Tensor* t, const char* what, ScalarType type, int index, at::IntArrayRef sizes) {
  return t ? dense(*t, what, type, index, sizes) : nullptr;
}

// [rows, cols] whose rows may lie further apart: address, and the leading dimension
void* spaced(const Tensor& t, const char* what, ScalarType type, int index, int64_t rows, int64_t cols, int64_t* ld) {
  if (t.scalar_type() != type || !on(t, index) || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    wrong("%s must be a %s [%lld, %lld] tensor on GPU %d", what, type_name(type), (long long)rows, (long long)cols, index);
  if (cols > 1 && t.stride(1) != 1) wrong("%s must have contiguous rows", what);
  *ld = rows > 1 ? t.stride(0) : cols;
  return t.data_ptr();
}

Tensor empty(at::IntArrayRef sizes, ScalarType type, const Tensor& like) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
}

int64_t whole(PyObject* o) {
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
// an argument of the C ABI that is an int: what does not fit is refused there
int small(PyObject* o) {
  const int64_t v = whole(o);
  return v < -1 || v > (1 << 20) ? -1 : (int)v;
}
// the stream that a call runs on; false: the current GPU is another one
bool stream_for(PyObject* o, int index, hipStream_t* s) {
  if (o == Py_None) {
    if (c10::hip::current_device() != index) return false;
    *s = c10::hip::getCurrentHIPStream((c10::DeviceIndex)index).stream();
    return true;
  }
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw python_error();
  *s = static_cast<hipStream_t>(p);
  return true;
}
PyObject* elsewhere() {
  Py_INCREF(Py_NotImplemented);
  return Py_NotImplemented;
}

ScalarType out_dtype(int out_type) {
  if (out_type != CR_OUT_BF16 && out_type != CR_OUT_F32) wrong("the output type is OUT.BF16 or OUT.F32");
  return out_type == CR_OUT_F32 ? ScalarType::Float : ScalarType::BFloat16;
}
cr_out float_type(const Tensor& t, const char* what) {
  if (t.scalar_type() == ScalarType::BFloat16) return CR_OUT_BF16;
  if (t.scalar_type() == ScalarType::Float) return CR_OUT_F32;
  wrong("%s must be bfloat16 or float32", what);
}

PyObject* pack(std::initializer_list<const Tensor*> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) {
    PyObject* o;
    if (t) {
      o = THPVariable_Wrap(*t);
    } else {
      o = Py_None;
      Py_INCREF(o);
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}
PyObject* refused(cr_status st) { return PyLong_FromLong((long)st); }

// A given tensor that a call has written: its version changes, so that autograd refuses a backward
// pass that needs what it held before. Tensors of inference mode have none.
void written(const Tensor* t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}
// a call that enqueued something, all of it or (with a launch that failed) a part
bool ran(cr_status st) { return st == CR_OK || st == CR_ERR_HIP; }

// Without the interpreter's lock: outputs are allocated and the call is launched, either of
// which may wait for the GPU, and so for what another thread of the interpreter does. Between
// this and its end nothing of Python's is touched.
struct Unlocked {
  PyThreadState* thread = PyEval_SaveThread();
  Unlocked() = default;
  // An interpreter that has ended meanwhile unwinds the thread instead of returning to it. What the call holds
  // is not to be given back then, so the thread waits here for the end of the process.
  ~Unlocked() {
    try {
      PyEval_RestoreThread(thread);
    } catch (...) {
      for (;;) pause();
    }
  }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;
};

// Every entry runs inside this: Wrong -> ValueError, torch's errors as torch turns them.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Wrong& w) {
    PyErr_SetString(PyExc_ValueError, w.text);
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
// the microscaled 4-bit linear
// ---------------------------------------------------------------------------
// x, rot_group, codes, scales, stream
PyObject* mx_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const Tensor& x = tensor(a[0], "x");
    const int index = gpu_of(x, "x");
    hipStream_t stream;
    if (!stream_for(a[4], index, &stream)) return elsewhere();
    if (x.dim() != 2) wrong("x is [rows, K]");
    const int64_t rows = x.size(0), K = x.size(1), tiles = (K + 127) / 128;
    int64_t ldx;
    const void* px = spaced(x, "x", ScalarType::BFloat16, index, rows, K, &ldx);
    const Tensor *gc = tensor_or_none(a[2], "codes"), *gs = tensor_or_none(a[3], "scales");
    dense_or_null(gc, "codes", ScalarType::Byte, index, {tiles, rows, 64});
    dense_or_null(gs, "scales", ScalarType::Byte, index, {tiles, rows, 4});
    const int rot_group = small(a[1]);
    Tensor codes, scales;
    cr_status st;
    {
      const Unlocked free;
      codes = gc ? *gc : empty({tiles, rows, 64}, ScalarType::Byte, x);
      scales = gs ? *gs : empty({tiles, rows, 4}, ScalarType::Byte, x);
      st = mxfp4_quantize(px, ldx, rows, K, rot_group, codes.data_ptr(), scales.data_ptr(), stream);
    }
    if (ran(st))
      for (const Tensor* t : {gc, gs}) written(t);
    return st ? refused(st) : pack({&codes, &scales});
  });
}

struct MxPair {
  int64_t tiles, rows;
  void *codes, *scales;
};
MxPair mx_pair(const Tensor& codes, const Tensor& scales, const char* what, int index) {
  char name[32];
  if (codes.dim() != 3 || codes.size(2) != 64) wrong("%s codes are uint8 [ceil(K/128), rows, 64]", what);
  MxPair p;
  p.tiles = codes.size(0);
  p.rows = codes.size(1);
  std::snprintf(name, sizeof name, "%s codes", what);
  p.codes = dense(codes, name, ScalarType::Byte, index, {p.tiles, p.rows, 64});
  std::snprintf(name, sizeof name, "%s scales", what);
  p.scales = dense(scales, name, ScalarType::Byte, index, {p.tiles, p.rows, 4});
  return p;
}

// codes, scales, K, rot_group, out_type, out, stream
PyObject* mx_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const Tensor& codes = tensor(a[0], "codes");
    const int index = gpu_of(codes, "codes");
    hipStream_t stream;
    if (!stream_for(a[6], index, &stream)) return elsewhere();
    const MxPair p = mx_pair(codes, tensor(a[1], "scales"), "the", index);
    const int64_t K = whole(a[2]);
    if (K < 0 || K > p.tiles * 128 || p.tiles != (K + 127) / 128) wrong("K does not fit the codes' tiles");
    const int rot_group = small(a[3]), type = small(a[4]);
    const ScalarType dt = out_dtype(type);
    const Tensor* go = tensor_or_none(a[5], "out");
    int64_t ldo = K;
    if (go) spaced(*go, "out", dt, index, p.rows, K, &ldo);
    Tensor out;
    cr_status st;
    {
      const Unlocked free;
      out = go ? *go : empty({p.rows, K}, dt, codes);
      st = mxfp4_dequantize(p.codes, p.scales, p.rows, K, rot_group, out.data_ptr(), (cr_out)type, ldo, stream);
    }
    if (ran(st)) written(go);
    return st ? refused(st) : THPVariable_Wrap(out);
  });
}

// a_codes, a_scales, w_codes, w_scales, bias, out_type, out, stream
PyObject* mx_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const Tensor& ac = tensor(a[0], "a_codes");
    const int index = gpu_of(ac, "a_codes");
    hipStream_t stream;
    if (!stream_for(a[7], index, &stream)) return elsewhere();
    const MxPair p = mx_pair(ac, tensor(a[1], "a_scales"), "a", index);
    const MxPair w = mx_pair(tensor(a[2], "w_codes"), tensor(a[3], "w_scales"), "w", index);
    if (p.tiles != w.tiles) wrong("a and w have different K");
    const void* pb = dense_or_null(tensor_or_none(a[4], "bias"), "bias", ScalarType::BFloat16, index, {w.rows});
    const int type = small(a[5]);
    const ScalarType dt = out_dtype(type);
    const Tensor* go = tensor_or_none(a[6], "out");
    int64_t ldc = w.rows;
    if (go) spaced(*go, "out", dt, index, p.rows, w.rows, &ldc);
    Tensor out;
    cr_status st;
    {
      const Unlocked free;
      out = go ? *go : empty({p.rows, w.rows}, dt, ac);
      st = mxfp4_gemm(p.codes, p.scales, w.codes, w.scales, pb, out.data_ptr(), (cr_out)type, ldc, p.rows, w.rows, p.tiles * 128,
                      stream);
    }
    if (ran(st)) written(go);
    return st ? refused(st) : THPVariable_Wrap(out);
  });
}

// ---------------------------------------------------------------------------
// layer norm
// ---------------------------------------------------------------------------
struct Affine {
  int64_t S, ldw, ldb;
  cr_out type;
  const void *w, *b;
  const int32_t* off;
  std::vector<int64_t> shape;      // of their gradients
};
// weight, bias [C], or [S, C] (rows may lie further apart) with seg_offsets [S + 1]
Affine affine(const Tensor* w, const Tensor* b, const Tensor* off, int index, int64_t C) {
  Affine r{1, C, C, CR_OUT_F32, nullptr, nullptr, nullptr, {C}};
  if (off) {
    if (off->dim() != 1 || off->size(0) < 1) wrong("seg_offsets is int32 [S + 1]");
    r.S = off->size(0) - 1;
    r.off = static_cast<const int32_t*>(dense(*off, "seg_offsets", ScalarType::Int, index, {r.S + 1}));
    r.shape = {r.S, C};
  }
  if (const Tensor* first = w ? w : b) {
    r.type = float_type(*first, "weight and bias");
    const ScalarType dt = first->scalar_type();
    if (off) {
      r.w = w ? spaced(*w, "weight", dt, index, r.S, C, &r.ldw) : nullptr;
      r.b = b ? spaced(*b, "bias", dt, index, r.S, C, &r.ldb) : nullptr;
    } else {
      r.w = dense_or_null(w, "weight", dt, index, r.shape);
      r.b = dense_or_null(b, "bias", dt, index, r.shape);
    }
  }
  return r;
}
int count_of(int64_t S) { return S > (1 << 20) ? -1 : (int)S; }

// x, weight, bias, seg_offsets, eps, one_plus, out_type, out, mean, rstd, stream
PyObject* norm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Tensor& x = tensor(a[0], "x");
    const int index = gpu_of(x, "x");
    hipStream_t stream;
    if (!stream_for(a[10], index, &stream)) return elsewhere();
    if (x.dim() != 2) wrong("x is [M, C]");
    const int64_t M = x.size(0), C = x.size(1);
    const cr_out x_type = float_type(x, "x");
    int64_t ldx, ldy = C;
    const void* px = spaced(x, "x", x.scalar_type(), index, M, C, &ldx);
    const Affine f = affine(tensor_or_none(a[1], "weight"), tensor_or_none(a[2], "bias"), tensor_or_none(a[3], "seg_offsets"), index, C);
    const int type = small(a[6]);
    const ScalarType dt = out_dtype(type);
    const Tensor *go = tensor_or_none(a[7], "out"), *gm = tensor_or_none(a[8], "mean"), *gr = tensor_or_none(a[9], "rstd");
    if (go) spaced(*go, "out", dt, index, M, C, &ldy);
    dense_or_null(gm, "mean", ScalarType::Float, index, {M});
    dense_or_null(gr, "rstd", ScalarType::Float, index, {M});
    const double eps = real(a[4]);
    const bool plus = truth(a[5]);
    Tensor out, mean, rstd;
    cr_status st;
    {
      const Unlocked free;
      out = go ? *go : empty({M, C}, dt, x);
      mean = gm ? *gm : empty({M}, ScalarType::Float, x);
      rstd = gr ? *gr : empty({M}, ScalarType::Float, x);
      st = convrot_layer_norm_forward(px, x_type, ldx, f.w, f.ldw, f.b, f.ldb, f.type, plus, f.off, count_of(f.S), eps, out.data_ptr(),
                                      (cr_out)type, ldy, static_cast<float*>(mean.data_ptr()), static_cast<float*>(rstd.data_ptr()), M,
                                      C, stream);
    }
    if (ran(st))
      for (const Tensor* t : {go, gm, gr}) written(t);
    return st ? refused(st) : pack({&out, &mean, &rstd});
  });
}

// dy, x, mean, rstd, weight, seg_offsets, one_plus, dx_base, dx_type, dx, d_weight, d_bias, want_dx, want_weights,
// accumulate, workspace, stream
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const Tensor& dy = tensor(a[0], "dy");
    const int index = gpu_of(dy, "dy");
    hipStream_t stream;
    if (!stream_for(a[16], index, &stream)) return elsewhere();
    if (dy.dim() != 2) wrong("dy is [M, C]");
    const int64_t M = dy.size(0), C = dy.size(1);
    const bool want_dx = truth(a[12]), want_w = truth(a[13]), accumulate = truth(a[14]);
    if (!want_dx && !want_w) wrong("nothing is wanted");
    const Tensor& x = tensor(a[1], "x");
    const cr_out dy_type = float_type(dy, "dy"), x_type = float_type(x, "x");
    int64_t lddy, ldx, ldb = C, lddx = C;
    const void* pdy = spaced(dy, "dy", dy.scalar_type(), index, M, C, &lddy);
    const void* px = spaced(x, "x", x.scalar_type(), index, M, C, &ldx);
    const float* pm = static_cast<const float*>(dense(tensor(a[2], "mean"), "mean", ScalarType::Float, index, {M}));
    const float* pr = static_cast<const float*>(dense(tensor(a[3], "rstd"), "rstd", ScalarType::Float, index, {M}));
    const Affine f = affine(tensor_or_none(a[4], "weight"), nullptr, tensor_or_none(a[5], "seg_offsets"), index, C);
    const int type = small(a[8]);
    const ScalarType dt = out_dtype(type);
    const Tensor *gb = tensor_or_none(a[7], "dx_base"), *gx = tensor_or_none(a[9], "dx"), *gw = tensor_or_none(a[10], "d_weight"),
                 *gd = tensor_or_none(a[11], "d_bias"), *gs = tensor_or_none(a[15], "workspace");
    if (accumulate && want_w && (!gw || !gd)) wrong("accumulate adds to given d_weight and d_bias");
    const void* pb = nullptr;
    Tensor dx, dw, db, ws;
    if (want_dx) {
      if (gb) pb = spaced(*gb, "dx_base", dt, index, M, C, &ldb);
      if (gx) spaced(*gx, "dx", dt, index, M, C, &lddx);
    }
    if (want_w) {
      dense_or_null(gw, "d_weight", ScalarType::Float, index, f.shape);
      dense_or_null(gd, "d_bias", ScalarType::Float, index, f.shape);
      if (gs && (!on(*gs, index) || !gs->is_contiguous())) wrong("workspace must be contiguous on GPU %d", index);
    }
    const bool plus = truth(a[6]);
    cr_status st;
    {
      const Unlocked free;
      if (want_dx) dx = gx ? *gx : empty({M, C}, dt, dy);
      if (want_w) {
        dw = gw ? *gw : empty(f.shape, ScalarType::Float, dy);
        db = gd ? *gd : empty(f.shape, ScalarType::Float, dy);
        const size_t need = convrot_layer_norm_backward_workspace_size(M, C, count_of(f.S));
        ws = gs ? *gs : empty({(int64_t)(need < 16 ? 16 : need)}, ScalarType::Byte, dy);
      }
      st = convrot_layer_norm_backward(pdy, dy_type, lddy, px, x_type, ldx, pm, pr, f.w, f.ldw, f.type, plus, f.off, count_of(f.S), pb,
                                       ldb, want_dx ? dx.data_ptr() : nullptr, (cr_out)type, lddx,
                                       want_w ? static_cast<float*>(dw.data_ptr()) : nullptr,
                                       want_w ? static_cast<float*>(db.data_ptr()) : nullptr, accumulate, M, C,
                                       want_w ? ws.data_ptr() : nullptr, want_w ? ws.nbytes() : 0, stream);
    }
    if (ran(st)) {
      if (want_dx) written(gx);
      if (want_w)
        for (const Tensor* t : {gw, gd, gs}) written(t);
    }
    return st ? refused(st) : pack({want_dx ? &dx : nullptr, want_w ? &dw : nullptr, want_w ? &db : nullptr, want_w ? &ws : nullptr});
  });
}

// ---------------------------------------------------------------------------
// optimizer step
// ---------------------------------------------------------------------------
// a list or tuple of tensors, which are held until the call has returned: the caller's list may change while the
// interpreter's lock is given up
struct Tensors {
  c10::SmallVector<PyObject*, 64> held;
  bool given;
  const char* what;
  Py_ssize_t n = 0;
  Tensors(PyObject* o, const char* what) : given(o != Py_None), what(what) {
    if (!given) return;
    PyObject* items = PySequence_Fast(o, "lists of tensors are wanted");
    if (!items) throw python_error();
    n = PySequence_Fast_GET_SIZE(items);
    held.append(PySequence_Fast_ITEMS(items), PySequence_Fast_ITEMS(items) + n);
    for (PyObject* t : held) Py_INCREF(t);
    Py_DECREF(items);
  }
  ~Tensors() {
    for (PyObject* t : held) Py_DECREF(t);
  }
  Tensors(const Tensors&) = delete;
  Tensors& operator=(const Tensors&) = delete;
  explicit operator bool() const { return given; }
  const Tensor& operator[](Py_ssize_t i) const { return tensor(held[(size_t)i], what); }
};

void* element(const Tensors& l, const Tensor& t, ScalarType type, int index, int64_t numel) {
  if (t.numel() != numel) wrong("%s must hold one tensor for each of params, of its size", l.what);
  if (t.scalar_type() != type || !on(t, index) || !t.is_contiguous())
    wrong("%s must be contiguous %s tensors on GPU %d", l.what, type_name(type), index);
  return t.data_ptr();
}
void* element(const Tensors& l, Py_ssize_t i, ScalarType type, int index, int64_t numel) { return element(l, l[i], type, index, numel); }

// Fills the moments of every entry; `sizes` from the first list.
void moments(std::vector<cr_adamw_tensor>& e, const Tensors& m, const Tensors& v, const Tensors& ms, const Tensors& vs, int index) {
  if ((bool)ms != (bool)vs) wrong("8-bit moments have exp_avg_scales and exp_avg_sq_scales");
  const Py_ssize_t n = (Py_ssize_t)e.size();
  for (const Tensors* l : {&m, &v, &ms, &vs})
    if (*l && l->n != n) wrong("%s must hold one tensor for each of params, of its size", l->what);
  if (!m || !v) wrong("exp_avgs and exp_avg_sqs are wanted");
  for (Py_ssize_t i = 0; i < n; ++i) {
    cr_adamw_tensor& t = e[(size_t)i];
    t.exp_avg = element(m, i, ms ? ScalarType::Char : ScalarType::Float, index, t.n);
    t.exp_avg_sq = element(v, i, ms ? ScalarType::Byte : ScalarType::Float, index, t.n);
    if (ms) {
      t.avg_scales = static_cast<float*>(element(ms, i, ScalarType::Float, index, (t.n + 255) / 256));
      t.sq_scales = static_cast<float*>(element(vs, i, ScalarType::Float, index, (t.n + 255) / 256));
    }
  }
}
int entries(const std::vector<cr_adamw_tensor>& e) { return e.size() > (1u << 20) ? -1 : (int)e.size(); }

// params, grads, exp_avgs, exp_avg_sqs, copies, exp_avg_scales, exp_avg_sq_scales, grad_scale, step, lr, beta1, beta2, eps,
// weight_decay, seed, stream
PyObject* adamw_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const Tensors p(a[0], "params"), g(a[1], "grads"), m(a[2], "exp_avgs"), v(a[3], "exp_avg_sqs"), c(a[4], "copies"),
        ms(a[5], "exp_avg_scales"), vs(a[6], "exp_avg_sq_scales");
    if (p.n < 1) wrong("params is empty");
    const int index = gpu_of(p[0], "params");
    hipStream_t stream;
    if (!stream_for(a[15], index, &stream)) return elsewhere();
    for (const Tensors* l : {&g, &c})
      if ((l == &g || *l) && l->n != p.n) wrong("%s must hold one tensor for each of params, of its size", l->what);
    const cr_out grad_type = float_type(g[0], "grads");
    const ScalarType gt = g[0].scalar_type();
    std::vector<cr_adamw_tensor> e((size_t)p.n);
    for (Py_ssize_t i = 0; i < p.n; ++i) {
      cr_adamw_tensor& t = e[(size_t)i];
      t = cr_adamw_tensor{};
      const Tensor& param = p[i];
      t.n = param.numel();
      t.param = element(p, param, ScalarType::Float, index, t.n);
      t.grad = element(g, i, gt, index, t.n);
      if (c) t.copy = element(c, i, ScalarType::BFloat16, index, t.n);
    }
    moments(e, m, v, ms, vs, index);
    const float* scale =
        static_cast<const float*>(dense_or_null(tensor_or_none(a[7], "grad_scale"), "grad_scale", ScalarType::Float, index, {1}));
    const double lr = real(a[9]), beta1 = real(a[10]), beta2 = real(a[11]), eps = real(a[12]), decay = real(a[13]);
    const int64_t step = whole(a[8]);
    const uint32_t seed = (uint32_t)whole(a[14]);
    cr_status st;
    {
      const Unlocked free;
      st = convrot_adamw_step(e.data(), entries(e), grad_type, ms ? 8 : 32, lr, beta1, beta2, eps, decay, step, scale, seed, stream);
    }
    // what a graph of the model can hold; the moments are the optimizer's own (252 tensors: 2 us of the host's for 10 with them)
    if (ran(st))
      for (const Tensors* l : {&p, &c})
        for (PyObject* t : l->held) written(&THPVariable_Unpack(t));
    return refused(st);
  });
}

// exp_avgs, exp_avg_sqs, exp_avg_scales, exp_avg_sq_scales, exp_avg_out, exp_avg_sq_out, stream
PyObject* adamw_moments(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const Tensors m(a[0], "exp_avgs"), v(a[1], "exp_avg_sqs"), ms(a[2], "exp_avg_scales"), vs(a[3], "exp_avg_sq_scales");
    if (m.n < 1) wrong("exp_avgs is empty");
    if (!ms || !vs) wrong("8-bit moments have exp_avg_scales and exp_avg_sq_scales");
    const int index = gpu_of(m[0], "exp_avgs");
    hipStream_t stream;
    if (!stream_for(a[6], index, &stream)) return elsewhere();
    std::vector<cr_adamw_tensor> e((size_t)m.n);
    int64_t total = 0;
    for (Py_ssize_t i = 0; i < m.n; ++i) {
      e[(size_t)i] = cr_adamw_tensor{};
      total += e[(size_t)i].n = m[i].numel();
    }
    moments(e, m, v, ms, vs, index);
    const Tensor *gm = tensor_or_none(a[4], "exp_avg_out"), *gv = tensor_or_none(a[5], "exp_avg_sq_out");
    dense_or_null(gm, "exp_avg_out", ScalarType::Float, index, {total});
    dense_or_null(gv, "exp_avg_sq_out", ScalarType::Float, index, {total});
    const Tensor& like = m[0];
    Tensor om, ov;
    cr_status st;
    {
      const Unlocked free;
      om = gm ? *gm : empty({total}, ScalarType::Float, like);
      ov = gv ? *gv : empty({total}, ScalarType::Float, like);
      st = convrot_adamw_moments(e.data(), entries(e), static_cast<float*>(om.data_ptr()), static_cast<float*>(ov.data_ptr()), stream);
    }
    if (ran(st))
      for (const Tensor* t : {gm, gv}) written(t);
    return st ? refused(st) : pack({&om, &ov});
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<mx_quantize>("mxfp4_quantize"),
                         method<mx_dequantize>("mxfp4_dequantize"),
                         method<mx_gemm>("mxfp4_gemm"),
                         method<norm_forward>("layer_norm_forward"),
                         method<norm_backward>("layer_norm_backward"),
                         method<adamw_step>("adamw_step"),
                         method<adamw_moments>("adamw_moments"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// Tensors are read through inlined code of the headers, which fits one torch.
PyMODINIT_FUNC PyInit__native() {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
  Py_XDECREF(torch);
  const char* text = version ? PyUnicode_AsUTF8(version) : nullptr;
  const bool same = text && !std::strcmp(text, BUILT_FOR_TORCH);
  if (text && !same) PyErr_Format(PyExc_ImportError, "built for torch %s, this is %s", BUILT_FOR_TORCH, text);
  Py_XDECREF(version);
  return same ? PyModule_Create(&module) : nullptr;
}
