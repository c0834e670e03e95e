// binding.cpp -- the Python module top_routing_grouped_gb300._fp8: the calls of the 8-bit operators
// (include/moe_fp8.h), of the rows around an expert stage (moe_rows.h) and of the optimiser's step (moe_optim.h)
// from torch tensors.  Each function checks types, shapes and layouts, as fp8.py, rows.py and optim.py document them,
// takes the current stream where none is given, and calls the library without the interpreter's lock.
//
// A call of a few rows takes the GPU two to five microseconds.  Checked in Python and passed on by ctypes,
// it cost the host 7.3 us (norm of one token, eight tensors: 4.1 us of checks, 1.2 of conversions, 2
// of the library and the launch); here it costs 2.1.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <memory>
#include <optional>
#include <string>
#include <vector>

#include "../../include/moe_fp8.h"
#include "../../include/moe_optim.h"
#include "../../include/moe_rows.h"

namespace {

using at::Tensor;

struct Refused {  // -> ValueError
  std::string what;
};
struct PyError {};  // the Python error is already set

// Types a tensor may have, in the order a message names them.
enum : unsigned { kF32 = 1, kBf16 = 2, kE4m3 = 4, kE8m0 = 8, kU8 = 16, kI32 = 32, kI64 = 64 };
constexpr unsigned kFloats = kF32 | kBf16, kScales = kE8m0 | kU8;

unsigned type_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::ScalarType::Float: return kF32;
    case at::ScalarType::BFloat16: return kBf16;
    case at::ScalarType::Float8_e4m3fn: return kE4m3;
    case at::ScalarType::Float8_e8m0fnu: return kE8m0;
    case at::ScalarType::Byte: return kU8;
    case at::ScalarType::Int: return kI32;
    case at::ScalarType::Long: return kI64;
    default: return 0;
  }
}

int32_t moe_dtype_of(unsigned type) { return type == kBf16 ? MOE_BF16 : MOE_F32; }

std::string names(unsigned types) {
  static constexpr const char* kNames[] = {"torch.float32", "torch.bfloat16", "torch.float8_e4m3fn", "torch.float8_e8m0fnu",
                                           "torch.uint8", "torch.int32", "torch.int64"};
  std::string s;
  for (int i = 0; i < 7; ++i)
    if (types >> i & 1) s += (s.empty() ? "" : " or ") + std::string(kNames[i]);
  return s;
}

using Shape = std::initializer_list<int64_t>;

[[noreturn]] void refuse(at::IntArrayRef shape, unsigned types, const char* name, const char* how) {
  std::string s;
  for (int64_t v : shape) s += (s.empty() ? "" : ", ") + std::to_string(v);
  if (shape.size() == 1) s += ",";
  throw Refused{std::string(name) + " must be a " + how + " (" + s + ") tensor of " + names(types)};
}

const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A tensor of two dimensions and one of these types, or what it says.
const Tensor& matrix(PyObject* o, unsigned types, const char* what) {
  const Tensor* t = tensor(o);
  if (!t || t->dim() != 2 || (types && !(type_of(*t) & types))) throw Refused{what};
  return *t;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return v;
}

template <typename P>
P handle(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw PyError{};
  return static_cast<P>(p);
}

struct Release {
  void operator()(PyObject* o) const { Py_DECREF(o); }
};

std::unique_ptr<PyObject, Release> attribute(PyObject* o, const char* name) {
  PyObject* v = PyObject_GetAttrString(o, name);
  if (!v) throw PyError{};
  return std::unique_ptr<PyObject, Release>(v);
}

// A call's arguments.  Types, shapes and layouts are checked as the arguments are taken; where the
// tensors lie, at the end (stream), which also makes their device the current one for the call.
struct Args {
  const char* on_host = nullptr;    // the first tensor outside GPU memory
  const char* elsewhere = nullptr;  // the first one on another GPU than those before it
  c10::DeviceIndex device = -1;     // theirs
  std::optional<c10::cuda::CUDAGuard> guard;

  void* address(const Tensor& t, const char* name) {
    if (!t.is_cuda()) {
      if (!on_host) on_host = name;
    } else if (device < 0) {
      device = (c10::DeviceIndex)t.get_device();
    } else if (t.get_device() != device && !elsewhere) {
      elsewhere = name;
    }
    return t.data_ptr();
  }

  // The address of a row-major contiguous tensor of this shape and one of these types.
  void* rows(PyObject* o, Shape shape, unsigned types, const char* name) {
    return array(o, at::IntArrayRef(shape.begin(), shape.size()), types, name);
  }

  void* array(PyObject* o, at::IntArrayRef shape, unsigned types, const char* name) {
    const Tensor* t = tensor(o);
    if (!t || !(type_of(*t) & types) || !t->sizes().equals(shape) || !t->is_contiguous()) refuse(shape, types, name, "contiguous");
    return address(*t, name);
  }

  void* maybe(PyObject* o, Shape shape, unsigned types, const char* name) {
    return o == Py_None ? nullptr : rows(o, shape, types, name);
  }

  // The address and row pitch of a 2-D tensor whose rows are contiguous and separate.
  void* pitched(PyObject* o, int64_t n, int64_t c, unsigned types, const char* name, int64_t* ld) {
    const Tensor* t = tensor(o);
    if (!t || !(type_of(*t) & types) || t->dim() != 2 || t->size(0) != n || t->size(1) != c) refuse({n, c}, types, name, "row-contiguous");
    *ld = c;
    if (!t->is_contiguous()) {
      if ((t->stride(1) != 1 && c != 1) || (t->stride(0) < c && n != 1)) refuse({n, c}, types, name, "row-contiguous");
      if (t->stride(0) > c) *ld = t->stride(0);
    }
    return address(*t, name);
  }

  // The address and size of a workspace.
  void* bytes(PyObject* o, size_t* n) {
    const Tensor* t = tensor(o);
    if (!t || type_of(*t) != kU8 || !t->is_contiguous())
      throw Refused{"workspaces and checkpoints must be contiguous uint8 tensors in GPU memory"};
    *n = (size_t)t->numel();
    return address(*t, "workspace");
  }

  void* maybe_bytes(PyObject* o, size_t* n) {
    *n = 0;
    return o == Py_None ? nullptr : bytes(o, n);
  }

  // The given torch.cuda.Stream, or (None) the current stream of the tensors' device.
  void* stream(PyObject* o) {
    if (on_host) throw Refused{std::string(on_host) + " must be in GPU memory"};
    if (elsewhere) throw Refused{std::string(elsewhere) + " must be on the device of the tensors before it"};
    if (o == Py_None) {
      make_current();
      return c10::cuda::getCurrentCUDAStream(device).stream();
    }
    void* p = handle<void*>(attribute(o, "cuda_stream").get());
    if (PyObject_HasAttrString(o, "device_index") && integer(attribute(o, "device_index").get()) != device)
      throw Refused{"the stream must be on the tensors' device"};
    make_current();
    return p;
  }

  void make_current() {
    if (c10::cuda::device_count() > 1) guard.emplace(device);
  }
};

// One Python function: kArgs arguments, body -> status.
template <int kArgs, typename Body>
PyObject* call(PyObject* const* a, Py_ssize_t n, Body body) {
  try {
    if (n != kArgs) throw Refused{"expected " + std::to_string(kArgs) + " arguments"};
    Args in;
    return PyLong_FromLong(body(in, a));
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
  } catch (const PyError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The library, without the interpreter's lock.
template <typename F>
long unlocked(F f) {
  PyThreadState* s = PyEval_SaveThread();
  const long status = f();
  PyEval_RestoreThread(s);
  return status;
}

#define ARGS PyObject*, PyObject *const *args, Py_ssize_t nargs
#define U8(p) static_cast<uint8_t*>(p)
#define FL(p) static_cast<float*>(p)

PyObject* quantize(ARGS) {  // x, q, scales, stream
  return call<4>(args, nargs, [](Args& in, PyObject* const* a) {
    const Tensor& x = matrix(a[0], kFloats, "x must be a 2-D fp32 or bf16 tensor");
    const int64_t n = x.size(0), c = x.size(1);
    int64_t ld;
    void *px = in.pitched(a[0], n, c, kFloats, "x", &ld), *q = in.rows(a[1], {n, c}, kE4m3, "q");
    void *s = in.rows(a[2], {n, moe_fp8_scale_cols(c)}, kScales, "scales"), *st = in.stream(a[3]);
    const int32_t dt = moe_dtype_of(type_of(x));
    return unlocked([=] { return moe_fp8_quantize(px, dt, n, c, ld, 1, 0, q, U8(s), st); });
  });
}

PyObject* quantize_weights(ARGS) {  // w, q, scales, stream
  return call<4>(args, nargs, [](Args& in, PyObject* const* a) {
    const Tensor* w = tensor(a[0]);
    if (!w || w->dim() != 3) throw Refused{"w must be a 3-D fp32 or bf16 tensor"};
    const int64_t E = w->size(0), n = w->size(1), c = w->size(2);
    void *pw = in.rows(a[0], {E, n, c}, kFloats, "w"), *q = in.rows(a[1], {E, n, c}, kE4m3, "q");
    void *s = in.rows(a[2], {E, (n + 127) / 128, moe_fp8_scale_cols(c)}, kScales, "scales"), *st = in.stream(a[3]);
    const int32_t dt = moe_dtype_of(type_of(*w));
    return unlocked([=] { return moe_fp8_quantize(pw, dt, E * n, c, c, 128, n, q, U8(s), st); });
  });
}

PyObject* rmsnorm(ARGS) {  // x, weight, residual, residual_out, out, q, scales, rstd, eps, stream
  return call<10>(args, nargs, [](Args& in, PyObject* const* a) {
    const Tensor& x = matrix(a[0], kFloats, "x must be a 2-D fp32 or bf16 tensor");
    const int64_t T = x.size(0), d = x.size(1);
    const unsigned t = type_of(x);
    int64_t ldx, ldr = d;
    void *px = in.pitched(a[0], T, d, t, "x", &ldx), *pr = a[2] == Py_None ? nullptr : in.pitched(a[2], T, d, t, "residual", &ldr);
    void *w = in.maybe(a[1], {d}, kF32, "weight"), *ro = in.maybe(a[3], {T, d}, t, "residual_out"), *out = in.maybe(a[4], {T, d}, t, "out");
    void *q = in.maybe(a[5], {T, d}, kE4m3, "q"), *s = in.maybe(a[6], {T, moe_fp8_scale_cols(d)}, kScales, "scales");
    void* rs = in.maybe(a[7], {T}, kF32, "rstd");
    const double eps = PyFloat_AsDouble(a[8]);
    if (eps == -1.0 && PyErr_Occurred()) throw PyError{};
    void* st = in.stream(a[9]);
    if (d > INT32_MAX) throw Refused{"x has too many columns"};
    return unlocked([=] {
      return moe_rmsnorm(px, pr, FL(w), moe_dtype_of(t), T, (int32_t)d, ldx, ldr, (float)eps, ro, out, q, U8(s), FL(rs), st);
    });
  });
}

PyObject* rmsnorm_backward(ARGS) {  // dout, r, weight, rstd, dx, dweight, workspace, dresidual, stream
  return call<9>(args, nargs, [](Args& in, PyObject* const* a) {
    const Tensor& r = matrix(a[1], kFloats, "r must be a 2-D fp32 or bf16 tensor");
    const int64_t T = r.size(0), d = r.size(1);
    const unsigned t = type_of(r);
    int64_t ldr;
    void *pr = in.pitched(a[1], T, d, t, "r", &ldr), *pd = in.rows(a[0], {T, d}, kFloats, "dout");
    void *w = in.maybe(a[2], {d}, kF32, "weight"), *rs = in.rows(a[3], {T}, kF32, "rstd"), *dres = in.maybe(a[7], {T, d}, t, "dresidual");
    void *dx = in.rows(a[4], {T, d}, t, "dx"), *dw = in.maybe(a[5], {d}, kF32, "dweight");
    size_t n;
    void *ws = in.maybe_bytes(a[6], &n), *st = in.stream(a[8]);
    const int32_t ddt = moe_dtype_of(type_of(THPVariable_Unpack(a[0])));
    if (d > INT32_MAX) throw Refused{"r has too many columns"};
    return unlocked([=] {
      return moe_rmsnorm_backward(pd, ddt, pr, FL(w), FL(rs), dres, moe_dtype_of(t), T, (int32_t)d, ldr, dx, FL(dw), ws, n, st);
    });
  });
}

PyObject* matmul(ARGS) {  // plan, (max_rows, K, n, E, segments, bf16 out), seg_counts, a, a_scales, w, w_scales, out, workspace, stream
  return call<15>(args, nargs, [](Args& in, PyObject* const* a) {
    const auto plan = handle<moe_fp8_plan_t>(a[0]);
    const int64_t R = integer(a[1]), K = integer(a[2]), N = integer(a[3]), E = integer(a[4]), S = integer(a[5]);
    const unsigned ot = integer(a[6]) ? kBf16 : kF32;
    a += 7;
    void *seg = in.maybe(a[0], {S}, kI32, "seg_counts"), *pa = in.rows(a[1], {R, K}, kE4m3, "a");
    void *sa = in.rows(a[2], {R, moe_fp8_scale_cols(K)}, kScales, "a_scales"), *w = in.rows(a[3], {E, N, K}, kE4m3, "w");
    void *sw = in.rows(a[4], {E, (N + 127) / 128, moe_fp8_scale_cols(K)}, kScales, "w_scales"), *out = in.rows(a[5], {R, N}, ot, "out");
    size_t n;
    void *ws = in.bytes(a[6], &n), *st = in.stream(a[7]);
    return unlocked([=] { return moe_fp8_matmul(plan, static_cast<int32_t*>(seg), pa, U8(sa), w, U8(sw), out, ws, n, st); });
  });
}

// The experts' weights and factors: w1, s1, w3, s3, w2, s2.
struct Experts {
  void *w1, *s1, *w3, *s3, *w2, *s2;
  Experts(Args& in, PyObject* const* a, int64_t E, int64_t d, int64_t F) {
    const int64_t sd = moe_fp8_scale_cols(d), sF = moe_fp8_scale_cols(F), bF = (F + 127) / 128, bd = (d + 127) / 128;
    w1 = in.rows(a[0], {E, F, d}, kE4m3, "w1");
    s1 = in.rows(a[1], {E, bF, sd}, kScales, "s1");
    w3 = in.rows(a[2], {E, F, d}, kE4m3, "w3");
    s3 = in.rows(a[3], {E, bF, sd}, kScales, "s3");
    w2 = in.rows(a[4], {E, d, F}, kE4m3, "w2");
    s2 = in.rows(a[5], {E, bd, sF}, kScales, "s2");
  }
};

PyObject* experts(ARGS) {  // plan, (max_rows, d, E, segments, F), seg_counts, x_rows, x_scales, gates, weights..., y_rows, workspace, stream
  return call<19>(args, nargs, [](Args& in, PyObject* const* a) {
    const auto plan = handle<moe_fp8_plan_t>(a[0]);
    const int64_t R = integer(a[1]), d = integer(a[2]), E = integer(a[3]), S = integer(a[4]), F = integer(a[5]);
    a += 6;
    void *seg = in.maybe(a[0], {S}, kI32, "seg_counts"), *x = in.rows(a[1], {R, d}, kE4m3, "x_rows");
    void *sx = in.rows(a[2], {R, moe_fp8_scale_cols(d)}, kScales, "x_scales"), *g = in.rows(a[3], {R}, kF32, "gates");
    const Experts w(in, a + 4, E, d, F);
    size_t n;
    void *y = in.rows(a[10], {R, d}, kBf16, "y_rows"), *ws = in.bytes(a[11], &n), *st = in.stream(a[12]);
    return unlocked([=] {
      return moe_fp8_expert_forward(plan, static_cast<int32_t*>(seg), x, U8(sx), FL(g), w.w1, U8(w.s1), w.w3, U8(w.s3), w.w2,
                                    U8(w.s2), y, ws, n, st);
    });
  });
}

PyObject* layer(ARGS) {  // plan, (T, d, E, F, bf16 out), x, x_q, x_scales, w_router, bias, weights..., y, workspace, stream
  return call<20>(args, nargs, [](Args& in, PyObject* const* a) {
    const auto plan = handle<moe_plan_t>(a[0]);
    const int64_t T = integer(a[1]), d = integer(a[2]), E = integer(a[3]), F = integer(a[4]);
    const unsigned ot = integer(a[5]) ? kBf16 : kF32;
    a += 6;
    void *x = in.rows(a[0], {T, d}, kBf16, "x"), *xq = in.rows(a[1], {T, d}, kE4m3, "x_q");
    void *sx = in.rows(a[2], {T, moe_fp8_scale_cols(d)}, kScales, "x_scales"), *wr = in.rows(a[3], {E, d}, kBf16, "w_router");
    void* bias = in.maybe(a[4], {E}, kF32, "bias");
    const Experts w(in, a + 5, E, d, F);
    size_t n;
    void *y = in.rows(a[11], {T, d}, ot, "y"), *ws = in.bytes(a[12], &n), *st = in.stream(a[13]);
    return unlocked([=] {
      return moe_fp8_forward(plan, x, xq, U8(sx), wr, FL(bias), w.w1, U8(w.s1), w.w3, U8(w.s3), w.w2, U8(w.s2), y, ws, n, st);
    });
  });
}

PyObject* checkpoint_save(ARGS) {  // a, b, qa, sa, qb, sb, stream
  return call<7>(args, nargs, [](Args& in, PyObject* const* p) {
    const Tensor& t = matrix(p[0], 0, "a must be 2-D");
    const int64_t n = t.size(0), F = t.size(1), sc = moe_fp8_scale_cols(F);
    void *a = in.rows(p[0], {n, F}, kBf16, "a"), *b = in.rows(p[1], {n, F}, kBf16, "b");
    void *qa = in.rows(p[2], {n, F}, kE4m3, "qa"), *sa = in.rows(p[3], {n, sc}, kScales, "sa");
    void *qb = in.rows(p[4], {n, F}, kE4m3, "qb"), *sb = in.rows(p[5], {n, sc}, kScales, "sb"), *st = in.stream(p[6]);
    if (F > INT32_MAX) throw Refused{"a has too many columns"};
    return unlocked([=] { return moe_checkpoint_save_rows(a, b, n, (int32_t)F, qa, U8(sa), qb, U8(sb), st); });
  });
}

// A checkpoint's values and factors: qa, sa, qb, sb.
struct Kept {
  int64_t n, F;
  void *qa, *sa, *qb, *sb;
  Kept(Args& in, PyObject* const* p) {
    const Tensor& t = matrix(p[0], 0, "qa must be 2-D");
    n = t.size(0);
    F = t.size(1);
    if (F > INT32_MAX) throw Refused{"qa has too many columns"};
    const int64_t sc = moe_fp8_scale_cols(F);
    qa = in.rows(p[0], {n, F}, kE4m3, "qa");
    sa = in.rows(p[1], {n, sc}, kScales, "sa");
    qb = in.rows(p[2], {n, F}, kE4m3, "qb");
    sb = in.rows(p[3], {n, sc}, kScales, "sb");
  }
};

PyObject* checkpoint_restore(ARGS) {  // qa, sa, qb, sb, a, b, h, stream
  return call<8>(args, nargs, [](Args& in, PyObject* const* p) {
    const Kept k(in, p);
    void *a = in.maybe(p[4], {k.n, k.F}, kBf16, "a"), *b = in.maybe(p[5], {k.n, k.F}, kBf16, "b");
    void *h = in.maybe(p[6], {k.n, k.F}, kBf16, "h"), *st = in.stream(p[7]);
    return unlocked(
        [=] { return moe_checkpoint_restore_rows(k.qa, U8(k.sa), k.qb, U8(k.sb), k.n, (int32_t)k.F, a, b, h, st); });
  });
}

PyObject* checkpoint_backward(ARGS) {  // qa, sa, qb, sb, dh, da, db, h, stream
  return call<9>(args, nargs, [](Args& in, PyObject* const* p) {
    const Kept k(in, p);
    void *dh = in.rows(p[4], {k.n, k.F}, kBf16, "dh"), *da = in.rows(p[5], {k.n, k.F}, kBf16, "da");
    void *db = in.rows(p[6], {k.n, k.F}, kBf16, "db"), *h = in.maybe(p[7], {k.n, k.F}, kBf16, "h"), *st = in.stream(p[8]);
    return unlocked(
        [=] { return moe_checkpoint_backward_rows(k.qa, U8(k.sa), k.qb, U8(k.sb), dh, k.n, (int32_t)k.F, da, db, h, st); });
  });
}

// The rows that a dispatch moves: x, x_rows, x_scales, row_scales, gates, row_gates.
struct Moved {
  int64_t d, ldx, R, scale_bytes = 0;
  int32_t elem_bytes;
  void *x, *x_rows, *x_scales = nullptr, *row_scales = nullptr, *gates = nullptr, *row_gates = nullptr;
  Moved(Args& in, int64_t T, int64_t k, PyObject* px, PyObject* po, PyObject* pxs, PyObject* prs, PyObject* pg, PyObject* prg) {
    const Tensor &t = matrix(px, kFloats | kE4m3, "x must be a 2-D fp32, bf16 or e4m3 tensor"), &o = matrix(po, 0, "x_rows must be 2-D");
    const unsigned type = type_of(t);
    d = t.size(1);
    R = o.size(0);
    elem_bytes = type == kE4m3 ? 1 : type == kBf16 ? 2 : 4;
    x = in.pitched(px, T, d, type, "x", &ldx);
    x_rows = in.rows(po, {R, d}, type, "x_rows");
    if ((pxs == Py_None) != (prs == Py_None)) throw Refused{"x_scales and row_scales go together"};
    if ((pg == Py_None) != (prg == Py_None)) throw Refused{"gates and row_gates go together"};
    if (pxs != Py_None) {
      if (type != kE4m3) throw Refused{"only e4m3 rows have scales"};
      scale_bytes = moe_fp8_scale_cols(d);
      x_scales = in.rows(pxs, {T, scale_bytes}, kScales, "x_scales");
      row_scales = in.rows(prs, {R, scale_bytes}, kScales, "row_scales");
    }
    if (pg != Py_None) {
      gates = in.rows(pg, {T, k}, kF32, "gates");
      row_gates = in.rows(prg, {R}, kF32, "row_gates");
    }
  }
};

// The sort's arrays: idx, counts, slot_pos, row_slot.
struct Sorted {
  int64_t T, k, E;
  int32_t idx_bytes;
  void *idx, *counts, *slot_pos, *row_slot;
  Sorted(Args& in, PyObject* pi, PyObject* pc, PyObject* ps, PyObject* pr) {
    const Tensor &t = matrix(pi, kI32 | kI64, "idx must be a 2-D int32 or int64 tensor"), *c = tensor(pc);
    if (!c || c->dim() != 1) throw Refused{"counts must be a 1-D int32 tensor"};
    T = t.size(0);
    k = t.size(1);
    E = c->size(0);
    if (k > INT32_MAX || E > INT32_MAX) throw Refused{"idx has too many columns, or counts too many values"};
    idx_bytes = type_of(t) == kI64 ? 8 : 4;
    idx = in.rows(pi, {T, k}, kI32 | kI64, "idx");
    counts = in.rows(pc, {E}, kI32, "counts");
    slot_pos = in.rows(ps, {T, k}, kI32, "slot_pos");
    row_slot = in.maybe(pr, {T * k}, kI32, "row_slot");
  }
};

#define I32(p) static_cast<int32_t*>(p)

PyObject* rows_sort(ARGS) {  // idx, counts, slot_pos, row_slot, workspace, stream
  return call<6>(args, nargs, [](Args& in, PyObject* const* p) {
    const Sorted s(in, p[0], p[1], p[2], p[3]);
    size_t n;
    void *ws = in.maybe_bytes(p[4], &n), *st = in.stream(p[5]);
    return unlocked([=] {
      return moe_rows_sort(s.idx, s.idx_bytes, s.T, (int32_t)s.k, (int32_t)s.E, I32(s.counts), I32(s.slot_pos), I32(s.row_slot), ws, n, st);
    });
  });
}

PyObject* rows_gather(ARGS) {  // slot_pos, x, x_rows, x_scales, row_scales, gates, row_gates, stream
  return call<8>(args, nargs, [](Args& in, PyObject* const* p) {
    const Tensor& t = matrix(p[0], kI32, "slot_pos must be a 2-D int32 tensor");
    const int64_t T = t.size(0), k = t.size(1);
    if (k > INT32_MAX) throw Refused{"slot_pos has too many columns"};
    void* pos = in.rows(p[0], {T, k}, kI32, "slot_pos");
    const Moved m(in, T, k, p[1], p[2], p[3], p[4], p[5], p[6]);
    void* st = in.stream(p[7]);
    return unlocked([=] {
      return moe_rows_gather(I32(pos), T, (int32_t)k, m.x, m.elem_bytes, m.d, m.ldx, m.R, m.x_rows, U8(m.x_scales), U8(m.row_scales),
                             m.scale_bytes, FL(m.gates), FL(m.row_gates), st);
    });
  });
}

PyObject* rows_dispatch(ARGS) {  // idx, x, counts, slot_pos, x_rows, workspace, row_slot, x_scales, row_scales, gates, row_gates, stream
  return call<12>(args, nargs, [](Args& in, PyObject* const* p) {
    const Sorted s(in, p[0], p[2], p[3], p[6]);
    const Moved m(in, s.T, s.k, p[1], p[4], p[7], p[8], p[9], p[10]);
    size_t n;
    void *ws = in.maybe_bytes(p[5], &n), *st = in.stream(p[11]);
    return unlocked([=] {
      return moe_rows_dispatch(s.idx, s.idx_bytes, s.T, (int32_t)s.k, (int32_t)s.E, I32(s.counts), I32(s.slot_pos), I32(s.row_slot), m.x,
                               m.elem_bytes, m.d, m.ldx, m.R, m.x_rows, U8(m.x_scales), U8(m.row_scales), m.scale_bytes, FL(m.gates),
                               FL(m.row_gates), ws, n, st);
    });
  });
}

PyObject* rows_combine(ARGS) {  // y_rows, slot_pos, out, gates, residual, stream
  return call<6>(args, nargs, [](Args& in, PyObject* const* p) {
    const Tensor &y = matrix(p[0], kFloats, "y_rows must be a 2-D fp32 or bf16 tensor"), &o = matrix(p[2], kFloats, "out must be a 2-D fp32 or bf16 tensor");
    const Tensor& sp = matrix(p[1], kI32, "slot_pos must be a 2-D int32 tensor");
    const int64_t R = y.size(0), d = y.size(1), T = sp.size(0), k = sp.size(1);
    if (k > INT32_MAX) throw Refused{"slot_pos has too many columns"};
    const unsigned ty = type_of(y), to = type_of(o);
    void *py = in.rows(p[0], {R, d}, ty, "y_rows"), *pos = in.rows(p[1], {T, k}, kI32, "slot_pos"), *out = in.rows(p[2], {T, d}, to, "out");
    void *g = in.maybe(p[3], {T, k}, kF32, "gates"), *res = in.maybe(p[4], {T, d}, to, "residual"), *st = in.stream(p[5]);
    return unlocked(
        [=] { return moe_rows_combine(py, moe_dtype_of(ty), R, I32(pos), FL(g), T, (int32_t)k, d, res, out, moe_dtype_of(to), st); });
  });
}

PyObject* rows_combine_backward(ARGS) {  // dout, slot_pos, gates, y_rows, dy_rows, dgates, stream
  return call<7>(args, nargs, [](Args& in, PyObject* const* p) {
    const Tensor &o = matrix(p[0], kFloats, "dout must be a 2-D fp32 or bf16 tensor"), &sp = matrix(p[1], kI32, "slot_pos must be a 2-D int32 tensor");
    const int64_t T = sp.size(0), k = sp.size(1), d = o.size(1);
    if (k > INT32_MAX) throw Refused{"slot_pos has too many columns"};
    PyObject* any = p[3] != Py_None ? p[3] : p[4];
    if (any == Py_None) throw Refused{"y_rows or dy_rows is needed"};
    const Tensor& y = matrix(any, kFloats, "y_rows and dy_rows must be 2-D fp32 or bf16 tensors");
    const int64_t R = y.size(0);
    const unsigned ty = type_of(y);
    void *po = in.rows(p[0], {T, d}, kFloats, "dout"), *pos = in.rows(p[1], {T, k}, kI32, "slot_pos"), *g = in.maybe(p[2], {T, k}, kF32, "gates");
    void *py = in.maybe(p[3], {R, d}, ty, "y_rows"), *dy = in.maybe(p[4], {R, d}, ty, "dy_rows"), *dg = in.maybe(p[5], {T, k}, kF32, "dgates");
    void* st = in.stream(p[6]);
    const int32_t dt = moe_dtype_of(type_of(o));
    return unlocked(
        [=] { return moe_rows_combine_backward(po, dt, I32(pos), FL(g), T, (int32_t)k, d, R, py, dy, moe_dtype_of(ty), FL(dg), st); });
  });
}

// A Python sequence of n (n < 0: any number of) items.
struct Items {
  std::unique_ptr<PyObject, Release> seq;
  Py_ssize_t n;
  Items(PyObject* o, Py_ssize_t want, const char* name) : seq(PySequence_Fast(o, name)) {
    if (!seq) {
      PyErr_Clear();
      throw Refused{std::string(name) + " must be a list"};
    }
    n = PySequence_Fast_GET_SIZE(seq.get());
    if (want >= 0 && n != want) throw Refused{std::string(name) + " must have " + std::to_string(want) + " entries"};
  }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq.get(), i); }
};

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError{};
  return v;
}

// params, masters, grads, m, v, m_scales, v_scales, decays, lr, lr_device, beta1, beta2, eps, seed, grad_factor, steps, ticket, stream
PyObject* adamw(ARGS) {
  return call<18>(args, nargs, [](Args& in, PyObject* const* p) {
    const Items ps(p[0], -1, "params");
    const Items ws(p[1], ps.n, "masters"), gs(p[2], ps.n, "grads"), ms(p[3], ps.n, "m"), vs(p[4], ps.n, "v"), mss(p[5], ps.n, "m_scales"),
        vss(p[6], ps.n, "v_scales"), ds(p[7], ps.n, "weight_decay");
    std::vector<moe_adamw_tensor> list(ps.n);
    for (Py_ssize_t i = 0; i < ps.n; ++i) {
      moe_adamw_tensor& t = list[i];
      const Tensor* q = tensor(ps[i]);
      if (!q || !(type_of(*q) & kFloats) || !q->is_contiguous()) throw Refused{"params must be contiguous fp32 or bf16 tensors"};
      const at::IntArrayRef shape = q->sizes();
      const bool small = mss[i] != Py_None;
      t.n = q->numel();
      const int64_t blocks = (t.n + 127) / 128;
      t.param = in.address(*q, "a parameter");
      t.master = ws[i] == Py_None ? nullptr : FL(in.array(ws[i], shape, kF32, "a master"));
      t.grad = in.array(gs[i], shape, kFloats, "a gradient");
      t.m = in.array(ms[i], shape, small ? kE4m3 : kF32, "m");
      t.v = in.array(vs[i], shape, small ? kE4m3 : kF32, "v");
      t.m_scales = U8(in.maybe(mss[i], {blocks}, kScales, "m_scales"));
      t.v_scales = U8(in.maybe(vss[i], {blocks}, kScales, "v_scales"));
      t.weight_decay = (float)real(ds[i]);
      t.param_dtype = moe_dtype_of(type_of(*q));
      t.grad_dtype = moe_dtype_of(type_of(*tensor(gs[i])));
    }
    moe_adamw_config c{};
    c.lr = real(p[8]);
    c.lr_device = FL(in.maybe(p[9], {1}, kF32, "lr"));
    c.beta1 = real(p[10]);
    c.beta2 = real(p[11]);
    c.eps = real(p[12]);
    c.seed = PyLong_AsUnsignedLongLongMask(p[13]);
    if (c.seed == (uint64_t)-1 && PyErr_Occurred()) throw PyError{};
    float* factor = FL(in.maybe(p[14], {1}, kF32, "grad_factor"));
    int64_t* steps = static_cast<int64_t*>(in.rows(p[15], {1}, kI64, "steps"));
    uint32_t* ticket = reinterpret_cast<uint32_t*>(in.rows(p[16], {1}, kI32, "ticket"));
    void* st = in.stream(p[17]);
    if (ps.n > INT32_MAX) throw Refused{"too many tensors"};
    return unlocked([&] { return moe_adamw(list.data(), (int32_t)list.size(), &c, factor, steps, ticket, st); });
  });
}

PyObject* grad_norm(ARGS) {  // grads, norm, factor, max_norm, workspace, stream
  return call<6>(args, nargs, [](Args& in, PyObject* const* p) {
    const Items gs(p[0], -1, "grads");
    std::vector<moe_grad_tensor> list(gs.n);
    for (Py_ssize_t i = 0; i < gs.n; ++i) {
      const Tensor* q = tensor(gs[i]);
      if (!q || !(type_of(*q) & kFloats) || !q->is_contiguous()) throw Refused{"grads must be contiguous fp32 or bf16 tensors"};
      list[i] = {in.address(*q, "a gradient"), q->numel(), moe_dtype_of(type_of(*q))};
    }
    float *norm = FL(in.rows(p[1], {1}, kF32, "norm")), *factor = FL(in.maybe(p[2], {1}, kF32, "factor"));
    const float most = (float)real(p[3]);
    size_t n;
    void *ws = in.maybe_bytes(p[4], &n), *st = in.stream(p[5]);
    if (gs.n > INT32_MAX) throw Refused{"too many tensors"};
    return unlocked([&] { return moe_grad_norm(list.data(), (int32_t)list.size(), most, norm, factor, ws, n, st); });
  });
}

#define FUNCTION(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr }
PyMethodDef kFunctions[] = {FUNCTION(quantize),          FUNCTION(quantize_weights),   FUNCTION(rmsnorm),
                            FUNCTION(rmsnorm_backward),  FUNCTION(matmul),             FUNCTION(experts),
                            FUNCTION(layer),             FUNCTION(checkpoint_save),    FUNCTION(checkpoint_restore),
                            FUNCTION(checkpoint_backward), FUNCTION(rows_sort),    FUNCTION(rows_gather),
                            FUNCTION(rows_dispatch),     FUNCTION(rows_combine),       FUNCTION(rows_combine_backward),
                            FUNCTION(adamw),             FUNCTION(grad_norm),          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fp8", "Calls of the 8-bit operators, the sorted rows and the optimiser's step.", -1, kFunctions, nullptr, nullptr, nullptr,
                       nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8(void) { return PyModule_Create(&kModule); }
