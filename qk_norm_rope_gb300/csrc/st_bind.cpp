// Python binding of the serving calls. A decoding step makes them for every
// layer on small tensors, where marshalling through ctypes costs several times
// the C call; here tensors are read, outputs allocated and the stream looked up
// in C++. Arguments are positional and complete (the Python layer fills in
// defaults); errors raise the StError class given to init().
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>
#include <string>

#include "st_rope_attn.h"

namespace {

PyObject* g_error = nullptr;  // the StError class

struct Refused : std::exception {
  int status;
  std::string msg;
  Refused(int s, std::string m) : status(s), msg(std::move(m)) {}
};

// One call's tensors: st_tensor views of them, and the one device they live on.
struct Call {
  int dev = -1;

  const at::Tensor* tensor(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Refused(ST_ERR_INVALID_ARG, std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) throw Refused(ST_ERR_INVALID_ARG, "all tensors must live on a CUDA device");
    const int d = t.get_device();
    if (dev < 0) dev = d;
    else if (d != dev)
      throw Refused(ST_ERR_INVALID_ARG, "tensors live on cuda:" + std::to_string(dev) + " and on cuda:" + std::to_string(d));
    return &t;
  }

  static void fill(const at::Tensor& t, st_tensor* s, const char* name) {
    switch (t.scalar_type()) {
      case at::kBFloat16: s->dtype = ST_BF16; break;
      case at::kHalf: s->dtype = ST_F16; break;
      case at::kFloat: s->dtype = ST_F32; break;
      case at::kBool: s->dtype = ST_BOOL; break;
      case at::kInt: s->dtype = ST_I32; break;
      case at::kLong: s->dtype = ST_I64; break;
      case at::kFloat8_e4m3fn: s->dtype = ST_E4M3; break;
      case at::kChar: s->dtype = ST_I8; break;
      default: throw Refused(ST_ERR_DTYPE, std::string("unsupported dtype of ") + name);
    }
    const int64_t n = t.dim();
    if (n > 4) throw Refused(ST_ERR_SHAPE, "tensors have at most 4 dims");
    s->data = t.numel() > 0 ? t.data_ptr() : nullptr;
    s->ndim = static_cast<int32_t>(n);
    for (int64_t a = 0; a < n; ++a) {
      s->shape[a] = t.size(a);
      s->stride[a] = t.stride(a);
    }
  }

  // The view of `o`, or NULL for None.
  st_tensor* view(PyObject* o, st_tensor* s, const char* name) {
    const at::Tensor* t = tensor(o, name);
    if (!t) return nullptr;
    fill(*t, s, name);
    return s;
  }
};

// torch.empty on a CUDA device (its allocator, the device's current stream)
// without the way through the dispatcher.
at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType ty, int dev) {
  if (dev < 0) throw Refused(ST_ERR_INVALID_ARG, "no tensor was given");
  return at::Tensor(at::detail::empty_cuda(shape, ty, at::Device(at::kCUDA, static_cast<at::DeviceIndex>(dev)), std::nullopt));
}

// An output: the caller's tensor, or a new one.
struct Out {
  at::Tensor t;
  PyObject* given = nullptr;  // borrowed
  st_tensor s;
  void take(Call& c, PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType ty) {
    if (o != Py_None) {
      given = o;
      Call::fill(*c.tensor(o, name), &s, name);
    } else {
      t = new_tensor(shape, ty, c.dev);
      Call::fill(t, &s, name);
    }
  }
  PyObject* py() {
    if (given) {
      Py_INCREF(given);
      return given;
    }
    return THPVariable_Wrap(t);
  }
};

int64_t dim_of(const at::Tensor& t, int64_t a, const char* name) {
  if (t.dim() <= a) throw Refused(ST_ERR_SHAPE, std::string(name) + " has too few dims");
  return t.size(a);
}

void check(int status) {
  if (status != ST_OK) throw Refused(status, st_last_error());
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused(-1, "");
  return v;
}

// Runs `body` with C++ exceptions turned into Python ones.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused& e) {
    if (e.status >= 0 && !PyErr_Occurred()) {
      PyObject* x = PyObject_CallFunction(g_error, "is", e.status, e.msg.c_str());
      if (x) {
        PyErr_SetObject(g_error, x);
        Py_DECREF(x);
      }
    }
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// fn(stream) on device `dev`'s current stream, that device being current.
template <class F>
void launch(int dev, F&& fn) {
  if (dev < 0) throw Refused(ST_ERR_INVALID_ARG, "no tensor was given");
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = fn(stream);
  Py_END_ALLOW_THREADS
  check(status);
}

struct Cache {
  st_tensor k, v, pages, ks, vs;
  st_kv_cache c;
  st_kv_scales sc;
  const st_kv_scales* scales;  // NULL where neither is given
  at::ScalarType type;
  // a: k, v, pages, k_scale, v_scale
  void take(Call& call, PyObject* const* a) {
    const at::Tensor* kt = call.tensor(a[0], "cache.k");
    if (!kt) throw Refused(ST_ERR_INVALID_ARG, "cache.k is None");
    type = kt->scalar_type();
    Call::fill(*kt, &k, "cache.k");
    c.k = &k;
    c.v = call.view(a[1], &v, "cache.v");
    c.pages = call.view(a[2], &pages, "cache.pages");
    sc.k = call.view(a[3], &ks, "cache.k_scale");
    sc.v = call.view(a[4], &vs, "cache.v_scale");
    scales = sc.k || sc.v || held() ? &sc : nullptr;
  }
  bool held() const { return type == at::kFloat8_e4m3fn || type == at::kChar; }
};

// q, k, v, wq, wk, eps, ids, cos, sin, cos_k, sin_k, axes, theta, cache (5), lens, counts, q_rot
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 21, [&]() -> PyObject* {
    Call c;
    st_tensor s[12];
    Cache kv;
    st_rope r;
    std::memset(&r, 0, sizeof(r));
    const at::Tensor* qt = c.tensor(a[0], "q");
    if (!qt) throw Refused(ST_ERR_INVALID_ARG, "q is None");
    st_tensor *q = c.view(a[0], &s[0], "q"), *k = c.view(a[1], &s[1], "k"), *v = c.view(a[2], &s[2], "v");
    st_tensor *wq = c.view(a[3], &s[3], "q_norm_w"), *wk = c.view(a[4], &s[4], "k_norm_w");
    const float eps = static_cast<float>(number(a[5]));
    r.ids = c.view(a[6], &s[5], "ids");
    r.cos = c.view(a[7], &s[6], "cos");
    r.sin = c.view(a[8], &s[7], "sin");
    r.cos_k = c.view(a[9], &s[8], "cos_k");
    r.sin_k = c.view(a[10], &s[9], "sin_k");
    PyObject* axes = PySequence_Fast(a[11], "axes_dim must be a sequence");
    if (!axes) throw Refused(-1, "");
    const Py_ssize_t na = PySequence_Fast_GET_SIZE(axes);
    for (Py_ssize_t i = 0; i < na && i < 8; ++i) r.axes_dim[i] = static_cast<int32_t>(PyLong_AsLong(PySequence_Fast_GET_ITEM(axes, i)));
    Py_DECREF(axes);
    if (PyErr_Occurred()) throw Refused(-1, "");
    r.n_axes = static_cast<int32_t>(na);
    r.theta = number(a[12]);
    kv.take(c, a + 13);
    st_tensor *lens = c.view(a[18], &s[10], "lens"), *counts = c.view(a[19], &s[11], "counts");
    Out o;
    o.take(c, a[20], "q_rot", qt->sizes(), kv.held() && v ? c.tensor(a[2], "v")->scalar_type() : kv.type);
    launch(c.dev, [&](void* st) { return st_cache_append_held(q, k, v, wq, wk, eps, &r, &kv.c, kv.scales, lens, counts, &o.s, st); });
    return o.py();
  });
}

int32_t count(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused(-1, "");
  if (v != static_cast<int32_t>(v)) throw Refused(ST_ERR_INVALID_ARG, std::string(name) + " is out of range");
  return static_cast<int32_t>(v);
}

// q_rot, cache (5), lens, counts, parents, scale, o, lse, workspace, window, sinks, shared
PyObject* cache_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    Call c;
    st_tensor s[5];
    Cache kv;
    const at::Tensor* qt = c.tensor(a[0], "q_rot");
    if (!qt) throw Refused(ST_ERR_INVALID_ARG, "q_rot is None");
    st_tensor* q = c.view(a[0], &s[0], "q_rot");
    kv.take(c, a + 1);
    st_tensor *lens = c.view(a[6], &s[1], "lens"), *counts = c.view(a[7], &s[2], "counts"), *par = c.view(a[8], &s[3], "parents");
    const float scale = static_cast<float>(number(a[9]));
    const st_cache_attn_opts opts{kv.scales, count(a[13], "window"), count(a[14], "sinks"), c.view(a[15], &s[4], "shared")};
    const int64_t B = dim_of(*qt, 0, "q_rot"), T = dim_of(*qt, 1, "q_rot"), H = dim_of(*qt, 2, "q_rot");
    Out o, lse;
    o.take(c, a[10], "o", qt->sizes(), qt->scalar_type());
    lse.take(c, a[11], "lse", {B, H, T}, at::kFloat);
    at::Tensor ws;
    void* wp;
    size_t wn;
    if (a[12] == Py_None) {
      wn = st_cache_attn_opt_workspace_size(q, &kv.c, &opts, par);
      // a size of 0: refused arguments, for which the call itself has the status (it
      // plans first and needs no workspace to refuse)
      if (wn == 0) {
        check(st_cache_attn_opt(q, &kv.c, &opts, lens, counts, par, scale, &o.s, &lse.s, nullptr, 0, nullptr));
        throw Refused(ST_ERR_INVALID_ARG, "the workspace has no size");
      }
      ws = new_tensor({static_cast<int64_t>(wn)}, at::kByte, c.dev);
      wp = ws.data_ptr();
    } else {
      const at::Tensor* w = c.tensor(a[12], "workspace");
      if (!w->is_contiguous()) throw Refused(ST_ERR_INVALID_ARG, "the workspace must be contiguous");
      wp = w->numel() > 0 ? w->data_ptr() : nullptr;
      wn = w->nbytes();
    }
    launch(c.dev, [&](void* st) { return st_cache_attn_opt(q, &kv.c, &opts, lens, counts, par, scale, &o.s, &lse.s, wp, wn, st); });
    PyObject *x = o.py(), *y = lse.py();
    PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
  });
}

// target, draft, tokens, parents, counts, u_accept, u_sample, path, n_accepted, next_token
PyObject* tree_verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    Call c;
    st_tensor s[7];
    st_tensor *p = c.view(a[0], &s[0], "target_probs"), *q = c.view(a[1], &s[1], "draft_probs");
    const at::Tensor* tt = c.tensor(a[2], "tokens");
    if (!tt) throw Refused(ST_ERR_INVALID_ARG, "tokens is None");
    st_tensor* tok = c.view(a[2], &s[2], "tokens");
    st_tensor *par = c.view(a[3], &s[3], "parents"), *counts = c.view(a[4], &s[4], "counts");
    st_tensor *ua = c.view(a[5], &s[5], "u_accept"), *us = c.view(a[6], &s[6], "u_sample");
    const int64_t B = dim_of(*tt, 0, "tokens"), T = dim_of(*tt, 1, "tokens");
    Out path, acc, next;
    path.take(c, a[7], "path", {B, T}, at::kInt);
    acc.take(c, a[8], "n_accepted", {B}, at::kInt);
    next.take(c, a[9], "next_token", {B}, tt->scalar_type());
    launch(c.dev, [&](void* st) { return st_tree_verify(p, q, tok, par, counts, ua, us, &path.s, &acc.s, &next.s, st); });
    PyObject *x = path.py(), *y = acc.py(), *z = next.py();
    PyObject* r = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    Py_XDECREF(z);
    return r;
  });
}

// cache (5), start, rows, n_rows, lens
PyObject* cache_keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    Call c;
    st_tensor s[3];
    Cache kv;
    kv.take(c, a);
    const at::Tensor* st0 = c.tensor(a[5], "start");
    if (!st0) throw Refused(ST_ERR_INVALID_ARG, "start is None");
    st_tensor *start = c.view(a[5], &s[0], "start"), *rows = c.view(a[6], &s[1], "rows"), *cnt = c.view(a[7], &s[2], "n_rows");
    Out lens;
    lens.take(c, a[8], "lens", st0->sizes(), at::kInt);
    launch(c.dev, [&](void* st) { return st_cache_keep_held(&kv.c, kv.scales, start, rows, cnt, &lens.s, st); });
    return lens.py();
  });
}

// cache (5), start, T, counts, dtype (a torch.dtype or None), k, v
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    Call c;
    st_tensor s[2];
    Cache kv;
    kv.take(c, a);
    st_tensor *start = c.view(a[5], &s[0], "start"), *counts = c.view(a[7], &s[1], "counts");
    const int64_t T = count(a[6], "n_rows");
    if (T < 0) throw Refused(ST_ERR_INVALID_ARG, "n_rows must be at least 0");
    at::ScalarType ty = kv.held() ? at::kBFloat16 : kv.type;
    if (a[8] != Py_None) {
      if (!THPDtype_Check(a[8])) throw Refused(ST_ERR_INVALID_ARG, "dtype must be a torch.dtype");
      ty = reinterpret_cast<THPDtype*>(a[8])->scalar_type;
    }
    const at::Tensor *kt = c.tensor(a[0], "cache.k"), *pt = c.tensor(a[2], "cache.pages");
    if (!pt) throw Refused(ST_ERR_INVALID_ARG, "cache.pages is None");
    const int64_t B = dim_of(*pt, 0, "cache.pages"), H = dim_of(*kt, 2, "cache.k"), D = dim_of(*kt, 3, "cache.k");
    Out k, v;
    k.take(c, a[9], "k", {B, T, H, D}, ty);
    v.take(c, a[10], "v", {B, T, H, D}, ty);
    launch(c.dev, [&](void* st) { return st_cache_read(&kv.c, kv.scales, start, counts, &k.s, &v.s, st); });
    PyObject *x = k.py(), *y = v.py();
    PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
  });
}

PyObject* init(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

#define ST_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef kMethods[] = {{"init", init, METH_O, nullptr},
                          {"cache_append", ST_FAST(cache_append)},
                          {"cache_attn", ST_FAST(cache_attn)},
                          {"tree_verify", ST_FAST(tree_verify)},
                          {"cache_keep", ST_FAST(cache_keep)},
                          {"cache_read", ST_FAST(cache_read)},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "st_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_st_bind(void) { return PyModule_Create(&kModule); }
