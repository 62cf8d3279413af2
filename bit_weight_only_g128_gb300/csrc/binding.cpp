// The binding's calls of the decoder layer's operators (norm, rotation and
// append, attention), as a CPython module: argument checks, allocation of the
// results and the call of the C ABI in one native step, for calls whose
// kernels take a few microseconds. The entry points come from the library that
// the package has loaded (bind), the results' memory and the current stream
// from PyTorch. The package's layer.py documents the functions.
#include <Python.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "w4a16.h"

namespace {

struct Library {
  decltype(&w4a16_rms_norm) rms_norm;
  decltype(&w4a16_rope_append) rope_append;
  decltype(&w4a16_attn_workspace_size) attn_workspace_size;
  decltype(&w4a16_attn_decode) attn_decode;
  decltype(&w4a16_attn_prompt) attn_prompt;
} lib;
PyObject* on_error = nullptr;   // (code, entry point): raises the package's error
PyObject* workspace_of = nullptr;  // (bytes, device, stream): the stream's workspace
PyObject *name_k, *name_v, *name_k_scale, *name_v_scale, *name_cuda_stream;

// A Python exception that is set (or is set by the text).
struct Raised {};

[[noreturn]] void refuse(const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  PyErr_SetString(PyExc_ValueError, buf);
  throw Raised();
}

std::string text(const at::Device& d) { return d.str(); }
std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}
const char* text(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kChar: return "torch.int8";
    case at::kByte: return "torch.uint8";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return at::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

int flags16(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kHalf) return 0;
  if (t.scalar_type() == at::kBFloat16) return W4A16_BF16;
  refuse("%s must be float16 or bfloat16, got %s", name, text(t.scalar_type()));
}

void check_place(const at::Tensor& t, const char* name, at::ScalarType type, const at::Device& dev) {
  if (t.scalar_type() != type) refuse("%s must be %s, got %s", name, text(type), text(t.scalar_type()));
  if (!t.is_cuda() || t.device() != dev) refuse("%s must be a CUDA tensor on %s", name, text(dev).c_str());
}

// Row stride of a 2-D tensor [rows, cols] with adjacent columns.
int64_t rows_of(const at::Tensor& t, const char* name, int64_t cols, at::ScalarType type, const at::Device& dev) {
  check_place(t, name, type, dev);
  if (t.dim() != 2 || t.size(1) != cols) refuse("%s must have %lld columns, got shape %s", name, (long long)cols, text(t.sizes()).c_str());
  if (cols > 1 && t.stride(1) != 1) refuse("%s's rows must be contiguous", name);
  return t.size(0) > 1 ? t.stride(0) : cols;
}

// Pointer of a contiguous tensor of n elements.
template <class T>
T* flat(const at::Tensor& t, const char* name, int64_t n, at::ScalarType type, const at::Device& dev) {
  check_place(t, name, type, dev);
  if (t.numel() != n || !t.is_contiguous())
    refuse("%s must be contiguous with %lld elements, got shape %s", name, (long long)n, text(t.sizes()).c_str());
  return static_cast<T*>(t.data_ptr());
}

// A new contiguous tensor on a CUDA device (without the dispatcher's round).
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
  return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

at::Tensor result(PyObject* given, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
  if (given == Py_None) return fresh(shape, type, dev);
  const at::Tensor& t = tensor(given, name);
  int64_t n = 1;
  for (int64_t s : shape) n *= s;
  flat<void>(t, name, n, type, dev);
  return t;
}

// The call's stream: the current one of the tensors' device, or the given
// torch.cuda.Stream, which is then the current one while results and workspace
// are allocated (and the workspace's zeros written): they belong to it. The
// library works on the current device (its SM count, error word and launches),
// so that is the tensors' for the call.
struct CallStream {
  void* ptr;
  c10::cuda::OptionalCUDAGuard device;  // (empty where it is current already: one query less)
  c10::cuda::OptionalCUDAStreamGuard guard;

  CallStream(PyObject* o, const at::Device& dev) {
    if (c10::cuda::current_device() != dev.index()) device.set_device(dev);
    if (o == Py_None) {
      ptr = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
      return;
    }
    PyObject* s = PyObject_GetAttr(o, name_cuda_stream);
    if (!s) throw Raised();
    ptr = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (!ptr && PyErr_Occurred()) throw Raised();
    guard.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(ptr), dev.index()));
  }
};

int int32_of(int64_t v, const char* name) {
  if (v > 0x7fffffff) refuse("%s=%lld is above 2^31 - 1", name, (long long)v);
  return (int)v;
}

void check(int rc, const char* where) {
  if (rc == 0) return;
  PyObject* r = PyObject_CallFunction(on_error, "is", rc, where);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, where);
  throw Raised();
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

PyObject* wrap(const at::Tensor& given, PyObject* o) {
  if (o == Py_None) return wrap(given);
  Py_INCREF(o);
  return o;
}

// A new tuple of new references.
PyObject* tuple(PyObject* a, PyObject* b, PyObject* c = nullptr) {
  PyObject* t = a && b ? PyTuple_New(c ? 3 : 2) : nullptr;
  if (!t) {
    Py_XDECREF(a);
    Py_XDECREF(b);
    Py_XDECREF(c);
    throw Raised();
  }
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  if (c) PyTuple_SET_ITEM(t, 2, c);
  return t;
}

// Runs a call, turning C++ exceptions into Python's.
template <class F>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t want, F&& call) {
  if (nargs != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, nargs);
    return nullptr;
  }
  if (!on_error) {
    PyErr_SetString(PyExc_RuntimeError, "no library is bound");
    return nullptr;
  }
  try {
    return call();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// rms_norm(x, weight, residual, eps, quant, out, residual_out, stream)
PyObject* rms_norm(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded(nargs, 8, [&]() -> PyObject* {
    const at::Tensor& x = tensor(args[0], "x");
    const int flags = flags16(x, "x");
    if (x.dim() != 2) refuse("x must be [M, K], got shape %s", text(x.sizes()).c_str());
    const int64_t M = x.size(0), K = x.size(1);
    const at::Device dev = x.device();
    const at::ScalarType type = x.scalar_type();
    const int64_t ldx = rows_of(x, "x", K, type, dev);
    const auto* w = flat<uint16_t>(tensor(args[1], "weight"), "weight", K, type, dev);
    const double eps = PyFloat_AsDouble(args[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised();
    const CallStream stream(args[7], dev);
    const uint16_t* r = nullptr;
    uint16_t* hp = nullptr;
    int64_t ldr = 0, ldh = 0;
    at::Tensor h;
    if (args[2] != Py_None) {
      const at::Tensor& res = tensor(args[2], "residual");
      ldr = rows_of(res, "residual", K, type, dev);
      if (res.size(0) != M) refuse("residual has %lld rows, x has %lld", (long long)res.size(0), (long long)M);
      r = static_cast<uint16_t*>(res.data_ptr());
      h = args[6] == Py_None ? fresh({M, K}, type, dev) : tensor(args[6], "residual_out");
      ldh = rows_of(h, "residual_out", K, type, dev);
      if (h.size(0) != M) refuse("residual_out has %lld rows, x has %lld", (long long)h.size(0), (long long)M);
      hp = static_cast<uint16_t*>(h.data_ptr());
    } else if (args[6] != Py_None) {
      refuse("residual_out goes with residual");
    }
    bool int8 = false, codes = false;
    if (args[4] != Py_None) {
      const char* q = PyUnicode_Check(args[4]) ? PyUnicode_AsUTF8(args[4]) : nullptr;
      int8 = q && std::string(q) == "int8";
      codes = q && std::string(q) == "codes";
      if (!int8 && !codes) {
        PyErr_Format(PyExc_ValueError, "quant must be None, 'int8' or 'codes', got %R", args[4]);
        throw Raised();
      }
    }
    const at::Tensor y = result(args[5], "out", {M, K}, int8 ? at::kChar : type, dev);
    at::Tensor scale;
    float* sp = nullptr;
    if (int8 || codes) {
      scale = fresh({M}, at::kFloat, dev);
      sp = scale.data_ptr<float>();
    }
    void* yp = y.data_ptr();
    check(lib.rms_norm(static_cast<uint16_t*>(x.data_ptr()), ldx, r, ldr, w, int32_of(M, "M"), int32_of(K, "K"), (float)eps, flags,
                       int8 || codes ? nullptr : static_cast<uint16_t*>(yp), codes ? static_cast<uint16_t*>(yp) : nullptr,
                       int8 ? static_cast<int8_t*>(yp) : nullptr, sp, hp, ldh, stream.ptr),
          "w4a16_rms_norm");
    // (not by the pointers: those of no rows are null)
    const bool quant = int8 || codes, residual = args[2] != Py_None;
    PyObject* yo = wrap(y, args[5]);
    if (!quant && !residual) return yo;
    if (!quant) return tuple(yo, wrap(h, args[6]));
    if (!residual) return tuple(yo, wrap(scale));
    return tuple(yo, wrap(scale), wrap(h, args[6]));
  });
}

// The tensors of a KVCache, checked against 16-bit type `type` on `dev`.
struct Cache {
  void *k, *v;
  const float *k_scale = nullptr, *v_scale = nullptr;
  int pages, heads, page_size, dim, flags = 0;

  Cache(PyObject* o, at::ScalarType type, const at::Device& dev) {
    Held ko(o, name_k), vo(o, name_v), kso(o, name_k_scale), vso(o, name_v_scale);
    const at::Tensor &kt = tensor(ko.o, "cache k"), &vt = tensor(vo.o, "cache v");
    if (kt.dim() != 4 || vt.sizes() != kt.sizes())
      refuse("cache k and v must be [pages, kv_heads, page_size, head_dim] alike, got %s and %s", text(kt.sizes()).c_str(),
             text(vt.sizes()).c_str());
    pages = int32_of(kt.size(0), "pages");
    heads = int32_of(kt.size(1), "kv_heads");
    page_size = int32_of(kt.size(2), "page_size");
    dim = int32_of(kt.size(3), "head_dim");
    if (kt.scalar_type() == at::kFloat8_e4m3fn) {
      if (kso.o == Py_None || vso.o == Py_None) refuse("a float8_e4m3fn cache needs k_scale and v_scale");
      flags = W4A16_CACHE_E4M3;
      k_scale = flat<float>(tensor(kso.o, "k_scale"), "k_scale", heads, at::kFloat, dev);
      v_scale = flat<float>(tensor(vso.o, "v_scale"), "v_scale", heads, at::kFloat, dev);
    } else {
      if (kso.o != Py_None || vso.o != Py_None) refuse("scales go with a float8_e4m3fn cache only");
      if (kt.scalar_type() != type)
        refuse("the cache must be %s or float8_e4m3fn, got %s", text(type), text(kt.scalar_type()));
    }
    if (vt.scalar_type() != kt.scalar_type() || !kt.is_cuda() || kt.device() != dev || vt.device() != dev)
      refuse("cache k and v must be CUDA tensors of one type on %s", text(dev).c_str());
    if (!kt.is_contiguous() || !vt.is_contiguous()) refuse("cache k and v must be contiguous");
    k = kt.data_ptr();
    v = vt.data_ptr();
  }

 private:
  struct Held {
    PyObject* o;
    Held(PyObject* from, PyObject* name) : o(PyObject_GetAttr(from, name)) {
      if (!o) throw Raised();
    }
    ~Held() { Py_XDECREF(o); }
  };
};

// rope_append(qkv, cos_sin, positions, slots, cache, interleaved, out, stream)
PyObject* rope_append(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded(nargs, 8, [&]() -> PyObject* {
    const at::Tensor& qkv = tensor(args[0], "qkv");
    const int flags = flags16(qkv, "qkv");
    const at::Device dev = qkv.device();
    const at::ScalarType type = qkv.scalar_type();
    const Cache c(args[4], type, dev);
    if (qkv.dim() != 2 || c.dim == 0 || qkv.size(1) % c.dim || qkv.size(1) / c.dim <= 2 * c.heads)
      refuse("qkv must be [T, (heads + 2 * %d) * %d], got shape %s", c.heads, c.dim, text(qkv.sizes()).c_str());
    const int64_t T = qkv.size(0), cols = qkv.size(1);
    const int heads = int32_of(cols / c.dim - 2 * c.heads, "heads");
    const int64_t ld = rows_of(qkv, "qkv", cols, type, dev);
    const at::Tensor& cs = tensor(args[1], "cos_sin");
    if (cs.dim() != 2) refuse("cos_sin must be [table_len, rotary], got shape %s", text(cs.sizes()).c_str());
    const auto* table = flat<float>(cs, "cos_sin", cs.numel(), at::kFloat, dev);
    const auto* pos = flat<int32_t>(tensor(args[2], "positions"), "positions", T, at::kInt, dev);
    const auto* slots = flat<int64_t>(tensor(args[3], "slots"), "slots", T, at::kLong, dev);
    const int interleaved = PyObject_IsTrue(args[5]);
    if (interleaved < 0) throw Raised();
    const CallStream stream(args[7], dev);
    const at::Tensor q = result(args[6], "out", {T, heads, c.dim}, type, dev);
    check(lib.rope_append(static_cast<uint16_t*>(qkv.data_ptr()), ld, table, int32_of(cs.size(0), "table_len"),
                          int32_of(cs.size(1), "rotary"), pos, slots, int32_of(T, "tokens"), heads, c.heads, c.dim,
                          static_cast<uint16_t*>(q.data_ptr()), c.k, c.v, c.k_scale, c.v_scale, c.pages, c.page_size,
                          flags | c.flags | (interleaved ? W4A16_ROPE_INTERLEAVED : 0), stream.ptr),
          "w4a16_rope_append");
    return wrap(q, args[6]);
  });
}

// attend(q, cache, table, starts, lens, scale, out, return_lse, workspace, stream);
// starts None: a row per sequence
PyObject* attend(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded(nargs, 10, [&]() -> PyObject* {
    const at::Tensor& q = tensor(args[0], "q");
    const int flags = flags16(q, "q");
    const at::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const Cache c(args[1], type, dev);
    if (q.dim() != 3 || q.size(2) != c.dim) refuse("q must be [tokens, heads, %d], got shape %s", c.dim, text(q.sizes()).c_str());
    const int64_t T = q.size(0), heads = q.size(1);
    if (q.stride(2) != 1 || (heads > 1 && q.stride(1) != c.dim)) refuse("q's heads must be adjacent");
    const int64_t ldq = T > 1 ? q.stride(0) : heads * c.dim;
    const at::Tensor& table = tensor(args[2], "table");
    if (table.dim() != 2) refuse("table must be [batch, pages], got shape %s", text(table.sizes()).c_str());
    const int64_t batch = table.size(0), most = table.size(1);
    const int64_t ldt = rows_of(table, "table", most, at::kInt, dev);
    const bool decode = args[3] == Py_None;
    if (decode && T != batch) refuse("q has %lld rows, the table %lld", (long long)T, (long long)batch);
    const auto* lens = flat<int32_t>(tensor(args[4], "lens"), "lens", batch, at::kInt, dev);
    const auto* starts = decode ? nullptr : flat<int32_t>(tensor(args[3], "starts"), "starts", batch + 1, at::kInt, dev);
    double scale;
    if (args[5] == Py_None) {
      scale = 1.0 / std::sqrt((double)c.dim);
    } else {
      scale = PyFloat_AsDouble(args[5]);
      if (scale == -1.0 && PyErr_Occurred()) throw Raised();
    }
    const CallStream stream(args[9], dev);
    const at::Tensor out = result(args[6], "out", {T, heads, c.dim}, type, dev);
    const int want_lse = PyObject_IsTrue(args[7]);
    if (want_lse < 0) throw Raised();
    at::Tensor lse;
    if (want_lse) lse = fresh({T, heads}, at::kFloat, dev);
    float* lp = want_lse ? lse.data_ptr<float>() : nullptr;
    const int t32 = int32_of(T, "tokens"), b32 = int32_of(batch, "batch"), h32 = int32_of(heads, "heads"),
              m32 = int32_of(most, "max_pages");
    size_t need = 0;
    if (T > 0) check(lib.attn_workspace_size(t32, b32, h32, c.heads, c.dim, &need), "w4a16_attn_workspace_size");
    at::Tensor ws;
    if (args[8] != Py_None) {
      ws = tensor(args[8], "workspace");
      if (!ws.is_cuda() || ws.device() != dev || !ws.is_contiguous())
        refuse("workspace must be a contiguous CUDA tensor on %s", text(dev).c_str());
    } else if (need) {
      PyObject* o = PyObject_CallFunction(workspace_of, "niK", (Py_ssize_t)need, (int)dev.index(),
                                          (unsigned long long)(uintptr_t)stream.ptr);
      if (!o) throw Raised();
      ws = THPVariable_Unpack(o);
      Py_DECREF(o);
    }
    void* wp = ws.defined() ? ws.data_ptr() : nullptr;
    const size_t wb = ws.defined() ? ws.nbytes() : 0;
    auto* qp = static_cast<uint16_t*>(q.data_ptr());
    auto* op = static_cast<uint16_t*>(out.data_ptr());
    const auto* tp = static_cast<int32_t*>(table.data_ptr());
    if (decode)
      check(lib.attn_decode(qp, ldq, c.k, c.v, c.k_scale, c.v_scale, c.pages, c.page_size, tp, ldt, m32, lens, b32, h32, c.heads,
                            c.dim, (float)scale, op, lp, wp, wb, flags | c.flags, stream.ptr),
            "w4a16_attn_decode");
    else
      check(lib.attn_prompt(qp, ldq, c.k, c.v, c.k_scale, c.v_scale, c.pages, c.page_size, tp, ldt, m32, starts, lens, t32, b32,
                            h32, c.heads, c.dim, (float)scale, op, lp, wp, wb, flags | c.flags, stream.ptr),
            "w4a16_attn_prompt");
    PyObject* o = wrap(out, args[6]);
    return want_lse ? tuple(o, wrap(lse)) : o;
  });
}

// bind(addresses of the five entry points, error function, workspace function)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 7) {
    PyErr_SetString(PyExc_TypeError, "7 arguments expected");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
      return nullptr;
    }
  }
  lib.rms_norm = reinterpret_cast<decltype(lib.rms_norm)>(p[0]);
  lib.rope_append = reinterpret_cast<decltype(lib.rope_append)>(p[1]);
  lib.attn_workspace_size = reinterpret_cast<decltype(lib.attn_workspace_size)>(p[2]);
  lib.attn_decode = reinterpret_cast<decltype(lib.attn_decode)>(p[3]);
  lib.attn_prompt = reinterpret_cast<decltype(lib.attn_prompt)>(p[4]);
  Py_INCREF(args[5]);
  Py_INCREF(args[6]);
  Py_XDECREF(on_error);
  Py_XDECREF(workspace_of);
  on_error = args[5];
  workspace_of = args[6];
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&bind)), METH_FASTCALL, nullptr},
    {"rms_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&rms_norm)), METH_FASTCALL, nullptr},
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&rope_append)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&attend)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  name_k = PyUnicode_InternFromString("k");
  name_v = PyUnicode_InternFromString("v");
  name_k_scale = PyUnicode_InternFromString("k_scale");
  name_v_scale = PyUnicode_InternFromString("v_scale");
  name_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (!name_k || !name_v || !name_k_scale || !name_v_scale || !name_cuda_stream) return nullptr;
  return PyModule_Create(&module);
}
