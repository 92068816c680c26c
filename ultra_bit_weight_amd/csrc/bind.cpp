// Argument checks and marshalling of the attention entry points for Python.
//
// A decode step calls them once a layer, for kernels of two to five
// microseconds, so the checks of the binding (shapes, types, devices, strides of
// up to ten tensors) are done here on the tensors themselves: about 1 us a call
// against 4 us through Python attributes.  No computation: every function checks,
// calls the C ABI (include/sherry.h) and returns its status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <dlfcn.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "sherry.h"

namespace {

struct Refused {};  // a Python exception is set

[[noreturn]] void type_error(const char* name) {
  PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
  throw Refused{};
}
[[noreturn]] void value_error(const std::string& text) {
  PyErr_SetString(PyExc_ValueError, text.c_str());
  throw Refused{};
}

std::string text(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}
std::string text(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return "float16";
    case at::kBFloat16: return "bfloat16";
    case at::kFloat: return "float32";
    case at::kInt: return "int32";
    case at::kLong: return "int64";
    default: return c10::toString(t);
  }
}
std::string text(const at::Tensor& t) {
  return text(t.scalar_type()) + " " + text(t.sizes()) + " with strides " + text(t.strides()) +
         " on " + t.device().str();
}

int device_of(const at::Tensor& t) { return t.device().is_cuda() ? t.device().index() : -1; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(name);
  return THPVariable_Unpack(o);
}
bool none(PyObject* o) { return o == Py_None; }

sherry_dtype fp_dtype(const at::Tensor& t, const char* name, bool f32) {
  switch (t.scalar_type()) {
    case at::kHalf: return SHERRY_F16;
    case at::kBFloat16: return SHERRY_BF16;
    case at::kFloat:
      if (f32) return SHERRY_F32;
      [[fallthrough]];
    default: value_error(std::string(name) + " has dtype " + text(t.scalar_type()) + ", expected " +
                         (f32 ? "float32, float16 or bfloat16" : "float16 or bfloat16"));
  }
}

[[noreturn]] void refuse(const at::Tensor& t, const char* name, const char* layout, at::ScalarType dt,
                         at::IntArrayRef shape, int dev) {
  value_error(std::string(name) + " must be " + layout + " " + text(dt) + " " + text(shape) + " on " +
              (dev >= 0 ? "GPU " + std::to_string(dev) : std::string("the GPU")) + ", got " + text(t));
}

struct Rows {
  void* p;
  int64_t st, sh;
};
// [tokens, heads, head_dim] with unit stride along head_dim
Rows rows(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dt, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.sizes() != shape || t.scalar_type() != dt || device_of(t) != dev || (t.stride(2) != 1 && shape[2] > 1))
    refuse(t, name, "unit-stride (along head_dim)", dt, shape, dev);
  return {t.data_ptr(), t.stride(0), t.stride(1)};
}
void* flat(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dt, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.sizes() != shape || t.scalar_type() != dt || device_of(t) != dev || !t.is_contiguous())
    refuse(t, name, "contiguous", dt, shape, dev);
  return t.data_ptr();
}
const at::Tensor& dims(PyObject* o, const char* name, int64_t n, const char* layout) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != n) value_error(std::string(name) + " must be " + layout + ", got shape " + text(t.sizes()));
  return t;
}
void on_gpu(int dev) {
  if (dev < 0) value_error("tensors must be on the GPU");
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
// an int argument of the C ABI: one that does not fit is as wrong as a negative one
int32_t integer32(PyObject* o) {
  const int64_t v = integer(o);
  return v < 0 || v > INT32_MAX ? -1 : static_cast<int32_t>(v);
}
// a size that the C ABI takes as an int: a larger one is refused there like the largest
int32_t small(int64_t v) { return static_cast<int32_t>(v > INT32_MAX ? INT32_MAX : v); }
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
hipStream_t stream(PyObject* o) { return reinterpret_cast<hipStream_t>(static_cast<uintptr_t>(integer(o))); }

decltype(&sherry_qk_norm_rope) g_rope;
decltype(&sherry_kv4_write) g_write;
decltype(&sherry_kv4_read) g_read;
decltype(&sherry_kv4_attn) g_attn;

// The call itself without the interpreter's lock: a launch waits when its queue
// is full.  The caller's frame holds the tensors and the cache.
template <class F, class... A>
PyObject* call(F f, A... args) {
  int status;
  Py_BEGIN_ALLOW_THREADS status = f(args...);
  Py_END_ALLOW_THREADS return PyLong_FromLong(status);
}

// The cache's descriptor (a sherry_kv4_cache at an address that the Python
// object keeps) and its device.
struct Cache {
  const sherry_kv4_cache* desc;
  int dev;
  Cache(PyObject* address, PyObject* device)
      : desc(reinterpret_cast<const sherry_kv4_cache*>(static_cast<uintptr_t>(integer(address)))),
        dev(static_cast<int>(integer(device))) {}
};

// q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved, q_out, k_out, stream
PyObject* rope(PyObject* const* a) {
  static const char* kHeads = "[tokens, heads, head_dim]";
  const at::Tensor& q = dims(a[0], "q", 3, kHeads);
  const int dev = device_of(q);
  const at::ScalarType x_st = q.scalar_type();
  const sherry_dtype x_dt = fp_dtype(q, "q", true);
  const at::Tensor& q_out = tensor(a[9], "q_out");
  const at::ScalarType y_st = q_out.scalar_type();
  const sherry_dtype y_dt = fp_dtype(q_out, "q_out", true);
  const int64_t n = q.size(0), d = q.size(2);
  auto side = [&](PyObject* x, PyObject* y, PyObject* w, const char* xn, const char* yn, const char* wn) {
    const int64_t shape[3] = {n, dims(x, xn, 3, kHeads).size(1), d};
    const Rows xr = rows(x, xn, shape, x_st, dev), yr = rows(y, yn, shape, y_st, dev);
    void* wp = none(w) ? nullptr : flat(w, wn, {d}, at::kFloat, dev);
    return sherry_heads{xr.p, yr.p, static_cast<const float*>(wp), xr.st, xr.sh, yr.st, yr.sh,
                        small(shape[1])};
  };
  const sherry_heads qs = side(a[0], a[9], a[5], "q", "q_out", "q_weight");
  sherry_heads ks{};
  const bool has_k = !none(a[1]);
  if (has_k)
    ks = side(a[1], a[10], a[6], "k", "k_out", "k_weight");
  else if (!none(a[10]) || !none(a[6]))
    value_error("k_out and k_weight need k");
  const at::Tensor& cos = dims(a[2], "cos", 2, "[max_pos, rot_dim / 2]");
  const float* cp = static_cast<const float*>(flat(a[2], "cos", cos.sizes(), at::kFloat, dev));
  const float* sp = static_cast<const float*>(flat(a[3], "sin", cos.sizes(), at::kFloat, dev));
  const int64_t* pp = static_cast<const int64_t*>(flat(a[4], "positions", {n}, at::kLong, dev));
  const float eps = static_cast<float>(real(a[7]));
  const int inter = PyObject_IsTrue(a[8]);
  on_gpu(dev);
  const int64_t rot = 2 * cos.size(1);
  return call(g_rope, &qs, has_k ? &ks : nullptr, x_dt, y_dt, n, small(d), small(rot), inter, cp, sp, cos.size(0), pp,
              eps, stream(a[11]));
}

// cache, device, k, v, slots, stream
template <bool kWrite>
PyObject* kv_rows(PyObject* const* a) {
  const Cache c(a[0], a[1]);
  const at::Tensor& slots = dims(a[4], "slots", 1, "[n]");
  const int64_t* sp = static_cast<const int64_t*>(flat(a[4], "slots", slots.sizes(), at::kLong, c.dev));
  const char *kn = kWrite ? "k" : "k_out", *vn = kWrite ? "v" : "v_out";
  const at::Tensor& k = tensor(a[2], kn);
  const sherry_dtype dt = fp_dtype(k, kn, true);
  const int64_t shape[3] = {slots.size(0), c.desc->n_kv_heads, c.desc->head_dim};
  const Rows kr = rows(a[2], kn, shape, k.scalar_type(), c.dev), vr = rows(a[3], vn, shape, k.scalar_type(), c.dev);
  on_gpu(c.dev);
  if constexpr (kWrite)
    return call(g_write, c.desc, kr.p, vr.p, dt, shape[0], kr.st, kr.sh, vr.st, vr.sh, sp, stream(a[5]));
  else
    return call(g_read, c.desc, kr.p, vr.p, dt, shape[0], kr.st, kr.sh, vr.st, vr.sh, sp, stream(a[5]));
}

// cache, device, q, page_table, kv_lens, cu_q, max_q, max_kv, scale, out, lse, workspace, stream
PyObject* attn(PyObject* const* a) {
  const Cache c(a[0], a[1]);
  const at::Tensor& q = dims(a[2], "q", 3, "[tokens, heads, head_dim]");
  const sherry_dtype dt = fp_dtype(q, "q", false);
  const int64_t n = q.size(0), hq = q.size(1);
  const int64_t shape[3] = {n, hq, c.desc->head_dim};
  const Rows qr = rows(a[2], "q", shape, q.scalar_type(), c.dev), yr = rows(a[9], "out", shape, q.scalar_type(), c.dev);
  const at::Tensor& table = dims(a[3], "page_table", 2, "[n_seqs, width]");
  const int64_t seqs = table.size(0), width = table.size(1);
  if (table.scalar_type() != at::kInt || device_of(table) != c.dev || (table.stride(1) != 1 && width > 1))
    refuse(table, "page_table", "unit-stride (along its rows)", at::kInt, table.sizes(), c.dev);
  const int32_t* lens = static_cast<const int32_t*>(flat(a[4], "kv_lens", {seqs}, at::kInt, c.dev));
  const int32_t* cu = none(a[5]) ? nullptr : static_cast<const int32_t*>(flat(a[5], "cu_q", {seqs + 1}, at::kInt, c.dev));
  float* lse = none(a[10]) ? nullptr : static_cast<float*>(flat(a[10], "lse", {n, hq}, at::kFloat, c.dev));
  const at::Tensor& ws = tensor(a[11], "workspace");
  const size_t ws_bytes = ws.numel() * ws.element_size();
  if (!ws.is_contiguous() || (ws_bytes && device_of(ws) != c.dev))
    value_error("workspace must be contiguous and on the cache's device, got " + text(ws));
  const int32_t max_q = integer32(a[6]);
  const int64_t max_kv = integer(a[7]);
  const float scale = static_cast<float>(real(a[8]));
  on_gpu(c.dev);
  return call(g_attn, c.desc, qr.p, dt, n, small(hq), qr.st, qr.sh, cu, small(seqs), max_q, max_kv,
              static_cast<const int32_t*>(table.data_ptr()), small(width), table.stride(0), lens, scale, yr.p, yr.st,
              yr.sh, lse, ws_bytes ? ws.data_ptr() : nullptr, ws_bytes, stream(a[12]));
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {  // no C++ exception leaves a C entry
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// attach(path): the library whose C ABI the calls go to
PyObject* attach(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* lib = dlopen(p, RTLD_NOW);
  if (!lib) {
    PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
    return nullptr;
  }
  auto find = [&](const char* name, auto& f) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(lib, name));
    if (!f) PyErr_Format(PyExc_RuntimeError, "%s has no %s", p, name);
    return f != nullptr;
  };
  if (!find("sherry_qk_norm_rope", g_rope) || !find("sherry_kv4_write", g_write) || !find("sherry_kv4_read", g_read) ||
      !find("sherry_kv4_attn", g_attn))
    return nullptr;
  Py_RETURN_NONE;
}

#define SHERRY_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f))
PyMethodDef kMethods[] = {
    {"attach", attach, METH_O, "attach(path): use this build of the library"},
    {"qk_norm_rope", SHERRY_FAST((&entry<rope, 12>)), METH_FASTCALL, nullptr},
    {"kv4_write", SHERRY_FAST((&entry<kv_rows<true>, 6>)), METH_FASTCALL, nullptr},
    {"kv4_read", SHERRY_FAST((&entry<kv_rows<false>, 6>)), METH_FASTCALL, nullptr},
    {"kv4_attn", SHERRY_FAST((&entry<attn, 13>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_sherry_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sherry_bind() { return PyModule_Create(&kModule); }
