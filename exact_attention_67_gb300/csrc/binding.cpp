// binding.cpp -- the Python side of the paged-cache calls: checks the tensors and
// calls the C ABI (include/exattn.h).  Compiled by the host compiler into
// _build/_exattn_binding.so, a Python module that paged.py forwards to.
//
// These calls are made once a layer and token when serving, on kernels of a few
// microseconds; through ctypes and Python's own attribute reads a call took 14
// to 27 us on the host, of which the C call was 4 to 7; through this module an
// append takes 2.5, an attention call 5.8.  Nothing here computes and nothing is
// kept from call to call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <string>
#include <utility>
#include <vector>

#include "exattn.h"

namespace {

// A refusal: the Python exception and its text.
struct Refused {
  PyObject* type;
  std::string text;
};

[[noreturn]] void bad_value(const std::string& text) { throw Refused{PyExc_ValueError, text}; }
[[noreturn]] void bad_type(const std::string& text) { throw Refused{PyExc_TypeError, text}; }

std::string shape_of(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// A bf16/f16 view with `dims` axes, d contiguous, of the given type if any.
const at::Tensor& operand(PyObject* o, const char* name, int dims, const at::Tensor* like = nullptr) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf)
    bad_type(std::string(name) + " must be bfloat16 or float16");
  if (t.dim() != dims)
    bad_value(std::string(name) + " must have " + std::to_string(dims) + " axes, got " + shape_of(t));
  if (t.size(dims - 1) > 1 && t.stride(dims - 1) != 1)
    bad_value(std::string(name) + ": the d axis must be contiguous (stride 1)");
  if (like && t.scalar_type() != like->scalar_type()) bad_value(std::string(name) + " must be of the first tensor's type");
  return t;
}

const at::Tensor& same(PyObject* o, const char* name, const at::Tensor& like) {
  const at::Tensor& t = operand(o, name, static_cast<int>(like.dim()), &like);
  if (t.sizes() != like.sizes()) bad_value(std::string(name) + " must be " + shape_of(like) + ", got " + shape_of(t));
  return t;
}

const at::Tensor& int32(PyObject* o, const char* name, std::initializer_list<int64_t> shape) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kInt) bad_type(std::string(name) + " must be int32");
  if (t.sizes() != at::IntArrayRef(shape)) bad_value(std::string(name) + ": unexpected shape " + shape_of(t));
  if (t.dim() && t.size(-1) > 1 && t.stride(-1) != 1) bad_value(std::string(name) + ": the last axis must be contiguous");
  return t;
}

int rotary_dim(const at::Tensor& f) {
  if (f.scalar_type() != at::kDouble || f.dim() != 1 || !f.is_contiguous())
    bad_value("inv_freq must be a contiguous float64 tensor [rot_dim / 2] (rotary_frequencies)");
  return static_cast<int>(2 * f.numel());
}

exattn_strides strides4(const at::Tensor& t) { return {t.stride(0), t.stride(1), t.stride(2)}; }
exattn_strides strides3(const at::Tensor& t) { return {0, t.stride(1), t.stride(0)}; }
int dtype_of(const at::Tensor& t) { return t.scalar_type() == at::kHalf ? EXATTN_DTYPE_F16 : EXATTN_DTYPE_BF16; }

// An extent or count as the C ABI takes it.
int as_int(int64_t n, const char* name) {
  if (n < 0 || n > INT32_MAX) bad_value(std::string(name) + " is out of range");
  return static_cast<int>(n);
}
int as_int(PyObject* o, const char* name) {
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
  if (n < INT32_MIN || n > INT32_MAX) bad_value(std::string(name) + " is out of range");
  return static_cast<int>(n);
}
float as_float(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return static_cast<float>(x);
}
int truth(PyObject* o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) throw Refused{nullptr, ""};
  return t;
}

// The one CUDA device of a call's tensors, made current for the call's length,
// and its stream: the given one (a torch stream or a raw handle) or, for None,
// the device's current one.
class OnDevice {
 public:
  explicit OnDevice(const at::Tensor& first) : dev_(first.is_cuda() ? first.get_device() : -1) {
    if (dev_ < 0) bad_value("all device operands must be CUDA tensors");
  }
  void also(const at::Tensor& t) const {
    if (!t.is_cuda()) bad_value("all device operands must be CUDA tensors");
    if (t.get_device() != dev_) bad_value("operands are on different devices");
  }
  void* enter(PyObject* stream) {
    void* s;
    if (stream == Py_None) {
      s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev_)).stream();
    } else if (PyLong_Check(stream)) {
      s = PyLong_AsVoidPtr(stream);
      if (!s && PyErr_Occurred()) throw Refused{nullptr, ""};
    } else {
      PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
      if (!h) throw Refused{nullptr, ""};
      s = PyLong_AsVoidPtr(h);
      Py_DECREF(h);
      if (!s && PyErr_Occurred()) throw Refused{nullptr, ""};
    }
    const int now = c10::cuda::current_device();
    if (now != dev_) {
      c10::cuda::set_device(static_cast<c10::DeviceIndex>(dev_));
      back_ = now;
    }
    return s;
  }
  ~OnDevice() {
    if (back_ < 0) return;
    try {
      c10::cuda::set_device(static_cast<c10::DeviceIndex>(back_));
    } catch (...) {  // the call's own status or error stands
    }
  }

 private:
  int dev_, back_ = -1;
};

// Other Python threads may run while the C call launches (or waits for room in a
// launch queue).
class WithoutGil {
 public:
  WithoutGil() : state_(PyEval_SaveThread()) {}
  ~WithoutGil() { PyEval_RestoreThread(state_); }

 private:
  PyThreadState* state_;
};

struct Cache {
  const at::Tensor &k, &v;
  int pages, heads, page_size;
};
Cache cache(PyObject* k, PyObject* v, const at::Tensor& tokens) {
  const at::Tensor& kc = operand(k, "k_cache", 4, &tokens);
  if (kc.size(3) != tokens.size(2))
    bad_value("k_cache and v_cache must be [num_pages, Hkv, page_size, d] of the tokens' d, got " + shape_of(kc));
  return {kc, same(v, "v_cache", kc), as_int(kc.size(0), "num_pages"), as_int(kc.size(1), "Hkv"),
          as_int(kc.size(2), "page_size")};
}

struct Tables {
  int B, pages;
  int64_t row;
  const int *table, *seqlens, *cu;
};
Tables tables(OnDevice& on, PyObject* page_table, PyObject* seqlens, PyObject* cu_seqlens, int64_t total) {
  const at::Tensor& t = tensor(page_table, "page_table");
  if (t.dim() != 2) bad_value("page_table must be [B, max_pages], got " + shape_of(t));
  const int64_t B = t.size(0);
  int32(page_table, "page_table", {B, t.size(1)});
  const at::Tensor& s = int32(seqlens, "seqlens", {B});
  on.also(t);
  on.also(s);
  const int* cu = nullptr;
  if (cu_seqlens != Py_None) {
    const at::Tensor& c = int32(cu_seqlens, "cu_seqlens", {B + 1});
    on.also(c);
    cu = static_cast<const int*>(c.data_ptr());
  } else if (B == 0 || total % B) {
    bad_value("without cu_seqlens the " + std::to_string(total) + " new tokens must divide evenly over " +
              std::to_string(B) + " sequences");
  }
  return {as_int(B, "B"), as_int(t.size(1), "max_pages"), B > 1 ? t.stride(0) : t.size(1),
          static_cast<const int*>(t.data_ptr()), static_cast<const int*>(s.data_ptr()), cu};
}

// q and k (which may be missing) with their outputs; p: positions, inv_freq, interleaved, inverse, factor, stream.
// [B, H, N, d] tensors with positions [N] or [B, N], or packed [total, H, d] ones with positions [total].
int rotary_call(const at::Tensor& q, const at::Tensor& qo, const at::Tensor* kt, const at::Tensor* kot, PyObject* const* p) {
  const bool packed = q.dim() == 3;
  const int dims = packed ? 3 : 4, h = 1, n = packed ? 0 : 2;
  auto strides = [&](const at::Tensor& t) { return packed ? strides3(t) : strides4(t); };
  OnDevice on(q);
  on.also(qo);
  const int64_t B = packed ? 1 : q.size(0), N = q.size(n), d = q.size(dims - 1);
  const void* k = nullptr;
  void* ko = nullptr;
  exattn_strides sk{}, sko{};
  int Hk = 0;
  if (kt) {
    if ((!packed && kt->size(0) != B) || kt->size(n) != N || kt->size(dims - 1) != d)
      bad_value("k must be laid out like q but for its heads, got " + shape_of(*kt));
    on.also(*kt);
    on.also(*kot);
    k = kt->data_ptr();
    ko = kot->data_ptr();
    sk = strides(*kt);
    sko = strides(*kot);
    Hk = as_int(kt->size(h), "Hk");
  }
  const bool shared = packed || tensor(p[0], "positions").dim() == 1;
  const at::Tensor& pos = shared ? int32(p[0], "positions", {N}) : int32(p[0], "positions", {B, N});
  const at::Tensor& f = tensor(p[1], "inv_freq");
  const int rot = rotary_dim(f);
  on.also(pos);
  on.also(f);
  const int il = truth(p[2]), inverse = truth(p[3]);
  const float factor = as_float(p[4]);
  if (q.numel() == 0 && (Hk == 0 || B * N == 0)) return EXATTN_OK;
  void* stream = on.enter(p[5]);
  const WithoutGil threads;
  return attn_rotary(dtype_of(q), q.data_ptr(), strides(q), qo.data_ptr(), strides(qo), as_int(q.size(h), "Hq"), k, sk, ko,
                     sko, Hk, static_cast<const int*>(pos.data_ptr()), shared || B <= 1 ? 0 : pos.stride(0),
                     static_cast<const double*>(f.data_ptr()), rot, il, inverse, factor, as_int(B, "B"), as_int(N, "N"),
                     as_int(d, "d"), stream);
}

const at::Tensor& rotary_operand(PyObject* o, const char* name, const at::Tensor* q) {
  const int dims = q ? static_cast<int>(q->dim()) : tensor(o, name).dim() == 3 ? 3 : 4;
  return operand(o, name, dims, q);
}

// (q, q_out, k, k_out, positions, inv_freq, interleaved, inverse, factor, stream)
PyObject* rotary(PyObject* const* p) {
  const at::Tensor& q = rotary_operand(p[0], "q", nullptr);
  const at::Tensor& qo = same(p[1], "q_out", q);
  if ((p[2] == Py_None) != (p[3] == Py_None)) bad_value("k and k_out go together");
  if (p[2] == Py_None) return PyLong_FromLong(rotary_call(q, qo, nullptr, nullptr, p + 4));
  const at::Tensor& k = rotary_operand(p[2], "k", &q);
  return PyLong_FromLong(rotary_call(q, qo, &k, &same(p[3], "k_out", k), p + 4));
}

// (q, k or None, positions, inv_freq, interleaved, inverse, factor, stream) -> (status, q_out, k_out or None): the
// outputs made here, which takes a third of the time that two calls from Python do.
PyObject* rotary_new(PyObject* const* p) {
  const at::Tensor& q = rotary_operand(p[0], "q", nullptr);
  const at::Tensor* k = p[1] == Py_None ? nullptr : &rotary_operand(p[1], "k", &q);
  const at::Tensor qo = at::empty_like(q);
  at::Tensor ko;
  if (k) ko = at::empty_like(*k);
  const int status = rotary_call(q, qo, k, k ? &ko : nullptr, p + 2);
  PyObject* const out = PyTuple_New(3);
  if (!out) throw Refused{nullptr, ""};
  PyTuple_SET_ITEM(out, 0, PyLong_FromLong(status));
  PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(qo));
  PyTuple_SET_ITEM(out, 2, k ? THPVariable_Wrap(ko) : Py_NewRef(Py_None));
  return out;
}

// (k, v, k_cache, v_cache, page_table, seqlens, cu_seqlens, q, q_out, inv_freq, interleaved, factor, stream)
int cache_append(PyObject* const* p) {
  const at::Tensor& k = operand(p[0], "k", 3);
  const at::Tensor& v = same(p[1], "v", k);
  OnDevice on(k);
  on.also(v);
  const Cache c = cache(p[2], p[3], k);
  on.also(c.k);
  on.also(c.v);
  if (c.heads != k.size(1)) bad_value("k and v must have the cache's " + std::to_string(c.heads) + " heads");
  const int64_t total = k.size(0);
  const Tables t = tables(on, p[4], p[5], p[6], total);
  if ((p[7] == Py_None) != (p[8] == Py_None) || (p[7] != Py_None && p[9] == Py_None))
    bad_value("q, q_out and inv_freq go together");
  const void* q = nullptr;
  void* qo = nullptr;
  exattn_strides sq{}, sqo{};
  int Hq = 0, rot = 0;
  const double* f = nullptr;
  if (p[7] != Py_None) {
    const at::Tensor& qt = operand(p[7], "q", 3, &k);
    if (qt.size(0) != total || qt.size(2) != k.size(2)) bad_value("q must be [total, Hq, d] like k, got " + shape_of(qt));
    const at::Tensor& qot = same(p[8], "q_out", qt);
    on.also(qt);
    on.also(qot);
    q = qt.data_ptr();
    qo = qot.data_ptr();
    sq = strides3(qt);
    sqo = strides3(qot);
    Hq = as_int(qt.size(1), "Hq");
  }
  if (p[9] != Py_None) {
    const at::Tensor& ft = tensor(p[9], "inv_freq");
    rot = rotary_dim(ft);
    on.also(ft);
    f = static_cast<const double*>(ft.data_ptr());
  }
  const int il = truth(p[10]);
  const float factor = as_float(p[11]);
  if (total == 0) return EXATTN_OK;
  void* stream = on.enter(p[12]);
  const WithoutGil threads;
  return attn_cache_append(dtype_of(k), q, sq, qo, sqo, Hq, k.data_ptr(), strides3(k), v.data_ptr(), strides3(v),
                           c.k.data_ptr(), strides4(c.k), c.v.data_ptr(), strides4(c.v), c.heads, c.pages, c.page_size,
                           t.table, t.row, t.pages, t.seqlens, t.cu, t.B, as_int(total, "total"), as_int(k.size(2), "d"), f,
                           rot, il, factor, stream);
}

// (q, k_cache, v_cache, o, lse, page_table, seqlens, cu_seqlens, max_seqlen_q, max_seqlen_k, causal, scale, workspace,
//  stream, window)
int fwd_paged(PyObject* const* p) {
  const at::Tensor& q = operand(p[0], "q", 3);
  OnDevice on(q);
  const Cache c = cache(p[1], p[2], q);
  const at::Tensor& o = same(p[3], "o", q);
  const at::Tensor& lse = tensor(p[4], "lse");
  const int64_t total = q.size(0), Hq = q.size(1);
  if (lse.scalar_type() != at::kFloat || lse.sizes() != at::IntArrayRef({Hq, total}) || !lse.is_contiguous())
    bad_value("lse must be contiguous float32 [Hq, total]");
  on.also(c.k);
  on.also(c.v);
  on.also(o);
  on.also(lse);
  const Tables t = tables(on, p[5], p[6], p[7], total);
  void* ws = nullptr;
  size_t ws_bytes = 0;
  if (p[12] != Py_None) {
    const at::Tensor& w = tensor(p[12], "workspace");
    on.also(w);
    if (!w.is_contiguous()) bad_value("workspace must be contiguous");
    ws = w.data_ptr();
    ws_bytes = w.nbytes();
  }
  const int mq = as_int(p[8], "max_seqlen_q"), mk = as_int(p[9], "max_seqlen_k"), causal = truth(p[10]);
  const float scale = as_float(p[11]);
  const int window = as_int(p[14], "window");
  if (total == 0) return EXATTN_OK;
  void* stream = on.enter(p[13]);
  const WithoutGil threads;
  return attn_fwd_paged(dtype_of(q), q.data_ptr(), strides3(q), c.k.data_ptr(), strides4(c.k), c.v.data_ptr(),
                        strides4(c.v), o.data_ptr(), strides3(o), static_cast<float*>(lse.data_ptr()), c.pages,
                        c.page_size, t.table, t.row, t.pages, t.seqlens, t.cu, t.B, as_int(Hq, "Hq"), c.heads,
                        as_int(total, "total"), mq, mk, as_int(q.size(2), "d"), causal, window, scale, ws, ws_bytes, stream);
}

// Host page numbers: an int32 tensor, or any sequence of ints (into `own`).
const int* pages(PyObject* o, const char* name, std::vector<int>* own, size_t* n) {
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cpu()) bad_value(std::string(name) + ": page numbers are host data (page tables are kept on the host)");
    if (t.dim() != 1 || t.scalar_type() != at::kInt || !t.is_contiguous())
      bad_value(std::string(name) + " must be contiguous 1-D int32 page numbers");
    *n = static_cast<size_t>(t.numel());
    return static_cast<const int*>(t.data_ptr());
  }
  PyObject* s = PySequence_Fast(o, "page numbers must be an int32 tensor or a sequence");
  if (!s) throw Refused{nullptr, ""};
  *n = static_cast<size_t>(PySequence_Fast_GET_SIZE(s));
  try {
    own->resize(*n);
    for (size_t i = 0; i < *n; ++i) (*own)[i] = as_int(PySequence_Fast_GET_ITEM(s, static_cast<Py_ssize_t>(i)), name);
  } catch (...) {
    Py_DECREF(s);
    throw;
  }
  Py_DECREF(s);
  return own->data();
}

// (pool, src, dst, stream)
int cache_copy(PyObject* const* p) {
  const at::Tensor& pool = tensor(p[0], "pool");
  OnDevice on(pool);
  if (pool.dim() < 3) bad_value("pool must be [slabs, num_pages, ...], got " + shape_of(pool));
  // A page is dense if its axes, by their strides, follow one another.
  std::vector<std::pair<int64_t, int64_t>> axes;
  for (int64_t i = 2; i < pool.dim(); ++i)
    if (pool.size(i) != 1) axes.emplace_back(pool.stride(i), pool.size(i));
  std::sort(axes.begin(), axes.end());
  int64_t each = 1;
  for (const auto& [stride, extent] : axes) {
    if (stride != each) bad_value("each page of the pool must be one dense block");
    each *= extent;
  }
  std::vector<int> own_src, own_dst;
  size_t n = 0, m = 0;
  const int* src = pages(p[1], "src", &own_src, &n);
  const int* dst = pages(p[2], "dst", &own_dst, &m);
  if (n != m) bad_value("src and dst must be of one length");
  if (n == 0) return EXATTN_OK;
  const int64_t size = pool.element_size();
  void* stream = on.enter(p[3]);
  const WithoutGil threads;
  return attn_cache_copy(pool.data_ptr(), pool.stride(0) * size, pool.stride(1) * size, each * size,
                         as_int(pool.size(0), "slabs"), as_int(pool.size(1), "num_pages"), src, dst,
                         as_int(static_cast<int64_t>(n), "n"), stream);
}

// The status of a C call as a Python int.
template <int (*F)(PyObject* const*)>
PyObject* status(PyObject* const* p) {
  return PyLong_FromLong(F(p));
}

// Refusals and errors as exceptions.
template <PyObject* (*F)(PyObject* const*), int ARGS>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != ARGS) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", ARGS, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    if (r.type) PyErr_SetString(r.type, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyMethodDef kMethods[] = {
    {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<rotary, 10>)), METH_FASTCALL, nullptr},
    {"rotary_new", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<rotary_new, 8>)), METH_FASTCALL, nullptr},
    {"cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<status<cache_append>, 13>)),
     METH_FASTCALL, nullptr},
    {"fwd_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<status<fwd_paged>, 15>)), METH_FASTCALL,
     nullptr},
    {"cache_copy", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<status<cache_copy>, 4>)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_exattn_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__exattn_binding() { return PyModule_Create(&kModule); }
