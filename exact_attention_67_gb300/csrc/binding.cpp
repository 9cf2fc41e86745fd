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
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <ATen/ops/zeros.h>
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

// What the calls that turn q and k (which may be missing) share.  [B, H, N, d] tensors with positions [N] or [B, N],
// or packed [total, H, d] ones with positions [total].
struct Turned {
  bool packed, empty;
  int64_t B, N, d, pos_stride;
  int Hq, Hk, rot;
  const int* pos;
  const double* freq;
  exattn_strides strides(const at::Tensor& t) const { return packed ? strides3(t) : strides4(t); }
};
Turned turned(OnDevice& on, const at::Tensor& q, const at::Tensor* k, PyObject* positions, PyObject* inv_freq) {
  Turned t{};
  t.packed = q.dim() == 3;
  const int dims = t.packed ? 3 : 4, h = 1, n = t.packed ? 0 : 2;
  t.B = t.packed ? 1 : q.size(0);
  t.N = q.size(n);
  t.d = q.size(dims - 1);
  t.Hq = as_int(q.size(h), "Hq");
  if (k) {
    if ((!t.packed && k->size(0) != t.B) || k->size(n) != t.N || k->size(dims - 1) != t.d)
      bad_value("k must be laid out like q but for its heads, got " + shape_of(*k));
    on.also(*k);
    t.Hk = as_int(k->size(h), "Hk");
  }
  const bool shared = t.packed || tensor(positions, "positions").dim() == 1;
  const at::Tensor& pos = shared ? int32(positions, "positions", {t.N}) : int32(positions, "positions", {t.B, t.N});
  const at::Tensor& f = tensor(inv_freq, "inv_freq");
  t.rot = rotary_dim(f);
  on.also(pos);
  on.also(f);
  t.pos = static_cast<const int*>(pos.data_ptr());
  t.pos_stride = shared || t.B <= 1 ? 0 : pos.stride(0);
  t.freq = static_cast<const double*>(f.data_ptr());
  t.empty = q.numel() == 0 && (t.Hk == 0 || t.B * t.N == 0);
  return t;
}

// A tensor's place and strides; nothing where it is missing.
struct Place {
  void* at = nullptr;
  exattn_strides s{};
  Place(const Turned& t, const at::Tensor* x) {
    if (!x) return;
    at = x->data_ptr();
    s = t.strides(*x);
  }
};

// q and k (which may be missing) with their outputs; p: positions, inv_freq, interleaved, inverse, factor, stream.
int rotary_call(const at::Tensor& q, const at::Tensor& qo, const at::Tensor* kt, const at::Tensor* kot, PyObject* const* p) {
  OnDevice on(q);
  on.also(qo);
  if (kot) on.also(*kot);
  const Turned t = turned(on, q, kt, p[0], p[1]);
  const int il = truth(p[2]), inverse = truth(p[3]);
  const float factor = as_float(p[4]);
  if (t.empty) return EXATTN_OK;
  const Place k(t, kt), ko(t, kot);
  void* stream = on.enter(p[5]);
  const WithoutGil threads;
  return attn_rotary(dtype_of(q), q.data_ptr(), t.strides(q), qo.data_ptr(), t.strides(qo), t.Hq, k.at, k.s, ko.at, ko.s, t.Hk,
                     t.pos, t.pos_stride, t.freq, t.rot, il, inverse, factor, as_int(t.B, "B"), as_int(t.N, "N"),
                     as_int(t.d, "d"), stream);
}

// Gains [d] of the norms, or nothing (all 1); of one type if both are given.
struct Gains {
  const void *q = nullptr, *k = nullptr;
  at::ScalarType type = at::kFloat;
  int dtype() const {
    return type == at::kFloat ? EXATTN_DTYPE_F32 : type == at::kHalf ? EXATTN_DTYPE_F16 : EXATTN_DTYPE_BF16;
  }
};
Gains gains(const OnDevice& on, PyObject* q, PyObject* k, int64_t d, const char* q_name = "q_gain",
            const char* k_name = "k_gain") {
  Gains g;
  bool first = true;
  auto one = [&](PyObject* o, const char* name) -> const void* {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kHalf && t.scalar_type() != at::kBFloat16)
      bad_type(std::string(name) + " must be float32, bfloat16 or float16");
    if (t.dim() != 1 || t.size(0) != d || !t.is_contiguous())
      bad_value(std::string(name) + " must be a contiguous tensor [d], got " + shape_of(t));
    on.also(t);
    if (!first && t.scalar_type() != g.type) bad_value("the gains must be of one type");
    first = false;
    g.type = t.scalar_type();
    return t.data_ptr();
  };
  g.q = one(q, q_name);
  g.k = one(k, k_name);
  return g;
}

// p: positions, inv_freq, q_gain, k_gain, interleaved, factor, eps, stream.
int norm_call(const at::Tensor& q, const at::Tensor& qo, const at::Tensor* kt, const at::Tensor* kot, PyObject* const* p) {
  OnDevice on(q);
  on.also(qo);
  if (kot) on.also(*kot);
  const Turned t = turned(on, q, kt, p[0], p[1]);
  const Gains g = gains(on, p[2], p[3], t.d);
  const int il = truth(p[4]);
  const float factor = as_float(p[5]), eps = as_float(p[6]);
  if (t.empty) return EXATTN_OK;
  const Place k(t, kt), ko(t, kot);
  void* stream = on.enter(p[7]);
  const WithoutGil threads;
  return attn_norm_rotary(dtype_of(q), q.data_ptr(), t.strides(q), qo.data_ptr(), t.strides(qo), t.Hq, k.at, k.s, ko.at, ko.s,
                          t.Hk, t.pos, t.pos_stride, t.freq, t.rot, il, factor, g.q, g.k, g.dtype(), eps, as_int(t.B, "B"),
                          as_int(t.N, "N"), as_int(t.d, "d"), stream);
}

const at::Tensor& rotary_operand(PyObject* o, const char* name, const at::Tensor* q) {
  const int dims = q ? static_cast<int>(q->dim()) : tensor(o, name).dim() == 3 ? 3 : 4;
  return operand(o, name, dims, q);
}

using TurnCall = int (*)(const at::Tensor&, const at::Tensor&, const at::Tensor*, const at::Tensor*, PyObject* const*);

// (q, q_out, k, k_out, ...F's)
template <TurnCall F>
PyObject* turn_into(PyObject* const* p) {
  const at::Tensor& q = rotary_operand(p[0], "q", nullptr);
  const at::Tensor& qo = same(p[1], "q_out", q);
  if ((p[2] == Py_None) != (p[3] == Py_None)) bad_value("k and k_out go together");
  if (p[2] == Py_None) return PyLong_FromLong(F(q, qo, nullptr, nullptr, p + 4));
  const at::Tensor& k = rotary_operand(p[2], "k", &q);
  return PyLong_FromLong(F(q, qo, &k, &same(p[3], "k_out", k), p + 4));
}

PyObject* tensor_or_none(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

// (status, tensors...), tensors that are not defined as None
PyObject* answer(int status, std::initializer_list<at::Tensor> ts) {
  PyObject* const out = PyTuple_New(static_cast<Py_ssize_t>(1 + ts.size()));
  if (!out) throw Refused{nullptr, ""};
  PyTuple_SET_ITEM(out, 0, PyLong_FromLong(status));
  Py_ssize_t i = 1;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(out, i++, tensor_or_none(t));
  return out;
}

// (q, k or None, ...F's) -> (status, q_out, k_out or None): the outputs made here, which takes a third of the time
// that two calls from Python do.
template <TurnCall F>
PyObject* turn_new(PyObject* const* p) {
  const at::Tensor& q = rotary_operand(p[0], "q", nullptr);
  const at::Tensor* k = p[1] == Py_None ? nullptr : &rotary_operand(p[1], "k", &q);
  at::Tensor qo, ko;
  {
    const at::AutoDispatchBelowAutograd plain;  // new tensors: nothing for autograd to record
    qo = at::empty_like(q);
    if (k) ko = at::empty_like(*k);
  }
  const int status = F(q, qo, k, k ? &ko : nullptr, p + 2);
  return answer(status, {qo, ko});
}

// The operands of the norms' gradient; dk, k, dk_out may be missing.
struct NormGrad {
  const at::Tensor &dq, &q, &dqo;
  const at::Tensor *dk, *k, *dko;
  void *dq_gain, *dk_gain, *ws;
  size_t ws_bytes;
};

// p: interleaved, factor, eps, then `stream`.
int norm_grad_call(OnDevice& on, const Turned& t, const Gains& g, const NormGrad& c, PyObject* const* p, PyObject* stream_of) {
  const int il = truth(p[0]);
  const float factor = as_float(p[1]), eps = as_float(p[2]);
  if (t.empty) return EXATTN_OK;
  const Place dk(t, c.dk), k(t, c.k), dko(t, c.dko);
  void* stream = on.enter(stream_of);
  const WithoutGil threads;
  return attn_norm_rotary_backward(dtype_of(c.q), c.dq.data_ptr(), t.strides(c.dq), c.q.data_ptr(), t.strides(c.q),
                                   c.dqo.data_ptr(), t.strides(c.dqo), t.Hq, dk.at, dk.s, k.at, k.s, dko.at, dko.s, t.Hk, t.pos,
                                   t.pos_stride, t.freq, t.rot, il, factor, g.q, g.k, g.dtype(), eps, c.dq_gain, c.dk_gain,
                                   as_int(t.B, "B"), as_int(t.N, "N"), as_int(t.d, "d"), c.ws, c.ws_bytes, stream);
}

struct Workspace {
  void* at = nullptr;
  size_t bytes = 0;
  Workspace(const OnDevice& on, PyObject* o) {
    if (o == Py_None) return;
    const at::Tensor& w = tensor(o, "workspace");
    on.also(w);
    if (!w.is_contiguous()) bad_value("workspace must be contiguous");
    at = w.data_ptr();
    bytes = w.nbytes();
  }
};

// (dq, q, dq_out, dk, k, dk_out, positions, inv_freq, q_gain, k_gain, dq_gain, dk_gain, interleaved, factor, eps,
//  workspace, stream)
int norm_grad(PyObject* const* p) {
  const at::Tensor& q = rotary_operand(p[1], "q", nullptr);
  OnDevice on(q);
  const at::Tensor &dq = same(p[0], "dq", q), &dqo = same(p[2], "dq_out", q);
  on.also(dq);
  on.also(dqo);
  if ((p[3] == Py_None) != (p[4] == Py_None) || (p[3] == Py_None) != (p[5] == Py_None))
    bad_value("dk, k and dk_out go together");
  const at::Tensor *dk = nullptr, *k = nullptr, *dko = nullptr;
  if (p[4] != Py_None) {
    k = &rotary_operand(p[4], "k", &q);
    dk = &same(p[3], "dk", *k);
    dko = &same(p[5], "dk_out", *k);
    on.also(*dk);
    on.also(*dko);
  }
  const Turned t = turned(on, q, k, p[6], p[7]);
  Gains g = gains(on, p[8], p[9], t.d);
  const Gains dg = gains(on, p[10], p[11], t.d, "dq_gain", "dk_gain");
  if (!g.q && !g.k) g.type = dg.type;
  if ((dg.q || dg.k) && dg.type != g.type) bad_value("the gains' gradients must be of the gains' type");
  const Workspace ws(on, p[15]);
  return norm_grad_call(on, t, g, {dq, q, dqo, dk, k, dko, const_cast<void*>(dg.q), const_cast<void*>(dg.k), ws.at, ws.bytes},
                        p + 12, p[16]);
}

// (dq, dk or None, q, k or None, positions, inv_freq, q_gain, k_gain, want_q, want_k, interleaved, factor, eps, stream)
// -> (status, gradients of q, k, q_gain and k_gain; None where missing or not wanted)
PyObject* norm_grad_new(PyObject* const* p) {
  const at::Tensor& q = rotary_operand(p[2], "q", nullptr);
  OnDevice on(q);
  const at::Tensor& dq = same(p[0], "dq", q);
  on.also(dq);
  if ((p[1] == Py_None) != (p[3] == Py_None)) bad_value("dk and k go together");
  const at::Tensor *dk = nullptr, *k = nullptr;
  if (p[3] != Py_None) {
    k = &rotary_operand(p[3], "k", &q);
    dk = &same(p[1], "dk", *k);
    on.also(*dk);
  }
  const Turned t = turned(on, q, k, p[4], p[5]);
  const Gains g = gains(on, p[6], p[7], t.d);
  const at::AutoDispatchBelowAutograd plain;  // new tensors: nothing for autograd to record
  const at::Tensor dqo = at::empty_like(q);
  at::Tensor dko, dqg, dkg;
  if (k) dko = at::empty_like(*k);
  const auto options = q.options().dtype(g.type);
  auto fresh = [&]() { return t.empty ? at::zeros({t.d}, options) : at::empty({t.d}, options); };
  if (g.q && truth(p[8])) dqg = fresh();
  if (g.k && truth(p[9])) dkg = t.Hk ? fresh() : at::zeros({t.d}, options);
  const size_t bytes = t.empty ? 0
                               : attn_norm_rotary_backward_workspace_size(as_int(t.B, "B"), as_int(t.N, "N"), as_int(t.d, "d"));
  const at::Tensor ws = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
  const int status = norm_grad_call(on, t, g,
                                    {dq, q, dqo, dk, k, k ? &dko : nullptr, dqg.defined() ? dqg.data_ptr() : nullptr,
                                     dkg.defined() ? dkg.data_ptr() : nullptr, ws.data_ptr(), bytes},
                                    p + 10, p[13]);
  return answer(status, {dqo, dko, dqg, dkg});
}

// (k, v, k_cache, v_cache, page_table, seqlens, cu_seqlens, q, q_out, inv_freq, interleaved, factor, stream, q_gain,
//  k_gain, eps); with gains, normalised on the way
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
  const Gains g = gains(on, p[13], p[14], k.size(2));
  const bool normed = g.q || g.k;
  if ((p[7] == Py_None) != (p[8] == Py_None) || (p[7] != Py_None && p[9] == Py_None && !normed))
    bad_value("q, q_out and inv_freq go together");
  if (normed && (!g.k || (p[7] == Py_None) != !g.q)) bad_value("gains are given for k, and for q where it is");
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
  const float factor = as_float(p[11]), eps = as_float(p[15]);
  if (total == 0) return EXATTN_OK;
  void* stream = on.enter(p[12]);
  const WithoutGil threads;
  if (normed)
    return attn_cache_append_norm(dtype_of(k), q, sq, qo, sqo, Hq, k.data_ptr(), strides3(k), v.data_ptr(), strides3(v),
                                  c.k.data_ptr(), strides4(c.k), c.v.data_ptr(), strides4(c.v), c.heads, c.pages, c.page_size,
                                  t.table, t.row, t.pages, t.seqlens, t.cu, t.B, as_int(total, "total"),
                                  as_int(k.size(2), "d"), f, rot, il, factor, g.q, g.k, g.dtype(), eps, stream);
  return attn_cache_append(dtype_of(k), q, sq, qo, sqo, Hq, k.data_ptr(), strides3(k), v.data_ptr(), strides3(v),
                           c.k.data_ptr(), strides4(c.k), c.v.data_ptr(), strides4(c.v), c.heads, c.pages, c.page_size,
                           t.table, t.row, t.pages, t.seqlens, t.cu, t.B, as_int(total, "total"), as_int(k.size(2), "d"), f,
                           rot, il, factor, stream);
}

// The operands of an attention over pages.
struct Attend {
  const at::Tensor& q;
  OnDevice on;
  const Cache c;
  const at::Tensor &o, &lse;
  int64_t total, Hq;
  Tables t;
  // p: q, k_cache, v_cache, o, lse, page_table, seqlens, cu_seqlens
  explicit Attend(PyObject* const* p)
      : q(operand(p[0], "q", 3)), on(q), c(cache(p[1], p[2], q)), o(same(p[3], "o", q)), lse(tensor(p[4], "lse")),
        total(q.size(0)), Hq(q.size(1)), t{} {
    if (lse.scalar_type() != at::kFloat || lse.sizes() != at::IntArrayRef({Hq, total}) || !lse.is_contiguous())
      bad_value("lse must be contiguous float32 [Hq, total]");
    on.also(c.k);
    on.also(c.v);
    on.also(o);
    on.also(lse);
    t = tables(on, p[5], p[6], p[7], total);
  }
};

// (q, k_cache, v_cache, o, lse, page_table, seqlens, cu_seqlens, max_seqlen_q, max_seqlen_k, causal, scale, workspace,
//  stream, window)
int fwd_paged(PyObject* const* p) {
  Attend a(p);
  const Workspace ws(a.on, p[12]);
  const int mq = as_int(p[8], "max_seqlen_q"), mk = as_int(p[9], "max_seqlen_k"), causal = truth(p[10]);
  const float scale = as_float(p[11]);
  const int window = as_int(p[14], "window");
  if (a.total == 0) return EXATTN_OK;
  void* stream = a.on.enter(p[13]);
  const Tables& t = a.t;
  const WithoutGil threads;
  return attn_fwd_paged(dtype_of(a.q), a.q.data_ptr(), strides3(a.q), a.c.k.data_ptr(), strides4(a.c.k), a.c.v.data_ptr(),
                        strides4(a.c.v), a.o.data_ptr(), strides3(a.o), static_cast<float*>(a.lse.data_ptr()), a.c.pages,
                        a.c.page_size, t.table, t.row, t.pages, t.seqlens, t.cu, t.B, as_int(a.Hq, "Hq"), a.c.heads,
                        as_int(a.total, "total"), mq, mk, as_int(a.q.size(2), "d"), causal, window, scale, ws.at, ws.bytes,
                        stream);
}

// (q, k_cache, v_cache, o, lse, page_table, seqlens, cu_seqlens, cu_groups, prefix_lens, max_seqlen_q, max_seqlen_k,
//  max_group_q, causal, scale, workspace, stream)
int fwd_paged_shared(PyObject* const* p) {
  Attend a(p);
  const Tables& t = a.t;
  const int64_t groups = tensor(p[8], "cu_groups").numel() - 1;
  const at::Tensor &cg = int32(p[8], "cu_groups", {groups + 1}), &pl = int32(p[9], "prefix_lens", {t.B});
  a.on.also(cg);
  a.on.also(pl);
  const Workspace ws(a.on, p[15]);
  const int mq = as_int(p[10], "max_seqlen_q"), mk = as_int(p[11], "max_seqlen_k"), mg = as_int(p[12], "max_group_q");
  const int causal = truth(p[13]);
  const float scale = as_float(p[14]);
  if (a.total == 0) return EXATTN_OK;
  void* stream = a.on.enter(p[16]);
  const WithoutGil threads;
  return attn_fwd_paged_shared(
      dtype_of(a.q), a.q.data_ptr(), strides3(a.q), a.c.k.data_ptr(), strides4(a.c.k), a.c.v.data_ptr(), strides4(a.c.v),
      a.o.data_ptr(), strides3(a.o), static_cast<float*>(a.lse.data_ptr()), a.c.pages, a.c.page_size, t.table, t.row, t.pages,
      t.seqlens, t.cu, static_cast<const int*>(cg.data_ptr()), static_cast<const int*>(pl.data_ptr()), t.B,
      static_cast<int>(std::max<int64_t>(groups, 0)), as_int(a.Hq, "Hq"), a.c.heads, as_int(a.total, "total"), mq, mk, mg,
      as_int(a.q.size(2), "d"), causal, scale, ws.at, ws.bytes, stream);
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

template <PyObject* (*F)(PyObject* const*), int ARGS>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<F, ARGS>)), METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {
    method<turn_into<rotary_call>, 10>("rotary"),
    method<turn_new<rotary_call>, 8>("rotary_new"),
    method<turn_into<norm_call>, 12>("norm_rotary"),
    method<turn_new<norm_call>, 10>("norm_rotary_new"),
    method<status<norm_grad>, 17>("norm_rotary_grad"),
    method<norm_grad_new, 14>("norm_rotary_grad_new"),
    method<status<cache_append>, 16>("cache_append"),
    method<status<fwd_paged>, 15>("fwd_paged"),
    method<status<fwd_paged_shared>, 17>("fwd_paged_shared"),
    method<status<cache_copy>, 4>("cache_copy"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_exattn_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__exattn_binding() { return PyModule_Create(&kModule); }
