// kvq_bind.cpp -- the part of the Python binding that a serving step runs many
// times: checks of arguments, allocation of outputs and marshalling for the
// rotary positions and the block-scaled 8-bit cache.  A step's calls are a few
// microseconds on the GPU each, and the same work done in Python with ctypes
// took 9 to 14 us a call.  kvq.py holds the documented functions; it hands over
// the addresses of the loaded library's entry points (connect), so this module
// serves whichever build of the library is in use.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "kvq.h"

namespace {

using at::Tensor;

decltype(&kvq_rope) f_rope;
decltype(&kvq_b8_append) f_append;
decltype(&kvq_b8_gather) f_gather;
decltype(&kvq_b8_attn_workspace) f_workspace;
decltype(&kvq_b8_attn) f_attn;
decltype(&kvq_b8_attn_mass) f_mass;
decltype(&kvq_b8_evict) f_evict;
PyObject *g_check;  // kvq._check(name, status): raises on a status other than 0

[[noreturn]] void raise(PyObject *type, const std::string &what) {
  PyErr_SetString(type, what.c_str());
  throw python_error();
}
[[noreturn]] void bad_value(const std::string &what) { raise(PyExc_ValueError, what); }
[[noreturn]] void bad_type(const std::string &what) { raise(PyExc_TypeError, what); }

// ---------------------------------------------------------------- arguments
const Tensor *optional_tensor(PyObject *o, const char *name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const Tensor &tensor(PyObject *o, const char *name) {
  const Tensor *t = optional_tensor(o, name);
  if (t == nullptr) bad_type(std::string(name) + " must be a tensor");
  return *t;
}
int32_t integer(PyObject *o, const char *name) {
  PyObject *n = PyNumber_Index(o);
  if (n == nullptr) throw python_error();
  const long long v = PyLong_AsLongLong(n);
  Py_DECREF(n);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < INT32_MIN || v > INT32_MAX) bad_value(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}
double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
void count(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) bad_type("expected " + std::to_string(want) + " arguments, got " + std::to_string(got));
}

kvq_dtype dtype_of(const Tensor &t) {
  if (t.scalar_type() == at::kFloat) return KVQ_F32;
  if (t.scalar_type() == at::kBFloat16) return KVQ_BF16;
  bad_type(std::string("expected float32 or bfloat16, got ") + c10::toString(t.scalar_type()));
}
void int32s(const char *name, const Tensor &t, int64_t numel) {
  if (t.scalar_type() != at::kInt || t.numel() != numel || !t.is_contiguous())
    bad_value(std::string(name) + " must be a contiguous int32 tensor of " + std::to_string(numel) +
              " values");
}
// The library launches on the current device: tensors have to be there.
void here(int dev, const char *name, const Tensor *t) {
  if (t != nullptr && (!t->is_cuda() || t->get_device() != dev))
    bad_value(std::string(name) + " must be on the current CUDA device (cuda:" +
              std::to_string(dev) + "), got " + t->device().str());
}

// [..., heads, dim] seen as tokens x heads: the leading dims must step through
// memory as one
kvq_heads heads_of(const char *name, const Tensor &t) {
  const int64_t nd = t.dim();
  if (nd < 3 || (t.stride(nd - 1) != 1 && t.size(nd - 1) != 1))
    bad_value(std::string(name) + " must be [..., heads, dim] with dim contiguous");
  int64_t step = 0, span = 1;
  for (int64_t d = nd - 3; d >= 0; d--) {
    if (t.size(d) == 1) continue;
    if (span == 1)
      step = t.stride(d);
    else if (t.stride(d) != step * span)
      bad_value(std::string(name) + ": its tokens do not lie at one stride");
    span *= t.size(d);
  }
  // the stride of a dim of size 1 says nothing
  return {t.data_ptr(), step, t.size(nd - 2) != 1 ? t.stride(nd - 2) : 0, (int32_t)t.size(nd - 2)};
}

// A call's stream (0 with none given: torch's current one), made current for
// the allocations, so that memory of theirs is not handed out again while the
// call's stream still uses it.
struct OnStream {
  cudaStream_t stream;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  OnStream(PyObject *o, int dev) {
    if (o == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(dev).stream();
      return;
    }
    PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
    if (h == nullptr) throw python_error();
    stream = reinterpret_cast<cudaStream_t>(PyLong_AsUnsignedLongLong(h));
    Py_DECREF(h);
    if (PyErr_Occurred()) throw python_error();
    guard.emplace(c10::cuda::getStreamFromExternal(stream, dev));
  }
};

Tensor empty(at::IntArrayRef sizes, at::ScalarType dtype, int dev) {
  return at::detail::empty_cuda(sizes, dtype, at::Device(at::kCUDA, dev), std::nullopt);
}

// a library call with the interpreter released, as a full launch queue blocks
template <class F, class... A>
kvq_status call(F f, A... args) {
  PyThreadState *state = PyEval_SaveThread();
  const kvq_status st = f(args...);
  PyEval_RestoreThread(state);
  return st;
}

void check(const char *name, kvq_status st) {
  if (st == KVQ_OK) return;
  PyObject *r = PyObject_CallFunction(g_check, "si", name, (int)st);
  Py_XDECREF(r);
  throw python_error();
}

PyObject *wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject *none() { Py_RETURN_NONE; }

// what B8Cache hands over: (address of its descriptor, its K codes)
struct Cache {
  const kvq_b8_cache *c;
  const Tensor *codes;
};
Cache cache_of(PyObject *o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) bad_type("cache must be a B8Cache");
  void *p = PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 0));
  if (p == nullptr) throw python_error();
  return {static_cast<const kvq_b8_cache *>(p), &tensor(PyTuple_GET_ITEM(o, 1), "cache")};
}

kvq_rope_spec rope_of(PyObject *inv_freq, PyObject *interleaved, PyObject *factor, const Tensor **f) {
  const Tensor &t = tensor(inv_freq, "inv_freq");
  if (t.scalar_type() != at::kDouble || t.dim() != 1 || !t.is_contiguous())
    bad_value("inv_freq must be a contiguous float64 vector");
  const int inter = PyObject_IsTrue(interleaved);
  if (inter < 0) throw python_error();
  *f = &t;
  return {static_cast<const double *>(t.data_ptr()), (int32_t)(2 * t.numel()), inter, (float)real(factor)};
}

// ---------------------------------------------------------------- rope
// q, k, positions, inv_freq, interleaved, factor, inverse, q_out, k_out, stream
PyObject *bind_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const Tensor &q = tensor(a[0], "q"), &pos = tensor(a[2], "positions");
  const Tensor *k = optional_tensor(a[1], "k"), *f = nullptr;
  const Tensor *qo = optional_tensor(a[7], "q_out"), *ko = optional_tensor(a[8], "k_out");
  const kvq_rope_spec spec = rope_of(a[3], a[4], a[5], &f);
  const int inverse = PyObject_IsTrue(a[6]);
  if (inverse < 0) throw python_error();
  const kvq_heads hq = heads_of("q", q);
  const int64_t dim = q.size(-1), tokens = q.numel() / std::max<int64_t>(dim * hq.num_heads, 1);
  if (qo != nullptr && (qo->sizes() != q.sizes() || qo->scalar_type() != q.scalar_type()))
    bad_value("q_out must have q's shape and dtype");
  if (k == nullptr && ko != nullptr) bad_value("k_out without k");
  if (k != nullptr) {
    const int64_t nd = q.dim();
    if (k->dim() != nd || k->sizes().slice(0, nd - 2) != q.sizes().slice(0, nd - 2) ||
        k->size(nd - 1) != dim || k->scalar_type() != q.scalar_type() ||
        (ko != nullptr && (ko->sizes() != k->sizes() || ko->scalar_type() != k->scalar_type())))
      bad_value("k and k_out must match q's tokens, dim and dtype");
  }
  int32s("positions", pos, tokens);
  const kvq_dtype dt = dtype_of(q);
  const int dev = c10::cuda::current_device();
  here(dev, "q", &q), here(dev, "k", k), here(dev, "positions", &pos), here(dev, "inv_freq", f);
  here(dev, "q_out", qo), here(dev, "k_out", ko);
  if (tokens > INT32_MAX) bad_value("too many tokens");
  OnStream on(a[9], dev);
  Tensor qn, kn;
  if (qo == nullptr) qn = empty(q.sizes(), q.scalar_type(), dev), qo = &qn;
  if (k != nullptr && ko == nullptr) kn = empty(k->sizes(), k->scalar_type(), dev), ko = &kn;
  const kvq_heads hqo = heads_of("q_out", *qo);
  kvq_heads hk, hko;
  if (k != nullptr) hk = heads_of("k", *k), hko = heads_of("k_out", *ko);
  if (tokens > 0) {
    check("kvq_rope", call(f_rope, &spec, dt, (int32_t)dim, (int32_t)tokens, pos.const_data_ptr<int32_t>(),
                             inverse, &hq, &hqo, k ? &hk : nullptr, k ? &hko : nullptr, on.stream));
  }
  PyObject *r0 = qn.defined() ? wrap(std::move(qn)) : Py_NewRef(a[7]);
  PyObject *r1 = kn.defined() ? wrap(std::move(kn)) : Py_NewRef(a[8]);
  PyObject *r = PyTuple_New(2);
  PyTuple_SET_ITEM(r, 0, r0);
  PyTuple_SET_ITEM(r, 1, r1);
  return r;
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- append
// cache, k, v, start_pos, new_lens, inv_freq or None, interleaved, factor,
// positions, stream
PyObject *bind_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &start = tensor(a[3], "start_pos");
  const Tensor *lens = optional_tensor(a[4], "new_lens"), *at = optional_tensor(a[8], "positions");
  const Tensor *f = nullptr;
  if (k.dim() != 4 || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type())
    bad_value("k and v must have the same [batch, t_new, Hkv, dim] shape and dtype");
  const Cache c = cache_of(a[0]);
  const int64_t batch = k.size(0), t_new = k.size(1);
  if (k.size(2) != c.c->num_kv_heads || k.size(3) != c.c->head_dim)
    bad_value("k and v do not match the cache's heads");
  int32s("start_pos", start, batch);
  if (lens) int32s("new_lens", *lens, batch);
  kvq_rope_spec spec;
  const bool turned = a[5] != Py_None;
  if (turned) spec = rope_of(a[5], a[6], a[7], &f);
  if (at) {
    if (!turned) bad_value("positions without rope");
    int32s("positions", *at, batch * t_new);
  }
  const kvq_dtype dt = dtype_of(k);
  const int dev = c10::cuda::current_device();
  here(dev, "cache", c.codes), here(dev, "k", &k), here(dev, "v", &v), here(dev, "start_pos", &start);
  here(dev, "new_lens", lens), here(dev, "positions", at), here(dev, "inv_freq", f);
  if (batch == 0 || t_new == 0) return none();
  if (batch > INT32_MAX || t_new > INT32_MAX) bad_value("too many tokens");
  OnStream on(a[9], dev);
  const kvq_heads hk = heads_of("k", k), hv = heads_of("v", v);
  check("kvq_b8_append",
        call(f_append, c.c, &hk, &hv, dt, (int32_t)batch, (int32_t)t_new, start.const_data_ptr<int32_t>(),
                 lens ? lens->const_data_ptr<int32_t>() : nullptr, turned ? &spec : nullptr,
                 at ? at->const_data_ptr<int32_t>() : nullptr, on.stream));
  return none();
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- gather
// cache, first, ends, count, fp32 (else bf16), k_out, v_out, stream
PyObject *bind_gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const Cache c = cache_of(a[0]);
  const Tensor &first = tensor(a[1], "first"), &ends = tensor(a[2], "ends");
  const int32_t cnt = integer(a[3], "count");
  const at::ScalarType dtype = a[4] == Py_True ? at::kFloat : at::kBFloat16;
  const Tensor *ko = optional_tensor(a[5], "k_out"), *vo = optional_tensor(a[6], "v_out");
  const int64_t batch = first.numel();
  int32s("first", first, batch);
  int32s("ends", ends, batch);
  if (cnt < 0) check("kvq_b8_gather", KVQ_ERR_INVALID_ARG);
  const int64_t shape[4] = {batch, cnt, c.c->num_kv_heads, c.c->head_dim};
  const at::ScalarType got = ko ? ko->scalar_type() : vo ? vo->scalar_type() : dtype;
  for (const Tensor *t : {ko, vo})
    if (t != nullptr && (t->sizes() != at::IntArrayRef(shape) || t->scalar_type() != got || !t->is_contiguous()))
      bad_value("k_out and v_out must be contiguous [batch, count, Hkv, dim] tensors of one dtype");
  const int dev = c10::cuda::current_device();
  here(dev, "cache", c.codes), here(dev, "first", &first), here(dev, "ends", &ends);
  here(dev, "k_out", ko), here(dev, "v_out", vo);
  OnStream on(a[7], dev);
  Tensor kn, vn;
  if (ko == nullptr) kn = empty(shape, got, dev), ko = &kn;
  if (vo == nullptr) vn = empty(shape, got, dev), vo = &vn;
  check("kvq_b8_gather",
        call(f_gather, c.c, (int32_t)batch, first.const_data_ptr<int32_t>(), ends.const_data_ptr<int32_t>(),
                 cnt, dtype_of(*ko), ko->data_ptr(), vo->data_ptr(), on.stream));
  PyObject *r = PyTuple_New(2);
  PyTuple_SET_ITEM(r, 0, kn.defined() ? wrap(std::move(kn)) : Py_NewRef(a[5]));
  PyTuple_SET_ITEM(r, 1, vn.defined() ? wrap(std::move(vn)) : Py_NewRef(a[6]));
  return r;
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- attention
// the queries of a call; its tensors have to be looked over by `here`
kvq_b8_queries queries_of(const Cache &c, const Tensor &q, const Tensor &lens, const Tensor *cu,
                          PyObject *max_len, PyObject *scale, PyObject *max_q) {
  if (q.dim() != 3 || q.size(2) != c.c->head_dim || q.size(1) % c.c->num_kv_heads)
    bad_value("q must be [queries, Hq, dim] with the cache's dim and Hq a multiple of its kv heads");
  const int64_t batch = lens.numel();
  int32s("seq_lens", lens, batch);
  kvq_b8_queries d = {};
  d.max_q = 1;
  if (cu == nullptr) {
    if (q.size(0) != batch) bad_value("without cu_q there is one query per sequence");
  } else {
    if (max_q == Py_None) bad_value("cu_q needs max_q");
    int32s("cu_q", *cu, batch + 1);
    d.d_cu_q = cu->const_data_ptr<int32_t>();
    d.max_q = integer(max_q, "max_q");
  }
  if (q.size(0) > INT32_MAX || batch > INT32_MAX) bad_value("too many queries");
  d.q = heads_of("q", q);
  d.dtype = dtype_of(q);
  d.batch = (int32_t)batch;
  d.total_q = (int32_t)q.size(0);
  d.d_seq_lens = lens.const_data_ptr<int32_t>();
  d.max_seq_len = integer(max_len, "max_seq_len");
  d.scale = (float)real(scale);
  return d;
}
void lse_shape(const Tensor &lse, const Tensor &q) {
  if (lse.dim() != 2 || q.dim() != 3 || lse.size(0) != q.size(0) || lse.size(1) != q.size(1) ||
      lse.scalar_type() != at::kFloat || !lse.is_contiguous())
    bad_value("lse must be a contiguous fp32 [queries, Hq] tensor");
}

// cache, q, seq_lens, max_seq_len, scale, cu_q, max_q, return_lse, out, lse,
// workspace, stream
PyObject *bind_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 12);
  const Cache c = cache_of(a[0]);
  const Tensor &q = tensor(a[1], "q"), &lens = tensor(a[2], "seq_lens");
  const Tensor *cu = optional_tensor(a[5], "cu_q"), *out = optional_tensor(a[8], "out");
  const Tensor *lse = optional_tensor(a[9], "lse"), *ws = optional_tensor(a[10], "workspace");
  const kvq_b8_queries d = queries_of(c, q, lens, cu, a[3], a[4], a[6]);
  if (out != nullptr &&
      (out->sizes() != q.sizes() || out->scalar_type() != q.scalar_type() || !out->is_contiguous()))
    bad_value("out must be a contiguous tensor of q's shape and dtype");
  if (lse != nullptr) lse_shape(*lse, q);
  const int dev = c10::cuda::current_device();
  here(dev, "cache", c.codes), here(dev, "q", &q), here(dev, "seq_lens", &lens);
  here(dev, "cu_q", cu), here(dev, "out", out), here(dev, "lse", lse), here(dev, "workspace", ws);
  OnStream on(a[11], dev);
  Tensor on_, ln, wn;
  if (out == nullptr) on_ = empty(q.sizes(), q.scalar_type(), dev), out = &on_;
  const int want_lse = PyObject_IsTrue(a[7]);
  if (want_lse < 0) throw python_error();
  if (lse == nullptr && want_lse)
    ln = empty({q.size(0), q.size(1)}, at::kFloat, dev), lse = &ln;
  size_t bytes = 0;
  if (ws != nullptr) {
    bytes = ws->numel() * ws->element_size();
  } else {
    bytes = f_workspace(c.c, d.dtype, d.q.num_heads, d.batch, d.max_q, d.max_seq_len);
    if (bytes) wn = empty({(int64_t)bytes}, at::kByte, dev), ws = &wn;
  }
  check("kvq_b8_attn", call(f_attn, c.c, &d, out->data_ptr(), lse ? lse->data_ptr<float>() : nullptr,
                              ws ? ws->data_ptr() : nullptr, bytes, on.stream));
  PyObject *r0 = on_.defined() ? wrap(std::move(on_)) : Py_NewRef(a[8]);
  if (!want_lse) return r0;
  PyObject *r = PyTuple_New(2);
  PyTuple_SET_ITEM(r, 0, r0);
  PyTuple_SET_ITEM(r, 1, ln.defined() ? wrap(std::move(ln)) : Py_NewRef(a[9]));
  return r;
  END_HANDLE_TH_ERRORS
}

void mass_shape(const char *name, const Tensor &t, const Cache &c, int64_t batch, int64_t tokens) {
  if (t.dim() != 3 || t.size(0) != batch || t.size(1) != c.c->num_kv_heads || t.size(2) < tokens ||
      t.scalar_type() != at::kFloat || !t.is_contiguous())
    bad_value(std::string(name) + " must be a contiguous fp32 [" + std::to_string(batch) + ", " +
              std::to_string(c.c->num_kv_heads) + ", >= " + std::to_string(tokens) + "] tensor");
}

// cache, q, lse, seq_lens, max_seq_len, scale, mass, cu_q, max_q, stream
PyObject *bind_mass(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const Cache c = cache_of(a[0]);
  const Tensor &q = tensor(a[1], "q"), &lse = tensor(a[2], "lse"), &lens = tensor(a[3], "seq_lens");
  const Tensor &mass = tensor(a[6], "mass"), *cu = optional_tensor(a[7], "cu_q");
  const kvq_b8_queries d = queries_of(c, q, lens, cu, a[4], a[5], a[8]);
  lse_shape(lse, q);
  mass_shape("mass", mass, c, d.batch, d.max_seq_len);
  const int dev = c10::cuda::current_device();
  here(dev, "cache", c.codes), here(dev, "q", &q), here(dev, "lse", &lse);
  here(dev, "seq_lens", &lens), here(dev, "mass", &mass), here(dev, "cu_q", cu);
  OnStream on(a[9], dev);
  check("kvq_b8_attn_mass", call(f_mass, c.c, &d, lse.const_data_ptr<float>(), mass.data_ptr<float>(),
                                   mass.size(2), on.stream));
  return none();
  END_HANDLE_TH_ERRORS
}

// cache, into, mass, seq_lens, max_seq_len, keep, recent, sinks, mass_out, stream
PyObject *bind_evict(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const Cache c = cache_of(a[0]), to = cache_of(a[1]);
  const Tensor &mass = tensor(a[2], "mass"), &lens = tensor(a[3], "seq_lens");
  const Tensor *mo = optional_tensor(a[8], "mass_out");
  const int32_t max_len = integer(a[4], "max_seq_len"), keep = integer(a[5], "keep");
  const int32_t recent = integer(a[6], "recent"), sinks = integer(a[7], "sinks");
  const int64_t batch = lens.numel(), hkv = c.c->num_kv_heads;
  int32s("seq_lens", lens, batch);
  mass_shape("mass", mass, c, batch, max_len);
  if (keep < 1) check("kvq_b8_evict", KVQ_ERR_INVALID_ARG);
  if (mo != nullptr) mass_shape("mass_out", *mo, c, batch, keep);
  const int dev = c10::cuda::current_device();
  here(dev, "cache", c.codes), here(dev, "into", to.codes), here(dev, "mass", &mass);
  here(dev, "seq_lens", &lens), here(dev, "mass_out", mo);
  if (batch > INT32_MAX) bad_value("too many sequences");
  OnStream on(a[9], dev);
  Tensor ln = empty({batch}, at::kInt, dev), kept = empty({batch, hkv, keep}, at::kInt, dev), mn;
  if (mo == nullptr) mn = empty({batch, hkv, keep}, at::kFloat, dev), mo = &mn;
  check("kvq_b8_evict",
        call(f_evict, c.c, to.c, (int32_t)batch, lens.const_data_ptr<int32_t>(), max_len,
                mass.const_data_ptr<float>(), mass.size(2), keep, recent, sinks,
                ln.data_ptr<int32_t>(), kept.data_ptr<int32_t>(), mo->data_ptr<float>(),
                mo->size(2), on.stream));
  PyObject *r = PyTuple_New(3);
  PyTuple_SET_ITEM(r, 0, wrap(std::move(ln)));
  PyTuple_SET_ITEM(r, 1, wrap(std::move(kept)));
  PyTuple_SET_ITEM(r, 2, mn.defined() ? wrap(std::move(mn)) : Py_NewRef(a[8]));
  return r;
  END_HANDLE_TH_ERRORS
}

// check function, addresses of the seven entry points
PyObject *bind_connect(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  void *p[7];
  for (int i = 0; i < 7; i++) {
    p[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (p[i] == nullptr) bad_type("connect needs the addresses of the entry points");
  }
  f_rope = reinterpret_cast<decltype(f_rope)>(p[0]);
  f_append = reinterpret_cast<decltype(f_append)>(p[1]);
  f_gather = reinterpret_cast<decltype(f_gather)>(p[2]);
  f_workspace = reinterpret_cast<decltype(f_workspace)>(p[3]);
  f_attn = reinterpret_cast<decltype(f_attn)>(p[4]);
  f_mass = reinterpret_cast<decltype(f_mass)>(p[5]);
  f_evict = reinterpret_cast<decltype(f_evict)>(p[6]);
  Py_XSETREF(g_check, Py_NewRef(a[0]));
  return none();
  END_HANDLE_TH_ERRORS
}

#define KVQ_FN(name) {#name, (PyCFunction)(void (*)(void))bind_##name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KVQ_FN(connect), KVQ_FN(rope), KVQ_FN(append), KVQ_FN(gather),
                         KVQ_FN(attn),    KVQ_FN(mass), KVQ_FN(evict),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "kvq_bind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// KVQ_BIND_KEY: the Python and torch that this module is built for; the loader
// looks for it in the file before it loads the module
PyMODINIT_FUNC PyInit_kvq_bind() {
  PyObject *m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "key", KVQ_BIND_KEY) < 0) Py_CLEAR(m);
  return m;
}
