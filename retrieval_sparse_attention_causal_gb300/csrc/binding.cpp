// Python binding of the decoding operators, on the side of the tensors: argument checks,
// outputs and scratch from PyTorch's allocator, the device and stream of the tensors, and
// the call into the C ABI, in one native function each.
//
// A decoding step is many short calls.  Through ctypes the checks and conversions of a call
// take longer than its kernels (24 us for a rotary call whose kernel takes 2); here a call
// costs little more than its allocations and its launch.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/gca.h"

namespace {

using at::Tensor;
using Args = PyObject* const*;

struct Refused {  // becomes a Python exception of this type
  PyObject* type;
  std::string what;
};
void need(bool ok, const char* what) {
  if (!ok) throw Refused{PyExc_ValueError, what};
}
struct Failed { gca_status status; };  // becomes a GCAError
void check(gca_status s) {
  if (s != GCA_OK) throw Failed{s};
}
PyObject* g_error = nullptr;  // the GCAError class

// ---------------------------------------------------------------- arguments
const Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(what) + " must be a tensor"};
  return THPVariable_Unpack(o);
}
const Tensor* optional(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }
long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int as_int(PyObject* o, const char* what) {
  const long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) throw Refused{PyExc_ValueError, std::string(what) + " is out of range"};
  return (int)v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

gca_dtype dtype_of(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return GCA_BF16;
  if (t.scalar_type() == at::kFloat) return GCA_F32;
  throw Refused{PyExc_TypeError, std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + " (bfloat16 or float32)"};
}

// The device of a call's tensors, made current.
class On {
 public:
  void add(const Tensor* t) {
    if (!t) return;
    need(t->is_cuda(), "tensors must live on a CUDA device");
    const int d = t->get_device();
    if (dev_ < 0) dev_ = d;
    need(d == dev_, "tensors must live on one device");
  }
  void enter() { guard_.set_index(dev_); }
  int device() const { return dev_; }
  gca_stream_t stream() const { return reinterpret_cast<gca_stream_t>(c10::cuda::getCurrentCUDAStream(dev_).stream()); }
  at::TensorOptions options(at::ScalarType t) const { return at::TensorOptions().dtype(t).device(at::kCUDA, dev_); }

 private:
  int dev_ = -1;
  c10::cuda::OptionalCUDAGuard guard_;
};

// The stride of an axis of one is no address: any number may stand there.
gca_heads heads(const Tensor& t) {
  return gca_heads{t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0, t.size(2) > 1 ? t.stride(2) : 0};
}
bool unit(const Tensor& t) { return t.size(3) == 1 || t.stride(3) == 1; }
bool is(const Tensor& t, at::ScalarType type, at::IntArrayRef shape) {
  return t.scalar_type() == type && t.sizes() == shape && t.is_contiguous();
}
void need_int32(const Tensor& t, at::IntArrayRef shape, const char* what) {
  if (is(t, at::kInt, shape)) return;
  std::string s = std::string(what) + " must be a contiguous int32 [";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  throw Refused{PyExc_ValueError, s + "] tensor"};
}
PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}
PyObject* pair(PyObject* a, PyObject* b) {
  if (!a || !b) {
    Py_XDECREF(a);
    Py_XDECREF(b);
    throw python_error();
  }
  PyObject* t = PyTuple_New(2);
  if (!t) throw python_error();
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  return t;
}

// ---------------------------------------------------------------- error words and scratch
constexpr int64_t kErrBytes = 256;
std::mutex g_mu;
std::vector<Tensor>& words() {
  static auto* w = new std::vector<Tensor>;  // not destroyed: CUDA may be gone by then
  return *w;
}

// The default error word of a device, zeroed when it is made.
Tensor error_word(int dev) {
  std::lock_guard<std::mutex> lk(g_mu);
  auto& w = words();
  if ((int)w.size() <= dev) w.resize(dev + 1);
  if (!w[dev].defined()) {
    need(c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None,
         "call cache_workspace(device), or any of these operators, once before a capture");
    c10::cuda::CUDAGuard guard(dev);
    w[dev] = at::zeros({kErrBytes}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, dev));
    c10::cuda::getCurrentCUDAStream(dev).synchronize();  // other streams' kernels may set it
  }
  return w[dev];
}
struct Word {
  Tensor t;
  void* p;
  size_t n;
  Word(const Tensor* given, const On& on) : t(given ? *given : error_word(on.device())), p(t.data_ptr()), n((size_t)t.numel()) {}
};
struct Scratch {
  Tensor t;
  void* p;
  size_t n;
  Scratch(size_t bytes, const On& on) : t(at::empty({(int64_t)bytes}, on.options(at::kByte))), p(t.data_ptr()), n(bytes) {}
};

// ---------------------------------------------------------------- rotary positions
// q, k, freq, positions, interleaved, gain, q_out, k_out, backward
PyObject* rotary(Args a) {
  const Tensor& q = tensor(a[0], "q");
  const Tensor* k = optional(a[1], "k");
  const Tensor& freq = tensor(a[2], "freq");
  const Tensor* pos = optional(a[3], "positions");
  const Tensor *qo = optional(a[6], "q_out"), *ko = optional(a[7], "k_out");
  const gca_dtype dt = dtype_of(q);
  need(q.dim() == 4 && unit(q), "q must be [B, L, H, dh] with unit stride in its last dim");
  const int64_t B = q.size(0), L = q.size(1), H = q.size(2), dh = q.size(3), Hkv = k ? k->size(2) : 0;
  if (k)
    need(k->dim() == 4 && k->size(0) == B && k->size(1) == L && k->size(3) == dh && k->scalar_type() == q.scalar_type() && unit(*k),
         "k must be [B, L, Hkv, dh] like q, with unit stride in its last dim");
  need(freq.scalar_type() == at::kLong && freq.dim() == 1 && freq.is_contiguous(), "freq must be what rotary_frequencies returned");
  int64_t pos_bs = 0;
  if (pos) {
    const int64_t nd = pos->dim();
    need(pos->scalar_type() == at::kInt && ((nd == 1 && pos->size(0) == L) || (nd == 2 && pos->size(1) == L && (pos->size(0) == B || pos->size(0) == 1))) &&
             (L == 1 || pos->stride(nd - 1) == 1),
         "positions must be int32 [B, L] or [L], with unit stride in the last dim");
    if (nd == 2 && pos->size(0) == B && B > 1) pos_bs = pos->stride(0);
  }
  need(k || !ko, "k_out needs k");
  On on;
  for (const Tensor* t : {&q, k, &freq, pos, qo, ko}) on.add(t);
  on.enter();
  Tensor q_new, k_new;
  if (!qo) q_new = at::empty({B, L, H, dh}, on.options(q.scalar_type()));
  if (k && !ko) k_new = at::empty({B, L, Hkv, dh}, on.options(q.scalar_type()));
  const Tensor& qt = qo ? *qo : q_new;
  const Tensor& kt = ko ? *ko : k_new;
  need(qt.sizes() == q.sizes() && qt.scalar_type() == q.scalar_type() && unit(qt), "q_out must be like q");
  if (k) need(kt.sizes() == k->sizes() && kt.scalar_type() == k->scalar_type() && unit(kt), "k_out must be like k");
  const gca_heads hq = heads(q), hqo = heads(qt), hk = k ? heads(*k) : gca_heads{}, hko = k ? heads(kt) : gca_heads{};
  need(B <= INT32_MAX && L <= INT32_MAX && H <= INT32_MAX && Hkv <= INT32_MAX && dh <= INT32_MAX && freq.size(0) < (1 << 20),
       "a size is out of range");
  check(gca_rotary(&hq, k ? &hk : nullptr, &hqo, k ? &hko : nullptr, dt, (int)B, (int)L, (int)H, (int)Hkv, (int)dh, 2 * (int)freq.size(0),
                   (int)integer(a[4]), (int)integer(a[8]), static_cast<const uint64_t*>(freq.data_ptr()),
                   pos ? static_cast<const int32_t*>(pos->data_ptr()) : nullptr, pos_bs, (float)number(a[5]), on.stream()));
  return pair(qo ? same(a[6]) : wrap(q_new), k ? (ko ? same(a[7]) : wrap(k_new)) : same(Py_None));
}

// ---------------------------------------------------------------- pools
// k_pages, v_pages, table, lengths, refs (or None): the state as the tensors have it at this call.  Nothing
// of it is kept: a tensor that was replaced or resized since the last call is seen as it is.
gca_cache pool_of(Args a, On& on) {
  const Tensor &k = tensor(a[0], "k_pages"), &v = tensor(a[1], "v_pages"), &table = tensor(a[2], "table"), &len = tensor(a[3], "lengths");
  const Tensor* refs = optional(a[4], "refs");
  need(k.dim() == 4 && k.size(1) == GCA_CHUNK && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type() && k.is_contiguous() && v.is_contiguous(),
       "k_pages, v_pages must be contiguous [pages, 64, heads, dh] tensors of one type");
  need(table.scalar_type() == at::kInt && table.dim() == 2 && table.is_contiguous(), "table must be a contiguous int32 [slots, width] tensor");
  need_int32(len, {table.size(0)}, "lengths");
  if (refs) need_int32(*refs, {k.size(0)}, "refs");
  for (const Tensor* t : {&k, &v, &table, &len, refs}) on.add(t);
  need(k.size(0) <= INT32_MAX && k.size(2) <= INT32_MAX && k.size(3) <= INT32_MAX && table.size(0) <= INT32_MAX && table.size(1) <= INT32_MAX,
       "a size is out of range");
  return gca_cache{k.data_ptr(), v.data_ptr(), dtype_of(k), (int)k.size(2), (int)k.size(3), (int)k.size(0),
                   static_cast<int32_t*>(table.data_ptr()), (int)table.size(0), (int)table.size(1),
                   static_cast<int32_t*>(len.data_ptr()), refs ? static_cast<int32_t*>(refs->data_ptr()) : nullptr};
}
// k_pages, v_pages, table, lengths, refs: refused where a call on them would be.
PyObject* check_pool(Args a) {
  On on;
  pool_of(a, on);
  Py_RETURN_NONE;
}

// ---------------------------------------------------------------- attention
// q, k_new, v_new | mask, positions, window, scale, out, lse, ws
PyObject* attend(const gca_cache& c, On& on, Args x, Args y) {
  const Tensor &q = tensor(x[0], "q"), &kn = tensor(x[1], "k_new"), &vn = tensor(x[2], "v_new");
  const Tensor *mask = optional(y[0], "mask"), *pos = optional(y[1], "positions"), *out = optional(y[4], "out"), *lse = optional(y[5], "lse"),
               *ws = optional(y[6], "ws");
  const int window = as_int(y[2], "window");
  need(q.dim() == 4 && q.size(3) == c.dh && dtype_of(q) == c.dtype && unit(q),
       "q must be [B, T, H, dh] of the pages' type and head dim, with unit stride in its last dim");
  const int64_t B = q.size(0), T = q.size(1), H = q.size(2), dh = q.size(3);
  for (const Tensor* t : {&kn, &vn})
    need(t->dim() == 4 && t->size(0) == B && t->size(1) == T && t->size(2) == c.heads && t->size(3) == dh &&
             t->scalar_type() == q.scalar_type() && unit(*t),
         "k_new, v_new must be [B, T, heads, dh] of the pages' type, with unit stride in the last dim");
  if (mask) need(is(*mask, at::kLong, {B, T, (T + 63) / 64}), "mask must be a contiguous int64 [B, T, ceil(T/64)] tensor");
  if (pos) need_int32(*pos, {B, T}, "positions");
  if (out) need(out->sizes() == q.sizes() && out->scalar_type() == q.scalar_type() && out->is_contiguous(), "out must be contiguous, like q");
  if (lse) need(is(*lse, at::kFloat, {B, T, H}), "lse must be a contiguous float32 [B, T, H] tensor");
  need(B >= 1 && B <= INT32_MAX && T >= 1 && T <= GCA_MAX_DRAFT && H <= INT32_MAX, "B must be >= 1 and T in 1..256");
  for (const Tensor* t : {&q, &kn, &vn, mask, pos, out, lse, ws}) on.add(t);
  on.enter();
  const float scale = y[3] == Py_None ? 1.0f / std::sqrt((float)dh) : (float)number(y[3]);
  Tensor o_new, l_new;
  if (!out) o_new = at::empty({B, T, H, dh}, on.options(q.scalar_type()));
  if (!lse) l_new = at::empty({B, T, H}, on.options(at::kFloat));
  const Word w(ws, on);
  const Scratch s(gca_tree_attention_scratch_size((int)B, (int)T, (int)H, c.heads, c.dh, c.width, window, c.dtype), on);
  const gca_heads hq = heads(q), hk = heads(kn), hv = heads(vn);
  check(gca_tree_attention(&hq, &hk, &hv, &c, (int)B, (int)T, (int)H, mask ? static_cast<const uint64_t*>(mask->data_ptr()) : nullptr,
                           pos ? static_cast<const int32_t*>(pos->data_ptr()) : nullptr, window, scale, out ? out->data_ptr() : o_new.data_ptr(),
                           static_cast<float*>(lse ? lse->data_ptr() : l_new.data_ptr()), w.p, w.n, s.p, s.n, on.stream()));
  return pair(out ? same(y[4]) : wrap(o_new), lse ? same(y[5]) : wrap(l_new));
}
// q, k_new, v_new, the cache's five, mask, positions, window, scale, out, lse, ws
PyObject* tree_attention(Args a) {
  On on;
  const gca_cache c = pool_of(a + 3, on);
  return attend(c, on, a, a + 8);
}
// parents, lengths, ws
PyObject* tree_plan(Args a) {
  const Tensor &parents = tensor(a[0], "parents"), &len = tensor(a[1], "lengths");
  const Tensor* ws = optional(a[2], "ws");
  need(parents.dim() == 2, "parents must be int32 [B, T]");
  const int64_t B = parents.size(0), T = parents.size(1);
  need_int32(parents, {B, T}, "parents");
  need(len.scalar_type() == at::kInt && len.dim() == 1 && len.size(0) >= B && len.is_contiguous(),
       "lengths must be a contiguous int32 tensor of B entries or more");
  need(B <= INT32_MAX && T <= INT32_MAX, "a size is out of range");
  On on;
  for (const Tensor* t : {&parents, &len, ws}) on.add(t);
  on.enter();
  Tensor mask = at::empty({B, T, (T + 63) / 64}, on.options(at::kLong)), pos = at::empty({B, T}, on.options(at::kInt));
  const Word w(ws, on);
  check(gca_tree_plan(static_cast<const int32_t*>(parents.data_ptr()), static_cast<const int32_t*>(len.data_ptr()), (int)B, (int)T,
                      static_cast<uint64_t*>(mask.data_ptr()), static_cast<int32_t*>(pos.data_ptr()), w.p, w.n, on.stream()));
  return pair(wrap(mask), wrap(pos));
}

// ---------------------------------------------------------------- page operations
const int32_t* ints(const Tensor* t) { return t ? static_cast<const int32_t*>(t->data_ptr()) : nullptr; }
const int32_t* entries(const Tensor* slots, int64_t n, const gca_cache& c) {
  need(n >= 1 && n <= INT32_MAX, "a call needs an entry");
  if (slots) need_int32(*slots, {n}, "slots");
  else need(n <= c.slots, "without `slots` entry i is slot i: there are more entries than slots");
  return ints(slots);
}
// The cache's five, then: k_new, v_new, counts, path, slots, ws
PyObject* append(Args a) {
  const Tensor &k = tensor(a[5], "k_new"), &v = tensor(a[6], "v_new"), &counts = tensor(a[7], "counts");
  const Tensor *path = optional(a[8], "path"), *slots = optional(a[9], "slots"), *ws = optional(a[10], "ws");
  On on;
  const gca_cache c = pool_of(a, on);
  for (const Tensor* t : {&k, &v, &counts, path, slots, ws}) on.add(t);
  need(k.dim() == 4, "k_new, v_new must be [n, T, heads, dh]");
  const int64_t n = k.size(0), T = k.size(1);
  for (const Tensor* t : {&k, &v})
    need(t->dim() == 4 && t->size(0) == n && t->size(1) == T && t->size(2) == c.heads && t->size(3) == c.dh && dtype_of(*t) == c.dtype && unit(*t),
         "k_new, v_new must be [n, T, heads, dh] of the pages' type, with unit stride in the last dim");
  need_int32(counts, {n}, "counts");
  if (path) need_int32(*path, {n, T}, "path");
  const int32_t* ids = entries(slots, n, c);
  need(T <= INT32_MAX, "a size is out of range");
  on.enter();
  const Word w(ws, on);
  const Scratch s(gca_cache_append_scratch_size((int)n, (int)T), on);
  const gca_heads hk = heads(k), hv = heads(v);
  check(gca_cache_append(&c, &hk, &hv, (int)n, (int)T, ids, ints(&counts), ints(path), w.p, w.n, s.p, s.n, on.stream()));
  Py_RETURN_NONE;
}
// src, dst, ws
PyObject* fork(Args a) {
  const Tensor &src = tensor(a[5], "src"), &dst = tensor(a[6], "dst");
  const Tensor* ws = optional(a[7], "ws");
  On on;
  const gca_cache c = pool_of(a, on);
  for (const Tensor* t : {&src, &dst, ws}) on.add(t);
  need(src.dim() == 1 && src.size(0) >= 1 && src.size(0) <= INT32_MAX, "src and dst must be int32 [n]");
  need_int32(src, {src.size(0)}, "src");
  need_int32(dst, {src.size(0)}, "dst");
  on.enter();
  const Word w(ws, on);
  check(gca_cache_fork(&c, (int)src.size(0), ints(&src), ints(&dst), w.p, w.n, on.stream()));
  Py_RETURN_NONE;
}
// begin, end, slots, release, ws
PyObject* trim(Args a) {
  const Tensor *begin = optional(a[5], "begin"), *end = optional(a[6], "end"), *slots = optional(a[7], "slots"), *ws = optional(a[9], "ws");
  On on;
  const gca_cache c = pool_of(a, on);
  for (const Tensor* t : {begin, end, slots, ws}) on.add(t);
  const Tensor* first = begin ? begin : end ? end : slots;
  need(!first || first->dim() == 1, "begin, end and slots must be int32 [n]");
  const int64_t n = first ? first->size(0) : c.slots;
  if (begin) need_int32(*begin, {n}, "begin");
  if (end) need_int32(*end, {n}, "end");
  const int32_t* ids = entries(slots, n, c);
  on.enter();
  const Word w(ws, on);
  check(gca_cache_trim(&c, (int)n, ids, ints(begin), ints(end), (int)integer(a[8]), w.p, w.n, on.stream()));
  Py_RETURN_NONE;
}
// ws
PyObject* compact(Args a) {
  const Tensor* ws = optional(a[5], "ws");
  On on;
  const gca_cache c = pool_of(a, on);
  on.add(ws);
  on.enter();
  Tensor live = at::empty({1}, on.options(at::kInt));
  const Word w(ws, on);
  const Scratch s(gca_cache_compact_scratch_size(c.pages), on);
  check(gca_cache_compact(&c, static_cast<int32_t*>(live.data_ptr()), w.p, w.n, s.p, s.n, on.stream()));
  return wrap(live);
}
// idx, slots, ws
PyObject* lookup(Args a) {
  const Tensor& idx = tensor(a[5], "idx");
  const Tensor *slots = optional(a[6], "slots"), *ws = optional(a[7], "ws");
  On on;
  const gca_cache c = pool_of(a, on);
  for (const Tensor* t : {&idx, slots, ws}) on.add(t);
  need(idx.scalar_type() == at::kInt && idx.dim() >= 2 && idx.is_contiguous() && idx.numel() >= 1 && idx.numel() <= INT32_MAX,
       "idx must be a contiguous int32 [n, ...] tensor");
  const int64_t n = idx.size(0);
  if (slots) need_int32(*slots, {n}, "slots");
  on.enter();
  Tensor out = at::empty_like(idx);
  const Word w(ws, on);
  check(gca_cache_lookup(&c, (int)n, (int)(idx.numel() / n), ints(slots), ints(&idx), static_cast<int32_t*>(out.data_ptr()), w.p, w.n, on.stream()));
  return wrap(out);
}
PyObject* error_word_of(Args a) { return wrap(error_word(as_int(a[0], "device"))); }
PyObject* set_error(Args a) {
  Py_INCREF(a[0]);
  g_error = a[0];
  Py_RETURN_NONE;
}

// ---------------------------------------------------------------- module
template <PyObject* (*F)(Args), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const Failed& f) {
    PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", (int)f.status, gca_last_error_detail()) : nullptr;
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
      PyErr_SetString(PyExc_RuntimeError, gca_last_error_detail());
    }
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}
template <PyObject* (*F)(Args), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {
    method<rotary, 9>("rotary"), method<check_pool, 5>("check_pool"), method<tree_attention, 15>("tree_attention"),
    method<tree_plan, 3>("tree_plan"), method<append, 11>("append"), method<fork, 8>("fork"), method<trim, 10>("trim"),
    method<compact, 6>("compact"), method<lookup, 8>("lookup"),
    method<error_word_of, 1>("error_word"), method<set_error, 1>("set_error"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_gca_decoding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__gca_decoding() { return PyModule_Create(&g_module); }
