// Compiled half of the Python binding of the serving operators (kda.py): checks of the tensors,
// allocation of the outputs and the call of the C entry point. These calls are made once or more
// per layer and token, and at small sizes their host time is what bounds them: the same checks in
// Python took 9-14 us a call on the GPU machine's cores, the launch itself 2.
//
// Every function takes all its arguments by position (kda.py has the signatures), returns what
// kda.py returns, or the kda_status as an int where the C call refused; it raises TypeError and
// ValueError for tensors of the wrong type or shape. Contiguity, types and shapes are checked
// here, values by the C entry point.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>

#include "../../include/kda.h"

namespace {

using at::Tensor;
constexpr int64_t kPage = 64;

[[noreturn]] void refuse(PyObject* type, const char* what, const char* name) {
  PyErr_Format(type, "%s %s", name, what);
  throw python_error();
}
void require(bool ok, const char* what, const char* name) {
  if (!ok) refuse(PyExc_ValueError, what, name);
}
void require_type(bool ok, const char* what, const char* name) {
  if (!ok) refuse(PyExc_TypeError, what, name);
}

const Tensor* opt(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  require_type(THPVariable_Check(o), "must be a tensor or None", name);
  return &THPVariable_Unpack(o);
}
const Tensor& need(PyObject* o, const char* name) {
  require_type(THPVariable_Check(o), "must be a tensor", name);
  return THPVariable_Unpack(o);
}

// The tensors of a call, all on one device: the current one, whose stream the call runs on.
struct Devices {
  c10::Device first{c10::DeviceType::CPU};
  bool any = false, mixed = false;
  void see(const Tensor& t) {
    if (!any) first = t.device();
    mixed |= any && t.device() != first;
    any = true;
  }
  void check() const {
    require(!mixed && first.is_cuda() && first.index() == c10::cuda::current_device(),
            "must be on the current CUDA device", "tensors");
  }
};

kda_dtype code_of(at::ScalarType t, const char* name) {
  require_type(t == at::kBFloat16 || t == at::kFloat, "must be bfloat16 or float32", name);
  return t == at::kBFloat16 ? KDA_BF16 : KDA_F32;
}

// Pointer of a contiguous tensor of n entries of a type (nullptr for none).
template <class P = void>
P* vec(Devices& d, const Tensor* t, at::ScalarType type, int64_t n, const char* name) {
  if (!t) return nullptr;
  require_type(t->scalar_type() == type, "has the wrong type", name);
  require(t->numel() == n && t->is_contiguous(), "must be contiguous and of the right size", name);
  d.see(*t);
  return static_cast<P*>(t->data_ptr());
}

// Token stride of [tokens, H, d] rows whose heads are contiguous (any token stride).
int64_t heads(Devices& d, const Tensor& t, at::IntArrayRef shape, at::ScalarType type,
              const char* name) {
  require_type(t.scalar_type() == type, "has the wrong type", name);
  require(t.sizes() == shape && t.stride(2) == 1 && (t.stride(1) == shape[2] || shape[1] <= 1),
          "must be [tokens, heads, d] with contiguous heads", name);
  d.see(t);
  return shape[0] > 1 ? t.stride(0) : shape[1] * shape[2];
}

int as_int(int64_t v, const char* name) {
  require(v >= 0 && v <= 0x7fffffff, "is too large", name);
  return (int)v;
}

double as_double(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
bool as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}
uint32_t* status_of(Devices& d, PyObject* o) {
  const Tensor* t = opt(o, "status");
  if (!t) return nullptr;
  require_type(t->scalar_type() == at::kInt, "must be int32", "status");
  require(t->numel() >= 1, "must hold a word", "status");
  d.see(*t);
  return static_cast<uint32_t*>(t->data_ptr());
}

// The stream of a call (None: the current one). While this lives, tensors are allocated on it: the
// allocator orders the uses of a block by the stream that it was allocated on, so a block that was
// freed while another stream still works on it is not written by this call ahead of that work.
// Made once the tensors of the call are known to be on the current device.
struct CallStream {
  kda_stream_t s;
  std::optional<c10::cuda::CUDAStream> caller;  // the current stream, where it is another one
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  explicit CallStream(PyObject* o) {
    const auto current = c10::cuda::getCurrentCUDAStream();
    s = (kda_stream_t)current.stream();
    if (o == Py_None) return;
    s = (kda_stream_t)PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw python_error();
    if (s == (kda_stream_t)current.stream()) return;
    caller = current;
    guard.emplace(c10::cuda::getStreamFromExternal((cudaStream_t)s, current.device_index()));
  }
};

// An output: the caller's tensor, or a new one.
struct Out {
  PyObject* given = nullptr;
  Tensor made;
  const Tensor* t = nullptr;
  void set(PyObject* o, at::IntArrayRef shape, const at::TensorOptions& opts, const char* name) {
    if (o != Py_None) {
      given = o;
      t = &need(o, name);
    } else {
      made = at::empty(shape, opts);
      t = &made;
    }
  }
  // A tensor made on the call's stream goes to the caller, whose current stream is the one that it
  // is likely used on: its memory is not handed out again before that stream has come so far.
  void handed_to(const CallStream& c) const {
    if (c.caller && made.defined())
      c10::cuda::CUDACachingAllocator::recordStream(made.storage().data_ptr(), *c.caller);
  }
  PyObject* object() const {
    if (!given) return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
  }
};
PyObject* tuple_of(std::initializer_list<PyObject*> items) {
  PyObject* r = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (!r || !o) throw python_error();
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}
PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  throw python_error();
}

// Lets other Python threads run during a C call (a launch waits where the queue is full). Every
// argument is converted before.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

struct Cache {
  void *kc, *vc;
  float *ks, *vs;
  const int32_t* table;
  int64_t n_pages, H, d;
  int max_pages;
};
// a: page_table, k_cache, k_scale, v_cache, v_scale
Cache cache_of(Devices& dv, PyObject* const* a, int64_t rows) {
  const Tensor &table = need(a[0], "page_table"), &kc = need(a[1], "k_cache"),
               &ks = need(a[2], "k_scale"), &vc = need(a[3], "v_cache"), &vs = need(a[4], "v_scale");
  const auto type = kc.scalar_type();
  require_type((type == at::kFloat8_e4m3fn || type == at::kByte) && vc.scalar_type() == type,
               "must be float8_e4m3fn (or uint8 codes)", "the caches");
  require(kc.dim() == 4 && kc.size(2) == kPage && vc.sizes() == kc.sizes() && kc.is_contiguous() &&
              vc.is_contiguous(),
          "must both be contiguous [n_pages, Hkv, 64, d]", "the caches");
  Cache c;
  c.n_pages = kc.size(0);
  c.H = kc.size(1);
  c.d = kc.size(3);
  for (const Tensor* s : {&ks, &vs})
    require(s->dim() == 2 && s->size(0) == c.n_pages && s->size(1) == c.H,
            "must be [n_pages, Hkv]", "the scales");
  require(table.dim() == 2 && table.size(0) == rows,
          "must be [rows, max_pages], a row for each entry of start", "page_table");
  c.max_pages = as_int(table.size(1), "max_pages");
  dv.see(kc);
  dv.see(vc);
  c.kc = kc.data_ptr();
  c.vc = vc.data_ptr();
  c.ks = vec<float>(dv, &ks, at::kFloat, ks.numel(), "k_scale");
  c.vs = vec<float>(dv, &vs, at::kFloat, vs.numel(), "v_scale");
  c.table = vec<int32_t>(dv, &table, at::kInt, table.numel(), "page_table");
  return c;
}

// q, k, q_weight, k_weight, eps, l2, cos_sin, positions, interleaved, q_out, k_out, status, stream
PyObject* head_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 13);
  const Tensor *q = opt(a[0], "q"), *k = opt(a[1], "k");
  require_type(q || k, "must not both be None", "q and k");
  const Tensor& x = q ? *q : *k;
  require(x.dim() == 3, "must be [tokens, heads, d]", "q and k");
  const auto type = x.scalar_type();
  const kda_dtype dt = code_of(type, "q and k");
  const int64_t T = x.size(0), d = x.size(2);
  Devices dv;
  Out out[2];
  int64_t stride[2] = {0, 0}, out_stride[2] = {0, 0};
  int H[2] = {0, 0};
  const void* src[2] = {nullptr, nullptr};
  void* dst[2] = {nullptr, nullptr};
  const Tensor* side[2] = {q, k};
  const char* name[2] = {"q", "k"};
  for (int i = 0; i < 2; ++i) {
    if (!side[i]) continue;
    const Tensor& t = *side[i];
    require(t.dim() == 3 && t.size(0) == T && t.size(2) == d,
            "must have the tokens and the head size of the other", name[i]);
    H[i] = as_int(t.size(1), name[i]);
    stride[i] = heads(dv, t, t.sizes(), type, name[i]);
  }
  const Tensor* table = opt(a[6], "cos_sin");
  require(!table || table->dim() == 2, "must be [n_pos, rot_dim]", "cos_sin");
  const float* cs = vec<float>(dv, table, at::kFloat, table ? table->numel() : 0, "cos_sin");
  const float* qw = vec<float>(dv, opt(a[2], "q_weight"), at::kFloat, d, "q_weight");
  const float* kw = vec<float>(dv, opt(a[3], "k_weight"), at::kFloat, d, "k_weight");
  const int32_t* pos = vec<int32_t>(dv, opt(a[7], "positions"), at::kInt, T, "positions");
  uint32_t* status = status_of(dv, a[11]);
  dv.check();
  const CallStream on(a[12]);
  for (int i = 0; i < 2; ++i) {
    if (!side[i]) continue;
    const Tensor& t = *side[i];
    out[i].set(a[9 + i], t.sizes(), at::TensorOptions().dtype(type).device(t.device()),
               i ? "k_out" : "q_out");
    out_stride[i] = heads(dv, *out[i].t, t.sizes(), type, i ? "k_out" : "q_out");
    src[i] = t.data_ptr();
    dst[i] = out[i].t->data_ptr();
  }
  dv.check();
  const int tokens = as_int(T, "tokens"), hd = as_int(d, "d");
  const int rot = table ? as_int(table->size(1), "rot_dim") : 0;
  const int64_t n_pos = table ? table->size(0) : 0;
  const float eps = (float)as_double(a[4]);
  const unsigned flags =
      (as_bool(a[5]) ? KDA_NORM_L2 : 0u) | (as_bool(a[8]) ? KDA_ROPE_INTERLEAVED : 0u);
  const kda_status st = [&] {
    NoGil g;
    return kda_head_norm_rope(dt, tokens, H[0], H[1], hd, src[0], stride[0], src[1], stride[1], qw,
                              kw, eps, flags, cs, n_pos, rot, pos, dst[0], out_stride[0], dst[1],
                              out_stride[1], status, on.s);
  }();
  if (st != KDA_OK) return PyLong_FromLong(st);
  for (const Out& o : out) o.handed_to(on);
  return tuple_of({q ? out[0].object() : none(), k ? out[1].object() : none()});
  END_HANDLE_TH_ERRORS
}

// k, v, start, page_table, k_cache, k_scale, v_cache, v_scale, cu_seqlens, lens, status, stream
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 12);
  const Tensor &k = need(a[0], "k"), &v = need(a[1], "v"), &start = need(a[2], "start");
  Devices dv;
  const int64_t rows = start.numel();
  const Cache c = cache_of(dv, a + 3, rows);
  const auto type = k.scalar_type();
  const kda_dtype dt = code_of(type, "k and v");
  require(k.dim() == 3 && k.size(1) == c.H && k.size(2) == c.d,
          "must be [tokens, Hkv, d] of the cache", "k and v");
  const int64_t ks = heads(dv, k, k.sizes(), type, "k");
  const int64_t vs = heads(dv, v, k.sizes(), type, "v");
  const int32_t* cu = vec<int32_t>(dv, opt(a[8], "cu_seqlens"), at::kInt, rows + 1, "cu_seqlens");
  const int32_t* st0 = vec<int32_t>(dv, &start, at::kInt, rows, "start");
  const int32_t* lens = vec<int32_t>(dv, opt(a[9], "lens"), at::kInt, rows, "lens");
  uint32_t* status = status_of(dv, a[10]);
  dv.check();
  const int nr = as_int(rows, "rows"), T = as_int(k.size(0), "tokens"), H = as_int(c.H, "Hkv"),
            d = as_int(c.d, "d");
  const CallStream on(a[11]);
  const kda_status st = [&] {
    NoGil g;
    return kda_cache_write(dt, nr, T, cu, st0, lens, H, d, k.data_ptr(), ks, v.data_ptr(), vs,
                           c.table, c.max_pages, c.kc, c.ks, c.vc, c.vs, c.n_pages, status, on.s);
  }();
  return st != KDA_OK ? PyLong_FromLong(st) : none();
  END_HANDLE_TH_ERRORS
}

at::ScalarType dtype_of(PyObject* o) {
  require_type(THPDtype_Check(o), "must be a torch.dtype", "dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// start, page_table, k_cache, k_scale, v_cache, v_scale, total_tokens, cu_seqlens, dtype, k, v,
// status, stream
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 13);
  const Tensor& start = need(a[0], "start");
  Devices dv;
  const int64_t rows = start.numel();
  const Cache c = cache_of(dv, a + 1, rows);
  const int64_t T = PyLong_AsLongLong(a[6]);
  if (T == -1 && PyErr_Occurred()) throw python_error();
  require(T >= 0, "must be >= 0", "total_tokens");
  const int32_t* cu = vec<int32_t>(dv, opt(a[7], "cu_seqlens"), at::kInt, rows + 1, "cu_seqlens");
  const int32_t* st0 = vec<int32_t>(dv, &start, at::kInt, rows, "start");
  // the outputs' type: the given tensors', else dtype
  const Tensor *kg = opt(a[9], "k"), *vg = opt(a[10], "v");
  const auto type = kg ? kg->scalar_type() : vg ? vg->scalar_type() : dtype_of(a[8]);
  const kda_dtype dt = code_of(type, "k and v");
  const int64_t shape[3] = {T, c.H, c.d};
  const auto opts = at::TensorOptions().dtype(type).device(start.device());
  uint32_t* status = status_of(dv, a[11]);
  dv.check();
  const CallStream on(a[12]);
  Out out[2];
  void* dst[2];
  for (int i = 0; i < 2; ++i) {
    out[i].set(a[9 + i], shape, opts, i ? "v" : "k");
    require(out[i].t->sizes() == at::IntArrayRef(shape), "must be [total_tokens, Hkv, d]",
            i ? "v" : "k");
    dst[i] = vec(dv, out[i].t, type, T * c.H * c.d, i ? "v" : "k");
  }
  dv.check();
  const int nr = as_int(rows, "rows"), total = as_int(T, "total_tokens"), H = as_int(c.H, "Hkv"),
            d = as_int(c.d, "d");
  const kda_status st = [&] {
    NoGil g;
    return kda_cache_read(dt, nr, total, cu, st0, H, d, c.table, c.max_pages, c.kc, c.ks, c.vc,
                          c.vs, c.n_pages, dst[0], dst[1], status, on.s);
  }();
  if (st != KDA_OK) return PyLong_FromLong(st);
  for (const Out& o : out) o.handed_to(on);
  return tuple_of({out[0].object(), out[1].object()});
  END_HANDLE_TH_ERRORS
}

// q, start, page_table, k_cache, k_scale, v_cache, v_scale, scale, lens, o, workspace, status,
// stream
PyObject* cache_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 13);
  const Tensor &q = need(a[0], "q"), &start = need(a[1], "start");
  Devices dv;
  const int64_t B = start.numel();
  const Cache c = cache_of(dv, a + 2, B);
  const auto type = q.scalar_type();
  const kda_dtype dt = code_of(type, "q");
  require(q.dim() >= 3 && q.size(-1) == c.d, "must be [.., Hq, d] with the cache's head size", "q");
  const int64_t Hq = q.size(-2), size = q.numel(), per = B * Hq * c.d;
  const int64_t W = per ? size / per : 0;
  require(W * per == size, "must hold batch x window tokens", "q");
  const void* qp = vec(dv, &q, type, size, "q");
  const int32_t* st0 = vec<int32_t>(dv, &start, at::kInt, B, "start");
  const int32_t* lens = vec<int32_t>(dv, opt(a[8], "lens"), at::kInt, B, "lens");
  uint32_t* status = status_of(dv, a[11]);
  dv.check();
  const CallStream on(a[12]);
  Out out, ws;
  out.set(a[9], q.sizes(), at::TensorOptions().dtype(type).device(q.device()), "o");
  void* op = vec(dv, out.t, type, size, "o");
  const int b = as_int(B, "batch"), w = as_int(W, "window"), hq = as_int(Hq, "Hq"),
            hkv = as_int(c.H, "Hkv"), d = as_int(c.d, "d");
  int64_t bytes = (int64_t)kda_cache_attention_workspace(b, w, hq, hkv, d);
  void* wp = nullptr;
  if (bytes > 0 || a[10] != Py_None) {
    ws.set(a[10], {bytes}, at::TensorOptions().dtype(at::kByte).device(q.device()), "workspace");
    require(ws.t->is_contiguous(), "must be contiguous", "workspace");
    dv.see(*ws.t);
    bytes = (int64_t)ws.t->nbytes();
    wp = ws.t->data_ptr();
  }
  dv.check();
  const float scale = (float)as_double(a[7]);
  const kda_status st = [&] {
    NoGil g;
    return kda_cache_attention(dt, b, w, hq, hkv, d, scale, qp, st0, lens, c.table, c.max_pages,
                               c.kc, c.ks, c.vc, c.vs, c.n_pages, op, wp, (size_t)bytes, status,
                               on.s);
  }();
  if (st != KDA_OK) return PyLong_FromLong(st);
  out.handed_to(on);
  return out.object();
  END_HANDLE_TH_ERRORS
}

// Row stride of [batch, places, vocab] rows at one stride, entries contiguous.
int64_t rows3(Devices& dv, const Tensor& t, at::IntArrayRef shape, at::ScalarType type,
              const char* name) {
  require_type(t.scalar_type() == type, "has the wrong type", name);
  require(t.sizes() == shape, "has the wrong shape", name);
  const int64_t s = shape[1] > 1 ? t.stride(1) : (shape[0] > 1 ? t.stride(0) : shape[2]);
  require((t.stride(2) == 1 || shape[2] <= 1) && (shape[0] <= 1 || t.stride(0) == shape[1] * s),
          "must have contiguous entries and evenly spaced rows", name);
  dv.see(t);
  return s;
}

// target_probs, draft_tokens, u_accept, u_sample, draft_probs, lens, write_slots, tokens,
// n_accepted, resume_slots, status, stream
PyObject* draft_verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 12);
  const Tensor &target = need(a[0], "target_probs"), &drafts = need(a[1], "draft_tokens"),
               &ua = need(a[2], "u_accept"), &us = need(a[3], "u_sample");
  const auto type = target.scalar_type();
  const kda_dtype dt = code_of(type, "target_probs");
  require(target.dim() == 3, "must be [batch, window + 1, vocab]", "target_probs");
  const int64_t B = target.size(0), W1 = target.size(1), W = W1 - 1, V = target.size(2);
  require(W >= 0, "must be [batch, window + 1, vocab]", "target_probs");
  for (const Tensor* t : {&drafts, &ua})
    require(t->dim() == 2 && t->size(0) == B && t->size(1) == W, "must be [batch, window]",
            "draft_tokens and u_accept");
  Devices dv;
  const int64_t ts = rows3(dv, target, target.sizes(), type, "target_probs");
  const Tensor* draft = opt(a[4], "draft_probs");
  int64_t ds = 0;
  const void* dp = nullptr;
  if (draft && W > 0) {
    const int64_t shape[3] = {B, W, V};
    ds = rows3(dv, *draft, shape, type, "draft_probs");
    dp = draft->data_ptr();
  }
  const int32_t* xp = vec<int32_t>(dv, &drafts, at::kInt, B * W, "draft_tokens");
  const float* uap = vec<float>(dv, &ua, at::kFloat, B * W, "u_accept");
  const float* usp = vec<float>(dv, &us, at::kFloat, B, "u_sample");
  const int32_t* lens = vec<int32_t>(dv, opt(a[5], "lens"), at::kInt, B, "lens");
  const int32_t* slots =
      vec<int32_t>(dv, opt(a[6], "write_slots"), at::kInt, B * W1, "write_slots");
  const auto opts = at::TensorOptions().dtype(at::kInt).device(target.device());
  uint32_t* status = status_of(dv, a[10]);
  dv.check();
  const CallStream on(a[11]);
  Out tokens, taken, resume;
  tokens.set(a[7], {B, W1}, opts, "tokens");
  taken.set(a[8], {B}, opts, "n_accepted");
  const bool has_resume = slots || a[9] != Py_None;
  if (has_resume) resume.set(a[9], {B}, opts, "resume_slots");
  int32_t* tp = vec<int32_t>(dv, tokens.t, at::kInt, B * W1, "tokens");
  int32_t* np = vec<int32_t>(dv, taken.t, at::kInt, B, "n_accepted");
  int32_t* rp = vec<int32_t>(dv, resume.t, at::kInt, B, "resume_slots");
  dv.check();
  const int b = as_int(B, "batch"), w = as_int(W, "window"), v = as_int(V, "vocab");
  const kda_status st = [&] {
    NoGil g;
    return kda_draft_verify(dt, b, w, v, target.data_ptr(), ts, dp, ds, xp, lens, uap, usp, slots,
                            tp, np, rp, status, on.s);
  }();
  if (st != KDA_OK) return PyLong_FromLong(st);
  for (const Out* o : {&tokens, &taken, &resume}) o->handed_to(on);
  return tuple_of({taken.object(), tokens.object(), has_resume ? resume.object() : none()});
  END_HANDLE_TH_ERRORS
}

#define KDA_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KDA_METHOD(head_norm_rope), KDA_METHOD(cache_write),
                         KDA_METHOD(cache_read),     KDA_METHOD(cache_attention),
                         KDA_METHOD(draft_verify),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_native(void) { return PyModule_Create(&module); }
