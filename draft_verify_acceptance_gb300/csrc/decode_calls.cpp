// decode_calls.cpp -- the ordinary calls of the decode-side and the tree
// operators, without the interpreter between their checks.
//
// A call of a server's step takes the GPU 5 to 15 us, and Python's checks,
// allocations and argument conversions took 20 to 30.  This module does them in
// one go for calls on the current device and stream without debug, out= or
// workspace= that no CUDA graph captures.  Anything else, and any argument that decode.py would refuse,
// returns NotImplemented: decode.py (tree.py) then makes the call itself, or says what is
// wrong with it.  (So no check here is looser than decode.py's, and there are
// no messages.)  Workspaces are decode.py's own, registered here as it makes
// them.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/TensorImpl.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/accumulate.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <initializer_list>
#include <vector>

#include "spec_tree.h"

namespace {

decltype(&spec_attention_workspace_size) attention_workspace_size;
decltype(&spec_paged_attention) attention;
decltype(&spec_cache_append) append;
decltype(&spec_cache_fork_workspace_size) fork_workspace_size;
decltype(&spec_cache_fork) fork_pages;
decltype(&spec_cache_compact_workspace_size) compact_workspace_size;
decltype(&spec_cache_compact) compact;
decltype(&spec_filtered_sample_workspace_size) sample_workspace_size;
decltype(&spec_filtered_sample) sample;
decltype(&spec_tree_attention_workspace_size) tree_workspace_size;
decltype(&spec_tree_attention) tree_attention;
decltype(&spec_cache_append_rotated) append_rotated;
decltype(&spec_tree_accept) tree_accept;
decltype(&spec_cache_keep) cache_keep;
PyObject *fork_result, *compact_result, *sample_result, *accept_result;

struct Workspace {
  long kind, device;
  unsigned long long stream;
  void* p;
  size_t bytes;
};
std::vector<Workspace> workspaces;  // a handful: kinds, devices and streams in use

PyObject* not_done() { Py_RETURN_NOTIMPLEMENTED; }

// One call's device and stream.
struct Where {
  int device;
  cudaStream_t stream;
};
bool where(const at::Tensor& t, Where* w) {
  if (!t.is_cuda()) return false;
  w->device = t.get_device();
  if (w->device != c10::cuda::current_device()) return false;
  w->stream = c10::cuda::getCurrentCUDAStream(w->device).stream();
  return true;
}

bool workspace(long kind, const Where& w, size_t bytes, void** p, size_t* have) {
  *p = nullptr;
  *have = 0;
  if (bytes == 0) return true;
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) return false;
  for (const Workspace& x : workspaces)
    if (x.kind == kind && x.device == w.device && x.stream == reinterpret_cast<unsigned long long>(w.stream)) {
      *p = x.p;
      *have = x.bytes;
      return x.bytes >= bytes;
    }
  return false;
}

// Arguments into out[0..n): up to `positional` by position, all by name.  The
// names that every call takes besides may only say "not given".
bool arguments(PyObject* const* args, Py_ssize_t given, PyObject* kwnames, const char* const* names, int positional, int n,
               PyObject** out) {
  static const char* const other[] = {"stream", "out", "workspace", "debug"};
  if (given > positional) return false;
  for (int i = 0; i < n; ++i) out[i] = i < given ? args[i] : nullptr;
  const Py_ssize_t named = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
  for (Py_ssize_t k = 0; k < named; ++k) {
    PyObject *name = PyTuple_GET_ITEM(kwnames, k), *value = args[given + k];
    int i = 0;
    while (i < n && PyUnicode_CompareWithASCIIString(name, names[i]) != 0) ++i;
    if (i < n) {
      if (out[i]) return false;
      out[i] = value;
      continue;
    }
    if (value != Py_None && value != Py_False) return false;
    bool known = false;
    for (const char* o : other) known |= PyUnicode_CompareWithASCIIString(name, o) == 0;
    if (!known) return false;
  }
  return true;
}

const at::Tensor* tensor(PyObject* o) { return o && THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A contiguous int32 vector of n elements.
bool ints(const at::Tensor* t, int64_t n, int device, const int32_t** p) {
  if (!t || t->scalar_type() != at::kInt || t->dim() != 1 || t->size(0) != n || !t->is_cuda() || t->get_device() != device ||
      !t->is_contiguous())
    return false;
  *p = static_cast<const int32_t*>(t->data_ptr());
  return true;
}

struct Table {
  const int32_t* p;
  int64_t stride;
  int pages;
};
bool table_of(const at::Tensor* t, int64_t B, int device, Table* out) {
  if (!t || t->scalar_type() != at::kInt || t->dim() != 2 || t->size(0) != B || !t->is_cuda() || t->get_device() != device)
    return false;
  const int64_t M = t->size(1);
  if (M > INT_MAX || (!t->is_contiguous() && M > 1 && t->stride(1) != 1)) return false;
  out->p = static_cast<const int32_t*>(t->data_ptr());
  out->pages = static_cast<int>(M);
  out->stride = t->is_contiguous() || B <= 1 ? M : t->stride(0);
  return out->stride == 0 || out->stride >= M;
}

bool cache_of(const at::Tensor* k, const at::Tensor* v, bool layered, int device, spec_cache_t* c) {
  if (!k || !v || k->scalar_type() != v->scalar_type() || !k->is_cuda() || !v->is_cuda() || k->get_device() != device ||
      v->get_device() != device)
    return false;
  if (k->scalar_type() == at::kBFloat16) c->dtype = SPEC_DTYPE_BF16;
  else if (k->scalar_type() == at::kFloat) c->dtype = SPEC_DTYPE_F32;
  else return false;
  const auto size = k->sizes(), stride = k->strides();
  const size_t dims = size.size();
  if ((dims != 4 && !(layered && dims == 5)) || size != v->sizes() || stride != v->strides()) return false;
  const size_t o = dims - 4;
  for (const int64_t n : size)
    if (n > INT_MAX) return false;
  const int64_t S = size[o + 1], H = size[o + 2], D = size[o + 3];
  if ((D > 1 && stride[o + 3] != 1) || (H > 1 && stride[o + 2] != D)) return false;
  c->k = k->data_ptr();
  c->v = v->data_ptr();
  c->layer_stride = o ? stride[0] : 0;
  c->page_stride = stride[o];
  c->token_stride = S > 1 ? stride[o + 1] : std::max<int64_t>(stride[o + 1], H * D);
  c->layers = o ? static_cast<int>(size[0]) : 1;
  c->pages = static_cast<int>(size[o]);
  c->page_size = static_cast<int>(S);
  c->heads = static_cast<int>(H);
  c->head_dim = static_cast<int>(D);
  return true;
}

// Tells autograd that a cache was changed in place.
void written(const at::Tensor* k, PyObject* v) {
  for (const at::Tensor* t : {k, tensor(v)})
    if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

at::Tensor make(at::IntArrayRef size, at::ScalarType type, int device) {
  return at::empty(size, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device))));
}

// Several 4-byte results in one allocation (one by one they took a third of a
// call's host time): tensors that share its storage.
class Results {
 public:
  Results(std::initializer_list<int64_t> sizes, int device) {
    int64_t total = 0;
    for (const int64_t n : sizes) total += rounded(n);
    buffer_ = make({total}, at::kInt, device);
  }
  // the next part, in the order of the sizes
  at::Tensor next(at::IntArrayRef size, at::ScalarType type) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(buffer_.storage()),
                                                     buffer_.key_set(), c10::scalarTypeToTypeMeta(type));
    impl->set_storage_offset(at_);
    impl->set_sizes_contiguous(size);
    at_ += rounded(c10::multiply_integers(size));
    return at::Tensor(std::move(impl));
  }

 private:
  static int64_t rounded(int64_t n) { return (n + 3) & ~static_cast<int64_t>(3); }
  at::Tensor buffer_;
  int64_t at_ = 0;
};

bool number(PyObject* o, float* f) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;
  const double d = PyFloat_AsDouble(o);
  if (d == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *f = static_cast<float>(d);
  return true;
}

bool whole(PyObject* o, int* i) {
  if (!PyLong_Check(o)) return false;
  int over = 0;
  const long n = PyLong_AsLongAndOverflow(o, &over);
  if (over || n < INT_MIN || n > INT_MAX) return false;
  *i = static_cast<int>(n);
  return true;
}

bool given(PyObject* o) { return o && o != Py_None; }

// Wraps tensors as a Python tuple's items; `type` (or a plain tuple) of them.
PyObject* result(PyObject* type, std::initializer_list<const at::Tensor*> tensors) {
  PyObject* items[8];
  size_t n = 0;
  for (const at::Tensor* t : tensors) {
    items[n] = t ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    if (!items[n++]) {
      while (n) Py_XDECREF(items[--n]);
      return nullptr;
    }
  }
  PyObject* r = PyObject_Vectorcall(type, items, n, nullptr);
  while (n) Py_DECREF(items[--n]);
  return r;
}

PyObject* call_attention(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
  static const char* const names[] = {"q", "k_pages", "v_pages", "page_table", "lengths", "scale", "return_lse"};
  PyObject* a[7];
  Where w;
  if (!arguments(args, n, kwnames, names, 6, 7, a)) return not_done();
  const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]);
  if (!q || !k || q->dim() != 4 || !where(*q, &w)) return not_done();
  spec_cache_t c;
  if (!cache_of(k, tensor(a[2]), false, w.device, &c) || q->scalar_type() != k->scalar_type()) return not_done();
  const int64_t B = q->size(0), Q = q->size(1), Hq = q->size(2), D = q->size(3);
  if (D != c.head_dim || c.heads < 1 || Hq % c.heads || (D > 1 && q->stride(3) != 1) || B > INT_MAX || Q > INT_MAX ||
      Hq > INT_MAX)
    return not_done();
  Table t;
  const int32_t* lengths;
  if (!table_of(tensor(a[3]), B, w.device, &t) || !ints(tensor(a[4]), B, w.device, &lengths)) return not_done();
  float scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  if (given(a[5]) && !number(a[5], &scale)) return not_done();
  if (a[6] && a[6] != Py_True && a[6] != Py_False) return not_done();
  const size_t need = attention_workspace_size(B, Q, Hq, c.heads, D, c.dtype);
  void* ws;
  size_t bytes;
  if (need == 0 || !workspace(0, w, need, &ws, &bytes)) return not_done();
  const at::Tensor out = make({B, Q, Hq, D}, q->scalar_type(), w.device);
  const bool with_lse = a[6] == Py_True;
  at::Tensor lse;
  if (with_lse) lse = make({B, Q, Hq}, at::kFloat, w.device);
  if (attention(q->data_ptr(), B > 1 ? q->stride(0) : 0, Q > 1 ? q->stride(1) : 0, Hq > 1 ? q->stride(2) : 0, &c, t.p, t.stride,
                t.pages, lengths, B, Q, Hq, scale, out.data_ptr(), with_lse ? lse.data_ptr<float>() : nullptr, ws, bytes,
                reinterpret_cast<spec_stream_t>(w.stream), nullptr) != SPEC_OK)
    return not_done();
  if (!with_lse) return THPVariable_Wrap(out);
  PyObject *x = THPVariable_Wrap(out), *y = THPVariable_Wrap(lse);
  PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

PyObject* call_append(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
  static const char* const names[] = {"k_new", "v_new", "k_pages", "v_pages", "page_table", "lengths", "starts"};
  PyObject* a[7];
  Where w;
  if (!arguments(args, n, kwnames, names, 7, 7, a)) return not_done();
  const at::Tensor *kn = tensor(a[0]), *vn = tensor(a[1]), *k = tensor(a[2]), *lens = tensor(a[5]);
  if (!kn || !vn || !k || !lens || lens->dim() != 1 || !where(*kn, &w)) return not_done();
  spec_cache_t c;
  if (!cache_of(k, tensor(a[3]), false, w.device, &c) || kn->scalar_type() != k->scalar_type() ||
      vn->scalar_type() != k->scalar_type() || !vn->is_cuda() || vn->get_device() != w.device || kn->sizes() != vn->sizes() ||
      kn->strides() != vn->strides())
    return not_done();
  const int64_t B = lens->size(0);
  const auto size = kn->sizes(), stride = kn->strides();
  const size_t dims = size.size();
  int64_t T, row;
  const int32_t *starts = nullptr, *lengths;
  if (given(a[6])) {
    if (dims != 3 || !ints(tensor(a[6]), B + 1, w.device, &starts)) return not_done();
    T = size[0];
    row = stride[0];
  } else {
    if (dims != 4 || size[0] != B || (B > 1 && size[1] > 1 && stride[0] != size[1] * stride[1])) return not_done();
    T = B * size[1];
    row = size[1] > 1 ? stride[1] : stride[0];
  }
  const int64_t H = size[dims - 2], D = size[dims - 1];
  if (H != c.heads || D != c.head_dim || T > INT_MAX || (D > 1 && stride[dims - 1] != 1) || (H > 1 && stride[dims - 2] != D))
    return not_done();
  Table t;
  if (!table_of(tensor(a[4]), B, w.device, &t) || !ints(lens, B, w.device, &lengths)) return not_done();
  if (append(kn->data_ptr(), vn->data_ptr(), T > 1 ? row : H * D, T, starts, &c, t.p, t.stride, t.pages, lengths, B,
             reinterpret_cast<spec_stream_t>(w.stream), nullptr) != SPEC_OK)
    return not_done();
  written(k, a[3]);
  Py_RETURN_NONE;
}

PyObject* call_fork(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
  static const char* const names[] = {"k_pages", "v_pages", "page_table", "lengths", "parents", "keep", "room"};
  PyObject* a[7];
  Where w;
  if (!arguments(args, n, kwnames, names, 7, 7, a)) return not_done();
  const at::Tensor *k = tensor(a[0]), *lens = tensor(a[3]), *par = tensor(a[4]);
  if (!k || !lens || !par || lens->dim() != 1 || par->dim() != 1 || !where(*k, &w)) return not_done();
  spec_cache_t c;
  Table t;
  const int32_t *lengths, *parents, *keep;
  const int64_t B = lens->size(0), C = par->size(0);
  int room = 0;
  if (!cache_of(k, tensor(a[1]), true, w.device, &c) || !table_of(tensor(a[2]), B, w.device, &t) ||
      !ints(lens, B, w.device, &lengths) || !ints(par, C, w.device, &parents) || !ints(tensor(a[5]), C, w.device, &keep) ||
      B > INT_MAX || C > INT_MAX || (a[6] && !whole(a[6], &room)))
    return not_done();
  void* ws;
  size_t bytes;
  if (!workspace(1, w, fork_workspace_size(c.pages, C), &ws, &bytes)) return not_done();
  Results r({C * t.pages, C, c.pages, c.pages, 1}, w.device);
  const at::Tensor table = r.next({C, t.pages}, at::kInt), lengths_new = r.next({C}, at::kInt),
                   refs = r.next({c.pages}, at::kInt), free = r.next({c.pages}, at::kInt), n_free = r.next({1}, at::kInt);
  if (fork_pages(&c, t.p, t.stride, t.pages, lengths, B, parents, keep, C, room, table.data_ptr<int>(),
                 lengths_new.data_ptr<int>(), refs.data_ptr<int>(), free.data_ptr<int>(), n_free.data_ptr<int>(), ws, bytes,
                 reinterpret_cast<spec_stream_t>(w.stream), nullptr) != SPEC_OK)
    return not_done();
  written(k, a[1]);
  return result(fork_result, {&table, &lengths_new, &refs, &free, &n_free, nullptr});
}

PyObject* call_compact(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
  static const char* const names[] = {"k_pages", "v_pages", "page_table"};
  PyObject* a[3];
  Where w;
  if (!arguments(args, n, kwnames, names, 3, 3, a)) return not_done();
  const at::Tensor *k = tensor(a[0]), *pt = tensor(a[2]);
  if (!k || !pt || pt->dim() != 2 || !where(*k, &w)) return not_done();
  spec_cache_t c;
  Table t;
  const int64_t B = pt->size(0);
  void* ws;
  size_t bytes;
  if (!cache_of(k, tensor(a[1]), true, w.device, &c) || B > INT_MAX || !table_of(pt, B, w.device, &t) ||
      !workspace(2, w, compact_workspace_size(c.pages), &ws, &bytes))
    return not_done();
  Results r({B * t.pages, c.pages, 1}, w.device);
  const at::Tensor table = r.next({B, t.pages}, at::kInt), refs = r.next({c.pages}, at::kInt), n_live = r.next({1}, at::kInt);
  if (compact(&c, t.p, t.stride, t.pages, B, table.data_ptr<int>(), refs.data_ptr<int>(), n_live.data_ptr<int>(), ws, bytes,
              reinterpret_cast<spec_stream_t>(w.stream), nullptr) != SPEC_OK)
    return not_done();
  written(k, a[1]);
  return result(compact_result, {&table, &refs, &n_live, nullptr});
}

// A sampling setting: absent, a number for every row, or one a row.
template <typename N>
bool setting(PyObject* o, at::ScalarType type, int64_t R, int device, bool (*scalar)(PyObject*, N*), N* value, const N** p) {
  *p = nullptr;
  if (!given(o)) return true;
  const at::Tensor* t = tensor(o);
  if (!t) return scalar(o, value);
  if (t->scalar_type() != type || t->numel() != R || !t->is_cuda() || t->get_device() != device || !t->is_contiguous())
    return false;
  *p = static_cast<const N*>(t->data_ptr());
  return true;
}

PyObject* call_sample(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
  static const char* const names[] = {"logits", "uniforms", "temperature", "top_k", "top_p", "min_p", "return_filtered"};
  PyObject* a[7];
  Where w;
  if (!arguments(args, n, kwnames, names, 3, 7, a)) return not_done();
  const at::Tensor *x = tensor(a[0]), *u = tensor(a[1]);
  if (!x || !u || x->dim() < 1 || !where(*x, &w)) return not_done();
  int dtype;
  if (x->scalar_type() == at::kBFloat16) dtype = SPEC_DTYPE_BF16;
  else if (x->scalar_type() == at::kFloat) dtype = SPEC_DTYPE_F32;
  else return not_done();
  const int64_t V = x->size(-1);
  if (V < 1 || V > (1 << 22)) return not_done();
  const at::IntArrayRef rows = x->sizes().slice(0, x->dim() - 1);
  const int64_t R = x->numel() / V;
  int64_t stride = V;
  if (!x->is_contiguous()) {
    if (x->dim() != 2 || x->stride(1) != 1 || x->stride(0) < V) return not_done();
    stride = x->stride(0);
  }
  if (R > INT_MAX || u->scalar_type() != at::kFloat || u->sizes() != rows || !u->is_cuda() || u->get_device() != w.device ||
      !u->is_contiguous())
    return not_done();
  float T = 1.f, top_p = 1.f, min_p = 0.f;
  int top_k = 0;
  const float *Ts, *ps, *ms;
  const int* ks;
  if (!setting<float>(a[2], at::kFloat, R, w.device, number, &T, &Ts) ||
      !setting<int>(a[3], at::kInt, R, w.device, whole, &top_k, &ks) ||
      !setting<float>(a[4], at::kFloat, R, w.device, number, &top_p, &ps) ||
      !setting<float>(a[5], at::kFloat, R, w.device, number, &min_p, &ms) ||
      (a[6] && a[6] != Py_True && a[6] != Py_False))
    return not_done();
  void* ws;
  size_t bytes;
  if (!workspace(3, w, sample_workspace_size(R, V, dtype), &ws, &bytes)) return not_done();
  const bool filtered = a[6] == Py_True;
  Results r({R, R, R}, w.device);
  const at::Tensor tokens = r.next(rows, at::kInt), p = r.next(rows, at::kFloat), n_kept = r.next(rows, at::kInt);
  at::Tensor out;
  if (filtered) out = make(x->sizes(), x->scalar_type(), w.device);
  if (sample(x->data_ptr(), stride, u->data_ptr<float>(), R, V, dtype, T, top_k, top_p, min_p, Ts, ks, ps, ms,
             tokens.data_ptr<int>(), p.data_ptr<float>(), n_kept.data_ptr<int>(), filtered ? out.data_ptr() : nullptr, ws, bytes,
             reinterpret_cast<spec_stream_t>(w.stream), nullptr) != SPEC_OK)
    return not_done();
  return result(sample_result, {&tokens, &p, &n_kept, filtered ? &out : nullptr, nullptr});
}

// A tree's parents: a row a sequence, or one for all.
bool parents_of(const at::Tensor* t, int64_t B, int64_t N, int device, const int32_t** p, int64_t* stride) {
  if (!t || t->scalar_type() != at::kInt || !t->is_cuda() || t->get_device() != device) return false;
  const int64_t dims = t->dim();
  if (dims < 1 || dims > 2 || t->size(dims - 1) != N || (dims == 2 && t->size(0) != B) || (N > 1 && t->stride(dims - 1) != 1))
    return false;
  *p = static_cast<const int32_t*>(t->data_ptr());
  *stride = dims == 1 ? 0 : B > 1 ? t->stride(0) : N;
  return *stride == 0 || *stride >= N;
}

PyObject* call_tree_attention(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
  static const char* const names[] = {"q", "k_pages", "v_pages", "page_table", "lengths", "parents", "scale", "return_lse"};
  PyObject* a[8];
  Where w;
  if (!arguments(args, n, kwnames, names, 7, 8, a)) return not_done();
  const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]);
  if (!q || !k || q->dim() != 4 || !where(*q, &w)) return not_done();
  spec_cache_t c;
  if (!cache_of(k, tensor(a[2]), false, w.device, &c) || q->scalar_type() != k->scalar_type()) return not_done();
  const int64_t B = q->size(0), N = q->size(1), Hq = q->size(2), D = q->size(3);
  if (D != c.head_dim || c.heads < 1 || Hq % c.heads || (D > 1 && q->stride(3) != 1) || B > INT_MAX ||
      N > SPEC_TREE_MAX_NODES || Hq > INT_MAX)
    return not_done();
  Table t;
  const int32_t *lengths, *parents;
  int64_t parents_stride;
  if (!table_of(tensor(a[3]), B, w.device, &t) || !ints(tensor(a[4]), B, w.device, &lengths) ||
      !parents_of(tensor(a[5]), B, N, w.device, &parents, &parents_stride))
    return not_done();
  float scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  if (given(a[6]) && !number(a[6], &scale)) return not_done();
  if (a[7] && a[7] != Py_True && a[7] != Py_False) return not_done();
  const size_t need = tree_workspace_size(B, N, Hq, c.heads, D, c.dtype);
  void* ws;
  size_t bytes;
  if (need == 0 || !workspace(4, w, need, &ws, &bytes)) return not_done();
  const at::Tensor out = make({B, N, Hq, D}, q->scalar_type(), w.device);
  const bool with_lse = a[7] == Py_True;
  at::Tensor lse;
  if (with_lse) lse = make({B, N, Hq}, at::kFloat, w.device);
  if (tree_attention(q->data_ptr(), B > 1 ? q->stride(0) : 0, N > 1 ? q->stride(1) : 0, Hq > 1 ? q->stride(2) : 0, &c, t.p,
                     t.stride, t.pages, lengths, parents, parents_stride, B, N, Hq, scale, out.data_ptr(),
                     with_lse ? lse.data_ptr<float>() : nullptr, ws, bytes, reinterpret_cast<spec_stream_t>(w.stream),
                     nullptr) != SPEC_OK)
    return not_done();
  if (!with_lse) return THPVariable_Wrap(out);
  PyObject *x = THPVariable_Wrap(out), *y = THPVariable_Wrap(lse);
  PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// New tokens' rows [lead..., heads, D] at one stride, heads contiguous.
bool rows_of(const at::Tensor& t, at::IntArrayRef lead, int64_t heads, int64_t D, int64_t T, int64_t* row) {
  const auto size = t.sizes(), stride = t.strides();
  const size_t m = lead.size();
  if (size.size() != m + 2 || size.slice(0, m) != lead || size[m] != heads || size[m + 1] != D) return false;
  if ((D > 1 && stride[m + 1] != 1) || (heads > 1 && stride[m] != D)) return false;
  if (T <= 1) *row = heads * D;
  else if (m == 1) *row = stride[0];
  else if (lead[0] > 1 && lead[1] > 1 && stride[0] != lead[1] * stride[1]) return false;
  else *row = lead[1] > 1 ? stride[1] : stride[0];
  return true;
}

PyObject* call_append_rotated(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
  static const char* const names[] = {"k_new", "v_new", "k_pages", "v_pages", "page_table", "lengths", "inv_freq", "q",
                                      "positions", "starts", "interleaved"};
  PyObject* a[11];
  Where w;
  if (!arguments(args, n, kwnames, names, 10, 11, a)) return not_done();
  const at::Tensor *kn = tensor(a[0]), *vn = tensor(a[1]), *k = tensor(a[2]), *lens = tensor(a[5]), *freq = tensor(a[6]);
  if (!kn || !vn || !k || !lens || !freq || lens->dim() != 1 || !where(*kn, &w)) return not_done();
  spec_cache_t c;
  if (!cache_of(k, tensor(a[3]), false, w.device, &c) || kn->scalar_type() != k->scalar_type() ||
      vn->scalar_type() != k->scalar_type() || !vn->is_cuda() || vn->get_device() != w.device || kn->sizes() != vn->sizes() ||
      kn->strides() != vn->strides())
    return not_done();
  const int64_t B = lens->size(0);
  const bool flat = given(a[9]);
  if (kn->dim() != (flat ? 3 : 4) || (!flat && kn->size(0) != B)) return not_done();
  const at::IntArrayRef lead = kn->sizes().slice(0, flat ? 1 : 2);
  const int64_t T = flat ? lead[0] : lead[0] * lead[1];
  int64_t row, q_row = 0, Hq = 0;
  const int32_t *starts = nullptr, *lengths, *positions = nullptr;
  if (B > INT_MAX || T > INT_MAX || !rows_of(*kn, lead, c.heads, c.head_dim, T, &row)) return not_done();
  if (flat && !ints(tensor(a[9]), B + 1, w.device, &starts)) return not_done();
  if (freq->scalar_type() != at::kFloat || freq->dim() != 1 || !freq->is_cuda() || freq->get_device() != w.device ||
      !freq->is_contiguous() || freq->size(0) > 1024)
    return not_done();
  if (given(a[8])) {
    const at::Tensor* p = tensor(a[8]);
    if (!p || p->scalar_type() != at::kInt || p->sizes() != lead || !p->is_cuda() || p->get_device() != w.device ||
        !p->is_contiguous())
      return not_done();
    positions = static_cast<const int32_t*>(p->data_ptr());
  }
  const at::Tensor* q = nullptr;
  if (given(a[7])) {
    q = tensor(a[7]);
    if (!q || q->scalar_type() != k->scalar_type() || q->dim() != kn->dim() || !q->is_cuda() || q->get_device() != w.device)
      return not_done();
    Hq = q->size(-2);
    if (Hq > INT_MAX || !rows_of(*q, lead, Hq, c.head_dim, T, &q_row)) return not_done();
  }
  if (a[10] && a[10] != Py_True && a[10] != Py_False) return not_done();
  Table t;
  if (!table_of(tensor(a[4]), B, w.device, &t) || !ints(lens, B, w.device, &lengths)) return not_done();
  at::Tensor out;
  if (q) out = make(q->sizes(), q->scalar_type(), w.device);
  if (append_rotated(kn->data_ptr(), vn->data_ptr(), row, T, starts, q ? q->data_ptr() : nullptr, q_row, Hq,
                     q ? out.data_ptr() : nullptr, Hq * c.head_dim, positions, freq->data_ptr<float>(), freq->size(0),
                     a[10] == Py_True, &c, t.p, t.stride, t.pages, lengths, B, reinterpret_cast<spec_stream_t>(w.stream),
                     nullptr) != SPEC_OK)
    return not_done();
  written(k, a[3]);
  if (!q) Py_RETURN_NONE;
  return THPVariable_Wrap(out);
}

// A contiguous int32 [B, N].
bool ints2(const at::Tensor* t, int64_t B, int64_t N, int device, const int32_t** p) {
  if (!t || t->scalar_type() != at::kInt || t->dim() != 2 || t->size(0) != B || t->size(1) != N || !t->is_cuda() ||
      t->get_device() != device || !t->is_contiguous())
    return false;
  *p = static_cast<const int32_t*>(t->data_ptr());
  return true;
}

PyObject* call_accept(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
  static const char* const names[] = {"tokens", "parents", "drawn"};
  PyObject* a[3];
  Where w;
  if (!arguments(args, n, kwnames, names, 3, 3, a)) return not_done();
  const at::Tensor* x = tensor(a[0]);
  if (!x || x->dim() != 2 || !where(*x, &w)) return not_done();
  const int64_t B = x->size(0), N = x->size(1);
  const int32_t *tokens, *parents, *drawn;
  int64_t parents_stride;
  if (B > INT_MAX || N > SPEC_TREE_MAX_NODES || !ints2(x, B, N, w.device, &tokens) ||
      !parents_of(tensor(a[1]), B, N, w.device, &parents, &parents_stride) || !ints2(tensor(a[2]), B, N, w.device, &drawn))
    return not_done();
  Results r({B, B * N, B * N}, w.device);
  const at::Tensor len = r.next({B}, at::kInt), out = r.next({B, N}, at::kInt), path = r.next({B, N}, at::kInt);
  if (tree_accept(tokens, parents, parents_stride, drawn, B, N, len.data_ptr<int>(), out.data_ptr<int>(), path.data_ptr<int>(),
                  reinterpret_cast<spec_stream_t>(w.stream), nullptr) != SPEC_OK)
    return not_done();
  // (the result type is a tuple without more, and made as one: its own constructor runs Python)
  PyTypeObject* type = reinterpret_cast<PyTypeObject*>(accept_result);
  PyObject* result = type->tp_alloc(type, 4);
  if (!result) return nullptr;
  const at::Tensor* items[] = {&len, &out, &path};
  for (int i = 0; i < 4; ++i) {
    PyObject* item = i < 3 ? THPVariable_Wrap(*items[i]) : Py_NewRef(Py_None);
    if (!item) {
      Py_DECREF(result);
      return nullptr;
    }
    PyTuple_SET_ITEM(result, i, item);
  }
  return result;
}

PyObject* call_keep(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
  static const char* const names[] = {"k_pages", "v_pages", "page_table", "lengths", "path"};
  PyObject* a[5];
  Where w;
  if (!arguments(args, n, kwnames, names, 5, 5, a)) return not_done();
  const at::Tensor *k = tensor(a[0]), *lens = tensor(a[3]), *p = tensor(a[4]);
  if (!k || !lens || !p || lens->dim() != 1 || p->dim() != 2 || !where(*k, &w)) return not_done();
  spec_cache_t c;
  Table t;
  const int32_t *lengths, *path;
  const int64_t B = lens->size(0), N = p->size(1);
  if (B > INT_MAX || N > INT_MAX || !cache_of(k, tensor(a[1]), true, w.device, &c) ||
      !table_of(tensor(a[2]), B, w.device, &t) || !ints(lens, B, w.device, &lengths) || !ints2(p, B, N, w.device, &path))
    return not_done();
  const at::Tensor out = make({B}, at::kInt, w.device);
  if (cache_keep(&c, t.p, t.stride, t.pages, lengths, B, path, N, out.data_ptr<int>(),
                 reinterpret_cast<spec_stream_t>(w.stream), nullptr) != SPEC_OK)
    return not_done();
  written(k, a[1]);
  return THPVariable_Wrap(out);
}

// C++ exceptions (an allocation that fails, say) are decode.py's to meet again
// and report.
template <PyObject* (*kCall)(PyObject*, PyObject* const*, Py_ssize_t, PyObject*)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
  try {
    return kCall(self, args, n, kwnames);
  } catch (...) {
    PyErr_Clear();
    return not_done();
  }
}

// The library's entry points by address, in this order, and the result types.
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[9];
  PyObject* r[3];
  if (!PyArg_ParseTuple(args, "(KKKKKKKKK)OOO", f, f + 1, f + 2, f + 3, f + 4, f + 5, f + 6, f + 7, f + 8, r, r + 1, r + 2))
    return nullptr;
  int i = 0;
  auto take = [&](auto& fn) { fn = reinterpret_cast<std::decay_t<decltype(fn)>>(f[i++]); };
  take(attention_workspace_size);
  take(attention);
  take(append);
  take(fork_workspace_size);
  take(fork_pages);
  take(compact_workspace_size);
  take(compact);
  take(sample_workspace_size);
  take(sample);
  fork_result = Py_NewRef(r[0]);
  compact_result = Py_NewRef(r[1]);
  sample_result = Py_NewRef(r[2]);
  Py_RETURN_NONE;
}

PyObject* bind_tree(PyObject*, PyObject* args) {
  unsigned long long f[5];
  PyObject* r;
  if (!PyArg_ParseTuple(args, "(KKKKK)O", f, f + 1, f + 2, f + 3, f + 4, &r)) return nullptr;
  int i = 0;
  auto take = [&](auto& fn) { fn = reinterpret_cast<std::decay_t<decltype(fn)>>(f[i++]); };
  take(tree_workspace_size);
  take(tree_attention);
  take(append_rotated);
  take(tree_accept);
  take(cache_keep);
  accept_result = Py_NewRef(r);
  Py_RETURN_NONE;
}

PyObject* register_workspace(PyObject*, PyObject* args) {
  Workspace w;
  unsigned long long p, bytes;
  if (!PyArg_ParseTuple(args, "llKKK", &w.kind, &w.device, &w.stream, &p, &bytes)) return nullptr;
  w.p = reinterpret_cast<void*>(p);
  w.bytes = bytes;
  for (Workspace& x : workspaces)
    if (x.kind == w.kind && x.device == w.device && x.stream == w.stream) {
      x = w;
      Py_RETURN_NONE;
    }
  workspaces.push_back(w);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         {"bind_tree", bind_tree, METH_VARARGS, nullptr},
                         {"register_workspace", register_workspace, METH_VARARGS, nullptr},
                         {"paged_attention", nullptr, 0, nullptr},
                         {"cache_append", nullptr, 0, nullptr},
                         {"cache_fork", nullptr, 0, nullptr},
                         {"cache_compact", nullptr, 0, nullptr},
                         {"filtered_sample", nullptr, 0, nullptr},
                         {"tree_attention", nullptr, 0, nullptr},
                         {"cache_append_rotated", nullptr, 0, nullptr},
                         {"tree_accept", nullptr, 0, nullptr},
                         {"cache_keep", nullptr, 0, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__decode_calls() {
  auto as = [](PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t, PyObject*)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
  };
  PyObject* (*calls[])(PyObject*, PyObject* const*, Py_ssize_t, PyObject*) = {
      guarded<call_attention>, guarded<call_append>, guarded<call_fork>, guarded<call_compact>, guarded<call_sample>,
      guarded<call_tree_attention>, guarded<call_append_rotated>, guarded<call_accept>, guarded<call_keep>};
  constexpr int kFirst = 3;  // in `methods`
  for (int i = 0; i < 9; ++i) {
    methods[kFirst + i].ml_meth = as(calls[i]);
    methods[kFirst + i].ml_flags = METH_FASTCALL | METH_KEYWORDS;
  }
  return PyModule_Create(&module);
}
