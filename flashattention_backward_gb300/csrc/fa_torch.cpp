// PyTorch binding of the paged-cache calls of include/fa.h: checks of the
// tensors, their addresses and strides, and the results' allocation.  Written
// against PyTorch's C++ interface because these calls are short: the kernels of
// a decoding step take a few microseconds, and the same checks and allocations
// from Python took 10 to 25 of the calling thread's: attention_decode at the
// smallest size 19 us a call against 5.5 from here, one row appended to each of
// 64 sequences 13 against 5.7.
//
// The library itself (libfa.so) knows nothing of PyTorch: paged.py hands its
// entry points over with bind().

#include <Python.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <optional>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fa.h"

namespace {

using at::Tensor;

struct Entries {
  decltype(&fa_decode_workspace_bytes) workspace_bytes;
  decltype(&fa_decode) decode;
  decltype(&fa_cache_append) append;
  decltype(&fa_cache_copy_pages) copy;
  decltype(&fa_pages_extend) extend;
  decltype(&fa_pages_fork) fork;
  decltype(&fa_pages_free) free;
  decltype(&fa_pages_compact) compact;
} g_fa;
PyObject* g_error = nullptr;  // FaError(code, what)

// A failed call, on its way to Python.
struct Failed {
  fa_status code;
  const char* what;
};

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

// No call here has a gradient, so none may be asked for one.
void no_gradient(const char* call, const Tensor& t) {
  TORCH_CHECK_VALUE(!(t.requires_grad() && at::GradMode::is_enabled()), call,
                    " has no gradient: call it under torch.no_grad()");
}

// The stream to launch on, after checking that `device` is the current one.
// given: an address as a Python int, or None for the current stream.
struct Stream {
  void* raw;
  bool given;
  at::Device device;
  Stream(const at::Device& d, PyObject* o) : given(o != Py_None), device(d) {
    const auto current = c10::cuda::current_device();
    TORCH_CHECK_VALUE(d.index() == current, "the tensors are on ", d, ", the current device is cuda:", (int)current);
    if (given) {
      raw = PyLong_AsVoidPtr(o);
      if (PyErr_Occurred()) throw python_error();
    } else {
      raw = c10::cuda::getCurrentCUDAStream(current).stream();
    }
  }
  c10::cuda::CUDAStream stream() const {
    return c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(raw), device.index());
  }
  // A tensor of the caller's, used on a stream that it gave: its memory may not
  // be handed out again before that stream is done with it.
  void lend(const Tensor& t) const {
    if (given) record(t, stream());
  }
  // A new tensor.  The allocator hands out memory that was freed while work of
  // the stream it was freed on was still using it, for that stream alone: so it
  // is asked for memory of the stream that the call runs on.
  Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    const c10::cuda::OptionalCUDAStreamGuard guard(given ? std::optional<c10::Stream>(stream().unwrap()) : std::nullopt);
    return at::empty(shape, at::TensorOptions().dtype(type).device(device));
  }
  // A new tensor for the caller, who may use it on the current stream and then
  // let it go.
  Tensor result(at::IntArrayRef shape, at::ScalarType type) const {
    Tensor t = empty(shape, type);
    if (given) record(t, c10::cuda::getCurrentCUDAStream(device.index()));
    return t;
  }

 private:
  static void record(const Tensor& t, const c10::cuda::CUDAStream& s) {
    if (t.defined() && t.numel() > 0) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), s);
  }
};

// The first three strides of a 4-D tensor with contiguous rows; the stride of
// a dimension of one element, which PyTorch leaves open, is set to a packed one.
struct RowStrides {
  int64_t s0, s1, s2;
  explicit RowStrides(const Tensor& t) {
    const auto n = t.sizes();
    const auto s = t.strides();
    TORCH_CHECK_VALUE(s[3] == 1, "the last dimension must be contiguous");
    const int64_t d = n[3];
    s2 = n[2] == 1 ? d : s[2];
    s1 = n[1] == 1 ? (s2 >= d ? n[2] * s2 : d) : s[1];
    s0 = n[0] == 1 ? std::max({n[1] * s1, n[2] * s2, d}) : s[0];
  }
  bool operator==(const RowStrides& o) const { return s0 == o.s0 && s1 == o.s1 && s2 == o.s2; }
};

int32_t as_int32(int64_t n, const char* what) {
  TORCH_CHECK_VALUE(n >= 0 && n <= INT32_MAX, what, " is out of range");
  return (int32_t)n;
}

const int32_t* set_table(fa_cache* c, const Tensor& t, const at::Device& device) {
  TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.dim() == 2 && t.device() == device,
                    "page_table must be a 2-D int32 tensor on ", device);
  c->S = as_int32(t.size(0), "the number of sequences");
  c->max_pages = as_int32(t.size(1), "the number of columns");
  TORCH_CHECK_VALUE(t.stride(1) == 1 || c->max_pages <= 1, "the rows of page_table must be contiguous");
  c->table_stride = c->S > 1 ? t.stride(0) : c->max_pages;
  return static_cast<const int32_t*>(t.data_ptr());
}

// Two pools and, unless it is None, the table over them.
struct Cache {
  fa_cache c{};
  at::Device device;
  const int32_t* table = nullptr;
  void *k, *v;
  at::ScalarType type;
  Cache(PyObject* k_pages, PyObject* v_pages, PyObject* page_table) : device(at::kCPU) {
    const Tensor &kt = tensor(k_pages, "k_pages"), &vt = tensor(v_pages, "v_pages");
    TORCH_CHECK_VALUE(kt.dim() == 4 && vt.sizes() == kt.sizes(),
                      "k_pages and v_pages must be [pages, kv_heads, page_rows, d] tensors of one shape");
    type = kt.scalar_type();
    TORCH_CHECK_TYPE(type == at::kBFloat16 || type == at::kFloat, "unsupported dtype ", type);
    TORCH_CHECK_VALUE(vt.scalar_type() == type, "k_pages and v_pages must share the dtype");
    device = kt.device();
    TORCH_CHECK_VALUE(device.is_cuda() && vt.device() == device, "the pools must be on one CUDA device");
    const RowStrides s(kt);
    TORCH_CHECK_VALUE(s == RowStrides(vt), "k_pages and v_pages must share their strides");
    c.num_pages = as_int32(kt.size(0), "the number of pages");
    c.H_kv = as_int32(kt.size(1), "the number of heads");
    c.page_rows = as_int32(kt.size(2), "page_rows");
    c.d = as_int32(kt.size(3), "d");
    c.dtype = type == at::kBFloat16 ? FA_BF16 : FA_FP32;
    c.S = c.max_pages = 1;
    c.stride_page = s.s0, c.stride_h = s.s1, c.stride_n = s.s2;
    c.table_stride = 1;
    k = kt.data_ptr();
    v = vt.data_ptr();
    if (page_table != Py_None) table = set_table(&c, tensor(page_table, "page_table"), device);
  }
};

// A table, lengths and references, for the page calls.
struct Pages {
  fa_cache c{};
  at::Device device;
  int32_t *table, *lengths, *refs;
  Pages(PyObject* page_table, PyObject* len, PyObject* ref, PyObject* page_rows);
};

// Address of a dense int32 tensor of that shape on that device.
int32_t* ints(PyObject* o, const char* name, at::IntArrayRef shape, const at::Device& device) {
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.sizes() == shape && t.device() == device && t.is_contiguous(), name,
                    " must be a contiguous int32 tensor of shape ", shape, " on ", device);
  return static_cast<int32_t*>(t.data_ptr());
}

Pages::Pages(PyObject* page_table, PyObject* len, PyObject* ref, PyObject* page_rows) : device(at::kCPU) {
  const Tensor& r = tensor(ref, "refs");
  TORCH_CHECK_VALUE(r.dim() == 1 && r.is_cuda(), "refs must be a 1-D CUDA tensor");
  device = r.device();
  const long rows = PyLong_AsLong(page_rows);
  if (rows == -1 && PyErr_Occurred()) throw python_error();
  c.num_pages = as_int32(r.size(0), "the number of pages");
  c.page_rows = rows < 0 || rows > INT32_MAX ? 0 : (int32_t)rows;  // 0 is refused by the library
  c.H_kv = 1;
  table = const_cast<int32_t*>(set_table(&c, tensor(page_table, "page_table"), device));
  lengths = ints(len, "lengths", {c.S}, device);
  refs = ints(ref, "refs", {c.num_pages}, device);
}

// The library's call, without the interpreter's lock: a full launch queue
// makes it wait.
template <class F, class... A>
void call(const char* what, F f, A... args) {
  fa_status code;
  Py_BEGIN_ALLOW_THREADS;
  code = f(args...);
  Py_END_ALLOW_THREADS;
  if (code != FA_OK) throw Failed{code, what};
}

void want(Py_ssize_t given, Py_ssize_t n) { TORCH_CHECK_TYPE(given == n, "expected ", n, " arguments, got ", given); }

// Python's view of a function of (arguments, count): exceptions become errors.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* python(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Failed& f) {
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)f.code, f.what);
    if (e) PyErr_SetObject(g_error, e);
    Py_XDECREF(e);
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* r = PyTuple_New(2);
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(b));
  return r;
}

// q, k_pages, v_pages, page_table, lengths, scale, workspace, out, stream
PyObject* decode(PyObject* const* a, Py_ssize_t n) {
  want(n, 9);
  const Tensor& q = tensor(a[0], "q");
  no_gradient("attention_decode", q);
  no_gradient("attention_decode", tensor(a[1], "k_pages"));
  no_gradient("attention_decode", tensor(a[2], "v_pages"));
  Cache cache(a[1], a[2], a[3]);
  const fa_cache& c = cache.c;
  TORCH_CHECK_VALUE(q.dim() == 4 && q.size(0) == c.S && q.size(2) == 1 && q.size(3) == c.d, "q must be a [", c.S,
                    ", heads, 1, ", c.d, "] tensor");
  TORCH_CHECK_VALUE(q.scalar_type() == cache.type && q.device() == cache.device,
                    "q must have the dtype and device of the pools");
  const Stream stream(cache.device, a[8]);
  const int32_t* lengths = ints(a[4], "lengths", {c.S}, cache.device);
  const int32_t heads = as_int32(q.size(1), "the number of heads");
  double scale = 1.0 / std::sqrt((double)c.d);
  if (a[5] != Py_None) {
    scale = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) throw python_error();
  }
  const RowStrides qs(q);
  Tensor o, L, workspace;
  if (a[7] == Py_None) {
    o = stream.result(q.sizes(), cache.type);
    L = stream.result(q.sizes().slice(0, 3), at::kFloat);
  } else {
    TORCH_CHECK_TYPE(PyTuple_Check(a[7]) && PyTuple_GET_SIZE(a[7]) == 2, "out must be a tuple (o, L)");
    o = tensor(PyTuple_GET_ITEM(a[7], 0), "out[0]");
    L = tensor(PyTuple_GET_ITEM(a[7], 1), "out[1]");
    no_gradient("attention_decode", o);
    no_gradient("attention_decode", L);
    TORCH_CHECK_VALUE(o.sizes() == q.sizes() && o.scalar_type() == cache.type && o.device() == cache.device,
                      "out[0] must have the shape, dtype and device of q");
    TORCH_CHECK_VALUE(L.sizes() == q.sizes().slice(0, 3) && L.scalar_type() == at::kFloat &&
                          L.device() == cache.device && L.is_contiguous(),
                      "out[1] must be a contiguous float32 tensor of shape ", q.sizes().slice(0, 3));
    stream.lend(o);
    stream.lend(L);
  }
  size_t bytes = g_fa.workspace_bytes(&c, heads);
  if (a[6] != Py_None) {
    workspace = tensor(a[6], "workspace");
    TORCH_CHECK_VALUE(workspace.device() == cache.device && workspace.is_contiguous(),
                      "workspace must be a contiguous tensor on ", cache.device);
    bytes = workspace.nbytes();
    stream.lend(workspace);
  } else if (bytes > 0) {
    workspace = stream.empty({(int64_t)bytes}, at::kByte);
  }
  const RowStrides os(o);
  call("fa_decode", g_fa.decode, &c, heads, (float)scale, (const void*)q.data_ptr(), qs.s0, qs.s1,
       (const void*)cache.k, (const void*)cache.v, cache.table, lengths, o.data_ptr(), os.s0, os.s1,
       static_cast<float*>(L.data_ptr()), workspace.defined() ? workspace.data_ptr() : nullptr, bytes, stream.raw);
  return pair(o, L);
}

// k, v, k_pages, v_pages, page_table, start, counts, stream
PyObject* append(PyObject* const* a, Py_ssize_t n) {
  want(n, 8);
  const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  no_gradient("cache_append", k);
  no_gradient("cache_append", v);
  no_gradient("cache_append", tensor(a[2], "k_pages"));
  no_gradient("cache_append", tensor(a[3], "v_pages"));
  Cache cache(a[2], a[3], a[4]);
  const fa_cache& c = cache.c;
  TORCH_CHECK_VALUE(k.dim() == 4 && k.size(0) == c.S && k.size(1) == c.H_kv && k.size(3) == c.d && v.sizes() == k.sizes(),
                    "k and v must be [", c.S, ", ", c.H_kv, ", rows, ", c.d, "] tensors");
  TORCH_CHECK_VALUE(k.scalar_type() == cache.type && v.scalar_type() == cache.type && k.device() == cache.device &&
                        v.device() == cache.device,
                    "k and v must have the dtype and device of the pools");
  const Stream stream(cache.device, a[7]);
  const int32_t* start = ints(a[5], "start", {c.S}, cache.device);
  const int32_t* counts = a[6] == Py_None ? nullptr : ints(a[6], "counts", {c.S}, cache.device);
  if (k.size(2) == 0) Py_RETURN_NONE;
  const RowStrides s(k);
  TORCH_CHECK_VALUE(s == RowStrides(v), "k and v must share their strides");
  call("fa_cache_append", g_fa.append, &c, as_int32(k.size(2), "the number of rows"), (const void*)k.data_ptr(),
       (const void*)v.data_ptr(), s.s0, s.s1, s.s2, cache.k, cache.v, cache.table, start, counts, stream.raw);
  Py_RETURN_NONE;
}

// k_pages, v_pages, moves, count, stream
PyObject* copy(PyObject* const* a, Py_ssize_t n) {
  want(n, 5);
  no_gradient("cache_copy_pages", tensor(a[0], "k_pages"));
  no_gradient("cache_copy_pages", tensor(a[1], "v_pages"));
  Cache cache(a[0], a[1], Py_None);
  const Tensor& moves = tensor(a[2], "moves");
  TORCH_CHECK_VALUE(moves.dim() == 2, "moves must be an [n, 3] tensor");
  const Stream stream(cache.device, a[4]);
  const int32_t* m = ints(a[2], "moves", {moves.size(0), 3}, cache.device);
  const int32_t* count = a[3] == Py_None ? nullptr : ints(a[3], "count", {1}, cache.device);
  call("fa_cache_copy_pages", g_fa.copy, &cache.c, as_int32(moves.size(0), "the number of moves"), m, count, cache.k,
       cache.v, stream.raw);
  Py_RETURN_NONE;
}

// page_table, lengths, refs, n_new, page_rows, stream
PyObject* extend(PyObject* const* a, Py_ssize_t n) {
  want(n, 6);
  Pages p(a[0], a[1], a[2], a[4]);
  const Stream stream(p.device, a[5]);
  const int32_t* n_new = ints(a[3], "n_new", {p.c.S}, p.device);
  Tensor start = stream.result({p.c.S}, at::kInt);
  call("fa_pages_extend", g_fa.extend, &p.c, p.table, p.lengths, p.refs, n_new, static_cast<int32_t*>(start.data_ptr()),
       stream.raw);
  return THPVariable_Wrap(start);
}

// page_table, lengths, refs, src, dst, page_rows, stream
PyObject* fork(PyObject* const* a, Py_ssize_t n) {
  want(n, 7);
  Pages p(a[0], a[1], a[2], a[5]);
  const Stream stream(p.device, a[6]);
  const Tensor& list = tensor(a[3], "src");
  TORCH_CHECK_VALUE(list.dim() == 1, "src must be a 1-D tensor");
  const int64_t pairs = list.size(0);
  const int32_t *src = ints(a[3], "src", {pairs}, p.device), *dst = ints(a[4], "dst", {pairs}, p.device);
  Tensor moves = stream.result({pairs, 3}, at::kInt);
  if (pairs > 0)
    call("fa_pages_fork", g_fa.fork, &p.c, as_int32(pairs, "the number of pairs"), src, dst, p.table, p.lengths, p.refs,
         static_cast<int32_t*>(moves.data_ptr()), stream.raw);
  return THPVariable_Wrap(moves);
}

// page_table, lengths, refs, sequences, page_rows, stream
PyObject* release(PyObject* const* a, Py_ssize_t n) {
  want(n, 6);
  Pages p(a[0], a[1], a[2], a[4]);
  const Stream stream(p.device, a[5]);
  const Tensor& list = tensor(a[3], "sequences");
  TORCH_CHECK_VALUE(list.dim() == 1, "sequences must be a 1-D tensor");
  const int32_t* sequences = ints(a[3], "sequences", {list.size(0)}, p.device);
  call("fa_pages_free", g_fa.free, &p.c, as_int32(list.size(0), "the number of sequences"), sequences, p.table,
       p.lengths, p.refs, stream.raw);
  Py_RETURN_NONE;
}

// page_table, lengths, refs, page_rows, out, stream
PyObject* compact(PyObject* const* a, Py_ssize_t n) {
  want(n, 6);
  Pages p(a[0], a[1], a[2], a[3]);
  const Stream stream(p.device, a[5]);
  int32_t *table_out = p.table, *refs_out = p.refs;
  if (a[4] != Py_None) {
    TORCH_CHECK_TYPE(PyTuple_Check(a[4]) && PyTuple_GET_SIZE(a[4]) == 2, "out must be a tuple (page_table, refs)");
    const Tensor &t = tensor(PyTuple_GET_ITEM(a[4], 0), "out[0]"), &old = tensor(a[0], "page_table");
    TORCH_CHECK_VALUE(t.sizes() == old.sizes() && t.strides() == old.strides() && t.scalar_type() == at::kInt &&
                          t.device() == p.device,
                      "out[0] must have the shape, strides, dtype and device of page_table");
    table_out = static_cast<int32_t*>(t.data_ptr());
    refs_out = ints(PyTuple_GET_ITEM(a[4], 1), "out[1]", {p.c.num_pages}, p.device);
  }
  Tensor moves = stream.result({p.c.num_pages / 2, 3}, at::kInt), count = stream.result({1}, at::kInt);
  call("fa_pages_compact", g_fa.compact, &p.c, (const int32_t*)p.table, (const int32_t*)p.lengths,
       (const int32_t*)p.refs, table_out, refs_out, static_cast<int32_t*>(moves.data_ptr()),
       static_cast<int32_t*>(count.data_ptr()), stream.raw);
  return pair(moves, count);
}

// k_pages, v_pages, page_table: the fields of fa_cache, in their order
PyObject* describe(PyObject* const* a, Py_ssize_t n) {
  want(n, 3);
  const Cache cache(a[0], a[1], a[2]);
  const fa_cache& c = cache.c;
  return Py_BuildValue("(iiiiiiiiLLLL)", c.num_pages, c.page_rows, c.H_kv, c.d, c.dtype, c.S, c.max_pages, c.reserved,
                       (long long)c.stride_page, (long long)c.stride_h, (long long)c.stride_n,
                       (long long)c.table_stride);
}

// FaError, then the addresses of the entry points in the order of Entries
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t kEntries = sizeof(Entries) / sizeof(void*);
  want(n, 1 + kEntries);
  void* p[kEntries];
  for (Py_ssize_t i = 0; i < kEntries; ++i) {
    p[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (PyErr_Occurred()) throw python_error();
  }
  memcpy(&g_fa, p, sizeof(g_fa));
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  Py_RETURN_NONE;
}

#define FA_METHOD(name, f) {name, (PyCFunction)(void (*)())python<f>, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FA_METHOD("bind", bind),       FA_METHOD("describe", describe), FA_METHOD("decode", decode),
                           FA_METHOD("append", append),   FA_METHOD("copy", copy),         FA_METHOD("extend", extend),
                           FA_METHOD("fork", fork),       FA_METHOD("free", release),      FA_METHOD("compact", compact),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&g_module); }
