// paged_bind.cpp — Python binding of the paged caches' and the rotary calls: checks the
// tensors, allocates what the caller left out and calls the C ABI (include/
// kvq.h).  A call on a small batch takes a few microseconds on the GPU, less
// than an interpreter needs to look at a dozen tensors, which is why these
// checks are compiled.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <map>
#include <mutex>
#include <string>
#include <tuple>
#include <type_traits>
#include <vector>

#include "kvq.h"

namespace {

PyObject* g_error_class = nullptr;  // kvq.KvqError(status, call)

// Raised by the checks; becomes a KvqError.
struct Refusal {
  int status;
  std::string what;
};

[[noreturn]] void refuse(const char* call, const std::string& what) {
  throw Refusal{KVQ_ERR_INVALID_ARG, std::string(call) + ": " + what};
}

void check(int status, const char* call) {
  if (status != KVQ_OK) throw Refusal{status, call};
}

const at::Tensor& tensor(const char* call, const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) refuse(call, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

long long number(const char* call, const char* name, PyObject* o, long long lo, long long hi) {
  PyObject* i = PyNumber_Index(o);
  long long v = 0;
  bool ok = i != nullptr;
  if (ok) {
    v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    ok = !(v == -1 && PyErr_Occurred());
  }
  if (!ok) {
    PyErr_Clear();
    refuse(call, std::string(name) + " must be a whole number");
  }
  if (v < lo || v > hi)
    refuse(call, std::string(name) + " must be between " + std::to_string(lo) + " and " +
                     std::to_string(hi) + ", not " + std::to_string(v));
  return v;
}
constexpr long long kIntMax = 0x7fffffff;

// The device of a call: every tensor of it is there.
struct Place {
  const char* call;
  int index = -1;
  void add(const char* name, const at::Tensor& x) {
    if (!x.is_cuda()) refuse(call, std::string(name) + " must be on a CUDA device");
    const int i = x.get_device();
    if (index < 0) index = i;
    if (i != index) refuse(call, std::string(name) + " must be on cuda:" + std::to_string(index));
  }
};

// Contiguous int32 of at least `size` elements.
const at::Tensor& ints(const char* call, const char* name, PyObject* o, int64_t size) {
  const at::Tensor& x = tensor(call, name, o);
  if (x.scalar_type() != at::kInt || !x.is_contiguous() || x.numel() < size)
    refuse(call, std::string(name) + " must be a contiguous int32 tensor of at least " +
                     std::to_string(size) + " elements");
  return x;
}
int* int_ptr(const at::Tensor& x) { return static_cast<int*>(x.data_ptr()); }

// block_table: [batch][max_pages].
const at::Tensor& table(const char* call, PyObject* o, int64_t batch) {
  const at::Tensor& x = ints(call, "block_table", o, 1);
  if (x.dim() != 2 || x.size(0) != batch)
    refuse(call, "block_table must be [" + std::to_string(batch) + "][max_pages]");
  return x;
}

struct Pool {
  kvq_paged_pool c;
  Pool(Place& place, PyObject* kp, PyObject* vp, PyObject* ks, PyObject* vs) {
    const char* call = place.call;
    const at::Tensor &k = tensor(call, "k_pages", kp), &v = tensor(call, "v_pages", vp);
    if (k.scalar_type() != at::kFloat8_e4m3fn || v.scalar_type() != at::kFloat8_e4m3fn ||
        k.dim() != 4 || v.sizes() != k.sizes() || !k.is_contiguous() || !v.is_contiguous())
      refuse(call, "k_pages and v_pages must be contiguous float8_e4m3fn tensors "
                   "[n_pages][n_kv_heads][page_size][head_dim]");
    const at::Tensor &sk = tensor(call, "k_scale", ks), &sv = tensor(call, "v_scale", vs);
    for (const at::Tensor* s : {&sk, &sv})
      if (s->scalar_type() != at::kFloat || s->dim() != 2 || s->size(0) != k.size(0) ||
          s->size(1) != k.size(1) || !s->is_contiguous())
        refuse(call, "k_scale and v_scale must be contiguous float32 tensors [n_pages][n_kv_heads]");
    for (int i = 0; i < 4; ++i)
      if (k.size(i) > kIntMax) throw Refusal{KVQ_ERR_UNSUPPORTED, call};
    c.k_pages = k.data_ptr();
    c.v_pages = v.data_ptr();
    c.k_scale = static_cast<float*>(sk.data_ptr());
    c.v_scale = static_cast<float*>(sv.data_ptr());
    c.n_pages = static_cast<int>(k.size(0));
    c.n_kv_heads = static_cast<int>(k.size(1));
    c.page_size = static_cast<int>(k.size(2));
    c.head_dim = static_cast<int>(k.size(3));
    place.add("k_pages", k);
    place.add("v_pages", v);
    place.add("k_scale", sk);
    place.add("v_scale", sv);
  }
};

struct Pool4 {
  kvq_paged4_pool c;
  Pool4(Place& place, PyObject* kc, PyObject* vc, PyObject* km, PyObject* vm) {
    const char* call = place.call;
    const at::Tensor &k = tensor(call, "k_codes", kc), &v = tensor(call, "v_codes", vc);
    if (k.scalar_type() != at::kByte || v.scalar_type() != at::kByte || k.dim() != 4 ||
        v.sizes() != k.sizes() || !k.is_contiguous() || !v.is_contiguous())
      refuse(call, "k_codes and v_codes must be contiguous uint8 tensors "
                   "[n_pages][n_kv_heads][page_size][head_dim / 2]");
    const at::Tensor &mk = tensor(call, "k_meta", km), &mv = tensor(call, "v_meta", vm);
    for (const at::Tensor* m : {&mk, &mv})
      if (m->scalar_type() != at::kHalf || m->dim() != 5 || m->size(0) != k.size(0) ||
          m->size(1) != k.size(1) || m->size(2) != k.size(2) || m->size(3) * 16 != k.size(3) ||
          m->size(4) != 2 || !m->is_contiguous())
        refuse(call, "k_meta and v_meta must be contiguous float16 tensors "
                     "[n_pages][n_kv_heads][page_size][head_dim / 32][2]");
    for (int i = 0; i < 4; ++i)
      if (k.size(i) > kIntMax / 2) throw Refusal{KVQ_ERR_UNSUPPORTED, call};
    c.k_codes = k.data_ptr();
    c.v_codes = v.data_ptr();
    c.k_meta = mk.data_ptr();
    c.v_meta = mv.data_ptr();
    c.n_pages = static_cast<int>(k.size(0));
    c.n_kv_heads = static_cast<int>(k.size(1));
    c.page_size = static_cast<int>(k.size(2));
    c.head_dim = static_cast<int>(2 * k.size(3));
    place.add("k_codes", k);
    place.add("v_codes", v);
    place.add("k_meta", mk);
    place.add("v_meta", mv);
  }
};

int dtype_of(const char* call, const char* name, const at::Tensor& x) {
  if (x.scalar_type() == at::kHalf) return KVQ_DTYPE_FP16;
  if (x.scalar_type() == at::kBFloat16) return KVQ_DTYPE_BF16;
  refuse(call, std::string(name) + " must be float16 or bfloat16");
}

// Token stride of x: [tokens][heads][dim], a token's heads and channels
// contiguous.
long long rows(const char* call, const char* name, const at::Tensor& x, int64_t heads,
               int64_t dim) {
  if (x.dim() != 3 || x.size(1) != heads || x.size(2) != dim || x.stride(2) != 1 ||
      (x.stride(1) != dim && heads != 1))
    refuse(call, std::string(name) + " must be [tokens][" + std::to_string(heads) + "][" +
                     std::to_string(dim) + "], a token's heads and channels contiguous");
  if (x.size(0) > kIntMax) throw Refusal{KVQ_ERR_UNSUPPORTED, call};
  return x.size(0) > 1 ? x.stride(0) : heads * dim;
}

cudaStream_t stream_of(const char* call, PyObject* o, int index) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(index).stream();
  PyObject* v = nullptr;
  if (PyLong_Check(o)) {
    v = Py_NewRef(o);
  } else {
    v = PyObject_GetAttrString(o, "cuda_stream");
  }
  void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
  Py_XDECREF(v);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse(call, "stream must be a stream or its address");
  }
  // (one name for as many streams as there are threads; memory is kept by name)
  if (p == cudaStreamPerThread) refuse(call, "stream must not be the per-thread default stream");
  return static_cast<cudaStream_t>(p);
}

int* error_ptr(Place& place, PyObject* o) {
  if (o == Py_None) return nullptr;
  const at::Tensor& x = ints(place.call, "error", o, 1);
  place.add("error", x);
  return int_ptr(x);
}

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType t, int index) {
  return at::detail::empty_cuda(sizes, t, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(index)),
                                std::nullopt);
}

// An output of a call on stream st: memory of st, as work still waiting on the
// current stream may use what that stream's allocations get again; and freed
// only behind the current stream's work, which reads it.
at::Tensor empty_on(cudaStream_t st, at::IntArrayRef sizes, at::ScalarType t, int index) {
  const c10::cuda::CUDAStream cur = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index));
  if (cur.stream() == st) return empty(sizes, t, index);
  const c10::cuda::CUDAStreamGuard guard(
      c10::cuda::getStreamFromExternal(st, static_cast<c10::DeviceIndex>(index)));
  at::Tensor x = empty(sizes, t, index);
  if (x.numel() > 0) c10::cuda::CUDACachingAllocator::recordStream(x.storage().data_ptr(), cur);
  return x;
}

// angles: fp32 [tokens][rotary_dim / 2][2].
const at::Tensor& angles_of(const char* call, PyObject* o, int64_t tokens, kvq_rotary* r, bool interleaved) {
  const at::Tensor& x = tensor(call, "angles", o);
  if (x.scalar_type() != at::kFloat || x.dim() != 3 || x.size(0) != tokens || x.size(2) != 2 ||
      x.size(1) > 1 << 20 || !x.is_contiguous())
    refuse(call, "angles must be a contiguous float32 tensor [" + std::to_string(tokens) + "][rotary_dim / 2][2]");
  r->angles = static_cast<const float*>(x.data_ptr());
  r->rotary_dim = static_cast<int>(2 * x.size(1));
  r->interleaved = interleaved ? 1 : 0;
  return x;
}
bool truth(const char* call, const char* name, PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(call, std::string(name) + " must be true or false");
  }
  return v != 0;
}

// The heads that a call turns: x [tokens][heads][dim], and out of the same type
// and shape (allocated at finish() when the caller gave none).
struct Turned {
  const at::Tensor* x = nullptr;
  at::Tensor out;
  long long xs = 0, os = 0;
  int64_t heads = 0, dim = 0;
  Turned() = default;
  Turned(const char* call, const char* xn, PyObject* xo, const char* on, PyObject* oo) {
    x = &tensor(call, xn, xo);
    dtype_of(call, xn, *x);
    if (x->dim() != 3) refuse(call, std::string(xn) + " must be [tokens][heads][head_dim]");
    heads = x->size(1);
    dim = x->size(2);
    if (heads > kIntMax || dim > kIntMax) throw Refusal{KVQ_ERR_UNSUPPORTED, call};
    xs = rows(call, xn, *x, heads, dim);
    os = heads * dim;
    if (oo != Py_None) {
      out = tensor(call, on, oo);
      if (out.scalar_type() != x->scalar_type() || out.sizes() != x->sizes())
        refuse(call, std::string(on) + " must have " + xn + "'s type and shape");
      os = rows(call, on, out, heads, dim);
    }
  }
  void add(Place& place, const char* xn, const char* on) const {
    place.add(xn, *x);
    if (out.defined()) place.add(on, out);
  }
  void finish(cudaStream_t st, int index) {
    if (!out.defined()) out = empty_on(st, x->sizes(), x->scalar_type(), index);
  }
};

// ---- workspaces ---------------------------------------------------------------
//
// Calls on one stream, over either kind of pages, run one after the other and share a workspace; the calls
// that a stream captures into one graph share another one, out of the
// capture's memory, whose counters the graph clears before their first use.
// So two graphs, or a graph and eager calls, never share.  A graph's workspace
// is the graph's: it lives as long as the graph and what is instantiated of it.
struct Workspace {
  at::Tensor mem;  // eager calls'
  void* at = nullptr;
  unsigned long long capture = 0;
};
using WorkKey = std::tuple<int, cudaStream_t, int, bool>;  // device, stream, head_dim, captured
std::mutex g_mu;
std::map<WorkKey, Workspace>& workspaces() {
  static auto* m = new std::map<WorkKey, Workspace>;  // outlives the interpreter's end
  return *m;
}

// Workspaces of graphs that are gone.  A graph is destroyed on a thread that may
// not call CUDA, so the next call frees them.
std::mutex g_gone_mu;
std::vector<at::Tensor*>& gone() {
  static auto* v = new std::vector<at::Tensor*>;
  return *v;
}
void CUDART_CB graph_gone(void* mem) {
  std::lock_guard<std::mutex> lock(g_gone_mu);
  gone().push_back(static_cast<at::Tensor*>(mem));
}
void free_gone() {
  std::vector<at::Tensor*> v;
  {
    std::lock_guard<std::mutex> lock(g_gone_mu);
    v.swap(gone());
  }
  for (at::Tensor* t : v) delete t;
}

// Makes `graph` keep `mem`.
bool keep_with_graph(cudaGraph_t graph, const at::Tensor& mem) {
  auto* held = new at::Tensor(mem);
  cudaUserObject_t object = nullptr;
  if (cudaUserObjectCreate(&object, held, graph_gone, 1, cudaUserObjectNoDestructorSync) != cudaSuccess) {
    delete held;
    return false;
  }
  if (cudaGraphRetainUserObject(graph, object, 1, cudaGraphUserObjectMove) == cudaSuccess) return true;
  cudaUserObjectRelease(object, 1);
  return false;
}

void* workspace(const char* call, int head_dim, int index, cudaStream_t st, size_t bytes) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  cudaGraph_t graph = nullptr;
  if (cudaStreamGetCaptureInfo(st, &status, &id, &graph) != cudaSuccess) {
    cudaGetLastError();
    throw Refusal{KVQ_ERR_CUDA, call};
  }
  const bool captured = status == cudaStreamCaptureStatusActive;
  free_gone();
  std::lock_guard<std::mutex> lock(g_mu);
  Workspace& w = workspaces()[WorkKey(index, st, head_dim, captured)];
  if (w.at == nullptr || (captured && w.capture != id)) {
    w.at = nullptr;
    const c10::cuda::CUDAStreamGuard guard(
        c10::cuda::getStreamFromExternal(st, static_cast<c10::DeviceIndex>(index)));
    at::Tensor mem = empty({static_cast<int64_t>(bytes)}, at::kByte, index);
    if (cudaMemsetAsync(mem.data_ptr(), 0, 1024, st) != cudaSuccess ||
        (captured && !keep_with_graph(graph, mem))) {
      cudaGetLastError();
      throw Refusal{KVQ_ERR_CUDA, call};
    }
    w.at = mem.data_ptr();
    w.capture = id;
    if (!captured) w.mem = std::move(mem);
  }
  return w.at;
}

int workspace_bytes(const kvq_paged_pool& p, size_t* n) { return kvq_paged_workspace_bytes(&p, n); }
int workspace_bytes(const kvq_paged4_pool& p, size_t* n) { return kvq_paged4_workspace_bytes(&p, n); }
template <typename... A>
int attend(const kvq_paged_pool* p, A... a) { return kvq_paged_attention(p, a...); }
template <typename... A>
int attend(const kvq_paged4_pool* p, A... a) { return kvq_paged4_attention(p, a...); }

template <typename... A>
int store_turned(const kvq_paged_pool* p, A... a) { return kvq_paged_append(p, a...); }
template <typename... A>
int store_turned(const kvq_paged4_pool* p, A... a) { return kvq_paged4_append(p, a...); }

// ---- the calls ------------------------------------------------------------------

template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refusal& r) {
    PyObject* e = PyObject_CallFunction(g_error_class ? g_error_class : PyExc_RuntimeError, "is",
                                        r.status, r.what.c_str());
    if (e != nullptr) {
      PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
      Py_DECREF(e);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

bool count_is(const char* call, Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", call, want, n);
  return false;
}

// (ctx_len, new_len, block_table, free_pages, n_free, page_size, n_tokens,
//  cu_new, seq_len, slots, n_left, error, stream, positions)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is("plan", n, 14)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* call = "kvq_paged_plan";
    Place place{call};
    const at::Tensor& ctx = ints(call, "ctx_len", a[0], 1);
    const int64_t batch = ctx.numel();
    const at::Tensor& nw = ints(call, "new_len", a[1], batch);
    const at::Tensor& tab = table(call, a[2], batch);
    const at::Tensor& fp = ints(call, "free_pages", a[3], 0);
    const at::Tensor& nf = ints(call, "n_free", a[4], 1);
    const int ps = static_cast<int>(number(call, "page_size", a[5], 1, kIntMax));
    const int64_t tokens = number(call, "n_tokens", a[6], 0, kIntMax);
    if (batch > kIntMax || tab.size(1) > kIntMax || fp.numel() > kIntMax)
      throw Refusal{KVQ_ERR_UNSUPPORTED, call};
    const char* names[4] = {"cu_new", "seq_len", "slots", "n_left"};
    const int64_t sizes[4] = {batch + 1, batch, tokens, 1};
    at::Tensor out[4];
    PyObject* ret[4];
    for (int i = 0; i < 4; ++i) {
      if (a[7 + i] == Py_None) continue;
      out[i] = ints(call, names[i], a[7 + i], sizes[i]);
    }
    const at::Tensor* positions = a[13] == Py_None ? nullptr : &ints(call, "positions", a[13], tokens);
    place.add("ctx_len", ctx);
    place.add("new_len", nw);
    place.add("block_table", tab);
    place.add("free_pages", fp);
    place.add("n_free", nf);
    for (int i = 0; i < 4; ++i)
      if (out[i].defined()) place.add(names[i], out[i]);
    if (positions) place.add("positions", *positions);
    int* err = error_ptr(place, a[11]);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(place.index));
    const cudaStream_t st = stream_of(call, a[12], place.index);
    for (int i = 0; i < 4; ++i)
      if (!out[i].defined()) out[i] = empty_on(st, {sizes[i]}, at::kInt, place.index);
    check(kvq_paged_plan_positions(int_ptr(ctx), int_ptr(nw), static_cast<int>(batch), int_ptr(tab),
                         static_cast<int>(tab.size(1)), int_ptr(fp), static_cast<int>(fp.numel()),
                         int_ptr(nf), ps, static_cast<int>(tokens), int_ptr(out[0]),
                         int_ptr(out[1]), int_ptr(out[2]), positions ? int_ptr(*positions) : nullptr, int_ptr(out[3]), err, st),
          call);
    for (int i = 0; i < 4; ++i)
      ret[i] = a[7 + i] != Py_None ? Py_NewRef(a[7 + i]) : THPVariable_Wrap(std::move(out[i]));
    PyObject* t = PyTuple_New(4);
    for (int i = 0; i < 4; ++i) PyTuple_SET_ITEM(t, i, ret[i]);
    return t;
  });
}

// (k, v, slots, k_pages, v_pages, k_scale, v_scale, error, stream)
PyObject* store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is("store", n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* call = "kvq_paged_store";
    const at::Tensor &k = tensor(call, "k", a[0]), &v = tensor(call, "v", a[1]);
    const int dt = dtype_of(call, "k", k);
    if (v.scalar_type() != k.scalar_type() || v.sizes() != k.sizes())
      refuse(call, "k and v must have the same type and shape");
    if (k.dim() != 3) refuse(call, "k must be [tokens][n_kv_heads][head_dim]");
    const at::Tensor& slots = ints(call, "slots", a[2], k.size(0));
    Place place{call};
    // (shapes first, so that a wrong one is told before a wrong device)
    const at::Tensor& kp = tensor(call, "k_pages", a[3]);
    long long ks = 0, vs = 0;
    if (kp.dim() == 4) {
      ks = rows(call, "k", k, kp.size(1), kp.size(3));
      vs = rows(call, "v", v, kp.size(1), kp.size(3));
    }
    const Pool pool(place, a[3], a[4], a[5], a[6]);
    place.add("k", k);
    place.add("v", v);
    place.add("slots", slots);
    int* err = error_ptr(place, a[7]);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(place.index));
    check(kvq_paged_store(&pool.c, k.data_ptr(), v.data_ptr(), dt, ks, vs, int_ptr(slots),
                          static_cast<int>(k.size(0)), err, stream_of(call, a[8], place.index)),
          call);
    Py_RETURN_NONE;
  });
}

// (q, k_pages, v_pages, k_scale, v_scale, block_table, cu_new, seq_len,
//  max_new, softmax_scale, window, out, workspace, error, stream); `P`: Pool, or
// Pool4 with codes and metadata in the pages' and scales' places
template <typename P>
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr bool four = std::is_same<P, Pool4>::value;
  if (!count_is(four ? "attention4" : "attention", n, 15)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* call = four ? "kvq_paged4_attention" : "kvq_paged_attention";
    Place place{call};
    const at::Tensor& q = tensor(call, "q", a[0]);
    const int dt = dtype_of(call, "q", q);
    if (q.dim() != 3) refuse(call, "q must be [tokens][n_q_heads][head_dim]");
    const at::Tensor& seq = ints(call, "seq_len", a[7], 1);
    const int64_t batch = seq.numel(), tokens = q.size(0), heads = q.size(1), dim = q.size(2);
    const at::Tensor& tab = table(call, a[5], batch);
    const at::Tensor& cu = ints(call, "cu_new", a[6], batch + 1);
    const int max_new = static_cast<int>(number(call, "max_new", a[8], 1, kIntMax));
    double scale = 0;
    if (a[9] == Py_None) {
      scale = 1.0 / std::sqrt(static_cast<double>(dim));
    } else {
      scale = PyFloat_AsDouble(a[9]);
      if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse(call, "softmax_scale must be a number");
      }
    }
    const int window = static_cast<int>(number(call, "window", a[10], 0, kIntMax));
    const at::Tensor& kp = tensor(call, four ? "k_codes" : "k_pages", a[1]);
    const long long qs = rows(call, "q", q, heads, kp.dim() == 4 ? kp.size(3) * (four ? 2 : 1) : dim);
    at::Tensor out;
    long long os = heads * dim;
    if (a[11] != Py_None) {
      out = tensor(call, "out", a[11]);
      if (out.scalar_type() != q.scalar_type() || out.sizes() != q.sizes())
        refuse(call, "out must have q's type and shape");
      os = rows(call, "out", out, heads, dim);
    }
    if (batch > kIntMax || tab.size(1) > kIntMax || heads > kIntMax)
      throw Refusal{KVQ_ERR_UNSUPPORTED, call};
    const P pool(place, a[1], a[2], a[3], a[4]);
    place.add("q", q);
    place.add("block_table", tab);
    place.add("cu_new", cu);
    place.add("seq_len", seq);
    if (out.defined()) place.add("out", out);
    int* err = error_ptr(place, a[13]);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(place.index));
    const cudaStream_t st = stream_of(call, a[14], place.index);
    if (!out.defined()) out = empty_on(st, q.sizes(), q.scalar_type(), place.index);
    void* ws = nullptr;
    size_t bytes = 0;
    if (a[12] == Py_None) {
      check(workspace_bytes(pool.c, &bytes), call);
      ws = workspace(call, pool.c.head_dim, place.index, st, bytes);
    } else {
      const at::Tensor& w = tensor(call, "workspace", a[12]);
      if (w.scalar_type() != at::kByte || !w.is_contiguous())
        refuse(call, "workspace must be a contiguous uint8 tensor");
      place.add("workspace", w);
      ws = w.data_ptr();
      bytes = static_cast<size_t>(w.numel());
    }
    check(attend(&pool.c, q.data_ptr(), dt, qs, out.data_ptr(), os, static_cast<int>(tokens),
                 static_cast<int>(heads), int_ptr(tab), static_cast<int>(tab.size(1)), int_ptr(cu),
                 int_ptr(seq), static_cast<int>(batch), max_new, static_cast<float>(scale), window, ws,
                 bytes, err, st),
          call);
    return a[11] != Py_None ? Py_NewRef(a[11]) : THPVariable_Wrap(std::move(out));
  });
}

// k and v of a store: types, shapes and strides.
struct Tokens {
  const at::Tensor *k, *v, *slots;
  int dtype;
  long long ks = 0, vs = 0;
  Tokens(const char* call, PyObject* ko, PyObject* vo, PyObject* so, const at::Tensor& pages, int64_t per) {
    k = &tensor(call, "k", ko);
    v = &tensor(call, "v", vo);
    dtype = dtype_of(call, "k", *k);
    if (v->scalar_type() != k->scalar_type() || v->sizes() != k->sizes())
      refuse(call, "k and v must have the same type and shape");
    if (k->dim() != 3) refuse(call, "k must be [tokens][n_kv_heads][head_dim]");
    slots = &ints(call, "slots", so, k->size(0));
    if (pages.dim() == 4) {
      ks = rows(call, "k", *k, pages.size(1), pages.size(3) * per);
      vs = rows(call, "v", *v, pages.size(1), pages.size(3) * per);
    }
  }
  void add(Place& place) const {
    place.add("k", *k);
    place.add("v", *v);
    place.add("slots", *slots);
  }
};

// (k, v, slots, k_pages, v_pages, k_scale, v_scale, angles, interleaved, q, q_out,
//  error, stream); `P`: Pool, or Pool4 with codes and metadata in the pages' and
// scales' places
template <typename P>
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr bool four = std::is_same<P, Pool4>::value;
  if (!count_is(four ? "append4" : "append", n, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* call = four ? "kvq_paged4_append" : "kvq_paged_append";
    const Tokens t(call, a[0], a[1], a[2], tensor(call, four ? "k_codes" : "k_pages", a[3]), four ? 2 : 1);
    const int64_t tokens = t.k->size(0);
    kvq_rotary rotary = {};
    Place place{call};
    const bool turns = a[7] != Py_None, queries = a[9] != Py_None;
    if (!turns && !four) refuse(call, "angles must be a tensor");
    if (!turns && queries) refuse(call, "angles must be given with q");
    if (!queries && a[10] != Py_None) refuse(call, "q_out must be given with q");
    const at::Tensor* angles = nullptr;
    if (turns) angles = &angles_of(call, a[7], tokens, &rotary, truth(call, "interleaved", a[8]));
    Turned q;
    if (queries) {
      q = Turned(call, "q", a[9], "q_out", a[10]);
      if (q.x->scalar_type() != t.k->scalar_type() || q.x->size(0) != tokens || q.dim != t.k->size(2))
        refuse(call, "q must have k's type, tokens and head_dim");
    }
    const P pool(place, a[3], a[4], a[5], a[6]);
    t.add(place);
    if (turns) place.add("angles", *angles);
    if (queries) q.add(place, "q", "q_out");
    int* err = error_ptr(place, a[11]);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(place.index));
    const cudaStream_t st = stream_of(call, a[12], place.index);
    if (queries) q.finish(st, place.index);
    check(store_turned(&pool.c, turns ? &rotary : nullptr, t.k->data_ptr(), t.v->data_ptr(), t.dtype, t.ks,
                       t.vs, int_ptr(*t.slots), static_cast<int>(tokens),
                       queries ? q.x->data_ptr() : nullptr, q.xs, queries ? q.out.data_ptr() : nullptr,
                       q.os, static_cast<int>(q.heads), err, st),
          call);
    if (!queries) Py_RETURN_NONE;
    return a[10] != Py_None ? Py_NewRef(a[10]) : THPVariable_Wrap(std::move(q.out));
  });
}

// (slots, k_codes, v_codes, k_meta, v_meta, k, v, error, stream)
PyObject* read4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is("read4", n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* call = "kvq_paged4_read";
    Place place{call};
    const at::Tensor& slots = ints(call, "slots", a[0], 0);
    const Pool4 pool(place, a[1], a[2], a[3], a[4]);
    const int64_t tokens = slots.numel();
    if (tokens > kIntMax) throw Refusal{KVQ_ERR_UNSUPPORTED, call};
    const int64_t sizes[3] = {tokens, pool.c.n_kv_heads, pool.c.head_dim};
    at::Tensor out[2];
    const char* names[2] = {"k", "v"};
    for (int i = 0; i < 2; ++i) {
      if (a[5 + i] == Py_None) continue;
      out[i] = tensor(call, names[i], a[5 + i]);
      if (out[i].scalar_type() != at::kHalf || out[i].sizes() != at::IntArrayRef(sizes, 3) ||
          !out[i].is_contiguous())
        refuse(call, std::string(names[i]) + " must be a contiguous float16 tensor [slots][n_kv_heads][head_dim]");
      place.add(names[i], out[i]);
    }
    place.add("slots", slots);
    int* err = error_ptr(place, a[7]);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(place.index));
    const cudaStream_t st = stream_of(call, a[8], place.index);
    for (int i = 0; i < 2; ++i)
      if (!out[i].defined()) out[i] = empty_on(st, at::IntArrayRef(sizes, 3), at::kHalf, place.index);
    check(kvq_paged4_read(&pool.c, int_ptr(slots), static_cast<int>(tokens), out[0].data_ptr(),
                          out[1].data_ptr(), err, st),
          call);
    PyObject* t = PyTuple_New(2);
    for (int i = 0; i < 2; ++i)
      PyTuple_SET_ITEM(t, i, a[5 + i] != Py_None ? Py_NewRef(a[5 + i]) : THPVariable_Wrap(std::move(out[i])));
    return t;
  });
}

// (positions, turns, magnitude, out, stream)
PyObject* angles(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is("angles", n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* call = "kvq_rotary_angles";
    Place place{call};
    const at::Tensor& pos = ints(call, "positions", a[0], 0);
    const at::Tensor& turns = tensor(call, "turns", a[1]);
    if (turns.scalar_type() != at::kLong || turns.dim() != 1 || !turns.is_contiguous() || turns.numel() < 1)
      refuse(call, "turns must be a contiguous int64 tensor [rotary_dim / 2]");
    const double magnitude = PyFloat_AsDouble(a[2]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      refuse(call, "magnitude must be a number");
    }
    if (pos.numel() > kIntMax || turns.numel() > kIntMax / 2) throw Refusal{KVQ_ERR_UNSUPPORTED, call};
    const int64_t sizes[3] = {pos.numel(), turns.numel(), 2};
    at::Tensor out;
    if (a[3] != Py_None) {
      out = tensor(call, "out", a[3]);
      if (out.scalar_type() != at::kFloat || out.sizes() != at::IntArrayRef(sizes, 3) || !out.is_contiguous())
        refuse(call, "out must be a contiguous float32 tensor [tokens][rotary_dim / 2][2]");
    }
    place.add("positions", pos);
    place.add("turns", turns);
    if (out.defined()) place.add("out", out);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(place.index));
    const cudaStream_t st = stream_of(call, a[4], place.index);
    if (!out.defined()) out = empty_on(st, at::IntArrayRef(sizes, 3), at::kFloat, place.index);
    check(kvq_rotary_angles(int_ptr(pos), static_cast<int>(pos.numel()),
                            static_cast<const int64_t*>(turns.data_ptr()), static_cast<int>(2 * turns.numel()),
                            static_cast<float>(magnitude), static_cast<float*>(out.data_ptr()), st),
          call);
    return a[3] != Py_None ? Py_NewRef(a[3]) : THPVariable_Wrap(std::move(out));
  });
}

// (x, angles, interleaved, out, stream)
PyObject* rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is("rotate", n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* call = "kvq_rotate";
    Place place{call};
    Turned x(call, "x", a[0], "out", a[3]);
    kvq_rotary rotary = {};
    const at::Tensor& ang = angles_of(call, a[1], x.x->size(0), &rotary, truth(call, "interleaved", a[2]));
    x.add(place, "x", "out");
    place.add("angles", ang);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(place.index));
    const cudaStream_t st = stream_of(call, a[4], place.index);
    x.finish(st, place.index);
    check(kvq_rotate(&rotary, x.x->data_ptr(), dtype_of(call, "x", *x.x), x.xs, x.out.data_ptr(), x.os,
                     static_cast<int>(x.x->size(0)), static_cast<int>(x.heads), static_cast<int>(x.dim), st),
          call);
    return a[3] != Py_None ? Py_NewRef(a[3]) : THPVariable_Wrap(std::move(x.out));
  });
}

PyObject* set_error_class(PyObject*, PyObject* c) {
  Py_XDECREF(g_error_class);
  g_error_class = Py_NewRef(c);
  Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef fast(const char* name, Fast f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {fast("plan", plan),
                           fast("store", store),
                           fast("attention", attention<Pool>),
                           fast("append", append<Pool>),
                           fast("append4", append<Pool4>),
                           fast("read4", read4),
                           fast("attention4", attention<Pool4>),
                           fast("angles", angles),
                           fast("rotate", rotate),
                           {"set_error_class", set_error_class, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_paged_bind", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_bind() { return PyModule_Create(&g_module); }
