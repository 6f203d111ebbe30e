// binding.cpp -- the Python calls of the 8-bit cache, and of normed and rotated rows, accumulated
// weights and eviction (of either cache): the checks of their tensors, outputs and scratch from
// torch's allocator, and one call of the C ABI each.
//
// The calls are made once per layer and step, and the smallest ones run for 2 to 6 us on the
// GPU: reading some forty properties of ten tensors from Python, and passing twenty arguments
// through ctypes, took longer than that (draft step 18.8 us a call on the host, 6.3 here; one token
// stored 8.5, 2.9; a short verification 20.4, 7.1).
#include <climits>
#include <string>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/vsd.h"

namespace {

constexpr int64_t kHistBins = 4096;  // of a scored verification's histogram

// ---------------------------------------------------------------- the library's calls
struct Calls {
  decltype(&vsd_append_kv_quant) append = nullptr;
  decltype(&vsd_read_kv_quant_zeroed) read = nullptr;
  decltype(&vsd_verify_quant_workspace_size) verify_size = nullptr;
  decltype(&vsd_verify_attn_collect_quant) verify = nullptr;
  decltype(&vsd_sparse_quant_workspace_size) sparse_size = nullptr;
  decltype(&vsd_sparse_decode_attn_quant) sparse = nullptr;
  decltype(&vsd_norm_rope) rope = nullptr;
  decltype(&vsd_norm_rope_append_kv) rope_append = nullptr;
  decltype(&vsd_norm_rope_append_kv_quant) rope_append_quant = nullptr;
  decltype(&vsd_accumulate_weights) weights = nullptr;
  decltype(&vsd_accumulate_weights_quant) weights_quant = nullptr;
  decltype(&vsd_compact_kv) compact = nullptr;
  decltype(&vsd_compact_kv_quant) compact_quant = nullptr;
  decltype(&vsd_select_topk) select = nullptr;
  PyObject* error = nullptr;  // VsdError(status, name)
};
Calls g_calls;

// What a call refuses, on its way to a Python exception.
struct Refused {
  PyObject* type;
  std::string what;
};

// A Python exception that is set already.
struct PythonError {};

[[noreturn]] void refuse(PyObject* type, const std::string& what) { throw Refused{type, what}; }

void check(vsd_status st, const char* call) {
  if (st == VSD_OK) return;
  PyObject* e = PyObject_CallFunction(g_calls.error, "is", static_cast<int>(st), call);
  if (e != nullptr) {
    PyErr_SetObject(g_calls.error, e);
    Py_DECREF(e);
  }
  throw PythonError{};
}

// ---------------------------------------------------------------- arguments
int as_int(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  if (v < INT_MIN || v > INT_MAX) refuse(PyExc_ValueError, std::string(name) + " is out of range");
  return static_cast<int>(v);
}

float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return static_cast<float>(v);
}

bool as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v != 0;
}

int dim_of(int64_t n, const char* name) {
  if (n > INT_MAX) refuse(PyExc_ValueError, std::string(name) + " is too large");
  return static_cast<int>(n);
}

const at::Tensor& as_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + ")";
}

// A contiguous tensor of the type on a GPU, of `dims` dimensions.
void need(const at::Tensor& t, at::ScalarType type, int64_t dims, const char* name) {
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " +
                                c10::toString(t.scalar_type()));
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
  if (t.dim() != dims)
    refuse(PyExc_ValueError, std::string(name) + " must have " + std::to_string(dims) +
                                 " dimensions, got shape " + text(t.sizes()));
  if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
}

// The same with the shape and the device.
void need(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, int dev, const char* name) {
  need(t, type, static_cast<int64_t>(shape.size()), name);
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
  if (t.get_device() != dev) refuse(PyExc_ValueError, std::string(name) + " is on another device");
}

void* pointer(const at::Tensor& t) { return t.data_ptr(); }

// A cache's tensors, and the part of the geometry that they give.
struct Cache {
  void *k, *v;
  float *ks, *vs;
};

Cache cache_of(PyObject* const* a, int dev, vsd_geom* geom) {
  const at::Tensor &k = as_tensor(a[0], "k_cache"), &v = as_tensor(a[1], "v_cache");
  const at::Tensor &ks = as_tensor(a[2], "k_scale"), &vs = as_tensor(a[3], "v_scale");
  need(k, at::kFloat8_e4m3fn, 4, "k_cache");
  if (k.get_device() != dev) refuse(PyExc_ValueError, "k_cache is on another device");
  need(v, at::kFloat8_e4m3fn, k.sizes(), dev, "v_cache");
  need(ks, at::kFloat, k.sizes().slice(0, 2), dev, "k_scale");
  need(vs, at::kFloat, k.sizes().slice(0, 2), dev, "v_scale");
  geom->num_blocks = dim_of(k.size(0), "num_blocks");
  geom->Hkv = dim_of(k.size(1), "Hkv");
  geom->page_size = dim_of(k.size(2), "page_size");
  geom->head_dim = dim_of(k.size(3), "head_dim");
  return Cache{pointer(k), pointer(v), static_cast<float*>(pointer(ks)), static_cast<float*>(pointer(vs))};
}

// int32 [B]
const int32_t* lengths(const at::Tensor& t, int64_t B, int dev, const char* name) {
  need(t, at::kInt, {B}, dev, name);
  return static_cast<const int32_t*>(pointer(t));
}

const int32_t* table_of(const at::Tensor& t, int64_t B, int dev, vsd_geom* geom) {
  need(t, at::kInt, 2, "block_table");
  need(t, at::kInt, {B, t.size(1)}, dev, "block_table");
  geom->max_blocks_per_seq = dim_of(t.size(1), "max_blocks_per_seq");
  return static_cast<const int32_t*>(pointer(t));
}

// ---------------------------------------------------------------- device, stream, memory
// The device of a call's first tensor made current, and its stream: the caller's, or the
// device's current one.  What a call allocates comes from torch's allocator tied to that
// stream, so that calls on other streams, and captured graphs, get memory of their own and
// it goes back in stream order.
struct Place {
  int dev;
  c10::cuda::CUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard on;
  cudaStream_t stream;

  Place(const at::Tensor& first, PyObject* raw) : dev(first.get_device()), device(static_cast<c10::DeviceIndex>(dev)) {
    if (raw != Py_None) {
      stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(raw));
      if (PyErr_Occurred()) throw PythonError{};
      on.reset_stream(c10::cuda::getStreamFromExternal(stream, static_cast<c10::DeviceIndex>(dev)));
    } else {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    }
  }

  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions(type).device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)));
  }
};

// Scratch: the caller's, or memory of the call's own.  A call is up to two launches that
// hand partial results on through it, made with the interpreter's lock released: memory that
// calls share would let a second thread's launch come between them (both threads on one
// stream).  Memory of its own belongs to the call until both launches are made, and goes back
// to its stream then; a captured call takes it from the graph's pool.  (One buffer kept for
// each stream, with a lock over a call's launches, would save 1.2 us of host time; it would
// keep the largest call's memory for good.)
struct Scratch {
  void* at = nullptr;
  size_t bytes = 0;
  at::Tensor keep;

  Scratch(PyObject* given, size_t need_bytes, const Place& p) {
    if (given != Py_None) {
      keep = as_tensor(given, "workspace");
      if (!keep.is_cuda() || keep.get_device() != p.dev || !keep.is_contiguous())
        refuse(PyExc_ValueError, "workspace must be contiguous and on the call's device");
    } else if (need_bytes == 0) {
      return;
    } else {
      keep = p.empty({static_cast<int64_t>(need_bytes)}, at::kByte);
    }
    at = pointer(keep);
    bytes = keep.nbytes();
  }
};

// An output: the caller's tensor, or a new one.
struct Output {
  PyObject* object = Py_None;  // borrowed, unless `made` holds a tensor
  at::Tensor made;
  void* at = nullptr;

  void take(PyObject* given, const Place& p, at::ScalarType type, at::IntArrayRef shape, const char* name) {
    if (given != Py_None) {
      object = given;
      const at::Tensor& t = as_tensor(given, name);
      need(t, type, shape, p.dev, name);
      at = pointer(t);
    } else {
      made = p.empty(shape, type);
      at = pointer(made);
    }
  }
  PyObject* result() const {
    if (made.defined()) return THPVariable_Wrap(made);
    Py_INCREF(object);
    return object;
  }
};

template <typename F>
vsd_status without_gil(F&& f) {
  vsd_status st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return st;
}

// The body of a call: C++ and torch errors become Python exceptions.
template <typename F>
PyObject* call(Py_ssize_t n, Py_ssize_t want, F&& body) {
  HANDLE_TH_ERRORS
  if (n != want || g_calls.error == nullptr) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or no library attached");
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  } catch (const PythonError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- the calls
// append(k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_table, pos_base, pos_offset,
//        n_valid, stream)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, [&]() -> PyObject* {
    const at::Tensor &kn = as_tensor(a[0], "k_new"), &vn = as_tensor(a[1], "v_new");
    need(kn, at::kBFloat16, 4, "k_new");
    const Place p(kn, a[10]);
    vsd_geom g;
    const Cache c = cache_of(a + 2, p.dev, &g);
    const int64_t B = kn.size(0);
    need(kn, at::kBFloat16, {B, kn.size(1), g.Hkv, g.head_dim}, p.dev, "k_new");
    need(vn, at::kBFloat16, kn.sizes(), p.dev, "v_new");
    const int32_t* bt = table_of(as_tensor(a[6], "block_table"), B, p.dev, &g);
    const int32_t* pos = lengths(as_tensor(a[7], "pos_base"), B, p.dev, "pos_base");
    const int32_t* nv = a[9] == Py_None ? nullptr : lengths(as_tensor(a[9], "n_valid"), B, p.dev, "n_valid");
    const int rows = dim_of(kn.size(1), "k_new"), offset = as_int(a[8], "pos_offset");
    g.B = dim_of(B, "B");
    g.Hq = g.Hkv;
    check(without_gil([&] {
            return g_calls.append(&g, rows, pointer(kn), pointer(vn), bt, pos, offset, nv, c.k, c.v, c.ks, c.vs,
                                  p.stream);
          }),
          "vsd_append_kv_quant");
    Py_RETURN_NONE;
  });
}

// read(k_cache, v_cache, k_scale, v_scale, block_table, pos_base, n, pos_offset, n_valid, k_out,
//      v_out, stream) -> (k_out, v_out)
PyObject* py_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 12, [&]() -> PyObject* {
    const at::Tensor& kc = as_tensor(a[0], "k_cache");
    need(kc, at::kFloat8_e4m3fn, 4, "k_cache");
    const Place p(kc, a[11]);
    vsd_geom g;
    const Cache c = cache_of(a, p.dev, &g);
    const at::Tensor& pt = as_tensor(a[5], "pos_base");
    need(pt, at::kInt, 1, "pos_base");
    const int64_t B = pt.size(0);
    const int32_t* pos = lengths(pt, B, p.dev, "pos_base");
    const int32_t* bt = table_of(as_tensor(a[4], "block_table"), B, p.dev, &g);
    const int32_t* nv = a[8] == Py_None ? nullptr : lengths(as_tensor(a[8], "n_valid"), B, p.dev, "n_valid");
    const int rows = as_int(a[6], "n"), offset = as_int(a[7], "pos_offset");
    if (rows < 0) refuse(PyExc_ValueError, "n is negative");
    g.B = dim_of(B, "B");
    g.Hq = g.Hkv;
    Output ko, vo;
    ko.take(a[9], p, at::kBFloat16, {B, rows, g.Hkv, g.head_dim}, "k_out");
    vo.take(a[10], p, at::kBFloat16, {B, rows, g.Hkv, g.head_dim}, "v_out");
    // (what a new output's memory held before must not show in the rows that are skipped)
    const unsigned zeroed = (ko.made.defined() ? VSD_READ_ZEROED_K : 0u) | (vo.made.defined() ? VSD_READ_ZEROED_V : 0u);
    check(without_gil([&] {
            return g_calls.read(&g, rows, c.k, c.v, c.ks, c.vs, bt, pos, offset, nv, ko.at, vo.at, zeroed,
                                p.stream);
          }),
          "vsd_read_kv_quant");
    return Py_BuildValue("(NN)", ko.result(), vo.result());
  });
}

// verify(q, k_cache, v_cache, k_scale, v_scale, block_table, prefix_len, P_max, scale, row0, row1,
//        logits, partial, score, score_hist, n_sink, n_recent, out, workspace, stream, collect,
//        scored) -> (out, logits, partial, score, score_hist)
PyObject* py_verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 22, [&]() -> PyObject* {
    const at::Tensor& q = as_tensor(a[0], "q");
    need(q, at::kBFloat16, 4, "q");
    const Place p(q, a[19]);
    vsd_geom g;
    const Cache c = cache_of(a + 1, p.dev, &g);
    const int64_t B = q.size(0);
    const int R = dim_of(q.size(1), "R"), P_max = as_int(a[7], "P_max");
    g.B = dim_of(B, "B");
    g.Hq = dim_of(q.size(2), "Hq");
    need(q, at::kBFloat16, {B, R, g.Hq, g.head_dim}, p.dev, "q");
    const int32_t* bt = table_of(as_tensor(a[5], "block_table"), B, p.dev, &g);
    const int32_t* pl = lengths(as_tensor(a[6], "prefix_len"), B, p.dev, "prefix_len");
    const float scale = as_float(a[8]);
    const int row0 = as_int(a[9], "row0"), row1 = a[10] == Py_None ? R - 1 : as_int(a[10], "row1");
    const int n_sink = as_int(a[15], "n_sink"), n_recent = as_int(a[16], "n_recent");
    const bool collect = as_bool(a[20]), scored = as_bool(a[21]);
    size_t bytes = 0;  // (its checks come before anything is allocated)
    check(g_calls.verify_size(&g, R, P_max, &bytes), "vsd_verify_quant_workspace_size");
    Output out, logits, partial, score, hist;
    out.take(a[17], p, at::kBFloat16, q.sizes(), "out");
    if (collect || a[11] != Py_None) logits.take(a[11], p, at::kFloat, {B, 2, g.Hq, P_max}, "logits");
    if (collect || scored || a[12] != Py_None) partial.take(a[12], p, at::kFloat, {B, g.Hkv, P_max}, "partial");
    if (scored) {
      score.take(a[13], p, at::kFloat, {B, P_max}, "score");
      hist.take(a[14], p, at::kInt, {B, kHistBins}, "score_hist");
    }
    const Scratch ws(a[18], bytes, p);
    check(without_gil([&] {
            return g_calls.verify(&g, R, pointer(q), c.k, c.v, c.ks, c.vs, bt, pl, row0, row1, P_max, scale,
                                  static_cast<float*>(logits.at), static_cast<float*>(partial.at),
                                  static_cast<float*>(score.at), static_cast<uint32_t*>(hist.at), n_sink, n_recent,
                                  out.at, ws.at, ws.bytes, p.stream);
          }),
          "vsd_verify_attn_collect_quant");
    return Py_BuildValue("(NNNNN)", out.result(), logits.result(), partial.result(), score.result(), hist.result());
  });
}

// sparse(q, k_cache, v_cache, k_scale, v_scale, block_table, idx, n_sel, tail_start, seq_len,
//        scale, max_tail, out, workspace, stream) -> out
PyObject* py_sparse(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 15, [&]() -> PyObject* {
    const at::Tensor& q = as_tensor(a[0], "q");
    need(q, at::kBFloat16, 3, "q");
    const Place p(q, a[14]);
    vsd_geom g;
    const Cache c = cache_of(a + 1, p.dev, &g);
    const int64_t B = q.size(0);
    g.B = dim_of(B, "B");
    g.Hq = dim_of(q.size(1), "Hq");
    need(q, at::kBFloat16, {B, g.Hq, g.head_dim}, p.dev, "q");
    const int32_t* bt = table_of(as_tensor(a[5], "block_table"), B, p.dev, &g);
    if ((a[6] == Py_None) != (a[7] == Py_None)) refuse(PyExc_ValueError, "idx and n_sel go together");
    int k_max = 0;
    const int32_t *idx = nullptr, *ns = nullptr;
    if (a[6] != Py_None) {
      const at::Tensor& it = as_tensor(a[6], "idx");
      need(it, at::kInt, 2, "idx");
      need(it, at::kInt, {B, it.size(1)}, p.dev, "idx");
      k_max = dim_of(it.size(1), "k_max");
      idx = static_cast<const int32_t*>(pointer(it));
      ns = lengths(as_tensor(a[7], "n_sel"), B, p.dev, "n_sel");
    }
    const int32_t* t0 = lengths(as_tensor(a[8], "tail_start"), B, p.dev, "tail_start");
    const int32_t* t1 = lengths(as_tensor(a[9], "seq_len"), B, p.dev, "seq_len");
    const float scale = as_float(a[10]);
    const int max_tail = as_int(a[11], "max_tail");
    size_t bytes = 0;
    check(g_calls.sparse_size(&g, k_max, max_tail, &bytes), "vsd_sparse_quant_workspace_size");
    Output out;
    out.take(a[12], p, at::kBFloat16, q.sizes(), "out");
    const Scratch ws(a[13], bytes, p);
    check(without_gil([&] {
            return g_calls.sparse(&g, pointer(q), c.k, c.v, c.ks, c.vs, bt, idx, ns, k_max, t0, t1, max_tail, scale,
                                  out.at, ws.at, ws.bytes, p.stream);
          }),
          "vsd_sparse_decode_attn_quant");
    return out.result();
  });
}

// A cache of either type: bf16 rows (no scales), or codes and their scales.
Cache any_cache(PyObject* const* a, int dev, vsd_geom* geom) {
  if (a[2] != Py_None || a[3] != Py_None) return cache_of(a, dev, geom);
  const at::Tensor &k = as_tensor(a[0], "k_cache"), &v = as_tensor(a[1], "v_cache");
  need(k, at::kBFloat16, 4, "k_cache");
  if (k.get_device() != dev) refuse(PyExc_ValueError, "k_cache is on another device");
  need(v, at::kBFloat16, k.sizes(), dev, "v_cache");
  geom->num_blocks = dim_of(k.size(0), "num_blocks");
  geom->Hkv = dim_of(k.size(1), "Hkv");
  geom->page_size = dim_of(k.size(2), "page_size");
  geom->head_dim = dim_of(k.size(3), "head_dim");
  return Cache{pointer(k), pointer(v), nullptr, nullptr};
}

// bf16 rows [B][n][heads][d], each contiguous, by their strides.
vsd_rows strided(const at::Tensor& t, at::IntArrayRef shape, int dev, const char* name) {
  if (t.scalar_type() != at::kBFloat16)
    refuse(PyExc_TypeError, std::string(name) + " must be BFloat16, got " + c10::toString(t.scalar_type()));
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
  if (t.get_device() != dev) refuse(PyExc_ValueError, std::string(name) + " is on another device");
  if (t.stride(3) != 1) refuse(PyExc_ValueError, std::string(name) + "'s rows must be contiguous");
  int64_t s[3];
  for (int i = 0; i < 3; ++i) {
    s[i] = t.size(i) > 1 ? t.stride(i) : 0;  // (a dimension of one element has no stride)
    if (s[i] % 8 != 0)
      refuse(PyExc_ValueError, std::string(name) + "'s strides must be multiples of 8 elements");
  }
  return vsd_rows{pointer(t), s[0], s[1], s[2]};
}

// rope(q, k, v, k_cache, v_cache, k_scale, v_scale, block_table, pos_base, turns, pos_offset,
//      rope_base, n_valid, q_weight, k_weight, eps, interleaved, amplitude, q_out, k_out, stream)
//   -> q_out with a cache; (q_out, k_out) where v and the cache are None
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 21, [&]() -> PyObject* {
    const at::Tensor& q = as_tensor(a[0], "q");
    if (!q.is_cuda()) refuse(PyExc_ValueError, "q must be a CUDA tensor");
    if (q.dim() != 4) refuse(PyExc_ValueError, "q must have 4 dimensions, got shape " + text(q.sizes()));
    const Place p(q, a[20]);
    const int64_t B = q.size(0), rows = q.size(1), d = q.size(3);
    const bool cached = a[3] != Py_None, with_k = cached || a[1] != Py_None;
    vsd_geom g;
    g.B = dim_of(B, "B");
    g.Hq = dim_of(q.size(2), "Hq");
    g.head_dim = dim_of(d, "head_dim");
    g.Hkv = g.Hq;
    Cache c{};
    const int32_t* bt = nullptr;
    if (cached) {
      c = any_cache(a + 3, p.dev, &g);
      bt = table_of(as_tensor(a[7], "block_table"), B, p.dev, &g);
    } else if (with_k) {
      const at::Tensor& k = as_tensor(a[1], "k");
      if (k.dim() != 4) refuse(PyExc_ValueError, "k must have 4 dimensions, got shape " + text(k.sizes()));
      g.Hkv = dim_of(k.size(2), "Hkv");
    }
    const vsd_rows qr = strided(q, {B, rows, g.Hq, g.head_dim}, p.dev, "q");
    vsd_rows kr{}, vr{};
    if (with_k) kr = strided(as_tensor(a[1], "k"), {B, rows, g.Hkv, g.head_dim}, p.dev, "k");
    if (cached) vr = strided(as_tensor(a[2], "v"), {B, rows, g.Hkv, g.head_dim}, p.dev, "v");
    const int32_t* pos = lengths(as_tensor(a[8], "pos_base"), B, p.dev, "pos_base");
    const int32_t* from = a[11] == Py_None ? nullptr : lengths(as_tensor(a[11], "rope_base"), B, p.dev, "rope_base");
    const int32_t* nv = a[12] == Py_None ? nullptr : lengths(as_tensor(a[12], "n_valid"), B, p.dev, "n_valid");
    vsd_rope r{};
    if (a[9] != Py_None) {
      const at::Tensor& t = as_tensor(a[9], "turns");
      need(t, at::kLong, 1, "turns");
      if (t.get_device() != p.dev) refuse(PyExc_ValueError, "turns is on another device");
      if (t.size(0) > INT_MAX / 2) refuse(PyExc_ValueError, "turns is too large");
      r.turns = static_cast<const int64_t*>(pointer(t));
      r.rot_dim = static_cast<int>(2 * t.size(0));
    }
    const auto weight = [&](PyObject* o, const char* name) -> const void* {
      if (o == Py_None) return nullptr;
      const at::Tensor& w = as_tensor(o, name);
      need(w, at::kBFloat16, {d}, p.dev, name);
      return pointer(w);
    };
    r.q_weight = weight(a[13], "q_weight");
    r.k_weight = weight(a[14], "k_weight");
    r.eps = as_float(a[15]);
    r.interleaved = as_bool(a[16]) ? 1 : 0;
    r.amplitude = as_float(a[17]);
    const int nrows = dim_of(rows, "q"), offset = as_int(a[10], "pos_offset");
    Output qo, ko;
    qo.take(a[18], p, at::kBFloat16, {B, rows, g.Hq, g.head_dim}, "q_out");
    if (with_k && !cached) ko.take(a[19], p, at::kBFloat16, {B, rows, g.Hkv, g.head_dim}, "k_out");
    // (what a new output's memory held before must not show in the rows behind n_valid)
    const unsigned zeroed = (qo.made.defined() ? VSD_ROPE_ZEROED_Q : 0u) | (ko.made.defined() ? VSD_ROPE_ZEROED_K : 0u);
    const char* name = !cached ? "vsd_norm_rope" : c.ks ? "vsd_norm_rope_append_kv_quant" : "vsd_norm_rope_append_kv";
    check(without_gil([&] {
            if (!cached)
              return g_calls.rope(&g, nrows, &qr, with_k ? &kr : nullptr, &r, pos, offset, nv, qo.at, ko.at, zeroed,
                                  p.stream);
            if (c.ks == nullptr)
              return g_calls.rope_append(&g, nrows, &qr, &kr, &vr, &r, bt, pos, offset, from, nv, qo.at, zeroed, c.k,
                                         c.v, p.stream);
            return g_calls.rope_append_quant(&g, nrows, &qr, &kr, &vr, &r, bt, pos, offset, from, nv, qo.at, zeroed,
                                             c.k, c.v, c.ks, c.vs, p.stream);
          }),
          name);
    if (cached) return qo.result();
    return Py_BuildValue("(NN)", qo.result(), ko.result());
  });
}

// weights(logits, q, k_cache, k_scale, block_table, prefix_len, weights, scale, rows, stream)
PyObject* py_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&]() -> PyObject* {
    const at::Tensor &q = as_tensor(a[1], "q"), &lg = as_tensor(a[0], "logits");
    need(q, at::kBFloat16, 4, "q");
    const Place p(q, a[9]);
    const at::Tensor& kc = as_tensor(a[2], "k_cache");
    const bool quant = a[3] != Py_None;
    need(kc, quant ? at::kFloat8_e4m3fn : at::kBFloat16, 4, "k_cache");
    if (kc.get_device() != p.dev) refuse(PyExc_ValueError, "k_cache is on another device");
    vsd_geom g;
    const int64_t B = q.size(0);
    const int R = dim_of(q.size(1), "R");
    g.B = dim_of(B, "B");
    g.Hq = dim_of(q.size(2), "Hq");
    g.num_blocks = dim_of(kc.size(0), "num_blocks");
    g.Hkv = dim_of(kc.size(1), "Hkv");
    g.page_size = dim_of(kc.size(2), "page_size");
    g.head_dim = dim_of(kc.size(3), "head_dim");
    need(q, at::kBFloat16, {B, R, g.Hq, g.head_dim}, p.dev, "q");
    const float* ks = nullptr;
    if (quant) {
      const at::Tensor& s = as_tensor(a[3], "k_scale");
      need(s, at::kFloat, {g.num_blocks, g.Hkv}, p.dev, "k_scale");
      ks = static_cast<const float*>(pointer(s));
    }
    const int32_t* bt = table_of(as_tensor(a[4], "block_table"), B, p.dev, &g);
    const int32_t* pl = lengths(as_tensor(a[5], "prefix_len"), B, p.dev, "prefix_len");
    need(lg, at::kFloat, 4, "logits");
    const int C = dim_of(lg.size(1), "logits"), P_max = dim_of(lg.size(3), "P_max");
    need(lg, at::kFloat, {B, C, g.Hq, P_max}, p.dev, "logits");
    const at::Tensor& w = as_tensor(a[6], "weights");
    need(w, at::kFloat, 3, "weights");
    need(w, at::kFloat, {B, g.Hkv, w.size(2)}, p.dev, "weights");
    const int stride = dim_of(w.size(2), "weights");
    if (stride < P_max) refuse(PyExc_ValueError, "weights must have room for every position of logits");
    const float scale = as_float(a[7]);
    int rows[16];
    if (C > 16) refuse(PyExc_ValueError, "logits has more than 16 rows");
    if (a[8] == Py_None) {  // all rows, or a verification's two collected ones (one of them, written twice)
      if (C != R && C != 2) refuse(PyExc_ValueError, "rows are needed for these logits");
      for (int c = 0; c < C; ++c) rows[c] = C == R ? c : c == 0 ? 0 : R == 1 ? -1 : R - 1;
    } else {
      PyObject* seq = PySequence_Fast(a[8], "rows must be a sequence of integers");
      if (seq == nullptr) throw PythonError{};
      const Py_ssize_t count = PySequence_Fast_GET_SIZE(seq);
      bool bad = count != C;
      for (int c = 0; c < C && !bad; ++c) {
        const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, c));
        bad = v < -1 || v >= R || PyErr_Occurred();
        rows[c] = static_cast<int>(v);
      }
      Py_DECREF(seq);
      if (PyErr_Occurred()) throw PythonError{};
      if (bad) refuse(PyExc_ValueError, "rows must name a verify row (or -1) for each row of logits");
    }
    check(without_gil([&] {
            const float* at = static_cast<const float*>(pointer(lg));
            float* to = static_cast<float*>(pointer(w));
            if (quant)
              return g_calls.weights_quant(&g, R, C, rows, at, pointer(q), pointer(kc), ks, bt, pl, P_max, scale, to,
                                           stride, p.stream);
            return g_calls.weights(&g, R, C, rows, at, pointer(q), pointer(kc), bt, pl, P_max, scale, to, stride,
                                   p.stream);
          }),
          quant ? "vsd_accumulate_weights_quant" : "vsd_accumulate_weights");
    Py_INCREF(a[6]);
    return a[6];
  });
}

// compact(k_cache, v_cache, k_scale, v_scale, block_table, dst_table, prefix_len, idx, n_sel,
//         weights, weights_out, stream) -> weights_out
PyObject* py_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 12, [&]() -> PyObject* {
    const at::Tensor& kc = as_tensor(a[0], "k_cache");
    if (!kc.is_cuda()) refuse(PyExc_ValueError, "k_cache must be a CUDA tensor");
    const Place p(kc, a[11]);
    vsd_geom g, other;
    const Cache c = any_cache(a, p.dev, &g);
    const at::Tensor& pt = as_tensor(a[6], "prefix_len");
    need(pt, at::kInt, 1, "prefix_len");
    const int64_t B = pt.size(0);
    const int32_t* pl = lengths(pt, B, p.dev, "prefix_len");
    const int32_t* bt = table_of(as_tensor(a[4], "block_table"), B, p.dev, &g);
    const int32_t* dt = table_of(as_tensor(a[5], "dst_table"), B, p.dev, &other);
    g.B = dim_of(B, "B");
    g.Hq = g.Hkv;
    const at::Tensor &it = as_tensor(a[7], "idx"), &nt = as_tensor(a[8], "n_sel");
    const bool heads = it.dim() == 3;
    need(it, at::kInt, heads ? 3 : 2, "idx");
    const int k = dim_of(it.size(heads ? 2 : 1), "idx");
    if (heads) {
      need(it, at::kInt, {B, g.Hkv, k}, p.dev, "idx");
      need(nt, at::kInt, {B, g.Hkv}, p.dev, "n_sel");
    } else {
      need(it, at::kInt, {B, k}, p.dev, "idx");
      need(nt, at::kInt, {B}, p.dev, "n_sel");
    }
    const float* w = nullptr;
    int ws = 0, wos = 0;
    Output wo;
    if (a[9] != Py_None) {
      const at::Tensor& wt = as_tensor(a[9], "weights");
      need(wt, at::kFloat, 3, "weights");
      need(wt, at::kFloat, {B, g.Hkv, wt.size(2)}, p.dev, "weights");
      w = static_cast<const float*>(pointer(wt));
      ws = dim_of(wt.size(2), "weights");
      if (a[10] != Py_None) {
        const at::Tensor& ot = as_tensor(a[10], "weights_out");
        need(ot, at::kFloat, 3, "weights_out");
        wos = dim_of(ot.size(2), "weights_out");
        if (wos < k) refuse(PyExc_ValueError, "weights_out must have room for every index");
        wo.take(a[10], p, at::kFloat, {B, g.Hkv, wos}, "weights_out");
      } else {
        wos = k;
        wo.take(Py_None, p, at::kFloat, {B, g.Hkv, wos}, "weights_out");
        wo.made.zero_();  // (a list that is refused leaves its row)
      }
      if (wos == 0) w = nullptr;  // (lists of no index: a tensor without elements has no address)
    } else if (a[10] != Py_None) {
      refuse(PyExc_ValueError, "weights_out needs weights");
    }
    check(without_gil([&] {
            const int32_t* idx = static_cast<const int32_t*>(pointer(it));
            const int32_t* ns = static_cast<const int32_t*>(pointer(nt));
            float* to = wos > 0 ? static_cast<float*>(wo.at) : nullptr;
            const int lists = heads ? g.Hkv : 1, dst = other.max_blocks_per_seq;
            if (c.ks != nullptr)
              return g_calls.compact_quant(&g, bt, dt, dst, pl, idx, ns, lists, k, c.k, c.v, c.ks, c.vs, w, ws, to,
                                           wos, p.stream);
            return g_calls.compact(&g, bt, dt, dst, pl, idx, ns, lists, k, c.k, c.v, w, ws, to, wos, p.stream);
          }),
          c.ks ? "vsd_compact_kv_quant" : "vsd_compact_kv");
    return wo.result();
  });
}

// select(partial, prefix_len, k, n_sink, n_recent, idx, n_sel, scores_out, want_scores, stream)
//   -> (idx, n_sel, scores_out)
PyObject* py_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&]() -> PyObject* {
    const at::Tensor &partial = as_tensor(a[0], "partial"), &pl = as_tensor(a[1], "prefix_len");
    need(partial, at::kFloat, 3, "partial");
    const Place p(partial, a[9]);
    const int rows = dim_of(partial.size(0), "n_rows"), Hkv = dim_of(partial.size(1), "Hkv");
    const int P_max = dim_of(partial.size(2), "P_max"), k = as_int(a[2], "k");
    const int n_sink = as_int(a[3], "n_sink"), n_recent = as_int(a[4], "n_recent");
    // (a length for each row, in any shape: [layers, sequences] too)
    need(pl, at::kInt, pl.sizes(), p.dev, "prefix_len");
    if (pl.numel() != rows)
      refuse(PyExc_ValueError, "prefix_len must have a length for each of " + std::to_string(rows) +
                                   " rows, got shape " + text(pl.sizes()));
    Output idx, ns, scores;
    idx.take(a[5], p, at::kInt, {rows, k}, "idx");
    ns.take(a[6], p, at::kInt, {rows}, "n_sel");
    if (as_bool(a[8]) || a[7] != Py_None) scores.take(a[7], p, at::kFloat, {rows, P_max}, "scores_out");
    check(without_gil([&] {
            return g_calls.select(rows, Hkv, static_cast<const float*>(pointer(partial)),
                                  static_cast<const int32_t*>(pointer(pl)), P_max, k, n_sink, n_recent,
                                  static_cast<int32_t*>(idx.at), static_cast<int32_t*>(ns.at),
                                  static_cast<float*>(scores.at), nullptr, 0, p.stream);
          }),
          "vsd_select_topk");
    return Py_BuildValue("(NNN)", idx.result(), ns.result(), scores.result());
  });
}

// attach(error class, addresses of the six library calls)
PyObject* py_attach(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "attach takes an exception class and six addresses");
    return nullptr;
  }
  void* at[6];
  for (int i = 0; i < 6; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_calls.append = reinterpret_cast<decltype(g_calls.append)>(at[0]);
  g_calls.read = reinterpret_cast<decltype(g_calls.read)>(at[1]);
  g_calls.verify_size = reinterpret_cast<decltype(g_calls.verify_size)>(at[2]);
  g_calls.verify = reinterpret_cast<decltype(g_calls.verify)>(at[3]);
  g_calls.sparse_size = reinterpret_cast<decltype(g_calls.sparse_size)>(at[4]);
  g_calls.sparse = reinterpret_cast<decltype(g_calls.sparse)>(at[5]);
  Py_INCREF(a[0]);
  g_calls.error = a[0];
  Py_RETURN_NONE;
}

// attach_more(addresses of the library calls of rows, weights and eviction, and of the selection)
PyObject* py_attach_more(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "attach_more takes eight addresses");
    return nullptr;
  }
  void* at[8];
  for (int i = 0; i < 8; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_calls.rope = reinterpret_cast<decltype(g_calls.rope)>(at[0]);
  g_calls.rope_append = reinterpret_cast<decltype(g_calls.rope_append)>(at[1]);
  g_calls.rope_append_quant = reinterpret_cast<decltype(g_calls.rope_append_quant)>(at[2]);
  g_calls.weights = reinterpret_cast<decltype(g_calls.weights)>(at[3]);
  g_calls.weights_quant = reinterpret_cast<decltype(g_calls.weights_quant)>(at[4]);
  g_calls.compact = reinterpret_cast<decltype(g_calls.compact)>(at[5]);
  g_calls.compact_quant = reinterpret_cast<decltype(g_calls.compact_quant)>(at[6]);
  g_calls.select = reinterpret_cast<decltype(g_calls.select)>(at[7]);
  Py_RETURN_NONE;
}

#define VSD_METHOD(name, fn) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(fn)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {VSD_METHOD("attach", py_attach), VSD_METHOD("append", py_append),
                           VSD_METHOD("read", py_read),     VSD_METHOD("verify", py_verify),
                           VSD_METHOD("sparse", py_sparse), VSD_METHOD("attach_more", py_attach_more),
                           VSD_METHOD("rope", py_rope),     VSD_METHOD("weights", py_weights),
                           VSD_METHOD("compact", py_compact), VSD_METHOD("select", py_select), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

// (built_for: the versions whose headers this was compiled with)
PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&g_module);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", VSD_BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
