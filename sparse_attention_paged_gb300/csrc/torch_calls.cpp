// torch_calls.cpp -- the tensor-level calls around the sparse attention as a
// CPython module over libdsa_indexer.so: tensors to pointers, strides and
// sizes, with the checks of types and shapes that the C ABI cannot make.
// A call through ctypes takes 20 us of host time for its 30 arguments, which
// is several times what the kernels of a small decode step take.
//
// Each function takes its arguments by position (the Python package gives
// them names and defaults), raises ValueError for a tensor of the wrong kind
// and returns the library's status.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "dsa_indexer.h"

namespace {

struct Refused : std::exception {
  std::string what_;
  explicit Refused(std::string w) : what_(std::move(w)) {}
  const char* what() const noexcept override { return what_.c_str(); }
};

void need(bool ok, const char* what) {
  if (!ok) throw Refused(what);
}

// An argument: a tensor, or null for None.
const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + ": a tensor expected");
  return &THPVariable_Unpack(o);
}

thread_local bool all_on_gpu;  // of the call under way

void* ptr(const at::Tensor* t) {
  if (!t) return nullptr;
  all_on_gpu &= t->is_cuda();
  return t->data_ptr();
}

// The given stream (an address), or torch's current one for None.
void* stream_of(PyObject* o) {
  if (o != Py_None) {
    void* s = PyLong_AsVoidPtr(o);
    if (!s && PyErr_Occurred()) throw std::exception();
    return s;
  }
  return c10::cuda::getCurrentCUDAStream().stream();
}

// The library's call, once every argument has been looked at.
template <typename F, typename... A>
int launch(F f, PyObject* stream, A... a) {
  need(all_on_gpu, "expected a CUDA tensor (the library takes device pointers)");
  return f(a..., stream_of(stream));
}

long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::exception();
  return v;
}

int small(PyObject* o) {
  const long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) throw Refused("an integer past 32 bits");
  return (int)v;
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw std::exception();
  return (float)v;
}

int size32(int64_t v) {
  if (v > INT32_MAX) throw Refused("a size past 32 bits");
  return (int)v;
}

const int* ints(const at::Tensor* t, const char* name, int64_t n) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || t->dim() != 1 || !t->is_contiguous() || (n >= 0 && t->size(0) != n))
    throw Refused(std::string(name) + ": contiguous int32 [" + (n >= 0 ? std::to_string(n) : "n") + "] expected");
  return static_cast<const int*>(ptr(t));
}

const float* floats(const at::Tensor* t, const char* name, int64_t a, int64_t b = -1) {
  if (!t) return nullptr;
  const bool shape = b < 0 ? t->dim() == 1 && t->size(0) == a : t->dim() == 2 && t->size(0) == a && t->size(1) == b;
  if (t->scalar_type() != at::kFloat || !shape || !t->is_contiguous())
    throw Refused(std::string(name) + ": contiguous float32 of shape [" + std::to_string(a) +
                  (b < 0 ? "" : ", " + std::to_string(b)) + "] expected");
  return static_cast<const float*>(ptr(t));
}

int* status_word(PyObject* o) {
  const at::Tensor* t = tensor(o, "dev_status");
  if (!t) return nullptr;
  need(t->scalar_type() == at::kInt && t->numel() >= 1, "dev_status: an int32 tensor expected");
  return static_cast<int*>(ptr(t));
}

// A row-strided matrix of bf16 whose rows are contiguous.
void* rows_bf16(const at::Tensor* t, const char* what, int64_t n, int64_t width, long long* stride) {
  need(t && t->scalar_type() == at::kBFloat16 && t->dim() == 2 && (n < 0 || t->size(0) == n) &&
           t->size(1) == width && t->stride(1) == 1,
       what);
  *stride = t->size(0) > 1 ? t->stride(0) : width;
  return ptr(t);
}

struct Pool {
  void* at;
  long long stride;
  int pages;
};

Pool pool_of(const at::Tensor* t, int kv) {
  need(t && t->scalar_type() == at::kByte && t->dim() == 2 && t->stride(1) == 1,
       "cache: uint8 [pages, page bytes] expected");
  need(kv == DSA_KV_FP8_E4M3 || kv == DSA_KV_BF16, "kv_dtype: KV_FP8_E4M3 or KV_BF16");
  need(t->size(1) >= (kv == DSA_KV_BF16 ? 73728 : 41984), "cache: rows shorter than a page");
  return Pool{ptr(t), t->size(0) > 1 ? t->stride(0) : t->size(1), size32(t->size(0))};
}

struct Table {
  const int* at;
  long long stride;
  int W;
};

// An int32 [rows, W] table, or one row [W] or [1, W] that all share.
Table table_of(const at::Tensor* t, int64_t rows) {
  need(t && t->scalar_type() == at::kInt && (t->dim() == 1 || t->dim() == 2) && t->stride(t->dim() - 1) == 1,
       "block_table: int32 [rows, W] expected");
  const int W = size32(t->size(t->dim() - 1));
  if (t->dim() == 1 || t->size(0) == 1) return Table{static_cast<const int*>(ptr(t)), 0, W};
  need(t->size(0) == rows, "block_table: one row, or one per request");
  return Table{static_cast<const int*>(ptr(t)), t->stride(0), W};
}

// Every CUDA tensor among the arguments is on the current device, whose
// streams and SM count the library uses: an address of another device would
// fault in a kernel.  (Tensors of the host are refused by `launch`.)
void one_device(PyObject* const* a, Py_ssize_t n) {
  int first = -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    // numbers and None first: the general test of a type takes 40 ns
    if (a[i] == Py_None || PyLong_Check(a[i]) || PyFloat_Check(a[i]) || !THPVariable_Check(a[i])) continue;
    const at::Device d = THPVariable_Unpack(a[i]).device();
    if (!d.is_cuda()) continue;
    need(first < 0 || d.index() == first, "the tensors are on more than one CUDA device");
    first = d.index();
  }
  need(first < 0 || first == c10::cuda::current_device(),
       "the tensors are not on the current CUDA device (torch.cuda.set_device, or `with torch.cuda.device`)");
}

template <typename F>
PyObject* guarded(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, n);
    return nullptr;
  }
  try {
    all_on_gpu = true;
    one_device(a, n);
    return PyLong_FromLong(f());
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// q, k, positions, table, rot_offset, interleaved, norm, q_weight, k_weight,
// q_bias, k_bias, eps, q_out, k_out, dev_status, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 16, [&] {
    const at::Tensor *q = tensor(a[0], "q"), *k = tensor(a[1], "k");
    const at::Tensor *qo = tensor(a[12], "q_out"), *ko = tensor(a[13], "k_out");
    need(q && q->dim() == 3, "q: [T, Hq, D] expected");
    const int64_t T = q->size(0), D = q->size(2);
    const auto type = q->scalar_type();
    const int dtype = type == at::kBFloat16 ? DSA_BF16 : type == at::kHalf ? DSA_FP16 : type == at::kFloat ? DSA_FP32 : -1;
    need(dtype >= 0, "q: bfloat16, float16 or float32 expected");
    need(q->stride(2) == 1, "q: the last dimension must be contiguous");
    need(qo && qo->sizes() == q->sizes() && qo->scalar_type() == type && qo->stride(2) == 1, "q_out: like q");
    int64_t Hk = 0, kt = 0, kh = 0, kot = 0, koh = 0;
    if (k) {
      need(k->dim() == 3 && k->size(0) == T && k->size(2) == D && k->scalar_type() == type && k->stride(2) == 1,
           "k: [T, Hk, D] of q's type");
      need(ko && ko->sizes() == k->sizes() && ko->scalar_type() == type && ko->stride(2) == 1, "k_out: like k");
      Hk = k->size(1), kt = k->stride(0), kh = k->stride(1), kot = ko->stride(0), koh = ko->stride(1);
    }
    const int* positions = ints(tensor(a[2], "positions"), "positions", T);
    const float* table = nullptr;
    int max_pos = 0, rot = 0;
    if (positions) {
      const at::Tensor* t = tensor(a[3], "table");
      need(t && t->dim() == 2, "positions need a table [max_pos, rot_dims]");
      max_pos = size32(t->size(0)), rot = size32(t->size(1));
      table = floats(t, "table", max_pos, rot);
    }
    const float* qw = floats(tensor(a[7], "q_weight"), "q_weight", D);
    const float* kw = floats(tensor(a[8], "k_weight"), "k_weight", D);
    const float* qb = floats(tensor(a[9], "q_bias"), "q_bias", D);
    const float* kb = floats(tensor(a[10], "k_bias"), "k_bias", D);
    return launch(dsa_qk_norm_rope, a[15], ptr(q), q->stride(0), q->stride(1), size32(q->size(1)), ptr(k), kt, kh, size32(Hk),
                            size32(T), size32(D), dtype, small(a[6]), qw, kw, qb, kb, real(a[11]), positions, table,
                            max_pos, rot, small(a[4]), small(a[5]), ptr(qo), qo->stride(0), qo->stride(1),
                            k ? ptr(ko) : nullptr, kot, koh, status_word(a[14]));
  });
}

// latent, rope, slot_mapping, cache, kv_dtype, norm_weight, eps, positions,
// rope_table, interleaved, dev_status, stream
PyObject* latent_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 12, [&] {
    long long ls, rs;
    const at::Tensor* latent = tensor(a[0], "latent");
    void* c = rows_bf16(latent, "latent: bfloat16 [n, 512], rows contiguous", -1, 512, &ls);
    const int64_t rows = latent->size(0);
    void* r = rows_bf16(tensor(a[1], "rope"), "rope: bfloat16 [n, 64], rows contiguous", rows, 64, &rs);
    const int* slots = ints(tensor(a[2], "slot_mapping"), "slot_mapping", rows);
    const int kv = small(a[4]);
    const Pool pool = pool_of(tensor(a[3], "cache"), kv);
    const float* w = floats(tensor(a[5], "norm_weight"), "norm_weight", 512);
    const int* positions = ints(tensor(a[7], "positions"), "positions", rows);
    const float* table = nullptr;
    int max_pos = 0;
    if (positions) {
      const at::Tensor* t = tensor(a[8], "rope_table");
      need(t && t->dim() == 2, "positions need a rope_table [max_pos, 64]");
      max_pos = size32(t->size(0));
      table = floats(t, "rope_table", max_pos, 64);
    }
    return launch(dsa_latent_store, a[11], c, ls, r, rs, size32(rows), 512, 64, w, real(a[6]), positions, table, max_pos, small(a[9]),
                            slots, pool.at, pool.stride, pool.pages, kv, 64, status_word(a[10]));
  });
}

// cache, kv_dtype, block_table, cu_rows, n, starts, out, dev_status, stream
PyObject* latent_load(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 9, [&] {
    const at::Tensor* cu = tensor(a[3], "cu_rows");
    const int* cu_rows = ints(cu, "cu_rows", -1);
    need(cu_rows && cu->size(0) >= 1, "cu_rows: int32 [requests + 1] expected");
    const int64_t req = cu->size(0) - 1;
    const int* starts = ints(tensor(a[5], "starts"), "starts", req);
    const int rows = small(a[4]), kv = small(a[1]);
    long long stride;
    void* out = rows_bf16(tensor(a[6], "out"), "out: bfloat16 [n, 576], rows contiguous", rows, 576, &stride);
    const Pool pool = pool_of(tensor(a[0], "cache"), kv);
    const Table t = table_of(tensor(a[2], "block_table"), req);
    return launch(dsa_latent_load, a[8], pool.at, pool.stride, pool.pages, kv, 64, t.at, t.stride, t.W, starts, cu_rows, size32(req),
                           rows, 512, 64, out, stride, status_word(a[7]));
  });
}

// q_latent, q_rope, cache, kv_dtype, block_table, seqlens, scale, idx, out,
// lse, workspace, dev_status, stream
PyObject* latent_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 13, [&] {
    const at::Tensor *ql = tensor(a[0], "q_latent"), *qr = tensor(a[1], "q_rope"), *idx = tensor(a[7], "idx");
    const at::Tensor *out = tensor(a[8], "out"), *ws = tensor(a[10], "workspace");
    need(ql && ql->scalar_type() == at::kBFloat16 && ql->dim() == 3 && ql->size(2) == 512 && ql->stride(2) == 1,
         "q_latent: bfloat16 [rows, H, 512]");
    const int64_t rows = ql->size(0), H = ql->size(1);
    need(qr && qr->scalar_type() == at::kBFloat16 && qr->dim() == 3 && qr->size(0) == rows && qr->size(1) == H &&
             qr->size(2) == 64 && qr->stride(2) == 1,
         "q_rope: bfloat16 [rows, H, 64]");
    const int kv = small(a[3]);
    const int* seqlens = ints(tensor(a[5], "seqlens"), "seqlens", rows);
    int64_t k = 0, idx_stride = 0;
    if (idx) {
      need(idx->scalar_type() == at::kInt && idx->dim() == 2 && idx->size(0) == rows && idx->stride(1) == 1,
           "idx: int32 [rows, k]");
      // an empty tensor has no address, and no address stands for "no lists"
      need(idx->size(1) > 0 || rows == 0, "idx: lists of at least one entry (None: every position)");
      k = idx->size(1), idx_stride = rows > 1 ? idx->stride(0) : k;
    }
    need(out && out->scalar_type() == at::kBFloat16 && out->dim() == 3 && out->sizes() == ql->sizes() &&
             out->stride(2) == 1,
         "out: bfloat16 [rows, H, 512]");
    const float* lse = floats(tensor(a[9], "lse"), "lse", rows, H);
    need(ws && ws->scalar_type() == at::kFloat && ws->is_contiguous(), "workspace: contiguous float32");
    const Pool pool = pool_of(tensor(a[2], "cache"), kv);
    const Table t = table_of(tensor(a[4], "block_table"), rows);
    return launch(dsa_latent_attention, a[12], ptr(ql), ql->stride(0), ql->stride(1), ptr(qr), qr->stride(0), qr->stride(1),
                                size32(rows), size32(H), 512, 64, real(a[6]), pool.at, pool.stride, pool.pages, kv, 64,
                                t.at, t.stride, t.W, seqlens, static_cast<const int*>(ptr(idx)), idx_stride, size32(k),
                                ptr(out), out->stride(0), out->stride(1), const_cast<float*>(lse),
                                static_cast<float*>(ptr(ws)), ws->numel(), status_word(a[11]));
  });
}

// ---- the paged cache of keys and values with grouped heads ----

int* writable(const int* p) { return const_cast<int*>(p); }

int type16(const at::Tensor* t, const char* what) {
  need(t && (t->scalar_type() == at::kBFloat16 || t->scalar_type() == at::kHalf), what);
  return t->scalar_type() == at::kHalf ? DSA_FP16 : DSA_BF16;
}

// [n, heads, D] of 16-bit values, a head's values adjacent.
struct Heads {
  void* at;
  int64_t n, heads, dim;
  long long row, head;
  int dtype;
};

Heads heads_of(const at::Tensor* t, const char* what) {
  const int dtype = type16(t, what);
  need(t->dim() == 3 && t->stride(2) == 1, what);
  // a dimension of one has any stride
  return Heads{ptr(t), t->size(0), t->size(1), t->size(2), t->size(0) > 1 ? t->stride(0) : t->size(2),
               t->size(1) > 1 ? t->stride(1) : t->size(2), dtype};
}

// A cache [pages, 64, heads, D].
struct Cache {
  void* at;
  long long page, slot, head;
  int64_t pages, heads, dim;
  int kv;
};

Cache cache_of(const at::Tensor* t, const char* what) {
  need(t && t->dim() == 4 && t->size(1) == 64 && t->stride(3) == 1, what);
  const auto type = t->scalar_type();
  const int kv = type == at::kBFloat16 ? DSA_KV_BF16 : type == at::kHalf ? DSA_KV_FP16 : type == at::kFloat8_e4m3fn ? DSA_KV_FP8_E4M3 : -1;
  need(kv >= 0, what);
  return Cache{ptr(t), t->stride(0), t->stride(1), t->stride(2), t->size(0), t->size(2), t->size(3), kv};
}

const float* scales_of(const at::Tensor* t, const Cache& c, const char* what) {
  if (c.kv != DSA_KV_FP8_E4M3) {
    need(!t, "k_scale, v_scale: for an fp8 cache only");
    return nullptr;
  }
  need(t && t->scalar_type() == at::kFloat && t->dim() == 3 && t->size(0) == c.pages && t->size(1) == c.heads &&
           t->size(2) == 64 && t->is_contiguous(),
       what);
  return static_cast<const float*>(ptr(t));
}

constexpr const char* kKCache = "k_cache: [pages, 64, Hkv, D] of bfloat16, float16 or float8_e4m3fn, values adjacent";
constexpr const char* kVCache = "v_cache: like k_cache";
constexpr const char* kKScale = "k_scale: contiguous float32 [pages, Hkv, 64] for an fp8 cache";
constexpr const char* kVScale = "v_scale: contiguous float32 [pages, Hkv, 64] for an fp8 cache";

Cache values_of(const at::Tensor* t, const Cache& k) {
  const Cache v = cache_of(t, kVCache);
  need(v.kv == k.kv && v.pages == k.pages && v.heads == k.heads && v.dim == k.dim, kVCache);
  return v;
}

// lengths, new_tokens, free_pages, block_table, n, slots, positions, seqlens,
// cu_rows, used, dev_status, stream
PyObject* request_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 12, [&] {
    const at::Tensor *lengths = tensor(a[0], "lengths"), *free_pages = tensor(a[2], "free_pages");
    const int* held = ints(lengths, "lengths", -1);
    need(lengths, "lengths: int32 [requests] expected");
    const int64_t req = lengths->size(0);
    const at::Tensor* fresh = tensor(a[1], "new_tokens");
    need(fresh && free_pages, "new_tokens and free_pages: int32 tensors expected");
    const int* fresh_at = ints(fresh, "new_tokens", req);
    const int* pages = ints(free_pages, "free_pages", -1);
    const at::Tensor* t = tensor(a[3], "block_table");
    need(t && t->dim() == 2 && t->size(0) == req, "block_table: int32 [requests, W] expected");
    const Table table = table_of(t, req);
    const int rows = small(a[4]);
    const at::Tensor* slots = tensor(a[5], "slots");
    need(slots, "slots: int32 [n] expected");
    return launch(dsa_request_slots, a[11], held, fresh_at, size32(req), pages, size32(free_pages->size(0)),
                  writable(table.at), table.stride, table.W, 64, rows, writable(ints(slots, "slots", rows)),
                  writable(ints(tensor(a[6], "positions"), "positions", rows)),
                  writable(ints(tensor(a[7], "seqlens"), "seqlens", req)),
                  writable(ints(tensor(a[8], "cu_rows"), "cu_rows", req + 1)),
                  writable(ints(tensor(a[9], "used"), "used", 1)), status_word(a[10]));
  });
}

// k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, dev_status, stream
PyObject* kv_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 9, [&] {
    const Heads k = heads_of(tensor(a[0], "k"), "k: bfloat16 or float16 [n, Hkv, D], values adjacent");
    const Heads v = heads_of(tensor(a[1], "v"), "v: like k");
    need(v.n == k.n && v.heads == k.heads && v.dim == k.dim && v.dtype == k.dtype, "v: like k");
    const Cache kc = cache_of(tensor(a[3], "k_cache"), kKCache), vc = values_of(tensor(a[4], "v_cache"), kc);
    need(kc.heads == k.heads && kc.dim == k.dim, "k_cache: k's heads and values");
    const at::Tensor* slot_tensor = tensor(a[2], "slot_mapping");
    need(slot_tensor, "slot_mapping: int32 [n] expected");
    const int* slots = ints(slot_tensor, "slot_mapping", k.n);
    const float* ks = scales_of(tensor(a[5], "k_scale"), kc, kKScale);
    const float* vs = scales_of(tensor(a[6], "v_scale"), vc, kVScale);
    return launch(dsa_kv_store, a[8], k.at, k.row, k.head, v.at, v.row, v.head, size32(k.n), size32(k.heads), size32(k.dim),
                  k.dtype, slots, kc.at, kc.page, kc.slot, kc.head, vc.at, vc.page, vc.slot, vc.head,
                  const_cast<float*>(ks), const_cast<float*>(vs), size32(kc.pages), kc.kv, 64, status_word(a[7]));
  });
}

// bounds and their scales, for `pages` pages of `heads` heads of `dim` values
signed char* bounds_of(const at::Tensor* t, int64_t pages, int64_t heads, int64_t dim) {
  need(t && t->scalar_type() == at::kChar && t->dim() == 4 && t->size(0) == pages && t->size(1) == heads &&
           t->size(2) == 2 && t->size(3) == dim && t->is_contiguous(),
       "bounds: contiguous int8 [pages, Hkv, 2, D]");
  return static_cast<signed char*>(ptr(t));
}

// k_cache, block_table, starts, seqlens, max_tokens, bounds, bound_scale,
// k_scale, dev_status, stream
PyObject* block_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 10, [&] {
    const Cache c = cache_of(tensor(a[0], "k_cache"), kKCache);
    const at::Tensor* lens = tensor(a[3], "seqlens");
    need(lens, "seqlens: int32 [requests] expected");
    const int* seqlens = ints(lens, "seqlens", -1);
    const int64_t req = lens->size(0);
    const int* starts = ints(tensor(a[2], "starts"), "starts", req);
    const Table t = table_of(tensor(a[1], "block_table"), req);
    signed char* bounds = bounds_of(tensor(a[5], "bounds"), c.pages, c.heads, c.dim);
    const at::Tensor* scale = tensor(a[6], "bound_scale");
    need(scale, "bound_scale: float32 [pages, Hkv] expected");
    const float* unit = floats(scale, "bound_scale", c.pages, c.heads);
    const float* ks = scales_of(tensor(a[7], "k_scale"), c, kKScale);
    return launch(dsa_block_bounds, a[9], c.at, c.page, c.slot, c.head, ks, size32(c.pages), c.kv, size32(c.heads),
                  size32(c.dim), 64, t.at, t.stride, t.W, starts, seqlens, size32(req), small(a[4]), bounds,
                  const_cast<float*>(unit), status_word(a[8]));
  });
}

// q, bounds, bound_scale, block_table, seqlens, k, first, last, out,
// dev_status, stream
PyObject* block_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 11, [&] {
    const Heads q = heads_of(tensor(a[0], "q"), "q: bfloat16 or float16 [rows, Hq, D], values adjacent");
    const at::Tensor* b = tensor(a[1], "bounds");
    need(b && b->dim() == 4, "bounds: contiguous int8 [pages, Hkv, 2, D]");
    const int64_t pages = b->size(0), heads = b->size(1);
    signed char* bounds = bounds_of(b, pages, heads, q.dim);
    const at::Tensor* scale = tensor(a[2], "bound_scale");
    need(scale, "bound_scale: float32 [pages, Hkv] expected");
    const float* unit = floats(scale, "bound_scale", pages, heads);
    const at::Tensor* lens = tensor(a[4], "seqlens");
    need(lens, "seqlens: int32 [rows] expected");
    const int* seqlens = ints(lens, "seqlens", q.n);
    const Table t = table_of(tensor(a[3], "block_table"), q.n);
    const int k = small(a[5]);
    const at::Tensor* out = tensor(a[8], "out");
    need(out && out->scalar_type() == at::kInt && out->dim() == 3 && out->size(0) == q.n && out->size(1) == heads &&
             out->size(2) == k && out->is_contiguous(),
         "out: contiguous int32 [rows, Hkv, k]");
    return launch(dsa_block_select, a[10], q.at, q.row, q.head, size32(q.n), size32(q.heads), size32(heads), size32(q.dim),
                  q.dtype, bounds, unit, size32(pages), t.at, t.stride, t.W, 64, seqlens, k, small(a[6]), small(a[7]),
                  static_cast<int*>(ptr(out)), status_word(a[9]));
  });
}

// q, k_cache, v_cache, block_table, seqlens, scale, blocks, k_scale, v_scale,
// out, lse, workspace, dev_status, stream
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 14, [&] {
    const Heads q = heads_of(tensor(a[0], "q"), "q: bfloat16 or float16 [rows, Hq, D], values adjacent");
    const Cache kc = cache_of(tensor(a[1], "k_cache"), kKCache), vc = values_of(tensor(a[2], "v_cache"), kc);
    need(kc.dim == q.dim, "k_cache: q's values per head");
    const at::Tensor* lens = tensor(a[4], "seqlens");
    need(lens, "seqlens: int32 [rows] expected");
    const int* seqlens = ints(lens, "seqlens", q.n);
    const at::Tensor* b = tensor(a[6], "blocks");
    int64_t k = 0, b_row = 0, b_head = 0;
    if (b) {
      need(b->scalar_type() == at::kInt && b->dim() == 3 && b->size(0) == q.n && b->size(1) == kc.heads &&
               (b->stride(2) == 1 || b->size(2) == 1),
           "blocks: int32 [rows, Hkv, k]");
      // an empty tensor has no address, and no address stands for "no lists"
      need(b->size(2) > 0 || q.n == 0, "blocks: lists of at least one entry (None: every page)");
      k = b->size(2), b_row = b->stride(0), b_head = b->stride(1);
    }
    const Heads out = heads_of(tensor(a[9], "out"), "out: like q");
    need(out.n == q.n && out.heads == q.heads && out.dim == q.dim && out.dtype == q.dtype, "out: like q");
    const float* lse = floats(tensor(a[10], "lse"), "lse", q.n, q.heads);
    const at::Tensor* ws = tensor(a[11], "workspace");
    need(ws && ws->scalar_type() == at::kFloat && ws->is_contiguous(), "workspace: contiguous float32");
    const Table t = table_of(tensor(a[3], "block_table"), q.n);
    const float* ks = scales_of(tensor(a[7], "k_scale"), kc, kKScale);
    const float* vs = scales_of(tensor(a[8], "v_scale"), vc, kVScale);
    return launch(dsa_paged_attention, a[13], q.at, q.row, q.head, size32(q.n), size32(q.heads), size32(kc.heads),
                  size32(q.dim), q.dtype, real(a[5]), kc.at, kc.page, kc.slot, kc.head, vc.at, vc.page, vc.slot, vc.head,
                  ks, vs, size32(kc.pages), kc.kv, 64, t.at, t.stride, t.W, seqlens,
                  static_cast<const int*>(ptr(b)), b_row, b_head, size32(k), out.at, out.row, out.head,
                  const_cast<float*>(lse), static_cast<float*>(ptr(ws)), ws->numel(), status_word(a[12]));
  });
}

PyMethodDef methods[] = {
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, nullptr},
    {"latent_store", (PyCFunction)(void (*)(void))latent_store, METH_FASTCALL, nullptr},
    {"latent_load", (PyCFunction)(void (*)(void))latent_load, METH_FASTCALL, nullptr},
    {"latent_attention", (PyCFunction)(void (*)(void))latent_attention, METH_FASTCALL, nullptr},
    {"request_slots", (PyCFunction)(void (*)(void))request_slots, METH_FASTCALL, nullptr},
    {"kv_store", (PyCFunction)(void (*)(void))kv_store, METH_FASTCALL, nullptr},
    {"block_bounds", (PyCFunction)(void (*)(void))block_bounds, METH_FASTCALL, nullptr},
    {"block_select", (PyCFunction)(void (*)(void))block_select, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void (*)(void))paged_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dsa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dsa_torch(void) { return PyModule_Create(&module); }
