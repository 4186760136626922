// Native half of the Python binding of the serving operators: checks every argument and calls the C ABI.
//
// The checks are those of the rest of the binding (a CUDA tensor on the current device, contiguous, of the shape and
// type the call expects).  In Python they took 5 to 11 us a call, two or three times what the smallest of these kernels
// takes; here they take under 1 us.  The functions take every argument by position and return the call's status; the
// functions of the package give them names, defaults and documentation, and raise on a status that is not 0.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "hata.h"

namespace {

struct Raised {};  // a Python exception is set

[[noreturn]] void raise(PyObject* type, const std::string& message) {
  PyErr_SetString(type, message.c_str());
  throw Raised{};
}

std::string sizes_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

// The arguments of one call.
class Args {
 public:
  Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : args_(args) {
    if (n != want) raise(PyExc_TypeError, "expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
    Py_buffer view;
    if (PyObject_GetBuffer(args[0], &view, PyBUF_SIMPLE) != 0) throw Raised{};
    const bool ok = view.len == (Py_ssize_t)sizeof(hata_dims_t);
    if (ok) d = *static_cast<const hata_dims_t*>(view.buf);
    PyBuffer_Release(&view);
    if (!ok) raise(PyExc_TypeError, "dims must be a Dims");
    type = d.dtype == HATA_F32 ? at::kFloat : at::kBFloat16;
  }

  hata_dims_t d;
  at::ScalarType type;  // of q, K, V and outputs

  bool none(int i) const { return args_[i] == Py_None; }

  const at::Tensor& tensor(int i, const char* name) {
    if (none(i)) raise(PyExc_ValueError, std::string(name) + " is required");
    if (!THPVariable_Check(args_[i])) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(args_[i]);
  }

  // a tensor of this type on the current device, of any layout
  const at::Tensor& placed(int i, const char* name, at::ScalarType t) {
    const at::Tensor& x = tensor(i, name);
    if (!x.is_cuda() || x.get_device() != device())
      raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor on the current device (got " + x.device().str() + ")");
    if (x.scalar_type() != t)
      raise(PyExc_TypeError, std::string(name) + " must be torch." + python_name(t) + " (got torch." +
                                 python_name(x.scalar_type()) + ")");
    return x;
  }

  void* ptr(int i, const char* name, std::initializer_list<int64_t> shape, at::ScalarType t) {
    const at::Tensor& x = placed(i, name, t);
    const at::IntArrayRef want(shape.begin(), shape.size());
    if (x.sizes() != want)
      raise(PyExc_ValueError, std::string(name) + " must have shape " + sizes_of(want) + " (got " + sizes_of(x.sizes()) + ")");
    if (!x.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    return x.data_ptr();
  }
  void* maybe(int i, const char* name, std::initializer_list<int64_t> shape, at::ScalarType t) {
    return none(i) ? nullptr : ptr(i, name, shape, t);
  }
  int32_t* ints(int i, const char* name, std::initializer_list<int64_t> shape) {
    return static_cast<int32_t*>(ptr(i, name, shape, at::kInt));
  }
  int32_t* maybe_ints(int i, const char* name, std::initializer_list<int64_t> shape) {
    return none(i) ? nullptr : ints(i, name, shape);
  }

  long long integer(int i) {
    const long long v = PyLong_AsLongLong(args_[i]);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
  }
  int small(int i, const char* name) {
    const long long v = integer(i);
    if (v < INT32_MIN || v > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
    return (int)v;
  }
  double number(int i) {
    const double v = PyFloat_AsDouble(args_[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
  }
  bool truth(int i) {
    const int v = PyObject_IsTrue(args_[i]);
    if (v < 0) throw Raised{};
    return v != 0;
  }

  void* workspace(int i, size_t* bytes) {
    const at::Tensor& x = placed(i, "workspace", at::kByte);
    if (!x.is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
    *bytes = (size_t)x.numel();
    return x.data_ptr();
  }
  // None: the current stream of the current device; else a stream's handle
  void* stream(int i) {
    if (none(i)) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device()).stream();
    void* s = PyLong_AsVoidPtr(args_[i]);
    if (!s && PyErr_Occurred()) throw Raised{};
    return s;
  }

 private:
  PyObject* const* args_;
  int device_ = -1;

  int device() {  // asked for only once a CUDA tensor is there
    if (device_ < 0) device_ = c10::cuda::current_device();
    return device_;
  }
  static std::string python_name(at::ScalarType t) {
    switch (t) {
      case at::kFloat: return "float32";
      case at::kBFloat16: return "bfloat16";
      case at::kInt: return "int32";
      case at::kByte: return "uint8";
      case at::kShort: return "int16";
      case at::kDouble: return "float64";
      case at::kHalf: return "float16";
      case at::kLong: return "int64";
      default: return c10::toString(t);
    }
  }
};

// The interpreter lock is let go while a call is enqueued.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// A cache: [B][Hkv][max_seq][d], or (table given) pools [n_blocks][Hkv][bs][d] and their block table.
struct Cache {
  void *K, *V;
  int32_t* table = nullptr;
  int bs = 0, n_blocks = 0;
  bool paged;
};
Cache cache(Args& a, int k, int v, int table, int block, bool paged) {
  const hata_dims_t& d = a.d;
  Cache c;
  c.paged = paged;
  if (!paged) {
    c.K = a.ptr(k, "K", {d.batch, d.n_kv_heads, d.max_seq, d.head_dim}, a.type);
    c.V = a.ptr(v, "V", {d.batch, d.n_kv_heads, d.max_seq, d.head_dim}, a.type);
    return c;
  }
  c.bs = a.small(block, "block_size");
  const at::Tensor& pool = a.tensor(k, "K_pool");
  if (pool.dim() != 4) raise(PyExc_ValueError, "K_pool must be a tensor [n_blocks][Hkv][block_size][d]");
  if (pool.size(0) > INT32_MAX) raise(PyExc_ValueError, "K_pool has too many blocks");
  c.n_blocks = (int)pool.size(0);
  c.K = a.ptr(k, "K_pool", {c.n_blocks, d.n_kv_heads, c.bs, d.head_dim}, a.type);
  c.V = a.ptr(v, "V_pool", {c.n_blocks, d.n_kv_heads, c.bs, d.head_dim}, a.type);
  c.table = a.ints(table, "block_table", {d.batch, c.bs > 0 ? ((int64_t)d.max_seq + c.bs - 1) / c.bs : 0});
  return c;
}

// Codes of a cache's slots: packed 32-bit words, or one 16-bit code per slot; null for None.
void* codes(Args& a, int i, int64_t lead, int64_t slots) {
  if (a.none(i)) return nullptr;
  const hata_dims_t& d = a.d;
  const at::ScalarType t = a.tensor(i, "codes").scalar_type();
  const bool wide = d.hash_bits != 16;
  if (wide ? (t != at::kInt && t != at::kUInt32) : (t != at::kShort && t != at::kUInt16))
    raise(PyExc_TypeError, wide ? "codes must be int32 or uint32 tensors holding the packed words"
                                : "16-bit codes must be int16 or uint16 tensors, one code per token");
  if (wide) return a.ptr(i, "codes", {lead, d.n_kv_heads, slots, d.hash_bits / 32}, t);
  return a.ptr(i, "codes", {lead, d.n_kv_heads, slots}, t);
}

// [B][n_tok][heads][d] with each token's heads side by side and its tokens at one stride
void* token_rows(Args& a, int i, const char* name, int heads, int64_t n_tok, long long* stride) {
  const int64_t B = a.d.batch, D = a.d.head_dim;
  const at::Tensor& x = a.placed(i, name, a.type);
  const int64_t shape[4] = {B, n_tok, heads, D};
  if (x.sizes() != at::IntArrayRef(shape, 4))
    raise(PyExc_ValueError, std::string(name) + " must have shape " + sizes_of(at::IntArrayRef(shape, 4)) + " (got " +
                                sizes_of(x.sizes()) + ")");
  const at::IntArrayRef s = x.strides();
  if (s[3] != 1 || (heads > 1 && s[2] != D) || (n_tok > 1 && B > 1 && s[0] != n_tok * s[1]))
    raise(PyExc_ValueError, std::string(name) +
                                " must hold each token's heads side by side and its tokens at one stride (strides " +
                                sizes_of(s) + ")");
  *stride = n_tok > 1 ? s[1] : B > 1 ? s[0] : heads * D;
  return x.data_ptr();
}

// dims, q_in, k_in, v_in, q_weight, k_weight, eps, table, interleaved, n_new, positions, seq_lens, q_out, K, V,
// block_table, block_size, workspace, stream, paged
hata_status_t norm_rope(Args& a) {
  const hata_dims_t& d = a.d;
  const at::Tensor& q = a.tensor(1, "q_in");
  if (q.dim() != 4) raise(PyExc_ValueError, "q_in must be a tensor [B][n_tok][Hq][d]");
  const int64_t T = q.size(1);
  if (T > INT32_MAX) raise(PyExc_ValueError, "q_in has too many tokens");
  long long qs, ks, vs;
  void* qi = token_rows(a, 1, "q_in", d.n_q_heads, T, &qs);
  void* ki = token_rows(a, 2, "k_in", d.n_kv_heads, T, &ks);
  void* vi = token_rows(a, 3, "v_in", d.n_kv_heads, T, &vs);
  const float* wq = static_cast<const float*>(a.maybe(4, "q_weight", {d.head_dim}, at::kFloat));
  const float* wk = static_cast<const float*>(a.maybe(5, "k_weight", {d.head_dim}, at::kFloat));
  const float* table = nullptr;
  int n_pos = 0, rot = 0;
  if (!a.none(7)) {
    const at::Tensor& t = a.tensor(7, "table");
    if (t.dim() != 3 || t.size(0) > INT32_MAX || t.size(2) > 1024)
      raise(PyExc_ValueError, "table must be a tensor [n_pos][2][rot_dim / 2]");
    n_pos = (int)t.size(0);
    rot = 2 * (int)t.size(2);
    table = static_cast<const float*>(a.ptr(7, "table", {n_pos, 2, rot / 2}, at::kFloat));
  }
  const int32_t* n_new = a.maybe_ints(9, "n_new", {d.batch});
  const int32_t* positions = a.maybe_ints(10, "positions", {d.batch, T});
  const int32_t* lens = a.ints(11, "seq_lens", {d.batch});
  void* out = a.ptr(12, "q_out", {d.batch, d.n_q_heads, T, d.head_dim}, a.type);
  const Cache c = cache(a, 13, 14, 15, 16, a.truth(19));
  size_t bytes;
  void* ws = a.workspace(17, &bytes);
  const float eps = (float)a.number(6);
  const int inter = a.truth(8);
  void* st = a.stream(18);
  Unlocked unlocked;
  if (c.paged)
    return hata_norm_rope_paged(&d, (int)T, qi, qs, ki, ks, vi, vs, wq, wk, eps, table, n_pos, rot, inter, n_new, positions,
                                lens, out, c.K, c.V, c.table, c.bs, c.n_blocks, ws, bytes, st);
  return hata_norm_rope(&d, (int)T, qi, qs, ki, ks, vi, vs, wq, wk, eps, table, n_pos, rot, inter, n_new, positions, lens,
                        out, c.K, c.V, ws, bytes, st);
}

// dims, q, K, V, block_table, block_size, seq_lens, window, n_sink, scale, out, workspace, stream, paged
hata_status_t window_decode(Args& a) {
  const hata_dims_t& d = a.d;
  const void* q = a.ptr(1, "q", {d.batch, d.n_q_heads, d.head_dim}, a.type);
  const Cache c = cache(a, 2, 3, 4, 5, a.truth(13));
  const int32_t* lens = a.ints(6, "seq_lens", {d.batch});
  const int window = a.small(7, "window"), sink = a.small(8, "n_sink");
  const float scale = (float)a.number(9);
  void* out = a.ptr(10, "out", {d.batch, d.n_q_heads, d.head_dim}, a.type);
  size_t bytes;
  void* ws = a.workspace(11, &bytes);
  void* st = a.stream(12);
  Unlocked unlocked;
  if (c.paged)
    return hata_window_decode_paged(&d, q, c.K, c.V, c.table, c.bs, c.n_blocks, lens, window, sink, scale, out, ws, bytes,
                                    st);
  return hata_window_decode(&d, q, c.K, c.V, lens, window, sink, scale, out, ws, bytes, st);
}

// dims, q, K, V, seq_lens, window, n_sink, scale, out, workspace, stream
hata_status_t window_prefill(Args& a) {
  const hata_dims_t& d = a.d;
  const void* q = a.ptr(1, "q", {d.batch, d.n_q_heads, d.max_seq, d.head_dim}, a.type);
  const Cache c = cache(a, 2, 3, 0, 0, false);
  const int32_t* lens = a.ints(4, "seq_lens", {d.batch});
  void* out = a.ptr(8, "out", {d.batch, d.n_q_heads, d.max_seq, d.head_dim}, a.type);
  size_t bytes;
  void* ws = a.workspace(9, &bytes);
  const int window = a.small(5, "window"), sink = a.small(6, "n_sink");
  const float scale = (float)a.number(7);
  void* st = a.stream(10);
  Unlocked unlocked;
  return hata_window_prefill(&d, q, c.K, c.V, lens, window, sink, scale, out, ws, bytes, st);
}

// dims, q, K, V, block_table, block_size, seq_lens, n_new, mask, scale, out, workspace, stream, paged
hata_status_t tree_attention(Args& a) {
  const hata_dims_t& d = a.d;
  const at::Tensor& qt = a.tensor(1, "q");
  if (qt.dim() != 4) raise(PyExc_ValueError, "q must be a tensor [B][Hq][n_tok][d]");
  const int64_t T = qt.size(2);
  if (T > INT32_MAX) raise(PyExc_ValueError, "q has too many tokens");
  const void* q = a.ptr(1, "q", {d.batch, d.n_q_heads, T, d.head_dim}, a.type);
  const Cache c = cache(a, 2, 3, 4, 5, a.truth(13));
  const int32_t* lens = a.ints(6, "seq_lens", {d.batch});
  const int32_t* n_new = a.maybe_ints(7, "n_new", {d.batch});
  const uint32_t* mask = nullptr;
  if (!a.none(8)) {
    const bool word = a.tensor(8, "mask").scalar_type() == at::kUInt32;
    mask = static_cast<const uint32_t*>(a.ptr(8, "mask", {d.batch, T, (T + 31) / 32}, word ? at::kUInt32 : at::kInt));
  }
  const float scale = (float)a.number(9);
  void* out = a.ptr(10, "out", {d.batch, d.n_q_heads, T, d.head_dim}, a.type);
  size_t bytes;
  void* ws = a.workspace(11, &bytes);
  void* st = a.stream(12);
  Unlocked unlocked;
  if (c.paged)
    return hata_tree_attention_paged(&d, (int)T, q, c.K, c.V, c.table, c.bs, c.n_blocks, lens, n_new, mask, scale, out, ws,
                                     bytes, st);
  return hata_tree_attention(&d, (int)T, q, c.K, c.V, lens, n_new, mask, scale, out, ws, bytes, st);
}

// dims, parent, block_table, block_size, seq_lens, ref_count, workspace, stream
hata_status_t pages_fork(Args& a) {
  const hata_dims_t& d = a.d;
  const int bs = a.small(3, "block_size");
  const int64_t n = a.tensor(5, "ref_count").numel();
  if (n > INT32_MAX) raise(PyExc_ValueError, "ref_count has too many blocks");
  const int32_t* parent = a.ints(1, "parent", {d.batch});
  int32_t* table = a.ints(2, "block_table", {d.batch, bs > 0 ? ((int64_t)d.max_seq + bs - 1) / bs : 0});
  int32_t* lens = a.ints(4, "seq_lens", {d.batch});
  int32_t* ref = a.ints(5, "ref_count", {n});
  size_t bytes;
  void* ws = a.workspace(6, &bytes);
  void* st = a.stream(7);
  Unlocked unlocked;
  return hata_pages_fork(&d, parent, table, bs, (int)n, lens, ref, ws, bytes, st);
}

// dims, new_lens, K_pool, V_pool, codes_pool, block_table, block_size, seq_lens, ref_count, workspace, stream
hata_status_t pages_resize(Args& a) {
  const hata_dims_t& d = a.d;
  const int32_t* new_lens = a.ints(1, "new_lens", {d.batch});
  const Cache c = cache(a, 2, 3, 5, 6, true);
  void* cd = codes(a, 4, c.n_blocks, c.bs);
  int32_t* lens = a.ints(7, "seq_lens", {d.batch});
  int32_t* ref = a.ints(8, "ref_count", {c.n_blocks});
  size_t bytes;
  void* ws = a.workspace(9, &bytes);
  void* st = a.stream(10);
  Unlocked unlocked;
  return hata_pages_resize(&d, new_lens, c.K, c.V, cd, c.table, c.bs, c.n_blocks, lens, ref, ws, bytes, st);
}

// dims, keep, n_keep, n_new, seq_lens, K, V, codes, block_table, block_size, new_lens, workspace, stream, paged
hata_status_t compact_kv(Args& a) {
  const hata_dims_t& d = a.d;
  const at::Tensor& k = a.tensor(1, "keep");
  if (k.dim() != 2 || k.size(1) > INT32_MAX) raise(PyExc_ValueError, "keep must be a tensor [B][n_tok]");
  const int64_t T = k.size(1);
  const int32_t* keep = a.ints(1, "keep", {d.batch, T});
  const int32_t* n_keep = a.ints(2, "n_keep", {d.batch});
  const int32_t* n_new = a.maybe_ints(3, "n_new", {d.batch});
  const int32_t* lens = a.ints(4, "seq_lens", {d.batch});
  const Cache c = cache(a, 5, 6, 8, 9, a.truth(13));
  void* cd = c.paged ? codes(a, 7, c.n_blocks, c.bs) : codes(a, 7, d.batch, d.max_seq);
  int32_t* new_lens = a.maybe_ints(10, "new_lens", {d.batch});
  size_t bytes;
  void* ws = a.workspace(11, &bytes);
  void* st = a.stream(12);
  Unlocked unlocked;
  if (c.paged)
    return hata_compact_kv_paged(&d, (int)T, keep, n_keep, n_new, lens, c.K, c.V, cd, c.table, c.bs, c.n_blocks, new_lens, ws,
                                 bytes, st);
  return hata_compact_kv(&d, (int)T, keep, n_keep, n_new, lens, c.K, c.V, cd, new_lens, ws, bytes, st);
}

template <hata_status_t (*CALL)(Args&), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    Args a(args, n, N);
    return PyLong_FromLong(CALL(a));
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

#define HATA_ENTRY(name, n) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, n>)), METH_FASTCALL, nullptr }

PyMethodDef methods[] = {HATA_ENTRY(norm_rope, 20),     HATA_ENTRY(window_decode, 14),  HATA_ENTRY(window_prefill, 11),
                         HATA_ENTRY(tree_attention, 14), HATA_ENTRY(pages_fork, 8),     HATA_ENTRY(pages_resize, 11),
                         HATA_ENTRY(compact_kv, 14),     {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch and the interpreter whose headers this was compiled with; the package compares it with those it runs on.
PyMODINIT_FUNC PyInit__serving() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", HATA_BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
