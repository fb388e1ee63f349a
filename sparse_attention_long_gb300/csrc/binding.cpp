// Argument marshalling of the serving calls.  A server makes them several times per
// generated token, and checking ten tensors in Python takes longer than the
// kernels of a small step: dsa_cache_fork through ctypes takes 7.4 us of host time,
// of which the launch is 1.8; through here 2.1 us.
//
// Each function checks what the Python function of the same name checks and makes
// the call on the current stream of the current device.  It returns the library's
// status, or 1 without having done anything when some argument is not exactly what
// the call needs (or the call is for another device or stream): the Python function
// then goes its own way, which says what is wrong.
#include <Python.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "dsa.h"

namespace {

constexpr int kRefused = 1;

struct Lib {
  decltype(&dsa_cache_fork) fork;
  decltype(&dsa_cache_extend) extend;
  decltype(&dsa_cache_compact) compact;
  decltype(&dsa_cache_copy_pages) copy_pages;
  decltype(&dsa_cache_write) write;
  decltype(&dsa_tree_attn_fwd) tree;
  decltype(&dsa_tree_workspace_size) tree_size;
  decltype(&dsa_beam_select) beam;
  decltype(&dsa_beam_workspace_size) beam_size;
  decltype(&dsa_rope_apply) rope;
  decltype(&dsa_sample) sample;
  decltype(&dsa_tree_accept) accept;
} lib;
PyObject *cache_type, *tree_type, *beam_type, *rope_type, *sampler_type;      // of the ctypes structures

// sizes multiply to a tensor's element count; -1 matches none
int64_t times(int64_t a, int64_t b) {
  int64_t r;
  return a < 0 || b < 0 || __builtin_mul_overflow(a, b, &r) ? -1 : r;
}

struct Refused {};

// a copy of a ctypes structure
template <typename S>
S structure(PyObject* o, PyObject* type) {
  if ((PyObject*)Py_TYPE(o) != type) throw Refused();
  Py_buffer v;
  if (PyObject_GetBuffer(o, &v, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    throw Refused();
  }
  const bool fits = v.len == (Py_ssize_t)sizeof(S);
  S s{};
  if (fits) memcpy(&s, v.buf, sizeof(S));
  PyBuffer_Release(&v);
  if (!fits) throw Refused();
  return s;
}

class Args {
 public:
  // a strided CUDA tensor (torch.Tensor itself) on the device of the call's first one
  const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_CheckExact(o)) throw Refused();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided) throw Refused();
    if (device_ < 0) {
      device_ = t.get_device();
      if (device_ != c10::cuda::current_device()) throw Refused();
    } else if (t.get_device() != device_) {
      throw Refused();
    }
    return t;
  }
  void* exactly(PyObject* o, at::ScalarType type, int64_t n) {
    const at::Tensor& t = tensor(o);
    if (t.scalar_type() != type || t.numel() != n || !t.is_contiguous()) throw Refused();
    return t.data_ptr();
  }
  int32_t* ints(PyObject* o, int64_t n) { return static_cast<int32_t*>(exactly(o, at::kInt, n)); }
  int32_t* list(PyObject* o, int64_t least, int64_t* n = nullptr) {
    const at::Tensor& t = tensor(o);
    if (t.scalar_type() != at::kInt || t.numel() < least || !t.is_contiguous()) throw Refused();
    if (n) *n = t.numel();
    return static_cast<int32_t*>(t.data_ptr());
  }
  // (layers,) pages, rows, columns
  dsa_pool pool(PyObject* o, const dsa_cache& c, at::ScalarType* type, int64_t* columns) {
    const at::Tensor& t = tensor(o);
    const int64_t k = t.dim() - 3;                 // first dimension of the pages
    if ((k != 0 && k != 1) || t.size(k) != c.n_pages || t.size(k + 1) != c.page_rows) throw Refused();
    const int64_t D = t.size(k + 2), e = t.element_size(), page = c.page_rows * D * e;
    if ((D > 1 && t.stride(k + 2) != 1) || (c.page_rows > 1 && t.stride(k + 1) != D)) throw Refused();
    *type = t.scalar_type();
    *columns = D;
    const int64_t layers = k ? t.size(0) : 1;
    return dsa_pool{t.data_ptr(), layers, layers > 1 ? t.stride(0) * e : page,
                    c.n_pages > 1 ? t.stride(k) * e : page, D * e};
  }
  // n_tok rows of heads, leading dimensions at one stride
  dsa_rope_rows rope_rows(PyObject* o, const dsa_rope_part& p, int64_t n_tok) {
    const at::Tensor& t = tensor(o);
    int64_t k = t.dim() - 1;
    if (t.scalar_type() != (p.dtype == DSA_BF16 ? at::kBFloat16 : at::kFloat) || k < 0 || t.size(k) != p.dim ||
        (p.dim > 1 && t.stride(k) != 1))
      throw Refused();
    dsa_rope_rows r{t.data_ptr(), 0, 0};
    if (p.heads > 1) {
      if (--k < 0 || t.size(k) != p.heads) throw Refused();
      r.head_stride = t.stride(k);
    }
    int64_t n = 1;
    while (--k >= 0) {
      if (t.size(k) == 1) continue;
      if (n == 1) r.tok_stride = t.stride(k);
      else if (t.stride(k) != times(r.tok_stride, n)) throw Refused();
      n *= t.size(k);
    }
    if (n != n_tok) throw Refused();
    return r;
  }
  template <typename T>
  T* exactly_or_none(PyObject* o, at::ScalarType type, int64_t n) {
    return o == Py_None ? nullptr : static_cast<T*>(exactly(o, type, n));
  }
  void* workspace(PyObject* o, size_t need) {
    if (o == Py_None) {
      if (need != 0) throw Refused();
      return nullptr;
    }
    const at::Tensor& t = tensor(o);
    if ((size_t)t.numel() * t.element_size() < need || !t.is_contiguous()) throw Refused();
    return t.data_ptr();
  }
  dsa_stream_t stream() const { return (dsa_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device_).stream(); }

 private:
  int64_t device_ = -1;
};

// f() without the interpreter's lock, as a Python number; nothing is thrown across the boundary
template <typename F>
PyObject* answer(Py_ssize_t n, Py_ssize_t want, F f) {
  int rc = kRefused;
  if (n == want) {
    try {
      rc = f();
    } catch (...) {
      PyErr_Clear();
    }
  }
  return PyLong_FromLong(rc);
}
template <typename F>
int unlocked(F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}

PyObject* cache_fork(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return answer(n, 10, [&] {
    const dsa_cache c = structure<dsa_cache>(o[0], cache_type);
    const int64_t t = times(c.n_seqs, c.max_pages), s = c.n_seqs, p = c.n_pages;
    Args a;
    int32_t *parent = a.ints(o[1], s), *table = a.ints(o[2], t), *lens = a.ints(o[3], s), *refs = a.ints(o[4], p);
    int32_t *table2 = a.ints(o[5], t), *lens2 = a.ints(o[6], s), *refs2 = a.ints(o[7], p);
    int32_t *copies = a.list(o[8], times(3, s)), *n_copies = a.ints(o[9], 1);
    dsa_stream_t st = a.stream();
    return unlocked([&] { return lib.fork(&c, parent, table, lens, refs, table2, lens2, refs2, copies, n_copies, st); });
  });
}

PyObject* cache_extend(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return answer(n, 8, [&] {
    const dsa_cache c = structure<dsa_cache>(o[0], cache_type);
    const int64_t s = c.n_seqs, p = c.n_pages;
    Args a;
    int32_t *grow = a.ints(o[1], s), *table = a.ints(o[2], times(s, c.max_pages)), *lens = a.ints(o[3], s);
    int32_t *refs = a.ints(o[4], p), *lens2 = a.ints(o[5], s), *refs2 = a.ints(o[6], p);
    int64_t n_slots;
    int32_t* slots = a.list(o[7], 1, &n_slots);
    dsa_stream_t st = a.stream();
    return unlocked([&] { return lib.extend(&c, grow, table, lens, refs, lens2, refs2, slots, n_slots, st); });
  });
}

PyObject* cache_compact(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return answer(n, 9, [&] {
    const dsa_cache c = structure<dsa_cache>(o[0], cache_type);
    const int64_t t = times(c.n_seqs, c.max_pages), p = c.n_pages;
    Args a;
    int32_t *table = a.ints(o[1], t), *lens = a.ints(o[2], c.n_seqs), *refs = a.ints(o[3], p);
    int32_t *table2 = a.ints(o[4], t), *refs2 = a.ints(o[5], p), *map = a.ints(o[6], p);
    int32_t *copies = a.list(o[7], times(3, p / 2 + 1)), *n_copies = a.ints(o[8], 1);
    dsa_stream_t st = a.stream();
    return unlocked([&] { return lib.compact(&c, table, lens, refs, table2, refs2, map, copies, n_copies, st); });
  });
}

PyObject* cache_copy_pages(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return answer(n, 4, [&] {
    const dsa_cache c = structure<dsa_cache>(o[0], cache_type);
    Args a;
    at::ScalarType type;
    int64_t D, entries;
    const dsa_pool pool = a.pool(o[1], c, &type, &D);
    int32_t *copies = a.list(o[2], 3, &entries), *n_copies = a.ints(o[3], 1);
    dsa_stream_t st = a.stream();
    return unlocked([&] { return lib.copy_pages(&c, &pool, copies, n_copies, entries / 3, st); });
  });
}

PyObject* cache_write(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return answer(n, 5, [&] {
    const dsa_cache c = structure<dsa_cache>(o[0], cache_type);
    Args a;
    at::ScalarType type;
    int64_t D, n_slots;
    const dsa_pool pool = a.pool(o[1], c, &type, &D);
    const at::Tensor& rows = a.tensor(o[2]);
    const int64_t k = rows.dim() - 2;
    if ((k != 0 && k != 1) || (k ? rows.size(0) : 1) != pool.n_layers || rows.size(k + 1) != D ||
        rows.scalar_type() != type)
      throw Refused();
    const int64_t n_src = rows.size(k);
    if ((D > 1 && rows.stride(k + 1) != 1) || (n_src > 1 && rows.stride(k) != D)) throw Refused();
    int32_t* slots = a.list(o[3], 1, &n_slots);
    int32_t* index = o[4] == Py_None ? nullptr : a.ints(o[4], n_slots);
    if (!index && n_src < n_slots) throw Refused();
    const int64_t layer = pool.n_layers > 1 ? rows.stride(0) * (int64_t)rows.element_size() : 0;
    const void* src = rows.data_ptr();
    dsa_stream_t st = a.stream();
    return unlocked([&] { return lib.write(&c, &pool, src, n_src, layer, slots, index, n_slots, st); });
  });
}

PyObject* tree_attn_fwd(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return answer(n, 13, [&] {
    const dsa_cache c = structure<dsa_cache>(o[0], cache_type);
    const dsa_tree t = structure<dsa_tree>(o[1], tree_type);
    const at::ScalarType type = t.dtype == DSA_BF16 ? at::kBFloat16 : at::kFloat;
    const int64_t rows = times(t.n_tok, t.H);
    Args a;
    at::ScalarType pool_type;
    int64_t D;
    const void* q = a.exactly(o[2], type, times(rows, t.d_qk));
    const dsa_pool pool = a.pool(o[3], c, &pool_type, &D);
    if (pool_type != type || pool.n_layers != 1 || D != t.d_qk) throw Refused();
    int32_t *table = a.ints(o[4], times(c.n_seqs, c.max_pages)), *lens = a.ints(o[5], c.n_seqs);
    const void* kv = a.exactly(o[6], type, times(t.n_tok, t.d_qk));
    int32_t* start = a.ints(o[7], c.n_seqs + 1);
    void* mask = o[8] == Py_None ? nullptr : a.exactly(o[8], at::kLong, times(t.n_tok, t.mask_words));
    void* out = a.exactly(o[9], type, times(rows, t.d_v));
    float* m = static_cast<float*>(a.exactly(o[10], at::kFloat, rows));
    float* l = static_cast<float*>(a.exactly(o[11], at::kFloat, rows));
    void* ws = a.workspace(o[12], lib.tree_size(&c, &t));
    dsa_stream_t st = a.stream();
    return unlocked([&] {
      return lib.tree(&c, &t, q, &pool, table, lens, kv, start, static_cast<uint64_t*>(mask), out, m, l, ws, st);
    });
  });
}

PyObject* beam_select(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return answer(n, 9, [&] {
    const dsa_beam b = structure<dsa_beam>(o[0], beam_type);
    const int64_t rows = times(b.n_batch, b.beams_in), outs = times(b.n_batch, b.beams_out);
    Args a;
    const void* x = a.exactly(o[1], b.dtype == DSA_BF16 ? at::kBFloat16 : at::kFloat, times(rows, b.ld));
    float* scores = static_cast<float*>(a.exactly(o[2], at::kFloat, rows));
    void* fin = o[3] == Py_None ? nullptr : a.exactly(o[3], at::kByte, rows);
    int32_t *parent = a.ints(o[4], outs), *token = a.ints(o[5], outs);
    float* scores2 = static_cast<float*>(a.exactly(o[6], at::kFloat, outs));
    void* fin2 = o[7] == Py_None ? nullptr : a.exactly(o[7], at::kByte, outs);
    void* ws = a.workspace(o[8], lib.beam_size(&b));
    dsa_stream_t st = a.stream();
    return unlocked([&] {
      return lib.beam(&b, x, scores, static_cast<uint8_t*>(fin), parent, token, scores2, static_cast<uint8_t*>(fin2),
                      ws, st);
    });
  });
}

PyObject* rope_apply(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return answer(n, 5, [&] {
    const dsa_rope r = structure<dsa_rope>(o[0], rope_type);
    if (r.n_parts < 1 || r.n_parts > DSA_ROPE_PARTS || (o[4] != Py_True && o[4] != Py_False)) throw Refused();
    Args a;
    int64_t n_tok;
    int32_t* pos = a.list(o[1], 1, &n_tok);
    dsa_rope_rows rows[2][DSA_ROPE_PARTS];
    for (int side = 0; side < 2; ++side) {
      PyObject* s = o[2 + side];
      if (!PyTuple_CheckExact(s) && !PyList_CheckExact(s)) throw Refused();
      if (PySequence_Fast_GET_SIZE(s) != r.n_parts) throw Refused();
      for (int i = 0; i < r.n_parts; ++i) rows[side][i] = a.rope_rows(PySequence_Fast_GET_ITEM(s, i), r.part[i], n_tok);
    }
    const int transposed = o[4] == Py_True;
    dsa_stream_t st = a.stream();
    return unlocked([&] { return lib.rope(&r, n_tok, pos, rows[0], rows[1], transposed, st); });
  });
}

PyObject* sample(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return answer(n, 10, [&] {
    const dsa_sampler s = structure<dsa_sampler>(o[0], sampler_type);
    Args a;
    const void* x = a.exactly(o[1], s.dtype == DSA_BF16 ? at::kBFloat16 : at::kFloat, times(s.rows, s.ld));
    float* u = static_cast<float*>(a.exactly(o[2], at::kFloat, s.rows));
    float* temperature = a.exactly_or_none<float>(o[3], at::kFloat, s.requests);
    int32_t* top_k = a.exactly_or_none<int32_t>(o[4], at::kInt, s.requests);
    float* top_p = a.exactly_or_none<float>(o[5], at::kFloat, s.requests);
    float* min_p = a.exactly_or_none<float>(o[6], at::kFloat, s.requests);
    int32_t* index = a.exactly_or_none<int32_t>(o[7], at::kInt, s.rows);
    int32_t* token = a.ints(o[8], s.rows);
    float* prob = a.exactly_or_none<float>(o[9], at::kFloat, s.rows);
    dsa_stream_t st = a.stream();
    return unlocked([&] { return lib.sample(&s, x, u, temperature, top_k, top_p, min_p, index, token, prob, st); });
  });
}

PyObject* tree_accept(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return answer(n, 11, [&] {
    const dsa_cache c = structure<dsa_cache>(o[0], cache_type);
    const dsa_tree t = structure<dsa_tree>(o[1], tree_type);
    Args a;
    int32_t* start = a.ints(o[2], c.n_seqs + 1);
    const uint64_t* mask = a.exactly_or_none<uint64_t>(o[3], at::kLong, times(t.n_tok, t.mask_words));
    int32_t *drafted = a.ints(o[4], t.n_tok), *sampled = a.ints(o[5], t.n_tok), *n_new = a.ints(o[6], c.n_seqs);
    int32_t *rows = a.ints(o[7], t.n_tok), *tokens = a.ints(o[8], t.n_tok), *next = a.ints(o[9], c.n_seqs);
    if (!PyLong_CheckExact(o[10])) throw Refused();
    const long long eos = PyLong_AsLongLong(o[10]);
    if (eos == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused();
    }
    dsa_stream_t st = a.stream();
    return unlocked([&] { return lib.accept(&c, &t, start, mask, drafted, sampled, eos, n_new, rows, tokens, next, st); });
  });
}

// the library's functions (addresses, in Lib's order) and the ctypes structures
PyObject* bind(PyObject*, PyObject* const* o, Py_ssize_t n) {
  void* f[sizeof(Lib) / sizeof(void*)];
  constexpr Py_ssize_t kFunctions = sizeof(f) / sizeof(f[0]);
  PyObject** types[] = {&cache_type, &tree_type, &beam_type, &rope_type, &sampler_type};
  constexpr int kTypes = sizeof(types) / sizeof(types[0]);
  if (n != kFunctions + kTypes) {
    PyErr_SetString(PyExc_TypeError, "bind: wrong number of arguments");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < kFunctions; ++i) {
    f[i] = PyLong_AsVoidPtr(o[i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null address");
      return nullptr;
    }
  }
  memcpy(&lib, f, sizeof(lib));
  for (int i = 0; i < kTypes; ++i) Py_XSETREF(*types[i], Py_NewRef(o[kFunctions + i]));
  Py_RETURN_NONE;
}

#define METHOD(name) \
  { #name, (PyCFunction)(void*)name, METH_FASTCALL, nullptr }
PyMethodDef methods[] = {METHOD(bind),          METHOD(cache_fork),  METHOD(cache_extend),
                         METHOD(cache_compact), METHOD(cache_copy_pages), METHOD(cache_write),
                         METHOD(tree_attn_fwd), METHOD(beam_select),
                         METHOD(rope_apply),    METHOD(sample),      METHOD(tree_accept), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "stamp", DSA_STAMP) != 0) Py_CLEAR(m);  // see _build.binding_stamp
  return m;
}
