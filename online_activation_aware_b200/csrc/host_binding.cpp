// Python module `_host`: the paged entry points of libttq.so for torch tensors. A step of a few
// tokens is a few microseconds on the GPU, so what surrounds a launch is most of its time: checking
// ten tensors, allocating the result and passing twenty arguments took 11 us in Python and ctypes
// beside the 4 of the call itself (append of 64 tokens: 15.1 us a call, 4.9 here; plan and attention
// of one sequence 20.9, 8.4 here; a fork 7.8, 2.9 here). The functions check the tensors (one device,
// types, sizes, contiguity), run on the given stream or the device's current one, allocate what the
// caller does not pass from that stream's memory and call the C entry point, whose own checks
// follow; a status that is not OK goes to the Python function that raises it.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <optional>
#include <string>

#include "ttq.h"

namespace {

// The C entry points, by address (the Python package loads the library).
struct Entries {
  decltype(&ttq_attention_plan) plan;
  decltype(&ttq_paged_attention) attention;
  decltype(&ttq_qk_norm_rope_paged) write;
  decltype(&ttq_copy_pages) copy;
  decltype(&ttq_remap_pages) remap;
  decltype(&ttq_token_logprobs) logprobs;
} entry;
PyObject* raise_status = nullptr;   // raise_status(name, status) raises
PyObject* out_of_memory = nullptr;  // torch's exception type

struct Error {
  PyObject* type;  // null: a Python error is set already
  std::string text;
};

constexpr int64_t kAny = -1;      // any size
constexpr int64_t kMostTop = 32;  // alternatives of ttq_token_logprobs
using Sizes = std::initializer_list<int64_t>;

std::string sizes_text(const int64_t* s, size_t n) {
  std::string t = "[";
  for (size_t i = 0; i < n; ++i) t += (i ? ", " : "") + (s[i] == kAny ? std::string("any") : std::to_string(s[i]));
  return t + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Error{PyExc_TypeError, std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}
void check_sizes(const at::Tensor& t, const char* name, Sizes want) {
  bool same = t.dim() == static_cast<int64_t>(want.size());
  for (size_t i = 0; same && i < want.size(); ++i)
    same = want.begin()[i] == kAny || t.size(static_cast<int64_t>(i)) == want.begin()[i];
  if (!same)
    throw Error{PyExc_ValueError, std::string(name) + " must have shape " + sizes_text(want.begin(), want.size()) +
                                      ", got " + sizes_text(t.sizes().data(), t.sizes().size())};
}

// The tensors of a call: all on one CUDA device.
struct Device {
  int index = -1;
  void take(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) throw Error{PyExc_ValueError, std::string(name) + " must be a CUDA tensor"};
    const int at = t.get_device();
    if (index >= 0 && at != index)
      throw Error{PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(at) +
                                        ", the other tensors on cuda:" + std::to_string(index)};
    index = at;
  }
  void typed(const at::Tensor& t, const char* name, at::ScalarType type) {
    take(t, name);
    if (t.scalar_type() != type)
      throw Error{PyExc_TypeError, std::string(name) + " must be " + at::toString(type) + ", got " +
                                       at::toString(t.scalar_type())};
  }
  void* contiguous(const at::Tensor& t, const char* name, at::ScalarType type, Sizes want) {
    check_sizes(t, name, want);
    typed(t, name, type);
    if (!t.is_contiguous()) throw Error{PyExc_ValueError, std::string(name) + " must be contiguous"};
    return t.data_ptr();
  }
  void* contiguous(PyObject* o, const char* name, at::ScalarType type, Sizes want) {
    return contiguous(tensor(o, name), name, type, want);
  }
  // None: null
  void* optional(PyObject* o, const char* name, at::ScalarType type, Sizes want) {
    return o == Py_None ? nullptr : contiguous(o, name, type, want);
  }
};

// The device is current, and so is the stream that the call was given (None: the current one).
struct On {
  c10::cuda::OptionalCUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> given;
  cudaStream_t stream;
  int index;
  On(const Device& d, PyObject* o) : index(d.index) {
    if (c10::cuda::current_device() != index) device.set_index(static_cast<c10::DeviceIndex>(index));
    if (o == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
      return;
    }
    PyObject* handle = PyObject_GetAttrString(o, "cuda_stream");
    if (!handle) throw Error{nullptr, ""};
    stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(handle));
    Py_DECREF(handle);
    if (PyErr_Occurred()) throw Error{nullptr, ""};
    given.emplace(c10::cuda::getStreamFromExternal(stream, static_cast<c10::DeviceIndex>(index)));
  }
  at::Tensor fresh(c10::IntArrayRef sizes, at::ScalarType type) const {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(index)));
  }
};

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Error{nullptr, ""};
  return v;
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Error{nullptr, ""};
  return static_cast<float>(v);
}

// The sizes of an AttentionPlan, and its buffer.
struct PlanOf {
  int64_t seqs, tokens, max_new, heads, kv_heads, head_dim;
  void* buffer;
  size_t bytes;
  PlanOf(Device& d, PyObject* o) {
    static PyObject* const names[6] = {
        PyUnicode_InternFromString("seqs"),  PyUnicode_InternFromString("tokens"),   PyUnicode_InternFromString("max_new"),
        PyUnicode_InternFromString("heads"), PyUnicode_InternFromString("kv_heads"), PyUnicode_InternFromString("head_dim")};
    int64_t* to[6] = {&seqs, &tokens, &max_new, &heads, &kv_heads, &head_dim};
    for (int i = 0; i < 6; ++i) {
      PyObject* v = PyObject_GetAttr(o, names[i]);
      if (!v) throw Error{nullptr, ""};
      *to[i] = PyLong_AsLongLong(v);
      Py_DECREF(v);
      if (*to[i] == -1 && PyErr_Occurred()) throw Error{nullptr, ""};
    }
    PyObject* b = PyObject_GetAttrString(o, "buffer");
    if (!b) throw Error{nullptr, ""};
    at::Tensor t;
    if (THPVariable_Check(b)) t = THPVariable_Unpack(b);
    Py_DECREF(b);  // (the plan holds it)
    if (!t.defined()) throw Error{PyExc_TypeError, "a plan's buffer must be a tensor"};
    buffer = d.contiguous(t, "plan", at::kByte, {kAny});
    bytes = static_cast<size_t>(t.numel());
  }
};

// The pools of a layer and their table.
struct Pool {
  void *k, *v, *table;
  int64_t pages, page_size, width;
  Pool(Device& d, PyObject* ko, PyObject* vo, PyObject* to, int64_t seqs, int64_t kv_heads, int64_t head_dim) {
    const at::Tensor& kt = tensor(ko, "k_pages");
    k = d.contiguous(kt, "k_pages", at::kBFloat16, {kAny, kAny, kv_heads, head_dim});
    pages = kt.size(0);
    page_size = kt.size(1);
    v = d.contiguous(vo, "v_pages", at::kBFloat16, {pages, page_size, kv_heads, head_dim});
    const at::Tensor& tt = tensor(to, "page_table");
    table = d.contiguous(tt, "page_table", at::kInt, {seqs, kAny});
    width = tt.size(1);
  }
};

template <typename F>
void run(const char* name, F call) {
  ttq_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = call();
  Py_END_ALLOW_THREADS;
  if (st == TTQ_OK) return;
  PyObject* r = PyObject_CallFunction(raise_status, "si", name, static_cast<int>(st));
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
  throw Error{nullptr, ""};
}

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t want, F body) {
  if (given != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return body();
  } catch (const Error& e) {
    if (e.type) PyErr_SetString(e.type, e.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(out_of_memory ? out_of_memory : PyExc_MemoryError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <typename T>
T* as(void* p) {
  return static_cast<T*>(p);
}

// plan(plan, q_start, kv_len, window, prefix, stream)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    Device d;
    const PlanOf s(d, a[0]);
    void* start = d.contiguous(a[1], "q_start", at::kInt, {s.seqs + 1});
    void* len = d.contiguous(a[2], "kv_len", at::kInt, {s.seqs});
    const int64_t window = integer(a[3]);
    void* prefix = d.optional(a[4], "prefix", at::kInt, {s.seqs});
    const On on(d, a[5]);
    run("ttq_attention_plan", [&] {
      return entry.plan(as<int32_t>(start), as<int32_t>(len), as<int32_t>(prefix), window, s.seqs, s.tokens, s.max_new,
                        s.heads, s.kv_heads, s.head_dim, s.buffer, s.bytes, on.stream);
    });
    Py_RETURN_NONE;
  });
}

// attention(q, plan, k_pages, v_pages, page_table, softcap, slopes, out, stream) -> out
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    Device d;
    const PlanOf s(d, a[1]);
    const int64_t channels = s.heads * s.head_dim;
    if (q.dim() != 2 || q.size(0) != s.tokens || q.size(1) < channels || q.stride(1) != 1)
      throw Error{PyExc_ValueError, "q must be " + std::to_string(s.tokens) + " rows of at least " +
                                        std::to_string(channels) + " contiguous channels, got " +
                                        sizes_text(q.sizes().data(), q.sizes().size())};
    d.typed(q, "q", at::kBFloat16);
    const Pool p(d, a[2], a[3], a[4], s.seqs, s.kv_heads, s.head_dim);
    const float softcap = number(a[5]);
    void* slopes = d.optional(a[6], "slopes", at::kFloat, {s.heads});
    void* to = d.optional(a[7], "out", at::kBFloat16, {s.tokens, channels});
    const On on(d, a[8]);
    at::Tensor out;
    if (!to) {
      out = on.fresh({s.tokens, channels}, at::kBFloat16);
      to = out.data_ptr();
    }
    run("ttq_paged_attention", [&] {
      return entry.attention(q.data_ptr(), s.tokens > 1 ? q.stride(0) : channels, s.seqs, s.tokens, s.max_new, s.heads,
                             s.kv_heads, s.head_dim, p.k, p.v, p.pages, p.page_size, as<int32_t>(p.table), p.width,
                             softcap, as<float>(slopes), to, s.buffer, s.bytes, on.stream);
    });
    if (out.defined()) return THPVariable_Wrap(std::move(out));
    Py_INCREF(a[7]);
    return a[7];
  });
}

// write(qkv, heads, kv_heads, head_dim, q_norm, k_norm, eps, rope, q_start, kv_len, k_pages, v_pages, page_table, q,
//       stream) -> q
PyObject* write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const at::Tensor& qkv = tensor(a[0], "qkv");
    const int64_t heads = integer(a[1]), kv_heads = integer(a[2]), D = integer(a[3]);
    Device d;
    void* from = d.contiguous(qkv, "qkv", at::kBFloat16, {kAny, (heads + 2 * kv_heads) * D});
    const int64_t T = qkv.size(0);
    void* qn = d.contiguous(a[4], "q_norm", at::kBFloat16, {D});
    void* kn = d.contiguous(a[5], "k_norm", at::kBFloat16, {D});
    const float eps = number(a[6]);
    const at::Tensor& rope = tensor(a[7], "table");
    void* angles = d.contiguous(rope, "table", at::kFloat, {kAny, D / 2, 2});
    const at::Tensor& lens = tensor(a[9], "kv_len");
    void* len = d.contiguous(lens, "kv_len", at::kInt, {kAny});
    const int64_t seqs = lens.size(0);
    void* start = d.contiguous(a[8], "q_start", at::kInt, {seqs + 1});
    const Pool p(d, a[10], a[11], a[12], seqs, kv_heads, D);
    void* to = d.optional(a[13], "q", at::kBFloat16, {T, heads * D});
    const On on(d, a[14]);
    at::Tensor out;
    if (!to) {
      out = on.fresh({T, heads * D}, at::kBFloat16);
      to = out.data_ptr();
    }
    run("ttq_qk_norm_rope_paged", [&] {
      return entry.write(from, seqs, T, heads, kv_heads, D, qn, kn, eps, as<float>(angles), rope.size(0),
                         as<int32_t>(start), as<int32_t>(len), p.k, p.v, p.pages, p.page_size, as<int32_t>(p.table),
                         p.width, to, on.stream);
    });
    if (out.defined()) return THPVariable_Wrap(std::move(out));
    Py_INCREF(a[13]);
    return a[13];
  });
}

// copy(k_pool, v_pool, src, dst, stream)
PyObject* copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const at::Tensor &k = tensor(a[0], "k_pool"), &v = tensor(a[1], "v_pool"), &src = tensor(a[2], "src");
    const int64_t dims = k.dim();
    if (dims != 4 && dims != 5)
      throw Error{PyExc_ValueError,
                  "pools are [num_pages, page_size, kv_heads, head_dim], with the layers ahead or without"};
    if (k.sizes() != v.sizes()) throw Error{PyExc_ValueError, "v_pool must have the shape of k_pool"};
    Device d;
    for (const at::Tensor* t : {&k, &v}) {
      d.typed(*t, t == &k ? "k_pool" : "v_pool", k.scalar_type());
      if (!t->is_contiguous()) throw Error{PyExc_ValueError, "the pools must be contiguous"};
    }
    void* from = d.contiguous(src, "src", at::kInt, {kAny});
    const int64_t pairs = src.size(0);
    void* to = d.contiguous(a[3], "dst", at::kInt, {pairs});
    if (pairs > 0) {
      const On on(d, a[4]);
      const int64_t bytes = k.size(dims - 3) * k.size(dims - 2) * k.size(dims - 1) * static_cast<int64_t>(k.element_size());
      run("ttq_copy_pages", [&] {
        return entry.copy(k.data_ptr(), v.data_ptr(), dims == 5 ? k.size(0) : 1, k.size(dims - 4), bytes,
                          as<int32_t>(from), as<int32_t>(to), pairs, on.stream);
      });
    }
    Py_RETURN_NONE;
  });
}

// remap(table, mapping, out, stream) -> out
PyObject* remap(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    const at::Tensor &table = tensor(a[0], "table"), &mapping = tensor(a[1], "mapping");
    Device d;
    void* map = d.contiguous(mapping, "mapping", at::kInt, {kAny});
    d.typed(table, "table", at::kInt);
    if (!table.is_contiguous()) throw Error{PyExc_ValueError, "table must be contiguous"};
    at::Tensor out;
    if (a[2] != Py_None) {
      const at::Tensor& o = tensor(a[2], "out");
      d.typed(o, "out", at::kInt);
      if (o.sizes() != table.sizes() || !o.is_contiguous())
        throw Error{PyExc_ValueError, "out must be contiguous and have the shape of table"};
      out = o;
    }
    const On on(d, a[3]);
    if (!out.defined()) out = on.fresh(table.sizes(), at::kInt);
    run("ttq_remap_pages", [&] {
      return entry.remap(as<int32_t>(table.data_ptr()), table.numel(), as<int32_t>(map), mapping.size(0),
                         as<int32_t>(out.data_ptr()), on.stream);
    });
    if (a[2] == Py_None) return THPVariable_Wrap(std::move(out));
    Py_INCREF(a[2]);
    return a[2];
  });
}

// logprobs(logits, tokens, top, stream) -> dict
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "logits");
    if (x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1))
      throw Error{PyExc_ValueError, "logits must be rows of contiguous logits"};
    const int64_t rows = x.size(0), vocab = x.size(1), top = integer(a[2]);
    const at::ScalarType type = x.scalar_type();
    if (type != at::kBFloat16 && type != at::kHalf && type != at::kFloat)
      throw Error{PyExc_TypeError, std::string("logits must be bf16, fp16 or fp32, got ") + at::toString(type)};
    Device d;
    const at::Tensor& tokens = tensor(a[1], "tokens");
    check_sizes(tokens, "tokens", {rows});
    d.take(x, "logits");
    void* tok = d.contiguous(tokens, "tokens", at::kLong, {rows});
    const On on(d, a[3]);
    at::Tensor lp = on.fresh({rows}, at::kFloat), ent = on.fresh({rows}, at::kFloat), ids, lps;
    if (top > 0 && top <= std::min<int64_t>(vocab, kMostTop)) {  // (the entry point refuses the others)
      ids = on.fresh({rows, top}, at::kLong);
      lps = on.fresh({rows, top}, at::kFloat);
    }
    run("ttq_token_logprobs", [&] {
      return entry.logprobs(x.data_ptr(), type == at::kBFloat16 ? TTQ_BF16 : type == at::kHalf ? TTQ_FP16 : TTQ_FP32, rows,
                            vocab, rows > 1 ? x.stride(0) : vocab, as<int64_t>(tok), top, as<float>(lp.data_ptr()),
                            as<float>(ent.data_ptr()), ids.defined() ? as<int64_t>(ids.data_ptr()) : nullptr,
                            lps.defined() ? as<float>(lps.data_ptr()) : nullptr, on.stream);
    });
    PyObject* r = PyDict_New();
    auto put = [&](const char* name, at::Tensor&& t) {
      PyObject* o = THPVariable_Wrap(std::move(t));
      const bool ok = r && o && PyDict_SetItemString(r, name, o) == 0;
      Py_XDECREF(o);
      if (!ok) {
        Py_XDECREF(r);
        throw Error{nullptr, ""};
      }
    };
    put("logprob", std::move(lp));
    put("entropy", std::move(ent));
    if (ids.defined()) {
      put("top_ids", std::move(ids));
      put("top_logprobs", std::move(lps));
    }
    return r;
  });
}

// bind(addresses of the six entry points, raise_status, out_of_memory)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 6) throw Error{PyExc_TypeError, "six addresses"};
    void* p[6];
    for (int i = 0; i < 6; ++i) p[i] = reinterpret_cast<void*>(integer(PyTuple_GET_ITEM(a[0], i)));
    entry.plan = reinterpret_cast<decltype(entry.plan)>(p[0]);
    entry.attention = reinterpret_cast<decltype(entry.attention)>(p[1]);
    entry.write = reinterpret_cast<decltype(entry.write)>(p[2]);
    entry.copy = reinterpret_cast<decltype(entry.copy)>(p[3]);
    entry.remap = reinterpret_cast<decltype(entry.remap)>(p[4]);
    entry.logprobs = reinterpret_cast<decltype(entry.logprobs)>(p[5]);
    Py_INCREF(a[1]);
    Py_XSETREF(raise_status, a[1]);
    Py_INCREF(a[2]);
    Py_XSETREF(out_of_memory, a[2]);
    Py_RETURN_NONE;
  });
}

#define TTQ_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TTQ_METHOD(bind),  TTQ_METHOD(plan),     TTQ_METHOD(attention),       TTQ_METHOD(write), TTQ_METHOD(copy),
                         TTQ_METHOD(remap), TTQ_METHOD(logprobs), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TTQ_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
