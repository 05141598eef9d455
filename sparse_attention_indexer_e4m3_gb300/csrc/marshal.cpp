// Argument marshalling of the 4-bit cache's calls for Python: checks torch tensors, allocates the outputs
// and workspaces that the caller leaves out, and passes device pointers and the stream to the C ABI (whose
// addresses Python hands over once).  The calls themselves take a few microseconds on the GPU in a decoding step; checked
// in Python, tensor by tensor, each took 10 to 20 us on the host, here 3 to 6.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "dsa.h"

namespace {

struct Entry {
  decltype(&dsa_quantize_kv4_reserved) quantize_kv4_reserved;
  decltype(&dsa_dequantize_kv4) dequantize_kv4;
  decltype(&dsa_sparse_attn_kv4) sparse_attn_kv4;
  decltype(&dsa_sparse_attn_kv4_workspace_size) sparse_attn_kv4_workspace_size;
  decltype(&dsa_fork_pages) fork_pages;
  decltype(&dsa_reserve_pages) reserve_pages;
  decltype(&dsa_reserve_pages_workspace_size) reserve_pages_workspace_size;
  decltype(&dsa_compact_pages) compact_pages;
  decltype(&dsa_compact_pages_workspace_size) compact_pages_workspace_size;
  decltype(&dsa_copy_pages) copy_pages;
} g_abi;
PyObject* g_error = nullptr;  // DsaError

// A refusal: the Python exception to raise and its text.
struct Refusal {
  PyObject* kind;
  std::string text;
};
[[noreturn]] void bad_type(const std::string& text) { throw Refusal{PyExc_TypeError, text}; }
[[noreturn]] void bad_value(const std::string& text) { throw Refusal{PyExc_ValueError, text}; }

const char* type_name(at::ScalarType t) { return c10::toString(t); }

// A contiguous tensor argument of the given type and number of dimensions.
const at::Tensor& arg(PyObject* o, const char* name, at::ScalarType type, int dims) {
  if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a torch.Tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type) bad_type(std::string(name) + ": dtype " + type_name(t.scalar_type()) + " is not " + type_name(type));
  if (t.dim() != dims) bad_value(std::string(name) + " must have " + std::to_string(dims) + " dimensions");
  if (!t.is_contiguous()) bad_value(std::string(name) + " must be contiguous");
  return t;
}

void shape(const at::Tensor& t, const char* name, at::IntArrayRef want) {
  if (t.sizes() == want) return;
  std::string text = std::string(name) + " must have shape (";
  for (const int64_t n : want) text += std::to_string(n) + ", ";
  bad_value(text + ")");
}

int as_int(int64_t n, const char* name) {
  if (n < 0 || n > INT32_MAX) bad_value(std::string(name) + " is too large");
  return static_cast<int>(n);
}

// The current device and the stream of the call.  Every tensor has to lie on that device.
struct Where {
  c10::DeviceIndex device = -1;
  cudaStream_t stream = nullptr;   // of the call
  cudaStream_t current = nullptr;  // the caller's

  Where(PyObject* stream_object, std::initializer_list<const at::Tensor*> tensors) {
    for (const at::Tensor* t : tensors)
      if (t != nullptr && !t->is_cuda()) bad_value("tensors must be CUDA tensors");
    device = c10::cuda::current_device();
    for (const at::Tensor* t : tensors)
      if (t != nullptr && t->get_device() != device) bad_value("tensors must be on the current CUDA device");
    current = c10::cuda::getCurrentCUDAStream(device).stream();
    if (stream_object == Py_None) {
      stream = current;
    } else {
      PyObject* h = PyObject_GetAttrString(stream_object, "cuda_stream");
      if (h == nullptr) throw Refusal{nullptr, ""};
      stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(h));
      Py_DECREF(h);
      if (PyErr_Occurred()) throw Refusal{nullptr, ""};
    }
  }

  // A new tensor.  It is allocated for the stream that writes it: memory of the current stream's pool may still be in use
  // there by what held it last.  The caller gets it on the current stream, so it is not used anew before that
  // stream is done with it either.
  at::Tensor make(at::IntArrayRef sizes, at::ScalarType type) const {
    const at::AutoDispatchBelowADInplaceOrView below;  // nothing here is differentiated
    const at::TensorOptions options = at::TensorOptions().dtype(type).device(c10::Device(c10::DeviceType::CUDA, device));
    if (stream == current) return at::empty(sizes, options);
    at::Tensor t;
    {
      const c10::cuda::CUDAStreamGuard there(c10::cuda::getStreamFromExternal(stream, device));
      t = at::empty(sizes, options);
    }
    t.record_stream(c10::cuda::getCurrentCUDAStream(device).unwrap());
    return t;
  }
};

// The caller's tensor, or a new one.
at::Tensor out_arg(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef sizes) {
  if (o == Py_None) return at::Tensor();
  const at::Tensor& t = arg(o, name, type, static_cast<int>(sizes.size()));
  shape(t, name, sizes);
  return t;
}

template <class T>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
const uint16_t* bf16(const at::Tensor& t) { return ptr<const uint16_t>(t); }
const int32_t* i32(const at::Tensor& t) { return ptr<const int32_t>(t); }

void check(dsa_status st, const char* name) {
  if (st == DSA_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(st), name);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refusal{nullptr, ""};
}

PyObject* keep(PyObject* o) {
  Py_INCREF(o);
  return o;
}

struct Pool {
  const at::Tensor& cache;
  const at::Tensor& table;
  int P, rows, R, M;

  Pool(PyObject* cache_object, PyObject* table_object, int64_t D)
      : cache(arg(cache_object, "cache", at::kByte, 2)), table(arg(table_object, "table", at::kInt, 2)) {
    if (D != 64 && D != 128 && D != 256 && D != 512) bad_value("D must be 64, 128, 256 or 512");
    const int64_t row = D / 2 + D / 16 + 4, n = cache.size(1) / row;
    if (cache.size(1) != n * row || n < 16 || n > 256 || (n & (n - 1)) != 0)
      bad_value("cache pages of " + std::to_string(cache.size(1)) + " bytes hold no power of two in [16, 256] of rows of D = " +
                std::to_string(D));
    P = as_int(cache.size(0), "cache");
    rows = static_cast<int>(n);
    R = as_int(table.size(0), "table");
    M = as_int(table.size(1), "table");
  }
};

// Runs a call, turning refusals and C++ exceptions into Python ones.
template <class F>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t want, F f) {
  try {
    if (got != want) bad_type(std::string(name) + ": wrong number of arguments");
    return f();
  } catch (const Refusal& r) {
    if (r.kind != nullptr) PyErr_SetString(r.kind, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, name);
  }
  return nullptr;
}

int64_t long_of(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad_type(std::string(name) + " must be an int");
  }
  return v;
}

// (kv, cache, table, seq, pos, stream, lacking)
PyObject* quantize_kv4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("quantize_kv4", n, 7, [&] {
    const at::Tensor& kv = arg(a[0], "kv", at::kBFloat16, 2);
    const Pool c(a[1], a[2], kv.size(1));
    const at::Tensor& seq = arg(a[3], "seq", at::kInt, 1);
    const at::Tensor& pos = arg(a[4], "pos", at::kInt, 1);
    shape(seq, "seq", {kv.size(0)});
    shape(pos, "pos", {kv.size(0)});
    const at::Tensor lacking = out_arg(a[6], "lacking", at::kInt, {1});
    const Where w(a[5], {&kv, &c.cache, &c.table, &seq, &pos, lacking.defined() ? &lacking : nullptr});
    check(g_abi.quantize_kv4_reserved(bf16(kv), i32(seq), i32(pos), as_int(kv.size(0), "kv"), static_cast<int>(kv.size(1)),
                                      ptr<uint8_t>(c.cache), c.P, c.rows, i32(c.table), c.R, c.M,
                                      lacking.defined() ? i32(lacking) : nullptr, w.stream),
          "dsa_quantize_kv4_reserved");
    return keep(a[1]);
  });
}

// (cache, table, seq, pos, D, out, stream)
PyObject* dequantize_kv4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("dequantize_kv4", n, 7, [&] {
    const int64_t D = long_of(a[4], "D");
    const Pool c(a[0], a[1], D);
    const at::Tensor& seq = arg(a[2], "seq", at::kInt, 1);
    const at::Tensor& pos = arg(a[3], "pos", at::kInt, 1);
    const int64_t N = seq.size(0);
    shape(pos, "pos", {N});
    at::Tensor out = out_arg(a[5], "out", at::kBFloat16, {N, D});
    const Where w(a[6], {&c.cache, &c.table, &seq, &pos, out.defined() ? &out : nullptr});
    if (!out.defined()) out = w.make({N, D}, at::kBFloat16);
    check(g_abi.dequantize_kv4(ptr<const uint8_t>(c.cache), c.P, c.rows, i32(c.table), c.R, c.M, i32(seq), i32(pos),
                               as_int(N, "seq"), static_cast<int>(D), ptr<uint16_t>(out), w.stream),
          "dsa_dequantize_kv4");
    return a[5] != Py_None ? keep(a[5]) : THPVariable_Wrap(out);
  });
}

// (q, cache, table, seq, idx, start, attn_sink, scale, out, lse, workspace, stream)
PyObject* sparse_attn_kv4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("sparse_attn_kv4", n, 12, [&] {
    const at::Tensor& q = arg(a[0], "q", at::kBFloat16, 3);
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    const Pool c(a[1], a[2], D);
    const at::Tensor& seq = arg(a[3], "seq", at::kInt, 1);
    const at::Tensor& idx = arg(a[4], "idx", at::kInt, 2);
    shape(seq, "seq", {T});
    if (idx.size(0) != T) bad_value("idx must be [T, K]");
    const at::Tensor start = out_arg(a[5], "start", at::kInt, {T});
    const at::Tensor sink = out_arg(a[6], "attn_sink", at::kFloat, {H});
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) throw Refusal{nullptr, ""};
    at::Tensor out = out_arg(a[8], "out", at::kBFloat16, {T, H, D});
    const at::Tensor lse = out_arg(a[9], "lse", at::kFloat, {T, H});
    at::Tensor ws;
    if (a[10] != Py_None) ws = arg(a[10], "workspace", at::kByte, 1);
    const Where w(a[11], {&q, &c.cache, &c.table, &seq, &idx, start.defined() ? &start : nullptr, sink.defined() ? &sink : nullptr,
                          out.defined() ? &out : nullptr, lse.defined() ? &lse : nullptr, ws.defined() ? &ws : nullptr});
    if (!out.defined()) out = w.make({T, H, D}, at::kBFloat16);
    if (!ws.defined()) {
      const size_t need = g_abi.sparse_attn_kv4_workspace_size(as_int(T, "q"), as_int(H, "q"), static_cast<int>(D),
                                                               as_int(idx.size(1), "idx"));
      if (need > 0) ws = w.make({static_cast<int64_t>(need)}, at::kByte);
    }
    check(g_abi.sparse_attn_kv4(bf16(q), ptr<const uint8_t>(c.cache), c.P, c.rows, i32(c.table), c.R, c.M, i32(seq),
                                start.defined() ? i32(start) : nullptr, sink.defined() ? ptr<const float>(sink) : nullptr, i32(idx),
                                as_int(T, "q"), as_int(H, "q"), static_cast<int>(D), as_int(idx.size(1), "idx"),
                                static_cast<float>(scale), ptr<uint16_t>(out), lse.defined() ? ptr<float>(lse) : nullptr, ws.defined() ? ws.data_ptr() : nullptr,
                                ws.defined() ? static_cast<size_t>(ws.numel()) : 0, w.stream),
          "dsa_sparse_attn_kv4");
    return a[8] != Py_None ? keep(a[8]) : THPVariable_Wrap(out);
  });
}

// (table, parent, ref, table_out, stream)
PyObject* fork_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("fork_pages", n, 5, [&] {
    const at::Tensor& table = arg(a[0], "table", at::kInt, 2);
    const at::Tensor& parent = arg(a[1], "parent", at::kInt, 1);
    const at::Tensor& ref = arg(a[2], "ref", at::kInt, 1);
    shape(parent, "parent", {table.size(0)});
    at::Tensor out = out_arg(a[3], "table_out", at::kInt, table.sizes());
    const Where w(a[4], {&table, &parent, &ref, out.defined() ? &out : nullptr});
    if (!out.defined()) out = w.make(table.sizes(), at::kInt);
    check(g_abi.fork_pages(i32(table), i32(parent), as_int(table.size(0), "table"), as_int(table.size(1), "table"),
                           as_int(ref.size(0), "ref"), ptr<int32_t>(ref), ptr<int32_t>(out), w.stream),
          "dsa_fork_pages");
    return a[3] != Py_None ? keep(a[3]) : THPVariable_Wrap(out);
  });
}

// n elements of a one-dimensional tensor from `at` on, sharing its memory.
at::Tensor part_of(const at::Tensor& all, int64_t at, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(all.storage()), all.key_set(), all.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(n);
  return t;
}

// The outputs src [n], dst [n] and one [1] and the workspace of a page call: the caller's where given.
struct Lists {
  at::Tensor src, dst, one, ws;
  void* workspace = nullptr;
  size_t workspace_bytes = 0;

  Lists(PyObject* const* a, int64_t n, const char* name) {
    src = out_arg(a[0], "src", at::kInt, {n});
    dst = out_arg(a[1], "dst", at::kInt, {n});
    one = out_arg(a[2], name, at::kInt, {1});
    if (a[3] != Py_None) ws = arg(a[3], "workspace", at::kByte, 1);
  }
  const at::Tensor* given(const at::Tensor& t) const { return t.defined() ? &t : nullptr; }
  void fill(const Where& w, int64_t n, size_t need) {
    // one allocation for what is left out, the workspace last
    const int64_t scratch = ws.defined() ? 0 : static_cast<int64_t>((need + 3) / 4);
    const int64_t total = (src.defined() ? 0 : n) + (dst.defined() ? 0 : n) + (one.defined() ? 0 : 1) + scratch;
    const bool given = src.defined() && dst.defined() && one.defined() && scratch == 0;
    const at::Tensor all = given ? at::Tensor() : w.make({total}, at::kInt);
    int64_t at = 0;
    const auto take = [&](at::Tensor& t, int64_t count) {
      if (t.defined()) return;
      t = part_of(all, at, count);
      at += count;
    };
    take(src, n);
    take(dst, n);
    take(one, 1);
    if (ws.defined()) {
      workspace = ws.data_ptr();
      workspace_bytes = static_cast<size_t>(ws.numel());
    } else if (scratch > 0) {
      workspace = ptr<int32_t>(all) + at;
      workspace_bytes = static_cast<size_t>(scratch) * 4;
    }
  }
  PyObject* result(PyObject* const* a) const {
    PyObject* r = PyTuple_New(3);
    if (r == nullptr) throw Refusal{nullptr, ""};
    const at::Tensor* t[3] = {&src, &dst, &one};
    for (int i = 0; i < 3; ++i) PyTuple_SET_ITEM(r, i, a[i] != Py_None ? keep(a[i]) : THPVariable_Wrap(*t[i]));
    return r;
  }
};

// (table, ref, begin, end, page_rows, src, dst, lacking, workspace, stream)
PyObject* reserve_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("reserve_pages", n, 10, [&] {
    const at::Tensor& table = arg(a[0], "table", at::kInt, 2);
    const at::Tensor& ref = arg(a[1], "ref", at::kInt, 1);
    const at::Tensor& begin = arg(a[2], "begin", at::kInt, 1);
    const at::Tensor& end = arg(a[3], "end", at::kInt, 1);
    const int64_t R = table.size(0);
    shape(begin, "begin", {R});
    shape(end, "end", {R});
    const int rows = as_int(long_of(a[4], "page_rows"), "page_rows");
    const int P = as_int(ref.size(0), "ref");
    Lists l(a + 5, 2 * R, "lacking");
    const Where w(a[9], {&table, &ref, &begin, &end, l.given(l.src), l.given(l.dst), l.given(l.one), l.given(l.ws)});
    l.fill(w, 2 * R, g_abi.reserve_pages_workspace_size(P));
    check(g_abi.reserve_pages(ptr<int32_t>(table), ptr<int32_t>(ref), i32(begin), i32(end), as_int(R, "table"),
                              as_int(table.size(1), "table"), P, rows, ptr<int32_t>(l.src), ptr<int32_t>(l.dst),
                              ptr<int32_t>(l.one), l.workspace, l.workspace_bytes, w.stream),
          "dsa_reserve_pages");
    return l.result(a + 5);
  });
}

// (table, ref, src, dst, n_live, workspace, stream)
PyObject* compact_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("compact_pages", n, 7, [&] {
    const at::Tensor& table = arg(a[0], "table", at::kInt, 2);
    const at::Tensor& ref = arg(a[1], "ref", at::kInt, 1);
    const int P = as_int(ref.size(0), "ref");
    Lists l(a + 2, P / 2, "n_live");
    const Where w(a[6], {&table, &ref, l.given(l.src), l.given(l.dst), l.given(l.one), l.given(l.ws)});
    l.fill(w, P / 2, g_abi.compact_pages_workspace_size(P));
    check(g_abi.compact_pages(ptr<int32_t>(table), ptr<int32_t>(ref), as_int(table.size(0), "table"),
                              as_int(table.size(1), "table"), P, ptr<int32_t>(l.src), ptr<int32_t>(l.dst), ptr<int32_t>(l.one),
                              l.workspace, l.workspace_bytes, w.stream),
          "dsa_compact_pages");
    return l.result(a + 2);
  });
}

// (pages, src, dst, stream)
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("copy_pages", n, 4, [&] {
    if (!THPVariable_Check(a[0])) bad_type("pages must be a torch.Tensor");
    const at::Tensor& pages = THPVariable_Unpack(a[0]);
    if (pages.dim() < 2) bad_value("pages must be [P, ...]");
    if (!pages.is_contiguous()) bad_value("pages must be contiguous");
    const at::Tensor& src = arg(a[1], "src", at::kInt, 1);
    const at::Tensor& dst = arg(a[2], "dst", at::kInt, 1);
    shape(dst, "dst", src.sizes());
    const int64_t P = pages.size(0);
    if (P == 0) return keep(a[0]);
    const Where w(a[3], {&pages, &src, &dst});
    check(g_abi.copy_pages(pages.data_ptr(), static_cast<size_t>(pages.numel() / P) * pages.element_size(), as_int(P, "pages"),
                           i32(src), i32(dst), as_int(src.size(0), "src"), w.stream),
          "dsa_copy_pages");
    return keep(a[0]);
  });
}

// (addresses of the C ABI in Entry's order, DsaError)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("bind", n, 2, [&]() -> PyObject* {
    constexpr Py_ssize_t kEntries = sizeof(Entry) / sizeof(void*);
    if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != kEntries) bad_type("bind: the entry points' addresses");
    void* at[kEntries];
    for (Py_ssize_t i = 0; i < kEntries; ++i) at[i] = reinterpret_cast<void*>(long_of(PyTuple_GET_ITEM(a[0], i), "address"));
    static_assert(sizeof(Entry) == sizeof(at), "function pointers only");
    memcpy(static_cast<void*>(&g_abi), at, sizeof(at));
    Py_XDECREF(g_error);
    g_error = keep(a[1]);
    Py_RETURN_NONE;
  });
}

#define DSA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {DSA_METHOD(bind),          DSA_METHOD(quantize_kv4), DSA_METHOD(dequantize_kv4),
                           DSA_METHOD(sparse_attn_kv4), DSA_METHOD(fork_pages),   DSA_METHOD(reserve_pages),
                           DSA_METHOD(compact_pages), DSA_METHOD(copy_pages),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&g_module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
