// The calls of include/cosa_attn.h for Python: checks of the tensors and the call itself, without a Python object per check.
//
// A call from Python had nine microseconds of such checks (a tensor's type, size, layout, device and address are five
// method calls) before its kernel; here they are reads of the tensor.  Loaded as block_sparse_long_gb300._attn_call; the library's
// functions come by address, so this file needs only its header.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdarg>
#include <cstdint>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "cosa_attn.h"

namespace {

constexpr int64_t kRot = COSA_ATTN_ROPE_DIM;

decltype(&cosa_tree_attention) tree_attention_fn = nullptr;
decltype(&cosa_tree_commit) tree_commit_fn = nullptr;
decltype(&cosa_latent_rope) latent_rope_fn = nullptr;
decltype(&cosa_latent_attention) latent_attention_fn = nullptr;
decltype(&cosa_latent_prefill) latent_prefill_fn = nullptr;

struct Refused {};      // a Python exception is set

[[noreturn]] void refuse(const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(PyExc_ValueError, format, args);
  va_end(args);
  throw Refused{};
}

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    default: return "torch.uint8";
  }
}

// One call: its parameters (a copy, which takes the strides), and the device of its tensors (the first one sets it).
struct Call {
  cosa_attn_params p;
  int index = -1;

  explicit Call(PyObject* params) {
    Py_buffer view;
    if (PyObject_GetBuffer(params, &view, PyBUF_SIMPLE) != 0) throw Refused{};
    const bool fits = view.len == static_cast<Py_ssize_t>(sizeof p);
    if (fits) p = *static_cast<const cosa_attn_params*>(view.buf);
    PyBuffer_Release(&view);
    if (!fits) refuse("the parameters must be CosaAttnParams");
  }

  static const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse("%s must be a tensor, got %R", name, reinterpret_cast<PyObject*>(Py_TYPE(o)));
    return THPVariable_Unpack(o);
  }

  static void type(PyObject* o, const at::Tensor& t, const char* name, at::ScalarType want) {
    if (t.scalar_type() == want) return;
    PyObject* got = PyObject_GetAttrString(o, "dtype");
    if (got != nullptr) PyErr_Format(PyExc_ValueError, "%s must be %s, got %S", name, name_of(want), got);
    Py_XDECREF(got);
    throw Refused{};
  }

  void on_device(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    const int at = t.get_device();
    if (index >= 0 && at != index) refuse("%s is on cuda:%d, the other tensors on cuda:%d", name, at, index);
    index = at;
  }

  // Address of a contiguous tensor of at least `least` elements, or null for None.
  template <typename T>
  T* dense(PyObject* o, const char* name, at::ScalarType want, int64_t least) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    type(o, t, name, want);
    if (!t.is_contiguous()) refuse("%s must be contiguous", name);
    if (t.numel() < least) refuse("%s holds %lld elements; the parameters need at least %lld", name, (long long)t.numel(), (long long)least);
    on_device(t, name);
    return static_cast<T*>(t.data_ptr());
  }
  const int32_t* ints(PyObject* o, const char* name, int64_t least) { return dense<int32_t>(o, name, at::kInt, least); }
  void* bf16(PyObject* o, const char* name, int64_t least) { return dense<void>(o, name, at::kBFloat16, least); }

  // Address and strides of rows [tokens, heads, width] (heads 0: [tokens, width]), whose tokens and heads may lie apart.
  const void* rows(PyObject* o, const char* name, int64_t tokens, int64_t heads, int64_t width, int64_t* by_token, int64_t* by_head) {
    const at::Tensor& t = tensor(o, name);
    type(o, t, name, at::kBFloat16);
    const int64_t dims = heads ? 3 : 2;
    if (t.dim() != dims || t.size(dims - 1) != width || (heads && t.size(1) != heads)) {
      PyObject* shape = PyObject_GetAttrString(o, "shape");
      if (shape != nullptr) {
        if (heads) PyErr_Format(PyExc_ValueError, "%s must be [tokens, %lld, %lld], got %S", name, (long long)heads, (long long)width, shape);
        else PyErr_Format(PyExc_ValueError, "%s must be [tokens, %lld], got %S", name, (long long)width, shape);
      }
      Py_XDECREF(shape);
      throw Refused{};
    }
    const int64_t n = t.size(0), h = heads ? heads : 1;
    if (n < tokens) refuse("%s holds %lld tokens; the parameters need at least %lld", name, (long long)n, (long long)tokens);
    // the stride of a single token or head says nothing
    int64_t head = h > 1 ? t.stride(1) : width, token = n > 1 ? t.stride(0) : (h - 1) * head + width;
    if (n > 0) {
      if (t.stride(dims - 1) != 1) refuse("%s: the values of a head must be contiguous", name);
      if (head < width) refuse("%s: heads are %lld elements apart, a head has %lld", name, (long long)head, (long long)width);
      if (n > 1 && token < (h - 1) * head + width && (token < width || head < (n - 1) * token + width))
        refuse("%s: tokens are %lld elements apart, heads %lld: they overlap", name, (long long)token, (long long)head);
    }
    on_device(t, name);
    if (n <= 1) token += (8 - token % 8) % 8;
    *by_token = token;
    if (by_head != nullptr) *by_head = head;
    return t.data_ptr();
  }

  // Runs `call(status, stream)` on the tensors' device.
  template <typename F>
  PyObject* run(PyObject* status, PyObject* stream, F call) {
    int32_t* s = dense<int32_t>(status, "status", at::kInt, 1);
    void* to;
    if (stream == Py_None) {
      to = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    } else {
      PyObject* handle = PyObject_GetAttrString(stream, "cuda_stream");
      PyObject* where = handle != nullptr ? PyObject_GetAttrString(stream, "device") : nullptr;
      PyObject* number = where != nullptr ? PyObject_GetAttrString(where, "index") : nullptr;
      const long long device = number != nullptr ? PyLong_AsLongLong(number) : -1;
      to = number != nullptr ? PyLong_AsVoidPtr(handle) : nullptr;
      Py_XDECREF(handle);
      Py_XDECREF(where);
      Py_XDECREF(number);
      if (PyErr_Occurred()) throw Refused{};
      if (device != index) refuse("stream is on cuda:%lld, the tensors on cuda:%d", device, index);
    }
    int rc;
    if (c10::cuda::current_device() == index) {
      rc = call(s, to);
    } else {
      c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
      rc = call(s, to);
    }
    return PyLong_FromLong(rc);
  }

  int64_t tables() const { return static_cast<int64_t>(p.num_reqs) * p.max_pages_per_req; }
  int64_t slots() const { return static_cast<int64_t>(p.num_pages) * p.page_size; }
  int64_t query_rows() const { return static_cast<int64_t>(p.total_tokens) * p.num_q_heads; }
};

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

struct Workspace {
  void* at;
  size_t bytes;
};

Workspace workspace_of(Call& c, PyObject* o) {
  const at::Tensor& t = Call::tensor(o, "workspace");
  c.on_device(t, "workspace");
  if (!t.is_contiguous()) refuse("workspace must be contiguous");
  return {t.data_ptr(), static_cast<size_t>(t.nbytes())};
}

// p, q, cu_seqlens, k_cache, v_cache, page_table, kv_len, tree_mask, out, lse, workspace, status, stream
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    Call c(a[0]);
    cosa_attn_params& p = c.p;
    const int64_t cache = c.slots() * p.num_kv_heads * p.head_dim, rows = c.query_rows();
    const void* q = c.rows(a[1], "q", p.total_tokens, p.num_q_heads, p.head_dim, &p.q_stride, &p.q_head_stride);
    const int32_t* cu = c.ints(a[2], "cu_seqlens", int64_t{p.num_reqs} + 1);
    const void* k = c.bf16(a[3], "k_cache", cache);
    const void* v = c.bf16(a[4], "v_cache", cache);
    const int32_t* table = c.ints(a[5], "page_table", c.tables());
    const int32_t* len = c.ints(a[6], "kv_len", p.num_reqs);
    const int64_t* mask = c.dense<int64_t>(a[7], "tree_mask", at::kLong, p.total_tokens);
    void* out = c.bf16(a[8], "out", rows * p.head_dim);
    float* lse = c.dense<float>(a[9], "lse", at::kFloat, rows);
    const Workspace ws = workspace_of(c, a[10]);
    return c.run(a[11], a[12], [&](int32_t* status, void* stream) {
      return tree_attention_fn(&p, q, cu, k, v, table, len, mask, out, lse, ws.at, ws.bytes, status, stream);
    });
  });
}

// p, q_latent, q_rope, cu_seqlens, cache, page_table, kv_len, tree_mask, out, lse, workspace, status, stream
PyObject* latent_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    Call c(a[0]);
    cosa_attn_params& p = c.p;
    const int64_t rows = c.query_rows();
    const void* q = c.rows(a[1], "q_latent", p.total_tokens, p.num_q_heads, p.latent_dim, &p.q_stride, &p.q_head_stride);
    const void* r = c.rows(a[2], "q_rope", p.total_tokens, p.num_q_heads, kRot, &p.q_rope_stride, &p.q_rope_head_stride);
    const int32_t* cu = c.ints(a[3], "cu_seqlens", int64_t{p.num_reqs} + 1);
    const void* cache = c.bf16(a[4], "latent_cache", c.slots() * (p.latent_dim + kRot));
    const int32_t* table = c.ints(a[5], "page_table", c.tables());
    const int32_t* len = c.ints(a[6], "kv_len", p.num_reqs);
    const int64_t* mask = c.dense<int64_t>(a[7], "tree_mask", at::kLong, p.total_tokens);
    void* out = c.bf16(a[8], "out", rows * p.latent_dim);
    float* lse = c.dense<float>(a[9], "lse", at::kFloat, rows);
    const Workspace ws = workspace_of(c, a[10]);
    return c.run(a[11], a[12], [&](int32_t* status, void* stream) {
      return latent_attention_fn(&p, q, r, cu, cache, table, len, mask, out, lse, ws.at, ws.bytes, status, stream);
    });
  });
}

// p, cache_a, cache_b, cu_seqlens, page_table, kv_len, path, path_len, new_len, status, stream
PyObject* tree_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    Call c(a[0]);
    cosa_attn_params& p = c.p;
    void* cache[2] = {nullptr, nullptr};
    int64_t row = 0;
    for (int i = 0; i < 2; ++i) {
      if (i && a[2] == Py_None) break;
      const at::Tensor& t = Call::tensor(a[1 + i], "caches");
      if (t.scalar_type() != at::kBFloat16 || t.dim() < 3 || !t.is_contiguous())
        refuse("caches: one or two contiguous bf16 tensors [num_pages, page_size, ...]");
      int64_t elems = 1;
      for (int64_t d = 2; d < t.dim(); ++d) elems *= t.size(d);
      if (i == 0) row = elems;
      if (t.size(0) < p.num_pages || t.size(1) != p.page_size || elems != row || row > INT32_MAX)
        refuse("caches must be [%d, %d, ...] with equal rows", p.num_pages, p.page_size);
      cache[i] = t.data_ptr();
    }
    c.on_device(Call::tensor(a[1], "caches"), "caches");
    if (a[2] != Py_None) c.on_device(Call::tensor(a[2], "caches"), "caches");
    const int32_t* cu = c.ints(a[3], "cu_seqlens", int64_t{p.num_reqs} + 1);
    const int32_t* table = c.ints(a[4], "page_table", c.tables());
    const int32_t* len = c.ints(a[5], "kv_len", p.num_reqs);
    const int32_t* path = c.ints(a[6], "path", static_cast<int64_t>(p.num_reqs) * p.max_new_tokens);
    const int32_t* path_len = c.ints(a[7], "path_len", p.num_reqs);
    int32_t* new_len = c.dense<int32_t>(a[8], "new_len", at::kInt, p.num_reqs);
    return c.run(a[9], a[10], [&](int32_t* status, void* stream) {
      return tree_commit_fn(&p, cache[0], cache[1], static_cast<int32_t>(row), cu, table, len, path, path_len, new_len, status, stream);
    });
  });
}

// p, kv, q, weight, inv_freq, positions, cu_seqlens, start, q_out, c_out, k_out, cache, page_table, status, stream
PyObject* latent_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    Call c(a[0]);
    cosa_attn_params& p = c.p;
    const int64_t T = p.total_tokens;
    const void* kv = c.rows(a[1], "kv", T, 0, p.latent_dim + kRot, &p.k_stride, nullptr);
    const void* q = a[2] == Py_None ? nullptr : c.rows(a[2], "q", T, p.num_q_heads, kRot, &p.q_rope_stride, &p.q_rope_head_stride);
    const void* weight = c.bf16(a[3], "weight", p.latent_dim);
    const double* freq = c.dense<double>(a[4], "inv_freq", at::kDouble, kRot / 2);
    const int32_t* pos = c.ints(a[5], "positions", T);
    const int32_t* cu = c.ints(a[6], "cu_seqlens", int64_t{p.num_reqs} + 1);
    const int32_t* start = c.ints(a[7], "start", p.num_reqs);
    void* q_out = c.bf16(a[8], "q_out", c.query_rows() * kRot);
    void* c_out = c.bf16(a[9], "c_out", T * p.latent_dim);
    void* k_out = c.bf16(a[10], "k_out", T * kRot);
    void* cache = c.bf16(a[11], "latent_cache", c.slots() * (p.latent_dim + kRot));
    const int32_t* table = c.ints(a[12], "page_table", c.tables());
    return c.run(a[13], a[14], [&](int32_t* status, void* stream) {
      return latent_rope_fn(&p, kv, q, weight, freq, pos, cu, start, q_out, c_out, k_out, cache, table, status, stream);
    });
  });
}

// p, q_nope, q_rope, k_nope, k_rope, v, cu_seqlens, cu_kv, out, lse, status, stream
PyObject* latent_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    Call c(a[0]);
    cosa_attn_params& p = c.p;
    const int64_t H = p.num_q_heads, d = p.head_dim, rows = c.query_rows();
    const void* q = c.rows(a[1], "q_nope", p.total_tokens, H, d, &p.q_stride, &p.q_head_stride);
    const void* qr = c.rows(a[2], "q_rope", p.total_tokens, H, kRot, &p.q_rope_stride, &p.q_rope_head_stride);
    const void* k = c.rows(a[3], "k_nope", p.total_kv_tokens, H, d, &p.k_stride, &p.k_head_stride);
    const void* kr = c.rows(a[4], "k_rope", p.total_kv_tokens, 0, kRot, &p.k_rope_stride, nullptr);
    const void* v = c.rows(a[5], "v", p.total_kv_tokens, H, d, &p.v_stride, &p.v_head_stride);
    const int32_t* cu = c.ints(a[6], "cu_seqlens", int64_t{p.num_reqs} + 1);
    const int32_t* cu_kv = c.ints(a[7], "cu_kv", int64_t{p.num_reqs} + 1);
    void* out = c.bf16(a[8], "out", rows * d);
    float* lse = c.dense<float>(a[9], "lse", at::kFloat, rows);
    return c.run(a[10], a[11], [&](int32_t* status, void* stream) {
      return latent_prefill_fn(&p, q, qr, k, kr, v, cu, cu_kv, out, lse, status, stream);
    });
  });
}

// The library's functions, by address, in the order of the calls above.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    void* f[5];
    for (int i = 0; i < 5; ++i) {
      f[i] = PyLong_AsVoidPtr(a[i]);
      if (PyErr_Occurred()) throw Refused{};
    }
    tree_attention_fn = reinterpret_cast<decltype(tree_attention_fn)>(f[0]);
    latent_attention_fn = reinterpret_cast<decltype(latent_attention_fn)>(f[1]);
    tree_commit_fn = reinterpret_cast<decltype(tree_commit_fn)>(f[2]);
    latent_rope_fn = reinterpret_cast<decltype(latent_rope_fn)>(f[3]);
    latent_prefill_fn = reinterpret_cast<decltype(latent_prefill_fn)>(f[4]);
    Py_RETURN_NONE;
  });
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"tree_attention", fast(tree_attention), METH_FASTCALL, nullptr},
                         {"latent_attention", fast(latent_attention), METH_FASTCALL, nullptr},
                         {"tree_commit", fast(tree_commit), METH_FASTCALL, nullptr},
                         {"latent_rope", fast(latent_rope), METH_FASTCALL, nullptr},
                         {"latent_prefill", fast(latent_prefill), METH_FASTCALL, nullptr},
                         {"bind", fast(bind), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_call", "Checked calls of libcosa_attn.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_call() { return PyModule_Create(&module); }
