// Native half of the Python binding for the serving calls: checks the tensors of a call, reads
// their shapes and pointers, and calls the C ABI (include/pa.h) with the GIL released.
//
// A small call on the GPU takes 4 to 8 us; the same checks made from Python, tensor by tensor, and
// the marshalling of some 20 arguments took the host 8 to 12 us before its launches' own 2 to 4.
// Positional arguments only: binding.py has the names, defaults and documentation.  A function
// returns the PA_* code; a tensor of the wrong type, device or shape raises ValueError.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdexcept>
#include <string>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pa.h"

namespace {

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

void require(bool ok, const char* what) {
  if (!ok) throw Refused(what);
}

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kI64 = at::kLong, kU8 = at::kByte;

// The arguments of one call.  Tensors are contiguous and on the current device.
class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t given, Py_ssize_t wanted) : a_(a) {
    if (given != wanted) throw Refused("wrong number of arguments");
  }
  const at::Tensor& tensor(int i, const char* name, at::ScalarType type) {
    if (!THPVariable_Check(a_[i])) throw Refused(std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(a_[i]);
    if (t.scalar_type() != type)
      throw Refused(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (!t.is_cuda() || t.device().index() != device())
      throw Refused(std::string(name) + " must be a CUDA tensor on the current device");
    if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
    return t;
  }
  int integer(int i) {
    const long v = PyLong_AsLong(a_[i]);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    if (v < INT32_MIN || v > INT32_MAX) throw Refused("an integer argument does not fit 32 bits");
    return static_cast<int>(v);
  }
  double real(int i) {
    const double v = PyFloat_AsDouble(a_[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
  }
  // None: the current stream of the current device; otherwise a stream handle.
  void* stream(int i) {
    if (a_[i] == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device())).stream();
    void* s = PyLong_AsVoidPtr(a_[i]);
    if (!s && PyErr_Occurred()) throw Raised();
    return s;
  }
  struct Raised {};  // a Python exception is set

 private:
  int device() {
    if (device_ < 0) device_ = c10::cuda::current_device();
    return device_;
  }
  PyObject* const* a_;
  int device_ = -1;
};

int size32(const at::Tensor& t, int d) {
  const int64_t n = t.size(d);
  if (n > INT32_MAX) throw Refused("a dimension does not fit 32 bits");
  return static_cast<int>(n);
}

bool is(const at::Tensor& t, std::initializer_list<int64_t> shape) { return t.sizes() == at::IntArrayRef(shape); }

// Runs one binding function: exceptions become Python ones, the result its PA_* code.
template <typename F>
PyObject* guarded(F&& body) {
  try {
    return PyLong_FromLong(body());
  } catch (const Args::Raised&) {
    return nullptr;
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <typename F>
int without_gil(F&& call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call();
  Py_END_ALLOW_THREADS
  return rc;
}

struct Cache {
  const at::Tensor& k;
  const at::Tensor& v;
  int num_blocks, kv_heads, block_size, head_dim;
  Cache(Args& a, int i, at::ScalarType type)
      : k(a.tensor(i, "k_cache", type)), v(a.tensor(i + 1, "v_cache", type)) {
    require(k.dim() == 4, "k_cache must be [num_blocks, num_kv_heads, block_size, head_dim]");
    require(v.sizes() == k.sizes(), "k_cache and v_cache differ in shape");
    num_blocks = size32(k, 0);
    kv_heads = size32(k, 1);
    block_size = size32(k, 2);
    head_dim = size32(k, 3);
  }
  float* scales(Args& a, int i) const {
    const at::Tensor& s = a.tensor(i, "kv_scale", kF32);
    require(is(s, {num_blocks, kv_heads, 2}), "kv_scale must be [num_blocks, num_kv_heads, 2]");
    return static_cast<float*>(s.data_ptr());
  }
};

pa_dims dims_of(const at::Tensor& q, const Cache& c) {
  require(q.dim() == 3 && q.size(2) == c.head_dim, "q must be [rows, num_q_heads, head_dim of the caches]");
  return pa_dims{size32(q, 1), c.kv_heads, c.head_dim, c.block_size};
}

// The 4-bit cache: one tensor of records.
struct Cache4 {
  const at::Tensor& t;
  int num_blocks, kv_heads;
  Cache4(Args& a, int i) : t(a.tensor(i, "cache", kU8)) {
    require(t.dim() == 3 && t.size(2) == PA_INT4_RECORD_BYTES, "cache must be [num_blocks, num_kv_heads, 2208]");
    num_blocks = size32(t, 0);
    kv_heads = size32(t, 1);
  }
  pa_dims dims(const at::Tensor& q) const {
    require(q.dim() == 3 && q.size(2) == 128, "q must be [rows, num_q_heads, 128]");
    return pa_dims{size32(q, 1), kv_heads, 128, 16};
  }
};

pa_rope rope_of(const at::Tensor& cos_sin, int layout) {
  require(cos_sin.dim() == 2, "cos_sin must be [max_pos, rotary_dim]");
  return pa_rope{size32(cos_sin, 1), layout};
}

template <typename T>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// kind, theta, factor, original_max_pos, low, high, magnitude, rotary_dim, max_pos, out, stream
PyObject* rope_table(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 11);
    const pa_rope_scaling s{a.real(1), a.real(2), a.real(3), a.real(4), a.real(5), a.real(6), a.integer(0)};
    const int R = a.integer(7), P = a.integer(8);
    const at::Tensor& out = a.tensor(9, "out", kF32);
    require(is(out, {P, R}), "out must be [max_pos, rotary_dim]");
    void* stream = a.stream(10);
    return without_gil([&] { return pa_rope_table(&s, R, P, ptr<float>(out), stream); });
  });
}

// q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, (kv_scale,) layout, q_out, stream
template <bool kBlock>
PyObject* rope_store(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, kBlock ? 12 : 11);
    const at::Tensor& q = a.tensor(0, "q", kBf16);
    const at::Tensor& k = a.tensor(1, "k", kBf16);
    const at::Tensor& v = a.tensor(2, "v", kBf16);
    const at::Tensor& pos = a.tensor(3, "positions", kI32);
    const at::Tensor& cs = a.tensor(4, "cos_sin", kF32);
    const at::Tensor& slots = a.tensor(5, "slot_mapping", kI64);
    const Cache c(a, 6, kBlock ? kU8 : kBf16);
    float* scale = kBlock ? c.scales(a, 8) : nullptr;
    constexpr int rest = kBlock ? 9 : 8;
    const pa_rope rope = rope_of(cs, a.integer(rest));
    const at::Tensor& out = a.tensor(rest + 1, "q_out", kBf16);
    const pa_dims d = dims_of(q, c);
    const int T = size32(q, 0);
    require(is(k, {T, c.kv_heads, c.head_dim}) && k.sizes() == v.sizes(), "k and v must be [rows of q, num_kv_heads, head_dim]");
    require(out.sizes() == q.sizes(), "q_out must have the shape of q");
    require(is(pos, {T}) && is(slots, {T}), "positions and slot_mapping must be [rows of q]");
    const int P = size32(cs, 0);
    void* stream = a.stream(rest + 2);
    return without_gil([&] {
      if (kBlock)
        return pa_rope_kv_store_fp8_block(&d, &rope, T, q.data_ptr(), out.data_ptr(), k.data_ptr(), v.data_ptr(), ptr<int32_t>(pos),
                                          ptr<float>(cs), P, ptr<int64_t>(slots), c.k.data_ptr(), c.v.data_ptr(), scale,
                                          c.num_blocks, stream);
      return pa_rope_kv_store_form(&d, &rope, T, q.data_ptr(), out.data_ptr(), k.data_ptr(), v.data_ptr(), ptr<int32_t>(pos),
                                   ptr<float>(cs), P, ptr<int64_t>(slots), c.k.data_ptr(), c.v.data_ptr(), c.num_blocks, stream);
    });
  });
}

struct Batch {
  const at::Tensor& tables;
  const at::Tensor& lens;
  int max_blocks;
  Batch(Args& a, int i, int num_seqs)
      : tables(a.tensor(i, "block_tables", kI32)), lens(a.tensor(i + 1, "context_lens", kI32)) {
    require(tables.dim() == 2 && tables.size(0) == num_seqs, "block_tables must be [num_seqs, max_blocks]");
    require(is(lens, {num_seqs}), "context_lens must be [num_seqs]");
    max_blocks = size32(tables, 1);
  }
};

// q, k_cache, v_cache, kv_scale, block_tables, context_lens, max_context_len, scale, partition_tokens,
// workspace, out, stream
PyObject* decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 12);
    const at::Tensor& q = a.tensor(0, "q", kBf16);
    const Cache c(a, 1, kU8);
    const float* scale = c.scales(a, 3);
    const pa_dims d = dims_of(q, c);
    const int S = size32(q, 0);
    const Batch b(a, 4, S);
    const at::Tensor& ws = a.tensor(9, "workspace", kF32);
    const at::Tensor& out = a.tensor(10, "out", kBf16);
    require(out.sizes() == q.sizes(), "out must have the shape of q");
    const int max_ctx = a.integer(6), P = a.integer(8);
    const float sm = static_cast<float>(a.real(7));
    void* stream = a.stream(11);
    return without_gil([&] {
      return pa_decode_fp8_block(&d, S, q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), scale, c.num_blocks,
                                 ptr<int32_t>(b.tables), b.max_blocks, ptr<int32_t>(b.lens), max_ctx, sm, P, ws.data_ptr(),
                                 static_cast<size_t>(ws.numel()) * 4, out.data_ptr(), stream);
    });
  });
}

// q, k, v, cos_sin, k_cache, v_cache, kv_scale, block_tables, context_lens, max_context_len, scale, layout,
// partition_tokens, workspace, out, flags, stream
PyObject* decode_step(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 17);
    const at::Tensor& q = a.tensor(0, "q", kBf16);
    const at::Tensor& k = a.tensor(1, "k", kBf16);
    const at::Tensor& v = a.tensor(2, "v", kBf16);
    const at::Tensor& cs = a.tensor(3, "cos_sin", kF32);
    const Cache c(a, 4, kU8);
    float* scale = c.scales(a, 6);
    const pa_dims d = dims_of(q, c);
    const int S = size32(q, 0);
    const Batch b(a, 7, S);
    require(is(k, {S, c.kv_heads, c.head_dim}) && k.sizes() == v.sizes(), "k and v must be [num_seqs, num_kv_heads, head_dim]");
    const pa_rope rope = rope_of(cs, a.integer(11));
    const at::Tensor& ws = a.tensor(13, "workspace", kF32);
    const at::Tensor& out = a.tensor(14, "out", kBf16);
    require(out.sizes() == q.sizes(), "out must have the shape of q");
    const int max_ctx = a.integer(9), P = a.integer(12), rows = size32(cs, 0);
    const unsigned flags = static_cast<unsigned>(a.integer(15));
    const float sm = static_cast<float>(a.real(10));
    void* stream = a.stream(16);
    return without_gil([&] {
      return pa_decode_step_fp8_block(&d, &rope, S, q.data_ptr(), k.data_ptr(), v.data_ptr(), ptr<float>(cs), rows,
                                      c.k.data_ptr(), c.v.data_ptr(), scale, c.num_blocks, ptr<int32_t>(b.tables),
                                      b.max_blocks, ptr<int32_t>(b.lens), max_ctx, sm, P, ws.data_ptr(),
                                      static_cast<size_t>(ws.numel()) * 4, out.data_ptr(), flags, stream);
    });
  });
}

// q, q_start, k_cache, v_cache, kv_scale, block_tables, context_lens, max_query_len, max_context_len, scale,
// out, stream
PyObject* prefill(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 12);
    const at::Tensor& q = a.tensor(0, "q", kBf16);
    const at::Tensor& starts = a.tensor(1, "q_start", kI32);
    const Cache c(a, 2, kU8);
    const float* scale = c.scales(a, 4);
    const pa_dims d = dims_of(q, c);
    require(starts.dim() == 1 && starts.size(0) >= 1, "q_start must be [num_seqs + 1]");
    const int S = size32(starts, 0) - 1;
    const Batch b(a, 5, S);
    const at::Tensor& out = a.tensor(10, "out", kBf16);
    require(out.sizes() == q.sizes(), "out must have the shape of q");
    const int T = size32(q, 0), max_q = a.integer(7), max_ctx = a.integer(8);
    const float sm = static_cast<float>(a.real(9));
    void* stream = a.stream(11);
    return without_gil([&] {
      return pa_prefill_fp8_block(&d, S, T, q.data_ptr(), ptr<int32_t>(starts), max_q, c.k.data_ptr(), c.v.data_ptr(), scale,
                                  c.num_blocks, ptr<int32_t>(b.tables), b.max_blocks, ptr<int32_t>(b.lens), max_ctx, sm,
                                  out.data_ptr(), stream);
    });
  });
}

// q, k, v, positions, cos_sin, slot_mapping, cache, layout, q_out, stream
PyObject* rope_store_int4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 10);
    const at::Tensor& q = a.tensor(0, "q", kBf16);
    const at::Tensor& k = a.tensor(1, "k", kBf16);
    const at::Tensor& v = a.tensor(2, "v", kBf16);
    const at::Tensor& pos = a.tensor(3, "positions", kI32);
    const at::Tensor& cs = a.tensor(4, "cos_sin", kF32);
    const at::Tensor& slots = a.tensor(5, "slot_mapping", kI64);
    const Cache4 c(a, 6);
    const pa_rope rope = rope_of(cs, a.integer(7));
    const at::Tensor& out = a.tensor(8, "q_out", kBf16);
    const pa_dims d = c.dims(q);
    const int T = size32(q, 0);
    require(is(k, {T, c.kv_heads, 128}) && k.sizes() == v.sizes(), "k and v must be [rows of q, num_kv_heads, 128]");
    require(out.sizes() == q.sizes(), "q_out must have the shape of q");
    require(is(pos, {T}) && is(slots, {T}), "positions and slot_mapping must be [rows of q]");
    const int P = size32(cs, 0);
    void* stream = a.stream(9);
    return without_gil([&] {
      return pa_rope_kv_store_int4(&d, &rope, T, q.data_ptr(), out.data_ptr(), k.data_ptr(), v.data_ptr(), ptr<int32_t>(pos),
                                   ptr<float>(cs), P, ptr<int64_t>(slots), c.t.data_ptr(), c.num_blocks, stream);
    });
  });
}

// cache, row_start, first (or None), block_tables, max_rows, k_out, v_out, stream
PyObject* read_kv_int4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 8);
    const Cache4 c(a, 0);
    const at::Tensor& starts = a.tensor(1, "row_start", kI32);
    require(starts.dim() == 1 && starts.size(0) >= 1, "row_start must be [num_seqs + 1]");
    const int S = size32(starts, 0) - 1;
    const int32_t* first = nullptr;
    if (args[2] != Py_None) {
      const at::Tensor& f = a.tensor(2, "first", kI32);
      require(is(f, {S}), "first must be [num_seqs]");
      first = ptr<int32_t>(f);
    }
    const at::Tensor& tables = a.tensor(3, "block_tables", kI32);
    require(tables.dim() == 2 && tables.size(0) == S, "block_tables must be [num_seqs, max_blocks]");
    const int max_rows = a.integer(4), max_blocks = size32(tables, 1);
    const at::Tensor& k = a.tensor(5, "k_out", kBf16);
    const at::Tensor& v = a.tensor(6, "v_out", kBf16);
    require(k.dim() == 3 && k.size(1) == c.kv_heads && k.size(2) == 128 && k.sizes() == v.sizes(),
            "k_out and v_out must be [rows, num_kv_heads, 128]");
    const int rows = size32(k, 0);
    const pa_dims d{c.kv_heads, c.kv_heads, 128, 16};
    void* stream = a.stream(7);
    return without_gil([&] {
      return pa_read_kv_int4(&d, S, rows, ptr<int32_t>(starts), first, max_rows, c.t.data_ptr(), c.num_blocks,
                             ptr<int32_t>(tables), max_blocks, k.data_ptr(), v.data_ptr(), stream);
    });
  });
}

// q, cache, block_tables, context_lens, max_context_len, scale, partition_tokens, workspace, out, stream
PyObject* decode_int4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 10);
    const at::Tensor& q = a.tensor(0, "q", kBf16);
    const Cache4 c(a, 1);
    const pa_dims d = c.dims(q);
    const int S = size32(q, 0);
    const Batch b(a, 2, S);
    const at::Tensor& ws = a.tensor(7, "workspace", kF32);
    const at::Tensor& out = a.tensor(8, "out", kBf16);
    require(out.sizes() == q.sizes(), "out must have the shape of q");
    const int max_ctx = a.integer(4), P = a.integer(6);
    const float sm = static_cast<float>(a.real(5));
    void* stream = a.stream(9);
    return without_gil([&] {
      return pa_decode_int4(&d, S, q.data_ptr(), c.t.data_ptr(), c.num_blocks, ptr<int32_t>(b.tables), b.max_blocks,
                            ptr<int32_t>(b.lens), max_ctx, sm, P, ws.data_ptr(), static_cast<size_t>(ws.numel()) * 4,
                            out.data_ptr(), stream);
    });
  });
}

// q, k, v, cos_sin, cache, block_tables, context_lens, max_context_len, scale, layout, partition_tokens, workspace,
// out, flags, stream
PyObject* decode_step_int4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 15);
    const at::Tensor& q = a.tensor(0, "q", kBf16);
    const at::Tensor& k = a.tensor(1, "k", kBf16);
    const at::Tensor& v = a.tensor(2, "v", kBf16);
    const at::Tensor& cs = a.tensor(3, "cos_sin", kF32);
    const Cache4 c(a, 4);
    const pa_dims d = c.dims(q);
    const int S = size32(q, 0);
    const Batch b(a, 5, S);
    require(is(k, {S, c.kv_heads, 128}) && k.sizes() == v.sizes(), "k and v must be [num_seqs, num_kv_heads, 128]");
    const pa_rope rope = rope_of(cs, a.integer(9));
    const at::Tensor& ws = a.tensor(11, "workspace", kF32);
    const at::Tensor& out = a.tensor(12, "out", kBf16);
    require(out.sizes() == q.sizes(), "out must have the shape of q");
    const int max_ctx = a.integer(7), P = a.integer(10), rows = size32(cs, 0);
    const unsigned flags = static_cast<unsigned>(a.integer(13));
    const float sm = static_cast<float>(a.real(8));
    void* stream = a.stream(14);
    return without_gil([&] {
      return pa_decode_step_int4(&d, &rope, S, q.data_ptr(), k.data_ptr(), v.data_ptr(), ptr<float>(cs), rows, c.t.data_ptr(),
                                 c.num_blocks, ptr<int32_t>(b.tables), b.max_blocks, ptr<int32_t>(b.lens), max_ctx, sm, P,
                                 ws.data_ptr(), static_cast<size_t>(ws.numel()) * 4, out.data_ptr(), flags, stream);
    });
  });
}

// q, q_start, cache, block_tables, context_lens, max_query_len, max_context_len, scale, out, stream
PyObject* prefill_int4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 10);
    const at::Tensor& q = a.tensor(0, "q", kBf16);
    const at::Tensor& starts = a.tensor(1, "q_start", kI32);
    const Cache4 c(a, 2);
    const pa_dims d = c.dims(q);
    require(starts.dim() == 1 && starts.size(0) >= 1, "q_start must be [num_seqs + 1]");
    const int S = size32(starts, 0) - 1;
    const Batch b(a, 3, S);
    const at::Tensor& out = a.tensor(8, "out", kBf16);
    require(out.sizes() == q.sizes(), "out must have the shape of q");
    const int T = size32(q, 0), max_q = a.integer(5), max_ctx = a.integer(6);
    const float sm = static_cast<float>(a.real(7));
    void* stream = a.stream(9);
    return without_gil([&] {
      return pa_prefill_int4(&d, S, T, q.data_ptr(), ptr<int32_t>(starts), max_q, c.t.data_ptr(), c.num_blocks,
                             ptr<int32_t>(b.tables), b.max_blocks, ptr<int32_t>(b.lens), max_ctx, sm, out.data_ptr(), stream);
    });
  });
}

// cached_lens, new_lens, block_tables, free_blocks, num_free, num_free_out, num_blocks, num_tokens, context_lens,
// q_start, positions, slot_mapping, granted, stream
PyObject* plan_step(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 14);
    const at::Tensor& cached = a.tensor(0, "cached_lens", kI32);
    const at::Tensor& fresh = a.tensor(1, "new_lens", kI32);
    const at::Tensor& tables = a.tensor(2, "block_tables", kI32);
    const at::Tensor& pool = a.tensor(3, "free_blocks", kI32);
    const at::Tensor& left = a.tensor(4, "num_free", kI32);
    const at::Tensor& left_out = a.tensor(5, "num_free_out", kI32);
    const int num_blocks = a.integer(6), T = a.integer(7);
    const at::Tensor& ctx = a.tensor(8, "context_lens", kI32);
    const at::Tensor& starts = a.tensor(9, "q_start", kI32);
    const at::Tensor& pos = a.tensor(10, "positions", kI32);
    const at::Tensor& slots = a.tensor(11, "slot_mapping", kI64);
    const at::Tensor& granted = a.tensor(12, "granted", kI32);
    require(cached.dim() == 1 && fresh.sizes() == cached.sizes(), "cached_lens and new_lens must be [num_seqs]");
    const int S = size32(cached, 0);
    require(tables.dim() == 2 && tables.size(0) == S, "block_tables must be [num_seqs, max_blocks]");
    require(pool.dim() == 1 && left.numel() == 1 && left_out.numel() == 1,
            "free_blocks must be [capacity], num_free and num_free_out [1]");
    require(is(ctx, {S}) && is(starts, {S + 1}) && is(granted, {S}) && is(pos, {T}) && is(slots, {T}),
            "the plan does not fit these sequences and rows");
    const pa_dims d{1, 1, 128, 16};  // the plan depends on the block size alone
    const int max_blocks = size32(tables, 1), capacity = size32(pool, 0);
    void* stream = a.stream(13);
    return without_gil([&] {
      return pa_plan_step(&d, S, ptr<int32_t>(cached), ptr<int32_t>(fresh), ptr<int32_t>(tables), max_blocks,
                          ptr<int32_t>(pool), capacity, ptr<int32_t>(left), ptr<int32_t>(left_out), num_blocks, T,
                          ptr<int32_t>(ctx), ptr<int32_t>(starts), ptr<int32_t>(pos), ptr<int64_t>(slots),
                          ptr<int32_t>(granted), stream);
    });
  });
}

#define PA_FAST(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {PA_FAST("rope_table", rope_table),
                          PA_FAST("rope_kv_store_form", rope_store<false>),
                          PA_FAST("rope_kv_store_fp8_block", rope_store<true>),
                          PA_FAST("decode_fp8_block", decode),
                          PA_FAST("decode_step_fp8_block", decode_step),
                          PA_FAST("prefill_fp8_block", prefill),
                          PA_FAST("plan_step", plan_step),
                          PA_FAST("rope_kv_store_int4", rope_store_int4),
                          PA_FAST("read_kv_int4", read_kv_int4),
                          PA_FAST("decode_int4", decode_int4),
                          PA_FAST("decode_step_int4", decode_step_int4),
                          PA_FAST("prefill_int4", prefill_int4),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_pa_torch", "Native half of binding.py.", -1, kMethods,
                       nullptr,               nullptr,     nullptr,                      nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_torch() { return PyModule_Create(&kModule); }
