// The Python calls of the operators around paged attention, of those on pages and of the biased
// attention, for the common case.
//
// A decode step's operators run for a few microseconds each, less than Python needs to look
// at a dozen tensors. These functions make the same checks as step.py, pool.py and biased.py and call the same C
// entry points (whose addresses step.py hands over); they allocate the outputs as torch does,
// on the current stream. Anything unusual - another type, device or layout, an argument that
// an entry point refuses, an exception - returns None without a trace: the Python then makes the
// call itself and says what was wrong.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "pagedattn.h"

namespace {

decltype(&pa_build_block_tables) build_block_tables_fn;
decltype(&pa_qk_norm_rope) qk_norm_rope_fn;
decltype(&pa_update_page_bounds) update_page_bounds_fn;
decltype(&pa_select_pages) select_pages_fn;
decltype(&pa_sparse_paged_attention) sparse_paged_attention_fn;
decltype(&pa_fork_block_tables) fork_block_tables_fn;
decltype(&pa_compact_block_tables) compact_block_tables_fn;
decltype(&pa_copy_pages) copy_pages_fn;
decltype(&pa_biased_paged_attention) biased_paged_attention_fn;
decltype(&pa_pool_workspace_size) pool_workspace_size_fn;
decltype(&pa_biased_workspace_size) biased_workspace_size_fn;

struct Unusual {};

void need(bool ok) {
  if (!ok) throw Unusual();
}

const at::Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

bool is_none(PyObject* o) { return o == Py_None; }

int64_t integer(PyObject* o) {
  need(PyLong_Check(o));
  const int64_t v = PyLong_AsLongLong(o);
  need(v >= INT32_MIN && v <= INT32_MAX);
  return v;
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    throw Unusual();
  }
  return (float)v;
}

// one that is not 0 in 32 bits unless it is 0
float real_or_0(PyObject* o) {
  const float v = real(o);
  need(v != 0.f || PyFloat_AsDouble(o) == 0.);
  return v;
}

// the device that the call's tensors are on, which must be the current one
struct Call {
  c10::Device device;
  explicit Call(const at::Tensor& t) : device(t.device()) {
    need(t.is_cuda() && device.index() == c10::cuda::current_device());
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
  const at::Tensor& whole(PyObject* o, at::ScalarType type, int64_t dim) const {
    const at::Tensor& t = tensor(o);
    need(t.scalar_type() == type && t.device() == device && t.dim() == dim && t.is_contiguous());
    return t;
  }
  int32_t* ints(PyObject* o, int64_t n) const {
    const at::Tensor& t = whole(o, at::kInt, 1);
    need(t.size(0) == n);
    return (int32_t*)t.data_ptr();
  }
  uint32_t* error(PyObject* o) const {
    if (is_none(o)) return nullptr;
    const at::Tensor& t = tensor(o);
    need(t.scalar_type() == at::kInt && t.device() == device && t.numel() == 1);
    return (uint32_t*)t.data_ptr();
  }
  // the stride of a 2-D tensor with contiguous rows of `width`
  int64_t rows(const at::Tensor& t, at::ScalarType type, int64_t width) const {
    need(t.scalar_type() == type && t.device() == device && t.dim() == 2 && t.size(1) == width && t.stride(1) == 1 &&
         t.size(0) > 0);
    const int64_t stride = t.stride(0);
    return t.size(0) > 1 ? stride : ((stride > width ? stride : width) + 7) / 8 * 8;
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(device));
  }
};

int32_t dtype_code(at::ScalarType t) {
  need(t == at::kHalf || t == at::kBFloat16);
  return t == at::kHalf ? PA_FLOAT16 : PA_BFLOAT16;
}

int32_t i32(int64_t v) {
  need(v >= 0 && v <= INT32_MAX);
  return (int32_t)v;
}

// (batch_size, columns) of the batch description
struct Batch {
  const int32_t *cum, *past, *table;
  int32_t size, columns;
  Batch(const Call& call, PyObject* cum_o, PyObject* past_o, PyObject* table_o) {
    const at::Tensor& p = call.whole(past_o, at::kInt, 1);
    const at::Tensor& t = call.whole(table_o, at::kInt, 2);
    size = i32(p.size(0));
    columns = i32(t.size(1));
    need(t.size(0) == size);
    cum = call.ints(cum_o, (int64_t)size + 1);
    past = (const int32_t*)p.data_ptr();
    table = (const int32_t*)t.data_ptr();
  }
};

// An entry point called without the interpreter's lock, as ctypes makes its calls: a launch
// waits while the stream's queue is full, and what it waits for may be another Python thread.
// (The arguments are plain values, worked out before.)
template <typename... P, typename... A>
pa_status unlocked(pa_status (*f)(P...), A... args) {
  struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
  } now;
  return f(args...);
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  try {
    need(n == want);
    at::AutoDispatchBelowADInplaceOrView guard;
    return f();
  } catch (...) {
  }
  if (PyErr_Occurred()) PyErr_Clear();
  Py_RETURN_NONE;
}

// tensors of their own over pieces of one allocation of int32
at::Tensor piece_of(const at::Tensor& all, int64_t at, at::IntArrayRef shape) {
  at::Tensor piece = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
  piece.unsafeGetTensorImpl()->set_storage_offset(at);
  piece.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return piece;
}

// (past, query_lens, held, table, ring, state, block_size, num_tokens) -> the six outputs
PyObject* build_block_tables(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor& table = tensor(v[3]);
    const Call call(table);
    call.whole(v[3], at::kInt, 2);
    const int64_t B = table.size(0), N = integer(v[7]);
    need(N >= 0);
    const at::Tensor& ring = call.whole(v[4], at::kInt, 1);
    const int32_t *past = call.ints(v[0], B), *q = call.ints(v[1], B), *held = call.ints(v[2], B),
                  *state = call.ints(v[5], 2);
    const int64_t sizes[6] = {B + 1, N, N, B, 2, 1};
    const at::Tensor all = call.empty({2 * (B + N + 2)}, at::kInt);
    int32_t* p = (int32_t*)all.data_ptr();
    need(unlocked(build_block_tables_fn, past, q, held, (int32_t*)table.data_ptr(), (int32_t*)ring.data_ptr(), state,
                  i32(B), i32(N), i32(table.size(1)), (int32_t)integer(v[6]), i32(ring.size(0)), p, p + B + 1,
                  p + B + 1 + N, p + B + 1 + 2 * N, p + 2 * B + 1 + 2 * N, (uint32_t*)(p + 2 * B + 3 + 2 * N),
                  call.stream()) == PA_OK);
    PyObject* out = PyTuple_New(6);
    need(out != nullptr);
    int64_t at = 0;
    for (int i = 0; i < 6; ++i) {
      PyTuple_SET_ITEM(out, i, THPVariable_Wrap(piece_of(all, at, {sizes[i]})));
      at += sizes[i];
    }
    return out;
  });
}

// (query, key, positions, heads, kv_heads, q_weight, k_weight, eps, rotary_dim, theta, interleaved)
PyObject* qk_norm_rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor &query = tensor(v[0]), &key = tensor(v[1]);
    const Call call(query);
    const at::ScalarType type = query.scalar_type();
    const int32_t code = dtype_code(type);
    const int64_t nh = integer(v[3]), kvh = integer(v[4]);
    need(nh > 0 && kvh > 0 && query.dim() == 2 && query.size(1) % nh == 0);
    const int64_t N = query.size(0), hs = query.size(1) / nh;
    const int64_t qs = call.rows(query, type, nh * hs), ks = call.rows(key, type, kvh * hs);
    need(key.size(0) == N);
    auto weight = [&](PyObject* o) -> const void* {
      if (is_none(o)) return nullptr;
      const at::Tensor& w = call.whole(o, type, 1);
      need(w.size(0) == hs);
      return w.data_ptr();
    };
    const pa_qk_prep prep = {weight(v[5]), weight(v[6]), real(v[7]), real(v[9]), (int32_t)integer(v[8]), 0};
    const int interleaved = PyObject_IsTrue(v[10]);
    need(interleaved >= 0);
    const int32_t* positions = call.ints(v[2], N);
    const at::Tensor qo = call.empty({N, nh * hs}, type), ko = call.empty({N, kvh * hs}, type);
    need(unlocked(qk_norm_rope_fn, query.data_ptr(), key.data_ptr(), positions, &prep, interleaved, i32(N), i32(nh),
                  i32(kvh), i32(hs), code, qs, ks, qo.data_ptr(), ko.data_ptr(), nh * hs, kvh * hs,
                  call.stream()) == PA_OK);
    PyObject* out = PyTuple_New(2);
    need(out != nullptr);
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(qo));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(ko));
    return out;
  });
}

const at::Tensor& bounds_of(const Call& call, PyObject* bounds, PyObject* scale, int64_t kvh, const float** s) {
  const at::Tensor& b = call.whole(bounds, at::kChar, 4);
  const at::Tensor& c = call.whole(scale, at::kFloat, 2);
  need(b.size(1) == kvh && b.size(2) == 2 && c.size(0) == kvh && c.size(1) == b.size(3));
  *s = (const float*)c.data_ptr();
  return b;
}

// (key_cache, bounds, scale, cum, past, table, num_tokens, error) -> True
PyObject* update_page_bounds(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor& cache = tensor(v[0]);
    const Call call(cache);
    const int32_t code = dtype_code(cache.scalar_type());
    call.whole(v[0], cache.scalar_type(), 4);
    const float* scale;
    const at::Tensor& bounds = bounds_of(call, v[1], v[2], cache.size(2), &scale);
    need(bounds.size(0) == cache.size(0) && bounds.size(3) == cache.size(3));
    const Batch b(call, v[3], v[4], v[5]);
    pa_sparse_dims d{};
    d.num_tokens = i32(integer(v[6]));
    d.batch_size = b.size;
    d.num_heads = d.kv_num_heads = i32(cache.size(2));
    d.head_size = i32(cache.size(3));
    d.num_blocks = i32(cache.size(0));
    d.block_size = i32(cache.size(1));
    d.max_blocks_per_sequence = b.columns;
    d.dtype = code;
    need(unlocked(update_page_bounds_fn, cache.data_ptr(), (int8_t*)bounds.data_ptr(), scale, b.cum, b.past, b.table,
                  &d, call.error(v[7]), call.stream()) == PA_OK);
    Py_RETURN_TRUE;
  });
}

// (query, bounds, scale, cum, past, table, heads, kv_heads, block_size, top_k, query_block, sink, local, error)
PyObject* select_pages(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const at::Tensor& query = tensor(v[0]);
    const Call call(query);
    const at::ScalarType type = query.scalar_type();
    const float* scale;
    pa_sparse_dims d{};
    d.dtype = dtype_code(type);
    d.num_heads = i32(integer(v[6]));
    d.kv_num_heads = i32(integer(v[7]));
    const at::Tensor& bounds = bounds_of(call, v[1], v[2], d.kv_num_heads, &scale);
    const int64_t hs = bounds.size(3);
    const Batch b(call, v[3], v[4], v[5]);
    d.query_stride = call.rows(query, type, d.num_heads * hs);
    d.num_tokens = i32(query.size(0));
    d.batch_size = b.size;
    d.head_size = i32(hs);
    d.num_blocks = i32(bounds.size(0));
    d.block_size = i32(integer(v[8]));
    d.max_blocks_per_sequence = b.columns;
    d.top_k = i32(integer(v[9]));
    d.query_block = i32(integer(v[10]));
    d.sink_pages = i32(integer(v[11]));
    d.local_pages = i32(integer(v[12]));
    uint32_t* error = call.error(v[13]);
    const at::Tensor out = call.empty({query.size(0), d.kv_num_heads, d.top_k}, at::kInt);
    need(unlocked(select_pages_fn, query.data_ptr(), (const int8_t*)bounds.data_ptr(), scale, b.cum, b.past, b.table,
                  &d, (int32_t*)out.data_ptr(), error, call.stream()) == PA_OK);
    return THPVariable_Wrap(out);
  });
}

// (query, key_cache, value_cache, cum, past, table, selected, heads, kv_heads, scale, query_block, lse, error)
PyObject* sparse_paged_attention(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const at::Tensor& query = tensor(v[0]);
    const Call call(query);
    const at::ScalarType type = query.scalar_type();
    pa_sparse_dims d{};
    d.dtype = dtype_code(type);
    const at::Tensor &k = call.whole(v[1], type, 4), &value = call.whole(v[2], type, 4);
    need(value.sizes() == k.sizes());
    const Batch b(call, v[3], v[4], v[5]);
    const int64_t N = query.size(0);
    const at::Tensor& selected = call.whole(v[6], at::kInt, 3);
    d.num_heads = i32(integer(v[7]));
    d.kv_num_heads = i32(integer(v[8]));
    need(k.size(2) == d.kv_num_heads && selected.size(0) == N && selected.size(1) == d.kv_num_heads);
    d.query_stride = call.rows(query, type, d.num_heads * k.size(3));
    d.num_tokens = i32(N);
    d.batch_size = b.size;
    d.head_size = i32(k.size(3));
    d.num_blocks = i32(k.size(0));
    d.block_size = i32(k.size(1));
    d.max_blocks_per_sequence = b.columns;
    d.top_k = i32(selected.size(2));
    d.query_block = i32(integer(v[10]));
    d.local_pages = 1;
    float* lse = nullptr;
    if (!is_none(v[11])) {
      const at::Tensor& l = call.whole(v[11], at::kFloat, 2);
      need(l.size(0) == N && l.size(1) == d.num_heads);
      lse = (float*)l.data_ptr();
    }
    uint32_t* error = call.error(v[12]);
    const float scale = real(v[9]);
    const at::Tensor out = call.empty({N, d.num_heads * k.size(3)}, type);
    need(unlocked(sparse_paged_attention_fn, query.data_ptr(), k.data_ptr(), value.data_ptr(), b.cum, b.past,
                  b.table, (const int32_t*)selected.data_ptr(), scale, out.data_ptr(), lse, &d, error,
                  call.stream()) == PA_OK);
    return THPVariable_Wrap(out);
  });
}

const uint8_t* pinned_of(const Call& call, PyObject* o, int64_t blocks) {
  if (is_none(o)) return nullptr;
  const at::Tensor& t = tensor(o);
  need(t.scalar_type() == at::kBool || t.scalar_type() == at::kByte);
  need(t.device() == call.device && t.dim() == 1 && t.size(0) == blocks && t.is_contiguous());
  return (const uint8_t*)t.data_ptr();
}

PyObject* tuple_of(std::initializer_list<at::Tensor> pieces) {
  PyObject* out = PyTuple_New((Py_ssize_t)pieces.size());
  need(out != nullptr);
  Py_ssize_t i = 0;
  for (const at::Tensor& t : pieces) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(t));
  return out;
}

// (parents, past, held, table, ring, state, pinned, block_size, num_blocks) -> the six outputs
PyObject* fork_block_tables(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& table = tensor(v[3]);
    const Call call(table);
    call.whole(v[3], at::kInt, 2);
    const int64_t B = table.size(0), cols = table.size(1), blocks = integer(v[8]);
    const at::Tensor &parents = call.whole(v[0], at::kInt, 1), &ring = call.whole(v[4], at::kInt, 1);
    const int64_t N = parents.size(0);
    const int32_t *past = call.ints(v[1], B), *held = call.ints(v[2], B), *state = call.ints(v[5], 2);
    const uint8_t* pins = pinned_of(call, v[6], blocks);
    const size_t bytes = pool_workspace_size_fn(i32(blocks));
    need(bytes > 0);
    const at::Tensor all = call.empty({N * (cols + 4) + 3}, at::kInt), ws = call.empty({(int64_t)bytes}, at::kByte);
    int32_t* p = (int32_t*)all.data_ptr();  // copies, table, past, held, state, error
    const int64_t t = 2 * N, q = t + N * cols, h = q + N, s = h + N;
    need(unlocked(fork_block_tables_fn, (const int32_t*)parents.data_ptr(), past, held, (const int32_t*)table.data_ptr(),
                  (int32_t*)ring.data_ptr(), state, pins, i32(B), i32(N), i32(cols), (int32_t)integer(v[7]),
                  i32(blocks), i32(ring.size(0)), p + q, p + h, p + t, p, p + s, (uint32_t*)(p + s + 2),
                  ws.data_ptr(), bytes, call.stream()) == PA_OK);
    return tuple_of({piece_of(all, q, {N}), piece_of(all, h, {N}), piece_of(all, t, {N, cols}), piece_of(all, 0, {N, 2}),
                     piece_of(all, s, {2}), piece_of(all, s + 2, {1})});
  });
}

// (held, table, ring, pinned, num_blocks, max_moves) -> the five outputs
PyObject* compact_block_tables(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor& table = tensor(v[1]);
    const Call call(table);
    call.whole(v[1], at::kInt, 2);
    const int64_t B = table.size(0), cols = table.size(1), blocks = integer(v[4]), moves = integer(v[5]);
    need(moves >= 0);
    const int32_t* held = call.ints(v[0], B);
    const at::Tensor& ring = call.whole(v[2], at::kInt, 1);
    const uint8_t* pins = pinned_of(call, v[3], blocks);
    const size_t bytes = pool_workspace_size_fn(i32(blocks));
    need(bytes > 0);
    const at::Tensor all = call.empty({2 * moves + B * cols + 4}, at::kInt), ws = call.empty({(int64_t)bytes}, at::kByte);
    int32_t* p = (int32_t*)all.data_ptr();  // copies, table, state, end, error
    const int64_t t = 2 * moves, s = t + B * cols;
    need(unlocked(compact_block_tables_fn, held, (const int32_t*)table.data_ptr(), (int32_t*)ring.data_ptr(), pins,
                  i32(B), i32(cols), i32(blocks), i32(ring.size(0)), i32(moves), p + t, p, p + s, p + s + 2,
                  (uint32_t*)(p + s + 3), ws.data_ptr(), bytes, call.stream()) == PA_OK);
    return tuple_of({piece_of(all, t, {B, cols}), piece_of(all, 0, {moves, 2}), piece_of(all, s, {2}),
                     piece_of(all, s + 2, {1}), piece_of(all, s + 3, {1})});
  });
}

// (tensors, copies, error) -> True
PyObject* copy_pages(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    need(PyList_Check(v[0]) || PyTuple_Check(v[0]));
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(v[0]);
    need(count > 0 && count <= PA_MAX_COPY_TENSORS);
    const at::Tensor& copies = tensor(v[1]);
    const Call call(copies);
    call.whole(v[1], at::kInt, 2);
    need(copies.size(1) == 2);
    pa_page_tensor pages[PA_MAX_COPY_TENSORS];
    int64_t blocks = 0;
    for (Py_ssize_t i = 0; i < count; ++i) {
      const at::Tensor& t = tensor(PySequence_Fast_ITEMS(v[0])[i]);
      need(t.device() == call.device && t.dim() > 0 && t.is_contiguous());
      if (i == 0) blocks = t.size(0);
      need(t.size(0) == blocks && blocks > 0);
      pages[i] = {t.data_ptr(), t.numel() / blocks * (int64_t)t.element_size()};
    }
    uint32_t* error = call.error(v[2]);
    need(unlocked(copy_pages_fn, (const pa_page_tensor*)pages, (int32_t)count, i32(blocks),
                  (const int32_t*)copies.data_ptr(), i32(copies.size(0)), error, call.stream()) == PA_OK);
    Py_RETURN_TRUE;
  });
}

// (query, key_cache, value_cache, cum, past, table, heads, kv_heads, scale, softcap, slopes, window, first_keys,
//  prefix_lens, max_query_len, lse, error)
PyObject* biased_paged_attention(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const at::Tensor& query = tensor(v[0]);
    const Call call(query);
    const at::ScalarType type = query.scalar_type();
    pa_biased_dims d{};
    d.dtype = dtype_code(type);
    const at::Tensor &k = call.whole(v[1], type, 4), &value = call.whole(v[2], type, 4);
    need(value.sizes() == k.sizes());
    const Batch b(call, v[3], v[4], v[5]);
    const int64_t N = query.size(0);
    d.num_heads = i32(integer(v[6]));
    d.kv_num_heads = i32(integer(v[7]));
    need(k.size(2) == d.kv_num_heads);
    d.query_stride = call.rows(query, type, d.num_heads * k.size(3));
    d.num_tokens = i32(N);
    d.batch_size = b.size;
    d.head_size = i32(k.size(3));
    d.num_blocks = i32(k.size(0));
    d.block_size = i32(k.size(1));
    d.max_blocks_per_sequence = b.columns;
    d.max_query_len = i32(integer(v[14]));
    pa_score_rules rules{};
    rules.softcap = real_or_0(v[9]);
    rules.window = i32(integer(v[11]));
    if (!is_none(v[10])) {
      const at::Tensor& s = call.whole(v[10], at::kFloat, 1);
      need(s.size(0) == d.num_heads);
      rules.slopes = (const float*)s.data_ptr();
    }
    if (!is_none(v[12])) rules.first_keys = call.ints(v[12], N);
    if (!is_none(v[13])) rules.prefix_lens = call.ints(v[13], b.size);
    float* lse = nullptr;
    if (!is_none(v[15])) {
      const at::Tensor& l = call.whole(v[15], at::kFloat, 2);
      need(l.size(0) == N && l.size(1) == d.num_heads);
      lse = (float*)l.data_ptr();
    }
    uint32_t* error = call.error(v[16]);
    const float scale = real_or_0(v[8]);
    const size_t bytes = biased_workspace_size_fn(d.head_size);
    need(bytes > 0);
    const at::Tensor out = call.empty({N, d.num_heads * k.size(3)}, type);
    const c10::DataPtr ws = c10::GetAllocator(c10::DeviceType::CUDA)->allocate(bytes);  // (no tensor: 0.5 us less)
    need(unlocked(biased_paged_attention_fn, query.data_ptr(), k.data_ptr(), value.data_ptr(), b.cum, b.past, b.table,
                  scale, (const pa_score_rules*)&rules, out.data_ptr(), lse, (const pa_biased_dims*)&d, error,
                  ws.get(), bytes, call.stream()) == PA_OK);
    return THPVariable_Wrap(out);
  });
}

// (six addresses): the entry points of the four functions above, then the sizes of their workspaces
PyObject* bind_pool(PyObject*, PyObject* const* v, Py_ssize_t n) {
  void* p[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind_pool takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(v[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is null");
      return nullptr;
    }
  }
  fork_block_tables_fn = reinterpret_cast<decltype(fork_block_tables_fn)>(p[0]);
  compact_block_tables_fn = reinterpret_cast<decltype(compact_block_tables_fn)>(p[1]);
  copy_pages_fn = reinterpret_cast<decltype(copy_pages_fn)>(p[2]);
  biased_paged_attention_fn = reinterpret_cast<decltype(biased_paged_attention_fn)>(p[3]);
  pool_workspace_size_fn = reinterpret_cast<decltype(pool_workspace_size_fn)>(p[4]);
  biased_workspace_size_fn = reinterpret_cast<decltype(biased_workspace_size_fn)>(p[5]);
  Py_RETURN_NONE;
}

// (five addresses): the entry points of libpagedattn.so that the first five functions call, in their order
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
  void* p[5];
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
    return nullptr;
  }
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(v[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is null");
      return nullptr;
    }
  }
  build_block_tables_fn = reinterpret_cast<decltype(build_block_tables_fn)>(p[0]);
  qk_norm_rope_fn = reinterpret_cast<decltype(qk_norm_rope_fn)>(p[1]);
  update_page_bounds_fn = reinterpret_cast<decltype(update_page_bounds_fn)>(p[2]);
  select_pages_fn = reinterpret_cast<decltype(select_pages_fn)>(p[3]);
  sparse_paged_attention_fn = reinterpret_cast<decltype(sparse_paged_attention_fn)>(p[4]);
  Py_RETURN_NONE;
}

#define PA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PA_METHOD(build_block_tables), PA_METHOD(qk_norm_rope),           PA_METHOD(update_page_bounds),
                         PA_METHOD(select_pages),       PA_METHOD(sparse_paged_attention), PA_METHOD(bind),
                         PA_METHOD(fork_block_tables),  PA_METHOD(compact_block_tables),   PA_METHOD(copy_pages),
                         PA_METHOD(biased_paged_attention), PA_METHOD(bind_pool),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step_binding(void) { return PyModule_Create(&module); }
