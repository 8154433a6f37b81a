// C ABI of the operators around paged attention (include/pagedattn.h): argument checks and
// launches. No allocation and no synchronisation; a workspace only where the caller gives one.
#include <cmath>
#include <initializer_list>

#include "ops.cuh"

namespace {

bool aligned(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool all_aligned(uintptr_t a, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, a)) return false;
  return true;
}

// (the page operators go over a row's columns in parts, and count past the last one in 32 bits)
constexpr int32_t kMostColumns = INT32_MAX - 1024;

// memory that a call reads or writes
struct Range {
  uintptr_t from, to;
  Range(const void* p, int64_t bytes)
      : from(reinterpret_cast<uintptr_t>(p)), to(p && bytes > 0 ? from + (uintptr_t)bytes : from) {}
  bool meets(const Range& r) const { return from < r.to && r.from < to; }
};

// whether each of `written` is apart from the others and from all of `read`
bool all_apart(std::initializer_list<Range> written, std::initializer_list<Range> read) {
  for (const Range* w = written.begin(); w != written.end(); ++w) {
    for (const Range* o = written.begin(); o != w; ++o)
      if (w->meets(*o)) return false;
    for (const Range& r : read)
      if (w->meets(r)) return false;
  }
  return true;
}

pa_status launched(cudaError_t e, const char* what, int kernels = 1) {
  if (e) return pa::cuda_fail(e, what);
  while (kernels-- > 0) pa::count_launch();
  return PA_OK;
}

pa_status check_batch_dims(const pa_sparse_dims* d) {
  if (!d || d->reserved != 0) return PA_ERR_INVALID_ARGUMENT;
  if (d->num_tokens < 0 || d->batch_size < 0 || d->num_blocks < 0 || d->max_blocks_per_sequence < 0 ||
      (d->num_tokens > 0 && d->batch_size == 0))
    return PA_ERR_INVALID_ARGUMENT;
  if (d->num_heads <= 0 || d->kv_num_heads <= 0 || d->num_heads % d->kv_num_heads != 0 || d->block_size <= 0 ||
      d->head_size <= 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (d->dtype != PA_FLOAT16 && d->dtype != PA_BFLOAT16) return PA_ERR_UNSUPPORTED;
  if (d->head_size != 64 && d->head_size != 128 && d->head_size != 256) return PA_ERR_UNSUPPORTED;
  if (d->block_size % 16 != 0) return PA_ERR_UNSUPPORTED;
  // (positions are counted in 32 bits, a tile past the last one among them)
  if ((int64_t)d->num_blocks * d->block_size > INT32_MAX ||
      (int64_t)d->max_blocks_per_sequence * d->block_size > INT32_MAX - 4096)
    return PA_ERR_UNSUPPORTED;
  if ((int64_t)d->num_heads * d->head_size > 65536 || d->kv_num_heads > 65535) return PA_ERR_UNSUPPORTED;
  // (query blocks and touched pages are numbered with room for every sequence)
  if ((int64_t)d->num_tokens + 2 * (int64_t)d->batch_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
  if (d->num_tokens > 0 && (d->num_blocks == 0 || d->max_blocks_per_sequence == 0)) return PA_ERR_INVALID_ARGUMENT;
  return PA_OK;
}

pa_status check_selection_dims(const pa_sparse_dims* d) {
  if (d->top_k <= 0 || d->query_block <= 0) return PA_ERR_INVALID_ARGUMENT;
  if (d->query_stride < (int64_t)d->num_heads * d->head_size || d->query_stride % 8 != 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (d->top_k > PA_MAX_SELECTED_PAGES || (int64_t)d->query_block * (d->num_heads / d->kv_num_heads) > 1024)
    return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

void fill(pa::PageArgs& a, const pa_sparse_dims* d, const int32_t* cum, const int32_t* past, const int32_t* table,
          uint32_t* error) {
  a.cum = cum;
  a.past = past;
  a.table = table;
  a.error = error;
  a.N = d->num_tokens;
  a.B = d->batch_size;
  a.nh = d->num_heads;
  a.kvh = d->kv_num_heads;
  a.G = d->num_heads / d->kv_num_heads;
  a.hs = d->head_size;
  a.num_blocks = d->num_blocks;
  a.bs = d->block_size;
  a.max_blocks = d->max_blocks_per_sequence;
  a.top_k = d->top_k;
  a.R = d->query_block;
  a.sink = d->sink_pages;
  a.local = d->local_pages;
  a.q_stride = d->query_stride;
}

}  // namespace

extern "C" {

pa_status pa_build_block_tables(const int32_t* past_seqlens, const int32_t* query_lens, const int32_t* blocks_held,
                                int32_t* block_table, int32_t* free_blocks, const int32_t* free_state,
                                int32_t batch_size, int32_t num_tokens, int32_t max_blocks_per_sequence,
                                int32_t block_size, int32_t free_capacity, int32_t* cumulative_sequence_length,
                                int32_t* slot_mapping, int32_t* positions, int32_t* blocks_held_out,
                                int32_t* free_state_out, uint32_t* error, void* stream) {
  if (batch_size < 0 || num_tokens < 0 || max_blocks_per_sequence <= 0 || block_size <= 0 || free_capacity <= 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (batch_size > PA_MAX_TABLE_REQUESTS || num_tokens == INT32_MAX ||
      (int64_t)max_blocks_per_sequence * block_size > INT32_MAX ||
      (int64_t)batch_size * max_blocks_per_sequence > INT32_MAX || free_capacity > (1 << 30))
    return PA_ERR_UNSUPPORTED;
  if (!all_aligned(4, {free_blocks, free_state, cumulative_sequence_length, free_state_out, error}))
    return PA_ERR_INVALID_ARGUMENT;
  if (batch_size > 0 && !all_aligned(4, {past_seqlens, query_lens, blocks_held, block_table, blocks_held_out}))
    return PA_ERR_INVALID_ARGUMENT;
  if (num_tokens > 0 && !all_aligned(4, {slot_mapping, positions})) return PA_ERR_INVALID_ARGUMENT;
  // the kernel's CTAs read the old counts while others write the new ones
  if ((batch_size > 0 && blocks_held_out == blocks_held) || free_state_out == free_state) return PA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  if (!pa::device_sms(&sms)) return pa::cuda_fail(cudaGetLastError(), "device query");
  pa::TableArgs a{};
  a.past = past_seqlens;
  a.query_lens = query_lens;
  a.held = blocks_held;
  a.table = block_table;
  a.ring = free_blocks;
  a.state = free_state;
  a.cum = cumulative_sequence_length;
  a.slots = slot_mapping;
  a.positions = positions;
  a.held_out = blocks_held_out;
  a.state_out = free_state_out;
  a.error = error;
  a.B = batch_size;
  a.N = num_tokens;
  a.max_blocks = max_blocks_per_sequence;
  a.bs = block_size;
  a.cap = free_capacity;
  return launched(pa::launch_tables(a, sms, static_cast<cudaStream_t>(stream)), "tables_kernel launch");
}

pa_status pa_qk_norm_rope(const void* query, const void* key, const int32_t* positions, const pa_qk_prep* prep,
                          int32_t interleaved, int32_t num_tokens, int32_t num_heads, int32_t kv_num_heads,
                          int32_t head_size, int32_t dtype, int64_t query_stride, int64_t key_stride,
                          void* query_out, void* key_out, int64_t query_out_stride, int64_t key_out_stride,
                          void* stream) {
  if (!prep || prep->reserved != 0 || num_tokens < 0 || num_heads <= 0 || kv_num_heads <= 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (dtype != PA_FLOAT16 && dtype != PA_BFLOAT16) return PA_ERR_UNSUPPORTED;
  if (head_size != 64 && head_size != 128 && head_size != 256) return PA_ERR_UNSUPPORTED;
  const int32_t d = prep->rotary_dim;
  if (d < 0 || d > head_size || d % 16 != 0) return PA_ERR_UNSUPPORTED;
  if (d > 0 && !(prep->rope_theta > 0.f)) return PA_ERR_INVALID_ARGUMENT;
  if ((prep->q_norm_weight || prep->k_norm_weight) && !(prep->norm_eps > 0.f)) return PA_ERR_INVALID_ARGUMENT;
  const int64_t qw = (int64_t)num_heads * head_size, kw = (int64_t)kv_num_heads * head_size;
  if (qw > 65536 || kw > 65536) return PA_ERR_UNSUPPORTED;
  if (query_stride < qw || query_out_stride < qw || key_stride < kw || key_out_stride < kw || query_stride % 8 ||
      query_out_stride % 8 || key_stride % 8 || key_out_stride % 8)
    return PA_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return PA_OK;
  if (!all_aligned(16, {query, key, query_out, key_out}) || !aligned(positions, 4) ||
      (prep->q_norm_weight && !aligned(prep->q_norm_weight, 16)) ||
      (prep->k_norm_weight && !aligned(prep->k_norm_weight, 16)))
    return PA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  if (!pa::device_sms(&sms)) return pa::cuda_fail(cudaGetLastError(), "device query");
  pa::RotateArgs a{};
  a.query = static_cast<const uint16_t*>(query);
  a.key = static_cast<const uint16_t*>(key);
  a.query_out = static_cast<uint16_t*>(query_out);
  a.key_out = static_cast<uint16_t*>(key_out);
  a.q_weight = static_cast<const uint16_t*>(prep->q_norm_weight);
  a.k_weight = static_cast<const uint16_t*>(prep->k_norm_weight);
  a.positions = positions;
  a.q_stride = query_stride;
  a.k_stride = key_stride;
  a.qo_stride = query_out_stride;
  a.ko_stride = key_out_stride;
  a.N = num_tokens;
  a.nh = num_heads;
  a.kvh = kv_num_heads;
  a.rotary_dim = d;
  a.interleaved = interleaved != 0;
  a.eps = prep->norm_eps;
  // the fp32 rotary table fl32(theta^(-2u/d)), formed in double and rounded once; a thread's
  // calls with one base and dimension (a model's) form it once
  struct Table {
    float theta = 0.f, freq[128];
    int32_t d = 0;
  };
  static thread_local Table table;
  if (d > 0 && (table.d != d || table.theta != prep->rope_theta)) {
    for (int u = 0; u < d / 2; ++u) table.freq[u] = (float)std::pow((double)prep->rope_theta, -2.0 * u / d);
    table.d = d;
    table.theta = prep->rope_theta;
  }
  for (int u = 0; u < d / 2; ++u) a.inv_freq[u] = table.freq[u];
  return launched(pa::launch_rotate(a, dtype == PA_BFLOAT16, head_size, sms, static_cast<cudaStream_t>(stream)),
                  "rotate_kernel launch");
}

pa_status pa_update_page_bounds(const void* key_cache, int8_t* page_bounds, const float* bound_scale,
                                const int32_t* cumulative_sequence_length, const int32_t* past_seqlens,
                                const int32_t* block_table, const pa_sparse_dims* dims, uint32_t* error,
                                void* stream) {
  if (pa_status st = check_batch_dims(dims)) return st;
  if (dims->num_tokens == 0) return PA_OK;
  if (!all_aligned(16, {key_cache, page_bounds}) ||
      !all_aligned(4, {bound_scale, cumulative_sequence_length, past_seqlens, block_table}) ||
      (error && !aligned(error, 4)))
    return PA_ERR_INVALID_ARGUMENT;
  pa::PageArgs a{};
  fill(a, dims, cumulative_sequence_length, past_seqlens, block_table, error);
  a.key_cache = static_cast<const uint16_t*>(key_cache);
  a.bounds = page_bounds;
  a.scale = bound_scale;
  return launched(pa::launch_bounds(a, dims->dtype == PA_BFLOAT16, static_cast<cudaStream_t>(stream)),
                  "bounds_kernel launch");
}

pa_status pa_select_pages(const void* query, const int8_t* page_bounds, const float* bound_scale,
                          const int32_t* cumulative_sequence_length, const int32_t* past_seqlens,
                          const int32_t* block_table, const pa_sparse_dims* dims, int32_t* selected, uint32_t* error,
                          void* stream) {
  if (pa_status st = check_batch_dims(dims)) return st;
  if (pa_status st = check_selection_dims(dims)) return st;
  if (dims->sink_pages < 0 || dims->local_pages < 1 ||
      (int64_t)dims->sink_pages + dims->local_pages + (dims->query_block + dims->block_size - 2) / dims->block_size >
          dims->top_k)
    return PA_ERR_INVALID_ARGUMENT;
  if (dims->max_blocks_per_sequence > PA_MAX_SCORED_PAGES) return PA_ERR_UNSUPPORTED;
  if (dims->num_tokens == 0) return PA_OK;
  if (!all_aligned(16, {query, page_bounds}) ||
      !all_aligned(4, {bound_scale, cumulative_sequence_length, past_seqlens, block_table, selected}) ||
      (error && !aligned(error, 4)))
    return PA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  if (!pa::device_sms(&sms)) return pa::cuda_fail(cudaGetLastError(), "device query");
  pa::PageArgs a{};
  fill(a, dims, cumulative_sequence_length, past_seqlens, block_table, error);
  a.query = static_cast<const uint16_t*>(query);
  a.bounds = const_cast<int8_t*>(page_bounds);
  a.scale = bound_scale;
  a.selected = selected;
  return launched(pa::launch_select(a, dims->dtype == PA_BFLOAT16, sms, static_cast<cudaStream_t>(stream)),
                  "select_kernel launch");
}

pa_status pa_sparse_paged_attention(const void* query, const void* key_cache, const void* value_cache,
                                    const int32_t* cumulative_sequence_length, const int32_t* past_seqlens,
                                    const int32_t* block_table, const int32_t* selected, float scale, void* output,
                                    float* lse, const pa_sparse_dims* dims, uint32_t* error, void* stream) {
  if (pa_status st = check_batch_dims(dims)) return st;
  if (pa_status st = check_selection_dims(dims)) return st;
  // (a query block's tiles are numbered in 32 bits, with room for every sequence)
  const int32_t R = dims->query_block, G = dims->num_heads / dims->kv_num_heads;
  if (!pa::takes_rows_kernel(R, G) &&
      ((int64_t)dims->num_tokens / R + dims->batch_size) * pa::ceil_div(R, pa::rows_of_tile(R, G)) > INT32_MAX)
    return PA_ERR_UNSUPPORTED;
  if (dims->num_tokens == 0) return PA_OK;
  if (!all_aligned(16, {query, key_cache, value_cache, output}) ||
      !all_aligned(4, {cumulative_sequence_length, past_seqlens, block_table, selected}) ||
      (lse && !aligned(lse, 4)) || (error && !aligned(error, 4)))
    return PA_ERR_INVALID_ARGUMENT;
  int sms = 0;
  if (!pa::device_sms(&sms)) return pa::cuda_fail(cudaGetLastError(), "device query");
  pa::PageArgs a{};
  fill(a, dims, cumulative_sequence_length, past_seqlens, block_table, error);
  a.query = static_cast<const uint16_t*>(query);
  a.key_cache = static_cast<const uint16_t*>(key_cache);
  a.value_cache = static_cast<const uint16_t*>(value_cache);
  a.selected = const_cast<int32_t*>(selected);
  a.output = output;
  a.lse = lse;
  const float sc = scale == 0.0f ? 1.0f / std::sqrt((float)dims->head_size) : scale;
  a.scale_log2 = sc * 1.4426950408889634f;
  return launched(pa::launch_sparse(a, dims->dtype == PA_BFLOAT16, sms, static_cast<cudaStream_t>(stream)),
                  "sparse attention launch");
}

size_t pa_pool_workspace_size(int32_t num_blocks) {
  if (num_blocks <= 0 || num_blocks > PA_MAX_POOL_PAGES) return 0;
  return pa::pool_workspace(num_blocks, true, nullptr, nullptr);
}

pa_status pa_fork_block_tables(const int32_t* parents, const int32_t* past_seqlens, const int32_t* blocks_held,
                               const int32_t* block_table, int32_t* free_blocks, const int32_t* free_state,
                               const uint8_t* pinned, int32_t batch_size, int32_t new_batch_size,
                               int32_t max_blocks_per_sequence, int32_t block_size, int32_t num_blocks,
                               int32_t free_capacity, int32_t* past_seqlens_out, int32_t* blocks_held_out,
                               int32_t* block_table_out, int32_t* copies, int32_t* free_state_out, uint32_t* error,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (batch_size < 0 || new_batch_size < 0 || max_blocks_per_sequence <= 0 || block_size <= 0 || num_blocks <= 0 ||
      free_capacity <= 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (batch_size > PA_MAX_TABLE_REQUESTS || new_batch_size > PA_MAX_TABLE_REQUESTS || num_blocks > PA_MAX_POOL_PAGES ||
      max_blocks_per_sequence > kMostColumns ||
      (int64_t)max_blocks_per_sequence * block_size > INT32_MAX ||
      (int64_t)batch_size * max_blocks_per_sequence > INT32_MAX ||
      (int64_t)new_batch_size * max_blocks_per_sequence > INT32_MAX || free_capacity > (1 << 30))
    return PA_ERR_UNSUPPORTED;
  if (!all_aligned(4, {free_blocks, free_state, free_state_out, error}) || !aligned(workspace, 16))
    return PA_ERR_INVALID_ARGUMENT;
  if (batch_size > 0 && !all_aligned(4, {past_seqlens, blocks_held, block_table})) return PA_ERR_INVALID_ARGUMENT;
  if (new_batch_size > 0 &&
      (!all_aligned(4, {parents, past_seqlens_out, blocks_held_out, block_table_out}) || !aligned(copies, 8)))
    return PA_ERR_INVALID_ARGUMENT;
  // rows are read while others are written
  const int64_t B = batch_size, n = new_batch_size, width = max_blocks_per_sequence;
  if (!all_apart({{past_seqlens_out, 4 * n}, {blocks_held_out, 4 * n}, {block_table_out, 4 * n * width}, {copies, 8 * n},
                  {free_state_out, 8}, {error, 4}, {free_blocks, 4 * (int64_t)free_capacity},
                  {workspace, (int64_t)pa::pool_workspace(num_blocks, true, nullptr, nullptr)}},
                 {{parents, 4 * n}, {past_seqlens, 4 * B}, {blocks_held, 4 * B}, {block_table, 4 * B * width},
                  {free_state, 8}, {pinned, num_blocks}}))
    return PA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < pa::pool_workspace(num_blocks, true, nullptr, nullptr)) return PA_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if (!pa::device_sms(&sms)) return pa::cuda_fail(cudaGetLastError(), "device query");
  pa::PoolArgs a{};
  pa::pool_workspace(num_blocks, true, &a, static_cast<uint8_t*>(workspace));
  a.parents = parents;
  a.past = past_seqlens;
  a.held = blocks_held;
  a.table = block_table;
  a.ring = free_blocks;
  a.state = free_state;
  a.pinned = pinned;
  a.past_out = past_seqlens_out;
  a.held_out = blocks_held_out;
  a.table_out = block_table_out;
  a.copies = reinterpret_cast<int2*>(copies);
  a.state_out = free_state_out;
  a.error = error;
  a.B = batch_size;
  a.Bn = new_batch_size;
  a.max_blocks = max_blocks_per_sequence;
  a.bs = block_size;
  a.num_blocks = num_blocks;
  a.cap = free_capacity;
  int kernels = 0;
  const cudaError_t e = pa::launch_fork(a, sms, static_cast<cudaStream_t>(stream), &kernels);
  return launched(e, "fork launch", kernels);
}

pa_status pa_compact_block_tables(const int32_t* blocks_held, const int32_t* block_table, int32_t* free_blocks,
                                  const uint8_t* pinned, int32_t batch_size, int32_t max_blocks_per_sequence,
                                  int32_t num_blocks, int32_t free_capacity, int32_t max_moves,
                                  int32_t* block_table_out, int32_t* copies, int32_t* free_state_out,
                                  int32_t* pages_end, uint32_t* error, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  if (batch_size < 0 || max_blocks_per_sequence <= 0 || num_blocks <= 0 || free_capacity <= 0 || max_moves < 0)
    return PA_ERR_INVALID_ARGUMENT;
  if (batch_size > PA_MAX_TABLE_REQUESTS || num_blocks > PA_MAX_POOL_PAGES || max_moves > PA_MAX_POOL_PAGES ||
      max_blocks_per_sequence > kMostColumns ||
      (int64_t)batch_size * max_blocks_per_sequence > INT32_MAX || free_capacity > (1 << 30))
    return PA_ERR_UNSUPPORTED;
  if (!all_aligned(4, {free_blocks, free_state_out, pages_end, error}) || !aligned(workspace, 16))
    return PA_ERR_INVALID_ARGUMENT;
  if (batch_size > 0 && !all_aligned(4, {blocks_held, block_table, block_table_out})) return PA_ERR_INVALID_ARGUMENT;
  if (max_moves > 0 && !aligned(copies, 8)) return PA_ERR_INVALID_ARGUMENT;
  // (a table that is renamed in place is one: each entry is read and written by one thread)
  const int64_t B = batch_size, entries = B * max_blocks_per_sequence;
  if (!all_apart({{block_table_out, 4 * entries}, {copies, 8 * (int64_t)max_moves}, {free_state_out, 8}, {pages_end, 4},
                  {error, 4}, {free_blocks, 4 * (int64_t)free_capacity},
                  {workspace, (int64_t)pa::pool_workspace(num_blocks, false, nullptr, nullptr)}},
                 {{blocks_held, 4 * B}, {block_table, block_table_out == block_table ? 0 : 4 * entries}, {pinned, num_blocks}}))
    return PA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < pa::pool_workspace(num_blocks, false, nullptr, nullptr)) return PA_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if (!pa::device_sms(&sms)) return pa::cuda_fail(cudaGetLastError(), "device query");
  pa::PoolArgs a{};
  pa::pool_workspace(num_blocks, false, &a, static_cast<uint8_t*>(workspace));
  a.held = blocks_held;
  a.table = block_table;
  a.ring = free_blocks;
  a.pinned = pinned;
  a.table_out = block_table_out;
  a.copies = reinterpret_cast<int2*>(copies);
  a.state_out = free_state_out;
  a.pages_end = pages_end;
  a.error = error;
  a.B = batch_size;
  a.max_blocks = max_blocks_per_sequence;
  a.num_blocks = num_blocks;
  a.cap = free_capacity;
  a.max_moves = max_moves;
  int kernels = 0;
  const cudaError_t e = pa::launch_compact(a, sms, static_cast<cudaStream_t>(stream), &kernels);
  return launched(e, "compaction launch", kernels);
}

pa_status pa_copy_pages(const pa_page_tensor* tensors, int32_t num_tensors, int32_t num_blocks, const int32_t* copies,
                        int32_t num_copies, uint32_t* error, void* stream) {
  if (num_tensors < 0 || num_blocks < 0 || num_copies < 0) return PA_ERR_INVALID_ARGUMENT;
  if (num_tensors > PA_MAX_COPY_TENSORS || num_copies > PA_MAX_COPIES) return PA_ERR_UNSUPPORTED;
  if (num_tensors == 0 || num_copies == 0) return PA_OK;
  if (!tensors || !aligned(copies, 8) || (error && !aligned(error, 4))) return PA_ERR_INVALID_ARGUMENT;
  pa::CopyArgs a{};
  for (int32_t t = 0; t < num_tensors; ++t) {
    const int64_t bytes = tensors[t].page_bytes;
    if (bytes <= 0 || !aligned(tensors[t].data, 16)) return PA_ERR_INVALID_ARGUMENT;
    if (bytes % 16 != 0 || bytes > INT32_MAX) return PA_ERR_UNSUPPORTED;
    a.data[t] = static_cast<uint8_t*>(tensors[t].data);
    a.bytes[t] = bytes;
  }
  int sms = 0;
  if (!pa::device_sms(&sms)) return pa::cuda_fail(cudaGetLastError(), "device query");
  a.copies = reinterpret_cast<const int2*>(copies);
  a.error = error;
  a.n = num_copies;
  a.num_tensors = num_tensors;
  a.num_blocks = num_blocks;
  return launched(pa::launch_copy_pages(a, sms, static_cast<cudaStream_t>(stream)), "copy_pages_kernel launch");
}

// the rows kernel's two slots per CTA: partial results, their (m, l), and the CTAs' records
size_t pa_biased_workspace_size(int32_t head_size) {
  if (head_size != 64 && head_size != 128 && head_size != 256) return 0;
  const size_t slots = 2 * (size_t)PA_BIASED_CTAS;
  return slots * 16 * (size_t)head_size * 4 + slots * 16 * 8 + slots * 16;
}

pa_status pa_biased_paged_attention(const void* query, const void* key_cache, const void* value_cache,
                                    const int32_t* cumulative_sequence_length, const int32_t* past_seqlens,
                                    const int32_t* block_table, float scale, const pa_score_rules* rules, void* output,
                                    float* lse, const pa_biased_dims* dims, uint32_t* error, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  if (!dims || dims->reserved != 0 || !rules || rules->reserved != 0) return PA_ERR_INVALID_ARGUMENT;
  const pa_sparse_dims d = {dims->num_tokens, dims->batch_size, dims->num_heads, dims->kv_num_heads, dims->head_size,
                            dims->num_blocks, dims->block_size, dims->max_blocks_per_sequence, dims->dtype,
                            1, 1, 0, 1, 0, dims->query_stride};
  if (pa_status st = check_batch_dims(&d)) return st;
  if (pa_status st = check_selection_dims(&d)) return st;
  const float sc = scale == 0.0f ? 1.0f / std::sqrt((float)dims->head_size) : scale;
  if (!std::isfinite(sc * 1.4426950408889634f) || rules->window < 0 || dims->max_query_len < 0) return PA_ERR_INVALID_ARGUMENT;
  // (a cap so small or large that a score in units of it, or it in powers of two, is none is no cap)
  if (rules->softcap != 0.f && !(rules->softcap >= 1e-30f && rules->softcap <= 1e30f && std::isfinite(sc / rules->softcap)))
    return PA_ERR_INVALID_ARGUMENT;
  // (rows, heads and blocks of rows are numbered in 32 bits)
  if (((int64_t)dims->num_tokens + dims->batch_size) * dims->num_heads > INT32_MAX) return PA_ERR_UNSUPPORTED;
  if (dims->num_tokens == 0) return PA_OK;
  if (!all_aligned(16, {query, key_cache, value_cache, output, workspace}) ||
      !all_aligned(4, {cumulative_sequence_length, past_seqlens, block_table}) || (lse && !aligned(lse, 4)) ||
      (error && !aligned(error, 4)) || (rules->slopes && !aligned(rules->slopes, 4)) ||
      (rules->first_keys && !aligned(rules->first_keys, 4)) || (rules->prefix_lens && !aligned(rules->prefix_lens, 4)))
    return PA_ERR_INVALID_ARGUMENT;
  // (rows are read again after others have been written)
  const int64_t row = (int64_t)dims->num_heads * dims->head_size;
  const uintptr_t q0 = (uintptr_t)query, q1 = q0 + 2 * ((dims->num_tokens - 1) * dims->query_stride + row);
  const uintptr_t o0 = (uintptr_t)output, o1 = o0 + 2 * dims->num_tokens * row;
  if (o0 < q1 && q0 < o1) return PA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < pa_biased_workspace_size(dims->head_size)) return PA_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if (!pa::device_sms(&sms)) return pa::cuda_fail(cudaGetLastError(), "device query");
  pa::BiasedArgs a{};
  a.query = static_cast<const uint16_t*>(query);
  a.key_cache = static_cast<const uint16_t*>(key_cache);
  a.value_cache = static_cast<const uint16_t*>(value_cache);
  a.cum = cumulative_sequence_length;
  a.past = past_seqlens;
  a.table = block_table;
  a.first = rules->first_keys;
  a.prefix = rules->prefix_lens;
  a.slopes = rules->slopes;
  a.output = output;
  a.lse = lse;
  a.error = error;
  a.q_stride = dims->query_stride;
  a.N = dims->num_tokens;
  a.B = dims->batch_size;
  a.nh = dims->num_heads;
  a.kvh = dims->kv_num_heads;
  a.G = dims->num_heads / dims->kv_num_heads;
  a.hs = dims->head_size;
  a.num_blocks = dims->num_blocks;
  a.bs = dims->block_size;
  a.max_blocks = dims->max_blocks_per_sequence;
  a.window = rules->window;
  a.max_rows = dims->max_query_len;
  a.scale_log2 = sc * 1.4426950408889634f;
  if (rules->softcap > 0.f) {
    a.scale_cap = sc / rules->softcap;
    a.cap_log2 = rules->softcap * 1.4426950408889634f;
  }
  const size_t slots = 2 * (size_t)PA_BIASED_CTAS;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = a.part_o + slots * 16 * (size_t)dims->head_size;
  a.records = reinterpret_cast<int4*>(a.part_ml + slots * 16 * 2);
  int kernels = 0;
  const cudaError_t e = pa::launch_biased(a, dims->dtype == PA_BFLOAT16, sms, static_cast<cudaStream_t>(stream), &kernels);
  return launched(e, "biased attention launch", kernels);
}

}  // extern "C"
