// C ABI of the operators around paged attention (include/pagedattn.h): argument checks and
// launches. No allocation, no synchronisation, no workspace.
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

pa_status launched(cudaError_t e, const char* what) {
  if (e) return pa::cuda_fail(e, what);
  pa::count_launch();
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

}  // extern "C"
