// Shared declarations of the operators around paged attention: block tables, Q/K norm and
// rotation, page bounds, page selection and attention over selected pages.
#pragma once

#include "common.cuh"
#include "rules.h"

namespace pa {

// ---- host helpers defined with the paged-attention entry points (api.cu) -------------------
pa_status cuda_fail(cudaError_t e, const char* what);  // records the message for pa_last_error
void count_launch();
bool device_sms(int* sms);  // SMs of the current device
// 3-D map over a cache of 16-bit values viewed as (head_size, kv_heads, slots), box 64 x 1 x
// rows, 128-byte swizzle
bool cache_map_16(CUtensorMap* m, const void* base, bool bf16, int hs, int kvh, int64_t slots, int rows);
// 3-D map over query rows viewed as (head_size, heads, rows) with rows `stride` elements apart,
// box 64 x heads x rows, 128-byte swizzle
bool query_block_map(CUtensorMap* m, const void* base, bool bf16, int hs, int nh, int64_t n, int64_t stride, int heads,
                     int rows);

// products of packed fp32 pairs
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// ---- batch lookup without a plan -----------------------------------------------------------
// Work units are numbered so that sequence b's begin at cum[b] / div + mul * b: a CTA finds
// its sequence from its own index by searching that increasing function, and no kernel has to
// lay the units out first. (With mul = 1 there is room for ceil(q_b / div) units per
// sequence, with mul = 2 for one more, as rows that start inside a page touch; unused numbers
// in between belong to no unit.) The largest b with cum[b] / div + mul * b <= u, by a whole
// warp, 32 candidates a step; -1 if there is none.
//
// A sequence's rows and history; ok is false for lengths that do not belong to a batch
// of N rows and tables of max_blocks pages (such a sequence is skipped).
struct Seq {
  int b, c0, q, past;
  bool ok;
};
__device__ __forceinline__ Seq make_seq(int b, int c0, int c1, int past, int N, int max_blocks, int bs) {
  Seq s;
  s.b = b;
  s.c0 = c0;
  s.q = c1 - c0;
  s.past = past;
  s.ok = c0 >= 0 && c1 >= c0 && c1 <= N && past >= 0 && (int64_t)past + s.q <= (int64_t)max_blocks * bs;
  return s;
}

// The sequence of unit u: the largest b with cum[b] / div + mul * b <= u, found by a whole warp,
// 32 candidates a step; the last step's loads bring the lengths with them. ok is false where
// there is none.
__device__ __forceinline__ Seq find_seq(const int32_t* cum, const int32_t* past, int B, int div, int mul, int u,
                                        int N, int max_blocks, int bs, int lane) {
  int lo = 0, n = B;
  for (;;) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const bool in = i < lo + n;
    const int c = in ? cum[i] : 0;
    int c_next = 0, p = 0;
    if (step == 1 && in) c_next = cum[i + 1], p = past[i];
    const unsigned m = __ballot_sync(0xffffffffu, in && c / div + mul * i <= u);
    if (m == 0) return Seq{-1, 0, 0, 0, false};
    const int k = 31 - __clz(m);
    if (step == 1)
      return make_seq(lo + k, __shfl_sync(0xffffffffu, c, k), __shfl_sync(0xffffffffu, c_next, k),
                      __shfl_sync(0xffffffffu, p, k), N, max_blocks, bs);
    n = min(step, lo + n - (lo + k * step));
    lo += k * step;
  }
}

// the checks of the whole batch, by one CTA: sets PA_DEVERR_BAD_BATCH
__device__ __forceinline__ void check_batch(const int32_t* cum, const int32_t* past, int B, int N, int max_blocks,
                                            int bs, uint32_t* err) {
  if (!err) return;
  bool bad = threadIdx.x == 0 && cum[0] != 0;
  for (int b = threadIdx.x; b < B; b += blockDim.x) bad |= !make_seq(b, cum[b], cum[b + 1], past[b], N, max_blocks, bs).ok;
  if (bad) atomicOr(err, PA_DEVERR_BAD_BATCH);
}

// ---- clusters ------------------------------------------------------------------------------
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address in CTA `rank` of the cluster that `p` has in this one
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// ---- argument records ----------------------------------------------------------------------
struct TableArgs {
  const int32_t *past, *query_lens, *held;
  int32_t *table, *ring;
  const int32_t* state;
  int32_t *cum, *slots, *positions, *held_out, *state_out;
  uint32_t* error;
  int32_t B, N, max_blocks, bs, cap;
};

struct RotateArgs {
  const uint16_t *query, *key, *q_weight, *k_weight;
  uint16_t *query_out, *key_out;
  const int32_t* positions;
  int64_t q_stride, k_stride, qo_stride, ko_stride;  // elements between rows
  int32_t N, nh, kvh, rotary_dim, interleaved;
  int32_t split;  // warps that share a row's heads
  float eps;
  float inv_freq[128];
};

struct PageArgs {
  const uint16_t *query, *key_cache, *value_cache;
  int8_t* bounds;      // (num_blocks, kvh, 2, hs): minimum, then maximum codes
  const float* scale;  // (kvh, hs)
  const int32_t *cum, *past, *table;
  int32_t* selected;   // (N, kvh, top_k)
  void* output;
  float* lse;
  uint32_t* error;
  int64_t q_stride;
  int32_t N, B, nh, kvh, G, hs, num_blocks, bs, max_blocks;
  int32_t top_k, R, sink, local;
  float scale_log2;
};

// forks and compactions of block tables (pool.cu)
struct PoolArgs {
  const int32_t *parents, *past, *held, *table, *state;
  const uint8_t* pinned;  // per page, or null
  int32_t *ring, *past_out, *held_out, *table_out, *state_out, *pages_end;
  int2* copies;
  uint32_t* error;
  // the workspace: the error word and the marks, cleared first (clear_words 16-byte words), then
  // the words of bits and the chunks' totals
  uint4* clear;
  int64_t clear_words;
  uint32_t* ws_error;
  uint8_t *marks, *old_marks;  // per page
  int32_t* keeper;             // per page (fork)
  uint4* words;
  int2* chunks;
  int32_t *first_child, *last;  // per old row (fork, else null): its lowest new row, its partly filled page
  uint32_t* row_bits;          // 32 new rows each (fork)
  int32_t* holes;              // per page (compact)
  int32_t B, Bn, max_blocks, bs, num_blocks, num_chunks, cap, max_moves;
  int32_t row_blocks;  // blocks of the last kernel that write rows, the others pages
};
// bytes of the workspace of num_blocks pages; fills in its pointers where `a` is given
inline size_t pool_workspace(int32_t num_blocks, bool fork, PoolArgs* a, uint8_t* base) {
  const size_t chunks = (size_t)ceil_div(num_blocks, 1024), pages = chunks * 1024, rows = PA_MAX_TABLE_REQUESTS;
  size_t off = 16;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 16);
    return at;
  };
  const size_t marks = take(pages), old_marks = take(fork ? pages : 0), keeper = take(fork ? 4 * pages : 0), cleared = off;
  const size_t words = take(pages / 2), totals = take(8 * chunks), child = take(fork ? 4 * rows : 0), last = take(fork ? 4 * rows : 0),
               row_bits = take(fork ? rows / 8 : 0), holes = take(fork ? 0 : 4 * pages);
  if (a) {
    a->clear = reinterpret_cast<uint4*>(base);
    a->clear_words = (int64_t)(cleared / 16);
    a->ws_error = reinterpret_cast<uint32_t*>(base);
    a->marks = base + marks;
    a->old_marks = base + old_marks;
    a->keeper = reinterpret_cast<int32_t*>(base + keeper);
    a->words = reinterpret_cast<uint4*>(base + words);
    a->chunks = reinterpret_cast<int2*>(base + totals);
    a->first_child = fork ? reinterpret_cast<int32_t*>(base + child) : nullptr;
    a->last = fork ? reinterpret_cast<int32_t*>(base + last) : nullptr;
    a->row_bits = reinterpret_cast<uint32_t*>(base + row_bits);
    a->holes = reinterpret_cast<int32_t*>(base + holes);
    a->num_chunks = (int32_t)chunks;
  }
  return off;
}

struct CopyArgs {
  uint8_t* data[PA_MAX_COPY_TENSORS];
  int64_t bytes[PA_MAX_COPY_TENSORS];  // of a page
  const int2* copies;
  uint32_t* error;
  int32_t n, num_tensors, num_blocks, pieces;
};

// attention with capped or biased scores and ranges of keys (biased.cu)
struct BiasedArgs {
  const uint16_t *query, *key_cache, *value_cache;
  const int32_t *cum, *past, *table, *first, *prefix;  // first, prefix: or null
  const float* slopes;                                 // or null
  void* output;
  float* lse;
  uint32_t* error;
  int64_t q_stride;
  int32_t N, B, nh, kvh, G, hs, num_blocks, bs, max_blocks;
  int32_t window, max_rows;  // 0: none
  int32_t after_tiles;       // the rows kernel runs beside the tile kernel: it starts without waiting for it
  // s log2(e) of a score q.k is q.k * scale_log2, or with a cap cap_log2 * tanh(q.k * scale_cap)
  float scale_log2, scale_cap, cap_log2;
  // split pieces of the rows kernel: two slots per CTA, and what they hold
  float *part_o, *part_ml;
  int4* records;
};

cudaError_t launch_fork(const PoolArgs& a, int sms, cudaStream_t s, int* kernels);
cudaError_t launch_compact(const PoolArgs& a, int sms, cudaStream_t s, int* kernels);
cudaError_t launch_copy_pages(CopyArgs& a, int sms, cudaStream_t s);
int biased_ctas(int hs, int sms);  // CTAs of the rows kernel
cudaError_t launch_biased(const BiasedArgs& a, bool bf16, int sms, cudaStream_t s, int* kernels);
cudaError_t launch_tables(const TableArgs& a, int sms, cudaStream_t s);
cudaError_t launch_rotate(const RotateArgs& a, bool bf16, int hs, int sms, cudaStream_t s);
cudaError_t launch_bounds(const PageArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_select(const PageArgs& a, bool bf16, int sms, cudaStream_t s);
cudaError_t launch_sparse(const PageArgs& a, bool bf16, int sms, cudaStream_t s);

// A launch that may start before the kernel before it has finished (its blocks wait for that
// kernel's results) and whose CTAs along z form one cluster each. `most` is the largest smem of
// any call of this kernel: the limit is the function's, for all host threads, so that every
// call sets it to the same.
template <typename... KArgs, typename... Actual>
inline cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, size_t most,
                                   cudaStream_t s, Actual&&... args) {
  // (up to 48 KB with the kernel's static arrays need no attribute)
  if (smem > 12 * 1024)
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most)) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = grid.z;
  cfg.attrs = attr;
  cfg.numAttrs = grid.z > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Actual&&>(args)...);
}

// numbers of query blocks (units of div rows, with mul numbers to spare per sequence)
inline int64_t query_blocks(const PageArgs& a) { return a.R == 1 ? a.N : (int64_t)a.N / a.R + a.B; }

}  // namespace pa
