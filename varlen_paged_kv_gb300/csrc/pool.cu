// The pages of a pool as requests fork, end and are compacted, and the copies that this takes.
//
// fork_block_tables makes the rows of a new batch from rows of the old one; compact_block_tables
// moves the highest pages in use into the lowest free ones. Both ask of every page of the pool
// what the tables hold it for. Small batches over small pools do all of it in one CTA, with
// the pages' marks as bits in shared memory (one launch: a fork of 64 rows 7.6 us instead of 9.4 with
// the kernels below, a compaction 8.0 instead of 10.0). Others take a few short kernels over a workspace:
//   clear   the marks; the fork's first new row of each old one
//   mark    every held table entry stores a byte at its page (the same byte from whoever
//           stores it, so without atomics); a row that would write into its last page next
//           leaves its number there by an atomic maximum (of Bn - row: the lowest row stays)
//   words   the marks as bits, 32 pages a word, with counts before each word inside its chunk of
//           1024 pages and the chunks' totals; the fork's rows that copy as bits
//   lists   (compaction) the holes in order
//   finish  every CTA scans the chunks' totals (1024 at most) itself; a page's rank among the
//           pages of its kind is then its chunk's sum, its word's and a population count. Tables,
//           ring and copies are written from that, each entry by itself.
// Every order (of pages given out, given back and moved) is one of page or row numbers, so results
// do not depend on the order in which CTAs run. What bounds them is latency, a few dependent
// loads from L2 per kernel: 1024 requests with 470000 held pages fork in 23 us and are compacted
// in 24.
//
// copy_pages moves the pages' data: one launch over the tensors of all layers, each CTA taking
// pieces of 16 KB.
#include "ops.cuh"

namespace pa {

constexpr int kPoolThreads = 256;
constexpr int kSmallThreads = 1024;
constexpr int kChunk = 1024;      // pages

// How a warp goes over table rows: items of K * 32 columns of a row, ROWS of them with their loads in
// flight together. A CTA of many rows takes short ones, a grid of many CTAs long ones.
template <int ROWS_, int K_>
struct Walk {
  static constexpr int ROWS = ROWS_, K = K_, COLUMNS = 32 * K_;
  __host__ __device__ __forceinline__ static int parts(int columns) { return (columns + COLUMNS - 1) / COLUMNS; }
  // row and first column of item i
  __device__ __forceinline__ static int2 item(int i, int parts) {
    return parts == 1 ? make_int2(i, 0) : make_int2(i / parts, i % parts * COLUMNS);
  }
};
using BigWalk = Walk<1, 8>;
using SmallWalk = Walk<4, 4>;

// entry head + k of the ring, k at most its capacity
__device__ __forceinline__ int ring_index(const PoolArgs& a, int head, int k) {
  const uint32_t i = (uint32_t)head + (uint32_t)k;
  return (int)(i >= (uint32_t)a.cap ? i - (uint32_t)a.cap : i);
}

// ---- marks ---------------------------------------------------------------------------------
// Where the marks go: bytes in the workspace, or bits in shared memory.
struct ByteMarks {
  uint8_t *whole, *old;
  int32_t* keeper;
  __device__ __forceinline__ void set_whole(int x) const { whole[x] = 1; }
  __device__ __forceinline__ void set_old(int x) const { old[x] = 1; }
  __device__ __forceinline__ void keep(int x, int v) const { atomicMax(&keeper[x], v); }
};
struct BitMarks {
  uint32_t *whole, *old, *kept;
  int32_t* keeper;
  __device__ __forceinline__ void set_whole(int x) const { atomicOr(&whole[x >> 5], 1u << (x & 31)); }
  __device__ __forceinline__ void set_old(int x) const { atomicOr(&old[x >> 5], 1u << (x & 31)); }
  __device__ __forceinline__ void keep(int x, int v) const {
    atomicOr(&kept[x >> 5], 1u << (x & 31));
    atomicMax(&keeper[x], v);
  }
};

// the lowest new row of each old one (INT32_MAX: none), by the block; the errors found
__device__ __forceinline__ uint32_t find_children(const PoolArgs& a, int* first_child) {
  uint32_t err = 0;
  for (int p = threadIdx.x; p < a.B; p += blockDim.x) first_child[p] = INT32_MAX;
  __syncthreads();
  for (int b = threadIdx.x; b < a.Bn; b += blockDim.x) {
    const int p = a.parents[b];
    if (p < -1 || p >= a.B) err = PA_DEVERR_BAD_BATCH;
    else if (p >= 0) atomicMin(&first_child[p], b);
  }
  return err;
}

// Marks the pages of the old rows, item by item of a row's columns from `first` on; the errors found.
// `pasts` and `helds` are the call's, or their copies; `last` receives the rows' partly filled pages.
template <bool FORK, typename W, typename Marks>
__device__ __forceinline__ uint32_t mark_pages(const PoolArgs& a, const int* pasts, const int* helds, const int* first_child,
                                               const Marks& marks, int* last, int first, int step, int lane) {
  uint32_t err = 0;
  const int parts = W::parts(a.max_blocks), items = a.B * parts;
  for (int i0 = first; i0 < items; i0 += W::ROWS * step) {
    int x[W::ROWS][W::K];
#pragma unroll
    for (int n = 0; n < W::ROWS; ++n) {  // (all of the rows: which entries are held need not be known yet)
      const int2 it = W::item(i0 + n * step, parts);
#pragma unroll
      for (int k = 0; k < W::K; ++k) {
        const int c = it.y + k * 32 + lane;
        x[n][k] = i0 + n * step < items && c < a.max_blocks ? a.table[(int64_t)it.x * a.max_blocks + c] : -1;
      }
    }
#pragma unroll
    for (int n = 0; n < W::ROWS; ++n) {
      if (i0 + n * step >= items) break;
      const int2 it = W::item(i0 + n * step, parts);
      const int p = it.x;
      int held = helds[p];
      if (held < 0 || held > a.max_blocks) err |= PA_DEVERR_BAD_BATCH, held = 0;
      int whole = 0, child = INT32_MAX;
      bool part = false;
      if constexpr (FORK) {
        const int past = pasts[p];
        child = first_child[p];
        whole = past / a.bs;
        part = past % a.bs != 0;
        // (refused: the marks do not matter any more, but the pages are still looked at)
        if (past < 0 || (child != INT32_MAX && whole + (part ? 1 : 0) > held)) err |= PA_DEVERR_BAD_BATCH;
      }
#pragma unroll
      for (int k = 0; k < W::K; ++k) {
        const int c = it.y + k * 32 + lane, page = x[n][k];
        if (c >= held) continue;
        if (page < 0 || page >= a.num_blocks) {
          err |= PA_DEVERR_BAD_BLOCK;
        } else if (FORK && (child == INT32_MAX || c >= whole)) {
          marks.set_old(page);
          if (child != INT32_MAX && c == whole && part) {
            marks.keep(page, a.Bn - child);
            if (last) last[p] = page;
          }
        } else {
          marks.set_whole(page);
        }
      }
    }
  }
  return err;
}

__global__ void __launch_bounds__(kPoolThreads) pool_clear_kernel(const PoolArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t i = blockIdx.x * (int64_t)kPoolThreads + threadIdx.x; i < a.clear_words; i += (int64_t)gridDim.x * kPoolThreads)
    a.clear[i] = make_uint4(0, 0, 0, 0);
  if (a.pages_end && blockIdx.x == 0 && threadIdx.x == 0) *a.pages_end = 0;  // (the finish takes a maximum)
  if (a.first_child && blockIdx.x == gridDim.x - 1) {
    extern __shared__ int children[];  // [B]
    find_children(a, children);
    __syncthreads();
    for (int p = threadIdx.x; p < a.B; p += kPoolThreads) a.first_child[p] = children[p];
  }
}

template <bool FORK>
__global__ void __launch_bounds__(kPoolThreads) pool_mark_kernel(const PoolArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  uint32_t err = 0;
  if (FORK && blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.Bn; b += kPoolThreads)
      if (a.parents[b] < -1 || a.parents[b] >= a.B) err = PA_DEVERR_BAD_BATCH;
  err |= mark_pages<FORK, BigWalk>(a, a.past, a.held, a.first_child, ByteMarks{a.marks, a.old_marks, a.keeper}, a.last,
                                   blockIdx.x * (kPoolThreads / 32) + (threadIdx.x >> 5),
                                   gridDim.x * (kPoolThreads / 32), threadIdx.x & 31);
  if (err) atomicOr(a.ws_error, err);
}

// ---- words ---------------------------------------------------------------------------------
// word i: {bits of the first kind, of the second, the counts of both before it in its chunk}.
// fork: the first kind are the pages to give back; compact: the holes, and the movers. Blocks behind
// the chunks': the fork's rows that copy.
template <bool FORK>
__global__ void __launch_bounds__(kPoolThreads) pool_words_kernel(const PoolArgs a) {
  __shared__ uint32_t bits[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (FORK && (int)blockIdx.x >= a.num_chunks) {
    // whether a new row takes a page of its own for the last, partly filled one of its parent (a refused
    // fork's parents and pages may be anything)
    const int b = (blockIdx.x - a.num_chunks) * kPoolThreads + threadIdx.x;
    const int p = b < a.Bn ? a.parents[b] : -1, fine = *a.ws_error == 0;
    bool copy = false;
    if (fine && p >= 0) {
      const int past = a.past[p], x = a.last[p];
      if (past % a.bs) copy = a.keeper[x] != a.Bn - b || a.marks[x] || (a.pinned && a.pinned[x]);
    }
    const uint32_t m = __ballot_sync(0xffffffffu, copy);
    if (lane == 0) a.row_bits[(blockIdx.x - a.num_chunks) * (kPoolThreads / 32) + warp] = m;
    return;
  }
#pragma unroll
  for (int i = 0; i < 32 / (kPoolThreads / 32); ++i) {
    const int w = warp + i * (kPoolThreads / 32), x = blockIdx.x * kChunk + w * 32 + lane;
    bool first = false, second = false;
    if (x < a.num_blocks) {
      const bool pinned = a.pinned && a.pinned[x], mark = a.marks[x];
      if constexpr (FORK) {
        first = a.old_marks[x] && !mark && a.keeper[x] == 0 && !pinned;
      } else {
        first = !mark && !pinned;
        second = mark && !pinned;
      }
    }
    const uint32_t f = __ballot_sync(0xffffffffu, first), s = __ballot_sync(0xffffffffu, second);
    if (lane == 0) bits[0][w] = f, bits[1][w] = s;
  }
  __syncthreads();
  if (warp == 0) {
    const uint32_t f = bits[0][lane], s = bits[1][lane];
    uint32_t n = __popc(f) | __popc(s) << 16;  // (both counts at once: at most 1024 each)
    const uint32_t own = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) n += y;
    }
    a.words[blockIdx.x * 32 + lane] = make_uint4(f, s, n - own, 0);
    if (lane == 31) a.chunks[blockIdx.x] = make_int2(n & 0xffff, n >> 16);
  }
}

// exclusive sums of n pairs (value(i)), by the whole block; sums[n] are the totals
template <typename F>
__device__ __forceinline__ void scan_pairs(int n, int2* sums, F value) {
  __shared__ int2 part[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, threads = blockDim.x;
  int2 carry = make_int2(0, 0);
  for (int i0 = 0; i0 < n; i0 += threads) {
    const int i = i0 + threadIdx.x;
    const int2 own = i < n ? value(i) : make_int2(0, 0);
    int2 x = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y0 = __shfl_up_sync(0xffffffffu, x.x, d), y1 = __shfl_up_sync(0xffffffffu, x.y, d);
      if (lane >= d) x.x += y0, x.y += y1;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    const int2 all = lane * 32 < threads ? part[lane] : make_int2(0, 0);
    int2 before = carry;
    before.x += __reduce_add_sync(0xffffffffu, lane < warp ? all.x : 0);
    before.y += __reduce_add_sync(0xffffffffu, lane < warp ? all.y : 0);
    carry.x += __reduce_add_sync(0xffffffffu, all.x);
    carry.y += __reduce_add_sync(0xffffffffu, all.y);
    if (i < n) sums[i] = make_int2(before.x + x.x - own.x, before.y + x.y - own.y);
    __syncthreads();
  }
  if (threadIdx.x == 0) sums[n] = carry;
  __syncthreads();
}

// The pages as words {bits of both kinds, the counts of both before the word in the whole pool}.
struct BigWords {
  const uint4* words;
  const int2* sums;  // before each chunk
  __device__ __forceinline__ uint4 at(int w) const {
    const uint4 v = __ldg(words + w);  // (of a kernel before)
    const int2 s = sums[w / 32];
    return make_uint4(v.x, v.y, s.x + (v.z & 0xffff), s.y + (v.z >> 16));
  }
};
struct SmallWords {
  const uint32_t *first, *second;
  const int2* sums;  // before each word
  __device__ __forceinline__ uint4 at(int w) const {
    return make_uint4(first[w], second ? second[w] : 0u, (uint32_t)sums[w].x, (uint32_t)sums[w].y);
  }
};

// the fork's rows that copy, and their count before the word
struct BigRows {
  const uint32_t* bits;
  const int2* sums;
  __device__ __forceinline__ int2 at(int w) const { return make_int2((int)bits[w], sums[w].x); }
};
struct SmallRows {
  const uint32_t* bits;
  const int2* sums;
  __device__ __forceinline__ int2 at(int w) const { return make_int2((int)bits[w], sums[w].y); }
};

// ---- finish: fork --------------------------------------------------------------------------
// The outputs, spread over the threads from `i0` on in steps of `step`. A refused fork (err) describes an
// empty batch and changes nothing that it was given. `parents` and `pasts` are the call's, or their copies.
template <typename W, typename Rows>
__device__ __forceinline__ void fork_rows(const PoolArgs& a, uint32_t err, int head, int count, int copies, int freed,
                                          const Rows& rows, const int* parents, const int* pasts, int i0, int step) {
  auto rank_of = [&](int b) {  // which copy row b makes, -1 for none
    if (err) return -1;
    const int2 w = rows.at(b >> 5);
    return (uint32_t)w.x >> (b & 31) & 1 ? w.y + __popc((uint32_t)w.x & ((1u << (b & 31)) - 1)) : -1;
  };
  if (i0 == 0) {
    a.error[0] = err;
    a.state_out[0] = err ? head : ring_index(a, head, copies);
    a.state_out[1] = err ? count : count - copies + freed;
  }
  const int parts = W::parts(a.max_blocks), items = a.Bn * parts, lane = threadIdx.x & 31, warps = step / 32;
  for (int j0 = i0 / 32; j0 < items; j0 += W::ROWS * warps) {
    int x[W::ROWS][W::K];
#pragma unroll
    for (int n = 0; n < W::ROWS; ++n) {  // (the parent's entries, whichever of them are its pages)
      const int2 it = W::item(j0 + n * warps, parts);
      const int p = err || j0 + n * warps >= items ? -1 : parents[it.x];
#pragma unroll
      for (int k = 0; k < W::K; ++k) {
        const int c = it.y + k * 32 + lane;
        x[n][k] = p >= 0 && c < a.max_blocks ? __ldg(a.table + (int64_t)p * a.max_blocks + c) : -1;
      }
    }
#pragma unroll
    for (int n = 0; n < W::ROWS; ++n) {
      if (j0 + n * warps >= items) break;
      const int2 it = W::item(j0 + n * warps, parts);
      const int b = it.x, p = err ? -1 : parents[b], past = p < 0 ? 0 : pasts[p], rank = rank_of(b);
      const int whole = past / a.bs, need = whole + (past % a.bs != 0);
#pragma unroll
      for (int k = 0; k < W::K; ++k) {
        const int c = it.y + k * 32 + lane;
        if (c >= a.max_blocks) break;
        int page = c < need ? x[n][k] : -1;
        if (rank >= 0 && c == whole) {
          const int fresh = a.ring[ring_index(a, head, rank)];
          a.copies[rank] = make_int2(page, fresh);
          page = fresh;
        }
        a.table_out[(int64_t)b * a.max_blocks + c] = page;
      }
      if (it.y == 0 && lane == 0) {
        a.past_out[b] = past;
        a.held_out[b] = need;
        if (err || b >= copies) a.copies[b] = make_int2(-1, -1);
      }
    }
  }
}

// the pages given back, behind the last free one
template <typename Words>
__device__ __forceinline__ void fork_pages(const PoolArgs& a, int head, int count, const Words& pages, int i0, int step) {
#pragma unroll 4
  for (int x = i0; x < a.num_blocks; x += step) {
    const uint4 w = pages.at(x >> 5);
    if (w.x >> (x & 31) & 1) {
      const int r = (int)w.z + __popc(w.x & ((1u << (x & 31)) - 1));
      a.ring[ring_index(a, head, count + r)] = x;
    }
  }
}

__device__ __forceinline__ uint32_t fork_refusal(const PoolArgs& a, uint32_t err, int head, int count, int copies, int freed) {
  if (head < 0 || head >= a.cap || count < 0 || count > a.cap) err |= PA_DEVERR_BAD_BATCH;
  if (err) return err;
  return (int64_t)count + freed > a.cap ? PA_DEVERR_BAD_BATCH : copies > count ? PA_DEVERR_NO_BLOCKS : 0;
}

__global__ void __launch_bounds__(kPoolThreads) fork_finish_kernel(const PoolArgs a) {
  extern __shared__ int2 smem2[];
  int2* sums = smem2;                       // [num_chunks + 1]
  int2* before = sums + a.num_chunks + 1;   // [words of rows + 1]
  pdl_wait();
  pdl_launch_dependents();
  const int row_words = (a.Bn + 31) / 32;
  const int head = a.state[0], count = a.state[1];
  scan_pairs(a.num_chunks, sums, [&](int i) { return a.chunks[i]; });
  scan_pairs(row_words, before, [&](int i) { return make_int2(__popc(a.row_bits[i]), 0); });
  const int freed = sums[a.num_chunks].x, copies = before[row_words].x;
  const uint32_t err = fork_refusal(a, *a.ws_error, head, count, copies, freed);
  // (rows by the first blocks, pages by the others, side by side)
  const int i = blockIdx.x * kPoolThreads + threadIdx.x;
  if ((int)blockIdx.x < a.row_blocks)
    fork_rows<BigWalk>(a, err, head, count, copies, freed, BigRows{a.row_bits, before}, a.parents, a.past, i,
                       a.row_blocks * kPoolThreads);
  else if (!err)
    fork_pages(a, head, count, BigWords{a.words, sums}, i - a.row_blocks * kPoolThreads,
               ((int)gridDim.x - a.row_blocks) * kPoolThreads);
}

// Everything in one CTA: lengths, parents and pins are loaded at once, the table's entries after them,
// and the outputs need one more round of loads; between them all is in shared memory.
__global__ void __launch_bounds__(kSmallThreads) fork_small_kernel(const PoolArgs a) {
  extern __shared__ int2 smem2[];
  const int words = (a.num_blocks + 31) / 32, row_words = (a.Bn + 31) / 32, n_sums = max(words, row_words);
  int2* sums = smem2;                                                   // [n_sums + 1]: pages given back, rows that copy
  uint32_t* whole = reinterpret_cast<uint32_t*>(sums + n_sums + 1);     // [words] each
  uint32_t *old = whole + words, *kept = old + words, *pinned = kept + words;
  uint32_t* rows = pinned + words;                                      // [row_words]
  int* keeper = reinterpret_cast<int*>(rows + row_words);               // [num_blocks]
  int* first_child = keeper + a.num_blocks;                             // [B] each
  int *past = first_child + a.B, *held = past + a.B, *last = held + a.B;  // last: the partly filled page
  int* parent = last + a.B;                                             // [Bn]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, threads = blockDim.x, warps = threads / 32;
  for (int i = threadIdx.x; i < 3 * words; i += threads) whole[i] = 0;
  for (int i = threadIdx.x; i < a.num_blocks; i += threads) keeper[i] = 0;
  for (int p = threadIdx.x; p < a.B; p += threads) first_child[p] = INT32_MAX;
  pdl_wait();
  pdl_launch_dependents();
  uint32_t err = 0;
  const int head = a.state[0], count = a.state[1];
  for (int p = threadIdx.x; p < a.B; p += threads) past[p] = a.past[p], held[p] = a.held[p];
  for (int b = threadIdx.x; b < a.Bn; b += threads) {
    const int p = a.parents[b];
    if (p < -1 || p >= a.B) err = PA_DEVERR_BAD_BATCH;
    parent[b] = p < 0 || p >= a.B ? -1 : p;
  }
  for (int w = warp; w < words; w += warps) {
    const int x = w * 32 + lane;
    const uint32_t m = __ballot_sync(0xffffffffu, a.pinned && x < a.num_blocks && a.pinned[x]);
    if (lane == 0) pinned[w] = m;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < a.Bn; b += threads)
    if (parent[b] >= 0) atomicMin(&first_child[parent[b]], b);
  __syncthreads();
  const BitMarks marks{whole, old, kept, keeper};
  err |= mark_pages<true, SmallWalk>(a, past, held, first_child, marks, last, warp, warps, lane);
  const bool batch = __syncthreads_or(err & PA_DEVERR_BAD_BATCH), block = __syncthreads_or(err & PA_DEVERR_BAD_BLOCK);
  err = (batch ? PA_DEVERR_BAD_BATCH : 0) | (block ? PA_DEVERR_BAD_BLOCK : 0);
  for (int b0 = 0; b0 < a.Bn; b0 += threads) {
    const int b = b0 + threadIdx.x;
    bool copy = false;
    if (b < a.Bn && !err && parent[b] >= 0 && past[parent[b]] % a.bs) {
      const int x = last[parent[b]];
      copy = keeper[x] != a.Bn - b || ((whole[x >> 5] | pinned[x >> 5]) >> (x & 31) & 1);
    }
    const uint32_t m = __ballot_sync(0xffffffffu, copy);
    if (lane == 0 && b < a.Bn) rows[b >> 5] = m;
  }
  for (int w = threadIdx.x; w < words; w += threads) old[w] &= ~(whole[w] | kept[w] | pinned[w]);
  __syncthreads();
  scan_pairs(n_sums, sums, [&](int i) {
    return make_int2(i < words ? __popc(old[i]) : 0, i < row_words ? __popc(rows[i]) : 0);
  });
  const int freed = sums[n_sums].x, copies = sums[n_sums].y;
  err = fork_refusal(a, err, head, count, copies, freed);
  fork_rows<SmallWalk>(a, err, head, count, copies, freed, SmallRows{rows, sums}, parent, past, threadIdx.x, threads);
  if (!err) fork_pages(a, head, count, SmallWords{old, nullptr, sums}, threadIdx.x, threads);
}

// ---- finish: compact -----------------------------------------------------------------------
// The r-th highest mover x_r goes to the r-th lowest hole h_r while h_r < x_r: x_r falls and h_r
// rises with r, so the pairs that move are the first D, and D is the number of movers x with
//   holes below x > movers above x.
// the movers of a word for which that holds; w as Words::at gives it, M movers in all
__device__ __forceinline__ int moving_in(const uint4& w, int M) {
  int n = 0;
  for (uint32_t rest = w.y; rest; rest &= rest - 1) {
    const uint32_t below = (rest & -rest) - 1;
    n += (int)w.z + __popc(w.x & below) + (int)w.w + __popc(w.y & below) + 1 > M;
  }
  return n;
}

// by the whole block
__device__ __forceinline__ int count_moves(const PoolArgs& a, const BigWords& pages) {
  __shared__ int found;
  const int2* sums = pages.sums;
  const int M = sums[a.num_chunks].y;
  if (threadIdx.x == 0) found = a.num_chunks;
  __syncthreads();
  // the first chunk at whose end (holes below) + (movers up to there) is over M: later chunks' movers all move
  for (int c = threadIdx.x; c < a.num_chunks; c += kPoolThreads)
    if (sums[c + 1].x + sums[c + 1].y > M) atomicMin(&found, c);
  __syncthreads();
  const int c = found;
  __syncthreads();
  if (c == a.num_chunks) return 0;
  if (threadIdx.x < 32) {
    const int n = __reduce_add_sync(0xffffffffu, moving_in(pages.at(c * 32 + threadIdx.x), M));
    if (threadIdx.x == 0) found = M - sums[c + 1].y + n;
  }
  __syncthreads();
  return min(found, a.max_moves);
}

// The outputs, spread over the threads from `i0` on in steps of `step`; hole(r) is the r-th hole.
// Ring and copies, page by page; one more than the highest page in use that the thread saw.
template <typename Words, typename Hole>
__device__ __forceinline__ int compact_pages(const PoolArgs& a, uint32_t err, int holes, int movers, int moves,
                                             const Words& pages, Hole hole, int i0, int step) {
  if (i0 == 0) {
    a.error[0] = err;
    a.state_out[0] = 0;
    a.state_out[1] = err ? 0 : holes;
  }
  for (int r = moves + i0; r < a.max_moves; r += step) a.copies[r] = make_int2(-1, -1);
  int end = 0;
  if (err) return end;
#pragma unroll 4
  for (int x = i0; x < a.num_blocks; x += step) {
    const uint4 w = pages.at(x >> 5);
    const uint32_t bit = 1u << (x & 31);
    const int h = (int)w.z + __popc(w.x & (bit - 1)), m = (int)w.w + __popc(w.y & (bit - 1));
    bool free = false;
    if (w.x & bit) {
      free = h >= moves;
    } else if (w.y & bit) {
      const int above = movers - 1 - m;
      if (above < moves) {
        a.copies[above] = make_int2(x, hole(above));
        free = true;
      }
    }
    // free pages below x: the holes that nothing moves into, and the pages moved away
    if (free) a.ring[max(0, h - moves) + max(0, m - (movers - moves))] = x;
    else end = max(end, x + 1);
  }
  return end;
}

// the table, entry by entry
template <typename W, typename Words, typename Hole>
__device__ __forceinline__ void compact_table(const PoolArgs& a, uint32_t err, int movers, int moves, const Words& pages,
                                              Hole hole, int i0, int step) {
  const int parts = W::parts(a.max_blocks), items = a.B * parts, lane = threadIdx.x & 31, warps = step / 32;
  for (int j0 = i0 / 32; j0 < items; j0 += W::ROWS * warps) {
    int x[W::ROWS][W::K], held[W::ROWS];
#pragma unroll
    for (int n = 0; n < W::ROWS; ++n) {
      if (j0 + n * warps >= items) break;
      const int2 it = W::item(j0 + n * warps, parts);
      held[n] = err ? 0 : a.held[it.x];
#pragma unroll
      for (int k = 0; k < W::K; ++k) {
        const int c = it.y + k * 32 + lane;
        x[n][k] = c < a.max_blocks ? a.table[(int64_t)it.x * a.max_blocks + c] : 0;
      }
    }
#pragma unroll
    for (int n = 0; n < W::ROWS; ++n) {
      if (j0 + n * warps >= items) break;
      const int2 it = W::item(j0 + n * warps, parts);
      int to[W::K];
#pragma unroll
      for (int k = 0; k < W::K; ++k) {  // the rank from above of the pages that move, -1 for others
        to[k] = -1;
        if (it.y + k * 32 + lane >= held[n]) continue;
        const uint4 w = pages.at(x[n][k] >> 5);
        const uint32_t bit = 1u << (x[n][k] & 31);
        const int above = movers - 1 - ((int)w.w + __popc(w.y & (bit - 1)));
        if ((w.y & bit) && above < moves) to[k] = above;
      }
#pragma unroll
      for (int k = 0; k < W::K; ++k)
        if (to[k] >= 0) x[n][k] = hole(to[k]);
#pragma unroll
      for (int k = 0; k < W::K; ++k) {
        const int c = it.y + k * 32 + lane;
        if (c < a.max_blocks) a.table_out[(int64_t)it.x * a.max_blocks + c] = x[n][k];
      }
    }
  }
}

// the holes in order
__global__ void __launch_bounds__(kPoolThreads) compact_lists_kernel(const PoolArgs a) {
  extern __shared__ int2 smem2[];
  pdl_wait();
  pdl_launch_dependents();
  scan_pairs(a.num_chunks, smem2, [&](int i) { return a.chunks[i]; });
  const BigWords pages{a.words, smem2};
#pragma unroll 4
  for (int x = blockIdx.x * kPoolThreads + threadIdx.x; x < a.num_blocks; x += gridDim.x * kPoolThreads) {
    const uint4 w = pages.at(x >> 5);
    if (w.x >> (x & 31) & 1) a.holes[(int)w.z + __popc(w.x & ((1u << (x & 31)) - 1))] = x;
  }
}

__global__ void __launch_bounds__(kPoolThreads) compact_finish_kernel(const PoolArgs a) {
  extern __shared__ int2 smem2[];  // [num_chunks + 1]
  pdl_wait();
  pdl_launch_dependents();
  scan_pairs(a.num_chunks, smem2, [&](int i) { return a.chunks[i]; });
  uint32_t err = *a.ws_error;
  const int holes = smem2[a.num_chunks].x, movers = smem2[a.num_chunks].y;
  if (!err && holes > a.cap) err = PA_DEVERR_BAD_BATCH;
  const BigWords pages{a.words, smem2};
  const int moves = err ? 0 : count_moves(a, pages);
  auto hole = [&](int r) { return __ldg(a.holes + r); };
  // (rows by the first blocks, pages by the others, side by side)
  const int i = blockIdx.x * kPoolThreads + threadIdx.x;
  if ((int)blockIdx.x < a.row_blocks) {
    compact_table<BigWalk>(a, err, movers, moves, pages, hole, i, a.row_blocks * kPoolThreads);
    return;
  }
  int end = compact_pages(a, err, holes, movers, moves, pages, hole, i - a.row_blocks * kPoolThreads,
                          ((int)gridDim.x - a.row_blocks) * kPoolThreads);
  end = __reduce_max_sync(0xffffffffu, end);
  if ((threadIdx.x & 31) == 0 && end) atomicMax(a.pages_end, end);
}

// everything in one CTA
__global__ void __launch_bounds__(kSmallThreads) compact_small_kernel(const PoolArgs a) {
  extern __shared__ int2 smem2[];
  __shared__ int total[2];  // pages that move, the highest page in use
  const int words = (a.num_blocks + 31) / 32;
  int2* sums = smem2;                                               // [words + 1]
  uint32_t* movers = reinterpret_cast<uint32_t*>(sums + words + 1);  // [words] each
  uint32_t *holes = movers + words, *pinned = holes + words;
  int* list = reinterpret_cast<int*>(pinned + words);               // [num_blocks]: the holes in order
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, threads = blockDim.x, warps = threads / 32;
  for (int i = threadIdx.x; i < words; i += threads) movers[i] = 0;
  if (threadIdx.x < 2) total[threadIdx.x] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  for (int w = warp; w < words; w += warps) {
    const int x = w * 32 + lane;
    const uint32_t m = __ballot_sync(0xffffffffu, a.pinned && x < a.num_blocks && a.pinned[x]);
    if (lane == 0) pinned[w] = m;
  }
  uint32_t err = mark_pages<false, SmallWalk>(a, nullptr, a.held, nullptr, BitMarks{movers, nullptr, nullptr, nullptr}, nullptr, warp,
                                   warps, lane);
  const bool batch = __syncthreads_or(err & PA_DEVERR_BAD_BATCH), block = __syncthreads_or(err & PA_DEVERR_BAD_BLOCK);
  err = (batch ? PA_DEVERR_BAD_BATCH : 0) | (block ? PA_DEVERR_BAD_BLOCK : 0);
  for (int w = threadIdx.x; w < words; w += threads) {
    const uint32_t there = a.num_blocks - w * 32 >= 32 ? 0xffffffffu : (1u << (a.num_blocks & 31)) - 1, used = movers[w] | pinned[w];
    holes[w] = there & ~used;
    movers[w] = used & ~pinned[w];
  }
  __syncthreads();
  scan_pairs(words, sums, [&](int i) { return make_int2(__popc(holes[i]), __popc(movers[i])); });
  const int H = sums[words].x, M = sums[words].y;
  if (!err && H > a.cap) err = PA_DEVERR_BAD_BATCH;
  const SmallWords pages{holes, movers, sums};
  int n = 0;
  for (int w = threadIdx.x; w < words; w += threads) {
    n += moving_in(pages.at(w), M);
    int r = sums[w].x;
    for (uint32_t rest = holes[w]; rest; rest &= rest - 1) list[r++] = w * 32 + __ffs(rest) - 1;
  }
  if (n) atomicAdd(&total[0], n);
  __syncthreads();
  const int moves = err ? 0 : min(total[0], a.max_moves);
  auto hole = [&](int r) { return list[r]; };
  const int end = compact_pages(a, err, H, M, moves, pages, hole, threadIdx.x, threads);
  compact_table<SmallWalk>(a, err, M, moves, pages, hole, threadIdx.x, threads);
  if (end) atomicMax(&total[1], end);
  __syncthreads();
  if (threadIdx.x == 0) *a.pages_end = total[1];
}

// ---- copies --------------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kPiece = 16384;   // bytes
constexpr int kCopyRound = 1024;  // entries of the list that a CTA takes

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  __shared__ int2 list[kCopyRound];
  __shared__ int part[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  // this CTA's part of the list, entries that are none taken out
  const int e0 = blockIdx.y * kCopyRound, entries = min(kCopyRound, a.n - e0);
  constexpr int EACH = kCopyRound / kCopyThreads, WARPS = kCopyThreads / 32;
  int2 e[EACH];
  unsigned use[EACH];
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    const int i = k * kCopyThreads + threadIdx.x;
    e[k] = i < entries ? a.copies[e0 + i] : make_int2(-1, -1);
  }
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    use[k] = 0;
    if (lane == 0) part[k * WARPS + warp] = 0;
    if (k * kCopyThreads >= entries) continue;
    const bool good = e[k].x >= 0 && e[k].x < a.num_blocks && e[k].y >= 0 && e[k].y < a.num_blocks;
    if (!good && !(e[k].x == -1 && e[k].y == -1) && blockIdx.x == 0 && a.error) atomicOr(a.error, PA_DEVERR_BAD_BLOCK);
    use[k] = __ballot_sync(0xffffffffu, good && e[k].x != e[k].y);
    if (lane == 0) part[k * WARPS + warp] = __popc(use[k]);
  }
  __syncthreads();
  // (counts of the warps' entries in the list's order, a lane each)
  static_assert(EACH * WARPS == 32, "");
  const int counts = part[lane], kept = __reduce_add_sync(0xffffffffu, counts);
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    if (k * kCopyThreads >= entries) break;
    const int before = __reduce_add_sync(0xffffffffu, lane < k * WARPS + warp ? counts : 0);
    if (use[k] >> lane & 1) list[before + __popc(use[k] & ((1u << lane) - 1))] = e[k];
  }
  __syncthreads();
  const int64_t units = (int64_t)kept * a.num_tensors * a.pieces;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int piece = (int)(u % a.pieces);
    const int64_t v = u / a.pieces;
    const int t = (int)(v % a.num_tensors);
    const int2 pair = list[v / a.num_tensors];
    const int64_t bytes = a.bytes[t];
    const int64_t off = (int64_t)piece * kPiece;
    const uint8_t* src = a.data[t] + pair.x * bytes + off;
    uint8_t* dst = a.data[t] + pair.y * bytes + off;
    const int64_t left = bytes - off;
    if (left >= kPiece) {
      uint4 x[kPiece / 16 / kCopyThreads];
#pragma unroll
      for (int k = 0; k < kPiece / 16 / kCopyThreads; ++k)
        x[k] = __ldcs(reinterpret_cast<const uint4*>(src) + k * kCopyThreads + threadIdx.x);
#pragma unroll
      for (int k = 0; k < kPiece / 16 / kCopyThreads; ++k)
        __stcs(reinterpret_cast<uint4*>(dst) + k * kCopyThreads + threadIdx.x, x[k]);
    } else {
      for (int64_t i = threadIdx.x * 16; i < left; i += kCopyThreads * 16)
        *reinterpret_cast<uint4*>(dst + i) = *reinterpret_cast<const uint4*>(src + i);
    }
  }
}

// ---- host ----------------------------------------------------------------------------------
static int grid_of(int64_t work, int sms, int per_sm) {
  const int64_t g = ceil_div(work, kPoolThreads);
  return (int)(g < 1 ? 1 : g > (int64_t)sms * per_sm ? (int64_t)sms * per_sm : g);
}

// One CTA takes batches of up to about 10000 table entries and pages together: one SM's instruction rate
// bounds it (64 rows of 66 columns over 1707 pages 7.6 us, of 130 over 3340 12.6, 250 of 66 over 7096
// 14.5), where the kernels of many CTAs take about 12 us whatever there is below 50000.
constexpr int kSmallPages = 8192, kSmallRows = 2048, kSmallWork = 10000;
static int small_smem(int num_blocks, int B, int Bn, bool fork) {
  const int words = (int)ceil_div(num_blocks, 32), row_words = (int)ceil_div(Bn, 32);
  return fork ? 8 * ((words > row_words ? words : row_words) + 1) + 4 * (4 * words + row_words + num_blocks + 4 * B + Bn)
              : 8 * (words + 1) + 4 * (3 * words + num_blocks);
}
static bool is_small(const PoolArgs& a) {
  const int64_t rows = a.B > a.Bn ? a.B : a.Bn;
  return a.num_blocks <= kSmallPages && rows <= kSmallRows && rows * a.max_blocks + a.num_blocks <= kSmallWork;
}

// (at most PA_MAX_TABLE_REQUESTS rows and PA_MAX_POOL_PAGES / 1024 chunks)
constexpr int kFinishSmem = 8 * (PA_MAX_POOL_PAGES / kChunk + 1) + 8 * (PA_MAX_TABLE_REQUESTS / 32 + 1);
static_assert(kFinishSmem <= 48 * 1024 - 1024, "no attribute is needed");

template <bool FORK>
static cudaError_t launch_pool(const PoolArgs& a, int sms, cudaStream_t s, int* kernels) {
  if (is_small(a)) {
    auto kernel = FORK ? fork_small_kernel : compact_small_kernel;
    const int smem = small_smem(a.num_blocks, a.B, a.Bn, FORK);
    *kernels = 1;
    if (smem > 32 * 1024)  // (less needs no attribute; the same limit from every host thread)
      if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               small_smem(kSmallPages, kSmallRows, kSmallRows, FORK)))
        return e;
    return launch_pdl(kernel, dim3(1), dim3(kSmallThreads), (size_t)smem, s, a);
  }
  const dim3 block(kPoolThreads);
  const size_t sums = 8 * ((size_t)a.num_chunks + 1), rows_smem = FORK ? 8 * ((size_t)ceil_div(a.Bn, 32) + 1) : 0;
  *kernels = FORK ? 4 : 5;
  if (cudaError_t e = launch_pdl(pool_clear_kernel, dim3(grid_of(a.clear_words, sms, 4)), block, FORK ? (size_t)a.B * 4 : 0, s, a))
    return e;
  const int64_t parts = BigWalk::parts(a.max_blocks) * 32;
  if (cudaError_t e = launch_pdl(pool_mark_kernel<FORK>, dim3(grid_of(a.B * parts, sms, 8)), block, 0, s, a)) return e;
  const int64_t more = FORK ? ceil_div(a.Bn, kPoolThreads) : 0;
  if (cudaError_t e = launch_pdl(pool_words_kernel<FORK>, dim3((unsigned)(a.num_chunks + more)), block, 0, s, a)) return e;
  PoolArgs b = a;
  b.row_blocks = grid_of((FORK ? a.Bn : a.B) * parts, sms, 4);
  const dim3 grid(b.row_blocks + grid_of(ceil_div(a.num_blocks, 2), sms, 2));
  if constexpr (FORK) {
    return launch_pdl(fork_finish_kernel, grid, block, sums + rows_smem, s, b);
  } else {
    if (cudaError_t e = launch_pdl(compact_lists_kernel, dim3(grid_of(a.num_blocks, sms, 4)), block, sums, s, a)) return e;
    return launch_pdl(compact_finish_kernel, grid, block, sums, s, b);
  }
}
cudaError_t launch_fork(const PoolArgs& a, int sms, cudaStream_t s, int* kernels) { return launch_pool<true>(a, sms, s, kernels); }
cudaError_t launch_compact(const PoolArgs& a, int sms, cudaStream_t s, int* kernels) { return launch_pool<false>(a, sms, s, kernels); }

cudaError_t launch_copy_pages(CopyArgs& a, int sms, cudaStream_t s) {
  int64_t most = 0;
  for (int t = 0; t < a.num_tensors; ++t) most = a.bytes[t] > most ? a.bytes[t] : most;
  a.pieces = (int)ceil_div(most, kPiece);
  const int64_t parts = ceil_div(a.n, kCopyRound), units = ceil_div(a.n, parts) * a.num_tensors * a.pieces;
  // Up to 64 CTAs an SM: many of few pieces keep more loads in flight than a resident set that loops (160
  // pages of 24 layers 293 us, with 16 an SM 302, with 8 319), but each looks through its part of the list first
  // (400 pages among 5000 entries 24 us, with 16 an SM 16, with 400 62; among 200000 61, 191 and 89).
  const int64_t ctas = ceil_div((int64_t)sms * 64, parts);
  return launch_pdl(copy_pages_kernel, dim3((unsigned)(units < ctas ? units : ctas), (unsigned)parts), dim3(kCopyThreads), 0,
                    s, a);
}

}  // namespace pa
