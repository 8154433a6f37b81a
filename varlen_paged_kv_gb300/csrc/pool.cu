// The pages of a pool as requests fork, end and are compacted, and the copies that this takes.
//
// fork_block_tables makes the rows of a new batch from rows of the old one; compact_block_tables
// moves the highest pages in use into the lowest free ones. Both ask of every page of the pool
// what the tables hold it for, so both run as four short kernels over a workspace of marks:
//   clear   the marks
//   mark    every held table entry stores a byte at its page (the same byte from whoever
//           stores it, so without atomics); a row that would write into its last page next
//           leaves its number there by an atomic maximum (of Bn - row: the lowest row stays)
//   words   the marks as bits, 32 pages a word, with counts before each word inside its chunk of
//           1024 pages and the chunks' totals
//   finish  every CTA scans the chunks' totals (1024 at most) itself; a page's rank among the
//           pages of its kind is then its chunk's sum, its word's and a population count, and the
//           r-th page of a kind is found by bisection in them. Tables, ring and copies are
//           written from that, each entry by itself.
// Every order (of pages given out, given back and moved) is one of page or row numbers, so results
// do not depend on the order in which CTAs run.
//
// copy_pages moves the pages' data: one launch over the tensors of all layers, each CTA taking
// pieces of 16 KB.
#include "ops.cuh"

namespace pa {

constexpr int kPoolThreads = 256;
constexpr int kChunk = 1024;      // pages
constexpr int kColumns = 256;     // columns of a table row that a warp takes at a time

// ---- clear ---------------------------------------------------------------------------------
__global__ void __launch_bounds__(kPoolThreads) pool_clear_kernel(uint4* p, int64_t n) {
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t i = blockIdx.x * (int64_t)kPoolThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kPoolThreads)
    p[i] = make_uint4(0, 0, 0, 0);
}

// ---- mark ----------------------------------------------------------------------------------
template <bool FORK>
__global__ void __launch_bounds__(kPoolThreads) pool_mark_kernel(const PoolArgs a) {
  extern __shared__ int first_child[];  // FORK: the lowest new row of each old one
  pdl_wait();
  pdl_launch_dependents();
  uint32_t err = 0;
  if (!FORK && blockIdx.x == 0 && threadIdx.x == 0) *a.pages_end = 0;  // (the finish takes a maximum)
  if constexpr (FORK) {
    for (int p = threadIdx.x; p < a.B; p += kPoolThreads) first_child[p] = INT32_MAX;
    __syncthreads();
    for (int b = threadIdx.x; b < a.Bn; b += kPoolThreads) {
      const int p = a.parents[b];
      if (p < -1 || p >= a.B) err = PA_DEVERR_BAD_BATCH;
      else if (p >= 0) atomicMin(&first_child[p], b);
    }
    __syncthreads();
  }
  const int lane = threadIdx.x & 31;
  const int parts = (a.max_blocks + kColumns - 1) / kColumns;
  const int64_t items = (int64_t)a.B * parts, step = (int64_t)gridDim.x * (kPoolThreads / 32);
  for (int64_t i = blockIdx.x * (int64_t)(kPoolThreads / 32) + (threadIdx.x >> 5); i < items; i += step) {
    const int p = (int)(i / parts), c0 = (int)(i % parts) * kColumns;
    const int held = a.held[p];
    if (held < 0 || held > a.max_blocks) {
      err |= PA_DEVERR_BAD_BATCH;
      continue;
    }
    int whole = 0, child = INT32_MAX;
    bool part = false;
    if constexpr (FORK) {
      const int past = a.past[p];
      child = first_child[p];
      whole = past / a.bs;
      part = past % a.bs != 0;
      if (past < 0 || (child != INT32_MAX && whole + (part ? 1 : 0) > held)) {
        err |= PA_DEVERR_BAD_BATCH;
        continue;
      }
    }
    int x[kColumns / 32];
#pragma unroll
    for (int k = 0; k < kColumns / 32; ++k) {
      const int c = c0 + k * 32 + lane;
      x[k] = c < held ? a.table[(int64_t)p * a.max_blocks + c] : -1;
      if (c < held && (x[k] < 0 || x[k] >= a.num_blocks)) err |= PA_DEVERR_BAD_BLOCK, x[k] = -1;
    }
#pragma unroll
    for (int k = 0; k < kColumns / 32; ++k) {
      const int c = c0 + k * 32 + lane;
      if (x[k] < 0) continue;
      if (FORK && (child == INT32_MAX || c >= whole)) {
        a.old_marks[x[k]] = 1;
        if (child != INT32_MAX && c == whole && part) atomicMax(&a.keeper[x[k]], a.Bn - child);
      } else {
        a.marks[x[k]] = 1;
      }
    }
  }
  if (err) atomicOr(a.ws_error, err);
}

// ---- words ---------------------------------------------------------------------------------
// word i: {bits of the first kind, of the second, the counts of both before it in its chunk}.
// fork: the first kind are the pages to give back; compact: the holes, and the movers.
template <bool FORK>
__global__ void __launch_bounds__(kPoolThreads) pool_words_kernel(const PoolArgs a) {
  __shared__ uint32_t bits[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int w = warp; w < 32; w += kPoolThreads / 32) {
    const int x = blockIdx.x * kChunk + w * 32 + lane;
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

// exclusive sums of the chunks' totals, and the totals at [chunks]
__device__ __forceinline__ void scan_chunks(const PoolArgs& a, int2* sums) {
  __shared__ int2 part[kPoolThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int2 carry = make_int2(0, 0);
  const int n = a.num_chunks;
  for (int i0 = 0; i0 < n; i0 += kPoolThreads) {
    const int i = i0 + threadIdx.x;
    const int2 own = i < n ? a.chunks[i] : make_int2(0, 0);
    int2 x = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y0 = __shfl_up_sync(0xffffffffu, x.x, d), y1 = __shfl_up_sync(0xffffffffu, x.y, d);
      if (lane >= d) x.x += y0, x.y += y1;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int2 before = carry;
    for (int w = 0; w < kPoolThreads / 32; ++w) {
      if (w < warp) before.x += part[w].x, before.y += part[w].y;
      carry.x += part[w].x, carry.y += part[w].y;
    }
    if (i < n) sums[i] = make_int2(before.x + x.x - own.x, before.y + x.y - own.y);
    __syncthreads();
  }
  if (threadIdx.x == 0) sums[n] = carry;
  __syncthreads();
}

// ---- finish: fork --------------------------------------------------------------------------
__global__ void __launch_bounds__(kPoolThreads) fork_finish_kernel(const PoolArgs a) {
  extern __shared__ int smem[];
  int2* sums = reinterpret_cast<int2*>(smem);          // [num_chunks + 1]
  int* rank = smem + 2 * (a.num_chunks + 1);           // [Bn]: which copy a row makes, -1 for none
  __shared__ int part[kPoolThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  uint32_t err = *a.ws_error;
  const int head = a.state[0], count = a.state[1];
  if (head < 0 || head >= a.cap || count < 0 || count > a.cap) err |= PA_DEVERR_BAD_BATCH;
  scan_chunks(a, sums);
  const int freed = sums[a.num_chunks].x;
  int copies = 0;
  if (!err) {  // (the rows' parents and pages are what they should be)
    for (int b0 = 0; b0 < a.Bn; b0 += kPoolThreads) {
      const int b = b0 + threadIdx.x;
      bool copy = false;
      if (b < a.Bn) {
        const int p = a.parents[b], past = p < 0 ? 0 : a.past[p];
        if (past % a.bs) {
          const int x = a.table[(int64_t)p * a.max_blocks + past / a.bs];
          copy = a.keeper[x] != a.Bn - b || a.marks[x] || (a.pinned && a.pinned[x]);
        }
      }
      const unsigned m = __ballot_sync(0xffffffffu, copy);
      if (lane == 0) part[warp] = __popc(m);
      __syncthreads();
      int before = copies;
      for (int w = 0; w < kPoolThreads / 32; ++w) {
        if (w < warp) before += part[w];
        copies += part[w];
      }
      if (b < a.Bn) rank[b] = copy ? before + __popc(m & ((1u << lane) - 1)) : -1;
      __syncthreads();
    }
    if ((int64_t)count + freed > a.cap) err = PA_DEVERR_BAD_BATCH;
    else if (copies > count) err = PA_DEVERR_NO_BLOCKS;
  }
  // A refused fork describes an empty batch and changes nothing that it was given.
  const int i0 = blockIdx.x * kPoolThreads + threadIdx.x, step = gridDim.x * kPoolThreads;
  if (i0 == 0) {
    a.error[0] = err;
    a.state_out[0] = err ? head : (int)(((int64_t)head + copies) % a.cap);
    a.state_out[1] = err ? count : count - copies + freed;
  }
  for (int b = i0; b < a.Bn; b += step) {
    const int p = err ? -1 : a.parents[b], past = p < 0 ? 0 : a.past[p];
    a.past_out[b] = past;
    a.held_out[b] = past / a.bs + (past % a.bs != 0);
    if (err || b >= copies) a.copies[b] = make_int2(-1, -1);
    if (!err && rank[b] >= 0)
      a.copies[rank[b]] = make_int2(a.table[(int64_t)p * a.max_blocks + past / a.bs],
                                    a.ring[((int64_t)head + rank[b]) % a.cap]);
  }
  const int parts = (a.max_blocks + kColumns - 1) / kColumns;
  const int64_t items = (int64_t)a.Bn * parts, stride = (int64_t)gridDim.x * (kPoolThreads / 32);
  for (int64_t i = blockIdx.x * (int64_t)(kPoolThreads / 32) + warp; i < items; i += stride) {
    const int b = (int)(i / parts), c0 = (int)(i % parts) * kColumns;
    const int p = err ? -1 : a.parents[b], past = p < 0 ? 0 : a.past[p];
    const int whole = past / a.bs, need = whole + (past % a.bs != 0);
    const int fresh = !err && rank[b] >= 0 && whole >= c0 && whole < c0 + kColumns
                          ? a.ring[((int64_t)head + rank[b]) % a.cap] : -1;
    int x[kColumns / 32];
#pragma unroll
    for (int k = 0; k < kColumns / 32; ++k) {
      const int c = c0 + k * 32 + lane;
      x[k] = c < need ? a.table[(int64_t)p * a.max_blocks + c] : -1;
      if (!err && rank[b] >= 0 && c == whole) x[k] = fresh;
    }
#pragma unroll
    for (int k = 0; k < kColumns / 32; ++k) {
      const int c = c0 + k * 32 + lane;
      if (c < a.max_blocks) a.table_out[(int64_t)b * a.max_blocks + c] = x[k];
    }
  }
  if (err) return;
  for (int x = i0; x < a.num_blocks; x += step) {  // the pages given back, behind the last free one
    const uint4 w = a.words[x >> 5];
    if (w.x >> (x & 31) & 1) {
      const int r = sums[x / kChunk].x + (w.z & 0xffff) + __popc(w.x & ((1u << (x & 31)) - 1));
      a.ring[((int64_t)head + count + r) % a.cap] = x;
    }
  }
}

// ---- finish: compact -----------------------------------------------------------------------
// The r-th highest mover x_r goes to the r-th lowest hole h_r while h_r < x_r: x_r falls and h_r
// rises with r, so the pairs that move are the first D, and D is the number of movers x with
//   holes below x > movers above x.
struct Compaction {
  int holes, movers, moves;
};

// by the whole block; `sums` as scan_chunks leaves it
__device__ __forceinline__ int count_moves(const PoolArgs& a, const int2* sums) {
  __shared__ int found;
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
    const int lane = threadIdx.x;
    const uint4 w = a.words[c * 32 + lane];
    const int h0 = sums[c].x + (w.z & 0xffff), m0 = sums[c].y + (w.z >> 16);
    int n = 0;  // movers of this word that move
    for (uint32_t rest = w.y; rest; rest &= rest - 1) {
      const uint32_t below = (rest & -rest) - 1;
      n += h0 + __popc(w.x & below) + m0 + __popc(w.y & below) + 1 > M;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
    if (lane == 0) found = M - sums[c + 1].y + n;
  }
  __syncthreads();
  return min(found, a.max_moves);
}

// the r-th hole
__device__ __forceinline__ int hole_at(const PoolArgs& a, const int2* sums, int r) {
  int lo = 0, n = a.num_chunks;  // the last chunk with at most r holes before it
  while (n > 1) {
    const int half = n >> 1;
    if (sums[lo + half].x <= r) lo += half, n -= half;
    else n = half;
  }
  r -= sums[lo].x;
  int w = lo * 32;
#pragma unroll
  for (int d = 16; d; d >>= 1)
    if ((int)(a.words[w + d].z & 0xffff) <= r) w += d;
  const uint4 word = a.words[w];
  r -= word.z & 0xffff;
  uint32_t bits = word.x;
  int at = 0;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const int low = __popc(bits & ((1u << d) - 1));
    if (low <= r) r -= low, at += d, bits >>= d;
  }
  return w * 32 + at;
}

__global__ void __launch_bounds__(kPoolThreads) compact_finish_kernel(const PoolArgs a) {
  extern __shared__ int smem[];
  int2* sums = reinterpret_cast<int2*>(smem);  // [num_chunks + 1]
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  scan_chunks(a, sums);
  uint32_t err = *a.ws_error;
  const int holes = sums[a.num_chunks].x, movers = sums[a.num_chunks].y;
  if (!err && holes > a.cap) err = PA_DEVERR_BAD_BATCH;
  const int moves = err ? 0 : count_moves(a, sums);
  // where page x goes: itself, or the hole of its rank from above
  auto moved = [&](int x) {
    const uint4 w = a.words[x >> 5];
    if (!(w.y >> (x & 31) & 1)) return x;
    const int above = movers - 1 - (sums[x / kChunk].y + (int)(w.z >> 16) + __popc(w.y & ((1u << (x & 31)) - 1)));
    return above < moves ? hole_at(a, sums, above) : x;
  };
  const int i0 = blockIdx.x * kPoolThreads + threadIdx.x, step = gridDim.x * kPoolThreads;
  if (i0 == 0) {
    a.error[0] = err;
    a.state_out[0] = 0;
    a.state_out[1] = err ? 0 : holes;
  }
  for (int r = moves + i0; r < a.max_moves; r += step) a.copies[r] = make_int2(-1, -1);
  int end = 0;
  if (!err)
    for (int x = i0; x < a.num_blocks; x += step) {
      const uint4 w = a.words[x >> 5];
      const uint32_t bit = 1u << (x & 31);
      const int h = sums[x / kChunk].x + (w.z & 0xffff) + __popc(w.x & (bit - 1));
      const int m = sums[x / kChunk].y + (int)(w.z >> 16) + __popc(w.y & (bit - 1));
      bool free = false;
      if (w.x & bit) {
        free = h >= moves;
      } else if (w.y & bit) {
        const int above = movers - 1 - m;
        if (above < moves) {
          a.copies[above] = make_int2(x, hole_at(a, sums, above));
          free = true;
        }
      }
      // free pages below x: the holes that nothing moves into, and the pages moved away
      if (free) a.ring[max(0, h - moves) + max(0, m - (movers - moves))] = x;
      else end = max(end, x + 1);
    }
  end = __reduce_max_sync(0xffffffffu, end);
  if (lane == 0 && end) atomicMax(a.pages_end, end);
  const int parts = (a.max_blocks + kColumns - 1) / kColumns;
  const int64_t items = (int64_t)a.B * parts, stride = (int64_t)gridDim.x * (kPoolThreads / 32);
  for (int64_t i = blockIdx.x * (int64_t)(kPoolThreads / 32) + (threadIdx.x >> 5); i < items; i += stride) {
    const int b = (int)(i / parts), c0 = (int)(i % parts) * kColumns;
    const int held = err ? 0 : a.held[b];
#pragma unroll
    for (int k = 0; k < kColumns / 32; ++k) {
      const int c = c0 + k * 32 + lane;
      if (c >= a.max_blocks) break;
      const int x = a.table[(int64_t)b * a.max_blocks + c];
      a.table_out[(int64_t)b * a.max_blocks + c] = c < held ? moved(x) : x;
    }
  }
}

// ---- copies --------------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kPiece = 16384;   // bytes
constexpr int kCopyRound = 1024;  // entries of the list looked at together

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  __shared__ int2 list[kCopyRound];
  __shared__ int part[kCopyThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  for (int e0 = 0; e0 < a.n; e0 += kCopyRound) {
    int kept = 0;
    for (int i0 = 0; i0 < kCopyRound; i0 += kCopyThreads) {
      const int i = e0 + i0 + threadIdx.x;
      const int2 e = i < a.n && i < e0 + kCopyRound ? a.copies[i] : make_int2(-1, -1);
      const bool none = e.x == -1 && e.y == -1;
      const bool good = e.x >= 0 && e.x < a.num_blocks && e.y >= 0 && e.y < a.num_blocks;
      if (!none && !good && blockIdx.x == 0 && a.error) atomicOr(a.error, PA_DEVERR_BAD_BLOCK);
      const bool use = good && e.x != e.y;
      const unsigned m = __ballot_sync(0xffffffffu, use);
      if (lane == 0) part[warp] = __popc(m);
      __syncthreads();
      int before = kept;
      for (int w = 0; w < kCopyThreads / 32; ++w) {
        if (w < warp) before += part[w];
        kept += part[w];
      }
      if (use) list[before + __popc(m & ((1u << lane) - 1))] = e;
      __syncthreads();
    }
    const int64_t units = (int64_t)kept * a.num_tensors * a.pieces;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
      const int piece = (int)(u % a.pieces);
      const int64_t v = u / a.pieces;
      const int t = (int)(v % a.num_tensors);
      const int2 e = list[v / a.num_tensors];
      const int64_t bytes = a.bytes[t];
      const int64_t off = (int64_t)piece * kPiece;
      const uint8_t* src = a.data[t] + e.x * bytes + off;
      uint8_t* dst = a.data[t] + e.y * bytes + off;
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
    __syncthreads();
  }
}

// ---- host ----------------------------------------------------------------------------------
static int grid_of(int64_t work, int sms, int per_sm) {
  const int64_t g = ceil_div(work, kPoolThreads);
  return (int)(g < 1 ? 1 : g > (int64_t)sms * per_sm ? (int64_t)sms * per_sm : g);
}

// (at most PA_MAX_TABLE_REQUESTS rows and PA_MAX_POOL_PAGES / 1024 chunks)
constexpr int kMarkSmem = PA_MAX_TABLE_REQUESTS * 4;
constexpr int kFinishSmem = 8 * (PA_MAX_POOL_PAGES / kChunk + 1) + PA_MAX_TABLE_REQUESTS * 4;
static_assert(kMarkSmem <= 48 * 1024 && kFinishSmem <= 48 * 1024 - 256, "no attribute is needed");

template <bool FORK>
static cudaError_t launch_pool(const PoolArgs& a, int sms, cudaStream_t s) {
  const dim3 block(kPoolThreads);
  if (cudaError_t e = launch_pdl(pool_clear_kernel, dim3(grid_of(a.clear_words, sms, 4)), block, 0, s, a.clear, a.clear_words)) return e;
  const int64_t parts = ceil_div(a.max_blocks, kColumns) * 32;
  if (cudaError_t e = launch_pdl(pool_mark_kernel<FORK>, dim3(grid_of(a.B * parts, sms, 4)), block,
                                 FORK ? (size_t)a.B * 4 : 0, s, a))
    return e;
  if (cudaError_t e = launch_pdl(pool_words_kernel<FORK>, dim3(a.num_chunks), block, 0, s, a)) return e;
  const int64_t rows = FORK ? a.Bn : a.B, work = rows * parts > a.num_blocks ? rows * parts : a.num_blocks;
  if constexpr (FORK)
    return launch_pdl(fork_finish_kernel, dim3(grid_of(work, sms, 4)), block,
                      8 * ((size_t)a.num_chunks + 1) + (size_t)a.Bn * 4, s, a);
  else
    return launch_pdl(compact_finish_kernel, dim3(grid_of(work, sms, 4)), block, 8 * ((size_t)a.num_chunks + 1), s, a);
}
cudaError_t launch_fork(const PoolArgs& a, int sms, cudaStream_t s) { return launch_pool<true>(a, sms, s); }
cudaError_t launch_compact(const PoolArgs& a, int sms, cudaStream_t s) { return launch_pool<false>(a, sms, s); }

cudaError_t launch_copy_pages(CopyArgs& a, int sms, cudaStream_t s) {
  int64_t most = 0;
  for (int t = 0; t < a.num_tensors; ++t) most = a.bytes[t] > most ? a.bytes[t] : most;
  a.pieces = (int)ceil_div(most, kPiece);
  const int64_t units = (int64_t)a.n * a.num_tensors * a.pieces;
  const int64_t g = units < (int64_t)sms * 8 ? units : (int64_t)sms * 8;
  return launch_pdl(copy_pages_kernel, dim3((unsigned)g), dim3(kCopyThreads), 0, s, a);
}

}  // namespace pa
