// Block tables and slot maps from the requests' lengths, with the pages taken from and
// returned to a ring of free pages on the GPU.
//
// Over the requests b = 0 .. B - 1, with need_b = ceil((past_b + q_b) / bs) for q_b > 0:
//   cum    exclusive prefix sums of the new rows max(q_b, 0);
//   grow   exclusive prefix sums of max(need_b - held_b, 0): request b's new columns
//          held_b .. need_b - 1 take the free pages head + grow_b .. of the ring, in order;
//   back   exclusive prefix sums of held_b over the finished requests (q_b = -1): their
//          pages go behind the ring's last free page, in order.
// Row i of request b is at position p = past_b + i - cum_b, in slot page(p / bs) * bs + p % bs.
//
// One kernel, no scratch memory and no communication between its CTAs: every CTA scans all B
// requests itself (12 bytes each, from L2) into shared memory, then writes its share of the
// rows, new table columns and returned pages, finding an entry's request by binary search in
// the scanned sums. Columns and ring entries that the call writes are read by none of its
// CTAs (a new column's page is read from the ring, and the ring has room behind its last
// free page for all returned ones), so no order between CTAs is needed. Latency, not bytes,
// bounds it (a call moves a few hundred KB at most): 64 decoding requests take 3.6 us, 1024
// requests with 28000 rows 6.8 us.
#include "ops.cuh"

namespace pa {

constexpr int kTableThreads = 512;
constexpr uint32_t kSumCap = 0x7fffffffu;

// adding with a ceiling keeps prefix sums ordered and associative whatever the lengths say
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSumCap); }

// the last i in [0, n) with sums[i] <= x, given sums[0] = 0 (entries with equal sums are empty)
__device__ __forceinline__ int last_at_most(const uint32_t* sums, int n, uint32_t x) {
  int lo = 0;
  while (n > 1) {
    const int half = n >> 1;
    if (sums[lo + half] <= x) lo += half, n -= half;
    else n = half;
  }
  return lo;
}

__global__ void __launch_bounds__(kTableThreads) tables_kernel(const TableArgs a) {
  extern __shared__ uint32_t sm[];
  uint32_t* cum = sm;                    // [B + 1] each
  uint32_t* grow = cum + a.B + 1;
  uint32_t* back = grow + a.B + 1;
  __shared__ uint32_t part[3][kTableThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  bool bad = false;
  pdl_wait();
  pdl_launch_dependents();
  uint32_t carry[3] = {0, 0, 0};
  for (int b0 = 0; b0 < a.B; b0 += kTableThreads) {
    const int b = b0 + tid;
    uint32_t v[3] = {0, 0, 0};
    if (b < a.B) {
      const int past = a.past[b], q = a.query_lens[b], held = a.held[b];
      const int64_t need = q > 0 ? ((int64_t)past + q + a.bs - 1) / a.bs : 0;
      if (past < 0 || q < -1 || held < 0 || held > a.max_blocks || need > a.max_blocks) {
        bad = true;
      } else {
        v[0] = max(q, 0);
        v[1] = max((int)need - held, 0);
        v[2] = q < 0 ? held : 0;
      }
    }
    uint32_t x[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      x[k] = v[k];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x[k], d);
        if (lane >= d) x[k] = sat_add(x[k], y);
      }
      if (lane == 31) part[k][warp] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint32_t before = carry[k], all = carry[k];
      for (int w = 0; w < kTableThreads / 32; ++w) {
        if (w < warp) before = sat_add(before, part[k][w]);
        all = sat_add(all, part[k][w]);
      }
      carry[k] = all;
      if (b < a.B) (k == 0 ? cum : k == 1 ? grow : back)[b + 1] = sat_add(before, x[k]);
    }
    __syncthreads();
  }
  if (tid == 0) cum[0] = grow[0] = back[0] = 0;
  const int head = a.state[0], count = a.state[1];
  uint32_t err = 0;
  if (__syncthreads_or(bad) || carry[0] > (uint32_t)a.N || head < 0 || head >= a.cap || count < 0 || count > a.cap ||
      (uint64_t)count + carry[2] > (uint64_t)a.cap)
    err = PA_DEVERR_BAD_BATCH;
  else if (carry[1] > (uint32_t)count)
    err = PA_DEVERR_NO_BLOCKS;
  // (unsigned: the step past the last of up to 2^31 - 2 rows must not turn negative)
  const uint32_t i0 = blockIdx.x * kTableThreads + tid, step = gridDim.x * kTableThreads;
  if (i0 == 0) {
    a.error[0] = err;
    a.cum[0] = 0;
    a.state_out[0] = err ? head : (int)(((int64_t)head + carry[1]) % a.cap);
    a.state_out[1] = err ? count : count - (int)carry[1] + (int)carry[2];
  }
  if (err) {  // refused: nothing changes, and the step has no rows
    for (uint32_t b = i0; b < (uint32_t)a.B; b += step) a.cum[b + 1] = 0, a.held_out[b] = a.held[b];
    for (uint32_t i = i0; i < (uint32_t)a.N; i += step) a.slots[i] = a.positions[i] = -1;
    return;
  }
  for (uint32_t b = i0; b < (uint32_t)a.B; b += step) {
    a.cum[b + 1] = (int)cum[b + 1];
    a.held_out[b] = a.query_lens[b] < 0 ? 0 : a.held[b] + (int)(grow[b + 1] - grow[b]);
  }
  // rows: consecutive threads have consecutive rows, mostly of one request
  const int max_page = (0x7fffffff - (a.bs - 1)) / a.bs;
  for (uint32_t i = i0; i < (uint32_t)a.N; i += step) {
    int slot = -1, pos = -1;
    if (i < carry[0]) {
      const int b = last_at_most(cum, a.B, i);
      pos = a.past[b] + (int)(i - cum[b]);
      const int col = pos / a.bs, held = a.held[b];
      const int page = col < held ? a.table[(int64_t)b * a.max_blocks + col]
                                  : a.ring[((int64_t)head + grow[b] + (col - held)) % a.cap];
      if (page >= 0 && page <= max_page) slot = page * a.bs + pos % a.bs;
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
  for (uint32_t k = i0; k < carry[1]; k += step) {  // new columns
    const int b = last_at_most(grow, a.B, k);
    a.table[(int64_t)b * a.max_blocks + a.held[b] + (int)(k - grow[b])] = a.ring[((int64_t)head + k) % a.cap];
  }
  for (uint32_t k = i0; k < carry[2]; k += step) {  // returned pages
    const int b = last_at_most(back, a.B, k);
    a.ring[((int64_t)head + count + k) % a.cap] = a.table[(int64_t)b * a.max_blocks + (int)(k - back[b])];
  }
}

cudaError_t launch_tables(const TableArgs& a, int sms, cudaStream_t s) {
  const int64_t smem = 3 * ((int64_t)a.B + 1) * 4;
  constexpr int most = 3 * (PA_MAX_TABLE_REQUESTS + 1) * 4;
  if (smem > 32 * 1024)  // (less needs no attribute; the same limit from every host thread)
    if (cudaError_t e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most)) return e;
  const int64_t work = a.N > a.B ? a.N : a.B;
  int64_t grid = ceil_div(work, kTableThreads);
  grid = grid < 1 ? 1 : grid > sms ? sms : grid;
  return launch_pdl(tables_kernel, dim3((unsigned)grid), dim3(kTableThreads), (size_t)smem, s, a);
}

}  // namespace pa
