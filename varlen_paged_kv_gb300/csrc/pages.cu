// Page bounds of a paged key cache, and the pages that a cheap score selects from them.
//
// Bounds. For every page, KV head g and channel c, the least and the largest code of the
// page's keys, code(x) = min(max(rint(x / s_gc), -127), 127) with a caller-given scale (the
// INT8 cache's code rule). The code never decreases with x, so the bounds are the codes of
// the keys' minimum and maximum: exact, whatever the order.
//
// Score. A block of R consecutive query rows of a sequence shares one selection per KV head.
// For one query row q, sum_c max(q_c lo_c, q_c hi_c) bounds q.k for every key k inside the
// page's bounds (in units of the scales); with q split by sign it is sum_c q+_c hi_c - q-_c
// lo_c, linear in (q+, q-), so the sum of the bounds over the block's R rows and the group's
// G heads is one product with the summed parts: the cost does not grow with R or G. The
// summed parts enter as 8-bit codes, so a score is a whole number below 2^24 and the
// selection is exact: the top_k pages by (score, lowest index), always with the first
// `sink` pages, the last `local` pages up to the block's first row, and the pages that hold
// the block's rows.
#include "ops.cuh"

namespace pa {

// ---- bounds --------------------------------------------------------------------------------

constexpr int kBoundChunks = 32;  // 16-byte chunks (8 channels) of a key row per CTA
constexpr int kBoundGroups = 8;   // keys read side by side

__device__ __forceinline__ int key_code(float x, float s) {
  return (int)fminf(fmaxf(rintf(__fdiv_rn(x, s)), -127.f), 127.f);
}

template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16) asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF16>
__device__ __forceinline__ float half_of(uint32_t w, int e) {
  const uint32_t b = (w >> (16 * e)) & 0xFFFFu;
  if constexpr (BF16) return __uint_as_float(b << 16);
  else return __half2float(__ushort_as_half((unsigned short)b));
}

// One CTA takes one touched page and 256 channels of it: eight groups of 32 threads read the
// page's new keys, eight keys side by side, 16 bytes a thread, and keep the running minimum
// and maximum in the keys' own type; the groups meet in shared memory and the first converts
// to codes, joining the page's old bounds when the page holds keys from before the call. Only
// the call's own rows are read. Bytes bound it on prompts (one read of the new keys); a decode
// step is a chain of dependent loads (lengths, table, key, bounds).
template <bool BF16>
__global__ void __launch_bounds__(kBoundChunks * kBoundGroups) bounds_kernel(const PageArgs a) {
  const int chunk_in = threadIdx.x % kBoundChunks, group = threadIdx.x / kBoundChunks, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_batch(a.cum, a.past, a.B, a.N, a.max_blocks, a.bs, a.error);
  const int u = blockIdx.x;
  const int b = find_seq(a.cum, a.B, a.bs, 2, u, lane);
  if (b < 0) return;
  const Seq s = load_seq(a.cum, a.past, b, a.N, a.max_blocks, a.bs);
  if (!s.ok || s.q == 0) return;
  const int page = s.past / a.bs + (u - (s.c0 / a.bs + 2 * b));
  const int end = s.past + s.q;
  if ((int64_t)page * a.bs >= end) return;
  const int phys = a.table[(int64_t)b * a.max_blocks + page];
  if (phys < 0 || phys >= a.num_blocks) {
    if (threadIdx.x == 0 && a.error) atomicOr(a.error, PA_DEVERR_BAD_BLOCK);
    return;
  }
  const int k0 = max(s.past - page * a.bs, 0), k1 = min(end - page * a.bs, a.bs);
  const int chunks = a.kvh * a.hs / 8, chunk = blockIdx.y * kBoundChunks + chunk_in;
  const bool on = chunk < chunks;
  const uint32_t inf = BF16 ? 0x7F807F80u : 0x7C007C00u;
  uint32_t lo[4] = {inf, inf, inf, inf}, hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) hi[i] = inf | 0x80008000u;
  if (on) {
    const uint4* src = reinterpret_cast<const uint4*>(a.key_cache + (int64_t)phys * a.bs * a.kvh * a.hs) + chunk;
#pragma unroll 8
    for (int k = k0 + group; k < k1; k += kBoundGroups) {
      const uint4 v = src[(int64_t)k * chunks];
      lo[0] = min2<BF16>(lo[0], v.x), hi[0] = max2<BF16>(hi[0], v.x);
      lo[1] = min2<BF16>(lo[1], v.y), hi[1] = max2<BF16>(hi[1], v.y);
      lo[2] = min2<BF16>(lo[2], v.z), hi[2] = max2<BF16>(hi[2], v.z);
      lo[3] = min2<BF16>(lo[3], v.w), hi[3] = max2<BF16>(hi[3], v.w);
    }
  }
  __shared__ uint32_t part[kBoundGroups][8][kBoundChunks];
#pragma unroll
  for (int i = 0; i < 4; ++i) part[group][i][chunk_in] = lo[i], part[group][4 + i][chunk_in] = hi[i];
  __syncthreads();
  if (group != 0 || !on) return;
  for (int o = 1; o < kBoundGroups; ++o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = min2<BF16>(lo[i], part[o][i][chunk_in]);
      hi[i] = max2<BF16>(hi[i], part[o][4 + i][chunk_in]);
    }
  }
  const int c = chunk * 8, g = c / a.hs;
  int8_t* dst = a.bounds + (((int64_t)phys * a.kvh + g) * 2) * a.hs + c % a.hs;
  const bool join = page * a.bs < s.past;  // the page held keys before this call
  uint2 old_lo = make_uint2(0, 0), old_hi = old_lo;
  if (join) old_lo = *reinterpret_cast<const uint2*>(dst), old_hi = *reinterpret_cast<const uint2*>(dst + a.hs);
  uint32_t out_lo[2] = {0, 0}, out_hi[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float sc = __ldg(a.scale + c + e);
    int x = key_code(half_of<BF16>(lo[e / 2], e & 1), sc), y = key_code(half_of<BF16>(hi[e / 2], e & 1), sc);
    if (join) {
      x = min(x, (int)(int8_t)((e < 4 ? old_lo.x : old_lo.y) >> (8 * (e & 3))));
      y = max(y, (int)(int8_t)((e < 4 ? old_hi.x : old_hi.y) >> (8 * (e & 3))));
    }
    out_lo[e / 4] |= (uint32_t)(x & 0xFF) << (8 * (e & 3));
    out_hi[e / 4] |= (uint32_t)(y & 0xFF) << (8 * (e & 3));
  }
  *reinterpret_cast<uint2*>(dst) = make_uint2(out_lo[0], out_lo[1]);
  *reinterpret_cast<uint2*>(dst + a.hs) = make_uint2(out_hi[0], out_hi[1]);
}

cudaError_t launch_bounds(const PageArgs& a, bool bf16, cudaStream_t s) {
  const int64_t units = (int64_t)a.N / a.bs + 2 * (int64_t)a.B;
  const dim3 grid((unsigned)units, (unsigned)ceil_div(a.kvh * a.hs / 8, kBoundChunks));
  if (bf16) bounds_kernel<true><<<grid, kBoundChunks * kBoundGroups, 0, s>>>(a);
  else bounds_kernel<false><<<grid, kBoundChunks * kBoundGroups, 0, s>>>(a);
  return cudaGetLastError();
}

// ---- selection -----------------------------------------------------------------------------

constexpr int kSelThreads = 256;

// unsigned bytes times signed bytes, added to c
__device__ __forceinline__ int dot4_us(uint32_t u, uint32_t s, int c) {
  int d;
  asm("dp4a.u32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(u), "r"(s), "r"(c));
  return d;
}

template <bool BF16>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const PageArgs a) {
  extern __shared__ int score[];  // [max_blocks]
  __shared__ uint32_t qcode[2][64];  // codes of the summed negative (0) and positive (1) parts
  __shared__ int red[kSelThreads / 32][2];
  __shared__ float redf[kSelThreads / 32];
  int* list = score + a.max_blocks;  // [top_k]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.y;
  if (blockIdx.x == 0 && g == 0) check_batch(a.cum, a.past, a.B, a.N, a.max_blocks, a.bs, a.error);
  const int u = blockIdx.x;
  const int b = find_seq(a.cum, a.B, a.R, a.R == 1 ? 0 : 1, u, lane);
  if (b < 0) return;
  const Seq s = load_seq(a.cum, a.past, b, a.N, a.max_blocks, a.bs);
  if (!s.ok) return;
  const int j0 = (u - (a.R == 1 ? s.c0 : s.c0 / a.R + b)) * a.R;
  if (j0 >= s.q || j0 < 0) return;
  const int rows = min(a.R, s.q - j0);
  const int own = (s.past + j0) / a.bs, last = (s.past + j0 + rows - 1) / a.bs;
  const int n = last + 1;                                    // pages of the block's history
  const int begin = min(a.sink, n);                          // pages [begin, end) compete
  const int end = max(begin, min(n, own - a.local + 1));
  const int want = a.top_k - (n - (end - begin));            // of which this many are taken
  int* out = a.selected + ((int64_t)(s.c0 + j0) * a.kvh + g) * a.top_k;
  const int64_t row_step = (int64_t)a.kvh * a.top_k;
  if (want >= end - begin) {  // every page
    for (int r = 0; r < rows; ++r)
      for (int i = tid; i < a.top_k; i += kSelThreads) out[r * row_step + i] = i < n ? i : -1;
    return;
  }
  // ---- the block's codes: 12-bit codes of every row in units of the block's largest value,
  // summed by sign, rescaled to 8 bits ----
  const uint16_t* q = a.query + (int64_t)(s.c0 + j0) * a.q_stride + (int64_t)g * a.G * a.hs;
  const int c = tid;  // (hs <= 256 = threads: thread c sums channel c)
  const float sc = c < a.hs ? a.scale[g * a.hs + c] : 0.f;
  auto value = [&](int r, int h) {
    const uint16_t bits = q[(int64_t)r * a.q_stride + h * a.hs + c];
    const float x = __fmul_rn(BF16 ? __uint_as_float((uint32_t)bits << 16) : __half2float(__ushort_as_half(bits)), sc);
    return isfinite(x) ? x : 0.f;
  };
  float most = 0.f;
  if (c < a.hs)
    for (int r = 0; r < rows; ++r)
      for (int h = 0; h < a.G; ++h) most = fmaxf(most, fabsf(value(r, h)));
  for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) redf[warp] = most;
  __syncthreads();
  for (int i = 0; i < kSelThreads / 32; ++i) most = fmaxf(most, redf[i]);
  const float fine = most > 1e-30f ? __fdiv_rn(4095.f, most) : 0.f;
  int plus = 0, minus = 0;
  if (c < a.hs)
    for (int r = 0; r < rows; ++r)
      for (int h = 0; h < a.G; ++h) {
        const int t = __float2int_rn(__fmul_rn(value(r, h), fine));
        plus += max(t, 0);
        minus += max(-t, 0);
      }
  int big = max(plus, minus);
  big = __reduce_max_sync(0xffffffffu, big);
  if (lane == 0) red[warp][0] = big;
  __syncthreads();
  for (int i = 0; i < kSelThreads / 32; ++i) big = max(big, red[i][0]);
  big = max(big, 1);
  if (c < a.hs) {
    // (510 * plus + big) / (2 big): 510 * 1024 rows * 4095 stays below 2^31
    reinterpret_cast<uint8_t*>(qcode[1])[c] = (uint8_t)((uint32_t)(510 * plus + big) / (uint32_t)(2 * big));
    reinterpret_cast<uint8_t*>(qcode[0])[c] = (uint8_t)((uint32_t)(510 * minus + big) / (uint32_t)(2 * big));
  }
  __syncthreads();
  // ---- scores ----
  const int words = a.hs / 4;
  for (int i = begin + tid; i < end; i += kSelThreads) {
    const int phys = a.table[(int64_t)b * a.max_blocks + i];
    int d = 0;
    if (phys >= 0 && phys < a.num_blocks) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(a.bounds + ((int64_t)phys * a.kvh + g) * 2 * a.hs);
      int neg = 0;
      for (int k = 0; k < words; ++k) {
        neg = dot4_us(qcode[0][k], p[k], neg);
        d = dot4_us(qcode[1][k], p[words + k], d);
      }
      d -= neg;
    } else if (a.error) {
      atomicOr(a.error, PA_DEVERR_BAD_BLOCK);
    }
    score[i] = d;
  }
  __syncthreads();
  // ---- the largest threshold that at least `want` scores reach, by bisection; each warp
  // counts its own contiguous part ----
  const int per = (int)align_up(ceil_div(end - begin, kSelThreads / 32), 32);
  const int i0 = min(end, begin + warp * per), i1 = min(end, i0 + per);
  int lo = -(1 << 24), hi = 1 << 24;  // count(score >= lo) >= want > count(score >= hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    int cnt = 0;
    for (int i = i0 + lane; i < i1; i += 32) cnt += score[i] >= mid;
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) red[warp][0] = cnt;
    __syncthreads();
    cnt = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) cnt += red[w][0];
    __syncthreads();
    if (cnt >= want) lo = mid;
    else hi = mid;
  }
  // ---- the taken pages in order: those above the threshold, and of those at it the first ----
  int above = 0, at = 0;
  for (int i = i0 + lane; i < i1; i += 32) above += score[i] > lo, at += score[i] == lo;
  above = __reduce_add_sync(0xffffffffu, above);
  at = __reduce_add_sync(0xffffffffu, at);
  if (lane == 0) red[warp][0] = above, red[warp][1] = at;
  __syncthreads();
  int all_above = 0, before_above = 0, before_at = 0;
  for (int w = 0; w < kSelThreads / 32; ++w) {
    if (w < warp) before_above += red[w][0], before_at += red[w][1];
    all_above += red[w][0];
  }
  const int ties = want - all_above;
  for (int i = i0; i < i1; i += 32) {
    const int x = i + lane < i1 ? score[i + lane] : INT32_MIN;
    const unsigned up = __ballot_sync(0xffffffffu, i + lane < i1 && x > lo);
    const unsigned eq = __ballot_sync(0xffffffffu, i + lane < i1 && x == lo);
    const unsigned below = (1u << lane) - 1;
    const int eq_rank = before_at + __popc(eq & below);
    if ((up >> lane & 1) || ((eq >> lane & 1) && eq_rank < ties))
      list[begin + before_above + __popc(up & below) + min(eq_rank, ties)] = i + lane;
    before_above += __popc(up);
    before_at += __popc(eq);
  }
  for (int i = tid; i < begin; i += kSelThreads) list[i] = i;
  for (int i = end + tid; i < n; i += kSelThreads) list[begin + want + i - end] = i;
  __syncthreads();
  for (int r = 0; r < rows; ++r)
    for (int i = tid; i < a.top_k; i += kSelThreads) out[r * row_step + i] = list[i];
}

cudaError_t launch_select(const PageArgs& a, bool bf16, int /*sms*/, cudaStream_t s) {
  const size_t smem = ((size_t)a.max_blocks + a.top_k) * 4;
  const dim3 grid((unsigned)query_blocks(a), (unsigned)a.kvh);
  auto kernel = bf16 ? select_kernel<true> : select_kernel<false>;
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) return e;
  kernel<<<grid, kSelThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace pa
