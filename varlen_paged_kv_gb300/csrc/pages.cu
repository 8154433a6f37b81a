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
// summed parts enter as 8-bit codes, so a score is a whole number below 2^24 (an estimate of
// that bound: codes are rounded to the nearest and clipped, not outward) and the selection is exact: the top_k pages by (score, lowest index), always with the first
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
// the call's own rows are read. A decode step is a chain of dependent loads (lengths, table,
// key, bounds): 3.8 us for 64 rows of 8 heads of 128; prompts add one round of loads that are
// all in flight at once: 5.0 us for 4 prompts of 2048 (16.8 MB, 2.5 us at HBM's rate).
template <bool BF16>
__global__ void __launch_bounds__(kBoundChunks * kBoundGroups) bounds_kernel(const PageArgs a) {
  const int chunk_in = threadIdx.x % kBoundChunks, group = threadIdx.x / kBoundChunks, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0) check_batch(a.cum, a.past, a.B, a.N, a.max_blocks, a.bs, a.error);
  const int u = blockIdx.x;
  const Seq s = find_seq(a.cum, a.past, a.B, a.bs, 2, u, a.N, a.max_blocks, a.bs, lane);
  if (!s.ok || s.q == 0) return;
  const int page = s.past / a.bs + (u - (s.c0 / a.bs + 2 * s.b));
  const int end = s.past + s.q;
  if ((int64_t)page * a.bs >= end) return;
  const int phys = a.table[(int64_t)s.b * a.max_blocks + page];
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
  return launch_pdl(bf16 ? bounds_kernel<true> : bounds_kernel<false>, grid, dim3(kBoundChunks * kBoundGroups), 0, s, a);
}

// ---- selection -----------------------------------------------------------------------------

constexpr int kSelLoads = 8;     // 16-byte loads in flight per lane while scoring
constexpr int kSelBins = 2048;   // of the histograms that find the threshold

// unsigned bytes times signed bytes, added to c
__device__ __forceinline__ int dot4_us(uint32_t u, uint32_t s, int c) {
  int d;
  asm("dp4a.u32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(u), "r"(s), "r"(c));
  return d;
}

// what a select CTA holds beside its scores and list
template <int HS, int T>
struct SelShared {
  static constexpr int kWarps = T / 32;
  static constexpr int kSums = kWarps * 2 * HS > kSelBins ? kWarps * 2 * HS : kSelBins;
  __align__(16) uint8_t code[2][256];  // 8-bit codes: negative (0), positive (1) parts
  union {
    int hist[kSums];
    __align__(16) float sums[kWarps][2][HS];  // a warp's sums of t and of |t| per channel
  };
  int warp_a[kWarps], warp_b[kWarps];
  float warp_f[kWarps];
  int found[3];
  int n_close, close[32];  // the distances left when few are
};

template <bool BF16>
__device__ __forceinline__ uint64_t f2_unpack(uint32_t w) {
  return f2_make(half_of<BF16>(w, 0), half_of<BF16>(w, 1));
}

// The block's codes into sh.code: 12-bit codes t of every row in units of the block's largest
// product, summed by sign, rescaled to 8 bits. A thread holds up to HOLD 16-byte pieces of
// the rows in registers between finding the largest value and rounding by it, so that up to
// HOLD * T / (HS / 8) rows are read from memory once (more are read twice). On prompts its
// instructions are most of the kernel's (issue slots 59% busy, the rest mostly waits for those
// rows), so it runs on packed pairs: rounding to a whole number is adding and taking off 1.5 * 2^23, and the sums by sign come from those of t and |t| (whole numbers below 2^23,
// so exact in fp32). Products that are not finite are left out in a second form of the
// same steps.
template <int HS, bool BF16, int T>
__device__ void query_codes(const PageArgs& a, int row0, int rows, int g, SelShared<HS, T>& sh) {
  constexpr int CH = HS / 8, GROUPS = T / CH, HOLD = T == 256 ? 8 : 4, WARPS = T / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = tid % CH * 8, group = tid / CH, total = rows * a.G;
  const uint16_t* q = a.query + (int64_t)row0 * a.q_stride + (int64_t)g * a.G * HS + c;
  uint64_t sc[4];
  if (reinterpret_cast<uintptr_t>(a.scale) % 16 == 0) {
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(a.scale + g * HS + c));
    const float4 s1 = __ldg(reinterpret_cast<const float4*>(a.scale + g * HS + c) + 1);
    sc[0] = f2_make(s0.x, s0.y), sc[1] = f2_make(s0.z, s0.w), sc[2] = f2_make(s1.x, s1.y), sc[3] = f2_make(s1.z, s1.w);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      sc[e] = f2_make(__ldg(a.scale + g * HS + c + 2 * e), __ldg(a.scale + g * HS + c + 2 * e + 1));
  }
  auto load = [&](int r) {
    return __ldg(reinterpret_cast<const uint4*>(q + (int64_t)(r / a.G) * a.q_stride + (int64_t)(r % a.G) * HS));
  };
  uint4 held[HOLD];
#pragma unroll
  for (int k = 0; k < HOLD; ++k)
    held[k] = group + k * GROUPS < total ? load(group + k * GROUPS) : make_uint4(0, 0, 0, 0);
  // Per channel the largest |q| first, on the 16-bit patterns (their order is that of the values):
  // the scale is positive and rounding keeps the order, so its product is the largest product.
  // A channel that reaches infinity or NaN, or whose product does, takes the exact way.
  uint32_t widest16[4] = {0, 0, 0, 0};
  float most = 0.f;
  auto widest = [&](const uint4& v, bool filter) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!filter) {
        widest16[e] = max_u16x2(widest16[e], w[e] & 0x7FFF7FFFu);
      } else {
        float x0, x1;
        f2_split(f2_mul(f2_unpack<BF16>(w[e]), sc[e]), x0, x1);
        most = fmax3(most, isfinite(x0) ? fabsf(x0) : 0.f, isfinite(x1) ? fabsf(x1) : 0.f);
      }
    }
  };
  auto every = [&](auto&& f) {  // the thread's pieces
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
      if (k * GROUPS < total) f(held[k]);  // (a decode step has pieces for the first only)
    for (int r = group + HOLD * GROUPS; r < total; r += GROUPS) f(load(r));
  };
  every([&](const uint4& v) { widest(v, false); });
  bool odd = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float x0, x1;
    f2_split(f2_mul(f2_unpack<BF16>(widest16[e]), sc[e]), x0, x1);
    odd |= !isfinite(x0) || !isfinite(x1);
    most = fmax3(most, fabsf(x0), fabsf(x1));
  }
  const bool filter = __syncthreads_or(odd);
  if (filter) {
    most = 0.f;
    every([&](const uint4& v) { widest(v, true); });
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) sh.warp_f[warp] = most;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WARPS; ++i) most = fmaxf(most, sh.warp_f[i]);
  const float fine = most > 1e-30f ? __fdiv_rn(4095.f, most) : 0.f;
  const uint64_t fine2 = f2_make(fine, fine);
  constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: adding it leaves a whole number
  uint64_t sum[4];
  float mag[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = f2_make(0.f, 0.f), mag[2 * e] = mag[2 * e + 1] = 0.f;
  auto add = [&](const uint4& v, bool filter) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint64_t x2 = f2_mul(f2_unpack<BF16>(w[e]), sc[e]);
      float x0, x1;
      if (filter) {
        f2_split(x2, x0, x1);
        x2 = f2_make(isfinite(x0) ? x0 : 0.f, isfinite(x1) ? x1 : 0.f);
      }
      // (scalar sums: a product and a sum on packed pairs may become one fma, which rounds once)
      f2_split(f2_mul(x2, fine2), x0, x1);
      x0 = __fadd_rn(__fadd_rn(x0, kWhole), -kWhole);
      x1 = __fadd_rn(__fadd_rn(x1, kWhole), -kWhole);
      sum[e] = f2_add(sum[e], f2_make(x0, x1));
      mag[2 * e] += fabsf(x0);
      mag[2 * e + 1] += fabsf(x1);
    }
  };
  if (!filter) every([&](const uint4& v) { add(v, false); });
  else every([&](const uint4& v) { add(v, true); });
  float tot[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) f2_split(sum[e], tot[2 * e], tot[2 * e + 1]);
#pragma unroll
  for (int o = CH; o < 32; o <<= 1)  // (lanes CH apart hold the same channels)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      tot[e] += __shfl_xor_sync(0xffffffffu, tot[e], o);
      mag[e] += __shfl_xor_sync(0xffffffffu, mag[e], o);
    }
  if (lane < CH) {
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      *reinterpret_cast<float4*>(&sh.sums[warp][0][c + e]) = make_float4(tot[e], tot[e + 1], tot[e + 2], tot[e + 3]);
      *reinterpret_cast<float4*>(&sh.sums[warp][1][c + e]) = make_float4(mag[e], mag[e + 1], mag[e + 2], mag[e + 3]);
    }
  }
  __syncthreads();
  constexpr int MINE = (HS + T - 1) / T;  // channels of a thread
  int plus[MINE], minus[MINE], big = 0;
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    float t = 0.f, m = 0.f;
    if (tid + i * T < HS) {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) t += sh.sums[w][0][tid + i * T], m += sh.sums[w][1][tid + i * T];
    }
    plus[i] = (int)((m + t) * 0.5f), minus[i] = (int)((m - t) * 0.5f);
    big = max(big, max(plus[i], minus[i]));
  }
  big = __reduce_max_sync(0xffffffffu, big);
  if (lane == 0) sh.warp_a[warp] = big;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WARPS; ++i) big = max(big, sh.warp_a[i]);
  big = max(big, 1);
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    if (tid + i * T >= HS) break;
    // (510 plus + big) / (2 big): 510 * 1024 rows * 4095 stays below 2^31
    sh.code[1][tid + i * T] = (uint8_t)((uint32_t)(510 * plus[i] + big) / (uint32_t)(2 * big));
    sh.code[0][tid + i * T] = (uint8_t)((uint32_t)(510 * minus[i] + big) / (uint32_t)(2 * big));
  }
  __syncthreads();
}

// Scores of pages [i0, i1) of a history into `put(page, score)`. A page's 2 * HS bytes are CH
// 16-byte pieces: a lane keeps the query codes of its own piece in registers and takes it from
// kSelLoads * 32 / CH pages at once; the pieces' sums meet by a transposing reduction, so that
// every lane ends with one page's score (or shares one).
template <int HS, int T, typename Put>
__device__ void score_pages(const PageArgs& a, const int* table, int g, int i0, int i1, const SelShared<HS, T>& sh, Put put) {
  constexpr int CH = HS / 8;             // pieces of a page: half minimum, half maximum codes
  constexpr int PER = 32 / CH;           // pages per load of the warp
  constexpr int BATCH = kSelLoads * PER;  // pages per step
  constexpr int WARPS = T / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int piece = lane % CH, sub = lane / CH;
  const bool upper = piece >= CH / 2;
  const uint4 q = *reinterpret_cast<const uint4*>(sh.code[upper ? 1 : 0] + piece % (CH / 2) * 16);
  const int8_t* base = a.bounds + (int64_t)g * 2 * HS + piece * 16;
  const int64_t page_bytes = (int64_t)a.kvh * 2 * HS;
  bool bad = false;
  auto entry = [&](int i) { return lane < BATCH && i + lane < i1 ? __ldg(table + i + lane) : -1; };
  int next = entry(i0 + warp * BATCH);
  for (int i = i0 + warp * BATCH; i < i1; i += WARPS * BATCH) {
    const int phys = next < a.num_blocks ? next : -1;
    next = entry(i + WARPS * BATCH);  // a step ahead
    bad |= phys < 0 && lane < BATCH && i + lane < i1;
    uint4 v[kSelLoads];
#pragma unroll
    for (int k = 0; k < kSelLoads; ++k) {
      const int p = __shfl_sync(0xffffffffu, phys, k * PER + sub);
      v[k] = p >= 0 ? __ldg(reinterpret_cast<const uint4*>(base + p * page_bytes)) : make_uint4(0, 0, 0, 0);
    }
    int d[kSelLoads];
#pragma unroll
    for (int k = 0; k < kSelLoads; ++k) {
      const int x = dot4_us(q.x, v[k].x, dot4_us(q.y, v[k].y, dot4_us(q.z, v[k].z, dot4_us(q.w, v[k].w, 0))));
      d[k] = upper ? x : -x;
    }
    // halve the values a lane holds while summing over the pieces: after the step of bit o
    // the lanes with that bit set keep the upper half
    int first = 0;
#pragma unroll
    for (int o = CH / 2, n = kSelLoads; o >= 1; o >>= 1) {
      if (n > 1) {
        n >>= 1;
        const bool hi = lane & o;
#pragma unroll
        for (int k = 0; k < n; ++k) {
          const int send = hi ? d[k] : d[k + n], keep = hi ? d[k + n] : d[k];
          d[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
        first += hi ? n : 0;
      } else {
        d[0] += __shfl_xor_sync(0xffffffffu, d[0], o);
      }
    }
    // lanes that differ in the bits left over hold the same
    constexpr int SAME = CH > kSelLoads ? CH / kSelLoads : 1;
    if (lane % SAME == 0) {
#pragma unroll
      for (int k = 0; k < (CH < kSelLoads ? kSelLoads / CH : 1); ++k) {
        const int page = i + (first + k) * PER + sub;
        if (page < i1) put(page, d[k]);
      }
    }
  }
  if (bad && a.error) atomicOr(a.error, PA_DEVERR_BAD_BLOCK);
}

// The CTAs of a cluster score a share of the pages each into the first one's shared memory,
// which then finds the want-th best score and writes the list: the largest score first, a
// histogram of the distances from it in 2048 bins, then the bin that the want-th falls in: at
// most 32 scores are ranked directly, more go through further histograms. Bytes bound the
// scoring of long histories (2 HS bytes a page and head: 8 rows with up to 8192 pages read 84 MB
// and take 30 us, of which the scores 16); short ones are a chain of latencies (64 rows with up
// to 65 pages 8.1 us); prompts wait in turn for the query rows, which are read twice, and for the
// arithmetic on them (4 prompts of 2048 in blocks of 32: 59 us; DRAM 15%, issue slots 59% busy).
template <int HS, bool BF16, int T>
__global__ void __launch_bounds__(T, T == 256 ? 3 : 1024 / T) select_kernel(const PageArgs a) {
  constexpr int WARPS = T / 32;
  extern __shared__ int score[];  // [max_blocks], then the list [top_k]
  __shared__ SelShared<HS, T> sh;
  int* list = score + a.max_blocks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.y, rank = blockIdx.z, C = gridDim.z;
  pdl_wait();
  if (blockIdx.x == 0 && g == 0 && rank == 0) check_batch(a.cum, a.past, a.B, a.N, a.max_blocks, a.bs, a.error);
  const int u = blockIdx.x;
  if (a.R == 1) {  // (the row is known: its query heads are on their way while the lengths are looked up)
    const char* q = reinterpret_cast<const char*>(a.query + (int64_t)u * a.q_stride + (int64_t)g * a.G * HS);
    for (int i = tid * 128; i < a.G * HS * 2; i += T * 128) prefetch_l2(q + i);
  }
  const Seq s = find_seq(a.cum, a.past, a.B, a.R, a.R == 1 ? 0 : 1, u, a.N, a.max_blocks, a.bs, lane);
  if (!s.ok) return;
  const int j0 = (u - (a.R == 1 ? s.c0 : s.c0 / a.R + s.b)) * a.R;
  if (j0 >= s.q || j0 < 0) return;
  const int rows = min(a.R, s.q - j0);
  const int own = (s.past + j0) / a.bs, last = (s.past + j0 + rows - 1) / a.bs;
  const int n = last + 1;                                    // pages of the block's history
  const int begin = min(a.sink, n);                          // pages [begin, end) compete
  const int end = max(begin, min(n, own - a.local + 1));
  const int want = a.top_k - (n - (end - begin));            // of which this many are taken
  int* out = a.selected + ((int64_t)(s.c0 + j0) * a.kvh + g) * a.top_k;
  const int64_t row_step = (int64_t)a.kvh * a.top_k;
  if (want >= end - begin) {  // every page (all CTAs of a cluster agree)
    if (rank == 0)
      for (int i = tid; i < rows * a.top_k; i += T) {
        const int k = i % a.top_k;
        out[i / a.top_k * row_step + k] = k < n ? k : -1;
      }
    return;
  }
  query_codes<HS, BF16, T>(a, s.c0 + j0, rows, g, sh);
  const int* table = a.table + (int64_t)s.b * a.max_blocks;
  const int count = end - begin;
  if (C == 1) {
    score_pages<HS, T>(a, table, g, begin, end, sh, [&](int page, int d) { score[page - begin] = d; });
    __syncthreads();
  } else {
    cluster_sync();  // (the first CTA runs before it is written to)
    const uint32_t first = cluster_addr(score, 0);
    score_pages<HS, T>(a, table, g, begin + (int)((int64_t)count * rank / C), begin + (int)((int64_t)count * (rank + 1) / C),
                    sh, [&](int page, int d) {
                      asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(first + (uint32_t)(page - begin) * 4), "r"(d)
                                   : "memory");
                    });
    cluster_sync();
    if (rank != 0) return;
  }
  // ---- the threshold: scores above `cut` are taken, and the first `ties` of those at it ----
  int top = INT32_MIN, low = INT32_MAX;
  for (int i = tid; i < count; i += T) top = max(top, score[i]), low = min(low, score[i]);
  top = __reduce_max_sync(0xffffffffu, top);
  low = __reduce_min_sync(0xffffffffu, low);
  if (lane == 0) sh.warp_a[warp] = top, sh.warp_b[warp] = low;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) top = max(top, sh.warp_a[w]), low = min(low, sh.warp_b[w]);
  // distances top - score from `from` on, below `from + span`, in bins of 2^shift
  uint32_t from = 0, span = (uint32_t)(top - low) + 1;
  int ties = want;  // still to be taken among them
  constexpr int MINE = kSelBins / T;  // bins of a thread
  for (;;) {
    const int bits = 32 - __clz(span - 1 | 1), shift = max(bits - 11, 0);
#pragma unroll
    for (int k = 0; k < MINE; k += 4) *reinterpret_cast<int4*>(sh.hist + tid * MINE + k) = make_int4(0, 0, 0, 0);
    if (tid == 0) sh.n_close = 0;
    __syncthreads();
    for (int i = tid; i < count; i += T) {
      const uint32_t x = (uint32_t)(top - score[i]) - from;
      if (x < span) atomicAdd(&sh.hist[x >> shift], 1);
    }
    __syncthreads();
    int h[MINE], sum = 0;
#pragma unroll
    for (int k = 0; k < MINE; k += 4) {
      const int4 v = *reinterpret_cast<const int4*>(sh.hist + tid * MINE + k);
      h[k] = v.x, h[k + 1] = v.y, h[k + 2] = v.z, h[k + 3] = v.w;
      sum += (v.x + v.y) + (v.z + v.w);
    }
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) sh.warp_a[warp] = inc;
    __syncthreads();
    int before = inc - sum;
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
      if (w < warp) before += sh.warp_a[w];
    if (before < ties && ties <= before + sum) {  // the want-th falls in one of this thread's bins
#pragma unroll
      for (int k = 0; k < MINE; ++k) {
        if (before < ties && ties <= before + h[k]) {
          sh.found[0] = tid * MINE + k, sh.found[1] = ties - before, sh.found[2] = h[k];
        }
        before += h[k];
      }
    }
    if (ties == 0 && tid == 0) sh.found[0] = sh.found[1] = sh.found[2] = 0;  // (nothing to take: above all)
    __syncthreads();
    from += (uint32_t)sh.found[0] << shift;
    ties = sh.found[1];
    if (shift == 0 || ties == 0) break;
    span = min(span - ((uint32_t)sh.found[0] << shift), 1u << shift);
    if (span == 1) break;
    if (sh.found[2] <= 32) {
      // few are left: every warp ranks them by comparing each with each
      for (int i = tid; i < count; i += T) {
        const uint32_t x = (uint32_t)(top - score[i]) - from;
        if (x < span) sh.close[atomicAdd(&sh.n_close, 1)] = (int)x;
      }
      __syncthreads();
      const int left = sh.n_close, mine = lane < left ? sh.close[lane] : INT32_MAX;
      int rank = 0, fewer = 0;  // those before this one, and those strictly before
      for (int j = 0; j < left; ++j) {
        const int y = __shfl_sync(0xffffffffu, mine, j);
        fewer += y < mine;
        rank += y < mine || (y == mine && j < lane);
      }
      const unsigned m = __ballot_sync(0xffffffffu, lane < left && rank == ties - 1);
      const int at = __ffs(m) - 1;
      from += (uint32_t)__shfl_sync(0xffffffffu, mine, at);
      ties -= __shfl_sync(0xffffffffu, fewer, at);
      break;
    }
  }
  const int cut = top - (int)from;
  // ---- the taken pages in order, each warp a contiguous part: lane k keeps the masks of the
  // part's k-th 32 scores, the warps exchange their counts, and each lane writes its own ----
  const int per = (int)align_up(ceil_div(count, WARPS), 32);
  const int i0 = min(count, warp * per), i1 = min(count, i0 + per);
  int n_up = 0, n_eq = 0;  // of this warp
  constexpr int ROUNDS = 2;  // 2 * 32 * 32 scores a warp: 32768 by sixteen warps
  unsigned up[ROUNDS], eq[ROUNDS];
  int up_at[ROUNDS], eq_at[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    up[r] = eq[r] = 0;
    for (int k = 0; k < 32; ++k) {
      const int i = i0 + (r * 32 + k) * 32;
      if (i >= i1) break;
      const int x = i + lane < i1 ? score[i + lane] : INT32_MIN;
      const unsigned u1 = __ballot_sync(0xffffffffu, x > cut), e1 = __ballot_sync(0xffffffffu, x == cut);
      if (lane == k) up[r] = u1, eq[r] = e1;
    }
    int a1 = __popc(up[r]), e1 = __popc(eq[r]);
    const int a0 = a1, e0 = e1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, a1, d), z = __shfl_up_sync(0xffffffffu, e1, d);
      if (lane >= d) a1 += y, e1 += z;
    }
    up_at[r] = n_up + a1 - a0, eq_at[r] = n_eq + e1 - e0;
    n_up += __shfl_sync(0xffffffffu, a1, 31);
    n_eq += __shfl_sync(0xffffffffu, e1, 31);
  }
  __syncthreads();
  if (lane == 0) sh.warp_a[warp] = n_up, sh.warp_b[warp] = n_eq;
  __syncthreads();
  int before_up = 0, before_eq = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w)
    if (w < warp) before_up += sh.warp_a[w], before_eq += sh.warp_b[w];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    int above = before_up + up_at[r], equal = before_eq + eq_at[r];
    for (unsigned m = up[r] | eq[r]; m; m &= m - 1) {
      const int bit = __ffs(m) - 1;
      const bool is_eq = eq[r] >> bit & 1;
      if (!is_eq || equal < ties)
        list[begin + above + min(equal, ties)] = begin + i0 + (r * 32 + lane) * 32 + bit;
      if (is_eq) ++equal;
      else ++above;
    }
  }
  for (int i = tid; i < begin; i += T) list[i] = i;
  for (int i = end + tid; i < n; i += T) list[begin + want + i - end] = i;
  __syncthreads();
  for (int i = tid; i < rows * a.top_k; i += T) out[i / a.top_k * row_step + i % a.top_k] = list[i % a.top_k];
}

template <int HS, bool BF16>
static cudaError_t launch_select_t(const PageArgs& a, int sms, cudaStream_t s) {
  auto bytes = [](size_t columns, size_t top_k) { return (columns + top_k) * 4; };
  const size_t smem = bytes(a.max_blocks, a.top_k);
  const int64_t items = items_of_batch(a.N, a.B, a.R, 1, 1) * a.kvh;
  // CTAs that share the pages of a block: as many as run at once, each with a step of pages (at
  // most eight, the portable cluster; sixteen took 0.4 us more on one request of 2048 pages, and
  // twice as many as run at once 37 us instead of 30 on 8 long decode rows; 16 rows of 2048
  // pages in blocks of 16, counted as one block, 25 us instead of 16)
  const int c = cluster_size(items, 2 * (int64_t)sms, a.max_blocks, 128, 8);
  const dim3 grid((unsigned)query_blocks(a), (unsigned)a.kvh, (unsigned)c);
  // Threads by the longest history the table can hold. Short ones are chains of latencies that
  // more CTAs per SM overlap (tables of 544 pages, 4 prompts of 2048 rows: 58 us with 128
  // threads, 67 with 256, 86 with 512; 65 pages, 64 decode rows: 8.2, 11.0, 18.4 us), long ones
  // a stream of bounds and a last CTA's passes over the scores (8193 pages, 8 decode rows: 63,
  // 41, 33 us; 1025 pages, 32 drafts of 4: 18.4, 15.4, 16.1 us). The host knows the table's width,
  // not the histories: short ones in a wide table take the long ones' threads and shared memory (64 decode rows of
  // up to 65 pages: 8.1 us in 66 to 768 columns, 9.8 up to 4096, 16.9 in 8192, 23.4 in 32768), so
  // a table cut to the longest history of the step is worth its while.
  auto launch = [&](auto kernel, int threads, int columns) {
    return launch_clusters(kernel, grid, threads, smem, bytes(columns, PA_MAX_SELECTED_PAGES), s, a);
  };
  if (a.max_blocks <= 768) return launch(select_kernel<HS, BF16, 128>, 128, 768);
  if (a.max_blocks <= 4096) return launch(select_kernel<HS, BF16, 256>, 256, 4096);
  return launch(select_kernel<HS, BF16, 512>, 512, PA_MAX_SCORED_PAGES);
}

cudaError_t launch_select(const PageArgs& a, bool bf16, int sms, cudaStream_t s) {
#define PA_SELECT(HS) (bf16 ? launch_select_t<HS, true>(a, sms, s) : launch_select_t<HS, false>(a, sms, s))
  return a.hs == 64 ? PA_SELECT(64) : a.hs == 128 ? PA_SELECT(128) : PA_SELECT(256);
#undef PA_SELECT
}

}  // namespace pa
