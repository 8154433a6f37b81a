// Attention over the paged cache with capped scores, biases that grow with the distance, and a
// range of keys for every row.
//
// Row j of a sequence is at position p = past + j and sees the keys [lo, hi): lo the largest of 0,
// first_keys[row] and p - window + 1, hi the smaller of past + q and max(p + 1, prefix). Its score
// of key t for head h is s = scale q.k, then cap * tanh(s / cap), then - slope_h |p - t|; softmax
// and P V in fp32, rounded once to T. A row without keys gives zeros and an lse of -inf. Keys
// before the first and behind the last that a row of an item sees are not read, and pages between that no row sees (rows
// without keys among packed documents) are not reported, so neither need be there (a window's old pages).
//
// Two kernels, by the rows that share a KV head's keys:
//   biased_rows_kernel  sequences of up to 16 such rows (decode steps, short drafts): bound by the
//                       bytes of K and V; the work is cut into equal shares whatever the lengths,
//                       and biased_merge_kernel joins what a cut went through;
//   biased_tile_kernel  longer ones (prompts, wide groups): tcgen05, 128 rows against tiles of 64 keys.
#include "biased.cuh"

namespace pa {

constexpr int kBiThreads = 160;      // rows kernel: four consumer warps and a producer
constexpr int kBiCost = 3;           // what an item costs beside its tiles, in tiles
constexpr int kMergeThreads = 256;

// ---- few rows: equal shares of all tiles ----------------------------------------------------
// All (sequence, KV head, 16 rows) units stand in a row, each as long as its 64-key tiles and
// kBiCost; CTA c of C takes the c-th C-th of that. What a CTA has of a unit is an item: its
// tiles go through a ring of K and V tiles (TMA, one box per page segment, 128-byte swizzle);
// each of four consumer warps takes 16 keys of every tile (S = Q K^T by mma.sync, an online
// softmax in registers, O += P V, bf16 with P as two bf16 terms); the warps' (m, l, O) meet in
// shared memory. A whole unit is written out, a piece of one goes to one of the CTA's two slots
// (2c: its unit began with an earlier CTA; 2c + 1: it goes on with the next) and the merge
// kernel joins the slots in order. Every warp walks the units by itself.
template <int HS>
struct BiRows {
  static constexpr int kStages = 3;
  static constexpr int kTileBytes = kBiTile * HS * 2;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStride = HS + 4;                      // floats between rows of a partial result
  static constexpr int kComb = kStages * kStageBytes;         // float [16][kStride]
  static constexpr int kMl = kComb + 16 * kStride * 4;        // float [2][4][16]: m and l of the warps
  static constexpr int kCl = kMl + 2 * 4 * 16 * 4;            // float [2][16]: m and l of the CTA
  static constexpr int kPre = kCl + 2 * 16 * 4;               // int64 [kBiThreads + 1]: costs before each thread's sequences
  static constexpr int kBars = kPre + (kBiThreads + 2) * 8;
  static constexpr int kAbort = kBars + 2 * kStages * 8;      // abort flag, error word, rows to redo
  static constexpr int kBytes = kAbort + 16 + 1024;
};
static_assert(2 * (BiRows<128>::kBytes + 1024) <= 233472 && BiRows<256>::kBytes <= 232448, "rows kernel's shared memory");

struct BiItem {
  int b, c0, q, past, prefix;
  int r_first, n_rows, g;  // rows r = j * G + head of the sequence, from r_first
  int ta, te;              // tiles
  Keys keys;               // of all rows of the sequence
  bool first, last;        // the unit's first, last tiles
};

struct BiWalk {
  int64_t pos, end, base;  // the CTA's share; where sequence b begins
  int b, u;                // the next unit
  bool loaded;
  Seq s;
  Keys keys;
  int prefix, units, chunks, t0, nt;

  // by a whole warp: CTA c's share of all costs, `pre` the costs before each thread's run of sequences
  __device__ __forceinline__ void begin(const int64_t* pre, int run, int c, int ctas, int lane) {
    const int64_t W = pre[kBiThreads];
    const int C = (int)min((int64_t)ctas, max(W / (kBiCost + 1), (int64_t)1));
    pos = c < C ? W * c / C : W;
    end = c < C ? W * (c + 1) / C : W;
    loaded = false;
    int k = 0;  // the thread whose sequences hold the share's beginning
#pragma unroll
    for (int i = 0; i < kBiThreads / 32; ++i) k += __popc(__ballot_sync(0xffffffffu, pre[i * 32 + lane + 1] <= pos));
    k = min(k, kBiThreads - 1);
    b = k * run;
    base = pre[k];
  }
  // by a whole warp: the sequence's lengths and keys
  __device__ __forceinline__ void load(const BiasedArgs& a, int lane) {
    s = seq_at(a, b);
    units = 0;
    loaded = true;
    if (!short_rows(a, s)) return;
    prefix = a.prefix ? a.prefix[b] : 0;
    keys = {INT32_MAX, 0};
    if (a.first) {
      for (int j = lane; j < s.q; j += 32) keys = join(keys, keys_of_row(a, s, prefix, j));
      keys.lo = __reduce_min_sync(0xffffffffu, keys.lo);
      keys.hi = __reduce_max_sync(0xffffffffu, keys.hi);
    } else {
      keys = join(keys_of_row(a, s, prefix, 0), keys_of_row(a, s, prefix, s.q - 1));
    }
    const int2 t = tiles_of(keys);
    t0 = t.x;
    nt = t.y - t.x;
    chunks = (int)(((int64_t)s.q * a.G + 15) / 16);
    units = a.kvh * chunks;
  }
  // the rank-th of C equal shares of the sequence's tiles (`loaded` is taken back: the only item)
  __device__ __forceinline__ bool only(const BiasedArgs& a, int g, int rank, int C, BiItem& it) {
    if (!loaded) return false;
    loaded = false;
    it.b = b, it.c0 = s.c0, it.q = s.q, it.past = s.past, it.prefix = prefix;
    it.g = g;
    it.r_first = 0;
    it.n_rows = s.q * a.G;
    it.ta = t0 + (int)((int64_t)nt * rank / C), it.te = t0 + (int)((int64_t)nt * (rank + 1) / C);
    it.keys = keys;
    it.first = it.last = true;
    return true;
  }
  __device__ __forceinline__ bool next(const BiasedArgs& a, int lane, BiItem& it) {
    for (;;) {
      if (b >= a.B || base >= end) return false;
      if (!loaded) {
        load(a, lane);
        u = base < pos && units ? (int)((pos - base) / (nt + kBiCost)) : 0;
      }
      const int cost = nt + kBiCost;
      if (u >= units) {
        if (units) base += (int64_t)units * cost;
        ++b;
        loaded = false;
        continue;
      }
      const int64_t start = base + (int64_t)u * cost;
      if (start >= end) return false;
      const int unit = u++;
      int64_t x = 0, y = 0;
      if (nt == 0) {
        if (start < pos) continue;
      } else {
        x = max(max(pos, start) - start - kBiCost, (int64_t)0);
        y = max(min(end, start + cost) - start - kBiCost, (int64_t)0);
        if (y <= x) continue;
      }
      it.b = b, it.c0 = s.c0, it.q = s.q, it.past = s.past, it.prefix = prefix;
      it.g = unit / chunks;
      it.r_first = unit % chunks * 16;
      it.n_rows = min(16, s.q * a.G - it.r_first);
      it.ta = t0 + (int)x, it.te = t0 + (int)y;
      it.keys = keys;
      it.first = x == 0, it.last = y == nt;
      return true;
    }
  }
};

//
// CLUSTER: few units over short tables. The CTAs of a cluster (a column of the grid) share one unit's
// tiles, no costs are summed up and no merge follows: every CTA learns all (m, l) of the cluster and
// sums a share of the columns over it. One row of 2048 keys: 8.0 us where equal shares and a merge
// take 12.6; but a cluster's CTAs are at most eight, and a unit is not cut between clusters.
template <int HS, bool BF16, bool CLUSTER>
__global__ void __launch_bounds__(kBiThreads, HS == 256 ? 1 : 2)
    biased_rows_kernel(const __grid_constant__ BiasedArgs a, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const int seg_rows) {
  using L = BiRows<HS>;
  constexpr int NKS = HS / 16, ND = HS / 8;
  constexpr float kLift = BF16 ? 1.f : 32768.f;  // of the weights on their way into P V
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  float* comb = reinterpret_cast<float*>(smem + L::kComb);
  float* ml = reinterpret_cast<float*>(smem + L::kMl);
  float* cl = reinterpret_cast<float*>(smem + L::kCl);
  int64_t* pre = reinterpret_cast<int64_t*>(smem + L::kPre);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* empty = full + L::kStages;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kAbort);
  uint32_t* err = reinterpret_cast<uint32_t*>(smem + L::kAbort + 4);
  uint32_t* redo = reinterpret_cast<uint32_t*>(smem + L::kAbort + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    *abort = 0;
    *err = 0;
    *redo = 0;
    fence_mbar_init();
  }
  // Beside the tile kernel, whose every CTA has waited for what came before and let this one start, there is
  // nothing to wait for but at the end, by one CTA for all: this kernel must not be over before that one, since
  // what comes next waits for this one only. What came before is complete then and has left its writes in L2; that
  // they are what the loads below see, which the wait says elsewhere, a fence says here (and the loads are plain
  // ones: none may take its value from a cache that is not coherent).
  if (a.after_tiles) acquire_earlier_kernels();
  else pdl_wait();
  pdl_launch_dependents();
  const int c = blockIdx.x, rank = blockIdx.z;
  const bool waits = a.after_tiles && c == 0 && rank == 0;
  BiWalk walk;
  if (c == 0 && rank == 0) check_biased_batch(a);
  if constexpr (CLUSTER) {
    __syncthreads();  // the barriers are there
    walk.b = c / a.kvh;
    walk.load(a, lane);
    if (walk.units == 0) {  // (all CTAs of a cluster agree)
      if (waits) pdl_wait();
      return;
    }
  } else {
    // the costs of all sequences, each thread those of a run of them
    const int run = (a.B + kBiThreads - 1) / kBiThreads;
    {
      int64_t mine = 0;
      for (int i = 0; i < run; ++i) {
        const int b = threadIdx.x * run + i;
        if (b >= a.B) break;
        const Seq s = seq_at(a, b);
        if (!short_rows(a, s)) continue;
        const int prefix = a.prefix ? a.prefix[b] : 0;
        Keys k = join(keys_of_row(a, s, prefix, 0), keys_of_row(a, s, prefix, s.q - 1));
        if (a.first)
          for (int j = 1; j < s.q - 1; ++j) k = join(k, keys_of_row(a, s, prefix, j));
        const int2 t = tiles_of(k);
        mine += (int64_t)a.kvh * (((int64_t)s.q * a.G + 15) / 16) * (t.y - t.x + kBiCost);
      }
      pre[threadIdx.x + 1] = mine;
    }
    __syncthreads();
    if (warp == 0) {  // sums, five threads' costs a lane
      int64_t v[kBiThreads / 32], sum = 0;
#pragma unroll
      for (int i = 0; i < kBiThreads / 32; ++i) sum += pre[lane * (kBiThreads / 32) + i + 1], v[i] = sum;
      int64_t x = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
#pragma unroll
      for (int i = 0; i < kBiThreads / 32; ++i) pre[lane * (kBiThreads / 32) + i + 1] = x - sum + v[i];
      if (lane == 0) pre[0] = 0;
    }
    __syncthreads();
    walk.begin(pre, run, c, gridDim.x, lane);
    if (walk.pos >= walk.end) {
      if (threadIdx.x == 0) a.records[2 * c] = make_int4(0, 0, 0, 0), a.records[2 * c + 1] = make_int4(0, 0, 0, 0);
      if (waits) pdl_wait();
      return;
    }
  }
  BiItem it;
  int n = 0;  // tiles so far

  if (warp == 4) {
    // ---- producer ----
    const int nseg = kBiTile / seg_rows, oob = a.num_blocks * a.bs;
    int4 head = make_int4(0, 0, 0, 0);
    int cont = 0, head_b = 0;
    while (CLUSTER ? walk.only(a, c % a.kvh, rank, gridDim.z, it) : walk.next(a, lane, it)) {
      if (it.first && !it.last) head = make_int4(it.n_rows, it.c0, it.r_first, it.g), head_b = it.b;
      if (!it.first) cont = it.last ? 2 : 1;
      const int* table = a.table + (int64_t)it.b * a.max_blocks;
      auto slot = [&](int t) {  // this lane's segment of tile t: its first cache row
        const int v = t * kBiTile + lane * seg_rows;
        if (lane >= nseg || t >= it.te || v >= it.keys.hi || v + seg_rows <= it.keys.lo) return oob;
        const int page = v / a.bs, phys = table[page];
        if (unlikely(phys < 0 || phys >= a.num_blocks)) {
          // (reported if a row of the item sees one of these keys: with up to 16 rows in all, the gaps between their
          // ranges are shorter than 16 keys, and of a wider group an item has two rows at most)
          Seq sq;
          sq.c0 = it.c0, sq.q = it.q, sq.past = it.past;
          auto sees = [&](int r) {
            const Keys k = keys_of_row(a, sq, it.prefix, r / a.G);
            return k.lo < v + seg_rows && k.hi > v;
          };
          if (CLUSTER || a.G <= 16 || sees(it.r_first) || sees(it.r_first + it.n_rows - 1)) atomicOr(err, PA_DEVERR_BAD_BLOCK);
          return oob;
        }
        return phys * a.bs + (v - page * a.bs);
      };
      int z = slot(it.ta);
      for (int t = it.ta; t < it.te; ++t, ++n) {
        const int s = n % L::kStages, z_next = slot(t + 1);
        if (lane == 0) {
          mbar_wait(&empty[s], ((n / L::kStages) & 1) ^ 1, abort, err);
          mbar_arrive_expect_tx(&full[s], L::kStageBytes);
        }
        __syncwarp();
        if (lane < nseg) {
          uint8_t* dst = smem + s * L::kStageBytes + lane * seg_rows * 128;
#pragma unroll
          for (int h = 0; h < HS / 64; ++h) {
            tma_load_3d(dst + h * kBiTile * 128, &tmK, &full[s], h * 64, it.g, z);
            tma_load_3d(dst + L::kTileBytes + h * kBiTile * 128, &tmV, &full[s], h * 64, it.g, z);
          }
        }
        __syncwarp();
        z = z_next;
      }
    }
    if (!CLUSTER && lane == 0) a.records[2 * c] = head, a.records[2 * c + 1] = make_int4(cont, head_b, 0, 0);
  } else {
    // ---- consumers: warp w has keys 16w .. 16w + 15 of every tile ----
    const int w = warp, tq = lane & 3, gq = lane >> 2;
    const int mi = lane >> 3, rr = lane & 7;
    while (CLUSTER ? walk.only(a, c % a.kvh, rank, gridDim.z, it) : walk.next(a, lane, it)) {
      Seq sq;
      sq.c0 = it.c0, sq.q = it.q, sq.past = it.past;
      uint32_t qa[NKS][4];  // Q as the A operand: rows gq and gq + 8
      Keys k[2];
      int pos[2];
      float slope[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = it.r_first + gq + 8 * i, rc = min(r, it.r_first + it.n_rows - 1);  // (padding rows borrow the last row's keys)
        const int j = rc / a.G, h = it.g * a.G + rc % a.G;
        const uint32_t* p = reinterpret_cast<const uint32_t*>(a.query + (int64_t)(it.c0 + j) * a.q_stride + (int64_t)h * HS + tq * 2);
#pragma unroll
        for (int ks = 0; ks < NKS; ++ks) {
          qa[ks][i] = rc == r ? p[ks * 8] : 0u;
          qa[ks][i + 2] = rc == r ? p[ks * 8 + 4] : 0u;
        }
        k[i] = keys_of_row(a, sq, it.prefix, j);
        pos[i] = it.past + j;
        slope[i] = a.slopes ? a.slopes[h] * 1.4426950408889634f : 0.f;
      }
      // keys that some row sees, and those that all see
      const int some_lo = __reduce_min_sync(0xffffffffu, min(k[0].lo, k[1].lo));
      const int some_hi = __reduce_max_sync(0xffffffffu, max(k[0].hi, k[1].hi));
      const int all_lo = __reduce_max_sync(0xffffffffu, max(k[0].lo, k[1].lo));
      const int all_hi = __reduce_min_sync(0xffffffffu, min(k[0].hi, k[1].hi));
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      float o[ND][4];
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
      for (int t = it.ta; t < it.te; ++t, ++n) {
        const int s = n % L::kStages;
        mbar_wait(&full[s], (n / L::kStages) & 1, abort, err);
        const uint32_t kb = smem_u32(smem + s * L::kStageBytes), vb = kb + L::kTileBytes;
        const int v0 = t * kBiTile + 16 * w;  // the warp's first key
        if (v0 < some_hi && v0 + 16 > some_lo) {
          float sa[2][4] = {}, sb[2][4] = {};  // keys 0-7 and 8-15; even and odd k-steps
          {
            const int key = 16 * w + (mi >> 1) * 8 + rr;
#pragma unroll
            for (int ks = 0; ks < NKS; ++ks) {
              const int cc = ks * 2 + (mi & 1);
              uint32_t b0, b1, b2, b3;
              ldsm_x4(kb + (cc >> 3) * (kBiTile * 128) + key * 128 + (((cc & 7) ^ (key & 7)) << 4), b0, b1, b2, b3);
              mma16816<BF16>((ks & 1) ? sb[0] : sa[0], qa[ks], b0, b1);
              mma16816<BF16>((ks & 1) ? sb[1] : sa[1], qa[ks], b2, b3);
            }
          }
          float x[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = sa[i][e] + sb[i][e];
          if (a.cap_log2 != 0.f) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[i][e] = a.cap_log2 * tanh_of(x[i][e] * a.scale_cap);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[i][e] *= a.scale_log2;
          }
          if (a.slopes) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int away = abs(pos[e >> 1] - (v0 + i * 8 + tq * 2 + (e & 1)));
                x[i][e] = fmaf(-slope[e >> 1], (float)away, x[i][e]);
              }
          }
          if (v0 < all_lo || v0 + 16 > all_hi) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int key = v0 + i * 8 + tq * 2 + (e & 1);
                if (key < k[e >> 1].lo || key >= k[e >> 1].hi) x[i][e] = -INFINITY;
              }
          }
          float mx0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
          float mx1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
#pragma unroll
          for (int d = 1; d < 4; d <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
          }
          const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
          const float ms0 = mn0 == -INFINITY ? 0.f : mn0, ms1 = mn1 == -INFINITY ? 0.f : mn1;  // (no key yet)
          const float al0 = fast_exp2(m0 - ms0), al1 = fast_exp2(m1 - ms1);
          m0 = mn0;
          m1 = mn1;
          float p[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            p[i][0] = fast_exp2(x[i][0] - ms0);
            p[i][1] = fast_exp2(x[i][1] - ms0);
            p[i][2] = fast_exp2(x[i][2] - ms1);
            p[i][3] = fast_exp2(x[i][3] - ms1);
          }
          l0 = l0 * al0 + ((p[0][0] + p[0][1]) + (p[1][0] + p[1][1]));
          l1 = l1 * al1 + ((p[0][2] + p[0][3]) + (p[1][2] + p[1][3]));
          // P as the A operand: fp16 rounds the weights once (2^-11, as the output is rounded), lifted
          // to at most 2^15 so that only those below 2^-29 of the largest are subnormal; bf16, whose
          // one rounding would be 2^-8, keeps them as two terms
          uint32_t ph[4], pl[4];
          if constexpr (BF16) {
            split_bf16x2(p[0][0], p[0][1], ph[0], pl[0]);
            split_bf16x2(p[0][2], p[0][3], ph[1], pl[1]);
            split_bf16x2(p[1][0], p[1][1], ph[2], pl[2]);
            split_bf16x2(p[1][2], p[1][3], ph[3], pl[3]);
          } else {
            ph[0] = pack2<false>(p[0][0] * kLift, p[0][1] * kLift);
            ph[1] = pack2<false>(p[0][2] * kLift, p[0][3] * kLift);
            ph[2] = pack2<false>(p[1][0] * kLift, p[1][1] * kLift);
            ph[3] = pack2<false>(p[1][2] * kLift, p[1][3] * kLift);
          }
          if (!__all_sync(0xffffffffu, al0 == 1.f && al1 == 1.f)) {
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d][0] *= al0, o[d][1] *= al0, o[d][2] *= al1, o[d][3] *= al1;
          }
          // keys that no row sees may be unwritten cache rows: their V is cleared, so that no NaN
          // meets a weight of 0
          const int key = 16 * w + (mi & 1) * 8 + rr;
          auto pv = [&](uint32_t mlo, uint32_t mhi) {
#pragma unroll
            for (int dp = 0; dp < ND / 2; ++dp) {
              const int cc = 2 * dp + (mi >> 1);
              uint32_t w0, w1, w2, w3;
              ldsm_x4_t(vb + (cc >> 3) * (kBiTile * 128) + key * 128 + (((cc & 7) ^ (key & 7)) << 4), w0, w1, w2, w3);
              w0 &= mlo, w2 &= mlo, w1 &= mhi, w3 &= mhi;
              mma16816<BF16>(o[2 * dp], ph, w0, w1);
              mma16816<BF16>(o[2 * dp + 1], ph, w2, w3);
              if constexpr (BF16) {
                mma16816<BF16>(o[2 * dp], pl, w0, w1);
                mma16816<BF16>(o[2 * dp + 1], pl, w2, w3);
              }
            }
          };
          if (v0 >= some_lo && v0 + 16 <= some_hi) {
            pv(0xffffffffu, 0xffffffffu);
          } else {
            auto keep = [&](int first_key) {  // the two keys of a register
              return (first_key >= some_lo && first_key < some_hi ? 0xFFFFu : 0u) |
                     (first_key + 1 >= some_lo && first_key + 1 < some_hi ? 0xFFFF0000u : 0u);
            };
            pv(keep(v0 + 2 * tq), keep(v0 + 8 + 2 * tq));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
      }
      // ---- the four warps' results of the item ----
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
      }
      // scores of NaN alone leave no maximum but a sum of NaN, which must not be taken for a row
      // without keys
      if (m0 == -INFINITY && l0 != l0) m0 = 0.f;
      if (m1 == -INFINITY && l1 != l1) m1 = 0.f;
      if (tq == 0) {
        ml[w * 16 + gq] = m0, ml[w * 16 + gq + 8] = m1;
        ml[64 + w * 16 + gq] = l0, ml[64 + w * 16 + gq + 8] = l1;
      }
      named_bar_sync(1, 128);
      float f[2];
      bool none[2];  // no keys (O may be anything); a factor that is 0 in 32 bits makes NaN of an infinity, which redo_row settles
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = gq + 8 * i;
        const float M = fmaxf(fmaxf(ml[r], ml[16 + r]), fmaxf(ml[32 + r], ml[48 + r]));
        const float m = i ? m1 : m0;
        none[i] = m == -INFINITY;
        f[i] = none[i] ? 0.f : fast_exp2(m - M) * (1.f / kLift);
      }
      // up to four rows: the warps' side by side; more: the warps in turn add into the same rows
      const bool side = it.n_rows <= 4;
      for (int turn = 0; turn < (side ? 1 : 4); ++turn) {
        if (side || turn == w) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = gq + 8 * i;
            if (r >= it.n_rows) continue;
            float* dst = comb + (side ? w * 4 + r : r) * L::kStride + tq * 2;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              float2 y = none[i] ? make_float2(0.f, 0.f) : make_float2(o[d][2 * i] * f[i], o[d][2 * i + 1] * f[i]);
              if (!side && turn > 0) {
                const float2 old = *reinterpret_cast<float2*>(dst + d * 8);
                y.x += old.x, y.y += old.y;
              }
              *reinterpret_cast<float2*>(dst + d * 8) = y;
            }
          }
        }
        named_bar_sync(1, 128);
      }
      const bool whole = it.first && it.last;
      const int slot = 2 * c + (it.first ? 1 : 0);
      for (int i = threadIdx.x; i < it.n_rows * (HS / 4); i += 128) {
        const int r = i / (HS / 4), cc = i % (HS / 4) * 4;
        float4 x = *reinterpret_cast<float4*>(comb + r * L::kStride + cc);
        if (side)
          for (int v = 1; v < 4; ++v) {
            const float4 y = *reinterpret_cast<float4*>(comb + (v * 4 + r) * L::kStride + cc);
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
          }
        const float M = fmaxf(fmaxf(ml[r], ml[16 + r]), fmaxf(ml[32 + r], ml[48 + r]));
        float S = 0.f;
        for (int v = 0; v < 4; ++v)
          if (ml[v * 16 + r] != -INFINITY) S += ml[64 + v * 16 + r] * fast_exp2(ml[v * 16 + r] - M);
        if constexpr (CLUSTER) {
          *reinterpret_cast<float4*>(comb + r * L::kStride + cc) = x;
          if (cc == 0) cl[r] = M, cl[16 + r] = S;
        } else if (whole) {
          const int rs = it.r_first + r;
          const int64_t at = (int64_t)(it.c0 + rs / a.G) * a.nh + it.g * a.G + rs % a.G;
          const float inv = M == -INFINITY ? 0.f : 1.f / S;
          uint2 out = make_uint2(pack_out<BF16>(x.x * inv, x.y * inv), pack_out<BF16>(x.z * inv, x.w * inv));
          if (M == -INFINITY) out = make_uint2(0, 0);
          else if (S == S && !finite4(x.x * inv, x.y * inv, x.z * inv, x.w * inv)) *redo = 1;
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.output) + at * HS + cc) = out;
          if (a.lse && cc == 0) a.lse[at] = M == -INFINITY ? -INFINITY : (M + fast_log2(S)) * 0.69314718055994531f;
        } else {
          *reinterpret_cast<float4*>(a.part_o + ((int64_t)slot * 16 + r) * HS + cc) = x;
          if (cc == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * 16 + r) * 2) = make_float2(M, S);
        }
      }
      named_bar_sync(1, 128);  // the combining buffers are free again
    }
  }
  if constexpr (CLUSTER) {
    const int C = gridDim.z;
    cluster_sync();  // all results of the cluster
    const int c0 = HS / 4 * rank / C, nc = HS / 4 * (rank + 1) / C - c0;  // this CTA's share of the columns, in quads
    for (int i = threadIdx.x; i < it.n_rows * nc; i += kBiThreads) {
      const int r = i / nc, cc = (c0 + i % nc) * 4;
      float M = -INFINITY, S = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < C; ++k) M = fmaxf(M, ld_cluster(cluster_addr(cl + r, k)));
      for (int k = 0; k < C; ++k) {
        const float m = ld_cluster(cluster_addr(cl + r, k));
        if (m == -INFINITY) continue;
        const float f = fast_exp2(m - M);
        S += f * ld_cluster(cluster_addr(cl + 16 + r, k));
        const float4 y = ld_cluster4(cluster_addr(comb + r * L::kStride + cc, k));
        x[0] += f * y.x, x[1] += f * y.y, x[2] += f * y.z, x[3] += f * y.w;
      }
      const int64_t at = (int64_t)(it.c0 + r / a.G) * a.nh + it.g * a.G + r % a.G;
      const float inv = M == -INFINITY ? 0.f : 1.f / S;
      uint2 out = make_uint2(pack_out<BF16>(x[0] * inv, x[1] * inv), pack_out<BF16>(x[2] * inv, x[3] * inv));
      if (M == -INFINITY) out = make_uint2(0, 0);
      else if (S == S && !finite4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv)) atomicOr(redo, 1u << r);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.output) + at * HS + cc) = out;
      if (a.lse && cc == 0) a.lse[at] = M == -INFINITY ? -INFINITY : (M + fast_log2(S)) * 0.69314718055994531f;
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
    for (int r = warp; *redo && r < it.n_rows; r += kBiThreads / 32)  // (this CTA's columns)
      if (*redo >> r & 1)
        redo_row<HS, BF16>(a, it.b, it.c0, it.q, it.past, r / a.G, it.g * a.G + r % a.G, lane, c0 * 4, (c0 + nc) * 4);
  }
  __syncthreads();
  if (threadIdx.x == 0 && *err && a.error) atomicOr(a.error, *err);
  if constexpr (!CLUSTER) {
    // Rows of whole units that are not finite, as they stand in the output: after the last item, when no
    // warp waits for another any more, since a row of many keys may take longer than a wait's limit.
    if (*redo) {
      walk.begin(pre, (a.B + kBiThreads - 1) / kBiThreads, c, gridDim.x, lane);
      while (walk.next(a, lane, it)) {
        if (!it.first || !it.last) continue;
        for (int r = it.r_first + warp; r < it.r_first + it.n_rows; r += kBiThreads / 32) {
          const int j = r / a.G, h = it.g * a.G + r % a.G;
          const uint16_t* out = static_cast<const uint16_t*>(a.output) + ((int64_t)(it.c0 + j) * a.nh + h) * HS;
          constexpr uint32_t top = BF16 ? 0x7F80u : 0x7C00u;
          bool fine = true;
          for (int e = lane; e < HS; e += 32) fine = fine && (out[e] & top) != top;
          if (!__all_sync(0xffffffffu, fine))
            redo_row<HS, BF16>(a, it.b, it.c0, it.q, it.past, j, h, lane, 0, HS);
        }
      }
    }
  }
  if (waits) pdl_wait();
}

// The pieces of the units that the cuts between CTAs went through, in order: CTA c of the rows
// kernel began such a unit (record 2c), its next ones went on with it (record 2k + 1: 1, and 2 for
// the last; its second number is the sequence of the unit that record 2k begins). A lane has four columns of a row,
// eight warps share the pieces: what bounds it is latency, of its launch and of two loads, one after the other (the
// records, the pieces): 2.6 us behind one row of 200 keys, 3.7 behind 8 of 8000.
// (Four CTAs to an SM: with the registers that redo_row would take, two, 64 decode rows 120.5 us instead of 117.5.)
template <int HS, bool BF16>
__global__ void __launch_bounds__(kMergeThreads, 4) biased_merge_kernel(const __grid_constant__ BiasedArgs a, const int ctas) {
  constexpr int WARPS = kMergeThreads / 32;
  __shared__ float part[WARPS][6][32];
  pdl_wait();
  pdl_launch_dependents();
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 head = a.records[2 * c];
  auto record = [&](int k) { return k + lane < ctas ? a.records[2 * (k + lane) + 1].x : 0; };
  int rec = record(c + 1);  // (loaded beside the head)
  if (head.x == 0) return;
  int pieces = 1;
  for (int k = c + 1;; k += 32, rec = record(k)) {
    const unsigned end = __ballot_sync(0xffffffffu, rec != 1);
    const int n = end ? __ffs(end) - 1 : 32;
    pieces += n;
    if (end) {
      pieces += __shfl_sync(0xffffffffu, rec, n) == 2;
      break;
    }
  }
  unsigned again = 0;  // a bit for each row
  for (int i = blockIdx.y * 32 + lane; i - lane < head.x * (HS / 4); i += gridDim.y * 32) {
    const int r = min(i / (HS / 4), head.x - 1), cc = i % (HS / 4) * 4;
    float M = -INFINITY, S = 0.f;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](float m_in, float s_in, float4 y) {
      if (m_in == -INFINITY) return;
      const float m = fmaxf(M, m_in), f = fast_exp2(M - m), g = fast_exp2(m_in - m);  // (0 on the first piece with keys)
      M = m;
      S = S * f + s_in * g;
      x[0] = x[0] * f + y.x * g, x[1] = x[1] * f + y.y * g, x[2] = x[2] * f + y.z * g, x[3] = x[3] * f + y.w * g;
    };
#pragma unroll 4
    for (int p = warp; p < pieces; p += WARPS) {
      const int slot = p ? 2 * (c + p) : 2 * c + 1;
      const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (slot * 16 + r) * 2);
      add(ml.x, ml.y, *reinterpret_cast<const float4*>(a.part_o + ((int64_t)slot * 16 + r) * HS + cc));
    }
    __syncthreads();  // (the round before has been read)
    part[warp][0][lane] = M, part[warp][1][lane] = S;
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][2 + e][lane] = x[e];
    __syncthreads();
    if (warp != 0) continue;
#pragma unroll
    for (int w = 1; w < WARPS; ++w)
      add(part[w][0][lane], part[w][1][lane],
          make_float4(part[w][2][lane], part[w][3][lane], part[w][4][lane], part[w][5][lane]));
    const int rs = head.z + r;
    const int64_t at = (int64_t)(head.y + rs / a.G) * a.nh + head.w * a.G + rs % a.G;
    const float inv = M == -INFINITY ? 0.f : 1.f / S;
    uint2 out = make_uint2(pack_out<BF16>(x[0] * inv, x[1] * inv), pack_out<BF16>(x[2] * inv, x[3] * inv));
    if (M == -INFINITY) out = make_uint2(0, 0);
    const bool there = i < head.x * (HS / 4);
    if (there) {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.output) + at * HS + cc) = out;
      if (a.lse && cc == 0) a.lse[at] = M == -INFINITY ? -INFINITY : (M + fast_log2(S)) * 0.69314718055994531f;
    }
    if (there && M != -INFINITY && S == S && !finite4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv)) again |= 1u << r;
  }
  // rows to look at again, this block's columns of them (here, where little else is alive: called in the loop above, it
  // cost 2 of 117 us of 64 decode rows)
  if (warp != 0) return;
  __syncwarp();
  again = __reduce_or_sync(0xffffffffu, again);
  const int from = (blockIdx.y * 32) % (HS / 4) * 4;
  for (; again; again &= again - 1) {
    const int row = __ffs(again) - 1, rr = head.z + row, b = a.records[2 * c + 1].y;
    redo_row<HS, BF16>(a, b, head.y, a.cum[b + 1] - head.y, a.past[b], rr / a.G, head.w * a.G + rr % a.G, lane, from,
                       min(from + 128, HS));
  }
}


// ---- host ----------------------------------------------------------------------------------
int biased_ctas(int hs, int sms) {
  const int n = sms * (hs == 256 ? 1 : 2);
  return n < PA_BIASED_CTAS ? n : PA_BIASED_CTAS;
}

template <int HS, bool BF16>
static cudaError_t launch_biased_merge(const BiasedArgs& a, int ctas, cudaStream_t s) {
  return launch_pdl(biased_merge_kernel<HS, BF16>, dim3(ctas, 4), dim3(kMergeThreads), 0, s, a, ctas);
}

static int divisor(int a, int b) {
  while (b) {
    const int t = a % b;
    a = b;
    b = t;
  }
  return a;
}

template <int HS, bool BF16>
static cudaError_t launch_biased_rows(const BiasedArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int seg,
                                      int sms, cudaStream_t s, int* kernels, int* merge) {
  const int ctas = biased_ctas(HS, sms);
  constexpr int smem = BiRows<HS>::kBytes;
  // Clusters where two to eight CTAs for each unit run at once and none has many tiles, by the table's
  // width or the window: up to 8, or 16 where they are over half of what runs at once; else equal shares,
  // which do not mind how lengths differ. Random lengths up to l, clusters against equal shares: 1 x 200
  // keys 5.9 us and 9.9, 1 x 4000 12.9 and 13.7, 1 x 8000 16.7 and 14.5, 4 x 8000 22.9 and 26.1, 8 x 4000
  // 23.6 and 27.1, 1 x 60000 73 and 37.
  const int64_t units = (int64_t)a.B * a.kvh, tiles = ceil_div(keys_in_reach(a, 16), kBiTile) + 1;
  const int cl = cluster_size(units, ctas, tiles, 1, 8);
  if (a.G <= 16 && cl > 1 && tiles <= (int64_t)cl * (2 * units * cl > ctas ? 16 : 8)) {
    *kernels += 1;
    return launch_clusters(biased_rows_kernel<HS, BF16, true>, dim3((unsigned)units, 1, cl), kBiThreads, smem, smem, s, a, tk,
                           tv, seg);
  }
  *kernels += 1;
  if (cudaError_t e = cudaFuncSetAttribute(biased_rows_kernel<HS, BF16, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))
    return e;
  if (cudaError_t e = launch_pdl(biased_rows_kernel<HS, BF16, false>, dim3(ctas), dim3(kBiThreads), smem, s, a, tk, tv, seg))
    return e;
  *merge = ctas;
  return cudaSuccess;
}

cudaError_t launch_biased(const BiasedArgs& args, bool bf16, int sms, cudaStream_t s, int* kernels) {
  BiasedArgs a = args;
  *kernels = 0;
  const int seg = divisor(a.bs, kBiTile);
  const int64_t slots = (int64_t)a.num_blocks * a.bs;
  CUtensorMap tk, tv, tq;
  if (!cache_map_16(&tk, a.key_cache, bf16, a.hs, a.kvh, slots, seg) ||
      !cache_map_16(&tv, a.value_cache, bf16, a.hs, a.kvh, slots, seg))
    return cudaErrorInvalidValue;
  // Sequences of up to 16 rows per KV head are the rows kernel's, longer ones the tile kernel's (groups
  // of over 128 heads, more than a tile's rows, are all the rows kernel's); a kernel that can have none is
  // not launched. The tile kernel comes first, so that the rows' bytes fill what its last CTAs leave free (8 chunks
  // of 512 and 24 decode rows 321 us, in the other order 331, with the rows on 120 CTAs through all of the tiles' time
  // 325; the chunks alone 261: a rows CTA takes the place of a tile's), and the merge of the rows kernel's results last.
  int merge = 0;
#define PA_TYPES(F, HS, ...) (bf16 ? F<HS, true>(__VA_ARGS__) : F<HS, false>(__VA_ARGS__))
#define PA_SIZES(F, ...) (a.hs == 64 ? PA_TYPES(F, 64, __VA_ARGS__) : a.hs == 128 ? PA_TYPES(F, 128, __VA_ARGS__) : PA_TYPES(F, 256, __VA_ARGS__))
  if (a.G <= 128 && (a.max_rows == 0 || (int64_t)a.max_rows * a.G > 16)) {
    const int rows = 128 / a.G;
    if (!query_block_map(&tq, a.query, bf16, a.hs, a.nh, a.N, a.q_stride, a.G, rows)) return cudaErrorInvalidValue;
    *kernels += 1;
    if (cudaError_t e = bf16 ? launch_biased_tile_bf16(a, tq, tk, tv, seg, rows, sms, s)
                             : launch_biased_tile_f16(a, tq, tk, tv, seg, rows, sms, s))
      return e;
    a.after_tiles = 1;
  }
  if (a.G <= 16 || a.G > 128)
    if (cudaError_t e = PA_SIZES(launch_biased_rows, a, tk, tv, seg, sms, s, kernels, &merge)) return e;
  if (merge == 0) return cudaSuccess;
  *kernels += 1;
  return PA_SIZES(launch_biased_merge, a, merge, s);
#undef PA_SIZES
#undef PA_TYPES
}

}  // namespace pa
