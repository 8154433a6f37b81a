// Attention of query rows over the pages selected for them.
//
// A block of R consecutive rows of a sequence shares, per KV head g, a list of logical pages
// in ascending order; row j of the sequence attends, for the G query heads of g, the keys t <=
// past + j of those pages: softmax(scale q.k) V in fp32, rounded once to T. A row without any
// key gives zeros and an lse of -inf.
//
// One CTA (or a cluster that shares the keys) takes one block and KV head: its R * G query
// rows are the rows of one matrix product against each 64-key tile of the list, so every
// gathered K and V element is loaded once for all of them. The list is read as one string
// of "virtual" keys v = 0 .. n_list * block_size - 1 (page list[v / bs], offset v % bs): only
// the last pages can reach past a row, so all tiles but the last few need no mask, and no
// tile has a hole. Nothing is planned and nothing is kept in memory: the CTA finds its
// sequence from its index (find_seq) and the partial results of a cluster meet in its CTAs'
// shared memory, so that calls share no state.
//
// Two kernels, by the rows that share a list:
//   sparse_rows_kernel  up to 16 (decode steps): bound by the bytes of K and V;
//   sparse_tile_kernel  more (prompts, drafts of wide groups): tcgen05, bound by the softmax.
#include "ops.cuh"

namespace pa {

constexpr int kSpTile = 64;  // keys per tile

// ---- a CTA's work item ---------------------------------------------------------------------
struct SparseItem {
  int rows;    // rows of the batch in this item (0: nothing to do)
  int row0;    // the first of them
  int pos0;    // its position
  int n_list;  // pages in the list
  int v_end;   // virtual keys up to the last row's position
  int v_mask;  // virtual keys that every row sees
};

// By one warp: rows [sub, sub + sub_rows) of query block u and the list of pages of KV head
// g, as (logical, physical) pairs; entries that are no page of the block's history in
// ascending order are passed over (and reported, unless -1), pages behind the last row too.
__device__ __forceinline__ SparseItem sparse_item(const PageArgs& a, int u, int sub, int sub_rows, int g, int2* list,
                                                  int lane) {
  constexpr int E = 4;  // entries per lane and step: their loads, then their table loads, are in flight together
  SparseItem it{};
  int e[E];
  auto entries = [&](const int* sel, int i) {
#pragma unroll
    for (int k = 0; k < E; ++k) e[k] = i + 32 * k + lane < a.top_k ? sel[i + 32 * k + lane] : -1;
  };
  if (a.R == 1) entries(a.selected + ((int64_t)u * a.kvh + g) * a.top_k, 0);  // (u < N is the row)
  const Seq s = find_seq(a.cum, a.past, a.B, a.R, a.R == 1 ? 0 : 1, u, a.N, a.max_blocks, a.bs, lane);
  if (!s.ok) return it;
  const int j0 = (u - (a.R == 1 ? s.c0 : s.c0 / a.R + s.b)) * a.R;
  if (j0 < 0 || j0 + sub >= s.q) return it;
  it.rows = min(min(a.R - sub, sub_rows), s.q - j0 - sub);
  it.row0 = s.c0 + j0 + sub;
  it.pos0 = s.past + j0 + sub;
  const int last = it.pos0 + it.rows - 1;
  const int visible = (s.past + min(j0 + a.R, s.q) - 1) / a.bs + 1;
  const int whole = (it.pos0 + 1) / a.bs;  // pages below are seen whole by every row
  const int* sel = a.selected + ((int64_t)(s.c0 + j0) * a.kvh + g) * a.top_k;
  const int* table = a.table + (int64_t)s.b * a.max_blocks;
  int kept = 0, top = -1, last_page = -1, n_whole = 0;
  for (int i = 0; i < a.top_k; i += 32 * E) {
    if (a.R != 1 || i > 0) entries(sel, i);
    int phys[E];
#pragma unroll
    for (int k = 0; k < E; ++k) phys[k] = e[k] >= 0 && e[k] < visible ? table[e[k]] : -1;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      if (i + 32 * k >= a.top_k) break;
      int m = e[k];  // the largest entry up to this lane
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, m, d);
        if (lane >= d) m = max(m, y);
      }
      int before = __shfl_up_sync(0xffffffffu, m, 1);
      before = max(top, lane ? before : -1);
      bool use = e[k] >= 0 && e[k] < visible && e[k] > before && phys[k] >= 0 && phys[k] < a.num_blocks;
      if (!use && e[k] != -1 && a.error) atomicOr(a.error, PA_DEVERR_BAD_BLOCK);
      use = use && (int64_t)e[k] * a.bs <= last;
      const unsigned mask = __ballot_sync(0xffffffffu, use);
      if (use) list[kept + __popc(mask & ((1u << lane) - 1))] = make_int2(e[k], phys[k]);
      n_whole += __popc(__ballot_sync(0xffffffffu, use && e[k] < whole));
      if (mask) last_page = __shfl_sync(0xffffffffu, e[k], 31 - __clz(mask));
      kept += __popc(mask);
      top = max(top, __shfl_sync(0xffffffffu, m, 31));
    }
  }
  it.n_list = kept;
  it.v_mask = n_whole * a.bs;
  it.v_end = kept * a.bs;
  if (kept && last - last_page * a.bs + 1 < a.bs) it.v_end -= a.bs - (last - last_page * a.bs + 1);
  return it;
}

// ---- up to 16 rows per list: warp-level MMA --------------------------------------------------
// A CTA streams its share of the list's tiles through a ring of K and V tiles (TMA, one box
// per page segment, 128-byte swizzle); four consumer warps take 16 keys of every tile each:
// S = Q K^T, an online softmax in registers, O += P V (bf16: P as two bf16 terms). The warps'
// (m, l, O) meet in shared memory, then those of the cluster's CTAs: every CTA learns all
// (m, l), scales its own O by 2^(m - M) / L, and sums a share of the columns over the cluster
// in CTA order. The bytes in flight are what keeps HBM busy: two CTAs of three 32 KB stages
// per SM, as the dense decode kernel has. 64 rows of 32 + 8 heads of 128, 16 pages of 64 each:
// 46 us, 5.8 TB/s; one row of 32 pages of 64 in clusters of eight: 7.8 us, of which a third
// before the first tile and a third after the last.
template <int HS>
struct RowsSmem {
  static constexpr int kStages = 3;
  static constexpr int kTileBytes = kSpTile * HS * 2;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStride = HS + 4;  // floats between rows of a partial result
  static constexpr int kMl = kStages * kStageBytes;           // float [2][4][16]: m and l of the warps
  static constexpr int kCl = kMl + 2 * 4 * 16 * 4;            // float [2][16]: m and l of the CTA
  static constexpr int kBars = kCl + 2 * 16 * 4;
  static constexpr int kAbort = kBars + 2 * kStages * 8;      // abort flag, error word
  static constexpr int kItem = kAbort + 16;
  static constexpr int kList = kItem + 32;
  static_assert(4 * 16 * kStride * 4 <= kStages * kStageBytes, "partial results lie over the ring");
  static size_t bytes(int top_k) { return kList + (size_t)top_k * 8 + 1024; }
};
constexpr int kRowsThreads = 160;

template <int HS, bool BF16>
__global__ void __launch_bounds__(kRowsThreads, HS == 256 ? 1 : 2)
    sparse_rows_kernel(const PageArgs a, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const int seg_rows, const int chunks) {
  using L = RowsSmem<HS>;
  constexpr int NKS = HS / 16, ND = HS / 8;
  constexpr float kLift = BF16 ? 1.f : 32768.f;  // of the weights on their way into P V
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  float* ml = reinterpret_cast<float*>(smem + L::kMl);
  float* cl = reinterpret_cast<float*>(smem + L::kCl);
  float* part = reinterpret_cast<float*>(smem);  // [4][16][kStride], once the ring is done
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* empty = full + L::kStages;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kAbort);
  uint32_t* err = reinterpret_cast<uint32_t*>(smem + L::kAbort + 4);
  SparseItem* item_s = reinterpret_cast<SparseItem*>(smem + L::kItem);
  int2* list = reinterpret_cast<int2*>(smem + L::kList);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.y / chunks, r_first = blockIdx.y % chunks * 16;  // rows r = j * G + head of the item
  const int rank = blockIdx.z, C = gridDim.z;                            // the cluster is a column of the grid
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    *abort = 0;
    *err = 0;
    fence_mbar_init();
  }
  pdl_wait();
  if (warp == 4) {
    const SparseItem it = sparse_item(a, blockIdx.x, 0, a.R, g, list, lane);
    if (lane == 0) *item_s = it;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && rank == 0)
    check_batch(a.cum, a.past, a.B, a.N, a.max_blocks, a.bs, a.error);
  __syncthreads();
  const SparseItem it = *item_s;
  const int n_rows = min(16, it.rows * a.G - r_first);  // (all CTAs of a cluster agree)
  if (n_rows <= 0) return;
  const int tiles = (it.v_end + kSpTile - 1) / kSpTile;
  const int t0 = (int)((int64_t)tiles * rank / C), t1 = (int)((int64_t)tiles * (rank + 1) / C);

  const int tq = lane & 3, gq = lane >> 2;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  float o[ND][4];
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;

  if (warp == 4) {
    // ---- producer ----
    const int nseg = kSpTile / seg_rows, oob = a.num_blocks * a.bs;
    for (int t = t0; t < t1; ++t) {
      const int s = (t - t0) % L::kStages;
      const uint32_t ph = ((t - t0) / L::kStages) & 1;
      if (lane == 0) {
        mbar_wait(&empty[s], ph ^ 1, abort, err);
        mbar_arrive_expect_tx(&full[s], L::kStageBytes);
      }
      __syncwarp();
      if (lane < nseg) {
        const int v = t * kSpTile + lane * seg_rows, i = v / a.bs;
        const int z = i < it.n_list ? list[i].y * a.bs + (v - i * a.bs) : oob;  // (past the list: zeros)
        uint8_t* dst = smem + s * L::kStageBytes + lane * seg_rows * 128;
#pragma unroll
        for (int h = 0; h < HS / 64; ++h) {
          tma_load_3d(dst + h * kSpTile * 128, &tmK, &full[s], h * 64, g, z);
          tma_load_3d(dst + L::kTileBytes + h * kSpTile * 128, &tmV, &full[s], h * 64, g, z);
        }
      }
      __syncwarp();
    }
  } else {
    // ---- consumers: warp w has keys 16w .. 16w + 15 of every tile ----
    const int w = warp;
    uint32_t qa[NKS][4];  // Q as the A operand: rows gq and gq + 8
    {
      const uint32_t* p[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r_first + gq + 8 * i;
        p[i] = gq + 8 * i < n_rows
                   ? reinterpret_cast<const uint32_t*>(a.query + (int64_t)(it.row0 + r / a.G) * a.q_stride +
                                                       (int64_t)(g * a.G + r % a.G) * HS + tq * 2)
                   : nullptr;
      }
#pragma unroll
      for (int ks = 0; ks < NKS; ++ks) {
        qa[ks][0] = p[0] ? __ldg(p[0] + ks * 8) : 0u;
        qa[ks][2] = p[0] ? __ldg(p[0] + ks * 8 + 4) : 0u;
        qa[ks][1] = p[1] ? __ldg(p[1] + ks * 8) : 0u;
        qa[ks][3] = p[1] ? __ldg(p[1] + ks * 8 + 4) : 0u;
      }
    }
    // the last position of the thread's two rows (padding rows borrow the last row's)
    const int lim0 = it.pos0 + min((r_first + gq) / a.G, it.rows - 1);
    const int lim1 = it.pos0 + min((r_first + gq + 8) / a.G, it.rows - 1);
    const int mi = lane >> 3, rr = lane & 7;
    for (int t = t0; t < t1; ++t) {
      const int s = (t - t0) % L::kStages;
      mbar_wait(&full[s], ((t - t0) / L::kStages) & 1, abort, err);
      const uint32_t kb = smem_u32(smem + s * L::kStageBytes), vb = kb + L::kTileBytes;
      const int v0 = t * kSpTile + 16 * w;  // the warp's first virtual key
      if (v0 < it.v_end) {
        float sa[2][4] = {}, sb[2][4] = {};  // keys 0-7 and 8-15; even and odd k-steps
        {
          const int key = 16 * w + (mi >> 1) * 8 + rr;
#pragma unroll
          for (int ks = 0; ks < NKS; ++ks) {
            const int c = ks * 2 + (mi & 1);
            uint32_t b0, b1, b2, b3;
            ldsm_x4(kb + (c >> 3) * (kSpTile * 128) + key * 128 + (((c & 7) ^ (key & 7)) << 4), b0, b1, b2, b3);
            mma16816<BF16>((ks & 1) ? sb[0] : sa[0], qa[ks], b0, b1);
            mma16816<BF16>((ks & 1) ? sb[1] : sa[1], qa[ks], b2, b3);
          }
        }
        float x[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] = (sa[n][e] + sb[n][e]) * a.scale_log2;
        if (v0 + 16 > it.v_mask) {  // (16 keys never straddle a page)
          const int i = v0 / a.bs, base = list[i].x * a.bs + (v0 - i * a.bs);
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (base + n * 8 + tq * 2 + (e & 1) > (e < 2 ? lim0 : lim1)) x[n][e] = -INFINITY;
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
        for (int n = 0; n < 2; ++n) {
          p[n][0] = fast_exp2(x[n][0] - ms0);
          p[n][1] = fast_exp2(x[n][1] - ms0);
          p[n][2] = fast_exp2(x[n][2] - ms1);
          p[n][3] = fast_exp2(x[n][3] - ms1);
        }
        l0 = l0 * al0 + ((p[0][0] + p[0][1]) + (p[1][0] + p[1][1]));
        l1 = l1 * al1 + ((p[0][2] + p[0][3]) + (p[1][2] + p[1][3]));
        // P as the A operand: fp16 rounds the weights once (2^-11, the output's own rounding and the
        // dense call's choice; errors of 2.8e-4 where weights of 32 bits leave 2.1e-4 on 64 decode rows),
        // lifted from at most 1 to at most 2^15, so that only those below 2^-29 of the largest are
        // subnormal and have absolute errors, of 2^-40: without it many small ones beside a large
        // one were lost; bf16, whose one rounding would be 2^-8, keeps them as two terms
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
        // keys past the last row may be unwritten cache rows: their V is cleared, so that no
        // NaN meets a weight of 0
        const int key = 16 * w + (mi & 1) * 8 + rr;
        auto pv = [&](uint32_t mlo, uint32_t mhi) {
#pragma unroll
          for (int dp = 0; dp < ND / 2; ++dp) {
            const int c = 2 * dp + (mi >> 1);
            uint32_t w0, w1, w2, w3;
            ldsm_x4_t(vb + (c >> 3) * (kSpTile * 128) + key * 128 + (((c & 7) ^ (key & 7)) << 4), w0, w1, w2, w3);
            w0 &= mlo, w2 &= mlo, w1 &= mhi, w3 &= mhi;
            mma16816<BF16>(o[2 * dp], ph, w0, w1);
            mma16816<BF16>(o[2 * dp + 1], ph, w2, w3);
            if constexpr (BF16) {
              mma16816<BF16>(o[2 * dp], pl, w0, w1);
              mma16816<BF16>(o[2 * dp + 1], pl, w2, w3);
            }
          }
        };
        if (v0 + 16 <= it.v_end) {
          pv(0xffffffffu, 0xffffffffu);
        } else {
          const int k0 = v0 + 2 * tq, k8 = k0 + 8;
          pv((k0 < it.v_end ? 0xFFFFu : 0u) | (k0 + 1 < it.v_end ? 0xFFFF0000u : 0u),
             (k8 < it.v_end ? 0xFFFFu : 0u) | (k8 + 1 < it.v_end ? 0xFFFF0000u : 0u));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    // scores of NaN alone leave no maximum but a sum of NaN, which the merge must not take for a
    // row without keys
    if (m0 == -INFINITY && l0 != l0) m0 = 0.f;
    if (m1 == -INFINITY && l1 != l1) m1 = 0.f;
    if (tq == 0) {
      ml[w * 16 + gq] = m0, ml[w * 16 + gq + 8] = m1;
      ml[64 + w * 16 + gq] = l0, ml[64 + w * 16 + gq + 8] = l1;
    }
  }
  __syncthreads();  // (m, l) of the warps; the ring has been read
  // the CTA's (m, l) of each row, then the cluster's
  if (threadIdx.x < 16) {
    const int r = threadIdx.x;
    float M = fmaxf(fmaxf(ml[r], ml[16 + r]), fmaxf(ml[32 + r], ml[48 + r])), S = 0.f;
    for (int w = 0; w < 4; ++w)
      if (ml[w * 16 + r] != -INFINITY) S += ml[64 + w * 16 + r] * fast_exp2(ml[w * 16 + r] - M);
    cl[r] = M, cl[16 + r] = S;
  }
  if (warp < 4) {
    // the warp's rows relative to the CTA's maximum, side by side over the ring
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = gq + 8 * i;
      const float M = fmaxf(fmaxf(ml[r], ml[16 + r]), fmaxf(ml[32 + r], ml[48 + r]));
      const float m = i ? m1 : m0;
      f[i] = m == -INFINITY ? 0.f : fast_exp2(m - M) * (1.f / kLift);
    }
    float* dst = part + warp * 16 * L::kStride;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      if (gq < n_rows)
        *reinterpret_cast<float2*>(dst + gq * L::kStride + d * 8 + tq * 2) = make_float2(o[d][0] * f[0], o[d][1] * f[0]);
      if (gq + 8 < n_rows)
        *reinterpret_cast<float2*>(dst + (gq + 8) * L::kStride + d * 8 + tq * 2) =
            make_float2(o[d][2] * f[1], o[d][3] * f[1]);
    }
  }
  __syncthreads();
  if (C > 1) {
    // the four warps' partials added in place, then the cluster's CTAs read each other's
    for (int i = threadIdx.x; i < n_rows * (HS / 4); i += kRowsThreads) {
      float* p = part + i / (HS / 4) * L::kStride + i % (HS / 4) * 4;
      float4 x = *reinterpret_cast<float4*>(p);
      for (int w = 1; w < 4; ++w) {
        const float4 y = *reinterpret_cast<float4*>(p + w * 16 * L::kStride);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      *reinterpret_cast<float4*>(p) = x;
    }
    cluster_sync();
  }
  // this CTA's share of the columns, in quads
  const int c0 = HS / 4 * rank / C, c1 = HS / 4 * (rank + 1) / C, nc = c1 - c0;
  for (int i = threadIdx.x; i < n_rows * nc; i += kRowsThreads) {
    const int r = i / nc, c = c0 + i % nc;
    float x[4] = {0.f, 0.f, 0.f, 0.f}, M = -INFINITY, S = 0.f;
    if (C > 1) {
      for (int k = 0; k < C; ++k) M = fmaxf(M, ld_cluster(cluster_addr(cl + r, k)));
      for (int k = 0; k < C; ++k) {
        const float m = ld_cluster(cluster_addr(cl + r, k));
        if (m == -INFINITY) continue;
        const float f = fast_exp2(m - M);
        S += f * ld_cluster(cluster_addr(cl + 16 + r, k));
        const float4 y = ld_cluster4(cluster_addr(part + r * L::kStride + c * 4, k));
        x[0] += f * y.x, x[1] += f * y.y, x[2] += f * y.z, x[3] += f * y.w;
      }
    } else {
      M = cl[r], S = cl[16 + r];
      for (int w = 0; w < 4; ++w) {
        const float4 y = *reinterpret_cast<float4*>(part + (w * 16 + r) * L::kStride + c * 4);
        x[0] += y.x, x[1] += y.y, x[2] += y.z, x[3] += y.w;
      }
    }
    const float inv = S > 0.f ? 1.f / S : 0.f;
    const int64_t row = it.row0 + (r_first + r) / a.G;
    const int h = g * a.G + (r_first + r) % a.G;
    uint2 out = make_uint2(pack2<BF16>(x[0] * inv, x[1] * inv), pack2<BF16>(x[2] * inv, x[3] * inv));
    if (!(S > 0.f) && M == -INFINITY) out = make_uint2(0, 0);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.output) + (row * a.nh + h) * HS + c * 4) = out;
    if (a.lse && c == 0)
      a.lse[row * a.nh + h] = M == -INFINITY ? -INFINITY : (M + fast_log2(S)) * 0.69314718055994531f;
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another reads its shared memory
  if (threadIdx.x == 0 && *err && a.error) atomicOr(a.error, *err);
}

// ---- more rows per list: tcgen05 -------------------------------------------------------------
// The up to 128 rows r = j * G + head of a block are one M = 128 tile (TMA lays them out so
// from a (channel, head, row) view of the query; rows past the item are computed and not
// stored). Warp 0 gathers K and V tiles (two stages), warp 1 issues S_t = Q K_t^T into one of
// two S buffers in TMEM and O += P_t V_t, warps 2 .. 9 are the softmax: two threads share a
// row (TMEM lets a warp at 32 of the 128 lanes), read 32 of its 64 scores each, exchange their
// maxima through shared memory, write P over the scores (fp16, or bf16 hi and lo terms) and
// rescale O in TMEM when the maximum grew by more than 2^8 (fp16: 2^4). S_{t+1} is issued before P_t is waited for, so
// the tensor core works during the softmax; two CTAs share an SM (one with 256-wide heads)
// and fill each other's gaps, the prologue included. 4 prompts of 2048 rows in blocks of 32, 32
// pages of 64, bf16: 335 us (821 TFLOP/s, P V counted once); its loads alone take 206 us (10.5
// TB/s from L2), with the products 264 us, so L2, tensor pipe and softmax each wait for the
// others about half of the time, and two stages of K and V are what fits twice on an SM.
template <int HS>
struct TileSmem {
  static constexpr int kStages = 2;
  static constexpr int kQBytes = 128 * HS * 2;
  static constexpr int kTileBytes = kSpTile * HS * 2;
  static constexpr int kRing = kQBytes;                             // K tiles, then V tiles
  static constexpr int kBars = kRing + 2 * kStages * kTileBytes;    // 1 + 4 * kStages + 3 * 2 barriers
  static constexpr int kNumBars = 1 + 4 * kStages + 6;
  static constexpr int kAbort = kBars + kNumBars * 8;               // abort flag, error word, TMEM address
  static constexpr int kItem = (kAbort + 12 + 15) / 16 * 16;
  static constexpr int kMl = kItem + 32;                            // float [2][128]: m and l of the rows
  static constexpr int kX = kMl + 2 * 128 * 4;                      // float [2][128][2]: maxima and sums of half rows
  static constexpr int kList = kX + 2 * 128 * 2 * 4;
  static constexpr uint32_t kTmem = HS == 256 ? 512 : 256;          // S, S, O at columns 0, 64, 128
  static_assert(128 * HS * 4 <= 2 * kStages * kTileBytes, "the cluster's partial result lies over the ring");
  // At least a third of an SM's shared memory, so that no more CTAs share an SM than find TMEM
  // there: a CTA that waited for TMEM while its cluster waits for it could wait for ever.
  static size_t bytes(int top_k) {
    const size_t need = kList + (size_t)top_k * 8 + 1024;
    return need < 80 * 1024 ? 80 * 1024 : need;
  }
};
constexpr int kTileThreads = 320;

template <int HS, bool BF16>
__global__ void __launch_bounds__(kTileThreads, HS == 256 ? 1 : 2)
    sparse_tile_kernel(const PageArgs a, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const int seg_rows, const int sub_rows, const int chunks) {
  using L = TileSmem<HS>;
  constexpr int HALVES = HS / 64, KSTEPS = HS / 16;
  constexpr uint32_t IDESC_QK = idesc_f16(BF16, 128, kSpTile, false), IDESC_PV = idesc_f16(BF16, 128, HS, true);
  constexpr uint32_t kO = 128;  // TMEM column of O
  // The row's reference m_used may lag behind its maximum by kLag before O is rescaled. fp16
  // weights are lifted by 2^kLift, to 2^15 at most, so that only those below 2^-25 of the largest
  // are subnormal and have absolute errors, of 2^-36; l is lifted with them.
  constexpr float kLag = BF16 ? 8.f : 4.f, kLift = BF16 ? 0.f : 11.f, kUnlift = BF16 ? 1.f : 1.f / 2048;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* k_full = q_full + 1;
  uint64_t* k_empty = k_full + L::kStages;
  uint64_t* v_full = k_empty + L::kStages;
  uint64_t* v_empty = v_full + L::kStages;
  uint64_t* s_full = v_empty + L::kStages;  // [2]
  uint64_t* p_full = s_full + 2;            // [2]
  uint64_t* o_done = p_full + 2;            // [2]
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kAbort);
  uint32_t* err = reinterpret_cast<uint32_t*>(smem + L::kAbort + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kAbort + 8);
  SparseItem* item_s = reinterpret_cast<SparseItem*>(smem + L::kItem);
  float* ml = reinterpret_cast<float*>(smem + L::kMl);
  float2* half = reinterpret_cast<float2*>(smem + L::kX);  // [2][128]
  int2* list = reinterpret_cast<int2*>(smem + L::kList);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.y, u = blockIdx.x / chunks, sub = blockIdx.x % chunks * sub_rows;
  const int rank = blockIdx.z, C = gridDim.z;
  if (threadIdx.x == 32) {
    mbar_init(q_full, 1);
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 256);
      mbar_init(&o_done[i], 1);
    }
    *abort = 0;
    *err = 0;
    fence_mbar_init();
  }
  pdl_wait();
  if (warp == 0) {
    const SparseItem it = sparse_item(a, u, sub, sub_rows, g, list, lane);
    if (lane == 0) *item_s = it;
  }
  if (blockIdx.x == 0 && g == 0 && rank == 0) check_batch(a.cum, a.past, a.B, a.N, a.max_blocks, a.bs, a.error);
  __syncthreads();
  const SparseItem it = *item_s;
  if (it.rows <= 0) return;  // (all CTAs of a cluster agree)
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tiles = (it.v_end + kSpTile - 1) / kSpTile;
  const int t0 = (int)((int64_t)tiles * rank / C), n = (int)((int64_t)tiles * (rank + 1) / C) - t0;

  const int row = (warp & 3) * 32 + lane;  // (softmax warps) the thread's TMEM lane
  const int side = warp >= 6;              // and its half of the row's columns
  const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
  const int j = row / a.G;                  // its row in the item
  const bool live = warp >= 2 && j < it.rows && row < sub_rows * a.G;
  const bool any_live = __any_sync(0xffffffffu, live);
  float m_used = -INFINITY, l = 0.f;

  if (warp == 0) {
    // ---- producer ----
    if (n > 0) {
      const int nseg = kSpTile / seg_rows, oob = a.num_blocks * a.bs;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, (uint32_t)(sub_rows * a.G * HS * 2));
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
          tma_load_3d(smem + h * 128 * 128, &tmQ, q_full, h * 64, g * a.G, it.row0);
      }
      // tiles are asked for in the order in which the products free their stages: K_{t+2} (after
      // Q K_t) before V_{t+1} (after P V_{t-1})
      auto slot = [&](int t) {  // this lane's segment of tile t: its first cache row
        const int v = (t0 + t) * kSpTile + lane * seg_rows, i = v / a.bs;
        return lane < nseg && t < n && i < it.n_list ? list[i].y * a.bs + (v - i * a.bs) : oob;
      };
      auto load = [&](int t, const CUtensorMap* map, uint64_t* full, uint64_t* empty, uint8_t* ring) {
        if (t < 0 || t >= n) return;
        const int s = t % L::kStages, z = slot(t);
        if (lane == 0) {
          mbar_wait(&empty[s], ((t / L::kStages) & 1) ^ 1, abort, err);
          mbar_arrive_expect_tx(&full[s], L::kTileBytes);
        }
        __syncwarp();
        if (lane < nseg)
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
            tma_load_3d(ring + s * L::kTileBytes + h * kSpTile * 128 + lane * seg_rows * 128, map, &full[s], h * 64, g, z);
        __syncwarp();
      };
      for (int t = -2; t < n; ++t) {
        load(t + 2, &tmK, k_full, k_empty, smem + L::kRing);
        load(t + 1, &tmV, v_full, v_empty, smem + L::kRing + L::kStages * L::kTileBytes);
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer ----
    const uint64_t qdesc = sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t kdesc = sdesc_sw128(smem_u32(smem + L::kRing), 16, 1024);
    const uint64_t vdesc = sdesc_sw128(smem_u32(smem + L::kRing + L::kStages * L::kTileBytes), kSpTile * 128, 1024);
    auto issue_qk = [&](int t) {
      const int s = t % L::kStages;
      mbar_wait(&k_full[s], (t / L::kStages) & 1, abort, err);
      tc_fence_after();
      if (elect_one()) {
        const uint64_t kd = kdesc + (uint64_t)((s * L::kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < KSTEPS; ++kk)
          tc_mma_ss(tmem + (t & 1) * kSpTile, qdesc + (uint64_t)((kk >> 2) * (128 * 128 >> 4) + (kk & 3) * 2),
                    kd + (uint64_t)((kk >> 2) * (kSpTile * 128 >> 4) + (kk & 3) * 2), IDESC_QK, kk > 0 ? 1u : 0u);
        tc_commit(&s_full[t & 1]);
        tc_commit(&k_empty[s]);
      }
      __syncwarp();
    };
    if (n > 0) {
      mbar_wait(q_full, 0, abort, err);
      issue_qk(0);
    }
    for (int t = 0; t < n; ++t) {
      if (t + 1 < n) {
        if (t > 0) mbar_wait(&o_done[(t - 1) & 1], ((t - 1) >> 1) & 1, abort, err);  // P_{t-1}, in that S buffer, has been read
        issue_qk(t + 1);
      }
      const int s = t % L::kStages;
      mbar_wait(&v_full[s], (t / L::kStages) & 1, abort, err);
      const int valid = it.v_end - (t0 + t) * kSpTile;
      if (valid < kSpTile) {
        // rows past the last position may be unwritten: cleared, so that no NaN meets a
        // weight of 0 (whole 128-byte rows: the swizzle stays inside)
        uint8_t* vt = smem + L::kRing + (L::kStages + s) * L::kTileBytes;
        const int rows = kSpTile - valid;
        for (int c = lane; c < rows * 8 * HALVES; c += 32)
          *reinterpret_cast<uint4*>(vt + c / (rows * 8) * (kSpTile * 128) + (valid + c % (rows * 8) / 8) * 128 +
                                    c % 8 * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      mbar_wait(&p_full[t & 1], (t >> 1) & 1, abort, err);
      __syncwarp();
      tc_fence_after();
      if (elect_one()) {
        const uint64_t vd = vdesc + (uint64_t)((s * L::kTileBytes) >> 4);
        const uint32_t p = tmem + (t & 1) * kSpTile;
#pragma unroll
        for (int kk = 0; kk < kSpTile / 16; ++kk) {
          tc_mma_ts(tmem + kO, p + p_col(kk), vd + (uint64_t)(kk * (16 * 128 >> 4)), IDESC_PV,
                    kk > 0 || t > 0 ? 1u : 0u);
          if constexpr (BF16)
            tc_mma_ts(tmem + kO, p + p_col(kk) + 16, vd + (uint64_t)(kk * (16 * 128 >> 4)), IDESC_PV, 1u);
        }
        tc_commit(&o_done[t & 1]);
        tc_commit(&v_empty[s]);
      }
      __syncwarp();
    }
  } else {
    // ---- softmax ----
    // (S, P and O each signal on two barriers in turn: not every wait is made by every warp, and a
    // parity tells a phase from the next only, so a barrier must not be two phases ahead of or
    // behind one that waits; P_{t-2} V is done once S_t is, and P_t V is not before this warp's P_t)
    constexpr int COLS = kSpTile / 2, OCOLS = HS / 2;
    const float c = a.scale_log2;
    const float none = c > 0.f ? -INFINITY : INFINITY;  // a score whose product with c is -inf
    const int lim = it.pos0 + min(j, it.rows - 1);
    const uint32_t o_tmem = tmem + lane_off + kO + side * OCOLS;
    const int bar = 1 + (warp & 3);  // of the two warps of a lane quarter
    for (int t = 0; t < n; ++t) {
      mbar_wait(&s_full[t & 1], (t >> 1) & 1, abort, err);
      if (!any_live) {  // rows past the item: whatever their P holds stays in their rows of O
        mbar_arrive(&p_full[t & 1]);
        continue;
      }
      tc_fence_after();
      const uint32_t st = tmem + lane_off + (t & 1) * kSpTile;
      uint32_t r[COLS];
      tmem_ld_x32(st + side * COLS, r);
      const int v0 = (t0 + t) * kSpTile + side * COLS;
      if (v0 + COLS > it.v_mask) {
#pragma unroll
        for (int k = 0; k < COLS / 16; ++k) {  // (16 keys never straddle a page)
          const int v = v0 + 16 * k, i = v / a.bs;
          const int base = i < it.n_list ? list[i].x * a.bs + (v - i * a.bs) : INT32_MAX - 16;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (base + e > lim) r[16 * k + e] = __float_as_uint(none);
        }
      }
      float mc[4] = {none, none, none, none};
      if (c > 0.f) {
#pragma unroll
        for (int e = 0; e < COLS; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mc[k] = fmax3(mc[k], __uint_as_float(r[e + 2 * k]), __uint_as_float(r[e + 2 * k + 1]));
      } else {
#pragma unroll
        for (int e = 0; e < COLS; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mc[k] = fmin3(mc[k], __uint_as_float(r[e + 2 * k]), __uint_as_float(r[e + 2 * k + 1]));
      }
      const float best = c > 0.f ? fmax3(fmaxf(mc[0], mc[1]), mc[2], mc[3]) : fmin3(fminf(mc[0], mc[1]), mc[2], mc[3]);
      float2* hx = half + (t & 1) * 128 + row;
      (side ? hx->y : hx->x) = best * c;
      named_bar_sync(bar, 64);
      const float2 both = *hx;
      const float m_new = fmaxf(m_used, fmaxf(both.x, both.y));
      const bool grow = __any_sync(0xffffffffu, live && m_new > m_used + kLag);
      float alpha = 1.f;
      if (grow) {
        // (fp16: a whole number, which kLift is taken off exactly)
        const float to = BF16 ? m_new : ceilf(m_new);
        alpha = m_new == -INFINITY ? 1.f : fast_exp2(m_used - to);  // 0 on a row's first keys
        m_used = to;
        l *= alpha;
      }
      const float neg_m = m_used == -INFINITY ? 0.f : kLift - m_used;  // (no key yet: every weight is 0)
      const uint64_t c2 = f2_make(c, c), nm2 = f2_make(neg_m, neg_m);
      uint64_t lsum = f2_make(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < COLS / 16; ++k) {
        uint32_t* q = r + k * 16;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x0, x1;
          f2_split(f2_fma(f2_make(__uint_as_float(q[2 * e]), __uint_as_float(q[2 * e + 1])), c2, nm2), x0, x1);
          const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
          lsum = f2_add(lsum, f2_make(p0, p1));
          if constexpr (BF16) split_bf16x2(p0, p1, q[2 * e], q[2 * e + 1]);
          else q[2 * e] = pack2<false>(p0, p1);
        }
        const uint32_t p = st + p_col(side * (COLS / 16) + k);
        tmem_st_x8_nowait(p, q[0], q[2], q[4], q[6], q[8], q[10], q[12], q[14]);
        if constexpr (BF16) tmem_st_x8_nowait(p + 16, q[1], q[3], q[5], q[7], q[9], q[11], q[13], q[15]);
      }
      float s0, s1;
      f2_split(lsum, s0, s1);
      l += s0 + s1;
      if (t > 0 && grow) {  // O holds P_0 V .. P_{t-1} V once the last product is done
        mbar_wait(&o_done[(t - 1) & 1], ((t - 1) >> 1) & 1, abort, err);
        tc_fence_after();
#pragma unroll 1
        for (int cc = 0; cc < OCOLS; cc += 32) {
          uint32_t ov[32];
          tmem_ld_x32(o_tmem + cc, ov);
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
          tmem_st_x32(o_tmem + cc, ov);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[t & 1]);
    }
    if (n > 0) {
      mbar_wait(&o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, abort, err);
      tc_fence_after();
    }
    // the row's sum from its halves (the two warps have the same maximum)
    (side ? half[row].y : half[row].x) = l;
    named_bar_sync(bar, 64);
    l = half[row].x + half[row].y;
    if (m_used == -INFINITY && l != l) m_used = 0.f;  // scores of NaN alone: not a row without keys
    if (C > 1 && side == 0) ml[row] = m_used, ml[128 + row] = l;
  }

  uint16_t* out = static_cast<uint16_t*>(a.output);
  if (C == 1) {
    if (warp >= 2) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int64_t at = (int64_t)(it.row0 + j) * a.nh + g * a.G + row % a.G;
      if (live && a.lse && side == 0)
        a.lse[at] = m_used == -INFINITY ? -INFINITY : (m_used + fast_log2(l * kUnlift)) * 0.69314718055994531f;
#pragma unroll 1
      for (int cc = side * (HS / 2); cc < (side + 1) * (HS / 2); cc += 32) {
        uint32_t ov[32];
        if (n > 0) {
          tmem_ld_x32(tmem + lane_off + kO + cc, ov);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = 0u;
        }
        if (live) {
          const bool some = m_used != -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = some ? pack2<BF16>(__uint_as_float(ov[e + 2 * k]) * inv, __uint_as_float(ov[e + 2 * k + 1]) * inv) : 0u;
            *reinterpret_cast<uint4*>(out + at * HS + cc + e) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  } else {
    // every row's share of the cluster's result: O 2^(m - M) / L, quads of a row rotated by the
    // row so that a warp's stores spread over the banks
    cluster_sync();  // all (m, l)
    float* part = reinterpret_cast<float*>(smem + L::kRing);
    if (warp >= 2) {
      float M = -INFINITY, S = 0.f;
      for (int k = 0; k < C; ++k) M = fmaxf(M, ld_cluster(cluster_addr(ml + row, k)));
      for (int k = 0; k < C; ++k) {
        const float m = ld_cluster(cluster_addr(ml + row, k));
        if (m != -INFINITY) S += fast_exp2(m - M) * ld_cluster(cluster_addr(ml + 128 + row, k));
      }
      const float f = m_used == -INFINITY ? 0.f : fast_exp2(m_used - M) / S;
      if (rank == 0 && live && a.lse && side == 0)
        a.lse[(int64_t)(it.row0 + j) * a.nh + g * a.G + row % a.G] =
            M == -INFINITY ? -INFINITY : (M + fast_log2(S * kUnlift)) * 0.69314718055994531f;
#pragma unroll 1
      for (int cc = side * (HS / 2); any_live && cc < (side + 1) * (HS / 2); cc += 32) {
        uint32_t ov[32];
        if (n > 0) tmem_ld_x32(tmem + lane_off + kO + cc, ov);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (n > 0 && f != 0.f)
            x = make_float4(__uint_as_float(ov[e]) * f, __uint_as_float(ov[e + 1]) * f, __uint_as_float(ov[e + 2]) * f,
                            __uint_as_float(ov[e + 3]) * f);
          const int quad = ((cc + e) / 4 + row) % (HS / 4);
          *reinterpret_cast<float4*>(part + row * HS + quad * 4) = x;
        }
      }
    }
    cluster_sync();
    const int M = it.rows * a.G;  // rows of the item, a share of them summed by each CTA
    const int r0 = M * rank / C, r1 = M * (rank + 1) / C;
    for (int i = threadIdx.x; i < (r1 - r0) * (HS / 4); i += kTileThreads) {
      const int r = r0 + i / (HS / 4), quad = i % (HS / 4);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < C; ++k) {
        const float4 y = ld_cluster4(cluster_addr(part + r * HS + (quad + r) % (HS / 4) * 4, k));
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      const int64_t at = (int64_t)(it.row0 + r / a.G) * a.nh + g * a.G + r % a.G;
      *reinterpret_cast<uint2*>(out + at * HS + quad * 4) = make_uint2(pack2<BF16>(x.x, x.y), pack2<BF16>(x.z, x.w));
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }
  tc_fence_before();
  __syncthreads();  // (no warp waits any more: whichever gave up has said so)
  if (threadIdx.x == 0 && *err && a.error) atomicOr(a.error, *err);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
}

// ---- host ------------------------------------------------------------------------------------

static int common_divisor(int a, int b) {
  while (b) {
    const int t = a % b;
    a = b;
    b = t;
  }
  return a;
}

// The CTAs of a cluster share an item's tiles, as many as run at once. (More cost more than they
// balance: twice as many 8 long decode rows 26.6 us instead of 18.5 and 32 drafts of 4 in 256-wide
// heads 39.2 instead of 29.5, eight times as many 64 one-row sequences in blocks of 16, of 32 pages of
// 64, 208 us instead of 90. Idle sequences that are counted cost less: a chunk of 512 in blocks of
// 32 beside 63 of them takes 43.9 us in clusters of one instead of 40.1 of two.)
template <int HS, bool BF16>
static cudaError_t launch_rows(const PageArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int seg, int sms,
                               cudaStream_t s) {
  const int chunks = (int)ceil_div((int64_t)a.R * a.G, 16);
  const int tiles = (int)ceil_div((int64_t)a.top_k * a.bs, kSpTile);
  const int64_t items = items_of_batch(a.N, a.B, a.R, chunks, ceil_div(a.G, 16)) * a.kvh;
  const int c = cluster_size(items, (int64_t)sms * (HS == 256 ? 1 : 2), tiles, 2, 8);
  const dim3 grid((unsigned)query_blocks(a), (unsigned)(a.kvh * chunks), (unsigned)c);
  return launch_clusters(sparse_rows_kernel<HS, BF16>, grid, kRowsThreads, RowsSmem<HS>::bytes(a.top_k),
                         RowsSmem<HS>::bytes(PA_MAX_SELECTED_PAGES), s, a, tk, tv, seg, chunks);
}

template <int HS, bool BF16>
static cudaError_t launch_tile(const PageArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               int seg, int sub_rows, int sms, cudaStream_t s) {
  const int chunks = (int)ceil_div(a.R, sub_rows);
  const int tiles = (int)ceil_div((int64_t)a.top_k * a.bs, kSpTile);
  const int64_t items = items_of_batch(a.N, a.B, sub_rows, 1, 1) * a.kvh;
  const int c = cluster_size(items, (int64_t)sms * (HS == 256 ? 1 : 2), tiles, 4, 8);
  const dim3 grid((unsigned)(query_blocks(a) * chunks), (unsigned)a.kvh, (unsigned)c);
  return launch_clusters(sparse_tile_kernel<HS, BF16>, grid, kTileThreads, TileSmem<HS>::bytes(a.top_k),
                         TileSmem<HS>::bytes(PA_MAX_SELECTED_PAGES), s, a, tq, tk, tv, seg, sub_rows, chunks);
}

cudaError_t launch_sparse(const PageArgs& a, bool bf16, int sms, cudaStream_t s) {
  const int seg = common_divisor(a.bs, kSpTile);
  const int64_t slots = (int64_t)a.num_blocks * a.bs;
  CUtensorMap tk, tv, tq;
  if (!cache_map_16(&tk, a.key_cache, bf16, a.hs, a.kvh, slots, seg) ||
      !cache_map_16(&tv, a.value_cache, bf16, a.hs, a.kvh, slots, seg))
    return cudaErrorInvalidValue;
  // Up to 16 rows on a list take the warp-level kernel, which has one row tile, more the tcgen05
  // kernel, whatever share of its 128 rows they fill: 64 decode requests with 16 pages of 64 take
  // 46.9 us against 51.8 with 4 rows, 52.2 against 55.6 with 16, and 65.5 against 55.7 with 20 (a
  // second pass over the list). Groups of over 128 heads are more than a tile's rows.
  if (takes_rows_kernel(a.R, a.G)) {
#define PA_ROWS(HS) (bf16 ? launch_rows<HS, true>(a, tk, tv, seg, sms, s) : launch_rows<HS, false>(a, tk, tv, seg, sms, s))
    return a.hs == 64 ? PA_ROWS(64) : a.hs == 128 ? PA_ROWS(128) : PA_ROWS(256);
#undef PA_ROWS
  }
  const int sub_rows = rows_of_tile(a.R, a.G);
  if (!query_block_map(&tq, a.query, bf16, a.hs, a.nh, a.N, a.q_stride, a.G, sub_rows)) return cudaErrorInvalidValue;
#define PA_TILE(HS)                                                    \
  (bf16 ? launch_tile<HS, true>(a, tq, tk, tv, seg, sub_rows, sms, s) \
        : launch_tile<HS, false>(a, tq, tk, tv, seg, sub_rows, sms, s))
  return a.hs == 64 ? PA_TILE(64) : a.hs == 128 ? PA_TILE(128) : PA_TILE(256);
#undef PA_TILE
}

}  // namespace pa
