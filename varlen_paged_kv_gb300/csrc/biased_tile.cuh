// biased_tile_kernel: the biased attention of sequences of more than 16 rows per KV head.
//
// The up to 128 rows r = j * G + head of 128 / G consecutive rows of a sequence are one M = 128
// tile (TMA lays them out so from a (channel, head, row) view of the query; rows past the item are
// computed and not stored). Warp 0 loads K and V tiles of 64 keys (two stages), warp 1 issues
// S_t = Q K_t^T into one of two S buffers in TMEM and O += P_t V_t, the others are the softmax: a
// thread takes its row's 64 scores through the cap, the bias and the mask, writes P over them
// (fp16, or bf16 hi and lo terms) and rescales O in TMEM when the maximum grew by more than 2^8
// (fp16: 2^7). With 256-wide heads, one CTA to an SM, two threads share a row, take 32 of its
// scores each and exchange their maxima through shared memory; with narrower ones two CTAs share an
// SM and fill each other's gaps (there two threads a row were slower, 4 prompts of 2048 872 us
// instead of 746). S_{t+1} is issued before P_t is waited for, so the tensor core works during the
// softmax. What bounds it is that softmax: 4 prompts of 2048 with a cap and a bias take 638 us in bf16, 1020 TFLOP/s
// (P V counted once), 540 in fp16, and 470 in fp16 without cap and bias, 1383 TFLOP/s.
// The load of S brings the row's largest magnitude (or score) with it; finding it score by score took
// 738 us instead of 723 (before the steps below), and 344 instead of 329 for chunks with a cap and a window.
// Where a batch has few tiles of rows, the CTAs of a cluster share an item's keys and add their
// results through each other's shared memory.
//
// RULES (1: a cap, 2: a bias) are the call's: the softmax's code is long, and what it jumps over for other
// calls' rules costs fetches (chunks with a cap and a window 340 us instead of 352 with all of it in one kernel).
#pragma once

#include "biased.cuh"

namespace pa {

template <int HS>
struct BiTile {
  static constexpr int kStages = 2;
  static constexpr int kQBytes = 128 * HS * 2;
  static constexpr int kTileBytes = kBiTile * HS * 2;
  static constexpr int kRing = kQBytes;                             // K tiles, then V tiles
  static constexpr int kBars = kRing + 2 * kStages * kTileBytes;    // 1 + 4 * kStages + 3 * 2 barriers
  static constexpr int kNumBars = 1 + 4 * kStages + 6;
  static constexpr int kAbort = kBars + kNumBars * 8;               // abort flag, error word, TMEM address
  static constexpr int kItem = (kAbort + 12 + 15) / 16 * 16;
  static constexpr int kMl = kItem + 64;                            // float [2][128]: m and l of the rows
  static constexpr int kX = kMl + 2 * 128 * 4;                      // float [2][128][2]: maxima and sums of half rows
  static constexpr int kRedo = kX + 2 * 128 * 2 * 4;                // uint32 [5]: rows whose result is not finite, pages to report
  static constexpr uint32_t kTmem = HS == 256 ? 512 : 256;          // S, S, O at columns 0, 64, 128
  static_assert(128 * HS * 4 <= 2 * kStages * kTileBytes, "the cluster's partial result lies over the ring");
  // At least a third of an SM's shared memory, so that no more CTAs share an SM than find TMEM
  // there: a CTA that waited for TMEM while its cluster waits for it could wait for ever.
  static constexpr int kNeed = kRedo + 32 + 1024;
  static constexpr int kBytes = kNeed < 80 * 1024 ? 80 * 1024 : kNeed;
};

// tcgen05.ld 32x32b of COLS consecutive columns of this thread's TMEM lane, with the largest of them, or of their
// magnitudes, on the way (NaN passed over, as fmaxf does)
template <int COLS, bool ABS>
__device__ __forceinline__ float tmem_ld_max(uint32_t taddr, uint32_t* r) {
  float m;
  if constexpr (COLS == 64 && ABS) {
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x64.max.abs.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, %64, [%65];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=f"(m)
        : "r"(taddr)
        : "memory");
  } else if constexpr (COLS == 64) {
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x64.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, %64, [%65];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=f"(m)
        : "r"(taddr)
        : "memory");
  } else if constexpr (ABS) {
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.abs.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(m)
        : "r"(taddr)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(m)
        : "r"(taddr)
        : "memory");
  }
  return m;
}

// softmax threads that share a row, and the threads of a CTA
__host__ __device__ constexpr int bi_sides(int hs) { return hs == 256 ? 2 : 1; }
__host__ __device__ constexpr int bi_threads(int hs) { return 64 + 128 * bi_sides(hs); }

// a CTA's work item: some rows of one sequence
struct TileItem {
  int rows, row0, pos0, b;  // rows of the batch (0: none), the first of them, its position, the sequence
  int prefix, total;        // keys of the sequence
  int lo, hi;               // keys that some row sees
  int all_lo, all_hi;       // keys that all rows see that see any
};

__device__ __forceinline__ TileItem tile_item(const BiasedArgs& a, int u, int sub_rows, int lane) {
  TileItem it{};
  Seq s = find_seq(a.cum, a.past, a.B, sub_rows, 1, u, a.N, a.max_blocks, a.bs, lane);
  s.ok = s.ok && (a.max_rows == 0 || s.q <= a.max_rows);
  if (!s.ok || short_rows(a, s)) return it;
  const int j0 = (u - (s.c0 / sub_rows + s.b)) * sub_rows;
  if (j0 < 0 || j0 >= s.q) return it;
  it.rows = min(sub_rows, s.q - j0);
  it.row0 = s.c0 + j0;
  it.pos0 = s.past + j0;
  it.b = s.b;
  it.prefix = a.prefix ? a.prefix[s.b] : 0;
  it.total = s.past + s.q;
  Keys some{INT32_MAX, 0}, all{0, INT32_MAX};
  for (int j = lane; j < it.rows; j += 32) {
    const Keys k = keys_of_row(a, s, it.prefix, j0 + j);
    some = join(some, k);
    if (k.hi > 0) all = {max(all.lo, k.lo), min(all.hi, k.hi)};
  }
  it.lo = __reduce_min_sync(0xffffffffu, some.lo);
  it.hi = __reduce_max_sync(0xffffffffu, some.hi);
  it.all_lo = __reduce_max_sync(0xffffffffu, all.lo);
  it.all_hi = __reduce_min_sync(0xffffffffu, all.hi);
  return it;
}

// Reports the pages outside the pool among those of the keys [from, to), unless none of the sequence's `rows` rows from
// j0 on sees a key of such a page: where rows that see nothing lie between documents, the keys of a block of rows have
// gaps, and what stands in the table for a page in one must not be reported. By the whole block, at its end, and only
// where a producer met such a page (asked there, it cost 4 of 321 us of chunks whose tables are good).
static __device__ __noinline__ void report_pages(const BiasedArgs& a, int b, int c0, int q_len, int past, int prefix, int j0,
                                                 int rows, int from, int to) {
  Seq s;
  s.c0 = c0, s.q = q_len, s.past = past;
  for (int page = from / a.bs + (int)threadIdx.x; (int64_t)page * a.bs < to; page += (int)blockDim.x) {
    const int phys = a.table[(int64_t)b * a.max_blocks + page], v = page * a.bs;
    if (phys >= 0 && phys < a.num_blocks) continue;
    for (int j = j0 + rows - 1; j >= j0; --j) {  // (later rows mostly see more)
      const Keys k = keys_of_row(a, s, prefix, j);
      if (k.lo >= min(v + a.bs, to) || k.hi <= max(v, from)) continue;
      atomicOr(a.error, PA_DEVERR_BAD_BLOCK);
      break;
    }
  }
}

// N products q.k of a row as scores in powers of two, consecutive keys from v0 on: capped, less their
// distance's share (`slope` is minus the slope, `away` the distance of the first key; with `after` some keys may lie
// behind the row), plus `shift`. `level` says how the cap is taken: kNear and kMid, by polynomials in whose reach all
// scores are; kFar, by the exponential, 2^-21 of the cap off wherever a score is; kAny, each score by what suits it,
// for caps so large that this matters. 4 prompts of 2048 whose scores reach 0.1, 0.25, 0.4 and all of their cap take
// 638, 750, 784 and 920 us (848, 1204 and 3757 the last three where each score past 0.75 chose its form by a branch), 980 up to
// a cap of 170, and with kAny, at one of 200, 1500.
// On packed pairs: a score takes 2, 4 and 3 instruction slots and none, none and two more of the special function unit's,
// half a slot with a bias, where one score at a time took 13.
constexpr int kNear = 1, kMid = 2, kFar = 3, kAny = 4;
template <bool CAP, bool BIAS, int N>
__device__ __forceinline__ void bend_scores(const BiasedArgs& a, uint32_t* r, int level, float slope, float away, bool after,
                                            float shift) {
  auto pair = [&](int e) { return f2_make(__uint_as_float(r[e]), __uint_as_float(r[e + 1])); };
  auto put = [&](int e, uint64_t v) {
    float x, y;
    f2_split(v, x, y);
    r[e] = __float_as_uint(x), r[e + 1] = __float_as_uint(y);
  };
  const float scale = CAP ? a.scale_cap : a.scale_log2, cl = a.cap_log2;
  if (BIAS && unlikely(after)) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float x = __uint_as_float(r[e]) * scale;
      r[e] = __float_as_uint(fmaf(slope, fabsf(away - (float)e), CAP ? cl * tanh_of(x) : x) + shift);
    }
    return;
  }
  // without a key behind the row the bias is slope * away - slope * e, exact enough in this form: its
  // rounding, 2^-23 of the bias, only shows where the bias itself has not made the weight small
  const float base = fmaf(slope, away, shift);
  const uint64_t all = f2_make(base, base);
  uint64_t eight[4] = {};  // the bias of the eight keys from each eighth one on, and of that key
  if constexpr (BIAS) {
#pragma unroll
    for (int k = 0; k < 4; ++k) eight[k] = f2_make(-slope * (float)(2 * k), -slope * (float)(2 * k + 1));
  }
  uint64_t from = all;
  auto bias_of = [&](int e) {
    if constexpr (!BIAS) return all;
    if (e % 8 == 0) {
      const float x = fmaf(-slope, (float)e, base);
      from = f2_make(x, x);
    }
    return f2_add(eight[e % 8 / 2], from);
  };
  const uint64_t sc = f2_make(scale, scale);
  if constexpr (!CAP) {
#pragma unroll
    for (int e = 0; e < N; e += 2) put(e, f2_fma(pair(e), sc, bias_of(e)));
  } else if (likely(level == kNear)) {
    // cap * tanh(u) with u = scale * r as r times a polynomial in r^2 (for scales whose fifth power is
    // a normal number)
    const float s1 = cl * scale, s2 = scale * scale, s3 = s1 * s2, s5 = s3 * s2;
    const uint64_t c0 = f2_make(kTanh3[0] * s1, kTanh3[0] * s1), c1 = f2_make(kTanh3[1] * s3, kTanh3[1] * s3),
                   c2 = f2_make(kTanh3[2] * s5, kTanh3[2] * s5);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const uint64_t x = pair(e), z = f2_mul(x, x);
      put(e, f2_fma(f2_fma(f2_fma(c2, z, c1), z, c0), x, bias_of(e)));
    }
  } else if (level == kMid) {
    uint64_t k[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) k[i] = f2_make(kTanh6[i] * cl, kTanh6[i] * cl);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const uint64_t x = f2_mul(pair(e), sc), z = f2_mul(x, x);
      uint64_t y = k[5];
#pragma unroll
      for (int i = 4; i >= 0; --i) y = f2_fma(y, z, k[i]);
      put(e, f2_fma(y, x, bias_of(e)));
    }
  } else if (level == kFar) {
    const uint64_t twice = f2_make(scale * 2.8853900818f, scale * 2.8853900818f), one = f2_make(1.f, 1.f);
    const uint64_t less = f2_make(-2.f * cl, -2.f * cl), more = f2_make(cl, cl);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      float x, y;
      f2_split(f2_mul(pair(e), twice), x, y);
      f2_split(f2_add(f2_make(fast_exp2(x), fast_exp2(y)), one), x, y);
      put(e, f2_fma(f2_make(rcp_approx(x), rcp_approx(y)), less, f2_add(bias_of(e), more)));
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float x = cl * tanh_of(__uint_as_float(r[e]) * scale), y = cl * tanh_of(__uint_as_float(r[e + 1]) * scale);
      put(e, f2_add(f2_make(x, y), bias_of(e)));
    }
  }
}

// two weights as bf16 pairs hi + lo: hi their upper 16 bits as they are, lo the rest rounded, so that
// the sum is 2^-17 off at most
__device__ __forceinline__ void cut_bf16x2(uint64_t p, uint32_t& hi, uint32_t& lo) {
  float p0, p1;
  f2_split(p, p0, p1);
  hi = prmt(__float_as_uint(p0), __float_as_uint(p1), 0x7632u);
  float r0, r1;  // (minus the rest: 4 prompts of 2048 26 us faster than with the upper part masked out and added)
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; sub.rn.f32.bf16 %0, l, %3; sub.rn.f32.bf16 %1, h, %4;}"
      : "=f"(r0), "=f"(r1)
      : "r"(hi), "f"(p0), "f"(p1));
  lo = pack2<true>(r0, r1) ^ 0x80008000u;
}

// The weights 2^(r c + shift) (c is 1 where SCALED is not set, and the shift 0) of COLS scores, written to
// TMEM from column `p` on as the A operand of P V: fp16, or bf16 hi and lo terms. Returns their sum.
template <int COLS, bool BF16, bool SCALED>
__device__ __forceinline__ float weigh(uint32_t* r, float c, float shift, uint32_t p, int first_block) {
  const uint64_t c2 = f2_make(c, c), sh = f2_make(shift, shift);
  uint64_t sum = f2_make(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < COLS / 16; ++k) {
    uint32_t* q = r + k * 16;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float x0 = __uint_as_float(q[2 * e]), x1 = __uint_as_float(q[2 * e + 1]);
      if constexpr (SCALED) f2_split(f2_fma(f2_make(x0, x1), c2, sh), x0, x1);
      const uint64_t w = f2_make(fast_exp2(x0), fast_exp2(x1));
      sum = f2_add(sum, w);
      if constexpr (BF16) {
        cut_bf16x2(w, q[2 * e], q[2 * e + 1]);
      } else {
        f2_split(w, x0, x1);
        q[2 * e] = pack2<false>(x0, x1);
      }
    }
    const uint32_t at = p + p_col(first_block + k);
    tmem_st_x8_nowait(at, q[0], q[2], q[4], q[6], q[8], q[10], q[12], q[14]);
    if constexpr (BF16) tmem_st_x8_nowait(at + 16, q[1], q[3], q[5], q[7], q[9], q[11], q[13], q[15]);
  }
  float s0, s1;
  f2_split(sum, s0, s1);
  return s0 + s1;
}

__device__ __forceinline__ Keys keys_of_item_row(const BiasedArgs& a, const TileItem& it, int j) {
  Seq s;
  s.c0 = it.row0, s.past = it.pos0, s.q = it.total - it.pos0;  // (the item's rows counted from 0)
  return keys_of_row(a, s, it.prefix, j);
}

template <int HS, bool BF16, int RULES>
__global__ void __launch_bounds__(bi_threads(HS), HS == 256 ? 1 : 2)
    biased_tile_kernel(const __grid_constant__ BiasedArgs a, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const int seg_rows, const int sub_rows) {
  using L = BiTile<HS>;
  constexpr int HALVES = HS / 64, KSTEPS = HS / 16, SIDES = bi_sides(HS), THREADS = bi_threads(HS);
  constexpr uint32_t IDESC_QK = idesc_f16(BF16, 128, kBiTile, false), IDESC_PV = idesc_f16(BF16, 128, HS, true);
  constexpr uint32_t kO = 128;  // TMEM column of O
  // The row's reference m_used may lag behind its maximum by kLag before O is rescaled. fp16
  // weights are lifted by 2^kLift, to 2^15 at most, so that only those below 2^-22 of the reference
  // are subnormal and have absolute errors, of 2^-33; l is lifted with them.
  constexpr float kLag = BF16 ? 8.f : 7.f, kLift = BF16 ? 0.f : 8.f, kUnlift = BF16 ? 1.f : 1.f / 256;
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
  TileItem* item_s = reinterpret_cast<TileItem*>(smem + L::kItem);
  float* ml = reinterpret_cast<float*>(smem + L::kMl);
  float2* half = reinterpret_cast<float2*>(smem + L::kX);  // [2][128]
  uint32_t* redo = reinterpret_cast<uint32_t*>(smem + L::kRedo);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Later rows see more keys, so their items start first, those of all heads: 4 prompts of 2048 634 us instead of 670
  // with one head after the other, whose last CTAs leave SMs idle. (Sequences by length, too, make that 624, but 8
  // chunks and 24 decode rows 323 instead of 321 and one chunk and 7 decode rows 69 instead of 65.)
  const int i = gridDim.x - 1 - blockIdx.x, g = i % a.kvh, u = i / a.kvh;
  const int rank = blockIdx.z, C = gridDim.z;  // the cluster is a column of the grid
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
      mbar_init(&p_full[i], 128 * SIDES);
      mbar_init(&o_done[i], 1);
    }
    *abort = 0;
    *err = 0;
    for (int i = 0; i < 5; ++i) redo[i] = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();  // (the rows kernel starts when the last CTA has: beside the tiles that are left)
  if (warp == 0) {
    const TileItem it = tile_item(a, u, sub_rows, lane);
    if (lane == 0) *item_s = it;
  }
  if (i == 0 && rank == 0) check_biased_batch(a);
  __syncthreads();
  const TileItem it = *item_s;
  if (it.rows <= 0) return;  // (all CTAs of a cluster agree)
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int2 tiles = tiles_of(Keys{it.lo, it.hi});
  const int t0 = tiles.x + (int)((int64_t)(tiles.y - tiles.x) * rank / C);
  const int n = tiles.x + (int)((int64_t)(tiles.y - tiles.x) * (rank + 1) / C) - t0;
  // Tiles are taken from the last to the first: with a bias the near keys' scores are the large ones, and
  // in this order a row's maximum is there from the beginning (in the other it grows with every tile,
  // and O is rescaled with it: 4 prompts of 2048 with everything 1031 us instead of 760).
  const int last = t0 + n - 1;

  const int row = (warp & 3) * 32 + lane;  // (softmax warps) the thread's TMEM lane
  const int side = SIDES == 2 && warp >= 6;  // and, where two threads share a row, its half of the columns
  const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
  const int j = row / a.G;                  // its row in the item
  const bool live = warp >= 2 && j < it.rows && row < sub_rows * a.G;
  const bool any_live = __any_sync(0xffffffffu, live);
  float m_used = -INFINITY, l = 0.f;

  if (warp == 0) {
    // ---- producer ----
    if (n > 0) {
      const int nseg = kBiTile / seg_rows, oob = a.num_blocks * a.bs;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, (uint32_t)(sub_rows * a.G * HS * 2));
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
          tma_load_3d(smem + h * 128 * 128, &tmQ, q_full, h * 64, g * a.G, it.row0);
      }
      const int* table = a.table + (int64_t)it.b * a.max_blocks;
      auto slot = [&](int t) {  // this lane's segment of tile t: its first cache row
        const int v = (last - t) * kBiTile + lane * seg_rows;
        if (lane >= nseg || t >= n || v >= it.hi || v + seg_rows <= it.lo) return oob;
        const int page = v / a.bs, phys = table[page];
        if (unlikely(phys < 0 || phys >= a.num_blocks)) {
          redo[4] = 1;
          return oob;
        }
        return phys * a.bs + (v - page * a.bs);
      };
      auto load = [&](int t, int z, const CUtensorMap* map, uint64_t* full, uint64_t* empty, uint8_t* ring) {
        if (t < 0 || t >= n) return;
        const int s = t % L::kStages;
        if (lane == 0) {
          mbar_wait(&empty[s], ((t / L::kStages) & 1) ^ 1, abort, err);
          mbar_arrive_expect_tx(&full[s], L::kTileBytes);
        }
        __syncwarp();
        if (lane < nseg)
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
            tma_load_3d(ring + s * L::kTileBytes + h * kBiTile * 128 + lane * seg_rows * 128, map, &full[s], h * 64, g, z);
        __syncwarp();
      };
      // tiles are asked for in the order in which the products free their stages: K_{t+2} (after
      // Q K_t) before V_{t+1} (after P V_{t-1}); a tile's pages are looked up a step before
      int z1 = oob, z2 = slot(0);  // of tiles t + 1 and t + 2
      for (int t = -2; t < n; ++t) {
        const int z3 = slot(t + 3);
        load(t + 2, z2, &tmK, k_full, k_empty, smem + L::kRing);
        load(t + 1, z1, &tmV, v_full, v_empty, smem + L::kRing + L::kStages * L::kTileBytes);
        z1 = z2;
        z2 = z3;
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer ----
    const uint64_t qdesc = sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t kdesc = sdesc_sw128(smem_u32(smem + L::kRing), 16, 1024);
    const uint64_t vdesc = sdesc_sw128(smem_u32(smem + L::kRing + L::kStages * L::kTileBytes), kBiTile * 128, 1024);
    auto issue_qk = [&](int t) {
      const int s = t % L::kStages;
      mbar_wait(&k_full[s], (t / L::kStages) & 1, abort, err);
      tc_fence_after();
      if (elect_one()) {
        const uint64_t kd = kdesc + (uint64_t)((s * L::kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < KSTEPS; ++kk)
          tc_mma_ss(tmem + (t & 1) * kBiTile, qdesc + (uint64_t)((kk >> 2) * (128 * 128 >> 4) + (kk & 3) * 2),
                    kd + (uint64_t)((kk >> 2) * (kBiTile * 128 >> 4) + (kk & 3) * 2), IDESC_QK, kk > 0 ? 1u : 0u);
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
      // rows that no row of the item sees may be unwritten: cleared, so that no NaN meets a
      // weight of 0 (whole 128-byte rows: the swizzle stays inside)
      const int k0 = (last - t) * kBiTile, front = max(it.lo - k0, 0), back = min(it.hi - k0, kBiTile);
      if (front > 0 || back < kBiTile) {
        uint8_t* vt = smem + L::kRing + (L::kStages + s) * L::kTileBytes;
        const int rows = front + kBiTile - back;
        for (int c = lane; c < rows * 8 * HALVES; c += 32) {
          const int r = c % (rows * 8) / 8;
          *reinterpret_cast<uint4*>(vt + c / (rows * 8) * (kBiTile * 128) + (r < front ? r : back + r - front) * 128 +
                                    c % 8 * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      mbar_wait(&p_full[t & 1], (t >> 1) & 1, abort, err);
      __syncwarp();
      tc_fence_after();
      if (elect_one()) {
        const uint64_t vd = vdesc + (uint64_t)((s * L::kTileBytes) >> 4);
        const uint32_t p = tmem + (t & 1) * kBiTile;
#pragma unroll
        for (int kk = 0; kk < kBiTile / 16; ++kk) {
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
    constexpr int COLS = kBiTile / SIDES, OCOLS = HS / SIDES;
    const int jc = min(j, it.rows - 1), h = g * a.G + min(row % a.G, a.G - 1);  // (rows past the item borrow the last row's keys)
    const Keys keys = keys_of_item_row(a, it, jc);
    const bool seeing = keys.hi > 0;  // (a row without keys is worked on as its neighbours, its result dropped)
    const bool works = live && seeing;
    const int pos = it.pos0 + jc;
    constexpr bool cap = RULES & 1, bias = RULES & 2, bent = cap || bias;
    const float span = fabsf(a.scale_cap);
    // the polynomial's coefficients hold; and kFar's error, 2^-21 of the cap, is 2^-13 of a power of two at most
    const bool short_form = span > 1e-6f && span < 1e6f && a.cap_log2 < 1e6f, far_form = a.cap_log2 <= 256.f;
    const float slope = bias ? -a.slopes[h] * 1.4426950408889634f : 0.f;
    const float c = bent ? 1.f : a.scale_log2;  // what the scores below are still multiplied by
    const float none = c > 0.f ? -INFINITY : INFINITY;  // a score whose product with c is -inf
    const uint32_t o_tmem = tmem + lane_off + kO + side * OCOLS;
    [[maybe_unused]] const int bar = 1 + (warp & 3);  // of the two warps of a lane quarter
    for (int t = 0; t < n; ++t) {
      mbar_wait(&s_full[t & 1], (t >> 1) & 1, abort, err);
      if (!any_live) {  // rows past the item: whatever their P holds stays in their rows of O
        mbar_arrive(&p_full[t & 1]);
        continue;
      }
      tc_fence_after();
      const uint32_t st = tmem + lane_off + (t & 1) * kBiTile;
      uint32_t r[COLS];
      const float most = tmem_ld_max<COLS, bent>(st + side * COLS, r);
      const int v0 = (last - t) * kBiTile + side * COLS;
      // With a cap or a bias the scores are bent first. The largest |q.k| of the row's keys tells how far
      // the cap bends them and bounds the scores from above, so that a maximum is only looked for where
      // the bound is over what the row's reference may lag behind; else the reference goes into the
      // bend (where two threads share a row they would have to agree: there it is always looked for).
      bool find_max = true;
      if constexpr (bent) {
        const float u = most * fabsf(cap ? a.scale_cap : a.scale_log2), away = (float)(pos - v0);
        float top = u;
        int level = 0;
        if (cap) {
          // (rows past the item may hold anything)
          const bool near = __all_sync(0xffffffffu, u <= kTanhNear || !works);
          level = near && short_form                                      ? kNear
                  : __all_sync(0xffffffffu, u <= kTanhMid || !works) ? kMid
                  : far_form                                         ? kFar
                                                                     : kAny;
          top = a.cap_log2 * fminf(u, 1.f);
        }
        const bool after = v0 + COLS > it.pos0 && it.prefix > it.pos0;
        if constexpr (SIDES == 1) {
          // (the bias of the nearest or farthest key, whichever is more; a key behind the row may be as near as 0)
          const float far = after ? fmaxf(fabsf(away), fabsf(away - (COLS - 1))) : away;
          top += fmaxf(slope * far, slope * (after ? 0.f : fmaxf(away - (COLS - 1), 0.f)));
          find_max = __any_sync(0xffffffffu, works && !(top <= m_used + kLag));
        }
        const float shift = find_max || m_used == -INFINITY ? 0.f : kLift - m_used;
        // The common cases by themselves, and in halves, the second loaded again when the first is done: with half
        // of the registers the compiler finds a better order (4 prompts of 2048 667 us instead of 698; kMid 764
        // instead of 863; kFar too: 920 instead of 985, but 20 us more for the others).
        auto by_halves = [&](int lv) {
#pragma unroll
          for (int k = 0; k < COLS / 32; ++k) {
            uint32_t* x = r + 32 * k;
            if (k) tmem_ld_x32(st + 32 * k, x);
            bend_scores<cap, bias, 32>(a, x, lv, slope, away - (float)(32 * k), false, shift);
            l += weigh<32, BF16, false>(x, 1.f, 0.f, st, 2 * k);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&p_full[t & 1]);
        };
        if (SIDES == 1 && !find_max && !after && level < kAny && v0 >= it.all_lo && v0 + COLS <= it.all_hi) {
          if (!cap || level == kNear) {
            by_halves(kNear);
            continue;
          }
          if (level == kMid) {
            by_halves(kMid);
            continue;
          }
        }
        bend_scores<cap, bias, COLS>(a, r, level, slope, away, after, shift);
      }
      // (v0 and the bounds of all rows are the warp's: most tiles need neither side, few need both)
      if (unlikely(v0 < it.all_lo)) {
        const int lo = keys.lo - v0;
#pragma unroll
        for (int e = 0; e < COLS; ++e)
          if (e < lo) r[e] = __float_as_uint(none);
      }
      if (unlikely(v0 + COLS > it.all_hi)) {
        const int hi = keys.hi - v0;
#pragma unroll
        for (int e = 0; e < COLS; ++e)
          if (e >= hi) r[e] = __float_as_uint(none);
      }
      bool grow = false;
      float alpha = 1.f;
      if (find_max) {
        float mc[4] = {none, none, none, none};
        if (!bent && c > 0.f && v0 >= it.all_lo && v0 + COLS <= it.all_hi) {  // (the tile's keys are all rows')
          mc[0] = most;
        } else if (c > 0.f) {
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
        float m_new = fmaxf(m_used, best * c);
        if constexpr (SIDES == 2) {
          float2* hx = half + (t & 1) * 128 + row;
          (side ? hx->y : hx->x) = best * c;
          named_bar_sync(bar, 64);
          const float2 both = *hx;
          m_new = fmaxf(m_used, fmaxf(both.x, both.y));
        }
        grow = __any_sync(0xffffffffu, works && m_new > m_used + kLag);
        if (unlikely(grow)) {
          // (fp16: a whole number, which kLift is taken off exactly)
          const float to = BF16 ? m_new : ceilf(m_new);
          alpha = m_new == -INFINITY ? 1.f : fast_exp2(m_used - to);  // 0 on a row's first keys
          m_used = to;
          l *= alpha;
        }
        const float neg_m = m_used == -INFINITY ? 0.f : kLift - m_used;  // (no key yet: every weight is 0)
        l += weigh<COLS, BF16, true>(r, c, neg_m, st, side * (COLS / 16));
      } else {
        l += weigh<COLS, BF16, false>(r, 1.f, 0.f, st, 0);
      }
      if (unlikely(t > 0 && grow)) {  // O holds P_0 V .. P_{t-1} V once the last product is done
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
    if constexpr (SIDES == 2) {  // the row's sum from its halves (the two warps have the same maximum)
      (side ? half[row].y : half[row].x) = l;
      named_bar_sync(bar, 64);
      l = half[row].x + half[row].y;
    }
    if (m_used == -INFINITY && l != l) m_used = 0.f;  // scores of NaN alone: not a row without keys
    if (!seeing) m_used = -INFINITY, l = 0.f;
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
      for (int cc = side * (HS / SIDES); cc < (side + 1) * (HS / SIDES); cc += 32) {
        uint32_t ov[32];
        if (n > 0) {
          tmem_ld_x32(tmem + lane_off + kO + cc, ov);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = 0u;
        }
        if (live) {
          const bool some = m_used != -INFINITY;
          bool fine = true;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            fine = fine && finite4(__uint_as_float(ov[e]) * inv, __uint_as_float(ov[e + 1]) * inv,
                                   __uint_as_float(ov[e + 2]) * inv, __uint_as_float(ov[e + 3]) * inv);
          if (some && !fine && l == l) atomicOr(&redo[row >> 5], 1u << (row & 31));
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = some ? pack_sat<BF16>(__uint_as_float(ov[e + 2 * k]) * inv, __uint_as_float(ov[e + 2 * k + 1]) * inv) : 0u;
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
      for (int cc = side * (HS / SIDES); any_live && cc < (side + 1) * (HS / SIDES); cc += 32) {
        uint32_t ov[32];
        if (n > 0) tmem_ld_x32(tmem + lane_off + kO + cc, ov);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (n > 0 && m_used != -INFINITY)  // (a factor that is 0 in 32 bits makes NaN of an infinity: redo_row's)
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
    for (int i = threadIdx.x; i < (r1 - r0) * (HS / 4); i += THREADS) {
      const int r = r0 + i / (HS / 4), quad = i % (HS / 4);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < C; ++k) {
        const float4 y = ld_cluster4(cluster_addr(part + r * HS + (quad + r) % (HS / 4) * 4, k));
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      const int64_t at = (int64_t)(it.row0 + r / a.G) * a.nh + g * a.G + r % a.G;
      *reinterpret_cast<uint2*>(out + at * HS + quad * 4) = make_uint2(pack_sat<BF16>(x.x, x.y), pack_sat<BF16>(x.z, x.w));
      if (!finite4(x.x, x.y, x.z, x.w)) {
        bool lost = false;  // (a sum of weights that is NaN makes the row so)
        for (int k = 0; k < C; ++k) {
          const float sum = ld_cluster(cluster_addr(ml + 128 + r, k));
          lost = lost || sum != sum;
        }
        if (!lost) atomicOr(&redo[r >> 5], 1u << (r & 31));
      }
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }
  tc_fence_before();
  __syncthreads();  // (no warp waits any more: whichever gave up has said so)
  if (threadIdx.x == 0 && *err && a.error) atomicOr(a.error, *err);
  if (redo[4] && a.error)
    report_pages(a, it.b, it.row0, it.total - it.pos0, it.pos0, it.prefix, 0, it.rows, max(t0 * kBiTile, it.lo),
                 min((t0 + n) * kBiTile, it.hi));
  if (redo[0] | redo[1] | redo[2] | redo[3])
    for (int r = warp; r < it.rows * a.G; r += THREADS / 32)
      if (redo[r >> 5] >> (r & 31) & 1)  // (the item's rows counted from 0)
        redo_row<HS, BF16>(a, it.b, it.row0, it.total - it.pos0, it.pos0, r / a.G, g * a.G + r % a.G, lane, 0, HS);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
}

// The CTAs of a cluster share an item's tiles, as many as run at once.
template <int HS, bool BF16, int RULES>
static cudaError_t launch_biased_tile_of(const BiasedArgs& a, const CUtensorMap& tq, const CUtensorMap& tk,
                                         const CUtensorMap& tv, int seg, int sub_rows, int sms, cudaStream_t s) {
  const int64_t keys = keys_in_reach(a, sub_rows);
  const int64_t items = items_of_batch(a.N, a.B, sub_rows, 1, 1) * a.kvh;
  const int c = cluster_size(items, (int64_t)sms * (HS == 256 ? 1 : 2), ceil_div(keys, kBiTile), 4, 8);
  const dim3 grid((unsigned)((a.N / sub_rows + a.B) * a.kvh), 1, (unsigned)c);
  return launch_clusters(biased_tile_kernel<HS, BF16, RULES>, grid, bi_threads(HS), BiTile<HS>::kBytes, BiTile<HS>::kBytes, s,
                         a, tq, tk, tv, seg, sub_rows);
}

template <bool BF16>
static cudaError_t launch_biased_tile(const BiasedArgs& a, const CUtensorMap& tq, const CUtensorMap& tk,
                                      const CUtensorMap& tv, int seg, int sub_rows, int sms, cudaStream_t s) {
  const int rules = (a.cap_log2 != 0.f ? 1 : 0) + (a.slopes ? 2 : 0);
#define PA_TILE(HS, R) launch_biased_tile_of<HS, BF16, R>(a, tq, tk, tv, seg, sub_rows, sms, s)
#define PA_RULES(HS) (rules == 0 ? PA_TILE(HS, 0) : rules == 1 ? PA_TILE(HS, 1) : rules == 2 ? PA_TILE(HS, 2) : PA_TILE(HS, 3))
  return a.hs == 64 ? PA_RULES(64) : a.hs == 128 ? PA_RULES(128) : PA_RULES(256);
#undef PA_RULES
#undef PA_TILE
}

}  // namespace pa
