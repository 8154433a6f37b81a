// RMSNorm of every query and key head, then the rotary embedding, in one pass over the rows.
//
// A head x of HS values at position p becomes y_c = x_c / sqrt(mean x^2 + eps) * w_c (with a
// weight), then its first d = rotary_dim values are turned pairwise by the angles
// a_u = fl32(fl32(p) * fl32(theta^(-2u/d))), pairs (u, u + d/2) or, interleaved, (2u, 2u + 1);
// computed in fp32 and rounded once to T (the preparation that paged_attention can run before
// its cache write, here for rows that stay in tensors).
//
// Bytes bound it: every value is read once and written once. A head takes HS / 8 lanes, 16
// bytes each, so a warp takes 256 / HS heads a step; a lane keeps the same channels at every
// step, so sines, cosines and weights stay in registers over all heads of a row: the two
// lanes of a pair of halves compute four of their eight common angles each and exchange
// them. The arithmetic (about 60 instructions for a warp's 512 bytes) runs on packed pairs to
// stay below the bytes: 8001 rows of 16 + 2 heads of 256 take 29 us (147 MB, 5.1 TB/s; four steps
// in flight at seven blocks an SM; six or eight steps 32 us, two 34 to 38 us). Few rows are shared by several warps (`split`), each with some of the
// heads, so that a decode batch is not one warp's chain of steps.
#include "ops.cuh"

namespace pa {

constexpr int kRotThreads = 128;

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& w, uint64_t (&x)[4]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      x[i] = f2_make(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xFFFF0000u));
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
      x[i] = f2_make(f.x, f.y);
    }
  }
}

// Sine and cosine of a fp32 angle below 2^31, within about 2^-22: the angle in turns from the exact
// product with 1 / 2 pi in three parts (a product and its error by fma), whole turns taken off
// each part (exact), the rest summed from its smallest part. One path for every position.
__device__ __forceinline__ void sin_cos(float x, float* s, float* c) {
  constexpr float kHi = 0x1.45f3060000000p-3f, kLo = 0x1.b939100000000p-28f, kLo2 = 0x1.529fc20000000p-54f;  // 1 / 2 pi
  const float p = __fmul_rn(x, kHi), e = fmaf(x, kHi, -p), q = __fmul_rn(x, kLo), f = fmaf(x, kLo, -q);
  const float r = (p - rintf(p)) + ((e - rintf(e)) + ((q - rintf(q)) + fmaf(x, kLo2, f)));
  sincospif(2.f * r, s, c);
}

// what a lane holds for a row: x_c becomes x_c cs_c + x_partner sn_c (the sign of a pair's first
// value folded into sn)
struct Turn {
  uint64_t cs[4], sn[4];
  int partner;  // the lane with the other values of this lane's pairs
  bool on;
};

constexpr int kRotSteps = 4;  // steps in flight

// this lane's pieces of steps s .. s + kRotSteps - 1 (below s1) of one input's heads (H a step)
template <int HS>
__device__ __forceinline__ void load_steps(uint4 (&v)[kRotSteps], const uint16_t* src, int heads, int s, int s1,
                                           int lane) {
  constexpr int L = HS / 8, H = 32 / L;
#pragma unroll
  for (int u = 0; u < kRotSteps; ++u) {
    const int h = (s + u) * H + lane / L;
    v[u] = s + u < s1 && h < heads ? *(reinterpret_cast<const uint4*>(src + (int64_t)h * HS) + lane % L)
                                   : make_uint4(0, 0, 0, 0);
  }
}

// Steps [s0, s1) of one input's heads.
template <int HS, bool BF16, bool INTER>
__device__ __forceinline__ void rotate_heads(const uint16_t* src, uint16_t* dst, int heads, int s0, int s1,
                                             const uint16_t* weight, float eps, const Turn& t, bool any_turn, int lane) {
  constexpr int L = HS / 8, H = 32 / L, U = kRotSteps;
  const int l = lane % L, sub = lane / L;
  uint64_t w[4];
  if (weight) unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(weight) + l), w);
  for (int s = s0; s < s1; s += U) {
    uint4 v[U];
    load_steps<HS>(v, src, heads, s, s1, lane);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= s1) break;
      const int h = (s + u) * H + sub;
      uint64_t x[4];
      unpack8<BF16>(v[u], x);
      if (weight) {
        uint64_t ss2 = f2_make(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) ss2 = f2_fma(x[i], x[i], ss2);
        float s0f, s1f;
        f2_split(ss2, s0f, s1f);
        float ss = s0f + s1f;
#pragma unroll
        for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(fmaf(ss, 1.f / HS, eps));  // (2^-22.9 off at most)
        const uint64_t r2 = f2_make(r, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f2_mul(f2_mul(x[i], r2), w[i]);
      }
      if (any_turn) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a, b;
          f2_split(x[i], a, b);
          const uint64_t o = INTER ? f2_make(b, a)
                                   : f2_make(__shfl_sync(0xffffffffu, a, t.partner), __shfl_sync(0xffffffffu, b, t.partner));
          const uint64_t y = f2_fma(o, t.sn[i], f2_mul(x[i], t.cs[i]));
          x[i] = t.on ? y : x[i];
        }
      }
      if (h < heads) {
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a, b;
          f2_split(x[i], a, b);
          out[i] = pack2<BF16>(a, b);
        }
        *(reinterpret_cast<uint4*>(dst + (int64_t)h * HS) + l) = make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
  }
}

template <int HS, bool BF16, bool INTER>
__global__ void __launch_bounds__(kRotThreads, 7) rotate_kernel(const RotateArgs a) {
  constexpr int L = HS / 8, H = 32 / L;
  const int lane = threadIdx.x & 31, l = lane % L;
  const int64_t w = (int64_t)blockIdx.x * (kRotThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = w / a.split;
  const int part = (int)(w % a.split);
  pdl_wait();
  pdl_launch_dependents();
  if (row >= a.N) return;
  const int qs = (a.nh + H - 1) / H, steps = qs + (a.kvh + H - 1) / H;
  const int s0 = (int)((int64_t)steps * part / a.split), s1 = (int)((int64_t)steps * (part + 1) / a.split);
  const uint16_t *q = a.query + row * a.q_stride, *k = a.key + row * a.k_stride;
  const int pos = a.positions[row];
  if (pos < 0) return;  // a row of no sequence: left as it is
  const int d = a.rotary_dim, half = d / 2;
  Turn t;
  t.on = 8 * l < d;
  const bool lower = 8 * l < half;
  t.partner = INTER || !t.on ? lane : lower ? lane + d / 16 : lane - d / 16;
  if (d > 0) {
    // four angles: of this lane's pairs (interleaved), or of half of the eight it shares
    float sn[4], cs[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int u = INTER ? 4 * l + e : lower ? 8 * l + e : 8 * l - half + 4 + e;
      sin_cos((float)pos * a.inv_freq[t.on ? u : 0], &sn[e], &cs[e]);
    }
    if constexpr (INTER) {
#pragma unroll
      for (int e = 0; e < 4; ++e) t.cs[e] = f2_make(cs[e], cs[e]), t.sn[e] = f2_make(-sn[e], sn[e]);
    } else {
      float c8[8], s8[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float co = __shfl_sync(0xffffffffu, cs[e], t.partner), so = __shfl_sync(0xffffffffu, sn[e], t.partner);
        c8[e] = lower ? cs[e] : co, c8[4 + e] = lower ? co : cs[e];
        s8[e] = lower ? -sn[e] : so, s8[4 + e] = lower ? -so : sn[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) t.cs[e] = f2_make(c8[2 * e], c8[2 * e + 1]), t.sn[e] = f2_make(s8[2 * e], s8[2 * e + 1]);
    }
  }
  rotate_heads<HS, BF16, INTER>(q, a.query_out + row * a.qo_stride, a.nh, min(s0, qs), min(s1, qs), a.q_weight, a.eps, t,
                                d > 0, lane);
  rotate_heads<HS, BF16, INTER>(k, a.key_out + row * a.ko_stride, a.kvh, max(s0 - qs, 0), max(s1 - qs, 0), a.k_weight,
                                a.eps, t, d > 0, lane);
}

template <int HS>
static cudaError_t launch_rotate_t(RotateArgs a, bool bf16, int sms, cudaStream_t s) {
  // warps per row: enough that the launch has about 16 warps an SM, at most one per step (each
  // computes the row's angles: 8001 rows take 4 us more with two warps each, 64 rows 0.9 us less
  // with twenty than with five)
  const int steps = (int)(ceil_div(a.nh, 256 / HS) + ceil_div(a.kvh, 256 / HS));
  const int64_t want = ceil_div((int64_t)16 * sms, a.N);
  a.split = (int)(want < 1 ? 1 : want > steps ? steps : want);
  const int64_t grid = ceil_div((int64_t)a.N * a.split, kRotThreads / 32);
  auto kernel = bf16 ? (a.interleaved ? rotate_kernel<HS, true, true> : rotate_kernel<HS, true, false>)
                     : (a.interleaved ? rotate_kernel<HS, false, true> : rotate_kernel<HS, false, false>);
  return launch_pdl(kernel, dim3((unsigned)grid), dim3(kRotThreads), 0, s, a);
}

cudaError_t launch_rotate(const RotateArgs& a, bool bf16, int hs, int sms, cudaStream_t s) {
  if (hs == 64) return launch_rotate_t<64>(a, bf16, sms, s);
  if (hs == 128) return launch_rotate_t<128>(a, bf16, sms, s);
  return launch_rotate_t<256>(a, bf16, sms, s);
}

}  // namespace pa
