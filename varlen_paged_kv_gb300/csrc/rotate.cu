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
// step, so it computes its eight sines and cosines once per row and holds them, and the
// weights, in registers over all heads. Few rows are shared by several warps (`split`), each
// with some of the heads, so that a decode batch is not one warp's chain of steps.
#include "ops.cuh"

namespace pa {

constexpr int kRotThreads = 128;

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <int HS, bool BF16>
__global__ void __launch_bounds__(kRotThreads) rotate_kernel(const RotateArgs a) {
  constexpr int L = HS / 8;      // lanes per head
  constexpr int H = 32 / L;      // heads per warp and step
  constexpr int U = 4;           // steps in flight
  const int lane = threadIdx.x & 31, l = lane % L;
  const int64_t w = (int64_t)blockIdx.x * (kRotThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = w / a.split;
  const int part = (int)(w % a.split);
  if (row >= a.N) return;
  const int pos = a.positions[row];
  if (pos < 0) return;  // a row of no sequence: left as it is
  const int d = a.rotary_dim, half = d / 2;
  const bool rot = 8 * l < d, lower = 8 * l < half;
  float cs[8], sn[8];
  if (rot) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (a.interleaved && (e & 1)) {
        cs[e] = cs[e - 1], sn[e] = sn[e - 1];
      } else {
        const int c = 8 * l + e, u = a.interleaved ? c / 2 : lower ? c : c - half;
        sincosf((float)pos * a.inv_freq[u], &sn[e], &cs[e]);
      }
    }
    // the first value of a pair subtracts its partner's share
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (a.interleaved ? !(e & 1) : lower) sn[e] = -sn[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f;
  }
  // the lane with the other half of this lane's pairs
  const int partner = a.interleaved || !rot ? lane : lower ? lane + d / 16 : lane - d / 16;
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (a.q_weight) wq = __ldg(reinterpret_cast<const uint4*>(a.q_weight) + l);
  if (a.k_weight) wk = __ldg(reinterpret_cast<const uint4*>(a.k_weight) + l);
  const int heads = a.nh + a.kvh, steps = (heads + H - 1) / H;
  const int s0 = (int)((int64_t)steps * part / a.split), s1 = (int)((int64_t)steps * (part + 1) / a.split);
  for (int s = s0; s < s1; s += U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (s + u) * H + lane / L;
      if (s + u < s1 && h < heads) {
        const uint16_t* src = h < a.nh ? a.query + row * a.q_stride + (int64_t)h * HS
                                       : a.key + row * a.k_stride + (int64_t)(h - a.nh) * HS;
        v[u] = *(reinterpret_cast<const uint4*>(src) + l);
      } else {
        v[u] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= s1) break;
      const int h = (s + u) * H + lane / L;
      const bool is_q = h < a.nh;
      float x[8];
      unpack8<BF16>(v[u], x);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (is_q ? a.q_weight != nullptr : a.k_weight != nullptr) {
        const float r = 1.f / sqrtf(ss * (1.f / HS) + a.eps);
        float g[8];
        unpack8<BF16>(is_q ? wq : wk, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * r * g[e];
      }
      float y[8];
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = rot ? x[e] * cs[e] + x[e ^ 1] * sn[e] : x[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float o = __shfl_sync(0xffffffffu, x[e], partner);
          y[e] = rot ? x[e] * cs[e] + o * sn[e] : x[e];
        }
      }
      if (h < heads) {
        uint16_t* dst = is_q ? a.query_out + row * a.qo_stride + (int64_t)h * HS
                             : a.key_out + row * a.ko_stride + (int64_t)(h - a.nh) * HS;
        *(reinterpret_cast<uint4*>(dst) + l) = make_uint4(pack2<BF16>(y[0], y[1]), pack2<BF16>(y[2], y[3]),
                                                          pack2<BF16>(y[4], y[5]), pack2<BF16>(y[6], y[7]));
      }
    }
  }
}

template <int HS>
static cudaError_t launch_rotate_t(RotateArgs a, bool bf16, int sms, cudaStream_t s) {
  // warps per row: enough that the launch has about 16 warps an SM, at most one per step
  const int steps = (int)ceil_div(a.nh + a.kvh, 256 / HS);
  const int64_t want = ceil_div((int64_t)16 * sms, a.N);
  a.split = (int)(want < 1 ? 1 : want > steps ? steps : want);
  const int64_t grid = ceil_div((int64_t)a.N * a.split, kRotThreads / 32);
  if (bf16) rotate_kernel<HS, true><<<(unsigned)grid, kRotThreads, 0, s>>>(a);
  else rotate_kernel<HS, false><<<(unsigned)grid, kRotThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_rotate(const RotateArgs& a, bool bf16, int hs, int sms, cudaStream_t s) {
  if (hs == 64) return launch_rotate_t<64>(a, bf16, sms, s);
  if (hs == 128) return launch_rotate_t<128>(a, bf16, sms, s);
  return launch_rotate_t<256>(a, bf16, sms, s);
}

}  // namespace pa
