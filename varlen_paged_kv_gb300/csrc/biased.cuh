// What the kernels of the biased attention share: the scores' cap, the rows' keys, and rows that are
// computed again because their result is not finite.
#pragma once

#include "ops.cuh"

namespace pa {

constexpr int kBiTile = 64;          // keys per tile

// (where the compiler lays the rarer path out of line: the softmax's code is long, and what it jumps
// over costs fetches)
__device__ __forceinline__ bool likely(bool x) { return __builtin_expect(x, 1); }
__device__ __forceinline__ bool unlikely(bool x) { return __builtin_expect(x, 0); }

// ---- scores --------------------------------------------------------------------------------
// tanh as u times a polynomial in u^2 (minimax by weighted least squares on 4000 Chebyshev points) up to
// |u| = 0.25, 4.9e-8 off at most (with six terms up to 0.75, 9.5e-9), beyond that from the exponential,
// 1 - 2 / (1 + e^2u), 2^-21 off at most (an exponential, a sum, a reciprocal, a rounding); the instruction
// tanh.approx is 5e-4 off, which a cap of 50 would turn into scores 0.02 off.
constexpr float kTanhNear = 0.25f, kTanhMid = 0.75f;
__device__ constexpr float kTanh3[3] = {0.99999863f, -0.33315702f, 0.12762232f};
__device__ constexpr float kTanh6[6] = {0.99999983f, -0.33332471f, 0.1332058f, -0.05314926f, 0.01923724f, -0.00449346f};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float tanh_of(float u) {
  const float z = u * u, near = u * fmaf(fmaf(kTanh3[2], z, kTanh3[1]), z, kTanh3[0]);
  const float far = copysignf(1.f - 2.f * rcp_approx(1.f + fast_exp2(fabsf(u) * 2.8853900818f)), u);
  return fabsf(u) <= kTanhNear ? near : far;
}

// ---- ranges --------------------------------------------------------------------------------
struct Keys {
  int lo, hi;  // (lo >= hi: none, then lo = INT32_MAX and hi = 0)
};
__device__ __forceinline__ Keys keys_of_row(const BiasedArgs& a, const Seq& s, int prefix, int j) {
  const int p = s.past + j;
  Keys k;
  k.lo = a.first ? max(a.first[s.c0 + j], 0) : 0;
  if (a.window) k.lo = max(k.lo, p - a.window + 1);
  k.hi = min(max(p + 1, prefix), s.past + s.q);
  if (k.lo >= k.hi) k.lo = INT32_MAX, k.hi = 0;
  return k;
}
__device__ __forceinline__ Keys join(Keys x, Keys y) { return {min(x.lo, y.lo), max(x.hi, y.hi)}; }

__device__ __forceinline__ Seq seq_at(const BiasedArgs& a, int b) {
  Seq s = make_seq(b, a.cum[b], a.cum[b + 1], a.past[b], a.N, a.max_blocks, a.bs);
  s.ok = s.ok && (a.max_rows == 0 || s.q <= a.max_rows);
  return s;
}
// whether a sequence is the rows kernel's
__device__ __forceinline__ bool short_rows(const BiasedArgs& a, const Seq& s) {
  return s.ok && s.q > 0 && (a.G > 128 || (int64_t)s.q * a.G <= 16);
}

// the checks of the whole batch, by one CTA
__device__ __forceinline__ void check_biased_batch(const BiasedArgs& a) {
  if (!a.error) return;
  bool bad = threadIdx.x == 0 && a.cum[0] != 0;
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) bad |= !seq_at(a, b).ok;
  if (bad) atomicOr(a.error, PA_DEVERR_BAD_BATCH);
}

// ---- results ---------------------------------------------------------------------------------
// Two results as T. The fp16 weights were rounded on their way into P V and their sum was not, so a mean of values near
// 65504 may come out up to 2^-11 above it, where fp16 rounds to infinity: what is finite stays so.
template <bool BF16>
__device__ __forceinline__ uint32_t pack_out(float x, float y) {
  if constexpr (!BF16) {
    constexpr float top = 65504.f;
    if (fabsf(x) < INFINITY) x = fminf(fmaxf(x, -top), top);
    if (fabsf(y) < INFINITY) y = fminf(fmaxf(y, -top), top);
  }
  return pack2<BF16>(x, y);
}

// The same by the conversion alone, which holds infinities too: for rows that are computed again where they are not
// finite (one instruction for two results; 8 chunks and 24 decode rows 320 us, by pack_out 329).
template <bool BF16>
__device__ __forceinline__ uint32_t pack_sat(float x, float y) {
  if constexpr (BF16) return pack2<true>(x, y);
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
  return d;
}

// ---- rows whose result is not finite ---------------------------------------------------------
// The products P V run over all keys that some row of an item sees, with weights of 0 where a row does
// not, and 0 times a value that is not finite is NaN. So a row whose result is not finite is computed
// again, here, over its own keys alone, by one warp in fp32 (channels from .. to_channel - 1 of it): what is
// left is what those keys make of it. bf16 values as large as 32 bits hold come here too, where their sum by
// weights not yet divided by the weights' own sum overflowed; here it is their mean that is carried from key to key.
// (Slow, 0.1 ms for 5000 keys, but bounded, and over at the first key whose score or values are NaN throughout.)
template <int HS, bool BF16>
__device__ __noinline__ void redo_row(const BiasedArgs& a, int b, int c0, int q_len, int past, int j, int h, int lane,
                                      int from, int to_channel) {
  constexpr int E = HS / 32;  // channels of a lane
  Seq s;
  s.b = b, s.c0 = c0, s.q = q_len, s.past = past, s.ok = true;
  const Keys k = keys_of_row(a, s, a.prefix ? a.prefix[b] : 0, j);
  const int64_t row = c0 + j;
  auto value = [](uint16_t x) { return BF16 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x)); };
  float q[E], o[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) q[e] = value(a.query[row * a.q_stride + (int64_t)h * HS + lane * E + e]), o[e] = 0.f;
  for (int t = k.lo; t < k.hi; ++t) {
    const int phys = a.table[(int64_t)b * a.max_blocks + t / a.bs];
    const bool there = phys >= 0 && phys < a.num_blocks;  // (a page outside the pool reads as zeros)
    const int64_t at = (((int64_t)phys * a.bs + t % a.bs) * a.kvh + h / a.G) * HS + lane * E;
    float x = 0.f;
    for (int e = 0; e < E; ++e) x += q[e] * (there ? value(a.key_cache[at + e]) : 0.f);
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x = a.cap_log2 != 0.f ? a.cap_log2 * tanh_of(x * a.scale_cap) : x * a.scale_log2;
    if (a.slopes) x -= a.slopes[h] * 1.4426950408889634f * (float)abs(past + j - t);
    const float to = fmaxf(m, x), f = to == -INFINITY ? 1.f : fast_exp2(m - to);
    const float w = x == -INFINITY ? 0.f : fast_exp2(x - to);  // (NaN for a score of NaN, on the first key too)
    m = to;
    const float sum = l * f + w;
    const float old = sum == 0.f ? 1.f : l * f / sum, add = sum == 0.f ? 0.f : w / sum;  // (no weight yet: 0)
    l = sum;
    bool lost = true;
    for (int e = 0; e < E; ++e) {  // (the mean so far: no larger than its values)
      o[e] = o[e] * old + add * (there ? value(a.value_cache[at + e]) : 0.f);
      lost = lost && o[e] != o[e];
    }
    if (__all_sync(0xffffffffu, lost)) break;  // NaN throughout: no key changes that
  }
  uint16_t* out = static_cast<uint16_t*>(a.output) + (row * a.nh + h) * HS + lane * E;
  for (int e = 0; e < E; e += 2)
    if (lane * E + e >= from && lane * E + e < to_channel) *reinterpret_cast<uint32_t*>(out + e) = pack_out<BF16>(o[e], o[e + 1]);
}

__device__ __forceinline__ bool finite4(float x, float y, float z, float w) {
  // (a sum of magnitudes is finite where all are, but for an overflow, which only costs a second look)
  return fabsf(x) + fabsf(y) + fabsf(z) + fabsf(w) < INFINITY;
}

// the tiles of a sequence's rows
__device__ __forceinline__ int2 tiles_of(Keys k) {
  return k.hi > 0 ? make_int2(k.lo / kBiTile, (k.hi + kBiTile - 1) / kBiTile) : make_int2(0, 0);
}

// most keys that `rows` rows of a sequence see, by the table's width or the window
inline int64_t keys_in_reach(const BiasedArgs& a, int rows) {
  const int64_t keys = (int64_t)a.max_blocks * a.bs, reach = (int64_t)a.window + rows;
  return a.window && !a.prefix && reach < keys ? reach : keys;
}

// the tile kernel's launch (biased_tile.cuh), sub_rows rows of a sequence to a tile
cudaError_t launch_biased_tile_f16(const BiasedArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   int seg, int sub_rows, int sms, cudaStream_t s);
cudaError_t launch_biased_tile_bf16(const BiasedArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                    int seg, int sub_rows, int sms, cudaStream_t s);

}  // namespace pa
