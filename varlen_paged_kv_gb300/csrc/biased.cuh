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
// |u| = 0.25, 4.9e-8 off at most (with six terms up to 0.75, 1.4e-8), beyond that from the exponential,
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
// not, and 0 times a value that is not finite is NaN; a weight that is 0 in 32 bits only makes NaN of an infinity; and a
// sum of bf16 values by weights not yet divided by their own sum may be past 32 bits. So a row whose result is not finite is
// looked at again, here, over its own keys alone, by one warp (channels from .. to_channel - 1 of it, as they stand in
// the output). A channel in which the row sees an infinity or NaN is that, whatever the weights: one pass over the
// values says so, and is all there is to do if every other channel is finite already. Else the row is computed again in
// fp32, the mean so far carried from key to key, which is no larger than its values.
// (By a warp, 32 keys at a time, with the loads of 8 or 16 values in flight: a decode row of 50000 keys of 128 channels
// takes 2.5 ms to look at and 11 to compute again, 36 where a key followed the other; of 256 channels 8 and 39; a prompt of
// 8192 rows that all see one infinity 9 ms instead of 140. Rows whose sum of weights is NaN, as by a score of NaN, are NaN
// throughout and do not come here.)
template <int HS, bool BF16>
__device__ __noinline__ void redo_row(const BiasedArgs& a, int b, int c0, int q_len, int past, int j, int h, int lane,
                                      int from, int to_channel) {
  constexpr int E = HS / 32;  // channels of a lane
  constexpr uint32_t kTop = BF16 ? 0x7F80u : 0x7C00u;
  Seq s;
  s.b = b, s.c0 = c0, s.q = q_len, s.past = past, s.ok = true;
  const Keys k = keys_of_row(a, s, a.prefix ? a.prefix[b] : 0, j);
  const int64_t row = c0 + j;
  const int32_t* table = a.table + (int64_t)b * a.max_blocks;
  auto value = [](uint32_t x) { return BF16 ? __uint_as_float(x << 16) : __half2float(__ushort_as_half((uint16_t)x)); };
  // the cache row of this lane's key of the 32 from t on; -1 for one that the row does not see, which is left out, and
  // for one on a page outside the pool, which reads as zeros
  auto slot_of = [&](int t) {
    t += lane;
    const int phys = t >= k.lo && t < k.hi ? table[t / a.bs] : -1;
    return phys >= 0 && phys < a.num_blocks ? phys * a.bs + t % a.bs : -1;
  };
  const int stride = a.kvh * HS;  // of cache rows
  const int64_t head = (int64_t)(h / a.G) * HS;
  // the lane's channels of the V rows of keys i .. i + BATCH - 1 of 32, their loads in flight together
  constexpr int BATCH = E == 8 ? 8 : 16;
  auto load_values = [&](int slot, int i, uint32_t (&v)[BATCH][E / 2]) {
#pragma unroll
    for (int n = 0; n < BATCH; ++n) {
      const int row_n = __shfl_sync(0xffffffffu, slot, i + n);
      const uint16_t* p = a.value_cache + head + lane * E + (int64_t)max(row_n, 0) * stride;
      if constexpr (E == 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        v[n][0] = x.x, v[n][1] = x.y, v[n][2] = x.z, v[n][3] = x.w;
      } else if constexpr (E == 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        v[n][0] = x.x, v[n][1] = x.y;
      } else {
        v[n][0] = *reinterpret_cast<const uint32_t*>(p);
      }
#pragma unroll
      for (int e = 0; e < E / 2; ++e) v[n][e] = row_n < 0 ? 0u : v[n][e];
    }
  };
  uint16_t* out = static_cast<uint16_t*>(a.output) + (row * a.nh + h) * HS + lane * E;
  const int first = k.lo / 32 * 32;

  // The largest values seen, pairs of channels as signed 16-bit numbers, which order what is not negative as the values,
  // infinity and NaN behind them; and as unsigned ones, which do so with the magnitudes of what is negative.
  uint32_t top[E / 2] = {}, low[E / 2] = {};
  for (int t = first, slot = slot_of(first); t < k.hi; t += 32) {
    const int next = slot_of(t + 32);
#pragma unroll 1
    for (int i = 0; i < 32; i += BATCH) {
      uint32_t v[BATCH][E / 2];
      load_values(slot, i, v);
#pragma unroll
      for (int n = 0; n < BATCH; n += 2)
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          top[e] = __vimax3_s16x2(top[e], v[n][e], v[n + 1][e]);
          low[e] = __vimax3_u16x2(low[e], v[n][e], v[n + 1][e]);
        }
    }
    slot = next;
  }
  float o[E];
  bool given[E], settled = true;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const bool mine = lane * E + e >= from && lane * E + e < to_channel;
    const uint32_t now = mine ? out[e] : 0u;
    const uint32_t up = top[e / 2] >> (e & 1) * 16 & 0xffffu, down = low[e / 2] >> (e & 1) * 16 & 0xffffu;
    given[e] = up >= kTop || down >= (kTop | 0x8000u);
    o[e] = value(now);
    if (given[e]) o[e] = up < kTop ? value(down) : down < (kTop | 0x8000u) ? value(up) : NAN;
    else settled = settled && (now & kTop) != kTop && (BF16 || (now & 0x7FFFu) != 0x7BFFu);  // (fp16 may be held there)
  }
  if (!__all_sync(0xffffffffu, settled)) {
    const uint16_t* q = a.query + row * a.q_stride + (int64_t)h * HS;
    float mean[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) mean[e] = 0.f;
    for (int t = first, slot = slot_of(first); t < k.hi; t += 32) {
      const int next = slot_of(t + 32);
      const bool sees = t + lane >= k.lo && t + lane < k.hi;
      const uint16_t* key = a.key_cache + head + (int64_t)max(slot, 0) * stride;
      float x = 0.f;
#pragma unroll 4
      for (int c = 0; c < HS; c += 8) {
        const uint4 y = *reinterpret_cast<const uint4*>(q + c);
        const uint4 z = *reinterpret_cast<const uint4*>(key + c);
        const uint32_t ys[4] = {y.x, y.y, y.z, y.w}, zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x = fmaf(value(ys[e / 2] >> (e & 1) * 16 & 0xffffu), value(zs[e / 2] >> (e & 1) * 16 & 0xffffu), x);
      }
      if (slot < 0) x = 0.f;
      x = a.cap_log2 != 0.f ? a.cap_log2 * tanh_of(x * a.scale_cap) : x * a.scale_log2;
      if (a.slopes) x -= a.slopes[h] * 1.4426950408889634f * (float)abs(past + j - (t + lane));
      if (!sees) x = -INFINITY;
      float to = x;
#pragma unroll
      for (int d = 16; d; d >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, d));
      to = fmaxf(to, m);
      const float f = to == -INFINITY ? 1.f : fast_exp2(m - to);
      const float w = x == -INFINITY ? 0.f : fast_exp2(x - to);  // (NaN for a score of NaN)
      float sum = w;
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      sum += l * f;
      const float old = sum == 0.f ? 1.f : l * f / sum, add = sum == 0.f ? 0.f : w / sum;  // (no weight yet: 0)
      m = to;
      l = sum;
      if (sum != sum) break;  // NaN throughout: no key changes that
#pragma unroll
      for (int e = 0; e < E; ++e) mean[e] *= old;
#pragma unroll 1
      for (int i = 0; i < 32; i += BATCH) {
        uint32_t v[BATCH][E / 2];
        load_values(slot, i, v);
#pragma unroll
        for (int n = 0; n < BATCH; ++n) {
          const float share = __shfl_sync(0xffffffffu, add, i + n);
#pragma unroll
          for (int e = 0; e < E; ++e) mean[e] = fmaf(share, value(v[n][e / 2] >> (e & 1) * 16 & 0xffffu), mean[e]);
        }
      }
      slot = next;
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (l != l) o[e] = NAN;
      else if (!given[e]) o[e] = mean[e];
  }
#pragma unroll
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
