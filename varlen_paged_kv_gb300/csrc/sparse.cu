// Attention of every query row over the pages selected for it.
//
// Row i of sequence b at position p attends, for query head h of KV head g, the keys t <= p
// of the pages selected[i][g] (logical pages, strictly ascending, -1 for none):
// softmax(scale q.k) V in fp32, rounded once to T; a row without any key gives zeros and an
// lse of -inf.
#include "ops.cuh"

namespace pa {

constexpr int kSimpleWarps = 4;

template <bool BF16, int HS>
__global__ void __launch_bounds__(kSimpleWarps * 32) sparse_simple_kernel(const PageArgs a) {
  constexpr int E = HS / 32;
  extern __shared__ int list[];  // [2 * top_k]: logical and physical pages
  __shared__ float acc[kSimpleWarps][HS], mw[kSimpleWarps], lw[kSimpleWarps];
  __shared__ int n_list;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x, h = blockIdx.y, g = h / a.G;
  if (blockIdx.x == 0 && h == 0) check_batch(a.cum, a.past, a.B, a.N, a.max_blocks, a.bs, a.error);
  const int b = find_seq(a.cum, a.B, 1, 0, row, lane);
  if (b < 0) return;
  const Seq s = load_seq(a.cum, a.past, b, a.N, a.max_blocks, a.bs);
  if (!s.ok || row - s.c0 >= s.q) return;
  const int pos = s.past + row - s.c0;
  const int j0 = (row - s.c0) / a.R * a.R;  // the row's query block
  const int visible = (s.past + min(j0 + a.R, s.q) - 1) / a.bs + 1;
  if (warp == 0) {
    const int* sel = a.selected + ((int64_t)(s.c0 + j0) * a.kvh + g) * a.top_k;
    int kept = 0, top = -1;
    for (int i = 0; i < a.top_k; i += 32) {
      const int e = i + lane < a.top_k ? sel[i + lane] : -1;
      int m = e;  // the largest entry up to this lane
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, m, d);
        if (lane >= d) m = max(m, y);
      }
      int before = __shfl_up_sync(0xffffffffu, m, 1);
      before = max(top, lane ? before : -1);
      int phys = -1;
      bool use = e >= 0 && e < visible && e > before, bad = e < -1 || e >= visible || (e >= 0 && !use);
      if (use) {
        phys = a.table[(int64_t)b * a.max_blocks + e];
        if (phys < 0 || phys >= a.num_blocks) use = false, bad = true;
      }
      if (bad && a.error) atomicOr(a.error, PA_DEVERR_BAD_BLOCK);
      const unsigned mask = __ballot_sync(0xffffffffu, use);
      if (use) {
        const int at = kept + __popc(mask & ((1u << lane) - 1));
        list[at] = e;
        list[a.top_k + at] = phys;
      }
      kept += __popc(mask);
      top = max(top, __shfl_sync(0xffffffffu, m, 31));
    }
    if (lane == 0) n_list = kept;
  }
  __syncthreads();
  float q[E], o[E], m = -INFINITY, l = 0.f;
  auto get = [&](const uint16_t* p, float (&x)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      x[e] = BF16 ? __uint_as_float((uint32_t)p[lane * E + e] << 16) : __half2float(__ushort_as_half(p[lane * E + e]));
  };
  get(a.query + (int64_t)row * a.q_stride + (int64_t)h * HS, q);
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int t = warp; t < n_list * a.bs; t += kSimpleWarps) {
    const int i = t / a.bs, in = t % a.bs;
    if (list[i] * a.bs + in > pos) continue;
    const int64_t at = (((int64_t)list[a.top_k + i] * a.bs + in) * a.kvh + g) * HS;
    float k[E], d = 0.f;
    get(a.key_cache + at, k);
#pragma unroll
    for (int e = 0; e < E; ++e) d = fmaf(q[e], k[e], d);
#pragma unroll
    for (int x = 16; x; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
    d *= a.scale_log2;
    const float mn = fmaxf(m, d), al = exp2f(m - mn), p = exp2f(d - mn);
    m = mn;
    l = l * al + p;
    get(a.value_cache + at, k);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(p, k[e], o[e] * al);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) acc[warp][lane * E + e] = o[e];
  if (lane == 0) mw[warp] = m, lw[warp] = l;
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kSimpleWarps; ++w) M = fmaxf(M, mw[w]);
  for (int w = 0; w < kSimpleWarps; ++w)
    if (mw[w] != -INFINITY) L += lw[w] * exp2f(mw[w] - M);
  for (int c = threadIdx.x; c < HS; c += kSimpleWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kSimpleWarps; ++w)
      if (mw[w] != -INFINITY) x += acc[w][c] * exp2f(mw[w] - M);
    x = L > 0.f ? x / L : 0.f;
    reinterpret_cast<uint16_t*>(a.output)[((int64_t)row * a.nh + h) * HS + c] =
        BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(int64_t)row * a.nh + h] = L > 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

cudaError_t launch_sparse(const PageArgs& a, bool bf16, int /*sms*/, cudaStream_t s) {
  const dim3 grid((unsigned)a.N, (unsigned)a.nh);
  const size_t smem = (size_t)a.top_k * 8;
  auto go = [&](auto kernel) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) return e;
    kernel<<<grid, kSimpleWarps * 32, smem, s>>>(a);
    return cudaGetLastError();
  };
  if (a.hs == 64) return bf16 ? go(sparse_simple_kernel<true, 64>) : go(sparse_simple_kernel<false, 64>);
  if (a.hs == 128) return bf16 ? go(sparse_simple_kernel<true, 128>) : go(sparse_simple_kernel<false, 128>);
  return bf16 ? go(sparse_simple_kernel<true, 256>) : go(sparse_simple_kernel<false, 256>);
}

}  // namespace pa
