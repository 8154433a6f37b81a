// The fp16 kernels of biased_tile.cuh, compiled by themselves.
#include "biased_tile.cuh"

namespace pa {

cudaError_t launch_biased_tile_f16(const BiasedArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   int seg, int sub_rows, int sms, cudaStream_t s) {
  return launch_biased_tile<false>(a, tq, tk, tv, seg, sub_rows, sms, s);
}

}  // namespace pa
