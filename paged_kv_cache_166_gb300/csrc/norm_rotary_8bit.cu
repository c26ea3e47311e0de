// Norms of q and k for each head, rotary positions and the write of quantised k and v.
#include "norm_rotary.cuh"

namespace pkv {

int norm_rotary_8bit(const NormArgs& a, int32_t codes, int32_t dtype, bool interleaved,
                     cudaStream_t st) {
  return codes == PKV_FP8_E4M3 ? launch_norm_of<1>(a, dtype, interleaved, st)
                               : launch_norm_of<2>(a, dtype, interleaved, st);
}

}  // namespace pkv
