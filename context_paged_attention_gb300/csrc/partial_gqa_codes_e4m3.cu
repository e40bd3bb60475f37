// The decode kernel over pools of codes, E4M3 pools with modified scores (one
// file a pool type: they compile in parallel).
#include "partial_gqa_codes.cuh"

namespace cpattn {

int launch_gqa_codes_e4m3(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  return codes_dispatch<false, true>(a, s, err);
}

}  // namespace cpattn
