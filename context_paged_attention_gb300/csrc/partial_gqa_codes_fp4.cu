// The decode kernel over pools of codes, E2M1 pools (one file a pool type: they
// compile in parallel).
#include "partial_gqa_codes.cuh"

namespace cpattn {

int launch_gqa_codes_fp4(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  return a.has_mod ? codes_dispatch<true, true>(a, s, err) : codes_dispatch<true, false>(a, s, err);
}

}  // namespace cpattn
