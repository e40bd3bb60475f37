// Instantiations of the multi-token kernel (partial_gqa_ext_ws.cuh), one file a
// pool type so that they compile in parallel.
#include "partial_gqa_ext_ws.cuh"

namespace cpattn {

int launch_gqa_partial_ext_fp4(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  return a.has_mod ? ext_ws_dispatch<2, true>(a, s, err) : ext_ws_dispatch<2, false>(a, s, err);
}

}  // namespace cpattn
