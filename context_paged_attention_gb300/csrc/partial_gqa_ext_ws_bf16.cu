// Instantiations of the multi-token kernel (partial_gqa_ext_ws.cuh), one file a
// pool type so that they compile in parallel.
#include "partial_gqa_ext_ws.cuh"

namespace cpattn {

int launch_gqa_partial_ext_bf16(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  return a.has_mod ? ext_ws_dispatch<0, true>(a, s, err) : ext_ws_dispatch<0, false>(a, s, err);
}

int launch_gqa_partial_ext(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  if (a.kv_fp4) return launch_gqa_partial_ext_fp4(a, s, err);
  return a.kv_fp8 ? launch_gqa_partial_ext_e4m3(a, s, err) : launch_gqa_partial_ext_bf16(a, s, err);
}

}  // namespace cpattn
