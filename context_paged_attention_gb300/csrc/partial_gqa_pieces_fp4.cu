// The two-tile multi-token kernel over E2M1 pools (one file a pool type: they
// compile in parallel).
#include "partial_gqa_pieces.cuh"

namespace cpattn {

int launch_gqa_pieces_fp4(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  return a.has_mod ? pieces::dispatch<pieces::kFp4, true>(a, s, err) : pieces::dispatch<pieces::kFp4, false>(a, s, err);
}

}  // namespace cpattn
