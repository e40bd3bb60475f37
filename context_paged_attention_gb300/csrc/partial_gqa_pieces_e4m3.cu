// The two-tile multi-token kernel over e4m3 pools, modified scores (one file a
// pool type: they compile in parallel).
#include "partial_gqa_pieces.cuh"

namespace cpattn {

int launch_gqa_pieces_e4m3(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  return pieces::dispatch<pieces::kE4m3, true>(a, s, err);
}

}  // namespace cpattn
