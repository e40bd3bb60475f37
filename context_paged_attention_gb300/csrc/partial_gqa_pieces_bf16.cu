// The two-tile multi-token kernel over bf16 pools, modified scores (one file a
// pool type: they compile in parallel).
#include "partial_gqa_pieces.cuh"

namespace cpattn {

int launch_gqa_pieces_bf16(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  return pieces::dispatch<pieces::kBf16, true>(a, s, err);
}

}  // namespace cpattn
