// The paged attention kernels for heads of 64 elements.
#include "hs_paged_attention.cuh"

namespace hs {

cudaError_t paged_decode_d64(const PagedDecodeParams& p, const CUtensorMap& map, cudaStream_t st) {
  return pa::by_group<64>(p, map, st);
}

}  // namespace hs
