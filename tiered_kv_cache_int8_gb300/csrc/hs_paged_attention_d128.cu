// The paged attention kernels for heads of 128 elements.
#include "hs_paged_attention.cuh"

namespace hs {

cudaError_t paged_decode_d128(const PagedDecodeParams& p, const CUtensorMap& map, cudaStream_t st) {
  return pa::by_group<128>(p, map, st);
}

}  // namespace hs
