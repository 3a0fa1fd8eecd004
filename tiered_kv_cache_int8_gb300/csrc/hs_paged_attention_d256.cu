// The paged attention kernels for heads of 256 elements.
#include "hs_paged_attention.cuh"

namespace hs {

cudaError_t paged_decode_d256(const PagedDecodeParams& p, const CUtensorMap& map, cudaStream_t st) {
  return pa::by_group<256>(p.group, p.type, p.page_type, [&](auto k) { return k.launch(p, map, st); });
}

cudaError_t prepare_paged_d256(int group, int type, int page_type) {
  return pa::by_group<256>(group, type, page_type, [](auto k) { return k.prepare(); });
}

}  // namespace hs
