// The paged attention kernels for heads of 128 elements.
#include "hs_paged_attention.cuh"

namespace hs {

cudaError_t paged_decode_d128(const PagedDecodeParams& p, const CUtensorMap& map, cudaStream_t st) {
  return pa::by_group<128>(p.group, p.type, p.page_type, [&](auto k) { return k.launch(p, map, st); });
}

cudaError_t prepare_paged_d128(int group, int type, int page_type) {
  return pa::by_group<128>(group, type, page_type, [](auto k) { return k.prepare(); });
}

}  // namespace hs
