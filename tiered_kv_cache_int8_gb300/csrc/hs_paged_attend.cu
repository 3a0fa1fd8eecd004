// Host side of the prompt attention: the choice of the kernel and the workspace.
#include "hs_paged_attend.cuh"

namespace hs {

int64_t attend_workspace_bytes(int d, int ctas) {
  auto of = [&](auto c) {
    using C = decltype(c);
    return pt::ws_chain<C>(ctas) * sizeof(float) + (size_t)ctas * sizeof(pt::Chain);
  };
  const size_t n = d == 64    ? of(pt::Cfg<64, HS_BF16, PAGES_SAME>{})
                   : d == 128 ? of(pt::Cfg<128, HS_BF16, PAGES_SAME>{})
                              : of(pt::Cfg<256, HS_BF16, PAGES_SAME>{});
  return (int64_t)((n + 255) / 256 * 256);
}

int attend_box_rows(int d, int page_size) {
  return std::min(page_size, d == 256 ? pt::Cfg<256, HS_BF16, PAGES_SAME>::KT : pt::Cfg<128, HS_BF16, PAGES_SAME>::KT);
}

cudaError_t prepare_attend(int d, int type, int page_type) {
  return d == 64    ? pt::prepare_attend_of<64>(type, page_type)
         : d == 128 ? pt::prepare_attend_of<128>(type, page_type)
                    : pt::prepare_attend_of<256>(type, page_type);
}

cudaError_t launch_paged_attend(const PagedAttendParams& p, const CUtensorMap& map, cudaStream_t st) {
  return p.d == 64    ? pt::paged_attend_of<64>(p, map, st)
         : p.d == 128 ? pt::paged_attend_of<128>(p, map, st)
                      : pt::paged_attend_of<256>(p, map, st);
}

}  // namespace hs
