// The paged attention kernels for heads of 128: 16-bit and 8-bit pages.
#include "hs_paged_attention.cuh"

namespace hs {
namespace pa {

HS_PAGED_DECODE_OF(128, PAGES_SAME, false)
HS_PAGED_DECODE_OF(128, PAGES_E4M3, false)

}  // namespace pa
}  // namespace hs
