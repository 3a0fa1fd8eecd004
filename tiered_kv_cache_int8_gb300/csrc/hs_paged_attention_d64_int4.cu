// The paged attention kernels for heads of 64: 4-bit pages.
#include "hs_paged_attention.cuh"

namespace hs {
namespace pa {

HS_PAGED_DECODE_OF(64, PAGES_INT4, false)
HS_PAGED_DECODE_OF(64, PAGES_INT4, true)

}  // namespace pa
}  // namespace hs
