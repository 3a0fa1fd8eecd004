// The paged attention kernels for heads of 256: 4-bit pages.
#include "hs_paged_attention.cuh"

namespace hs {
namespace pa {

HS_PAGED_DECODE_OF(256, PAGES_INT4, false)
HS_PAGED_DECODE_OF(256, PAGES_INT4, true)

}  // namespace pa
}  // namespace hs
