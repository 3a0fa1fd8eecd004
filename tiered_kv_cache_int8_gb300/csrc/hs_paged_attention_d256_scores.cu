// The paged attention kernels for heads of 256: 16-bit and 8-bit pages, scores with a cap or a bias.
#include "hs_paged_attention.cuh"

namespace hs {
namespace pa {

HS_PAGED_DECODE_OF(256, PAGES_SAME, true)
HS_PAGED_DECODE_OF(256, PAGES_E4M3, true)

}  // namespace pa
}  // namespace hs
