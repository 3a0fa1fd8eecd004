// The prompt attention kernels for heads of 256 elements.
#include "hs_paged_attend.cuh"

namespace hs {
namespace pt {

HS_PAGED_ATTEND_OF(256)

}  // namespace pt
}  // namespace hs
