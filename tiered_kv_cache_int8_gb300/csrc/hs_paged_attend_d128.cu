// The prompt attention kernels for heads of 128 elements.
#include "hs_paged_attend.cuh"

namespace hs {
namespace pt {

HS_PAGED_ATTEND_OF(128)

}  // namespace pt
}  // namespace hs
