// The prompt attention kernels for heads of 64 elements.
#include "hs_paged_attend.cuh"

namespace hs {
namespace pt {

HS_PAGED_ATTEND_OF(64)

}  // namespace pt
}  // namespace hs
