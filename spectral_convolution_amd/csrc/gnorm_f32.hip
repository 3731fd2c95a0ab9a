// gnorm_f32.hip - the group norm kernels of f32 fields (gnorm.hip).

#include "gnorm_kernels.hpp"

namespace fno {

hipError_t gnorm_f32(const GnArgs &a, bool fwd, void *workspace, hipStream_t s) {
  return fwd ? gn_forward<DT_F32>(a, workspace, s) : gn_backward<DT_F32>(a, workspace, s);
}

}  // namespace fno
