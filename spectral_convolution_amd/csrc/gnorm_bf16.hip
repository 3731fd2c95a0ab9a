// gnorm_bf16.hip - the group norm kernels of bf16 fields (gnorm.hip).

#include "gnorm_kernels.hpp"

namespace fno {

hipError_t gnorm_bf16(const GnArgs &a, bool fwd, void *workspace, hipStream_t s) {
  return fwd ? gn_forward<DT_BF16>(a, workspace, s) : gn_backward<DT_BF16>(a, workspace, s);
}

}  // namespace fno
