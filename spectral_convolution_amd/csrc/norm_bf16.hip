// norm_bf16.hip - the norm kernels of bf16 fields and tokens (norm.hip launches them).

#include "norm_field.hpp"
#include "norm_token.hpp"

namespace fno {

NormPick norm_kernel_bf16(bool tok, int kind, bool fwd, int C, long tiles) {
  if (tok) return kind == kLayer ? tok_kernel<DT_BF16, kLayer>(fwd, C) : tok_kernel<DT_BF16, kRms>(fwd, C);
  const int w = field_waves(C, tiles);
  return kind == kLayer ? field_kernel<DT_BF16, kLayer>(fwd, C, w) : field_kernel<DT_BF16, kRms>(fwd, C, w);
}

}  // namespace fno
