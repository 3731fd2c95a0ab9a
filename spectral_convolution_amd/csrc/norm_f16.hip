// norm_f16.hip - the norm kernels of f16 fields and tokens (norm.hip launches them).

#include "norm_field.hpp"
#include "norm_token.hpp"

namespace fno {

const void *norm_kernel_f16(bool tok, int kind, bool fwd, int C, long tiles, int &threads, int &rpg) {
  if (tok)
    return kind == kLayer ? tok_kernel<DT_F16, kLayer>(fwd, C, threads, rpg) : tok_kernel<DT_F16, kRms>(fwd, C, threads, rpg);
  const int w = field_waves(C, tiles);
  threads = w == 1 ? 256 : 64 * w;
  rpg = w == 1 ? 4 : 1;
  if (fwd) return kind == kLayer ? field_kernel<DT_F16, kLayer, true>(C, w) : field_kernel<DT_F16, kRms, true>(C, w);
  return kind == kLayer ? field_kernel<DT_F16, kLayer, false>(C, w) : field_kernel<DT_F16, kRms, false>(C, w);
}

}  // namespace fno
