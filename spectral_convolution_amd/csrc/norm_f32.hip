// norm_f32.hip - the norm kernels of f32 fields and tokens (norm.hip launches them).

#include "norm_field.hpp"
#include "norm_token.hpp"

namespace fno {

const void *norm_kernel_f32(bool tok, int kind, bool fwd, int C, long tiles, int &threads, int &rpg) {
  if (tok)
    return kind == kLayer ? tok_kernel<DT_F32, kLayer>(fwd, C, threads, rpg) : tok_kernel<DT_F32, kRms>(fwd, C, threads, rpg);
  const int w = field_waves(C, tiles);
  threads = w == 1 ? 256 : 64 * w;
  rpg = w == 1 ? 4 : 1;
  if (fwd) return kind == kLayer ? field_kernel<DT_F32, kLayer, true>(C, w) : field_kernel<DT_F32, kRms, true>(C, w);
  return kind == kLayer ? field_kernel<DT_F32, kLayer, false>(C, w) : field_kernel<DT_F32, kRms, false>(C, w);
}

}  // namespace fno
