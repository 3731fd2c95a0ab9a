// mix_train_bf16.hip - the training channel mix on bf16 fields (mix_train.hip launches it).

#include "mix_train_half.hpp"

namespace fno {

MtPick mix_train_bf16(int O, int I) { return mh_pick<DT_BF16>(O, I); }

}  // namespace fno
