// mix_train_f16.hip - the training channel mix on f16 fields (mix_train.hip launches it).

#include "mix_train_half.hpp"

namespace fno {

MtPick mix_train_f16(int O, int I) { return mh_pick<DT_F16>(O, I); }

}  // namespace fno
