// fa_kern_bwds128.cu - the dK/dV and dQ passes for head_dim 128 with capped scores or a prefix
// (kFeatScore) in every combination of the other features.
#include "launch_impl.cuh"

namespace fa_host {

// kFeatScore with the 8 combinations of kFeatAlibi, kFeatKpad, kFeatDropout
FA_INSTANTIATE_BWD(128, 64) FA_INSTANTIATE_BWD(128, 65) FA_INSTANTIATE_BWD(128, 66)
FA_INSTANTIATE_BWD(128, 67) FA_INSTANTIATE_BWD(128, 72) FA_INSTANTIATE_BWD(128, 73)
FA_INSTANTIATE_BWD(128, 74) FA_INSTANTIATE_BWD(128, 75)

int take_status_bwds128() { return take_unit_status(); }

}  // namespace fa_host
