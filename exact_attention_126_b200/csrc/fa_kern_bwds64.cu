// fa_kern_bwds64.cu - the dK/dV and dQ passes for head_dim 64 with capped scores or a prefix
// (kFeatScore) in every combination of the other features.
#include "launch_impl.cuh"

namespace fa_host {

// kFeatScore with the 8 combinations of kFeatAlibi, kFeatKpad, kFeatDropout
FA_INSTANTIATE_BWD(64, 64) FA_INSTANTIATE_BWD(64, 65) FA_INSTANTIATE_BWD(64, 66)
FA_INSTANTIATE_BWD(64, 67) FA_INSTANTIATE_BWD(64, 72) FA_INSTANTIATE_BWD(64, 73)
FA_INSTANTIATE_BWD(64, 74) FA_INSTANTIATE_BWD(64, 75)

int take_status_bwds64() { return take_unit_status(); }

}  // namespace fa_host
