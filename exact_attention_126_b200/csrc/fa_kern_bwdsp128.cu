// fa_kern_bwdsp128.cu - the dK/dV and dQ passes for head_dim 128 with capped scores or a prefix
// (kFeatScore) on packed batches in every combination of the other features.
#include "launch_impl.cuh"

namespace fa_host {

// kFeatScore | kFeatPacked with the 8 combinations of kFeatAlibi, kFeatKpad, kFeatDropout
FA_INSTANTIATE_BWD(128, 96) FA_INSTANTIATE_BWD(128, 97) FA_INSTANTIATE_BWD(128, 98)
FA_INSTANTIATE_BWD(128, 99) FA_INSTANTIATE_BWD(128, 104) FA_INSTANTIATE_BWD(128, 105)
FA_INSTANTIATE_BWD(128, 106) FA_INSTANTIATE_BWD(128, 107)

int take_status_bwdsp128() { return take_unit_status(); }

}  // namespace fa_host
