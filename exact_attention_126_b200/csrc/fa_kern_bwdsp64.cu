// fa_kern_bwdsp64.cu - the dK/dV and dQ passes for head_dim 64 with capped scores or a prefix
// (kFeatScore) on packed batches in every combination of the other features.
#include "launch_impl.cuh"

namespace fa_host {

// kFeatScore | kFeatPacked with the 8 combinations of kFeatAlibi, kFeatKpad, kFeatDropout
FA_INSTANTIATE_BWD(64, 96) FA_INSTANTIATE_BWD(64, 97) FA_INSTANTIATE_BWD(64, 98)
FA_INSTANTIATE_BWD(64, 99) FA_INSTANTIATE_BWD(64, 104) FA_INSTANTIATE_BWD(64, 105)
FA_INSTANTIATE_BWD(64, 106) FA_INSTANTIATE_BWD(64, 107)

int take_status_bwdsp64() { return take_unit_status(); }

}  // namespace fa_host
