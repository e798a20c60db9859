// fa_kern_fwdsp64.cu - the forward kernel for head_dim 64 with capped scores or a prefix
// (kFeatScore) on packed batches in every combination of the other bf16 features.
#include "launch_impl.cuh"

namespace fa_host {

// kFeatScore | kFeatPacked with the 16 combinations of kFeatAlibi, kFeatKpad, kFeatResidual, kFeatDropout
FA_INSTANTIATE_FWD(64, 96) FA_INSTANTIATE_FWD(64, 97) FA_INSTANTIATE_FWD(64, 98)
FA_INSTANTIATE_FWD(64, 99) FA_INSTANTIATE_FWD(64, 100) FA_INSTANTIATE_FWD(64, 101)
FA_INSTANTIATE_FWD(64, 102) FA_INSTANTIATE_FWD(64, 103) FA_INSTANTIATE_FWD(64, 104)
FA_INSTANTIATE_FWD(64, 105) FA_INSTANTIATE_FWD(64, 106) FA_INSTANTIATE_FWD(64, 107)
FA_INSTANTIATE_FWD(64, 108) FA_INSTANTIATE_FWD(64, 109) FA_INSTANTIATE_FWD(64, 110)
FA_INSTANTIATE_FWD(64, 111)
// ... and without ALiBi with kFeatNoMax
FA_INSTANTIATE_FWD(64, 224) FA_INSTANTIATE_FWD(64, 226) FA_INSTANTIATE_FWD(64, 228)
FA_INSTANTIATE_FWD(64, 230) FA_INSTANTIATE_FWD(64, 232) FA_INSTANTIATE_FWD(64, 234)
FA_INSTANTIATE_FWD(64, 236) FA_INSTANTIATE_FWD(64, 238)

int take_status_fwdsp64() { return take_unit_status(); }

}  // namespace fa_host
