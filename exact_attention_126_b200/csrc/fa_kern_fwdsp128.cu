// fa_kern_fwdsp128.cu - the forward kernel for head_dim 128 with capped scores or a prefix
// (kFeatScore) on packed batches in every combination of the other bf16 features.
#include "launch_impl.cuh"

namespace fa_host {

// kFeatScore | kFeatPacked with the 16 combinations of kFeatAlibi, kFeatKpad, kFeatResidual, kFeatDropout
FA_INSTANTIATE_FWD(128, 96) FA_INSTANTIATE_FWD(128, 97) FA_INSTANTIATE_FWD(128, 98)
FA_INSTANTIATE_FWD(128, 99) FA_INSTANTIATE_FWD(128, 100) FA_INSTANTIATE_FWD(128, 101)
FA_INSTANTIATE_FWD(128, 102) FA_INSTANTIATE_FWD(128, 103) FA_INSTANTIATE_FWD(128, 104)
FA_INSTANTIATE_FWD(128, 105) FA_INSTANTIATE_FWD(128, 106) FA_INSTANTIATE_FWD(128, 107)
FA_INSTANTIATE_FWD(128, 108) FA_INSTANTIATE_FWD(128, 109) FA_INSTANTIATE_FWD(128, 110)
FA_INSTANTIATE_FWD(128, 111)
// ... and without ALiBi with kFeatNoMax
FA_INSTANTIATE_FWD(128, 224) FA_INSTANTIATE_FWD(128, 226) FA_INSTANTIATE_FWD(128, 228)
FA_INSTANTIATE_FWD(128, 230) FA_INSTANTIATE_FWD(128, 232) FA_INSTANTIATE_FWD(128, 234)
FA_INSTANTIATE_FWD(128, 236) FA_INSTANTIATE_FWD(128, 238)

int take_status_fwdsp128() { return take_unit_status(); }

}  // namespace fa_host
