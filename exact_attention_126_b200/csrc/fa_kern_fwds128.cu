// fa_kern_fwds128.cu - the forward kernel for head_dim 128 with capped scores or a prefix
// (kFeatScore) in every combination of the other bf16 features.
#include "launch_impl.cuh"

namespace fa_host {

// kFeatScore with the 16 combinations of kFeatAlibi, kFeatKpad, kFeatResidual, kFeatDropout
FA_INSTANTIATE_FWD(128, 64) FA_INSTANTIATE_FWD(128, 65) FA_INSTANTIATE_FWD(128, 66)
FA_INSTANTIATE_FWD(128, 67) FA_INSTANTIATE_FWD(128, 68) FA_INSTANTIATE_FWD(128, 69)
FA_INSTANTIATE_FWD(128, 70) FA_INSTANTIATE_FWD(128, 71) FA_INSTANTIATE_FWD(128, 72)
FA_INSTANTIATE_FWD(128, 73) FA_INSTANTIATE_FWD(128, 74) FA_INSTANTIATE_FWD(128, 75)
FA_INSTANTIATE_FWD(128, 76) FA_INSTANTIATE_FWD(128, 77) FA_INSTANTIATE_FWD(128, 78)
FA_INSTANTIATE_FWD(128, 79)
// ... and without ALiBi with kFeatNoMax
FA_INSTANTIATE_FWD(128, 192) FA_INSTANTIATE_FWD(128, 194) FA_INSTANTIATE_FWD(128, 196)
FA_INSTANTIATE_FWD(128, 198) FA_INSTANTIATE_FWD(128, 200) FA_INSTANTIATE_FWD(128, 202)
FA_INSTANTIATE_FWD(128, 204) FA_INSTANTIATE_FWD(128, 206)

int take_status_fwds128() { return take_unit_status(); }

}  // namespace fa_host
