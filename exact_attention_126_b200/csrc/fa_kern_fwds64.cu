// fa_kern_fwds64.cu - the forward kernel for head_dim 64 with capped scores or a prefix
// (kFeatScore) in every combination of the other bf16 features.
#include "launch_impl.cuh"

namespace fa_host {

// kFeatScore with the 16 combinations of kFeatAlibi, kFeatKpad, kFeatResidual, kFeatDropout
FA_INSTANTIATE_FWD(64, 64) FA_INSTANTIATE_FWD(64, 65) FA_INSTANTIATE_FWD(64, 66)
FA_INSTANTIATE_FWD(64, 67) FA_INSTANTIATE_FWD(64, 68) FA_INSTANTIATE_FWD(64, 69)
FA_INSTANTIATE_FWD(64, 70) FA_INSTANTIATE_FWD(64, 71) FA_INSTANTIATE_FWD(64, 72)
FA_INSTANTIATE_FWD(64, 73) FA_INSTANTIATE_FWD(64, 74) FA_INSTANTIATE_FWD(64, 75)
FA_INSTANTIATE_FWD(64, 76) FA_INSTANTIATE_FWD(64, 77) FA_INSTANTIATE_FWD(64, 78)
FA_INSTANTIATE_FWD(64, 79)
// ... and without ALiBi with kFeatNoMax
FA_INSTANTIATE_FWD(64, 192) FA_INSTANTIATE_FWD(64, 194) FA_INSTANTIATE_FWD(64, 196)
FA_INSTANTIATE_FWD(64, 198) FA_INSTANTIATE_FWD(64, 200) FA_INSTANTIATE_FWD(64, 202)
FA_INSTANTIATE_FWD(64, 204) FA_INSTANTIATE_FWD(64, 206)

int take_status_fwds64() { return take_unit_status(); }

}  // namespace fa_host
