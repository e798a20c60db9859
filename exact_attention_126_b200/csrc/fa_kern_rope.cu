// fa_kern_rope.cu - the kernels of fa_rope.cuh (per-head norm and rotary positions) and their
// launchers, for head_dim 64 and 128 and both pairings.
#include "fa_rope.cuh"
#include "launch.h"

namespace fa_host {

namespace {

int device_sms() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n;
}

fa_status_t status() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Warps per token: one, unless the tokens are too few to give every SM 16 warps (the
// latency of a few tokens' rows is then spread over more of them), and at most one per unit
// of rows a warp loads at once.
int warps_per_token(const fa::RopeArgs& a, int d, int sms) {
  int units = 0;
  const int rows = 32 / (d / 16);
  for (const fa::HeadRows& y : a.y) units += (y.heads + rows - 1) / rows;
  const long long want = ((long long)sms * 16 + a.tokens - 1) / a.tokens;
  return (int)(want < units ? (want < 1 ? 1 : want) : (units < 1 ? 1 : units));
}

}  // namespace

template <int D, bool kInter>
fa_status_t launch_rope_fwd_t(fa::RopeArgs a, cudaStream_t st) {
  const int sms = device_sms();
  a.splits = warps_per_token(a, D, sms);
  const long long blocks = ((long long)a.tokens * a.splits + fa::kRopeWarps - 1) / fa::kRopeWarps;
  const long long most = (long long)sms * 8;
  fa::fa_rope_fwd_kernel<D, kInter>
      <<<(unsigned)(blocks < most ? blocks : most), fa::kRopeThreads, 0, st>>>(a);
  return status();
}

template <int D, bool kInter>
fa_status_t launch_rope_bwd_t(fa::RopeArgs a, cudaStream_t st) {
  const int sms = device_sms();
  const bool gains = a.partial != nullptr;
  int blocks = 0;
  if (a.tokens > 0) {
    a.splits = warps_per_token(a, D, sms);
    const long long need =
        ((long long)a.tokens * a.splits + fa::kRopeWarps - 1) / fa::kRopeWarps;
    const int most = 2 * sms < fa::kRopeMaxBlocks ? 2 * sms : fa::kRopeMaxBlocks;
    blocks = (int)(need < most ? need : most);
    fa::fa_rope_bwd_kernel<D, kInter><<<blocks, fa::kRopeThreads, 0, st>>>(a);
    const fa_status_t s = status();
    if (s != FA_OK) return s;
  }
  if (!gains) return FA_OK;
  fa::fa_rope_reduce_kernel<D><<<2 * D / 32, 1024, 0, st>>>(a.partial, blocks, a.dw[0], a.dw[1]);
  return status();
}

fa_status_t launch_rope_fwd(const fa::RopeArgs& a, int d, bool interleaved, cudaStream_t st) {
  if (d == 64)
    return interleaved ? launch_rope_fwd_t<64, true>(a, st) : launch_rope_fwd_t<64, false>(a, st);
  return interleaved ? launch_rope_fwd_t<128, true>(a, st) : launch_rope_fwd_t<128, false>(a, st);
}

fa_status_t launch_rope_bwd(const fa::RopeArgs& a, int d, bool interleaved, cudaStream_t st) {
  if (d == 64)
    return interleaved ? launch_rope_bwd_t<64, true>(a, st) : launch_rope_bwd_t<64, false>(a, st);
  return interleaved ? launch_rope_bwd_t<128, true>(a, st) : launch_rope_bwd_t<128, false>(a, st);
}

}  // namespace fa_host
