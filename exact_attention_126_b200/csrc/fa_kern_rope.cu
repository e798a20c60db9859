// fa_kern_rope.cu - the kernels of fa_rope.cuh (per-head norm and rotary positions) and their
// launchers, for head_dim 64 and 128 and both pairings.
#include <atomic>

#include "fa_rope.cuh"
#include "launch.h"

namespace fa_host {

namespace {

// SMs of the current device (asked once per device).
int device_sms() {
  static std::atomic<int> cache[64];
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return n;
  if (dev < 64 && cache[dev].load(std::memory_order_relaxed) > 0)
    return cache[dev].load(std::memory_order_relaxed);
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
  if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

fa_status_t status() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Sets a.splits and returns the grid. A warp takes all units (fa_rope.cuh) of a token, unless
// that leaves SMs with fewer than 16 warps: then a token's units are dealt to several warps, so
// that the latency of a few tokens' rows is spread over as many warps as there are units.
int plan(fa::RopeArgs& a, int d) {
  const int sms = device_sms();
  const int rows = 32 / (d / 8);
  int units = 0;
  for (const fa::HeadRows& y : a.y) units += (y.heads + rows - 1) / rows;
  const long long want = ((long long)sms * 16 + a.tokens - 1) / a.tokens;
  a.splits = (int)(want < units ? want : units);
  if (a.splits < 1) a.splits = 1;
  const long long blocks = ((long long)a.tokens * a.splits + fa::kRopeWarps - 1) / fa::kRopeWarps;
  const long long most = (long long)sms * fa::kRopeBlocksPerSm;
  return (int)(blocks < most ? blocks : most);
}

template <int D, bool kInter>
fa_status_t fwd(fa::RopeArgs a, cudaStream_t st) {
  const int grid = plan(a, D);
  fa::fa_rope_fwd_kernel<D, kInter><<<grid, fa::kRopeThreads, 0, st>>>(a);
  return status();
}

template <int D, bool kInter>
fa_status_t bwd(fa::RopeArgs a, cudaStream_t st) {
  int blocks = 0;
  if (a.tokens > 0) {
    blocks = plan(a, D);
    if (blocks > fa::kRopeMaxBlocks) blocks = fa::kRopeMaxBlocks;
    fa::fa_rope_bwd_kernel<D, kInter><<<blocks, fa::kRopeThreads, 0, st>>>(a);
    const fa_status_t s = status();
    if (s != FA_OK) return s;
  }
  if (a.partial == nullptr) return FA_OK;
  fa::fa_rope_reduce_kernel<D><<<2 * D / 32, 1024, 0, st>>>(a.partial, blocks, a.dw[0], a.dw[1]);
  return status();
}

}  // namespace

fa_status_t launch_rope_fwd(const fa::RopeArgs& a, int d, bool interleaved, cudaStream_t st) {
  if (d == 64) return interleaved ? fwd<64, true>(a, st) : fwd<64, false>(a, st);
  return interleaved ? fwd<128, true>(a, st) : fwd<128, false>(a, st);
}

fa_status_t launch_rope_bwd(const fa::RopeArgs& a, int d, bool interleaved, cudaStream_t st) {
  if (d == 64) return interleaved ? bwd<64, true>(a, st) : bwd<64, false>(a, st);
  return interleaved ? bwd<128, true>(a, st) : bwd<128, false>(a, st);
}

}  // namespace fa_host
