// fa_kern_rope.cu - the kernels of fa_rope.cuh (per-head norm and rotary positions) and their
// launchers, for head_dim 64 and 128 and both pairings.
#include <atomic>

#include "fa_rope.cuh"
#include "tma_maps.h"
#include "launch.h"

namespace fa_host {

namespace {

// When the tile kernel runs, by the bytes of rows and the share of its tiles' token slots that hold
// a row (a sequence's last tile may hold few). Row / tile kernel in us, inputs from memory, kernels
// alone (3 x 16 heads of 64; 32 + 2 x 8 heads of 128):
//   one sequence     33 MB       50 MB       100 MB      200 MB      400 MB
//   d 64  forward    17 / 16     24 / 22     45 / 40     87 / 78    166 / 148
//         backward   29 / 24     40 / 34     72 / 58    134 / 104   254 / 196
//   d 128 forward    20 / 21     24 / 26     46 / 45     84 / 80    161 / 148
//         backward   34 / 31     39 / 38     72 / 65    131 / 116   251 / 211
//   short ones, 200 MB (share)   forward     backward
//   d 64   N 33  (52%)           85 / 121    133 / 172
//          N 65  (68%)           85 / 95     133 / 130
//          N 257 (89%)           82 / 80     129 / 109
//   d 128  N 17  (53%)           82 / 135    131 / 195
//          N 65  (81%)           82 / 92     131 / 131
//          N 257 (94%)           82 / 82     131 / 118
template <int D, bool kBwd>
bool tiles_pay(long long bytes, long long rows, long long slots) {
  constexpr long long kMinBytes = (D == 128 && !kBwd ? 96ll : 32ll) << 20;
  return bytes >= kMinBytes && 8 * rows >= 7 * slots;
}

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

// The tensor map of rows of one kind as the tile kernel takes them: (d, N, heads, B) boxes of
// kHeads heads x kTokens tokens. False where no map can be made of them (rows shared through a
// stride of 0, strides past the copy engine's).
bool rows_map(CUtensorMap* map, const fa::HeadRows& r, const fa::RopeArgs& a, int d, int tokens,
              int heads) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const bool packed = a.cu != nullptr;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)(packed ? a.tokens : a.N),
                              (cuuint64_t)r.heads, (cuuint64_t)(packed ? 1 : a.B)};
  cuuint64_t strides[3] = {(cuuint64_t)r.sn * 2, (cuuint64_t)r.sh * 2, (cuuint64_t)r.sb * 2};
  for (int i = 0; i < 3; ++i) {
    if (dims[i + 1] == 1) strides[i] = (cuuint64_t)d * 2;  // never stepped
    if (strides[i] == 0 || strides[i] >= (1ull << 40)) return false;
  }
  const cuuint32_t box[4] = {(cuuint32_t)d, (cuuint32_t)tokens, (cuuint32_t)heads, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, r.data, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launches the tile kernel if the problem is one for it: sequences of at least a tile of tokens,
// rows as tiles_pay has them, strides that a tensor map takes. Returns its blocks, 0 if it was not
// launched, -1 on an error.
template <int D, bool kInter, bool kBwd>
int tiles(const fa::RopeArgs& a, cudaStream_t st) {
  using T = fa::RopeTile<D, kBwd>;
  const int sms = device_sms();
  const int rows = a.cu != nullptr ? a.tokens : a.N;
  long long bytes = 0, items = 0;
  const long long per_kind =
      ((long long)rows + T::kTokens - 1) / T::kTokens * (a.cu != nullptr ? 1 : a.B);
  for (const fa::HeadRows& y : a.y) {
    bytes += (long long)a.tokens * y.heads * D * 2;
    if (y.heads > 0) items += per_kind;
  }
  if (rows < T::kTokens || !tiles_pay<D, kBwd>(bytes, a.tokens, per_kind * T::kTokens)) return 0;
  fa::RopeMaps m;
  for (int i = 0; i < 3; ++i) {
    if (a.y[i].heads == 0) continue;
    const bool ok = rows_map(&m.in[i], kBwd ? a.y[i] : a.x[i], a, D, T::kTokens, T::kHeads) &&
                    rows_map(&m.out[i], kBwd ? a.g[i] : a.y[i], a, D, T::kTokens, T::kHeads) &&
                    (!kBwd || i == 2 || !a.norm ||
                     rows_map(&m.x[i], a.x[i], a, D, T::kTokens, T::kHeads));
    if (!ok) return 0;
  }
  if (cudaFuncSetAttribute(fa::fa_rope_tile_kernel<D, kInter, kBwd>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           T::kSmemBytes) != cudaSuccess)
    return -1;
  long long grid = (long long)sms * fa::kRopeBlocksPerSm;
  if (grid > items) grid = items;
  if (grid > fa::kRopeMaxBlocks) grid = fa::kRopeMaxBlocks;
  fa::fa_rope_tile_kernel<D, kInter, kBwd>
      <<<(unsigned)grid, T::kThreads, T::kSmemBytes, st>>>(m, a);
  return status() == FA_OK ? (int)grid : -1;
}

template <int D, bool kInter>
fa_status_t fwd(fa::RopeArgs a, cudaStream_t st) {
  const int tiled = tiles<D, kInter, false>(a, st);
  if (tiled != 0) return tiled > 0 ? FA_OK : FA_ERR_CUDA;
  const int grid = plan(a, D);
  fa::fa_rope_fwd_kernel<D, kInter><<<grid, fa::kRopeThreads, 0, st>>>(a);
  return status();
}

template <int D, bool kInter>
fa_status_t bwd(fa::RopeArgs a, cudaStream_t st) {
  int blocks = 0;
  if (a.tokens > 0) {
    blocks = tiles<D, kInter, true>(a, st);
    if (blocks < 0) return FA_ERR_CUDA;
  }
  if (a.tokens > 0 && blocks == 0) {
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

int take_status_rope() {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, fa::g_fa_status, sizeof(int)) != cudaSuccess) return -1;
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(fa::g_fa_status, &zero, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

fa_status_t launch_rope_fwd(const fa::RopeArgs& a, int d, bool interleaved, cudaStream_t st) {
  if (d == 64) return interleaved ? fwd<64, true>(a, st) : fwd<64, false>(a, st);
  return interleaved ? fwd<128, true>(a, st) : fwd<128, false>(a, st);
}

fa_status_t launch_rope_bwd(const fa::RopeArgs& a, int d, bool interleaved, cudaStream_t st) {
  if (d == 64) return interleaved ? bwd<64, true>(a, st) : bwd<64, false>(a, st);
  return interleaved ? bwd<128, true>(a, st) : bwd<128, false>(a, st);
}

}  // namespace fa_host
