// Host-side check of the tile and mask logic (tiles.cuh) with a prefix, against the definition
// spelled out here: key c is visible from query r iff both lie below N and c <= r or c < prefix.
// Prints "OK" or the first mismatch and exits non-zero.
#define __host__
#define __device__
#include <cstdio>
#include "tiles.cuh"

using namespace fa;

static int fail(const char* what, const Mask& k, int a, int b) {
  std::printf("FAIL %s (N %d, prefix %d: %d %d)\n", what, k.N, k.prefix, a, b);
  return 1;
}

static int check(const Mask& k) {
  const int T = num_tiles(k.N), rows = T * kBlock;
  auto sees = [&](int r, int c) { return r < k.N && c < k.N && (c <= r || c < k.prefix); };
  for (int r = 0; r < rows; ++r)
    for (int c = 0; c < rows; ++c)
      if (sees(r, c) != is_visible(r, c, k)) return fail("is_visible", k, r, c);
  for (int m = 0; m < T; ++m)
    for (int j = 0; j < T; ++j) {
      bool any = false, all = true;
      for (int r = m * kBlock; r < (m + 1) * kBlock; ++r)
        for (int c = j * kBlock; c < (j + 1) * kBlock; ++c) {
          any = any || sees(r, c);
          all = all && sees(r, c);
        }
      int lo, hi;
      kv_tiles_for_q_tile(m, k, lo, hi);
      if (any != (lo <= j && j <= hi)) return fail("kv_tiles_for_q_tile", k, m, j);
      q_tiles_for_kv_tile(j, k, lo, hi);
      if (any != (lo <= m && m <= hi)) return fail("q_tiles_for_kv_tile", k, m, j);
      if (all != tile_all_visible(m, j, k)) return fail("tile_all_visible", k, m, j);
    }
  for (int w = 32; w <= 128; w *= 2)
    for (int base = 0; base < rows; base += w)
      for (int x = 0; x < rows; ++x) {
        int lo, hi;
        visible_keys(x, base, w, k, lo, hi);
        if (lo < 0 || lo > w || hi < -1 || hi > w - 1) return fail("visible_keys bounds", k, x, base);
        for (int c = 0; c < w; ++c)
          if ((lo <= c && c <= hi) != sees(x, base + c)) return fail("visible_keys", k, x, base + c);
        visible_queries(x, base, w, k, lo, hi);
        if (lo < 0 || lo > w || hi < -1 || hi > w - 1)
          return fail("visible_queries bounds", k, x, base);
        for (int r = 0; r < w; ++r)
          if ((lo <= r && r <= hi) != sees(base + r, x))
            return fail("visible_queries", k, x, base + r);
      }
  return 0;
}

int main() {
  const int Ns[6] = {1, 100, 127, 128, 129, 520};
  const int prefixes[9] = {0, 1, 31, 64, 127, 128, 129, 300, 520};
  for (int N : Ns)
    for (int p : prefixes) {
      Mask k{N, -1, 0};
      k.prefix = p < N ? p : N;
      if (check(k)) return 1;
    }
  std::printf("OK\n");
  return 0;
}
