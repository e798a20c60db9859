"""fa_fwd_score and fa_bwd_score without a GPU, and the tile ranges of a prefix by brute force."""
import ctypes
import shutil
import subprocess

import pytest

from exact_attention_126_b200 import build, fa

A = 0x10000
W = fa.fa_window_t


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fa.library()


def S(**kw):
    return ctypes.byref(fa.fa_score_t(**kw))


def test_refusals(lib):
    def fwd(score, opt=None, scale=0.125, causal=1, window=(-1, -1), q=A, d=64, N=128):
        return lib.fa_fwd_score(q, A, A, A, A, 1, 2, N, d, scale, causal, W(*window), opt, score,
                                None)

    def bwd(score, opt=None, causal=1, ws=A, n=1 << 20, dq=A):
        return lib.fa_bwd_score(A, A, A, A, A, A, dq, A, A, 1, 2, 128, 64, 0.125, causal,
                                W(-1, -1), opt, score, ws, n, None)

    for f in (fwd, bwd):
        assert f(S(softcap=-1.0)) == 1
        assert f(S(softcap=float("nan"))) == 1
        assert f(S(softcap=float("inf"))) == 1
        assert f(S(softcap=1e-40)) == 1
        assert f(S(prefix_lengths=A + 2)) == 3
        assert f(S(prefix_lengths=A), causal=0) == 1
        assert f(S(softcap=5.0), fa.fa_options_t(dropout_p=1.0)) == 1
        assert f(S(softcap=5.0), fa.fa_options_t(flags=1)) == 2
        assert f(S(prefix_lengths=A), fa.fa_options_t(flags=1)) == 2
    assert fwd(S(softcap=1e6), scale=0.1) == 1      # scale / c outside [1e-6, 1e6]
    assert fwd(S(softcap=1e-8), scale=0.1) == 1
    assert fwd(S(prefix_lengths=A), window=(5, 0)) == 2
    assert fwd(S(softcap=5.0), q=None) == 1
    assert fwd(S(softcap=5.0), q=A + 8) == 3
    assert fwd(S(softcap=5.0), d=96) == 2
    assert fwd(S(softcap=5.0), scale=0.0) == 1
    assert fwd(S(softcap=-5.0), N=0, q=None) == 0   # an empty problem launches nothing
    assert bwd(S(softcap=5.0), dq=None) == 1
    assert bwd(S(softcap=5.0), ws=None) == 1
    assert bwd(S(softcap=5.0), n=8) == 4


def test_struct_layout():
    assert ctypes.sizeof(fa.fa_score_t) == 16
    assert (fa.fa_score_t.prefix_lengths.offset, fa.fa_score_t.softcap.offset) == (0, 8)


PREFIX_CHECK = r"""
#define __host__
#define __device__
#include <cstdio>
#include <initializer_list>
#include "tiles.cuh"
using namespace fa;
int main() {
  const int Ns[] = {1, 5, 127, 128, 129, 300, 512};
  for (int N : Ns)
    for (int P : {0, 1, 64, 127, 128, 129, 200, N - 1, N}) {
      if (P < 0 || P > N) continue;
      const Mask k{N, -1, 0, P};
      const int T = num_tiles(N);
      for (int r = 0; r < N; ++r)
        for (int c = 0; c < N; ++c)
          if (is_visible(r, c, k) != (c <= r || c < P)) return std::puts("visible"), 1;
      for (int t = 0; t < T; ++t) {
        int lo, hi, want_lo = T, want_hi = -1, qlo, qhi, wq_lo = T, wq_hi = -1;
        kv_tiles_for_q_tile(t, k, lo, hi);
        q_tiles_for_kv_tile(t, k, qlo, qhi);
        for (int u = 0; u < T; ++u) {
          bool all = true, any = false, any_t = false;
          for (int r = t * kBlock; r < (t + 1) * kBlock; ++r)
            for (int c = u * kBlock; c < (u + 1) * kBlock; ++c) {
              any |= is_visible(r, c, k);
              all &= is_visible(r, c, k);
              any_t |= is_visible(c, r, k);  // query tile u, key tile t
            }
          if (any) { if (u < want_lo) want_lo = u; if (u > want_hi) want_hi = u; }
          if (any_t) { if (u < wq_lo) wq_lo = u; if (u > wq_hi) wq_hi = u; }
          if (tile_all_visible(t, u, k) && !all) return std::puts("all"), 1;
          if (all && !tile_all_visible(t, u, k)) return std::puts("not all"), 1;
        }
        if (lo != want_lo || hi != want_hi) return std::puts("key range"), 1;
        if (qlo != wq_lo || qhi != wq_hi) return std::puts("query range"), 1;
      }
      for (int width : {32, 64, 128})
        for (int base = 0; base < T * kBlock; base += width)
          for (int r = 0; r < T * kBlock; ++r) {
            int lo, hi, a, b;
            visible_keys(r, base, width, k, lo, hi);
            visible_queries(r, base, width, k, a, b);
            for (int c = 0; c < width; ++c) {
              if ((c >= lo && c <= hi) != is_visible(r, base + c, k)) return std::puts("keys"), 1;
              if ((c >= a && c <= b) != is_visible(base + c, r, k)) return std::puts("queries"), 1;
            }
          }
    }
  return 0;
}
"""


def test_tiles_of_a_prefix(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src = tmp_path / "prefix.cpp"
    src.write_text(PREFIX_CHECK)
    exe = tmp_path / "prefix"
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", build.CSRC, str(src), "-o", str(exe)],
                   check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout
