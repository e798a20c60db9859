// fa_rope.cuh - per-head RMS norm and rotary positions of queries and keys, forward and
// backward, between a fused projection and the attention kernels.
//
// A token of the projection's output has Hq + Hk + Hv rows of D values. For a row x of a
// query or key head with gain w and a token at position pos (one number per axis):
//
//   x^ = r x, r = 1 / sqrt(mean(x^2) + eps)        (without norm: x^ = x, no gain)
//   u  = w o x^
//   y  = R u: the pair (e, f) of rotation p turns by the angle pos[axis(p)] * inv_freq[p],
//        y_e = e cos - f sin, y_f = f cos + e sin; values past rotary_dim stay
//
// and value rows are carried along, so that one launch turns (B, N, H, D) views of the
// projection into the (B, H, N, D) (or packed (total, H, D)) tensors the attention takes.
// The backward, from dy: g = R^T dy, dw = sum over rows of g o x^, and
//   dx = r (w o g - x^ mean(w o g o x^)).
//
// Both kernels are bound by device memory: each value is read and written once (the backward
// reads dy and x). A warp owns one token (or a share of its rows when there are few tokens),
// so the cosines and sines of the token are computed once, by the warp's lanes side by side,
// and serve all of its heads. A row is spread over D / 16 lanes, 16 values (two 16-byte
// vectors) each, chosen so that both members of every pair sit in one lane: lane c holds
// values 16c .. 16c+15 of an interleaved row, and of a row with split halves values
// 8c .. 8c+7 of either half. The row sums of the norm then take log2(D / 16) shuffles, and
// several rows per warp are in flight before the first is used.
//
// Angles. Positions reach 2^31 and the fp32 product pos * inv_freq would lose the angle
// itself (at position 2^20 its rounding error is 0.06 radians). The frequency is therefore
// held in turns as a 64-bit fixed-point fraction, T = inv_freq / (2 pi) mod 1 in units of
// 2^-64: pos * T in wrapping integer arithmetic is the angle in turns, exactly reduced.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "rope_args.h"
#include "sm100.cuh"

namespace fa {

// One token as a warp sees it.
struct RopeToken {
  int b;
  int n;       // row: n of entry b, or packed: the token's index
  int place;   // place in its sequence
  bool live;   // within its sequence's real length
  bool owned;  // a row the call writes (packed: some sequence covers it)
};

__device__ __forceinline__ RopeToken rope_token(const RopeArgs& a, int t) {
  RopeToken k;
  if (a.cu == nullptr) {
    k.b = t / a.N;
    k.n = t - k.b * a.N;
    k.place = k.n;
    k.owned = true;
    k.live = a.seq_len == nullptr || k.n < __ldg(a.seq_len + k.b);
    return k;
  }
  // the last sequence that starts at or before t (empty ones before it are passed over)
  int lo = 0, hi = a.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu + mid + 1) <= t) {
      lo = mid + 1;
    } else {
      hi = mid;
    }
  }
  const int start = lo < a.B ? __ldg(a.cu + lo) : 0;
  k.b = lo;
  k.n = t;
  k.place = t - start;
  k.owned = k.live = lo < a.B && k.place >= 0 && k.place < a.N;
  return k;
}

// This lane's share of a row: two vectors of eight values at offsets oa and ob, holding the
// pairs (e[i], f[i]) of rotations 8 * chunk + i when `turns`.
template <int D>
struct RopeLane {
  static constexpr int kLanes = D / 16;      // lanes per row
  static constexpr int kRows = 32 / kLanes;  // rows a warp covers at once
  int sub;    // row of the warp's kRows
  int chunk;  // lane of the row
  int oa, ob;
  bool turns;

  __device__ __forceinline__ RopeLane(const RopeArgs& a, bool interleaved) {
    const int lane = threadIdx.x & 31;
    sub = lane / kLanes;
    chunk = lane % kLanes;
    turns = 16 * chunk < a.rot;
    const bool split = turns && !interleaved;
    oa = split ? 8 * chunk : 16 * chunk;
    ob = split ? a.rot / 2 + 8 * chunk : 16 * chunk + 8;
  }
};

// The sixteen values of a lane: first and second members of its eight pairs.
struct Pairs {
  float e[8], f[8];
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <bool kInter>
__device__ __forceinline__ void unpack_pairs(const uint4& a, const uint4& b, Pairs& p) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (kInter) {
      p.e[i] = bf_lo(w[i]);
      p.f[i] = bf_hi(w[i]);
    } else {
      p.e[i] = (i & 1) ? bf_hi(w[i / 2]) : bf_lo(w[i / 2]);
      p.f[i] = (i & 1) ? bf_hi(w[4 + i / 2]) : bf_lo(w[4 + i / 2]);
    }
  }
}

template <bool kInter>
__device__ __forceinline__ void pack_pairs(const Pairs& p, uint4& a, uint4& b) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kInter) {
      w[i] = pack_bf16x2(p.e[i], p.f[i]);
      w[4 + i] = pack_bf16x2(p.e[4 + i], p.f[4 + i]);
    } else {
      w[i] = pack_bf16x2(p.e[2 * i], p.e[2 * i + 1]);
      w[4 + i] = pack_bf16x2(p.f[2 * i], p.f[2 * i + 1]);
    }
  }
  a = make_uint4(w[0], w[1], w[2], w[3]);
  b = make_uint4(w[4], w[5], w[6], w[7]);
}

// Sixteen fp32 values in the order of unpack_pairs (gains; null = ones).
template <bool kInter>
__device__ __forceinline__ void load_gain(const float* w, int oa, int ob, Pairs& p) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = w != nullptr ? __ldg(w + oa + i) : 1.f;
    v[8 + i] = w != nullptr ? __ldg(w + ob + i) : 1.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p.e[i] = kInter ? v[2 * i] : v[i];
    p.f[i] = kInter ? v[2 * i + 1] : v[8 + i];
  }
}

// The rotations a lane computes for its warp: pairs lane and lane + 32, their frequencies in
// turns (2^-64) and their axes.
template <int D>
struct RopeTurns {
  static constexpr int kOwn = D / 64;  // pairs per lane: rot / 2 <= D / 2 over 32 lanes
  unsigned long long turn[kOwn];
  int axis[kOwn];

  __device__ __forceinline__ explicit RopeTurns(const RopeArgs& a) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int p = (threadIdx.x & 31) + 32 * i;
      turn[i] = 0;
      axis[i] = 0;
      if (p < a.rot / 2) {
        double t = (double)__ldg(a.inv_freq + p) * 0.15915494309189533577;  // 1 / (2 pi)
        t -= rint(t);
        turn[i] = (unsigned long long)__double2ll_rn(t * 18446744073709551616.0);
        if (a.pair_axis != nullptr) {
          const int x = __ldg(a.pair_axis + p);
          axis[i] = x < a.axes ? x : a.axes - 1;  // (no axis of its own: the last)
        }
      }
    }
  }

  // Writes the cosine and sine of each of the token's rotations to `cs` (this warp's D / 2
  // entries of shared memory) and loads those of this lane's pairs.
  __device__ __forceinline__ void compute(const RopeArgs& a, const RopeToken& k, int t,
                                          const RopeLane<D>& ln, float2* cs, float (&c)[8],
                                          float (&s)[8]) const {
    if (a.rot == 0) return;
    __syncwarp();  // the previous token's entries have been read
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int p = (threadIdx.x & 31) + 32 * i;
      if (p < a.rot / 2) {
        const long long pos =
            a.positions != nullptr ? __ldg(a.positions + (size_t)axis[i] * a.tokens + t) : k.place;
        const unsigned long long ph = (unsigned long long)pos * turn[i];
        // the top 32 bits as a signed fraction of a turn, in half turns
        float sn, cn;
        sincospif((float)(int)(unsigned)(ph >> 32) * 4.656612873077393e-10f, &sn, &cn);
        cs[p] = make_float2(cn, sn);
      }
    }
    __syncwarp();
    if (ln.turns) {
      const float4* src = reinterpret_cast<const float4*>(cs + 8 * ln.chunk);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = src[i];
        c[2 * i] = v.x;
        s[2 * i] = v.y;
        c[2 * i + 1] = v.z;
        s[2 * i + 1] = v.w;
      }
    }
  }
};

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = D / 32; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

__device__ __forceinline__ uint4 ld_vec(const __nv_bfloat16* p) {
  return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void st_vec(__nv_bfloat16* p, const uint4& v) {
  *reinterpret_cast<uint4*>(p) = v;
}

__device__ __forceinline__ __nv_bfloat16* token_rows(const HeadRows& r, const RopeToken& k,
                                                     bool packed) {
  return r.data + (packed ? 0 : k.b * r.sb) + k.n * r.sn;
}

// Units (of kRows heads) of rows a warp takes of a kind: it takes every a.splits-th unit of
// the token's queries, keys and values counted through; first unit for this kind, with
// `before` units in the kinds before it.
__device__ __forceinline__ int first_unit(int split, int before, int splits) {
  const int m = (split - before) % splits;
  return m < 0 ? m + splits : m;
}

// ------------------------------------------------------------------------------ forward
template <int D, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_fwd_kernel(const RopeArgs a) {
  using L = RopeLane<D>;
  constexpr int U = 4;  // rows per lane in flight
  __shared__ __align__(16) float2 cs_all[kRopeWarps][D / 2];
  const int warp = threadIdx.x >> 5;
  const L ln(a, kInter);
  const RopeTurns<D> turns(a);
  const bool packed = a.cu != nullptr;
  const long long items = (long long)a.tokens * a.splits;
  for (long long it = (long long)blockIdx.x * kRopeWarps + warp; it < items;
       it += (long long)gridDim.x * kRopeWarps) {
    const int t = (int)(it / a.splits);
    const int split = (int)(it - (long long)t * a.splits);
    const RopeToken k = rope_token(a, t);
    if (!k.owned) continue;
    float c[8], s[8];
    if (k.live) turns.compute(a, k, t, ln, cs_all[warp], c, s);
    int before = 0;
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      const int heads = a.x[part].heads;
      const int units = (heads + L::kRows - 1) / L::kRows;
      const __nv_bfloat16* x = token_rows(a.x[part], k, packed);
      __nv_bfloat16* y = token_rows(a.y[part], k, packed);
      Pairs w;
      int u = first_unit(split, before, a.splits);
      if (part < 2 && a.norm && u < units) load_gain<kInter>(a.w[part], ln.oa, ln.ob, w);
      for (; u < units; u += U * a.splits) {
        uint4 va[U], vb[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int h = (u + i * a.splits) * L::kRows + ln.sub;
          va[i] = vb[i] = make_uint4(0, 0, 0, 0);
          if (h < heads && k.live) {
            va[i] = ld_vec(x + h * a.x[part].sh + ln.oa);
            vb[i] = ld_vec(x + h * a.x[part].sh + ln.ob);
          }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (u + i * a.splits >= units) break;
          const int h = (u + i * a.splits) * L::kRows + ln.sub;
          if (part < 2 && k.live) {
            Pairs p;
            unpack_pairs<kInter>(va[i], vb[i], p);
            if (a.norm) {
              float ss = 0.f;
#pragma unroll
              for (int j = 0; j < 8; ++j) ss = fmaf(p.e[j], p.e[j], fmaf(p.f[j], p.f[j], ss));
              const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                p.e[j] = p.e[j] * r * w.e[j];
                p.f[j] = p.f[j] * r * w.f[j];
              }
            }
            if (ln.turns) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float e = p.e[j], f = p.f[j];
                p.e[j] = fmaf(e, c[j], -f * s[j]);
                p.f[j] = fmaf(f, c[j], e * s[j]);
              }
            }
            pack_pairs<kInter>(p, va[i], vb[i]);
          }
          if (h < heads) {
            st_vec(y + h * a.y[part].sh + ln.oa, va[i]);
            st_vec(y + h * a.y[part].sh + ln.ob, vb[i]);
          }
        }
      }
      before += units;
    }
  }
}

// ------------------------------------------------------------------------------ backward
// Gains' gradients: every lane adds up its sixteen columns over all rows it meets, a block
// adds its lanes in a fixed order and writes (2, D) sums to a.partial, and
// fa_rope_reduce_kernel adds the blocks: no atomics, so the result is the same on every run.
template <int D, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, 2) fa_rope_bwd_kernel(const RopeArgs a) {
  using L = RopeLane<D>;
  constexpr int U = 2;
  __shared__ __align__(16) float2 cs_all[kRopeWarps][D / 2];
  __shared__ float sums[kRopeWarps][2][D];
  const int warp = threadIdx.x >> 5;
  const L ln(a, kInter);
  const RopeTurns<D> turns(a);
  const bool packed = a.cu != nullptr;
  const long long items = (long long)a.tokens * a.splits;
  Pairs acc[2];
#pragma unroll
  for (int part = 0; part < 2; ++part)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[part < 2 ? part : 0].e[j] = acc[part < 2 ? part : 0].f[j] = 0.f;
  for (long long it = (long long)blockIdx.x * kRopeWarps + warp; it < items;
       it += (long long)gridDim.x * kRopeWarps) {
    const int t = (int)(it / a.splits);
    const int split = (int)(it - (long long)t * a.splits);
    const RopeToken k = rope_token(a, t);
    if (!k.owned) continue;
    float c[8], s[8];
    if (k.live) turns.compute(a, k, t, ln, cs_all[warp], c, s);
    int before = 0;
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      const int heads = a.y[part].heads;
      const int units = (heads + L::kRows - 1) / L::kRows;
      const bool normed = part < 2 && a.norm;
      const __nv_bfloat16* x = normed ? token_rows(a.x[part], k, packed) : nullptr;
      const __nv_bfloat16* y = token_rows(a.y[part], k, packed);
      __nv_bfloat16* g = token_rows(a.g[part], k, packed);
      Pairs w;
      int u = first_unit(split, before, a.splits);
      if (normed && u < units) load_gain<kInter>(a.w[part], ln.oa, ln.ob, w);
      for (; u < units; u += U * a.splits) {
        uint4 ya[U], yb[U], xa[U], xb[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int h = (u + i * a.splits) * L::kRows + ln.sub;
          ya[i] = yb[i] = xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
          if (h < heads && k.live) {
            ya[i] = ld_vec(y + h * a.y[part].sh + ln.oa);
            yb[i] = ld_vec(y + h * a.y[part].sh + ln.ob);
            if (normed) {
              xa[i] = ld_vec(x + h * a.x[part].sh + ln.oa);
              xb[i] = ld_vec(x + h * a.x[part].sh + ln.ob);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (u + i * a.splits >= units) break;
          const int h = (u + i * a.splits) * L::kRows + ln.sub;
          if (part < 2 && k.live) {
            Pairs d;
            unpack_pairs<kInter>(ya[i], yb[i], d);
            if (ln.turns) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float e = d.e[j], f = d.f[j];
                d.e[j] = fmaf(e, c[j], f * s[j]);
                d.f[j] = fmaf(f, c[j], -e * s[j]);
              }
            }
            if (a.norm) {
              Pairs p;
              unpack_pairs<kInter>(xa[i], xb[i], p);
              float ss = 0.f, sx = 0.f;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                ss = fmaf(p.e[j], p.e[j], fmaf(p.f[j], p.f[j], ss));
                sx = fmaf(d.e[j] * w.e[j], p.e[j], fmaf(d.f[j] * w.f[j], p.f[j], sx));
              }
              // (lanes of rows past the last head hold zeros: they add nothing)
              const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
              const float m = row_sum<D>(sx) * r * r * (1.f / D);  // times x: x^ mean(...)
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                acc[part < 2 ? part : 0].e[j] = fmaf(d.e[j], p.e[j] * r, acc[part < 2 ? part : 0].e[j]);
                acc[part < 2 ? part : 0].f[j] = fmaf(d.f[j], p.f[j] * r, acc[part < 2 ? part : 0].f[j]);
                d.e[j] = r * fmaf(-m, p.e[j], d.e[j] * w.e[j]);
                d.f[j] = r * fmaf(-m, p.f[j], d.f[j] * w.f[j]);
              }
            }
            pack_pairs<kInter>(d, ya[i], yb[i]);
          }
          if (h < heads) {
            st_vec(g + h * a.g[part].sh + ln.oa, ya[i]);
            st_vec(g + h * a.g[part].sh + ln.ob, yb[i]);
          }
        }
      }
      before += units;
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int part = 0; part < 2; ++part) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float e = acc[part < 2 ? part : 0].e[j], f = acc[part < 2 ? part : 0].f[j];
#pragma unroll
      for (int off = L::kLanes; off < 32; off <<= 1) {
        e += __shfl_xor_sync(0xffffffffu, e, off);
        f += __shfl_xor_sync(0xffffffffu, f, off);
      }
      if (ln.sub == 0) {
        // the columns of unpack_pairs' members
        const int ce = kInter ? (j < 4 ? ln.oa + 2 * j : ln.ob + 2 * (j - 4)) : ln.oa + j;
        const int cf = kInter ? ce + 1 : ln.ob + j;
        sums[warp][part][ce] = e;
        sums[warp][part][cf] = f;
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kRopeThreads) {
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kRopeWarps; ++q) v += (&sums[q][0][0])[i];
    a.partial[(size_t)blockIdx.x * 2 * D + i] = v;
  }
}

// Adds the blocks' sums: block b takes columns 32b .. 32b+31 of the 2 D (queries' gains, then
// keys'), each warp every 32nd block.
template <int D>
__global__ void __launch_bounds__(1024)
    fa_rope_reduce_kernel(const float* partial, int blocks, float* dwq, float* dwk) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float v = 0.f;
  for (int b = warp; b < blocks; b += 32) v += partial[(size_t)b * 2 * D + col];
  part[warp][lane] = v;
  __syncthreads();
  if (warp != 0) return;
  float sum = 0.f;
#pragma unroll
  for (int q = 0; q < 32; ++q) sum += part[q][lane];
  float* out = col < D ? dwq : dwk;
  if (out != nullptr) out[col < D ? col : col - D] = sum;
}

}  // namespace fa
