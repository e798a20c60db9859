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
// reads dy and x). A row is spread over D / 8 lanes, eight values each, chosen so that both
// members of every pair sit in one lane: lane c holds values 8c .. 8c+7 of an interleaved row,
// and of a row with split halves values 4c .. 4c+3 of either half. A warp covers 32 / (D / 8)
// rows at once (a unit) and owns one token (or a share of its units when tokens are few): the
// cosines and sines of the token are computed once, by the lanes side by side, and serve all of
// its heads. Units go in batches, queries first, then keys, then values; the loads of a batch are
// issued before the previous one is worked on.
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

// One token: where its rows lie and whether it takes part.
struct RopeToken {
  int b;
  int n;       // row: n of entry b, or packed: the token's index
  int place;   // place in its sequence
  bool live;   // within its sequence's real length
  bool owned;  // its rows are written (packed: some sequence covers it, or a.fill)
};

__device__ __forceinline__ RopeToken rope_token(const RopeArgs& a, int t) {
  RopeToken k;
  if (a.cu == nullptr) {
    k.b = t / a.N;
    k.n = t - k.b * a.N;
    k.place = k.n;
    k.owned = t < a.tokens;
    k.live = k.owned && (a.seq_len == nullptr || k.n < __ldg(a.seq_len + k.b));
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
  k.b = 0;
  k.n = t;
  k.place = t - start;
  k.live = t < a.tokens && lo < a.B && k.place >= 0 && k.place < a.N;
  k.owned = k.live || (a.fill && t < a.tokens);
  return k;
}

// This lane's share of a row: values at offsets oa .. oa+3 and ob .. ob+3, holding the pairs
// (e[i], f[i]) of rotations 4 * chunk + i when `turns`.
template <int D, bool kInter>
struct RopeLane {
  static constexpr int kLanes = D / 8;       // lanes per row
  static constexpr int kRows = 32 / kLanes;  // rows of a unit
  int sub;    // row of the unit
  int chunk;  // lane of the row
  int oa, ob;
  bool turns;

  __device__ __forceinline__ explicit RopeLane(const RopeArgs& a) {
    const int lane = threadIdx.x & 31;
    sub = lane / kLanes;
    chunk = lane % kLanes;
    turns = 8 * chunk < a.rot;
    const bool split = turns && !kInter;
    oa = split ? 4 * chunk : 8 * chunk;
    ob = split ? a.rot / 2 + 4 * chunk : 8 * chunk + 4;
  }
  // the column of member i (0 .. 3) of this lane's e and f
  __device__ __forceinline__ int col_e(int i) const { return kInter ? oa + 2 * i : oa + i; }
  __device__ __forceinline__ int col_f(int i) const { return kInter ? oa + 2 * i + 1 : ob + i; }
};

// A lane's eight values as they lie in memory.
struct RopeRaw {
  uint2 a, b;
};

// The eight values: first and second members of four pairs, two pairs per element.
struct Pairs {
  float2 e[2], f[2];
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <bool kInter>
__device__ __forceinline__ Pairs unpack_pairs(const RopeRaw& r) {
  Pairs p;
  if (kInter) {
    p.e[0] = make_float2(bf_lo(r.a.x), bf_lo(r.a.y));
    p.f[0] = make_float2(bf_hi(r.a.x), bf_hi(r.a.y));
    p.e[1] = make_float2(bf_lo(r.b.x), bf_lo(r.b.y));
    p.f[1] = make_float2(bf_hi(r.b.x), bf_hi(r.b.y));
  } else {
    p.e[0] = make_float2(bf_lo(r.a.x), bf_hi(r.a.x));
    p.e[1] = make_float2(bf_lo(r.a.y), bf_hi(r.a.y));
    p.f[0] = make_float2(bf_lo(r.b.x), bf_hi(r.b.x));
    p.f[1] = make_float2(bf_lo(r.b.y), bf_hi(r.b.y));
  }
  return p;
}

template <bool kInter>
__device__ __forceinline__ RopeRaw pack_pairs(const Pairs& p) {
  RopeRaw r;
  if (kInter) {
    r.a = make_uint2(pack_bf16x2(p.e[0].x, p.f[0].x), pack_bf16x2(p.e[0].y, p.f[0].y));
    r.b = make_uint2(pack_bf16x2(p.e[1].x, p.f[1].x), pack_bf16x2(p.e[1].y, p.f[1].y));
  } else {
    r.a = make_uint2(pack_bf16x2(p.e[0].x, p.e[0].y), pack_bf16x2(p.e[1].x, p.e[1].y));
    r.b = make_uint2(pack_bf16x2(p.f[0].x, p.f[0].y), pack_bf16x2(p.f[1].x, p.f[1].y));
  }
  return r;
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

  // Writes the cosine and sine of each rotation of token t (the place-th of its sequence) to `cs`
  // (D / 2 entries of shared memory); by all lanes of the warp.
  __device__ __forceinline__ void fill(const RopeArgs& a, int place, int t, float2* cs) const {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int p = (threadIdx.x & 31) + 32 * i;
      if (p < a.rot / 2) {
        const long long pos =
            a.positions != nullptr ? __ldg(a.positions + (size_t)axis[i] * a.tokens + t) : place;
        const unsigned long long ph = (unsigned long long)pos * turn[i];
        // the top 32 bits as a signed fraction of a turn, in half turns
        float sn, cn;
        sincospif((float)(int)(unsigned)(ph >> 32) * 4.656612873077393e-10f, &sn, &cn);
        cs[p] = make_float2(cn, sn);
      }
    }
  }

  // Loads those of this lane's pairs.
  template <typename Lane>
  __device__ __forceinline__ void read(const Lane& ln, const float2* cs, float2 (&c)[2],
                                       float2 (&s)[2]) const {
    if (!ln.turns) return;
    const float4* src = reinterpret_cast<const float4*>(cs + 4 * ln.chunk);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 v = src[i];
      c[i] = make_float2(v.x, v.z);
      s[i] = make_float2(v.y, v.w);
    }
  }

  template <typename Lane>
  __device__ __forceinline__ void compute(const RopeArgs& a, const RopeToken& k, int t,
                                          const Lane& ln, float2* cs, float2 (&c)[2],
                                          float2 (&s)[2]) const {
    if (a.rot == 0) return;
    __syncwarp();  // the previous token's entries have been read
    fill(a, k.place, t, cs);
    __syncwarp();
    read(ln, cs, c, s);
  }
};

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = D / 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// This lane's eight values of the first row it takes of a kind, and of the rows after it: steps of
// `step` 8-byte units (strides are multiples of 8 values, and a kind's rows span less than 2^34
// values, checked on the host: 32-bit products do).
struct RowWalk {
  const uint2* p;
  unsigned step;
  __device__ __forceinline__ const uint2* at(int i) const { return p + (size_t)((unsigned)i * step); }
};
__device__ __forceinline__ RowWalk walk_rows(const HeadRows& r, const RopeToken& k, int head,
                                             int heads_per_step) {
  return RowWalk{reinterpret_cast<const uint2*>(r.data) +
                     ((unsigned)k.b * (unsigned)(r.sb >> 2) + (unsigned)k.n * (unsigned)(r.sn >> 2) +
                      (unsigned)head * (unsigned)(r.sh >> 2)),
                 (unsigned)heads_per_step * (unsigned)(r.sh >> 2)};
}

template <bool kInter, typename Lane>
__device__ __forceinline__ RopeRaw load_row(const uint2* p, const Lane& ln) {
  RopeRaw r;
  if (kInter) {
    const uint4 v = *reinterpret_cast<const uint4*>(p + 2 * ln.chunk);
    r.a = make_uint2(v.x, v.y);
    r.b = make_uint2(v.z, v.w);
  } else {
    r.a = p[ln.oa >> 2];
    r.b = p[ln.ob >> 2];
  }
  return r;
}
template <bool kInter, typename Lane>
__device__ __forceinline__ void store_row(const uint2* p, const Lane& ln, const RopeRaw& r) {
  uint2* q = const_cast<uint2*>(p);
  if (kInter) {
    *reinterpret_cast<uint4*>(q + 2 * ln.chunk) = make_uint4(r.a.x, r.a.y, r.b.x, r.b.y);
  } else {
    q[ln.oa >> 2] = r.a;
    q[ln.ob >> 2] = r.b;
  }
}

// The gains of queries and keys in shared memory, each lane's e and f values side by side.
template <int D, typename Lane>
__device__ __forceinline__ void stage_gains(const RopeArgs& a, const Lane& ln,
                                            float4 (*gains)[D / 8][2]) {
  if (threadIdx.x < 2 * (D / 8)) {
    const int part = threadIdx.x / (D / 8);
    // (threads 0 .. D/8-1 of the block are lanes of chunk threadIdx % (D/8))
    const float* w = a.norm ? a.w[part] : nullptr;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = w != nullptr ? __ldg(w + ln.col_e(i)) : 1.f;
      v[4 + i] = w != nullptr ? __ldg(w + ln.col_f(i)) : 1.f;
    }
    gains[part][ln.chunk][0] = make_float4(v[0], v[1], v[2], v[3]);
    gains[part][ln.chunk][1] = make_float4(v[4], v[5], v[6], v[7]);
  }
  __syncthreads();
}
template <int D, typename Lane>
__device__ __forceinline__ Pairs lane_gain(const float4 (*gains)[D / 8][2], int part,
                                           const Lane& ln) {
  const float4 e = gains[part][ln.chunk][0], f = gains[part][ln.chunk][1];
  Pairs w;
  w.e[0] = make_float2(e.x, e.y);
  w.e[1] = make_float2(e.z, e.w);
  w.f[0] = make_float2(f.x, f.y);
  w.f[1] = make_float2(f.z, f.w);
  return w;
}

// The units of one kind that a warp takes of its token: heads first, first + splits * kRows, ...
struct RopeShare {
  int head;   // this lane's first head
  int units;  // steps it takes (some lanes may have no head in the last)
};
template <typename Lane>
__device__ __forceinline__ RopeShare rope_share(int heads, int split, int splits, const Lane& ln) {
  const int all = (heads + Lane::kRows - 1) / Lane::kRows;
  return RopeShare{split * Lane::kRows + ln.sub, all > split ? (all - split + splits - 1) / splits : 0};
}

// ------------------------------------------------------------------------------ forward
template <int D, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocksPerSm) fa_rope_fwd_kernel(const RopeArgs a) {
  using L = RopeLane<D, kInter>;
  constexpr int U = 4;  // units of a batch
  __shared__ __align__(16) float2 cs_all[kRopeWarps][D / 2];
  __shared__ float4 gains[2][D / 8][2];
  float2* const cs = cs_all[threadIdx.x >> 5];
  const L ln(a);
  stage_gains<D>(a, ln, gains);
  const RopeTurns<D> turns(a);
  const long long items = (long long)a.tokens * a.splits;
  const int stride = a.splits * L::kRows;
  for (long long item = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5); item < items;
       item += (long long)gridDim.x * kRopeWarps) {
    const int t = a.splits == 1 ? (int)item : (int)(item / a.splits);
    const int split = (int)(item - (long long)t * a.splits);
    const RopeToken k = rope_token(a, t);
    if (!k.owned) continue;
    RopeRaw now[U], then[U];
    auto load = [&](int part, int u, RopeRaw (&raw)[U]) {
      const RopeShare sh = rope_share(a.x[part].heads, split, a.splits, ln);
      const RowWalk w = walk_rows(a.x[part], k, sh.head, stride);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        raw[i].a = raw[i].b = make_uint2(0, 0);
        if (k.live && sh.head + (u + i) * stride < a.x[part].heads)
          raw[i] = load_row<kInter>(w.at(u + i), ln);
      }
    };
    load(0, 0, now);
    float2 c[2], s[2];
    if (k.live) turns.compute(a, k, t, ln, cs, c, s);
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      const int heads = a.y[part].heads;
      const RopeShare sh = rope_share(heads, split, a.splits, ln);
      if (sh.units == 0 && part < 2) load(part + 1, 0, now);
      const RowWalk wy = walk_rows(a.y[part], k, sh.head, stride);
      for (int u = 0; u < sh.units; u += U) {
        if (u + U < sh.units) {
          load(part, u + U, then);
        } else if (part < 2) {
          load(part + 1, 0, then);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (u + i >= sh.units) break;
          RopeRaw r = now[i];
          if (part < 2 && k.live) {
            Pairs p = unpack_pairs<kInter>(r);
            if (a.norm) {
              float2 ss = __fmul2_rn(p.e[0], p.e[0]);
              ss = __ffma2_rn(p.e[1], p.e[1], ss);
              ss = __ffma2_rn(p.f[0], p.f[0], ss);
              ss = __ffma2_rn(p.f[1], p.f[1], ss);
              const float2 rs = both(rsqrtf(row_sum<D>(ss.x + ss.y) * (1.f / D) + a.eps));
              const Pairs w = lane_gain<D>(gains, part, ln);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                p.e[j] = __fmul2_rn(__fmul2_rn(p.e[j], rs), w.e[j]);
                p.f[j] = __fmul2_rn(__fmul2_rn(p.f[j], rs), w.f[j]);
              }
            }
            if (ln.turns) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float2 e = p.e[j], f = p.f[j];
                p.e[j] = make_float2(fmaf(e.x, c[j].x, -f.x * s[j].x),
                                     fmaf(e.y, c[j].y, -f.y * s[j].y));
                p.f[j] = __ffma2_rn(e, s[j], __fmul2_rn(f, c[j]));
              }
            }
            r = pack_pairs<kInter>(p);
          }
          if (sh.head + (u + i) * stride < heads) store_row<kInter>(wy.at(u + i), ln, r);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) now[i] = then[i];
      }
    }
  }
}

// ------------------------------------------------------------------------------ backward
// Gains' gradients: every lane adds up its eight columns over all rows it meets, a block
// adds its lanes in a fixed order and writes (2, D) sums to a.partial, and
// fa_rope_reduce_kernel adds the blocks: no atomics, so the result is the same on every run.
template <int D, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocksPerSm) fa_rope_bwd_kernel(const RopeArgs a) {
  using L = RopeLane<D, kInter>;
  constexpr int U = 2;
  __shared__ __align__(16) float2 cs_all[kRopeWarps][D / 2];
  __shared__ float4 gains[2][D / 8][2];
  __shared__ float sums[kRopeWarps][2][D];
  const int warp = threadIdx.x >> 5;
  float2* const cs = cs_all[warp];
  const L ln(a);
  stage_gains<D>(a, ln, gains);
  const RopeTurns<D> turns(a);
  const long long items = (long long)a.tokens * a.splits;
  const int stride = a.splits * L::kRows;
  Pairs acc[2];
#pragma unroll
  for (int part = 0; part < 2; ++part)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[part].e[j] = acc[part].f[j] = both(0.f);
  for (long long item = (long long)blockIdx.x * kRopeWarps + warp; item < items;
       item += (long long)gridDim.x * kRopeWarps) {
    const int t = a.splits == 1 ? (int)item : (int)(item / a.splits);
    const int split = (int)(item - (long long)t * a.splits);
    const RopeToken k = rope_token(a, t);
    if (!k.owned) continue;
    RopeRaw dy0[U], dy1[U], x0[U], x1[U];
    auto load = [&](int part, int u, RopeRaw (&dy)[U], RopeRaw (&x)[U]) {
      const RopeShare sh = rope_share(a.y[part].heads, split, a.splits, ln);
      const RowWalk wy = walk_rows(a.y[part], k, sh.head, stride);
      const RowWalk wx = walk_rows(a.x[part], k, sh.head, stride);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        dy[i].a = dy[i].b = x[i].a = x[i].b = make_uint2(0, 0);
        if (k.live && sh.head + (u + i) * stride < a.y[part].heads) {
          dy[i] = load_row<kInter>(wy.at(u + i), ln);
          if (part < 2 && a.norm) x[i] = load_row<kInter>(wx.at(u + i), ln);
        }
      }
    };
    load(0, 0, dy0, x0);
    float2 c[2], s[2];
    if (k.live) turns.compute(a, k, t, ln, cs, c, s);
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      const int heads = a.g[part].heads;
      const RopeShare sh = rope_share(heads, split, a.splits, ln);
      if (sh.units == 0 && part < 2) load(part + 1, 0, dy0, x0);
      const RowWalk wg = walk_rows(a.g[part], k, sh.head, stride);
      for (int u = 0; u < sh.units; u += U) {
        if (u + U < sh.units) {
          load(part, u + U, dy1, x1);
        } else if (part < 2) {
          load(part + 1, 0, dy1, x1);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (u + i >= sh.units) break;
          RopeRaw r = dy0[i];
          if (part < 2 && k.live) {
            Pairs d = unpack_pairs<kInter>(r);
            if (ln.turns) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float2 e = d.e[j], f = d.f[j];
                d.e[j] = __ffma2_rn(f, s[j], __fmul2_rn(e, c[j]));
                d.f[j] = make_float2(fmaf(f.x, c[j].x, -e.x * s[j].x),
                                     fmaf(f.y, c[j].y, -e.y * s[j].y));
              }
            }
            if (a.norm) {
              const Pairs p = unpack_pairs<kInter>(x0[i]);
              const Pairs w = lane_gain<D>(gains, part, ln);
              float2 ss = __fmul2_rn(p.e[0], p.e[0]);
              ss = __ffma2_rn(p.e[1], p.e[1], ss);
              ss = __ffma2_rn(p.f[0], p.f[0], ss);
              ss = __ffma2_rn(p.f[1], p.f[1], ss);
              Pairs gx;  // g o x: the gain's gradient up to the row's r
              float2 sx = both(0.f);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                gx.e[j] = __fmul2_rn(d.e[j], p.e[j]);
                gx.f[j] = __fmul2_rn(d.f[j], p.f[j]);
                sx = __ffma2_rn(gx.e[j], w.e[j], __ffma2_rn(gx.f[j], w.f[j], sx));
              }
              float rs = rsqrtf(row_sum<D>(ss.x + ss.y) * (1.f / D) + a.eps);
              // (rows of no head add nothing, also with eps = 0)
              if (sh.head + (u + i) * stride >= heads) rs = 0.f;
              const float2 m = both(row_sum<D>(sx.x + sx.y) * rs * rs * (-1.f / D));
              const float2 r2 = both(rs);
              Pairs& sum = acc[part < 2 ? part : 0];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                sum.e[j] = __ffma2_rn(gx.e[j], r2, sum.e[j]);
                sum.f[j] = __ffma2_rn(gx.f[j], r2, sum.f[j]);
                d.e[j] = __fmul2_rn(__ffma2_rn(p.e[j], m, __fmul2_rn(d.e[j], w.e[j])), r2);
                d.f[j] = __fmul2_rn(__ffma2_rn(p.f[j], m, __fmul2_rn(d.f[j], w.f[j])), r2);
              }
            }
            r = pack_pairs<kInter>(d);
          }
          if (sh.head + (u + i) * stride < heads) store_row<kInter>(wg.at(u + i), ln, r);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          dy0[i] = dy1[i];
          x0[i] = x1[i];
        }
      }
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int part = 0; part < 2; ++part) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float e = j & 1 ? acc[part].e[j / 2].y : acc[part].e[j / 2].x;
      float f = j & 1 ? acc[part].f[j / 2].y : acc[part].f[j / 2].x;
#pragma unroll
      for (int off = L::kLanes; off < 32; off <<= 1) {
        e += __shfl_xor_sync(0xffffffffu, e, off);
        f += __shfl_xor_sync(0xffffffffu, f, off);
      }
      if (ln.sub == 0) {
        sums[warp][part][ln.col_e(j)] = e;
        sums[warp][part][ln.col_f(j)] = f;
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

// ------------------------------------------------------------------------------ tiles
// The same two computations on large problems, through shared memory: a tile is kTileTokens
// consecutive tokens of kTileHeads heads of one kind, [head][token][D], which the copy engine
// fetches from and puts to tensors of any strides. One thread issues the loads of a ring of
// stages, eight warps work on a full stage in place, and one thread issues the stores of the
// finished ones, so that loads and stores run while other stages are worked on, whatever the
// latency. A warp owns kRows tokens of each tile, one row per D / 8 lanes, and steps through the
// heads: cosines, sines and the gain stay in registers. Items (all heads of a kind for a tile of
// tokens) go queries first, then keys, then values, dealt to persistent blocks.
//   B32 N2048, 3 x 16 heads of 64: forward 143 us (805 MB, 5.6 TB/s), backward 193 us (1.07 GB,
//   5.6 TB/s); the kernels above take 160 and 252 us. Bound by device memory: a plain copy runs at
//   6.55 TB/s, rows of 128 bytes on one side cost the rest.
struct RopeMaps {
  CUtensorMap in[3];   // forward: x; backward: the incoming gradients y
  CUtensorMap out[3];  // forward: y; backward: g
  CUtensorMap x[2];    // backward with norm: x
};

template <int D, bool kBwd>
struct RopeTile {
  static constexpr int kRows = 32 / (D / 8);          // tokens of a warp
  static constexpr int kTokens = kRows * kRopeWarps;  // 32 (D = 64) or 16
  static constexpr int kHeads = 4;
  static constexpr int kBytes = kHeads * kTokens * D * 2;  // 16 KB
  static constexpr int kStage = kBwd ? 2 * kBytes : kBytes;
  static constexpr int kStages = kBwd ? 3 : 6;
  static constexpr int kThreads = kRopeThreads + 64;  // eight working warps, load warp, store warp
  static constexpr int kBar = kStages * kStage;       // full, done, empty barriers
  static constexpr int kMisc = (kBar + 3 * kStages * 8 + 15) / 16 * 16;
  static constexpr int kCs = kMisc + 16;              // cosines and sines of each warp's tokens
  static constexpr int kSums = kCs + kRopeWarps * kRows * (D / 2) * 8;
  static_assert(kCs % 16 == 0, "float4 loads of the cosines and sines");
  static constexpr int kSmemBytes = kSums + (kBwd ? kRopeWarps * 2 * D * 4 : 0) + 128;
};

// The items of a call: tiles of tokens per kind.
struct RopeItems {
  int per_entry;  // tiles of an entry's N rows (packed: of the tensor)
  int tiles;
  int ends[3];    // items of queries, of queries and keys, of all
};

template <int kTokens>
__device__ __forceinline__ RopeItems rope_items(const RopeArgs& a, const HeadRows (&y)[3]) {
  RopeItems r;
  const int rows = a.cu != nullptr ? a.tokens : a.N;
  r.per_entry = (rows + kTokens - 1) / kTokens;
  r.tiles = a.cu != nullptr ? r.per_entry : r.per_entry * a.B;
  int n = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (y[i].heads > 0) n += r.tiles;
    r.ends[i] = n;
  }
  return r;
}

// Item `it`: kind, entry, first row (n0 of entry b) and steps of kHeads heads.
struct RopeItem {
  int part, b, n0, steps;
};
template <int kTokens, int kHeads>
__device__ __forceinline__ RopeItem rope_item(const RopeItems& r, const HeadRows (&y)[3], int it) {
  RopeItem k;
  k.part = it < r.ends[0] ? 0 : (it < r.ends[1] ? 1 : 2);
  const int t = it - (k.part == 0 ? 0 : r.ends[k.part - 1]);
  k.b = t / r.per_entry;
  k.n0 = (t - k.b * r.per_entry) * kTokens;
  k.steps = (y[k.part].heads + kHeads - 1) / kHeads;
  return k;
}

// The token of row n0 + lane of an item's tile, for lanes below kTokens; `whole` (warp-wide):
// every row of the tile inside the tensor is one the call writes, so that the tile leaves as one.
template <int kTokens>
__device__ __forceinline__ RopeToken tile_token(const RopeArgs& a, const RopeItem& k, bool& whole) {
  const int lane = threadIdx.x & 31;
  const int n = k.n0 + (lane < kTokens ? lane : 0);
  RopeToken t;
  if (a.cu != nullptr) {
    t = rope_token(a, n < a.tokens ? n : a.tokens - 1);
    if (n >= a.tokens) t.live = t.owned = false;
    whole = __all_sync(0xffffffffu, t.owned || n >= a.tokens);
  } else {
    t.b = k.b;
    t.n = t.place = n;
    t.owned = n < a.N;
    t.live = t.owned && (a.seq_len == nullptr || n < __ldg(a.seq_len + k.b));
    whole = true;
  }
  return t;
}

// A lane's eight values of a row in shared memory at `p` (bytes). (At D = 64 the rows of a warp
// lie 128 bytes apart and the halves of two rows meet in the same banks; taking them in turns costs
// more instructions than it saves wavefronts: forward 145 -> 149 us on the problem above.)
template <bool kInter, typename Lane>
__device__ __forceinline__ RopeRaw tile_load(const uint8_t* p, const Lane& ln) {
  RopeRaw r;
  if (kInter) {
    const uint4 v = *reinterpret_cast<const uint4*>(p + 16 * ln.chunk);
    r.a = make_uint2(v.x, v.y);
    r.b = make_uint2(v.z, v.w);
  } else {
    r.a = *reinterpret_cast<const uint2*>(p + 2 * ln.oa);
    r.b = *reinterpret_cast<const uint2*>(p + 2 * ln.ob);
  }
  return r;
}
template <bool kInter, typename Lane>
__device__ __forceinline__ void tile_store(uint8_t* p, const Lane& ln, const RopeRaw& r) {
  if (kInter) {
    *reinterpret_cast<uint4*>(p + 16 * ln.chunk) = make_uint4(r.a.x, r.a.y, r.b.x, r.b.y);
  } else {
    *reinterpret_cast<uint2*>(p + 2 * ln.oa) = r.a;
    *reinterpret_cast<uint2*>(p + 2 * ln.ob) = r.b;
  }
}

template <int D, bool kInter, bool kBwd>
__global__ void __launch_bounds__(RopeTile<D, kBwd>::kThreads, kRopeBlocksPerSm)
    fa_rope_tile_kernel(const __grid_constant__ RopeMaps maps, const RopeArgs a) {
  using T = RopeTile<D, kBwd>;
  using L = RopeLane<D, kInter>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                             ~uintptr_t(127));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::kMisc);
  auto full = [&](int s) -> uint32_t { return sb + T::kBar + 8u * s; };
  auto done = [&](int s) -> uint32_t { return sb + T::kBar + 8u * (T::kStages + s); };
  auto empty = [&](int s) -> uint32_t { return sb + T::kBar + 8u * (2 * T::kStages + s); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(done(s), kRopeWarps);
      mbar_init(empty(s), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (kBwd)
    for (int i = threadIdx.x; i < kRopeWarps * 2 * D; i += T::kThreads)
      reinterpret_cast<float*>(smem + T::kSums)[i] = 0.f;
  __syncthreads();
  const RopeItems items = rope_items<T::kTokens>(a, a.y);

  if (warp == kRopeWarps) {
    // ------------------------------------------------------------------ loads
    if (lane == 0) {
      int n = 0;
      bool ok = true;
      for (int it = blockIdx.x; ok && it < items.ends[2]; it += gridDim.x) {
        const RopeItem k = rope_item<T::kTokens, T::kHeads>(items, a.y, it);
        const bool with_x = kBwd && k.part < 2 && a.norm;
        // a tile wholly past its entry's real length is only filled with zeros
        const bool dead = a.seq_len != nullptr && k.n0 >= __ldg(a.seq_len + k.b);
        for (int g = 0; g < k.steps; ++g, ++n) {
          const int s = n % T::kStages;
          if (!mbar_wait(empty(s), ((n / T::kStages) & 1) ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t dst = sb + s * T::kStage;
          if (dead) {
            mbar_arrive(full(s));  // nothing to fetch
            continue;
          }
          mbar_arrive_expect_tx(full(s), with_x ? 2 * T::kBytes : T::kBytes);
          tma_load_4d(dst, &maps.in[k.part], full(s), 0, k.n0, g * T::kHeads, k.b);
          if (with_x)
            tma_load_4d(dst + T::kBytes, &maps.x[k.part < 2 ? k.part : 0], full(s), 0, k.n0,
                        g * T::kHeads, k.b);
        }
      }
      // Drain: every copy issued must have landed before the block may exit.
      for (int s = 0; s < T::kStages; ++s)
        if (n > s) mbar_wait(full(s), ((n - 1 - s) / T::kStages) & 1, nullptr);
    }
  } else if (warp == kRopeWarps + 1) {
    // ------------------------------------------------------------------ stores
    int n = 0;
    bool ok = true;
    for (int it = blockIdx.x; ok && it < items.ends[2]; it += gridDim.x) {
      const RopeItem k = rope_item<T::kTokens, T::kHeads>(items, a.y, it);
      bool whole;
      tile_token<T::kTokens>(a, k, whole);
      for (int g = 0; g < k.steps; ++g, ++n) {
        const int s = n % T::kStages;
        if (!mbar_wait_warp(done(s), (n / T::kStages) & 1, abort_flag)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          // (the rows of a tile that does not leave as one were written by the working warps)
          if (whole)
            tma_store_4d(&maps.out[k.part], sb + s * T::kStage, 0, k.n0, g * T::kHeads, k.b);
          bulk_commit();
          // the previous stage's store has read it: its stage is free
          bulk_wait_read_but_one();
          if (n > 0) mbar_arrive(empty((n - 1) % T::kStages));
        }
        __syncwarp();
      }
    }
    if (lane == 0) bulk_wait_all();
  } else {
    // ------------------------------------------------------------------ working warps
    const L ln(a);
    const RopeTurns<D> turns(a);
    float2* const cs = reinterpret_cast<float2*>(smem + T::kCs) + warp * (T::kRows * (D / 2));
    const int mine = warp * T::kRows + ln.sub;  // this lane's token of a tile
    Pairs w, acc;
    int last_part = -1;
    auto flush = [&]() {
      // the gain's gradient over this warp's rows of one kind
      if (!kBwd || last_part < 0 || last_part > 1 || a.partial == nullptr) return;
      float* sums = reinterpret_cast<float*>(smem + T::kSums) + (warp * 2 + last_part) * D;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float e = j & 1 ? acc.e[j / 2].y : acc.e[j / 2].x;
        float f = j & 1 ? acc.f[j / 2].y : acc.f[j / 2].x;
#pragma unroll
        for (int off = L::kLanes; off < 32; off <<= 1) {
          e += __shfl_xor_sync(0xffffffffu, e, off);
          f += __shfl_xor_sync(0xffffffffu, f, off);
        }
        if (ln.sub == 0) {
          sums[ln.col_e(j)] = e;
          sums[ln.col_f(j)] = f;
        }
      }
    };
    int n = 0;
    bool ok = true;
    for (int it = blockIdx.x; ok && it < items.ends[2]; it += gridDim.x) {
      const RopeItem k = rope_item<T::kTokens, T::kHeads>(items, a.y, it);
      bool whole;
      const RopeToken t = tile_token<T::kTokens>(a, k, whole);
      const bool live = __shfl_sync(0xffffffffu, (int)t.live, mine) != 0;
      const bool owned = __shfl_sync(0xffffffffu, (int)t.owned, mine) != 0;
      const bool any_live = __any_sync(0xffffffffu, live);
      const int heads = a.y[k.part].heads;
      if (k.part != last_part) {
        flush();
        last_part = k.part;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          acc.e[j] = acc.f[j] = both(0.f);
          w.e[j] = w.f[j] = both(1.f);
          const float* gain = k.part < 2 && a.norm ? a.w[k.part] : nullptr;
          if (gain != nullptr) {
            w.e[j] = make_float2(__ldg(gain + ln.col_e(2 * j)), __ldg(gain + ln.col_e(2 * j + 1)));
            w.f[j] = make_float2(__ldg(gain + ln.col_f(2 * j)), __ldg(gain + ln.col_f(2 * j + 1)));
          }
        }
      }
      float2 c[2], s[2], ns[2];
      if (k.part < 2 && a.rot > 0) {
        __syncwarp();  // the previous item's entries have been read
#pragma unroll
        for (int j = 0; j < T::kRows; ++j) {
          const int place = __shfl_sync(0xffffffffu, t.place, warp * T::kRows + j);
          const int row = k.n0 + warp * T::kRows + j;
          const int at = a.cu != nullptr ? row : k.b * a.N + row;
          if (row < (a.cu != nullptr ? a.tokens : a.N))
            turns.fill(a, place, at, cs + j * (D / 2));
        }
        __syncwarp();
        turns.read(ln, cs + ln.sub * (D / 2), c, s);
#pragma unroll
        for (int j = 0; j < 2; ++j) ns[j] = make_float2(-s[j].x, -s[j].y);
      }
      for (int g = 0; g < k.steps; ++g, ++n) {
        const int st = n % T::kStages;
        if (!mbar_wait_warp(full(st), (n / T::kStages) & 1, abort_flag)) {
          ok = false;
          break;
        }
        uint8_t* const p0 = smem + st * T::kStage + mine * (D * 2);
#pragma unroll
        for (int hh = 0; hh < T::kHeads; ++hh) {
          if (g * T::kHeads + hh >= heads) break;
          uint8_t* const row = p0 + hh * (T::kTokens * D * 2);
          if (k.part == 2 && whole && live) continue;  // values stay as they came
          RopeRaw r = {};
          if (any_live) r = tile_load<kInter>(row, ln);
          if (k.part < 2 && any_live) {
            Pairs v = unpack_pairs<kInter>(r);
            if (!kBwd) {
              if (a.norm) {
                float2 ss = __fmul2_rn(v.e[0], v.e[0]);
                ss = __ffma2_rn(v.e[1], v.e[1], ss);
                ss = __ffma2_rn(v.f[0], v.f[0], ss);
                ss = __ffma2_rn(v.f[1], v.f[1], ss);
                const float2 rs = both(rsqrtf(row_sum<D>(ss.x + ss.y) * (1.f / D) + a.eps));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  v.e[j] = __fmul2_rn(__fmul2_rn(v.e[j], rs), w.e[j]);
                  v.f[j] = __fmul2_rn(__fmul2_rn(v.f[j], rs), w.f[j]);
                }
              }
              if (ln.turns) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const float2 e = v.e[j], f = v.f[j];
                  v.e[j] = __ffma2_rn(f, ns[j], __fmul2_rn(e, c[j]));
                  v.f[j] = __ffma2_rn(e, s[j], __fmul2_rn(f, c[j]));
                }
              }
            } else {
              if (ln.turns) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const float2 e = v.e[j], f = v.f[j];
                  v.e[j] = __ffma2_rn(f, s[j], __fmul2_rn(e, c[j]));
                  v.f[j] = __ffma2_rn(e, ns[j], __fmul2_rn(f, c[j]));
                }
              }
              if (a.norm) {
                const Pairs x = unpack_pairs<kInter>(tile_load<kInter>(row + T::kBytes, ln));
                float2 ss = __fmul2_rn(x.e[0], x.e[0]);
                ss = __ffma2_rn(x.e[1], x.e[1], ss);
                ss = __ffma2_rn(x.f[0], x.f[0], ss);
                ss = __ffma2_rn(x.f[1], x.f[1], ss);
                Pairs gx;  // g o x: the gain's gradient up to the row's r
                float2 sx = both(0.f);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  gx.e[j] = __fmul2_rn(v.e[j], x.e[j]);
                  gx.f[j] = __fmul2_rn(v.f[j], x.f[j]);
                  sx = __ffma2_rn(gx.e[j], w.e[j], __ffma2_rn(gx.f[j], w.f[j], sx));
                }
                const float rs = rsqrtf(row_sum<D>(ss.x + ss.y) * (1.f / D) + a.eps);
                const float2 m = both(row_sum<D>(sx.x + sx.y) * rs * rs * (-1.f / D));
                const float2 r2 = both(rs);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  if (live) {  // (rows past a length add nothing)
                    acc.e[j] = __ffma2_rn(gx.e[j], r2, acc.e[j]);
                    acc.f[j] = __ffma2_rn(gx.f[j], r2, acc.f[j]);
                  }
                  v.e[j] = __fmul2_rn(__ffma2_rn(x.e[j], m, __fmul2_rn(v.e[j], w.e[j])), r2);
                  v.f[j] = __fmul2_rn(__ffma2_rn(x.f[j], m, __fmul2_rn(v.f[j], w.f[j])), r2);
                }
              }
            }
            r = pack_pairs<kInter>(v);
          }
          if (!live) r.a = r.b = make_uint2(0, 0);
          tile_store<kInter>(row, ln, r);
          if (!whole && owned) {
            const HeadRows& o = kBwd ? a.g[k.part] : a.y[k.part];
            const RopeToken tok{0, k.n0 + mine, 0, true, true};
            store_row<kInter>(walk_rows(o, tok, g * T::kHeads + hh, 1).p, ln, r);
          }
        }
        fence_async_smem();
        mbar_arrive_warp(done(st));
      }
    }
    flush();
  }
  __syncthreads();
  if (!kBwd || a.partial == nullptr) return;
  const float* sums = reinterpret_cast<const float*>(smem + T::kSums);
  for (int i = threadIdx.x; i < 2 * D; i += T::kThreads) {
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kRopeWarps; ++q) v += sums[q * 2 * D + i];
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
