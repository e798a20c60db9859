// score.cuh - scores capped by a tanh: y = c tanh(s / c), and the weights the backward forms from
// them.
//
// With u = s / c the capped score in log2 units is c log2(e) tanh(u). Its derivative with respect
// to s is 1 - tanh(u)^2, which the backward multiplies into dS.
//
// tanh costs two special-function operations (tanh u = 1 - 2 / (1 + e^(2u))), three times what the
// softmax itself needs per score, and that unit is a co-ceiling of the attention kernels. But a cap
// is chosen so that few scores come near it: for |u| <= 0.4 an odd polynomial of degree 7 (u times a
// cubic in u^2, my minimax fit of tanh(u) / u on that range, relative error 1e-7) takes five packed
// fp32 instructions per two scores and keeps the relative accuracy of small scores, which matters
// for large caps. A warp whose scores all lie there takes it; otherwise the exact form. The powers
// of 1 / c are multiplied into the coefficients, so that s itself is what the polynomial takes.
#pragma once

#include "sm100.cuh"
#include "tiles.cuh"

namespace fa {

struct CapArgs {
  int on;       // 0: the scores are not capped
  float limit;  // |Q K^T| up to which the polynomial holds: 0.4 c / scale
  float mul;    // c log2(e): turns tanh(u) into log2 units
  float exp2u;  // 2 log2(e) scale / c
  float a[4];   // the polynomial in (Q K^T)^2
};

// The arguments for a cap c of scores scaled by `scale`; c = 0: none.
inline CapArgs make_cap(float c, float scale) {
  CapArgs r = {};
  if (!(c > 0.f)) return r;
  const double u = (double)scale / c;
  r.on = 1;
  r.limit = (float)(0.4 / u);
  r.mul = (float)(c * 1.4426950408889634);
  r.exp2u = (float)(2.0 * 1.4426950408889634 * u);
  const double fit[4] = {0.999999902, -0.333313625, 0.132709767, -0.047553602};
  double p = u;
  for (int i = 0; i < 4; ++i) {
    r.a[i] = (float)(fit[i] * p);
    p *= u * u;
  }
  return r;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x <- tanh(u) of the N scores x of each lane of a warp.
template <int N>
__device__ __forceinline__ void cap_tanh(float (&x)[N], const CapArgs& cap) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; i += 2)
    m[(i >> 1) & 3] = fmax3(m[(i >> 1) & 3], fabsf(x[i]), fabsf(x[i + 1]));
  if (__any_sync(0xffffffffu, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) > cap.limit)) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = fmaf(-2.f, rcp(ex2(x[i] * cap.exp2u) + 1.f), 1.f);
    return;
  }
  const float2 a0 = make_float2(cap.a[0], cap.a[0]), a1 = make_float2(cap.a[1], cap.a[1]);
  const float2 a2 = make_float2(cap.a[2], cap.a[2]), a3 = make_float2(cap.a[3], cap.a[3]);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 s = make_float2(x[i], x[i + 1]);
    const float2 z = __fmul2_rn(s, s);
    float2 p = __ffma2_rn(z, a3, a2);
    p = __ffma2_rn(p, z, a1);
    p = __ffma2_rn(p, z, a0);
    p = __fmul2_rn(p, s);
    x[i] = p.x;
    x[i + 1] = p.y;
  }
}

// Bits lo .. hi of a word (none when lo > hi), 0 <= lo <= 32, -1 <= hi <= 31.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  if (lo > hi) return 0u;
  return (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo);
}

template <bool kMask, bool kCap, bool kDrop, typename Add>
__device__ __forceinline__ void score_weights_t(float (&p)[32], uint32_t (&pk)[16], float mul,
                                                uint32_t vis, uint32_t keep, float ks, Add add) {
#pragma unroll
  for (int r = 0; r < 32; r += 4) {
    const float4 b4 = add(r);
    const float b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const float t0 = p[r + e], t1 = p[r + e + 1];
      const float2 x = __ffma2_rn(make_float2(t0, t1), make_float2(mul, mul),
                                  make_float2(b[e], b[e + 1]));
      float w0 = ex2(x.x), w1 = ex2(x.y);
      if (kMask) {
        w0 = ((vis >> (r + e)) & 1u) ? w0 : 0.f;
        w1 = ((vis >> (r + e + 1)) & 1u) ? w1 : 0.f;
      }
      pk[(r + e) / 2] =
          kDrop ? pack_bf16x2(((keep >> (r + e)) & 1u) ? w0 * ks : 0.f,
                              ((keep >> (r + e + 1)) & 1u) ? w1 * ks : 0.f)
                : pack_bf16x2(w0, w1);
      if (kCap) {
        // 1 - tanh^2, the cap's derivative, goes into the weight that dS is formed from
        const float2 g = __ffma2_rn(make_float2(-t0, -t1), make_float2(t0, t1),
                                    make_float2(1.f, 1.f));
        const float2 v = __fmul2_rn(make_float2(w0, w1), g);
        w0 = v.x;
        w1 = v.y;
      }
      p[r + e] = w0;
      p[r + e + 1] = w1;
    }
  }
}

// The backward's weights of 32 scores p of a lane: caps them (cap.on), forms
// P = 2^(p * mul + add) (add(r): four addends from r on), zero where `vis` has no bit, packs P
// (kDrop: the weights that multiplied V, kept ones times ks) in bf16 to pk, and leaves in p
// what dP - delta is multiplied by: P, with a cap times its derivative.
template <bool kDrop, typename Add>
__device__ __forceinline__ void score_weights(float (&p)[32], uint32_t (&pk)[16],
                                              const CapArgs& cap, float mul, uint32_t vis,
                                              uint32_t keep, float ks, Add add) {
  const bool all = __all_sync(0xffffffffu, vis == ~0u);
  if (cap.on) {
    cap_tanh(p, cap);
    if (all)
      score_weights_t<false, true, kDrop>(p, pk, mul, vis, keep, ks, add);
    else
      score_weights_t<true, true, kDrop>(p, pk, mul, vis, keep, ks, add);
  } else if (all) {
    score_weights_t<false, false, kDrop>(p, pk, mul, vis, keep, ks, add);
  } else {
    score_weights_t<true, false, kDrop>(p, pk, mul, vis, keep, ks, add);
  }
}

}  // namespace fa
