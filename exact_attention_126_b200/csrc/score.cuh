// score.cuh - scores capped by a tanh: y = c tanh(s / c), and the weights the backward forms from
// them.
//
// With u = s / c the capped score in log2 units is c log2(e) tanh(u). Its derivative with respect
// to s is 1 - tanh(u)^2, which the backward multiplies into dS.
//
// tanh costs two special-function operations (tanh u = 1 - 2 / (1 + e^(2u))), three times what the
// softmax itself needs per score, and that unit is a co-ceiling of the attention kernels. But a cap
// is chosen so that few scores come near it. A warp whose scores all have |u| <= 0.25 takes an odd
// polynomial of degree 5 (s times a quadratic in s^2, the powers of 1 / c multiplied into its
// coefficients: four packed fp32 instructions per two scores; relative error 4e-7), one whose
// scores have |u| <= 0.625 one of degree 9 (1.1e-7), and only others the exact form. Both are my
// minimax fits of tanh(u) / u in u^2; they keep the relative accuracy of small scores, which
// matters for large caps. (One polynomial of degree 7 up to 0.4, at an earlier step of these kernels:
// 849 and 1962 us for the forward and backward of B32 H16 N2048 d64 causal, against 813 and 1895.)
// What a problem takes therefore depends on its scores: that one with cap 50 and the residual takes
// 649 and 1813 us where they have a deviation of 2, 830 and 2223 at 8, 1081 and 2665 at 50, where most
// lie on the cap.
#pragma once

#include "sm100.cuh"
#include "tiles.cuh"

namespace fa {

struct CapArgs {
  int on;            // 0: the scores are not capped
  float near_limit;  // |Q K^T| up to which the short polynomial holds: 0.25 c / scale
  float limit;       // ... and the long one: kCapLimit c / scale
  float mul;         // c log2(e): turns tanh(u) into log2 units
  float scale;       // scale / c
  float near[3];     // the short polynomial in (Q K^T)^2
  float near2[3];    // ... times mul
};

// The arguments for a cap c of scores scaled by `scale`; c = 0: none.
inline CapArgs make_cap(float c, float scale) {
  CapArgs r = {};
  if (!(c > 0.f)) return r;
  const double u = (double)scale / c;
  r.on = 1;
  r.near_limit = (float)(0.25 / u);
  r.limit = (float)(0.625 / u);
  r.mul = (float)(c * 1.4426950408889634);
  const double near[3] = {0.999999604, -0.333219082, 0.128416134};
  double p = u;
  for (int i = 0; i < 3; ++i) {
    r.near[i] = (float)(near[i] * p);
    p *= u * u;
  }
  for (int i = 0; i < 3; ++i) r.near2[i] = r.near[i] * r.mul;
  r.scale = (float)u;
  return r;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest magnitude of a lane's N scores.
template <int N>
__device__ __forceinline__ float cap_amax(const float (&x)[N]) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; i += 2)
    m[(i >> 1) & 3] = fmax3(m[(i >> 1) & 3], fabsf(x[i]), fabsf(x[i + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// x <- x times the polynomial of K coefficients in x^2.
template <int K, int N>
__device__ __forceinline__ void cap_poly(float (&x)[N], const float (&a)[K]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 s = make_float2(x[i], x[i + 1]);
    const float2 z = __fmul2_rn(s, s);
    float2 p = __ffma2_rn(z, make_float2(a[K - 1], a[K - 1]), make_float2(a[K - 2], a[K - 2]));
#pragma unroll
    for (int k = K - 3; k >= 0; --k) p = __ffma2_rn(p, z, make_float2(a[k], a[k]));
    p = __fmul2_rn(p, s);
    x[i] = p.x;
    x[i + 1] = p.y;
  }
}

__device__ __forceinline__ float cap_exact(float u) {
  return fmaf(-2.f, rcp(ex2(u * (2.f * kLog2e)) + 1.f), 1.f);
}

// u <- tanh(u) where some score of the warp lies past the short polynomial's range; `exact`: past
// the long one's. The exact form's error of 2e-7 in tanh is c log2(e) times that in the exponent:
// past kCapCoarse (2^-12 in a weight, an eighth of P's rounding to bf16) scores that the long
// polynomial covers keep it, whatever other scores their warp holds. kLarge: such caps occur.
constexpr float kCapLimit = 0.625f;
constexpr float kCapCoarse = 1024.f;

template <bool kLarge, int N>
__device__ __forceinline__ void cap_far(float (&u)[N], const CapArgs& cap, bool exact) {
  const float a[5] = {0.999999893f, -0.333319542f, 0.133045259f, -0.0518218645f, 0.0150509423f};
  if (exact) {
    if (kLarge && cap.mul > kCapCoarse) {
      float y[N];  // (in local memory, for a loop: unrolled, the backward takes 1.5% longer)
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = u[i];
#pragma unroll 1
      for (int i = 0; i < N; ++i) {
        const float x = y[i], z = x * x;
        const float p = x * fmaf(fmaf(fmaf(fmaf(a[4], z, a[3]), z, a[2]), z, a[1]), z, a[0]);
        y[i] = fabsf(x) > kCapLimit ? cap_exact(x) : p;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] = y[i];
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = cap_exact(u[i]);
  } else {
    cap_poly<5>(u, a);
  }
}

// Its scores scaled first, their largest magnitude taken anew: kept from the check of the short
// polynomial, it costs every tile a register, and the backward 3% (B32 H16 N2048 d64 causal, cap 50:
// 1900 -> 1845 us).
template <int N>
__device__ __forceinline__ void cap_far(float (&x)[N], const CapArgs& cap) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] *= cap.scale;
  cap_far<true>(x, cap, __any_sync(0xffffffffu, cap_amax(x) > kCapLimit) != 0);
}

// x <- tanh(u) of the N scores x of each lane of a warp.
template <int N>
__device__ __forceinline__ void cap_tanh(float (&x)[N], const CapArgs& cap) {
  if (__builtin_expect(!__any_sync(0xffffffffu, cap_amax(x) > cap.near_limit), 1)) {
    cap_poly<3>(x, cap.near);
  } else {
    cap_far(x, cap);
  }
}

// x <- c log2(e) tanh(u), c log2(e) at most kCapNoMax.
template <int N>
__device__ __forceinline__ void cap_log2(float (&x)[N], const CapArgs& cap) {
  const float m = cap_amax(x);
  if (__builtin_expect(!__any_sync(0xffffffffu, m > cap.near_limit), 1)) {
    cap_poly<3>(x, cap.near2);
  } else {
    // (here the kept maximum is the faster: cap 20, 797 us against 820)
    const bool exact = __any_sync(0xffffffffu, m > cap.limit) != 0;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= cap.scale;
    cap_far<false>(x, cap, exact);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= cap.mul;
  }
}

// The same for scores x that also lie in tensor memory at `t` (and may be overwritten there). The
// rarer forms run in a loop over 32 columns in tensor memory: unrolled over 64 scores, code that
// hardly ever runs would push what does out of the instruction cache (head_dim 128, B2 H32 N4096
// causal: 498 us unrolled, 449 us as a loop).
template <int N>
__device__ __forceinline__ void cap_tanh_tmem(float (&x)[N], const CapArgs& cap, uint32_t t) {
  if (__builtin_expect(!__any_sync(0xffffffffu, cap_amax(x) > cap.near_limit), 1)) {
    cap_poly<3>(x, cap.near);
    return;
  }
#pragma unroll 1
  for (int q = 0; q < N / 32; ++q) {
    uint32_t u[32];
    tmem_ld32(t + 32 * q, u);
    tmem_wait_ld();
    reg_fence(u);
    float y[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(u[i]);
    cap_far(y, cap);
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(y[i]);
    tmem_st32(t + 32 * q, u);
  }
  tmem_wait_st();
  uint32_t u[N];
#pragma unroll
  for (int q = 0; q < N / 32; ++q)
    tmem_ld32(t + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(u + 32 * q));
  tmem_wait_ld();
  reg_fence(u);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __uint_as_float(u[i]);
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
