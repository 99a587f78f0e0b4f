// Score shapes of the attention kernels: a tanh cap, a bias that falls with the
// distance between query and key, and a prefix every query sees.
//
// With x = scale * q.k (times k_scale for an e4m3 cache), all in units of the
// argument of softmax's exp:
//
//   x <- cap * tanh(x / cap)             cap > 0
//   x <- x - slope[head] * |pos - t|     slopes given
//   key t visible iff t <= pos or t < prefix (both within kv_len and window)
//
// The kernels hold scores in base 2 (y = x * log2 e). tanh comes from
// tanh(a) = 1 - 2 / (1 + e^(2a)): with u = 2 a log2 e = raw * cap_arg,
//
//   y = C - 2 C / (1 + 2^u),   C = cap * log2 e,
//
// one ex2 and one reciprocal per score. What matters is the absolute error of
// y (softmax exponentiates it): a few 2^-24 of C, about 2e-5 at cap 50, far
// below the rounding of P to 16 bits; it grows with the cap, which is why caps
// above UA_MAX_SOFTCAP are refused. 2^u overflowing to infinity gives y = C,
// underflowing to zero y = -C.
#pragma once

#include <cstdint>

#include "sm100.cuh"
#include "ua_device.cuh"

namespace ua {

// What a kernel instance applies (template argument): nothing, or at least
// the prefix mask, plus the cap and / or the bias.
constexpr int kShapePlain = 0;
constexpr int kShapePrefix = 1;
constexpr int kShapeCap = 2;
constexpr int kShapeBias = 4;

inline int shape_of(const ScoreShape& s) {
  if (s.cap_log2 <= 0.f && s.slopes == nullptr && s.prefix_lens == nullptr) return kShapePlain;
  return kShapePrefix | (s.cap_log2 > 0.f ? kShapeCap : 0) | (s.slopes ? kShapeBias : 0);
}

// Reciprocal to within an ulp or so; 1 / inf = 0.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap * tanh(raw scaled score / cap) in base 2, from u = raw * cap_arg.
__device__ __forceinline__ float cap_score(float u, float cap_log2) {
  return fmaf(-2.f * cap_log2, rcp_approx(1.f + ex2(u)), cap_log2);
}

// N raw scores of one row, keys at pos + rel0 .. pos + rel0 + N - 1, to shaped
// base-2 scores. c: raw score -> base 2; u_mult: raw score -> cap argument
// (SHAPE has kShapeCap); slope2: slope * log2 e (kShapeBias).
template <int N, int SHAPE>
__device__ __forceinline__ void shape_row(float (&x)[N], float c, float u_mult, float cap_log2,
                                          float slope2, int rel0) {
  constexpr bool kCap = (SHAPE & kShapeCap) != 0, kBias = (SHAPE & kShapeBias) != 0;
  if constexpr (kCap) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = cap_score(x[i] * u_mult, cap_log2);
  }
  if constexpr (kBias) {
    const float mult = kCap ? 1.f : c;
    const float rel = static_cast<float>(rel0);
#pragma unroll
    for (int i = 0; i < N; ++i)
      x[i] = fmaf(x[i], mult, -slope2 * fabsf(rel + static_cast<float>(i)));
  }
}

}  // namespace ua
