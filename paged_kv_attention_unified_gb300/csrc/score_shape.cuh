// Score shapes of the attention kernels: a tanh cap, a bias that falls with the
// distance between query and key, a prefix every query sees, and first keys
// (sinks) that stay visible under a window.
//
// With x = scale * q.k (times k_scale for an e4m3 cache), all in units of the
// argument of softmax's exp:
//
//   x <- cap * tanh(x / cap)             cap > 0
//   x <- x - slope[head] * |pos - t|     slopes given
//   key t visible iff (t <= pos or t < prefix) and (t > pos - window or t < sinks)
//
// The kernels hold scores in base 2 (y = x * log2 e). tanh comes from
// tanh(a) = 1 - 2 / (1 + e^(2a)): with u = 2 a log2 e = raw * cap_arg,
//
//   y = C - 2 C / (1 + 2^u),   C = cap * log2 e,
//
// one ex2 and one reciprocal per score. 2^u overflowing to infinity gives y =
// C, underflowing to zero y = -C. The prefill kernels, which issue slots
// bound, use it only where some score of a warp's key tile exceeds half the
// cap (or the tile is masked), and else
//
//   tanh(a) = a P(a^2), P of degree 3 fitted on |a| <= 1/2 to a relative
//   5.5e-7 (least maximum error, by iterated weighted least squares),
//
// on the paired multiply-add pipe.
// What matters is the absolute error of y (softmax exponentiates it): both
// forms stay within 2^-21 of the cap or so, about 2e-5 at cap 50, far below
// the rounding of P to 16 bits; it grows with the cap, which is why caps above
// UA_MAX_SOFTCAP are refused.
#pragma once

#include <cstdint>

#include "sm100.cuh"
#include "ua_device.cuh"

namespace ua {

// What a kernel instance applies (template argument): nothing, or at least
// the prefix mask and the sinks, plus the cap and / or the bias.
constexpr int kShapePlain = 0;
constexpr int kShapePrefix = 1;
constexpr int kShapeCap = 2;
constexpr int kShapeBias = 4;

inline int shape_of(const ScoreShape& s) {
  if (s.cap_log2 <= 0.f && s.slopes == nullptr && s.prefix_lens == nullptr && s.sinks <= 0)
    return kShapePlain;
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

// The distance bias of one row in base 2, -slope2 * (|pos - t| - shift), with
// softmax's freedom to move a row's scores by a constant: negative slopes
// favour the far keys, so that the farthest visible one gets no bias there (as
// the row's own key does under a positive slope) and the scores that count keep
// their precision however long the context. Slopes are held to 2^27 over the
// row's reach (131072 keys: 1024 a key, which leaves the neighbour of a favoured
// key 2^-1024): unfavoured scores then stay within 2^27 and their rounding,
// some 2^4, within binary32's range of 2^x between the maximum and the
// exponentials of a key tile.
struct RowBias {
  float slope2 = 0.f;
  int shift = 0;
};
// before, after: distances from the row to the first and the last key it sees.
__device__ __forceinline__ RowBias row_bias(float slope, int before, int after) {
  const int reach = max(before, after);
  const float most = 134217728.f / static_cast<float>(max(reach, 1024));
  RowBias b;
  b.slope2 = fminf(fmaxf(slope * kLog2e, -most), most);
  b.shift = b.slope2 < 0.f ? reach : 0;
  return b;
}

// Row maximum (of the magnitudes: ABS) with independent 3-input partial
// maxima; NaN is passed over (it reaches the output by itself).
template <bool ABS, int N>
__device__ __forceinline__ float row_max(const float (&x)[N]) {
  using namespace sm100;
  constexpr int kAcc = 4;
  auto v = [](float f) { return ABS ? fabsf(f) : f; };
  float part[kAcc];
#pragma unroll
  for (int a = 0; a < kAcc; ++a) part[a] = v(x[a]);
#pragma unroll
  for (int i = kAcc; i < N; i += 2)
    part[(i / 2) % kAcc] = fmax3(part[(i / 2) % kAcc], v(x[i]), v(x[i + 1]));
  return fmaxf(fmax3(part[0], part[1], part[2]), part[3]);
}

// What a prefill softmax row needs for its scores, constant over its key
// tiles, and its softmax of one key tile of KEYS scores in tensor memory.
//
// KEYS 128 (the two-query-tile kernel, whose softmax warps compete with the
// MMA issuer for issue slots): 32 columns at a time, in loops that are not
// unrolled over them, the scores read from tensor memory once for the maximum
// and once for the exponentials. The shaping makes the code per score long;
// unrolled over 128 scores held in registers, the plain kernel's way, the
// softmax warps run out of the instruction cache. Capped dense causal prefill,
// 4 x 4096 tokens, 32 heads of 128: unrolled with ex2 and reciprocal 881 us,
// unrolled with the polynomial 728 us, in loops over 16, 32 and 64 columns 671,
// 643 and 723 us; 600 us with the maximum left out where no score can move the
// reference and masks taken as bits. Without a cap: 505 us, the plain kernel;
// with a distance bias 566 us (691 when every rise towards the row moved the
// reference), with both 779 us.
// KEYS 64 (the wide kernel, one query tile at a time, its products issued at
// N = 64): unrolled, held in registers (head_dim 256 on the same batch 1206
// us; when it was 1211, in loops 1397 us and with a row shared by two threads
// 1300 us; uncapped 1067 us).
template <int SHAPE, bool F8, int KEYS>
struct RowSoftmax {
  static constexpr bool kCap = (SHAPE & kShapeCap) != 0, kBias = (SHAPE & kShapeBias) != 0;
  static constexpr float kSlack = 8.f;  // log2 units by which scores may exceed the reference
  static constexpr int N = KEYS == 128 ? 32 : KEYS;  // columns at a time
  float c, cap_log2;     // raw score -> base 2; the cap in base 2
  float a0, a1, a2, a3;  // base-2 capped score = raw (a0 + a1 raw^2 + a2 raw^4 + a3 raw^6) ...
  float small;           // ... for |raw| up to this
  RowBias bias;
  float m = -INFINITY, l = 0.f;  // reference (a lagging running maximum) and sum

  __device__ __forceinline__ RowSoftmax(float c_, float cap_log2_, const RowBias& bias_)
      : c(c_), cap_log2(cap_log2_), bias(bias_) {
    if constexpr (kCap) {
      const float k = c / cap_log2, k2 = k * k;  // raw score -> argument of tanh
      a0 = c * 0.99999946f;
      a1 = c * -0.33326318f * k2;
      a2 = c * 0.13190296f * k2 * k2;
      a3 = c * -0.04440221f * k2 * k2 * k2;
      // a factor beyond 2^16 leaves the coefficients without range
      small = fabsf(k) <= 65536.f ? 0.5f / fabsf(k) : -1.f;
    }
  }

  // A row's place in a key tile.
  struct Place {
    int rel0;            // first key, relative to the row
    int lo_col, hi_col;  // visible columns ...
    int sink_col;        // ... and those below it (0: none)
    bool after;          // (bias) the warp has visible keys after their rows
  };

  __device__ __forceinline__ static void load(uint32_t taddr, float (&x)[N]) {
    uint32_t v[N / 32][32];
#pragma unroll
    for (int b = 0; b < N / 32; ++b) sm100::tmem_ld32(taddr + 32 * b, v[b]);
#pragma unroll
    for (int b = 0; b < N / 32; ++b) sm100::tmem_wait_ld(v[b]);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __uint_as_float(v[i / 32][i % 32]);
  }

  // Raw scores of the columns ch .. ch + N - 1 to base-2 scores minus sub, -inf
  // where not visible. SMALL: by the polynomial. OPEN: all of them visible. The
  // bias is slope * (rel + shift) as long as visible keys lie at or before their
  // rows.
  template <bool SMALL, bool OPEN>
  __device__ __forceinline__ void scores(float (&x)[N], int ch, const Place& at, float sub) const {
    using namespace sm100;
    const float slope2 = bias.slope2;
    const float rel = static_cast<float>(at.rel0 + ch + (kBias ? bias.shift : 0));
    // What is added to a score: -sub, and the bias of its pair of keys.
    const bool after = kBias && !OPEN && at.after;  // (the bias is added further down)
    const float step = kBias && !after ? slope2 : 0.f;
    const uint64_t step2 = f2_pack(step, step);
    const uint64_t first = kBias ? f2_pack(fmaf(rel, step, -sub), fmaf(rel + 1.f, step, -sub))
                                 : f2_pack(-sub, -sub);
    auto add = [&](int i) {
      const float f = static_cast<float>(i);
      return kBias && i > 0 ? f2_fma(f2_pack(f, f), step2, first) : first;
    };
    if constexpr (kCap && !SMALL) {
      const float u_mult = c * (2.f * kLog2e / cap_log2);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = cap_score(x[i] * u_mult, cap_log2);
#pragma unroll
      for (int i = 0; i < N; i += 2)
        f2_unpack(f2_add(f2_pack(x[i], x[i + 1]), add(i)), x[i], x[i + 1]);
    } else {
      const uint64_t b0 = f2_pack(kCap ? a0 : c, kCap ? a0 : c), b1 = f2_pack(a1, a1),
                     b2 = f2_pack(a2, a2), b3 = f2_pack(a3, a3);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const uint64_t raw = f2_pack(x[i], x[i + 1]);
        uint64_t poly = b0;
        if constexpr (kCap) {
          const uint64_t sq = f2_mul(raw, raw);
          poly = f2_fma(f2_fma(f2_fma(b3, sq, b2), sq, b1), sq, b0);
        }
        f2_unpack(f2_fma(raw, poly, add(i)), x[i], x[i + 1]);
      }
    }
    if (after) {
      const float key = static_cast<float>(at.rel0 + ch), shift = static_cast<float>(bias.shift);
#pragma unroll
      for (int i = 0; i < N; ++i)
        x[i] = fmaf(-slope2, fabsf(key + static_cast<float>(i)) - shift, x[i]);
    }
    if constexpr (!OPEN) {
      static_assert(N == 32, "one bit per column");
      const int lo = at.lo_col - ch, hi = at.hi_col - ch;
      auto below = [](int n) { return n >= N ? ~0u : (n <= 0 ? 0u : (1u << n) - 1u); };
      const uint32_t seen = below(hi) & (~below(lo) | below(at.sink_col - ch));
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!(seen & (1u << i))) x[i] = -INFINITY;
    }
  }

  // P = 2^x of N exponents over columns that have been read (bf16 pairs, or
  // e4m3 quadruples); the unrounded P are added to sum.
  __device__ __forceinline__ static void store_p(uint32_t p_tmem, const float (&x)[N],
                                                 uint64_t (&sum)[4]) {
    using namespace sm100;
    uint32_t pk[F8 ? N / 4 : N / 2];
    float q0 = 0.f, q1 = 0.f;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float p0 = ex2(x[2 * i]), p1 = ex2(x[2 * i + 1]);
      sum[i % 4] = f2_add(sum[i % 4], f2_pack(p0, p1));
      if constexpr (F8) {
        if (i % 2 == 0) {
          q0 = p0;
          q1 = p1;
        } else {
          pk[i / 2] = to_e4m3x4(q0, q1, p0, p1);
        }
      } else {
        pk[i] = pack2<false>(p0, p1);
      }
    }
    tmem_st(p_tmem, pk);
  }

  // Moves the reference for a tile whose largest score is top; returns the
  // factor for what was accumulated before. Under a bias the scores rise from
  // key tile to key tile towards the row, by slope * KEYS each, and every move
  // rescales O: a moved reference is put ahead by the rise still to come, up to
  // 2^48 (bf16 P and binary32 sums keep their relative precision there; e4m3 P
  // has no range to spare).
  __device__ __forceinline__ float move(float top, int rel0) {
    const float m_old = m, m_new = fmaxf(m, top);
    float lead = 0.f;
    if constexpr (kBias && !F8)
      lead = fminf(fmaxf(-bias.slope2 * static_cast<float>(rel0 + KEYS - 1), 0.f), 48.f);
    if (m_new > -INFINITY && (m == -INFINITY || m_new > m + kSlack)) m = m_new + lead;
    return m == m_old ? 1.f : (m_old == -INFINITY ? 0.f : ex2(m_old - m));
  }
  __device__ __forceinline__ float subtrahend() const { return m == -INFINITY ? 0.f : m; }

  template <bool SMALL, bool OPEN>
  __device__ __forceinline__ float tile_max(uint32_t s_tmem, const Place& at) const {
    float top = -INFINITY;
#pragma unroll 1
    for (int ch = 0; ch < KEYS; ch += N) {
      float x[N];
      load(s_tmem + ch, x);
      scores<SMALL, OPEN>(x, ch, at, 0.f);
      top = fmaxf(top, row_max<false>(x));
    }
    return top;
  }
  template <bool SMALL, bool OPEN>
  __device__ __forceinline__ void tile_p(uint32_t s_tmem, const Place& at, uint64_t (&sum)[4]) const {
#pragma unroll 1
    for (int ch = 0; ch < KEYS; ch += N) {
      float x[N];
      load(s_tmem + ch, x);
      scores<SMALL, OPEN>(x, ch, at, subtrahend());
      store_p(s_tmem + ch / (F8 ? 4 : 2), x, sum);
    }
  }

  // One key tile: scores at s_tmem, keys from pos + rel0 on, columns [lo_col,
  // hi_col) and those below sink_col and hi_col visible, to P. Returns the factor
  // for what was accumulated before. Whole warps call it together.
  __device__ __forceinline__ float tile(uint32_t s_tmem, int rel0, int lo_col, int hi_col,
                                        int sink_col) {
    using namespace sm100;
    if (sink_col >= lo_col) lo_col = 0;  // one run
    uint64_t sum[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) sum[a] = f2_pack(0.f, 0.f);
    float alpha;
    if constexpr (KEYS == N) {
      alpha = whole_tile(s_tmem, rel0, lo_col, hi_col, sink_col, sum);
    } else {
      const bool after = kBias && __any_sync(0xffffffffu, rel0 + min(hi_col, KEYS) > 1);
      alpha = tile_by_columns(s_tmem, Place{rel0, max(lo_col, 0), hi_col, sink_col, after}, sum);
    }
    sum[0] = f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3]));
    float lo, hi;
    f2_unpack(sum[0], lo, hi);
    l = l * alpha + (lo + hi);
    return alpha;
  }

 private:
  __device__ __forceinline__ float tile_by_columns(uint32_t s_tmem, const Place& at,
                                                   uint64_t (&sum)[4]) {
    const bool open =
        __all_sync(0xffffffffu, at.hi_col >= KEYS && at.lo_col <= 0) && !at.after;
    bool is_small = true, settled = false;  // settled: no score can move a reference
    if constexpr (kCap) {
      float amax = 0.f;
#pragma unroll 1
      for (int ch = 0; ch < KEYS; ch += N) {
        float x[N];
        load(s_tmem + ch, x);
        amax = fmaxf(amax, row_max<true>(x));
      }
      is_small = __all_sync(0xffffffffu, amax <= small);
      float bound = amax * fabsf(c);  // |cap tanh(x / cap)| <= |x|
      if constexpr (kBias) {  // the largest bias is at one of the ends, or at most 0 at the row itself
        const float first = static_cast<float>(abs(at.rel0) - bias.shift);
        const float last = static_cast<float>(abs(at.rel0 + KEYS - 1) - bias.shift);
        const float ends = fmaxf(-bias.slope2 * first, -bias.slope2 * last);
        bound += at.rel0 <= 0 && at.rel0 + KEYS > 0 ? fmaxf(ends, 0.f) : ends;
      }
      settled = __all_sync(0xffffffffu, bound <= m + kSlack);
    }
    float top = -INFINITY;
    if (!settled)
      top = open ? (is_small ? tile_max<true, true>(s_tmem, at) : tile_max<false, true>(s_tmem, at))
                 : (is_small ? tile_max<true, false>(s_tmem, at)
                             : tile_max<false, false>(s_tmem, at));
    const float alpha = move(top, at.rel0);
    if (open) {
      if (is_small) tile_p<true, true>(s_tmem, at, sum);
      else tile_p<false, true>(s_tmem, at, sum);
    } else {
      if (is_small) tile_p<true, false>(s_tmem, at, sum);
      else tile_p<false, false>(s_tmem, at, sum);
    }
    return alpha;
  }

  __device__ __forceinline__ float whole_tile(uint32_t s_tmem, int rel0, int lo_col, int hi_col,
                                              int sink_col, uint64_t (&sum)[4]) {
    using namespace sm100;
    float x[N];
    load(s_tmem, x);
    if constexpr (kCap) {
      float b0 = a0, b1 = a1, b2 = a2, b3 = a3;
      if (!__all_sync(0xffffffffu, row_max<true>(x) <= small)) {
        const float u_mult = c * (2.f * kLog2e / cap_log2);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = cap_score(x[i] * u_mult, cap_log2);
        b0 = 1.f;  // the polynomial below leaves them as they are
        b1 = b2 = b3 = 0.f;
      }
      const uint64_t c0 = f2_pack(b0, b0), c1 = f2_pack(b1, b1), c2 = f2_pack(b2, b2),
                     c3 = f2_pack(b3, b3);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const uint64_t raw = f2_pack(x[i], x[i + 1]);
        const uint64_t sq = f2_mul(raw, raw);
        f2_unpack(f2_mul(raw, f2_fma(f2_fma(f2_fma(c3, sq, c2), sq, c1), sq, c0)), x[i], x[i + 1]);
      }
    }
    if constexpr (kBias) {
      // Key tiles with no key after its row, most of them, take the bias in
      // pairs, slope * (rel + shift), as above (head_dim 192, 6 prompts of 1500
      // tokens after 1500, 32 heads: 1005 us, 1251 with the distances one by one).
      const float mult = kCap ? 1.f : c, slope2 = bias.slope2;
      if (__all_sync(0xffffffffu, rel0 + N <= 1)) {
        const float first = static_cast<float>(rel0 + bias.shift);
        const uint64_t m2 = f2_pack(mult, mult), step2 = f2_pack(slope2, slope2);
        const uint64_t base = f2_pack(first * slope2, (first + 1.f) * slope2);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const float f = static_cast<float>(i);
          f2_unpack(f2_fma(f2_pack(x[i], x[i + 1]), m2, f2_fma(f2_pack(f, f), step2, base)), x[i],
                    x[i + 1]);
        }
      } else {
        const float rel = static_cast<float>(rel0), shift = static_cast<float>(bias.shift);
#pragma unroll
        for (int i = 0; i < N; ++i)
          x[i] = fmaf(x[i], mult, -slope2 * (fabsf(rel + static_cast<float>(i)) - shift));
      }
    }
    // a prefix alone leaves the scores raw until the exponents
    const bool raw = !kCap && !kBias, flip = raw && c < 0.f;
    if (flip) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = -x[i];
    }
    if (sink_col > 0 && lo_col > 0) {  // sinks, then keys that the window has passed
      if (lo_col >= N) {
        hi_col = min(hi_col, sink_col);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i >= sink_col && i < lo_col) x[i] = -INFINITY;
      }
      lo_col = 0;
    }
    if (hi_col < N || lo_col > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i >= hi_col || i < lo_col) x[i] = -INFINITY;
    }
    const float mult = raw ? fabsf(c) : 1.f;
    const float alpha = move(row_max<false>(x) * mult, rel0);
    const float sub = subtrahend();
    const uint64_t nsub = f2_pack(-sub, -sub), m2 = f2_pack(mult, mult);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint64_t y = f2_pack(x[i], x[i + 1]);
      f2_unpack(raw ? f2_fma(y, m2, nsub) : f2_add(y, nsub), x[i], x[i + 1]);
    }
    store_p(s_tmem, x, sum);
    return alpha;
  }
};

}  // namespace ua
