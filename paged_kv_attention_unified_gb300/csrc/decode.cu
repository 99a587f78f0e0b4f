// Split-KV decode kernel (K-D): a bandwidth-bound pass over the paged cache.
//
// Work unit: one ua_tile = up to 8 packed (token, head) rows of one sequence
// and KV head (all query heads of a GQA group share one K/V stream, as in the
// packed Q tile of "vllm_triton_unified_attention_notes") over one key range
// [kv_lo, kv_hi) -- a whole range, or one split piece whose partial result is
// merged later by the log-sum-exp combine (FlashDecoding, "Fused Attention"
// notes; run_flash_splitkv_fwd in "flashatten takeaways EP2 工程").
//
// Design for sm_103a. Decode is HBM-bound (about 4-16 flop per cache byte).
// Each warp owns a ring of shared-memory stages; one lane issues, per 16-key
// step, one TMA box of K and one of V (the 16 slots of one KV head in one
// page) a few steps ahead of the math, and the warp reads the landed page
// into registers and keeps the math on the tensor pipe with m16n8k16 MMAs in
// a transposed orientation:
//   S^T[key, row]  = K[key, :] . Q[row, :]      (M = 16 keys, N = 8 rows)
//   O^T[d, row]   += V^T[d, key] . P^T[key, row] (M = 16 dims, N = 8 rows)
// Keys on M and the GQA rows on N waste no MMA rows when 8 query heads share
// a KV head. The score fragment becomes the PV operand with one movmatrix
// transpose per 8x8 block. Because the contraction index of both products
// and the M index of the second may be permuted freely, the kernel assigns
// keys and head dimensions to lanes so that the shared-memory fragment reads
// take the minimum number of wavefronts (4 lanes x 16 B of one K row, 8 lanes
// x 16 B of one V row, with the 128-byte swizzle of the staged page).
// Online softmax in base 2 ("Fused Attention" notes, _attn_fwd_inner): running
// max m, running sum l, rescale factor 2^(m_old - m_new). Optionally a unified
// max (FlashDecoding++, "Fused Attention" notes): a preset reference replaces
// the first step's max, with the running max as the fallback.
// Four warps per CTA take interleaved 16-key steps of the tile's range and
// merge their (m, l, O) through shared memory at the end. A split piece
// leaves its normalised partial and base-2 lse in the workspace; with arrival
// counters given, the last piece of a group to finish merges the group in the
// same launch (otherwise the combine kernel does).
// Over an e4m3 cache with block scales every step lies in one page, so the key
// scale multiplies the step's scores, and the value scale vs the weights of its
// codes: l sums the weights as they are, O is held in a unit of the warp's
// (ValueUnit) and takes weights times vs / unit where f16 has room for those, and
// the product of a step times vs / unit in binary32 where it has not. Weights have
// the range that they have without scales, whatever the scales of a row's pages.
#include <type_traits>

#include "score_shape.cuh"
#include "sm100.cuh"
#include "ua_device.cuh"
#include "planner.h"
#include "ua_kernels.h"

namespace ua {

namespace {

// Values per shared-memory load: as many as fill 16 bytes, else 8 or 4 bytes,
// dividing the n values a lane reads per row.
constexpr int load_vals(int n, int elt) {
  int v = 16 / elt;
  while (v * elt > 4 && n % v != 0) v /= 2;
  return v;
}

// Head dims: any multiple of 32 up to 256.
template <int D, bool FP8>
struct DecodeCfg {
  static_assert(D % 32 == 0 && D >= 32 && D <= 256, "head_dim");
  static constexpr int ELT = FP8 ? 1 : 2;                       // cache element bytes
  static constexpr int KVALS = D / 4;                           // K values per row per lane
  static constexpr int KE = load_vals(KVALS, ELT);              // K values per load
  static constexpr int KW = KVALS * ELT / 4;                    // ... as 32-bit words
  static constexpr int NKL = KVALS / KE;                        // K loads per row
  static constexpr int VVALS = D / 8;                           // V values per key per lane
  static constexpr int VE = load_vals(VVALS, ELT);              // V values per load
  static constexpr int VW = VVALS * ELT / 4;
  static constexpr int NVL = VVALS / VE;
  static constexpr int VLB = VE * ELT;                          // bytes per V load (16, 8 or 4)
  static constexpr int NC = D / 16;                             // MMA chunks along D
  static constexpr int QW = KVALS / 2;                          // Q words (16-bit pairs)
  static_assert(KVALS % KE == 0 && VVALS % VE == 0 && KE * ELT >= 4 && VLB >= 4, "loads");
};

// A load of B bytes (16, 8 or 4) from shared memory into consecutive words.
template <int B>
__device__ __forceinline__ void lds_words(uint32_t* w, const uint8_t* src, bool ok) {
  if constexpr (B == 16) {
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (ok) x = *reinterpret_cast<const uint4*>(src);
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
  } else if constexpr (B == 8) {
    uint2 x = make_uint2(0u, 0u);
    if (ok) x = *reinterpret_cast<const uint2*>(src);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    w[0] = ok ? *reinterpret_cast<const uint32_t*>(src) : 0u;
  }
}

constexpr int kWarps = kDecodeWarps;
constexpr int kThreads = kWarps * 32;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// How far a unified-max reference may sit above a row's first max (log2
// units): P values down to 2^-64 times the largest are still normal bf16
// numbers, while f16 P (the e4m3 path) has no range to spare beyond what the
// running-max path already uses (largest P in [1, 2^8]).
template <bool FP8>
constexpr float kUnifiedAbove = FP8 ? 0.0f : 64.0f;

// Key slot (0..15) of a step held as MMA row m of S^T. Chosen so that the
// PV contraction slots 2t, 2t+1, 2t+8, 2t+9 of lane t are keys 4t..4t+3.
__device__ __forceinline__ int key_of_row(int m) {
  return (m < 8) ? ((m & 1) ? 2 * m - 1 : 2 * m) : ((m & 1) ? 2 * m - 15 : 2 * m - 14);
}

// Head-dimension index of K/Q value u (0..D/4-1) of lane t.
template <int D, bool FP8>
__device__ __forceinline__ int k_dim(int u, int t) {
  using C = DecodeCfg<D, FP8>;
  return (u / C::KE) * 4 * C::KE + t * C::KE + (u % C::KE);
}

// Head-dimension index of V value v (0..D/8-1) of lane group g.
template <int D, bool FP8>
__device__ __forceinline__ int v_dim(int v, int g) {
  using C = DecodeCfg<D, FP8>;
  return (v / C::VE) * 8 * C::VE + g * C::VE + (v % C::VE);
}

// Shared-memory layout of one 16-key page of K or V as TMA lands it. Rows of
// at least 128 bytes arrive as 128-byte-wide panels (16 rows each) with the
// 128-byte swizzle: the 16-byte chunk c of row r sits at chunk c ^ (r % 8).
// The fragment reads below touch 8 rows at one column (K) or 4 whole rows (V)
// per instruction; with the swizzle both take the minimum of 4 wavefronts
// (unswizzled, the 8 K rows at a 256-byte stride share half of the banks).
// The e4m3 path keeps plain rows: its K reads are half as many and its
// conversion work leaves no issue slots for the swizzled address arithmetic
// (measured: slower with the swizzle). So do bf16 rows that are not a whole
// number of 128-byte panels (head dims 32, 96, 160, 224).
template <int D, bool FP8>
struct PageLayout {
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  static constexpr bool kSwizzle = !FP8 && kRowBytes % 128 == 0;
  static constexpr int kBoxDims = kSwizzle ? 128 / (FP8 ? 1 : 2) : D;  // elements per box row
  static constexpr int kPanels = kSwizzle ? kRowBytes / 128 : 1;
  static constexpr int kPanelBytes = 16 * (kSwizzle ? 128 : kRowBytes);
  // Byte address of row `key`, byte `o` of the row (o a multiple of 8).
  __device__ static __forceinline__ int at(int key, int o) {
    if constexpr (kSwizzle) {
      const int within = o & 127;
      return (o >> 7) * kPanelBytes + key * 128 + ((((within >> 4) ^ (key & 7))) << 4) +
             (within & 15);
    } else {
      return key * kRowBytes + o;
    }
  }
};

template <int D, bool FP8>
struct StepRegs {
  uint32_t k[2][DecodeCfg<D, FP8>::KW];   // K rows key_of_row(g), key_of_row(g+8)
  uint32_t v[4][DecodeCfg<D, FP8>::VW];   // V rows 4t .. 4t+3
};

// Registers of one 16-key step from its shared-memory stage: kp / vp hold the
// step's K and V rows (16 rows of head_dim elements, as the TMA box lands).
// Keys at or beyond kv_hi read as zero (the page may hold anything there).
template <int D, bool FP8>
__device__ __forceinline__ void read_k(StepRegs<D, FP8>& r, const uint8_t* kp, int base,
                                       int kv_hi, int g, int t) {
  using C = DecodeCfg<D, FP8>;
  using PL = PageLayout<D, FP8>;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int key = key_of_row(g + 8 * h);
    const bool ok = base + key < kv_hi;
    constexpr int kB = C::KE * C::ELT;  // bytes per load
#pragma unroll
    for (int l = 0; l < C::NKL; ++l)
      lds_words<kB>(&r.k[h][l * (kB / 4)], kp + PL::at(key, (l * 4 * C::KE + t * C::KE) * C::ELT),
                    ok);
  }
}

template <int D, bool FP8>
__device__ __forceinline__ void read_v(StepRegs<D, FP8>& r, const uint8_t* vp, int base,
                                       int kv_hi, int g, int t) {
  using C = DecodeCfg<D, FP8>;
  using PL = PageLayout<D, FP8>;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int key = 4 * t + j;
    const bool ok = base + key < kv_hi;
#pragma unroll
    for (int l = 0; l < C::NVL; ++l)
      lds_words<C::VLB>(&r.v[j][l * (C::VLB / 4)],
                        vp + PL::at(key, (l * 8 * C::VE + g * C::VE) * C::ELT), ok);
  }
}

// Head dims above 128 read V only after the softmax, so that the K and V
// fragments of a step are never live together (register budget).
template <int D>
constexpr bool kLateV = D > 128;

// Per-warp online-softmax state for the two rows (columns n = 2t, 2t+1) a lane
// holds, plus its O^T accumulator fragments.
template <int D>
struct WarpState {
  float acc[D / 16][4];
  float m[2];
  float l[2];  // lane-partial sums; reduced over the 8 lane groups at the end
};

struct StepMask {
  int kv_hi;       // keys >= kv_hi are outside the range
  int hi_full;     // keys < hi_full are visible to every row (upper side)
  int lo_full;     // keys >= lo_full are visible to every row (lower side)
  int pos[2];      // query position of the lane's two rows
  int last[2];     // last key the causal mask leaves them (pos, or the prefix's last key)
  int causal;
  int window;
  int sinks;       // (SHAPED instances) keys below it stay visible under the window
  float phi2;      // unified max in log2 units of the scaled score; NaN: off
  // Score shape (SHAPED instances): the cap, 0 for none, with its argument's
  // multiplier, and the distance biases of the two rows.
  float cap_log2, cap_arg;
  RowBias bias[2];
};

// The block scales of a step's page (SCALED instances): keys, values.
struct StepScale {
  float k, v;
};

// The unit of a warp's O accumulators over a cache with block scales, a power of
// two: a step's values count v / unit of a code's. While that lies in [1, 2^7] it
// goes into the weights before they are rounded to f16 (which are at most 2^8, so
// nothing overflows, and no weight is smaller than without scales). The unit
// follows the pages in steps of exact products. It stays within [2^-60, 2^22] and
// at 2^-64 of the largest scale so far or above: then O, at most 2^8 a key times 448
// of those, stays below 2^128 for 2^31 keys, and what the quietest page (2^-100)
// adds beside the loudest (2^100) is a number of binary32. Pages of one step pair 2^12
// apart all along, the slowest case (64 x 4096 keys, us): head_dim 64 74.0 -> 75.9, 128
// 94.8 -> 94.9, 256 172.2 -> 173.5.
struct ValueUnit {
  float inv = 0.f, top = 0.f;  // 1 / unit (0: nothing taken yet); the largest scale so far
  __device__ __forceinline__ static float power(float x) {  // 2^floor(log2 x)
    return __uint_as_float(__float_as_uint(x) & 0x7f800000u);
  }
  __device__ __forceinline__ static float inverse(float x) {  // of a power of two
    return __uint_as_float((254u << 23) - __float_as_uint(x));
  }
  __device__ __forceinline__ bool near(float least, float most) const {
    return least * inv >= 1.f && most * inv <= 128.f;
  }
  // A unit for pages with scales from least to most; returns old / new.
  __device__ __forceinline__ float follow(float least, float most) {
    top = fmaxf(top, most);
    const float unit = fminf(fmaxf(fmaxf(power(least) * 0.125f, power(top) * 0x1p-64f), 0x1p-60f), 0x1p22f);
    const float factor = inv > 0.f ? unit * inv : 1.f;  // new / old
    inv = inverse(unit);
    return inverse(factor);
  }
};

template <int D, bool FP8, bool SHAPED>
__device__ __forceinline__ void compute_step(WarpState<D>& st, StepRegs<D, FP8>& r,
                                             const uint8_t* vp, int kv_hi,
                                             const uint32_t (&qb)[D / 16][2], const float (&cc)[2],
                                             const StepMask& mk, int base, int g, int t) {
  using C = DecodeCfg<D, FP8>;
  // S^T = K Q^T for the 16 keys of this step, in two independent accumulation
  // chains (even and odd head-dim chunks) that are added at the end: half the
  // dependent MMA latency per step.
  float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
  for (int c = 0; c < C::NC; ++c) {
    uint32_t a[4];
    if constexpr (FP8) {
      e4m3x4_to_f16x2x2(r.k[0][c], a[0], a[2]);
      e4m3x4_to_f16x2x2(r.k[1][c], a[1], a[3]);
    } else {
      a[0] = r.k[0][2 * c];
      a[1] = r.k[1][2 * c];
      a[2] = r.k[0][2 * c + 1];
      a[3] = r.k[1][2 * c + 1];
    }
    mma16816<FP8>(s[c & 1], a, qb[c][0], qb[c][1]);
  }
  float x[4];
  x[0] = (s[0][0] + s[1][0]) * cc[0];
  x[1] = (s[0][1] + s[1][1]) * cc[1];
  x[2] = (s[0][2] + s[1][2]) * cc[0];
  x[3] = (s[0][3] + s[1][3]) * cc[1];
  if constexpr (SHAPED) {
    // HBM-bound: one instance applies whatever the call asks for (uniform
    // branches; without a bias the slopes are zero).
    if (mk.cap_log2 > 0.f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = cap_score(x[e] * mk.cap_arg, mk.cap_log2);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = base + key_of_row(g + 8 * (e >> 1));
      const RowBias& b = mk.bias[e & 1];
      x[e] = fmaf(-b.slope2, static_cast<float>(abs(mk.pos[e & 1] - key) - b.shift), x[e]);
    }
  }
  // Masking (a select, so that nothing read from outside the visible set can
  // reach the result) only on steps that straddle a bound.
  if (base < mk.lo_full || base + 16 > mk.hi_full) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = base + key_of_row(g + 8 * (e >> 1));
      const int pos = mk.pos[e & 1];
      bool ok = key < mk.kv_hi;
      if (mk.causal) ok = ok && key <= (SHAPED ? mk.last[e & 1] : pos);
      if (mk.window > 0) ok = ok && (key > pos - mk.window || (SHAPED && key < mk.sinks));
      x[e] = ok ? x[e] : -INFINITY;
    }
  }
  // Row max over the 16 keys: the lane's two keys, then the 8 lane groups.
  float mx[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 4));
    mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 8));
    mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 16));
  }
  // The reference max moves only when the row max grew by more than 2^8
  // (log2 units 8): P and l use the same stale reference, so the result is
  // exact up to rounding, P stays below 2^8, and the O rescale (a multiply of
  // every accumulator) runs only on the rare steps where some row moved.
  // With a unified max phi2, a row's first visible step takes phi2 as its
  // reference when its max lies in [phi2 - kUnifiedAbove, phi2 + 8]; outside
  // that range (overflow or underflow risk) it falls back to its own max, and
  // later steps move the reference up as above.
  float p[4], alpha[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const bool first = st.m[j] == -INFINITY;
    const float m_new = fmaxf(st.m[j], mx[j]);
    const bool grow = first || (m_new > st.m[j] + kRescaleThreshold);
    float m_use = grow ? m_new : st.m[j];
    if (first && mx[j] <= mk.phi2 + kRescaleThreshold && mx[j] >= mk.phi2 - kUnifiedAbove<FP8>)
      m_use = mk.phi2;
    // Rows with nothing visible yet keep m = -inf; subtract 0 instead so that
    // no -inf - -inf appears.
    const float sub = (m_use == -INFINITY) ? 0.f : m_use;
    alpha[j] = grow ? ex2(st.m[j] - sub) : 1.f;
    p[j] = ex2(x[j] - sub);
    p[j + 2] = ex2(x[j + 2] - sub);
    st.l[j] = st.l[j] * alpha[j] + p[j] + p[j + 2];
    st.m[j] = m_use;
  }
  if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
    for (int c = 0; c < C::NC; ++c) {
      st.acc[c][0] *= alpha[0];
      st.acc[c][2] *= alpha[0];
      st.acc[c][1] *= alpha[1];
      st.acc[c][3] *= alpha[1];
    }
  }
  if constexpr (kLateV<D>) read_v<D, FP8>(r, vp, base, kv_hi, g, t);
  // P^T as the B operand of the PV product: transpose the two 8x8 blocks.
  const uint32_t pb0 = movmatrix_trans(pack2<FP8>(p[0], p[1]));
  const uint32_t pb1 = movmatrix_trans(pack2<FP8>(p[2], p[3]));
  // O^T += V^T P^T.
#pragma unroll
  for (int c = 0; c < C::NC; ++c) {
    uint32_t a[4];
    if constexpr (FP8) {
      const uint32_t sel = (c & 1) ? 0x7362u : 0x5140u;
      const uint32_t lo = __byte_perm(r.v[0][c >> 1], r.v[1][c >> 1], sel);
      const uint32_t hi = __byte_perm(r.v[2][c >> 1], r.v[3][c >> 1], sel);
      e4m3x4_to_f16x2x2(lo, a[0], a[1]);
      e4m3x4_to_f16x2x2(hi, a[2], a[3]);
    } else {
      a[0] = __byte_perm(r.v[0][c], r.v[1][c], 0x5410u);
      a[1] = __byte_perm(r.v[0][c], r.v[1][c], 0x7632u);
      a[2] = __byte_perm(r.v[2][c], r.v[3][c], 0x5410u);
      a[3] = __byte_perm(r.v[2][c], r.v[3][c], 0x7632u);
    }
    mma16816<FP8>(st.acc[c], a, pb0, pb1);
  }
}

// Steps a warp takes at a time over a cache with block scales. The e4m3 path
// waits for its own chain (shared memory, conversions, products, row maximum,
// exponentials, products) more than for memory; two steps in one chain share the
// maximum and the rescale and leave twice as many independent instructions (8 x
// 131072 keys, 64 and 8 heads of 128: one step 399 us, two 394, and 367 with the
// page layout below; 64 x 512 to 8192 keys 130, 126 and 108.5).
template <bool SCALED>
constexpr int kStepsAtOnce = SCALED ? 2 : 1;

// Key slot of MMA row m of S^T over a cache with block scales: 0 5 2 7 4 1 6 3,
// and 8 more. Rows of whole 128-byte panels arrive swizzled (chunk c of row r at
// c ^ (r % 8)); a 16-byte shared-memory read takes its lanes eight at a time, two
// lane groups g and all four t. Those read K rows that differ in bit 2, at chunks
// t and 4 + t, and V rows 0, 2, 4, 6 (or 5, 7, 1, 3) at two neighbouring chunks:
// eight different ones either way, so that no read has bank conflicts (with plain
// rows and keys 4t .. 4t + 3 to a lane a step's reads take 96 wavefronts at head_dim
// 128, so 32).
__device__ __forceinline__ int scaled_key_of_row(int m) { return m ^ ((m & 1) << 2); }

template <int D>
struct ScaledPage {
  using C = DecodeCfg<D, true>;
  static constexpr bool kSwizzle = D % 128 == 0;
  static constexpr int kBoxDims = kSwizzle ? 128 : D;  // elements per box row
  static constexpr int kPanels = D / kBoxDims;
  static constexpr int kRow = kBoxDims;                // bytes between rows of a panel
  static constexpr int kPanelBytes = 16 * kRow;
  __device__ static __forceinline__ int at(int key, int o) {
    if constexpr (kSwizzle)
      return (o >> 7) * kPanelBytes + key * 128 + ((((o >> 4) & 7) ^ (key & 7)) << 4) + (o & 15);
    else
      return key * D + o;
  }
  // This lane's reads of a step: K row scaled_key_of_row(g) (and 8 rows on), V rows
  // scaled_key_of_row(2t) and (2t + 1) (and 8 rows on).
  int k[C::NKL], v[2][C::NVL], k_key, v_key[2];
  __device__ __forceinline__ ScaledPage(int g, int t) {
    k_key = scaled_key_of_row(g);
#pragma unroll
    for (int l = 0; l < C::NKL; ++l) k[l] = at(k_key, l * 4 * C::KE + t * C::KE);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      v_key[j] = scaled_key_of_row(2 * t + j);
#pragma unroll
      for (int l = 0; l < C::NVL; ++l) v[j][l] = at(v_key[j], l * 8 * C::VE + g * C::VE);
    }
  }
  // Rows at or beyond `rows` read as zero (the page may hold anything there); ALL: none is.
  template <bool ALL>
  __device__ __forceinline__ void read_k(StepRegs<D, true>& r, const uint8_t* page, int rows) const {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int l = 0; l < C::NKL; ++l)
        lds_words<C::KE>(&r.k[h][l * (C::KE / 4)], page + k[l] + h * 8 * kRow,
                         ALL || k_key + 8 * h < rows);
  }
  template <bool ALL>
  __device__ __forceinline__ void read_v(StepRegs<D, true>& r, const uint8_t* page, int rows) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int l = 0; l < C::NVL; ++l)
        lds_words<C::VLB>(&r.v[j][l * (C::VLB / 4)], page + v[j & 1][l] + (j >> 1) * 8 * kRow,
                          ALL || v_key[j & 1] + 8 * (j >> 1) < rows);
  }
};

// The two steps at base[0] and base[1] (their K and V rows at kp and vp): as
// compute_step, with one reference for both. A step past kv_hi contributes nothing.
// release() refills the stages, by the whole warp: at the end, and above head_dim
// 128, where an SM holds half as many warps, as soon as nothing of them is left to
// be read (16 x 30000 keys, head_dim 192: 320 / 267 us; head_dim 256, 64 x 4096: 199 /
// 178; but at 128, 8 x 131072 343 / 359 us).
template <int D, bool SHAPED, class Release>
__device__ __forceinline__ void compute_two_scaled(WarpState<D>& st, const uint8_t* const (&kp)[2],
                                                   const uint8_t* const (&vp)[2], int kv_hi,
                                                   const uint32_t (&qb)[D / 16][2],
                                                   const float (&cq)[2], const StepMask& mk,
                                                   const StepScale (&scale)[2], ValueUnit& unit,
                                                   const int (&base)[2], const ScaledPage<D>& page,
                                                   int g, const Release& release) {
  using C = DecodeCfg<D, true>;
  StepRegs<D, true> r[2];
  const bool all = base[1] + 16 <= kv_hi;  // (the second step is the later one)
  auto read_v = [&]() {
#pragma unroll
    for (int n = 0; n < 2; ++n)
      if (all) page.template read_v<true>(r[n], vp[n], 16);
      else page.template read_v<false>(r[n], vp[n], kv_hi - base[n]);
  };
#pragma unroll
  for (int n = 0; n < 2; ++n)
    if (all) page.template read_k<true>(r[n], kp[n], 16);
    else page.template read_k<false>(r[n], kp[n], kv_hi - base[n]);
  float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
  for (int c = 0; c < C::NC; ++c) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      uint32_t a[4];
      e4m3x4_to_f16x2x2(r[n].k[0][c], a[0], a[2]);
      e4m3x4_to_f16x2x2(r[n].k[1][c], a[1], a[3]);
      mma16816<true>(s[n], a, qb[c][0], qb[c][1]);
    }
  }
  read_v();
  float x[2][4];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const float cc[2] = {cq[0] * scale[n].k, cq[1] * scale[n].k};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = base[n] + page.k_key + 8 * (e >> 1);
      x[n][e] = s[n][e] * cc[e & 1];
      if constexpr (SHAPED) {
        if (mk.cap_log2 > 0.f) x[n][e] = cap_score(x[n][e] * mk.cap_arg, mk.cap_log2);
        const RowBias& b = mk.bias[e & 1];
        x[n][e] = fmaf(-b.slope2, static_cast<float>(abs(mk.pos[e & 1] - key) - b.shift), x[n][e]);
      }
    }
    if (base[n] < mk.lo_full || base[n] + 16 > mk.hi_full) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = base[n] + page.k_key + 8 * (e >> 1);
        const int pos = mk.pos[e & 1];
        bool ok = key < mk.kv_hi;
        if (mk.causal) ok = ok && key <= (SHAPED ? mk.last[e & 1] : pos);
        if (mk.window > 0) ok = ok && (key > pos - mk.window || (SHAPED && key < mk.sinks));
        x[n][e] = ok ? x[n][e] : -INFINITY;
      }
    }
  }
  float top[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    top[j] = fmaxf(fmaxf(x[0][j], x[0][j + 2]), fmaxf(x[1][j], x[1][j + 2]));
    top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 4));
    top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 8));
    top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
  }
  if constexpr (kLateV<D>) release();
  float p[2][4], alpha[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float mx = top[j];
    const bool first = st.m[j] == -INFINITY;
    const float m_new = fmaxf(st.m[j], mx);
    const bool grow = first || (m_new > st.m[j] + kRescaleThreshold);
    float m_use = grow ? m_new : st.m[j];
    if (first && mx <= mk.phi2 + kRescaleThreshold && mx >= mk.phi2 - kUnifiedAbove<true>)
      m_use = mk.phi2;
    const float sub = (m_use == -INFINITY) ? 0.f : m_use;
    alpha[j] = grow ? ex2(st.m[j] - sub) : 1.f;
    st.l[j] *= alpha[j];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      p[n][j] = ex2(x[n][j] - sub);
      p[n][j + 2] = ex2(x[n][j + 2] - sub);
      st.l[j] += p[n][j] + p[n][j + 2];
    }
    st.m[j] = m_use;
  }
  // (the scales are the same for the whole warp)
  const float least = fminf(scale[0].v, scale[1].v), most = fmaxf(scale[0].v, scale[1].v);
  bool near = unit.near(least, most);
  if (!near) {
    const float shrink = unit.follow(least, most);
    alpha[0] *= shrink;
    alpha[1] *= shrink;
    near = unit.near(least, most);
  }
  if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
    for (int c = 0; c < C::NC; ++c) {
      st.acc[c][0] *= alpha[0];
      st.acc[c][2] *= alpha[0];
      st.acc[c][1] *= alpha[1];
      st.acc[c][3] *= alpha[1];
    }
  }
  // A step's V codes of chunk c as an f16 operand.
  auto v_operand = [&](int n, int c, uint32_t (&a)[4]) {
    const uint32_t sel = (c & 1) ? 0x7362u : 0x5140u;
    const uint32_t lo = __byte_perm(r[n].v[0][c >> 1], r[n].v[1][c >> 1], sel);
    const uint32_t hi = __byte_perm(r[n].v[2][c >> 1], r[n].v[3][c >> 1], sel);
    e4m3x4_to_f16x2x2(lo, a[0], a[1]);
    e4m3x4_to_f16x2x2(hi, a[2], a[3]);
  };
  if (near) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float f = scale[n].v * unit.inv;
      const uint32_t pb0 = movmatrix_trans(pack2<true>(p[n][0] * f, p[n][1] * f));
      const uint32_t pb1 = movmatrix_trans(pack2<true>(p[n][2] * f, p[n][3] * f));
#pragma unroll
      for (int c = 0; c < C::NC; ++c) {
        uint32_t a[4];
        v_operand(n, c, a);
        mma16816<true>(st.acc[c], a, pb0, pb1);
      }
    }
  } else {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float f = scale[n].v * unit.inv;
      const uint32_t pb0 = movmatrix_trans(pack2<true>(p[n][0], p[n][1]));
      const uint32_t pb1 = movmatrix_trans(pack2<true>(p[n][2], p[n][3]));
#pragma unroll
      for (int c = 0; c < C::NC; ++c) {
        uint32_t a[4];
        v_operand(n, c, a);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        mma16816<true>(o, a, pb0, pb1);
#pragma unroll
        for (int e = 0; e < 4; ++e) st.acc[c][e] = fmaf(o[e], f, st.acc[c][e]);
      }
    }
  }
  if constexpr (!kLateV<D>) release();
}

// Shared memory of one CTA: a ring of R stages per warp, each holding the K
// and V rows (16 x head_dim, in the page layout above) of one 16-key step as
// TMA lands them; then one mbarrier per stage. After the loop the ring is
// reused for the cross-warp merge. The sizes come from the scheduler's copy of
// the decode geometry, which also sizes splits by the CTAs an SM holds.
template <int D, bool FP8>
struct Ring {
  static constexpr int kElt = FP8 ? 1 : 2;
  static constexpr int kRowBytes = D * kElt;
  static constexpr int kStage = decode_stage_bytes(D, kElt);
  static constexpr int kStages = decode_ring_stages(D, kElt);
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kBars = kRing;
  static constexpr int kMisc = kBars + 8 * kWarps * kStages;
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;  // slack for 1024-byte alignment (swizzle atoms)
  static constexpr int kCtasPerSm = decode_ctas_per_sm(D, kElt);
  static_assert(kAlloc == decode_smem_bytes(D, kElt), "decode shared memory");
  static_assert(kWarps * (UA_DECODE_ROWS * (D + 2) + 1) * 4 <= kRing, "merge buffers alias the ring");
};

template <int D, bool FP8, bool SCALED>
using KernelPage = std::conditional_t<SCALED, ScaledPage<D>, PageLayout<D, FP8>>;

template <int D, bool FP8, bool SHAPED, bool SCALED>
__global__ void __launch_bounds__(kThreads, Ring<D, FP8>::kCtasPerSm)
    decode_kernel(const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const KernelParams p) {
  using C = DecodeCfg<D, FP8>;
  using RC = Ring<D, FP8>;
  constexpr int R = RC::kStages;
  extern __shared__ uint8_t dsm_raw[];
  uint8_t* dsm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(dsm + RC::kBars);
  volatile int32_t* never = reinterpret_cast<volatile int32_t*>(dsm + RC::kMisc);
  // merge buffers (valid only after the loop; they alias the ring)
  float (*red_acc)[UA_DECODE_ROWS][D] = reinterpret_cast<float (*)[UA_DECODE_ROWS][D]>(dsm);
  float (*red_m)[UA_DECODE_ROWS] =
      reinterpret_cast<float (*)[UA_DECODE_ROWS]>(dsm + kWarps * UA_DECODE_ROWS * D * 4);
  float (*red_l)[UA_DECODE_ROWS] = red_m + kWarps;
  [[maybe_unused]] float* const red_unit = red_l[kWarps];  // (SCALED: 1 / the warp's unit of O)

  const ua_tile tile = p.tiles[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0 && p.span_start != nullptr) atomicMin(p.span_start, sm100::globaltimer_ns());
  auto stamp_end = [&]() {
    if (threadIdx.x == 0 && p.span_end != nullptr) atomicMax(p.span_end, sm100::globaltimer_ns());
  };
  if (threadIdx.x == 0) {
    *never = 0;
    for (int i = 0; i < kWarps * R; ++i) sm100::mbar_init(&bars[i], 1);
    sm100::fence_mbar_init();
  }
  __syncthreads();

  // Per-sequence values from the device arrays; every range is clamped so
  // that disagreeing host/device lengths cannot send a read out of bounds.
  const int q_start = p.cu_query_lens[tile.seq];
  const int qlen = p.cu_query_lens[tile.seq + 1] - q_start;
  const int kv_len = p.kv_lens[tile.seq];
  const int ctx = kv_len - qlen;
  const int nrows = min(tile.nrows, qlen * p.qpk - tile.row0);
  const int kv_hi = min(min(tile.kv_hi, kv_len), p.max_blocks_per_seq * p.block_size);
  const int kv_lo = tile.kv_lo;

  // ---- Q fragments (B operand of S^T = K Q^T): row n = g of the tile.
  uint32_t qb[C::NC][2];
  float cc[2];
  {
    uint32_t qw[C::QW];
    const bool row_ok = g < nrows;
    const int r = tile.row0 + (row_ok ? g : 0);
    const int tok = q_start + r / p.qpk;
    const int head = tile.kv_head * p.qpk + r % p.qpk;
    const uint8_t* qrow = reinterpret_cast<const uint8_t*>(p.q) +
                          (static_cast<int64_t>(tok) * p.num_q_heads + head) * D * 2;
#pragma unroll
    for (int l = 0; l < C::NKL; ++l) {
#pragma unroll
      for (int h = 0; h < C::KE / 8; ++h) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (row_ok) x = *reinterpret_cast<const uint4*>(qrow + (l * 4 * C::KE + t * C::KE + 8 * h) * 2);
        const int w = l * (C::KE / 2) + 4 * h;
        qw[w + 0] = x.x;
        qw[w + 1] = x.y;
        qw[w + 2] = x.z;
        qw[w + 3] = x.w;
      }
    }
    if constexpr (FP8) {
      // f16 operands for the e4m3 path: scale each Q row by a power of two so
      // that its largest magnitude lies in [2^14, 2^15); exact for every
      // element within 2^-29 of the row maximum. The factor is undone in the
      // per-row score multiplier.
      float amax = 0.f;
#pragma unroll
      for (int w = 0; w < C::QW; ++w) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qw[w]));
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      int e = 0;
      if (amax > 0.f && amax < INFINITY) {
        int E;
        frexpf(amax, &E);
        e = min(max(15 - E, -126), 126);
      }
      const float up = __int_as_float((127 + e) << 23);
      const float down = __int_as_float((127 - e) << 23);
#pragma unroll
      for (int w = 0; w < C::QW; ++w) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qw[w]));
        qw[w] = pack2<true>(f.x * up, f.y * up);
      }
      const float row_mult = p.score_scale_log2 * down;
      cc[0] = __shfl_sync(0xffffffffu, row_mult, 4 * (2 * t));
      cc[1] = __shfl_sync(0xffffffffu, row_mult, 4 * (2 * t + 1));
    } else {
      cc[0] = cc[1] = p.score_scale_log2;
    }
#pragma unroll
    for (int c = 0; c < C::NC; ++c) {
      qb[c][0] = qw[2 * c];
      qb[c][1] = qw[2 * c + 1];
    }
  }

  // ---- Visibility of the lane's two rows (columns n = 2t, 2t+1).
  StepMask mk;
  mk.kv_hi = kv_hi;
  mk.causal = p.causal;
  mk.window = p.window;
  mk.phi2 = p.unified_max_on ? p.unified_max_log2 : __int_as_float(0x7fc00000);
  {
    const int last = max(nrows - 1, 0);
    const int min_pos = ctx + tile.row0 / p.qpk;
    const int max_pos = ctx + (tile.row0 + last) / p.qpk;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = 2 * t + j;
      mk.pos[j] = (n < nrows) ? ctx + (tile.row0 + n) / p.qpk : max_pos;
    }
    mk.hi_full = p.causal ? min(kv_hi, min_pos + 1) : kv_hi;
    mk.lo_full = p.window > 0 ? max_pos - p.window + 1 : INT_MIN;
    if constexpr (SHAPED) {
      mk.sinks = p.shape.sinks;
      const int prefix = p.shape.prefix_lens ? p.shape.prefix_lens[tile.seq] : 0;
      mk.cap_log2 = p.shape.cap_log2;
      mk.cap_arg = p.shape.cap_arg;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = 2 * t + j;
        mk.last[j] = max(mk.pos[j], prefix - 1);
        // (of the whole row: the same in every split piece)
        if (p.shape.slopes && n < nrows)
          mk.bias[j] = row_bias(
              p.shape.slopes[tile.kv_head * p.qpk + (tile.row0 + n) % p.qpk],
              p.window > 0 && p.shape.sinks <= 0 ? min(mk.pos[j], p.window - 1) : mk.pos[j],
              (p.causal ? min(kv_len - 1, mk.last[j]) : kv_len - 1) - mk.pos[j]);
      }
      if (p.causal) mk.hi_full = min(kv_hi, max(min_pos + 1, prefix));
    }
  }

  WarpState<D> st_state;
#pragma unroll
  for (int c = 0; c < C::NC; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) st_state.acc[c][e] = 0.f;
  st_state.m[0] = st_state.m[1] = -INFINITY;
  st_state.l[0] = st_state.l[1] = 0.f;

  // ---- Stream the key range: warp w takes steps w, w+4, w+8, ...; each step
  // is one TMA box of K and one of V (16 keys of one page) into the warp's ring.
  int nsteps = kv_hi > kv_lo ? (kv_hi - kv_lo + 15) / 16 : 0;
  int gap_lo = INT_MAX, gap = 0;  // a range that spans the keys behind the sinks passes over them
  if constexpr (SHAPED) {
    const KeyGap no_row = gap_within(
        key_gap(p.shape.sinks, p.window, ctx + tile.row0 / p.qpk, kKeyStep), kv_lo, kv_hi);
    if (no_row.hi > no_row.lo) {
      gap_lo = no_row.lo;
      gap = no_row.hi - no_row.lo;
      nsteps -= gap / 16;
    }
  }
  const int my_n = nsteps > warp ? (nsteps - warp + kWarps - 1) / kWarps : 0;
  auto step_base = [&](int k) {
    const int at = kv_lo + 16 * (warp + kWarps * k);
    return SHAPED && at >= gap_lo ? at + gap : at;
  };
  uint8_t* ring = dsm + warp * R * RC::kStage;
  uint64_t* wbar = bars + warp * R;
  // Page ids, 32 steps at a time: lane l holds the page of step 32c + l.
  // SCALED: and the page's scales, of this chunk of steps and of the one before
  // (a step is computed at most a ring after it was issued). The copy at a refill
  // waits for loads that are a chunk old; the new ones are waited for by the first
  // step that needs them.
  // A step's slot in its page is looked up with the page where a step's place costs the
  // arithmetic of a gap too (8 x 131072 keys, e4m3, 64 and 8 heads, capped: 375 us, 391
  // with both at the copies, 386 without a gap), or scales come with the page anyway.
  constexpr bool kSlotWithPage = SCALED || SHAPED;
  int32_t ids = -1, slots = 0;
  StepScale of_issue{1.f, 1.f}, of_before{1.f, 1.f};
  int issue_chunk = 0;
  auto refill_ids = [&](int c) {
    const int k = 32 * c + lane;
    ids = k < my_n ? p.block_tables[static_cast<int64_t>(tile.seq) * p.max_blocks_per_seq +
                                    step_base(k) / p.block_size]
                   : -1;
    if constexpr (kSlotWithPage) slots = step_base(k) % p.block_size;
    if constexpr (SCALED) {
      of_before = of_issue;
      issue_chunk = c;
      of_issue = StepScale{1.f, 1.f};
      if (ids >= 0 && static_cast<int64_t>(ids) < p.num_blocks) {
        const int64_t at = static_cast<int64_t>(ids) * p.num_kv_heads + tile.kv_head;
        of_issue = StepScale{usable_scale(__ldg(p.k_scales + at)), usable_scale(__ldg(p.v_scales + at))};
      }
    }
  };
  auto scale_of = [&](int k) {
    StepScale s{1.f, 1.f};
    if constexpr (SCALED) {
      const bool issued_last = (k >> 5) == issue_chunk;
      s.k = __shfl_sync(0xffffffffu, issued_last ? of_issue.k : of_before.k, k & 31);
      s.v = __shfl_sync(0xffffffffu, issued_last ? of_issue.v : of_before.v, k & 31);
    }
    return s;
  };
  // Whole-warp call: every lane takes part in the shuffle, lane 0 issues.
  auto issue = [&](int k) {
    const int32_t id = __shfl_sync(0xffffffffu, ids, k & 31);
    [[maybe_unused]] int32_t slot = 0;
    if constexpr (kSlotWithPage) slot = __shfl_sync(0xffffffffu, slots, k & 31);
    if (lane == 0) {
      const int base = step_base(k);
      int32_t blk = static_cast<int32_t>(p.num_blocks);  // out of range: TMA fills zeros
      if (id >= 0 && static_cast<int64_t>(id) < p.num_blocks) blk = id;
      else record_error(p.err, UA_ERR_BOUNDS);
      const int st = k % R;
      uint8_t* stage = ring + st * RC::kStage;
      sm100::fence_proxy_async_smem();
      sm100::mbar_arrive_expect_tx(&wbar[st], RC::kStage);
      using PL = KernelPage<D, FP8, SCALED>;
#pragma unroll
      for (int pn = 0; pn < PL::kPanels; ++pn) {
        sm100::tma_load_4d(stage + pn * PL::kPanelBytes, &map_k, &wbar[st], pn * PL::kBoxDims,
                           tile.kv_head, kSlotWithPage ? slot : base % p.block_size, blk);
        sm100::tma_load_4d(stage + 16 * RC::kRowBytes + pn * PL::kPanelBytes, &map_v, &wbar[st],
                           pn * PL::kBoxDims, tile.kv_head, kSlotWithPage ? slot : base % p.block_size, blk);
      }
    }
  };
  [[maybe_unused]] ValueUnit unit;
  int issued = 0, done = 0;
  if (my_n > 0) {
    refill_ids(0);
    for (; issued < my_n && issued < R; ++issued) issue(issued);
    constexpr int N = kStepsAtOnce<SCALED>;
    [[maybe_unused]] const ScaledPage<D> page(g, t);
    static_assert(N == 1 || N == 2, "one step or two");
    for (; N == 2 && done < my_n; done += 2) {
      const int more = min(done + 1, my_n - 1);  // (the last step's place where there is no second)
      const bool ok = __all_sync(
          0xffffffffu,
          sm100::mbar_wait(&wbar[done % R], (done / R) & 1, never, p.timeout_ns) &&
              sm100::mbar_wait(&wbar[more % R], (more / R) & 1, never, p.timeout_ns));
      if (!ok) {
        record_error(p.err, UA_ERR_DEVICE_TIMEOUT);
        break;
      }
      if constexpr (N == 2) {
        const uint8_t* const kp[2] = {ring + done % R * RC::kStage, ring + more % R * RC::kStage};
        const uint8_t* const vp[2] = {kp[0] + 16 * RC::kRowBytes, kp[1] + 16 * RC::kRowBytes};
        const int base[2] = {step_base(done), done + 1 < my_n ? step_base(done + 1) : kv_hi};
        const StepScale scale[2] = {scale_of(done), scale_of(more)};
        auto refill = [&]() {
          // orders every lane's reads before the first lane's proxy fence and copies
          __syncwarp();
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (issued >= my_n) break;
            if ((issued & 31) == 0) refill_ids(issued >> 5);
            issue(issued);
            ++issued;
          }
        };
        compute_two_scaled<D, SHAPED>(st_state, kp, vp, kv_hi, qb, cc, mk, scale, unit, base, page,
                                      g, refill);
      }
    }
    StepRegs<D, FP8> r;
    for (; N == 1 && done < my_n; ++done) {
      const int st = done % R;
      const bool ok = __all_sync(0xffffffffu, sm100::mbar_wait(&wbar[st], (done / R) & 1, never,
                                                                p.timeout_ns));
      if (!ok) {
        record_error(p.err, UA_ERR_DEVICE_TIMEOUT);
        break;
      }
      const uint8_t* stage = ring + st * RC::kStage;
      const uint8_t* vstage = stage + 16 * RC::kRowBytes;
      read_k<D, FP8>(r, stage, step_base(done), kv_hi, g, t);
      if constexpr (!kLateV<D>) read_v<D, FP8>(r, vstage, step_base(done), kv_hi, g, t);
      compute_step<D, FP8, SHAPED>(st_state, r, vstage, kv_hi, qb, cc, mk, step_base(done), g, t);
      __syncwarp();  // every lane has consumed the stage: it may be refilled
      if (issued < my_n) {
        if ((issued & 31) == 0) refill_ids(issued >> 5);
        issue(issued);
        ++issued;
      }
    }
    // Copies still in flight (only after a timeout) complete before exit.
    if (lane == 0)
      for (int k = done; k < issued; ++k)
        sm100::mbar_wait(&wbar[k % R], (k / R) & 1, never, p.timeout_ns);
    __syncwarp();
  }
  __syncthreads();  // the ring is reused for the merge below

  // ---- Merge the four warps.
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    st_state.l[j] += __shfl_xor_sync(0xffffffffu, st_state.l[j], 4);
    st_state.l[j] += __shfl_xor_sync(0xffffffffu, st_state.l[j], 8);
    st_state.l[j] += __shfl_xor_sync(0xffffffffu, st_state.l[j], 16);
  }
  if (g == 0) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      red_m[warp][2 * t + j] = st_state.m[j];
      red_l[warp][2 * t + j] = st_state.l[j];
    }
  }
  if constexpr (SCALED) {
    if (lane == 0) red_unit[warp] = unit.inv;
  }
#pragma unroll
  for (int c = 0; c < C::NC; ++c) {
    const int d0 = v_dim<D, FP8>(2 * c, g);
    red_acc[warp][2 * t][d0] = st_state.acc[c][0];
    red_acc[warp][2 * t + 1][d0] = st_state.acc[c][1];
    red_acc[warp][2 * t][d0 + 1] = st_state.acc[c][2];
    red_acc[warp][2 * t + 1][d0 + 1] = st_state.acc[c][3];
  }
  __syncthreads();

  constexpr int kSeg = D / 16;  // dims per thread in the epilogue
  const int n = threadIdx.x / 16;
  const int d0 = (threadIdx.x % 16) * kSeg;
  const bool row_ok = n < nrows;
  float M = -INFINITY, L = 0.f;
  [[maybe_unused]] float inv_unit = INFINITY;  // SCALED: of the merged O, the largest of the warps'
  float o[kSeg];
#pragma unroll
  for (int e = 0; e < kSeg; ++e) o[e] = 0.f;
  if (row_ok) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_m[w][n]);
    if constexpr (SCALED) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (red_unit[w] > 0.f) inv_unit = fminf(inv_unit, red_unit[w]);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = red_m[w][n];
      float f = (mw == -INFINITY) ? 0.f : ex2(mw - M);
      L += f * red_l[w][n];
      if constexpr (SCALED) {
        if (red_unit[w] > 0.f) f *= inv_unit * ValueUnit::inverse(red_unit[w]);
      }
#pragma unroll
      for (int e = 0; e < kSeg; ++e) o[e] += f * red_acc[w][n][d0 + e];
    }
  }
  // bf16 output row n of this tile, scaled by `mult`.
  auto store_out = [&](const float* vals, float mult) {
    const int r = tile.row0 + n;
    const int tok = q_start + r / p.qpk;
    const int head = tile.kv_head * p.qpk + r % p.qpk;
    uint32_t packed[kSeg / 2];
#pragma unroll
    for (int e = 0; e < kSeg / 2; ++e)
      packed[e] = pack2<false>(vals[2 * e] * mult, vals[2 * e + 1] * mult);
    uint8_t* dst = reinterpret_cast<uint8_t*>(p.out) +
                   ((static_cast<int64_t>(tok) * p.num_q_heads + head) * D + d0) * 2;
    if constexpr (kSeg % 8 == 0) {
#pragma unroll
      for (int i = 0; i < kSeg / 8; ++i)
        *reinterpret_cast<uint4*>(dst + 16 * i) =
            make_uint4(packed[4 * i], packed[4 * i + 1], packed[4 * i + 2], packed[4 * i + 3]);
    } else if constexpr (kSeg % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kSeg / 4; ++i)
        *reinterpret_cast<uint2*>(dst + 8 * i) = make_uint2(packed[2 * i], packed[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < kSeg / 2; ++i) *reinterpret_cast<uint32_t*>(dst + 4 * i) = packed[i];
    }
  };
  const float inv = !(L > 0.f) ? 0.f
                    : SCALED   ? ValueUnit::inverse(inv_unit) / L
                               : p.v_scale / L;
  if (tile.slot < 0) {
    if (row_ok) store_out(o, inv);
    stamp_end();
    return;
  }
  // Split piece: normalised partial row and its base-2 log-sum-exp.
  if (row_ok) {
    float* wo = p.ws_o + (static_cast<int64_t>(tile.slot) * UA_DECODE_ROWS + n) * D + d0;
    if constexpr (kSeg % 4 == 0) {
#pragma unroll
      for (int e = 0; e < kSeg; e += 4)
        *reinterpret_cast<float4*>(wo + e) =
            make_float4(o[e] * inv, o[e + 1] * inv, o[e + 2] * inv, o[e + 3] * inv);
    } else {
#pragma unroll
      for (int e = 0; e < kSeg; e += 2)
        *reinterpret_cast<float2*>(wo + e) = make_float2(o[e] * inv, o[e + 1] * inv);
    }
    if (threadIdx.x % 16 == 0)
      p.ws_lse[static_cast<int64_t>(tile.slot) * UA_DECODE_ROWS + n] =
          L > 0.f ? M + log2f(L) : -INFINITY;
  }
  if (p.split_counters == nullptr) {  // a separate combine kernel merges the pieces
    stamp_end();
    return;
  }
  // Fused combine: the last piece of a group to finish merges all of them
  // (weights 2^(lse_s - lse*)), then re-arms the group's counter for the next call.
  __shared__ int s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int ns = p.groups[tile.group].nsplits;
    s_last = atomicAdd(&p.split_counters[tile.group], 1) == ns - 1;
  }
  __syncthreads();
  if (!s_last) {
    stamp_end();
    return;
  }
  __threadfence();
  const ua_combine_group grp = p.groups[tile.group];
  if (row_ok) {
    const float* lse = p.ws_lse + static_cast<int64_t>(grp.slot0) * UA_DECODE_ROWS + n;
    float Mx = -INFINITY;
    for (int sp = 0; sp < grp.nsplits; ++sp) Mx = fmaxf(Mx, __ldcg(lse + sp * UA_DECODE_ROWS));
    float W = 0.f;
    float acc[kSeg];
#pragma unroll
    for (int e = 0; e < kSeg; ++e) acc[e] = 0.f;
    for (int sp = 0; sp < grp.nsplits; ++sp) {
      const float l = __ldcg(lse + sp * UA_DECODE_ROWS);
      if (l == -INFINITY) continue;
      const float w = ex2(l - Mx);
      W += w;
      const float* src =
          p.ws_o + ((static_cast<int64_t>(grp.slot0) + sp) * UA_DECODE_ROWS + n) * D + d0;
      if constexpr (kSeg % 4 == 0) {
#pragma unroll
        for (int e = 0; e < kSeg; e += 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(src + e));
          acc[e] += w * v.x;
          acc[e + 1] += w * v.y;
          acc[e + 2] += w * v.z;
          acc[e + 3] += w * v.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < kSeg; e += 2) {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(src + e));
          acc[e] += w * v.x;
          acc[e + 1] += w * v.y;
        }
      }
    }
    store_out(acc, W > 0.f ? 1.f / W : 0.f);
  }
  if (threadIdx.x == 0) p.split_counters[tile.group] = 0;
  stamp_end();
}

template <int D, bool FP8, bool SHAPED, bool SCALED = false>
cudaError_t launch_decode_as(const KernelParams& p, cudaStream_t stream, bool after_prefill) {
  CUtensorMap mk, mv;
  const int elt = FP8 ? 1 : 2;
  using PL = KernelPage<D, FP8, SCALED>;
  // one box = the 16 key rows of one KV head in one page, one 128-byte panel
  // of head dims (swizzled) or the whole row
  cudaError_t e = encode_kv_page_map(&mk, p.k_cache, elt, D, p.num_kv_heads, p.block_size,
                                     p.num_blocks, PL::kBoxDims, 16, PL::kSwizzle);
  if (e == cudaSuccess)
    e = encode_kv_page_map(&mv, p.v_cache, elt, D, p.num_kv_heads, p.block_size, p.num_blocks,
                           PL::kBoxDims, 16, PL::kSwizzle);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> smem_set{0};
  e = set_smem_once(decode_kernel<D, FP8, SHAPED, SCALED>, Ring<D, FP8>::kAlloc, smem_set);
  if (e != cudaSuccess) return e;
  if (!after_prefill) {
    decode_kernel<D, FP8, SHAPED, SCALED>
        <<<p.num_tiles, kThreads, Ring<D, FP8>::kAlloc, stream>>>(mk, mv, p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.num_tiles));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Ring<D, FP8>::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_kernel<D, FP8, SHAPED, SCALED>, mk, mv, p);
}

template <int D, bool FP8>
cudaError_t launch_decode_d(const KernelParams& p, cudaStream_t stream, bool after_prefill) {
  if constexpr (FP8) {
    if (p.k_scales != nullptr)
      return shape_of(p.shape) == kShapePlain
                 ? launch_decode_as<D, FP8, false, true>(p, stream, after_prefill)
                 : launch_decode_as<D, FP8, true, true>(p, stream, after_prefill);
  }
  return shape_of(p.shape) == kShapePlain ? launch_decode_as<D, FP8, false>(p, stream, after_prefill)
                                          : launch_decode_as<D, FP8, true>(p, stream, after_prefill);
}

}  // namespace

cudaError_t launch_decode(const KernelParams& p, int head_dim, int kv_dtype, cudaStream_t stream,
                          bool after_prefill) {
  if (p.num_tiles <= 0) return cudaSuccess;
  const bool a = after_prefill;
  const bool f8 = kv_dtype != UA_KV_BF16;
  switch (head_dim) {
    case 32: return f8 ? launch_decode_d<32, true>(p, stream, a) : launch_decode_d<32, false>(p, stream, a);
    case 64: return f8 ? launch_decode_d<64, true>(p, stream, a) : launch_decode_d<64, false>(p, stream, a);
    case 96: return f8 ? launch_decode_d<96, true>(p, stream, a) : launch_decode_d<96, false>(p, stream, a);
    case 128: return f8 ? launch_decode_d<128, true>(p, stream, a) : launch_decode_d<128, false>(p, stream, a);
    case 160: return f8 ? launch_decode_d<160, true>(p, stream, a) : launch_decode_d<160, false>(p, stream, a);
    case 192: return f8 ? launch_decode_d<192, true>(p, stream, a) : launch_decode_d<192, false>(p, stream, a);
    case 224: return f8 ? launch_decode_d<224, true>(p, stream, a) : launch_decode_d<224, false>(p, stream, a);
    case 256: return f8 ? launch_decode_d<256, true>(p, stream, a) : launch_decode_d<256, false>(p, stream, a);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ua
