// Rotary append: rotates a step's queries and new keys to their positions and
// writes the keys and values into the paged cache, in one launch (the append
// kernel of append.cu with the rotation in front of it).
//
// Pair (a, b) of a head at position p, with frequency w_i (radians per
// position) and amplitude m:
//   c = m cos(p w_i), s = m sin(p w_i):  a' = a c - b s,  b' = b c + a s
// for i < rotary_dim / 2, where the pair is (x[i], x[i + rotary_dim / 2])
// (half layout) or (x[2i], x[2i + 1]) (interleaved); elements from rotary_dim
// on pass unchanged. Rotation in binary32, one rounding at the end: bf16 for
// q and a bf16 cache, e4m3(x / scale) with the quotient in binary32 for an
// e4m3 cache.
//
// Angles. p w_i grows to many turns (131072 radians for the first pair of a
// long context), where a binary32 product has lost the angle's fraction. The
// frequency is held in turns (w / 2 pi) as an unevaluated sum of two floats
// and the position as two exact floats (p = 4096 p1 + p0); the products'
// exact remainders (fma) are kept and whole turns removed before the parts
// are added, which leaves an error below 2^-22 turns up to |p| = 2^24.
#include <cstdint>

#include "planner.h"
#include "ua_device.cuh"
#include "ua_kernels.h"

namespace ua {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;  // rotary_dim / 2 at head_dim 256

// (cos, sin) of 2 pi * p * (f_hi + f_lo).
__device__ __forceinline__ float2 rotation(int32_t p, float f_hi, float f_lo) {
  const float p1 = static_cast<float>(p >> 12) * 4096.f, p0 = static_cast<float>(p & 4095);
  const float t1 = __fmul_rn(p1, f_hi), t0 = __fmul_rn(p0, f_hi);
  const float e1 = __fmaf_rn(p1, f_hi, -t1), e0 = __fmaf_rn(p0, f_hi, -t0);
  const float low = __fmaf_rn(p1, f_lo, e1) + __fmaf_rn(p0, f_lo, e0);
  float r = (t1 - rintf(t1)) + (t0 - rintf(t0));  // each part in [-1/2, 1/2]
  r = (r - rintf(r)) + low;
  float2 cs;
  sincospif(2.f * r, &cs.y, &cs.x);
  return cs;
}

__device__ __forceinline__ float bf16_at(const void* p, int64_t i) {
  return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

// One CTA per append tile (up to 8 new tokens of one sequence).
template <bool FP8>
__global__ void __launch_bounds__(kThreads)
    rope_append_kernel(const __grid_constant__ RopeTable rope, const RopeAppendParams p) {
  __shared__ float2 turn[kAppendTokens][kMaxPairs];
  const ua_tile tile = p.tiles[blockIdx.x];
  const int pairs = p.rotary_dim / 2;
  for (int x = threadIdx.x; x < tile.nrows * pairs; x += kThreads) {
    const int w = x / pairs, i = x % pairs;
    const int32_t pos = p.positions ? p.positions[tile.row0 + w] : tile.kv_lo + w;
    const float2 cs = rotation(pos, rope.hi[i], rope.lo[i]);
    turn[w][i] = make_float2(cs.x * rope.amplitude, cs.y * rope.amplitude);
  }
  __syncthreads();
  const int d = p.head_dim;
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  for (int w = 0; w < tile.nrows; ++w) {
    const int64_t j = tile.row0 + w;
    const int pos = tile.kv_lo + w;
    int32_t blk = -1;
    if (pos >= 0 && pos / p.block_size < p.max_blocks_per_seq)
      blk = p.block_tables[static_cast<int64_t>(tile.seq) * p.max_blocks_per_seq +
                           pos / p.block_size];
    const bool ok = blk >= 0 && static_cast<int64_t>(blk) < p.num_blocks;
    if (!ok && threadIdx.x == 0) record_error(p.err, UA_ERR_BOUNDS);
    const int64_t dst_row = (static_cast<int64_t>(blk) * p.block_size + pos % p.block_size) *
                            p.num_kv_heads;
    // One head at a time per warp, so that in place (q_out == q) every element
    // of a head is read before any is written.
    for (int h = threadIdx.x / 32; h < heads; h += kThreads / 32) {
      const bool is_q = h < p.num_q_heads, is_v = h >= p.num_q_heads + p.num_kv_heads;
      const int hh = is_q ? h : (is_v ? h - p.num_q_heads - p.num_kv_heads : h - p.num_q_heads);
      const void* src = is_q ? p.q : (is_v ? p.v_new : p.k_new);
      const int64_t base =
          j * (is_q ? p.q_stride : (is_v ? p.v_stride : p.k_stride)) + static_cast<int64_t>(hh) * d;
      float y[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int e = (threadIdx.x & 31) + 32 * u;
        if (e >= d) break;
        const float a = bf16_at(src, base + e);
        y[u] = a;
        if (is_v || e >= p.rotary_dim) continue;
        const bool first = p.interleaved ? (e & 1) == 0 : e < pairs;
        const int i = p.interleaved ? e / 2 : (first ? e : e - pairs);
        const int other = p.interleaved ? e ^ 1 : (first ? e + pairs : e - pairs);
        const float b = bf16_at(src, base + other);
        const float2 cs = turn[w][i];
        y[u] = first ? fmaf(a, cs.x, -b * cs.y) : fmaf(a, cs.x, b * cs.y);
      }
      __syncwarp();
      if (!is_q && !ok) continue;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int e = (threadIdx.x & 31) + 32 * u;
        if (e >= d) break;
        if (is_q) {
          reinterpret_cast<__nv_bfloat16*>(
              p.q_out)[(j * p.num_q_heads + hh) * d + e] = __float2bfloat16_rn(y[u]);
        } else {
          void* cache = is_v ? p.v_cache : p.k_cache;
          const int64_t at = (dst_row + hh) * d + e;
          if constexpr (FP8)
            reinterpret_cast<uint8_t*>(cache)[at] = static_cast<uint8_t>(
                to_e4m3x4(__fdiv_rn(y[u], is_v ? p.v_scale : p.k_scale), 0.f, 0.f, 0.f) & 0xFFu);
          else
            reinterpret_cast<__nv_bfloat16*>(cache)[at] = __float2bfloat16_rn(y[u]);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeTable& rope, const RopeAppendParams& p,
                               cudaStream_t stream) {
  if (p.num_tiles <= 0) return cudaSuccess;
  if (p.tiles == nullptr || p.rotary_dim > 2 * kMaxPairs || p.rotary_dim > p.head_dim)
    return cudaErrorInvalidValue;
  if (p.fp8)
    rope_append_kernel<true><<<p.num_tiles, kThreads, 0, stream>>>(rope, p);
  else
    rope_append_kernel<false><<<p.num_tiles, kThreads, 0, stream>>>(rope, p);
  return cudaGetLastError();
}

}  // namespace ua
