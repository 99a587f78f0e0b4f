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
// q and a bf16 cache, e4m3(x / scale) from a binary32 quotient for an e4m3
// cache.
//
// Angles. p w_i grows to many turns (131072 radians for the first pair of a
// long context), where a binary32 product has lost the angle's fraction. The
// frequency is held in turns (w / 2 pi) as an unevaluated sum of two floats
// and the position as two exact floats (p = 4096 p1 + p0); the products'
// exact remainders (fma) are kept and whole turns removed before the parts
// are added, which leaves an error below 2^-22 turns up to |p| = 2^24.
//
// HBM-bound: per token Hq d 2 B read and written, 2 Hkv d 2 B read and
// 2 Hkv d elt written. Two CTAs of 4 warps per append tile of the plan (up to 8
// new tokens of one sequence): the 8 warps take one token each, or share the
// tile's tokens when there are fewer (a decode step has one), a warp taking as
// many whole heads at a time as its 32 lanes hold, with eight such steps'
// loads in flight. A lane owns one unit of a head:
// 32 bytes, two 16-byte chunks that hold whole pairs -- chunks u and
// u + rotary_dim / 16 in the half layout, 2u and 2u + 1 otherwise -- so that a
// rotation needs no other lane's data, in place is safe, and a lane's eight
// (cos, sin) stay in registers over all heads of its token. They come from a
// table in shared memory that the CTA fills once (rotary_dim / 2 sines per
// token) while the first loads are under way.
// When the half layout's pairs do not fall on whole chunks (rotary_dim not a
// multiple of 16), a lane owns 16 consecutive elements and reads their
// partners from its warp's copy of the heads in shared memory: element e < 2P
// pairs with (e + P) mod 2P, so the partners of eight words are nine words mod
// P at places that stay the same for every head, shifted by half a word when P
// is odd. Elements that pass unchanged take cos 1, sin -0 and partner 0, which
// leaves every value as it is (-0 too). Prompts of 4 x 4096 tokens, 64 heads of
// 128 with 100 rotated 140 us, against 123 us aligned (196 with a read and a
// division of the index per element; with 2, 4, 6 and 8 heads in flight
// instead of 3 151, 147, 140 and 138 us, but chunks of 3850 tokens and 32
// heads 14.1, 16.8, 17.4 and 16.5 instead of 14.1).
#include <cmath>
#include <cstdint>

#include "rope_device.cuh"

namespace ua {

namespace {

using namespace rope_device;

template <bool FP8, Layout LAYOUT, bool AXES>
__global__ void __launch_bounds__(kThreads)
    rope_append_kernel(const __grid_constant__ RopeTable rope, const RopeAppendParams p,
                       const RopeScale k_scale, const RopeScale v_scale) {
  rope_append_block<FP8, LAYOUT, AXES>(rope, p, k_scale, v_scale, blockIdx.x);
}

RopeScale split_scale(float scale) {
  int e = 0;
  const float mant = 2.f * std::frexp(scale, &e);
  return {std::ldexp(1.f, 1 - e), mant, 1.f / mant};
}

template <bool FP8, bool AXES>
cudaError_t launch(const RopeTable& rope, const RopeAppendParams& p, cudaStream_t stream) {
  const RopeScale ks = split_scale(p.k_scale), vs = split_scale(p.v_scale);
  const int grid = p.num_tiles * kParts;
  if (p.interleaved)
    rope_append_kernel<FP8, kInterleaved, AXES><<<grid, kThreads, 0, stream>>>(rope, p, ks, vs);
  else if (p.rotary_dim % 16 == 0)
    rope_append_kernel<FP8, kHalf, AXES><<<grid, kThreads, 0, stream>>>(rope, p, ks, vs);
  else
    rope_append_kernel<FP8, kHalfOdd, AXES><<<grid, kThreads, 0, stream>>>(rope, p, ks, vs);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append(const RopeTable& rope, const RopeAppendParams& p,
                               cudaStream_t stream) {
  if (p.num_tiles <= 0) return cudaSuccess;
  if (p.tiles == nullptr || p.rotary_dim > 2 * kMaxPairs || p.rotary_dim > p.head_dim ||
      p.head_dim % 32 != 0)
    return cudaErrorInvalidValue;
  if (p.positions != nullptr && p.axes > 1)
    return p.fp8 ? launch<true, true>(rope, p, stream) : launch<false, true>(rope, p, stream);
  return p.fp8 ? launch<true, false>(rope, p, stream) : launch<false, false>(rope, p, stream);
}

}  // namespace ua
