// Append into an e4m3 cache with block scales: a step's new keys (turned to their
// positions, or as they are) and values, quantised with one scale for each page
// and KV head, in one launch with the rotation of the queries.
//
// Scale of a page and head (K and V each have their own), with amax the largest
// finite magnitude among the new elements (after the rotation, in binary32):
//   first new slot 0     scale = 2^k, the least k with amax <= 448 2^k (at least
//                        2^-100, at most 2^100; nothing but zeros: 2^-100)
//   earlier tokens       scale = old 2^n, the least n >= 0 with amax <= 448 old 2^n;
//                        their codes are divided by 2^n (exact but for what
//                        becomes subnormal)
// then code = e4m3(x / scale), as the other appends round. Powers of two lose
// nothing against any other scale: e4m3 has the same relative step in every
// binade, and 2^15 between its largest and its least normal value. An old scale
// outside [2^-100, 2^100] (a page that was never written) counts as none.
//
// One CTA of 4 warps per (page written to, run of heads, K or V). A warp owns one
// head, or a part of one head's tokens where pages are long or heads are few: as
// many tokens at a time as its 32 lanes hold, a lane owning the same 32 bytes of
// a head as in the rotary append (rope_device.cuh), four such steps in flight.
// A page that takes several rounds is written under the scale so far, and what came
// before its last growth once more at the end (32 KV heads, 128-slot pages, 4 x 4096
// tokens: 149 us; with the largest magnitude found in a pass of its own 394). (cos,
// sin) come from a table in shared memory, filled once a round for the CTA's heads.
// Bytes: 2 B read and 1 B written per new element of K and V, 4 B per element of q.
// 4 x 4096 tokens, 32 heads and 8 of 128, 16-slot pages: 75 us, the queries' part
// alone 42 (at the rate of HBM), the cache's 33 (15 at that rate: the angles' sines
// and the chain of loads, maximum and stores of a CTA); without rotation 23. Rotary dims
// that 16 does not divide: 100 of 128 rotated 112 us, 72 of 96 107 (71 with all 96; the
// pairs' partners come through shared memory and 200 bytes a thread are spilled). The two
// parts run one after the other: mixed CTA by CTA the same work takes 86 us, its two
// bodies do not fit the instruction cache together.
#include <cstdint>

#include "rope_device.cuh"

namespace ua {

namespace {

using namespace rope_device;

constexpr int kSteps = 4;  // token steps a warp holds in registers

// Tokens one warp holds in a round.
__host__ __device__ constexpr int warp_tokens(int head_dim) { return kSteps * (32 / (head_dim / 16)); }

// The table of a round's (cos, sin): pair i of a token at 8 units of pairs by
// remainder, so that lanes of neighbouring units read neighbouring places, and a row
// to a token with as much again between rows as the lanes of one token read.
__host__ __device__ constexpr int turn_units(int pairs) { return (pairs + 7) / 8; }
__host__ __device__ constexpr int turn_row(int pairs) { return 9 * turn_units(pairs); }
__device__ __forceinline__ int turn_at(int i, int pairs) {
  return (i & 7) * turn_units(pairs) + (i >> 3);
}
// At most 4 warps' tokens, 512 / head_dim * 4 of them, of head_dim / 2 pairs.
constexpr int kMostSmem = kWarps * kSteps * 512 / 16 * 9 * static_cast<int>(sizeof(float2));

constexpr uint32_t kLeastScale = (127u - 100u) << 23, kMostScale = (127u + 100u) << 23;

// The least 2^k with amax <= 448 * 2^k, within the limits (448 = 1.75 * 2^8).
__device__ __forceinline__ float fresh_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int k = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(min(max(k, 27), 227) << 23);
}

// The least n >= 0 with amax <= 448 old 2^n that leaves the scale within its limit.
__device__ __forceinline__ int doublings(float amax, float old) {
  const uint32_t a = __float_as_uint(amax), l = __float_as_uint(448.f * old);
  const int n = static_cast<int>(a >> 23) - static_cast<int>(l >> 23) +
                ((a & 0x7fffffu) > (l & 0x7fffffu) ? 1 : 0);
  return min(max(n, 0), static_cast<int>((kMostScale - __float_as_uint(old)) >> 23));
}

// How the keys of a launch are turned.
enum Turn { kTurnHalf, kTurnInterleaved, kTurnHalfOdd, kTurnNone };
constexpr Layout layout_of(Turn t) {
  return t == kTurnHalfOdd ? kHalfOdd : (t == kTurnInterleaved ? kInterleaved : kHalf);
}

// The block-th CTA of the cache's part.
template <Turn TURN, bool AXES>
__device__ __forceinline__ void fill_block(const RopeTable& rope, const FillParams& p, int block) {
  extern __shared__ float2 turn[];  // [tokens of a round][pairs]
  __shared__ uint32_t copy[TURN == kTurnHalfOdd ? kWarps * 32 * kUnitWords : 1];
  __shared__ float largest[2][kWarps];
  __shared__ int rounds_again[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_v = block & 1;
  const int groups = (p.num_kv_heads + p.heads_per_cta - 1) / p.heads_per_cta;
  const ua_tile tile = p.tiles[(block >> 1) / groups];
  const int share = p.warps_per_head;
  const int in_cta = warp / share, part = warp - in_cta * share;
  const int head = (block >> 1) % groups * p.heads_per_cta + in_cta;
  const bool active = in_cta < p.heads_per_cta && head < p.num_kv_heads;

  const int logical = tile.kv_lo / p.block_size, first = tile.kv_lo - logical * p.block_size;
  int32_t blk = -1;
  if (tile.kv_lo >= 0 && logical < p.max_blocks_per_seq)
    blk = p.block_tables[static_cast<int64_t>(tile.seq) * p.max_blocks_per_seq + logical];
  if (blk < 0 || static_cast<int64_t>(blk) >= p.num_blocks) {
    if (threadIdx.x == 0) record_error(p.err, UA_ERR_BOUNDS);
    return;
  }
  const int d = p.head_dim, pairs = TURN == kTurnNone ? 0 : p.rotary_dim / 2;
  const int units = d / 16, at_once = 32 / units;
  const int slot = lane / units, u = lane - slot * units;
  const bool mine = active && slot < at_once;
  const bool turns = !is_v && TURN != kTurnNone &&
                     (TURN == kTurnInterleaved ? 8 * u < pairs : 16 * u < 2 * pairs);
  const bool apart = TURN == kTurnHalf && turns;
  const int off0 = apart ? 8 * u : 16 * u;
  const int off1 = apart ? 8 * u + pairs : 16 * u + 8;

  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  const __nv_bfloat16* const src = static_cast<const __nv_bfloat16*>(is_v ? p.v_new : p.k_new) +
                                   tile.row0 * stride + static_cast<int64_t>(head) * d;
  uint8_t* const dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                       (static_cast<int64_t>(blk) * p.block_size * p.num_kv_heads + head) * d;
  const int64_t dst_stride = static_cast<int64_t>(p.num_kv_heads) * d;
  float* const scale_at =
      (is_v ? p.v_scales : p.k_scales) + static_cast<int64_t>(blk) * p.num_kv_heads + head;
  float old = 0.f;
  if (active && first > 0) {
    old = *scale_at;
    if (!(old >= __uint_as_float(kLeastScale) && old <= __uint_as_float(kMostScale))) old = 0.f;
  }

  // kTurnHalfOdd: where a unit's partner words are in the warp's copy (rope_device.cuh).
  uint32_t* const heads_copy = copy + warp * 32 * kUnitWords;
  const int turning = pairs - 8 * u, shift = (pairs & 1) * 16;
  int place[9];
  if constexpr (TURN == kTurnHalfOdd) {
#pragma unroll
    for (int i = 0; i < 9; ++i) {
      int word = 8 * u + pairs / 2 + i;
      if (word >= pairs) word -= pairs;
      if (word >= pairs || slot >= at_once) word = 0;  // not used
      place[i] = (slot >= at_once ? 0 : slot * units * kUnitWords) + word + word / 8;
    }
  }

  const int round_tokens = kSteps * at_once * share;
  const int rounds = (tile.nrows + round_tokens - 1) / round_tokens;
  const int lane_token = part * kSteps * at_once + slot;  // in its round, of the first step
  float x[kSteps][16];
  // The round's elements of this lane, turned, into x.
  auto take = [&](int r) {
    uint4 c0[kSteps], c1[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int tok = r * round_tokens + lane_token + i * at_once;
      c0[i] = c1[i] = make_uint4(0u, 0u, 0u, 0u);
      if (mine && tok < tile.nrows) {
        c0[i] = ld_row(src + tok * stride + off0);
        c1[i] = ld_row(src + tok * stride + off1);
      }
    }
    if constexpr (TURN != kTurnNone) {
      if (!is_v) {
        const int tokens = min(round_tokens, tile.nrows - r * round_tokens);
        __syncthreads();  // the round before has been read
        // a pair to a thread, or two threads and more
        const int wide = 32 - __clz(max(pairs - 1, 1));  // threads to a token, as a power of two
        const int i = threadIdx.x & ((1 << wide) - 1);
        const int at = turn_at(i, pairs);
        if (i < pairs) {
          const PairFrequency<AXES> f(rope, p.positions, p.positions_stride, i);
          for (int t = threadIdx.x >> wide; t < tokens; t += kThreads >> wide) {
            const int tok = r * round_tokens + t;
            turn[t * turn_row(pairs) + at] = f.at(tile.row0 + tok, tile.kv_lo + tok);
          }
        }
        __syncthreads();
      }
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      float(&y)[16] = x[i];
      {
        float lo[8], hi[8];
        widen8(c0[i], lo);
        widen8(c1[i], hi);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = lo[k], y[8 + k] = hi[k];
      }
      if constexpr (TURN != kTurnNone) {
        if (is_v) continue;  // (the whole CTA)
        if constexpr (TURN == kTurnHalfOdd) {
          __syncwarp();  // the copy of the step before has been read
          uint32_t* own = heads_copy + lane * kUnitWords;
          own[0] = c0[i].x, own[1] = c0[i].y, own[2] = c0[i].z, own[3] = c0[i].w;
          own[4] = c1[i].x, own[5] = c1[i].y, own[6] = c1[i].z, own[7] = c1[i].w;
          __syncwarp();
        }
        const int tok = r * round_tokens + lane_token + i * at_once;
        if (!mine || !turns || tok >= tile.nrows) continue;
        const float2* cs = turn + (lane_token + i * at_once) * turn_row(pairs);
        if constexpr (TURN == kTurnHalf) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 t = cs[turn_at(8 * u + k, pairs)];
            const float a = y[k], b = y[8 + k];
            y[k] = fmaf(a, t.x, -b * t.y);
            y[8 + k] = fmaf(b, t.x, a * t.y);
          }
        } else if constexpr (TURN == kTurnInterleaved) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (8 * u + k >= pairs) continue;
            const float2 t = cs[turn_at(8 * u + k, pairs)];
            const float a = y[2 * k], b = y[2 * k + 1];
            y[2 * k] = fmaf(a, t.x, -b * t.y);
            y[2 * k + 1] = fmaf(b, t.x, a * t.y);
          }
        } else {
          uint32_t word = heads_copy[place[0]];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t next = heads_copy[place[k + 1]];
            const uint32_t b = k < turning ? __funnelshift_r(word, next, shift) : 0u;
            word = next;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int at = 16 * u + 2 * k + e;
              if (at >= 2 * pairs) continue;
              const float2 t = cs[turn_at(at < pairs ? at : at - pairs, pairs)];
              const float partner = e ? bf16_hi(b) : bf16_lo(b);
              y[2 * k + e] = fmaf(y[2 * k + e], t.x, partner * (at < pairs ? -t.y : t.y));
            }
          }
        }
      }
    }
  };

  // Round after round: the scale so far, and the round's codes under it. Rounds
  // written before the scale grew for the last time are written again after the
  // last (they come from L2, most pages have none: a page's first tokens are
  // nearly as loud as all of them).
  float scale = 0.f, amax = 0.f;
  RopeScale div;
  int grown = 0;  // rounds before the last growth
  int turns_left = rounds;
  for (int it = 0; it < turns_left; ++it) {
    const bool again = it >= rounds;
    const int r = again ? it - rounds : it;
    take(r);
    if (!again) {
      // The largest finite magnitude of the round's elements (fmax3 passes over NaN).
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int k = 0; k < 16; k += 2) top = sm100::fmax3(top, fabsf(x[i][k]), fabsf(x[i][k + 1]));
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
      if (top == INFINITY) {
        top = 0.f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(x[i][k]) < INFINITY ? fabsf(x[i][k]) : 0.f);
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
      }
      if (share > 1) {
        if (lane == 0) largest[r & 1][warp] = top;
        __syncthreads();  // (also: every warp of a head has read the old scale)
        for (int w = 0; w < share; ++w) top = fmaxf(top, largest[r & 1][in_cta * share + w]);
      }
      amax = fmaxf(amax, top);
      const float now = old > 0.f
                            ? __uint_as_float(__float_as_uint(old) + (doublings(amax, old) << 23))
                            : fresh_scale(amax);
      if (now != scale) {
        scale = now;
        grown = r;
        const uint32_t bits = __float_as_uint(scale);
        div.shift = __uint_as_float((254u << 23) - (bits & 0x7f800000u));
        div.mant = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
        div.inv = __frcp_rn(div.mant);
      }
      if (r == rounds - 1 && rounds > 1) {
        // a round that one warp needs again is one for the whole CTA (`take` waits for all)
        if (lane == 0) rounds_again[warp] = grown;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) turns_left = max(turns_left, rounds + rounds_again[w]);
      }
    }
    if (again && r >= grown) continue;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int tok = r * round_tokens + lane_token + i * at_once;
      if (!mine || tok >= tile.nrows) continue;
      float lo[8], hi[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) lo[k] = x[i][k], hi[k] = x[i][8 + k];
      uint2 a, b;
      if (div.mant == 1.f) {  // a power of two, as the rule makes them: an exact product
#pragma unroll
        for (int k = 0; k < 8; ++k) lo[k] *= div.shift, hi[k] *= div.shift;
        a = make_uint2(to_e4m3x4(lo[0], lo[1], lo[2], lo[3]), to_e4m3x4(lo[4], lo[5], lo[6], lo[7]));
        b = make_uint2(to_e4m3x4(hi[0], hi[1], hi[2], hi[3]), to_e4m3x4(hi[4], hi[5], hi[6], hi[7]));
      } else {
        a = quantize8(lo, div);
        b = quantize8(hi, div);
      }
      uint8_t* row = dst + (first + tok) * dst_stride;
      if (off1 == off0 + 8) {
        *reinterpret_cast<uint4*>(row + off0) = make_uint4(a.x, a.y, b.x, b.y);
      } else {
        *reinterpret_cast<uint2*>(row + off0) = a;
        *reinterpret_cast<uint2*>(row + off1) = b;
      }
    }
  }
  if (active && part == 0 && lane == 0) *scale_at = scale;
  const int n = old > 0.f ? doublings(amax, old) : 0;
  // Earlier tokens of a page whose scale grew.
  if (n > 0 && mine) {
    const float down = __uint_as_float(static_cast<uint32_t>(127 - min(n, 126)) << 23);
    auto divided = [&](uint32_t codes) {
      uint32_t lo, hi;
      e4m3x4_to_f16x2x2(codes, lo, hi);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      return to_e4m3x4(f.x * down, f.y * down, g.x * down, g.y * down);
    };
    for (int tok = part * at_once + slot; tok < first; tok += share * at_once) {
      uint4* at = reinterpret_cast<uint4*>(dst + tok * dst_stride + 16 * u);
      const uint4 c = *at;
      *at = make_uint4(divided(c.x), divided(c.y), divided(c.z), divided(c.w));
    }
  }
}

template <Turn TURN, bool AXES>
__global__ void __launch_bounds__(kThreads, 4)
    fill_kernel(const __grid_constant__ RopeTable rope, const FillParams p, const RopeAppendParams q,
                int fill_blocks) {
  const int block = blockIdx.x;
  if (block < fill_blocks) {
    fill_block<TURN, AXES>(rope, p, block);
  } else if constexpr (TURN != kTurnNone) {
    const RopeScale one{1.f, 1.f, 1.f};  // (no cache rows here)
    rope_append_block<false, layout_of(TURN), AXES>(rope, q, one, one, block - fill_blocks);
  }
}

template <Turn TURN, bool AXES = false>
cudaError_t launch(const RopeTable& rope, const FillParams& p, const RopeAppendParams& q, int smem,
                   cudaStream_t stream) {
  const int groups = (p.num_kv_heads + p.heads_per_cta - 1) / p.heads_per_cta;
  const int64_t fill_blocks = int64_t{2} * p.num_tiles * groups;
  const int64_t blocks = fill_blocks + (TURN == kTurnNone ? 0 : int64_t{kParts} * q.num_tiles);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_once(fill_kernel<TURN, AXES>, kMostSmem, smem_set);
  if (e != cudaSuccess) return e;
  fill_kernel<TURN, AXES><<<static_cast<unsigned>(blocks), kThreads, smem, stream>>>(
      rope, p, q, static_cast<int>(fill_blocks));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fill(const RopeTable* rope, FillParams p, RopeAppendParams q, int sms,
                        cudaStream_t stream) {
  if (p.num_tiles <= 0) return cudaSuccess;
  if (p.tiles == nullptr || p.head_dim % 32 != 0 || p.head_dim > 256) return cudaErrorInvalidValue;
  // A head to a warp, but for heads that leave warps without one, and for so few
  // CTAs that SMs go without: then a head's tokens are shared out, in fewer rounds.
  const int per_warp = warp_tokens(p.head_dim);
  int share = p.num_kv_heads == 1 ? 4 : (p.num_kv_heads == 2 ? 2 : 1);
  auto ctas = [&]() { return int64_t{2} * p.num_tiles * ((p.num_kv_heads * share + kWarps - 1) / kWarps); };
  while (share < kWarps && share * per_warp < p.max_rows && ctas() < 2 * sms) share *= 2;
  p.warps_per_head = share;
  p.heads_per_cta = kWarps / share < p.num_kv_heads ? kWarps / share : p.num_kv_heads;
  if (rope == nullptr) return launch<kTurnNone>(RopeTable{}, p, q, 0, stream);
  if (p.rotary_dim > 2 * kMaxPairs || p.rotary_dim > p.head_dim) return cudaErrorInvalidValue;
  const int tokens = per_warp * share < p.max_rows ? per_warp * share : p.max_rows;
  const int smem = tokens * turn_row(p.rotary_dim / 2) * static_cast<int>(sizeof(float2));
  if (smem > kMostSmem) return cudaErrorInvalidValue;
  q.num_kv_heads = 0;
  const bool axes = p.positions != nullptr && p.axes > 1;
  if (p.interleaved)
    return axes ? launch<kTurnInterleaved, true>(*rope, p, q, smem, stream)
                : launch<kTurnInterleaved>(*rope, p, q, smem, stream);
  if (p.rotary_dim % 16 == 0)
    return axes ? launch<kTurnHalf, true>(*rope, p, q, smem, stream)
                : launch<kTurnHalf>(*rope, p, q, smem, stream);
  return axes ? launch<kTurnHalfOdd, true>(*rope, p, q, smem, stream)
              : launch<kTurnHalfOdd>(*rope, p, q, smem, stream);
}

}  // namespace ua
