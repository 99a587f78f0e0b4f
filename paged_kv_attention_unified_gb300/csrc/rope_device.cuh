// Device parts of the rotary append (rope.cu) that the append into a cache with
// block scales (fill.cu) shares: angles, rotations, quotients, and the append of
// one CTA's tokens.
#pragma once

#include <cstdint>

#include "planner.h"
#include "sm100.cuh"
#include "ua_device.cuh"
#include "ua_kernels.h"

namespace ua {
namespace rope_device {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kParts = kAppendTokens / kWarps;  // CTAs per append tile
constexpr int kMaxPairs = 128;  // rotary_dim / 2 at head_dim 256
static_assert(kAppendTokens == 8, "a tile's eight warps share its tokens by shifts");

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

// 16 bytes of a row that may be rewritten in place (no read-only path).
__device__ __forceinline__ uint4 ld_row(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// A frequency of the launch's parameter block through a generic address. As a
// constant-bank access the lanes' different indexes are taken one by one.
__device__ __forceinline__ float ld_param(const float* p) {
  float r;
  asm volatile("ld.f32 %0, [%1];" : "=f"(r) : "l"(p));
  return r;
}

__device__ __forceinline__ int ld_param(const uint8_t* p) {
  uint32_t r;
  asm volatile("ld.u8 %0, [%1];" : "=r"(r) : "l"(p));
  return static_cast<int>(r);
}

// (cos, sin) of pair i of a token, with the amplitude: at its position on the
// pair's axis (AXES; positions: axis a of row j at a * stride + j), on one axis, or
// at `slot_pos` without positions. (An instance for one axis: chunks of 3850 tokens
// 13.5 us, 14.7 with the axis looked up.)
template <bool AXES>
__device__ __forceinline__ float2 pair_turn(const RopeTable& rope, const int32_t* positions,
                                            int64_t stride, int row, int slot_pos, int i) {
  int32_t at;
  if constexpr (AXES) at = positions[ld_param(rope.axis + i) * stride + row];
  else at = positions ? positions[row] : slot_pos;
  const float2 cs = rotation(at, ld_param(rope.hi + i), ld_param(rope.lo + i));
  return make_float2(cs.x * rope.amplitude, cs.y * rope.amplitude);
}

// The same for one pair at many tokens.
template <bool AXES>
struct PairFrequency {
  float hi, lo, amplitude;
  const int32_t* row;  // the pair's axis of the positions, or null
  __device__ __forceinline__ PairFrequency(const RopeTable& rope, const int32_t* positions,
                                           int64_t stride, int i)
      : hi(ld_param(rope.hi + i)), lo(ld_param(rope.lo + i)), amplitude(rope.amplitude),
        row(positions) {
    if constexpr (AXES) row += ld_param(rope.axis + i) * stride;
  }
  __device__ __forceinline__ float2 at(int token, int slot_pos) const {
    const float2 cs = rotation(row ? row[token] : slot_pos, hi, lo);
    return make_float2(cs.x * amplitude, cs.y * amplitude);
  }
};

// Eight values of a chunk as binary32, and back.
__device__ __forceinline__ void widen8(uint4 w, float (&x)[8]) {
  x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
  return make_uint4(pack2<false>(x[0], x[1]), pack2<false>(x[2], x[3]), pack2<false>(x[4], x[5]),
                    pack2<false>(x[6], x[7]));
}
// An e4m3 cache's scale = mant / shift, |mant| in [1, 2), shift a power of two.
struct RopeScale {
  float shift, mant, inv;  // inv = 1 / mant
};

// x / scale of two values for rounding to e4m3: the product with the rounded reciprocal, off
// by two ulp at most, corrected by its remainder (as in P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990), which leaves half an ulp of binary32
// and 2^-20 ulp more. Clamped at 1024, beyond which e4m3 saturates, so that the
// remainder of an overflow stays a number; a zero keeps its sign. A true
// division per element took prompts of 4 x 4096 tokens with an e4m3 cache 183
// us, this 129 us (138 without the paired arithmetic).
__device__ __forceinline__ void quotients(float x0, float x1, const RopeScale& s, float& q0,
                                          float& q1) {
  using namespace sm100;
  const uint64_t inv = f2_pack(s.inv, s.inv);
  const uint64_t y = f2_mul(f2_pack(x0, x1), f2_pack(s.shift, s.shift));
  float a0, a1;
  f2_unpack(f2_mul(y, inv), a0, a1);
  const uint64_t q = f2_pack(fminf(fmaxf(a0, -1024.f), 1024.f), fminf(fmaxf(a1, -1024.f), 1024.f));
  f2_unpack(f2_fma(f2_fma(q, f2_pack(-s.mant, -s.mant), y), inv, q), q0, q1);
  q0 = copysignf(q0, a0);
  q1 = copysignf(q1, a1);
}
__device__ __forceinline__ uint2 quantize8(const float (&x)[8], const RopeScale& s) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) quotients(x[i], x[i + 1], s, q[i], q[i + 1]);
  return make_uint2(to_e4m3x4(q[0], q[1], q[2], q[3]), to_e4m3x4(q[4], q[5], q[6], q[7]));
}

// How a lane's two chunks hold its pairs.
enum Layout {
  kHalf,         // a in the first chunk, b in the second (rotary_dim a multiple of 16)
  kInterleaved,  // neighbours
  kHalfOdd,      // 16 consecutive elements, partners through shared memory
};

// Words between the 32-byte units of a warp's copy: odd, so that lanes reading
// the same place of their units hit different banks.
constexpr int kUnitWords = 9;

// One CTA of the rotary append, the block-th: the body of rope_append_kernel
// (rope.cu). With num_kv_heads 0 it turns the queries alone. AXES: positions of
// several axes are given.
template <bool FP8, Layout LAYOUT, bool AXES>
__device__ __forceinline__ void rope_append_block(const RopeTable& rope, const RopeAppendParams& p,
                                                  const RopeScale& k_scale,
                                                  const RopeScale& v_scale, int block) {
  constexpr int kUnroll = LAYOUT == kHalfOdd ? 3 : 8;  // heads per lane with loads in flight
  constexpr int kTurns = LAYOUT == kHalfOdd ? 16 : 8;  // (cos, sin) a lane holds
  __shared__ float2 turn[kWarps][kMaxPairs];
  __shared__ uint32_t copy[LAYOUT == kHalfOdd ? kWarps * kUnroll * 32 * kUnitWords : 1];
  const ua_tile tile = p.tiles[block / kParts];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d = p.head_dim, pairs = p.rotary_dim / 2;
  const int units = d / 16;       // units of a head: 2 .. 16
  const int at_once = 32 / units;  // heads a warp holds
  const int slot = lane / units, u = lane - slot * units;
  // The tile's eight warps (of kParts CTAs): 8, 4, 2 or 1 to a token. The
  // tokens of this CTA are w0 .. w0 + tokens - 1 of the tile.
  const int log_share = tile.nrows <= 1 ? 3 : (tile.nrows <= 2 ? 2 : (tile.nrows <= 4 ? 1 : 0));
  const int tile_warp = block % kParts * kWarps + warp;
  const int w = tile_warp >> log_share, part = tile_warp & ((1 << log_share) - 1);
  const int w0 = (block % kParts * kWarps) >> log_share;
  const int tokens = min(max(kWarps >> log_share, 1), tile.nrows - w0);
  if (tokens <= 0) return;
  const bool has_token = w < tile.nrows;
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  const int64_t j = tile.row0 + (has_token ? w : 0);
  const int pos = tile.kv_lo + (has_token ? w : 0);

  const bool turns = LAYOUT == kInterleaved ? 8 * u < pairs : 16 * u < p.rotary_dim;
  const bool apart = LAYOUT == kHalf && turns;
  const int off0 = apart ? 8 * u : 16 * u;
  const int off1 = apart ? 8 * u + pairs : 16 * u + 8;

  const __nv_bfloat16* const q_row = static_cast<const __nv_bfloat16*>(p.q) + j * p.q_stride;
  const __nv_bfloat16* const k_row = static_cast<const __nv_bfloat16*>(p.k_new) + j * p.k_stride;
  const __nv_bfloat16* const v_row = static_cast<const __nv_bfloat16*>(p.v_new) + j * p.v_stride;
  const int first_k = p.num_q_heads, first_v = p.num_q_heads + p.num_kv_heads;
  const int stride = at_once << log_share;  // heads between a warp's steps

  uint4 c0[kUnroll], c1[kUnroll];
  auto mine = [&](int h) { return has_token && slot < at_once && h < heads; };
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = h0 + i * stride + slot;
      if (!mine(h)) continue;
      const bool is_v = h >= first_v;
      const __nv_bfloat16* src = h < first_k ? q_row + h * d
                                 : is_v      ? v_row + (h - first_v) * d
                                             : k_row + (h - first_k) * d;
      c0[i] = ld_row(src + (is_v ? 16 * u : off0));
      c1[i] = ld_row(src + (is_v ? 16 * u + 8 : off1));
    }
  };
  load(part * at_once);

  int32_t blk = -1;
  if (pos >= 0 && pos / p.block_size < p.max_blocks_per_seq)
    blk = p.block_tables[static_cast<int64_t>(tile.seq) * p.max_blocks_per_seq +
                         pos / p.block_size];
  const bool page_ok = blk >= 0 && static_cast<int64_t>(blk) < p.num_blocks;
  if (!page_ok && has_token && lane == 0 && part == 0) record_error(p.err, UA_ERR_BOUNDS);
  const int64_t cache_row =
      (static_cast<int64_t>(blk) * p.block_size + pos % p.block_size) * p.num_kv_heads;

  for (int x = threadIdx.x; x < tokens * pairs; x += kThreads) {
    const int t = x / pairs, i = x - t * pairs;
    turn[t][i] = pair_turn<AXES>(rope, p.positions, p.positions_stride, tile.row0 + w0 + t,
                                 tile.kv_lo + w0 + t, i);
  }
  __syncthreads();
  if (!has_token) return;
  // cos and sin of this lane's pairs; kHalfOdd: of its elements, the sine with
  // the sign its partner takes.
  float co[kTurns], si[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int e = 16 * u + i;
    const int pair = LAYOUT == kHalfOdd ? (e < pairs ? e : e - pairs) : 8 * u + i;
    const float2 cs = turn[w - w0][min(pair, pairs - 1)];
    co[i] = cs.x;
    si[i] = LAYOUT == kHalfOdd && e < pairs ? -cs.y : cs.y;
    if (LAYOUT == kHalfOdd && e >= p.rotary_dim) co[i] = 1.f, si[i] = -0.f;
  }
  // kHalfOdd: where the partners' words are in a copy, and how many of the
  // lane's words turn.
  uint32_t* const heads_copy = copy + warp * kUnroll * 32 * kUnitWords;
  const int turning = pairs - 8 * u, shift = (pairs & 1) * 16;
  int place[9];
  if constexpr (LAYOUT == kHalfOdd) {
#pragma unroll
    for (int i = 0; i < 9; ++i) {
      int word = 8 * u + pairs / 2 + i;
      if (word >= pairs) word -= pairs;
      if (word >= pairs || slot >= at_once) word = 0;  // not used
      place[i] = (slot >= at_once ? 0 : slot * units * kUnitWords) + word + word / 8;
    }
  }

  for (int h0 = part * at_once; h0 < heads;) {
    if constexpr (LAYOUT == kHalfOdd) {
      __syncwarp();  // the copies of the round before have been read
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        uint32_t* own = heads_copy + (i * 32 + lane) * kUnitWords;
        own[0] = c0[i].x, own[1] = c0[i].y, own[2] = c0[i].z, own[3] = c0[i].w;
        own[4] = c1[i].x, own[5] = c1[i].y, own[6] = c1[i].z, own[7] = c1[i].w;
      }
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int h = h0 + i * stride + slot;
      const bool is_v = h >= first_v;
      float x0[8], x1[8];
      widen8(c0[i], x0);
      widen8(c1[i], x1);
      if constexpr (LAYOUT == kHalfOdd) {
        if (!is_v && turns) {
          const uint32_t* heads_i = heads_copy + i * 32 * kUnitWords;
          uint32_t word = heads_i[place[0]];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t next = heads_i[place[k + 1]];
            const uint32_t b = k < turning ? __funnelshift_r(word, next, shift) : 0u;
            word = next;
            float& lo = k < 4 ? x0[2 * (k % 4)] : x1[2 * (k % 4)];
            float& hi = k < 4 ? x0[2 * (k % 4) + 1] : x1[2 * (k % 4) + 1];
            lo = fmaf(lo, co[2 * k], bf16_lo(b) * si[2 * k]);
            hi = fmaf(hi, co[2 * k + 1], bf16_hi(b) * si[2 * k + 1]);
          }
        }
      } else if (!is_v && turns) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if constexpr (LAYOUT == kHalf) {
            const float a = x0[k], b = x1[k];
            x0[k] = fmaf(a, co[k], -b * si[k]);
            x1[k] = fmaf(b, co[k], a * si[k]);
          } else {
            float& lo = k < 4 ? x0[2 * (k % 4)] : x1[2 * (k % 4)];
            float& hi = k < 4 ? x0[2 * (k % 4) + 1] : x1[2 * (k % 4) + 1];
            if (8 * u + k < pairs) {
              const float a = lo, b = hi;
              lo = fmaf(a, co[k], -b * si[k]);
              hi = fmaf(b, co[k], a * si[k]);
            }
          }
        }
      }
      if (!mine(h)) continue;
      const int o0 = is_v ? 16 * u : off0, o1 = is_v ? 16 * u + 8 : off1;
      if (h < first_k) {
        __nv_bfloat16* dst =
            static_cast<__nv_bfloat16*>(p.q_out) + (j * p.num_q_heads + h) * d;
        *reinterpret_cast<uint4*>(dst + o0) = narrow8(x0);
        *reinterpret_cast<uint4*>(dst + o1) = narrow8(x1);
      } else if (page_ok) {
        const int64_t at = (cache_row + h - (is_v ? first_v : first_k)) * d;
        void* cache = is_v ? p.v_cache : p.k_cache;
        if constexpr (FP8) {
          const RopeScale scale = is_v ? v_scale : k_scale;
          uint8_t* dst = static_cast<uint8_t*>(cache) + at;
          const uint2 lo = quantize8(x0, scale), hi = quantize8(x1, scale);
          if (o1 == o0 + 8) {
            *reinterpret_cast<uint4*>(dst + o0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
          } else {
            *reinterpret_cast<uint2*>(dst + o0) = lo;
            *reinterpret_cast<uint2*>(dst + o1) = hi;
          }
        } else {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(cache) + at;
          *reinterpret_cast<uint4*>(dst + o0) = narrow8(x0);
          *reinterpret_cast<uint4*>(dst + o1) = narrow8(x1);
        }
      }
    }
    h0 += kUnroll * stride;
    if (h0 < heads) load(h0);
  }
}

}  // namespace rope_device
}  // namespace ua
