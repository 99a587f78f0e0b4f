// Staging kernel for prefill over an fp8 (e4m3) cache: widens the keys and
// values the prefill tiles will read from the paged e4m3 cache into a bf16
// staging cache of 128-slot pages, so that the tcgen05 prefill kernel (bf16
// operands) runs on it unchanged.
//
// The widening is exact and scale-free: an e4m3 code has 4 significant bits
// and an exponent within [-9, 8], so its value is a bf16 value; k_scale is
// folded into the score scale and v_scale into the output scale of the
// prefill launch, as for the oracle's dequantised values (code * scale).
// Conversion chain: e4m3x2 -> f16x2 (hardware, exact) -> f32 -> bf16x2
// (exact: no rounding happens for such values). NaN codes stay NaN.
//
// One to sixteen CTAs per staging page (the plan's stage tiles): 8 warps, one key
// row (all KV heads, contiguous in both caches) per warp at a time, 16-byte loads
// (four in flight per lane and cache) before the stores; source pages
// through the block table; rows past the sequence's length are not written
// (the prefill kernel masks those keys and zeroes those value rows); keys that no
// query sees (between the sinks and the first window) are staged as zeros, their
// pages not looked up.
// A cache with block scales is staged as code * scale, rounded to bf16 (exact for
// powers of two), with a scale of each row's page and head.
// HBM-bound: per staged key Hkv * d bytes read per cache, twice that written.
#include <cstdint>
#include <cuda_fp16.h>

#include "planner.h"
#include "ua_device.cuh"
#include "ua_kernels.h"

namespace ua {

namespace {

constexpr int kStageWarps = 8;

// f16x2 -> bf16x2 (exact for widened e4m3 values), element order kept.
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h2) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  uint32_t b2;
  // the first source operand lands in the upper half
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b2) : "f"(f.y), "f"(f.x));
  return b2;
}

template <bool SCALED>
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h2, float scale) {
  if constexpr (!SCALED) return f16x2_to_bf16x2(h2);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  return pack2<false>(f.x * scale, f.y * scale);
}

// Sixteen codes (16 bytes, lowest first) -> sixteen bf16 values (2 x 16 bytes).
template <bool SCALED>
__device__ __forceinline__ void widen16(uint4 c, float scale, uint4& lo, uint4& hi) {
  uint32_t h[8];
  e4m3x4_to_f16x2x2(c.x, h[0], h[1]);
  e4m3x4_to_f16x2x2(c.y, h[2], h[3]);
  e4m3x4_to_f16x2x2(c.z, h[4], h[5]);
  e4m3x4_to_f16x2x2(c.w, h[6], h[7]);
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = f16x2_to_bf16x2<SCALED>(h[i], scale);
  lo = make_uint4(b[0], b[1], b[2], b[3]);
  hi = make_uint4(b[4], b[5], b[6], b[7]);
}

constexpr int kUnroll = 4;  // 16-byte loads per lane in flight per cache

// GAPS: a tile may hold keys that no query sees (5 chunks of 300 to 1100 tokens over 100
// to 2500, where there are none: 2 us of 148 for looking).
template <bool SCALED, bool GAPS>
__global__ void __launch_bounds__(kStageWarps * 32) stage_kernel(const StageParams p, int parts) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const ua_tile tile = p.tiles[blockIdx.x / parts];
  const int first = tile.kv_lo + blockIdx.x % parts * (kStagePage / parts);
  const int last = min(tile.kv_hi, first + kStagePage / parts);
  const int chunks = p.row_elems / 16;  // 16 codes per load
  const int32_t* table = p.block_tables + static_cast<int64_t>(tile.seq) * p.max_blocks_per_seq;
  for (int t = first + w; t < last; t += kStageWarps) {
    if (t / p.block_size >= p.max_blocks_per_seq) break;
    if (GAPS && t >= tile.slot && t < tile.group) {  // seen by no query
      const int64_t row = (static_cast<int64_t>(tile.row0) * kStagePage + (t - tile.kv_lo)) * 2 * chunks;
      for (int c = lane; c < 2 * chunks; c += 32) {
        reinterpret_cast<uint4*>(p.k_dst)[row + c] = make_uint4(0u, 0u, 0u, 0u);
        reinterpret_cast<uint4*>(p.v_dst)[row + c] = make_uint4(0u, 0u, 0u, 0u);
      }
      continue;
    }
    const int32_t blk = table[t / p.block_size];
    if (blk < 0 || static_cast<int64_t>(blk) >= p.num_blocks) {
      if (lane == 0) record_error(p.err, UA_ERR_BOUNDS);
      continue;
    }
    const int64_t src_row = static_cast<int64_t>(blk) * p.block_size + t % p.block_size;
    const int64_t dst_row = static_cast<int64_t>(tile.row0) * kStagePage + (t - tile.kv_lo);
    const uint4* ks = reinterpret_cast<const uint4*>(p.k_src) + src_row * chunks;
    const uint4* vs = reinterpret_cast<const uint4*>(p.v_src) + src_row * chunks;
    uint4* kd = reinterpret_cast<uint4*>(p.k_dst) + dst_row * 2 * chunks;
    uint4* vd = reinterpret_cast<uint4*>(p.v_dst) + dst_row * 2 * chunks;
    for (int c0 = 0; c0 < chunks; c0 += 32 * kUnroll) {
      uint4 kc[kUnroll], vc[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int c = c0 + u * 32 + lane;
        if (c < chunks) {
          kc[u] = ld_stream_v4(ks + c);
          vc[u] = ld_stream_v4(vs + c);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int c = c0 + u * 32 + lane;
        if (c >= chunks) continue;
        float k_scale = 1.f, v_scale = 1.f;
        if constexpr (SCALED) {
          const int64_t at = static_cast<int64_t>(blk) * p.num_kv_heads + c / p.head_chunks;
          k_scale = usable_scale(__ldg(p.k_scales + at));
          v_scale = usable_scale(__ldg(p.v_scales + at));
        }
        uint4 lo, hi;
        widen16<SCALED>(kc[u], k_scale, lo, hi);
        kd[2 * c] = lo;
        kd[2 * c + 1] = hi;
        widen16<SCALED>(vc[u], v_scale, lo, hi);
        vd[2 * c] = lo;
        vd[2 * c + 1] = hi;
      }
    }
  }
}

}  // namespace

cudaError_t launch_stage(const StageParams& p, int sms, cudaStream_t stream) {
  if (p.num_tiles <= 0) return cudaSuccess;
  if (p.row_elems % 16 != 0 || p.tiles == nullptr) return cudaErrorInvalidValue;
  static_assert(kStagePage == 16 * kStageWarps, "a row per warp with sixteen CTAs to a page");
  // A warp's 16 rows of a page are a chain of table lookups, loads and stores;
  // eight CTAs to a page leave it two, sixteen one. Measured with one / eight /
  // sixteen: 8 heads of 128, 8 pages 20.6 / 8.0 / 6.8 us, 81 pages 27.3 / 17.9 /
  // 17.8, 649 pages 132.9 / 90.2 / 96.0; 32 heads, 16 pages 71 / 17 / 16, 64
  // pages 66 / 50 / 45, 192 pages 157 / 124 / 119. Only with wide rows (several
  // load rounds each) and pages for most of the SMs, in one wave, is one CTA to a
  // page the faster, with one / sixteen: 32 heads, 102 pages 70.5 / 66.7, 108 pages
  // 71.5 / 71.0, 116 pages 73.1 / 78.6, 152 pages 81 / 98, 156 pages 144 / 99; 24
  // heads, 108 pages 59.2 / 54.2, 116 pages 59.4 / 59.1, 128 pages 61.9 / 62.4.
  const bool wide_rows = p.row_elems / 16 > 32 * kUnroll;
  const bool fills = 4 * p.num_tiles > 3 * sms && p.num_tiles <= sms;
  const int parts = !wide_rows ? 8 : (fills ? 1 : 16);
  auto* const kernel = p.k_scales ? (p.gaps ? stage_kernel<true, true> : stage_kernel<true, false>)
                                  : (p.gaps ? stage_kernel<false, true> : stage_kernel<false, false>);
  kernel<<<p.num_tiles * parts, kStageWarps * 32, 0, stream>>>(p, parts);
  return cudaGetLastError();
}

}  // namespace ua
