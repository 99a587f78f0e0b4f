// The pages of a prefill kernel's key tile, for its TMA producers.
#pragma once

#include "planner.h"
#include "sm100.cuh"
#include "ua_device.cuh"
#include "ua_kernels.h"

namespace ua {

// One lane's copy of a tile of KEYS keys: panel lane % PANELS of box lane / PANELS,
// a box being p.rows_per_box keys of one page. The lanes of the producer warp look
// their pages up together: one by one, between the copies of a single thread, each
// cost a memory latency, which bounded the kernels over small pages. Four prompts
// of 4096 tokens, 32 heads and 8 KV heads in 16-slot pages, one thread / all lanes:
// head_dim 64 624 / 400 us, 128 804 / 476 (475 in 128-slot pages), 256 2184 / 1025,
// 128 with a window of 1024 405 / 281. A tile ahead of the copies the same lookups
// cost where they save nothing: 32 KV heads in 128-slot pages 515 / 497 us, ahead
// 589 (the CTAs of a head drift apart and find less of its keys in L2).
// SHAPED: there may be sinks. (The instances without them do no arithmetic of the gap,
// here and in the kernels: it cost head_dim 192 2 %, 911 / 927 us for 4 x 4096 tokens
// and 32 KV heads in 128-slot pages, and 256 1.4 %, 1029 / 1041.)
template <int KEYS, int PANELS, bool SHAPED>
struct TilePages {
  static_assert(KEYS / 16 * PANELS <= 32, "a copy to a lane");
  int32_t id;   // the page, as the block table has it
  bool wanted;  // the box holds keys of the range
  int slot;     // its first slot in the page

  __device__ __forceinline__ static int box(int lane) { return lane / PANELS; }

  __device__ __forceinline__ void fetch(const PrefillParams& p, int lane, int seq, int ctx,
                                        int base, int kv_hi) {
    const int key = base + box(lane) * p.rows_per_box;
    wanted = box(lane) * p.rows_per_box < KEYS && key < kv_hi;
    if constexpr (SHAPED) {
      // Boxes whose keys lie between the sinks and the first query's window are not
      // looked up: a session may have given such pages back.
      const KeyGap unseen = key_gap(p.shape.sinks, p.window, ctx, 1);
      wanted = wanted && !(key >= unseen.lo && key + p.rows_per_box <= unseen.hi);
    }
    id = -1;
    slot = 0;
    if (wanted) {
      const int page = key / p.block_size;
      slot = key - page * p.block_size;
      id = p.block_tables[static_cast<int64_t>(seq) * p.max_blocks_per_seq + page];
    }
  }

  // The lane's copy of the fetched tile. Every page id is checked; a missing or
  // out-of-range page is loaded from an out-of-range block coordinate, which TMA
  // fills with zeros.
  __device__ __forceinline__ void copy(const CUtensorMap* map, const PrefillParams& p, int lane,
                                       int kv_head, uint8_t* dst, int panel_bytes, int panel_dims,
                                       uint32_t full) const {
    if (box(lane) * p.rows_per_box >= KEYS) return;
    int32_t blk = static_cast<int32_t>(p.num_blocks);
    if (wanted) {
      if (id >= 0 && static_cast<int64_t>(id) < p.num_blocks) blk = id;
      else record_error(p.err, UA_ERR_BOUNDS);
    }
    const int pn = lane % PANELS;
    sm100::tma_load_4d(dst + pn * panel_bytes + box(lane) * p.rows_per_box * 128, map, full,
                       pn * panel_dims, kv_head, slot, blk);
  }
};

}  // namespace ua
