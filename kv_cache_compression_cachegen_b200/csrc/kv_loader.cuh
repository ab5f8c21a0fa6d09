// kv_loader.cuh -- the warps that bring K and V from the pages to shared memory.
//
// Tiles of K and V take turns in a ring of stages.  A tile is [64-channel
// block][key][64 channels] in the 128-byte swizzle (16-byte chunk index xor key
// mod 8), as the tensor cores and ldmatrix both take it.  Two warps bring half
// of a tile's keys each.  A weight of zero does not hide a value that is not
// finite, so keys that no row of the item sees need care:
//   load_kv     brings zeros for them: by TMA where all of the half can be seen
//               and lies in runs of eight rows or more, else row by row
//               (cp.async; a page may end anywhere in a tile)
//   load_boxes  brings whole TMA boxes, for a reader that hides the rest by
//               itself; what no row sees is there or is left from before
#pragma once

#include "attend.cuh"
#include "tcgen05.cuh"

namespace cg {

constexpr int kLoadWarps = 2;

// The ring, as both sides see it.
struct Ring {
  uint32_t smem;         // stage 0
  uint32_t full, empty;  // barriers, 8 bytes a stage
  // keys of a unit whose page is not in the pool, a bit each, by unit number mod 4
  uint32_t (*no_page)[4];
  volatile int* dead;
};

// DC: 64-channel blocks of a head.  wk: 0 or 1, which of the two warps.  False
// where a wait ran out.
template <int DC, int kTile, int kKeys, int kStages>
__device__ __forceinline__ bool load_kv(const AttnParams& p, Walk<kTile, kKeys>& w,
                                        const Ring& ring, const CUtensorMap* k_map,
                                        const CUtensorMap* v_map, int box, int wk) {
  constexpr int kBlock = kKeys * 128, kStage = DC * kBlock;
  constexpr int kMine = kKeys / kLoadWarps;  // rows of a tile that are this warp's
  constexpr int kOwn = kMine / 32;           // of these, a lane's
  constexpr int kLanes = 8 * DC;             // lanes of a row (16 bytes each)
  constexpr int kPer = 32 / kLanes;          // rows a warp copies at a time
  // Halves that came by cp.async are passed on kLag tiles behind the one that is
  // being asked for, when they have landed, so that more are on their way.
  constexpr int kLag = kStages > 3 ? 2 : 1;
  const int lane = threadIdx.x & 31;
  const int c = lane % kLanes, sub = lane / kLanes, D = p.dim;
  const int64_t step = int64_t(p.kv_heads) * D;
  const int boxes = box > 0 ? kMine / box * DC : 0;
  uint32_t stage = 0, phase = 1, tiles = 0, unit_count = 0;
  uint32_t copied = 0;  // the latest tiles, a bit each: this warp's half came by cp.async
  bool ok = true;
  const auto pass_on = [&](uint32_t behind) {
    if ((copied >> (behind - 1)) & 1) {
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.full + 8 * ((stage + kStages - behind) % kStages));
    }
  };
  while (ok && w.next(p)) {
    const Item& it = w.it;
    const bool prefix = it.request < 0;
    const int32_t* table = prefix ? p.prefix_table : p.tables + int64_t(it.request) * p.max_pages;
    const int64_t col = int64_t(w.head) * D + 8 * c;
    // Lane i has the warp's keys i, i + 32, ... of the unit; their pages are
    // looked up a unit ahead.  -2: no row of the item sees the key.
    int key_ahead[kOwn], page_ahead[kOwn], mine[kOwn];
    const auto look_up = [&](int u) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        page_ahead[i] = -2;
        key_ahead[i] = 0;
        if (u < w.last) {
          const int key = unit_key<kKeys>(it.span, u) + kMine * wk + 32 * i + lane;
          if (key < it.span.hi && (key >= it.span.lo || key < it.span.sink_end))
            page_ahead[i] = max(-1, __ldg(table + div_of(key, p.page_div)));
          key_ahead[i] = key;
        }
      }
    };
    look_up(w.first);
    for (int u = w.first; ok && u < w.last; ++u, ++unit_count) {
      uint32_t holes[kOwn];
      bool there = box > 0;  // every key of the warp's half can be read
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const bool hole = page_ahead[i] == -1 || page_ahead[i] >= p.num_pages;
        mine[i] = -1;
        if (page_ahead[i] >= 0 && !hole)
          mine[i] = page_ahead[i] * p.page_tokens +
                    (key_ahead[i] - div_of(key_ahead[i], p.page_div) * p.page_tokens);
        holes[i] = __ballot_sync(~0u, hole);
        there = there && mine[i] >= 0;
        if (holes[i] != 0 && lane == 0) report(p.status, CG_ERR_MISMATCH);
      }
      there = __all_sync(~0u, there);
      look_up(u + 1);
      for (int kv = 0; kv < 2; ++kv) {
        if (!(ok = mbar_wait(ring.empty + 8 * stage, phase, ring.dead))) break;
        if (kv == 0 && lane == 0) {
#pragma unroll
          for (int i = 0; i < kOwn; ++i) ring.no_page[unit_count & 3][wk * kOwn + i] = holes[i];
        }
        __syncwarp();
        const uint32_t tile = ring.smem + stage * kStage;
        if (there) {
          // whole boxes of keys that follow one another in a page
          if (lane == 0) mbar_expect(ring.full + 8 * stage, kMine * 128 * DC);
          __syncwarp();
          for (int i0 = 0; i0 < boxes; i0 += 32) {
            const int i = i0 + lane, b = i % DC, key = i / DC * box;
            int row = __shfl_sync(~0u, mine[0], key & 31);
            if constexpr (kOwn == 2) {
              const int upper = __shfl_sync(~0u, mine[kOwn - 1], key & 31);
              if (key >= 32) row = upper;
            }
            if (i < boxes)
              tma_load3(tile + b * kBlock + (kMine * wk + key) * 128, kv ? v_map : k_map, 64 * b,
                        w.head, row, ring.full + 8 * stage);
          }
        } else {
          const uint16_t* pool = (kv ? p.v_pool : p.k_pool) + col;
          const uint32_t dst = tile + (c >> 3) * kBlock;
          // the rows first, then the copies, so that eight are asked for at once
#pragma unroll
          for (int o = 0; o < kOwn; ++o)
            for (int i0 = 0; i0 < 32; i0 += 8 * kPer) {
              int src[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                src[i] = __shfl_sync(~0u, mine[o], (i0 + i * kPer + sub) & 31);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int key = kMine * wk + 32 * o + i0 + i * kPer + sub;
                if (8 * c < D && i0 + i * kPer < 32)
                  cp_async16(dst + key * 128 + (((c & 7) ^ (key & 7)) << 4),
                             src[i] >= 0 ? pool + src[i] * step : pool, src[i] >= 0 ? 16 : 0);
              }
            }
        }
        cp_async_commit();
        if (tiles >= kLag) {
          cp_async_wait<kLag>();
          pass_on(kLag);
        }
        copied = (copied << 1) | (there ? 0u : 1u);
        ++tiles;
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
    }
  }
  if (kLag > 1 && tiles > 1) {
    cp_async_wait<1>();
    pass_on(2);
  }
  cp_async_wait<0>();
  if (tiles > 0) pass_on(1);
  return ok;
}

// The same by boxes alone (box > 0), without zeros.
template <int DC, int kTile, int kKeys, int kStages>
__device__ __forceinline__ bool load_boxes(const AttnParams& p, Walk<kTile, kKeys>& w,
                                           const Ring& ring, const CUtensorMap* k_map,
                                           const CUtensorMap* v_map, int box, int wk) {
  constexpr int kBlock = kKeys * 128, kStage = DC * kBlock;
  constexpr int kMine = kKeys / kLoadWarps;
  static_assert(kMine / 8 * DC <= 32 && kMine <= 64, "a lane has at most one box");
  const int lane = threadIdx.x & 31;
  const int b = lane % DC, own = lane / DC * box;  // the lane's box: channels, first key
  uint32_t stage = 0, phase = 1, unit_count = 0;
  // One unit: where the lane's box lies; looked up while the unit before is issued.
  struct Ahead {
    int page, row_in_page, head;  // page -2: no row of the item sees the box
    bool unit;
  } next;
  const int32_t* table = nullptr;
  int u = 0;
  w.last = 0;
  const auto look_up = [&]() {
    next.unit = true;
    while (u >= w.last) {
      if (!w.next(p)) {
        next.unit = false;
        return;
      }
      u = w.first;
      table = w.it.request < 0 ? p.prefix_table : p.tables + int64_t(w.it.request) * p.max_pages;
    }
    const int key = unit_key<kKeys>(w.it.span, u) + kMine * wk + own;
    next.page = -2;
    next.head = w.head;
    if (own < kMine && key < w.it.span.hi &&
        (key + box > w.it.span.lo || key < w.it.span.sink_end)) {
      const int col = div_of(key, p.page_div);
      next.row_in_page = key - col * p.page_tokens;
      next.page = max(-1, __ldg(table + col));
    }
    ++u;
  };
  look_up();
  for (; next.unit; ++unit_count) {
    const Ahead now = next;
    look_up();
    const bool hole = now.page == -1 || now.page >= p.num_pages;
    const bool mine = now.page >= 0 && !hole;
    const int row = mine ? now.page * p.page_tokens + now.row_in_page : 0;
    const uint32_t bytes = __popc(__ballot_sync(~0u, mine)) * box * 128;
    uint32_t holes[2] = {0, 0};
    if (__any_sync(~0u, hole)) {
      const uint64_t bits = hole ? (box < 64 ? (1ull << box) - 1 : ~0ull) << own : 0ull;
      holes[0] = __reduce_or_sync(~0u, uint32_t(bits));
      holes[1] = __reduce_or_sync(~0u, uint32_t(bits >> 32));
      if (lane == 0) report(p.status, CG_ERR_MISMATCH);
    }
    for (int kv = 0; kv < 2; ++kv) {
      if (!mbar_wait(ring.empty + 8 * stage, phase, ring.dead)) return false;
      if (lane == 0) {
        if (kv == 0) {
#pragma unroll
          for (int i = 0; i < kMine / 32; ++i)
            ring.no_page[unit_count & 3][wk * (kMine / 32) + i] = holes[i];
        }
        mbar_expect(ring.full + 8 * stage, bytes);
      }
      __syncwarp();
      if (mine)
        tma_load3(ring.smem + stage * kStage + b * kBlock + (kMine * wk + own) * 128,
                  kv ? v_map : k_map, 64 * b, now.head, row, ring.full + 8 * stage);
      if (++stage == kStages) stage = 0, phase ^= 1;
    }
  }
  return true;
}

}  // namespace cg
