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
constexpr uint32_t kNoted = 8;

// The ring, as both sides see it.
struct Ring {
  uint32_t smem;         // stage 0
  uint32_t full, empty;  // barriers, 8 bytes a stage
  // Keys of a unit whose page is not in the pool, a bit each, by unit number mod
  // kNoted: a unit's note is written over when the stage of the unit kNoted behind
  // it is free, which at up to twelve stages is after the unit was read.
  uint32_t (*no_page)[4];
  volatile int* dead;  // and the beat behind it: mbar_wait's state
};

// DC: 64-channel blocks of a head.  wk: 0 or 1, which of the two warps.  False
// where a wait ran out.
template <int DC, int kTile, int kKeys, int kStages>
__device__ __forceinline__ bool load_kv(const AttnParams& p, Walk<kTile, kKeys>& w,
                                        const Ring& ring, const CUtensorMap* k_map,
                                        const CUtensorMap* v_map, int box, int wk) {
  static_assert(kStages / 2 + 1 <= int(kNoted), "");
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
  uint32_t stage = 0, phase = 1, unit_count = 0;
  uint32_t copied = 0;  // the latest tiles, a bit each: this warp's half came by cp.async
  bool ok = true;
  const auto pass_on = [&](int behind) {
    if ((copied >> (behind - 1)) & 1) {
      if (behind == kLag) cp_async_wait<kLag>();
      else cp_async_wait<0>();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.full + 8 * ((stage + kStages - behind) % kStages));
    }
  };
  while (ok && w.next(p)) {
    const Item& it = w.it;
    const bool prefix = it.request < 0;
    const int32_t* table = prefix ? p.prefix_table : p.tables + int64_t(it.request) * p.max_pages;
    const int head = __shfl_sync(~0u, w.head, 0);
    const int64_t col = int64_t(head) * D + 8 * c;
    // Lane i has the warp's keys i, i + 32, ... of the unit; their pages are
    // looked up a unit ahead.  Key -1: no row of the item sees it.
    int key_ahead[kOwn], page_ahead[kOwn], mine[kOwn];
    const auto look_up = [&](int u) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        key_ahead[i] = -1;
        if (u < w.last) {
          const int key = unit_key<kKeys>(it.span, u) + kMine * wk + 32 * i + lane;
          if (key < it.span.hi && (key >= it.span.lo || key < it.span.sink_end)) {
            key_ahead[i] = key;
            page_ahead[i] = __ldg(table + div_of(key, p.page_div));
          }
        }
      }
    };
    look_up(w.first);
    for (int u = w.first; ok && u < w.last; ++u, ++unit_count) {
      uint32_t holes[kOwn];
      bool there = box > 0;  // every key of the warp's half can be read
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const bool sees_it = key_ahead[i] >= 0;
        const bool hole = sees_it && (page_ahead[i] < 0 || page_ahead[i] >= p.num_pages);
        mine[i] = -1;
        if (sees_it && !hole)
          mine[i] = page_ahead[i] * p.page_tokens +
                    (key_ahead[i] - div_of(key_ahead[i], p.page_div) * p.page_tokens);
        holes[i] = __ballot_sync(~0u, hole);
        there = there && mine[i] >= 0;
        if (holes[i] != 0 && lane == 0) report(p.status, CG_ERR_MISMATCH);
      }
      there = __all_sync(~0u, there);
      int rows[kMine / 8];  // of the boxes: before the copies, which keep their order
#pragma unroll
      for (int i = 0; i < kMine / 8; ++i) {
        const int key = i * box;
        rows[i] = __shfl_sync(~0u, kOwn == 2 && key >= 32 ? mine[kOwn - 1] : mine[0], key & 31);
      }
      look_up(u + 1);
      for (int kv = 0; kv < 2; ++kv) {
        // the same in all lanes, as the compiler can see: addresses stay uniform
        ok = __all_sync(~0u, mbar_wait(ring.empty + 8 * stage, phase, ring.dead));
        if (!ok) break;
        if (kv == 0 && lane < kOwn)
          ring.no_page[unit_count % kNoted][wk * kOwn + lane] = lane == 0 ? holes[0] : holes[kOwn - 1];
        const uint32_t tile = ring.smem + stage * kStage;
        if (there) {
          // whole boxes of keys that follow one another in a page
          __syncwarp();
          mbar_expect(ring.full + 8 * stage, kMine * 128 * DC);
#pragma unroll
          for (int i = 0; i < kMine / 8; ++i)
            if (i * box < kMine) {
#pragma unroll
              for (int b = 0; b < DC; ++b)
                tma_load3(tile + b * kBlock + (kMine * wk + i * box) * 128, kv ? v_map : k_map,
                          64 * b, head, rows[i], ring.full + 8 * stage);
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
        pass_on(kLag);
        copied = (copied << 1) | (there ? 0u : 1u);
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
    }
  }
  // the last ones: nothing follows them
  cp_async_wait<0>();
  if (kLag > 1) pass_on(2);
  pass_on(1);
  return ok;
}

// The same by boxes alone (box > 0), without zeros.
template <int DC, int kTile, int kKeys, int kStages>
__device__ __forceinline__ bool load_boxes(const AttnParams& p, Walk<kTile, kKeys>& w,
                                           const Ring& ring, const CUtensorMap* k_map,
                                           const CUtensorMap* v_map, int box, int wk) {
  static_assert(kStages / 2 + 1 <= int(kNoted), "");
  constexpr int kBlock = kKeys * 128, kStage = DC * kBlock;
  constexpr int kMine = kKeys / kLoadWarps;
  static_assert(kMine / 8 <= 32 && kMine <= 64, "a lane has at most one box's keys");
  const int lane = threadIdx.x & 31;
  const int own = lane * box;  // the lane's keys: its box's first
  uint32_t stage = 0, phase = 1, unit_count = 0;
  // One unit: where the lane's keys lie; looked up while the unit before comes.
  struct Ahead {
    int page, row_in_page, head;
    bool unit, seen;  // seen: some row of the item sees some of the keys
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
    next.head = w.head;
    next.seen = own < kMine && key < w.it.span.hi &&
                (key + box > w.it.span.lo || key < w.it.span.sink_end);
    if (next.seen) {
      const int col = div_of(key, p.page_div);
      next.row_in_page = key - col * p.page_tokens;
      next.page = __ldg(table + col);
    }
    ++u;
  };
  look_up();
  while (__all_sync(~0u, next.unit)) {
    const Ahead now = next;
    const bool hole = now.seen && (now.page < 0 || now.page >= p.num_pages);
    const bool mine = now.seen && !hole;
    const int row = now.page * p.page_tokens + now.row_in_page;
    const uint32_t there = __ballot_sync(~0u, mine);
    const int head = __shfl_sync(~0u, now.head, 0);
    uint32_t holes[2] = {0, 0};
    if (__any_sync(~0u, hole)) {
      const uint64_t bits = hole ? (box < 64 ? (1ull << box) - 1 : ~0ull) << own : 0ull;
      holes[0] = __reduce_or_sync(~0u, uint32_t(bits));
      holes[1] = __reduce_or_sync(~0u, uint32_t(bits >> 32));
      if (lane == 0) report(p.status, CG_ERR_MISMATCH);
    }
    for (int kv = 0; kv < 2; ++kv) {
      if (!__all_sync(~0u, mbar_wait(ring.empty + 8 * stage, phase, ring.dead))) return false;
      if (kv == 0 && lane < kMine / 32)
        ring.no_page[unit_count % kNoted][wk * (kMine / 32) + lane] = holes[lane & 1];
      __syncwarp();
      mbar_expect(ring.full + 8 * stage, __popc(there) * box * (128 * DC));
      const uint32_t dst = ring.smem + stage * kStage + kMine * wk * 128;
      // A lane asks for its own box.  (One lane asking for all in turn, as above,
      // leaves 128 single tokens behind a 4,096 window at 364 us, this at 338.)
      if (mine) {
#pragma unroll
        for (int b = 0; b < DC; ++b)
          tma_load3_own(dst + b * kBlock + lane * box * 128, kv ? v_map : k_map, 64 * b, head, row,
                        ring.full + 8 * stage);
      }
      if (kv == 0) look_up();  // the next unit, while this one's keys come
      if (++stage == kStages) stage = 0, phase ^= 1;
    }
    ++unit_count;
  }
  return true;
}

}  // namespace cg
