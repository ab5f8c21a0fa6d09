// attend.cuh -- what the attention kernels share: their parameters, which
// keys a request's rows see, and how the work is dealt to the CTAs.
//
// Two kernels.  Requests with at most 16 query rows a kv head (tokens times
// heads of a group: single tokens, a few at most) are bound by the bytes of K
// and V and go to the rows kernel; the others, and a shared prefix under the
// rows of a whole batch, are matrix products and go to the tile kernel.
//
// Work.  An *item* is one request's tile of query rows at one kv head; a row
// is a (token, query head of the group) pair, token-major, so that the heads
// that share a kv head share its loads.  An item's keys are cut into units of
// kKeys keys, aligned in the sequence; its units are those that hold a sink
// followed by those from the window's start to the last row.  All
// units of all items, request by request and head by head, form one line that
// is cut into equal shares, one a CTA, whatever the lengths: one long request
// among short ones, or a batch of one, fills the machine.  A CTA whose share
// holds an item whole writes its output; an item cut between CTAs leaves a
// piece (unnormalised sums, running maximum and sum) with each, and a second
// kernel joins them.  Everything about the cut follows from the lengths, so
// the join needs no flags and the workspace no clearing, and the order of
// every sum is fixed.
#pragma once

#include <atomic>
#include <cuda.h>  // tensor-map types only; the encoder is looked up at run time

#include "paged.cuh"
#include "shares.cuh"

namespace cg {

constexpr int kRowTile = 16;   // query rows of an item of the rows kernel (one matrix tile)
constexpr int kRowKeys = 64;   // keys of a unit there
constexpr int kScanSlots = 1024;  // slots of a line that every CTA sums up by itself

// The line of work of one of the two kernels, in the workspace.
struct Cut {
  int first, row, rows;  // first packed row of q, first row of the tile, rows in it
  int head, c0, c1;      // kv head, CTAs that have pieces; c1 < c0: nothing was cut here
};

struct Lane {
  int64_t* cum;   // [slots + 1] units of one head before each slot
  Cut* cuts;      // [ctas] by each CTA: the item that its share begins in the middle of
  float* pieces;  // [2 * ctas][tile][dim] unnormalised outputs of cut items
  float2* stats;  // [2 * ctas][tile] (maximum in log2 units, sum)
  int ctas;       // CTAs of the kernel's grid, 0: not launched
  int in_step;    // give every tile of the prefix equal shares at equal places
  int tile;       // query rows of an item
};

struct AttnParams {
  const uint16_t* q;
  uint16_t* out;
  float* lse;  // [num_tokens][q_heads] or null
  int64_t q_stride, out_stride;
  const int32_t *q_starts, *kv_lens, *tables, *prefix_table;
  const uint16_t *k_pool, *v_pool;  // the layer's halves of the pool
  int32_t* status;
  int num_requests, num_tokens, max_q, q_heads, kv_heads, group, dim;
  int num_pages, page_tokens, max_pages;
  FastDiv page_div, group_div;
  int window, sinks;
  int prefix_tokens, shared;
  float scale_log2;  // scale * log2(e)
  uint32_t q_flip;    // sign bits of a negative scale, applied to q
  int prefix_small;   // the rows of the whole batch fit the rows kernel
  int tiled;          // requests above the rows kernel's size may be there (max_q)
  int planned;        // the lines are too long for that: a kernel before has summed them up
  Lane rows, tiles;
  // shared: items that one CTA finished, [own, prefix][num_tokens][q_heads][dim]
  float* whole;
  float2* whole_stats;
};

// What one request brings: its packed query rows and its keys.
struct Request {
  int first, tokens;  // rows of q
  int keys;           // tokens in the pool
  int row0;           // position of its first new token among the keys (may be negative)
};

constexpr int kMostKeys = 0x7FFFFF00;  // a unit's last key is counted in 31 bits

// False (and the request is left out) where the lengths do not fit the call.
__device__ __forceinline__ bool load_request(const AttnParams& p, int r, Request& q) {
  const int a = p.q_starts[r], b = p.q_starts[r + 1], keys = p.kv_lens[r];
  q.first = a;
  q.tokens = 0;
  q.keys = 0;
  q.row0 = 0;
  if (a < 0 || b < a || b > p.num_tokens || b - a > p.max_q || keys < 0 || keys > kMostKeys ||
      int64_t(keys) > int64_t(p.max_pages) * p.page_tokens)
    return false;
  q.tokens = b - a;
  q.keys = keys;
  q.row0 = keys - q.tokens;
  return true;
}

// The keys that rows at positions [p0, p1] may see between them: [0, sink_end)
// and [lo, hi), and the units that hold them.
struct Span {
  int sink_end, lo, hi;
  int sink_units, first_unit, units;
};

template <int kKeys>
__device__ __forceinline__ Span span_of(int p0, int p1, int window, int sinks) {
  Span s;
  s.hi = p1 + 1 > 0 ? p1 + 1 : 0;
  s.lo = (window > 0 && p0 >= window) ? p0 - window + 1 : 0;
  s.sink_end = sinks < s.lo ? sinks : s.lo;
  s.sink_units = (s.sink_end + kKeys - 1) / kKeys;
  s.first_unit = s.lo / kKeys > s.sink_units ? s.lo / kKeys : s.sink_units;
  const int last = (s.hi + kKeys - 1) / kKeys;
  s.units = s.sink_units + (last > s.first_unit ? last - s.first_unit : 0);
  if (s.hi == 0) s.units = 0;
  return s;
}

// Whether a row at position `at` sees a key.
__device__ __forceinline__ bool sees(int key, int at, int window, int sinks) {
  return key <= at && (window == 0 || at - key < window || key < sinks);
}

// First key of the u-th unit.
template <int kKeys>
__device__ __forceinline__ int unit_key(const Span& s, int u) {
  return (u < s.sink_units ? u : s.first_unit + u - s.sink_units) * kKeys;
}

struct Item {
  Request req;
  Span span;
  int request;    // whose table, -1: the prefix's
  int row, rows;  // first row of the tile among the request's rows, rows in it
};

// Slots of the kernels' lines.  Rows kernel: one a request.  Tile kernel:
// request r's tiles start at slot floor(first row / kTile) + r, which leaves room
// for every tile whatever the lengths; a slot without a tile costs nothing.
// The prefix's tiles come last.
template <int kTile>
__device__ __forceinline__ int own_slots(const AttnParams& p) {
  if (kTile == kRowTile) return p.num_requests;
  return p.tiled ? int(int64_t(p.num_tokens) * p.group / kTile) + p.num_requests : 0;
}

template <int kTile>
__device__ __forceinline__ int total_slots(const AttnParams& p) {
  const bool prefix = p.shared && (p.prefix_small != 0) == (kTile == kRowTile);
  return own_slots<kTile>(p) +
         (prefix ? int((int64_t(p.num_tokens) * p.group + kTile - 1) / kTile) : 0);
}

// The most rows that an item of the rows kernel can have: a request's, or the
// whole batch's under a prefix.
inline int64_t most_rows(const AttnParams& p) {
  const int64_t tokens =
      p.shared && p.prefix_small ? p.num_tokens : (p.max_q < p.num_tokens ? p.max_q : p.num_tokens);
  return tokens * p.group;
}
constexpr int row_ctas_per_sm(int dim, int64_t rows) {
  return dim > 128 && rows > 8 ? 1 : kRowCtasPerSm;
}

// Query rows of a kv head in the whole batch.
__device__ __forceinline__ int batch_rows(const AttnParams& p) {
  int n = p.q_starts[p.num_requests];
  n = n < 0 ? 0 : (n > p.num_tokens ? p.num_tokens : n);
  return n * p.group;
}

template <int kTile>
__device__ __forceinline__ int slot_base(const AttnParams& p, int r) {
  return kTile == kRowTile ? r : FirstSlots{p.q_starts, p.num_tokens, p.group, kTile}(r);
}

// What an item costs besides its units (queries, output, an empty pipeline), in
// units, so that shares of many short items are not longer than others.  Tiles at
// 1, 2, 3, 4, 5 and 8: 24 questions behind 10,752 shared tokens 323, 243, 198, 173,
// 176 and 185 us; prompts of up to 8,192 tokens 1,397, 1,248, 1,199 and 1,194 at
// the first four.
template <int kTile>
__host__ __device__ constexpr int item_cost() {
  return kTile == kRowTile ? 1 : 4;
}

// The item of slot x and its units for each kv head; 0 where it holds no rows.
template <int kTile, int kKeys>
__device__ __forceinline__ int slot_item(const AttnParams& p, int x, Item& it) {
  const int own = own_slots<kTile>(p);
  if (x >= own) {
    it.request = -1;
    it.req.first = 0;
    it.req.tokens = batch_rows(p) / p.group;
    it.req.keys = p.prefix_tokens;
    it.req.row0 = p.prefix_tokens - 1;  // where a row sees all of the prefix
    it.row = (x - own) * kTile;
  } else {
    int lo = x;
    if (kTile != kRowTile)
      lo = last_not_above(p.num_requests, x, FirstSlots{p.q_starts, p.num_tokens, p.group, kTile});
    it.request = lo;
    if (!load_request(p, lo, it.req)) {
      report(p.status, CG_ERR_MISMATCH);
      return 0;
    }
    if ((it.req.tokens * p.group <= kRowTile) != (kTile == kRowTile)) return 0;
    it.row = kTile == kRowTile ? 0 : (x - slot_base<kTile>(p, lo)) * kTile;
  }
  const int rows = it.req.tokens * p.group;
  if (it.row < 0 || it.row >= rows) return 0;
  it.rows = rows - it.row < kTile ? rows - it.row : kTile;
  if (it.request < 0) {
    it.span = span_of<kKeys>(p.prefix_tokens - 1, p.prefix_tokens - 1, 0, 0);
  } else {
    const int t0 = div_of(it.row, p.group_div), t1 = div_of(it.row + it.rows - 1, p.group_div);
    it.span = span_of<kKeys>(it.req.row0 + t0, it.req.row0 + t1, p.window, p.sinks);
  }
  // an item without a visible key still has its rows to write
  return (it.span.units > 0 ? it.span.units : 1) + item_cost<kTile>();
}

// Position of a row of an item among its keys (at the last one for the prefix).
__device__ __forceinline__ int row_position(const AttnParams& p, const Item& it, int row) {
  return it.request < 0 ? it.req.row0 : it.req.row0 + div_of(row, p.group_div);
}

// CTAs that get a share: no share is empty.  In step: where a prefix is larger
// than the L2 cache, its row tiles should read the same keys at the same time,
// and do if each has the same number of shares (the line goes tile by tile, and
// all have the same units).  Taken where it leaves no more than a tenth of the
// CTAs without work: 96 single tokens of 64 heads behind 79,872 tokens (three
// tiles a kv head) went from 304 to 289 us.
template <int kTile>
__device__ __forceinline__ int shares_of(const AttnParams& p, const Lane& lane, int64_t units) {
  int c = units < lane.ctas ? int(units) : lane.ctas;
  if (lane.in_step) {
    const int tiles = (batch_rows(p) + kTile - 1) / kTile;
    if (tiles > 1 && c / tiles * tiles * 10 >= c * 9) c = c / tiles * tiles;
  }
  return c;
}

// Row of the pool that holds a key, or -1 where the table has no such page.
__device__ __forceinline__ int pool_row(const AttnParams& p, const int32_t* table, int key) {
  const int col = div_of(key, p.page_div);
  const int page = __ldg(table + col);
  if (page < 0 || page >= p.num_pages) {
    report(p.status, CG_ERR_MISMATCH);
    return -1;
  }
  return page * p.page_tokens + (key - col * p.page_tokens);
}

__device__ __forceinline__ void prefetch_line(const void* p) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

// Units of one head before each slot of a line, and of the whole line behind
// the last.  All threads of a block; blockDim.x at most 1024.
template <int kTile, int kKeys>
__device__ void sum_line(const AttnParams& p, int64_t* cum) {
  __shared__ int64_t warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int slots = total_slots<kTile>(p);
  int64_t base = 0;
  for (int x0 = 0; x0 < slots; x0 += blockDim.x) {
    const int x = x0 + threadIdx.x;
    Item it;
    const int64_t own = x < slots ? slot_item<kTile, kKeys>(p, x, it) : 0;
    int64_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(~0u, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    const int64_t w = lane < warps ? warp_sum[lane] : 0;
    int64_t wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(~0u, wi, o);
      if (lane >= o) wi += up;
    }
    const int64_t before = base + __shfl_sync(~0u, wi - w, warp) + sum - own;
    if (x < slots) cum[x] = before;
    base += __shfl_sync(~0u, wi, 31);
    __syncthreads();
  }
  if (threadIdx.x == 0) cum[slots] = base;
  __syncthreads();
}

// The slot that holds unit u of a line: the last one with heads * cum[x] <= u.
__device__ __forceinline__ int slot_of(const int64_t* cum, int slots, int heads, int64_t u) {
  int x = 0, hi = slots - 1;
  while (x < hi) {
    const int mid = (x + hi + 1) >> 1;
    if (cum[mid] * heads <= u) x = mid;
    else hi = mid - 1;
  }
  return x;
}

// One CTA's share of a line, item by item.
template <int kTile, int kKeys>
struct Walk {
  int64_t u, u_end, share0, cum, units;
  int x, slots, ctas;
  int known = -1;  // the slot that `it` and `cost` are of
  // the current part: units [first, last) of an item of `cost` units at `head`
  Item it;
  int64_t item0;  // its first unit
  int cost, head, first, last, piece;
  bool whole;

  // All threads of the block; cum_s has room for kScanSlots + 1.
  __device__ __forceinline__ bool begin(const AttnParams& p, const Lane& lane, int64_t* cum_s) {
    // the lengths are looked at in an order that waits: have their lines come first
    for (int i = 32 * threadIdx.x; i <= p.num_requests; i += 32 * blockDim.x) {
      prefetch_line(p.q_starts + i);
      if (i < p.num_requests) prefetch_line(p.kv_lens + i);
    }
    slots = total_slots<kTile>(p);
    item0 = share0 = 0;
    if (slots <= 32) return begin_warp(p, lane);
    const int64_t* line = lane.cum;
    if (!p.planned) {
      sum_line<kTile, kKeys>(p, cum_s);
      line = cum_s;
      if (blockIdx.x == 0)  // for the join
        for (int i = threadIdx.x; i <= slots; i += blockDim.x) lane.cum[i] = cum_s[i];
    }
    units = line[slots] * p.kv_heads;
    if (!take_share(p, lane)) return false;
    x = slot_of(line, slots, p.kv_heads, u);
    cum = line[x];
    return true;
  }

  // A short line: every warp sums it up by itself, a slot a lane, and nothing waits.
  __device__ __forceinline__ bool begin_warp(const AttnParams& p, const Lane& lane) {
    const int at = threadIdx.x & 31;
    const int64_t own = at < slots ? slot_item<kTile, kKeys>(p, at, it) : 0;
    int64_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(~0u, sum, o);
      if (at >= o) sum += up;
    }
    const int64_t total = __shfl_sync(~0u, sum, 31);
    if (blockIdx.x == 0 && threadIdx.x < 32) {
      if (at < slots) lane.cum[at] = sum - own;
      if (at == 0) lane.cum[slots] = total;
    }
    units = total * p.kv_heads;
    const bool any = take_share(p, lane);
    const uint32_t before =
        __ballot_sync(~0u, any && at < slots && (sum - own) * p.kv_heads <= u);
    x = any ? 31 - __clz(before) : 0;
    cum = __shfl_sync(~0u, sum - own, x);
    return any;
  }

  __device__ __forceinline__ bool take_share(const AttnParams& p, const Lane& lane) {
    ctas = shares_of<kTile>(p, lane, units);
    if (int(blockIdx.x) >= ctas) return false;
    u = share_of(blockIdx.x, units, ctas);
    u_end = share_of(blockIdx.x + 1, units, ctas);
    share0 = u;
    return true;
  }

  __device__ __forceinline__ bool next(const AttnParams& p) {
    while (u < u_end && x < slots) {
      if (known != x) {
        cost = slot_item<kTile, kKeys>(p, x, it);
        known = x;
      }
      if (cost == 0 || u >= (cum + cost) * p.kv_heads) {
        cum += cost;
        ++x;
        continue;
      }
      head = int(uint32_t(u - cum * p.kv_heads) / uint32_t(cost));  // a slot's units fit 31 bits
      item0 = cum * p.kv_heads + int64_t(head) * cost;
      const int from = int(u - item0);
      const int to = int((item0 + cost < u_end ? item0 + cost : u_end) - item0);
      whole = from == 0 && to == cost;
      piece = 2 * int(blockIdx.x) + (item0 >= share0 ? 1 : 0);
      u = item0 + to;
      // the first units of an item's cost stand for what an item takes by itself
      first = max(0, from - item_cost<kTile>());
      last = min(it.span.units, max(0, to - item_cost<kTile>()));
      return true;
    }
    return false;
  }

  // One thread, after the first next() (or none): what the join has to know.
  __device__ __forceinline__ void note_cut(const Lane& lane, bool any) const {
    Cut cut{0, 0, 0, 0, 0, -1};
    // an item over several shares is joined at its first cut
    if (any && item0 < share0 && cta_of(item0, units, ctas) + 1 == int(blockIdx.x))
      cut = Cut{it.req.first, it.row, it.rows, head, int(blockIdx.x) - 1,
                cta_of(item0 + cost - 1, units, ctas)};
    lane.cuts[blockIdx.x] = cut;
  }
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Weight of a part with maximum m (log2 units) under the common maximum; a part
// that saw no key has none.  (A NaN among its scores is in its sums.)
__device__ __forceinline__ float weight_of(float m, float top) {
  return m == top ? (m == -__builtin_huge_valf() ? 0.f : 1.f) : exp2_fast(m - top);
}

constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718056f;
}

// Programmatic dependent launch: let the next kernel of the stream start, and
// wait for the one before to have finished and written its results.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Allow a kernel its dynamic shared memory, once on each device.
template <typename... Args>
cudaError_t allow_smem(void (*kernel)(Args...), int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

template <typename... Args>
cudaError_t launch_after(void (*kernel)(Args...), unsigned grid, unsigned threads, size_t smem,
                         cudaStream_t stream, bool early, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Tensor maps (attend_maps.cu) of one half (K or V) of the layer's pool in boxes
// of `box` rows, and of the queries in boxes of 128 rows of a kv head.  False
// where there is none for this geometry.
struct KvMaps {
  CUtensorMap k, v;
  int box;  // 0: none
};
KvMaps kv_maps(const AttnParams& p, int most_rows, bool bf16);
bool query_map(CUtensorMap* map, const AttnParams& p, bool bf16);

// attend_tile.cu, attend_rows.cu
int tile_rows(int dim);  // query rows of an item of the tile kernel
cudaError_t launch_tiles(const AttnParams& p, bool bf16, cudaStream_t stream);
cudaError_t launch_rows(const AttnParams& p, bool bf16, bool early, cudaStream_t stream);

}  // namespace cg
