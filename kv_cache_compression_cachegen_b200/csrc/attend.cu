// attend.cu -- attention over the paged pool: the workspace, the launches, and
// the join of what several CTAs computed of one row.
#include <algorithm>
#include <cmath>
#include <limits>

#include "attend.cuh"

namespace cg {
namespace {

constexpr int64_t kInStepBytes = 64 << 20;  // half of the L2 cache

// Block 0 sums up the rows kernel's line, block 1 the tile kernel's.
template <int kTile, int kKeys>
__global__ void __launch_bounds__(1024) plan_kernel(AttnParams p) {
  if (blockIdx.x == 0) sum_line<kRowTile, kRowKeys>(p, p.rows.cum);
  else sum_line<kTile, kKeys>(p, p.tiles.cum);
}

// The parts of one row of one item: pieces of CTAs c0 to c1, or one whole.
struct Part {
  int c0, c1, in_tile;
  int64_t whole_at;  // in p.whole, if one CTA had all of the item
  const Lane* lane;

  __device__ __forceinline__ int count() const { return c1 - c0 + 1; }
  __device__ __forceinline__ void at(const AttnParams& p, int i, const float2*& stat,
                                     const float*& values) const {
    if (c0 == c1) {
      stat = p.whole_stats + whole_at;
      values = p.whole + whole_at * p.dim;
    } else {
      // an item begins in its first CTA's share and is at the head of the others'
      const int64_t k = int64_t(2 * (c0 + i) + (i == 0 ? 1 : 0)) * lane->tile + in_tile;
      stat = lane->stats + k;
      values = lane->pieces + k * p.dim;
    }
  }
};

constexpr int kJoinThreads = 256;
constexpr int kRowLanes = 8;  // threads of a row
constexpr int kJoinRows = kJoinThreads / kRowLanes;

// Eight threads join one (token, query head) row, each kQuads times four
// channels.  Four parts at a time are asked for together, their maxima and
// sums with their values: most rows have no more, and wait once.
template <typename T, int kQuads, int kParts>
__device__ __forceinline__ void join_row(const AttnParams& p, const Part (&part)[kParts], int t,
                                         int qh) {
  const int lane = threadIdx.x % kRowLanes, D = p.dim;
  const int n0 = part[0].count(), n = n0 + (kParts > 1 ? part[kParts - 1].count() : 0);
  float mm = kNegInf, ll = 0.f;
  float4 o[kQuads];
#pragma unroll
  for (int q = 0; q < kQuads; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += 4) {
    float2 st[4];
    float4 v[4][kQuads];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      st[i] = make_float2(kNegInf, 0.f);
#pragma unroll
      for (int q = 0; q < kQuads; ++q) v[i][q] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + i < n) {
        const float2* stat;
        const float* values;
        if (kParts > 1 && i0 + i >= n0) part[kParts - 1].at(p, i0 + i - n0, stat, values);
        else part[0].at(p, i0 + i, stat, values);
        st[i] = *stat;
#pragma unroll
        for (int q = 0; q < kQuads; ++q)
          if (4 * (q * kRowLanes + lane) < D)
            v[i][q] = *reinterpret_cast<const float4*>(values + 4 * (q * kRowLanes + lane));
      }
    }
    float top = mm;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fmaxf(top, st[i].x);
    const float f0 = weight_of(mm, top);
    mm = top;
    ll *= f0;
#pragma unroll
    for (int q = 0; q < kQuads; ++q) o[q].x *= f0, o[q].y *= f0, o[q].z *= f0, o[q].w *= f0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = weight_of(st[i].x, top);
      ll += st[i].y * f;
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        o[q].x += v[i][q].x * f, o[q].y += v[i][q].y * f;
        o[q].z += v[i][q].z * f, o[q].w += v[i][q].w * f;
      }
    }
  }
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
  uint16_t* out = p.out + int64_t(t) * p.out_stride + int64_t(qh) * D;
#pragma unroll
  for (int q = 0; q < kQuads; ++q)
    if (4 * (q * kRowLanes + lane) < D)
      *reinterpret_cast<uint2*>(out + 4 * (q * kRowLanes + lane)) =
          make_uint2(T::pack(o[q].x * inv, o[q].y * inv), T::pack(o[q].z * inv, o[q].w * inv));
  if (lane == 0 && p.lse != nullptr) p.lse[int64_t(t) * p.q_heads + qh] = log_sum(mm, ll);
}

// Without a prefix only items that were cut are joined, each at its first cut,
// which the CTA behind it has noted.
template <typename T, int kTile>
__global__ void __launch_bounds__(kJoinThreads) cuts_kernel(AttnParams p) {
  wait_for_previous();
  constexpr int kBlocks = kTile / kJoinRows;  // blocks of a cut of the tile kernel's line
  int b = int(blockIdx.x) - p.rows.ctas, r = threadIdx.x / kRowLanes;
  const Lane& line = b < 0 ? p.rows : p.tiles;
  if (b < 0) {
    b += p.rows.ctas;
  } else {
    r += b % kBlocks * kJoinRows;
    b /= kBlocks;
  }
  const Cut cut = line.cuts[b];
  if (cut.c1 < cut.c0 || r >= cut.rows) return;
  const int row = cut.row + r, tok = div_of(row, p.group_div);
  const Part part[1] = {Part{cut.c0, cut.c1, r, 0, &line}};
  join_row<T, kTile == 256 ? 4 : 8>(p, part, cut.first + tok,
                                    cut.head * p.group + row - tok * p.group);
}

// With a prefix every row has two items, its own and the prefix's.
template <int kTile>
__device__ __forceinline__ Part find_part(const AttnParams& p, const Lane& line, bool prefix,
                                          int request, int row, int head, int64_t whole_at) {
  Part part;
  part.lane = &line;
  part.whole_at = whole_at;
  const int x = (prefix ? own_slots<kTile>(p) : slot_base<kTile>(p, request)) + row / kTile;
  part.in_tile = row % kTile;
  const int64_t cum = line.cum[x], cost = line.cum[x + 1] - cum;
  const int64_t units = line.cum[total_slots<kTile>(p)] * p.kv_heads;
  const int ctas = shares_of<kTile>(p, line, units);
  const int64_t item0 = cum * p.kv_heads + head * cost;
  part.c0 = cta_of(item0, units, ctas);
  part.c1 = cta_of(item0 + cost - 1, units, ctas);
  return part;
}

template <typename T, int kTile>
__global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(AttnParams p) {
  wait_for_previous();
  const int row_id = blockIdx.x * kJoinRows + threadIdx.x / kRowLanes;
  if (row_id >= p.num_tokens * p.q_heads) return;
  const int t = row_id / p.q_heads, qh = row_id - t * p.q_heads;
  if (t >= p.q_starts[p.num_requests]) return;
  const int lo = last_not_above(p.num_requests, t, FirstRows{p.q_starts});
  Request req;
  if (!load_request(p, lo, req) || t < req.first || t >= req.first + req.tokens) return;
  const int head = div_of(qh, p.group_div), member = qh - head * p.group;
  const int64_t rows = int64_t(p.num_tokens) * p.q_heads;
  const int own = (t - req.first) * p.group + member, of_all = t * p.group + member;
  const Part part[2] = {
      req.tokens * p.group <= kRowTile
          ? find_part<kRowTile>(p, p.rows, false, lo, own, head, row_id)
          : find_part<kTile>(p, p.tiles, false, lo, own, head, row_id),
      p.prefix_small ? find_part<kRowTile>(p, p.rows, true, lo, of_all, head, rows + row_id)
                     : find_part<kTile>(p, p.tiles, true, lo, of_all, head, rows + row_id)};
  join_row<T, kTile == 256 ? 4 : 8>(p, part, t, qh);
}

// Of the current device.
cudaError_t multiprocessors(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  *sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (*sms == 0) {
    err = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (err == cudaSuccess && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  }
  return err;
}

uint64_t up256(uint64_t v) { return (v + 255) & ~uint64_t(255); }

struct Workspace {
  uint64_t row_cum, row_cuts, row_pieces, row_stats, tile_cum, tile_cuts, tile_pieces, tile_stats,
      whole, whole_stats, total;
};

Workspace workspace_of(const cg_shape& s, int Hq, int tokens, int requests, bool shared) {
  const uint64_t D = s.head_dim, group = Hq / s.num_kv_heads;
  const uint64_t tile = tile_rows(s.head_dim);
  const uint64_t row_slots = uint64_t(requests) + 1;
  const uint64_t tile_slots = 2 * (tokens * group / tile) + requests + 1;
  // without a request or a batch of more than 16 rows the tile kernel has no work
  const uint64_t tile_ctas = tokens * group > kRowTile ? kMaxCtas : 0;
  const uint64_t rows = shared ? uint64_t(2) * tokens * Hq : 0;
  Workspace w;
  uint64_t at = 0;
  const auto take = [&at](uint64_t bytes) {
    const uint64_t here = at;
    at = up256(at + bytes);
    return here;
  };
  w.row_cum = take((row_slots + 1) * 8);
  w.row_cuts = take(kMaxRowCtas * sizeof(Cut));
  w.row_pieces = take(uint64_t(2) * kMaxRowCtas * kRowTile * D * 4);
  w.row_stats = take(uint64_t(2) * kMaxRowCtas * kRowTile * 8);
  w.tile_cum = take((tile_slots + 1) * 8);
  w.tile_cuts = take(tile_ctas * sizeof(Cut));
  w.tile_pieces = take(2 * tile_ctas * tile * D * 4);
  w.tile_stats = take(2 * tile_ctas * tile * 8);
  w.whole = take(rows * D * 4);
  w.whole_stats = take(rows * 8);
  w.total = at;
  return w;
}

template <typename T, int kTile, int kKeys>
cudaError_t launch_all(AttnParams& p, int sms, cudaStream_t stream) {
  p.rows.ctas = std::min(kMaxRowCtas, sms * row_ctas_per_sm(p.dim, most_rows(p)));
  p.rows.tile = kRowTile;
  const bool tiles = p.tiled || (p.shared && !p.prefix_small);
  p.tiles.ctas = tiles ? std::min(kMaxCtas, sms) : 0;
  p.tiles.tile = kTile;
  p.tiles.in_step = p.shared && !p.tiled && !p.prefix_small &&
                    int64_t(p.prefix_tokens) * p.kv_heads * p.dim * 4 > kInStepBytes;
  const int64_t rows = int64_t(p.num_tokens) * p.group;
  const int64_t slots = (tiles ? 2 * (rows / kTile) : 0) + p.num_requests + 1;
  p.planned = slots > kScanSlots;
  cudaError_t err = cudaSuccess;
  if (p.planned) {
    plan_kernel<kTile, kKeys><<<tiles ? 2 : 1, 1024, 0, stream>>>(p);
    err = cudaGetLastError();
  }
  if (err == cudaSuccess && tiles) err = launch_tiles(p, T::kBf16, stream);
  if (err == cudaSuccess) err = launch_rows(p, T::kBf16, tiles, stream);
  if (err != cudaSuccess) return err;
  if (p.shared) {
    const int64_t all = int64_t(p.num_tokens) * p.q_heads;
    return launch_after(shared_join_kernel<T, kTile>, unsigned((all + kJoinRows - 1) / kJoinRows),
                        kJoinThreads, 0, stream, true, p);
  }
  return launch_after(cuts_kernel<T, kTile>,
                      unsigned(p.rows.ctas + kTile / kJoinRows * p.tiles.ctas), kJoinThreads, 0,
                      stream, true, p);
}

template <typename T>
cudaError_t launch_type(AttnParams& p, int sms, cudaStream_t stream) {
  return p.dim <= 128 ? launch_all<T, 256, 128>(p, sms, stream)
                      : launch_all<T, 128, 64>(p, sms, stream);
}

}  // namespace

uint64_t attention_workspace(const cg_shape& s, int32_t num_q_heads, int32_t max_tokens,
                             int32_t max_requests, bool shared) {
  return workspace_of(s, num_q_heads, max_tokens, max_requests, shared).total;
}

cudaError_t launch_attention(const cg_attention_args& a, const cg_shape& s,
                             const int32_t* prefix_table, int32_t prefix_tokens, bool shared,
                             cudaStream_t stream) {
  int sms = 0;
  const cudaError_t err = multiprocessors(&sms);
  if (err != cudaSuccess) return err;
  AttnParams p{};
  p.q = a.q_dev;
  p.out = a.out_dev;
  p.lse = a.lse_dev;
  p.q_stride = a.q_stride;
  p.out_stride = a.out_stride;
  p.q_starts = a.q_starts_dev;
  p.kv_lens = a.kv_lens_dev;
  p.tables = a.block_tables_dev;
  p.prefix_table = prefix_table;
  const int64_t half_pool =
      int64_t(a.num_pages) * a.page_tokens * s.num_kv_heads * s.head_dim;
  p.k_pool = a.pool_dev + int64_t(a.layer) * 2 * half_pool;
  p.v_pool = p.k_pool + half_pool;
  p.status = a.status_dev;
  p.num_requests = a.num_requests;
  p.num_tokens = a.num_tokens;
  p.max_q = a.max_q;
  p.q_heads = a.num_q_heads;
  p.kv_heads = s.num_kv_heads;
  p.group = a.num_q_heads / s.num_kv_heads;
  p.dim = s.head_dim;
  p.num_pages = a.num_pages;
  p.page_tokens = a.page_tokens;
  p.max_pages = a.max_pages;
  p.page_div = fast_div(uint32_t(a.page_tokens));
  p.group_div = fast_div(uint32_t(p.group));
  p.window = a.window;
  p.sinks = a.sinks;
  p.prefix_tokens = prefix_tokens;
  p.shared = shared;
  // a negative scale is the positive one with q's signs turned, so that the
  // largest product is the largest score
  // (a scale of zero is the smallest number, so that a hidden score, -infinity, stays
  // that: scores are zero to within 2^-20 all the same)
  p.scale_log2 = std::max(std::fabs(a.scale) * 1.44269504089f,
                          std::numeric_limits<float>::denorm_min());
  p.q_flip = std::signbit(a.scale) ? 0x80008000u : 0u;
  p.prefix_small = int64_t(p.num_tokens) * p.group <= kRowTile;
  p.tiled = int64_t(p.max_q) * p.group > kRowTile && !p.prefix_small;
  uint8_t* w = static_cast<uint8_t*>(a.workspace_dev);
  const Workspace ws = workspace_of(s, a.num_q_heads, a.num_tokens, a.num_requests, shared);
  p.rows.cum = reinterpret_cast<int64_t*>(w + ws.row_cum);
  p.rows.cuts = reinterpret_cast<Cut*>(w + ws.row_cuts);
  p.rows.pieces = reinterpret_cast<float*>(w + ws.row_pieces);
  p.rows.stats = reinterpret_cast<float2*>(w + ws.row_stats);
  p.tiles.cum = reinterpret_cast<int64_t*>(w + ws.tile_cum);
  p.tiles.cuts = reinterpret_cast<Cut*>(w + ws.tile_cuts);
  p.tiles.pieces = reinterpret_cast<float*>(w + ws.tile_pieces);
  p.tiles.stats = reinterpret_cast<float2*>(w + ws.tile_stats);
  p.whole = reinterpret_cast<float*>(w + ws.whole);
  p.whole_stats = reinterpret_cast<float2*>(w + ws.whole_stats);
  return a.dtype == CG_DTYPE_F16 ? launch_type<F16>(p, sms, stream)
                                 : launch_type<BF16>(p, sms, stream);
}

}  // namespace cg
