// attend.cu -- attention over the paged pool: the workspace, the launches, and
// the join of what several CTAs computed of one row.
#include <algorithm>
#include <cmath>

#include "attend.cuh"

namespace cg {
namespace {

constexpr int kMaxCtas = 160;  // of either kernel, one an SM

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
  __device__ __forceinline__ int64_t at(int i) const {
    // an item begins in its first CTA's share and is at the head of the others'
    return int64_t(2 * (c0 + i) + (i == 0 ? 1 : 0)) * lane->tile + in_tile;
  }
  __device__ __forceinline__ float2 stat(const AttnParams& p, int i) const {
    return c0 == c1 ? p.whole_stats[whole_at] : lane->stats[at(i)];
  }
  __device__ __forceinline__ const float* values(const AttnParams& p, int i) const {
    return c0 == c1 ? p.whole + whole_at * p.dim : lane->pieces + at(i) * p.dim;
  }
};

// One warp joins one (token, query head) row: the lanes first look at the
// parts' maxima, then add up the parts, a lane four channels of each.
template <typename T, int kParts>
__device__ __forceinline__ void join_row(const AttnParams& p, const Part (&part)[kParts], int t,
                                         int qh) {
  const int lane = threadIdx.x & 31, D = p.dim;
  const int n0 = part[0].count(), n = n0 + (kParts > 1 ? part[kParts - 1].count() : 0);
  const auto of = [&](int i) -> const Part& { return kParts > 1 && i >= n0 ? part[kParts - 1] : part[0]; };
  float mm = kNegInf;
  for (int i = lane; i < n; i += 32) mm = fmaxf(mm, of(i).stat(p, i < n0 ? i : i - n0).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, o));
  float ll = 0.f;
  float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int mine = i0 + lane, have = min(32, n - i0);
    float f = 0.f;
    if (mine < n) {
      const float2 st = of(mine).stat(p, mine < n0 ? mine : mine - n0);
      f = weight_of(st.x, mm);
      ll += st.y * f;
    }
#pragma unroll 8
    for (int i = 0; i < have; ++i) {
      const int k = i0 + i;
      const float fk = __shfl_sync(~0u, f, i);
      const float* src = of(k).values(p, k < n0 ? k : k - n0) + 4 * lane;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (128 * h + 4 * lane < D) {
          const float4 v = *reinterpret_cast<const float4*>(src + 128 * h);
          o[h].x += v.x * fk, o[h].y += v.y * fk, o[h].z += v.z * fk, o[h].w += v.w * fk;
        }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) ll += __shfl_xor_sync(~0u, ll, x);
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (128 * h + 4 * lane < D)
      *reinterpret_cast<uint2*>(p.out + int64_t(t) * p.out_stride + int64_t(qh) * D + 128 * h +
                                4 * lane) =
          make_uint2(T::pack(o[h].x * inv, o[h].y * inv), T::pack(o[h].z * inv, o[h].w * inv));
  if (lane == 0 && p.lse != nullptr) p.lse[int64_t(t) * p.q_heads + qh] = log_sum(mm, ll);
}

constexpr int kJoinWarps = 8;

// Without a prefix only items that were cut are joined.  A line with c shares
// has c - 1 cuts; the warps of a cut take the rows of the item that it goes
// through, if it is the item's first cut.
template <typename T, int kTile, int kKeys>
__device__ __forceinline__ void join_cut(const AttnParams& p, const Lane& line, int cut, int first,
                                         int step) {
  const int slots = total_slots<kTile>(p), H = p.kv_heads;
  const int64_t units = line.cum[slots] * H;
  const int ctas = shares_of(line, units);
  if (cut >= ctas) return;
  const int64_t u = share_of(cut, units, ctas);
  const int x = slot_of(line.cum, slots, H, u);
  const int64_t cum = line.cum[x], cost = line.cum[x + 1] - cum;
  const int head = int(uint32_t(u - cum * H) / uint32_t(cost));
  const int64_t item0 = cum * H + head * cost;
  if (item0 == u) return;  // between two items
  Part part[1];
  part[0].lane = &line;
  part[0].c0 = cta_of(item0, units, ctas);
  if (part[0].c0 != cut - 1) return;
  part[0].c1 = cta_of(item0 + cost - 1, units, ctas);
  Item it;
  if (slot_item<kTile, kKeys>(p, x, it) == 0) return;
  for (int r = first; r < it.rows; r += step) {
    const int row = it.row + r, tok = div_of(row, p.group_div);
    part[0].in_tile = r;
    join_row<T>(p, part, it.req.first + tok, head * p.group + row - tok * p.group);
  }
}

template <typename T, int kTile, int kKeys>
__global__ void __launch_bounds__(32 * kJoinWarps) cuts_kernel(AttnParams p) {
  wait_for_previous();
  const int warp = threadIdx.x >> 5;
  constexpr int kRowBlocks = kRowTile / kJoinWarps;  // blocks of a cut of the rows kernel's line
  constexpr int kTileBlocks = 8;
  const int rows_first = kRowBlocks * (p.rows.ctas - 1);
  int b = blockIdx.x;
  if (b < rows_first) {
    join_cut<T, kRowTile, kRowKeys>(p, p.rows, 1 + b / kRowBlocks,
                                    b % kRowBlocks * kJoinWarps + warp, kRowTile);
  } else {
    b -= rows_first;
    join_cut<T, kTile, kKeys>(p, p.tiles, 1 + b / kTileBlocks, b % kTileBlocks * kJoinWarps + warp,
                              kTileBlocks * kJoinWarps);
  }
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
  const int64_t cost = line.cum[x + 1] - line.cum[x];
  const int64_t units = line.cum[total_slots<kTile>(p)] * p.kv_heads;
  const int ctas = shares_of(line, units);
  const int64_t item0 = line.cum[x] * p.kv_heads + head * cost;
  part.c0 = cta_of(item0, units, ctas);
  part.c1 = cta_of(item0 + cost - 1, units, ctas);
  return part;
}

template <typename T, int kTile>
__global__ void __launch_bounds__(32 * kJoinWarps) shared_join_kernel(AttnParams p) {
  wait_for_previous();
  const int row_id = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (row_id >= p.num_tokens * p.q_heads) return;
  const int t = row_id / p.q_heads, qh = row_id - t * p.q_heads;
  if (t >= p.q_starts[p.num_requests]) return;
  const int lo = request_of(p, t);
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
  join_row<T>(p, part, t, qh);
}

uint64_t up256(uint64_t v) { return (v + 255) & ~uint64_t(255); }

struct Workspace {
  uint64_t row_cum, row_pieces, row_stats, tile_cum, tile_pieces, tile_stats, whole, whole_stats,
      total;
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
  w.row_pieces = take(uint64_t(2) * kMaxCtas * kRowTile * D * 4);
  w.row_stats = take(uint64_t(2) * kMaxCtas * kRowTile * 8);
  w.tile_cum = take((tile_slots + 1) * 8);
  w.tile_pieces = take(2 * tile_ctas * tile * D * 4);
  w.tile_stats = take(2 * tile_ctas * tile * 8);
  w.whole = take(rows * D * 4);
  w.whole_stats = take(rows * 8);
  w.total = at;
  return w;
}

template <typename T, int kTile, int kKeys>
cudaError_t launch_all(AttnParams& p, int sms, cudaStream_t stream) {
  p.rows.ctas = std::min(kMaxCtas, sms);
  p.rows.tile = kRowTile;
  const bool tiles = p.tiled || (p.shared && !p.prefix_small);
  p.tiles.ctas = tiles ? std::min(kMaxCtas, sms) : 0;
  p.tiles.tile = kTile;
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
    return launch_after(shared_join_kernel<T, kTile>,
                        unsigned((all + kJoinWarps - 1) / kJoinWarps), 32 * kJoinWarps, 0, stream,
                        true, p);
  }
  const unsigned blocks = kRowTile / kJoinWarps * (p.rows.ctas - 1) + 8 * std::max(0, p.tiles.ctas - 1);
  return launch_after(cuts_kernel<T, kTile, kKeys>, std::max(1u, blocks), 32 * kJoinWarps, 0,
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
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
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
  p.scale_log2 = std::fabs(a.scale) * 1.44269504089f;
  p.q_flip = std::signbit(a.scale) ? 0x80008000u : 0u;
  p.prefix_small = int64_t(p.num_tokens) * p.group <= kRowTile;
  p.tiled = int64_t(p.max_q) * p.group > kRowTile && !p.prefix_small;
  uint8_t* w = static_cast<uint8_t*>(a.workspace_dev);
  const Workspace ws = workspace_of(s, a.num_q_heads, a.num_tokens, a.num_requests, shared);
  p.rows.cum = reinterpret_cast<int64_t*>(w + ws.row_cum);
  p.rows.pieces = reinterpret_cast<float*>(w + ws.row_pieces);
  p.rows.stats = reinterpret_cast<float2*>(w + ws.row_stats);
  p.tiles.cum = reinterpret_cast<int64_t*>(w + ws.tile_cum);
  p.tiles.pieces = reinterpret_cast<float*>(w + ws.tile_pieces);
  p.tiles.stats = reinterpret_cast<float2*>(w + ws.tile_stats);
  p.whole = reinterpret_cast<float*>(w + ws.whole);
  p.whole_stats = reinterpret_cast<float2*>(w + ws.whole_stats);
  return a.dtype == CG_DTYPE_F16 ? launch_type<F16>(p, sms, stream)
                                 : launch_type<BF16>(p, sms, stream);
}

}  // namespace cg
