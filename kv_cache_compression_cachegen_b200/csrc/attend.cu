// attend.cu -- attention over the paged pool for few query rows a kv head
// (single tokens, and the heads of a group), and the join of cut items.
//
//     o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),   s_j = (q . k_j) scale log2(e)
//
// in one pass over the keys with a running maximum m.  A row of K and V serves
// at most 16 query rows, so the bytes of K and V bound it.  They go from
// memory to registers in the layout that the matrix instruction wants, with no
// shared memory and no barrier between a load and its use:
//   - K: the product sums over the channels, so their order is free.  A lane
//     takes 16 bytes of a key's row, and those eight channels are its share of
//     two k-steps; the query's fragments are laid out the same.
//   - V: the product sums over the keys, so a fragment register holds two
//     keys' values of one channel.  A lane loads the same eight channels of
//     four keys and interleaves them by byte permutes; which channel is which
//     output column is free again.
// Each warp takes 16 keys of a unit, keeps its own maximum, sum and output,
// and the four warps of a CTA are joined once per item.
#include <algorithm>
#include <cmath>

#include "attend.cuh"

namespace cg {
namespace {

constexpr int kRowWarps = 4;
static_assert(kRowKeys == 16 * kRowWarps, "each warp takes 16 keys of a unit");
constexpr int kRowThreads = 32 * kRowWarps;
constexpr int kMaxRowCtas = 160 * 4;
constexpr int kMaxTileCtas = 160;

// Units of one head before each slot of a line.  One block.
template <int kTile, int kKeys>
__device__ void plan_line(const AttnParams& p, int64_t* cum) {
  __shared__ int64_t warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slots = total_slots<kTile>(p);
  int64_t base = 0;
  for (int x0 = 0; x0 < slots; x0 += 1024) {
    const int x = x0 + threadIdx.x;
    Item it;
    int64_t own = x < slots ? slot_item<kTile, kKeys>(p, x, it) : 0, sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(~0u, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int64_t w = warp_sum[lane], wi = w;
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
}

// Block 0 plans the rows kernel, block 1 the tile kernel.
template <int kTile, int kKeys>
__global__ void __launch_bounds__(1024) plan_kernel(AttnParams p) {
  if (blockIdx.x == 0) plan_line<kRowTile, kRowKeys>(p, p.rows.cum);
  else plan_line<kTile, kKeys>(p, p.tiles.cum);
}

// DB: 32-channel blocks of a head (K), VB: 64-channel blocks (V).
template <typename T, int DB>
__global__ void __launch_bounds__(kRowThreads, DB <= 4 ? 3 : 1) rows_kernel(AttnParams p) {
  constexpr int VB = (DB + 1) / 2;
  extern __shared__ float smem[];  // [kRowWarps][16][VB * 64] outputs
  __shared__ float stat_m[kRowWarps][16], stat_l[kRowWarps][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int H = p.kv_heads, D = p.dim;
  Walk<kRowTile, kRowKeys> w;
  if (!w.begin(p, p.rows)) return;
  while (w.next(p)) {
    const Item& it = w.it;
    const int head = w.head;
    // The two query rows of this lane's quad and their positions.
    uint32_t qf[DB][2][4];
    int pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = it.row + g + 8 * i;
      const int tok = div_of(row, p.group_div);
      const bool real = g + 8 * i < it.rows;
      pos[i] = row_position(p, it, row);
      const uint16_t* src = p.q + int64_t(it.req.first + tok) * p.q_stride +
                            int64_t(head * p.group + (row - tok * p.group)) * D;
#pragma unroll
      for (int b = 0; b < DB; ++b) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (real && 32 * b + 8 * c < D) v = *reinterpret_cast<const uint4*>(src + 32 * b + 8 * c);
        qf[b][0][i] = v.x ^ p.q_flip;
        qf[b][0][2 + i] = v.y ^ p.q_flip;
        qf[b][1][i] = v.z ^ p.q_flip;
        qf[b][1][2 + i] = v.w ^ p.q_flip;
      }
    }
    const bool prefix = it.request < 0;
    const int32_t* table = prefix ? p.prefix_table : p.tables + int64_t(it.request) * p.max_pages;
    const uint16_t* kb = p.k_pool + int64_t(head) * D;
    const uint16_t* vb = p.v_pool + int64_t(head) * D;
    const int64_t step = int64_t(H) * D;
    const int window = prefix ? 0 : p.window, sinks = prefix ? 0 : p.sinks;
    const int tok0 = div_of(it.row, p.group_div);
    const int tok1 = div_of(it.row + it.rows - 1, p.group_div);

    float acc[VB][8][4];
#pragma unroll
    for (int b = 0; b < VB; ++b)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[b][j][e] = 0.f;
    float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};  // m in log2 units

    for (int unit = w.first; unit < w.last; ++unit) {
      const int key0 = unit_key<kRowKeys>(it.span, unit) + 16 * warp;
      int mine = -1;  // pool row of key0 + (lane & 15); -1: no row of the tile sees it
      {
        const int key = key0 + (lane & 15);
        if (key < it.span.hi && (key >= it.span.lo || key < it.span.sink_end))
          mine = pool_row(p, table, key);
      }
      if (__all_sync(~0u, mine < 0)) continue;
      // S = Q K^T for 16 keys, as two tiles of 8
      float s[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int row = __shfl_sync(~0u, mine, g + 8 * t);
        const uint16_t* src = kb + row * step + 8 * c;
        uint4 kf[DB];
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          kf[b] = make_uint4(0, 0, 0, 0);
          if (row >= 0 && 32 * b + 8 * c < D)
            kf[b] = __ldg(reinterpret_cast<const uint4*>(src + 32 * b));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          T::mma(s[t], qf[b][0], kf[b].x, kf[b].y);
          T::mma(s[t], qf[b][1], kf[b].z, kf[b].w);
        }
      }
      // V of this lane's four keys
      int vrow[4];
      uint4 vf[VB][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vrow[i] = __shfl_sync(~0u, mine, 2 * c + (i & 1) + 8 * (i >> 1));
        const uint16_t* src = vb + vrow[i] * step + 8 * g;
#pragma unroll
        for (int b = 0; b < VB; ++b) {
          vf[b][i] = make_uint4(0, 0, 0, 0);
          if (vrow[i] >= 0 && 64 * b + 8 * g < D)
            vf[b][i] = __ldg(reinterpret_cast<const uint4*>(src + 64 * b));
        }
      }
      // s[t][e]: row e / 2, key 2 c + (e & 1) + 8 t of the sixteen
      float most[2] = {kNegInf, kNegInf};
      bool hidden = false;  // a key was loaded that one of the lane's rows does not see
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + 2 * c + (e & 1) + 8 * t;
          const bool in = vrow[2 * t + (e & 1)] >= 0;
          const bool see = in && sees(key, pos[e >> 1], window, sinks);
          hidden |= in && !see;
          s[t][e] = see ? s[t][e] * p.scale_log2 : kNegInf;
          most[e >> 1] = fmaxf(most[e >> 1], s[t][e]);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        most[i] = fmaxf(most[i], __shfl_xor_sync(~0u, most[i], 1));
        most[i] = fmaxf(most[i], __shfl_xor_sync(~0u, most[i], 2));
        most[i] = fmaxf(most[i], m[i]);
        const float f = m[i] == most[i] ? 1.f : exp2_fast(m[i] - most[i]);
        m[i] = most[i];
        l[i] *= f;
#pragma unroll
        for (int b = 0; b < VB; ++b)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[b][j][2 * i] *= f, acc[b][j][2 * i + 1] *= f;
      }
      float pr[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pr[t][e] = s[t][e] == kNegInf ? 0.f : exp2_fast(s[t][e] - m[e >> 1]);
          l[e >> 1] += pr[t][e];
        }
      // P is rounded to the pool's type for the matrix product, half a step of
      // it relative to each weight; the sum l is not.
      const uint32_t a[4] = {T::pack(pr[0][0], pr[0][1]), T::pack(pr[0][2], pr[0][3]),
                             T::pack(pr[1][0], pr[1][1]), T::pack(pr[1][2], pr[1][3])};
      // A weight of zero does not hide a value that is not finite.  Where rows of
      // several positions share such a value, each position takes the product
      // by itself, with the values it does not see put to zero.
      int steps = 1;
      if (__any_sync(~0u, hidden)) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int b = 0; b < VB; ++b)
            bad |= T::not_finite(vf[b][i].x) | T::not_finite(vf[b][i].y) |
                   T::not_finite(vf[b][i].z) | T::not_finite(vf[b][i].w);
        if (__any_sync(~0u, bad)) steps = tok1 - tok0 + 1;
      }
      if (steps > 1) {
        for (int i = 0; i < steps; ++i) {
          const int at = it.req.row0 + tok0 + i;
          uint32_t keep[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            keep[k] = sees(key0 + 2 * c + (k & 1) + 8 * (k >> 1), at, window, sinks) ? ~0u : 0u;
#pragma unroll
          for (int b = 0; b < VB; ++b)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
              const auto word = [&](int k) {
                return reinterpret_cast<const uint32_t*>(&vf[b][k])[j / 2] & keep[k];
              };
              float part[4] = {0.f, 0.f, 0.f, 0.f};
              T::mma(part, a, __byte_perm(word(0), word(1), sel),
                     __byte_perm(word(2), word(3), sel));
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (pos[e >> 1] == at) acc[b][j][e] += part[e];
            }
        }
        continue;
      }
#pragma unroll
      for (int b = 0; b < VB; ++b) {
        const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vf[b][0]);
        const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vf[b][1]);
        const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vf[b][2]);
        const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vf[b][3]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
          T::mma(acc[b][j], a, __byte_perm(v0[j / 2], v1[j / 2], sel),
                 __byte_perm(v2[j / 2], v3[j / 2], sel));
        }
      }
    }

    // Join the warps: sums over the quad, then the maximum over the warps.
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(~0u, l[i], 1);
      l[i] += __shfl_xor_sync(~0u, l[i], 2);
      if (c == 0) {
        stat_m[warp][g + 8 * i] = m[i];
        stat_l[warp][g + 8 * i] = l[i];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = kNegInf;
      for (int k = 0; k < kRowWarps; ++k) top = fmaxf(top, stat_m[k][g + 8 * i]);
      const float f = weight_of(m[i], top);
      // this lane has channels 64 b + 16 c + 0 .. 15 of its rows
      float* dst = smem + (warp * 16 + g + 8 * i) * (VB * 64) + 16 * c;
#pragma unroll
      for (int b = 0; b < VB; ++b)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dst[64 * b + j] = acc[b][j][2 * i] * f;
          dst[64 * b + 8 + j] = acc[b][j][2 * i + 1] * f;
        }
    }
    __syncthreads();
    // Thread: four channels of a row at a time.
    const int quads = D / 4;
    for (int i = threadIdx.x; i < it.rows * quads; i += kRowThreads) {
      const int row = i / quads, d = (i - row * quads) * 4;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < kRowWarps; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(smem + (k * 16 + row) * (VB * 64) + d);
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
      }
      float mm = kNegInf, ll = 0.f;
      for (int k = 0; k < kRowWarps; ++k) mm = fmaxf(mm, stat_m[k][row]);
      for (int k = 0; k < kRowWarps; ++k) ll += stat_l[k][row] * weight_of(stat_m[k][row], mm);
      const int tok = div_of(it.row + row, p.group_div);
      const int64_t t = it.req.first + tok;
      const int qh = head * p.group + it.row + row - tok * p.group;
      if (!w.whole) {
        const int64_t at = int64_t(w.piece) * kRowTile + row;
        *reinterpret_cast<float4*>(p.rows.pieces + at * D + d) = o;
        if (d == 0) p.rows.stats[at] = make_float2(mm, ll);
      } else if (p.shared) {
        const int64_t at = (int64_t(prefix) * p.num_tokens + t) * p.q_heads + qh;
        *reinterpret_cast<float4*>(p.whole + at * D + d) = o;
        if (d == 0) p.whole_stats[at] = make_float2(mm, ll);
      } else {
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        *reinterpret_cast<uint2*>(p.out + t * p.out_stride + int64_t(qh) * D + d) =
            make_uint2(T::pack(o.x * inv, o.y * inv), T::pack(o.z * inv, o.w * inv));
        if (d == 0 && p.lse != nullptr) p.lse[t * p.q_heads + qh] = log_sum(mm, ll);
      }
    }
    __syncthreads();  // smem is written again
  }
}

// Where the parts of one row of a line lie.
struct Part {
  int c0, c1, in_tile;  // CTAs that hold units of the row's item; the row in the tile
  int64_t item0, units, whole_at;
  int ctas;
  const Lane* lane;

  template <int kTile>
  __device__ void find(const AttnParams& p, const Lane& l, bool prefix, int request, int row,
                       int head) {
    lane = &l;
    const int x = (prefix ? own_slots<kTile>(p) : slot_base<kTile>(p, request)) + row / kTile;
    in_tile = row % kTile;
    const int64_t cost = l.cum[x + 1] - l.cum[x];
    units = l.cum[total_slots<kTile>(p)] * p.kv_heads;
    ctas = shares_of(l, units);
    item0 = l.cum[x] * p.kv_heads + head * cost;
    c0 = cta_of(item0, units, ctas);
    c1 = cta_of(item0 + cost - 1, units, ctas);
  }
  __device__ bool whole() const { return c0 == c1; }
  __device__ int64_t at(int cta) const {
    return int64_t(2 * cta + (item0 >= units * cta / ctas ? 1 : 0)) * lane->tile + in_tile;
  }
  __device__ float2 stat(const AttnParams& p, int cta) const {
    return whole() ? p.whole_stats[whole_at] : lane->stats[at(cta)];
  }
  __device__ const float* values(const AttnParams& p, int cta) const {
    return whole() ? p.whole + whole_at * p.dim : lane->pieces + at(cta) * p.dim;
  }
};

// One warp joins one (token, query head) row from its pieces.
template <typename T, int kDim>
__global__ void __launch_bounds__(256) join_kernel(AttnParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row_id = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row_id >= int64_t(p.num_tokens) * p.q_heads) return;
  const int t = int(row_id / p.q_heads), qh = int(row_id - int64_t(t) * p.q_heads);
  if (t >= p.q_starts[p.num_requests]) return;
  const int head = div_of(qh, p.group_div), member = qh - head * p.group;
  int lo = 0, hi = p.num_requests - 1;  // the last request that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.q_starts[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  Request req;
  if (!load_request(p, lo, req) || t < req.first || t >= req.first + req.tokens) return;

  const int D = p.dim;
  // the parts of the row: its own item's, and its prefix item's
  Part part[2];
  const int parts = p.shared ? 2 : 1;
  for (int k = 0; k < parts; ++k) {
    const int row = (k ? t : t - req.first) * p.group + member;
    const bool small = k ? p.prefix_small != 0 : req.tokens * p.group <= kRowTile;
    if (small) part[k].find<kRowTile>(p, p.rows, k != 0, lo, row, head);
    else if (kDim <= 128) part[k].find<256>(p, p.tiles, k != 0, lo, row, head);
    else part[k].find<128>(p, p.tiles, k != 0, lo, row, head);
    part[k].whole_at = int64_t(k) * p.num_tokens * p.q_heads + row_id;
  }
  if (!p.shared && part[0].whole()) return;  // written by the CTA that had all of it

  float mm = kNegInf;
  for (int k = 0; k < parts; ++k)
    for (int cta = part[k].c0; cta <= part[k].c1; ++cta) mm = fmaxf(mm, part[k].stat(p, cta).x);
  float ll = 0.f;
  float4 o[2];  // channels 4 * lane and 128 + 4 * lane
#pragma unroll
  for (int h = 0; h < 2; ++h) o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < parts; ++k)
    for (int cta = part[k].c0; cta <= part[k].c1; ++cta) {
      const float2 st = part[k].stat(p, cta);
      const float f = weight_of(st.x, mm);
      ll += st.y * f;
      const float* src = part[k].values(p, cta);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (128 * h + 4 * lane < D) {
          const float4 v = *reinterpret_cast<const float4*>(src + 128 * h + 4 * lane);
          o[h].x += v.x * f, o[h].y += v.y * f, o[h].z += v.z * f, o[h].w += v.w * f;
        }
    }
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (128 * h + 4 * lane < D)
      *reinterpret_cast<uint2*>(p.out + int64_t(t) * p.out_stride + int64_t(qh) * D + 128 * h +
                                4 * lane) =
          make_uint2(T::pack(o[h].x * inv, o[h].y * inv), T::pack(o[h].z * inv, o[h].w * inv));
  if (lane == 0 && p.lse != nullptr)
    p.lse[row_id] = log_sum(mm, ll);
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
  const uint64_t tile_ctas = tokens * group > kRowTile ? kMaxTileCtas : 0;
  const uint64_t rows = shared ? uint64_t(2) * tokens * Hq : 0;
  Workspace w;
  uint64_t at = 0;
  const auto take = [&at](uint64_t bytes) {
    const uint64_t here = at;
    at = up256(at + bytes);
    return here;
  };
  w.row_cum = take((row_slots + 1) * 8);
  w.row_pieces = take(uint64_t(2) * kMaxRowCtas * kRowTile * D * 4);
  w.row_stats = take(uint64_t(2) * kMaxRowCtas * kRowTile * 8);
  w.tile_cum = take((tile_slots + 1) * 8);
  w.tile_pieces = take(2 * tile_ctas * tile * D * 4);
  w.tile_stats = take(2 * tile_ctas * tile * 8);
  w.whole = take(rows * D * 4);
  w.whole_stats = take(rows * 8);
  w.total = at;
  return w;
}

template <typename T, int DB>
cudaError_t launch_rows(const AttnParams& p, cudaStream_t stream) {
  const int smem = kRowWarps * 16 * ((DB + 1) / 2) * 64 * 4;
  if (smem > 48 * 1024) {
    const cudaError_t err = cudaFuncSetAttribute(
        rows_kernel<T, DB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
  }
  rows_kernel<T, DB><<<p.rows.ctas, kRowThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(AttnParams& p, int sms, bool bf16, cudaStream_t stream) {
  p.rows.ctas = std::min(kMaxRowCtas, sms * (p.dim <= 128 ? 3 : 1));
  p.rows.tile = kRowTile;
  p.tiles.tile = tile_rows(p.dim);
  const bool tiles = p.tiled || (p.shared && !p.prefix_small);
  p.tiles.ctas = tiles ? std::min(kMaxTileCtas, sms) : 0;
  if (p.dim <= 128) plan_kernel<256, 128><<<tiles ? 2 : 1, 1024, 0, stream>>>(p);
  else plan_kernel<128, 64><<<tiles ? 2 : 1, 1024, 0, stream>>>(p);
  cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess && tiles) err = launch_tiles(p, bf16, stream);
  if (err == cudaSuccess)
    err = p.dim <= 64 ? launch_rows<T, 2>(p, stream)
                      : (p.dim <= 128 ? launch_rows<T, 4>(p, stream) : launch_rows<T, 8>(p, stream));
  if (err != cudaSuccess) return err;
  const int64_t rows = int64_t(p.num_tokens) * p.q_heads;
  const unsigned grid = unsigned((rows + 7) / 8);
  if (p.dim <= 128) join_kernel<T, 128><<<grid, 256, 0, stream>>>(p);
  else join_kernel<T, 256><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
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
  return a.dtype == CG_DTYPE_F16 ? launch_type<F16>(p, sms, false, stream)
                                 : launch_type<BF16>(p, sms, true, stream);
}

}  // namespace cg
