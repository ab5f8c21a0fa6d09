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

#include "attend.cuh"

namespace cg {
namespace {

constexpr int kRowTile = 16;   // query rows of an item (one matrix tile)
constexpr int kRowWarps = 4;
constexpr int kRowKeys = 16 * kRowWarps;  // keys of a unit
constexpr int kRowThreads = 32 * kRowWarps;
constexpr int kMaxRowCtas = 160 * 4;
constexpr float kNegInf = -__builtin_huge_valf();

struct Item {
  Request req;
  Span span;
  int row, rows;   // first row of the tile among the request's rows, rows in it
  int tokens0;     // first token of the tile
  bool prefix;
};

// Slots: request r's tiles start at slot floor(first row / 16) + r, which leaves
// room for every tile whatever the lengths; slots that hold no tile cost nothing.
__device__ __forceinline__ int num_slots(const AttnParams& p) {
  return int(int64_t(p.num_tokens) * p.group / kRowTile) + p.num_requests;
}

__device__ __forceinline__ int slot_base(const AttnParams& p, int r) {
  int a = p.q_starts[r];
  a = a < 0 ? 0 : (a > p.num_tokens ? p.num_tokens : a);
  return int(int64_t(a) * p.group / kRowTile) + r;
}

// Units of slot x (for each kv head); 0 where it holds no rows.
__device__ int slot_item(const AttnParams& p, int x, Item& it) {
  const int slots = num_slots(p);
  it.prefix = x >= slots;
  if (it.prefix) {
    int n = p.q_starts[p.num_requests];
    n = n < 0 ? 0 : (n > p.num_tokens ? p.num_tokens : n);
    it.req.first = 0;
    it.req.tokens = n;
    it.req.keys = p.prefix_tokens;
    it.req.row0 = p.prefix_tokens;  // every row stands behind the prefix
    it.row = (x - slots) * kRowTile;
  } else {
    int lo = 0, hi = p.num_requests - 1;  // the last request whose slots start at or before x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (slot_base(p, mid) <= x) lo = mid;
      else hi = mid - 1;
    }
    if (!load_request(p, lo, it.req)) {
      report(p.status, CG_ERR_MISMATCH);
      return 0;
    }
    it.row = (x - slot_base(p, lo)) * kRowTile;
  }
  const int rows = it.req.tokens * p.group;
  if (it.row < 0 || it.row >= rows) return 0;
  it.rows = rows - it.row < kRowTile ? rows - it.row : kRowTile;
  if (it.prefix) {
    it.span = span_of<kRowKeys>(p.prefix_tokens - 1, p.prefix_tokens - 1, 0, 0);
  } else {
    const int t0 = div_of(it.row, p.group_div), t1 = div_of(it.row + it.rows - 1, p.group_div);
    it.span = span_of<kRowKeys>(it.req.row0 + t0, it.req.row0 + t1, p.window, p.sinks);
  }
  // an item without a visible key still has its rows to write
  return it.span.units > 0 ? it.span.units : 1;
}

__device__ __forceinline__ int total_slots(const AttnParams& p) {
  return num_slots(p) +
         (p.shared ? int((int64_t(p.num_tokens) * p.group + kRowTile - 1) / kRowTile) : 0);
}

// Fill row_cum: units of one head before each slot.  One block.
__global__ void __launch_bounds__(1024) plan_kernel(AttnParams p) {
  __shared__ int64_t warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slots = total_slots(p);
  int64_t base = 0;
  for (int x0 = 0; x0 < slots; x0 += 1024) {
    const int x = x0 + threadIdx.x;
    Item it;
    int64_t own = x < slots ? slot_item(p, x, it) : 0, sum = own;
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
    if (x < slots) p.row_cum[x] = before;
    base += __shfl_sync(~0u, wi, 31);
    __syncthreads();
  }
  if (threadIdx.x == 0) p.row_cum[slots] = base;
}

// CTAs that get a share: no share is empty.
__device__ __forceinline__ int shares_of(const AttnParams& p, int64_t units) {
  return units < p.row_ctas ? int(units) : p.row_ctas;
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

// DB: 32-channel blocks of a head (K), VB: 64-channel blocks (V).
template <typename T, int DB>
__global__ void __launch_bounds__(kRowThreads, DB <= 4 ? 3 : 1) rows_kernel(AttnParams p) {
  constexpr int VB = (DB + 1) / 2;
  extern __shared__ float smem[];  // [kRowWarps][16][VB * 64] outputs
  __shared__ float stat_m[kRowWarps][16], stat_l[kRowWarps][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int slots = total_slots(p), H = p.kv_heads, D = p.dim;
  const int64_t per_head = p.row_cum[slots];
  const int64_t units = per_head * H;
  if (units == 0) return;
  const int ctas = shares_of(p, units);
  if (int(blockIdx.x) >= ctas) return;
  int64_t u = units * blockIdx.x / ctas;
  const int64_t u_end = units * (blockIdx.x + 1) / ctas;
  const int64_t share0 = u;

  int x = 0;  // the slot that holds unit u: the last one with H * row_cum[x] <= u
  {
    int hi = slots - 1;
    while (x < hi) {
      const int mid = (x + hi + 1) >> 1;
      if (p.row_cum[mid] * H <= u) x = mid;
      else hi = mid - 1;
    }
  }
  int64_t cum = p.row_cum[x];

  while (u < u_end && x < slots) {
    Item it;
    const int cost = slot_item(p, x, it);
    if (cost == 0 || u >= (cum + cost) * H) {
      cum += cost;
      ++x;
      continue;
    }
    const int head = int((u - cum * H) / cost);
    const int64_t item0 = cum * H + int64_t(head) * cost;
    const int first = int(u - item0);
    const int last = int((item0 + cost < u_end ? item0 + cost : u_end) - item0);
    const bool whole = first == 0 && last == cost;

    // The two query rows of this lane's quad and their positions.
    uint32_t qf[DB][2][4];
    int pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = it.row + g + 8 * i;
      const int tok = div_of(row, p.group_div);
      const bool real = g + 8 * i < it.rows;
      pos[i] = it.prefix ? it.req.keys : it.req.row0 + tok;
      const uint16_t* src = p.q + int64_t(it.req.first + tok) * p.q_stride +
                            int64_t(head * p.group + (row - tok * p.group)) * D;
#pragma unroll
      for (int b = 0; b < DB; ++b) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (real && 32 * b + 8 * c < D) v = *reinterpret_cast<const uint4*>(src + 32 * b + 8 * c);
        qf[b][0][i] = v.x;
        qf[b][0][2 + i] = v.y;
        qf[b][1][i] = v.z;
        qf[b][1][2 + i] = v.w;
      }
    }
    const int32_t* table = it.prefix ? p.prefix_table : nullptr;
    if (!it.prefix) {
      // the request of the slot: found again from its first row
      int lo = 0, hi = p.num_requests - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (slot_base(p, mid) <= x) lo = mid;
        else hi = mid - 1;
      }
      table = p.tables + int64_t(lo) * p.max_pages;
    }
    const uint16_t* kb = p.k_pool + int64_t(head) * D;
    const uint16_t* vb = p.v_pool + int64_t(head) * D;
    const int64_t step = int64_t(H) * D;
    const int window = it.prefix ? 0 : p.window, sinks = it.prefix ? 0 : p.sinks;
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

    for (int unit = first; unit < last && it.span.units > 0; ++unit) {
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
      for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, stat_m[w][g + 8 * i]);
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
    const int piece = 2 * int(blockIdx.x) + (item0 >= share0 ? 1 : 0);
    for (int i = threadIdx.x; i < it.rows * quads; i += kRowThreads) {
      const int row = i / quads, d = (i - row * quads) * 4;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < kRowWarps; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(smem + (w * 16 + row) * (VB * 64) + d);
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
      }
      float mm = kNegInf, ll = 0.f;
      for (int w = 0; w < kRowWarps; ++w) mm = fmaxf(mm, stat_m[w][row]);
      for (int w = 0; w < kRowWarps; ++w) ll += stat_l[w][row] * weight_of(stat_m[w][row], mm);
      const int tok = div_of(it.row + row, p.group_div);
      const int64_t t = it.req.first + tok;
      const int qh = head * p.group + it.row + row - tok * p.group;
      if (!whole) {
        *reinterpret_cast<float4*>(p.row_pieces + (int64_t(piece) * kRowTile + row) * D + d) = o;
        if (d == 0) p.row_stats[piece * kRowTile + row] = make_float2(mm, ll);
      } else if (p.shared) {
        const int64_t at = (int64_t(it.prefix) * p.num_tokens + t) * p.q_heads + qh;
        *reinterpret_cast<float4*>(p.whole + at * D + d) = o;
        if (d == 0) p.whole_stats[at] = make_float2(mm, ll);
      } else {
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        *reinterpret_cast<uint2*>(p.out + t * p.out_stride + int64_t(qh) * D + d) =
            make_uint2(T::pack(o.x * inv, o.y * inv), T::pack(o.z * inv, o.w * inv));
        if (d == 0 && p.lse != nullptr)
          p.lse[t * p.q_heads + qh] = ll == 0.f ? kNegInf : (mm + log2f(ll)) * 0.69314718056f;
      }
    }
    __syncthreads();  // smem is written again
    u = item0 + last;
  }
}

// One warp joins one (token, query head) row from its pieces.
template <typename T>
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

  const int slots = total_slots(p), H = p.kv_heads, D = p.dim;
  const int64_t units = p.row_cum[slots] * H;
  const int ctas = shares_of(p, units);
  // the pieces of the row's own item, and of its prefix item
  int c0[2] = {0, 0}, c1[2] = {-1, -1}, in_tile[2] = {0, 0};
  int64_t item0[2] = {0, 0};
  bool whole[2] = {false, false};
  for (int k = 0; k < (p.shared ? 2 : 1); ++k) {
    const int row = (k ? t : t - req.first) * p.group + member;
    const int x = (k ? num_slots(p) : slot_base(p, lo)) + row / kRowTile;
    in_tile[k] = row % kRowTile;
    const int64_t cost = p.row_cum[x + 1] - p.row_cum[x];
    item0[k] = p.row_cum[x] * H + head * cost;
    c0[k] = cta_of(item0[k], units, ctas);
    c1[k] = cta_of(item0[k] + cost - 1, units, ctas);
    whole[k] = c0[k] == c1[k];
  }
  if (!p.shared && whole[0]) return;  // written by the CTA that had all of it

  float mm = kNegInf;
  const auto at_piece = [&](int k, int cta) -> int64_t {
    const int64_t share0 = units * cta / ctas;
    return int64_t(2 * cta + (item0[k] >= share0 ? 1 : 0)) * kRowTile + in_tile[k];
  };
  const auto stat = [&](int k, int cta) -> float2 {
    return whole[k] ? p.whole_stats[int64_t(k) * p.num_tokens * p.q_heads + row_id]
                    : p.row_stats[at_piece(k, cta)];
  };
  for (int k = 0; k < 2; ++k)
    for (int cta = c0[k]; cta <= c1[k]; ++cta) mm = fmaxf(mm, stat(k, cta).x);
  float ll = 0.f;
  float4 o[2];  // channels 4 * lane and 128 + 4 * lane
#pragma unroll
  for (int h = 0; h < 2; ++h) o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < 2; ++k)
    for (int cta = c0[k]; cta <= c1[k]; ++cta) {
      const float2 st = stat(k, cta);
      const float f = weight_of(st.x, mm);
      ll += st.y * f;
      const float* src = whole[k] ? p.whole + (int64_t(k) * p.num_tokens * p.q_heads + row_id) * D
                                  : p.row_pieces + at_piece(k, cta) * D;
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
    p.lse[row_id] = ll == 0.f ? kNegInf : (mm + log2f(ll)) * 0.69314718056f;
}

uint64_t up256(uint64_t v) { return (v + 255) & ~uint64_t(255); }

struct Workspace {
  uint64_t row_cum, row_pieces, row_stats, whole, whole_stats, total;
};

Workspace workspace_of(const cg_shape& s, int Hq, int tokens, int requests, bool shared) {
  const uint64_t D = s.head_dim, group = Hq / s.num_kv_heads;
  const uint64_t slots = 2 * (tokens * group / kRowTile) + requests + 1;
  Workspace w;
  w.row_cum = 0;
  w.row_pieces = up256(w.row_cum + (slots + 1) * 8);
  w.row_stats = up256(w.row_pieces + uint64_t(2) * kMaxRowCtas * kRowTile * D * 4);
  w.whole = up256(w.row_stats + uint64_t(2) * kMaxRowCtas * kRowTile * 8);
  const uint64_t rows = shared ? uint64_t(2) * tokens * Hq : 0;
  w.whole_stats = up256(w.whole + rows * D * 4);
  w.total = up256(w.whole_stats + rows * 8);
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
  rows_kernel<T, DB><<<p.row_ctas, kRowThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(AttnParams& p, int sms, cudaStream_t stream) {
  p.row_ctas = std::min(kMaxRowCtas, sms * (p.dim <= 128 ? 3 : 1));
  plan_kernel<<<1, 1024, 0, stream>>>(p);
  cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess)
    err = p.dim <= 64 ? launch_rows<T, 2>(p, stream)
                      : (p.dim <= 128 ? launch_rows<T, 4>(p, stream) : launch_rows<T, 8>(p, stream));
  if (err != cudaSuccess) return err;
  const int64_t rows = int64_t(p.num_tokens) * p.q_heads;
  join_kernel<T><<<unsigned((rows + 7) / 8), 256, 0, stream>>>(p);
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
  p.scale_log2 = a.scale * 1.44269504089f;
  uint8_t* w = static_cast<uint8_t*>(a.workspace_dev);
  const Workspace ws = workspace_of(s, a.num_q_heads, a.num_tokens, a.num_requests, shared);
  p.row_cum = reinterpret_cast<int64_t*>(w + ws.row_cum);
  p.row_pieces = reinterpret_cast<float*>(w + ws.row_pieces);
  p.row_stats = reinterpret_cast<float2*>(w + ws.row_stats);
  p.whole = reinterpret_cast<float*>(w + ws.whole);
  p.whole_stats = reinterpret_cast<float2*>(w + ws.whole_stats);
  return a.dtype == CG_DTYPE_F16 ? launch_type<F16>(p, sms, stream)
                                 : launch_type<BF16>(p, sms, stream);
}

}  // namespace cg
