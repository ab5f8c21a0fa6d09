// attend_tile.cu -- attention over the paged pool as matrix products: chunks of
// query rows, and a shared prefix under the rows of a whole batch.
//
// One CTA an SM, its roles by warp:
//   warps 0-3, 4-7   softmax of query tile 0 and 1 (128 rows each, a row a
//                    thread): scores out of tensor memory, running maximum and
//                    sum, weights back into tensor memory; output of the item
//   warps 10, 11     K and V from the pages to shared memory (kv_loader.cuh)
//   warp 9           deals the items; queries to shared memory, as soon as the
//                    last product with the item's before has read them
//   warp 8           issues the products:
//                      S = Q K^T   both operands in shared memory
//                      O += P V    P in tensor memory, V along its channels
// The two query tiles take turns: while one's scores are in softmax the tensor
// cores work on the other's products.
//
// The running maximum m moves only when a score passes it by 2^8: until then
// weights up to 2^8 are in range of fp16 and bf16 alike, nothing is lost, and
// the output need not be read back from tensor memory to be rescaled.
#include "attend.cuh"
#include "kv_loader.cuh"

namespace cg {
namespace {

constexpr int kThreads = 384;  // up to 168 registers a thread; a softmax thread takes 150
constexpr int kMmaWarp = 8, kQueryWarp = 9, kLoadWarp = 10;
constexpr float kSlack = 8.f;  // log2 of how far a weight may pass one

template <int DC>
struct Geometry {
  static constexpr int kTiles = DC <= 2 ? 2 : 1;      // query tiles of 128 rows
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kKeys = DC <= 2 ? 128 : 64;    // keys of a unit
  static constexpr int kStages = 4;                   // K and V tiles in flight
  // Pairs j of 16 with (j & kPolynomial) == 4 go to exp2_pair: an eighth of a row
  // with up to 64 channels, a sixteenth beyond.  Two prompts of 8,192 tokens, 64
  // channels: 943 us, without any 977.  128 channels: 1,075, without 1,114, an
  // eighth or a quarter 1,060 to 1,086 (and 1,066 for the sixteenth beside them).
  static constexpr int kPolynomial = DC == 1 ? 7 : 15;
  static constexpr int kQBytes = 128 * 128;           // a 64-channel block of a query tile
  static constexpr int kBlock = kKeys * 128;          // a 64-channel block of a K or V tile
  static constexpr int kStage = DC * kBlock;
  // Output rows pass through shared memory on their way out, 64 bytes of each of a
  // warp's 32 rows at a time, so that four lanes write 64 bytes of a row and not
  // each lane 16 of its own: 148 requests of 64 tokens behind 64, an item an SM,
  // took 75.0 us instead of 85.3, one item 22.8 instead of 24.1.  Rows 80 bytes
  // apart: no bank conflicts.
  static constexpr int kPitch = 80, kOutBytes = 32 * kPitch;
  static constexpr int kOut = kTiles * DC * kQBytes + kStages * kStage;
  static constexpr int kSmem = kOut + 4 * kTiles * kOutBytes + 1024;
  // Tensor memory columns of scores, weights and outputs (of tile 1: kStep on).
  // Products are only sure to follow one another in order where their shapes
  // are alike, so the next scores may overwrite weights that a product still
  // reads only there: with 65 to 128 channels, where there is no room for both,
  // both products are made 128 x 128 (columns behind the channels are not
  // read).  Elsewhere the weights have columns of their own.
  static constexpr uint32_t kS = 0, kSStep = 128;
  static constexpr uint32_t kP = DC == 1 ? 256 : (DC == 2 ? 0 : 64);
  static constexpr uint32_t kPStep = DC == 1 ? 64 : 128;
  static constexpr uint32_t kO = DC == 1 ? 384 : 256;
  static constexpr uint32_t kOStep = DC == 1 ? 64 : 128;
};

struct Bars {
  uint32_t q_full, q_free, s_full, o_full;  // each the first of its two
  uint32_t p_full;                          // of the halves of each tile's weights
  uint32_t item_full, item_free;                    // of kItems
};

// One part of an item, as the query warp deals it to the softmax warps and the
// products; those have no registers to spare for the walk over the line.
constexpr int kItems = 4;
struct Deal {
  int first, last;             // units
  int sink_units, first_unit;  // of its span
  int rows, row;               // 0 rows: the share is done
  int token0, row0, request;   // first packed row of the request, its position, its number or -1
  int head, piece, whole;
};

// 2^x of two values without the special-function unit, for the few of a unit's
// weights that the multiply-add pipe has time for: n = round(x) by adding
// 1.5 * 2^23, a polynomial for 2^(x - n) on [-1/2, 1/2], n added to the exponent.
// The coefficients are the minimax ones of degree 5 for the relative error (Remez
// exchange), 2^-23.7, and 2^-22 as evaluated in fp32 -- what ex2.approx has.
// Below -126 the result runs out of exponent, as ex2.approx.ftz's does: at -127 and
// under it is one unit in the last place above zero, 2^-149, which rounds to a weight
// of zero in both types, so that the value of a hidden key (score -infinity) cannot
// show, however large.  (r is not negative at -127, so the exponent does not wrap.)
__device__ __forceinline__ float2 exp2_pair(float2 x) {
  const float2 magic = make_float2(12582912.f, 12582912.f);
  const float2 minus = make_float2(-12582912.f, -12582912.f);
  x = make_float2(fmaxf(x.x, -127.f), fmaxf(x.y, -127.f));
  const float2 t = add_pair(x, magic);
  const float2 n = add_pair(t, minus);
  const float2 r = fma_pair(n, make_float2(-1.f, -1.f), x);
  float2 y = make_float2(0.0013276472f, 0.0013276472f);
  y = fma_pair(y, r, make_float2(0.009675541f, 0.009675541f));
  y = fma_pair(y, r, make_float2(0.05550713f, 0.05550713f));
  y = fma_pair(y, r, make_float2(0.2402212f, 0.2402212f));
  y = fma_pair(y, r, make_float2(0.69314694f, 0.69314694f));
  y = fma_pair(y, r, make_float2(1.0000001f, 1.0000001f));
  return make_float2(__uint_as_float(__float_as_uint(y.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(y.y) + (__float_as_uint(t.y) << 23)));
}

// The lowest n bits.
__device__ __forceinline__ uint32_t below(int n) {
  return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u);
}

// A weight of zero does not hide an infinity or a NaN in the matrix product.  Of a
// warp's rows whose outputs are not finite (`odd` lanes; a lane's row stands at
// `pos`), those that a value which is not finite and which they do not see has met,
// a bit each: only these are computed again.  The others' own keys made them so,
// all rows behind one bad token perhaps.
template <typename T, int kKeys>
__device__ __forceinline__ uint32_t rows_met(const AttnParams& p, const Deal& it, int pos,
                                             bool odd) {
  const int lane = threadIdx.x & 31;
  const bool prefix = it.request < 0;
  const int32_t* table = prefix ? p.prefix_table : p.tables + int64_t(it.request) * p.max_pages;
  const int window = prefix ? 0 : p.window, sinks = prefix ? 0 : p.sinks;
  const int p0 = prefix ? it.row0 : it.row0 + div_of(it.row, p.group_div);
  const int p1 = prefix ? it.row0 : it.row0 + div_of(it.row + it.rows - 1, p.group_div);
  const Span span = span_of<kKeys>(p0, p1, window, sinks);  // outside of it zeros were loaded
  const int64_t step = int64_t(p.kv_heads) * p.dim;
  const int past = window == 0 ? 0 : int(max(0ll, (long long)pos - window + 1));
  bool met = false;
  for (int u = it.first; u < it.last; ++u) {
    const int key0 = unit_key<kKeys>(span, u), end = key0 + kKeys - 1;
    const bool whole = end <= pos && (window == 0 || pos - key0 < window || end < sinks);
    if (__all_sync(~0u, !odd || met || whole)) continue;
    for (int from = key0; from < key0 + kKeys; from += 32) {
      const int key = from + lane;
      const int at = key < span.hi && (key >= span.lo || key < span.sink_end)
                         ? pool_row(p, table, key)
                         : -1;
      bool bad = false;
      if (at >= 0) {
        const uint16_t* v = p.v_pool + at * step + int64_t(it.head) * p.dim;
#pragma unroll 4
        for (int d = 0; d < p.dim; d += 8) {
          const uint4 x = *reinterpret_cast<const uint4*>(v + d);
          bad |= T::not_finite(x.x) | T::not_finite(x.y) | T::not_finite(x.z) | T::not_finite(x.w);
        }
      }
      const uint32_t seen = below(pos + 1 - from) & (~below(past - from) | below(sinks - from));
      met |= (__ballot_sync(~0u, bad) & ~seen) != 0;
    }
  }
  return __ballot_sync(~0u, odd && met);
}

// Rows computed again by a warp from the definition, kRedo at a time, which share
// the loads of K and V: rows[i] of the item, at[i] its position.  A lane has a key's
// scores, and four channels of each row's output, 128 channels apart.  `beat` counts
// on, for those who wait meanwhile.  40 requests of 20,000 keys, 4 kv heads of 64
// under two, 120 rows of each head before a bad value: 84 ms; one at a time 114.
// Four take 62, but with registers that the usual way then spills (chunks 5 % longer).
constexpr int kRedo = 2;
template <typename T, int kKeys>
__device__ __forceinline__ void recompute_rows(const AttnParams& p, const Deal& it,
                                               const int (&rows)[kRedo], const int (&at)[kRedo],
                                               int* beat, float (&o)[kRedo][2][4],
                                               float (&m)[kRedo], float (&l)[kRedo]) {
  const int lane = threadIdx.x & 31, head = it.head;
  const bool prefix = it.request < 0;
  const int32_t* table = prefix ? p.prefix_table : p.tables + int64_t(it.request) * p.max_pages;
  const int window = prefix ? 0 : p.window, sinks = prefix ? 0 : p.sinks;
  const uint16_t* q[kRedo];
#pragma unroll
  for (int i = 0; i < kRedo; ++i) {
    const int tok = div_of(rows[i], p.group_div);
    q[i] = p.q + int64_t(it.token0 + tok) * p.q_stride +
           int64_t(head * p.group + rows[i] - tok * p.group) * p.dim;
    m[i] = kNegInf;
    l[i] = 0.f;  // of this lane's keys
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][h][e] = 0.f;
  }
  const int64_t step = int64_t(p.kv_heads) * p.dim;
  const auto eight = [](uint4 v, float2 (&f)[4]) {
    f[0] = T::unpack(v.x), f[1] = T::unpack(v.y), f[2] = T::unpack(v.z), f[3] = T::unpack(v.w);
  };
  for (int u = it.first; u < it.last; ++u) {
    const int unit = u < it.sink_units ? u : it.first_unit + u - it.sink_units;
    for (int k0 = 0; k0 < kKeys; k0 += 32) {
      const int key = unit * kKeys + k0 + lane;
      bool any = false;
#pragma unroll
      for (int i = 0; i < kRedo; ++i) any |= sees(key, at[i], window, sinks);
      const int from = any ? pool_row(p, table, key) : -1;
      if (__all_sync(~0u, from < 0)) continue;
      float s[kRedo], w[kRedo];
#pragma unroll
      for (int i = 0; i < kRedo; ++i) s[i] = 0.f;
      if (from >= 0) {
        const uint16_t* k = p.k_pool + from * step + int64_t(head) * p.dim;
#pragma unroll 2
        for (int d = 0; d < p.dim; d += 8) {
          float2 a[4], b[4];
          eight(*reinterpret_cast<const uint4*>(k + d), b);
#pragma unroll
          for (int i = 0; i < kRedo; ++i) {
            uint4 x = *reinterpret_cast<const uint4*>(q[i] + d);
            x.x ^= p.q_flip, x.y ^= p.q_flip, x.z ^= p.q_flip, x.w ^= p.q_flip;
            eight(x, a);
#pragma unroll
            for (int c = 0; c < 4; ++c) s[i] = fmaf(a[c].x, b[c].x, fmaf(a[c].y, b[c].y, s[i]));
          }
        }
      }
      uint32_t seen[kRedo];
#pragma unroll
      for (int i = 0; i < kRedo; ++i) {
        const bool mine = from >= 0 && sees(key, at[i], window, sinks);
        seen[i] = __ballot_sync(~0u, mine);
        s[i] = mine ? s[i] * p.scale_log2 : kNegInf;
        float top = s[i];
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
        top = fmaxf(top, m[i]);
        const float f = weight_of(m[i], top);
        m[i] = top;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][h][e] *= f;
        w[i] = s[i] == kNegInf ? 0.f : exp2_fast(s[i] - top);
        l[i] = l[i] * f + w[i];
      }
#pragma unroll 1
      for (int j0 = 0; j0 < 32; j0 += 4) {
        uint2 x[4][2];  // the values of four keys on their way together
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int src = __shfl_sync(~0u, from, j0 + j);
          const uint16_t* v = p.v_pool + src * step + int64_t(head) * p.dim + 4 * lane;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            x[j][h] = make_uint2(0, 0);
            if (src >= 0 && 128 * h + 4 * lane < p.dim)
              x[j][h] = *reinterpret_cast<const uint2*>(v + 128 * h);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < kRedo; ++i) {
            const float wj = __shfl_sync(~0u, w[i], j0 + j);
            if (!((seen[i] >> (j0 + j)) & 1)) continue;  // the same for the whole warp
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (128 * h >= p.dim) break;
              const float2 a = T::unpack(x[j][h].x), b = T::unpack(x[j][h].y);
              o[i][h][0] = fmaf(wj, a.x, o[i][h][0]);
              o[i][h][1] = fmaf(wj, a.y, o[i][h][1]);
              o[i][h][2] = fmaf(wj, b.x, o[i][h][2]);
              o[i][h][3] = fmaf(wj, b.y, o[i][h][3]);
            }
          }
      }
      if (lane == 0) atomicAdd(beat, 1);
    }
  }
#pragma unroll
  for (int i = 0; i < kRedo; ++i)
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l[i] += __shfl_xor_sync(~0u, l[i], x);
}

// Of a warp's 32 rows from `first` on, those named in `maybe`: see rows_met.  Not
// inlined: the few registers and instructions of the usual way stay together.
template <typename T, int kRows, int kKeys>
__device__ __noinline__ void redo_rows(const AttnParams& p, const Deal& it, int first,
                                       uint32_t maybe, int* beat) {
  const int lane = threadIdx.x & 31, D = p.dim;
  const bool prefix = it.request < 0, direct = it.whole && !p.shared;
  const int mine = it.row + min(first + lane, it.rows - 1);
  const int pos = prefix ? it.row0 : it.row0 + div_of(mine, p.group_div);
  uint32_t again = rows_met<T, kKeys>(p, it, pos, (maybe >> lane) & 1);
  __syncwarp();  // what other lanes have stored of these rows comes before
  while (again) {
    int rows[kRedo], at[kRedo];
    uint32_t here = 0;  // which of them there are
#pragma unroll
    for (int i = 0; i < kRedo; ++i) {
      rows[i] = i > 0 && again == 0 ? rows[0] : it.row + first + __ffs(again) - 1;
      at[i] = prefix ? it.row0 : it.row0 + div_of(rows[i], p.group_div);
      if (again != 0) here |= 1u << i;
      again &= again - 1;
    }
    float o[kRedo][2][4], m[kRedo], l[kRedo];
    recompute_rows<T, kKeys>(p, it, rows, at, beat, o, m, l);
#pragma unroll
    for (int i = 0; i < kRedo; ++i) {
      if (!((here >> i) & 1)) continue;
      const int tok = div_of(rows[i], p.group_div);
      const int64_t t = it.token0 + tok;
      const int qh = it.head * p.group + rows[i] - tok * p.group;
      const int64_t piece = int64_t(it.piece) * kRows + rows[i] - it.row;
      const int64_t whole = (int64_t(prefix) * p.num_tokens + t) * p.q_heads + qh;
      const float scale = direct ? (l[i] == 0.f ? 0.f : 1.f / l[i]) : 1.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int d = 128 * h + 4 * lane;
        if (d >= D) continue;
        const float(&v)[4] = o[i][h];
        if (direct)
          *reinterpret_cast<uint2*>(p.out + t * p.out_stride + int64_t(qh) * D + d) = make_uint2(
              T::pack(v[0] * scale, v[1] * scale), T::pack(v[2] * scale, v[3] * scale));
        else
          *reinterpret_cast<float4*>(
              (it.whole ? p.whole + whole * D : p.tiles.pieces + piece * D) + d) =
              make_float4(v[0], v[1], v[2], v[3]);
      }
      if (lane == 0) {
        if (!direct)
          (it.whole ? p.whole_stats[whole] : p.tiles.stats[piece]) = make_float2(m[i], l[i]);
        else if (p.lse != nullptr)
          p.lse[t * p.q_heads + qh] = log_sum(m[i], l[i]);
      }
    }
  }
  __syncwarp();
}

template <typename T, int DC>
__global__ void __launch_bounds__(kThreads, 1)
    tile_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ KvMaps maps,
                const __grid_constant__ CUtensorMap q_map, int by_map) {
  using G = Geometry<DC>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars_mem[2 * G::kStages + 12 + 2 * kItems];
  __shared__ Deal deals[kItems];
  __shared__ uint32_t tmem_slot;
  __shared__ int dead_mem[2];
  __shared__ __align__(16) uint32_t no_page[kNoted][4];
  const int warp = __shfl_sync(~0u, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t q_smem = base;
  const uint32_t kv_smem = base + G::kTiles * DC * G::kQBytes;
  volatile int* dead = dead_mem;
  const uint32_t bars = smem_addr(bars_mem);
  const Ring ring{kv_smem, bars, bars + 8 * G::kStages, no_page, dead_mem};
  Bars bar;
  bar.q_full = ring.empty + 8 * G::kStages;
  bar.q_free = bar.q_full + 16;
  bar.s_full = bar.q_free + 16;
  bar.p_full = bar.s_full + 16;
  bar.o_full = bar.p_full + 32;
  bar.item_full = bar.o_full + 16;
  bar.item_free = bar.item_full + 8 * kItems;

  let_next_start();
  if (threadIdx.x == 32 * kLoadWarp && maps.box > 0) {
    prefetch_map(&maps.k);
    prefetch_map(&maps.v);
  }
  if (threadIdx.x == 32 * kQueryWarp && by_map) prefetch_map(&q_map);
  if (threadIdx.x == 0) {
    dead_mem[0] = dead_mem[1] = 0;
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(ring.full + 8 * i, kLoadWarps);
      mbar_init(ring.empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar.q_full + 8 * i, 1);
      mbar_init(bar.q_free + 8 * i, 1);
      mbar_init(bar.s_full + 8 * i, 1);
      mbar_init(bar.p_full + 16 * i, 4);
      mbar_init(bar.p_full + 16 * i + 8, 4);
      mbar_init(bar.o_full + 8 * i, 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar.item_full + 8 * i, 1);
      mbar_init(bar.item_free + 8 * i, 4 * G::kTiles + 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&tmem_slot), 512);
  Walk<G::kRows, G::kKeys> w;
  const bool any = w.begin(p, p.tiles, reinterpret_cast<int64_t*>(smem_raw));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, tmem_slot, 0);
  const int D = p.dim;

  if (warp < 8) {
    const int tile = warp >> 2;
    const int r = threadIdx.x & 127;  // row in the tile, lane of tensor memory
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + lanes + G::kS + tile * G::kSStep;
    const uint32_t t_p = tmem + lanes + G::kP + tile * G::kPStep;
    const uint32_t t_o = tmem + lanes + G::kO + tile * G::kOStep;
    uint32_t s_phase = 0, o_phase = 0, unit_count = 0;
    bool ok = any && tile < G::kTiles;
    for (uint32_t n = 0; ok; ++n) {
      const Deal& it = deals[n % kItems];
      if (!(ok = mbar_wait(bar.item_full + 8 * (n % kItems), (n / kItems) & 1, dead))) break;
      if (it.rows == 0) break;
      const int first = it.first, last = it.last;
      const int sink_units = it.sink_units, key_shift = (it.first_unit - it.sink_units) * G::kKeys;
      if (it.rows <= 128 * tile) {  // no rows in this tile
        unit_count += last - first;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.item_free + 8 * (n % kItems));
        continue;
      }
      const bool real = 128 * tile + r < it.rows;
      const bool prefix = it.request < 0;
      const int row = it.row + (real ? 128 * tile + r : it.rows - 1);
      const int pos = prefix ? it.row0 : it.row0 + div_of(row, p.group_div);
      const int window = prefix ? 0 : p.window, sinks = prefix ? 0 : p.sinks;
      float m = kNegInf, l = 0.f;
      bool mixed = false;  // some unit had keys that a row does not see
      for (int u = first; u < last; ++u, ++unit_count) {
        const int key0 = u * G::kKeys + (u < sink_units ? 0 : key_shift);
        // the whole unit is seen by the row, or its keys are hidden one by one
        const int end = key0 + G::kKeys - 1;
        const bool full = __all_sync(
            ~0u, end <= pos && (window == 0 || pos - key0 < window || end < sinks));
        if (!(ok = mbar_wait(bar.s_full + 8 * tile, s_phase, dead))) break;
        s_phase ^= 1;
        tc_fence_after();
        const uint32_t* hole = no_page[unit_count % kNoted];
        uint32_t holes = 0;
#pragma unroll
        for (int i = 0; i < G::kKeys / 32; ++i) holes |= hole[i];
        const bool hide = !full || holes != 0;
        mixed |= hide;
        // keys before `past` are behind the window
        const int past = window == 0 ? 0 : int(max(0ll, (long long)pos - window + 1));
        // 64 scores at a time, twice: first the maximum, then the weights.  Loops, and
        // the scores read again, rather than a row's 128 in registers and all of it
        // unrolled: the first pass over more instructions costs a short item more
        // than the second load.  148 requests of 64 tokens behind 64: 75.5 us against
        // 87.9; two prompts of 8,192 tokens: 1,015 against 1,036, with 64 channels 890
        // against 871.  32 at a time wait for twice as many loads: 75.3, 1,060, 915.
        uint32_t raw[64];
        const auto scores = [&](int i) {
          tmem_load64(t_s + 64 * i, raw);
          if (hide) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int from = key0 + 64 * i + 32 * w;
              const uint32_t seen = below(pos + 1 - from) &
                                    (~below(past - from) | below(sinks - from)) & ~hole[2 * i + w];
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((seen >> j) & 1)) raw[32 * w + j] = __float_as_uint(kNegInf);
            }
          }
        };
        float top[2] = {kNegInf, kNegInf};  // NaN if any score is
#pragma unroll 1
        for (int i = 0; i < G::kKeys / 64; ++i) {
          scores(i);
#pragma unroll
          for (int j = 0; j < 64; j += 4) {
            top[0] = max3_nan(top[0], __uint_as_float(raw[j]), __uint_as_float(raw[j + 1]));
            top[1] = max3_nan(top[1], __uint_as_float(raw[j + 2]), __uint_as_float(raw[j + 3]));
          }
        }
        const float most = max3_nan(top[0], top[1], kNegInf) * p.scale_log2;
        const bool move = !(most <= m + kSlack);
        if (__any_sync(~0u, move)) {
          const float next = move ? max3_nan(m, most, kNegInf) : m;
          const float f = m == next ? 1.f : exp2_fast(m - next);
          m = next;
          l *= f;
          if (u > first) {
            // the products into O so far are done: S came after them
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_load16(t_o + c, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_store16(t_o + c, o);
            }
          }
        }
        // NaN for a maximum that is not finite: the polynomial would not show it
        const float shift = m == kNegInf ? 0.f : (m - m) - m;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
        const float2 shift2 = make_float2(shift, shift);
        // By halves of the unit, so that the product with the first half's values
        // runs while the second half is computed.
#pragma unroll 1
        for (int i = 0; i < G::kKeys / 64; ++i) {
          scores(i);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            uint32_t weights[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 x = fma_pair(make_float2(__uint_as_float(raw[32 * w + 2 * j]),
                                                    __uint_as_float(raw[32 * w + 2 * j + 1])),
                                        scale2, shift2);
              // a few on the multiply-add pipe: see exp2_pair
              const float2 e = (j & G::kPolynomial) == 4
                                   ? exp2_pair(x)
                                   : make_float2(exp2_fast(x.x), exp2_fast(x.y));
              sum[j & 1] = add_pair(sum[j & 1], e);
              // rounded to the pool's type for the product with V: half a step of it
              // relative to each weight; the sum is not
              weights[j] = T::pack(e.x, e.y);
            }
            // (where the weights take their scores' place, it is one already read)
            tmem_store16(t_p + 32 * i + 16 * w, weights);
          }
          constexpr int kHalves = 128 / G::kKeys;  // of the unit in 64 scores
          tmem_store_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0)
            for (int h = i * kHalves; h < (i + 1) * kHalves; ++h)
              mbar_arrive(bar.p_full + 8 * (2 * tile + h));
        }
        // nothing seen so far: exp2_pair leaves 2^-149 where the weight is zero
        l = m == kNegInf ? 0.f : l + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
      }
      if (!ok) break;
      // ---- the rows' output
      const bool none = first >= last;
      if (!none) {
        if (!(ok = mbar_wait(bar.o_full + 8 * tile, o_phase, dead))) break;
        o_phase ^= 1;
        tc_fence_after();
      }
      const int tok = div_of(row, p.group_div);
      const int64_t t = it.token0 + tok;
      const int qh = it.head * p.group + row - tok * p.group;
      const bool direct = it.whole && !p.shared;
      const int64_t piece = int64_t(it.piece) * G::kRows + 128 * tile + r;
      const int64_t whole = (int64_t(prefix) * p.num_tokens + t) * p.q_heads + qh;
      char* const mine =
          !real    ? nullptr
          : direct ? reinterpret_cast<char*>(p.out + t * p.out_stride + int64_t(qh) * D)
          : it.whole ? reinterpret_cast<char*>(p.whole + whole * D)
                     : reinterpret_cast<char*>(p.tiles.pieces + piece * D);
      // this lane stores 16 bytes of rows 8 i + lane / 4
      char* rows[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        rows[i] = reinterpret_cast<char*>(
                      __shfl_sync(~0u, reinterpret_cast<unsigned long long>(mine), 8 * i + (lane >> 2)));
      const uint32_t pass = base + G::kOut + warp * G::kOutBytes;
      const uint32_t give = pass + lane * G::kPitch, take = pass + (lane >> 2) * G::kPitch + 16 * (lane & 3);
      // 64 bytes of each row through shared memory, `bytes` of them the row's
      const auto put = [&](const uint32_t (&words)[16], int offset, int bytes) {
#pragma unroll
        for (int k = 0; k < 4; ++k) st_shared16(give + 16 * k, words + 4 * k);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = ld_shared16(take + 8 * i * G::kPitch);
          if (rows[i] != nullptr && 16 * (lane & 3) < bytes)
            *reinterpret_cast<uint4*>(rows[i] + offset + 16 * (lane & 3)) = v;
        }
        __syncwarp();
      };
      float2 odd2 = make_float2(l - l, 0.f);  // NaN once a sum is not finite
      const float2 zero2 = make_float2(0.f, 0.f);
      uint32_t words[16];
      if (direct) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float2 inv2 = make_float2(inv, inv);
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (none) {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0;
          } else {
            tmem_load32(t_o + c, o);  // past the channels, where those are no multiple of 32
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 v = make_float2(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1]));
            if (j < 8 || c + 16 < D) odd2 = fma_pair(v, zero2, odd2);
            const float2 y = fma_pair(v, inv2, zero2);
            words[j] = T::pack(y.x, y.y);
          }
          put(words, 2 * c, 2 * (D - c));
        }
      } else {
        for (int c = 0; c < D; c += 16) {
          if (none) {
#pragma unroll
            for (int j = 0; j < 16; ++j) words[j] = 0;
          } else {
            tmem_load16(t_o + c, words);
          }
#pragma unroll
          for (int j = 0; j < 16; j += 2)
            odd2 = fma_pair(make_float2(__uint_as_float(words[j]), __uint_as_float(words[j + 1])),
                            zero2, odd2);
          put(words, 4 * c, 64);
        }
      }
      const bool odd = !(odd2.x + odd2.y == 0.f);
      if (real) {
        if (!direct) (it.whole ? p.whole_stats[whole] : p.tiles.stats[piece]) = make_float2(m, l);
        else if (p.lse != nullptr) p.lse[t * p.q_heads + qh] = log_sum(m, l);
      }
      // rows whose outputs are not finite, where some keys were hidden (a sum of weights
      // that is not finite makes all of the row so, and comes of keys that it sees)
      const uint32_t maybe = __ballot_sync(~0u, real && mixed && odd && l - l == 0.f);
      if (maybe != 0)
        redo_rows<T, G::kRows, G::kKeys>(p, it, 128 * tile + 32 * (warp & 3), maybe, dead_mem + 1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.item_free + 8 * (n % kItems));
    }
    if (!ok && any && tile < G::kTiles && lane == 0) report(p.status, CG_ERR_CUDA);
  } else {
    if (warp >= kLoadWarp) {
      if (any)
        load_kv<DC, G::kRows, G::kKeys, G::kStages>(p, w, ring, &maps.k, &maps.v, maps.box,
                                                    warp - kLoadWarp);
    } else if (warp == kQueryWarp) {
      // ---- queries
      uint32_t q_phase = 3;  // a bit for each query tile
      bool ok = any;
      if (!any && lane == 0) w.note_cut(p.tiles, false);
      const auto deal = [&](uint32_t n, bool more) {
        if (!mbar_wait(bar.item_free + 8 * (n % kItems), ((n / kItems) & 1) ^ 1, dead)) return false;
        if (lane == 0) {
          const Item& it = w.it;
          deals[n % kItems] = Deal{w.first, max(w.first, w.last), it.span.sink_units,
                                   it.span.first_unit, more ? it.rows : 0, it.row, it.req.first,
                                   it.req.row0, it.request, w.head, w.piece, w.whole};
          mbar_arrive(bar.item_full + 8 * (n % kItems));
        }
        __syncwarp();
        return true;
      };
      bool more = ok && w.next(p);
      if (ok && lane == 0) w.note_cut(p.tiles, more);
      ok = ok && deal(0, more);
      // an item is dealt before the queries of the one before it are waited for
      for (uint32_t n = 1; ok && more; ++n) {
        const int rows = w.it.rows, row = w.it.row, token0 = w.it.req.first;
        const int first_head = w.head * p.group;
        const bool none = w.first >= w.last;
        more = w.next(p);
        if (!(ok = deal(n, more))) break;
        if (none) continue;
        for (int tile = 0; tile < (rows > 128 ? 2 : 1); ++tile) {
          if (!(ok = mbar_wait(bar.q_free + 8 * tile, (q_phase >> tile) & 1, dead))) break;
          q_phase ^= 1u << tile;
          const uint32_t dst = q_smem + tile * DC * G::kQBytes;
          const int row0 = row + 128 * tile;
          if (by_map) {
            // rows behind the item's are other tokens' or zeros, and are not used
            mbar_expect(bar.q_full + 8 * tile, DC * G::kQBytes);
            const int head = __shfl_sync(~0u, first_head, 0);
            const int token = __shfl_sync(~0u, token0 + div_of(row0, p.group_div), 0);
            for (int b = 0; b < DC; ++b)
              tma_load3(dst + b * G::kQBytes, &q_map, 64 * b, head, token, bar.q_full + 8 * tile);
            continue;
          }
#pragma unroll 4
          for (int i = 0; i < 128; i += 4) {  // eight lanes a row
            const int r = i + (lane >> 3), c = lane & 7, at = row0 + r;
            const int tok = div_of(at, p.group_div);
            const uint16_t* src = p.q + int64_t(token0 + tok) * p.q_stride +
                                  int64_t(first_head + at - tok * p.group) * D + 8 * c;
#pragma unroll
            for (int b = 0; b < DC; ++b) {
              uint4 v = make_uint4(0, 0, 0, 0);
              if (128 * tile + r < rows && 64 * b + 8 * c < D)
                v = *reinterpret_cast<const uint4*>(src + 64 * b);
              v.x ^= p.q_flip, v.y ^= p.q_flip, v.z ^= p.q_flip, v.w ^= p.q_flip;
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                               dst + b * G::kQBytes + r * 128 + ((c ^ (r & 7)) << 4)),
                           "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                           : "memory");
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar.q_full + 8 * tile);
        }
      }
    } else if (warp == kMmaWarp) {
      // ---- the products
      constexpr bool kBf16 = T::kBf16;
      const uint32_t qk = mma_desc(kBf16, false, 128, G::kKeys);
      const uint32_t pv = mma_desc(kBf16, true, 128, DC == 2 ? 128 : D);
      uint32_t stage = 0, phase = 0, q_phase = 0, p_phase = 0;  // a bit for each query tile
      bool ok = __shfl_sync(~0u, any, 0);
      const auto wait = [&](uint32_t b, uint32_t parity) {
        return __all_sync(~0u, mbar_wait(b, parity, dead)) != 0;
      };
      const auto step = [&]() {
        if (++stage == G::kStages) stage = 0, phase ^= 1;
      };
      // operand descriptors of stage and tile 0; others are a 16-byte count away
      const uint64_t q_desc = smem_desc(q_smem, 16, 1024);
      const uint64_t k_desc = smem_desc(kv_smem, 16, 1024);
      const uint64_t v_desc = smem_desc(kv_smem, G::kBlock, 1024);
      const auto scores = [&](int tile, uint32_t at, bool final) {
        const uint32_t dst = tmem + G::kS + tile * G::kSStep;
        const uint64_t a = q_desc + tile * (DC * G::kQBytes >> 4);
        const uint64_t b = k_desc + at * (G::kStage >> 4);
#pragma unroll 1
        for (int c = 0; 64 * c < D; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (64 * c + 16 * k < D)
              mma_ss(dst, a + c * (G::kQBytes >> 4) + 2 * k, b + c * (G::kBlock >> 4) + 2 * k, qk,
                     c > 0 || k > 0);
        mma_commit(bar.s_full + 8 * tile);
        if (final) mma_commit(bar.q_free + 8 * tile);
      };
      const auto outputs = [&](int tile, uint32_t at, int half, bool add) {
        const uint32_t dst = tmem + G::kO + tile * G::kOStep;
        const uint32_t a = tmem + G::kP + tile * G::kPStep + half * (G::kKeys / 4);
        const uint64_t b = v_desc + at * (G::kStage >> 4) + half * (G::kKeys / 2 * 128 >> 4);
#pragma unroll
        for (int k = 0; k < G::kKeys / 32; ++k)
          mma_ts(dst, a + 8 * k, b + (k * 2048 >> 4), pv, k > 0 || add);
      };
      for (uint32_t n = 0; ok; ++n) {
        const Deal& it = deals[n % kItems];
        if (!(ok = wait(bar.item_full + 8 * (n % kItems), (n / kItems) & 1))) break;
        // from lane 0: the same in all lanes, as the compiler can see
        const int rows = __shfl_sync(~0u, it.rows, 0);
        const int first = __shfl_sync(~0u, it.first, 0), last = __shfl_sync(~0u, it.last, 0);
        if (lane == 0) mbar_arrive(bar.item_free + 8 * (n % kItems));
        if (rows == 0) break;
        const int active = rows > 128 ? 2 : 1;
        if (first >= last) continue;
        if (!(ok = wait(ring.full + 8 * stage, phase))) break;
        uint32_t k_stage = stage;
        step();
        for (int tile = 0; tile < active; ++tile) {
          if (!(ok = wait(bar.q_full + 8 * tile, (q_phase >> tile) & 1))) break;
          q_phase ^= 1u << tile;
          tc_fence_after();
          scores(tile, k_stage, first + 1 == last);
        }
        if (!ok) break;
        mma_commit(ring.empty + 8 * k_stage);
        for (int u = first; ok && u < last; ++u) {
          const bool more = u + 1 < last;
          if (!(ok = wait(ring.full + 8 * stage, phase))) break;
          const uint32_t v_stage = stage;
          step();
          if (more) {
            if (!(ok = wait(ring.full + 8 * stage, phase))) break;
            k_stage = stage;
            step();
          }
          for (int tile = 0; tile < active; ++tile) {
            if (!(ok = wait(bar.p_full + 16 * tile, (p_phase >> tile) & 1))) break;
            tc_fence_after();
            outputs(tile, v_stage, 0, u > first);
            if (!(ok = wait(bar.p_full + 16 * tile + 8, (p_phase >> tile) & 1))) break;
            p_phase ^= 1u << tile;
            tc_fence_after();
            outputs(tile, v_stage, 1, true);
            if (tile + 1 == active) mma_commit(ring.empty + 8 * v_stage);
            if (more) scores(tile, k_stage, u + 2 == last);
            else mma_commit(bar.o_full + 8 * tile);
          }
          if (!ok) break;
          if (more) mma_commit(ring.empty + 8 * k_stage);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  let_settle(dead);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

template <typename T, int DC>
cudaError_t launch(const AttnParams& p, cudaStream_t stream) {
  using G = Geometry<DC>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t err = allow_smem(tile_kernel<T, DC>, G::kSmem, done);
  if (err != cudaSuccess) return err;
  CUtensorMap q_map{};
  const int by_map = query_map(&q_map, p, T::kBf16);
  tile_kernel<T, DC><<<p.tiles.ctas, kThreads, G::kSmem, stream>>>(
      p, kv_maps(p, G::kKeys / kLoadWarps, T::kBf16), q_map, by_map);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const AttnParams& p, cudaStream_t stream) {
  if (p.dim <= 64) return launch<T, 1>(p, stream);
  if (p.dim <= 128) return launch<T, 2>(p, stream);
  return launch<T, 4>(p, stream);
}

}  // namespace

int tile_rows(int dim) { return dim <= 128 ? Geometry<2>::kRows : Geometry<4>::kRows; }

cudaError_t launch_tiles(const AttnParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_type<BF16>(p, stream) : launch_type<F16>(p, stream);
}

}  // namespace cg
