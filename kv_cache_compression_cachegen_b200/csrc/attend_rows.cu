// attend_rows.cu -- attention over the paged pool for few query rows a kv head:
// single tokens with the heads of a group, a few tokens at most.
//
//     o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),   s_j = (q . k_j) scale log2(e)
//
// in one pass over the keys with a running maximum m.  A row of K and V serves
// at most 16 query rows, so the bytes of K and V bound it, and all that counts
// is that enough of them are on their way: two CTAs an SM, whose rings of stages
// (kv_loader.cuh) take most of the shared memory, 96 KB each; while one is at the
// end of an item the other reads on.  Four warps read a CTA's
// stages, 16 keys of each unit a warp, with the matrix instructions of
// a warp (the tensor-memory products want 128 rows).  The keys, and then the
// channels, are the 16 rows of those, the query rows their 8 columns,
//     S^T = K Q^T,   O^T = V^T P^T,
// so that up to eight query rows take one product and not a half-empty larger
// one: an m16n8k16 holds an SM's quarter for 32 cycles, and two products for
// each would take longer than the bytes.  Each warp keeps a maximum, sums and
// outputs of its own, joined once an item.
#include <algorithm>

#include "attend.cuh"
#include "kv_loader.cuh"

namespace cg {
namespace {

constexpr int kWarps = 4;  // that compute
constexpr int kThreads = 32 * (kWarps + kLoadWarps);
constexpr int kJoinBytes = 8704;
constexpr float kSlack = 8.f;  // log2 of how far a weight may pass one
static_assert(kRowKeys == 16 * kWarps, "each warp takes 16 keys of a unit");
static_assert(kJoinBytes >= (kScanSlots + 1) * 8, "the line's sums lie there at first");

template <int DC, int NR>
struct Shape {
  // Two CTAs an SM, but one where sixteen rows have more than 128 channels: 168
  // registers a thread hold neither those rows' sums nor their queries.  14 requests
  // of 113 keys, 32 kv heads of 256 under 16 rows each: 70 us against 91 with two;
  // of 5,001 keys 823 against 1,083.  (Sixteen rows of 65 to 128 channels spill 150
  // bytes at two CTAs, and more than 128 channels 72 at eight rows and 322 at sixteen.)
  static constexpr int kCtasPerSm = row_ctas_per_sm(64 * DC, 8 * NR);
  static constexpr int kStages = (DC == 4 ? 3 : (DC == 2 ? 6 : 12)) * kRowCtasPerSm / kCtasPerSm;
  static constexpr int kStage = DC * kRowKeys * 128;
  // a row of a warp's output for the join: four channels more, so that the four
  // rows that a store touches fall on different banks
  static constexpr int kPitch = 64 * DC + 4;
  static constexpr int kJoinRows = kJoinBytes / (kWarps * kPitch * 4) >= 4 ? 4 : 2;
  static constexpr int kSmem = kStages * kStage + kJoinBytes + 1024;
  static_assert(kJoinRows * kWarps * kPitch * 4 <= kJoinBytes, "");
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// The transpose of an 8 x 8 matrix of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}

// NR: products of eight query rows, 1 or 2.
template <typename T, int DC, int NR>
__global__ void __launch_bounds__(kThreads, Shape<DC, NR>::kCtasPerSm)
    rows_kernel(AttnParams p, const __grid_constant__ KvMaps maps) {
  using S = Shape<DC, NR>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * S::kStages];
  __shared__ uint32_t no_page[kNoted][4];
  __shared__ int dead_mem[2];
  __shared__ float stat_m[kWarps][16], stat_l[kWarps][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
  float* join = reinterpret_cast<float*>(smem_raw + (base - smem_addr(smem_raw)) +
                                         S::kStages * S::kStage);
  Ring ring{base, smem_addr(bars), smem_addr(bars) + 8 * S::kStages, no_page, dead_mem};

  let_next_start();
  if (threadIdx.x == 32 * kWarps && maps.box > 0) {
    prefetch_map(&maps.k);
    prefetch_map(&maps.v);
  }
  if (threadIdx.x == 0) {
    dead_mem[0] = dead_mem[1] = 0;
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(ring.full + 8 * i, kLoadWarps);
      mbar_init(ring.empty + 8 * i, kWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  Walk<kRowTile, kRowKeys> w;
  const bool any = w.begin(p, p.rows, reinterpret_cast<int64_t*>(join));
  __syncthreads();

  if (!any && threadIdx.x == 0) w.note_cut(p.rows, false);
  if (any && warp >= kWarps) {
    if (maps.box > 0)
      load_boxes<DC, kRowTile, kRowKeys, S::kStages>(p, w, ring, &maps.k, &maps.v, maps.box,
                                                     warp - kWarps);
    else
      load_kv<DC, kRowTile, kRowKeys, S::kStages>(p, w, ring, nullptr, nullptr, 0, warp - kWarps);
  } else if (any) {
    const int g = lane >> 2, c = lane & 3, D = p.dim;
    // this lane's part of an ldmatrix address: K tiles by key, V tiles transposed
    const int k_key = 16 * warp + (lane & 15), k_half = lane >> 4;
    const int v_key = 16 * warp + ((lane >> 4) << 3) + (lane & 7), v_half = (lane >> 3) & 1;
    const auto at = [](int key, int chunk) {  // byte of a 16-byte chunk in a tile
      return uint32_t((chunk >> 3) * (kRowKeys * 128) + key * 128 + (((chunk & 7) ^ (key & 7)) << 4));
    };
    uint32_t stage = 0, phase = 0, unit_count = 0;
    bool ok = true;
    const auto release = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.empty + 8 * stage);
      if (++stage == S::kStages) stage = 0, phase ^= 1;
    };
    // Query row g (and g + 8), loaded while the item before is joined.
    uint32_t qf[4 * DC][2 * NR];
    const auto load_queries = [&]() {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const int row = w.it.row + g + 8 * n;
        const int tok = div_of(row, p.group_div);
        const bool real = g + 8 * n < w.it.rows;
        const uint16_t* src = p.q + int64_t(w.it.req.first + tok) * p.q_stride +
                              int64_t(w.head * p.group + (row - tok * p.group)) * D + 2 * c;
#pragma unroll
        for (int k = 0; k < 4 * DC; ++k) {
          qf[k][2 * n] = qf[k][2 * n + 1] = 0;
          if (real && 16 * k < D) {
            qf[k][2 * n] = *reinterpret_cast<const uint32_t*>(src + 16 * k);
            qf[k][2 * n + 1] = *reinterpret_cast<const uint32_t*>(src + 16 * k + 8);
          }
        }
      }
    };
    bool more = w.next(p);
    if (more) load_queries();
    if (threadIdx.x == 0) w.note_cut(p.rows, more);
    while (more) {
      const Item it = w.it;
      const int head = w.head, piece = w.piece, first = w.first, last = w.last;
      const bool whole = w.whole;
      const bool prefix = it.request < 0;
      const int window = prefix ? 0 : p.window, sinks = prefix ? 0 : p.sinks;
      const int tok0 = div_of(it.row, p.group_div);
      const int tok1 = div_of(it.row + it.rows - 1, p.group_div);
      const int pos0 = prefix ? it.req.row0 : it.req.row0 + tok0;
      const int pos1 = prefix ? it.req.row0 : it.req.row0 + tok1;
      // this lane's scores: keys g and g + 8, query rows 8 n + 2 c + e
      int pos[NR][2];
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) pos[n][e] = row_position(p, it, it.row + 8 * n + 2 * c + e);
      if (p.q_flip != 0) {
#pragma unroll
        for (int k = 0; k < 4 * DC; ++k)
#pragma unroll
          for (int i = 0; i < 2 * NR; ++i) qf[k][i] ^= p.q_flip;
      }
      // channels 16 k + g and 8 on, of the same rows
      float acc[4 * DC][NR][4];
#pragma unroll
      for (int k = 0; k < 4 * DC; ++k)
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[k][n][e] = 0.f;
      float m[NR][2], l[NR][2];  // m in log2 units
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) m[n][e] = kNegInf, l[n][e] = 0.f;

      for (int u = first; u < last; ++u, ++unit_count) {
        const int key0 = unit_key<kRowKeys>(it.span, u) + 16 * warp;
        const bool used = key0 < it.span.hi && (key0 + 16 > it.span.lo || key0 < it.span.sink_end);
        if (!(ok = mbar_wait(ring.full + 8 * stage, phase, ring.dead))) break;
        float s[NR][4];
        uint32_t holes = 0;
        if (used) {
          const uint32_t tile = ring.smem + stage * S::kStage;
          float half[2][NR][4];  // two chains of products
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) half[0][n][e] = half[1][n][e] = 0.f;
#pragma unroll
          for (int k = 0; k < 4 * DC; ++k)
            if (16 * k < D) {
              uint32_t a[4];
              ldmatrix4(a, tile + at(k_key, 2 * k + k_half));
#pragma unroll
              for (int n = 0; n < NR; ++n)
                T::mma(half[k & 1][n], a, qf[k][2 * n], qf[k][2 * n + 1]);
            }
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = half[0][n][e] + half[1][n][e];
          holes = (no_page[unit_count % kNoted][warp >> 1] >> (16 * (warp & 1))) & 0xFFFFu;
        }
        release();
        bool full = true, mixed = false;
        uint32_t keep[2] = {~0u, ~0u};  // keys 2 c, 2 c + 1 and 8 on that some row sees
        uint32_t b[NR][2];
        if (used) {
          full = holes == 0 && key0 + 15 <= pos0 &&
                 (window == 0 || pos1 - key0 < window || key0 + 15 < sinks);
          mixed = !full && tok0 != tok1;
          if (!full) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              keep[h] = 0;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int j = 2 * c + e + 8 * h, key = key0 + j;
                if (key < it.span.hi && (key >= it.span.lo || key < it.span.sink_end) &&
                    !((holes >> j) & 1))
                  keep[h] |= e ? 0xFFFF0000u : 0xFFFFu;
              }
            }
          }
          // s[n][e]: key g + 8 * (e >> 1), query row 8 n + 2 c + (e & 1)
          float most[NR][2];
          bool move = false;
#pragma unroll
          for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[n][e] *= p.scale_log2;
              if (!full) {
                const int j = g + 8 * (e >> 1);
                if (((holes >> j) & 1) || !sees(key0 + j, pos[n][e & 1], window, sinks))
                  s[n][e] = kNegInf;
              }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              most[n][e] = fmaxf(s[n][e], s[n][2 + e]);
              move |= most[n][e] > m[n][e] + kSlack;
            }
          }
          // The maximum moves only when a score passes it by 2^8: weights up to
          // that are in range of both types, and nothing is rescaled until then.
          if (__any_sync(~0u, move)) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1)
                  most[n][e] = fmaxf(most[n][e], __shfl_xor_sync(~0u, most[n][e], x));
                const float next = fmaxf(m[n][e], most[n][e]);
                const float f = m[n][e] == next ? 1.f : exp2_fast(m[n][e] - next);
                m[n][e] = next;
                l[n][e] *= f;
#pragma unroll
                for (int k = 0; k < 4 * DC; ++k) acc[k][n][e] *= f, acc[k][n][2 + e] *= f;
              }
          }
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            float w8[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              w8[e] = s[n][e] == kNegInf ? 0.f : exp2_fast(s[n][e] - m[n][e & 1]);
              l[n][e & 1] += w8[e];
            }
            // Rounded to the pool's type for the product with V: half a step of it
            // relative to each weight; the sum l is not.
            b[n][0] = transpose8(T::pack(w8[0], w8[1]));
            b[n][1] = transpose8(T::pack(w8[2], w8[3]));
          }
        }
        if (!(ok = mbar_wait(ring.full + 8 * stage, phase, ring.dead))) break;
        if (used) {
          const uint32_t tile = ring.smem + stage * S::kStage;
          // A weight of zero does not hide a value that is not finite.  Where rows
          // of several positions share such a value, each position takes the
          // product by itself, with the values it does not see put to zero.
          bool bad = false;
          if (mixed) {
#pragma unroll 1
            for (int k = 0; 16 * k < D; ++k) {
              uint32_t a[4];
              ldmatrix4_t(a, tile + at(v_key, 2 * k + v_half));
              bad |= T::not_finite(a[0] & keep[0]) | T::not_finite(a[1] & keep[0]) |
                     T::not_finite(a[2] & keep[1]) | T::not_finite(a[3] & keep[1]);
            }
            bad = __any_sync(~0u, bad);
          }
          if (!bad) {
#pragma unroll
            for (int k = 0; k < 4 * DC; ++k)
              if (16 * k < D) {
                uint32_t a[4];
                ldmatrix4_t(a, tile + at(v_key, 2 * k + v_half));
                if (!full) a[0] &= keep[0], a[1] &= keep[0], a[2] &= keep[1], a[3] &= keep[1];
#pragma unroll
                for (int n = 0; n < NR; ++n) T::mma(acc[k][n], a, b[n][0], b[n][1]);
              }
          } else {
            for (int here = pos0; here <= pos1; ++here) {
              uint32_t seen[2];
#pragma unroll
              for (int h = 0; h < 2; ++h)
                seen[h] = keep[h] &
                          ((sees(key0 + 2 * c + 8 * h, here, window, sinks) ? 0xFFFFu : 0u) |
                           (sees(key0 + 2 * c + 1 + 8 * h, here, window, sinks) ? 0xFFFF0000u : 0u));
#pragma unroll
              for (int k = 0; k < 4 * DC; ++k)
                if (16 * k < D) {
                  uint32_t a[4];
                  ldmatrix4_t(a, tile + at(v_key, 2 * k + v_half));
                  a[0] &= seen[0], a[1] &= seen[0], a[2] &= seen[1], a[3] &= seen[1];
#pragma unroll
                  for (int n = 0; n < NR; ++n) {
                    float part[4] = {0.f, 0.f, 0.f, 0.f};
                    T::mma(part, a, b[n][0], b[n][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      if (pos[n][e & 1] == here) acc[k][n][e] += part[e];
                  }
                }
            }
          }
        }
        release();
      }

      more = w.next(p);
      if (more) load_queries();

      // Join the warps: sums over the lanes of a row, then under the common maximum.
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(~0u, l[n][e], x);
          if (g == 0) {
            stat_m[warp][8 * n + 2 * c + e] = m[n][e];
            stat_l[warp][8 * n + 2 * c + e] = l[n][e];
          }
        }
      compute_sync();
      float f[NR][2];
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = kNegInf;
#pragma unroll
          for (int k = 0; k < kWarps; ++k) top = fmaxf(top, stat_m[k][8 * n + 2 * c + e]);
          f[n][e] = weight_of(m[n][e], top);
        }
      const int quads = D / 4;
      for (int r0 = 0; r0 < it.rows; r0 += S::kJoinRows) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = 8 * n + 2 * c + e - r0;
            if (row < 0 || row >= S::kJoinRows) continue;
            float* dst = join + (warp * S::kJoinRows + row) * S::kPitch + g;
#pragma unroll
            for (int k = 0; k < 4 * DC; ++k) {
              dst[16 * k] = acc[k][n][e] * f[n][e];
              dst[16 * k + 8] = acc[k][n][2 + e] * f[n][e];
            }
          }
        compute_sync();
        // thread: four channels of a row
        const int rows = min(S::kJoinRows, it.rows - r0);
        for (int i = threadIdx.x; i < rows * quads; i += 32 * kWarps) {
          const int r = i / quads, row = r0 + r, d = (i - r * quads) * 4;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          float mm = kNegInf, ll = 0.f;
#pragma unroll
          for (int k = 0; k < kWarps; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(
                join + (k * S::kJoinRows + r) * S::kPitch + d);
            o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
            mm = fmaxf(mm, stat_m[k][row]);
          }
#pragma unroll
          for (int k = 0; k < kWarps; ++k) ll += stat_l[k][row] * weight_of(stat_m[k][row], mm);
          const int tok = div_of(it.row + row, p.group_div);
          const int64_t t = it.req.first + tok;
          const int qh = head * p.group + it.row + row - tok * p.group;
          if (!whole) {
            const int64_t to = int64_t(piece) * kRowTile + row;
            *reinterpret_cast<float4*>(p.rows.pieces + to * D + d) = o;
            if (d == 0) p.rows.stats[to] = make_float2(mm, ll);
          } else if (p.shared) {
            const int64_t to = (int64_t(prefix) * p.num_tokens + t) * p.q_heads + qh;
            *reinterpret_cast<float4*>(p.whole + to * D + d) = o;
            if (d == 0) p.whole_stats[to] = make_float2(mm, ll);
          } else {
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            *reinterpret_cast<uint2*>(p.out + t * p.out_stride + int64_t(qh) * D + d) =
                make_uint2(T::pack(o.x * inv, o.y * inv), T::pack(o.z * inv, o.w * inv));
            if (d == 0 && p.lse != nullptr) p.lse[t * p.q_heads + qh] = log_sum(mm, ll);
          }
        }
        compute_sync();  // join and the statistics are written again
      }
      // A wait that ran out: all warps are at this item and leave together.
      if (*ring.dead != 0) break;
    }
    if (!ok && lane == 0) report(p.status, CG_ERR_CUDA);
  }
  __syncthreads();
  let_settle(ring.dead);
  // this kernel may have started before the tile kernel was done; the join
  // waits for this one, and so for both
  wait_for_previous();
}

template <typename T, int DC, int NR>
cudaError_t launch(const AttnParams& p, bool early, cudaStream_t stream) {
  using S = Shape<DC, NR>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t err = allow_smem(rows_kernel<T, DC, NR>, S::kSmem, done);
  if (err != cudaSuccess) return err;
  return launch_after(rows_kernel<T, DC, NR>, p.rows.ctas, kThreads, S::kSmem, stream, early, p,
                      kv_maps(p, kRowKeys / kLoadWarps, T::kBf16));
}

template <typename T, int DC>
cudaError_t launch_dim(const AttnParams& p, bool early, cudaStream_t stream) {
  return most_rows(p) > 8 ? launch<T, DC, 2>(p, early, stream) : launch<T, DC, 1>(p, early, stream);
}

template <typename T>
cudaError_t launch_type(const AttnParams& p, bool early, cudaStream_t stream) {
  if (p.dim <= 64) return launch_dim<T, 1>(p, early, stream);
  if (p.dim <= 128) return launch_dim<T, 2>(p, early, stream);
  return launch_dim<T, 4>(p, early, stream);
}

}  // namespace

cudaError_t launch_rows(const AttnParams& p, bool bf16, bool early, cudaStream_t stream) {
  return bf16 ? launch_type<BF16>(p, early, stream) : launch_type<F16>(p, early, stream);
}

}  // namespace cg
