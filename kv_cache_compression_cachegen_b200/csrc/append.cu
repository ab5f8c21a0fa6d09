// append.cu -- cg_rope_table and cg_append_qkv: norms of queries and keys for
// each head, the position rotation in the same pass, and the new keys and
// values written to their places in the paged pool.
//
//     y = x * rsqrt(mean(x^2) + eps) * w                 (x itself without a weight)
//     (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)   for the rotated pairs
//
// All of it fp32, rounded once when it is stored.  Every value is read and
// written once, so HBM bounds it.  A group of lanes holds one head's vector,
// eight values (16 bytes) a lane, so the mean is a shuffle reduction inside
// the group and the partner of a value that is rot/2 away is in another lane
// of the group.  A group takes several heads of one token at a time: their
// loads are in flight together and share the token's row of the table.
#include "paged.cuh"

namespace cg {
namespace {

constexpr int kThreads = 128;
constexpr int64_t kResident = 148 * 2048;  // threads of all SMs

__global__ void rope_kernel(int32_t max_positions, int32_t half, double theta, float* out) {
  const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= int64_t(max_positions) * half) return;
  const int64_t pos = i / half;
  const int k = int(i - pos * half);
  // 64 bits: an angle of position 2^17 in 32 bits would be off by up to 2^-8.
  double s, c;
  sincos(double(pos) * pow(theta, -double(k) / half), &s, &c);
  out[pos * 2 * half + k] = float(c);
  out[pos * 2 * half + half + k] = float(s);
}

struct AppendParams {
  const uint16_t *q, *k, *v, *q_weight, *k_weight;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  uint16_t *q_out, *k_pool, *v_pool;
  const float* rope;
  const int32_t* positions;
  const int64_t* slots;
  int64_t num_tokens, num_slots;
  float eps;
  int max_positions, rot, interleaved, q_heads, kv_heads, dim;
  int units;    // head groups of a token
  int by_four;  // a lane's four angles of a row of the table lie on 16 bytes
  int32_t* status;
};

// Large calls (several heads a group) go past the cache: their values are read
// once, and what they write is more than stays there.
template <int HEADS>
__device__ __forceinline__ uint4 load(const uint16_t* p) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
  return HEADS > 1 ? __ldcs(q) : *q;
}
template <int HEADS>
__device__ __forceinline__ void store(uint16_t* p, uint4 v) {
  if (HEADS > 1) __stcs(reinterpret_cast<uint4*>(p), v);
  else *reinterpret_cast<uint4*>(p) = v;
}

// How a lane comes by the partners and angles of its values.
enum Turn {
  kNone,         // no rotation
  kHalves,       // rot/2 apart, a multiple of eight: the partners are in another lane
  kInterleaved,  // next to each other
  kScattered     // any other: partners are read again, from L1
};

// LANES: lanes of a head's vector (a power of two >= dim / 8).  HEADS: heads a
// group of lanes takes at a time, all of one token.
template <typename T, int LANES, int HEADS, Turn TURN>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendParams p) {
  const int64_t group = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / LANES;
  const int lane = threadIdx.x % LANES;
  const int64_t t = group / p.units;
  const int e0 = lane * 8;
  const int head0 = int(group - t * p.units) * HEADS;
  const int heads = p.q_heads + 2 * p.kv_heads;
  const int first_v = p.q_heads + p.kv_heads;
  const bool have = t < p.num_tokens && e0 < p.dim;

  // the values first: nothing decides whether they can be read
  const uint16_t* src[HEADS];
  uint4 raw[HEADS];
#pragma unroll
  for (int u = 0; u < HEADS; ++u) {
    const int h = head0 + u;
    raw[u] = make_uint4(0, 0, 0, 0);
    src[u] = h < p.q_heads  ? p.q + t * p.q_stride + int64_t(h) * p.dim
             : h < first_v ? p.k + t * p.k_stride + int64_t(h - p.q_heads) * p.dim
                           : p.v + t * p.v_stride + int64_t(h - first_v) * p.dim;
    if (have && h < heads) raw[u] = load<HEADS>(src[u] + e0);
  }
  int64_t slot = -1;
  int pos = 0;
  if (t < p.num_tokens) {
    slot = p.slots[t];
    if (TURN != kNone) pos = p.positions[t];
    // a bad row is left out whole; only a negative slot is one on purpose
    if (slot >= 0 &&
        (slot >= p.num_slots || (TURN != kNone && (pos < 0 || pos >= p.max_positions)))) {
      if (lane == 0) report(p.status, CG_ERR_MISMATCH);
      slot = -1;
    }
  }
  const bool live = have && slot >= 0;

  const int half = p.rot / 2;
  const bool turn = TURN != kNone && e0 < p.rot;
  const int partner = e0 < half ? lane + half / 8 : lane - half / 8;  // kHalves
  float co[8], si[8];  // y <- y co + partner si
  if (TURN != kNone) {
#pragma unroll
    for (int i = 0; i < 8; ++i) co[i] = 1.f, si[i] = 0.f;
    if (live && turn && head0 < first_v) {
      const float* row = p.rope + int64_t(pos) * p.rot;
      if (TURN == kHalves) {
        const float4* c = reinterpret_cast<const float4*>(row + (e0 < half ? e0 : e0 - half));
        const float4* s = reinterpret_cast<const float4*>(row + (e0 < half ? e0 + half : e0));
        const float sign = e0 < half ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 a = __ldg(c + i), b = __ldg(s + i);
          co[4 * i] = a.x, co[4 * i + 1] = a.y, co[4 * i + 2] = a.z, co[4 * i + 3] = a.w;
          si[4 * i] = sign * b.x, si[4 * i + 1] = sign * b.y;
          si[4 * i + 2] = sign * b.z, si[4 * i + 3] = sign * b.w;
        }
      } else if (TURN == kInterleaved && p.by_four) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(row + e0 / 2));
        const float4 b = __ldg(reinterpret_cast<const float4*>(row + half + e0 / 2));
        co[0] = co[1] = a.x, co[2] = co[3] = a.y, co[4] = co[5] = a.z, co[6] = co[7] = a.w;
        si[0] = -b.x, si[1] = b.x, si[2] = -b.y, si[3] = b.y;
        si[4] = -b.z, si[5] = b.z, si[6] = -b.w, si[7] = b.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = e0 + i;
          if (e < p.rot) {
            const int a = p.interleaved ? e >> 1 : (e < half ? e : e - half);
            co[i] = __ldg(row + a);
            si[i] = __ldg(row + half + a);
            if (p.interleaved ? !(e & 1) : e < half) si[i] = -si[i];  // y_a c - y_b s
          }
        }
      }
    }
  }

  const unsigned group_mask =
      LANES == 32 ? ~0u : ((1u << LANES) - 1u) << ((threadIdx.x & 31) / LANES * LANES);
#pragma unroll
  for (int u = 0; u < HEADS; ++u) {
    const int h = head0 + u;
    if (h >= first_v) continue;  // the same for the whole group
    const uint16_t* weight = h < p.q_heads ? p.q_weight : p.k_weight;
    float y[8];
    const uint32_t in[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = T::unpack(in[i]);
      y[2 * i] = f.x;
      y[2 * i + 1] = f.y;
    }
    float r = 1.f;
    if (weight != nullptr) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(y[i], y[i], sum);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(group_mask, sum, o, LANES);
      r = rsqrtf(sum / float(p.dim) + p.eps);
      if (e0 < p.dim) {
        const uint4 w4 = *reinterpret_cast<const uint4*>(weight + e0);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = T::unpack(w[i]);
          y[2 * i] *= r * f.x;
          y[2 * i + 1] *= r * f.y;
        }
      }
    }
    if (TURN != kNone) {
      float z[8];
      if (TURN == kInterleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = y[i ^ 1];
      } else if (TURN == kHalves) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = __shfl_sync(group_mask, y[i], partner, LANES);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = e0 + i;
          z[i] = 0.f;
          if (live && e < p.rot) {
            const int b = e < half ? e + half : e - half;
            z[i] = T::unpack(src[u][b]).x;
            if (weight != nullptr) z[i] *= r * T::unpack(weight[b]).x;
          }
        }
        __syncwarp(group_mask);  // q_out may be q: all partners are read before any value is stored
      }
      if (turn) {
        // A lane may hold the last turned channels and the first that are not: those
        // keep their value whatever lies beside it.  (With halves rot is a multiple
        // of 16, and a lane has the one or the other.)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (TURN == kHalves || e0 + i < p.rot) y[i] = fmaf(z[i], si[i], y[i] * co[i]);
      }
    }
    raw[u] = make_uint4(T::pack(y[0], y[1]), T::pack(y[2], y[3]), T::pack(y[4], y[5]),
                        T::pack(y[6], y[7]));
  }
  if (!live) return;
#pragma unroll
  for (int u = 0; u < HEADS; ++u) {
    const int h = head0 + u;
    if (h >= heads) break;
    uint16_t* dst =
        h < p.q_heads ? p.q_out + t * p.q_out_stride + int64_t(h) * p.dim
        : h < first_v ? p.k_pool + (slot * p.kv_heads + h - p.q_heads) * int64_t(p.dim)
                      : p.v_pool + (slot * p.kv_heads + h - first_v) * int64_t(p.dim);
    store<HEADS>(dst + e0, raw[u]);
  }
}

template <typename T, int LANES, Turn TURN>
cudaError_t launch_turn(AppendParams& p, cudaStream_t stream) {
  const int heads = p.q_heads + 2 * p.kv_heads;
  const auto go = [&](auto kernel, int per) {
    p.units = (heads + per - 1) / per;
    const int64_t threads = p.num_tokens * p.units * LANES;
    kernel<<<unsigned((threads + kThreads - 1) / kThreads), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
  };
  // One head a group while the machine holds all groups at once: nothing hides
  // a group's latency then but its own shortness.  Four beyond, whose loads are
  // on their way together and share the token's angles.  64 tokens of 48 heads
  // of 128: 2.7 us and 4.0; 10,752 tokens of 96: 167 us and 92.
  if (p.num_tokens * heads * LANES <= kResident)
    return go(append_kernel<T, LANES, 1, TURN>, 1);
  return go(append_kernel<T, LANES, 4, TURN>, 4);
}

template <typename T, int LANES>
cudaError_t launch_lanes(AppendParams& p, cudaStream_t stream) {
  if (p.rot == 0) return launch_turn<T, LANES, kNone>(p, stream);
  if (p.interleaved) return launch_turn<T, LANES, kInterleaved>(p, stream);
  // the table's rows are read 16 bytes at a time
  if (p.rot % 16 == 0 && p.by_four)
    return launch_turn<T, LANES, kHalves>(p, stream);
  return launch_turn<T, LANES, kScattered>(p, stream);
}

template <typename T>
cudaError_t launch_type(AppendParams& p, cudaStream_t stream) {
  if (p.dim <= 16) return launch_lanes<T, 2>(p, stream);
  if (p.dim <= 32) return launch_lanes<T, 4>(p, stream);
  if (p.dim <= 64) return launch_lanes<T, 8>(p, stream);
  if (p.dim <= 128) return launch_lanes<T, 16>(p, stream);
  return launch_lanes<T, 32>(p, stream);
}

}  // namespace

cudaError_t launch_rope_table(int32_t max_positions, int32_t rot_dim, double theta, float* out,
                              cudaStream_t stream) {
  const int64_t n = int64_t(max_positions) * (rot_dim / 2);
  rope_kernel<<<unsigned((n + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
      max_positions, rot_dim / 2, theta, out);
  return cudaGetLastError();
}

cudaError_t launch_append(const cg_append_args& a, const cg_shape& s, cudaStream_t stream) {
  AppendParams p{};
  p.q = a.q_dev;
  p.k = a.k_dev;
  p.v = a.v_dev;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_out = a.q_out_dev;
  p.q_out_stride = a.q_out_stride;
  p.q_weight = a.q_weight_dev;
  p.k_weight = a.k_weight_dev;
  p.eps = a.eps;
  p.rope = a.rope_dev;
  p.max_positions = a.max_positions;
  p.by_four = a.rot_dim % 8 == 0 && (reinterpret_cast<uintptr_t>(a.rope_dev) & 15) == 0;
  p.rot = a.rot_dim;
  p.interleaved = a.interleaved;
  p.positions = a.positions_dev;
  p.slots = a.slots_dev;
  p.num_tokens = a.num_tokens;
  p.num_slots = int64_t(a.num_pages) * a.page_tokens;
  p.q_heads = a.num_q_heads;
  p.kv_heads = s.num_kv_heads;
  p.dim = s.head_dim;
  const int64_t half_pool = p.num_slots * s.num_kv_heads * s.head_dim;  // one (layer, K or V)
  p.k_pool = a.pool_dev + int64_t(a.layer) * 2 * half_pool;
  p.v_pool = p.k_pool + half_pool;
  p.status = a.status_dev;
  return a.dtype == CG_DTYPE_F16 ? launch_type<F16>(p, stream) : launch_type<BF16>(p, stream);
}

}  // namespace cg
