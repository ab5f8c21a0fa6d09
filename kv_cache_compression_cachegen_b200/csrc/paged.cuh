// paged.cuh -- definitions shared by the paged serving operators (block
// tables, the query/key/value append and attention over the paged pool).
// Their semantics are specified in include/cachegen.h.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cachegen.h"

namespace cg {

constexpr int kMaxRequests = 8192;  // the tables kernel keeps three int32 per request on chip

// n / d for 0 <= n < 2^31 and d >= 1: with s = ceil(log2 d) and
// m = ceil(2^(31+s) / d) < 2^32, floor(n * m / 2^(31+s)) is exact (Granlund
// and Montgomery, "Division by Invariant Integers using Multiplication").
struct FastDiv {
  uint32_t d, m, s;
};

inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((uint64_t(1) << f.s) < d) ++f.s;
  f.m = uint32_t(((uint64_t(1) << (31 + f.s)) + d - 1) / d);
  return f;
}

__device__ __forceinline__ int div_of(int n, const FastDiv& f) {
  return int((uint64_t(uint32_t(n)) * f.m) >> (31 + f.s));
}

__device__ __forceinline__ void report(int32_t* status, int32_t code) {
  atomicCAS(status, int32_t(CG_OK), code);
}

// Type of a pool: fp16 or bf16 values, moved as 32-bit pairs.
struct F16 {
  static constexpr bool kBf16 = false;
  __device__ static __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  // An infinity or a NaN in either half.
  __device__ static __forceinline__ bool not_finite(uint32_t v) {
    return (v & 0x7C00u) == 0x7C00u || (v & 0x7C000000u) == 0x7C000000u;
  }
  // C += A (16x16, row major) * B (16x8, column major), fp32 accumulators.
  __device__ static __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

struct BF16 {
  static constexpr bool kBf16 = true;
  __device__ static __forceinline__ float2 unpack(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
  }
  __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ static __forceinline__ bool not_finite(uint32_t v) {
    return (v & 0x7F80u) == 0x7F80u || (v & 0x7F800000u) == 0x7F800000u;
  }
  __device__ static __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

cudaError_t launch_extend_tables(const cg_extend_args& a, cudaStream_t stream);
cudaError_t launch_rope_table(int32_t max_positions, int32_t rot_dim, double theta, float* out,
                              cudaStream_t stream);
cudaError_t launch_append(const cg_append_args& a, const cg_shape& s, cudaStream_t stream);
uint64_t attention_workspace(const cg_shape& s, int32_t num_q_heads, int32_t max_tokens,
                             int32_t max_requests, bool shared);
cudaError_t launch_attention(const cg_attention_args& a, const cg_shape& s,
                             const int32_t* prefix_table, int32_t prefix_tokens, bool shared,
                             cudaStream_t stream);

}  // namespace cg
