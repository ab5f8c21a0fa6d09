// shares.cuh -- how a line of units of work is dealt to CTAs.  Plain integer
// arithmetic that also compiles for the host, where it is tested.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define CG_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define CG_HOST_DEVICE inline
#endif

namespace cg {

constexpr int kRowCtasPerSm = 2;  // CTAs of the rows kernel on an SM
constexpr int kMaxCtas = 160;     // of the tile kernel, one an SM
constexpr int kMaxRowCtas = kMaxCtas * kRowCtasPerSm;

// Shorter lines are dealt in 32 bits, whose divisions are several times cheaper:
// the products below stay under 2^32 for the most CTAs that either kernel has.
constexpr int64_t kNarrowUnits = int64_t(1) << 23;
static_assert(kNarrowUnits * kMaxRowCtas <= int64_t(1) << 32, "units times CTAs in 32 bits");

// CTA that holds unit u when `units` are dealt to `ctas`: share c is
// [c * units / ctas, (c + 1) * units / ctas).
CG_HOST_DEVICE int cta_of(int64_t u, int64_t units, int ctas) {
  if (units < kNarrowUnits) return int((uint32_t(u + 1) * uint32_t(ctas) - 1) / uint32_t(units));
  return int(((u + 1) * ctas - 1) / units);
}

// First unit of share c.
CG_HOST_DEVICE int64_t share_of(int c, int64_t units, int ctas) {
  if (units < kNarrowUnits) return uint32_t(units) * uint32_t(c) / uint32_t(ctas);
  return units * c / ctas;
}

}  // namespace cg
