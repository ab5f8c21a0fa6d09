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

// The index that a bisection of [0, n) finds for the last one with at(i) <= x.
// Where `at` does not rise all the way (lengths that a call should not have been
// given) all users still find the same one, which is what matters: the line's
// sums, the walks over it and the joins have to agree on a slot's request.
template <typename At>
CG_HOST_DEVICE int last_not_above(int n, int x, const At& at) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at(mid) <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// First slots of requests whose rows begin at `starts` in a batch of `tokens`, in a
// line of tiles of `tile` rows a kv head.
struct FirstSlots {
  const int32_t* starts;
  int tokens, group, tile;
  CG_HOST_DEVICE int operator()(int r) const {
    int a = starts[r];
    a = a < 0 ? 0 : (a > tokens ? tokens : a);
    return int(int64_t(a) * group / tile) + r;
  }
};

// First rows.
struct FirstRows {
  const int32_t* starts;
  CG_HOST_DEVICE int operator()(int r) const { return starts[r]; }
};

}  // namespace cg
