// attend.cuh -- what the attention kernels share: their parameters, which
// keys a request's rows see, and how the work is dealt to the CTAs.
//
// Work.  An *item* is one request's tile of query rows at one kv head; a row
// is a (token, query head of the group) pair, token-major, so that the heads
// that share a kv head share its loads.  An item's keys are cut into units of
// kKeys keys, aligned in the sequence; its units are the tiles that hold a
// sink followed by the tiles from the window's start to the last row.  All
// units of all items, request by request and head by head, form one line that
// is cut into equal shares, one a CTA, whatever the lengths: one long request
// among short ones, or a batch of one, fills the machine.  A CTA whose share
// holds an item whole writes its output; an item cut between CTAs leaves a
// piece (unnormalised sums, running maximum and sum) with each, and a second
// kernel joins them.  Everything about the cut follows from the lengths, so
// the join needs no flags and the workspace no clearing, and the order of
// every sum is fixed.
#pragma once

#include "paged.cuh"

namespace cg {

struct AttnParams {
  const uint16_t* q;
  uint16_t* out;
  float* lse;  // [num_tokens][q_heads] or null
  int64_t q_stride, out_stride;
  const int32_t *q_starts, *kv_lens, *tables, *prefix_table;
  const uint16_t *k_pool, *v_pool;  // the layer's halves of the pool
  int32_t* status;
  int num_requests, num_tokens, max_q, q_heads, kv_heads, group, dim;
  int num_pages, page_tokens, max_pages;
  FastDiv page_div, group_div;
  int window, sinks;
  int prefix_tokens, shared;
  float scale_log2;  // scale * log2(e)
  // workspace
  int64_t* row_cum;   // [slots + 1] units of a head before each slot of the rows kernel
  float* row_pieces;  // [2 * row_ctas][kRowTile][dim]
  float2* row_stats;  // [2 * row_ctas][kRowTile] (maximum in log2 units, sum)
  float* whole;       // shared: [2][num_tokens][q_heads][dim], items that one CTA finished
  float2* whole_stats;
  int row_ctas;
};

// What one request brings: its packed query rows and its keys.
struct Request {
  int first, tokens;  // rows of q
  int keys;           // tokens in the pool
  int row0;           // position of its first new token among the keys (may be negative)
};

// False (and the request is left out) where the lengths do not fit the call.
__device__ __forceinline__ bool load_request(const AttnParams& p, int r, Request& q) {
  const int a = p.q_starts[r], b = p.q_starts[r + 1], keys = p.kv_lens[r];
  q.first = a;
  q.tokens = 0;
  q.keys = 0;
  q.row0 = 0;
  if (a < 0 || b < a || b > p.num_tokens || b - a > p.max_q || keys < 0 ||
      int64_t(keys) > int64_t(p.max_pages) * p.page_tokens)
    return false;
  q.tokens = b - a;
  q.keys = keys;
  q.row0 = keys - q.tokens;
  return true;
}

// The keys that rows at positions [p0, p1] may see between them: [0, sink_end)
// and [lo, hi), and the units that hold them.
struct Span {
  int sink_end, lo, hi;
  int sink_units, first_unit, units;
};

template <int kKeys>
__device__ __forceinline__ Span span_of(int p0, int p1, int window, int sinks) {
  Span s;
  s.hi = p1 + 1 > 0 ? p1 + 1 : 0;
  s.lo = (window > 0 && p0 >= window) ? p0 - window + 1 : 0;
  s.sink_end = sinks < s.lo ? sinks : s.lo;
  s.sink_units = (s.sink_end + kKeys - 1) / kKeys;
  s.first_unit = s.lo / kKeys > s.sink_units ? s.lo / kKeys : s.sink_units;
  const int last = (s.hi + kKeys - 1) / kKeys;
  s.units = s.sink_units + (last > s.first_unit ? last - s.first_unit : 0);
  if (s.hi == 0) s.units = 0;
  return s;
}

// Whether a row at position `at` sees a key.
__device__ __forceinline__ bool sees(int key, int at, int window, int sinks) {
  return key <= at && (window == 0 || at - key < window || key < sinks);
}

// First key of the u-th unit.
template <int kKeys>
__device__ __forceinline__ int unit_key(const Span& s, int u) {
  return (u < s.sink_units ? u : s.first_unit + u - s.sink_units) * kKeys;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Weight of a part with maximum m (log2 units) under the common maximum; a part
// that saw no key has none.  (A NaN among its scores is in its sums.)
__device__ __forceinline__ float weight_of(float m, float top) {
  return m == top ? (m == -__builtin_huge_valf() ? 0.f : 1.f) : exp2_fast(m - top);
}

// CTA that holds unit u when `units` are dealt to `ctas`: share c is
// [c * units / ctas, (c + 1) * units / ctas).
__device__ __forceinline__ int cta_of(int64_t u, int64_t units, int ctas) {
  return int(((u + 1) * ctas - 1) / units);
}

}  // namespace cg
