// tables.cu -- cg_extend_tables: block tables and slot maps from request lengths.
//
// With P tokens a page, request r needs
//     need_r = ceil((held_r + added_r) / P) - ceil(held_r / P)
// new pages; they are dealt from the free list in request order, so both the
// pages and the packed token rows of a request start at an exclusive prefix
// sum over the requests.  The work is a few bytes a token, so the kernel is
// one launch whose time is latency: every CTA of one cluster scans all the
// lengths itself (two loads a request, from L2 after the first CTA) instead of
// passing prefixes on through memory, keeps the prefixes on chip, and fills
// its share of the outputs, finding each token's request by binary search.
// A cluster, and not a grid: its barrier separates the reads of the lengths,
// the free list and the tables from the writes, so the outputs may be the
// inputs' own buffers, and makes the call all or nothing on an error.
#include <climits>

#include "paged.cuh"

namespace cg {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
}

// Pages that n >= 0 tokens take.
__device__ __forceinline__ int pages_of(int n, const FastDiv& div) {
  const int q = div_of(n, div);
  return q + (n != q * int(div.d));
}

// The first request from lo to hi whose inclusive sum passes t (hi's does).
__device__ __forceinline__ int request_behind(const int32_t* end, int lo, int hi, int t) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Give every CTA of the cluster the first code (in rank order) that any of them found.
__device__ int32_t cluster_first(int32_t mine, int32_t* slots, int rank, int size) {
  if (threadIdx.x < size) {
    const uint32_t here = uint32_t(__cvta_generic_to_shared(&slots[rank]));
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(threadIdx.x));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there), "r"(mine) : "memory");
  }
  cluster_sync();
  int32_t all = CG_OK;
  for (int i = 0; i < size; ++i)
    if (all == CG_OK) all = slots[i];
  return all;
}

// kPer: tokens of a thread at a time.
template <int kPer>
__global__ void __launch_bounds__(kThreads, 1) extend_kernel(cg_extend_args a, FastDiv div) {
  extern __shared__ int32_t smem[];
  const int B = a.num_requests;
  int32_t* held_s = smem;            // [B]
  int32_t* tok_end = smem + B;       // [B] inclusive sum of added
  int32_t* page_end = smem + 2 * B;  // [B] inclusive sum of need
  __shared__ long long warp_tok[kWarps], warp_page[kWarps];
  __shared__ int32_t err_s, codes[16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = int(cluster_rank()), size = int(cluster_size());
  const int P = a.page_tokens;
  const long long capacity = (long long)a.max_pages * P;
  if (tid == 0) err_s = CG_OK;
  const int32_t taken = *a.taken_dev;
  __syncthreads();
  cluster_sync();  // every CTA of the cluster runs before another writes to its shared memory

  long long tok_base = 0, page_base = 0;  // sums of the requests before this block of them
  for (int r0 = 0; r0 < B; r0 += kThreads) {
    const int r = r0 + tid;
    long long added = 0, need = 0;
    if (r < B) {
      const int32_t h = a.held_dev[r], n = a.added_dev[r];
      held_s[r] = h;
      if (h < 0 || n < 0) {
        atomicCAS(&err_s, CG_OK, int32_t(CG_ERR_MISMATCH));
      } else if ((long long)h + n > capacity ||
                 (long long)a.position_base + h + n > (long long)INT_MAX) {
        atomicCAS(&err_s, CG_OK, int32_t(CG_ERR_CAPACITY));
      } else {
        added = n;
        need = pages_of(h + n, div) - pages_of(h, div);
      }
    }
    long long t = added, p = need;  // inclusive scans over the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long tu = __shfl_up_sync(~0u, t, o), pu = __shfl_up_sync(~0u, p, o);
      if (lane >= o) t += tu, p += pu;
    }
    if (lane == 31) warp_tok[warp] = t, warp_page[warp] = p;
    __syncthreads();
    long long tw = warp_tok[lane], pw = warp_page[lane];  // kWarps == 32
    const long long own_t = tw, own_p = pw;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long tu = __shfl_up_sync(~0u, tw, o), pu = __shfl_up_sync(~0u, pw, o);
      if (lane >= o) tw += tu, pw += pu;
    }
    const long long tb = __shfl_sync(~0u, tw - own_t, warp), pb = __shfl_sync(~0u, pw - own_p, warp);
    t += tok_base + tb;
    p += page_base + pb;
    if (r < B) {
      // beyond these limits the call fails and the prefixes are not used
      tok_end[r] = int32_t(t < INT_MAX ? t : INT_MAX);
      page_end[r] = int32_t(p < INT_MAX ? p : INT_MAX);
    }
    tok_base += __shfl_sync(~0u, tw, 31);
    page_base += __shfl_sync(~0u, pw, 31);
    __syncthreads();  // warp_tok is written again
  }

  int32_t err = err_s;
  __syncthreads();  // every thread has read it before the checks below write it
  if (err == CG_OK && (taken < 0 || taken > a.num_free)) err = CG_ERR_MISMATCH;
  if (err == CG_OK && (tok_base > a.max_tokens || page_base > a.num_free - taken))
    err = CG_ERR_CAPACITY;
  const int total = int(tok_base), pages = int(page_base);
  const int first = rank * kThreads + tid, step = size * kThreads;
  if (err == CG_OK) {
    // every page the call will use must lie in the pool
    for (int i = first; i < pages; i += step) {
      const int32_t page = a.free_pages_dev[taken + i];
      if (page < 0 || page >= a.num_pages) atomicCAS(&err_s, CG_OK, int32_t(CG_ERR_MISMATCH));
    }
    for (int r = first; r < B; r += step) {
      const int h = held_s[r], n = tok_end[r] - (r ? tok_end[r - 1] : 0);
      const int full = div_of(h, div);
      if (n > 0 && h != full * P) {
        const int32_t page = a.block_tables_dev[(long long)r * a.max_pages + full];
        if (page < 0 || page >= a.num_pages) atomicCAS(&err_s, CG_OK, int32_t(CG_ERR_MISMATCH));
      }
    }
    __syncthreads();
    err = err_s;
  }
  err = cluster_first(err, codes, rank, size);  // also: everything is read before anything is written

  if (err != CG_OK) {
    if (rank == 0 && tid == 0) {
      report(a.status_dev, err);
      *a.taken_out_dev = taken;
      a.q_starts_dev[0] = 0;
    }
    for (int r = first; r < B; r += step) {
      a.kv_lens_dev[r] = held_s[r];
      a.q_starts_dev[r + 1] = 0;
    }
    for (int t = first; t < a.max_tokens; t += step) {
      a.slots_dev[t] = -1;
      a.positions_dev[t] = -1;
    }
    return;
  }

  if (rank == 0 && tid == 0) {
    *a.taken_out_dev = taken + pages;
    a.q_starts_dev[0] = 0;
  }
  for (int r = first; r < B; r += step) {
    const int end = tok_end[r];
    a.kv_lens_dev[r] = held_s[r] + (end - (r ? tok_end[r - 1] : 0));
    a.q_starts_dev[r + 1] = end;
  }
  // A token in its request's partly filled last page reads that page's table
  // entry, which no thread writes; all others take their page from the free
  // list.  A warp takes kPer * 32 tokens that follow one another and looks for
  // the requests of the first and the last: where those are one, no lane has to
  // search.  Their pages' entries are asked for together.
  constexpr int kChunk = 32 * kPer;
  for (int64_t c0 = int64_t(first >> 5) * kChunk; c0 < a.max_tokens; c0 += int64_t(step) * kPer) {
    int r0 = 0, r1 = B - 1;
    if (kPer > 1 && c0 < total) {
      r0 = request_behind(tok_end, 0, B - 1, int(c0));
      r1 = request_behind(tok_end, r0, B - 1, int(min(c0 + kChunk - 1, int64_t(total) - 1)));
    }
    int32_t page[kPer], row[kPer], pos[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t t = c0 + 32 * i + lane;
      page[i] = row[i] = 0;
      pos[i] = -1;
      if (t < total) {
        const int r = request_behind(tok_end, r0, r1, int(t));
        const int at = held_s[r] + int(t) - (r ? tok_end[r - 1] : 0);
        const int col = div_of(at, div), have = pages_of(held_s[r], div);
        page[i] = *(col < have
                        ? a.block_tables_dev + (long long)r * a.max_pages + col
                        : a.free_pages_dev + taken + (r ? page_end[r - 1] : 0) + (col - have));
        row[i] = at - col * P;
        pos[i] = a.position_base + at;
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t t = c0 + 32 * i + lane;
      if (t >= a.max_tokens) break;
      a.slots_dev[t] = pos[i] < 0 ? -1 : int64_t(page[i]) * P + row[i];
      a.positions_dev[t] = pos[i];
    }
  }
  for (int i = first; i < pages; i += step) {
    const int lo = request_behind(page_end, 0, B - 1, i);
    const int have = pages_of(held_s[lo], div);
    a.block_tables_dev[(long long)lo * a.max_pages + have + i - (lo ? page_end[lo - 1] : 0)] =
        a.free_pages_dev[taken + i];
  }
}

template <int kPer>
cudaError_t launch(const cg_extend_args& a, int ctas, cudaStream_t stream) {
  const size_t smem = size_t(a.num_requests) * 12;
  if (smem > 48 * 1024 - 2048) {
    const cudaError_t err = cudaFuncSetAttribute(
        extend_kernel<kPer>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRequests * 12);
    if (err != cudaSuccess) return err;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, extend_kernel<kPer>, a, fast_div(uint32_t(a.page_tokens)));
}

}  // namespace

cudaError_t launch_extend_tables(const cg_extend_args& a, cudaStream_t stream) {
  // One CTA while a thread has at most four tokens to write; eight beyond, the
  // largest portable cluster.
  return a.max_tokens > 4 * kThreads || a.num_requests > kThreads ? launch<4>(a, 8, stream)
                                                                  : launch<1>(a, 1, stream);
}

}  // namespace cg
