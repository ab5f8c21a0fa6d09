// attend_maps.cu -- the TMA tensor maps of the attention kernels.
#include <algorithm>

#include "attend.cuh"

namespace cg {
namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    cudaDriverEntryPointQueryResult found;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// [rows][heads][channels] in boxes of 64 channels of `heads` heads of `rows`
// rows, in the 128-byte swizzle; what lies outside is zeros.
bool encode(CUtensorMap* map, const uint16_t* base, bool bf16, int dim, int heads, int64_t rows,
            int64_t row_stride, int box_heads, int box_rows) {
  if (encode_fn() == nullptr || row_stride * 2 >= (int64_t(1) << 40)) return false;
  const cuuint64_t dims[3] = {cuuint64_t(dim), cuuint64_t(heads), cuuint64_t(rows)};
  const cuuint64_t strides[2] = {cuuint64_t(dim) * 2, cuuint64_t(row_stride) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_rows)}, ones[3] = {1, 1, 1};
  return encode_fn()(map,
                     bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                     const_cast<uint16_t*>(base), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

KvMaps kv_maps(const AttnParams& p, int most_rows, bool bf16) {
  // Keys that follow one another in a page for certain: the largest power of
  // two in its size.  The swizzle needs eight; smaller pages come row by row.
  KvMaps m{};
  m.box = std::min(p.page_tokens & -p.page_tokens, most_rows);
  const int64_t rows = int64_t(p.num_pages) * p.page_tokens, stride = int64_t(p.kv_heads) * p.dim;
  if (m.box < 8 || !encode(&m.k, p.k_pool, bf16, p.dim, p.kv_heads, rows, stride, 1, m.box) ||
      !encode(&m.v, p.v_pool, bf16, p.dim, p.kv_heads, rows, stride, 1, m.box))
    m.box = 0;
  return m;
}

bool query_map(CUtensorMap* map, const AttnParams& p, bool bf16) {
  // 128 rows are whole tokens only where the group divides 128, and a copy
  // cannot turn signs
  return 128 % p.group == 0 && p.q_flip == 0 &&
         encode(map, p.q, bf16, p.dim, p.q_heads, p.num_tokens, p.q_stride, p.group,
                128 / p.group);
}

}  // namespace cg
