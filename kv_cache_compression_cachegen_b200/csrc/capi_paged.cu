// capi_paged.cu -- the extern "C" entry points of the paged serving calls
// (declared and documented in include/cachegen.h).  Argument checks happen
// here, on the host, before anything is enqueued.
#include <cmath>

#include "cg_common.cuh"
#include "paged.cuh"

namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool missing16(const void* p) { return p == nullptr || !aligned(p, 16); }
bool missing4(const void* p) { return p == nullptr || !aligned(p, 4); }

cg_status check_heads(const cg_shape* s, int32_t num_q_heads) {
  if (s == nullptr || s->num_layers < 1 || s->num_kv_heads < 1 || s->head_dim < 1)
    return CG_ERR_INVALID_ARG;
  if (s->num_layers > cg::kMaxLayers || s->num_kv_heads > cg::kMaxHeads ||
      s->head_dim > cg::kMaxHeadDim || s->head_dim % 16 != 0)
    return CG_ERR_UNSUPPORTED;
  if (num_q_heads < 1 || num_q_heads % s->num_kv_heads != 0) return CG_ERR_INVALID_ARG;
  if (num_q_heads / s->num_kv_heads > 64) return CG_ERR_UNSUPPORTED;
  return CG_OK;
}

cg_status check_pool(const cg_shape* s, const void* pool, int32_t layer, int32_t num_pages,
                     int32_t page_tokens, cg_dtype dtype) {
  if (missing16(pool) || layer < 0 || layer >= s->num_layers || num_pages < 1 || page_tokens < 1 ||
      (dtype != CG_DTYPE_F16 && dtype != CG_DTYPE_BF16))
    return CG_ERR_INVALID_ARG;
  // rows of the pool are counted in 31 bits
  if (int64_t(num_pages) * page_tokens > 0x7FFFFFFF) return CG_ERR_UNSUPPORTED;
  return CG_OK;
}

bool bad_rows(const void* p, int64_t stride, int64_t width) {
  return missing16(p) || stride < width || stride % 8 != 0;
}

cg_status from_cuda(cudaError_t err) { return err == cudaSuccess ? CG_OK : CG_ERR_CUDA; }

cg_status check_batch(int32_t num_q_heads, int32_t max_tokens, int32_t max_requests) {
  if (max_tokens < 1 || max_requests < 1) return CG_ERR_INVALID_ARG;
  // query rows of a kv head, and rows of the output, are counted in 31 bits
  if (max_requests > cg::kMaxRequests || int64_t(max_tokens) * num_q_heads > 0x3FFFFFFF)
    return CG_ERR_UNSUPPORTED;
  return CG_OK;
}

cg_status attention(const cg_shape* shape, const cg_attention_args* a, const int32_t* prefix_table,
                    int32_t prefix_tokens, bool shared, cudaStream_t stream) {
  if (a == nullptr) return CG_ERR_INVALID_ARG;
  cg_status st = check_heads(shape, a->num_q_heads);
  if (st == CG_OK)
    st = check_pool(shape, a->pool_dev, a->layer, a->num_pages, a->page_tokens, a->dtype);
  if (st == CG_OK) st = check_batch(a->num_q_heads, a->num_tokens, a->num_requests);
  if (st != CG_OK) return st;
  const int64_t width = int64_t(a->num_q_heads) * shape->head_dim;
  if (bad_rows(a->q_dev, a->q_stride, width) || bad_rows(a->out_dev, a->out_stride, width) ||
      a->max_q < 1 || a->max_pages < 1 || a->window < 0 || a->sinks < 0 ||
      !std::isfinite(a->scale) || missing4(a->q_starts_dev) || missing4(a->kv_lens_dev) ||
      missing4(a->block_tables_dev) || missing4(a->status_dev) ||
      (a->lse_dev != nullptr && !aligned(a->lse_dev, 4)))
    return CG_ERR_INVALID_ARG;
  if (a->out_dev == a->q_dev) return CG_ERR_INVALID_ARG;
  if (shared && (a->window != 0 || a->sinks != 0 || prefix_tokens < 0 ||
                 (prefix_tokens > 0 && missing4(prefix_table))))
    return CG_ERR_INVALID_ARG;
  if (shared && prefix_tokens > 0x7FFFFF00) return CG_ERR_UNSUPPORTED;
  const uint64_t need =
      cg::attention_workspace(*shape, a->num_q_heads, a->num_tokens, a->num_requests, shared);
  if (a->workspace_bytes < need) return CG_ERR_CAPACITY;
  if (a->workspace_dev == nullptr || !aligned(a->workspace_dev, 256)) return CG_ERR_INVALID_ARG;
  return from_cuda(
      cg::launch_attention(*a, *shape, prefix_table, prefix_tokens, shared, stream));
}

}  // namespace

extern "C" {

cg_status cg_extend_tables(const cg_extend_args* a, cudaStream_t stream) {
  if (a == nullptr || a->num_requests < 1 || a->page_tokens < 1 || a->num_pages < 1 ||
      a->max_pages < 1 || a->num_free < 0 || a->max_tokens < 1 || a->position_base < 0)
    return CG_ERR_INVALID_ARG;
  if (missing4(a->held_dev) || missing4(a->added_dev) || missing4(a->taken_dev) ||
      (a->num_free > 0 && missing4(a->free_pages_dev)) || missing4(a->taken_out_dev) ||
      missing4(a->block_tables_dev) || missing4(a->kv_lens_dev) || missing4(a->q_starts_dev) ||
      a->slots_dev == nullptr || !aligned(a->slots_dev, 8) || missing4(a->positions_dev) ||
      missing4(a->status_dev))
    return CG_ERR_INVALID_ARG;
  if (a->num_requests > cg::kMaxRequests) return CG_ERR_UNSUPPORTED;
  return from_cuda(cg::launch_extend_tables(*a, stream));
}

cg_status cg_rope_table(int32_t max_positions, int32_t rot_dim, double theta, float* out_dev,
                        cudaStream_t stream) {
  if (max_positions < 1 || rot_dim < 2 || rot_dim % 2 != 0 || !(theta > 0.0) ||
      !std::isfinite(theta) || missing4(out_dev))
    return CG_ERR_INVALID_ARG;
  if (rot_dim > cg::kMaxHeadDim) return CG_ERR_UNSUPPORTED;
  return from_cuda(cg::launch_rope_table(max_positions, rot_dim, theta, out_dev, stream));
}

cg_status cg_append_qkv(const cg_shape* shape, const cg_append_args* a, cudaStream_t stream) {
  if (a == nullptr) return CG_ERR_INVALID_ARG;
  cg_status st = check_heads(shape, a->num_q_heads);
  if (st == CG_OK)
    st = check_pool(shape, a->pool_dev, a->layer, a->num_pages, a->page_tokens, a->dtype);
  if (st == CG_OK) st = check_batch(a->num_q_heads, a->num_tokens, 1);
  if (st != CG_OK) return st;
  const int64_t width = int64_t(a->num_q_heads) * shape->head_dim;
  const int64_t kv_width = int64_t(shape->num_kv_heads) * shape->head_dim;
  if (bad_rows(a->q_dev, a->q_stride, width) || bad_rows(a->k_dev, a->k_stride, kv_width) ||
      bad_rows(a->v_dev, a->v_stride, kv_width) ||
      bad_rows(a->q_out_dev, a->q_out_stride, width) || a->slots_dev == nullptr ||
      !aligned(a->slots_dev, 8) || missing4(a->status_dev) || a->rot_dim < 0 ||
      a->rot_dim % 2 != 0 || a->rot_dim > shape->head_dim || !(a->eps >= 0.f) ||
      !std::isfinite(a->eps))
    return CG_ERR_INVALID_ARG;
  if ((a->q_weight_dev != nullptr && !aligned(a->q_weight_dev, 16)) ||
      (a->k_weight_dev != nullptr && !aligned(a->k_weight_dev, 16)))
    return CG_ERR_INVALID_ARG;
  if (a->rot_dim > 0 &&
      (missing4(a->rope_dev) || missing4(a->positions_dev) || a->max_positions < 1))
    return CG_ERR_INVALID_ARG;
  // in place only row for row
  if (a->q_out_dev == a->q_dev && a->q_out_stride != a->q_stride) return CG_ERR_INVALID_ARG;
  return from_cuda(cg::launch_append(*a, *shape, stream));
}

cg_status cg_attention_workspace_bytes(const cg_shape* shape, int32_t num_q_heads,
                                       int32_t max_tokens, int32_t max_requests, int32_t shared,
                                       uint64_t* bytes) {
  cg_status st = check_heads(shape, num_q_heads);
  if (st == CG_OK) st = check_batch(num_q_heads, max_tokens, max_requests);
  if (st != CG_OK) return st;
  if (bytes == nullptr) return CG_ERR_INVALID_ARG;
  *bytes = cg::attention_workspace(*shape, num_q_heads, max_tokens, max_requests, shared != 0);
  return CG_OK;
}

cg_status cg_attention_paged(const cg_shape* shape, const cg_attention_args* args,
                             cudaStream_t stream) {
  return attention(shape, args, nullptr, 0, false, stream);
}

cg_status cg_attention_shared(const cg_shape* shape, const cg_attention_args* args,
                              const int32_t* prefix_table_dev, int32_t prefix_tokens,
                              cudaStream_t stream) {
  return attention(shape, args, prefix_table_dev, prefix_tokens, true, stream);
}

}  // extern "C"
