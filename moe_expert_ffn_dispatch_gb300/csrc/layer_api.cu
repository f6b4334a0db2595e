// C entry points of the decoder-layer operators (moe_layer.h): argument
// checks and the choice of launch.  Nothing here throws or allocates.
#include <cmath>

#include "layer_ops.cuh"

namespace {

bool at(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool act(int32_t dt) { return dt == MOE_LAYER_BF16 || dt == MOE_LAYER_FP16; }

constexpr int32_t kMostRows = 2147483647 - (1 << 20);

int done(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// SM count of the current device, asked once a device; 0 if it cannot be asked
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

bool w8_sizes(int32_t m, int32_t n, int32_t k) {
  return m >= 0 && m <= 1000000 && n >= 1 && n <= kMostRows && k >= 16 && k <= 65536 && k % 16 == 0;
}

int check_cache(const moe_layer_kv_cache_t& c) {
  if (!c.k || !c.v || !c.k_scale || !c.v_scale) return MOE_ERR_INVALID_ARG;
  if (c.num_pages < 1 || c.kv_heads < 1 || c.kv_heads > 1024) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (c.head_dim != 64 && c.head_dim != 128) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!at(c.k, 16) || !at(c.v, 16) || !at(c.k_scale, 4) || !at(c.v_scale, 4) || c.page_stride % 16 ||
      c.head_stride % 16)
    return MOE_ERR_ALIGNMENT;
  if (c.page_stride < 0 || c.head_stride < 0 || c.scale_stride < 0) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_layer_add_rmsnorm_quant(const moe_layer_norm_args_t* a, void* stream) {
  if (!a || !act(a->dtype) || (a->weight_dtype != a->dtype && a->weight_dtype != MOE_LAYER_FP32))
    return MOE_ERR_INVALID_ARG;
  if (a->rows < 0 || a->hidden < 1 || a->hidden > 16384) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!(a->eps >= 0.0f) || !std::isfinite(a->eps)) return MOE_ERR_INVALID_ARG;
  if (a->rows == 0) return MOE_OK;
  if (!a->x || !a->weight || !a->q || !a->q_scale || (a->residual == nullptr) != (a->residual_out == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (a->x_stride < a->hidden ||
      (a->residual && (a->residual_stride < a->hidden || a->residual_out_stride < a->hidden)))
    return MOE_ERR_INVALID_ARG;
  if (!at(a->x, 2) || !at(a->weight, a->weight_dtype == MOE_LAYER_FP32 ? 4 : 2) || !at(a->residual, 2) ||
      !at(a->residual_out, 2) || !at(a->y_out, 2) || !at(a->smooth, 4) || !at(a->q_scale, 4))
    return MOE_ERR_ALIGNMENT;
  return done(moe_layer::launch_norm(*a, sm_count(), static_cast<cudaStream_t>(stream)));
}

int moe_layer_w4_linear(const moe_layer_w4_args_t* a, void* stream) {
  if (!a || (!act(a->x_dtype) && a->x_dtype != MOE_LAYER_INT8) || (!act(a->out_dtype) && a->out_dtype != MOE_LAYER_FP32) ||
      (!act(a->scale_dtype) && a->scale_dtype != MOE_LAYER_FP32))
    return MOE_ERR_INVALID_ARG;
  // (the last round of tiles can go 16 x 16 x SMs rows past n, and row numbers are 32 bits)
  if (a->m < 0 || a->m > 1000000 || a->n < 1 || a->n > kMostRows || a->k < 32 || a->k > 65536 || a->group < 32 ||
      (a->group != 32 && a->group != 64 && a->group % 128) || a->k % a->group)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a->m == 0) return MOE_OK;
  if (!a->x || !a->w || !a->w_scale || !a->y || (a->x_scale != nullptr) != (a->x_dtype == MOE_LAYER_INT8) ||
      a->x_stride < a->k)
    return MOE_ERR_INVALID_ARG;
  const int xsize = a->x_dtype == MOE_LAYER_INT8 ? 1 : 2;
  if (!at(a->x, 16) || a->x_stride * xsize % 16 || !at(a->w, 16) ||
      !at(a->w_scale, a->scale_dtype == MOE_LAYER_FP32 ? 4 : 2) || !at(a->x_scale, 4) ||
      !at(a->y, a->out_dtype == MOE_LAYER_FP32 ? 4 : 2))
    return MOE_ERR_ALIGNMENT;
  const int sms = sm_count();
  if (!sms) return MOE_ERR_CUDA;
  return done(moe_layer::launch_w4(*a, sms, static_cast<cudaStream_t>(stream)));
}

int moe_layer_kv_append(const moe_layer_kv_append_args_t* a, void* stream) {
  if (!a || !act(a->dtype)) return MOE_ERR_INVALID_ARG;
  if (int rc = check_cache(a->cache)) return rc;
  if (a->tokens < 0 || a->batch < 0 || a->batch > 4096 || a->max_pages < 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a->tokens == 0 || a->batch == 0 || a->max_pages == 0) return MOE_OK;
  if (!a->k_new || !a->v_new || !a->page_table || !a->start) return MOE_ERR_INVALID_ARG;
  if (!a->cu_tokens && a->tokens != a->batch) return MOE_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(a->cache.kv_heads) * a->cache.head_dim;
  if (a->k_stride < row || a->v_stride < row || a->table_stride < a->max_pages) return MOE_ERR_INVALID_ARG;
  if (!at(a->k_new, 16) || !at(a->v_new, 16) || a->k_stride % 8 || a->v_stride % 8 || !at(a->page_table, 4) ||
      !at(a->start, 4) || !at(a->cu_tokens, 4))
    return MOE_ERR_ALIGNMENT;
  return done(moe_layer::launch_append(*a, static_cast<cudaStream_t>(stream)));
}

int moe_layer_kv_attention_workspace_size(int32_t head_dim, size_t* workspace_bytes) {
  if (!workspace_bytes) return MOE_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MOE_ERR_UNSUPPORTED_SHAPE;
  const int sms = sm_count();
  if (!sms) return MOE_ERR_CUDA;
  *workspace_bytes = moe_layer::attention_workspace(head_dim, sms);
  return MOE_OK;
}

int moe_layer_kv_attention(const moe_layer_kv_attention_args_t* a, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (!a || !act(a->dtype)) return MOE_ERR_INVALID_ARG;
  if (int rc = check_cache(a->cache)) return rc;
  if (a->tokens < 0 || a->batch < 0 || a->batch > 4096 || a->max_pages < 0 || a->max_q < 1 || a->group_size < 1 ||
      a->group_size > 128 || a->max_q > (1 << 24))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a->window < 0 || std::isnan(a->sm_scale)) return MOE_ERR_INVALID_ARG;
  if (a->tokens == 0 || a->batch == 0) return MOE_OK;
  if (!a->q || !a->out || (!a->page_table && a->max_pages > 0) || !a->seq_lens || !workspace) return MOE_ERR_INVALID_ARG;
  if (!a->cu_q && (a->tokens != a->batch || a->max_q != 1)) return MOE_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(a->cache.kv_heads) * a->group_size * a->cache.head_dim;
  if (a->q_stride < row || a->table_stride < a->max_pages) return MOE_ERR_INVALID_ARG;
  if (!at(a->q, 16) || !at(a->out, 16) || a->q_stride % 8 || !at(a->page_table, 4) || !at(a->seq_lens, 4) ||
      !at(a->cu_q, 4) || !at(workspace, 256))
    return MOE_ERR_ALIGNMENT;
  const int sms = sm_count();
  if (!sms) return MOE_ERR_CUDA;
  if (workspace_bytes < moe_layer::attention_workspace(a->cache.head_dim, sms)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return done(moe_layer::launch_attention(*a, workspace, sms, static_cast<cudaStream_t>(stream)));
}

int moe_layer_kv_attention_status(const void* workspace, void* stream) {
  if (!workspace) return MOE_ERR_INVALID_ARG;
  if (!at(workspace, 256)) return MOE_ERR_ALIGNMENT;
  int32_t words[4] = {0, 0, 0, 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(words, workspace, sizeof(words), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return MOE_ERR_CUDA;
  return words[1] ? MOE_ERR_DEVICE_TIMEOUT : MOE_OK;
}

int moe_layer_norm_add_rmsnorm_quant(const moe_layer_norm_pair_args_t* a, void* stream) {
  if (!a || !act(a->dtype) || (a->weight_dtype != a->dtype && a->weight_dtype != MOE_LAYER_FP32))
    return MOE_ERR_INVALID_ARG;
  if (a->rows < 0 || a->hidden < 1 || a->hidden > 16384) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!(a->eps >= 0.0f) || !std::isfinite(a->eps) || !std::isfinite(a->branch_scale)) return MOE_ERR_INVALID_ARG;
  if (a->rows == 0) return MOE_OK;
  if (!a->x || !a->residual || !a->post_weight || !a->weight || !a->residual_out ||
      (a->q == nullptr) != (a->q_scale == nullptr) || (!a->q && !a->y_out))
    return MOE_ERR_INVALID_ARG;
  if (a->x_stride < a->hidden || a->residual_stride < a->hidden || a->residual_out_stride < a->hidden ||
      (a->gate && a->gate_stride != 0 && a->gate_stride < a->hidden))
    return MOE_ERR_INVALID_ARG;
  const size_t wsize = a->weight_dtype == MOE_LAYER_FP32 ? 4 : 2;
  if (!at(a->x, 2) || !at(a->residual, 2) || !at(a->gate, 2) || !at(a->residual_out, 2) || !at(a->y_out, 2) ||
      !at(a->post_weight, wsize) || !at(a->weight, wsize) || !at(a->smooth, 4) || !at(a->q_scale, 4))
    return MOE_ERR_ALIGNMENT;
  return done(moe_layer::launch_norm_pair(*a, static_cast<cudaStream_t>(stream)));
}

int moe_layer_w8_linear_workspace_size(int32_t m, int32_t n, int32_t k, size_t* workspace_bytes) {
  if (!workspace_bytes) return MOE_ERR_INVALID_ARG;
  if (!w8_sizes(m, n, k)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const int sms = sm_count();
  if (!sms) return MOE_ERR_CUDA;
  *workspace_bytes = m ? moe_layer::w8_workspace(m, n, k, sms) : 0;
  return MOE_OK;
}

int moe_layer_w8_linear(const moe_layer_w8_args_t* a, void* workspace, size_t workspace_bytes, void* stream) {
  if (!a || (!act(a->out_dtype) && a->out_dtype != MOE_LAYER_FP32) ||
      (!act(a->scale_dtype) && a->scale_dtype != MOE_LAYER_FP32))
    return MOE_ERR_INVALID_ARG;
  if (!w8_sizes(a->m, a->n, a->k)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a->m == 0) return MOE_OK;
  if (!a->x || !a->x_scale || !a->w || !a->w_scale || !a->y || a->x_stride < a->k) return MOE_ERR_INVALID_ARG;
  if (!at(a->x, 16) || a->x_stride % 16 || !at(a->w, 16) || !at(a->x_scale, 4) ||
      !at(a->w_scale, a->scale_dtype == MOE_LAYER_FP32 ? 4 : 2) || !at(a->y, a->out_dtype == MOE_LAYER_FP32 ? 4 : 2) ||
      !at(workspace, 256))
    return MOE_ERR_ALIGNMENT;
  const int sms = sm_count();
  if (!sms) return MOE_ERR_CUDA;
  const size_t need = moe_layer::w8_workspace(a->m, a->n, a->k, sms);
  if (need && !workspace) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return done(moe_layer::launch_w8(*a, workspace, sms, static_cast<cudaStream_t>(stream)));
}

int moe_layer_w8_linear_status(const void* workspace, void* stream) {
  return moe_layer_kv_attention_status(workspace, stream);  // the same words
}

int moe_layer_page_plan(const moe_layer_page_plan_args_t* a, void* stream) {
  if (!a) return MOE_ERR_INVALID_ARG;
  if (a->batch < 0 || a->batch > 4096 || a->max_pages < 0 || a->num_pages < 0 || a->num_free < 0 || a->tokens < 0 ||
      static_cast<int64_t>(a->batch) * a->max_pages > INT32_MAX)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a->page_size != 16 && a->page_size != 32 && a->page_size != 64 && a->page_size != 128)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!a->taken_out || !a->unplaced || !a->cu_tokens ||
      (a->batch > 0 && (!a->held || !a->new_tokens || !a->seq_lens || (a->max_pages > 0 && !a->page_table))) ||
      (a->num_free > 0 && !a->free_pages) || (a->batch > 0 && a->table_stride < a->max_pages))
    return MOE_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(a->page_table), static_cast<const void*>(a->held),
                        static_cast<const void*>(a->new_tokens), static_cast<const void*>(a->free_pages),
                        static_cast<const void*>(a->taken), static_cast<const void*>(a->taken_out),
                        static_cast<const void*>(a->unplaced), static_cast<const void*>(a->cu_tokens),
                        static_cast<const void*>(a->seq_lens), static_cast<const void*>(a->sequence),
                        static_cast<const void*>(a->position)})
    if (!at(p, 4)) return MOE_ERR_ALIGNMENT;
  if (!at(a->slot, 8)) return MOE_ERR_ALIGNMENT;
  return done(moe_layer::launch_page_plan(*a, static_cast<cudaStream_t>(stream)));
}

int moe_layer_token_logprobs(const moe_layer_logprobs_args_t* a, void* stream) {
  if (!a || (!act(a->dtype) && a->dtype != MOE_LAYER_FP32) || (a->tokens_64 != 0 && a->tokens_64 != 1))
    return MOE_ERR_INVALID_ARG;
  if (a->rows < 0 || a->vocab < 1 || a->num_tokens < 0 || a->top < 0 || a->top > 32 || a->top > a->vocab)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a->rows == 0) return MOE_OK;
  if (!a->logits || a->logits_stride < a->vocab || (a->num_tokens > 0 && (!a->tokens || !a->logprob)) ||
      (a->top > 0 && (!a->top_logprob || !a->top_id)))
    return MOE_ERR_INVALID_ARG;
  if (!at(a->logits, a->dtype == MOE_LAYER_FP32 ? 4 : 2) || !at(a->tokens, a->tokens_64 ? 8 : 4) || !at(a->logprob, 4) ||
      !at(a->entropy, 4) || !at(a->top_logprob, 4) || !at(a->top_id, 4))
    return MOE_ERR_ALIGNMENT;
  const int sms = sm_count();
  if (!sms) return MOE_ERR_CUDA;
  return done(moe_layer::launch_logprobs(*a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
