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

}  // extern "C"
