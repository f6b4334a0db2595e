/* moe_layer.h -- C ABI of the decoder-layer operators around the fused MoE
 * expert block (moe_fused.h), in the same library.
 *
 *   moe_layer_add_rmsnorm_quant  residual addition, RMS norm, per-token INT8
 *                                quantisation (the block's own quant convention)
 *   moe_layer_w4_linear          products with 4-bit weights and group scales for
 *                                few tokens (projections, output head, router gate)
 *   moe_layer_kv_append          quantised write of new keys and values into a
 *                                paged INT8 cache, one scale a page and head
 *   moe_layer_kv_attention       attention of new tokens over that cache
 *
 * Conventions are those of moe_fused.h: device pointers owned by the caller,
 * no device memory allocated here, work enqueued asynchronously on `stream`
 * (a cudaStream_t as void*) of the current device, MOE_OK or a negative
 * MOE_ERR_* code, nothing launched by a call that returns an error.  There is
 * no handle and no state: a call reads nothing that an earlier call left in
 * the workspace.  Strides count elements, and the innermost dimension is
 * contiguous.  Pointers need only the alignment that each call states.
 */
#ifndef MOE_LAYER_H
#define MOE_LAYER_H

#include <stddef.h>
#include <stdint.h>

#include "moe_fused.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define MOE_LAYER_BF16 0
#define MOE_LAYER_FP16 1
#define MOE_LAYER_FP32 2
#define MOE_LAYER_INT8 3

/* Residual addition, RMS norm and INT8 quant, row t of `rows`, in fp32:
 *   s = x[t] + residual[t]          (x[t] without residual)
 *   residual_out[t] = T(s)          T: rounding to `dtype`, to nearest even
 *   y = s * (1 / sqrt(mean(s^2) + eps)) * weight
 *   y_out[t] = T(y)
 *   z = y * smooth                  (y without smooth)
 *   a = max(max|z|, 1e-4), m = 127 / a
 *   q[t] = clamp(rne(z * m), -127, 127), q_scale[t] = 1 / m
 * The norm and the quant take the unrounded s and y.  A row that holds a NaN
 * or an infinity gets a NaN scale, so that q * q_scale is NaN.
 * x, residual, residual_out: [rows, hidden] of `dtype` (BF16 or FP16) with
 * their own row strides (>= hidden); residual_out may be residual itself
 * (same stride) and y_out may be x.  residual and residual_out are both
 * given or both NULL.  weight: [hidden] of `weight_dtype` (`dtype` or FP32).
 * smooth: [hidden] fp32 or NULL.  y_out: [rows, hidden] of `dtype` or NULL.
 * q: [rows, hidden], q_scale: [rows].  1 <= hidden <= 16384 (any number),
 * rows >= 0.  Every pointer aligned to its element. */
typedef struct {
  const void* x;
  const void* residual;
  const void* weight;
  const float* smooth;
  void* residual_out;
  void* y_out;
  int8_t* q;
  float* q_scale;
  int64_t x_stride;
  int64_t residual_stride;
  int64_t residual_out_stride;
  int32_t rows;
  int32_t hidden;
  int32_t dtype;
  int32_t weight_dtype;
  float eps;
} moe_layer_norm_args_t;
int moe_layer_add_rmsnorm_quant(const moe_layer_norm_args_t* args, void* stream);

/* Products with 4-bit weights:
 *   y[m, n] = x_scale[m] * sum over groups g of w_scale[n, g] *
 *             sum over k in g of x[m, k] * (code[n, k] - zero[n, g])
 * x: [m, k] of `x_dtype` (BF16, FP16, or INT8 codes with x_scale [m] fp32;
 * x_scale is NULL for the other two), row stride x_stride (a multiple of 16
 * bytes; 16-byte aligned base).  w: [n, k/2] uint8, 16-byte aligned, the code
 * of an even k in the low four bits, of the next k in the high four.  w_scale:
 * [n, k/group] of `scale_dtype` (BF16, FP16 or FP32).  w_zero: [n, k/group]
 * uint8 in 0..15 (the low four bits count), NULL for 8 everywhere.  y: [m, n]
 * of `out_dtype` (BF16, FP16 or FP32), dense.
 * group: 32, 64 or a multiple of 128; k: a multiple of group, 32 <= k <=
 * 65536; 1 <= n < 2^31 - 2^20; 0 <= m <= 1000000.  x is held in fp16 with a
 * power of two for every 128 k of a row: exact but for elements 2^18 below the
 * largest of them, which keep a step of 2^-28 of it.  Products are exact, sums are
 * fp32, y is rounded once; elements of x and y below 2^-110 may lose bits or
 * vanish.  A row of x that holds a NaN or an infinity gives no finite value in its
 * own row of y and touches no other.  The call is made for few rows (the weights
 * are read once for every 16 rows of x); it is right for any m. */
typedef struct {
  const void* x;
  const float* x_scale;
  const uint8_t* w;
  const void* w_scale;
  const uint8_t* w_zero;
  void* y;
  int64_t x_stride;
  int32_t m;
  int32_t n;
  int32_t k;
  int32_t group;
  int32_t x_dtype;
  int32_t scale_dtype;
  int32_t out_dtype;
} moe_layer_w4_args_t;
int moe_layer_w4_linear(const moe_layer_w4_args_t* args, void* stream);

/* A paged INT8 cache of keys and values.  Page p holds page_size tokens of
 * every kv head; the value of token slot s, channel d of head h is
 *   k[p, h, s, d] * k_scale[p, h]         (v likewise)
 * with k, v: int8, each head's [page_size, head_dim] contiguous, 16-byte
 * aligned, page and head strides in elements (multiples of 16), and the scales
 * fp32 [num_pages, kv_heads] with a page stride (heads contiguous).
 * Row b of page_table ([batch, max_pages] int32, row stride table_stride)
 * lists the pages of sequence b in order; entries past its length are not read
 * (without any, max_pages is 0 and page_table may be NULL: no keys).
 * page_size: 16, 32, 64 or 128; head_dim: 64 or 128; 1 <= kv_heads <= 1024;
 * 0 <= batch <= 4096. */
typedef struct {
  int8_t* k;
  int8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t page_stride;
  int64_t head_stride;
  int64_t scale_stride;
  int32_t num_pages;
  int32_t kv_heads;
  int32_t page_size;
  int32_t head_dim;
} moe_layer_kv_cache_t;

/* Write new keys and values.  Sequence b gets tokens cu_tokens[b] ..
 * cu_tokens[b + 1] - 1 of k_new / v_new (token b alone when cu_tokens is
 * NULL) at positions start[b], start[b] + 1, ...  For every touched page and
 * head, K and V each by themselves:
 *   a page that the call starts (its slot 0 is written): scale = max(amax,
 *     1e-4) / 127 over the new tokens that it gets;
 *   a page that already holds tokens: scale' = max(scale, amax / 127); if it
 *     grew, the codes held below the first new slot become
 *     clamp(rne(code * (scale / scale')), -127, 127);
 *   new codes = clamp(rne(x * (1 / scale')), -127, 127).
 * (Slots are filled in order: what a started page held before is forgotten.)
 * A NaN or an infinity among a page's tokens becomes the scale of that page and
 * head, and with it all that they hold.
 * k_new, v_new: [tokens, kv_heads, head_dim] of `dtype` (BF16 or FP16) with
 * token strides (multiples of 8) and heads dense, 16-byte aligned.  A token whose page-table
 * entry is outside [0, num_pages) or whose position is outside [0, max_pages *
 * page_size) is not written.  No page may appear twice among those written. */
typedef struct {
  moe_layer_kv_cache_t cache;
  const void* k_new;
  const void* v_new;
  const int32_t* page_table;
  const int32_t* start;
  const int32_t* cu_tokens;
  int64_t k_stride;
  int64_t v_stride;
  int64_t table_stride;
  int32_t tokens;
  int32_t batch;
  int32_t max_pages;
  int32_t dtype;
} moe_layer_kv_append_args_t;
int moe_layer_kv_append(const moe_layer_kv_append_args_t* args, void* stream);

/* Attention over the cache.  Sequence b has the query tokens cu_q[b] ..
 * cu_q[b + 1] - 1 (token b alone when cu_q is NULL), qlen of them, and
 * seq_lens[b] keys, its query tokens' own (already appended) among them.
 * Query token j stands at position p = seq_lens[b] - qlen + j (whatever max_q
 * is) and sees the keys i with 0 <= i <= p, and i > p - window where window > 0.
 * Query head n uses kv head n / group_size:
 *   out[t, n] = sum_i softmax_i(sm_scale * <q[t, n], key_i>) * value_i
 * and zeros where no key is seen.  Keys on a page-table entry outside [0,
 * num_pages) are not seen.  A scale that is not finite reaches only the query
 * tokens that see a key of its page, whose outputs are then not finite; an element
 * of q that is not, its row.  Lengths are held to [0, max_pages * page_size].
 * q: [tokens, kv_heads * group_size, head_dim] of `dtype` (BF16 or FP16), token stride
 * q_stride (a multiple of 8), heads dense, 16-byte aligned.  out: the same
 * shape and type, dense, 16-byte aligned.  1 <= group_size <= 128.  max_q: the
 * largest number of query tokens of a sequence (1 without cu_q); a larger one in
 * cu_q leaves that sequence's tokens past the first max_q unwritten and the others
 * as they are.
 * Scores, softmax statistics and sums are fp32, exponentials and logarithms
 * (base 2) good to about 2^-22.  For the product with the values a softmax weight
 * times its page's scale of V is rounded to fp16: 11 bits down to 2^-21 of the
 * row's largest such product, below that a step of 2^-31 of it (for scales that lie
 * within 2^64 of one another).  Query rows are fp16 too, after a power of two a
 * row: elements below 2^-14 (fp16) or 2^-17 (bf16) of the row's largest keep a
 * step of 2^-24 of it.  Where max_q * group_size is 64 or more the products run on
 * the tensor memory units.
 * workspace: moe_layer_kv_attention_workspace_size bytes, 256-byte aligned,
 * no initial content needed; calls that share one must be ordered. */
typedef struct {
  moe_layer_kv_cache_t cache;
  const void* q;
  void* out;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  int64_t q_stride;
  int64_t table_stride;
  int32_t tokens;
  int32_t batch;
  int32_t max_pages;
  int32_t max_q;
  int32_t group_size;
  int32_t window;
  int32_t dtype;
  float sm_scale;
} moe_layer_kv_attention_args_t;
/* Bytes for any call with this head_dim on the current device. */
int moe_layer_kv_attention_workspace_size(int32_t head_dim, size_t* workspace_bytes);
int moe_layer_kv_attention(const moe_layer_kv_attention_args_t* args, void* workspace, size_t workspace_bytes,
                           void* stream);
/* Synchronise `stream` and say whether a wait inside the last call that used
 * `workspace` gave up (MOE_ERR_DEVICE_TIMEOUT; its output is then not to be
 * used).  Every wait inside a kernel is bounded.  A call without tokens or
 * sequences does not use the workspace; one that no call has used, and whose
 * first 256 bytes are not zero, has nothing to say. */
int moe_layer_kv_attention_status(const void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LAYER_H */
