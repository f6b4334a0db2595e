// Quantised write of new keys and values into the paged INT8 cache.
//
// One CTA takes one page and one kv head, K and V: the new tokens that fall on
// that page are at most twice page_size x head_dim elements, which stay in
// registers between the maximum and the rounding.  Each page is touched by
// one CTA alone, so nothing is atomic.  Bound by memory (2 bytes read and 1
// written an element) for prompts (4 ragged ones, 5035 tokens of 8 heads: 7.7 us),
// by latency for single tokens (64 of them: 2.3 us).  fp16 rows take more registers
// than bf16 ones (80 for 64 at pages of 64 x 128, 180 for 128 at 128 x 128), for 7.0
// us in place of 6.7 and 8.8 in place of 7.8 on prompts that start their pages.
//
// The CTAs know only bounds of the ragged lengths.  Sequence b owns the unit
// numbers from cu[b] / P + 2 b on, which leaves it floor(n / P) + 2, at least
// the pages that n tokens can touch; spare units end at once.
#include "layer_ops.cuh"

namespace moe_layer {
namespace {

// CHUNKS: chunks of 8 elements that a thread has at most
template <typename T, int D, int THREADS, int CHUNKS>
__global__ void __launch_bounds__(THREADS) kv_append_kernel(const moe_layer_kv_append_args_t a) {
  constexpr int kRowChunks = D / 8;  // of a token
  __shared__ uint32_t s_max[2][THREADS / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int P = a.cache.page_size;
  const int u = blockIdx.x, head = blockIdx.y;

  int b = u, tok0 = u, n = 1, unit = 0;
  if (a.cu_tokens) {
    // the last b with cu[b] / P + 2 b <= u: 33-ary search, one probe a lane
    int lo = 0, hi = a.batch;  // the answer lies in [lo, hi)
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = lo + lane * step;
      const bool ok = at < hi && a.cu_tokens[at] / P + 2 * at <= u;
      const int k = 31 - __clz(__ballot_sync(0xffffffffu, ok) | 1u);
      lo += k * step;
      hi = min(hi, lo + step);
    }
    b = lo;
    tok0 = max(a.cu_tokens[b], 0);
    n = min(a.cu_tokens[b + 1], a.tokens) - tok0;
    unit = u - (a.cu_tokens[b] / P + 2 * b);
  }
  const int start = a.start[b];
  if (n <= 0 || start < 0) return;
  const int64_t index = start / P + unit;  // page of the sequence
  const int64_t first = index * P;
  const int lo = static_cast<int>(max(static_cast<int64_t>(start) - first, static_cast<int64_t>(0)));
  const int hi = static_cast<int>(min(static_cast<int64_t>(start) + n - first, static_cast<int64_t>(P)));
  if (hi <= lo || index >= a.max_pages) return;
  const int page = a.page_table[b * a.table_stride + index];
  if (page < 0 || page >= a.cache.num_pages) return;

  const int64_t t_lo = tok0 + (first + lo - start);  // the token at slot lo
  const int64_t code_at = page * a.cache.page_stride + head * a.cache.head_stride;
  const int64_t scale_at = page * a.cache.scale_stride + head;
  const int chunks = (hi - lo) * kRowChunks;
  uint4 v[2][CHUNKS];
  float old[2];
  uint32_t top[2] = {0u, 0u};
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const T* src = static_cast<const T*>(kv ? a.v_new : a.k_new) + head * D;
    const int64_t stride = kv ? a.v_stride : a.k_stride;
    old[kv] = lo > 0 ? (kv ? a.cache.v_scale : a.cache.k_scale)[scale_at] : 0.0f;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int i = c * THREADS + tid;
      v[kv][c] = make_uint4(0, 0, 0, 0);
      if (i < chunks)
        v[kv][c] = *reinterpret_cast<const uint4*>(src + (t_lo + i / kRowChunks) * stride + (i % kRowChunks) * 8);
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const uint32_t w[4] = {v[kv][c].x, v[kv][c].y, v[kv][c].z, v[kv][c].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack2<T>(w[j]);
        top[kv] = max(top[kv], max(abs_bits(f.x), abs_bits(f.y)));
      }
    }
    top[kv] = __reduce_max_sync(0xffffffffu, top[kv]);
    if (lane == 0) s_max[kv][tid >> 5] = top[kv];
  }
  __syncthreads();  // and every thread has read the old scales
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint32_t most = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) most = max(most, s_max[kv][w]);
    float amax = __uint_as_float(most);
    float to;
    if (lo == 0) {
      if (amax < kAmaxFloor) amax = kAmaxFloor;
      to = __fdiv_rn(amax, 127.0f);
    } else {
      const float grown = __fdiv_rn(amax, 127.0f);
      to = (grown > old[kv] || grown != grown) ? grown : old[kv];
    }
    int8_t* codes = (kv ? a.cache.v : a.cache.k) + code_at;
    if (lo > 0 && to > old[kv]) {
      // the page's scale grew: the codes that it holds move to the new one
      const float f = __fdiv_rn(old[kv], to);
      for (int i = tid; i < lo * D / 16; i += THREADS) {
        const uint4 q = reinterpret_cast<uint4*>(codes)[i];
        uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float s[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[e] = __fmul_rn(static_cast<float>(static_cast<int8_t>((w[j] >> (8 * e)) & 0xFFu)), f);
          w[j] = codes_of(s[0], s[1], s[2], s[3]);
        }
        reinterpret_cast<uint4*>(codes)[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    const float inv = __fdiv_rn(1.0f, to);
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int i = c * THREADS + tid;
      if (i < chunks) {
        const uint32_t w[4] = {v[kv][c].x, v[kv][c].y, v[kv][c].z, v[kv][c].w};
        uint32_t o[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = unpack2<T>(w[2 * j]), g = unpack2<T>(w[2 * j + 1]);
          o[j] = codes_of(__fmul_rn(f.x, inv), __fmul_rn(f.y, inv), __fmul_rn(g.x, inv), __fmul_rn(g.y, inv));
        }
        *reinterpret_cast<uint2*>(codes + (lo + i / kRowChunks) * D + (i % kRowChunks) * 8) = make_uint2(o[0], o[1]);
      }
    }
    if (__builtin_expect(to < 0x1p-126f, 0)) {
      // a held page's scale can be so small that its inverse is coarse or infinite: no code of -128 even so
#pragma unroll 1
      for (int i = tid; i < chunks; i += THREADS) {
        uint2* at = reinterpret_cast<uint2*>(codes + (lo + i / kRowChunks) * D + (i % kRowChunks) * 8);  // this thread's own
        *at = make_uint2(__vmaxs4(at->x, 0x81818181u), __vmaxs4(at->y, 0x81818181u));
      }
    }
    if (tid == 0) (kv ? a.cache.v_scale : a.cache.k_scale)[scale_at] = to;
  }
}

template <typename T, int D>
cudaError_t launch_typed(const moe_layer_kv_append_args_t& a, cudaStream_t s) {
  moe_layer_kv_append_args_t arg = a;
  void* args[] = {&arg};
  const int64_t most = a.cu_tokens ? static_cast<int64_t>(a.tokens) / a.cache.page_size + 2 * a.batch : a.batch;
  const dim3 grid(static_cast<unsigned>(most), a.cache.kv_heads);
  // single tokens: one chunk of 16 lanes at most, 128 threads for a page that has to be requantised
  if (!a.cu_tokens) return launch_after((const void*)kv_append_kernel<T, D, 128, 1>, grid, dim3(128), args, 0, s);
  const int chunks = a.cache.page_size * (D / 8) / 256;
  const void* k = chunks <= 1   ? (const void*)kv_append_kernel<T, D, 256, 1>
                  : chunks == 2 ? (const void*)kv_append_kernel<T, D, 256, 2>
                  : chunks == 4 ? (const void*)kv_append_kernel<T, D, 256, 4>
                                : (const void*)kv_append_kernel<T, D, 256, 8>;
  return launch_after(k, grid, dim3(256), args, 0, s);
}

}  // namespace

cudaError_t launch_append(const moe_layer_kv_append_args_t& a, cudaStream_t s) {
  if (a.dtype == MOE_LAYER_BF16)
    return a.cache.head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(a, s) : launch_typed<__nv_bfloat16, 128>(a, s);
  return a.cache.head_dim == 64 ? launch_typed<__half, 64>(a, s) : launch_typed<__half, 128>(a, s);
}

}  // namespace moe_layer
