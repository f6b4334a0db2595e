// Log probabilities of given tokens, entropy, and the top alternatives of rows
// of logits, in one pass over them.
//
// Every thread keeps a running maximum M of what it has seen and the sums
//   S = sum exp(l - M),  U = sum exp(l - M) (l - M)
// (in powers of two), moved to a new M as often as one turns up; sums of threads,
// warps and CTAs join the same way.  logprob(c) = (l_c - M) - log S, and the
// entropy is log S - U / S.
// The top logits are kept by warps: lane r holds the r-th best of what the warp
// has seen, as one number that orders by value and then by the lower index.  A
// thread's maximum of its 64 bytes, which the sums need anyway, says whether any
// of them can enter; the worst entry of any warp's full list bounds all of them.
// A row is one CTA's, or a cluster's where there are few rows.
#include "layer_ops.cuh"

namespace moe_layer {
namespace {

constexpr int kMaxWarps = 8;
constexpr int kMaxCluster = 8;
constexpr int kBlocks = 4;  // 16-byte blocks that a thread has in flight
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -INFINITY;

// Larger for larger values (-0 as 0); NaN does not get here.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t index) {
  return static_cast<uint64_t>(order_of(v)) << 32 | static_cast<uint32_t>(~index);
}

struct Sums {
  float m, s, u;  // u in powers of two
};
// the sums of a and b with one reference; a side without elements (m = -inf) adds nothing
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
  const float m = fmaxf(a.m, b.m);
  if (m == kNone) return Sums{m, __fadd_rn(a.s, b.s), 0.0f};  // a NaN stays one
  const float da = fmaxf(__fmul_rn(a.m - m, kLog2e), -200.0f), db = fmaxf(__fmul_rn(b.m - m, kLog2e), -200.0f);
  const float ea = exp2_fast(da), eb = exp2_fast(db);
  Sums r;
  r.m = m;
  r.s = __fmaf_rn(a.s, ea, __fmul_rn(b.s, eb));
  r.u = __fmaf_rn(ea, __fmaf_rn(a.s, da, a.u), __fmul_rn(eb, __fmaf_rn(b.s, db, b.u)));
  return r;
}

// what a CTA leaves for the join of its cluster
struct Part {
  Sums sums;
  uint64_t keys[32];
};

// one sorted list (lane 0 the best) of the best 32 of two
__device__ __forceinline__ uint64_t merge_lists(uint64_t a, uint64_t b) {
  const int lane = threadIdx.x & 31;
  const uint64_t other = __shfl_sync(0xffffffffu, b, 31 - lane);
  uint64_t v = a > other ? a : other;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
    v = ((lane & o) == 0) == (v > w) ? v : w;
  }
  return v;
}
// the lanes' values sorted, lane 0 the largest
__device__ __forceinline__ uint32_t sort_lanes(uint32_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const uint32_t w = __shfl_xor_sync(0xffffffffu, v, o);
      const bool larger = ((lane & o) == 0) == ((lane & size) == 0);
      v = larger ? max(v, w) : min(v, w);
    }
  }
  return v;
}

template <typename T>
struct Block {  // 16 bytes of a row
  static constexpr int kN = 16 / sizeof(T);
  __device__ static __forceinline__ void take(const uint4& b, float (&v)[kN]) {
    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 2) {
        const float2 f = unpack2<T>(w[j]);
        v[2 * j] = f.x, v[2 * j + 1] = f.y;
      } else {
        v[j] = __uint_as_float(w[j]);
      }
    }
  }
};
template <typename T>
__device__ __forceinline__ float widen(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else return static_cast<float>(v);
}

template <typename T>
__global__ void __launch_bounds__(kMaxWarps * 32, 4) logprobs_kernel(const moe_layer_logprobs_args_t a) {
  constexpr int N = Block<T>::kN, E = N * kBlocks;
  __shared__ Part s_part;
  __shared__ Sums s_sums[kMaxWarps];
  __shared__ uint64_t s_keys[kMaxWarps][32];
  __shared__ uint32_t s_bound;  // order of a value that `top` logits of the row reach
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  uint32_t rank, ctas;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const int64_t row = blockIdx.x / ctas;
  const int top = a.top;
  const T* p = static_cast<const T*>(a.logits) + row * a.logits_stride;
  // The row lies in 16-byte blocks of memory, `off` elements past the start of the first.  The first and the last may
  // hold elements that are not the row's: those are read one by one.
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
  const int64_t blocks = (off + static_cast<int64_t>(a.vocab) + N - 1) / N;
  const uint4* base = reinterpret_cast<const uint4*>(p - off);
  if (threadIdx.x == 0) s_bound = 0;
  __syncthreads();

  Sums sum{kNone, 0.0f, 0.0f};
  uint64_t list = 0;              // below every key
  uint64_t least = 0;             // the list's entry number `top`
  float bound = kNone;            // its value, or a larger one that `top` logits reach: smaller ones need not be looked at
  const int64_t tile = static_cast<int64_t>(nw) * 32 * kBlocks * ctas;
  for (int64_t t0 = (static_cast<int64_t>(rank) * nw + warp) * 32 * kBlocks; t0 < blocks; t0 += tile) {
    uint4 raw[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const int64_t n = t0 + b * 32 + lane, e = n * N - off;
      if (e >= 0 && e + N <= a.vocab) raw[b] = __ldcs(base + n);
    }
    float v[E];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const int64_t n = t0 + b * 32 + lane, e = n * N - off;
      float f[N];
      if (e >= 0 && e + N <= a.vocab) {
        Block<T>::take(raw[b], f);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] = e + j >= 0 && e + j < a.vocab ? widen<T>(p[e + j]) : kNone;
      }
#pragma unroll
      for (int j = 0; j < N; ++j) v[b * N + j] = f[j];
    }
    float most = v[0];
#pragma unroll
    for (int j = 1; j < E; ++j) most = fmaxf(most, v[j]);
    if (most > sum.m) {
      const float d = fmaxf(__fmul_rn(sum.m - most, kLog2e), -200.0f), e = exp2_fast(d);
      sum.u = __fmul_rn(e, __fmaf_rn(sum.s, d, sum.u));
      sum.s = __fmul_rn(sum.s, e);
      sum.m = most;
    }
    const float ref = sum.m == kNone ? 0.0f : sum.m;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float d = __fmul_rn(__fsub_rn(v[j], ref), kLog2e), e = exp2_fast(d);
      sum.s = __fadd_rn(sum.s, e);
      sum.u = __fmaf_rn(e, fmaxf(d, -200.0f), sum.u);  // (-inf has e = 0)
    }
    if (top == 0) continue;
    bound = fmaxf(bound, value_of(max(*static_cast<volatile uint32_t*>(&s_bound), order_of(kNone))));
    uint32_t hit = __ballot_sync(0xffffffffu, most >= bound);
    if (!hit) continue;
    if (__popc(hit) >= top) {  // `top` lanes hold a logit of at least their own maximum
      const uint32_t sorted = sort_lanes(order_of(most));
      bound = fmaxf(bound, value_of(__shfl_sync(0xffffffffu, sorted, top - 1)));
    }
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int64_t e = (t0 + (j / N) * 32 + lane) * N - off + j % N;
      const bool in = e >= 0 && e < a.vocab && v[j] >= bound;
      const uint64_t key = in ? key_of(v[j], static_cast<uint32_t>(e)) : 0;
      uint32_t todo = __ballot_sync(0xffffffffu, key > least);
      while (todo) {
        const int from = __ffs(todo) - 1;
        todo &= todo - 1;
        const uint64_t k = __shfl_sync(0xffffffffu, key, from);
        if (k <= least) continue;
        const int at = __popc(__ballot_sync(0xffffffffu, list > k));
        const uint64_t up = __shfl_up_sync(0xffffffffu, list, 1);
        list = lane < at ? list : lane == at ? k : up;
        least = __shfl_sync(0xffffffffu, list, top - 1);
      }
    }
    if (least) {
      const uint32_t o = static_cast<uint32_t>(least >> 32);
      bound = fmaxf(bound, value_of(o));
      if (lane == 0) atomicMax(&s_bound, o);
    }
  }

  // threads, warps, CTAs
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Sums b{__shfl_xor_sync(0xffffffffu, sum.m, o), __shfl_xor_sync(0xffffffffu, sum.s, o),
                 __shfl_xor_sync(0xffffffffu, sum.u, o)};
    sum = join(sum, b);
  }
  if (lane == 0) s_sums[warp] = sum;
  if (top) s_keys[warp][lane] = list;
  __syncthreads();
  if (warp == 0) {
    sum = s_sums[0];
    for (int w = 1; w < nw; ++w) {
      sum = join(sum, s_sums[w]);
      if (top) list = merge_lists(list, s_keys[w][lane]);
    }
    if (lane == 0) s_part.sums = sum;
    s_part.keys[lane] = list;
  }
  if (ctas > 1) {
    cluster_sync();
    if (warp == 0 && rank == 0) {
      const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(&s_part));
      for (uint32_t r = 1; r < ctas; ++r) {
        const Sums b{cluster_read(at, r), cluster_read(at + 4, r), cluster_read(at + 8, r)};
        sum = join(sum, b);
        if (top) {
          const uint32_t k = at + offsetof(Part, keys) + lane * 8;
          const uint64_t lo = __float_as_uint(cluster_read(k, r)), hi = __float_as_uint(cluster_read(k + 4, r));
          list = merge_lists(list, hi << 32 | lo);
        }
      }
    }
    cluster_sync();  // no CTA ends while its part is read
    if (rank != 0) return;
  }
  if (warp != 0) return;
  // a NaN anywhere is one in s; so is +inf (less itself)
  const bool broken = !(sum.s == sum.s), none = broken || sum.m == kNone;
  const float nan = __uint_as_float(0x7FC00000u);
  const float log_s = logf(sum.s);
  if (lane == 0 && a.entropy) a.entropy[row] = none ? nan : __fsub_rn(log_s, __fmul_rn(kLn2, __fdiv_rn(sum.u, sum.s)));
  if (lane < top) {
    const float l = value_of(static_cast<uint32_t>(list >> 32));
    a.top_id[row * top + lane] = broken ? -1 : static_cast<int32_t>(~static_cast<uint32_t>(list));
    a.top_logprob[row * top + lane] = none ? nan : __fsub_rn(__fsub_rn(l, sum.m), log_s);
  }
  for (int64_t j = lane; j < a.num_tokens; j += 32) {
    const int64_t i = row * a.num_tokens + j;
    const int64_t c = a.tokens_64 ? static_cast<const int64_t*>(a.tokens)[i] : static_cast<const int32_t*>(a.tokens)[i];
    float r = kNone;
    if (c >= 0 && c < a.vocab) r = __fsub_rn(__fsub_rn(widen<T>(p[c]), sum.m), log_s);
    a.logprob[i] = none ? nan : r;
  }
}

template <typename T>
cudaError_t launch_typed(const moe_layer_logprobs_args_t& a, int num_sms, cudaStream_t s) {
  constexpr int64_t kTile = 32 * kBlocks * (16 / sizeof(T));  // elements of a warp's step
  const int64_t steps = (a.vocab + kTile - 1) / kTile;
  int warps = 1, ctas = 1;
  while (warps < kMaxWarps && warps < steps) warps *= 2;
  while (ctas < kMaxCluster && ctas * warps < steps && static_cast<int64_t>(a.rows) * ctas < 2 * num_sms) ctas *= 2;
  moe_layer_logprobs_args_t arg = a;
  void* args[] = {&arg};
  return launch_after((const void*)logprobs_kernel<T>, dim3(static_cast<unsigned>(a.rows) * ctas), dim3(warps * 32), args, 0,
                      s, ctas);
}

}  // namespace

cudaError_t launch_logprobs(const moe_layer_logprobs_args_t& a, int num_sms, cudaStream_t s) {
  if (a.dtype == MOE_LAYER_BF16) return launch_typed<__nv_bfloat16>(a, num_sms, s);
  if (a.dtype == MOE_LAYER_FP16) return launch_typed<__half>(a, num_sms, s);
  return launch_typed<float>(a, num_sms, s);
}

}  // namespace moe_layer
