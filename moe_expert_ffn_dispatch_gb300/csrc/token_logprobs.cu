// Log probabilities of given tokens, entropy, and the top alternatives of rows
// of logits, in one pass over them.
//
// Every thread keeps the largest logit M that it has seen and the sums
//   S = sum 2^d,  U = sum 2^d d,   d = (l - M) log2(e),
// moved to a new M as often as a larger logit turns up; sums of threads, warps and
// CTAs join the same way.  log p(c) = (l_c - M) - log S and the entropy is log S - (U /
// S) ln 2.  -inf is raised to a number that gives 2^d = 0 and keeps 2^d d from being
// NaN, except where M itself is so far out (kHuge, kFarDown) that this would change it.
// The top logits are kept by warps: lane r holds the r-th best of what the warp
// has seen, as one number that orders by value and then by the lower index.  A
// thread's maximum of its 64 bytes, which the sums need anyway, says whether any
// of them can enter; only the elements of lanes that say so are looked at.  The bound
// that they have to reach is the k-th largest of the threads' M, which k logits reach
// and few others: taken over the CTA in its first step and its fourth.
// A row is a CTA's, or a cluster's where there are few rows, or a warp's where it is short.
// Bound by memory and instructions: 2039 x 130001 bf16 88 us without alternatives, 6.0
// TB/s of 6.8; 108 with five of them (issue 75 %), 132 with twenty: the search of lanes that
// can enter.  64 rows 8.5 / 14.5 us (twenty), one row of fp32 with five 9.3: latency of a few
// steps and of the joins.
#include <type_traits>

#include "layer_ops.cuh"

namespace moe_layer {
namespace {

constexpr int kMaxWarps = 8;
constexpr int kMaxCluster = 8;
constexpr int kRowWarps = 4;  // rows of a CTA whose warps have one each
constexpr int kBlocks = 4;    // 16-byte blocks that a thread has in flight
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -INFINITY;
constexpr float kHuge = 1e30f;

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

template <typename T>
struct Type;
// kDown: what -inf is raised to, so that d stays finite; kFarDown: nothing is lost by that where M is above it
template <>
struct Type<__nv_bfloat16> {
  static constexpr float kFarDown = -1e30f;
  static constexpr uint32_t kDown = 0xFE96FE96u;  // -1e38
  static __device__ __forceinline__ uint32_t raise(uint32_t w) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(kDown));
    return r;
  }
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};
template <>
struct Type<__half> {
  static constexpr float kFarDown = -60000.0f;
  static constexpr uint32_t kDown = 0xFBFFFBFFu;  // -65504
  static __device__ __forceinline__ uint32_t raise(uint32_t w) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(kDown));
    return r;
  }
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};
template <>
struct Type<float> {
  static constexpr float kFarDown = -1e30f;
  static __device__ __forceinline__ uint32_t raise(uint32_t w) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(w)), "f"(-1e38f));
    return __float_as_uint(r);
  }
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
};

template <typename T>
__device__ __forceinline__ float widen(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else return static_cast<float>(v);
}
// two elements from word w on: both of it, or (fp32) it and the next
template <typename T>
__device__ __forceinline__ float2 pair_at(const uint32_t* w) {
  if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
  else return unpack2<T>(w[0]);
}

struct Sums {
  float m, s, u;  // m: the largest logit
};
template <typename T>
__device__ __forceinline__ bool far_out(float m) { return !(m > Type<T>::kFarDown && m < kHuge); }
// d of a logit against the largest, m, or what sums with the reference l are to be multiplied by for m, as a power of two
__device__ __forceinline__ float exponent(float l, float m) { return __fmul_rn(__fsub_rn(l, m), kLog2e); }
// the sums of a and b with one reference; a side without elements (m = -inf) adds nothing
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
  const float m = fmaxf(a.m, b.m);
  if (m == kNone) return Sums{m, __fadd_rn(a.s, b.s), 0.0f};  // a NaN stays one
  const float da = a.m == m ? 0.0f : fmaxf(exponent(a.m, m), -200.0f), db = b.m == m ? 0.0f : fmaxf(exponent(b.m, m), -200.0f);
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

// the best 32 of two sorted lists of 32-bit numbers, sorted
__device__ __forceinline__ uint32_t merge_orders(uint32_t a, uint32_t b) {
  const int lane = threadIdx.x & 31;
  uint32_t v = max(a, __shfl_sync(0xffffffffu, b, 31 - lane));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint32_t w = __shfl_xor_sync(0xffffffffu, v, o);
    v = (lane & o) == 0 ? max(v, w) : min(v, w);
  }
  return v;
}

// WARP_ROW: a warp takes a row by itself, kRowWarps rows a CTA
template <typename T, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? kRowWarps * 32 : kMaxWarps * 32, WARP_ROW ? 8 : 4)
    logprobs_kernel(const moe_layer_logprobs_args_t a) {
  constexpr int N = 16 / sizeof(T), E = N * kBlocks;  // elements of a block, and of a thread's step
  __shared__ Part s_part[kMaxWarps];  // of warps, then (in the first CTA) of the cluster's CTAs
  __shared__ uint4 s_raw[WARP_ROW ? kRowWarps : kMaxWarps][32 * kBlocks];
  __shared__ uint32_t s_order[kMaxWarps][32];
  __shared__ uint32_t s_bound;  // order of a value that `top` logits of the row reach
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, own_warp = threadIdx.x >> 5;
  const int warp = WARP_ROW ? 0 : own_warp, nw = WARP_ROW ? 1 : blockDim.x >> 5;
  uint32_t rank = 0, ctas = 1;
  if constexpr (!WARP_ROW) {
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  }
  const int64_t row = WARP_ROW ? static_cast<int64_t>(blockIdx.x) * kRowWarps + own_warp : blockIdx.x / ctas;
  if (WARP_ROW && row >= a.rows) return;
  const int top = a.top;
  const T* p = static_cast<const T*>(a.logits) + row * a.logits_stride;
  // The row lies in 16-byte blocks of memory, `off` elements past the start of the first.  The first and the last may
  // hold elements that are not the row's: those are read one by one.
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
  const int64_t blocks = (off + static_cast<int64_t>(a.vocab) + N - 1) / N;
  const uint4* base = reinterpret_cast<const uint4*>(p - off);
  if constexpr (!WARP_ROW) {
    if (threadIdx.x == 0) s_bound = 0;
    __syncthreads();
  }

  Sums sum{kNone, 0.0f, 0.0f};
  uint64_t list = 0;              // below every key
  uint64_t least = 0;             // the list's entry number `top`
  float bound = kNone;            // its value, or a larger one that `top` logits reach: smaller ones need not be looked at
  const int64_t tile = static_cast<int64_t>(nw) * 32 * kBlocks * ctas;
  int64_t t0 = (static_cast<int64_t>(rank) * nw + warp) * 32 * kBlocks;
  // as many steps for every warp of the CTA: some have nothing left to read in the last
  const int64_t steps = (blocks - static_cast<int64_t>(rank) * nw * 32 * kBlocks + tile - 1) / tile;
  auto load = [&](int64_t at, uint32_t (&into)[4 * kBlocks]) {
    if (at > 0 && at + 32 * kBlocks < blocks) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        const uint4 u = __ldcs(base + at + b * 32 + lane);
        into[4 * b] = u.x, into[4 * b + 1] = u.y, into[4 * b + 2] = u.z, into[4 * b + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        const int64_t n = at + b * 32 + lane, e = n * N - off;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (e >= 0 && e + N <= a.vocab) {
          u = __ldcs(base + n);
          into[4 * b] = u.x, into[4 * b + 1] = u.y, into[4 * b + 2] = u.z, into[4 * b + 3] = u.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) {
              into[4 * b + j] = e + j >= 0 && e + j < a.vocab ? __float_as_uint(p[e + j]) : 0xFF800000u;
            } else {
              const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
              const uint32_t none = std::is_same<T, __half>::value ? 0xFC00u : 0xFF80u;
              const int64_t i = e + 2 * j;
              into[4 * b + j] = (i >= 0 && i < a.vocab ? h[i] : none) |
                               (i + 1 >= 0 && i + 1 < a.vocab ? h[i + 1] : none) << 16;
            }
          }
        }
      }
    }
  };
  uint32_t next[4 * kBlocks];  // the step after this one, on its way
  if (steps > 0) load(t0, next);
  for (int64_t step = 0; step < steps; ++step, t0 += tile) {
    uint32_t raw[4 * kBlocks];
#pragma unroll
    for (int j = 0; j < 4 * kBlocks; ++j) raw[j] = next[j];
    if (step + 1 < steps) load(t0 + tile, next);
    // the largest of these: of the words as they are, then of a word's elements
    uint32_t top_word = raw[0];
#pragma unroll
    for (int j = 1; j < 4 * kBlocks; ++j) top_word = Type<T>::most(top_word, raw[j]);
    float most;
    if constexpr (sizeof(T) == 4) {
      most = __uint_as_float(top_word);
    } else {
      const float2 f = unpack2<T>(top_word);
      most = fmaxf(f.x, f.y);
    }
    if (most > sum.m) {
      const float d = fmaxf(exponent(sum.m, most), -200.0f), e = exp2_fast(d);
      sum.u = __fmul_rn(e, __fmaf_rn(sum.s, d, sum.u));
      sum.s = __fmul_rn(sum.s, e);
      sum.m = most;
    }
    const float m = sum.m == kNone ? 0.0f : sum.m;  // (nothing but -inf yet, which adds nothing, or NaN)
    if (!far_out<T>(m)) {
      const uint64_t scale = pair_of(kLog2e, kLog2e), less = pair_of(-m, -m);
      uint64_t s2 = pair_of(0.0f, 0.0f), u2 = s2;
#pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        uint32_t w[2];
        if constexpr (sizeof(T) == 4) w[0] = Type<T>::raise(raw[2 * j]), w[1] = Type<T>::raise(raw[2 * j + 1]);
        else w[0] = Type<T>::raise(raw[j]);
        const float2 l = pair_at<T>(w);
        const uint64_t d2 = mul_pair(add_pair(pair_of(l.x, l.y), less), scale);
        const float2 d = of_pair(d2);
        const uint64_t e2 = pair_of(exp2_fast(d.x), exp2_fast(d.y));
        s2 = add_pair(s2, e2);
        u2 = fma_pair(e2, d2, u2);
      }
      const float2 s = of_pair(s2), u = of_pair(u2);
      sum.s = __fadd_rn(sum.s, __fadd_rn(s.x, s.y));
      sum.u = __fadd_rn(sum.u, __fadd_rn(u.x, u.y));
    } else {
#pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        const float2 l = pair_at<T>(raw + (sizeof(T) == 4 ? 2 * j : j));
        const float d0 = exponent(l.x, m), d1 = exponent(l.y, m), e0 = exp2_fast(d0), e1 = exp2_fast(d1);
        sum.s = __fadd_rn(sum.s, __fadd_rn(e0, e1));
        sum.u = __fmaf_rn(e0, fmaxf(d0, -200.0f), __fmaf_rn(e1, fmaxf(d1, -200.0f), sum.u));  // (-inf has 2^d = 0)
      }
    }
    if (top == 0) continue;
    if constexpr (!WARP_ROW) {
      if ((step == 0 && steps > 1) || (step == 3 && steps > 7 && top > 8)) {
        // the `top` largest of the threads' maxima
        uint32_t best = sort_lanes(order_of(sum.m));
        for (int half = nw >> 1; half > 0; half >>= 1) {
          if (warp >= half && warp < 2 * half) s_order[warp][lane] = best;
          __syncthreads();
          if (warp < half) best = merge_orders(best, s_order[warp + half][lane]);
        }
        if (warp == 0 && lane == top - 1) atomicMax(&s_bound, best);
        __syncthreads();
      }
    }
    if constexpr (!WARP_ROW) bound = fmaxf(bound, value_of(max(*static_cast<volatile uint32_t*>(&s_bound), order_of(kNone))));
    uint32_t hit = __ballot_sync(0xffffffffu, most >= bound);
    if (!hit) continue;
    if (__popc(hit) >= top && __popc(hit) > 2) {  // `top` lanes hold a logit of at least their own maximum
      const uint32_t sorted = sort_lanes(order_of(most));
      bound = fmaxf(bound, value_of(__shfl_sync(0xffffffffu, sorted, top - 1)));
      hit = __ballot_sync(0xffffffffu, most >= bound);
    }
    // what these lanes hold goes through shared memory, an element a lane
    uint4* mine = s_raw[own_warp];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
      if (most >= bound) mine[b * 32 + lane] = make_uint4(raw[4 * b], raw[4 * b + 1], raw[4 * b + 2], raw[4 * b + 3]);
    __syncwarp();
    while (hit) {
      const int from = __ffs(hit) - 1;
      hit &= hit - 1;
      const int b = lane / N, j = lane % N;  // (a lane past the thread's E elements has none)
      const int64_t e = (t0 + b * 32 + from) * N - off + j;
      float v = kNone;
      if (lane < E) v = widen<T>(reinterpret_cast<const T*>(mine + (b * 32 + from))[j]);
      const bool in = lane < E && e >= 0 && e < a.vocab && v >= bound;
      const uint64_t key = in ? key_of(v, static_cast<uint32_t>(e)) : 0;
      uint32_t todo = __ballot_sync(0xffffffffu, key > least);
      while (todo) {
        const int at = __ffs(todo) - 1;
        todo &= todo - 1;
        const uint64_t k = __shfl_sync(0xffffffffu, key, at);
        if (k <= least) continue;
        const int place = __popc(__ballot_sync(0xffffffffu, list > k));
        const uint64_t up = __shfl_up_sync(0xffffffffu, list, 1);
        list = lane < place ? list : lane == place ? k : up;
        least = __shfl_sync(0xffffffffu, list, top - 1);
      }
    }
    __syncwarp();  // the elements have been read
    if (least) {
      const uint32_t o = static_cast<uint32_t>(least >> 32);
      bound = fmaxf(bound, value_of(o));
      if (!WARP_ROW && lane == 0) atomicMax(&s_bound, o);
    }
  }

  // threads, warps, CTAs
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Sums b{__shfl_xor_sync(0xffffffffu, sum.m, o), __shfl_xor_sync(0xffffffffu, sum.s, o),
                 __shfl_xor_sync(0xffffffffu, sum.u, o)};
    sum = join(sum, b);
  }
  if constexpr (!WARP_ROW) {
    // n parts in shared memory, the first of them each warp's own, joined two by two
    auto join_parts = [&](int n) {
      for (int half = n >> 1; half > 0; half >>= 1) {
        if (warp < 2 * half) {
          if (lane == 0) s_part[warp].sums = sum;
          s_part[warp].keys[lane] = list;
        }
        __syncthreads();
        if (warp < half) {
          sum = join(sum, s_part[warp + half].sums);
          if (top) list = merge_lists(list, s_part[warp + half].keys[lane]);
        }
        __syncthreads();
      }
    };
    join_parts(nw);
    if (ctas > 1) {
      if (warp == 0) {
        if (lane == 0) s_part[0].sums = sum;
        s_part[0].keys[lane] = list;
      }
      cluster_sync();
      if (rank == 0 && warp < static_cast<int>(ctas)) {
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(&s_part[0]));
        const uint32_t k = at + offsetof(Part, keys) + lane * 8;
        sum = Sums{cluster_read(at, warp), cluster_read(at + 4, warp), cluster_read(at + 8, warp)};
        const uint64_t lo = __float_as_uint(cluster_read(k, warp)), hi = __float_as_uint(cluster_read(k + 4, warp));
        list = hi << 32 | lo;
      }
      cluster_sync();  // no CTA ends, and nothing is overwritten, while the parts are read
      if (rank != 0) return;
      join_parts(static_cast<int>(ctas));
    }
    if (warp != 0) return;
  }
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
  moe_layer_logprobs_args_t arg = a;
  void* args[] = {&arg};
  // A row's end (joins, lists) costs a warp about as much as four steps.  Where there are rows for every SM its warps are
  // as few as leave each eight steps (us with 1 warp a row / 4 / 8 warps, five alternatives: 2039 x 8000 17 / 19 / 27, x
  // 32000 39 / 39 / 44, x 130001 117 / 105 / 109); elsewhere a row is spread over up to 64 warps (8 / 16 / 32 / 64: 64 x
  // 130001 21 / 15 / 12 / 13, 8 x 130001 20 / 14 / 11 / 9, 256 x 130001 24 / 24 / 29 / 40).
  const bool many = a.rows >= 8 * num_sms;
  if (steps <= (many ? 8 : 2))
    return launch_after((const void*)logprobs_kernel<T, true>, dim3((static_cast<unsigned>(a.rows) + kRowWarps - 1) / kRowWarps),
                        dim3(kRowWarps * 32), args, 0, s);
  int warps = 1, ctas = 1;
  while (warps < kMaxWarps && warps * (many ? 8 : 1) < steps) warps *= 2;
  while (ctas < kMaxCluster && ctas * warps < steps && static_cast<int64_t>(a.rows) * ctas < 2 * num_sms) ctas *= 2;
  return launch_after((const void*)logprobs_kernel<T, false>, dim3(static_cast<unsigned>(a.rows) * ctas), dim3(warps * 32), args,
                      0, s, ctas);
}

}  // namespace

cudaError_t launch_logprobs(const moe_layer_logprobs_args_t& a, int num_sms, cudaStream_t s) {
  if (a.dtype == MOE_LAYER_BF16) return launch_typed<__nv_bfloat16>(a, num_sms, s);
  if (a.dtype == MOE_LAYER_FP16) return launch_typed<__half>(a, num_sms, s);
  return launch_typed<float>(a, num_sms, s);
}

}  // namespace moe_layer
