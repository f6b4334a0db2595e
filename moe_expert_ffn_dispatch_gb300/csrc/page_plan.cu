// The plan of a step's pages: prefix sums over the sequences of new tokens and
// of new pages, then the page table's new entries and every token's place.
//
// One launch: a cluster of CTAs, each of which takes the prefix sums of all
// sequences (at most 4096, into shared memory) and then its share of the pages
// and tokens, found by binary search.  What a token's page is follows from the
// sums and the list of free pages, not from the entries that the call writes, so
// nothing waits for the table; the one cluster barrier lets `taken` be replaced
// in place and the count of unplaced tokens start from zero.
// Bound by latency: 16 bytes a token and 16 a sequence are next to nothing.  A sequence
// with one token 2.6 us, 64 of them 4.3, 5 prompts of 5035 tokens 4.2, 1024 sequences with
// 33000 tokens 9.7, 4096 with 35000 14: the eight SMs that a cluster can be relied on to have.
// Threads a CTA, 256 / 512 / 1024: 64 sequences 4.3 / 4.7 / -, 5 prompts - / 4.2 / 6.9, 1024
// sequences - / 11.3 / 9.7.
#include "layer_ops.cuh"

namespace moe_layer {
namespace {

constexpr int kTokensAThread = 4;  // neighbours: one search, and wide stores where the buffers are aligned
constexpr int64_t kMost = 2147483647;

struct Sums {
  int64_t tokens, pages;
};

// inclusive sums over the threads of the CTA, and the CTA's total
template <int WARPS>
__device__ __forceinline__ Sums scan(Sums v, Sums* s_warp, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, v.tokens, o), p = __shfl_up_sync(0xffffffffu, v.pages, o);
    if (lane >= o) v.tokens += t, v.pages += p;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  // every warp adds up the warps before it, a lane each
  static_assert(WARPS <= 32, "a warp's lanes");
  Sums w{0, 0};
  if (lane < WARPS) w = s_warp[lane];
  Sums before{lane < warp ? w.tokens : 0, lane < warp ? w.pages : 0};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    w.tokens += __shfl_xor_sync(0xffffffffu, w.tokens, o), w.pages += __shfl_xor_sync(0xffffffffu, w.pages, o);
    before.tokens += __shfl_xor_sync(0xffffffffu, before.tokens, o);
    before.pages += __shfl_xor_sync(0xffffffffu, before.pages, o);
  }
  *total = w;
  v.tokens += before.tokens, v.pages += before.pages;
  return v;
}

// the last i of lo .. hi with from[i] <= x, which from[lo] is
__device__ __forceinline__ int find(const int32_t* from, int lo, int hi, int32_t x) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (from[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) page_plan_kernel(const moe_layer_page_plan_args_t a, int shift) {
  extern __shared__ int32_t s_mem[];
  __shared__ Sums s_warp[THREADS / 32];
  __shared__ int s_unplaced;
  grid_dependency_wait();
  grid_launch_dependents();
  const int n = a.batch, rank = blockIdx.x, ctas = gridDim.x;
  int32_t *s_cu = s_mem, *s_page = s_cu + n + 1, *s_held = s_page + n + 1;  // tokens and pages before, tokens held
  const int64_t cap = static_cast<int64_t>(a.max_pages) << shift;
  const int taken = a.taken ? max(0, *a.taken) : 0;
  if (threadIdx.x == 0) s_unplaced = 0;
  if (rank == 0 && threadIdx.x == 0) *a.unplaced = 0;

  // lengths to shared memory, then sums over a thread's neighbours and over the threads
#pragma unroll 4
  for (int b = threadIdx.x; b < n; b += THREADS) {
    s_held[b] = max(0, a.held[b]);
    s_cu[b] = max(0, a.new_tokens[b]);
  }
  __syncthreads();
  auto pages_of = [&](int64_t held, int64_t len) {
    const int64_t first = (held + a.page_size - 1) >> shift, last = (min(len, cap) + a.page_size - 1) >> shift;
    return max(static_cast<int64_t>(0), last - first);
  };
  const int each = (n + THREADS - 1) / THREADS;
  const int b0 = min(n, static_cast<int>(threadIdx.x) * each), b1 = min(n, b0 + each);
  Sums sum{0, 0};
  for (int b = b0; b < b1; ++b) {
    const int64_t held = s_held[b], more = s_cu[b];
    sum.tokens += more;
    sum.pages += pages_of(held, held + more);
  }
  Sums total;
  const Sums upto = scan<THREADS / 32>(sum, s_warp, &total);
  Sums at{upto.tokens - sum.tokens, upto.pages - sum.pages};
  for (int b = b0; b < b1; ++b) {
    const int64_t held = s_held[b], more = s_cu[b], len = held + more;
    s_cu[b] = static_cast<int32_t>(min(at.tokens, kMost));
    s_page[b] = static_cast<int32_t>(at.pages);
    if (rank == 0) {
      a.cu_tokens[b] = static_cast<int32_t>(min(at.tokens, kMost));
      a.seq_lens[b] = static_cast<int32_t>(min(len, kMost));
    }
    at.tokens += more;
    at.pages += pages_of(held, len);
  }
  const int32_t tokens = static_cast<int32_t>(min(total.tokens, kMost)), pages = static_cast<int32_t>(total.pages);
  if (threadIdx.x == 0) {
    s_cu[n] = tokens;
    s_page[n] = pages;
  }
  cluster_sync();  // every CTA has read `taken`; the count of unplaced tokens is zero; and this CTA's sums are there
  if (rank == 0 && threadIdx.x == 0) {
    a.cu_tokens[n] = tokens;
    *a.taken_out = static_cast<int32_t>(min(static_cast<int64_t>(taken) + pages, static_cast<int64_t>(a.num_free)));
  }
  // the entry of the free list that new page number p takes
  auto fresh = [&](int32_t p) -> int32_t {
    const int64_t i = static_cast<int64_t>(taken) + p;
    return i < a.num_free ? __ldg(a.free_pages + i) : -1;
  };
  const int64_t tid = static_cast<int64_t>(rank) * THREADS + threadIdx.x, step = static_cast<int64_t>(ctas) * THREADS;
  for (int64_t p = tid; p < pages; p += step) {
    const int b = find(s_page, 0, n - 1, static_cast<int32_t>(p));
    const int first = static_cast<int>((static_cast<int64_t>(s_held[b]) + a.page_size - 1) >> shift);
    a.page_table[b * a.table_stride + first + (p - s_page[b])] = fresh(static_cast<int32_t>(p));
  }
  int lost = 0;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.sequence) | reinterpret_cast<uintptr_t>(a.position) |
                      reinterpret_cast<uintptr_t>(a.slot)) & 15u) == 0;
  for (int64_t t0 = tid * kTokensAThread; t0 < a.tokens; t0 += step * kTokensAThread) {
    int b = t0 < tokens ? find(s_cu, 0, n - 1, static_cast<int32_t>(t0)) : 0;
    int64_t last_page = -1;
    int32_t page = -1, seq[kTokensAThread], pos[kTokensAThread];
    int64_t slot[kTokensAThread];
#pragma unroll
    for (int j = 0; j < kTokensAThread; ++j) {
      const int64_t t = t0 + j;
      seq[j] = pos[j] = -1;
      slot[j] = -1;
      if (t >= tokens || t >= a.tokens) continue;
      while (t >= s_cu[b + 1]) ++b, last_page = -1;
      const int64_t held = s_held[b], at_pos = held + (t - s_cu[b]);
      const int64_t in_table = at_pos >> shift, first = (held + a.page_size - 1) >> shift;
      if (in_table != last_page) {
        last_page = in_table;
        page = in_table >= a.max_pages ? -1
               : in_table < first      ? a.page_table[b * a.table_stride + in_table]
                                       : fresh(static_cast<int32_t>(s_page[b] + (in_table - first)));
      }
      seq[j] = b;
      pos[j] = static_cast<int32_t>(min(at_pos, kMost));
      if (page >= 0 && page < a.num_pages) slot[j] = (static_cast<int64_t>(page) << shift) + (at_pos & (a.page_size - 1));
      else ++lost;
    }
    if (wide && t0 + kTokensAThread <= a.tokens) {
      if (a.sequence) *reinterpret_cast<int4*>(a.sequence + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      if (a.position) *reinterpret_cast<int4*>(a.position + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (a.slot) {
        reinterpret_cast<longlong2*>(a.slot + t0)[0] = make_longlong2(slot[0], slot[1]);
        reinterpret_cast<longlong2*>(a.slot + t0)[1] = make_longlong2(slot[2], slot[3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kTokensAThread; ++j) {
        if (t0 + j >= a.tokens) continue;
        if (a.sequence) a.sequence[t0 + j] = seq[j];
        if (a.position) a.position[t0 + j] = pos[j];
        if (a.slot) a.slot[t0 + j] = slot[j];
      }
    }
  }
  lost = __reduce_add_sync(0xffffffffu, lost);
  if ((threadIdx.x & 31) == 0 && lost) atomicAdd(&s_unplaced, lost);
  __syncthreads();
  if (threadIdx.x == 0 && s_unplaced) atomicAdd(a.unplaced, s_unplaced);
}

}  // namespace

namespace {

template <int THREADS>
cudaError_t launch_threads(const moe_layer_page_plan_args_t& a, cudaStream_t s) {
  int shift = 0;
  while ((1 << shift) < a.page_size) ++shift;
  int ctas = 1;  // a thread each four tokens, as far as a cluster goes
  while (ctas < 8 && ctas * THREADS * kTokensAThread < a.tokens) ctas *= 2;
  moe_layer_page_plan_args_t arg = a;
  void* args[] = {&arg, &shift};
  const size_t smem = (3 * static_cast<size_t>(a.batch) + 2) * sizeof(int32_t);
  const void* k = (const void*)page_plan_kernel<THREADS>;
  static std::atomic<uint64_t> allowed{0};
  if (const cudaError_t e = allow_smem(k, 64 * 1024, allowed); e != cudaSuccess) return e;
  return launch_after(k, dim3(ctas), dim3(THREADS), args, smem, s, ctas);
}

}  // namespace

cudaError_t launch_page_plan(const moe_layer_page_plan_args_t& a, cudaStream_t s) {
  if (a.batch <= 256 && a.tokens <= 1024) return launch_threads<256>(a, s);
  if (a.batch <= 512 && a.tokens <= 16384) return launch_threads<512>(a, s);
  return launch_threads<1024>(a, s);
}

}  // namespace moe_layer
