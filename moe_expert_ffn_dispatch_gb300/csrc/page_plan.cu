// The plan of a step's pages: prefix sums over the sequences of new tokens and
// of new pages, then the page table's new entries and every token's place.
//
// One launch: a cluster of CTAs, each of which takes the prefix sums of all
// sequences (at most 4096, into shared memory) and then its share of the pages
// and tokens, found by binary search.  What a token's page is follows from the
// sums and the list of free pages, not from the entries that the call writes, so
// nothing waits for the table; the one cluster barrier lets `taken` be replaced
// in place and the count of unplaced tokens start from zero.
// Bound by latency: 16 bytes a token and 16 a sequence are next to nothing.
#include "layer_ops.cuh"

namespace moe_layer {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kTokensAThread = 4;
constexpr int64_t kMost = 2147483647;

struct Sums {
  int64_t tokens, pages;
};

// inclusive sums over the threads of the CTA, and the CTA's total
__device__ __forceinline__ Sums scan(Sums v, Sums* s_warp, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, v.tokens, o), p = __shfl_up_sync(0xffffffffu, v.pages, o);
    if (lane >= o) v.tokens += t, v.pages += p;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  Sums before{0, 0}, all{0, 0};
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    const Sums x = s_warp[w];
    if (w < warp) before.tokens += x.tokens, before.pages += x.pages;
    all.tokens += x.tokens, all.pages += x.pages;
  }
  *total = all;
  v.tokens += before.tokens, v.pages += before.pages;
  return v;
}

// the last i < n with from[i] <= x; from[0] = 0 <= x
__device__ __forceinline__ int find(const int32_t* from, int n, int32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (from[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const moe_layer_page_plan_args_t a, int shift) {
  extern __shared__ int32_t s_mem[];
  __shared__ Sums s_warp[kPlanWarps];
  __shared__ int s_unplaced;
  grid_dependency_wait();
  grid_launch_dependents();
  const int n = a.batch, rank = blockIdx.x, ctas = gridDim.x;
  int32_t *s_cu = s_mem, *s_page = s_cu + n + 1, *s_held = s_page + n + 1;  // tokens and pages before, tokens held
  const int64_t cap = static_cast<int64_t>(a.max_pages) << shift;
  const int taken = a.taken ? max(0, *a.taken) : 0;
  if (threadIdx.x == 0) s_unplaced = 0;
  if (rank == 0 && threadIdx.x == 0) *a.unplaced = 0;

  const int each = (n + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(n, static_cast<int>(threadIdx.x) * each), b1 = min(n, b0 + each);
  Sums sum{0, 0};
  for (int b = b0; b < b1; ++b) {
    const int64_t held = max(0, a.held[b]), len = held + max(0, a.new_tokens[b]);
    const int64_t first = (held + a.page_size - 1) >> shift;
    sum.tokens += len - held;
    sum.pages += max(static_cast<int64_t>(0), ((min(len, cap) + a.page_size - 1) >> shift) - first);
  }
  Sums total;
  const Sums upto = scan(sum, s_warp, &total);
  Sums at{upto.tokens - sum.tokens, upto.pages - sum.pages};
  for (int b = b0; b < b1; ++b) {
    const int64_t held = max(0, a.held[b]), len = held + max(0, a.new_tokens[b]);
    const int64_t first = (held + a.page_size - 1) >> shift;
    s_cu[b] = static_cast<int32_t>(min(at.tokens, kMost));
    s_page[b] = static_cast<int32_t>(at.pages);
    s_held[b] = static_cast<int32_t>(held);
    if (rank == 0) {
      a.cu_tokens[b] = static_cast<int32_t>(min(at.tokens, kMost));
      a.seq_lens[b] = static_cast<int32_t>(min(len, kMost));
    }
    at.tokens += len - held;
    at.pages += max(static_cast<int64_t>(0), ((min(len, cap) + a.page_size - 1) >> shift) - first);
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
  const int64_t tid = static_cast<int64_t>(rank) * kPlanThreads + threadIdx.x, step = static_cast<int64_t>(ctas) * kPlanThreads;
  for (int64_t p = tid; p < pages; p += step) {
    const int b = find(s_page, n, static_cast<int32_t>(p));
    const int first = static_cast<int>((static_cast<int64_t>(s_held[b]) + a.page_size - 1) >> shift);
    a.page_table[b * a.table_stride + first + (p - s_page[b])] = fresh(static_cast<int32_t>(p));
  }
  int lost = 0;
  for (int64_t t0 = tid * kTokensAThread; t0 < a.tokens; t0 += step * kTokensAThread) {
    int b = t0 < tokens ? find(s_cu, n, static_cast<int32_t>(t0)) : 0;
    int64_t last_page = -1;
    int32_t page = -1;
#pragma unroll
    for (int j = 0; j < kTokensAThread; ++j) {
      const int64_t t = t0 + j;
      if (t >= a.tokens) break;
      int32_t seq = -1, pos = -1;
      int64_t slot = -1;
      if (t < tokens) {
        while (t >= s_cu[b + 1]) ++b, last_page = -1;
        const int64_t held = s_held[b], at_pos = held + (t - s_cu[b]);
        const int64_t in_table = at_pos >> shift, first = (held + a.page_size - 1) >> shift;
        if (in_table != last_page) {
          last_page = in_table;
          page = in_table >= a.max_pages ? -1
                 : in_table < first      ? a.page_table[b * a.table_stride + in_table]
                                         : fresh(static_cast<int32_t>(s_page[b] + (in_table - first)));
        }
        seq = b;
        pos = static_cast<int32_t>(min(at_pos, kMost));
        if (page >= 0 && page < a.num_pages) slot = (static_cast<int64_t>(page) << shift) + (at_pos & (a.page_size - 1));
        else ++lost;
      }
      if (a.sequence) a.sequence[t] = seq;
      if (a.position) a.position[t] = pos;
      if (a.slot) a.slot[t] = slot;
    }
  }
  lost = __reduce_add_sync(0xffffffffu, lost);
  if ((threadIdx.x & 31) == 0 && lost) atomicAdd(&s_unplaced, lost);
  __syncthreads();
  if (threadIdx.x == 0 && s_unplaced) atomicAdd(a.unplaced, s_unplaced);
}

}  // namespace

cudaError_t launch_page_plan(const moe_layer_page_plan_args_t& a, cudaStream_t s) {
  int shift = 0;
  while ((1 << shift) < a.page_size) ++shift;
  int ctas = 1;  // a thread each four tokens, as far as a cluster goes
  while (ctas < 8 && ctas * kPlanThreads * kTokensAThread < a.tokens) ctas *= 2;
  moe_layer_page_plan_args_t arg = a;
  void* args[] = {&arg, &shift};
  const size_t smem = (3 * static_cast<size_t>(a.batch) + 2) * sizeof(int32_t);
  const void* k = (const void*)page_plan_kernel;
  static std::atomic<uint64_t> allowed{0};
  if (const cudaError_t e = allow_smem(k, 64 * 1024, allowed); e != cudaSuccess) return e;
  return launch_after(k, dim3(ctas), dim3(kPlanThreads), args, smem, s, ctas);
}

}  // namespace moe_layer
