// 8-bit products of more tokens than a few, on the tensor cores' tensor memory,
// exact in int32.
//
// The tensor cores of this chip have no integer kind: codes run as f16 (every
// integer in [-128, 127] is exact), sums as fp32 in tensor memory.  A product of two
// codes is at most 2^14, so 1024 consecutive k sum to at most 2^24, exactly; each
// accumulator covers 1024 k at most and is then drained into registers.  There sums
// stay fp32 as long as the largest that could have come together is below 2^24, which
// is exact too, and are int32 from then on: the conversion is the drain's slowest part.
//
// A tile is 128 weight rows (M, the tensor memory's lanes) by up to 128 tokens (N), or,
// for many tokens, 256 rows by up to 256 tokens of a pair of CTAs: each has 128 of the
// rows and half of the tokens, and the first issues products of both.  Weights arrive
// as int8 by TMA and are converted in the CTA into tensor memory, the products' A
// operand, so that they cross memory and L2 as bytes.  Tokens are the B operand, f16 in
// shared memory: up to 64 of them arrive as int8 too and are converted by every CTA;
// more are converted once, by a kernel before this one into the workspace, and arrive
// as f16.  One CTA with 224 tokens of its own moves 147 KB a step of 128 k through
// shared memory, all that it can in the step's time (4093 x 6144 x 4096 131 us for 121,
// with the tokens' conversion of then); of a pair each moves 90.
// A pair's tile has an accumulator for each half of the tokens, side by side, and takes
// two steps of one half, then of the other: at the end of 1024 k one accumulator is
// drained while two steps' products run into the other (a step of each in turn 137 us
// for 131).  Its halves need not be alike, so that tiles come in 32s of tokens: 19 x 24
// tiles of 224 fill 76 pairs six times, 16 x 24 of 256 five times and a bit (121 us for
// 128).  A tile of one half alternates between two accumulators.
// What bounds a step is how fast one warp can wait, issue and commit (about 100 cycles
// a wait, 40 a product) and the conversion's chain of waits, loads and stores (830
// cycles): weights and tokens of a step complete one barrier, and its products one other.
// Roles: warp 0 copies weights, warp 2 copies tokens, warp 1 issues products (the first
// CTA's of a pair), warps 4..7 convert weights (a row a thread), warps 8..15 drain and
// write.  Up to 64 tokens warps 4..7 and 8..11 convert weights and tokens of every other
// step, and warps 12..15 drain.
// Where there are fewer tiles than SMs a cluster shares k out, and adds its int32
// sums up over distributed shared memory, a share of the tile's columns each.
//
// Bound by: many tokens, the products (4093 x 6144 x 4096 116 us, 1.77 PFLOP/s; 7 us of
// it is the tokens' conversion before, the tensor pipe is busy for 172 of the 205
// thousand cycles after, the rest is the ends of 1024 k and of tiles); 16 tokens x 130001
// x 4096, memory (88 us, 6.1 TB/s); up to 128 tokens on ordinary sizes, latency (64 x 4096
// x 4096 10.3 us: 3 until the first weights, 3 for the steps, 2 for the sums over the
// cluster, launch).
#include "w8_linear.cuh"

#include <algorithm>

#include "device_prims.cuh"
#include "tensor_map.cuh"

namespace moe_layer {
namespace {

constexpr int kRows = 128;          // weight rows of a tile
constexpr int kStage = 128;         // k of a weight stage
constexpr int kAtom = 64;           // k of one 128-byte row of f16
constexpr int kChunk = 1024 / kStage;  // stages that a sum stays exact for
constexpr int kA16Cols = kStage / 2;  // of a converted weight stage in tensor memory
constexpr int kTmemCols = 512;
constexpr int kThreads = 512, kWidenThreads = 256;
// Registers a thread where a tile has two halves: 128 at launch, and what the drain warps have more the others give.
// (With one half nobody needs more, and the sums over a cluster are every warp's.)
constexpr int kLaunchRegs = 128, kRoleRegs = 64, kConvRegs = 96, kDrainRegs = 176;
static_assert(128 * kRoleRegs + 128 * kConvRegs + 256 * kDrainRegs <= kThreads * kLaunchRegs, "the split fits what the launch has");
constexpr int kA8Bytes = kRows * kStage;
constexpr int kSite = 2 << 8;       // of the waits, in the status
constexpr float kNan = NAN;
constexpr uint32_t kMostParts = 8;  // CTAs that share k out

// A tile: 128 weight rows by up to 64 or up to 128 tokens, or 256 weight rows by up to 256 tokens in two halves, for a
// pair of CTAs
enum Form { kFew = 0, kOne = 1, kTwo = 2 };

// Shared memory: tokens of each step, weight stages, barriers
template <int FORM>
struct Layout {
  static constexpr int kHalves = FORM == kTwo ? 2 : 1;
  static constexpr int kHalf = FORM == kFew ? 64 : 128;  // tokens of a half at most
  static constexpr int kAtomBytes = kHalf * kAtom * 2;  // (of a pair's tokens each CTA has one half)
  static constexpr int kSteps = 4;  // of tokens, and of converted weights
  static constexpr int kA8 = 6;     // weights (up to 64 tokens: and tokens) as they arrive
  static constexpr int kStageBytes = kA8Bytes + (FORM == kFew ? kHalf * kStage : 0);
  static constexpr int kOffA8 = kSteps * 2 * kAtomBytes, kOffBar = kOffA8 + kA8 * kStageBytes;
  static constexpr int kBytes = kOffBar + 512;
  static constexpr int kAccCols = 2 * kHalf;
  static constexpr int kDrainWarp0 = FORM == kFew ? 12 : 8, kDrainWarps = 16 - kDrainWarp0, kConvGroups = kDrainWarp0 / 4 - 1;
  static_assert(kSteps % kConvGroups == 0 && kA8 % kConvGroups == 0, "a group's slots");
  static_assert(kBytes + 1024 <= kMaxSmem, "shared memory");
  static_assert(kAccCols + kSteps * kA16Cols <= kTmemCols, "tensor memory");
  static_assert(kOffBar >= kHalf * kRows * 4, "the sums of a tile of one half fit the rings");
  // arrivals of a step: the converting warps (a pair's: of both CTAs), and the tokens' copy
  static constexpr int kConvArrivals = FORM == kTwo ? 8 : 4, kFull = kConvArrivals + (FORM == kFew ? 0 : 1);
  static constexpr int kDrained = kDrainWarps * kHalves;
};

struct Barriers {
  uint64_t a8_full[6], a8_empty[6], full[4], empty[4], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int abort, broken;
};
static_assert(sizeof(Barriers) <= 512, "");

struct alignas(64) Maps {
  CUtensorMap w;  // int8 [n, k], box {128, 128}, 128-byte swizzle
  CUtensorMap x;  // f16 [m, k], box {64, tokens of a half}, or int8, box {128, tokens}; 128-byte swizzle
  CUtensorMap y;  // of a pair: x is half of the first half's tokens, this half of the second's
};

struct Params {
  moe_layer_w8_args_t a;
  int32_t* status;
  int half;     // tokens of a tile of one half, a multiple of 16, or of the first of two, of 32
  int half1;    // of the second
  int blocks;   // tiles along m
  int64_t tiles;
};

// 16 codes -> 16 f16, exactly
__device__ __forceinline__ void widen16(const uint4& c, uint32_t* o) {
  half_pairs(c.x, o[0], o[1]);
  half_pairs(c.y, o[2], o[3]);
  half_pairs(c.z, o[4], o[5]);
  half_pairs(c.w, o[6], o[7]);
}

// The tokens as f16, dense; and the status words of the call.  2^shift threads a row, 8 codes at a time, so that loads and
// stores of a warp are whole lines (16 codes a thread of one long row, which takes a division, 4093 x 4096 4 us more).
__global__ void __launch_bounds__(kWidenThreads) w8_widen_kernel(const moe_layer_w8_args_t a, __half* x16, int32_t* status,
                                                                 int shift) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x < 8) status[threadIdx.x] = 0;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kWidenThreads >> shift) + (threadIdx.x >> shift);
  if (row >= a.m) return;
  const int pieces = a.k / 8, step = 1 << shift;
  const uint2* from = reinterpret_cast<const uint2*>(a.x + row * a.x_stride);
  uint4* to = reinterpret_cast<uint4*>(x16 + row * a.k);
  for (int c = threadIdx.x & (step - 1); c < pieces; c += 4 * step) {
    uint2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i * step < pieces) v[i] = from[c + i * step];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c + i * step >= pieces) continue;
      uint32_t o[4];
      half_pairs(v[i].x, o[0], o[1]);
      half_pairs(v[i].y, o[2], o[3]);
      to[c + i * step] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// Every copy that a producer issued has landed when this returns: the last phase
// armed on each slot of its ring has completed.  s, ph: the next slot and its parity.
__device__ __forceinline__ void drain_ring(uint64_t* full, int n, int s, uint32_t ph, bool wrapped, int32_t* status,
                                           int site) {
  for (int i = 0; i < n; ++i) {
    if (i < s) moe::mbar_wait_bounded(&full[i], ph, nullptr, status, site);
    else if (wrapped) moe::mbar_wait_bounded(&full[i], ph ^ 1u, nullptr, status, site);
  }
}

__device__ __forceinline__ void put(float* y, float v) { *y = v; }
__device__ __forceinline__ void put(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* y, float v) { *y = __float2half_rn(v); }

// `most` (at most 64) tokens of one weight row a lane, `stride` apart; every lane of the warp
template <typename T>
__device__ __forceinline__ void write_tokens(T* y, int64_t stride, const uint32_t (&acc)[64], float ws, float xs0, float xs1,
                                             int most, bool mine) {
#pragma unroll
  for (int j = 0; j < 64; ++j) {
    const float xs = __shfl_sync(0xffffffffu, j < 32 ? xs0 : xs1, j & 31);
    if (j < most && mine) put(y, scaled(__uint_as_float(acc[j]), ws, xs));
    y += stride;
  }
}

// 32 columns of this warp's 32 lanes, and the wait for them
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}

// the largest of |a|, |b| and |c|
__device__ __forceinline__ float most_of(float a, uint32_t b, uint32_t c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return d;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// the two halves of a cluster barrier
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// 16 bytes at shared address `at` of CTA `rank` of the cluster
__device__ __forceinline__ int4 cluster_read4(uint32_t at, uint32_t rank) {
  uint32_t remote;
  int4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(remote)
               : "memory");
  return v;
}

// ---- a pair of CTAs: what one thread of the first issues works on the tensor memory of both
__device__ __forceinline__ void pair_alloc(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(moe::smem_u32(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D (256 rows, 128 in each CTA) (+)= A (tensor memory, likewise) * B^T, whose N rows are half each CTA's
__device__ __forceinline__ void pair_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrive on `bar` of both CTAs once every product issued so far by this thread is done
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          moe::smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// `bar` of CTA `rank`, as an address in the cluster's shared memory
__device__ __forceinline__ uint32_t remote_of(uint64_t* bar, uint32_t rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(moe::smem_u32(bar)), "r"(rank));
  return remote;
}
// Arrive on `bar` of CTA `rank`.  What the arrival tells of is tensor memory whose stores (or loads) have been waited for:
// the tcgen05 fences on either side order it, and ask for an arrival of the cluster's scope, relaxed (a release, which
// waits for all that the thread did, took 1200 cycles a step more).
__device__ __forceinline__ void arrive_at(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote_of(bar, rank)) : "memory");
}
// moe::tma_load_2d into this CTA's shared memory, completing bytes on a barrier of either CTA of the pair
__device__ __forceinline__ void pair_tma_load_2d(void* dst, const void* tmap, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(moe::smem_u32(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// A wait's budget, for copies whose landing no barrier can show any more
__device__ __forceinline__ void wait_out_budget() {
  const uint64_t t0 = moe::global_timer_ns();
  while (moe::global_timer_ns() - t0 <= moe::kWaitBudgetNs) __nanosleep(100000);
}

// EARLY: slots of codes go back before the codes are converted
template <int FORM, bool EARLY>
__global__ void __launch_bounds__(kThreads, 1) w8_tc_kernel(const __grid_constant__ Maps maps, const Params p) {
  using L = Layout<FORM>;
  constexpr int HALVES = L::kHalves, kAccCols = L::kAccCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (moe::smem_u32(smem_raw) & 1023u)) & 1023u);
  Barriers& bar = *reinterpret_cast<Barriers*>(smem + L::kOffBar);
  const moe_layer_w8_args_t& a = p.a;
  // (handed round, so that the compiler knows it to be one number a warp and keeps what follows from it in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t in_cluster, ctas;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(in_cluster));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const int64_t first = blockIdx.x / ctas, step = gridDim.x / ctas;
  // a cluster shares k out, or is a pair that shares a tile
  const uint32_t rank = FORM == kTwo ? 0 : in_cluster, parts = FORM == kTwo ? 1 : ctas;
  const uint32_t side_of_pair = FORM == kTwo ? in_cluster : 0;
  constexpr int kTileRows = kRows * HALVES;
  const int tokens = HALVES == 2 ? p.half + p.half1 : p.half;
  const int stages = (a.k + kStage - 1) / kStage;
  const int kb0 = static_cast<int>(static_cast<int64_t>(stages) * rank / parts),
            kb1 = static_cast<int>(static_cast<int64_t>(stages) * (rank + 1) / parts);

  if (warp == 0) {
    if (lane < L::kA8) {
      moe::mbar_init(&bar.a8_full[lane], 1);
      moe::mbar_init(&bar.a8_empty[lane], 4);
    }
    if (lane < L::kSteps) {
      moe::mbar_init(&bar.full[lane], L::kFull);
      moe::mbar_init(&bar.empty[lane], 1);
    }
    if (lane < 2) {
      moe::mbar_init(&bar.acc_full[lane], 1);
      moe::mbar_init(&bar.acc_empty[lane], L::kDrained);
    }
    if (lane == 0) {
      moe::mbar_init(&bar.drain, 1);
      bar.abort = bar.broken = 0;
    }
    moe::fence_barrier_init();
  }
  if (warp == 1) {
    if constexpr (FORM == kTwo) pair_alloc(&bar.tmem, kTmemCols);
    else moe::tmem_alloc(&bar.tmem, kTmemCols);
  }
  if (warp == 2 && lane == 0) {
    prefetch_map(&maps.w);
    prefetch_map(&maps.x);
  }
  if constexpr (FORM == kTwo) cluster_sync();  // the other CTA's barriers are there
  else __syncthreads();
  moe::tc_fence_after();
  const uint32_t tmem = bar.tmem;
  volatile int* abort = &bar.abort;
  // A bounded wait of a whole warp, with one answer for all of its lanes.  The status words are the widening kernel's
  // to clear: what is reported before it is done would be lost, but nothing waits that long before it.  (Without one
  // there are no status words.)  A tile whose wait gave up is written as NaN.
  auto wait = [&](uint64_t* b, uint32_t parity, int site) {
    return __all_sync(0xffffffffu, moe::mbar_wait_bounded(b, parity, abort, p.status, kSite + site)) != 0;
  };
  // the same, where the other CTA of a pair arrives
  auto wait_both = [&](uint64_t* b, uint32_t parity, int site) {
    return __all_sync(0xffffffffu, moe::mbar_wait_bounded<FORM == kTwo>(b, parity, abort, p.status, kSite + site)) != 0;
  };
  // what completes a step, or empties an accumulator, does so at the CTA that issues the products
  auto arrive = [&](uint64_t* b) {
    if (side_of_pair) arrive_at(b, 0);
    else moe::mbar_arrive(b);
  };

  if constexpr (FORM == kFew) grid_dependency_wait();  // no kernel of this call's own has done so
  grid_launch_dependents();
  if (warp < 4) {
    if constexpr (HALVES == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
    if (warp == 0) {
      // ---------------------------------------------------- weights: what the call before this one left is complete
      // once the widening kernel runs, which waited for it
      int s = 0;
      uint32_t ph = 0;
      bool wrapped = false, ok = true;
      for (int64_t it = first; ok && it < p.tiles; it += step) {
        const int n0 = static_cast<int>(it / p.blocks) * kTileRows + static_cast<int>(side_of_pair) * kRows;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (wrapped && !wait(&bar.a8_empty[s], ph ^ 1u, 1)) {
            ok = false;
            break;
          }
          if (moe::elect_one()) {
            uint8_t* to = smem + L::kOffA8 + s * L::kStageBytes;
            moe::mbar_arrive_expect_tx(&bar.a8_full[s], kA8Bytes + (FORM == kFew ? p.half * kStage : 0));
            moe::tma_load_2d(to, &maps.w, kb * kStage, n0, &bar.a8_full[s]);
            if (FORM == kFew) moe::tma_load_2d(to + kA8Bytes, &maps.x, kb * kStage, 0, &bar.a8_full[s]);
          }
          __syncwarp();
          if (++s == L::kA8) s = 0, ph ^= 1u, wrapped = true;
        }
      }
      drain_ring(bar.a8_full, L::kA8, s, ph, wrapped, p.status, kSite + 2);
    } else if (FORM != kFew && warp == 2) {
      // ---------------------------------------------------- tokens
      grid_dependency_wait();
      int s = 0;
      uint32_t ph = 0;
      bool wrapped = false, ok = true;
      // One half's tokens; or, of a pair, half of each half's, so that the columns of a product (the first CTA's tokens,
      // then the second's) are neighbours.  Both CTAs' copies complete the first's barrier.
      const int box = p.half / HALVES, box1 = p.half1 / 2;
      const uint32_t bytes = 2 * tokens * kAtom * 2;  // of both CTAs
      for (int64_t it = first; ok && it < p.tiles; it += step) {
        const int m0 = static_cast<int>(it % p.blocks) * tokens;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (wrapped && !wait(&bar.empty[s], ph ^ 1u, 3)) {
            ok = false;
            break;
          }
          if (moe::elect_one()) {
            if (!side_of_pair) moe::mbar_arrive_expect_tx(&bar.full[s], bytes);
            const uint32_t landed = FORM == kTwo ? remote_of(&bar.full[s], 0) : 0;
#pragma unroll
            for (int a = 0; a < 2; ++a) {
              uint8_t* to = smem + (2 * s + a) * L::kAtomBytes;
              const int k = kb * kStage + a * kAtom;
              if constexpr (FORM == kTwo) {
                pair_tma_load_2d(to, &maps.x, k, m0 + side_of_pair * box, landed);
                pair_tma_load_2d(to + box * kAtom * 2, &maps.y, k, m0 + p.half + side_of_pair * box1, landed);
              } else {
                moe::tma_load_2d(to, &maps.x, k, m0, &bar.full[s]);
              }
            }
          }
          __syncwarp();
          if (++s == L::kSteps) s = 0, ph ^= 1u, wrapped = true;
        }
      }
      // (every step's products are done where nothing gave up: the tokens have landed; else: after the roles)
    } else if (warp == 1 && side_of_pair) {
      // the first CTA's products, which are of this one's memory too, are done
      moe::mbar_wait_bounded(&bar.drain, 0, nullptr, p.status, kSite + 8);
    } else if (warp == 1) {
      // ---------------------------------------------------- products
      const uint32_t idescs[2] = {moe::umma_idesc_f16(kTileRows, p.half), moe::umma_idesc_f16(kTileRows, p.half1)};
      const uint64_t b0 = moe::umma_desc_sw128(moe::smem_u32(smem));
      constexpr uint64_t kAtomAt = L::kAtomBytes >> 4;
      const uint64_t half_at = (p.half / HALVES * kAtom * 2) >> 4;
      // eight products of 16 k
      auto products = [&](uint32_t d, uint32_t at, uint64_t bd, uint32_t idesc, bool fresh) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t bk = bd + (k >> 2) * kAtomAt + 2 * (k & 3);
          if constexpr (FORM == kTwo) pair_mma_ts(d, at + 8 * k, bk, idesc, !fresh || k != 0);
          else moe::umma_f16_ts(d, at + 8 * k, bk, idesc, !fresh || k != 0);
        }
      };
      auto commit = [&](uint64_t* b) {
        if constexpr (FORM == kTwo) pair_commit(b);
        else moe::umma_commit(b);
      };
      int s = 0;
      uint32_t ph = 0;
      int64_t chunk = 0;
      bool ok = true;
      for (int64_t it = first; ok && it < p.tiles; it += step) {
        int kc = 0;  // step of the chunk
        for (int kb = kb0; ok && kb < kb1;) {
          const int steps = HALVES == 2 && kc + 1 < kChunk && kb + 1 < kb1 ? 2 : 1;
          const bool last = kc + steps == kChunk || kb + steps == kb1;
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            // the accumulator's uses so far: a half's own one a chunk, or two in turn
            const int buf = HALVES == 2 ? h : static_cast<int>(chunk & 1);
            const int64_t used = HALVES == 2 ? chunk : chunk >> 1;
            if (kc == 0 && used > 0) ok = ok && wait_both(&bar.acc_empty[buf], (used - 1) & 1, 7);
#pragma unroll
            for (int i = 0; i < HALVES; ++i) {
              if (i == steps) break;
              const int at = s + i < L::kSteps ? s + i : 0;
              if (h == 0) ok = ok && wait_both(&bar.full[at], s + i < L::kSteps ? ph : ph ^ 1u, 6);
              if (!ok) break;
              moe::tc_fence_after();
              if (moe::elect_one()) {
                products(tmem + buf * p.half, tmem + kAccCols + at * kA16Cols, b0 + 2 * at * kAtomAt + h * half_at,
                         idescs[h], kc + i == 0);
                if (h == HALVES - 1) commit(&bar.empty[at]);
                if (last && i + 1 == steps) commit(&bar.acc_full[buf]);
              }
              __syncwarp();
            }
          }
          s += steps;
          if (s >= L::kSteps) s -= L::kSteps, ph ^= 1u;
          kb += steps;
          if (last) ++chunk, kc = 0;
          else kc += steps;
        }
      }
      // nothing of this CTA is in flight when its tensor memory goes back
      if (moe::elect_one()) commit(&bar.drain);
      __syncwarp();
      moe::mbar_wait_bounded(&bar.drain, 0, nullptr, p.status, kSite + 8);
    }
  } else if (warp < L::kDrainWarp0) {
    if constexpr (HALVES == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    // ------------------------------------------------------ weights to f16, a row a thread, into tensor memory;
    // 16-byte chunk j of row r lies at chunk j ^ (r % 8) of its 128 bytes.  The next codes are loaded while these ones'
    // stores are on their way.  Two groups take steps in turn.
    constexpr int kGroups = L::kConvGroups;
    const int row = (warp & 3) * 32 + lane, group = (warp >> 2) - 1;
    const uint32_t to = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kAccCols;
    const int64_t mine = first < p.tiles ? (p.tiles - first + step - 1) / step : 0, n_stages = mine * (kb1 - kb0);
    int s8 = group, s = group;
    uint32_t p8 = 0, ph = 0;
    uint4 c[8];
    // Tokens (up to 64): 16 codes of a token are two chunks of its f16 row; a thread has one of each 16 tokens.
    const int tch = threadIdx.x & 7, tok0 = (threadIdx.x & 127) >> 3;  // (tok0 + 16 i) % 8 = tok0 % 8
    const int tok_from = kA8Bytes + tok0 * kStage + ((tch ^ (tok0 & 7)) << 4);
    const int tok_to = (tch >> 2) * L::kAtomBytes + tok0 * 128;
    const int j0 = (((tch & 3) * 2) ^ (tok0 & 7)) << 4, j1 = (((tch & 3) * 2 + 1) ^ (tok0 & 7)) << 4;
    uint4 x[4];
    // The copy that refills the slot is of the async proxy and can overtake loads that are still on their way to
    // registers (seen as rows whose last chunks were those of two steps on): the slot goes back once the codes have been
    // converted, so that they have arrived, or (EARLY) behind a proxy fence right after the loads.  The fence takes 100 cycles
    // a step (64 x 4096 x 4096 10.6 us for 10.2), but where CTAs of few tokens stream through tiles, the bytes that are on
    // their way sooner are worth more (16 x 130001 x 4096 88.3 us for 90.5).
    auto hand_back = [&]() {
      __syncwarp();
      if (lane == 0) moe::mbar_arrive(&bar.a8_empty[s8]);
      s8 += kGroups;
      if (s8 >= L::kA8) s8 -= L::kA8, p8 ^= 1u;
    };
    auto load = [&]() {
      if (!wait(&bar.a8_full[s8], p8, 9)) return false;
      const uint8_t* stage = smem + L::kOffA8 + s8 * L::kStageBytes;
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = *reinterpret_cast<const uint4*>(stage + row * kStage + ((j ^ (row & 7)) << 4));
      if constexpr (FORM == kFew) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (tok0 + 16 * i < p.half) x[i] = *reinterpret_cast<const uint4*>(stage + tok_from + i * 16 * kStage);
      }
      if constexpr (EARLY) {
        moe::fence_proxy_async_smem();
        hand_back();
      }
      return true;
    };
    bool ok = group < n_stages && load();
    for (int64_t k = group; ok && k < n_stages; k += kGroups) {
      if (k >= L::kSteps && !wait(&bar.empty[s], ph ^ 1u, 10)) break;
      moe::tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) widen16(c[4 * h + j], v + 8 * j);
        moe::tmem_st32(to + s * kA16Cols + 32 * h, v);
      }
      if constexpr (FORM == kFew) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (tok0 + 16 * i < p.half) {
            uint32_t o[8];
            widen16(x[i], o);
            uint8_t* at = smem + 2 * s * L::kAtomBytes + tok_to + i * 16 * 128;
            *reinterpret_cast<uint4*>(at + j0) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(at + j1) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
        moe::fence_proxy_async_smem();
      }
      if constexpr (!EARLY) hand_back();
      if (k + kGroups < n_stages) ok = load();
      moe::tmem_st_wait();  // also on the way out after a wait that gave up: no store left in flight
      moe::tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) arrive(&bar.full[s]);
      s += kGroups;
      if (s >= L::kSteps) s -= L::kSteps, ph ^= 1u;
    }
  } else {
    if constexpr (HALVES == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kDrainRegs));
    // ------------------------------------------------------ sums, and what they are written as
    const int q = warp & 3, side = (warp - L::kDrainWarp0) >> 2;  // lanes 32 q .., columns 64 side .. of each half
    const uint32_t from = tmem + (static_cast<uint32_t>(32 * q) << 16) + 64 * side;
    auto release = [&](int buf) {
      moe::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(&bar.acc_empty[buf]);
    };
    int64_t chunk = 0;
    bool ok = true;
    for (int64_t it = first; it < p.tiles; it += step) {
      // 64 tokens of each half, of one weight row: fp32, or int32 for those 32 whose bit of `whole` is set (one answer for
      // the warp's lanes); `reach`: what the sums of 32 are below in magnitude, while they are fp32
      uint32_t acc[HALVES][64];
      float reach[HALVES][2];
      uint32_t whole = 0;
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        reach[h][0] = reach[h][1] = 0.0f;
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[h][j] = 0;
      }
      for (int kb = kb0; ok && kb < kb1; kb += kChunk, ++chunk) {
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          const int buf = HALVES == 2 ? h : static_cast<int>(chunk & 1);
          const int64_t used = HALVES == 2 ? chunk : chunk >> 1;
          const int half = h == 0 ? p.half : p.half1;
          ok = ok && wait(&bar.acc_full[buf], used & 1, 11);
          if (!ok) break;
          moe::tc_fence_after();
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // columns past the half's last are read along with it, and not looked at
            if (64 * side + 32 * j < half) {
              uint32_t v[32];
              tmem_ld32(from + buf * p.half + 32 * j, v);
              if (j == 1 || 64 * side + 32 >= half) release(buf);  // what is still to come is in registers
              const uint32_t bit = 1u << (2 * h + j);
              if (!(whole & bit)) {
                float most = 0.0f;
#pragma unroll
                for (int e = 0; e < 16; e += 2) most = most_of(most, v[e], v[e + 1]);
                if (64 * side + 32 * j + 16 < half) {
#pragma unroll
                  for (int e = 16; e < 32; e += 2) most = most_of(most, v[e], v[e + 1]);
                }
                reach[h][j] = __fadd_ru(reach[h][j], most);
                if (__any_sync(0xffffffffu, reach[h][j] > 16777216.0f)) {
                  whole |= bit;
#pragma unroll
                  for (int e = 0; e < 32; ++e) acc[h][32 * j + e] = __float2int_rn(__uint_as_float(acc[h][32 * j + e]));
                }
              }
              if (!(whole & bit)) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  uint32_t* to = &acc[h][32 * j + e];
                  const float2 sum = of_pair(add_pair(pair_of(__uint_as_float(to[0]), __uint_as_float(to[1])),
                                                      pair_of(__uint_as_float(v[e]), __uint_as_float(v[e + 1]))));
                  to[0] = __float_as_uint(sum.x), to[1] = __float_as_uint(sum.y);
                }
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) acc[h][32 * j + e] += __float2int_rn(__uint_as_float(v[e]));
              }
            }
          }
          if (64 * side >= half) release(buf);
        }
      }
      if (parts > 1) {
        // every product is done, so the rings are at rest: they take this CTA's sums, [token][weight row]
        int32_t* sums = reinterpret_cast<int32_t*>(smem);
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (64 * side + j < p.half)
            sums[(64 * side + j) * kRows + 32 * q + lane] =
                whole >> (j >> 5) & 1 ? acc[0][j] : __float2int_rn(__uint_as_float(acc[0][j]));
        if (!ok && lane == 0) bar.broken = 1;
        break;
      }
      const int n = static_cast<int>(it / p.blocks) * kTileRows + static_cast<int>(side_of_pair) * kRows + 32 * q + lane;
      const int m0 = static_cast<int>(it % p.blocks) * tokens + 64 * side;
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (whole >> (2 * h + (j >> 5)) & 1) acc[h][j] = __float_as_uint(__int2float_rn(acc[h][j]));
      const float ws = !ok ? kNan : n < a.n ? scale_at(a.w_scale, n, a.scale_dtype) : 0.0f;
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const int row = m0 + h * p.half;
        const int most = min(min(64, (h == 0 ? p.half : p.half1) - 64 * side), a.m - row);  // tokens of mine that there are
        // their scales: a lane holds two, and hands them round
        const float xs0 = lane < most ? __ldg(a.x_scale + row + lane) : 0.0f;
        const float xs1 = lane + 32 < most ? __ldg(a.x_scale + row + lane + 32) : 0.0f;
        const int64_t at = static_cast<int64_t>(row) * a.n + n;
        if (a.out_dtype == MOE_LAYER_FP32) write_tokens(static_cast<float*>(a.y) + at, a.n, acc[h], ws, xs0, xs1, most, n < a.n);
        else if (a.out_dtype == MOE_LAYER_BF16)
          write_tokens(static_cast<__nv_bfloat16*>(a.y) + at, a.n, acc[h], ws, xs0, xs1, most, n < a.n);
        else write_tokens(static_cast<__half*>(a.y) + at, a.n, acc[h], ws, xs0, xs1, most, n < a.n);
      }
    }
  }
  // (of a pair: no CTA ends, or gives its tensor memory back, while the other's products or arrivals may be under way)
  if constexpr (FORM == kTwo) cluster_sync();
  else __syncthreads();
  // Tokens on their way into a CTA in which a wait gave up: converters that stopped never complete their steps' barriers,
  // so the CTA stays for as long as any other wait takes at most.  A CTA in which none did has drained all of its products,
  // which read every copy that there was.
  if (FORM != kFew && warp == 2 && *abort) wait_out_budget();
  if (warp == 1) {
    moe::tc_fence_after();
    if constexpr (FORM == kTwo) pair_dealloc(tmem, kTmemCols);
    else moe::tmem_dealloc(tmem, kTmemCols);
  }
  if constexpr (HALVES == 1) {
    if (parts > 1) {
      // each CTA adds up its share of the tokens, a thread four weight rows of one
      const int m0 = static_cast<int>(first % p.blocks) * p.half, row = (threadIdx.x & 31) * 4;
      const int n = static_cast<int>(first / p.blocks) * kRows + row;
      const int c0 = static_cast<int>(p.half * rank / parts), c1 = min(static_cast<int>(p.half * (rank + 1) / parts), a.m - m0);
      static_assert(L::kHalf <= 8 * (kThreads / 32), "tokens of a warp");
      float ws[4], xs[4];  // (two CTAs at least: four tokens a warp at most)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + warp + j * (kThreads / 32);
        ws[j] = n + j < a.n ? scale_at(a.w_scale, n + j, a.scale_dtype) : 0.0f;
        xs[j] = c < c1 ? __ldg(a.x_scale + m0 + c) : 0.0f;
      }
      cluster_sync();
      int broken = 0;
      int4 sum[4];
#pragma unroll
      for (uint32_t r = 0; r < kMostParts; ++r)
        if (r < parts) broken |= __float_as_int(cluster_read(moe::smem_u32(&bar.broken), r));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + warp + j * (kThreads / 32);
        int4 part[kMostParts];
        sum[j] = make_int4(0, 0, 0, 0);
        if (c >= c1) continue;
#pragma unroll
        for (uint32_t r = 0; r < kMostParts; ++r)
          if (r < parts) part[r] = cluster_read4(moe::smem_u32(smem) + (c * kRows + row) * 4, r);
#pragma unroll
        for (uint32_t r = 0; r < kMostParts; ++r)
          if (r < parts) sum[j].x += part[r].x, sum[j].y += part[r].y, sum[j].z += part[r].z, sum[j].w += part[r].w;
      }
      cluster_arrive();  // what this CTA reads of the others has been read
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + warp + j * (kThreads / 32);
        const int32_t v[4] = {sum[j].x, sum[j].y, sum[j].z, sum[j].w};
        if (c >= c1) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < a.n)
            store_y(a.y, static_cast<int64_t>(m0 + c) * a.n + n + e, scaled(v[e], broken ? kNan : ws[e], xs[j]), a.out_dtype);
      }
      cluster_wait();  // no CTA ends while its sums are read
    }
  }
  grid_dependency_wait();  // the next launch takes this grid's end for the widening kernel's too
}

struct Shape {
  int form, half, half1, blocks;
  int64_t tiles;
};

// The tiles that take the least time by a count of cycles, fitted to 33 sizes of 160..4093 tokens with every tile of
// them (of 500 times within 4 %, the tile chosen on average 1 % off the best): with one half of t tokens a step costs 525 +
// 1.4 t, a pair's 270 + 3.2 t and no less than the conversion of the weights, 830; a tile some more, and SMs work in rounds.
// A pair reads weights and tokens half as often and wins once there are tiles for all SMs (1024 x 4096 x 4096 28.7 us for
// 31.8; 512 x 4096 x 4096, where one half fills the SMs and a pair does not, 19.3 for 23.1).
Shape shape_of(int m, int n, int k, int num_sms) {
  const int64_t rows = (static_cast<int64_t>(n) + kRows - 1) / kRows;
  if (m <= 64) return Shape{kFew, (m + 15) / 16 * 16, 0, 1, rows};
  const int steps = (k + kStage - 1) / kStage;
  Shape s{};
  double best = 0;
  for (int form = kOne; form <= kTwo; ++form) {
    const int halves = form == kTwo ? 2 : 1, least = (m + 128 * halves - 1) / (128 * halves);
    if (form == kTwo && m <= 128) break;
    for (int b = least; b <= 2 * least; ++b) {
      // (a pair's product is of a multiple of 32 tokens)
      const int unit = form == kTwo ? 32 : 16, tokens = ((m + b - 1) / b + unit - 1) / unit * unit;
      const int half1 = form == kTwo ? tokens / 64 * 32 : 0, half = tokens - half1, blocks = (m + tokens - 1) / tokens;
      const int64_t tiles = (form == kTwo ? (rows + 1) / 2 : rows) * blocks, at_once = form == kTwo ? num_sms / 2 : num_sms;
      const int64_t rounds = (tiles + at_once - 1) / at_once;
      int parts = 1;  // of k, in a cluster
      if (form == kOne)
        while (parts < static_cast<int>(kMostParts) && tiles * (parts + 1) <= num_sms && steps >= 2 * (parts + 1)) ++parts;
      const double a_step = form == kTwo ? std::max(830.0, 270 + 3.2 * tokens) : (525 + 1.4 * tokens) / parts;
      const double cost = rounds * (steps * a_step + (form == kTwo ? 2800 : 900) + (parts > 1 ? 4600 : 0));
      if (best == 0 || cost < best) best = cost, s = Shape{form, half, half1, blocks, tiles};
    }
  }
  return s;
}

// How many clusters of `parts` CTAs the current device runs at once; asked once a device and size.
template <int FORM, bool EARLY>
int clusters_at_once(int parts) {
  static std::atomic<int> known[64][9];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = known[dev][parts].load(std::memory_order_relaxed)) > 0) return n - 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Layout<FORM>::kBytes + 1024;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, w8_tc_kernel<FORM, EARLY>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (dev < 64) known[dev][parts].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <int FORM, bool EARLY = false>
cudaError_t launch_tiles(const Maps& maps, const Params& p, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  const void* k = (const void*)w8_tc_kernel<FORM, EARLY>;
  if (const cudaError_t e = allow_smem(k, kMaxSmem, allowed, FORM == kTwo ? kLaunchRegs : 0); e != cudaSuccess) return e;
  int parts = 1;
  if constexpr (FORM != kTwo) {
    // clusters that share k out, as large as all of them run at once and have two steps a CTA
    const int steps = (p.a.k + kStage - 1) / kStage;
    for (int c = kMostParts; c > 1 && parts == 1; --c)
      if (p.tiles * c <= num_sms && steps >= 2 * c && clusters_at_once<FORM, EARLY>(c) >= p.tiles) parts = c;
  }
  Maps m = maps;
  Params arg = p;
  void* args[] = {&m, &arg};
  if constexpr (FORM == kTwo) {
    int64_t pairs = clusters_at_once<FORM, EARLY>(2);
    if (pairs < 1) pairs = num_sms / 2;
    if (p.tiles < pairs) pairs = p.tiles;
    return launch_after(k, dim3(static_cast<unsigned>(2 * pairs)), dim3(kThreads), args, Layout<FORM>::kBytes + 1024, s, 2);
  }
  const int64_t grid = parts > 1 ? p.tiles * parts : p.tiles < num_sms ? p.tiles : num_sms;
  return launch_after(k, dim3(static_cast<unsigned>(grid)), dim3(kThreads), args, Layout<FORM>::kBytes + 1024, s, parts);
}

}  // namespace

size_t w8_tc_workspace(int m, int, int k, int) { return m <= 64 ? 0 : 256 + static_cast<size_t>(m) * k * 2; }

cudaError_t launch_w8_tc(const moe_layer_w8_args_t& a, void* ws, int num_sms, cudaStream_t s) {
  const Shape shape = shape_of(a.m, a.n, a.k, num_sms);
  Maps maps{};
  if (!moe::encode_2d(&maps.w, a.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.n, a.k, kStage, kRows, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  Params p{a, nullptr, shape.half, shape.half1, shape.blocks, shape.tiles};
  if (shape.form == kFew) {
    if (!moe::encode_2d(&maps.x, a.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.m, a.k, kStage, shape.half,
                        CU_TENSOR_MAP_SWIZZLE_128B, a.x_stride))
      return cudaErrorInvalidValue;
    return p.tiles > num_sms ? launch_tiles<kFew, true>(maps, p, num_sms, s) : launch_tiles<kFew>(maps, p, num_sms, s);
  }
  p.status = static_cast<int32_t*>(ws);
  __half* x16 = reinterpret_cast<__half*>(static_cast<char*>(ws) + 256);
  if (!moe::encode_2d(&maps.x, x16, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a.m, a.k, kAtom,
                      shape.half / (shape.form == kTwo ? 2 : 1), CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if (shape.form == kTwo && !moe::encode_2d(&maps.y, x16, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a.m, a.k, kAtom, shape.half1 / 2,
                                            CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  moe_layer_w8_args_t arg = a;
  int shift = 0;  // a thread has one to four pieces of a row where it can
  while (shift < 8 && (8 << (shift + 2)) < a.k) ++shift;
  void* args[] = {&arg, &x16, &p.status, &shift};
  const int rows = kWidenThreads >> shift;
  const cudaError_t e = launch_after((const void*)w8_widen_kernel, dim3(static_cast<unsigned>((a.m + rows - 1) / rows)),
                                     dim3(kWidenThreads), args, 0, s);
  if (e != cudaSuccess) return e;
  return shape.form == kTwo ? launch_tiles<kTwo>(maps, p, num_sms, s) : launch_tiles<kOne>(maps, p, num_sms, s);
}

}  // namespace moe_layer
