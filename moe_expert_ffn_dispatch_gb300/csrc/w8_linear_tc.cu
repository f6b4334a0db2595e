// 8-bit products of more tokens than a few, on the tensor cores' tensor memory,
// exact in int32.
//
// The tensor cores of this chip have no integer kind: codes run as f16 (every
// integer in [-128, 127] is exact), sums as fp32 in tensor memory.  A product of two
// codes is at most 2^14, so 1024 consecutive k sum to at most 2^24, exactly; each
// accumulator covers 1024 k at most and is then drained into int32 registers.
//
// A tile is 128 weight rows (M, the tensor memory's lanes) by up to 256 tokens (N, in
// one or two halves of at most 128 columns).  Weights arrive as int8 by TMA and are
// converted in the CTA into tensor memory, the products' A operand, so that they
// cross memory and L2 as bytes.  Tokens are converted once by a kernel before this
// one, into the workspace, and arrive as f16 in shared memory.
// The two halves of a wide tile have an accumulator each, side by side: most steps of
// 128 k multiply both at once, the first and the last of a 1024 k the first half
// before the second, so that one is drained while the other's products run.  A tile
// of one half alternates between two accumulators.
// What bounds a step is how fast one warp can wait, issue and commit (about 100 cycles
// a wait, 40 a product): weights and tokens of a step complete one barrier, and its
// products one other.
// Roles: warp 0 copies weights, warp 2 copies tokens, warp 1 issues products, warps
// 4..7 convert weights (a row a thread), warps 8..15 drain and write.
// Where there are fewer tiles than SMs a cluster shares k out, and adds its int32
// sums up over distributed shared memory, a share of the tile's columns each.
#include "w8_linear.cuh"

#include "device_prims.cuh"
#include "tensor_map.cuh"

namespace moe_layer {
namespace {

constexpr int kRows = 128;          // weight rows of a tile
constexpr int kHalf = 128;          // tokens of a half at most
constexpr int kStage = 128;         // k of a weight stage
constexpr int kAtom = 64;           // k of one 128-byte row of f16
constexpr int kChunk = 1024 / kStage;  // stages that a sum stays exact for
constexpr int kA16Cols = kStage / 2;  // of a converted weight stage in tensor memory
constexpr int kAccCols = 2 * kHalf;
constexpr int kTmemCols = 512;
constexpr int kThreads = 512;
constexpr int kConvWarps = 4, kDrainWarps = 8;
// Registers a thread where a tile has two halves: 128 at launch, and what the drain warps have more the others give.
// (With one half nobody needs more, and the sums over a cluster are every warp's.)
constexpr int kRoleRegs = 72, kConvRegs = 104, kDrainRegs = 168;
static_assert(128 * kRoleRegs + 128 * kConvRegs + 256 * kDrainRegs <= kThreads * 128, "the split fits what the launch has");
constexpr int kA8Bytes = kRows * kStage;
constexpr int kSite = 2 << 8;       // of the waits, in the status

// HALVES: of a tile's tokens.  Shared memory: tokens of each step, weight stages, barriers
template <int HALVES>
struct Layout {
  static constexpr int kAtomBytes = HALVES * kHalf * kAtom * 2;
  static constexpr int kSteps = HALVES == 2 ? 3 : 4;  // tokens in shared memory, converted weights in tensor memory
  static constexpr int kA8 = HALVES == 2 ? 2 : 6;     // weights as they arrive
  static constexpr int kOffA8 = kSteps * 2 * kAtomBytes, kOffBar = kOffA8 + kA8 * kA8Bytes;
  static constexpr int kBytes = kOffBar + 512;
  static_assert(kBytes + 1024 <= kMaxSmem, "shared memory");
  static_assert(kAccCols + kSteps * kA16Cols <= kTmemCols, "tensor memory");
};
static_assert(Layout<1>::kOffBar >= kHalf * kRows * 4, "the sums of a tile of one half fit the rings");

struct Barriers {
  uint64_t a8_full[8], a8_empty[8], full[4], empty[4], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Barriers) <= 512, "");

struct alignas(64) Maps {
  CUtensorMap w;  // int8 [n, k], box {128, 128}, 128-byte swizzle
  CUtensorMap x;  // f16 [m, k], box {64, tokens of a tile}, 128-byte swizzle
};

struct Params {
  moe_layer_w8_args_t a;
  int32_t* status;
  int half;     // tokens of a half, a multiple of 16
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

// the tokens as f16, dense; and the status words of the call
__global__ void __launch_bounds__(256) w8_widen_kernel(const moe_layer_w8_args_t a, __half* x16, int32_t* status) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x < 8) status[threadIdx.x] = 0;
  const int chunks = a.k / 16;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<int64_t>(a.m) * chunks) return;
  const int64_t row = i / chunks;
  const int c = static_cast<int>(i - row * chunks);
  uint32_t o[8];
  widen16(*reinterpret_cast<const uint4*>(a.x + row * a.x_stride + c * 16), o);
  uint4* to = reinterpret_cast<uint4*>(x16 + i * 16);
  to[0] = make_uint4(o[0], o[1], o[2], o[3]);
  to[1] = make_uint4(o[4], o[5], o[6], o[7]);
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
__device__ __forceinline__ void write_tokens(T* y, int64_t stride, const int32_t (&acc)[64], float ws, float xs0, float xs1,
                                             int most, bool mine) {
#pragma unroll
  for (int j = 0; j < 64; ++j) {
    const float xs = __shfl_sync(0xffffffffu, j < 32 ? xs0 : xs1, j & 31);
    if (j < most && mine) put(y, scaled(acc[j], ws, xs));
    y += stride;
  }
}

// The same for the steps, whose barriers the converters complete too: where they have given up, a phase never completes
// and the copies get a while to land.
__device__ __forceinline__ void drain_steps(uint64_t* full, int n, int s, uint32_t ph, bool wrapped, volatile int* abort,
                                            int32_t* status, int site) {
  for (int i = 0; i < n; ++i) {
    const uint32_t parity = i < s ? ph : ph ^ 1u;
    if (i < s || wrapped) moe::mbar_wait_bounded(&full[i], parity, abort, status, site);
  }
  if (*abort)
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

template <int HALVES>
__global__ void __launch_bounds__(kThreads, 1) w8_tc_kernel(const __grid_constant__ Maps maps, const Params p) {
  using L = Layout<HALVES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (moe::smem_u32(smem_raw) & 1023u)) & 1023u);
  Barriers& bar = *reinterpret_cast<Barriers*>(smem + L::kOffBar);
  const moe_layer_w8_args_t& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank, parts;  // of the cluster that shares k out
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(parts));
  const int64_t first = blockIdx.x / parts, step = gridDim.x / parts;
  const int stages = (a.k + kStage - 1) / kStage;
  const int kb0 = static_cast<int>(static_cast<int64_t>(stages) * rank / parts),
            kb1 = static_cast<int>(static_cast<int64_t>(stages) * (rank + 1) / parts);

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kA8; ++i) {
      moe::mbar_init(&bar.a8_full[i], 1);
      moe::mbar_init(&bar.a8_empty[i], kConvWarps);
    }
    for (int i = 0; i < L::kSteps; ++i) {
      moe::mbar_init(&bar.full[i], kConvWarps + 1);
      moe::mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      moe::mbar_init(&bar.acc_full[i], 1);
      moe::mbar_init(&bar.acc_empty[i], kDrainWarps);
    }
    moe::mbar_init(&bar.drain, 1);
    bar.abort = 0;
    moe::fence_barrier_init();
  }
  if (warp == 1) moe::tmem_alloc(&bar.tmem, kTmemCols);
  __syncthreads();
  moe::tc_fence_after();
  const uint32_t tmem = bar.tmem;
  volatile int* abort = &bar.abort;
  // A bounded wait of a whole warp, with one answer for all of its lanes.  The status words are the widening kernel's
  // to clear: what is reported before it is done would be lost, but nothing waits that long before it.
  auto wait = [&](uint64_t* b, uint32_t parity, int site) {
    return __all_sync(0xffffffffu, moe::mbar_wait_bounded(b, parity, abort, p.status, kSite + site)) != 0;
  };

  if (warp < 4) {
    if constexpr (HALVES == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
    if (warp == 0) {
      // ---------------------------------------------------- weights: what the call before this one left is complete
      // once the widening kernel runs, which waited for it
      int s = 0;
      uint32_t ph = 0;
      bool wrapped = false, ok = true;
      for (int64_t it = first; ok && it < p.tiles; it += step) {
        const int n0 = static_cast<int>(it / p.blocks) * kRows;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (wrapped && !wait(&bar.a8_empty[s], ph ^ 1u, 1)) {
            ok = false;
            break;
          }
          if (moe::elect_one()) {
            moe::mbar_arrive_expect_tx(&bar.a8_full[s], kA8Bytes);
            moe::tma_load_2d(smem + L::kOffA8 + s * kA8Bytes, &maps.w, kb * kStage, n0, &bar.a8_full[s]);
          }
          __syncwarp();
          if (++s == L::kA8) s = 0, ph ^= 1u, wrapped = true;
        }
      }
      drain_ring(bar.a8_full, L::kA8, s, ph, wrapped, p.status, kSite + 2);
    } else if (warp == 2) {
      // ---------------------------------------------------- tokens
      grid_dependency_wait();
      int s = 0;
      uint32_t ph = 0;
      bool wrapped = false, ok = true;
      const int tokens = p.half * HALVES;
      for (int64_t it = first; ok && it < p.tiles; it += step) {
        const int m0 = static_cast<int>(it % p.blocks) * tokens;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (wrapped && !wait(&bar.empty[s], ph ^ 1u, 3)) {
            ok = false;
            break;
          }
          if (moe::elect_one()) {
            moe::mbar_arrive_expect_tx(&bar.full[s], 2 * tokens * kAtom * 2);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              moe::tma_load_2d(smem + (2 * s + h) * L::kAtomBytes, &maps.x, kb * kStage + h * kAtom, m0, &bar.full[s]);
          }
          __syncwarp();
          if (++s == L::kSteps) s = 0, ph ^= 1u, wrapped = true;
        }
      }
      // what it armed has landed, or (the converters having given up) is past where a barrier could tell
      drain_steps(bar.full, L::kSteps, s, ph, wrapped, abort, p.status, kSite + 4);
    } else if (warp == 1) {
      // ---------------------------------------------------- products
      const uint32_t idesc = moe::umma_idesc_f16(kRows, p.half), idesc_both = moe::umma_idesc_f16(kRows, HALVES * p.half);
      const uint64_t b0 = moe::umma_desc_sw128(moe::smem_u32(smem));
      constexpr uint64_t kAtomAt = L::kAtomBytes >> 4;
      const uint64_t half_at = (p.half * kAtom * 2) >> 4;
      // eight products of 16 k
      auto products = [&](uint32_t d, uint32_t at, uint64_t bd, uint32_t form, bool fresh) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          moe::umma_f16_ts(d, at + 8 * k, bd + (k >> 2) * kAtomAt + 2 * (k & 3), form, !fresh || k != 0);
      };
      int s = 0;
      uint32_t ph = 0;
      int64_t chunk = 0;
      bool ok = true;
      for (int64_t it = first; ok && it < p.tiles; it += step) {
        int kc = 0;  // step of the chunk
        for (int kb = kb0; kb < kb1; ++kb) {
          const bool last = kc + 1 == kChunk || kb + 1 == kb1;
          const uint32_t at = tmem + kAccCols + s * kA16Cols;
          const uint64_t bd = b0 + 2 * s * kAtomAt;
          if (HALVES == 2 && kc != 0 && !last) {
            ok = wait(&bar.full[s], ph, 5);
            if (!ok) break;
            moe::tc_fence_after();
            if (moe::elect_one()) {
              products(tmem, at, bd, idesc_both, false);
              moe::umma_commit(&bar.empty[s]);
            }
          } else {
            ok = wait(&bar.full[s], ph, 6);
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
              // the accumulator's uses so far: a half's own one a chunk, or two in turn
              const int buf = HALVES == 2 ? h : static_cast<int>(chunk & 1);
              const int64_t used = HALVES == 2 ? chunk : chunk >> 1;
              if (kc == 0 && used > 0) ok = ok && wait(&bar.acc_empty[buf], (used - 1) & 1, 7);
              if (!ok) break;
              moe::tc_fence_after();
              if (moe::elect_one()) {
                products(tmem + buf * p.half, at, bd + h * half_at, idesc, kc == 0);
                if (h == HALVES - 1) moe::umma_commit(&bar.empty[s]);
                if (last) moe::umma_commit(&bar.acc_full[buf]);
              }
              __syncwarp();
            }
            if (!ok) break;
          }
          __syncwarp();
          if (++s == L::kSteps) s = 0, ph ^= 1u;
          if (last) ++chunk, kc = 0;
          else ++kc;
        }
      }
      // nothing of this CTA is in flight when its tensor memory goes back
      if (moe::elect_one()) moe::umma_commit(&bar.drain);
      __syncwarp();
      moe::mbar_wait_bounded(&bar.drain, 0, nullptr, p.status, kSite + 8);
    }
  } else if (warp < 8) {
    if constexpr (HALVES == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    // ------------------------------------------------------ weights to f16, a row a thread, into tensor memory
    // (16-byte chunk j of row r lies at chunk j ^ (r % 8) of its 128 bytes).  The next stage's codes are loaded while
    // this one's stores are on their way.
    const int row = (warp - 4) * 32 + lane;
    const uint32_t to = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kAccCols;
    const int64_t mine = first < p.tiles ? (p.tiles - first + step - 1) / step : 0, n_stages = mine * (kb1 - kb0);
    int s8 = 0, s = 0;
    uint32_t p8 = 0, ph = 0;
    uint4 c[8];
    auto load = [&]() {
      if (!wait(&bar.a8_full[s8], p8, 9)) return false;
      const uint8_t* from = smem + L::kOffA8 + s8 * kA8Bytes + row * kStage;
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = *reinterpret_cast<const uint4*>(from + ((j ^ (row & 7)) << 4));
      __syncwarp();
      if (lane == 0) moe::mbar_arrive(&bar.a8_empty[s8]);
      if (++s8 == L::kA8) s8 = 0, p8 ^= 1u;
      return true;
    };
    bool ok = n_stages > 0 && load();
    for (int64_t k = 0; ok && k < n_stages; ++k) {
      if (k >= L::kSteps && !wait(&bar.empty[s], ph ^ 1u, 10)) break;
      moe::tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) widen16(c[4 * h + j], v + 8 * j);
        moe::tmem_st32(to + s * kA16Cols + 32 * h, v);
      }
      if (k + 1 < n_stages) ok = load();
      moe::tmem_st_wait();  // also on the way out after a wait that gave up: no store left in flight
      moe::tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) moe::mbar_arrive(&bar.full[s]);
      if (++s == L::kSteps) s = 0, ph ^= 1u;
    }
  } else {
    if constexpr (HALVES == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kDrainRegs));
    // ------------------------------------------------------ sums, and what they are written as
    const int q = warp & 3, side = (warp - 8) >> 2;  // lanes 32 q .., columns 64 side .. of each half
    const uint32_t from = tmem + (static_cast<uint32_t>(32 * q) << 16) + 64 * side;
    int64_t chunk = 0;
    bool ok = true;
    for (int64_t it = first; ok && it < p.tiles; it += step) {
      int32_t acc[HALVES][64];  // 64 tokens of each half, of one weight row
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[h][j] = 0;
      for (int kb = kb0; ok && kb < kb1; kb += kChunk, ++chunk) {
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          const int buf = HALVES == 2 ? h : static_cast<int>(chunk & 1);
          const int64_t used = HALVES == 2 ? chunk : chunk >> 1;
          ok = ok && wait(&bar.acc_full[buf], used & 1, 11);
          if (!ok) break;
          moe::tc_fence_after();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (64 * side + 16 * j < p.half) {
              uint32_t v[16];
              moe::tmem_ld16(from + buf * p.half + 16 * j, v);
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[h][16 * j + e] += __float2int_rn(__uint_as_float(v[e]));
            }
          }
          moe::tc_fence_before();
          __syncwarp();
          if (lane == 0) moe::mbar_arrive(&bar.acc_empty[buf]);
        }
      }
      if (parts > 1) {
        // every product is done, so the rings are at rest: they take this CTA's sums, [token][weight row]
        int32_t* sums = reinterpret_cast<int32_t*>(smem);
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (64 * side + j < p.half) sums[(64 * side + j) * kRows + 32 * q + lane] = acc[0][j];
        break;
      }
      if (!ok) break;
      const int n = static_cast<int>(it / p.blocks) * kRows + 32 * q + lane;
      const int m0 = static_cast<int>(it % p.blocks) * p.half * HALVES + 64 * side;
      const float ws = n < a.n ? scale_at(a.w_scale, n, a.scale_dtype) : 0.0f;
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const int row = m0 + h * p.half;
        const int most = min(min(64, p.half - 64 * side), a.m - row);  // tokens of mine that there are
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
  __syncthreads();
  if (warp == 1) {
    moe::tc_fence_after();
    moe::tmem_dealloc(tmem, kTmemCols);
  }
  if constexpr (HALVES == 1) {
    if (parts > 1) {
      // each CTA adds up its share of the tokens
      const int32_t* sums = reinterpret_cast<const int32_t*>(smem);
      cluster_sync();
      const int m0 = static_cast<int>(first % p.blocks) * p.half, row = threadIdx.x & (kRows - 1);
      const int n = static_cast<int>(first / p.blocks) * kRows + row;
      const int c0 = static_cast<int>(p.half * rank / parts), c1 = static_cast<int>(p.half * (rank + 1) / parts);
      const float ws = n < a.n ? scale_at(a.w_scale, n, a.scale_dtype) : 0.0f;
      for (int c = c0 + static_cast<int>(threadIdx.x / kRows); c < c1; c += kThreads / kRows) {
        int32_t sum = 0;
        for (uint32_t r = 0; r < parts; ++r)
          sum += __float_as_int(cluster_read(moe::smem_u32(sums + c * kRows + row), r));
        if (n < a.n && m0 + c < a.m)
          store_y(a.y, static_cast<int64_t>(m0 + c) * a.n + n, scaled(sum, ws, __ldg(a.x_scale + m0 + c)), a.out_dtype);
      }
      cluster_sync();  // no CTA ends while its sums are read
    }
  }
  grid_dependency_wait();  // the next launch takes this grid's end for the widening kernel's too
}

struct Shape {
  int halves, half, blocks, parts;
  int64_t tiles;
};
Shape shape_of(int m, int n, int k, int num_sms) {
  const int64_t rows = (static_cast<int64_t>(n) + kRows - 1) / kRows;
  Shape s{};
  if (m <= kHalf) {
    s = Shape{1, (m + 15) / 16 * 16, 1, 1, rows};
  } else {
    // tiles as wide as they go, narrower ones where that fills the last round of SMs better
    double best = 0;
    for (int blocks = (m + 255) / 256; blocks <= (m + 255) / 256 * 2; ++blocks) {
      const int half = ((m + blocks - 1) / blocks + 31) / 32 * 16;
      const int64_t tiles = rows * ((m + 2 * half - 1) / (2 * half));
      const double cost = static_cast<double>((tiles + num_sms - 1) / num_sms) * (2 * half + 16);
      if (best == 0 || cost < best) best = cost, s = Shape{2, half, (m + 2 * half - 1) / (2 * half), 1, tiles};
    }
  }
  const int stages = (k + kStage - 1) / kStage;
  if (s.halves == 1)
    while (s.parts < 8 && s.tiles * s.parts * 2 <= num_sms && stages >= s.parts * 4) s.parts *= 2;
  return s;
}

template <int HALVES>
cudaError_t launch_tiles(const Maps& maps, const Params& p, int parts, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  const void* k = (const void*)w8_tc_kernel<HALVES>;
  if (const cudaError_t e = allow_smem(k, kMaxSmem, allowed); e != cudaSuccess) return e;
  Maps m = maps;
  Params arg = p;
  void* args[] = {&m, &arg};
  const int64_t grid = parts > 1 ? p.tiles * parts : p.tiles < num_sms ? p.tiles : num_sms;
  return launch_after(k, dim3(static_cast<unsigned>(grid)), dim3(kThreads), args, Layout<HALVES>::kBytes + 1024, s, parts);
}

}  // namespace

size_t w8_tc_workspace(int m, int, int k, int) { return 256 + static_cast<size_t>(m) * k * 2; }

cudaError_t launch_w8_tc(const moe_layer_w8_args_t& a, void* ws, int num_sms, cudaStream_t s) {
  const Shape shape = shape_of(a.m, a.n, a.k, num_sms);
  moe_layer_w8_args_t arg = a;
  __half* x16 = reinterpret_cast<__half*>(static_cast<char*>(ws) + 256);
  Params p{a, static_cast<int32_t*>(ws), shape.half, shape.blocks, shape.tiles};
  Maps maps;
  if (!moe::encode_2d(&maps.w, a.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.n, a.k, kStage, kRows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !moe::encode_2d(&maps.x, x16, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a.m, a.k, kAtom, shape.halves * shape.half,
                      CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  void* args[] = {&arg, &x16, &p.status};
  const int64_t chunks = static_cast<int64_t>(a.m) * (a.k / 16);
  const cudaError_t e = launch_after((const void*)w8_widen_kernel, dim3(static_cast<unsigned>((chunks + 255) / 256)), dim3(256),
                                     args, 0, s);
  if (e != cudaSuccess) return e;
  return shape.halves == 2 ? launch_tiles<2>(maps, p, shape.parts, num_sms, s)
                           : launch_tiles<1>(maps, p, shape.parts, num_sms, s);
}

}  // namespace moe_layer
