// Products of INT8 codes with INT8 weights, exact in int32, with a scale a token
// and a scale a channel: up to 8 tokens, and the choice of kernel.
//
// Weight rows are the M side of mma.sync m16n8k32, tokens its N side.  A CTA takes 16
// weight rows at a time; its warps share out k in steps of 128 and add up in shared
// memory.  A lane loads 16 bytes of a weight row (and of a token) at a time, 64 apart:
// the four words of a load are k-words of four products, in the same order for weights
// and tokens, which is all that the sum asks for.
// Bound by memory: the weights once.  Each warp has the loads of its next steps in
// flight, those of the next 16 rows among them while it adds up these.
#include "w8_linear.cuh"

namespace moe_layer {
namespace {

constexpr int kFewTokens = 8;
constexpr int kFewWarps = 8, kFewThreads = kFewWarps * 32;
constexpr int kFewRows = 16;   // weight rows of a tile
constexpr int kStep = 128;     // k of a warp's step
constexpr int kRing = 4;       // steps in flight

// D(16x8, s32) += A(16x32, s8, row) * B(32x8, s8, col).  Lane = 4 g + t.  A: a0
// (row g, k 4t ..), a1 (row g+8), a2 (row g, k 16 + 4t ..), a3; B: b0 (k 4t ..,
// column g), b1 (k 16 + 4t ..); D: d0 d1 (row g, columns 2t, 2t+1), d2 d3 (row g+8).
__device__ __forceinline__ void mma_s8(int32_t (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__global__ void __launch_bounds__(kFewThreads, 2) w8_few_kernel(const moe_layer_w8_args_t a, int64_t tiles) {
  __shared__ int32_t s_part[2][kFewWarps][kFewTokens][kFewRows + 1];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int steps = (a.k + kStep - 1) / kStep;
  const int mine = warp < steps ? (steps - warp + kFewWarps - 1) / kFewWarps : 0;  // this warp's steps of a tile
  const bool has_x = g < a.m;
  const int8_t* x = a.x + (has_x ? g : 0) * a.x_stride;
  uint4 wv[kRing][2][2], xv[kRing][2];
  // the next step to load: of tile `lt`, the warp's step number `ls`
  int64_t lt = mine ? blockIdx.x : tiles;
  int ls = 0;
  auto load = [&](uint4 (&wr)[2][2], uint4 (&xr)[2]) {
    const int k0 = (warp + ls * kFewWarps) * kStep + 16 * t;
    const int64_t n0 = lt * kFewRows + g;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = k0 + 64 * j;
      const bool in = lt < tiles && k < a.k;
      xr[j] = wr[j][0] = wr[j][1] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (in && n0 + 8 * i < a.n) wr[j][i] = __ldcs(reinterpret_cast<const uint4*>(a.w + (n0 + 8 * i) * a.k + k));
      if (in && has_x) xr[j] = __ldg(reinterpret_cast<const uint4*>(x + k));
    }
    if (++ls >= mine) ls = 0, lt += gridDim.x;
  };
  if (mine) {
#pragma unroll
    for (int r = 0; r < kRing; ++r) load(wv[r], xv[r]);
  }
  int buf = 0, done = 0;  // steps of the tile that is multiplied
  int64_t tile = blockIdx.x;
  int32_t d[4] = {};
  // adds up a tile once its last step is done; false after the last tile
  auto finish = [&]() {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s_part[buf][warp][2 * t + (e & 1)][g + 8 * (e >> 1)] = d[e];
      d[e] = 0;
    }
    __syncthreads();  // (two buffers: the next tile's sums are written while these are read)
    for (int i = threadIdx.x; i < kFewTokens * kFewRows; i += kFewThreads) {
      const int tok = i / kFewRows, r = i % kFewRows;
      const int64_t n = tile * kFewRows + r;
      if (tok >= a.m || n >= a.n) continue;
      int32_t sum = 0;
#pragma unroll
      for (int q = 0; q < kFewWarps; ++q) sum += s_part[buf][q][tok][r];
      store_y(a.y, static_cast<int64_t>(tok) * a.n + n, scaled(sum, scale_at(a.w_scale, n, a.scale_dtype), a.x_scale[tok]),
              a.out_dtype);
    }
    buf ^= 1;
    done = 0;
    tile += gridDim.x;
    return tile < tiles;
  };
  if (!mine) {
    while (finish()) {
    }
    return;
  }
  while (true) {
#pragma unroll
    for (int r = 0; r < kRing; ++r) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mma_s8(d, wv[r][j][0].x, wv[r][j][1].x, wv[r][j][0].y, wv[r][j][1].y, xv[r][j].x, xv[r][j].y);
        mma_s8(d, wv[r][j][0].z, wv[r][j][1].z, wv[r][j][0].w, wv[r][j][1].w, xv[r][j].z, xv[r][j].w);
      }
      load(wv[r], xv[r]);
      if (++done == mine && !finish()) return;
    }
  }
}

}  // namespace

size_t w8_workspace(int m, int n, int k, int num_sms) { return m <= kFewTokens ? 0 : w8_tc_workspace(m, n, k, num_sms); }

cudaError_t launch_w8(const moe_layer_w8_args_t& a, void* ws, int num_sms, cudaStream_t s) {
  if (a.m > kFewTokens) return launch_w8_tc(a, ws, num_sms, s);
  moe_layer_w8_args_t arg = a;
  int64_t tiles = (static_cast<int64_t>(a.n) + kFewRows - 1) / kFewRows;
  void* args[] = {&arg, &tiles};
  const int64_t grid = tiles < 2 * num_sms ? tiles : 2 * num_sms;
  return launch_after((const void*)w8_few_kernel, dim3(static_cast<unsigned>(grid)), dim3(kFewThreads), args, 0, s);
}

}  // namespace moe_layer
