// Products of INT8 codes with INT8 weights, exact in int32, with a scale a token
// and a scale a channel: few tokens, and the choice of kernel.
//
// Weight rows are the M side of mma.sync m16n8k32, tokens its N side.  A CTA takes 16
// weight rows at a time; its warps share out k in steps of 128 and add up in shared
// memory.  A lane loads 16 bytes of a weight row (and of a token) at a time, 64 apart:
// the four words of a load are k-words of four products, in the same order for weights
// and tokens, which is all that the sum asks for.
// Bound by memory: the weights once.  Each warp has the loads of its next steps in
// flight, those of the next 16 rows among them while it adds up these: 8 x 130001 x
// 4096 84 us, 6.4 TB/s; 8 x 6144 x 4096 7.3 to 8 us, of which launch and first load are 3.
#include "w8_linear.cuh"

namespace moe_layer {
namespace {

constexpr int kFewWarps = 8, kFewThreads = kFewWarps * 32;
constexpr int kFewRows = 16;   // weight rows of a tile
constexpr int kStep = 128;     // k of a warp's step

// D(16x8, s32) += A(16x32, s8, row) * B(32x8, s8, col).  Lane = 4 g + t.  A: a0
// (row g, k 4t ..), a1 (row g+8), a2 (row g, k 16 + 4t ..), a3; B: b0 (k 4t ..,
// column g), b1 (k 16 + 4t ..); D: d0 d1 (row g, columns 2t, 2t+1), d2 d3 (row g+8).
__device__ __forceinline__ void mma_s8(int32_t (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: tokens in eights; RING: steps in flight
template <int NT, int RING>
__global__ void __launch_bounds__(kFewThreads, NT == 4 ? 1 : 2) w8_few_kernel(const moe_layer_w8_args_t a, int64_t tiles) {
  __shared__ int32_t s_part[2][kFewWarps][8 * NT][kFewRows + 1];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int steps = (a.k + kStep - 1) / kStep;
  const int mine = warp < steps ? (steps - warp + kFewWarps - 1) / kFewWarps : 0;  // this warp's steps of a tile
  const int8_t* x = a.x + g * a.x_stride;  // of the lane's first token; the others are 8 rows apart
  uint4 wv[RING][2][2], xv[RING][2][NT];
  // the next step to load: of tile `lt`, the warp's step number `ls`
  int64_t lt = mine ? blockIdx.x : tiles;
  int ls = 0;
  auto load = [&](uint4 (&wr)[2][2], uint4 (&xr)[2][NT]) {
    const int k0 = (warp + ls * kFewWarps) * kStep + 16 * t;
    const int64_t n0 = lt * kFewRows + g;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = k0 + 64 * j;
      const bool in = lt < tiles && k < a.k;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        wr[j][i] = make_uint4(0, 0, 0, 0);
        if (in && n0 + 8 * i < a.n) wr[j][i] = __ldcs(reinterpret_cast<const uint4*>(a.w + (n0 + 8 * i) * a.k + k));
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        xr[j][i] = make_uint4(0, 0, 0, 0);
        if (in && 8 * i + g < a.m) xr[j][i] = __ldg(reinterpret_cast<const uint4*>(x + 8 * i * a.x_stride + k));
      }
    }
    if (++ls >= mine) ls = 0, lt += gridDim.x;
  };
  if (mine) {
#pragma unroll
    for (int r = 0; r < RING; ++r) load(wv[r], xv[r]);
  }
  int buf = 0, done = 0;  // steps of the tile that is multiplied
  int64_t tile = blockIdx.x;
  int32_t d[NT][4] = {};
  // adds up a tile once its last step is done; false after the last tile
  auto finish = [&]() {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s_part[buf][warp][8 * i + 2 * t + (e & 1)][g + 8 * (e >> 1)] = d[i][e];
        d[i][e] = 0;
      }
    __syncthreads();  // (two buffers: the next tile's sums are written while these are read)
    for (int i = threadIdx.x; i < 8 * NT * kFewRows; i += kFewThreads) {
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
    for (int r = 0; r < RING; ++r) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const uint4 &lo = wv[r][j][0], &hi = wv[r][j][1], &xr = xv[r][j][i];
          mma_s8(d[i], lo.x, hi.x, lo.y, hi.y, xr.x, xr.y);
          mma_s8(d[i], lo.z, hi.z, lo.w, hi.w, xr.z, xr.w);
        }
      load(wv[r], xv[r]);
      if (++done == mine && !finish()) return;
    }
  }
}

template <int NT, int RING>
cudaError_t launch_few(const moe_layer_w8_args_t& a, int num_sms, cudaStream_t s) {
  moe_layer_w8_args_t arg = a;
  int64_t tiles = (static_cast<int64_t>(a.n) + kFewRows - 1) / kFewRows;
  void* args[] = {&arg, &tiles};
  const int64_t grid = tiles < 2 * num_sms ? tiles : 2 * num_sms;
  return launch_after((const void*)w8_few_kernel<NT, RING>, dim3(static_cast<unsigned>(grid)), dim3(kFewThreads), args, 0, s);
}

// The integer products take 8 tokens at a time and run at 158 TOPS; the other kernel needs 6 us for the smallest call.
// us, this one and the other: 16 x 2048 x 4096 4.9 / 7.7, 16 x 4096 x 4096 7.7 / 8.4, 16 x 6144 x 4096 11.6 / 11.0; 32 x
// 1024 x 1024 3.6 / 6.1, 32 x 2048 x 2048 5.4 / 7.1, 32 x 2048 x 4096 8.6 / 8.0; 8 x 130001 x 4096 84, 16 rows there 89.
bool few(int m, int n, int k) {
  const int64_t weights = static_cast<int64_t>(n) * k;
  return m <= 8 || (m <= 16 && weights <= 12 << 20) || (m <= 32 && weights <= 4 << 20);
}

}  // namespace

size_t w8_workspace(int m, int n, int k, int num_sms) { return few(m, n, k) ? 0 : w8_tc_workspace(m, n, k, num_sms); }

cudaError_t launch_w8(const moe_layer_w8_args_t& a, void* ws, int num_sms, cudaStream_t s) {
  if (!few(a.m, a.n, a.k)) return launch_w8_tc(a, ws, num_sms, s);
  if (a.m <= 8) return launch_few<1, 4>(a, num_sms, s);
  if (a.m <= 16) return launch_few<2, 3>(a, num_sms, s);
  return launch_few<4, 3>(a, num_sms, s);
}

}  // namespace moe_layer
