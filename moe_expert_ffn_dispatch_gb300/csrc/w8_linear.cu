// Products of INT8 codes with INT8 weights, exact in int32, with a scale a token
// and a scale a channel.
//
// Few tokens: weight rows are the M side of mma.sync m16n8k32, tokens its N side.
// A CTA takes 32 weight rows and up to 8 NT tokens; its warps share out k in steps
// of 128 and add up in shared memory.  A lane loads 16 bytes of a weight row (and
// of a token) at a time, 64 apart: the four words of a load are k-words of four
// products, in the same order for weights and tokens, which is all that the sum
// asks for.
#include "w8_linear.cuh"

namespace moe_layer {
namespace {

constexpr int kFewWarps = 8, kFewThreads = kFewWarps * 32;
constexpr int kFewRows = 32;   // weight rows of a CTA
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

template <int NT>
__global__ void __launch_bounds__(kFewThreads, 2) w8_few_kernel(const moe_layer_w8_args_t a) {
  __shared__ int32_t s_part[kFewWarps][8 * NT][kFewRows + 1];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kFewRows;
  const int m0 = blockIdx.y * 8 * NT;
  const int8_t *w[4], *x[NT];
  bool has_w[4], has_x[NT];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    has_w[i] = n0 + 8 * i + g < a.n;
    w[i] = a.w + (has_w[i] ? n0 + 8 * i + g : 0) * a.k;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    has_x[i] = m0 + 8 * i + g < a.m;
    x[i] = a.x + (has_x[i] ? m0 + 8 * i + g : 0) * a.x_stride;
  }
  int32_t d[2][NT][4] = {};
  const uint4 none = make_uint4(0, 0, 0, 0);
  for (int k0 = warp * kStep; k0 < a.k; k0 += kFewWarps * kStep) {
    uint4 wv[2][4], xv[2][NT];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = k0 + 64 * j + 16 * t;
      const bool in = k < a.k;
#pragma unroll
      for (int i = 0; i < 4; ++i) wv[j][i] = in && has_w[i] ? __ldcs(reinterpret_cast<const uint4*>(w[i] + k)) : none;
#pragma unroll
      for (int i = 0; i < NT; ++i) xv[j][i] = in && has_x[i] ? __ldg(reinterpret_cast<const uint4*>(x[i] + k)) : none;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          mma_s8(d[r][i], wv[j][2 * r].x, wv[j][2 * r + 1].x, wv[j][2 * r].y, wv[j][2 * r + 1].y, xv[j][i].x, xv[j][i].y);
          mma_s8(d[r][i], wv[j][2 * r].z, wv[j][2 * r + 1].z, wv[j][2 * r].w, wv[j][2 * r + 1].w, xv[j][i].z, xv[j][i].w);
        }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s_part[warp][8 * i + 2 * t + (e & 1)][16 * r + g + 8 * (e >> 1)] = d[r][i][e];
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * NT * kFewRows; i += kFewThreads) {
    const int tok = i / kFewRows, r = i % kFewRows;
    if (m0 + tok >= a.m || n0 + r >= a.n) continue;
    int32_t sum = 0;
#pragma unroll
    for (int q = 0; q < kFewWarps; ++q) sum += s_part[q][tok][r];
    store_y(a.y, static_cast<int64_t>(m0 + tok) * a.n + n0 + r,
            scaled(sum, scale_at(a.w_scale, n0 + r, a.scale_dtype), a.x_scale[m0 + tok]), a.out_dtype);
  }
}

template <int NT>
cudaError_t launch_few(const moe_layer_w8_args_t& a, cudaStream_t s) {
  moe_layer_w8_args_t arg = a;
  void* args[] = {&arg};
  const dim3 grid((a.n + kFewRows - 1) / kFewRows, (a.m + 8 * NT - 1) / (8 * NT));
  return launch_after((const void*)w8_few_kernel<NT>, grid, dim3(kFewThreads), args, 0, s);
}

}  // namespace

size_t w8_workspace(int m, int n, int k, int num_sms) { return m <= 8 ? 0 : w8_tc_workspace(m, n, k, num_sms); }

cudaError_t launch_w8(const moe_layer_w8_args_t& a, void* ws, int num_sms, cudaStream_t s) {
  if (a.m <= 8) return launch_few<1>(a, s);
  return launch_w8_tc(a, ws, num_sms, s);
}

}  // namespace moe_layer
