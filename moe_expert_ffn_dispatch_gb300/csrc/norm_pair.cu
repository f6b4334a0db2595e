// RMS norm of a block's output, gate and scale, residual addition, RMS norm and
// INT8 quant of the next block's input.
//
// Three reductions over the row (sum of squares of the block's output, of the new
// residual, then the maximum of |z|) and one pass over memory, as norm_quant.cu
// has it: the row stays in registers as fp32 between them, a CTA a row (a warp up
// to 1024 wide), every load of a row's own data issued before the first use, and the
// weights' a barrier ahead of theirs.
// Bound by memory: 4 bytes read (6 with a gate a token) and 2 to 5 written an
// element.  4093 x 4096 with a gate a token, y and no codes: 27.3 us, 6.1 TB/s of 6.8;
// 8 x 4096: 2.5 us, latency.  Five CTAs of 256 threads an SM, for which the compiler has 48
// registers a thread (three CTAs took 31.6 us); two elements an instruction (28.6 without).
// Past 4096 wide it spills: 2000 x 8192 32 us, 1000 x 16384 31.  Rows that are not 16-byte
// aligned go through shared memory and take twice the time (4093 x 4097 64 us, 2000 x 8191 53;
// issue 69 %, 61 instructions an element).
#include "norm_rows.cuh"

namespace moe_layer {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kRowWarps = 4;

template <bool ROW_WARP>
__device__ __forceinline__ float row_sum(float v, float* s_part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (!ROW_WARP) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0) s_part[warp] = v;
    __syncthreads();
    // every thread adds up the warps' sums, in one order
    v = s_part[0];
#pragma unroll
    for (int w = 1; w < kMaxWarps; ++w)
      if (w < nw) v = __fadd_rn(v, s_part[w]);
  } else {
    __syncwarp();
  }
  return v;
}

__device__ __forceinline__ float sum_of(uint64_t pair) {
  const float2 f = of_pair(pair);
  return __fadd_rn(f.x, f.y);
}
template <typename T>
__device__ __forceinline__ uint4 pack_pairs(const uint64_t (&v)[4]) {
  const float2 a = of_pair(v[0]), b = of_pair(v[1]), c = of_pair(v[2]), d = of_pair(v[3]);
  return make_uint4(pack2<T>(a.x, a.y), pack2<T>(b.x, b.y), pack2<T>(c.x, c.y), pack2<T>(d.x, d.y));
}

// ROW_WARP: a warp takes a row by itself, kRowWarps rows a CTA
template <typename T, typename W, int C, bool VEC, bool ROW_WARP>
__global__ void __launch_bounds__(ROW_WARP ? kRowWarps * 32 : C * 128, ROW_WARP ? 5 : VEC ? 10 / C : 8 / C)
    norm_pair_kernel(const moe_layer_norm_pair_args_t a) {
  __shared__ float s_sum[kMaxWarps], s_sum2[kMaxWarps];
  __shared__ uint32_t s_max[kMaxWarps];
  extern __shared__ __align__(16) uint4 s_rows[];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int nt = ROW_WARP ? 32 : blockDim.x, tid = ROW_WARP ? lane : threadIdx.x;
  const int h = a.hidden;
  const int64_t row = ROW_WARP ? static_cast<int64_t>(blockIdx.x) * kRowWarps + warp : blockIdx.x;
  if (ROW_WARP && row >= a.rows) return;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* res = static_cast<const T*>(a.residual) + row * a.residual_stride;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + row * a.gate_stride : nullptr;
  const bool own_gate = a.gate && a.gate_stride != 0;  // a row's own, rather than one that all rows share
  T* res_out = static_cast<T*>(a.residual_out) + row * a.residual_out_stride;
  T* y_out = a.y_out ? static_cast<T*>(a.y_out) + row * h : nullptr;
  const W *post = static_cast<const W*>(a.post_weight), *w = static_cast<const W*>(a.weight);
  // rows that are not VEC: x, then the new residual; the residual, then y; the gate, then the codes
  uint4 *buf_x = s_rows + (ROW_WARP ? warp * 3 * row_slots(C, 32) : 0), *buf_r = buf_x + row_slots(C, nt),
        *buf_g = buf_r + row_slots(C, nt);
  auto root = [&](float sum) { return __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(h)), a.eps)); };
  auto sync_row = [] {
    if constexpr (ROW_WARP) __syncwarp();
    else __syncthreads();
  };

  RowIn<T, C> xs, rs, gs;
  Chunk8<T, true> xr[C], rr[C], gr[C];
  // weights are loaded ahead of the barrier before their use where there are registers for it
  constexpr bool kAhead = ROW_WARP || (VEC && C == 2);
  Chunk8<W, VEC> wr[C];
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (c * nt + tid) * 8;
      xr[c].load(x, i, h);
      rr[c].load(res, i, h);
      if (gate) gr[c].load(gate, i, h);
    }
  } else {
    xs.load(x, row, a.rows - 1 - row, a.x_stride, tid, nt, h);
    rs.load(res, row, a.rows - 1 - row, a.residual_stride, tid, nt, h);
    if (own_gate) gs.load(gate, row, a.rows - 1 - row, a.gate_stride, tid, nt, h);
    xs.stage(buf_x, tid, nt);
    rs.stage(buf_r, tid, nt);
    if (own_gate) gs.stage(buf_g, tid, nt);
    sync_row();
  }

  if constexpr (kAhead) {
#pragma unroll
    for (int c = 0; c < C; ++c) wr[c].load(post, (c * nt + tid) * 8, h);
  }
  uint64_t v[C][4];  // pairs of neighbours; zeros past the row's end stay zeros, as weights and residual are zeros there
  uint64_t sums = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float f[8];
    if constexpr (VEC) xr[c].take(f);
    else take_row<T>(buf_x, c * nt + tid, xs.off, h, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[c][j] = pair_of(f[2 * j], f[2 * j + 1]);
      sums = fma_pair(v[c][j], v[c][j], sums);
    }
  }
  const float r1 = root(row_sum<ROW_WARP>(sum_of(sums), s_sum));

  // the new residual, and its sum of squares
  const uint64_t r1s = pair_of(r1, r1), scales = pair_of(a.branch_scale, a.branch_scale);
  sums = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int n = c * nt + tid, i = n * 8;
    float f[8];
    if constexpr (!kAhead) wr[c].load(post, i, h);
    wr[c].take(f);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[c][j] = mul_pair(mul_pair(v[c][j], r1s), pair_of(f[2 * j], f[2 * j + 1]));
    if (gate) {
      if constexpr (VEC) {
        gr[c].take(f);
      } else if (own_gate) {
        take_row<T>(buf_g, n, gs.off, h, f);
      } else {
        Chunk8<T, false> shared;
        shared.load(gate, i, h);
        shared.take(f);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[c][j] = mul_pair(v[c][j], pair_of(f[2 * j], f[2 * j + 1]));
    }
    if constexpr (VEC) rr[c].take(f);
    else take_row<T>(buf_r, n, rs.off, h, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[c][j] = fma_pair(scales, v[c][j], pair_of(f[2 * j], f[2 * j + 1]));
      sums = fma_pair(v[c][j], v[c][j], sums);
    }
    if constexpr (VEC) {
      if (i < h) *reinterpret_cast<uint4*>(res_out + i) = pack_pairs<T>(v[c]);
    } else {
      buf_x[n] = pack_pairs<T>(v[c]);  // every thread has taken x, at the sum's barrier
    }
  }
  if constexpr (kAhead) {
#pragma unroll
    for (int c = 0; c < C; ++c) wr[c].load(w, (c * nt + tid) * 8, h);
  }
  const float sum = row_sum<ROW_WARP>(sum_of(sums), s_sum2);
  if constexpr (!VEC) store_row(res_out, buf_x, tid, nt, h);
  const float r2 = root(sum);

  uint32_t top = 0;
  const uint64_t r2s = pair_of(r2, r2);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int n = c * nt + tid, i = n * 8;
    float f[8];
    if constexpr (!kAhead) wr[c].load(w, i, h);
    wr[c].take(f);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[c][j] = mul_pair(mul_pair(v[c][j], r2s), pair_of(f[2 * j], f[2 * j + 1]));
    if (y_out) {
      if constexpr (!VEC) buf_r[n] = pack_pairs<T>(v[c]);  // the residual has left it
      else if (i < h) *reinterpret_cast<uint4*>(y_out + i) = pack_pairs<T>(v[c]);
    }
    if (a.q) {
      if (a.smooth) {
        Chunk8<float, VEC> sr;
        sr.load(a.smooth, i, h);
        sr.take(f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[c][j] = mul_pair(v[c][j], pair_of(f[2 * j], f[2 * j + 1]));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 z = of_pair(v[c][j]);
        top = max(top, max(abs_bits(z.x), abs_bits(z.y)));
      }
    }
  }
  if (a.q) {  // the maximum of the row
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (!ROW_WARP) {
      if (lane == 0) s_max[warp] = top;
      __syncthreads();
      for (int w = 0; w < nw; ++w) top = max(top, s_max[w]);
    } else if constexpr (!VEC) {
      __syncwarp();
    }
  } else if constexpr (!VEC) {
    sync_row();
  }
  if constexpr (!VEC) {
    if (y_out) store_row(y_out, buf_r, tid, nt, h);
  }
  if (!a.q) return;
  // a NaN or an infinity in the row is a NaN here (infinity times r = 0), and so in the scale
  float amax = __uint_as_float(top >= 0x7F800000u ? 0x7FC00000u : top);
  if (amax < kAmaxFloor) amax = kAmaxFloor;
  const float m = __fdiv_rn(127.0f, amax);
  const uint64_t ms = pair_of(m, m);
  int8_t* q = a.q + row * h;
  uint2* codes = reinterpret_cast<uint2*>(buf_g);  // the gate has left it
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int n = c * nt + tid;
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 lo = of_pair(mul_pair(v[c][2 * j], ms)), hi = of_pair(mul_pair(v[c][2 * j + 1], ms));
      o[j] = codes_of(lo.x, lo.y, hi.x, hi.y);
    }
    if constexpr (!VEC) codes[n] = make_uint2(o[0], o[1]);
    else if (n * 8 < h) *reinterpret_cast<uint2*>(q + n * 8) = make_uint2(o[0], o[1]);
  }
  if constexpr (!VEC) {
    sync_row();
    store_codes(q, buf_g, tid, nt, h);
  }
  if (tid == 0) a.q_scale[row] = __fdiv_rn(1.0f, m);
}

template <typename T, typename W, int C, bool ROW_WARP>
cudaError_t launch_shape(const moe_layer_norm_pair_args_t& a, bool vec, cudaStream_t s) {
  const int chunks = (a.hidden + 7) / 8;
  const int nt = ROW_WARP ? kRowWarps * 32 : ((chunks + C - 1) / C + 31) / 32 * 32;
  const void* k = vec ? (const void*)norm_pair_kernel<T, W, C, true, ROW_WARP>
                      : (const void*)norm_pair_kernel<T, W, C, false, ROW_WARP>;
  moe_layer_norm_pair_args_t arg = a;
  void* args[] = {&arg};
  size_t smem = 0;
  if (!vec) {
    smem = (ROW_WARP ? kRowWarps * row_slots(C, 32) : row_slots(C, nt)) * 3 * sizeof(uint4);
    static std::atomic<uint64_t> allowed{0};
    if (const cudaError_t e = allow_smem(k, kMaxSmem / 2, allowed); e != cudaSuccess) return e;
  }
  return launch_after(k, dim3(ROW_WARP ? (a.rows + kRowWarps - 1) / kRowWarps : a.rows), dim3(nt), args, smem, s);
}

template <typename T, typename W>
cudaError_t launch_typed(const moe_layer_norm_pair_args_t& a, cudaStream_t s) {
  auto at = [](const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  const bool vec = a.hidden % 8 == 0 && at(a.x, 16) && a.x_stride % 8 == 0 && at(a.residual, 16) &&
                   a.residual_stride % 8 == 0 && at(a.residual_out, 16) && a.residual_out_stride % 8 == 0 &&
                   at(a.gate, 16) && a.gate_stride % 8 == 0 && at(a.post_weight, 16) && at(a.weight, 16) && at(a.q, 8) &&
                   at(a.y_out, 16) && at(a.smooth, 16);
  // The form goes by hidden alone, so that a row's results do not depend on
  // the rows beside it.
  if (a.hidden <= 512) return launch_shape<T, W, 2, true>(a, vec, s);
  if (a.hidden <= 1024) return launch_shape<T, W, 4, true>(a, vec, s);
  if (a.hidden <= 4096) return launch_shape<T, W, 2, false>(a, vec, s);
  return launch_shape<T, W, 4, false>(a, vec, s);
}

}  // namespace

cudaError_t launch_norm_pair(const moe_layer_norm_pair_args_t& a, cudaStream_t s) {
  if (a.dtype == MOE_LAYER_BF16)
    return a.weight_dtype == MOE_LAYER_FP32 ? launch_typed<__nv_bfloat16, float>(a, s)
                                            : launch_typed<__nv_bfloat16, __nv_bfloat16>(a, s);
  return a.weight_dtype == MOE_LAYER_FP32 ? launch_typed<__half, float>(a, s) : launch_typed<__half, __half>(a, s);
}

}  // namespace moe_layer
