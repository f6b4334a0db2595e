// Residual addition + RMS norm + per-token INT8 quant, one CTA a row.
//
// Two reductions over the row (sum of squares, then the maximum of |z|) and
// one pass over memory: the row stays in registers as fp32 between them.
// Bound by memory: 2 bytes read (4 with a residual) and 1 to 5 written an element.
#include "layer_ops.cuh"

namespace moe_layer {
namespace {

constexpr int kMaxWarps = 32;

// C chunks of 8 elements a thread.  VEC: a chunk is 8 neighbours, moved by
// 16-byte accesses (needs hidden % 8 == 0, aligned rows); otherwise the 8
// elements of a chunk lie a block apart and move one by one, for any hidden
// and alignment.
template <typename T, typename W, int C, bool VEC>
__global__ void __launch_bounds__(1024) add_rmsnorm_quant_kernel(const moe_layer_norm_args_t a) {
  __shared__ float s_sum[kMaxWarps];
  __shared__ uint32_t s_max[kMaxWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const int h = a.hidden;
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
  T* res_out = a.residual ? static_cast<T*>(a.residual_out) + row * a.residual_out_stride : nullptr;
  T* y_out = a.y_out ? static_cast<T*>(a.y_out) + row * h : nullptr;
  const W* w = static_cast<const W*>(a.weight);

  float v[C][8];
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (VEC) {
      const int i = (c * nt + tid) * 8;
      if (i < h) {
        const uint4 u = *reinterpret_cast<const uint4*>(x + i);
        const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = unpack2<T>(uw[j]);
          v[c][2 * j] = f.x;
          v[c][2 * j + 1] = f.y;
        }
        if (res) {
          const uint4 r = *reinterpret_cast<const uint4*>(res + i);
          const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2<T>(rw[j]);
            v[c][2 * j] = __fadd_rn(v[c][2 * j], f.x);
            v[c][2 * j + 1] = __fadd_rn(v[c][2 * j + 1], f.y);
            o[j] = pack2<T>(v[c][2 * j], v[c][2 * j + 1]);
          }
          *reinterpret_cast<uint4*>(res_out + i) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = 0.0f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = (c * 8 + j) * nt + tid;
        float f = 0.0f;
        if (i < h) {
          f = to_f32(x[i]);
          if (res) {
            f = __fadd_rn(f, to_f32(res[i]));
            res_out[i] = from_f32<T>(f);
          }
        }
        v[c][j] = f;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __fmaf_rn(v[c][j], v[c][j], sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = lane < nw ? s_sum[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float r = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(h)), a.eps));

  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (VEC) {
      const int i = (c * nt + tid) * 8;
      if (i < h) {
        float wv[8];
        if constexpr (sizeof(W) == 2) {
          const uint4 u = *reinterpret_cast<const uint4*>(w + i);
          const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2<W>(uw[j]);
            wv[2 * j] = f.x;
            wv[2 * j + 1] = f.y;
          }
        } else {
          const float4 p0 = *reinterpret_cast<const float4*>(w + i), p1 = *reinterpret_cast<const float4*>(w + i + 4);
          wv[0] = p0.x, wv[1] = p0.y, wv[2] = p0.z, wv[3] = p0.w;
          wv[4] = p1.x, wv[5] = p1.y, wv[6] = p1.z, wv[7] = p1.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = __fmul_rn(__fmul_rn(v[c][j], r), wv[j]);
        if (y_out) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = pack2<T>(v[c][2 * j], v[c][2 * j + 1]);
          *reinterpret_cast<uint4*>(y_out + i) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (a.smooth) {
          const float4 p0 = *reinterpret_cast<const float4*>(a.smooth + i),
                       p1 = *reinterpret_cast<const float4*>(a.smooth + i + 4);
          const float sv[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) v[c][j] = __fmul_rn(v[c][j], sv[j]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = (c * 8 + j) * nt + tid;
        if (i < h) {
          v[c][j] = __fmul_rn(__fmul_rn(v[c][j], r), to_f32(w[i]));
          if (y_out) y_out[i] = from_f32<T>(v[c][j]);
          if (a.smooth) v[c][j] = __fmul_rn(v[c][j], a.smooth[i]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, abs_bits(v[c][j]));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, lane < nw ? s_max[lane] : 0u);
  // a NaN or an infinity in the row is a NaN here (infinity times r = 0), and so in the scale
  float amax = __uint_as_float(top >= 0x7F800000u ? 0x7FC00000u : top);
  if (amax < kAmaxFloor) amax = kAmaxFloor;
  const float m = __fdiv_rn(127.0f, amax);

  int8_t* q = a.q + row * h;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (VEC) {
      const int i = (c * nt + tid) * 8;
      if (i < h) {
        uint32_t o[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j >> 2] |= code_of(__fmul_rn(v[c][j], m)) << ((j & 3) * 8);
        *reinterpret_cast<uint2*>(q + i) = make_uint2(o[0], o[1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = (c * 8 + j) * nt + tid;
        if (i < h) q[i] = static_cast<int8_t>(code_of(__fmul_rn(v[c][j], m)));
      }
    }
  }
  if (tid == 0) a.q_scale[row] = __fdiv_rn(1.0f, m);
}

template <typename T, typename W>
cudaError_t launch_typed(const moe_layer_norm_args_t& a, cudaStream_t s) {
  auto at = [](const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  const bool vec = a.hidden % 8 == 0 && at(a.x, 16) && a.x_stride % 8 == 0 && at(a.weight, 16) && at(a.q, 8) &&
                   (!a.residual || (at(a.residual, 16) && at(a.residual_out, 16) && a.residual_stride % 8 == 0 &&
                                    a.residual_out_stride % 8 == 0)) &&
                   (!a.y_out || at(a.y_out, 16)) && (!a.smooth || at(a.smooth, 16));
  const int chunks = (a.hidden + 7) / 8;
  const int per = chunks <= 512 ? 1 : 2;
  const int nt = ((chunks + per - 1) / per + 31) / 32 * 32;
  const void* k = per == 1 ? (vec ? (const void*)add_rmsnorm_quant_kernel<T, W, 1, true>
                                  : (const void*)add_rmsnorm_quant_kernel<T, W, 1, false>)
                           : (vec ? (const void*)add_rmsnorm_quant_kernel<T, W, 2, true>
                                  : (const void*)add_rmsnorm_quant_kernel<T, W, 2, false>);
  moe_layer_norm_args_t arg = a;
  void* args[] = {&arg};
  return launch_after(k, dim3(a.rows), dim3(nt), args, 0, s);
}

}  // namespace

cudaError_t launch_norm(const moe_layer_norm_args_t& a, int, cudaStream_t s) {
  if (a.dtype == MOE_LAYER_BF16)
    return a.weight_dtype == MOE_LAYER_FP32 ? launch_typed<__nv_bfloat16, float>(a, s)
                                            : launch_typed<__nv_bfloat16, __nv_bfloat16>(a, s);
  return a.weight_dtype == MOE_LAYER_FP32 ? launch_typed<__half, float>(a, s) : launch_typed<__half, __half>(a, s);
}

}  // namespace moe_layer
