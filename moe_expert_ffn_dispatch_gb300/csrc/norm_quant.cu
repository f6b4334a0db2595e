// Residual addition + RMS norm + per-token INT8 quant.
//
// Two reductions over the row (sum of squares, then the maximum of |z|) and
// one pass over memory: the row stays in registers as fp32 between them.  A
// CTA takes a row (a warp does, up to 1024 wide), and every load is issued
// before the first use, the weight's too, so that a row costs one trip to
// memory and two barriers.
// Bound by memory: 2 bytes read (4 with a residual) and 1 to 5 written an
// element.  4093 x 4096 with residual and y: 23.8 us, 6.3 TB/s of 6.8; 8 x 4096:
// 2.2 us, latency.  Rows that are not 16-byte aligned go one element
// at a time, 1.4 to 2.9 TB/s (4093 x 4097: 84 us); 16-byte reads shifted into
// place between lanes were no faster (91 us).
#include "layer_ops.cuh"

namespace moe_layer {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kRowWarps = 4;

// A thread holds C chunks of 8 neighbouring elements; a warp's 32 chunks are
// 256 neighbours.  VEC: a chunk moves by 16-byte accesses (needs hidden % 8 ==
// 0 and aligned rows).  Otherwise the warp moves its 256 elements one by one,
// neighbours by neighbouring lanes, and hands them round in shared memory, so
// that every thread holds the same elements in either form and the sums, and
// with them every result, do not depend on alignment.
// Raw holds a chunk's bits between the load, which a kernel issues early, and take.
template <typename E, bool VEC>
struct Raw {
  uint32_t w[VEC ? sizeof(E) * 2 : 8];
  __device__ __forceinline__ void load(const E* p, int i, int h) {
    if constexpr (VEC) {
#pragma unroll
      for (int k = 0; k < static_cast<int>(sizeof(E) / 2); ++k) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (i < h) u = reinterpret_cast<const uint4*>(p + i)[k];
        w[4 * k] = u.x, w[4 * k + 1] = u.y, w[4 * k + 2] = u.z, w[4 * k + 3] = u.w;
      }
    } else {
      const int lane = threadIdx.x & 31, first = i - lane * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = first + j * 32 + lane < h ? __float_as_uint(to_f32(p[first + j * 32 + lane])) : 0u;
    }
  }
  __device__ __forceinline__ void take(float* buf, float (&v)[8]) const {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(E) == 2) {
          const float2 f = unpack2<E>(w[j]);
          v[2 * j] = f.x;
          v[2 * j + 1] = f.y;
        } else {
          v[2 * j] = __uint_as_float(w[2 * j]);
          v[2 * j + 1] = __uint_as_float(w[2 * j + 1]);
        }
      }
    } else {
      const int lane = threadIdx.x & 31;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) buf[(j * 32 + lane) + (j * 32 + lane) / 8] = __uint_as_float(w[j]);  // 9 words a chunk: no bank twice
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = buf[lane * 9 + j];
    }
  }
};

template <typename E, bool VEC>
__device__ __forceinline__ void store8(E* p, int i, int h, float* buf, const float (&v)[8]) {
  if constexpr (VEC) {
    if (i < h) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = pack2<E>(v[2 * j], v[2 * j + 1]);
      *reinterpret_cast<uint4*>(p + i) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  } else {
    const int lane = threadIdx.x & 31, first = i - lane * 8;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) buf[lane * 9 + j] = v[j];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (first + j * 32 + lane < h) p[first + j * 32 + lane] = from_f32<E>(buf[(j * 32 + lane) + (j * 32 + lane) / 8]);
  }
}

// ROW_WARP: a warp takes a row by itself, kRowWarps rows a CTA
template <typename T, typename W, int C, bool VEC, bool ROW_WARP>
__global__ void __launch_bounds__(ROW_WARP ? kRowWarps * 32 : 512, ROW_WARP ? 6 : 2) add_rmsnorm_quant_kernel(const moe_layer_norm_args_t a) {
  __shared__ float s_sum[kMaxWarps];
  __shared__ uint32_t s_max[kMaxWarps];
  __shared__ float s_buf[VEC ? 1 : (ROW_WARP ? kRowWarps : kMaxWarps) * 32 * 9];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int nt = ROW_WARP ? 32 : blockDim.x, tid = ROW_WARP ? lane : threadIdx.x;
  float* buf = s_buf + (VEC ? 0 : warp * 32 * 9);
  const int h = a.hidden;
  const int64_t row = ROW_WARP ? static_cast<int64_t>(blockIdx.x) * kRowWarps + warp : blockIdx.x;
  if (ROW_WARP && row >= a.rows) return;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
  T* res_out = a.residual ? static_cast<T*>(a.residual_out) + row * a.residual_out_stride : nullptr;
  T* y_out = a.y_out ? static_cast<T*>(a.y_out) + row * h : nullptr;
  const W* w = static_cast<const W*>(a.weight);

  // every load of the row before the first use or store
  Raw<T, VEC> xr[C], rr[C];
  Raw<W, VEC> wr[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    xr[c].load(x, (c * nt + tid) * 8, h);
    if (res) rr[c].load(res, (c * nt + tid) * 8, h);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) wr[c].load(w, (c * nt + tid) * 8, h);
  float v[C][8];
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (c * nt + tid) * 8;
    xr[c].take(buf, v[c]);
    if (res) {
      float r[8];
      rr[c].take(buf, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = __fadd_rn(v[c][j], r[j]);
      store8<T, VEC>(res_out, i, h, buf, v[c]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __fmaf_rn(v[c][j], v[c][j], sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if constexpr (!ROW_WARP) {
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    sum = lane < nw ? s_sum[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  const float r = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(h)), a.eps));

  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (c * nt + tid) * 8;
    float f[8];
    wr[c].take(buf, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[c][j] = i + j < h ? __fmul_rn(__fmul_rn(v[c][j], r), f[j]) : 0.0f;
    if (y_out) store8<T, VEC>(y_out, i, h, buf, v[c]);
    if (a.smooth) {
      Raw<float, VEC> sr;
      sr.load(a.smooth, i, h);
      sr.take(buf, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = i + j < h ? __fmul_rn(v[c][j], f[j]) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, abs_bits(v[c][j]));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if constexpr (!ROW_WARP) {
    if (lane == 0) s_max[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, lane < nw ? s_max[lane] : 0u);
  }
  // a NaN or an infinity in the row is a NaN here (infinity times r = 0), and so in the scale
  float amax = __uint_as_float(top >= 0x7F800000u ? 0x7FC00000u : top);
  if (amax < kAmaxFloor) amax = kAmaxFloor;
  const float m = __fdiv_rn(127.0f, amax);

  int8_t* q = a.q + row * h;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (c * nt + tid) * 8;
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      o[j] = codes_of(__fmul_rn(v[c][4 * j], m), __fmul_rn(v[c][4 * j + 1], m), __fmul_rn(v[c][4 * j + 2], m),
                      __fmul_rn(v[c][4 * j + 3], m));
    if constexpr (VEC) {
      if (i < h) *reinterpret_cast<uint2*>(q + i) = make_uint2(o[0], o[1]);
    } else {
      uint8_t* b = reinterpret_cast<uint8_t*>(buf);
      __syncwarp();
      *reinterpret_cast<uint2*>(b + lane * 8) = make_uint2(o[0], o[1]);
      __syncwarp();
      const int first = i - lane * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (first + j * 32 + lane < h) q[first + j * 32 + lane] = static_cast<int8_t>(b[j * 32 + lane]);
    }
  }
  if (tid == 0) a.q_scale[row] = __fdiv_rn(1.0f, m);
}

template <typename T, typename W, int C, bool ROW_WARP>
cudaError_t launch_shape(const moe_layer_norm_args_t& a, bool vec, cudaStream_t s) {
  const int chunks = (a.hidden + 7) / 8;
  const int nt = ROW_WARP ? kRowWarps * 32 : ((chunks + C - 1) / C + 31) / 32 * 32;
  const void* k = vec ? (const void*)add_rmsnorm_quant_kernel<T, W, C, true, ROW_WARP>
                      : (const void*)add_rmsnorm_quant_kernel<T, W, C, false, ROW_WARP>;
  moe_layer_norm_args_t arg = a;
  void* args[] = {&arg};
  return launch_after(k, dim3(ROW_WARP ? (a.rows + kRowWarps - 1) / kRowWarps : a.rows), dim3(nt), args, 0, s);
}

template <typename T, typename W>
cudaError_t launch_typed(const moe_layer_norm_args_t& a, cudaStream_t s) {
  auto at = [](const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  const bool vec = a.hidden % 8 == 0 && at(a.x, 16) && a.x_stride % 8 == 0 && at(a.weight, 16) && at(a.q, 8) &&
                   (!a.residual || (at(a.residual, 16) && at(a.residual_out, 16) && a.residual_stride % 8 == 0 &&
                                    a.residual_out_stride % 8 == 0)) &&
                   (!a.y_out || at(a.y_out, 16)) && (!a.smooth || at(a.smooth, 16));
  // The form goes by hidden alone, so that a row's results do not depend on
  // the rows beside it.
  if (a.hidden <= 512) return launch_shape<T, W, 2, true>(a, vec, s);
  if (a.hidden <= 1024) return launch_shape<T, W, 4, true>(a, vec, s);
  if (a.hidden <= 4096) return launch_shape<T, W, 2, false>(a, vec, s);
  return launch_shape<T, W, 4, false>(a, vec, s);
}

}  // namespace

cudaError_t launch_norm(const moe_layer_norm_args_t& a, int, cudaStream_t s) {
  if (a.dtype == MOE_LAYER_BF16)
    return a.weight_dtype == MOE_LAYER_FP32 ? launch_typed<__nv_bfloat16, float>(a, s)
                                            : launch_typed<__nv_bfloat16, __nv_bfloat16>(a, s);
  return a.weight_dtype == MOE_LAYER_FP32 ? launch_typed<__half, float>(a, s) : launch_typed<__half, __half>(a, s);
}

}  // namespace moe_layer
