// Residual addition + RMS norm + per-token INT8 quant.
//
// Two reductions over the row (sum of squares, then the maximum of |z|) and
// one pass over memory: the row stays in registers as fp32 between them.  A
// CTA takes a row (a warp does, up to 1024 wide), and every load is issued
// before the first use, the weight's too, so that a row costs one trip to
// memory and two barriers.
// Bound by memory: 2 bytes read (4 with a residual) and 1 to 5 written an
// element.  4093 x 4096 with residual and y: 23.8 us, 6.3 TB/s of 6.8; 8 x 4096:
// 2.2 us, latency.  Rows that are not 16-byte aligned take about twice the
// instructions and four barriers: 4093 x 4097 48 us (element by element it was
// 84), 16000 x 1001 39, 16000 x 513 34 (54).  A weight in fp32 costs little up to
// 4096 wide (4093 x 4096 24.9 us for 23.9); beyond, its 32 values a thread do not fit
// the registers beside the row, and the spills show: 2000 x 8192 31 us for 24, 1000 x
// 16384 35 for 26, 2000 x 8191 57 for 47.
#include "norm_rows.cuh"

namespace moe_layer {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kRowWarps = 4;

// ROW_WARP: a warp takes a row by itself, kRowWarps rows a CTA
template <typename T, typename W, int C, bool VEC, bool ROW_WARP>
__global__ void __launch_bounds__(ROW_WARP ? kRowWarps * 32 : C * 128, ROW_WARP ? 6 : 8 / C)
    add_rmsnorm_quant_kernel(const moe_layer_norm_args_t a) {
  __shared__ float s_sum[kMaxWarps];
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
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
  T* res_out = a.residual ? static_cast<T*>(a.residual_out) + row * a.residual_out_stride : nullptr;
  T* y_out = a.y_out ? static_cast<T*>(a.y_out) + row * h : nullptr;
  int8_t* q = a.q + row * h;
  const W* w = static_cast<const W*>(a.weight);
  // rows that are not VEC: x, then y; the residual; the new residual, then the codes
  uint4 *buf_x = s_rows + (ROW_WARP ? warp * 3 * row_slots(C, 32) : 0), *buf_r = buf_x + row_slots(C, nt),
        *buf_o = buf_r + row_slots(C, nt);
  auto sync_row = [] {
    if constexpr (ROW_WARP) __syncwarp();
    else __syncthreads();
  };

  // every load of the row before the first use or store
  RowIn<T, C> xs, rs;
  Chunk8<T, true> xr[C], rr[C];
  Chunk8<W, VEC> wr[C];
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      xr[c].load(x, (c * nt + tid) * 8, h);
      if (res) rr[c].load(res, (c * nt + tid) * 8, h);
    }
  } else {
    xs.load(x, row, a.rows - 1 - row, a.x_stride, tid, nt, h);
    if (res) rs.load(res, row, a.rows - 1 - row, a.residual_stride, tid, nt, h);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) wr[c].load(w, (c * nt + tid) * 8, h);
  if constexpr (!VEC) {
    xs.stage(buf_x, tid, nt);
    if (res) rs.stage(buf_r, tid, nt);
    sync_row();
  }
  float v[C][8];
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int n = c * nt + tid;
    if constexpr (VEC) xr[c].take(v[c]);
    else take_row<T>(buf_x, n, xs.off, h, v[c]);
    if (res) {
      float r[8];
      if constexpr (VEC) rr[c].take(r);
      else take_row<T>(buf_r, n, rs.off, h, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = __fadd_rn(v[c][j], r[j]);
      if constexpr (!VEC) buf_o[n] = pack8<T>(v[c]);
      else if (n * 8 < h) *reinterpret_cast<uint4*>(res_out + n * 8) = pack8<T>(v[c]);
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
  } else if constexpr (!VEC) {
    __syncwarp();
  }
  if constexpr (!VEC) {  // x and the residual have been read, the new residual is there
    if (res) store_row(res_out, buf_o, tid, nt, h);
  }
  const float r = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(h)), a.eps));

  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int n = c * nt + tid, i = n * 8;
    float f[8];
    wr[c].take(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[c][j] = i + j < h ? __fmul_rn(__fmul_rn(v[c][j], r), f[j]) : 0.0f;
    if (y_out) {
      if constexpr (!VEC) buf_x[n] = pack8<T>(v[c]);
      else if (i < h) *reinterpret_cast<uint4*>(y_out + i) = pack8<T>(v[c]);
    }
    if (a.smooth) {
      Chunk8<float, VEC> sr;
      sr.load(a.smooth, i, h);
      sr.take(f);
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
  } else if constexpr (!VEC) {
    __syncwarp();
  }
  if constexpr (!VEC) {
    if (y_out) store_row(y_out, buf_x, tid, nt, h);
  }
  // a NaN or an infinity in the row is a NaN here (infinity times r = 0), and so in the scale
  float amax = __uint_as_float(top >= 0x7F800000u ? 0x7FC00000u : top);
  if (amax < kAmaxFloor) amax = kAmaxFloor;
  const float m = __fdiv_rn(127.0f, amax);

  uint2* codes = reinterpret_cast<uint2*>(buf_o);  // the new residual has left it
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int n = c * nt + tid;
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      o[j] = codes_of(__fmul_rn(v[c][4 * j], m), __fmul_rn(v[c][4 * j + 1], m), __fmul_rn(v[c][4 * j + 2], m),
                      __fmul_rn(v[c][4 * j + 3], m));
    if constexpr (!VEC) codes[n] = make_uint2(o[0], o[1]);
    else if (n * 8 < h) *reinterpret_cast<uint2*>(q + n * 8) = make_uint2(o[0], o[1]);
  }
  if constexpr (!VEC) {
    sync_row();
    store_codes(q, buf_o, tid, nt, h);
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
  size_t smem = 0;
  if (!vec) {
    smem = (ROW_WARP ? kRowWarps * row_slots(C, 32) : row_slots(C, nt)) * 3 * sizeof(uint4);
    static std::atomic<uint64_t> allowed{0};
    if (const cudaError_t e = allow_smem(k, kMaxSmem / 2, allowed); e != cudaSuccess) return e;
  }
  return launch_after(k, dim3(ROW_WARP ? (a.rows + kRowWarps - 1) / kRowWarps : a.rows), dim3(nt), args, smem, s);
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
