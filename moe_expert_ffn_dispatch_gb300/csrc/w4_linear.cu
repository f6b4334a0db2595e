// Products of a few rows of x with 4-bit weights and group scales.
//
// y^T = W x^T as mma.sync m16n8k16: 16 weight rows are the M side, 8 rows of
// x the N side, so that one row of x costs what eight do and the weights pass
// through registers once.  Codes become exact 16-bit floats (a code set into
// the mantissa of 1024 or 128, minus that and the zero point), products are
// exact, each group's sum is one fp32 accumulator chain and enters the row's
// sum through an fp32 fma with the group's scale.
//
// Bound by the weights' bytes.  A CTA has 16 warps in WR groups of rows x
// (16 / WR) parts of K; a warp streams its own 16-row tiles through a ring of
// 128-K steps by asynchronous copies, which needs no barrier, and the parts of K
// are summed in shared memory, in a fixed order.  x lies in shared memory,
// its elements in the order in which the codes leave a 32-bit word.
#include <type_traits>

#include "layer_ops.cuh"

namespace moe_layer {
namespace {

constexpr int kWarps = 16;
constexpr int kStepK = 128;                    // k of one ring stage
constexpr int kRowPitch = kStepK / 2 + 16;     // bytes of a weight row in a stage, padded against bank conflicts
constexpr int kStageBytes = 16 * kRowPitch;
constexpr int kXBudget = 128 * 1024;           // bytes of x in shared memory
// what fits beside 128 KB of x: ring stages of a warp, and halves of the buffer of partial sums
template <int NT>
constexpr int kStagesOf = NT == 1 ? 4 : 3;
template <int NT>
constexpr int kRedBufs = NT <= 2 ? 2 : 1;

struct W4Params {
  moe_layer_w4_args_t a;
  int kc;         // k of one piece of x that fits shared memory (multiple of 128)
  int pieces;     // pieces of kc that cover k
  int wr;         // row groups of a CTA: 1, 2, 4, 8 or 16
  int tiles;      // row tiles of 16 * wr rows
  int xpitch;     // bytes of a row of x in shared memory
  int ngroups;    // k / group
};

__device__ __forceinline__ float scale_at(const void* p, int64_t i, int dt) {
  if (dt == MOE_LAYER_FP32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t b = __ldg(static_cast<const uint16_t*>(p) + i);
  return dt == MOE_LAYER_BF16 ? __uint_as_float(static_cast<uint32_t>(b) << 16) : __half2float(__ushort_as_half(b));
}

// the 8 codes of a word as 4 pairs (0,4) (1,5) (2,6) (3,7), minus the zero
// point; zp: 128 + zero (bf16) or 1024 + zero (fp16) in both halves
template <typename T>
__device__ __forceinline__ void expand8(uint32_t w, uint32_t zp, uint32_t (&o)[4]) {
  constexpr uint32_t base = std::is_same_v<T, __half> ? 0x64006400u : 0x43004300u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = ((w >> (4 * i)) & 0x000F000Fu) | base;
    if constexpr (std::is_same_v<T, __half>) {
      const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&zp));
      o[i] = *reinterpret_cast<const uint32_t*>(&r);
    } else {
      const __nv_bfloat162 r =
          __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), *reinterpret_cast<const __nv_bfloat162*>(&zp));
      o[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}

template <typename T>
__device__ __forceinline__ uint32_t zero_word(uint32_t z) {
  if constexpr (std::is_same_v<T, __half>) return (0x6400u | z) * 0x10001u;
  return (0x4300u | z) * 0x10001u;
}

// 8 neighbouring elements of x as pairs (0,4) (1,5) (2,6) (3,7)
__device__ __forceinline__ uint4 pair04(uint4 v) {
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                    __byte_perm(v.y, v.w, 0x7632));
}

// NT: tiles of 8 rows of x.  GPS: groups of a 128-k step (1, 2 or 4)
template <typename T, int NT, int GPS>
__global__ void __launch_bounds__(kWarps * 32, 1) w4_linear_kernel(const W4Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kStages = kStagesOf<NT>;
  const moe_layer_w4_args_t& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int wr = p.wr, wk = kWarps / wr;
  const int row_group = warp / wk, kpart = warp - row_group * wk;
  const int m0 = blockIdx.y * (8 * NT);
  const int mrows = min(a.m - m0, 8 * NT);
  // x | rings | partial sums
  uint8_t* xs = smem;
  uint8_t* ring = smem + 8 * NT * p.xpitch + warp * (kStages * kStageBytes);
  float* red = reinterpret_cast<float*>(smem + 8 * NT * p.xpitch + kWarps * kStages * kStageBytes);
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const uint32_t xs_u = static_cast<uint32_t>(__cvta_generic_to_shared(xs));

  const int my_tiles = blockIdx.x < p.tiles ? (p.tiles - 1 - blockIdx.x) / gridDim.x + 1 : 0;
  const int steps_pp = p.kc / kStepK;                       // steps of a piece, all warps
  const int64_t row_bytes = a.k / 2;

  // position of the copies: tile, piece, step of this warp, ahead of the products
  int c_tile = blockIdx.x, c_piece = 0, c_step = kpart, c_slot = 0;
  const uint8_t* wbase = a.w;
  auto issue = [&]() {
    if (c_tile < p.tiles) {
      const int r0 = (c_tile * wr + row_group) * 16;
      // 16 rows x 64 bytes: lane i copies a quarter of rows i / 4 and i / 4 + 8
      const int kb = (c_piece * p.kc + c_step * kStepK) / 2 + t * 16;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = g + hh * 8;
        const int n = min(r0 + r, a.n - 1);
        const bool ok = kb < row_bytes;
        cp_async16(ring_u + c_slot * kStageBytes + r * kRowPitch + t * 16, wbase + n * row_bytes + (ok ? kb : 0), ok);
      }
      c_step += wk;
      if (c_step >= steps_pp || c_piece * p.kc + c_step * kStepK >= a.k) {
        c_step = kpart;
        if (++c_piece == p.pieces || c_piece * p.kc + c_step * kStepK >= a.k) {
          c_piece = 0;
          c_tile += gridDim.x;
        }
      }
    }
    c_slot = c_slot + 1 == kStages ? 0 : c_slot + 1;
    cp_async_commit();
  };
  // a warp whose part of K is empty issues nothing
  const bool any = kpart * kStepK < min(p.kc, a.k);
  if (!any) c_tile = p.tiles;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue();

  auto load_x = [&](int piece) {
    const int k0 = piece * p.kc;
    const int n8 = p.kc / 8;
    for (int i = tid; i < 8 * NT * n8; i += kWarps * 32) {
      const int m = i / n8, k8 = (i - m * n8) * 8;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (m < mrows && k0 + k8 < a.k) {
        const int64_t at = (m0 + m) * a.x_stride + k0 + k8;
        if (a.x_dtype == MOE_LAYER_INT8) {
          const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const int8_t*>(a.x) + at);
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t b = (j < 2 ? q.x : q.y) >> ((j & 1) * 16);
            o[j] = pack2<T>(static_cast<float>(static_cast<int8_t>(b & 0xFF)),
                            static_cast<float>(static_cast<int8_t>((b >> 8) & 0xFF)));
          }
          v = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + at);
        }
        v = pair04(v);
      }
      *reinterpret_cast<uint4*>(xs + m * p.xpitch + k8 * 2) = v;
    }
  };

  int slot = 0, buf = 0;
  for (int it = 0; it < my_tiles; ++it) {
    const int tile = blockIdx.x + it * gridDim.x;
    const int r0 = (tile * wr + row_group) * 16;
    const int64_t na = min(r0 + g, a.n - 1), nb = min(r0 + g + 8, a.n - 1);
    float acc[NT][4] = {};
    for (int piece = 0; piece < p.pieces; ++piece) {
      if (it == 0 || p.pieces > 1) {
        if (it > 0 || piece > 0) __syncthreads();  // the last piece is no longer read
        load_x(piece);
        __syncthreads();
      }
      const int k0 = piece * p.kc;
      for (int step = kpart; step < steps_pp && k0 + step * kStepK < a.k; step += wk) {
        // scales and zeros of this step's groups, asked for before the wait
        const int kk = k0 + step * kStepK;
        float sa[GPS], sb[GPS];
        uint32_t za[GPS], zb[GPS];
#pragma unroll
        for (int i = 0; i < GPS; ++i) {
          const int gi = min(GPS == 1 ? kk / a.group : kk / (kStepK / GPS) + i, p.ngroups - 1);
          sa[i] = scale_at(a.w_scale, na * p.ngroups + gi, a.scale_dtype);
          sb[i] = scale_at(a.w_scale, nb * p.ngroups + gi, a.scale_dtype);
          za[i] = zero_word<T>(a.w_zero ? __ldg(a.w_zero + na * p.ngroups + gi) & 15u : 8u);
          zb[i] = zero_word<T>(a.w_zero ? __ldg(a.w_zero + nb * p.ngroups + gi) & 15u : 8u);
        }
        cp_async_wait<kStages - 2>();
        __syncwarp();
        const uint32_t wa = ring_u + slot * kStageBytes + g * kRowPitch + t * 4;
        const uint32_t xa = xs_u + g * p.xpitch + (step * kStepK + t * 8) * 2;
        float part[NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          constexpr int jpg = 4 / GPS;  // words of a lane in a group
          const int gi = j / jpg;
          if (j % jpg == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n) part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0.0f;
          }
          uint32_t ea[4], eb[4];
          expand8<T>(lds32(wa + j * 16), za[gi], ea);
          expand8<T>(lds32(wa + 8 * kRowPitch + j * 16), zb[gi], eb);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 xv = lds128(xa + n * 8 * p.xpitch + j * 64);
            mma16816<T>(part[n], ea[0], eb[0], ea[1], eb[1], xv.x, xv.y);
            mma16816<T>(part[n], ea[2], eb[2], ea[3], eb[3], xv.z, xv.w);
          }
          if (j % jpg == jpg - 1) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              acc[n][0] = __fmaf_rn(sa[gi], part[n][0], acc[n][0]);
              acc[n][1] = __fmaf_rn(sa[gi], part[n][1], acc[n][1]);
              acc[n][2] = __fmaf_rn(sb[gi], part[n][2], acc[n][2]);
              acc[n][3] = __fmaf_rn(sb[gi], part[n][3], acc[n][3]);
            }
          }
        }
        __syncwarp();  // the stage is read before it is filled again
        issue();
        slot = slot + 1 == kStages ? 0 : slot + 1;
      }
    }
    // parts of K: red[buf][warp][x row][16 weight rows]
    float* mine = red + (buf * kWarps + warp) * (NT * 8 * 16);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mine[(n * 8 + 2 * t) * 16 + g] = acc[n][0];
      mine[(n * 8 + 2 * t + 1) * 16 + g] = acc[n][1];
      mine[(n * 8 + 2 * t) * 16 + g + 8] = acc[n][2];
      mine[(n * 8 + 2 * t + 1) * 16 + g + 8] = acc[n][3];
    }
    __syncthreads();
    const int cols = 16 * wr;
    for (int i = tid; i < mrows * cols; i += kWarps * 32) {
      const int m = i / cols, c = i - m * cols, n = tile * cols + c;
      if (n >= a.n) continue;
      const float* from = red + (buf * kWarps + (c >> 4) * wk) * (NT * 8 * 16) + m * 16 + (c & 15);
      float y = 0.0f;
      for (int q = 0; q < wk; ++q) y = __fadd_rn(y, from[q * (NT * 8 * 16)]);
      if (a.x_scale) y = __fmul_rn(y, a.x_scale[m0 + m]);
      const int64_t at = static_cast<int64_t>(m0 + m) * a.n + n;
      if (a.out_dtype == MOE_LAYER_FP32) static_cast<float*>(a.y)[at] = y;
      else if (a.out_dtype == MOE_LAYER_BF16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(y);
      else static_cast<__half*>(a.y)[at] = __float2half_rn(y);
    }
    // with two halves the other one is written while this one may still be read
    if constexpr (kRedBufs<NT> == 2) buf ^= 1;
    else __syncthreads();
  }
  cp_async_wait<0>();
}

template <typename T, int NT>
cudaError_t launch_nt(const moe_layer_w4_args_t& a, int num_sms, cudaStream_t s) {
  W4Params p;
  p.a = a;
  const int kpad = (a.k + kStepK - 1) / kStepK * kStepK;
  const int fit = kXBudget / (8 * NT * 2) / kStepK * kStepK;
  p.pieces = (kpad + fit - 1) / fit;
  p.kc = (kpad / kStepK + p.pieces - 1) / p.pieces * kStepK;
  p.pieces = (kpad + p.kc - 1) / p.kc;
  p.xpitch = p.kc * 2 + 64;  // a multiple of 128 plus 64: rows 2i and 2i + 1 of a 16-byte read fall on other banks
  p.ngroups = a.k / a.group;
  // as many row groups as still give every SM a tile, and no more parts of K than steps of K
  p.wr = 1;
  while (p.wr < kWarps && ((a.n + 32 * p.wr - 1) / (32 * p.wr) >= 16 * num_sms || p.kc / kStepK < kWarps / p.wr)) p.wr *= 2;
  p.tiles = (a.n + 16 * p.wr - 1) / (16 * p.wr);
  const int smem = 8 * NT * p.xpitch + kWarps * kStagesOf<NT> * kStageBytes + kRedBufs<NT> * kWarps * NT * 8 * 16 * 4;
  const int gps = a.group == 32 ? 4 : (a.group == 64 ? 2 : 1);
  const void* k = gps == 4 ? (const void*)w4_linear_kernel<T, NT, 4>
                           : (gps == 2 ? (const void*)w4_linear_kernel<T, NT, 2> : (const void*)w4_linear_kernel<T, NT, 1>);
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  void* args[] = {&p};
  const int gx = p.tiles < num_sms ? p.tiles : num_sms;
  return cudaLaunchKernel(k, dim3(gx, (a.m + 8 * NT - 1) / (8 * NT)), dim3(kWarps * 32), args, smem, s);
}

template <typename T>
cudaError_t launch_t(const moe_layer_w4_args_t& a, int num_sms, cudaStream_t s) {
  if (a.m <= 8) return launch_nt<T, 1>(a, num_sms, s);
  if (a.m <= 16) return launch_nt<T, 2>(a, num_sms, s);
  return launch_nt<T, 4>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_w4(const moe_layer_w4_args_t& a, int num_sms, cudaStream_t s) {
  // int8 codes are exact in fp16 and bf16; fp16 needs fewer operations a weight
  return a.x_dtype == MOE_LAYER_BF16 ? launch_t<__nv_bfloat16>(a, num_sms, s) : launch_t<__half>(a, num_sms, s);
}

}  // namespace moe_layer
