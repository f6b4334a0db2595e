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
// 128-k steps by asynchronous copies, which needs no barrier.  One part of K
// is written straight from the accumulators; several are summed in shared
// memory, in a fixed order.  x lies in shared memory, its elements in the
// order in which the codes leave a 32-bit word.
//
// k order.  Both operands may take the k of a group in any common order.  A
// lane takes neighbouring words of a weight row, as many as the group allows
// the four lanes of a row to take (4 words at groups of 128 and more, 2 at
// 64, 1 at 32), so that each product of 16 k stays inside one group.
#include <type_traits>

#include "layer_ops.cuh"

namespace moe_layer {
namespace {

constexpr int kWarps = 16;
constexpr int kStepK = 128;                    // k of one ring stage
constexpr int kStageBytes = 16 * kStepK / 2;   // 16 weight rows
constexpr int kXSmall = 66 * 1024;             // bytes of x that leave room for 8 stages of a warp
constexpr int kXMost = 130 * 1024;             // and for 4

struct W4Params {
  moe_layer_w4_args_t a;
  int kc;         // k of one piece of x that fits shared memory (multiple of 128)
  int pieces;     // pieces of kc that cover k
  int wr;         // row groups of a CTA: 1, 2, 4, 8 or 16
  int tiles;      // tiles of 16 weight rows
  int xpitch;     // bytes of a row of x in shared memory
  int ngroups;    // k / group
};

__device__ __forceinline__ float scale_at(const void* p, int64_t i, int dt) {
  if (dt == MOE_LAYER_FP32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t b = __ldg(static_cast<const uint16_t*>(p) + i);
  return dt == MOE_LAYER_BF16 ? __uint_as_float(static_cast<uint32_t>(b) << 16) : __half2float(__ushort_as_half(b));
}

// The 8 codes of a word as 4 pairs (0,4) (1,5) (2,6) (3,7), minus the zero
// point.  fp16: a code in the low bits of the mantissa of 1024 is 1024 + code,
// four bits higher 1024 + 16 code, which one exact fma turns into code - zero.
// bf16's mantissa holds the low position only.  zp: zero_words.
template <typename T>
__device__ __forceinline__ void expand8(uint32_t w, const uint32_t (&zp)[2], uint32_t (&o)[4]) {
  if constexpr (std::is_same_v<T, __half>) {
    const uint32_t sixteenth = 0x2C002C00u;  // 1 / 16
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = i ? w >> 8 : w;
      const uint32_t lo = (v & 0x000F000Fu) | 0x64006400u, hi = (v & 0x00F000F0u) | 0x64006400u;
      const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), *reinterpret_cast<const __half2*>(&zp[0]));
      const __half2 b = __hfma2(*reinterpret_cast<const __half2*>(&hi), *reinterpret_cast<const __half2*>(&sixteenth),
                                *reinterpret_cast<const __half2*>(&zp[1]));
      o[2 * i] = *reinterpret_cast<const uint32_t*>(&a);
      o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
      const __nv_bfloat162 r =
          __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), *reinterpret_cast<const __nv_bfloat162*>(&zp[0]));
      o[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}

// fp16: 1024 + zero, and -(64 + zero); bf16: 128 + zero
template <typename T>
__device__ __forceinline__ void zero_words(uint32_t z, uint32_t (&zp)[2]) {
  if constexpr (std::is_same_v<T, __half>) {
    zp[0] = (0x6400u | z) * 0x10001u;
    zp[1] = (0xD400u | (z << 4)) * 0x10001u;
  } else {
    zp[0] = (0x4300u | z) * 0x10001u;
    zp[1] = 0u;
  }
}

// where 16-byte chunk c of row r of a stage lies: reads of 16, 8 and 4 bytes
// a lane (8 rows x 4 lanes) all fall on different banks
__device__ __forceinline__ uint32_t stage_at(int r, int c) {
  const int s = ((r >> 2) & 1) | (r & 2);
  return r * 64 + ((c ^ s) << 4);
}

// 8 neighbouring elements of x as pairs (0,4) (1,5) (2,6) (3,7)
__device__ __forceinline__ uint4 pair04(uint4 v) {
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                    __byte_perm(v.y, v.w, 0x7632));
}

// NT: tiles of 8 rows of x.  GPS: groups of a 128-k step (1, 2 or 4)
template <typename T, int NT, int GPS, int kStages>
__global__ void __launch_bounds__(kWarps * 32, 1) w4_linear_kernel(const W4Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  grid_dependency_wait();
  grid_launch_dependents();
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

  // row group r of CTA c takes tiles (r + wr i) grid + c: every SM gets as many, to one
  const int first_tile = row_group * gridDim.x + blockIdx.x, next_tile = wr * gridDim.x;
  const int rounds = (p.tiles + next_tile - 1) / next_tile;  // the same for every warp
  const int steps_pp = p.kc / kStepK;                        // steps of a piece, all parts
  const int64_t row_bytes = a.k / 2;

  // position of the copies: tile, piece, step of this warp, ahead of the products
  int c_tile = first_tile, c_piece = 0, c_step = kpart, c_slot = 0;
  const int cr = lane >> 2, cc = lane & 3;  // this lane copies chunk cc of rows cr and cr + 8
  auto issue = [&]() {
    if (c_tile < p.tiles) {
      const int kb = (c_piece * p.kc + c_step * kStepK) / 2 + cc * 16;
      const bool ok = kb < row_bytes;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = cr + hh * 8, n = min(c_tile * 16 + r, a.n - 1);
        cp_async16(ring_u + c_slot * kStageBytes + stage_at(r, cc), a.w + n * row_bytes + (ok ? kb : 0), ok);
      }
      c_step += wk;
      if (c_step >= steps_pp || c_piece * p.kc + c_step * kStepK >= a.k) {
        c_step = kpart;
        if (++c_piece == p.pieces || c_piece * p.kc + c_step * kStepK >= a.k) {
          c_piece = 0;
          c_tile += next_tile;
        }
      }
    }
    c_slot = c_slot + 1 == kStages ? 0 : c_slot + 1;
    cp_async_commit();
  };
  // a warp whose part of K is empty issues nothing
  if (kpart * kStepK >= min(p.kc, a.k)) c_tile = p.tiles;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue();

  // x of one piece, 8 elements at a time, four loads in flight
  auto load_x = [&](int piece) {
    const int k0 = piece * p.kc, n8 = p.kc / 8, all = 8 * NT * n8;
    for (int base = tid; base < all; base += 4 * kWarps * 32) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = base + u * kWarps * 32, m = i / n8, k = k0 + (i - m * n8) * 8;
        v[u] = make_uint4(0, 0, 0, 0);
        if (m < mrows && k < a.k) {
          const int64_t at = (m0 + m) * a.x_stride + k;
          if (a.x_dtype == MOE_LAYER_INT8) {
            const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const int8_t*>(a.x) + at);
            v[u].x = q.x, v[u].y = q.y;
          } else {
            v[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + at);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = base + u * kWarps * 32;
        if (i >= all) break;
        const int m = i / n8, k8 = i - m * n8;
        uint4 x = v[u];
        if (a.x_dtype == MOE_LAYER_INT8) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t b = (j < 2 ? v[u].x : v[u].y) >> ((j & 1) * 16);
            o[j] = pack2<T>(static_cast<float>(static_cast<int8_t>(b & 0xFF)),
                            static_cast<float>(static_cast<int8_t>((b >> 8) & 0xFF)));
          }
          x = make_uint4(o[0], o[1], o[2], o[3]);
        }
        // block k8 of a step belongs to lane xt, word xj: it is read as block 4 xj + xt
        const int kk = k8 & 15;
        int xt, xj;
        if constexpr (GPS == 1) xt = kk >> 2, xj = kk & 3;
        else if constexpr (GPS == 2) xt = (kk & 7) >> 1, xj = (kk >> 3) * 2 + (kk & 1);
        else xt = kk & 3, xj = kk >> 2;
        *reinterpret_cast<uint4*>(xs + m * p.xpitch + ((k8 & ~15) + xj * 4 + xt) * 16) = pair04(x);
      }
    }
  };

  int slot = 0, buf = 0;
  for (int it = 0; it < rounds; ++it) {
    const int tile = first_tile + it * next_tile;
    const int64_t na = min(tile * 16 + g, a.n - 1), nb = min(tile * 16 + g + 8, a.n - 1);
    float acc[NT][4] = {};
    for (int piece = 0; piece < p.pieces; ++piece) {
      if (it == 0 || p.pieces > 1) {
        if (it > 0 || piece > 0) __syncthreads();  // the last piece is no longer read
        load_x(piece);
        __syncthreads();
      }
      const int k0 = piece * p.kc;
      if (tile < p.tiles) {
        for (int step = kpart; step < steps_pp && k0 + step * kStepK < a.k; step += wk) {
          // scales and zeros of this step's groups, asked for before the wait
          const int kk = k0 + step * kStepK;
          float sa[GPS], sb[GPS];
          uint32_t za[GPS][2], zb[GPS][2];
#pragma unroll
          for (int i = 0; i < GPS; ++i) {
            const int gi = min(GPS == 1 ? kk / a.group : kk / (kStepK / GPS) + i, p.ngroups - 1);
            sa[i] = scale_at(a.w_scale, na * p.ngroups + gi, a.scale_dtype);
            sb[i] = scale_at(a.w_scale, nb * p.ngroups + gi, a.scale_dtype);
            zero_words<T>(a.w_zero ? __ldg(a.w_zero + na * p.ngroups + gi) & 15u : 8u, za[i]);
            zero_words<T>(a.w_zero ? __ldg(a.w_zero + nb * p.ngroups + gi) & 15u : 8u, zb[i]);
          }
          cp_async_wait<kStages - 2>();
          __syncwarp();
          const uint32_t st = ring_u + slot * kStageBytes;
          uint32_t wa[4], wb[4];
          if constexpr (GPS == 1) {
            const uint4 u = lds128(st + stage_at(g, t)), v = lds128(st + stage_at(g + 8, t));
            wa[0] = u.x, wa[1] = u.y, wa[2] = u.z, wa[3] = u.w;
            wb[0] = v.x, wb[1] = v.y, wb[2] = v.z, wb[3] = v.w;
          } else if constexpr (GPS == 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint2 u = lds64(st + stage_at(g, 2 * i + (t >> 1)) + (t & 1) * 8);
              const uint2 v = lds64(st + stage_at(g + 8, 2 * i + (t >> 1)) + (t & 1) * 8);
              wa[2 * i] = u.x, wa[2 * i + 1] = u.y;
              wb[2 * i] = v.x, wb[2 * i + 1] = v.y;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              wa[i] = lds32(st + stage_at(g, i) + t * 4);
              wb[i] = lds32(st + stage_at(g + 8, i) + t * 4);
            }
          }
          const uint32_t xa = xs_u + g * p.xpitch + step * kStepK * 2 + t * 16;
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
            expand8<T>(wa[j], za[gi], ea);
            expand8<T>(wb[j], zb[gi], eb);
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
    }
    auto store = [&](int m, int n, float y) {
      if (a.x_scale) y = __fmul_rn(y, a.x_scale[m0 + m]);
      const int64_t at = static_cast<int64_t>(m0 + m) * a.n + n;
      if (a.out_dtype == MOE_LAYER_FP32) static_cast<float*>(a.y)[at] = y;
      else if (a.out_dtype == MOE_LAYER_BF16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(y);
      else static_cast<__half*>(a.y)[at] = __float2half_rn(y);
    };
    if (wk == 1) {
      if (tile < p.tiles) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = n * 8 + 2 * t + (e & 1), row = tile * 16 + g + 8 * (e >> 1);
            if (m < mrows && row < a.n) store(m, row, acc[n][e]);
          }
      }
      continue;
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
      const int m = i / cols, c = i - m * cols, rg = c >> 4;
      const int n = (rg * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x) + it * next_tile) * 16 + (c & 15);
      if (n >= a.n) continue;
      const float* from = red + (buf * kWarps + rg * wk) * (NT * 8 * 16) + m * 16 + (c & 15);
      float y = 0.0f;
      for (int q = 0; q < wk; ++q) y = __fadd_rn(y, from[q * (NT * 8 * 16)]);
      store(m, n, y);
    }
    // with two halves the other one is written while this one may still be read
    if constexpr (NT == 1) buf ^= 1;
    else __syncthreads();
  }
  cp_async_wait<0>();
}

template <typename T, int NT, int GPS, int kStages>
cudaError_t launch_stages(const W4Params& p, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  const void* k = (const void*)w4_linear_kernel<T, NT, GPS, kStages>;
  if (const cudaError_t e = allow_smem(k, kMaxSmem, allowed); e != cudaSuccess) return e;
  const int red = p.wr == kWarps ? 0 : (NT == 1 ? 2 : 1) * kWarps * NT * 8 * 16 * 4;
  const int smem = 8 * NT * p.xpitch + kWarps * kStages * kStageBytes + red;
  W4Params arg = p;
  void* args[] = {&arg};
  const int groups = (p.tiles + p.wr - 1) / p.wr;
  return launch_after(k, dim3(groups < num_sms ? groups : num_sms, (p.a.m + 8 * NT - 1) / (8 * NT)), dim3(kWarps * 32),
                      args, smem, s);
}

template <typename T, int NT, int GPS>
cudaError_t launch_gps(const W4Params& p, int num_sms, cudaStream_t s) {
  if constexpr (NT < 4)
    if (8 * NT * p.xpitch <= kXSmall) return launch_stages<T, NT, GPS, 8>(p, num_sms, s);
  return launch_stages<T, NT, GPS, 4>(p, num_sms, s);
}

template <typename T, int NT>
cudaError_t launch_nt(const moe_layer_w4_args_t& a, int num_sms, cudaStream_t s) {
  W4Params p;
  p.a = a;
  const int kpad = (a.k + kStepK - 1) / kStepK * kStepK;
  const int fit = (kXMost / (8 * NT) - 64) / 2 / kStepK * kStepK;
  p.pieces = (kpad + fit - 1) / fit;
  p.kc = (kpad / kStepK + p.pieces - 1) / p.pieces * kStepK;
  p.pieces = (kpad + p.kc - 1) / p.kc;
  p.xpitch = p.kc * 2 + 64;  // a multiple of 128 plus 64: rows 2i and 2i + 1 of a 16-byte read fall on other banks
  p.ngroups = a.k / a.group;
  p.tiles = (a.n + 15) / 16;
  // one part of K where every warp gets two tiles or more; else more parts,
  // but no more than a piece has steps
  p.wr = kWarps;
  while (p.wr > 1 && p.tiles < 2 * p.wr * num_sms && 2 * (kWarps / p.wr) <= p.kc / kStepK) p.wr /= 2;
  if (a.group == 32) return launch_gps<T, NT, 4>(p, num_sms, s);
  if (a.group == 64) return launch_gps<T, NT, 2>(p, num_sms, s);
  return launch_gps<T, NT, 1>(p, num_sms, s);
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
