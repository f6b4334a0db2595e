// Products of a few rows of x with 4-bit weights and group scales.
//
// y^T = W x^T as mma.sync m16n8k16 in fp16: weight rows are the M side, 8 rows
// of x the N side, so that one row of x costs what eight do and the weights
// pass through registers once.
//
// Codes.  A code masked out of its word is, as fp16 bits, the subnormal code x
// 2^-24 (or, four bits higher, code x 2^-20), which the matrix unit multiplies
// exactly: five operations turn a word into four pairs.  The elements of x
// that meet the higher position are stored as x / 16.  With X the sum of a
// group's x, sum x (code - zero) = sum x code - zero X: the second term is one
// fp32 fma a group.
//
// x.  Each 128 k of a row are scaled by a power of two to [2^8, 2^9) at their
// largest element, so x and x / 16 are exact in fp16 but for elements 2^18
// below the largest, which keep a step of 2^-28 of it: nothing that an fp32
// sum over them can tell.  Products are exact, a group's sum is one fp32
// accumulator chain and enters the row's sum through an fp32 fma with the
// group's scale and the power of two.  X and the row's sum are held times 2^-16,
// so that neither passes fp32 where x and y do not.
//
// Bound by the weights' bytes, and close behind by instructions (about 140 a KB
// of weights at one row, 180 at 16): 130001 x 4096 takes 55 us for one row (4.9
// TB/s of 6.8), 57 for 8, 74 for 16; groups of 32, with four times the scales and
// fp32 steps, 97 for 8 rows.  4096 x 4096 for one row 6 us, of which a
// launch and the first trip to memory are 3.6.  Every 16 rows of x read the
// weights again: 6144 x 4096 takes 12 us for 16 rows, 34 for 64, 244 for 512 and
// 1920 for 4096.  The tensor-memory product, with weights converted into tensor
// memory as its M side, has not been built here; it is what many rows would need.  A CTA has 16
// warps in WR groups of rows x (16 / WR) parts of K; a warp streams its own
// 16-row tiles through a ring of 128-k steps by asynchronous copies, which
// needs no barrier.  One part of K is written straight from the accumulators;
// several are summed in shared memory, in a fixed order.  Where tiles are
// few or a CTA's shared memory does not hold x (8 rows beyond k 8192, 16 beyond
// 4096), a cluster of up to 8 CTAs shares K, so that each lays out its part of x
// alone, and sums over distributed shared memory: 16 x 4096 x 14336 18 us, where
// CTAs that took x in pieces took 38; 64 x 8000 x 16384 113 (186).
//
// k order.  Both operands may take the k of a group in any common order.  A
// lane takes neighbouring words of a weight row, as many as the group allows
// the four lanes of a row to take (4 words at groups of 128 and more, 2 at
// 64, 1 at 32), so that each product of 16 k stays inside one group.
#include <climits>
#include <cstdint>

#include "layer_ops.cuh"

namespace moe_layer {
namespace {

constexpr int kWarps = 16;
constexpr int kRows = 16;                      // weight rows of a tile
constexpr int kStepK = 128;                    // k of one ring stage
constexpr int kStageBytes = kRows * kStepK / 2;
constexpr int kXSmall = 66 * 1024;             // bytes of x that leave room for 8 stages of a warp
constexpr int kXMost = 130 * 1024;             // and for 4
constexpr int kMostCtas = 8;                   // of a cluster

// bytes of a warp's own: the scales and scale x zero of 8 groups, or its partial sums
template <int NT>
constexpr int kPrivateOf = NT * 8 * kRows * 4 > 2 * 8 * kRows * 4 ? NT * 8 * kRows * 4 : 2 * 8 * kRows * 4;

struct W4Params {
  moe_layer_w4_args_t a;
  int kc;         // k of one piece of x that fits shared memory (whole steps of every part of K)
  int pieces;     // pieces of kc that cover k
  int wr;         // row groups of a CTA: 1, 2, 4 or 8
  int tiles;      // tiles of kRows weight rows
  int cs;         // CTAs of a cluster, which share K between them
  int cta_steps;  // steps of one of them (all, where cs is 1)
  int at_once;    // clusters that run at once
  int xpitch;     // bytes of a row of x in shared memory
  int ngroups;    // k / group
  int gsteps;     // steps of a group (1 for groups of 128 and less)
};

// bits of a scale, loaded early; its value
__device__ __forceinline__ uint32_t scale_bits(const void* p, int64_t i, int dt) {
  if (dt == MOE_LAYER_FP32) return __ldg(static_cast<const uint32_t*>(p) + i);
  return __ldg(static_cast<const uint16_t*>(p) + i);
}
__device__ __forceinline__ float scale_value(uint32_t b, int dt) {
  if (dt == MOE_LAYER_FP16) return __half2float(__ushort_as_half(static_cast<uint16_t>(b)));
  return __uint_as_float(dt == MOE_LAYER_BF16 ? b << 16 : b);
}

// a pair of fp16 times a power of two
__device__ __forceinline__ uint32_t half_mul(uint32_t v, float f) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 2^e, e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// where 16-byte chunk c of row r of a stage lies: reads of 16, 8 and 4 bytes
// a lane (8 rows x 4 lanes) all fall on different banks
__device__ __forceinline__ uint32_t stage_at(int r, int c) {
  const int s = ((r >> 2) & 1) | (r & 2);
  return r * 64 + ((c ^ s) << 4);
}

// NT: tiles of 8 rows of x.  GPS: groups of a 128-k step (1, 2 or 4)
// SPLIT: the CTAs of a cluster share K
template <int NT, int GPS, int kStages, bool SPLIT>
__global__ void __launch_bounds__(kWarps * 32, 1) w4_linear_kernel(const W4Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int M = 8 * NT;                            // rows of x of a CTA
  constexpr int kBlock = 8 / GPS;                      // steps whose scales come together: 8 groups
  constexpr int kPrivate = kPrivateOf<NT>;  // of a warp: scales and scale x zero of a block; its partial sums
  grid_dependency_wait();
  grid_launch_dependents();
  const moe_layer_w4_args_t& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int wr = p.wr, wk = kWarps / wr;
  const int row_group = warp / wk, kpart = warp - row_group * wk;
  const int m0 = blockIdx.y * M;
  const int mrows = min(a.m - m0, M);
  const int all_steps = (a.k + kStepK - 1) / kStepK, steps_pp = p.kc / kStepK;
  const int rank = SPLIT ? blockIdx.x % p.cs : 0, cid = SPLIT ? blockIdx.x / p.cs : blockIdx.x;
  const int ncl = SPLIT ? gridDim.x / p.cs : gridDim.x;
  const int s_base = SPLIT ? rank * p.cta_steps : 0;  // this CTA's steps: [s_base, s_base + steps)
  const int steps = SPLIT ? max(0, min(p.cta_steps, all_steps - s_base)) : all_steps;
  // x | of each group of a step and pair of rows, the sums and the powers of two [steps_pp * GPS][M / 2] | private | rings
  uint8_t* xs = smem;
  float4* xsum = reinterpret_cast<float4*>(smem + M * p.xpitch);
  float* priv = reinterpret_cast<float*>(xsum + steps_pp * GPS * (M / 2));
  float* mine = priv + warp * (kPrivate / 4);
  const uint32_t ring_u =
      static_cast<uint32_t>(__cvta_generic_to_shared(priv + kWarps * (kPrivate / 4))) + warp * (kStages * kStageBytes);
  const uint32_t xs_u = static_cast<uint32_t>(__cvta_generic_to_shared(xs));
  const uint32_t xsum_u = static_cast<uint32_t>(__cvta_generic_to_shared(xsum));

  // row group r of CTA (or cluster) c of C takes tiles (r + wr i) C + c: every SM gets as many, to one
  const int first_tile = row_group * ncl + cid, next_tile = wr * ncl;
  const int rounds = (p.tiles + next_tile - 1) / next_tile;  // the same for every warp
  const int run = steps_pp / wk;                             // steps of a part of K in a piece
  const int row_bytes = a.k / 2;
  // steps of this warp's part in a piece: [piece * steps_pp + kpart * run, ...)
  auto run_of = [&](int piece) { return min(run, steps - piece * steps_pp - kpart * run); };

  // the copies run ahead of the products: this lane copies chunk cc of rows cr and cr + 8
  const int cr = lane >> 2, cc = lane & 3;
  const int tail = (row_bytes & (kStepK / 2 - 1)) ? row_bytes & (kStepK / 2 - 1) : kStepK / 2;  // bytes of the last step
  int c_tile = first_tile, c_piece = 0, c_left = run_of(0);
  uint32_t c_slot = 0;
  const uint8_t *c_row0 = a.w, *c_row1 = a.w;
  bool c_last = false;  // the run ends with K, whose last step this lane may be past
  auto copy_run = [&]() {  // the start of a run
    const int step = c_piece * steps_pp + kpart * run, kb = (s_base + step) * (kStepK / 2) + cc * 16;
    c_row0 = a.w + static_cast<int64_t>(min(c_tile * kRows + cr, a.n - 1)) * row_bytes + kb;
    c_row1 = a.w + static_cast<int64_t>(min(c_tile * kRows + cr + 8, a.n - 1)) * row_bytes + kb;
    c_last = s_base + step + c_left == all_steps && cc * 16 >= tail;
  };
  if (c_left <= 0) c_tile = p.tiles;  // no part of K for this warp
  if (c_tile < p.tiles) copy_run();
  const uint32_t c_dst = ring_u + stage_at(cr, cc);  // row cr + 8 lies 512 bytes on
  auto issue = [&]() {
    if (c_tile < p.tiles) {
      const bool ok = !(c_last && c_left == 1);  // past the end of K: zeros
      cp_async16(c_dst + c_slot, ok ? c_row0 : a.w, ok);
      cp_async16(c_dst + c_slot + 8 * 64, ok ? c_row1 : a.w, ok);
      c_row0 += kStepK / 2;
      c_row1 += kStepK / 2;
      if (--c_left == 0) {
        if (++c_piece == p.pieces || run_of(c_piece) <= 0) {
          c_piece = 0;
          c_tile += next_tile;
        }
        c_left = run_of(c_piece);
        if (c_tile < p.tiles) copy_run();
      }
    }
    c_slot = (c_slot + kStageBytes) & (kStages * kStageBytes - 1);
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue();

  // Scales and zeros come 8 groups at a time: lane t of a quad loads groups 2t
  // and 2t + 1 of rows g and g + 8, one block ahead, and lays scale and
  // -scale x zero out as [group][g][row] for one 16-byte read a group.
  uint32_t sraw[2][2], zraw[2][2] = {{8u, 8u}, {8u, 8u}};
  int64_t s_row0 = 0, s_row1 = 0;
  auto scale_tile = [&](int tile) {
    s_row0 = static_cast<int64_t>(min(tile * kRows + g, a.n - 1)) * p.ngroups;
    s_row1 = static_cast<int64_t>(min(tile * kRows + g + 8, a.n - 1)) * p.ngroups;
  };
  auto load_scales = [&](int first_step) {
    const int v = first_step * GPS + 2 * t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int gi = min(GPS == 1 && p.gsteps > 1 ? (v + i) / p.gsteps : v + i, p.ngroups - 1);
      sraw[0][i] = scale_bits(a.w_scale, s_row0 + gi, a.scale_dtype);
      sraw[1][i] = scale_bits(a.w_scale, s_row1 + gi, a.scale_dtype);
      if (a.w_zero) {
        zraw[0][i] = __ldg(a.w_zero + s_row0 + gi) & 15u;
        zraw[1][i] = __ldg(a.w_zero + s_row1 + gi) & 15u;
      }
    }
  };
  if (kpart * run < steps) {
    scale_tile(min(first_tile, p.tiles - 1));
    load_scales(s_base + kpart * run);
  }
  const uint32_t mine_u = static_cast<uint32_t>(__cvta_generic_to_shared(mine));

  // x of one piece: 16 / (rows, as a power of two) warps a row, 8 elements a
  // lane, so 16 lanes hold the 128 k that share a power of two.  Rows past the
  // last are not written: a column of the products meets no other.
  const int row_shift = 31 - __clz(2 * mrows - 1);
  auto load_x_as = [&](auto type, int piece) {
    using X = decltype(type);
    constexpr bool kInt8 = sizeof(X) == 1;
    const int k0 = s_base * kStepK + piece * p.kc, n8 = p.kc / 8;
    const int m = warp & ((1 << row_shift) - 1), part = warp >> row_shift, parts = kWarps >> row_shift;
    if (m >= mrows) return;
    const X* row = static_cast<const X*>(a.x) + static_cast<int64_t>(m0 + m) * a.x_stride + k0;
    uint8_t* to = xs + m * p.xpitch;
    float* sums = reinterpret_cast<float*>(xsum) + (m >> 1) * 4 + (m & 1);
    for (int first = part * 32; first < n8; first += 8 * 32 * parts) {  // the same for every lane: sums cross lanes
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int k8 = first + u * 32 * parts + lane;
        v[u] = make_uint4(0, 0, 0, 0);
        if (k8 < n8 && k0 + k8 * 8 < a.k) {
          if constexpr (kInt8) {
            const uint2 q = *reinterpret_cast<const uint2*>(row + k8 * 8);
            v[u].x = q.x, v[u].y = q.y;
          } else {
            v[u] = *reinterpret_cast<const uint4*>(row + k8 * 8);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int k8 = first + u * 32 * parts + lane;
        if (k8 - lane >= n8) break;
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        // pairs (0,4) (1,5) (2,6) (3,7) x 2^(8 - e); the second and the last meet codes four bits higher
        uint4 x;
        float sum;
        int e = 7;  // codes of up to 127: [2^6, 2^7)
        if constexpr (kInt8) {
          half_pairs(__byte_perm(w[0], w[1], 0x5140), x.x, x.y);
          half_pairs(__byte_perm(w[0], w[1], 0x7362), x.z, x.w);
          x.x = half_mul(x.x, 2.0f), x.y = half_mul(x.y, 0.125f);
          x.z = half_mul(x.z, 2.0f), x.w = half_mul(x.w, 0.125f);
          sum = static_cast<float>(__dp4a(static_cast<int>(w[0]), 0x01010101, __dp4a(static_cast<int>(w[1]), 0x01010101, 0)));
        } else {
          // magnitudes are ordered as 16-bit integers
          uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                  __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
          top = max(top >> 16, top & 0xFFFFu);
          const float2 big = unpack2<X>(top);
          // an infinity or a NaN stays one; elements of 2^-110 and less may vanish
          e = min(max(static_cast<int>(__float_as_uint(big.x) >> 23), 17), 254) - 127;
          float f[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 h = unpack2<X>(w[j]);
            f[2 * j] = h.x, f[2 * j + 1] = h.y;
          }
          // times 2^-16, as all sums are: no x that fp32 holds makes one pass it on the way
          sum = __fadd_rn(__fadd_rn(__fmaf_rn(f[0], 0x1p-16f, __fmul_rn(f[1], 0x1p-16f)), __fmaf_rn(f[2], 0x1p-16f, __fmul_rn(f[3], 0x1p-16f))),
                          __fadd_rn(__fmaf_rn(f[4], 0x1p-16f, __fmul_rn(f[5], 0x1p-16f)), __fmaf_rn(f[6], 0x1p-16f, __fmul_rn(f[7], 0x1p-16f))));
          const float up = pow2(8 - e), up16 = pow2(4 - e);
          x.x = pack2<__half>(__fmul_rn(f[0], up), __fmul_rn(f[4], up));
          x.y = pack2<__half>(__fmul_rn(f[1], up16), __fmul_rn(f[5], up16));
          x.z = pack2<__half>(__fmul_rn(f[2], up), __fmul_rn(f[6], up));
          x.w = pack2<__half>(__fmul_rn(f[3], up16), __fmul_rn(f[7], up16));
        }
#pragma unroll
        for (int o = 1; o < 16 / GPS; o <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
        if (k8 < n8) {
          if (lane % (16 / GPS) == 0) {
            float* at = sums + (k8 / (16 / GPS)) * (M * 2);
            at[0] = kInt8 ? __fmul_rn(sum, 0x1p-16f) : sum;
            at[2] = pow2(e);
          }
          // block k8 of a step belongs to lane xt, word xj: it is read as block 4 xj + xt
          const int kk = k8 & 15;
          int xt, xj;
          if constexpr (GPS == 1) xt = kk >> 2, xj = kk & 3;
          else if constexpr (GPS == 2) xt = (kk & 7) >> 1, xj = (kk >> 3) * 2 + (kk & 1);
          else xt = kk & 3, xj = kk >> 2;
          *reinterpret_cast<uint4*>(to + ((k8 & ~15) + xj * 4 + xt) * 16) = x;
        }
      }
    }
  };
  auto load_x = [&](int piece) {
    if (a.x_dtype == MOE_LAYER_INT8) load_x_as(int8_t(), piece);
    else if (a.x_dtype == MOE_LAYER_BF16) load_x_as(__nv_bfloat16(), piece);
    else load_x_as(__half(), piece);
  };

  const uint32_t w_at = ring_u + (GPS == 1 ? stage_at(g, t) : 0);
  const int wr_shift = 31 - __clz(wr);
  uint32_t slot = 0;
  for (int it = 0; it < rounds; ++it) {
    const int tile = first_tile + it * next_tile;
    float acc[NT][4] = {};
    for (int piece = 0; piece < p.pieces; ++piece) {
      if (it == 0 || p.pieces > 1) {
        if (it > 0 || piece > 0) __syncthreads();  // the last piece is no longer read
        load_x(piece);
        __syncthreads();
      }
      const int todo = tile < p.tiles ? run_of(piece) : 0;
      const int s0 = s_base + piece * steps_pp + kpart * run;
      uint32_t xa = xs_u + g * p.xpitch + t * 16 + kpart * run * kStepK * 2;
      uint32_t xg = xsum_u + (kpart * run * GPS * (M / 2) + t) * 16;
      for (int base = 0; base < todo; base += kBlock) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float v0 = scale_value(sraw[0][i], a.scale_dtype), v1 = scale_value(sraw[1][i], a.scale_dtype);
          *reinterpret_cast<float4*>(mine + ((2 * t + i) * 8 + g) * 4) =
              make_float4(v0, v1, -__fmul_rn(v0, static_cast<float>(zraw[0][i])),
                          -__fmul_rn(v1, static_cast<float>(zraw[1][i])));
        }
        // the next block: of this run, of the next piece, or of the next tile
        if (base + kBlock < todo) {
          load_scales(s0 + base + kBlock);
        } else if (piece + 1 < p.pieces && run_of(piece + 1) > 0) {
          load_scales(s0 + steps_pp);
        } else if (tile + next_tile < p.tiles) {
          scale_tile(tile + next_tile);
          load_scales(s_base + kpart * run);
        }
        uint32_t sa = mine_u + g * 16;
        const int here = min(kBlock, todo - base);
        for (int b = 0; b < here; ++b) {
          cp_async_wait<kStages - 2>();
          __syncwarp();  // every lane's copies, and the block's scales
          const uint32_t st = w_at + slot;
          uint32_t w[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if constexpr (GPS == 1) {
              const uint4 u = lds128(st + r * 8 * 64);
              w[r][0] = u.x, w[r][1] = u.y, w[r][2] = u.z, w[r][3] = u.w;
            } else if constexpr (GPS == 2) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint2 u = lds64(st + stage_at(g, 2 * i + (t >> 1)) + (t & 1) * 8 + r * 8 * 64);
                w[r][2 * i] = u.x, w[r][2 * i + 1] = u.y;
              }
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) w[r][i] = lds32(st + stage_at(g, i) + t * 4 + r * 8 * 64);
            }
          }
#pragma unroll
          for (int q = 0; q < GPS; ++q) {  // groups of the step
            constexpr int kWords = 4 / GPS;
            float part[NT][4];
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
              const int j = q * kWords + i;
              const uint32_t wa = w[0][j], wb = w[1][j], va = wa >> 8, vb = wb >> 8;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const uint4 xv = lds128(xa + n * 8 * p.xpitch + j * 64);
                if (i == 0)
                  mma16816_first(part[n], wa & 0x000F000Fu, wb & 0x000F000Fu, wa & 0x00F000F0u, wb & 0x00F000F0u,
                                 xv.x, xv.y);
                else
                  mma16816(part[n], wa & 0x000F000Fu, wb & 0x000F000Fu, wa & 0x00F000F0u, wb & 0x00F000F0u, xv.x,
                           xv.y);
                mma16816(part[n], va & 0x000F000Fu, vb & 0x000F000Fu, va & 0x00F000F0u, vb & 0x00F000F0u, xv.z,
                         xv.w);
              }
            }
            const uint4 su = lds128(sa);
            sa += kRows * 8;
            const float sv[2] = {__uint_as_float(su.x), __uint_as_float(su.y)};
            const float zv[2] = {__uint_as_float(su.z), __uint_as_float(su.w)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint4 xu = lds128(xg + n * 64);
              const float x2[2] = {__uint_as_float(xu.x), __uint_as_float(xu.y)};
              const float p2[2] = {__uint_as_float(xu.z), __uint_as_float(xu.w)};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[n][e] = __fmaf_rn(zv[e >> 1], x2[e & 1],
                                      __fmaf_rn(__fmul_rn(sv[e >> 1], p2[e & 1]), part[n][e], acc[n][e]));
            }
            xg += M * 8;
          }
          xa += kStepK * 2;
          __syncwarp();  // the stage is read before it is filled again
          issue();
          slot = (slot + kStageBytes) & (kStages * kStageBytes - 1);
        }
      }
    }
    auto store = [&](int m, int n, float y) {
      y = __fmul_rn(y, 0x1p16f);
      if (a.x_scale) y = __fmul_rn(y, __ldg(a.x_scale + m0 + m));
      const int64_t at = static_cast<int64_t>(m0 + m) * a.n + n;
      if (a.out_dtype == MOE_LAYER_FP32) static_cast<float*>(a.y)[at] = y;
      else if (a.out_dtype == MOE_LAYER_BF16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(y);
      else static_cast<__half*>(a.y)[at] = __float2half_rn(y);
    };
    if (!SPLIT && wk == 1) {
      if (tile < p.tiles) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = n * 8 + 2 * t + (e & 1), row = tile * kRows + g + 8 * (e >> 1);
            if (m < mrows && row < a.n) store(m, row, acc[n][e]);
          }
      }
      continue;
    }
    // parts of K, in each warp's private memory: [x row][16 weight rows]
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) mine[(n * 8 + 2 * t + (e & 1)) * kRows + g + 8 * (e >> 1)] = acc[n][e];
    if constexpr (SPLIT) cluster_sync();
    else __syncthreads();
    const int cshift = wr_shift + 4;  // columns: 16 x wr
    const int sharers = SPLIT ? p.cs : 1;
    for (int i = rank * kWarps * 32 + tid; i < mrows << cshift; i += sharers * kWarps * 32) {
      const int m = i >> cshift, c = i & ((1 << cshift) - 1), rg = c >> 4;
      const int n = (rg * ncl + cid + it * next_tile) * kRows + (c & 15);
      const float* from = priv + rg * wk * (kPrivate / 4) + m * kRows + (c & 15);
      float y = 0.0f;
      if constexpr (SPLIT) {
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(from));
        for (int w = 0; w < sharers; ++w)
#pragma unroll 4
          for (int q = 0; q < wk; ++q) y = __fadd_rn(y, cluster_read(at + q * kPrivate, w));
      } else {
        for (int q = 0; q < wk; ++q) y = __fadd_rn(y, from[q * (kPrivate / 4)]);
      }
      if (n < a.n) store(m, n, y);
    }
    if constexpr (SPLIT) cluster_sync();
    else __syncthreads();  // the sums are read before the next block's scales take their place
  }
  cp_async_wait<0>();
}

// Clusters of `cs` CTAs, one CTA an SM, that the current device runs at once:
// fewer than SMs / cs, as a cluster lies within a part of the GPU (one cluster too
// many doubles the time: 16 x 16384 x 16384 92 us).  Asked once a device and size.
cudaError_t clusters_at_once(int cs, int num_sms, int& n) {
  static std::atomic<int> known[64][3];
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
  const int slot = cs == 2 ? 0 : cs == 4 ? 1 : 2;
  n = dev < 64 ? known[dev][slot].load(std::memory_order_relaxed) : 0;
  if (n > 0) return cudaSuccess;
  static std::atomic<uint64_t> allowed{0};
  const void* k = (const void*)w4_linear_kernel<1, 1, 4, true>;
  if (const cudaError_t e = allow_smem(k, kMaxSmem, allowed); e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cs;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms / cs * cs);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = kMaxSmem;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, k, &cfg); e != cudaSuccess) return e;
  if (n < 1) return cudaErrorInvalidConfiguration;
  n = n < num_sms / cs ? n : num_sms / cs;
  if (dev < 64) known[dev][slot].store(n, std::memory_order_relaxed);
  return cudaSuccess;
}

template <int NT, int GPS, int kStages, bool SPLIT>
cudaError_t launch_stages(const W4Params& p, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  const void* k = (const void*)w4_linear_kernel<NT, GPS, kStages, SPLIT>;
  if (const cudaError_t e = allow_smem(k, kMaxSmem, allowed); e != cudaSuccess) return e;
  const int smem = 8 * NT * (p.xpitch + p.kc / kStepK * GPS * 8) + kWarps * kPrivateOf<NT> +
                   kWarps * kStages * kStageBytes;
  W4Params arg = p;
  void* args[] = {&arg};
  const int groups = (p.tiles + p.wr - 1) / p.wr;
  return launch_after(k, dim3((groups < p.at_once ? groups : p.at_once) * p.cs, (p.a.m + 8 * NT - 1) / (8 * NT)),
                      dim3(kWarps * 32), args, smem, s, p.cs);
}

template <int NT, int GPS>
cudaError_t launch_gps(const W4Params& p, cudaStream_t s) {
  const bool small = 8 * NT * p.xpitch <= kXSmall;
  if (p.cs > 1)
    return small ? launch_stages<NT, GPS, 8, true>(p, s) : launch_stages<NT, GPS, 4, true>(p, s);
  return small ? launch_stages<NT, GPS, 8, false>(p, s) : launch_stages<NT, GPS, 4, false>(p, s);
}

template <int NT>
cudaError_t launch_nt(const moe_layer_w4_args_t& a, int num_sms, cudaStream_t s) {
  W4Params p;
  p.a = a;
  p.ngroups = a.k / a.group;
  p.gsteps = a.group > kStepK ? a.group / kStepK : 1;
  p.tiles = (a.n + kRows - 1) / kRows;
  const int all_steps = (a.k + kStepK - 1) / kStepK;
  const int fit = (kXMost / (8 * NT) - 64) / (2 * kStepK);  // steps of x that shared memory takes
  // CTAs that share K, and row groups: the split with the least work in the
  // longest warp, in steps of 128 k (cost: 64ths of one).  A tile costs about
  // one step beside its own, about six where parts of K are summed (130001 x
  // 4096 took 58 us in one part, 83 us in eight).  x costs a step for every 64
  // of its rows x steps, once; every round, and six steps a piece, in pieces.  A
  // cluster costs 1 + cs / 4 steps, and its sums twice as much from the
  // second round on.  So few tiles are split (16 x 4096 x 4096: 11.6 us by one CTA
  // each, 10.0 by two, 9.2 by four) and many are not (16 x 28672 x 4096: 27 us by
  // one, 30 by two; 64 x 40000 x 4096 123 and 148).
  const int rows = a.m < 8 * NT ? a.m : 8 * NT;
  int64_t best = INT64_MAX;
  p.wr = p.cs = 1;
  p.cta_steps = all_steps;
  p.at_once = num_sms;
  for (int cs = 1; cs <= kMostCtas; cs *= 2) {
    const int steps = (all_steps + cs - 1) / cs, pieces = (steps + fit - 1) / fit;
    if (cs > 1 && (cs - 1) * steps >= all_steps) break;  // nothing for the last CTA
    int at_once = num_sms;
    if (cs > 1)
      if (const cudaError_t e = clusters_at_once(cs, num_sms, at_once); e != cudaSuccess) return e;
    for (int wr = kWarps; wr >= 1; wr /= 2) {
      const int wk = kWarps / wr;
      if (wk > steps || wk > fit) break;
      const int64_t tiles_at_once = static_cast<int64_t>(wr) * at_once;
      const int64_t rounds = (p.tiles + tiles_at_once - 1) / tiles_at_once;
      int64_t cost = 64 * rounds * ((steps + wk - 1) / wk + (wk > 1 || cs > 1 ? 6 : 1));
      cost += pieces > 1 ? rounds * (static_cast<int64_t>(rows) * steps + 64 * 6 * pieces) : rows * steps;
      if (cs > 1) cost += 64 * 6 * (rounds - 1) + 32 * cs + 32;
      if (cost < best) {
        best = cost;
        p.wr = wr, p.cs = cs, p.cta_steps = steps, p.at_once = at_once;
      }
    }
  }
  const int steps = p.cta_steps;
  const int wk = kWarps / p.wr;
  // pieces of whole rounds of the parts of K
  p.kc = (steps + wk - 1) / wk * wk;
  if (p.kc > fit) {
    const int most = fit / wk * wk;
    p.pieces = (steps + most - 1) / most;
    p.kc = ((steps + p.pieces - 1) / p.pieces + wk - 1) / wk * wk;
  }
  p.pieces = (steps + p.kc - 1) / p.kc;
  p.kc *= kStepK;
  p.xpitch = p.kc * 2 + 64;  // a multiple of 128 plus 64: rows 2i and 2i + 1 of a 16-byte read fall on other banks
  if (a.group == 32) return launch_gps<NT, 4>(p, s);
  if (a.group == 64) return launch_gps<NT, 2>(p, s);
  return launch_gps<NT, 1>(p, s);
}

}  // namespace

cudaError_t launch_w4(const moe_layer_w4_args_t& a, int num_sms, cudaStream_t s) {
  return a.m <= 8 ? launch_nt<1>(a, num_sms, s) : launch_nt<2>(a, num_sms, s);
}

}  // namespace moe_layer
