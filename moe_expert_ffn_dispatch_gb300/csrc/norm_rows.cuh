// Rows of 16-bit elements in registers, for the kernels that norm them
// (norm_quant.cu, norm_pair.cu): whole rows in one trip to memory, at any
// alignment.
#pragma once

#include "layer_ops.cuh"

namespace moe_layer {
namespace {

// A thread holds C chunks of 8 neighbouring elements: chunk n of the row is
// thread n % threads' chunk n / threads.  VEC: a chunk moves by 16-byte
// accesses (needs hidden % 8 == 0 and aligned rows).  Otherwise memory is
// accessed in the 16-byte blocks that the row happens to lie in: with the row
// `off` elements past a boundary, block n is elements 8 n - off .. 8 n - off +
// 7, and a chunk is put together from its own thread's block and the next one,
// which its thread leaves in shared memory (stores the other way round).
// Elements in the row's first and last block go one by one.  Either form
// leaves every thread the same elements, so the sums, and with them every
// result, do not depend on alignment.

__device__ __forceinline__ int halves_past(const void* p) { return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) >> 1; }

// a row of 16-bit elements on its way to shared memory: blocks c * nt + tid, and one more there can be
template <typename E, int C>
struct RowIn {
  uint4 b[C + 1];
  int off, blocks;
  // Elements around the row come along, unused, where rows before or after it
  // put them inside the tensor; elsewhere the row's own are read one by one.
  __device__ __forceinline__ void load(const E* row, int64_t rows_before, int64_t rows_after, int64_t stride, int tid, int nt, int h) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
    off = halves_past(row);
    blocks = (off + h + 7) / 8;
    const bool before = rows_before * stride >= 8, after = rows_after * stride >= 8;
#pragma unroll
    for (int c = 0; c < C + 1; ++c) {
      const int n = c * nt + tid, e0 = n * 8 - off;
      b[c] = make_uint4(0, 0, 0, 0);
      if (n >= blocks) continue;
      if ((e0 >= 0 || before) && (e0 + 8 <= h || after)) {
        b[c] = *reinterpret_cast<const uint4*>(p + e0);
      } else {
        // (all on their way at once: a loop over them, 1000 x 16383 59.5 us for 54.4)
        uint32_t e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = e0 + j >= 0 && e0 + j < h ? p[e0 + j] : 0;
        b[c] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
      }
    }
  }
  __device__ __forceinline__ void stage(uint4* buf, int tid, int nt) const {
#pragma unroll
    for (int c = 0; c < C + 1; ++c)
      if (c * nt + tid < blocks) buf[c * nt + tid] = b[c];
  }
};

// The 8 elements that begin `at` elements (0..7) into slot n, from two wide accesses, which no banks
// conflict in (word by word four neighbours meet in each), and selects by what is one number a row.
__device__ __forceinline__ uint4 elements_at(const uint4* buf, int n, int at) {
  const uint4 a = buf[n], b = buf[n + 1];
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 6; ++j) w[j] = at & 4 ? w[j + 2] : w[j];
#pragma unroll
  for (int j = 0; j < 5; ++j) w[j] = at & 2 ? w[j + 1] : w[j];
  const int bits = (at & 1) * 16;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                    __funnelshift_r(w[3], w[4], bits));
}

// chunk n of a staged row
template <typename E>
__device__ __forceinline__ void take_row(const uint4* buf, int n, int off, int h, float (&v)[8]) {
  const uint4 u = elements_at(buf, n, off);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack2<E>(w[j]);
    v[2 * j] = f.x, v[2 * j + 1] = f.y;
  }
  if (n * 8 + 8 > h) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (n * 8 + j >= h) v[j] = 0.0f;
  }
}

// buf holds the chunks of a row: write the row
__device__ __forceinline__ void store_row(void* row, const uint4* buf, int tid, int nt, int h) {
  const int off = halves_past(row), blocks = (off + h + 7) / 8;
  uint16_t* p = static_cast<uint16_t*>(row);
  for (int n = tid; n < blocks; n += nt) {
    const int e0 = n * 8 - off;
    if (e0 >= 0 && e0 + 8 <= h) {
      *reinterpret_cast<uint4*>(p + e0) = elements_at(buf, off ? n - 1 : n, off ? 8 - off : 0);
    } else {
#pragma unroll 1
      for (int e = max(e0, 0); e < min(e0 + 8, h); ++e) p[e] = reinterpret_cast<const uint16_t*>(buf)[e];
    }
  }
}
// codes likewise, in blocks of 8 bytes
__device__ __forceinline__ void store_codes(int8_t* p, const uint4* buf, int tid, int nt, int h) {
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 7u), blocks = (off + h + 7) / 8;
  for (int n = tid; n < blocks; n += nt) {
    const int e0 = n * 8 - off;
    if (e0 >= 0 && e0 + 8 <= h) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(buf) + (e0 >> 2);
      *reinterpret_cast<uint2*>(p + e0) =
          make_uint2(__funnelshift_r(w[0], w[1], (e0 & 3) * 8), __funnelshift_r(w[1], w[2], (e0 & 3) * 8));
    } else {
#pragma unroll 1
      for (int e = max(e0, 0); e < min(e0 + 8, h); ++e) p[e] = reinterpret_cast<const int8_t*>(buf)[e];
    }
  }
}

// 8 elements from i on, of an aligned row or of a vector that all rows share (16-byte loads where that is aligned)
template <typename E, bool VEC>
struct Chunk8 {
  uint32_t w[sizeof(E) * 2];
  __device__ __forceinline__ void load(const E* p, int i, int h) {
    const bool wide = VEC ? i < h : (i + 8 <= h && (reinterpret_cast<uintptr_t>(p) & 15u) == 0);
#pragma unroll
    for (int k = 0; k < static_cast<int>(sizeof(E) / 2); ++k) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (wide) u = reinterpret_cast<const uint4*>(p + i)[k];
      w[4 * k] = u.x, w[4 * k + 1] = u.y, w[4 * k + 2] = u.z, w[4 * k + 3] = u.w;
    }
    if (!VEC && !wide) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (i + j >= h) continue;
        if constexpr (sizeof(E) == 2) w[j >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i + j]) << ((j & 1) * 16);
        else w[j] = __float_as_uint(p[i + j]);
      }
    }
  }
  __device__ __forceinline__ void take(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(E) == 2) {
        const float2 f = unpack2<E>(w[j]);
        v[2 * j] = f.x, v[2 * j + 1] = f.y;
      } else {
        v[2 * j] = __uint_as_float(w[2 * j]), v[2 * j + 1] = __uint_as_float(w[2 * j + 1]);
      }
    }
  }
};

template <typename E>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack2<E>(v[0], v[1]), pack2<E>(v[2], v[3]), pack2<E>(v[4], v[5]), pack2<E>(v[6], v[7]));
}

// slots of one of the three buffers that a row that is not VEC has in shared memory
__host__ __device__ constexpr int row_slots(int c, int nt) { return c * nt + 2; }

}  // namespace
}  // namespace moe_layer
