// Declarations and device helpers shared by the decoder-layer operators
// (layer_api.cu checks arguments and launches; norm_quant.cu, w4_linear.cu,
// kv_append.cu and kv_attention.cu hold the kernels).
#pragma once

#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "moe_layer.h"

namespace moe_layer {

// Launch functions: arguments are checked, sizes are not zero.
cudaError_t launch_norm(const moe_layer_norm_args_t& a, int num_sms, cudaStream_t s);
cudaError_t launch_w4(const moe_layer_w4_args_t& a, int num_sms, cudaStream_t s);
cudaError_t launch_append(const moe_layer_kv_append_args_t& a, cudaStream_t s);
size_t attention_workspace(int head_dim, int num_sms);
cudaError_t launch_attention(const moe_layer_kv_attention_args_t& a, void* ws, int num_sms, cudaStream_t s);

// Lets `kernel` have `most` bytes of dynamic shared memory on the current
// device, asking the runtime once a device and kernel (`done`: one bit a device).
inline cudaError_t allow_smem(const void* kernel, int most, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}
constexpr int kMaxSmem = 227 * 1024;  // dynamic shared memory that a block can have, less what a kernel has of its own

// Launch that may begin while the stream's previous kernel still runs: every
// kernel here starts with grid_dependency_wait, before it touches memory.
inline cudaError_t launch_after(const void* kernel, dim3 grid, dim3 block, void** args, size_t smem, cudaStream_t s,
                                int cluster = 1) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

// Wait until the preceding grid of the stream has completed and its memory is
// visible; let the next grid be placed.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" :::); }

constexpr float kAmaxFloor = 1e-4f;  // floor of an amax before 127 / amax, as in the block's quant

// two 16-bit elements of one 32-bit word, widened
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// four fp32 -> int8 codes of one word, round half to even; NaN gives 0.  The
// conversion saturates at -128 and 127; quotients by amax / 127 stay within
// 127.0001 of zero, so -128 does not occur where that quotient is a normal number.
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d) {
  uint32_t hi, r;
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(hi) : "r"(__float2int_rn(d)), "r"(__float2int_rn(c)), "r"(0));
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(__float2int_rn(b)), "r"(__float2int_rn(a)), "r"(hi));
  return r;
}

// four int8 codes -> two pairs of fp16: (0, 1) and (2, 3)
__device__ __forceinline__ void half_pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t off = 0x64806480u;  // 1152
  const uint32_t l = __byte_perm(u, 0x64646464u, 0x4140), h = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&l), *reinterpret_cast<const __half2*>(&off));
  const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&off));
  lo = *reinterpret_cast<const uint32_t*>(&a);
  hi = *reinterpret_cast<const uint32_t*>(&b);
}

// |v| as ordered bits: the unsigned maximum of these is the maximum |v|, and
// a NaN is above every number
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float log2_fast(float v) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// asynchronous 16-byte copy global -> shared; `ok` false fills with zeros and reads nothing
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// every thread of a cluster: what was written before is seen after
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// the float at shared address `at` of CTA `rank` of the cluster
__device__ __forceinline__ float cluster_read(uint32_t at, uint32_t rank) {
  uint32_t remote;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

// shared-memory reads by address: plain loads, which the compiler may move between barriers
__device__ __forceinline__ uint4 lds128(uint32_t a) { return *static_cast<const uint4*>(__cvta_shared_to_generic(a)); }
__device__ __forceinline__ uint2 lds64(uint32_t a) { return *static_cast<const uint2*>(__cvta_shared_to_generic(a)); }
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  return *static_cast<const uint32_t*>(__cvta_shared_to_generic(a));
}

// D(16x8, f32) += A(16x16, row) * B(16x8, col), fp16.  Lane = 4 g + t.  A: a0 (row
// g, k 2t..2t+1), a1 (row g+8, same k), a2 (row g, k 2t+8..2t+9), a3 (row
// g+8); B: b0 (k 2t..2t+1, column g), b1 (k 2t+8..2t+9); D: d0 d1 (row g,
// columns 2t, 2t+1), d2 d3 (row g+8).
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with a zero accumulator
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

}  // namespace moe_layer
