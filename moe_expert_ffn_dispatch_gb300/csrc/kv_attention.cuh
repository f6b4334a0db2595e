// What the two attention kernels share: the division of the work over the
// CTAs, and the records of units that several CTAs hold.
#pragma once

#include "layer_ops.cuh"

namespace moe_layer {

struct Record {  // a unit that several CTAs share, left by the CTA that holds its last piece
  int b, head, rt;  // b < 0: none
  int c0, c1;       // its CTAs
};

struct AttnParams {
  moe_layer_kv_attention_args_t a;
  float* part_o;      // [2 * grid][rows of a unit][D]
  float* part_ml;     // [2 * grid][rows of a unit][2]
  Record* records;    // [grid]: of the unit that a CTA finished; or of each unit, where row_tiles > 0
  int row_tiles;      // a unit's number is (b * kv_heads + head) * row_tiles + rt
  int32_t* status;    // [4] words of the workspace: a wait that gave up is noted here
  float scale_log2;   // sm_scale * log2(e)
  int page_shift;
};

// With x a score times log2(e) and v the page scale of V, a row's running sums
// are
//   O = sum v 2^(x - M) V  and  l = sum 2^(x - M + kSumShift)
// with one reference M, that of the products v 2^x (taken of the weights 2^x
// alone, a page with a large v would push all others out of fp16's range).  Each
// v 2^(x - M) is rounded to fp16.  M moves so that none passes 2^kWeightMost and
// the largest lands at 2^kWeightLand: what is 2^-21 of the largest still has 11
// bits, and a step below that is 2^-31 of it.
// A warp measures v in units of 2^base, the smallest of the first scales that it meets.  While
// log2 v lies in [kScaleLeast, kScaleMost] of that, l is the sum of the products
// divided by v; a weight too small for fp32 in that form is below 2^-46 of the
// row's largest.  Other scales (0, negative ones, and all that come after one
// above kScaleMost) take an exponential more.  One below kScaleLeast counts as
// that in M, which holds l in range.
// Landing nearer to 2^kWeightMost keeps more and moves M more often: chunks of 512 tokens over 5011 take 99 us
// at 2^11, 95 at 2^8 and 93 at 2^5.
constexpr float kWeightLand = 8.0f, kWeightMost = 15.0f;
constexpr float kScaleLeast = -50.0f, kScaleMost = 40.0f, kSumShift = 31.0f;

// log2 of the unit of V's scales, from the smallest that a lane has (where `counts`) and that is neither 0 nor
// not finite; infinity where there is none
__device__ __forceinline__ float scale_base(float v, bool counts) {
  const uint32_t b = abs_bits(v), least = __reduce_min_sync(0xffffffffu, counts && b != 0 && b < 0x7F800000u ? b : 0x7F800000u);
  return least < 0x7F800000u ? fmaxf(floorf(log2_fast(__uint_as_float(least))), -126.0f) : INFINITY;
}

// A row's sums at the end: l in [1, 2) (or 0, or not finite) relative to m, and what makes O relative to it
__device__ __forceinline__ float settle(float& m, float& l, float base) {
  if (!(l > 0.0f && l < INFINITY)) {
    if (l == 0.0f) m = -INFINITY;
    return 1.0f;
  }
  const int e = static_cast<int>(__float_as_uint(l) >> 23) - 127;
  l = __uint_as_float((__float_as_uint(l) & 0x7FFFFFu) | 0x3F800000u);
  m = __fadd_rn(m, static_cast<float>(e) - kSumShift);
  return exp2_fast(__fadd_rn(base, kSumShift - static_cast<float>(e)));
}

// What a sequence contributes, from its lengths.
struct SeqShape {
  int q0, qlen;     // query tokens that are computed
  int len;          // keys
  int pos0;         // position of query token q0: negative where there are more query tokens than keys
};

__device__ __forceinline__ SeqShape seq_shape(const moe_layer_kv_attention_args_t& a, int b) {
  SeqShape s;
  int end = b + 1;  // of the sequence's query tokens, those past max_q among them: the last stands at len - 1
  if (a.cu_q) {
    end = max(a.cu_q[b + 1], 0);
    s.q0 = min(max(a.cu_q[b], 0), a.tokens);
    s.qlen = min(max(min(end, a.tokens) - s.q0, 0), a.max_q);
  } else {
    s.q0 = b;
    s.qlen = 1;
  }
  const int64_t most = static_cast<int64_t>(a.max_pages) * a.cache.page_size;
  s.len = static_cast<int>(min(static_cast<int64_t>(max(a.seq_lens[b], 0)), most));
  s.pos0 = s.len - max(end - s.q0, 0);
  return s;
}

// Keys that the rows of tile rt (R rows) of a sequence see: [lo, hi)
struct KeyRange {
  int lo, hi;
};
template <int R>
__device__ __forceinline__ KeyRange keys_of(const moe_layer_kv_attention_args_t& a, const SeqShape& s, int rt) {
  const int64_t pos0 = s.pos0;
  const int last_row = min((rt + 1) * R, s.qlen * a.group_size) - 1;
  KeyRange k;
  k.hi = static_cast<int>(max(static_cast<int64_t>(0), pos0 + last_row / a.group_size + 1));
  k.lo = 0;
  if (a.window > 0)
    k.lo = static_cast<int>(min(max(static_cast<int64_t>(0), pos0 + rt * R / a.group_size - a.window + 1),
                                static_cast<int64_t>(k.hi)));
  return k;
}

// A stretch of a unit's pieces that one CTA takes.
struct Segment {
  int b, head, rt, rows;  // rows: query rows of the unit
  int tile0, tiles;       // the unit's pieces of TILE keys: the first, how many (1 at least)
  int ta, tb;             // of them, this stretch
  SeqShape s;
  KeyRange keys;          // that any row sees
  int64_t first_piece;    // where the unit's first piece lies in the sequence of work
};

// The work of all units (sequence, kv head, tile of R rows) in a row: each
// costs its pieces of TILE keys and COST more (its queries, a cold pipeline,
// the join).  CTA c of G takes [total c / G, total (c + 1) / G) of it.
template <int R, int TILE, int COST>
struct Schedule {
  int64_t* prefix;  // shared memory: [batch + 1]
  int4* shapes;     // shared memory: [batch], q0, qlen, len, pos0
  int64_t total, begin, end;  // of all the work; this CTA's
  int G;

  static __device__ __forceinline__ int pieces(const KeyRange& k) {
    return max(1, (k.hi + TILE - 1) / TILE - k.lo / TILE);
  }

  static __host__ __device__ size_t bytes(int batch) { return static_cast<size_t>(batch + 2) / 2 * 16 + batch * 16; }

  // by every thread of the CTA; carry: shared, one entry a warp
  template <int THREADS>
  __device__ __forceinline__ void build(const moe_layer_kv_attention_args_t& a, uint8_t* mem, int64_t* carry) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    prefix = reinterpret_cast<int64_t*>(mem);
    shapes = reinterpret_cast<int4*>(mem + (a.batch + 2) / 2 * 16);
    if (tid == 0) prefix[0] = 0;
    int64_t run = 0;
    for (int base = 0; base < a.batch; base += THREADS) {
      const int b = base + tid;
      int64_t v = 0;
      if (b < a.batch) {
        const SeqShape s = seq_shape(a, b);
        const int row_tiles = (s.qlen * a.group_size + R - 1) / R;
        int64_t one = 0;  // of one head
        for (int rt = 0; rt < row_tiles; ++rt) one += pieces(keys_of<R>(a, s, rt)) + COST;
        v = a.cache.kv_heads * one;
        shapes[b] = make_int4(s.q0, s.qlen, s.len, s.pos0);
      }
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (lane == 31) carry[warp] = v;
      __syncthreads();
      int64_t before = run, all = run;
      for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += carry[w];
        all += carry[w];
      }
      if (b < a.batch) prefix[b + 1] = before + v;
      run = all;
      __syncthreads();
    }
    total = run;
    G = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total));
    const int c = blockIdx.x;
    begin = c < G ? total * c / G : 0;
    end = c < G ? total * (c + 1) / G : 0;
  }

  // the stretch at `at`, which starts at `begin` and is moved on; false at the end
  __device__ __forceinline__ bool next(const moe_layer_kv_attention_args_t& a, int64_t& at, Segment& g) const {
    while (at < end) {
      int lo = 0, hi = a.batch;  // the b with prefix[b] <= at < prefix[b + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= at) lo = mid;
        else hi = mid;
      }
      const int4 sh = shapes[lo];
      g.b = lo;
      g.s.q0 = sh.x, g.s.qlen = sh.y, g.s.len = sh.z, g.s.pos0 = sh.w;
      const int64_t rel = at - prefix[lo], one = (prefix[lo + 1] - prefix[lo]) / a.cache.kv_heads;
      g.head = static_cast<int>(rel / one);
      int64_t rem = rel - g.head * one;
      g.rt = 0;
      while (true) {  // the unit of this head that holds `rem`
        g.keys = keys_of<R>(a, g.s, g.rt);
        g.tiles = pieces(g.keys);
        if (rem < g.tiles + COST) break;
        rem -= g.tiles + COST;
        ++g.rt;
      }
      g.tile0 = g.keys.lo / TILE;
      const int xa = static_cast<int>(rem), xb = static_cast<int>(min(static_cast<int64_t>(g.tiles + COST), xa + (end - at)));
      g.ta = max(0, xa - COST);
      g.tb = max(0, xb - COST);
      g.rows = min(R, g.s.qlen * a.group_size - g.rt * R);
      g.first_piece = at - xa + COST;
      at += xb - xa;
      if (g.tb > g.ta) return true;
    }
    return false;
  }

  // unit u of all that the shapes of the call allow, whole; false where this sequence has no such rows
  static __device__ __forceinline__ bool unit(const moe_layer_kv_attention_args_t& a, int u, Segment& g) {
    const int row_tiles = static_cast<int>((static_cast<int64_t>(a.max_q) * a.group_size + R - 1) / R);
    g.rt = u % row_tiles;
    g.head = u / row_tiles % a.cache.kv_heads;
    g.b = u / row_tiles / a.cache.kv_heads;
    g.s = seq_shape(a, g.b);
    g.rows = min(R, g.s.qlen * a.group_size - g.rt * R);
    if (g.rows <= 0) return false;
    g.keys = keys_of<R>(a, g.s, g.rt);
    g.tile0 = g.keys.lo / TILE;
    g.tiles = pieces(g.keys);
    g.ta = 0;
    g.tb = g.tiles;
    g.first_piece = 0;
    return true;
  }

  // the CTA that holds piece x: the last c with total c / G <= x
  __device__ __forceinline__ int cta_of(int64_t x) const {
    int64_t c = x * G / total;
    while (c + 1 < G && total * (c + 1) / G <= x) ++c;
    while (c > 0 && total * c / G > x) --c;
    return static_cast<int>(c);
  }
};

// Joins the parts of units that several CTAs shared (kv_attention.cu).  records: how many there are; rows: the
// most that a unit has; JW: warps that share a row's parts.
template <typename T, int D, int R, int JW>
cudaError_t launch_join(const AttnParams& p, int records, int rows, cudaStream_t s);

// kv_attention_chunk.cu: tensor-memory kernel for many query rows a kv head.
constexpr int kChunkRows = 256;
template <typename T, int D>
cudaError_t launch_chunk(const AttnParams& p, int num_sms, cudaStream_t s);
bool chunk_fits(int head_dim, int batch);  // its shared memory, which the batch's lengths share

}  // namespace moe_layer
