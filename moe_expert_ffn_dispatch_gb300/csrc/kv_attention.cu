// Attention of new tokens over the paged INT8 cache: the kernel for few query
// rows, the join of shared units, and the choice between the kernels.
//
// The query rows of one kv head (query tokens x group_size) are cut into
// tiles of 8 or 16.  A unit is (sequence, kv head, row tile).  The host knows
// how many there can be and how many keys a page table has room for, not the
// lengths, and by these takes one of two forms:
//
// Whole units, where a table or the window is short: a cluster of 8, 4, 2 or 1 CTAs, as many
// as let all units run at once, takes a unit, deals its slices out to the
// warps and joins them over distributed shared memory.  One launch: 1 context
// of 1009 tokens 5.2 us (the other form 9.3), 64 of 500 14.3 (23), 256 of 100 20
// (32).
//
// A schedule, where tables are long, for then one context may be far longer
// than the others: a unit's keys are cut into pieces of kTileTokens, all pieces
// of all units form one sequence of work, and the CTAs share it evenly, whatever
// the lengths are.  A CTA takes consecutive pieces, so only the first and the
// last unit that it meets can be shared with other CTAs.  Those leave (row
// reference, row sum, unnormalised output) in the workspace, and a second
// kernel joins them in CTA order.  64 contexts, one of 2000 tokens and the others
// of 50: 12.6 us (whole units 28); from 768 keys a CTA on the whole form loses on
// such lengths and wins on even ones (64 of 2000: 46 us for 52).
//
// Within a CTA each of 4 warps streams its own 16-token slices of keys and
// values through a ring of asynchronous copies and keeps a running softmax of
// its own (no barrier in the loop); the warps join in shared memory at the end
// of a unit.  Several small CTAs an SM hide one another's cold starts: 4 of
// them at 8 rows, 3 at 16 (8-warp CTAs, one an SM: 71 us where these take 52).
//
// Both products are transposed, S^T = K Q^T and O^T = V^T P^T (mma.sync
// m16n8k16, fp32 accumulators): tokens and channels are the 16-wide M side, 8
// query rows the N side, so 8 rows fill what they occupy (with rows on the M
// side the same kernel took 84 us where this one takes 68).  The weights turn
// from one layout into the other by movmatrix.  (The same shape on the
// tensor-memory product, keys as its 128-wide side and 8 rows as N, has not been
// built: each code would still be converted here, and written to tensor memory.)
//
// Arithmetic: the int8 codes become exact fp16 (a byte set into the mantissa
// of 1024, minus 1152).  A query row is scaled by a power of two to [1, 2) at
// its largest element, so bf16 rows are exact in fp16 as far as an fp32 sum
// can tell.  With x the scores times log2(e), the page scale of K and the
// row's power of two enter x in fp32.  The page scale of V enters the weight of
// the second product, which is rounded to fp16: 11 bits, where the output has 8
// or 11 (kv_attention.cuh).  Sums of weights are taken before that rounding, in
// fp32.
// Both products let the k index run over channels (or tokens) in whatever
// order makes shared-memory reads whole 16-byte chunks: a permuted sum is the
// same sum.
//
// Bound by the cache's bytes at 8 rows (two contexts of 200003 and 100000
// tokens, 8 kv heads of 128, 4 rows each: 100 us, 6.1 TB/s of 6.8; heads of 64:
// 59 us, 5.2 TB/s), by instructions at 16 (64 contexts of 2000 tokens: 77 us, 3.4
// TB/s).  More rows than 16 take more units, which convert every key again: 16
// contexts of 4000 tokens with 2 query tokens of 4 rows 32 us, with 4 46, with 8
// 70.
#include <climits>

#include "kv_attention.cuh"

namespace moe_layer {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSlice = 16;                       // tokens of a warp's ring stage
constexpr int kTileTokens = kSlice * kWarps;     // tokens of a piece of work
// NR: blocks of 8 query rows that a unit holds.  One block leaves registers for 16 warps on an SM, two for 12.
template <int NR>
constexpr int kCtasPerSm = NR == 1 ? 4 : 3;
template <int NR>
constexpr int kStagesOf = NR == 1 ? 3 : 4;
constexpr int kMaxSlots = 4096;                  // CTAs of a launch (at most 4 an SM)
// what a unit costs beside its pieces (its queries, a cold ring, the join of the warps), in pieces.  64 ragged
// contexts with 0, 2, 4 or 8: 69, 36.9, 33.8 and 36.8 us; 64 even ones of 2000 tokens 53.0, 52.4, 52.1 and 51.6.
constexpr int kUnitCost = 4;
// A cluster of CTAs takes a whole unit where the table (or the window) leaves no more keys than this for each of them
constexpr int kWholeKeys = 768;
constexpr int kWholeUnits = 1 << 20;  // a grid's size stays far below 2^31
// Query rows of a kv head (the longest sequence's) from which the tensor-memory kernel takes over.  Its time
// hardly depends on them up to 128, this kernel's grows with every 16.  us here / there at 32, 48, 64, 96 and 128
// rows: 16 contexts of 4000 tokens 70/91, 95/92, 118/93, 166/95, 212/97; 64 of 500 39/73, 57/74, 72/76, 105/78,
// 135/83; 4 of 2000 19/28, 19/29, 32/29, 39/30, 46/30; 1 of 4000 15/24, 15/24, 19/25, 19/26, 30/27.
constexpr int kChunkFrom = 64;

// position of channel chunk `c` (16 bytes) of token row `r` in a slice of [16][D] bytes
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  else return r * 64 + ((c ^ (((r >> 2) & 1) << 1)) << 4);
}
// token (0..7) of score column n (0..7).  D = 64: two rows share a 128-byte
// line, and this order puts the rows that are read together on other banks.
template <int D>
__device__ __forceinline__ int token_of(int n) {
  if constexpr (D == 128) return n;
  else return n ^ ((n >> 1) & 1);
}

// 8x8 matrix of 16-bit elements, transposed: lane 4 g + t gives (g, 2t..2t+1) and gets (2t..2t+1, g)
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// CS 0: the CTAs divide the work of all units by the schedule.  Otherwise a
// cluster of CS CTAs takes a unit, all of its pieces, and joins its parts itself.
template <typename T, int D, int NR, int CS>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<NR>) kv_attention_kernel(const AttnParams p) {
  constexpr int KS = D / 16;                   // k steps of the score product
  constexpr int NT = D / 16;                   // channel tiles of the output
  constexpr int R = 8 * NR;                    // rows of a unit
  constexpr int kStages = kStagesOf<NR>;
  constexpr int kSliceBytes = kSlice * D;      // of K; V follows
  constexpr int kStageBytes = 2 * kSliceBytes;
  constexpr int kRing = kStages * kStageBytes;
  constexpr int kCopies = kSliceBytes / 16 / 32;  // 16-byte copies of a lane for K (and for V)
  static_assert(kRing >= R * D * 4 + 8 * R, "the join reuses the ring");
  extern __shared__ __align__(128) uint8_t smem[];
  grid_dependency_wait();
  grid_launch_dependents();
  const moe_layer_kv_attention_args_t& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  using Work = Schedule<R, kTileTokens, kUnitCost>;
  Work work;
  constexpr int kShare = CS > 1 ? CS : 1;  // CTAs that share a unit's slices
  const int c = blockIdx.x, rank = c % kShare;
  if (c == 0 && tid == 0) p.status[1] = p.status[2] = 0;  // no wait of this kernel can give up
  if constexpr (CS == 0) {
    __shared__ int64_t s_carry[kWarps];
    work.template build<kThreads>(a, smem + kWarps * kRing, s_carry);
    if (tid == 0 && p.row_tiles == 0) p.records[c].b = -1;
  }

  uint8_t* ring = smem + warp * kRing;
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));

  Segment seg;
  int64_t at = 0;
  if constexpr (CS == 0) {
    at = work.begin;
  } else {
    if (!work.unit(a, c / kShare, seg)) return;  // the same for the whole cluster
  }
  while (CS > 0 || work.next(a, at, seg)) {
    const SeqShape& s = seg.s;
    const int b = seg.b, head = seg.head, rt = seg.rt, rows = seg.rows, ta = seg.ta, tb = seg.tb;
    const int64_t pos0 = s.pos0;
    // keys that any row of the tile sees, cut to this CTA's pieces
    const int64_t last = pos0 + (rt * R + rows - 1) / a.group_size;
    int64_t k_lo = static_cast<int64_t>(seg.tile0 + ta) * kTileTokens;
    const int64_t k_hi = min(static_cast<int64_t>(seg.tile0 + tb) * kTileTokens, static_cast<int64_t>(seg.keys.hi));
    k_lo = max(k_lo, static_cast<int64_t>(seg.keys.lo & ~(kSlice - 1)));
    // this warp's slices: first + kSpread i, from the slice of k_lo on
    constexpr int kSpread = kWarps * kShare;
    const int first = static_cast<int>(k_lo / kSlice) + rank * kWarps + warp;
    const int n = k_hi > static_cast<int64_t>(first) * kSlice
                      ? static_cast<int>(((k_hi + kSlice - 1) / kSlice - first + kSpread - 1) / kSpread)
                      : 0;

    // keys [all_lo, all_hi) are seen by every row of the tile; n_all: slices of
    // this warp that end there need no mask (rows past the last take part
    // with zero queries and are not stored)
    const int64_t all_hi = pos0 + rt * R / a.group_size + 1;
    const int64_t all_lo = a.window > 0 ? last - a.window + 1 : 0;

    // page, and scales, of the slices 32 at a time: lane i holds slice base + i
    auto look_up = [&](int base, int& page, float& ks, float& vs) {
      page = -1;
      ks = vs = 0.0f;
      const int i = base + lane;
      if (i < n) {
        const int64_t tok = static_cast<int64_t>(first + i * kSpread) * kSlice;
        const int pg = a.page_table[b * a.table_stride + (tok >> p.page_shift)];
        if (pg >= 0 && pg < a.cache.num_pages) {
          page = pg;
          ks = a.cache.k_scale[pg * a.cache.scale_stride + head];
          vs = a.cache.v_scale[pg * a.cache.scale_stride + head];
        }
      }
    };
    // log2 of the scales of V of the slices that come next, in units of 2^unit; infinity stands for any
    // that is not between kScaleLeast and kScaleMost, or beside a scale of K that is not finite
    float unit = INFINITY;
    auto log_scale = [&](int page, float ks, float vs) {
      if (unit == INFINITY) unit = scale_base(vs, true);
      const float lv = __fsub_rn(log2_fast(vs), unit);
      return page < 0 ? 0.0f : lv >= kScaleLeast && lv <= kScaleMost && fabsf(ks) < INFINITY ? lv : INFINITY;
    };
    int page0, page1;
    float ks0, vs0, ks1, vs1, lv0;
    look_up(0, page0, ks0, vs0);
    look_up(32, page1, ks1, vs1);
    const int in_page = a.cache.page_size - 1;
    const int8_t* k_head = a.cache.k + head * a.cache.head_stride + lane * 16;
    const int8_t* v_head = a.cache.v + head * a.cache.head_stride + lane * 16;
    // where this lane's copies of a slice go: the rows of copy x lie 512 bytes after those of copy x - 1, at the
    // same place in the swizzle or (D = 128) at the place that differs by 4 chunks
    const uint32_t to0 = chunk_at<D>(lane / (D / 16), lane % (D / 16));
    auto to = [&](int x) { return D == 128 ? (x & 1 ? to0 ^ 64u : to0) + x * 512 : to0 + x * 512; };
    auto issue = [&](int i, int rel_i) {  // slice i of this warp, rel_i from the base of page0
      const int page = rel_i < 32 ? __shfl_sync(0xffffffffu, page0, rel_i & 31) : __shfl_sync(0xffffffffu, page1, rel_i & 31);
      if (i < n) {
        const int64_t off = max(page, 0) * a.cache.page_stride + (((first + i * kSpread) * kSlice) & in_page) * D;
        const int8_t *kp = k_head + off, *vp = v_head + off;
        const uint32_t dst = ring_u + (i % kStages) * kStageBytes;
#pragma unroll
        for (int x = 0; x < kCopies; ++x) {
          cp_async16(dst + to(x), kp + x * 512, page >= 0);
          cp_async16(dst + kSliceBytes + to(x), vp + x * 512, page >= 0);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, i);

    // ---- rows of this tile: row r is query token r / group of the sequence
    int row_pos[NR][2];          // positions of rows 2t and 2t + 1 of each block, -1 past the last row
    float row_scale[NR][2];
    uint32_t qf[NR][KS][2];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const int r = g + 8 * nr, row = rt * R + r;
      const int j = row / a.group_size, hq = row - j * a.group_size;
      // lane t holds channels [t D / 4, (t + 1) D / 4) of row g of the block
      uint32_t w[KS * 2];
      if (r < rows) {
        const T* src = static_cast<const T*>(a.q) + static_cast<int64_t>(s.q0 + j) * a.q_stride +
                       static_cast<int64_t>(head * a.group_size + hq) * D + t * (D / 4);
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) {
          const uint4 u = reinterpret_cast<const uint4*>(src)[i];
          w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < KS * 2; ++i) w[i] = 0u;
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < KS * 2; ++i) {
        const float2 f = unpack2<T>(w[i]);
        top = max(top, max(abs_bits(f.x), abs_bits(f.y)));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // exponent of the largest element, inside what 2^-e can hold
      const int e = min(max(static_cast<int>(top >> 23), 1), 253);
      const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^(127 - e)
      // a query that is not finite makes every score NaN: scores of minus infinity alone would hide it
      const float up = top < 0x7F800000u ? __fmul_rn(__uint_as_float(static_cast<uint32_t>(e) << 23), p.scale_log2) : NAN;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const float2 f0 = unpack2<T>(w[2 * i]), f1 = unpack2<T>(w[2 * i + 1]);
        qf[nr][i][0] = pack2<__half>(__fmul_rn(f0.x, down), __fmul_rn(f0.y, down));
        qf[nr][i][1] = pack2<__half>(__fmul_rn(f1.x, down), __fmul_rn(f1.y, down));
      }
      const int pos = r < rows ? static_cast<int>(max(pos0 + j, static_cast<int64_t>(-1))) : -1;
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        row_scale[nr][e2] = __shfl_sync(0xffffffffu, up, (2 * t + e2) * 4);
        row_pos[nr][e2] = __shfl_sync(0xffffffffu, pos, (2 * t + e2) * 4);
      }
    }
    // whether a row sees this lane's key of a half slice: as many tokens back as the window has, or any (32 bits
    // do, as a key in front of the row is a large number without its sign)
    const uint32_t reach = a.window > 0 ? a.window : INT_MAX;
    auto sees = [&](int pos, int half, int64_t tok0) {
      return static_cast<uint32_t>(pos) - (static_cast<uint32_t>(tok0) + half * 8 + token_of<D>(g)) < reach;
    };
    float o[NR][NT][4];  // transposed: channels g D / 8 + 2 i and + 1 of column tile i, rows 2t and 2t + 1
    float m[NR][2], l[NR][2];
    bool far = false;  // a scale of V above kScaleMost has been met
    lv0 = log_scale(page0, ks0, vs0);
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
      for (int i = 0; i < NT; ++i) o[nr][i][0] = o[nr][i][1] = o[nr][i][2] = o[nr][i][3] = 0.0f;
      m[nr][0] = m[nr][1] = -INFINITY;
      l[nr][0] = l[nr][1] = 0.0f;
    }

    for (int i = 0; i < n; ++i) {
      const int ri = i & 31;
      if (ri == 0 && i > 0) {
        page0 = page1, ks0 = ks1, lv0 = log_scale(page1, ks1, vs1);
        look_up(i + 32, page1, ks1, vs1);
      }
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const uint32_t kb = ring_u + (i % kStages) * kStageBytes, vb = kb + kSliceBytes;
      const int page = __shfl_sync(0xffffffffu, page0, ri);
      const float ks = __shfl_sync(0xffffffffu, ks0, ri);
      float lv = __shfl_sync(0xffffffffu, lv0, ri);
      const int64_t tok0 = static_cast<int64_t>(first + i * kSpread) * kSlice;

      // scores, transposed: 16 tokens x 8 NR rows, in two chains of products
      float sc[NR][4], s2[NR][4];
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nr][e] = s2[nr][e] = 0.0f;
      {
        uint32_t w[2][KS];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = h * 8 + token_of<D>(g);
          if constexpr (D == 128) {
            const uint4 x = lds128(kb + chunk_at<D>(r, 2 * t)), y = lds128(kb + chunk_at<D>(r, 2 * t + 1));
            w[h][0] = x.x, w[h][1] = x.y, w[h][2] = x.z, w[h][3] = x.w;
            w[h][4] = y.x, w[h][5] = y.y, w[h][6] = y.z, w[h][7] = y.w;
          } else {
            const uint4 x = lds128(kb + chunk_at<D>(r, t));
            w[h][0] = x.x, w[h][1] = x.y, w[h][2] = x.z, w[h][3] = x.w;
          }
        }
#pragma unroll
        for (int q = 0; q < KS; ++q) {
          uint32_t a0, a1, a2, a3;
          half_pairs(w[0][q], a0, a2);
          half_pairs(w[1][q], a1, a3);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
            mma16816(q & 1 ? s2[nr] : sc[nr], a0, a1, a2, a3, qf[nr][q][0], qf[nr][q][1]);
        }
      }
      // x = score * scales * log2(e), masked where a row does not see the whole slice
      const bool whole = page >= 0 && tok0 >= all_lo && tok0 + kSlice <= all_hi;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sc[nr][e] = __fmul_rn(__fadd_rn(sc[nr][e], s2[nr][e]), __fmul_rn(ks, row_scale[nr][e & 1]));
      if (!whole) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (page < 0 || !sees(row_pos[nr][e & 1], e >> 1, tok0)) sc[nr][e] = -INFINITY;
          }
      }
      // The references move only when a product would pass what fp16 is to
      // hold: most slices rescale nothing.
      uint32_t sign = 0;
      float top[NR][2], rv = exp2_fast(__fsub_rn(kSumShift, lv));
      const bool odd = far || lv == INFINITY;
      bool move = odd;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[nr][e] = fmaxf(sc[nr][e], sc[nr][2 + e]);
          move |= top[nr][e] > m[nr][e] + (kWeightMost - lv);
        }
      if (__builtin_expect(__any_sync(0xffffffffu, move), 0)) {
        float lr = lv;
        if (odd && page >= 0) {
          const float k1 = a.cache.k_scale[page * a.cache.scale_stride + head], v1 = a.cache.v_scale[page * a.cache.scale_stride + head];
          rv = 0.0f;
          lv = __fsub_rn(log2_fast(fabsf(v1)), unit);
          if (v1 < 0.0f) sign = 0x80008000u;
          if (!(fabsf(k1) < INFINITY && fabsf(v1) < INFINITY)) {
            // a scale that is not finite makes the rows that see the page NaN, through
            // their sums, and stays out of what the rows share
            lv = -INFINITY;
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (sees(row_pos[nr][e & 1], e >> 1, tok0)) l[nr][e & 1] = NAN;
                sc[nr][e] = top[nr][e & 1] = -INFINITY;
              }
          }
          lr = fmaxf(lv, kScaleLeast);
          far = far || lv > kScaleMost;
        }
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          float corr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top[nr][e] = fmaxf(top[nr][e], __shfl_xor_sync(0xffffffffu, top[nr][e], x));
            const float mn = fmaxf(m[nr][e], __fadd_rn(top[nr][e], lr - kWeightLand));
            corr[e] = mn == m[nr][e] ? 1.0f : exp2_fast(__fsub_rn(m[nr][e], mn));
            m[nr][e] = mn;
            l[nr][e] = __fmul_rn(l[nr][e], corr[e]);
          }
#pragma unroll
          for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nr][q][e] = __fmul_rn(o[nr][q][e], corr[e & 1]);
          if (odd) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = __fsub_rn(sc[nr][e], m[nr][e & 1] == -INFINITY ? 0.0f : m[nr][e & 1]);
              l[nr][e & 1] = __fadd_rn(l[nr][e & 1], exp2_fast(__fadd_rn(x, kSumShift)));
            }
          }
        }
      }
      uint32_t pb[NR][2];  // weights: tokens 2t.. (and 2t + 8..) of row g
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float by = __fsub_rn(lv, m[nr][e] == -INFINITY ? 0.0f : m[nr][e]);
          sc[nr][e] = exp2_fast(__fadd_rn(sc[nr][e], by));
          sc[nr][2 + e] = exp2_fast(__fadd_rn(sc[nr][2 + e], by));
          l[nr][e] = __fmaf_rn(__fadd_rn(sc[nr][e], sc[nr][2 + e]), rv, l[nr][e]);
        }
        pb[nr][0] = transpose8x8(pack2<__half>(sc[nr][0], sc[nr][1]) ^ sign);
        pb[nr][1] = transpose8x8(pack2<__half>(sc[nr][2], sc[nr][3]) ^ sign);
      }
      // values: lane row g holds channels [g D / 8, (g + 1) D / 8), two a channel tile
      uint32_t w[4][NT / 2];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = (q >> 1) * 8 + token_of<D>(2 * t + (q & 1));
        if constexpr (D == 128) {
          const uint4 x = lds128(vb + chunk_at<D>(r, g));
          w[q][0] = x.x, w[q][1] = x.y, w[q][2] = x.z, w[q][3] = x.w;
        } else {
          const uint2 x = lds64(vb + chunk_at<D>(r, g >> 1) + (g & 1) * 8);
          w[q][0] = x.x, w[q][1] = x.y;
        }
      }
#pragma unroll
      for (int q = 0; q < NT / 2; ++q) {
        // bytes of tokens (2t, 2t + 1) side by side, then (2t + 8, 2t + 9)
        uint32_t lo0, lo1, lo2, lo3, hi0, hi1, hi2, hi3;
        half_pairs(__byte_perm(w[0][q], w[1][q], 0x5140), lo0, lo1);
        half_pairs(__byte_perm(w[0][q], w[1][q], 0x7362), lo2, lo3);
        half_pairs(__byte_perm(w[2][q], w[3][q], 0x5140), hi0, hi1);
        half_pairs(__byte_perm(w[2][q], w[3][q], 0x7362), hi2, hi3);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          mma16816(o[nr][2 * q], lo0, lo1, hi0, hi1, pb[nr][0], pb[nr][1]);
          mma16816(o[nr][2 * q + 1], lo2, lo3, hi2, hi3, pb[nr][0], pb[nr][1]);
        }
      }
      __syncwarp();  // the stage is read before it is filled again
      issue(i + kStages - 1, ri + kStages - 1);
    }
    cp_async_wait<0>();
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], x);
    __syncwarp();

    // ---- join the warps: O [R][D], then m [R], l [R] in each warp's ring
    float* wo = reinterpret_cast<float*>(ring);
    float* wm = wo + R * D;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nr * 8 + 2 * t + e;
        const float by = settle(m[nr][e], l[nr][e], unit == INFINITY ? 0.0f : unit);
#pragma unroll
        for (int q = 0; q < NT; ++q)
          *reinterpret_cast<float2*>(wo + r * D + g * (D / 8) + 2 * q) =
              make_float2(__fmul_rn(o[nr][q][e], by), __fmul_rn(o[nr][q][2 + e], by));
        if (g == 0) wm[r] = m[nr][e], wm[R + r] = l[nr][e];
      }
    __syncthreads();
    constexpr int kPerRow = kThreads / R, kEach = D / kPerRow;
    const int r = tid / kPerRow;
    float top = -INFINITY;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, reinterpret_cast<float*>(smem + w * kRing)[R * D + r]);
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, acc[kEach] = {};
    const int d0 = (tid % kPerRow) * kEach;
    for (int w = 0; w < kWarps; ++w) {
      const float* from = reinterpret_cast<float*>(smem + w * kRing);
      const float f = exp2_fast(__fsub_rn(from[R * D + r], base));
      sum = __fmaf_rn(from[R * D + R + r], f, sum);
#pragma unroll
      for (int i = 0; i < kEach; ++i) acc[i] = __fmaf_rn(from[r * D + d0 + i], f, acc[i]);
    }
    if constexpr (CS > 1) {
      // the CTA's part in place of its first warp's; each CTA joins R / CS rows
      static_assert(R % CS == 0, "");
      __syncthreads();
      float* mine = reinterpret_cast<float*>(smem);
#pragma unroll
      for (int i = 0; i < kEach; ++i) mine[r * D + d0 + i] = acc[i];
      if (tid % kPerRow == 0) mine[R * D + r] = top, mine[R * D + R + r] = sum;
      cluster_sync();
      const uint32_t part = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
      for (int i = tid; i < R / CS * (D / 2); i += kThreads) {  // two channels of a row
        const int jr = rank * (R / CS) + i / (D / 2), ch = i % (D / 2) * 2;
        if (jr >= rows) continue;
        float m1[CS], l1[CS], x1[CS], y1[CS];
#pragma unroll
        for (int w = 0; w < CS; ++w) {
          m1[w] = cluster_read(part + (R * D + jr) * 4, w);
          l1[w] = cluster_read(part + (R * D + R + jr) * 4, w);
          x1[w] = cluster_read(part + (jr * D + ch) * 4, w);
          y1[w] = cluster_read(part + (jr * D + ch + 1) * 4, w);
        }
        float most = -INFINITY, total = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 0; w < CS; ++w) most = fmaxf(most, m1[w]);
        const float from = most == -INFINITY ? 0.0f : most;
#pragma unroll
        for (int w = 0; w < CS; ++w) {
          const float f = exp2_fast(__fsub_rn(m1[w], from));
          total = __fmaf_rn(l1[w], f, total);
          x = __fmaf_rn(x1[w], f, x);
          y = __fmaf_rn(y1[w], f, y);
        }
        const int row = rt * R + jr, j = row / a.group_size, hq = row - j * a.group_size;
        const float inv = total > 0.0f ? __fdiv_rn(1.0f, total) : (total == 0.0f ? 0.0f : total);
        T* out = static_cast<T*>(a.out) +
                 (static_cast<int64_t>(s.q0 + j) * a.cache.kv_heads * a.group_size + head * a.group_size + hq) * D + ch;
        *reinterpret_cast<uint32_t*>(out) = pack2<T>(__fmul_rn(x, inv), __fmul_rn(y, inv));
      }
      cluster_sync();  // the parts are read before their CTA ends
      return;
    } else if (CS == 1 || (ta == 0 && tb == seg.tiles)) {
      if (CS == 0 && tid == 0 && p.row_tiles > 0) p.records[(b * a.cache.kv_heads + head) * p.row_tiles + rt].b = -1;
      if (r < rows) {
        const int row = rt * R + r, j = row / a.group_size, hq = row - j * a.group_size;
        const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : (sum == 0.0f ? 0.0f : sum);
        T* out = static_cast<T*>(a.out) +
                 (static_cast<int64_t>(s.q0 + j) * a.cache.kv_heads * a.group_size + head * a.group_size + hq) * D + d0;
#pragma unroll
        for (int i = 0; i < kEach; i += 2)
          *reinterpret_cast<uint32_t*>(out + i) = pack2<T>(__fmul_rn(acc[i], inv), __fmul_rn(acc[i + 1], inv));
      }
      if (CS == 1) return;
    } else {
      const int64_t slot = 2 * static_cast<int64_t>(c) + (ta > 0 ? 0 : 1);
      float* po = p.part_o + (slot * R + r) * D + d0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) po[i] = acc[i];
      if (tid % kPerRow == 0) {
        p.part_ml[(slot * R + r) * 2] = top;
        p.part_ml[(slot * R + r) * 2 + 1] = sum;
      }
      if (tb == seg.tiles && tid == 0) {
        const int at_record = p.row_tiles > 0 ? (b * a.cache.kv_heads + head) * p.row_tiles + rt : c;
        p.records[at_record] = Record{b, head, rt, work.cta_of(seg.first_piece), c};
      }
    }
    __syncthreads();
  }
}

}  // namespace

namespace {

// Joins the parts of a unit that several CTAs shared.  CTA (i, y) takes 16 /
// JW rows of the unit of record i, JW warps a row: a warp sums every JW-th
// part, a lane D / 32 channels, and the JW sums are added in a fixed
// order.  The maxima are read first, so that the parts' loads depend on
// nothing but their addresses.  Few units have many parts each (JW = 16,
// records by unit: the CTAs of most records would have nothing to do), many
// units few (JW = 4), units of 256 rows two or three (JW = 1).
constexpr int kJoinThreads = 512;
template <typename T, int D, int R, int JW>
__global__ void __launch_bounds__(kJoinThreads) kv_attention_join_kernel(const AttnParams p) {
  constexpr int kEach = D / 32, kRowsHere = 16 / JW;
  __shared__ float s_acc[kRowsHere][JW][D];
  __shared__ float s_sum[kRowsHere][JW];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r4 = warp / JW, part = warp % JW, r = blockIdx.y * kRowsHere + r4;
  const Record rec = p.records[blockIdx.x];
  const moe_layer_kv_attention_args_t& a = p.a;
  if (p.row_tiles > 0) {  // a sequence of fewer rows leaves no record
    const int b = blockIdx.x / p.row_tiles / a.cache.kv_heads, rt = blockIdx.x % p.row_tiles;
    if (rt * R >= seq_shape(a, b).qlen * a.group_size) return;
  }
  if (rec.b < 0) return;
  const int np = rec.c1 - rec.c0 + 1;
  // the first CTA left its part in slot 1, the others in slot 0
  auto slot_row = [&](int i) { return (2 * static_cast<int64_t>(rec.c0 + i) + (i == 0 ? 1 : 0)) * R + r; };
  float top = -INFINITY;
  for (int i = lane; i < np; i += 32) top = fmaxf(top, p.part_ml[slot_row(i) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float base = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f, acc[kEach] = {};
#pragma unroll (JW == 1 ? 8 : 4)
  for (int i = part; i < np; i += JW) {
    const int64_t at = slot_row(i);
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
    const float f = exp2_fast(__fsub_rn(ml.x, base));
    sum = __fmaf_rn(ml.y, f, sum);
#pragma unroll
    for (int e = 0; e < kEach; ++e) acc[e] = __fmaf_rn(p.part_o[at * D + lane * kEach + e], f, acc[e]);
  }
  if (lane == 0) s_sum[r4][part] = sum;
#pragma unroll
  for (int e = 0; e < kEach; ++e) s_acc[r4][part][lane * kEach + e] = acc[e];
  __syncthreads();
  const SeqShape s = seq_shape(a, rec.b);
  if (part != 0 || r >= min(R, s.qlen * a.group_size - rec.rt * R)) return;
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < JW; ++w) sum = __fadd_rn(sum, s_sum[r4][w]);
  const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : (sum == 0.0f ? 0.0f : sum);
  const int row = rec.rt * R + r, j = row / a.group_size, hq = row - j * a.group_size;
  T* out = static_cast<T*>(a.out) +
           (static_cast<int64_t>(s.q0 + j) * a.cache.kv_heads * a.group_size + rec.head * a.group_size + hq) * D;
#pragma unroll
  for (int e = 0; e < kEach; e += 2) {
    float v[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      v[z] = 0.0f;
#pragma unroll
      for (int w = 0; w < JW; ++w) v[z] = __fadd_rn(v[z], s_acc[r4][w][lane * kEach + e + z]);
    }
    *reinterpret_cast<uint32_t*>(out + lane * kEach + e) = pack2<T>(__fmul_rn(v[0], inv), __fmul_rn(v[1], inv));
  }
}

int grid_max(int num_sms, int per_sm) { return num_sms * per_sm < kMaxSlots ? num_sms * per_sm : kMaxSlots; }

template <typename T, int D, int NR, int CS>
cudaError_t launch_whole(const AttnParams& p, int64_t units, size_t smem, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  const void* k = (const void*)kv_attention_kernel<T, D, NR, CS>;
  if (const cudaError_t e = allow_smem(k, static_cast<int>(smem), allowed); e != cudaSuccess) return e;
  AttnParams arg = p;
  void* args[] = {&arg};
  return launch_after(k, dim3(static_cast<unsigned>(units) * CS), dim3(kThreads), args, smem, s, CS);
}

template <typename T, int D, int NR>
cudaError_t launch_rows(const AttnParams& p, int num_sms, cudaStream_t s) {
  const moe_layer_kv_attention_args_t& a = p.a;
  using Work = Schedule<8 * NR, kTileTokens, kUnitCost>;
  const size_t ring = kWarps * kStagesOf<NR> * 2 * kSlice * D;
  const int64_t keys = static_cast<int64_t>(a.max_pages) * a.cache.page_size;
  const int64_t rows = static_cast<int64_t>(a.max_q) * a.group_size;
  const int row_tiles = static_cast<int>((rows + 8 * NR - 1) / (8 * NR));
  const int64_t units = static_cast<int64_t>(a.batch) * a.cache.kv_heads * row_tiles;
  const int full = grid_max(num_sms, kCtasPerSm<NR>);
  AttnParams arg = p;
  // a cluster a unit: as many CTAs as let all units run at once
  const int share = units * 8 <= full ? 8 : units * 4 <= full ? 4 : units * 2 <= full ? 2 : 1;
  const int64_t seen = a.window > 0 && a.window + static_cast<int64_t>(8 * NR) < keys ? static_cast<int64_t>(a.window) + 8 * NR : keys;
  if (seen <= kWholeKeys * share && units <= kWholeUnits) {
    if (share == 8) return launch_whole<T, D, NR, 8>(arg, units, ring, s);
    if (share == 4) return launch_whole<T, D, NR, 4>(arg, units, ring, s);
    if (share == 2) return launch_whole<T, D, NR, 2>(arg, units, ring, s);
    return launch_whole<T, D, NR, 1>(arg, units, ring, s);
  }
  void* args[] = {&arg};
  static std::atomic<uint64_t> allowed{0};
  const void* k = (const void*)kv_attention_kernel<T, D, NR, 0>;
  cudaError_t e = allow_smem(k, kMaxSmem - 1024, allowed);
  if (e != cudaSuccess) return e;
  // no more CTAs than pieces of work there can be
  const int64_t tiles = (keys + kTileTokens - 1) / kTileTokens;
  const double most = static_cast<double>(units) * ((tiles > 0 ? tiles : 1) + kUnitCost);
  const int grid = most < full ? static_cast<int>(most) : full;
  const bool few = share == 8;
  if (few) arg.row_tiles = row_tiles;
  e = launch_after(k, dim3(grid), dim3(kThreads), args, ring + Work::bytes(a.batch), s);
  if (e != cudaSuccess) return e;
  const int most_rows = rows < 8 * NR ? static_cast<int>(rows) : 8 * NR;
  return few ? launch_join<T, D, 8 * NR, 16>(arg, static_cast<int>(units), most_rows, s)
             : launch_join<T, D, 8 * NR, 4>(arg, grid, most_rows, s);
}

template <typename T, int D>
cudaError_t launch_typed(const AttnParams& p, int num_sms, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.a.max_q) * p.a.group_size;
  if (rows <= 8) return launch_rows<T, D, 1>(p, num_sms, s);
  if (rows < kChunkFrom || !chunk_fits(D, p.a.batch)) return launch_rows<T, D, 2>(p, num_sms, s);
  return launch_chunk<T, D>(p, num_sms, s);
}

}  // namespace

template <typename T, int D, int R, int JW>
cudaError_t launch_join(const AttnParams& p, int records, int rows, cudaStream_t s) {
  AttnParams arg = p;
  void* args[] = {&arg};
  return launch_after((const void*)kv_attention_join_kernel<T, D, R, JW>, dim3(records, (rows + 16 / JW - 1) / (16 / JW)),
                      dim3(kJoinThreads), args, 0, s);
}
template cudaError_t launch_join<__nv_bfloat16, 64, kChunkRows, 1>(const AttnParams&, int, int, cudaStream_t);
template cudaError_t launch_join<__nv_bfloat16, 128, kChunkRows, 1>(const AttnParams&, int, int, cudaStream_t);
template cudaError_t launch_join<__half, 64, kChunkRows, 1>(const AttnParams&, int, int, cudaStream_t);
template cudaError_t launch_join<__half, 128, kChunkRows, 1>(const AttnParams&, int, int, cudaStream_t);

namespace {
// rows of all parts: 4 CTAs an SM of 8 or 3 of 16, or one of kChunkRows
constexpr size_t kStatusBytes = 256;
size_t part_rows(int num_sms) { return 2 * static_cast<size_t>(num_sms) * kChunkRows; }
static_assert(kChunkRows >= 3 * 16 && kChunkRows >= 4 * 8, "the parts of every kernel fit");
}  // namespace

size_t attention_workspace(int head_dim, int num_sms) {
  return kStatusBytes + part_rows(num_sms) * (head_dim + 2) * sizeof(float) + grid_max(num_sms, 4) * sizeof(Record);
}

cudaError_t launch_attention(const moe_layer_kv_attention_args_t& a, void* ws, int num_sms, cudaStream_t s) {
  AttnParams p;
  p.a = a;
  p.row_tiles = 0;
  p.status = static_cast<int32_t*>(ws);
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kStatusBytes);
  p.part_ml = p.part_o + part_rows(num_sms) * a.cache.head_dim;
  p.records = reinterpret_cast<Record*>(p.part_ml + part_rows(num_sms) * 2);
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  p.page_shift = 31 - __builtin_clz(static_cast<unsigned>(a.cache.page_size));
  if (a.dtype == MOE_LAYER_BF16)
    return a.cache.head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(p, num_sms, s)
                                  : launch_typed<__nv_bfloat16, 128>(p, num_sms, s);
  return a.cache.head_dim == 64 ? launch_typed<__half, 64>(p, num_sms, s) : launch_typed<__half, 128>(p, num_sms, s);
}

}  // namespace moe_layer
