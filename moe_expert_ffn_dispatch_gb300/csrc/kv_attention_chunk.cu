// Attention of many query rows a kv head (prompt chunks) over the paged INT8
// cache, on the tensor cores' tensor memory.
//
// A unit is (sequence, kv head, 256 query rows): two tiles A and B of 128
// rows that share every key and value.  For each piece of 128 keys
//   S = Q K^T        Q and K fp16 in shared memory, S in tensor memory;
//   P = weights      of S, a row a thread, written over S as fp16;
//   O += P V         P from tensor memory, V fp16 in shared memory.
// While one tile's weights are computed the other tile's products run:
//   S_A(i) | O_B(i-1) | S_B(i) | O_A(i) | S_A(i+1) ...
// all issued by one thread, which the tensor core runs in order, so a tile's
// S never overwrites weights that are still to be read.
//
// Roles: 8 warps of weights (4 a tile), 8 warps that turn int8 codes into fp16
// operands (exact), 1 warp that issues the products.  K and V have two stages
// each.  Keys lie [key][channel] in both operands; V's is the transposed
// (channel-contiguous) form.  The arithmetic of the weights is that of the
// kernel for few rows: row scaled by a power of two, page scale of K in the
// score, page scale of V in the weight.  The rows' references move by whole
// powers of two, and only when a weight would pass what fp16 is to hold, so that S
// is read once: weights of the same piece that are already written move with the
// reference (exactly, but for those that become subnormal).
//
// Bound by a tile's chain (S, weights, O: about 5000 cycles a piece, of which the
// products are 1100) at 42 % of the issue slots; two tiles overlap, a third has
// no room in tensor memory.  8 chunks of 512 tokens over 8192 keys (32 heads on
// 8, channels 128): 635 us, 839 TFLOP/s; channels 64: 539 us, 494 TFLOP/s.  A unit
// of fewer than 256 rows pays for 128 or 256: 16 contexts of 4000 keys and 64 rows
// take 94 us, with 256 rows 120.
#include "kv_attention.cuh"

#include "device_prims.cuh"

namespace moe_layer {
namespace {

constexpr int kTile = 128;
constexpr int kUnitCost = 4;  // in pieces; with 0, 2, 4 or 8 chunks of 512 tokens over 5011 take 163, 102, 95 and 105 us
constexpr int kSoftWarps = 8, kConvWarps = 8, kWarpMma = kSoftWarps + kConvWarps;
constexpr int kThreads = (kSoftWarps + kConvWarps + 4) * 32;  // warps in fours, which share a register limit
// Registers a thread: 96 at launch (640 x 96 = 61440 of the SM's 65536); the
// weights' warps take 120 once the others have gone down to 80 (256 x 120 + 256
// x 80 + 128 x 80 = 61440).  With 96 for all the weights' warps spill: 835 us in
// place of 632 (8 chunks of 512 tokens at 8192 keys, 32 heads on 8).
constexpr int kLaunchRegs = 96, kSoftRegs = 120, kConvRegs = 80, kMmaRegs = 80;
static_assert(256 * kSoftRegs + 256 * kConvRegs + 128 * kMmaRegs <= kThreads * kLaunchRegs, "the split fits what the launch has");
constexpr int kConvThreads = kConvWarps * 32;
constexpr int kSite = 1 << 8;  // of the waits, in the status

using Work = Schedule<kChunkRows, kTile, kUnitCost>;

// shared memory after 1024-byte alignment
template <int D>
struct Layout {
  static constexpr int kOperand = kTile * D * 2;  // one tile of Q, K or V: halves of 64 channels, [128][128 bytes] each
  static constexpr int kQ = 0, kK = 2 * kOperand, kV = 4 * kOperand, kMisc = 6 * kOperand;
  static constexpr int kWork = kMisc + 2560;
};

struct Barriers {
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full, drain;
  uint32_t tmem;
  int abort;
  int64_t carry[kThreads / 32];
  Work work;
  Segment seg[kThreads / 32];
};
static_assert(sizeof(Barriers) <= 2560, "");

// keys of a segment in pieces: the first, and how many
struct Pieces {
  int first, n;
  int lo, hi;       // keys that any row sees
  int64_t pos0;     // position of the first query token
};
__device__ __forceinline__ Pieces pieces_of(const Segment& g) {
  Pieces r;
  r.pos0 = g.s.pos0;
  r.lo = g.keys.lo, r.hi = g.keys.hi;
  r.first = g.tile0 + g.ta;
  r.n = max(0, min(g.tile0 + g.tb, (r.hi + kTile - 1) / kTile) - r.first);
  return r;
}

// byte address of 16-byte chunk ch (of 8 channels) of row r in an operand
__device__ __forceinline__ uint32_t operand_at(int r, int ch) {
  return (ch >> 3) * (kTile * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

// operand whose contiguous dimension is the N side: halves of 64 channels 16 KB apart, 8 keys every 1024 bytes
__device__ __forceinline__ uint64_t desc_transposed(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((kTile * 128) >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// 32 columns of this warp's 32 lanes, and the wait for them
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_chunk_kernel(const AttnParams p) {
  using L = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (moe::smem_u32(smem_raw) & 1023u)) & 1023u);
  Barriers& bar = *reinterpret_cast<Barriers*>(smem + L::kMisc);
  grid_dependency_wait();
  grid_launch_dependents();
  const moe_layer_kv_attention_args_t& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    p.records[blockIdx.x].b = -1;
    if (blockIdx.x == 0) p.status[moe::kStErrorFlags] = p.status[moe::kStErrorSite] = 0;
    moe::mbar_init(&bar.q_full, kSoftWarps * 32);
    for (int i = 0; i < 2; ++i) {
      moe::mbar_init(&bar.k_full[i], kConvThreads);
      moe::mbar_init(&bar.v_full[i], kConvThreads);
      moe::mbar_init(&bar.k_empty[i], 1);
      moe::mbar_init(&bar.v_empty[i], 1);
      moe::mbar_init(&bar.s_full[i], 1);
      moe::mbar_init(&bar.p_full[i], 128);
    }
    moe::mbar_init(&bar.o_full, 1);
    moe::mbar_init(&bar.drain, 1);
    bar.abort = 0;
    moe::fence_barrier_init();
  }
  if (warp == kWarpMma) moe::tmem_alloc(&bar.tmem, 512);
  {
    Work built;
    built.template build<kThreads>(a, smem + L::kWork, bar.carry);
    if (tid == 0) bar.work = built;
  }
  __syncthreads();
  moe::tc_fence_after();
  const uint32_t tmem = bar.tmem;
  volatile int* abort = &bar.abort;
  // a bounded wait of a whole warp, with one answer for all of its lanes
  auto wait = [&](uint64_t* b, uint32_t parity, int site) {
    return __all_sync(0xffffffffu, moe::mbar_wait_bounded(b, parity, abort, p.status, site)) != 0;
  };
  // columns: S of A and B, then O of A and B
  auto s_at = [&](int q) { return tmem + q * kTile; };
  auto o_at = [&](int q) { return tmem + 2 * kTile + q * D; };
  // what a warp works on lies in shared memory: registers are for the tiles
  const Work& work = bar.work;
  Segment& seg = bar.seg[warp];
  int64_t at = work.begin;
  auto next_segment = [&]() {
    Segment s;
    const bool more = work.next(a, at, s);
    __syncwarp();
    if (more && lane == 0) seg = s;
    __syncwarp();
    return more;
  };

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ------------------------------------------------ weights: a row a thread
    const int q = warp >> 2, r = (warp & 3) * 32 + lane;  // row of the tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t s_phase = 0, o_phase = 0;
    bool ok = true;
    while (ok && next_segment()) {
      const Pieces pc = pieces_of(seg);
      const int row = q * 128 + r;
      const bool mine = row < seg.rows, active = q * 128 < seg.rows;  // active: uniform over the tile
      const int grow = seg.rt * kChunkRows + row, j = grow / a.group_size, hq = grow - j * a.group_size;
      float m = -INFINITY, l = 0.0f, up = 0.0f;
      // of the warp: the unit of V's scales, and whether one above kScaleMost has been met
      float base = INFINITY;
      bool far = false;
      if (pc.n > 0) {
        // The rows of Q, each scaled by a power of two to [1, 2) at its largest
        // element: D / 8 lanes a row, 16 bytes a lane, 4 loads in flight.
        if (active) {
          constexpr int kLanes = D / 8, kRowsAt = 32 / kLanes;
          const int rl = lane / kLanes, ch = lane % kLanes;
#pragma unroll 1
          for (int r4 = 0; r4 < 32; r4 += 4 * kRowsAt) {
            uint4 u[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int rr = q * 128 + (warp & 3) * 32 + r4 + x * kRowsAt + rl;
              const int gr = seg.rt * kChunkRows + rr, jj = gr / a.group_size;
              u[x] = make_uint4(0, 0, 0, 0);
              if (rr < seg.rows)
                u[x] = *reinterpret_cast<const uint4*>(
                    static_cast<const T*>(a.q) + static_cast<int64_t>(seg.s.q0 + jj) * a.q_stride +
                    static_cast<int64_t>(seg.head * a.group_size + gr - jj * a.group_size) * D + ch * 8);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t w[4] = {u[x].x, u[x].y, u[x].z, u[x].w};
              uint32_t top = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = unpack2<T>(w[e]);
                top = max(top, max(abs_bits(f.x), abs_bits(f.y)));
              }
#pragma unroll
              for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
              const int e = min(max(static_cast<int>(top >> 23), 1), 253);
              const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
              uint32_t o[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const float2 f = unpack2<T>(w[z]);
                o[z] = pack2<__half>(__fmul_rn(f.x, down), __fmul_rn(f.y, down));
              }
              const int rr = (warp & 3) * 32 + r4 + x * kRowsAt + rl;
              *reinterpret_cast<uint4*>(smem + L::kQ + q * L::kOperand + operand_at(rr, ch)) = make_uint4(o[0], o[1], o[2], o[3]);
              // to the thread that has the row
              const float up1 = top < 0x7F800000u ? __fmul_rn(__uint_as_float(static_cast<uint32_t>(e) << 23), p.scale_log2) : NAN;
              const float mine_up = __shfl_sync(0xffffffffu, up1, ((lane - r4 - x * kRowsAt) & (kRowsAt - 1)) * kLanes);
              if (lane >= r4 + x * kRowsAt && lane < r4 + (x + 1) * kRowsAt) up = mine_up;
            }
          }
          moe::fence_proxy_async_smem();
        }
        moe::tc_fence_before();
        moe::mbar_arrive(&bar.q_full);
        const int64_t pos = mine ? pc.pos0 + j : 0;
        // page scales of the 8 blocks of 16 keys of a piece, by lanes 0 .. 7; one piece ahead
        int n_page = 0;
        float n_ks = 0.0f, n_vs = 0.0f;
        auto look_up = [&](int piece) {
          n_page = 0;
          n_ks = n_vs = 0.0f;
          const int tok = piece * kTile + lane * 16;
          if (lane < 8 && tok < pc.hi && tok + 16 > pc.lo) {
            const int pg = a.page_table[seg.b * a.table_stride + (tok >> p.page_shift)];
            n_page = -1;
            if (pg >= 0 && pg < a.cache.num_pages) {
              n_page = pg;
              n_ks = a.cache.k_scale[pg * a.cache.scale_stride + seg.head];
              n_vs = a.cache.v_scale[pg * a.cache.scale_stride + seg.head];
              if (!(fabsf(n_ks) < INFINITY)) n_ks = 0.0f, n_vs = NAN;  // a score of minus infinity would hide it
            }
          }
        };
        if (active) look_up(pc.first);
        for (int i = 0; active && i < pc.n; ++i) {
          const int key0 = (pc.first + i) * kTile;
          const int page = n_page;
          const float ks = n_ks, vs = n_vs;
          if (i + 1 < pc.n) look_up(pc.first + i + 1);
          // columns that this row sees: [c_lo, c_hi]
          int c_lo = 0, c_hi = kTile - 1;
          if (mine) {
            c_hi = static_cast<int>(max(min(pos - key0, static_cast<int64_t>(kTile - 1)), static_cast<int64_t>(-1)));
            if (a.window > 0)
              c_lo = static_cast<int>(max(min(pos - a.window + 1 - key0, static_cast<int64_t>(kTile)), static_cast<int64_t>(0)));
          }
          const uint32_t gone = __ballot_sync(0xffffffffu, page < 0);  // blocks on pages that do not exist
          const bool whole = gone == 0 && __all_sync(0xffffffffu, c_lo <= 0 && c_hi >= kTile - 1);
          // blocks that no row of the warp sees (lane i: block i); their scales do not count
          const int low = __reduce_min_sync(0xffffffffu, mine ? c_lo : kTile - 1);
          const int high = __reduce_max_sync(0xffffffffu, mine ? c_hi : -1);
          const bool hidden = page < 0 || 16 * lane > high || 16 * lane + 15 < low;
          // (nor does one that is not finite: the rows that see it take it in their weights)
          const bool counts = !hidden && lane < 8 && fabsf(vs) < INFINITY;
          if (base == INFINITY) base = scale_base(vs, counts);
          const float lv = __fsub_rn(log2_fast(fabsf(vs)), base);
          far = __any_sync(0xffffffffu, far || (counts && lv > kScaleMost));
          if (!wait(&bar.s_full[q], s_phase & 1, kSite + q)) {
            ok = false;
            break;
          }
          ++s_phase;
          moe::tc_fence_after();
          const uint32_t s_col = s_at(q) + lanes;
          // columns c .. c + 31 that this row sees, as bits
          auto bits_of = [&](int c) {
            const int lo = max(c_lo - c, 0), hi = min(c_hi - c, 31);
            uint32_t b = hi < lo ? 0u : (0xFFFFFFFFu >> (31 - hi)) & (0xFFFFFFFFu << lo);
            if ((gone >> (c >> 4)) & 1u) b &= 0xFFFF0000u;
            if ((gone >> (c >> 4)) & 2u) b &= 0x0000FFFFu;
            return b;
          };
          // S(i) is there, so the products of earlier pieces are done.  The stores have arrived when this
          // returns: a piece can scale O more than once.
          auto scale_o = [&](float corr) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float v[32];
              tmem_ld32(o_at(q) + lanes + c, v);
              uint32_t w[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__fmul_rn(v[e], corr));
              moe::tmem_st32(o_at(q) + lanes + c, w);
            }
            moe::tmem_st_wait();
          };
          // every scale of V an ordinary positive number (or no row sees its keys)
          if (!far && __all_sync(0xffffffffu, lane >= 8 || hidden || (counts && vs > 0.0f && lv >= kScaleLeast))) {
            const float lb = hidden ? 0.0f : lv, rv = hidden ? 0.0f : exp2_fast(__fsub_rn(kSumShift, lv));
#pragma unroll 1
            for (int c = 0; c < kTile; c += 32) {
              const uint32_t bits = whole ? 0xFFFFFFFFu : bits_of(c);
              uint32_t w[16];
              if (!whole && __all_sync(0xffffffffu, bits == 0)) {
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = 0u;
                tmem_st16(s_col + c / 2, w);
                continue;
              }
              const float ref = m == -INFINITY ? 0.0f : m;
              float v[32];
              tmem_ld32(s_col + c, v);
              float top = -INFINITY;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float f = __fmul_rn(__shfl_sync(0xffffffffu, ks, (c >> 4) + h), up);
                const float b = __fsub_rn(__shfl_sync(0xffffffffu, lb, (c >> 4) + h), ref);
                const uint64_t ff = pair_of(f, f), bb = pair_of(b, b);
#pragma unroll
                for (int e = h * 16; e < h * 16 + 16; e += 2) {
                  const float2 x = of_pair(fma_pair(pair_of(v[e], v[e + 1]), ff, bb));
                  v[e] = x.x, v[e + 1] = x.y;
                }
              }
              if (!whole) {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = bits & (1u << e) ? v[e] : -INFINITY;
              }
#pragma unroll
              for (int e = 0; e < 32; ++e) top = fmaxf(top, v[e]);
              // The reference moves, by whole powers of two, when a weight would
              // pass what fp16 holds (or is a row's first): what the row has so
              // far moves with it, this piece's weights among it.
              const bool fresh = m == -INFINITY && top > -INFINITY;
              if (__any_sync(0xffffffffu, top > kWeightMost || fresh)) {
                const float d = top > kWeightLand || fresh ? __fsub_rn(ceilf(top), kWeightLand) : 0.0f;
                const float corr = fresh ? 1.0f : exp2_fast(-d);  // a fresh row has nothing yet
                m = __fadd_rn(ref, d) + (m == -INFINITY && !fresh ? -INFINITY : 0.0f);
                l = __fmul_rn(l, corr);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __fsub_rn(v[e], d);
                moe::tmem_st_wait();
#pragma unroll 1
                for (int x = 0; x < c; x += 32) {
                  float pv[16];
                  tmem_ld16(s_col + x / 2, pv);
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    // (in fp32, as fp16 has no 2^-25: a weight of 2^15 outlives a step of 39)
                    const float2 f = unpack2<__half>(__float_as_uint(pv[e]));
                    w[e] = pack2<__half>(__fmul_rn(f.x, corr), __fmul_rn(f.y, corr));
                  }
                  tmem_st16(s_col + x / 2, w);
                  moe::tmem_st_wait();
                }
                if (i > 0) scale_o(corr);
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float r1 = __shfl_sync(0xffffffffu, rv, (c >> 4) + h);
                uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
                for (int e = h * 16; e < h * 16 + 16; e += 4) {
                  const float p0 = exp2_fast(v[e]), p1 = exp2_fast(v[e + 1]), p2 = exp2_fast(v[e + 2]), p3 = exp2_fast(v[e + 3]);
                  sum0 = add_pair(sum0, pair_of(p0, p1));
                  sum1 = add_pair(sum1, pair_of(p2, p3));
                  w[e / 2] = pack2<__half>(p0, p1);
                  w[e / 2 + 1] = pack2<__half>(p2, p3);
                }
                const float2 s2 = of_pair(add_pair(sum0, sum1));
                l = __fmaf_rn(__fadd_rn(s2.x, s2.y), r1, l);
              }
              tmem_st16(s_col + c / 2, w);  // columns that have been read
            }
          } else {
            // any scales: the maximum first, then the weights
            const float lr = fmaxf(lv, kScaleLeast), neg = vs < 0.0f ? -1.0f : 1.0f;
            const float ref0 = m == -INFINITY ? 0.0f : m;
            float top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < kTile; c += 32) {
              const uint32_t bits = bits_of(c);
              float v[32];
              tmem_ld32(s_col + c, v);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float f = __fmul_rn(__shfl_sync(0xffffffffu, ks, (c >> 4) + h), up);
                const float b = __fsub_rn(__shfl_sync(0xffffffffu, lr, (c >> 4) + h), ref0);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  top = fmaxf(top, bits & (1u << (h * 16 + e)) ? __fmaf_rn(v[h * 16 + e], f, b) : -INFINITY);
              }
            }
            const bool fresh = m == -INFINITY && top > -INFINITY;
            if (__any_sync(0xffffffffu, top > kWeightMost || fresh)) {
              const float d = top > kWeightLand || fresh ? __fsub_rn(ceilf(top), kWeightLand) : 0.0f;
              const float corr = fresh ? 1.0f : exp2_fast(-d);
              m = __fadd_rn(ref0, d) + (m == -INFINITY && !fresh ? -INFINITY : 0.0f);
              l = __fmul_rn(l, corr);
              if (i > 0) scale_o(corr);
            }
            const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll 1
            for (int c = 0; c < kTile; c += 32) {
              const uint32_t bits = bits_of(c);
              uint32_t w[16];
              float v[32];
              tmem_ld32(s_col + c, v);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float f = __fmul_rn(__shfl_sync(0xffffffffu, ks, (c >> 4) + h), up);
                const float vb = __shfl_sync(0xffffffffu, lv, (c >> 4) + h), sb = __shfl_sync(0xffffffffu, neg, (c >> 4) + h);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  float p2[2];
#pragma unroll
                  for (int z = 0; z < 2; ++z) {
                    // a scale that is not finite stays out of what is not seen
                    const bool on = bits & (1u << (h * 16 + e + z));
                    const float x = __fmaf_rn(v[h * 16 + e + z], f, -ref);
                    l = __fadd_rn(l, on ? exp2_fast(__fadd_rn(x, kSumShift)) : 0.0f);
                    p2[z] = on ? __fmul_rn(exp2_fast(__fadd_rn(x, vb)), sb) : 0.0f;
                  }
                  w[h * 8 + e / 2] = pack2<__half>(p2[0], p2[1]);
                }
              }
              tmem_st16(s_col + c / 2, w);  // columns that have been read
            }
          }
          moe::tmem_st_wait();
          moe::tc_fence_before();
          moe::mbar_arrive(&bar.p_full[q]);
        }
        if (!ok || !wait(&bar.o_full, o_phase & 1, kSite + 2)) break;
        ++o_phase;
        moe::tc_fence_after();
      }
      if (!active) continue;
      // ---- the rows' results
      const bool whole_unit = seg.ta == 0 && seg.tb == seg.tiles;
      float by = settle(m, l, base == INFINITY ? 0.0f : base);
      if (whole_unit) by = l > 0.0f ? __fdiv_rn(by, l) : (l == 0.0f ? 0.0f : l);
      const int64_t slot_row = (2 * static_cast<int64_t>(blockIdx.x) + (seg.ta > 0 ? 0 : 1)) * kChunkRows + row;
      T* out = static_cast<T*>(a.out) + (static_cast<int64_t>(seg.s.q0 + j) * a.cache.kv_heads * a.group_size +
                                         seg.head * a.group_size + hq) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float v[32];
        if (pc.n > 0) {
          tmem_ld32(o_at(q) + lanes + c, v);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __fmul_rn(v[e], by);
        if (whole_unit) {
          if (mine) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                w[x] = pack2<T>(v[e + 2 * x], v[e + 2 * x + 1]);
              *reinterpret_cast<uint4*>(out + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(p.part_o + slot_row * D + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
      if (!whole_unit) {
        p.part_ml[slot_row * 2] = m;
        p.part_ml[slot_row * 2 + 1] = l;
        if (seg.tb == seg.tiles && row == 0)
          p.records[blockIdx.x] = Record{seg.b, seg.head, seg.rt, work.cta_of(seg.first_piece), static_cast<int>(blockIdx.x)};
      }
    }
  } else if (warp < kWarpMma) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    // ------------------------------------------------ int8 codes to fp16 operands
    constexpr int kRowChunks = D / 16, kIt = kTile * kRowChunks / kConvThreads;  // 16-byte copies of a thread
    const int ct = tid - kSoftWarps * 32;
    const int cc = ct % kRowChunks, r0 = ct / kRowChunks;
    constexpr int kRowStep = kConvThreads / kRowChunks;
    // the codes come a piece ahead of the conversion, into the registers that it
    // has just emptied; their pages a piece ahead of that
    Pieces pc;
    pc.n = 0;
    int done = 0;  // pieces of the segment
    int page[kIt], head = 0, slot[kIt];
    auto pages_of_next = [&]() {  // false: no piece left
      while (done >= pc.n) {
        if (!next_segment()) return false;
        pc = pieces_of(seg);
        done = 0;
      }
      head = seg.head;
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        const int tok = (pc.first + done) * kTile + r0 + i * kRowStep;
        page[i] = tok < pc.hi ? a.page_table[seg.b * a.table_stride + (tok >> p.page_shift)] : -1;
        slot[i] = tok & (a.cache.page_size - 1);
      }
      ++done;
      return true;
    };
    uint4 ck[kIt], cv[kIt];
    auto fetch = [&](const int8_t* base, uint4 (&u)[kIt]) {
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        u[i] = make_uint4(0, 0, 0, 0);
        if (page[i] >= 0 && page[i] < a.cache.num_pages)
          u[i] = __ldg(reinterpret_cast<const uint4*>(base + page[i] * a.cache.page_stride + head * a.cache.head_stride +
                                                      slot[i] * D + cc * 16));
      }
    };
    // rows of a thread lie a multiple of 8 apart: one swizzle for all of them.
    // Lanes of the other half of the channels store in the other order: no bank twice
    static_assert(kRowStep % 8 == 0, "");
    const bool swap = cc & 4;
    const uint32_t first_at = operand_at(r0, 2 * cc + (swap ? 1 : 0)), second_at = operand_at(r0, 2 * cc + (swap ? 0 : 1));
    auto convert = [&](uint8_t* to, const uint4 (&u)[kIt]) {
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        uint32_t h[8];
        half_pairs(swap ? u[i].z : u[i].x, h[0], h[1]);
        half_pairs(swap ? u[i].w : u[i].y, h[2], h[3]);
        half_pairs(swap ? u[i].x : u[i].z, h[4], h[5]);
        half_pairs(swap ? u[i].y : u[i].w, h[6], h[7]);
        *reinterpret_cast<uint4*>(to + first_at + i * kRowStep * 128) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(to + second_at + i * kRowStep * 128) = make_uint4(h[4], h[5], h[6], h[7]);
      }
      moe::fence_proxy_async_smem();
    };
    uint32_t t = 0;
    bool ok = true;
    if (pages_of_next()) {
      fetch(a.cache.k, ck);
      fetch(a.cache.v, cv);
      bool more = pages_of_next();
      while (true) {
        const int st = t & 1;
        const uint32_t ph = (t >> 1) & 1;
        // Lanes wait for themselves, and the warp leaves or stays together: with one vote a piece in place
        // of one a wait, 8 chunks of 512 tokens over 8192 keys take 631 us and not 679.
        if (t >= 2) ok = moe::mbar_wait_bounded(&bar.k_empty[st], ph ^ 1, abort, p.status, kSite + 3);
        if (ok) {
          convert(smem + L::kK + st * L::kOperand, ck);
          moe::mbar_arrive(&bar.k_full[st]);
          if (more) fetch(a.cache.k, ck);
          if (t >= 2) ok = moe::mbar_wait_bounded(&bar.v_empty[st], ph ^ 1, abort, p.status, kSite + 4);
          if (ok) {
            convert(smem + L::kV + st * L::kOperand, cv);
            moe::mbar_arrive(&bar.v_full[st]);
          }
        }
        if (!__all_sync(0xffffffffu, ok)) break;
        ++t;
        if (!more) break;
        fetch(a.cache.v, cv);
        more = pages_of_next();
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    if (warp == kWarpMma) {
      // ------------------------------------------------ the products, by one lane
      const uint32_t idesc_s = moe::umma_idesc_f16(kTile, kTile);
      const uint32_t idesc_o = moe::umma_idesc_f16(kTile, D) | (1u << 16);  // V's contiguous dimension is N
      const uint64_t q_desc = moe::umma_desc_sw128(moe::smem_u32(smem + L::kQ));
      const uint64_t k_desc = moe::umma_desc_sw128(moe::smem_u32(smem + L::kK));
      const uint64_t v_desc = desc_transposed(moe::smem_u32(smem + L::kV));
      constexpr uint64_t kOp = L::kOperand >> 4, kHalf = (kTile * 128) >> 4;
      uint32_t t = 0, u = 0, np[2] = {0, 0};  // pieces, units, and weights taken of each tile
      bool ok = true;
      // S of tile q: 16 channels a product, 64 to a half
      auto product_s = [&](int q, int st) {
        if (moe::elect_one()) {
  #pragma unroll
          for (int k = 0; k < D / 16; ++k)
            moe::umma_f16(s_at(q), q_desc + q * kOp + (k >> 2) * kHalf + (k & 3) * 2,
                          k_desc + st * kOp + (k >> 2) * kHalf + (k & 3) * 2, idesc_s, k != 0);
          moe::umma_commit(&bar.s_full[q]);
        }
        __syncwarp();
      };
      // O of tile q: 16 keys a product
      auto product_o = [&](int q, uint32_t piece, bool first) {
        const int st = piece & 1;
        if (!wait(&bar.p_full[q], np[q] & 1, kSite + 5 + q)) return false;
        ++np[q];
        if (!wait(&bar.v_full[st], (piece >> 1) & 1, kSite + 7)) return false;
        moe::tc_fence_after();
        if (moe::elect_one()) {
  #pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            moe::umma_f16_ts(o_at(q), s_at(q) + k * 8, v_desc + st * kOp + k * (16 * 128 >> 4), idesc_o, !first || k != 0);
        }
        __syncwarp();
        return true;
      };
      auto commit = [&](uint64_t* b) {
        if (moe::elect_one()) moe::umma_commit(b);
        __syncwarp();
      };
      while (ok && next_segment()) {
        const Pieces pc = pieces_of(seg);
        if (pc.n == 0) continue;
        const bool two = seg.rows > 128;
        ok = wait(&bar.q_full, u & 1, kSite + 8);
        ++u;
        for (int i = 0; ok && i < pc.n; ++i, ++t) {
          ok = wait(&bar.k_full[t & 1], (t >> 1) & 1, kSite + 9);
          if (!ok) break;
          moe::tc_fence_after();
          product_s(0, t & 1);
          if (two) {
            if (i > 0) {
              ok = product_o(1, t - 1, i == 1);
              if (!ok) break;
              commit(&bar.v_empty[(t - 1) & 1]);
            }
            product_s(1, t & 1);
          }
          commit(&bar.k_empty[t & 1]);
          ok = product_o(0, t, i == 0);
          if (ok && !two) commit(&bar.v_empty[t & 1]);
        }
        if (ok && two) {
          ok = product_o(1, t - 1, pc.n == 1);
          if (ok) commit(&bar.v_empty[(t - 1) & 1]);
        }
        if (ok) commit(&bar.o_full);
      }
      // nothing of this CTA is in flight when its tensor memory goes back
      commit(&bar.drain);
      moe::mbar_wait_bounded(&bar.drain, 0, nullptr, p.status, kSite + 10);
      __syncwarp();
    }
  }
  moe::tc_fence_before();
  __syncthreads();
  moe::tc_fence_after();
  if (warp == kWarpMma) moe::tmem_dealloc(tmem, 512);
}

}  // namespace

template <typename T, int D>
size_t chunk_smem(int batch) {
  return 1024 + Layout<D>::kWork + Work::bytes(batch);
}

template <typename T, int D>
cudaError_t launch_chunk(const AttnParams& p, int num_sms, cudaStream_t s) {
  const moe_layer_kv_attention_args_t& a = p.a;
  static std::atomic<uint64_t> allowed{0};
  const void* k = (const void*)kv_attention_chunk_kernel<T, D>;
  cudaError_t e = allow_smem(k, kMaxSmem, allowed, kLaunchRegs);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (static_cast<int64_t>(a.max_pages) * a.cache.page_size + kTile - 1) / kTile;
  const int64_t rows = static_cast<int64_t>(a.max_q) * a.group_size;
  const double most = static_cast<double>(a.batch) * a.cache.kv_heads * ((rows + kChunkRows - 1) / kChunkRows) *
                      ((tiles > 0 ? tiles : 1) + kUnitCost);
  const int grid = most < num_sms ? static_cast<int>(most) : num_sms;
  AttnParams arg = p;
  void* args[] = {&arg};
  e = launch_after(k, dim3(grid), dim3(kThreads), args, chunk_smem<T, D>(a.batch), s);
  if (e != cudaSuccess) return e;
  return launch_join<T, D, kChunkRows, 1>(p, grid, rows < kChunkRows ? static_cast<int>(rows) : kChunkRows, s);
}
template cudaError_t launch_chunk<__nv_bfloat16, 64>(const AttnParams&, int, cudaStream_t);
template cudaError_t launch_chunk<__nv_bfloat16, 128>(const AttnParams&, int, cudaStream_t);
template cudaError_t launch_chunk<__half, 64>(const AttnParams&, int, cudaStream_t);
template cudaError_t launch_chunk<__half, 128>(const AttnParams&, int, cudaStream_t);

bool chunk_fits(int head_dim, int batch) {
  return (head_dim == 64 ? chunk_smem<__half, 64>(batch) : chunk_smem<__half, 128>(batch)) <= static_cast<size_t>(kMaxSmem);
}

}  // namespace moe_layer
