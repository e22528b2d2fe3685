// Attention of many query rows over the paged 8-bit cache on the 5th-generation tensor cores
// (prompt chunks; the formulas are those of qdq_kv_attn.cu).
//
// A unit is one or two groups of 128 rows (query token, head of the group) of one key/value head;
// its work is the tiles of 64 tokens that its rows see.  All units' tiles and their parts' costs in one
// line are cut into equal shares, one per CTA (causal tiles and ragged sequences differ in length), so a
// CTA takes the end of a unit, whole units and the start of another, part by part.  A unit cut by
// shares is joined from its parts' accumulators by the CTA that finishes last, in order.  For each tile:
//   S = Q K^T (128 x 64, f32 in TMEM), P = 2^(S - reference) in f16 written over S in TMEM,
//   O += P V (128 x D, f32 in TMEM).
// Codes are exact in f16, so K and V tiles are converted in registers, without their scales, into
// the 128-byte-swizzled layout the tensor core reads (V transposed on the way, four by four bytes); a
// block's key scale multiplies its 16 columns of S, its value scale the probabilities.
//   one part (16-bit activations): the queries are exact in f16 but for elements 2^-25 below the
//     row's largest, the probabilities are rounded to f16 (2^-11 relative, as the output is);
//   two parts (f32): queries and probabilities in two f16 parts each, twice the products.
//
// Warp roles (G groups of rows):
//   4 G softmax warps: one row per thread (a TMEM lane), so its maximum and sum need no exchange;
//              O is rescaled only when a reference has grown by 2^kLazy;
//   8 warps that convert the codes, as two sets of 4 taking alternate tiles, so that the loads and
//              the fence of one tile run beside the conversion of the other;
//   G warps that issue the products of a group (the first also allocates TMEM): S of tile i + 1 before P V
//              of tile i, so that the tensor core works while the softmax of a tile runs;
//   1 warp that brings the codes (bulk copies).
// Bound: the chain of a tile (codes converted, S, softmax, P V: 1.2 us a tile, no unit more than half busy)
// and what a part costs besides (queries 5 us, output 4 us, a join 8 us).  Measured: 2 prompts of 512 queries
// over 3500 to 4600 tokens, 24 / 8 heads of 128, bf16: 85 us, 0.56 PFLOP/s; the decode kernel took 278 us.
// One CTA per SM.  Two groups (head dims up to 128) share each tile's conversion.  Every wait is
// bounded; one that runs out makes the CTA's rows NaN and counts in qdq_pipeline_timeouts.
#include "qdq_kv_attn.cuh"

namespace qdq {

__device__ unsigned int g_attn_tc_timeouts = 0;

namespace {

constexpr int BN = 64;  // tokens per tile
constexpr int kMinShare = 8;  // places on the line: a shorter share saves less than its part costs
constexpr int kJoinSlots = 3;  // for joining parts
constexpr int kSoft = 4, kSet = 4;  // softmax warps per group of rows, warps per converting set

// ---- tcgen05 --------------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// 16 columns of this thread's lane, without waiting for them.
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's loads; the registers pass through, so that nothing reads them earlier.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Products issued by the lane whose `leader` is set, the whole warp running the same code.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t leader, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void named_bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Registers per thread of the calling warps' group of four.
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// K-major operand tile, rows of 128 bytes, 128-byte swizzle (16-byte chunk c of row r at c ^ (r % 8)).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
// kind::f16 with f16 operands (format 0), f32 accumulator, both K-major.
constexpr uint32_t idesc_f16(int m, int n) { return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24); }

template <int D, int PARTS, int G>
struct Cfg {
  static constexpr int kSub = D / 64;                    // 64-dim sub-tiles
  static constexpr uint32_t kQTile = kTcRows * 128;      // bytes of 128 rows of a sub-tile
  static constexpr uint32_t kQPart = G * kSub * kQTile;  // [group][sub-tile]
  static constexpr uint32_t kK = kSub * BN * 128, kV = D * 128;
  static constexpr uint32_t kRing = PARTS * kQPart + 2 * (kK + kV);
  static constexpr uint32_t kOCol = 2 * BN * G;  // S of group 0 (two), of group 1 (two) | O of group 0, of group 1
  static constexpr uint32_t kCols = kOCol + G * D <= 256 ? 256 : 512;
  static_assert(kOCol + G * D <= 512, "TMEM");
  // Codes wait in shared memory as stored, [keys | values, every 8 tokens 16 bytes further so that
  // the reads of 8 tokens' words meet different banks], brought by bulk copies (the converting
  // warps' proxy fences wait for a thread's loads in flight, not for these); 256 dims: no
  // room, plain loads.
  static constexpr bool kStaged = D <= 192;
  static constexpr uint32_t kStageV = BN * D, kVStep = 8 * D + 16;
  static constexpr uint32_t kStage = (kStageV + 8 * kVStep + 127) / 128 * 128;
  static constexpr uint32_t kFixed = 1024 + kRing + kTcSplitBlocks * uint32_t(sizeof(BlockAt));
  static constexpr uint32_t kLeft = 225 * 1024 - kFixed;
  // two sets of converting warps take alternate tiles, unless only one stage fits (two parts:
  // there the products take twice as long)
  static constexpr int kSets = kStaged && kLeft < 2 * kStage ? 1 : 2;
  static constexpr int kSlots = !kStaged ? 0 : kLeft >= 2 * kSets * kStage ? 2 : 1;  // stages per set
  static constexpr uint32_t kBytes = kFixed + kSets * kSlots * kStage;
  // more than half an SM's shared memory: one CTA per SM, as the columns of TMEM want it
  static constexpr uint32_t kSmem = kBytes > 116 * 1024 ? kBytes : 116 * 1024;
  static_assert(kSmem <= 225 * 1024, "shared memory");
  static constexpr int kConv = kSet * kSets;
  static constexpr int kThreads = 32 * (kSoft * G + kConv + G + 1);
  // joining parts: columns of 4 dims in a slot, warps that add
  static constexpr uint32_t join_bytes(int quads) { return 1024 + 2 * kTcRows * G * 4 + kJoinSlots * kTcRows * G * (quads * 16 + 4); }
  static constexpr int kJoinQuads = join_bytes(16) <= kSmem ? 16 : 8, kJoinWarps = kThreads >= 512 ? 16 : 8;
  static_assert(join_bytes(kJoinQuads) <= kSmem, "room for the join");
  // 19 warps are launched with 96 registers a thread: 8 softmax warps x 128 + 8 converting x 64
  // + 3 x 96 = 19 x 96; all have 96 again for the output
  static constexpr bool kShift = G == 2 && kSets == 2;
};

template <int G>
struct Bars {
  uint64_t stage[2][2], sread[2][2], kfull[2], vfull[2], kfree[2], sfull[G][2], pready[G][2], pvdone[G][2], drain, joined[kJoinSlots];
  static constexpr int kBars = 8 + 6 + 6 * G + 1 + kJoinSlots;
  long long sums[20], first, g0, g1, total;  // the share's state, kept here while a part runs (registers are short)
  uint32_t tmem;
  int abort, last, entry, shares;
};

// BENT: the scores have a cap or a bias.
template <int D, int PARTS, int G, bool BENT>
__global__ void __launch_bounds__(Cfg<D, PARTS, G>::kThreads, 1) attn_tc_kernel(const AttnArgs a) {
  using C = Cfg<D, PARTS, G>;
  constexpr int R = kTcRows * G, kThreads = C::kThreads, kConv = C::kConv;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t *kring = smem + PARTS * C::kQPart, *vring = kring + 2 * C::kK;
  BlockAt *s_blk = reinterpret_cast<BlockAt *>(smem + C::kRing);
  uint8_t *stages = smem + C::kRing + kTcSplitBlocks * sizeof(BlockAt);  // [set][slot]
  __shared__ Bars<G> bars;
  __shared__ float s_qs[R];
  const float ninf = __int_as_float(0xff800000), qnan = __int_as_float(0x7fffffff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();

  // ---- this CTA's share.  Entry e = (sequence, tile of rows); every entry has n_kv units of the same length.
  struct Entry {
    int s, q0, len, nq, rows, r0, nr, pos_lo, pos_hi, b_lo, b_hi, tiles;  // tiles: at least 1 where there are rows
    bool bad;
  };
  auto entry = [&](int e) {
    Entry x;
    x.s = e / a.tiles;
    x.r0 = e % a.tiles * R;
    x.q0 = a.cu_q ? int(ld_u1(a.cu_q + x.s)) : x.s;
    x.nq = a.cu_q ? int(ld_u1(a.cu_q + x.s + 1)) - x.q0 : 1;
    x.len = int(ld_u1(a.kv_len + x.s));
    x.rows = min(x.nq, a.max_q) * a.group;
    x.nr = min(R, x.rows - x.r0);
    x.bad = x.len < 0 || x.len > a.max_kv_len || (x.len + a.c.page_tokens - 1) / a.c.page_tokens > a.c.table_stride;
    x.tiles = 0;
    if (x.nr <= 0) return x;
    x.pos_lo = x.len - x.nq + int(a.query_of(x.r0));
    x.pos_hi = x.len - x.nq + int(a.query_of(x.r0 + x.nr - 1));
    x.b_lo = a.window > 0 ? max(0, x.pos_lo - a.window + 1) / kKvBlock : 0;
    x.b_hi = x.bad ? 0 : (x.pos_hi + kKvBlock) / kKvBlock;
    x.tiles = max(1, (x.b_hi - x.b_lo + 3) / 4);
    return x;
  };
  // An entry's unit on the line of all work: a part's cost in tiles, then its tiles, so that a share's end
  // in a unit's first kTcPartCost leaves the unit to the next CTA.
  auto line_of = [](const Entry &x) { return x.tiles ? x.tiles + kTcPartCost : 0; };
  const int n_entries = a.n_seqs * a.tiles, chunk = (n_entries + kThreads - 1) / kThreads;
  long long total = 0, g0, g1;  // the line's length; this CTA's share of it
  int shares;                   // CTAs that have a share
  {  // bars.entry, bars.first: the entry at g0 and its place
    long long mine = 0;
    for (int i = 0; i < chunk; ++i)
      if (tid * chunk + i < n_entries) mine += line_of(entry(tid * chunk + i));
    long long up = mine;  // inclusive sums over the threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += x;
    }
    if (lane == 31) bars.sums[warp] = up;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += bars.sums[w];
      total += bars.sums[w];
    }
    before += up - mine;
    total *= a.c.n_kv;
    before *= a.c.n_kv;
    mine *= a.c.n_kv;
    shares = int(min((long long)gridDim.x, max(1ll, total / kMinShare)));
    if (total == 0 || int(blockIdx.x) >= shares) return;
    g0 = total * blockIdx.x / shares;
    g1 = total * (blockIdx.x + 1) / shares;
    if (before <= g0 && g0 < before + mine) {  // one thread has the entry of g0
      int e = tid * chunk;
      for (;; ++e) {
        const long long n = (long long)line_of(entry(e)) * a.c.n_kv;
        if (g0 < before + n) break;
        before += n;
      }
      bars.entry = e;
      bars.first = before;
    }
  }
  if (warp == kSoft * G + kConv) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem)),
                 "r"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  if (tid == 0) {
    bars.g0 = g0;
    bars.g1 = g1;
    bars.total = total;
    bars.shares = shares;
  }
  // (volatile reads: the values are not to live in registers through a part)
  auto kept = [&](const long long &x) { return *reinterpret_cast<const volatile long long *>(&x); };
  bool started = false;
  for (;;) {  // part by part
    __syncthreads();  // the state is written; the part before is done with shared memory
    struct Unit {
      long long first;  // its place on the line
      int h, t0, t1, c_lo, nsplit;  // head, tiles of this part, first CTA with a part of it, parts
    };
    auto unit_of = [&](const Entry &en) {
      const long long at = kept(bars.g0), e0 = kept(bars.first), all = kept(bars.total);
      const int n = *reinterpret_cast<volatile int *>(&bars.shares);
      auto owner = [&](long long g) { return int(((g + 1) * n - 1) / all); };  // the CTA whose share has place g
      Unit u;
      u.h = int((at - e0) / line_of(en));
      u.first = e0 + (long long)u.h * line_of(en);
      u.t0 = int(max(0ll, at - u.first - kTcPartCost));
      u.t1 = int(min((long long)en.tiles, kept(bars.g1) - u.first - kTcPartCost));
      u.c_lo = owner(u.first + kTcPartCost);
      u.nsplit = owner(u.first + kTcPartCost + en.tiles - 1) - u.c_lo + 1;
      return u;
    };
    int s, q0, len, nq, r0, nr, pos_lo, pos_hi, c0, cn, h;
    bool bad;
    {
      const Entry en = entry(*reinterpret_cast<volatile int *>(&bars.entry));
      const Unit u = unit_of(en);
      if (u.t1 <= u.t0) break;  // a share that ends before its first unit's tiles
      s = en.s;
      q0 = en.q0;
      len = en.len;
      nq = en.nq;
      r0 = en.r0;
      nr = en.nr;
      pos_lo = en.pos_lo;
      pos_hi = en.pos_hi;
      bad = en.bad;
      h = u.h;
      c0 = en.b_lo + 4 * u.t0;
      cn = max(0, min(4 * (u.t1 - u.t0), en.b_hi - c0));
      if (!QDQ_GUARD(cn <= kTcSplitBlocks, QDQ_CHECK_SMEM)) break;
      if (u.nsplit > 1 && !QDQ_GUARD(int64_t(2) * (u.c_lo + u.nsplit) * (R * (D + 2)) <= a.room &&
                                         int64_t(bars.entry) * a.c.n_kv + h < a.units, QDQ_CHECK_OUT))
        break;
    }
    const int nt = (cn + 3) / 4;

    if (tid == 32 * (kSoft * G + kConv)) {
      if (started)
        for (int i = 0; i < Bars<G>::kBars; ++i) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(&bars.stage[0][0] + i)) : "memory");
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.stage[0][i], 1);
        mbar_init(&bars.stage[1][i], 1);
        mbar_init(&bars.sread[0][i], kSet);
        mbar_init(&bars.sread[1][i], kSet);
        mbar_init(&bars.kfull[i], kSet);
        mbar_init(&bars.vfull[i], kSet);
        mbar_init(&bars.kfree[i], G);
        for (int g = 0; g < G; ++g) {
          mbar_init(&bars.sfull[g][i], 1);
          mbar_init(&bars.pready[g][i], kSoft);
          mbar_init(&bars.pvdone[g][i], 1);
        }
      }
      mbar_init(&bars.drain, G);
      for (int i = 0; i < kJoinSlots; ++i) mbar_init(&bars.joined[i], 1);
      if (!started) bars.abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    started = true;
    const int64_t vplane = int64_t(a.c.page_tokens) * D;
    // copies of tile i's codes into its stage
    auto copy_tile = [&](int i) {
      if constexpr (C::kStaged) {
        const int set = i % C::kSets, n = i / C::kSets % C::kSlots;
        uint8_t *dst = stages + (set * C::kSlots + n) * C::kStage;
        uint64_t *bar = &bars.stage[set][n];
        int64_t at[4];
        uint32_t bytes = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          at[b] = s_blk[4 * i + b].k;
          bytes += at[b] >= 0 ? 32 * D : 0;
        }
        mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (at[b] < 0) continue;  // no such block: its part of the stage is not read
          const uint8_t *p = a.c.pages + at[b];
          bulk_copy_g2s(dst + b * 16 * D, p, 16 * D, bar);
          bulk_copy_g2s(dst + C::kStageV + (2 * b) * C::kVStep, p + vplane, 8 * D, bar);
          bulk_copy_g2s(dst + C::kStageV + (2 * b + 1) * C::kVStep, p + vplane + 8 * D, 8 * D, bar);
        }
      }
    };
    int copied = 0;  // tiles whose copies have been issued (the copying lane's)
    // the queries, scaled by a power of two per row, into f16 parts: D / 8 lanes to a row.  A lane
    // copies its 8 dims of all its rows into the tiles' space first (all copies in flight at once,
    // each read back by the lane that made it) and converts them in a small loop.
    if (warp < kSoft * G + kConv) {
      constexpr int LR = D / 8 == 24 ? 32 : D / 8, RW = 32 / LR;  // lanes and rows of a warp's copy
      constexpr int kWarps = kSoft * G + kConv, kStep = kWarps * RW;
      constexpr int kIter = (R + kStep - 1) / kStep;               // rows per lane
      constexpr int kRoom = int(2 * (C::kK + C::kV)) / (kWarps * 512 * PARTS);
      constexpr int kRound = kRoom < kIter ? kRoom : kIter;        // of them at a time
      static_assert(kRound > 0, "room for the raw queries");
      const int sub = lane / LR, d = lane % LR * 8;
      const uint32_t mine = smem_u32(kring) + uint32_t(warp * 32 + lane) * (16 * PARTS);  // + iteration * kWarps * 512 * PARTS
      const bool half = a.type == QDQ_TYPE_F16;
#pragma unroll 1
      for (int i0 = 0; i0 < kIter; i0 += kRound) {
#pragma unroll 1
        for (int i = 0; i < kRound; ++i) {
          const int r = (i0 + i) * kStep + warp * RW + sub;
          if (r < nr && d < D) {
            const int qi = int(a.query_of(r0 + r));
            const int64_t e = int64_t(q0 + qi) * a.q_stride + int64_t(h * a.group + (r0 + r - qi * a.group)) * D + d;
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine + i * (kWarps * 512 * PARTS) + 16 * p),
                           "l"(static_cast<const uint8_t *>(a.q) + (PARTS == 2 ? 4 * e + 16 * p : 2 * e))
                           : "memory");
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
        for (int i = 0; i < kRound; ++i) {
          const int r = (i0 + i) * kStep + warp * RW + sub;
          const bool in = r < nr && d < D;
          uint32_t w[4 * PARTS];
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[4 * p]), "=r"(w[4 * p + 1]), "=r"(w[4 * p + 2]), "=r"(w[4 * p + 3])
                         : "r"(mine + i * (kWarps * 512 * PARTS) + 16 * p)
                         : "memory");
#pragma unroll
            for (int e = 0; e < 4; ++e) w[4 * p + e] = in ? w[4 * p + e] : 0u;
          }
          float v[8], mx;  // the elements and the row's largest magnitude (by its bits: NaN is the largest)
          if constexpr (PARTS == 2) {
            uint32_t bits = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              v[e] = __uint_as_float(w[e]);
              bits = max(bits, w[e] & 0x7FFFFFFFu);
            }
#pragma unroll
            for (int o = LR / 2; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
            mx = __uint_as_float(bits);
          } else {
            uint32_t bits = 0;  // two halves
#pragma unroll
            for (int e = 0; e < 4; ++e) bits = __vmaxu2(bits, w[e] & 0x7FFF7FFFu);
#pragma unroll
            for (int o = LR / 2; o > 0; o >>= 1) bits = __vmaxu2(bits, __shfl_xor_sync(0xffffffffu, bits, o));
            bits = max(bits & 0xFFFFu, bits >> 16);
            mx = half ? __half2float(__ushort_as_half(uint16_t(bits))) : __uint_as_float(bits << 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = half ? unpack2(w[e], __half{}) : unpack2(w[e], __nv_bfloat16{});
              v[2 * e] = f.x;
              v[2 * e + 1] = f.y;
            }
          }
          const bool finite = mx < __int_as_float(0x7f800000);
          int ex = 13 - (int(__float_as_uint(mx) >> 23) - 127);
          ex = max(-120, min(120, ex));
          // the scale's sign goes into the queries, so that a larger product is a larger score
          float up = __uint_as_float(uint32_t(ex + 127) << 23);
          if (a.scale < 0.f) up = -up;
          if (d == 0 && r < R) {
            const float q = (finite ? __uint_as_float(uint32_t(127 - ex) << 23) : qnan) * fabsf(a.scale);
            s_qs[r] = a.softcap > 0.f ? q : q * kLog2e;
          }
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = v[2 * e] * up, y = v[2 * e + 1] * up;
            hi[e] = finite ? pack2(x, y, __half{}) : 0u;
            if constexpr (PARTS == 2) {
              const float2 back = unpack2(hi[e], __half{});
              lo[e] = finite ? pack2(x - back.x, y - back.y, __half{}) : 0u;
            }
          }
          if (r < R && d < D) {
            uint8_t *dst = smem + ((r / kTcRows) * C::kSub + d / 64) * C::kQTile + (r % kTcRows) * 128 + (((d % 64 / 8) ^ (r & 7)) << 4);
            *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if constexpr (PARTS == 2) *reinterpret_cast<uint4 *>(dst + C::kQPart) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    } else {
      // meanwhile the split's blocks: places and scales (past the last one: zeros, hidden from every row)
      const int64_t rec = kv_record_bytes(a.c.page_tokens, D);
#pragma unroll 2
      for (int i = tid - 32 * (kSoft * G + kConv); i < 4 * nt; i += kThreads - 32 * (kSoft * G + kConv)) {
        BlockAt e{-1, 0.f, 0.f, 0.f, 0.f};
        if (i < cn) {
          const int blk = c0 + i, b = blk % (a.c.page_tokens / kKvBlock);
          const int64_t at = kv_record_of(a.c, s, blk, h, rec);
          if (at >= 0) {
            const uint8_t *sc = a.c.pages + at + 2 * vplane + 4 * b;
            const float ks = __uint_as_float(ld_u1(sc)), vs = __uint_as_float(ld_u1(sc + 4 * (a.c.page_tokens / kKvBlock)));
            e = BlockAt{at + int64_t(b) * kKvBlock * D, ks, vs * kPScale, log2f(fmaxf(vs, kMinScale)), 0.f};
            if (vs >= kMinScale && vs < __int_as_float(0x7f800000)) e.inv = __frcp_rn(e.vs);
          } else {
            e.ks = qnan;  // no page: its codes count as 0, its scores are NaN
          }
        }
        s_blk[i] = e;
      }
      if constexpr (C::kStaged) {  // and the first tiles' copies
        named_bar_sync(4, 32 * (G + 1));
        if (tid == 32 * (kSoft * G + kConv + G))
          for (; copied < min(nt, C::kSets * C::kSlots); ++copied) copy_tile(copied);
        __syncwarp();
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;
    auto give_up = [&]() { *reinterpret_cast<volatile int *>(&bars.abort) = 1; };
    // a whole warp waits; false after the time limit
    auto wait = [&](uint64_t *bar, int phase) {
      if (__all_sync(0xffffffffu, mbar_wait(bar, uint32_t(phase) & 1u))) return true;
      give_up();
      return false;
    };

    const int grp = warp / kSoft;        // softmax warps: their group of rows
    const int lr = tid;                  // and their thread's row of the tile
    const int row = r0 + lr;
    float m = ninf, l = 0.f;             // its reference and sum
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t otm = tmem + lanes + C::kOCol + uint32_t(grp * D);  // its O
    if (warp < kSoft * G) {
      if constexpr (C::kShift) reg_inc<128>();
      const int qi = int(a.query_of(row));
      const int pos = len - nq + qi;
      const int lo_pos = a.window > 0 ? pos - a.window + 1 : 0;
      const float qs = s_qs[lr];
      const float slope = a.slopes && lr < nr ? __ldg(a.slopes + h * a.group + row - qi * a.group) * kLog2e : 0.f;
      // tokens that every row of the tile sees
      const int all_lo = a.window > 0 ? max(0, pos_hi - a.window + 1) : 0, all_hi = pos_lo + 1;
      for (int i = 0; i < nt; ++i) {
        const int b = i & 1;
        const uint32_t sp = tmem + lanes + uint32_t((2 * grp + b) * BN);
        if (!wait(&bars.sfull[grp][b], i >> 1)) break;
        tc_fence_after();
        const int j0 = (c0 + 4 * i) * kKvBlock;
        const bool whole = j0 >= all_lo && j0 + BN <= all_hi;
        const BlockAt *blk = s_blk + 4 * i;
        // moves the reference, l and O with it; false after a wait's time limit
        auto raise = [&](float m_new) {
          const float corr = m_new > m ? ex2(m - m_new) : 1.f;
          l *= corr;
          m = m_new;
          if (i > 0) {
            if (!wait(&bars.pvdone[grp][(i - 1) & 1], (i - 1) >> 1)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16_async(otm + c, o);
              tmem_wait_ld16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              tmem_st16(otm + c, o);
            }
          }
          return true;
        };
        if constexpr (BENT) {
          // Scores that need more than a factor (cap or bias, and the mask): transformed in their place in TMEM, then the
          // reference, then the probabilities, a block of 16 at a time in loops (unrolled over the tile this
          // was 30 KB of code, which eight warps fetched from far: a capped tile took 8 us).
          float most = ninf;  // the largest score plus log2 of its value scale
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[16];
            tmem_ld16_async(sp + 16 * c, x);
            tmem_wait_ld16(x);
            const float f = qs * blk[c].ks * (a.softcap > 0.f ? a.inv_cap : 1.f);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
            if (a.softcap > 0.f) {
              const float cap = a.softcap * kLog2e;
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(cap * tanh_of<PARTS == 2>(__uint_as_float(x[e])));
            }
            if (a.slopes) {
              const float at = float(pos - (j0 + 16 * c));
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(fmaf(-slope, at - float(e), __uint_as_float(x[e])));
            }
            if (!whole) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int j = j0 + 16 * c + e;
                if (j > pos || j < lo_pos) x[e] = __float_as_uint(ninf);
              }
            }
            float bm = __uint_as_float(x[0]);
#pragma unroll
            for (int e = 1; e < 16; ++e) bm = fmaxf(bm, __uint_as_float(x[e]));
            most = fmaxf(most, bm + blk[c].lv);
            tmem_st16(sp + 16 * c, x);
          }
          tmem_wait_st();
          const float m_new = fmaxf(m, most);
          if (__any_sync(0xffffffffu, m_new > m + (m == ninf ? 0.f : kLazy))) {
            if (!raise(m_new)) break;
          }
          const float mref = m == ninf ? 0.f : m;
          const float2 mm = f2(-mref, -mref);
          float sum = 0.f;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[16], hi[8], lo[PARTS == 2 ? 8 : 1];
            tmem_ld16_async(sp + 16 * c, x);
            tmem_wait_ld16(x);
            const float vs = blk[c].vs;
            float2 l2 = f2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 y = __fadd2_rn(f2_bits(x[2 * e], x[2 * e + 1]), mm), p = f2(ex2(y.x), ex2(y.y));
              l2 = __fadd2_rn(l2, p);
              float2 pv = __fmul2_rn(p, f2(vs, vs));
              if (y.x == ninf) pv.x = 0.f;  // a hidden token's scale may be NaN
              if (y.y == ninf) pv.y = 0.f;
              hi[e] = pack2(pv.x, pv.y, __half{});
              if constexpr (PARTS == 2) {
                const float2 back = unpack2(hi[e], __half{});
                lo[e] = pack2(pv.x - back.x, pv.y - back.y, __half{});
              }
            }
            sum += l2.x + l2.y;
            tmem_st8(sp + 16 * c, hi);  // over the block's own columns of S
            if constexpr (PARTS == 2) tmem_st8(sp + 16 * c + 8, lo);
          }
          l += sum;
        } else {
          // scores of one block of 16 of which some may be hidden (log2 units)
          auto transform = [&](int c, uint32_t *r) {
            const float fc = qs * blk[c].ks;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int j = j0 + 16 * c + e;
              float x = __uint_as_float(r[e]) * fc;
              if (j > pos || j < lo_pos) x = ninf;
              r[e] = __float_as_uint(x);
            }
          };
          uint32_t hi[4][8], lo[4][PARTS == 2 ? 8 : 1];
          float sum, most;  // of the tile's probabilities; largest sum of a block's times its value scale
          // the tile's probabilities for the present reference, from S in TMEM, a block of 16 at a time
          auto probabilities = [&](auto plain) {
            constexpr bool kPlain = decltype(plain)::value;
            const float mref = m == ninf ? 0.f : m;
            uint32_t r[2][16];
            tmem_ld16_async(sp, r[0]);
            sum = most = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t *x = r[c & 1];
              tmem_wait_ld16(x);
              if (c < 3) tmem_ld16_async(sp + 16 * (c + 1), r[(c + 1) & 1]);
              if constexpr (!kPlain) transform(c, x);
              // plain: the value scale goes into the exponent, p * vs = 2^(s - reference + log2 vs), and out of the
              // block's sum again (a product less per score; the exponent's rounding is within the scores')
              const float f = kPlain ? qs * blk[c].ks : 1.f, vs = blk[c].vs;
              const float off = kPlain ? blk[c].lv + (kLog2PScale - mref) : -mref;
              const float2 mm = f2(off, off);
              float2 l2, l3;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 y = kPlain ? __ffma2_rn(f2_bits(x[2 * e], x[2 * e + 1]), f2(f, f), mm)
                                        : __fadd2_rn(f2_bits(x[2 * e], x[2 * e + 1]), mm);
                const float2 p = f2(ex2(y.x), ex2(y.y));
                if (e == 0) l2 = p;
                else if (e == 1) l3 = p;
                else if (e & 1) l3 = __fadd2_rn(l3, p);
                else l2 = __fadd2_rn(l2, p);
                float2 pv = p;
                if constexpr (!kPlain) {  // a hidden token's scale may be NaN
                  pv = __fmul2_rn(p, f2(vs, vs));
                  if (y.x == ninf) pv.x = 0.f;
                  if (y.y == ninf) pv.y = 0.f;
                }
                hi[c][e] = pack2(pv.x, pv.y, __half{});
                if constexpr (PARTS == 2) {
                  const float2 back = unpack2(hi[c][e], __half{});
                  lo[c][e] = pack2(pv.x - back.x, pv.y - back.y, __half{});
                }
              }
              const float bs = (l2.x + l2.y) + (l3.x + l3.y);
              sum = kPlain ? fmaf(bs, blk[c].inv, sum) : sum + bs;
              most = fmaxf(most, kPlain ? bs : bs * vs);
            }
          };
          // the largest score plus log2 of its value scale
          auto largest = [&](bool plain) {
            float mx = ninf;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t x[16];
              tmem_ld16_async(sp + 16 * c, x);
              tmem_wait_ld16(x);
              if (!plain) transform(c, x);
              float bm = __uint_as_float(x[0]);
#pragma unroll
              for (int e = 1; e < 16; ++e) bm = fmaxf(bm, __uint_as_float(x[e]));
              mx = fmaxf(mx, plain ? fmaf(bm, qs * blk[c].ks, blk[c].lv) : bm + blk[c].lv);
            }
            return mx;
          };
          // Every p * vs of a block is at most the block's sum of p times vs: where those stay below
          // 2^15 (f16 ends at 2^16) with the reference there is, no maximum is looked for (64
          // comparisons less per row and tile).  Else, and for a row's first tile, the maximum moves
          // the reference and the probabilities are computed once more.
          const bool plain = whole && fminf(fminf(blk[0].inv, blk[1].inv), fminf(blk[2].inv, blk[3].inv)) > 0.f;
          bool again = __any_sync(0xffffffffu, m == ninf), ok = true;
          for (;;) {
            if (again) {  // the reference: see qdq_kv_attn.cu
              const float m_new = fmaxf(m, largest(plain));
              const bool grow = m_new > m + (m == ninf ? 0.f : kLazy);
              if (__any_sync(0xffffffffu, grow)) {
                ok = raise(m_new);
                if (!ok) break;
              }
            }
            if (plain)
              probabilities(std::true_type{});
            else
              probabilities(std::false_type{});
            if (again || !__any_sync(0xffffffffu, most > 32768.f || sum > 1e30f)) break;
            again = true;
          }
          if (!ok) break;
          l += sum;
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // over the block's own columns of S
            tmem_st8(sp + 16 * c, hi[c]);
            if constexpr (PARTS == 2) tmem_st8(sp + 16 * c + 8, lo[c]);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.pready[grp][b]);
      }
      if constexpr (C::kShift) {
        named_bar_sync(1 + grp, 32 * kSoft);  // a group of four warps meets between two changes of its registers
        reg_dec<96>();
        named_bar_arrive(3, 32 * (kSoft * G + kConv));
      }
    } else if (warp < kSoft * G + kConv) {
      // ---------------- codes to f16 tiles ----------------
      if constexpr (C::kShift) reg_dec<64>();
      const int set = (warp - kSoft * G) / kSet, w = (warp - kSoft * G) % kSet;  // tiles set, set + kSets, ...
      constexpr int KL = D / 32;            // 16-byte chunks of keys per thread: tokens 16 w .. 16 w + 15 of the tile
      constexpr int VG = (D / 32 + 3) / 4;  // groups of 32 dims of the values per warp
      uint4 kq[KL];
      uint2 vq[VG][8];
      const int vtc = lane & 7, vd = lane >> 3;  // 8-token chunk, 8-dim part of the group
      // chunk j of this thread's keys: row and 16-dim chunk of the warp's 16 tokens
      auto key_at = [&](int j, int &rr, int &ch) {
        const int u = lane + 32 * j;
        rr = u / (D / 16);
        ch = u % (D / 16);
      };
      uint8_t *my_stages = stages + set * C::kSlots * C::kStage;
      int n = 0, round = 0;  // slot, and how often it has been used
      for (int i = set; i < nt; i += C::kSets) {
        const int b = i & 1;
        const int64_t ak = s_blk[4 * i + w].k, av = s_blk[4 * i + vtc / 2].k;
        if constexpr (C::kStaged) {
          if (!wait(&bars.stage[set][n], round)) break;
          const uint8_t *st = my_stages + n * C::kStage;
#pragma unroll
          for (int j = 0; j < KL; ++j)
            kq[j] = ak < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4 *>(st + w * 16 * D + (lane + 32 * j) * 16);
#pragma unroll
          for (int g = 0; g < VG; ++g)
            if (w + 4 * g < D / 32) {
#pragma unroll
              for (int t = 0; t < 8; ++t)
                vq[g][t] = av < 0 ? make_uint2(0, 0)
                                  : *reinterpret_cast<const uint2 *>(st + C::kStageV + vtc * C::kVStep + t * D + (w + 4 * g) * 32 + vd * 8);
            }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.sread[set][n]);
          if (++n == C::kSlots) {
            n = 0;
            ++round;
          }
        } else {
#pragma unroll
          for (int j = 0; j < KL; ++j)
            kq[j] = ak < 0 ? make_uint4(0, 0, 0, 0) : ld_u4(a.c.pages + ak + (lane + 32 * j) * 16);
#pragma unroll
          for (int g = 0; g < VG; ++g)
            if (w + 4 * g < D / 32) {
#pragma unroll
              for (int t = 0; t < 8; ++t)
                vq[g][t] = av < 0 ? make_uint2(0, 0)
                                  : ld_u2(a.c.pages + av + vplane + ((vtc & 1) * 8 + t) * D + (w + 4 * g) * 32 + vd * 8);
            }
        }
        if (i >= 2 && !wait(&bars.kfree[b], (i - 2) >> 1)) break;  // S of tile i - 2 is done: its keys' tile is free
        uint8_t *kt = kring + b * C::kK, *vt = vring + b * C::kV;
#pragma unroll
        for (int j = 0; j < KL; ++j) {
          int rr, ch;
          key_at(j, rr, ch);
          rr += 16 * w;
          const uint32_t q[4] = {kq[j].x, kq[j].y, kq[j].z, kq[j].w};
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t u = q[e] ^ 0x80808080u;
            o[2 * e] = codes_f16<0x4140>(u);
            o[2 * e + 1] = codes_f16<0x4342>(u);
          }
          uint8_t *dst = kt + (ch / 4) * (BN * 128) + rr * 128;
          const int c = 2 * ch % 8;
          *reinterpret_cast<uint4 *>(dst + ((c ^ (rr & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4 *>(dst + (((c + 1) ^ (rr & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.kfull[b]);
        // P V of tile i - 2: its values' tile is free
        if (i >= 2 && !(wait(&bars.pvdone[0][b], (i - 2) >> 1) && (G == 1 || wait(&bars.pvdone[G - 1][b], (i - 2) >> 1)))) break;
#pragma unroll
        for (int g = 0; g < VG; ++g)
          if (w + 4 * g < D / 32) {
#pragma unroll
            for (int hw = 0; hw < 2; ++hw) {  // four dims
              uint32_t even[4], odd[4];       // pairs of tokens: dims 0, 1 and dims 2, 3
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const uint32_t x = (hw ? vq[g][2 * t].y : vq[g][2 * t].x) ^ 0x80808080u;
                const uint32_t y = (hw ? vq[g][2 * t + 1].y : vq[g][2 * t + 1].x) ^ 0x80808080u;
                even[t] = __byte_perm(x, y, 0x5140);
                odd[t] = __byte_perm(x, y, 0x7362);
              }
              const int d = (w + 4 * g) * 32 + vd * 8 + hw * 4;
              auto put = [&](int dd, uint32_t x, uint32_t y, uint32_t z, uint32_t u) {
                *reinterpret_cast<uint4 *>(vt + dd * 128 + ((vtc ^ (dd & 7)) << 4)) = make_uint4(x, y, z, u);
              };
              put(d, codes_f16<0x4140>(even[0]), codes_f16<0x4140>(even[1]), codes_f16<0x4140>(even[2]), codes_f16<0x4140>(even[3]));
              put(d + 1, codes_f16<0x4342>(even[0]), codes_f16<0x4342>(even[1]), codes_f16<0x4342>(even[2]), codes_f16<0x4342>(even[3]));
              put(d + 2, codes_f16<0x4140>(odd[0]), codes_f16<0x4140>(odd[1]), codes_f16<0x4140>(odd[2]), codes_f16<0x4140>(odd[3]));
              put(d + 3, codes_f16<0x4342>(odd[0]), codes_f16<0x4342>(odd[1]), codes_f16<0x4342>(odd[2]), codes_f16<0x4342>(odd[3]));
            }
          }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.vfull[b]);
      }
      if constexpr (C::kShift) {
        // not before the softmax warps have given theirs back: a set without a tile would take its
        // registers again before a softmax group had got them
        named_bar_sync(3, 32 * (kSoft * G + kConv));
        reg_inc<96>();
      }
    } else if (warp == kSoft * G + kConv + G) {
      // ---------------- copies of the codes ----------------
      if constexpr (C::kStaged) {
        if (lane == 0) {
          for (; copied < nt; ++copied) {
            const int set = copied % C::kSets, use = copied / C::kSets, n = use % C::kSlots;  // the set's use-th tile
            if (!mbar_wait(&bars.sread[set][n], uint32_t(use / C::kSlots - 1) & 1u)) {
              give_up();
              break;
            }
            copy_tile(copied);
          }
          // no copy may be in flight when the CTA ends, also after giving up: each stage's last one
          for (int i = max(0, copied - C::kSets * C::kSlots); i < copied; ++i)
            if (!mbar_wait(&bars.stage[i % C::kSets][i / C::kSets % C::kSlots], uint32_t(i / C::kSets / C::kSlots) & 1u))
              atomicAdd(&g_attn_tc_timeouts, 1u);
        }
        __syncwarp();
      }
    } else {
      // ---------------- products ----------------
      // a warp per group: one for both spent longer on its waits than the tensor core on the products
      const int g = warp - (kSoft * G + kConv);
      const uint32_t leader = elect_lane();
      const uint32_t q_base = smem_u32(smem) + g * C::kSub * C::kQTile, k_base = smem_u32(kring), v_base = smem_u32(vring);
      const uint32_t s_col = tmem + uint32_t(2 * g * BN), o_col = tmem + C::kOCol + uint32_t(g * D);
      auto scores = [&](int i) {  // S of tile i
        const int b = i & 1;
        tc_fence_after();
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(leader, s_col + uint32_t(b * BN), desc_sw128(q_base + part * C::kQPart + (k / 4) * C::kQTile + (k % 4) * 32),
                   desc_sw128(k_base + b * C::kK + (k / 4) * (BN * 128) + (k % 4) * 32), idesc_f16(kTcRows, BN), (part | k) != 0);
        mma_commit(leader, &bars.sfull[g][b]);
        mma_commit(leader, &bars.kfree[b]);
      };
      bool ok = true;
      if (nt > 0) {
        ok = wait(&bars.kfull[0], 0);
        if (ok) scores(0);
      }
      for (int i = 0; i < nt && ok; ++i) {
        const int b = i & 1;
        if (i + 1 < nt) {
          ok = wait(&bars.kfull[b ^ 1], (i + 1) >> 1);
          // the other S holds the probabilities of tile i - 1 until its products are done
          if (ok && i >= 1) ok = wait(&bars.pvdone[g][b ^ 1], (i - 1) >> 1);
          if (!ok) break;
          scores(i + 1);
        }
        ok = wait(&bars.vfull[b], i >> 1) && wait(&bars.pready[g][b], i >> 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
          for (int k = 0; k < BN / 16; ++k)
            mma_ts(leader, o_col, s_col + uint32_t(b * BN + 16 * k + 8 * part), desc_sw128(v_base + b * C::kV + k * 32),
                   idesc_f16(kTcRows, D), (i | part | k) != 0);
        mma_commit(leader, &bars.pvdone[g][b]);
      }
      mma_commit(leader, &bars.drain);
    }

    // ---------------- output ----------------
    __syncwarp();
    // every product has completed before the accumulators are read and TMEM is freed
    if (!wait(&bars.drain, 0) && lane == 0) atomicAdd(&g_attn_tc_timeouts, 1u);
    tc_fence_after();
    // and every commit's arrival has landed before the barriers are made anew for the next part
    if (tid == 0 && !*reinterpret_cast<volatile int *>(&bars.abort))
      for (int b = 0; b < 2 && b < nt; ++b) {
        const uint32_t last = uint32_t((nt - b + 1) / 2 - 1) & 1u;  // of the (nt - b + 1) / 2 uses
        bool done = mbar_wait(&bars.kfree[b], last);
        for (int g = 0; g < G; ++g) done = mbar_wait(&bars.sfull[g][b], last) && mbar_wait(&bars.pvdone[g][b], last) && done;
        if (!done) give_up();
      }
    __syncthreads();
    const bool lost = bad || *reinterpret_cast<volatile int *>(&bars.abort) != 0;
    if (tid == 0 && bars.abort) atomicAdd(&g_attn_tc_timeouts, 1u);
    constexpr int kPart = R * (D + 2);
    const int e_cur = *reinterpret_cast<volatile int *>(&bars.entry);
    const Entry en = entry(e_cur);
    const Unit u = unit_of(en);
    const int nsplit = u.nsplit;
    // a CTA keeps up to two parts of cut units: the first of its share, and another, which starts its unit
    const bool another = u.first > kept(bars.total) * u.c_lo / *reinterpret_cast<volatile int *>(&bars.shares);
    auto part_of = [&](int k) { return a.partial + (2 * int64_t(u.c_lo + k) + (k == 0 && another)) * kPart; };  // k-th part
    float *part = part_of(int(blockIdx.x) - u.c_lo);  // [four dims][row][4], maxima, sums
    if (warp < kSoft * G) {
      if (lost) l = qnan;
      const float inv = l == 0.f ? 0.f : (1.f / kPScale) / l;
      const bool in = lr < nr;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        if (nt > 0) {
          tmem_ld16_async(otm + c, o);
          tmem_wait_ld16(o);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0;
        }
        if (nsplit == 1) {
          if (in) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              store_out<D>(a, q0, h, row, c + e,
                           make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                       __uint_as_float(o[e + 3])),
                           inv);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<uint4 *>(part + (c + e) * R + 4 * lr) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (nsplit == 1) {
        if (in) store_lse(a, q0, h, row, m, l);
      } else {
        part[D * R + lr] = m;
        part[D * R + R + lr] = l;
      }
    }
    tc_fence_before();
    if (nsplit > 1) {
      // The CTA that finishes last joins the parts, in order.  Their accumulators (32 or 64 dims of all rows
      // at a time) and references come through a ring of bulk copies in the space of the tiles; a warp takes
      // 16 dims of 8 rows at a time, whole sectors of the output.  (Plain loads, 4 of 16 bytes in flight per thread,
      // took 10 us for two or three parts of 256 rows of 128.)
      asm volatile("fence.proxy.async;" ::: "memory");
      __threadfence();
      __syncthreads();
      if (tid == 0) bars.last = atomicInc(a.tickets + int64_t(e_cur) * a.c.n_kv + h, nsplit - 1) == uint32_t(nsplit - 1);
      __syncthreads();
      if (bars.last) {
        __threadfence();
        asm volatile("fence.proxy.async;" ::: "memory");
        constexpr int kJoinQuads = C::kJoinQuads, kJoinWarps = C::kJoinWarps;
        constexpr uint32_t kBytes = kJoinQuads * R * 16, kSlot = kBytes + R * 4;
        constexpr int kRows = R / (8 * kJoinWarps), kQuads = kJoinQuads / 4;  // rows and 4-dim columns per thread
        float *s_ref = reinterpret_cast<float *>(smem), *s_inv = s_ref + R;
        uint8_t *slots = smem + 2 * R * 4;
        const int items = D / (4 * kJoinQuads) * nsplit;  // 32 dims of one part each
        auto bring = [&](int j) {
          const float *p = part_of(j % nsplit);
          uint8_t *dst = slots + j % kJoinSlots * kSlot;
          uint64_t *bar = &bars.joined[j % kJoinSlots];
          mbar_arrive_expect_tx(bar, kSlot);
          bulk_copy_g2s(dst, p + int64_t(j / nsplit) * (kJoinQuads * R * 4), kBytes, bar);
          bulk_copy_g2s(dst + kBytes, p + D * R, R * 4, bar);
        };
        if (tid == 0)
          for (int j = 0; j < min(items, kJoinSlots); ++j) bring(j);
        __syncwarp();
        for (int r = tid; r < nr; r += kThreads) {
          float M = ninf, L = 0.f;
#pragma unroll 4
          for (int k = 0; k < nsplit; ++k) {
            const float mk = __ldcg(part_of(k) + D * R + r), lk = __ldcg(part_of(k) + (D + 1) * R + r);
            const float top = fmaxf(M, mk), ref = top == ninf ? 0.f : top;
            L = fmaf(lk, ex2(mk - ref), L * ex2(M - ref));
            M = top;
          }
          s_ref[r] = M == ninf ? 0.f : M;
          s_inv[r] = L == 0.f ? 0.f : (1.f / kPScale) / L;
          store_lse(a, q0, h, r0 + r, M, L);
        }
        __syncthreads();
        const int r1 = 8 * warp + (lane & 7), quad = lane >> 3;  // the thread's first row and column
        float4 v[kRows][kQuads];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int c = 0; c < kQuads; ++c) v[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        int64_t to[kRows];
        float ref[kRows], inv[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int r = min(r1 + 8 * kJoinWarps * i, R - 1);
          to[i] = out_at<D>(a, q0, h, r0 + r) + 4 * quad;
          ref[i] = s_ref[r];
          inv[i] = s_inv[r];
        }
        int k = 0;
        for (int j = 0; j < items; ++j) {
          const bool there = mbar_wait(&bars.joined[j % kJoinSlots], uint32_t(j / kJoinSlots) & 1u);
          if (!there) give_up();
          if (warp < kJoinWarps) {
            const uint8_t *slot = slots + j % kJoinSlots * kSlot;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
              const int r = r1 + 8 * kJoinWarps * i;
              const float w = there ? ex2(reinterpret_cast<const float *>(slot + kBytes)[r] - ref[i]) : qnan;
#pragma unroll
              for (int c = 0; c < kQuads; ++c) {
                const float4 x = reinterpret_cast<const float4 *>(slot)[(quad + 4 * c) * R + r];
                float4 &o = v[i][c];
                o = make_float4(fmaf(x.x, w, o.x), fmaf(x.y, w, o.y), fmaf(x.z, w, o.z), fmaf(x.w, w, o.w));
              }
            }
          }
          __syncthreads();  // the slot has been read
          if (tid == 0 && j + kJoinSlots < items) bring(j + kJoinSlots);
          if (++k == nsplit) {
            if (warp < kJoinWarps) {
#pragma unroll
              for (int i = 0; i < kRows; ++i) {
                const int r = r1 + 8 * kJoinWarps * i;
#pragma unroll
                for (int c = 0; c < kQuads; ++c) {
                  if (r < nr) store_at(a, to[i] + 16 * c, v[i][c], inv[i]);
                  v[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                to[i] += 4 * kJoinQuads;
              }
            }
            k = 0;
          }
        }
      }
    }
    // the next unit, where the share has tiles of it
    const long long next = u.first + line_of(en), end = kept(bars.first) + (long long)line_of(en) * a.c.n_kv;
    const bool more = next + kTcPartCost < kept(bars.g1);
    __syncthreads();  // every thread has read the state
    if (!more) break;
    if (tid == 0) {
      bars.g0 = next;
      if (next == end) {  // to the next entry that has tiles
        int e = e_cur;
        do ++e;
        while (entry(e).tiles == 0);
        bars.entry = e;
        bars.first = next;
      }
    }
  }
  __syncthreads();
  if (warp == kSoft * G + kConv) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(bars.tmem), "r"(C::kCols) : "memory");
  }
}

template <int D, int PARTS, int G>
cudaError_t run(const AttnArgs &a, cudaStream_t s) {
  using C = Cfg<D, PARTS, G>;
  const auto kernel = a.softcap > 0.f || a.slopes ? attn_tc_kernel<D, PARTS, G, true> : attn_tc_kernel<D, PARTS, G, false>;
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), int(C::kSmem));
  if (e != cudaSuccess) return e;
  return launch(kernel, dim3(a.splits), dim3(C::kThreads), C::kSmem, s, a);
}
template <int D, int PARTS>
cudaError_t run(const AttnArgs &a, int groups, cudaStream_t s) {
  if constexpr (D <= 128) {
    if (groups == 2) return run<D, PARTS, 2>(a, s);
  }
  return run<D, PARTS, 1>(a, s);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs &a, int head_dim, int parts, int groups, cudaStream_t s) {
  switch (head_dim) {
    case 64: return parts == 2 ? run<64, 2>(a, groups, s) : run<64, 1>(a, groups, s);
    case 128: return parts == 2 ? run<128, 2>(a, groups, s) : run<128, 1>(a, groups, s);
    case 192: return parts == 2 ? run<192, 2>(a, groups, s) : run<192, 1>(a, groups, s);
    default: return parts == 1 ? run<256, 1>(a, groups, s) : cudaErrorInvalidValue;
  }
}

QDQ_CHECK_READER(read_checks_attn_tc)

int read_attn_tc_timeouts() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_tc_timeouts, sizeof(v)) != cudaSuccess) return -1;
  if (v && cudaMemcpyToSymbol(g_attn_tc_timeouts, &zero, sizeof(zero)) != cudaSuccess) return -1;
  return int(v);
}

}  // namespace qdq
