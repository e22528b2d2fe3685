// The tensor-core kernel of attention over the paged 8-bit cache (many rows per cache head): included by the translation
// units that hold its instances, qdq_kv_attn_tc.cu (queries one after the other) and qdq_kv_tree_tc.cu (trees of
// drafted tokens).  How it works stands in qdq_kv_attn_tc.cu.
#pragma once

#include "qdq_kv_attn.cuh"

namespace qdq {

static __device__ unsigned int g_attn_tc_timeouts = 0;  // of this translation unit's kernels

namespace {

constexpr int BN = 64;  // tokens per tile
constexpr int kMinShare = 8;  // places on the line: a shorter share saves less than its part costs
constexpr int kJoinSlots = 3;  // for joining parts
constexpr int kPairs = 2;  // pairs of tiles whose codes are on the way or waiting (SPLIT)
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

// SPLIT: the two groups take alternate tiles of the same 128 rows, each with a tile of keys and one of values of its
// own, and are joined at the end of a part; one converting set takes the keys of the groups' tiles, the other the values.
template <int D, int PARTS, int G, bool SPLIT>
struct Cfg {
  static constexpr int kSub = D / 64;                    // 64-dim sub-tiles
  static constexpr uint32_t kQTile = kTcRows * 128;      // bytes of 128 rows of a sub-tile
  static constexpr int kRows = SPLIT ? 1 : G;            // groups of rows
  static constexpr uint32_t kQPart = kRows * kSub * kQTile;  // [group][sub-tile]
  static constexpr uint32_t kK = kSub * BN * 128, kV = D * 128;
  // tiles of keys: two pairs for SPLIT where they fit (two parts of queries leave no room)
  static constexpr int kKeys = SPLIT && PARTS == 1 ? 4 : 2;
  static constexpr uint32_t kRing = PARTS * kQPart + kKeys * kK + 2 * kV;
  static constexpr uint32_t kOCol = 2 * BN * G;  // S of group 0 (two), of group 1 (two) | O of group 0, of group 1
  static constexpr uint32_t kCols = kOCol + G * D <= 256 ? 256 : 512;
  static_assert(kOCol + G * D <= 512, "TMEM");
  // Codes wait in shared memory as stored, [keys | values, every 8 tokens 16 bytes further so that
  // the reads of 8 tokens' words meet different banks], brought by bulk copies (the converting
  // warps' proxy fences wait for a thread's loads in flight, not for these); 256 dims: no
  // room, plain loads.
  static constexpr bool kStaged = D <= 192;
  // (SPLIT: a pair of tiles' keys, then their values, unpadded, so that blocks that lie behind one another in a page come in
  // one copy; the lanes that read 8 tokens' words take different dims of them there)
  static constexpr uint32_t kStageV = BN * D, kVStep = 8 * D + (SPLIT ? 0 : 16);
  static constexpr uint32_t kStage = (kStageV + 8 * kVStep + 127) / 128 * 128;
  static constexpr int kMaxBlocks = SPLIT ? kTcTreeBlocks : kTcSplitBlocks;  // of one part
  static constexpr uint32_t kFixed = 1024 + kRing + kMaxBlocks * uint32_t(sizeof(BlockAt));
  static constexpr uint32_t kLeft = 225 * 1024 - kFixed;
  // two sets of converting warps take alternate tiles, unless only one stage fits (two parts:
  // there the products take twice as long)
  static constexpr int kSets = kStaged && kLeft < 2 * kStage ? 1 : 2;
  static_assert(!SPLIT || (kStaged && kSets == 2 && G == 2), "a converting set for the keys and one for the values");
  static constexpr int kSlots = !kStaged ? 0 : kLeft >= 2 * kSets * kStage ? 2 : 1;  // stages per set
  static constexpr uint32_t kBytes = kFixed + kSets * kSlots * kStage;
  // more than half an SM's shared memory: one CTA per SM, as the columns of TMEM want it
  static constexpr uint32_t kSmem = kBytes > 116 * 1024 ? kBytes : 116 * 1024;
  static_assert(kSmem <= 225 * 1024, "shared memory");
  static_assert(!SPLIT || kSets * kSlots == 2 * kPairs, "stages");
  static constexpr int kConv = kSet * kSets;
  static constexpr int kThreads = 32 * (kSoft * G + kConv + G + 1);
  // joining parts: columns of 4 dims in a slot, warps that add
  static constexpr uint32_t join_bytes(int quads) { return 1024 + 2 * kTcRows * kRows * 4 + kJoinSlots * kTcRows * kRows * (quads * 16 + 4); }
  static constexpr int kJoinQuads = join_bytes(16) <= kSmem ? 16 : 8, kJoinWarps = kThreads >= 512 ? 16 : 8;
  static_assert(join_bytes(kJoinQuads) <= kSmem, "room for the join");
  // 19 warps are launched with 96 registers a thread: 8 softmax warps x 128 + 8 converting x 64
  // + 3 x 96 = 19 x 96; all have 96 again for the output.  (SPLIT: what spills less: 131071 tokens bf16 136 us with
  // 128 and 64, 130 with 112 and 80, f32 164 and, with 120 and 72, 160.)
  static constexpr bool kShift = G == 2 && kSets == 2;
  static constexpr int kSoftRegs = !SPLIT ? 128 : PARTS == 1 ? 112 : 120, kConvRegs = 192 - kSoftRegs;
};

template <int N>
struct MoreBars {
  uint64_t kstage[N], kread[N], vstage[N], vread[N], kfull2[N], kfree2[N];
};
template <>
struct MoreBars<0> {};
// (SPLIT: those of a pair of tiles, one for each group; stage, sread, kfull and kfree stay unused, of vfull one is used)
template <int G, bool SPLIT>
struct Bars : MoreBars<SPLIT ? kPairs : 0> {
  uint64_t stage[2][2], sread[2][2], kfull[2], vfull[2], kfree[2], sfull[G][2], pready[G][2], pvdone[G][2], drain, joined[kJoinSlots];
  static constexpr int kBars = 8 + 6 + 6 * G + 1 + kJoinSlots + (SPLIT ? 6 * kPairs : 0);
  long long sums[20], first, g0, g1, total;  // the share's state, kept here while a part runs (registers are short)
  uint32_t tmem;
  int abort, last, entry, shares;
};

// Entry e = (sequence, tile of R rows).
struct TcEntry {
  int s, q0, len, nq, rows, r0, nr, pos_lo, pos_hi, b_lo, b_hi, tiles;  // tiles: at least 1 where there are rows
  bool bad;
};
template <bool TREE>
__device__ __forceinline__ TcEntry tc_entry(const AttnArgs &a, int e, int R) {
  TcEntry x;
  x.s = e / a.tiles;
  x.r0 = e % a.tiles * R;
  x.q0 = a.cu_q ? int(ld_u1(a.cu_q + x.s)) : x.s;
  x.nq = a.cu_q ? int(ld_u1(a.cu_q + x.s + 1)) - x.q0 : 1;
  x.len = int(ld_u1(a.kv_len + x.s));
  x.rows = min(x.nq, a.max_q) * a.group;
  x.nr = min(R, x.rows - x.r0);
  x.bad = x.len < 0 || x.len > a.max_kv_len || (x.len + a.c.page_tokens - 1) / a.c.page_tokens > a.c.table_stride ||
          (TREE && x.nq > a.max_q);
  x.tiles = 0;
  if (x.nr <= 0) return x;
  // (a tree's nodes stand anywhere from its root's position on, and their keys are the last ones)
  x.pos_lo = x.len - x.nq + (TREE ? 0 : int(a.query_of(x.r0)));
  x.pos_hi = TREE ? x.len - 1 : x.len - x.nq + int(a.query_of(x.r0 + x.nr - 1));
  x.b_lo = a.window > 0 ? max(0, x.pos_lo - a.window + 1) / kKvBlock : 0;
  x.b_hi = x.bad ? 0 : (x.pos_hi + kKvBlock) / kKvBlock;
  x.tiles = max(1, (x.b_hi - x.b_lo + 3) / 4);
  return x;
}

// BENT: the scores have a cap or a bias.  TREE: a sequence's queries are a tree of drafted tokens.
template <int D, int PARTS, int G, bool BENT, bool TREE>
__global__ void __launch_bounds__(Cfg<D, PARTS, G, TREE && G == 2>::kThreads, 1) attn_tc_kernel(const AttnArgs a) {
  constexpr bool SPLIT = TREE && G == 2;  // a tree rarely has more than 128 rows
  using C = Cfg<D, PARTS, G, SPLIT>;
  constexpr int R = kTcRows * C::kRows, kThreads = C::kThreads, kConv = C::kConv;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t *kring = smem + PARTS * C::kQPart, *vring = kring + C::kKeys * C::kK;
  BlockAt *s_blk = reinterpret_cast<BlockAt *>(smem + C::kRing);
  uint8_t *stages = smem + C::kRing + C::kMaxBlocks * sizeof(BlockAt);  // [set][slot]
  __shared__ Bars<G, SPLIT> bars;
  __shared__ float s_qs[R];
  __shared__ TreeNodes<TREE> s_tree;
  const float ninf = __int_as_float(0xff800000), qnan = __int_as_float(0x7fffffff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();

  // ---- this CTA's share.  Entry e = (sequence, tile of rows); every entry has n_kv units of the same length.
  using Entry = TcEntry;
  auto entry = [&](int e) { return tc_entry<TREE>(a, e, R); };
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
      if (!QDQ_GUARD(cn <= C::kMaxBlocks, QDQ_CHECK_SMEM)) break;
      if (u.nsplit > 1 && !QDQ_GUARD(int64_t(2) * (u.c_lo + u.nsplit) * (R * (D + 2)) <= a.room &&
                                         int64_t(bars.entry) * a.c.n_kv + h < a.units, QDQ_CHECK_OUT))
        break;
    }
    const int nt = (cn + 3) / 4;

    if (tid == 32 * (kSoft * G + kConv)) {
      if (started)
        for (int i = 0; i < Bars<G, SPLIT>::kBars; ++i) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(&bars) + 8 * i) : "memory");
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
      if constexpr (SPLIT)
        for (int i = 0; i < kPairs; ++i) {
          mbar_init(&bars.kstage[i], 1);
          mbar_init(&bars.kread[i], kSet);
          mbar_init(&bars.vstage[i], 1);
          mbar_init(&bars.vread[i], kSet);
          mbar_init(&bars.kfull2[i], kSet);
          mbar_init(&bars.kfree2[i], G);
        }
      mbar_init(&bars.drain, G);
      for (int i = 0; i < kJoinSlots; ++i) mbar_init(&bars.joined[i], 1);
      if (!started) bars.abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    started = true;
    const int64_t vplane = int64_t(a.c.page_tokens) * D;
    // block i of the part: its place and scales
    auto block_at = [&](int i) {
      BlockAt e{-1, 0.f, 0.f, 0.f, 0.f};
      if (i < cn) {
        const int blk = c0 + i, b = blk % (a.c.page_tokens / kKvBlock);
        const int64_t at = kv_record_of(a.c, s, blk, h, kv_record_bytes(a.c.page_tokens, D));
        if (at >= 0) {
          const uint8_t *sc = a.c.pages + at + 2 * vplane + 4 * b;
          const float ks = __uint_as_float(ld_u1(sc)), vs = __uint_as_float(ld_u1(sc + 4 * (a.c.page_tokens / kKvBlock)));
          e = BlockAt{at + int64_t(b) * kKvBlock * D, ks, vs * kPScale, log2f(fmaxf(vs, kMinScale)), 0.f};
          if (vs >= kMinScale && vs < __int_as_float(0x7f800000)) e.inv = __frcp_rn(e.vs);
        } else {
          e.ks = qnan;  // no page: its codes count as 0, its scores are NaN
        }
      }
      return e;
    };
    // copies of the p-th pair of tiles' keys or values into their stage (SPLIT), by a whole warp: a lane for each run of blocks
    // that lie behind one another.  (Bulk copies cost by their number: 24 of 1 and 2 KB a pair set the pace at 0.8 us a tile.)
    auto copy_pair = [&](int p, bool values) {
      if constexpr (SPLIT) {
        const int n = p % kPairs;
        uint64_t *bar = values ? &bars.vstage[n] : &bars.kstage[n];
        const int64_t at = lane < 8 && 8 * p + lane < 4 * nt ? s_blk[8 * p + lane].k : -1;  // no such block: not read
        const int64_t prev = __shfl_up_sync(0xffffffffu, (long long)at, 1);
        const bool first = at >= 0 && (lane == 0 || prev < 0 || at != prev + 16 * D);
        const uint32_t have = __ballot_sync(0xffffffffu, at >= 0), ends = __ballot_sync(0xffffffffu, first) | ~have;
        if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(__popc(have)) * 16 * D);
        __syncwarp();
        if (first) {
          const uint32_t bytes = uint32_t(__ffs(int(ends >> (lane + 1)))) * 16 * D;
          bulk_copy_g2s(stages + 2 * n * C::kStage + (values ? 2 * C::kStageV : 0) + lane * 16 * D,
                        a.c.pages + at + (values ? vplane : 0), bytes, bar);
        }
        __syncwarp();
      }
    };
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
    int copied = 0;  // tiles (SPLIT: pairs) whose copies have been issued (the copying lane's, or warp's)
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
#pragma unroll 2
      for (int i = tid - 32 * (kSoft * G + kConv); !SPLIT && i < 4 * nt; i += kThreads - 32 * (kSoft * G + kConv)) s_blk[i] = block_at(i);
      if constexpr (SPLIT) {  // the first of them (the others follow before their copies), and the first tiles' copies
        if (warp == kSoft * G + kConv + G) {
          if (lane < 4 * nt) s_blk[lane] = block_at(lane);
          __syncwarp();
        }
        named_bar_sync(4, 32 * (G + 1));
        if (warp == kSoft * G + kConv + G)
          for (; 2 * copied < nt && copied < kPairs; ++copied) {
            copy_pair(copied, false);
            copy_pair(copied, true);
          }
      } else if constexpr (C::kStaged) {  // and the first tiles' copies
        named_bar_sync(4, 32 * (G + 1));
        if (tid == 32 * (kSoft * G + kConv + G))
          for (; copied < min(nt, C::kSets * C::kSlots); ++copied) copy_tile(copied);
        __syncwarp();
      }
      if constexpr (TREE) {
        if (warp == kSoft * G + kConv + G) {  // one warp, two nodes to a lane
          const int nodes = min(nq, QDQ_MAX_TREE);
          s_tree.load(a.parent + q0, nodes, lane);
          s_tree.load(a.parent + q0, nodes, lane + 32);
          __syncwarp();
          s_tree.walk(nodes, a.window, lane);
          s_tree.walk(nodes, a.window, lane + 32);
          __syncwarp();
        }
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
    const int lr = SPLIT ? tid % kTcRows : tid;  // and their thread's row of the tile
    const int row = r0 + lr;
    float m = ninf, l = 0.f;             // its reference and sum
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t otm = tmem + lanes + C::kOCol + uint32_t(grp * D);  // its O
    if (warp < kSoft * G) {
      if constexpr (C::kShift) reg_inc<C::kSoftRegs>();
      const int qi = int(a.query_of(row));
      const int base = len - nq;  // a tree's first key
      const int pos = base + (TREE ? s_tree.depth_of(qi) : qi);
      const int lo_pos = a.window > 0 ? pos - a.window + 1 : 0;
      const float qs = TREE && s_tree.wrong(qi) ? qnan : s_qs[lr];
      uint64_t seen = 0;  // the row's drafted tokens
      if constexpr (TREE) seen = s_tree.seen_of(qi);
      const float slope = a.slopes && lr < nr ? __ldg(a.slopes + h * a.group + row - qi * a.group) * kLog2e : 0.f;
      // tokens that every row of the tile sees
      const int all_lo = a.window > 0 ? max(0, (TREE ? base + min(nq, QDQ_MAX_TREE) - 1 : pos_hi) - a.window + 1) : 0;
      const int all_hi = TREE ? base : pos_lo + 1;
      // the group's t-th tile is i
      for (int i = SPLIT ? grp : 0, t = 0; i < nt; i += SPLIT ? 2 : 1, ++t) {
        const int b = t & 1;
        const uint32_t sp = tmem + lanes + uint32_t((2 * grp + b) * BN);
        if (!wait(&bars.sfull[grp][b], t >> 1)) break;
        tc_fence_after();
        const int j0 = (c0 + 4 * i) * kKvBlock;
        const bool whole = j0 >= all_lo && j0 + BN <= all_hi;
        const BlockAt *blk = s_blk + 4 * i;
        // moves the reference, l and O with it; false after a wait's time limit
        auto raise = [&](float m_new) {
          const float corr = m_new > m ? ex2(m - m_new) : 1.f;
          l *= corr;
          m = m_new;
          if (t > 0) {
            if (!wait(&bars.pvdone[grp][(t - 1) & 1], (t - 1) >> 1)) return false;
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
              for (int e = 0; e < 16; ++e) {
                float far = at - float(e);
                if constexpr (TREE) {
                  const int node = j0 + 16 * c + e - base;
                  if (node >= 0) far = float(pos - base - s_tree.depth_of(node));
                }
                x[e] = __float_as_uint(fmaf(-slope, far, __uint_as_float(x[e])));
              }
            }
            if constexpr (TREE) {
              if (!whole) {
                const uint32_t see = tree_sees(seen, base, lo_pos, j0 + 16 * c);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (!((see >> e) & 1)) x[e] = __float_as_uint(ninf);
              }
            } else if (!whole) {
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
            const uint32_t see = TREE ? tree_sees(seen, base, lo_pos, j0 + 16 * c) : 0u;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int j = j0 + 16 * c + e;
              float x = __uint_as_float(r[e]) * fc;
              if (TREE ? !((see >> e) & 1) : j > pos || j < lo_pos) x = ninf;
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
      if constexpr (C::kShift) reg_dec<C::kConvRegs>();
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
      // the registers' codes into a tile of keys, and into one of values
      auto put_keys = [&](uint8_t *kt) {
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
      };
      // (8 tokens, chunk vc, of 8 dims from d0)
      auto put_values = [&](uint8_t *vt, const uint2 (&v)[8], int d0, int vc) {
#pragma unroll
        for (int hw = 0; hw < 2; ++hw) {  // four dims
          uint32_t even[4], odd[4];       // pairs of tokens: dims 0, 1 and dims 2, 3
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t x = (hw ? v[2 * t].y : v[2 * t].x) ^ 0x80808080u;
            const uint32_t y = (hw ? v[2 * t + 1].y : v[2 * t + 1].x) ^ 0x80808080u;
            even[t] = __byte_perm(x, y, 0x5140);
            odd[t] = __byte_perm(x, y, 0x7362);
          }
          const int d = d0 + hw * 4;
          auto put = [&](int dd, uint32_t x, uint32_t y, uint32_t z, uint32_t u) {
            *reinterpret_cast<uint4 *>(vt + dd * 128 + ((vc ^ (dd & 7)) << 4)) = make_uint4(x, y, z, u);
          };
          put(d, codes_f16<0x4140>(even[0]), codes_f16<0x4140>(even[1]), codes_f16<0x4140>(even[2]), codes_f16<0x4140>(even[3]));
          put(d + 1, codes_f16<0x4342>(even[0]), codes_f16<0x4342>(even[1]), codes_f16<0x4342>(even[2]), codes_f16<0x4342>(even[3]));
          put(d + 2, codes_f16<0x4140>(odd[0]), codes_f16<0x4140>(odd[1]), codes_f16<0x4140>(odd[2]), codes_f16<0x4140>(odd[3]));
          put(d + 3, codes_f16<0x4342>(odd[0]), codes_f16<0x4342>(odd[1]), codes_f16<0x4342>(odd[2]), codes_f16<0x4342>(odd[3]));
        }
      };
      if constexpr (SPLIT) {
        // a pair of tiles at a time: waits, fence and arrivals cost as much as the conversion of one
        constexpr int kKeyPairs = C::kKeys / 2;
        for (int p = 0; 2 * p < nt; ++p) {
          const int n = p % kPairs, tiles = min(2, nt - 2 * p);
          if (set == 0) {
            const int k = p % kKeyPairs;
            if (!wait(&bars.kstage[n], p / kPairs)) break;
            if (p >= kKeyPairs && !wait(&bars.kfree2[k], p / kKeyPairs - 1)) break;  // S of the tiles that were there is done
            for (int x = 0; x < tiles; ++x) {
              const uint8_t *st = stages + 2 * n * C::kStage + x * C::kStageV;
              const int64_t ak = s_blk[8 * p + 4 * x + w].k;
#pragma unroll
              for (int j = 0; j < KL; ++j)
                kq[j] = ak < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4 *>(st + w * 16 * D + (lane + 32 * j) * 16);
              put_keys(kring + (2 * k + x) * C::kK);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&bars.kread[n]);
              mbar_arrive(&bars.kfull2[k]);
            }
          } else {
            if (!wait(&bars.vstage[n], p / kPairs)) break;
            // P V of the pair before
            if (p >= 1 && !(wait(&bars.pvdone[0][(p - 1) & 1], (p - 1) >> 1) && wait(&bars.pvdone[1][(p - 1) & 1], (p - 1) >> 1))) break;
            for (int x = 0; x < tiles; ++x) {
              // A thread's 8 tokens and 8 dims: 16 lanes take 16 different dims (8 of them twice, heads of 64) of their
              // tokens, 8 lanes 8 different chunks of tokens, so that neither the reads nor the stores meet in one bank.
              if (D == 64 && w / 2 != x) continue;
              const int q = lane & 15, k = 2 * (D == 64 ? w & 1 : w) + (lane >> 4), vc = q & 7;
              const int d0 = D == 64 ? ((q + k + (q >> 3) * 4) & 7) * 8 : ((q + k) & 15) * 8;
              const uint8_t *st = stages + 2 * n * C::kStage + 2 * C::kStageV + x * C::kStageV + vc * 8 * D + d0;
              const int64_t av = s_blk[8 * p + 4 * x + vc / 2].k;
#pragma unroll
              for (int t = 0; t < 8; ++t) vq[0][t] = av < 0 ? make_uint2(0, 0) : *reinterpret_cast<const uint2 *>(st + t * D);
              put_values(vring + x * C::kV, vq[0], d0, vc);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&bars.vread[n]);
              mbar_arrive(&bars.vfull[0]);
            }
          }
        }
      } else {
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
          put_keys(kt);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.kfull[b]);
          // P V of tile i - 2: its values' tile is free
          if (i >= 2 && !(wait(&bars.pvdone[0][b], (i - 2) >> 1) && (G == 1 || wait(&bars.pvdone[G - 1][b], (i - 2) >> 1)))) break;
#pragma unroll
          for (int g = 0; g < VG; ++g)
            if (w + 4 * g < D / 32) put_values(vt, vq[g], (w + 4 * g) * 32 + vd * 8, vtc);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.vfull[b]);
        }
      }
      if constexpr (C::kShift) {
        // not before the softmax warps have given theirs back: a set without a tile would take its
        // registers again before a softmax group had got them
        named_bar_sync(3, 32 * (kSoft * G + kConv));
        reg_inc<96>();
      }
    } else if (warp == kSoft * G + kConv + G) {
      // ---------------- copies of the codes ----------------
      if constexpr (SPLIT) {
        // tile by tile, and the places of the next eight tiles' blocks, one to a lane, before those tiles' copies
        int keys = copied, values = copied;  // pairs whose copies have been issued
        bool ok = true;
        for (int batch = 0; 8 * batch < nt && ok; ++batch) {
          const int next = 32 * (batch + 1) + lane;
          BlockAt e{};
          if (next < 4 * nt) e = block_at(next);
          while (2 * values < min(nt, 8 * (batch + 1))) {
            const int n = values % kPairs, round = values / kPairs - 1;
            ok = wait(&bars.kread[n], round);
            if (!ok) break;
            copy_pair(keys++, false);
            ok = wait(&bars.vread[n], round);
            if (!ok) break;
            copy_pair(values++, true);
          }
          if (next < 4 * nt) s_blk[next] = e;
          __syncwarp();
        }
        // no copy may be in flight when the CTA ends, also after giving up: each stage's last one
        if (lane == 0) {
          bool done = true;
          for (int i = max(0, keys - kPairs); i < keys; ++i) done = mbar_wait(&bars.kstage[i % kPairs], uint32_t(i / kPairs) & 1u) && done;
          for (int i = max(0, values - kPairs); i < values; ++i)
            done = mbar_wait(&bars.vstage[i % kPairs], uint32_t(i / kPairs) & 1u) && done;
          if (!done) atomicAdd(&g_attn_tc_timeouts, 1u);
        }
        __syncwarp();
      } else if constexpr (C::kStaged) {
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
      const uint32_t q_base = smem_u32(smem) + (SPLIT ? 0 : g * C::kSub * C::kQTile), k_base = smem_u32(kring), v_base = smem_u32(vring);
      const uint32_t s_col = tmem + uint32_t(2 * g * BN), o_col = tmem + C::kOCol + uint32_t(g * D);
      const int mine = SPLIT ? (nt - g + 1) / 2 : nt;  // the group's tiles
      // where the keys and values of the group's t-th tile are, and whether they are there
      constexpr int kKeyPairs = C::kKeys / 2;
      auto k_slot = [&](int t) { return SPLIT ? t % kKeyPairs * 2 + g : t & 1; };
      auto v_slot = [&](int t) { return SPLIT ? g : t & 1; };
      auto keys_there = [&](int t) {
        if constexpr (SPLIT) return wait(&bars.kfull2[t % kKeyPairs], t / kKeyPairs);
        return wait(&bars.kfull[t & 1], t >> 1);
      };
      auto values_there = [&](int t) {
        if constexpr (SPLIT) return wait(&bars.vfull[0], t);
        return wait(&bars.vfull[t & 1], t >> 1);
      };
      auto scores = [&](int t) {  // S of the t-th tile
        const int b = t & 1;
        tc_fence_after();
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(leader, s_col + uint32_t(b * BN), desc_sw128(q_base + part * C::kQPart + (k / 4) * C::kQTile + (k % 4) * 32),
                   desc_sw128(k_base + k_slot(t) * C::kK + (k / 4) * (BN * 128) + (k % 4) * 32), idesc_f16(kTcRows, BN), (part | k) != 0);
        mma_commit(leader, &bars.sfull[g][b]);
        if constexpr (SPLIT)
          mma_commit(leader, &bars.kfree2[t % kKeyPairs]);
        else
          mma_commit(leader, &bars.kfree[t & 1]);
      };
      bool ok = true;
      if (mine > 0) {
        ok = keys_there(0);
        if (ok) scores(0);
      }
      for (int t = 0; t < mine && ok; ++t) {
        const int b = t & 1;
        if (t + 1 < mine) {
          ok = keys_there(t + 1);
          // the other S holds the probabilities of tile t - 1 until its products are done
          if (ok && t >= 1) ok = wait(&bars.pvdone[g][b ^ 1], (t - 1) >> 1);
          if (!ok) break;
          scores(t + 1);
        }
        ok = values_there(t) && wait(&bars.pready[g][b], t >> 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
          for (int k = 0; k < BN / 16; ++k)
            mma_ts(leader, o_col, s_col + uint32_t(b * BN + 16 * k + 8 * part), desc_sw128(v_base + v_slot(t) * C::kV + k * 32),
                   idesc_f16(kTcRows, D), (t | part | k) != 0);
        mma_commit(leader, &bars.pvdone[g][b]);
      }
      if constexpr (SPLIT) {
        // a last pair of one tile: its keys' place is free of the second group, too (not before the pair is there: the
        // first group may still have to free the pair before)
        if (g == 1 && (nt & 1) && ok && keys_there(nt >> 1)) mma_commit(leader, &bars.kfree2[(nt >> 1) % kKeyPairs]);
      }
      mma_commit(leader, &bars.drain);
    }

    // ---------------- output ----------------
    __syncwarp();
    // every product has completed before the accumulators are read and TMEM is freed
    if (!wait(&bars.drain, 0) && lane == 0) atomicAdd(&g_attn_tc_timeouts, 1u);
    tc_fence_after();
    // and every commit's arrival has landed before the barriers are made anew for the next part
    if (tid == 0 && !*reinterpret_cast<volatile int *>(&bars.abort)) {
      bool done = true;
      if constexpr (SPLIT) {
        const int pairs = (nt + 1) / 2;
        for (int k = 0; k < C::kKeys / 2 && k < pairs; ++k)
          done = mbar_wait(&bars.kfree2[k], uint32_t((pairs - 1 - k) / (C::kKeys / 2)) & 1u) && done;
        for (int g = 0; g < G; ++g)
          for (int b = 0; b < 2 && 2 * b + g < nt; ++b) {
            const uint32_t last = uint32_t(((nt - g + 1) / 2 - 1 - b) / 2) & 1u;  // of the group's tiles
            done = mbar_wait(&bars.sfull[g][b], last) && mbar_wait(&bars.pvdone[g][b], last) && done;
          }
      } else {
        for (int b = 0; b < 2 && b < nt; ++b) {
          const uint32_t last = uint32_t((nt - b + 1) / 2 - 1) & 1u;  // of the (nt - b + 1) / 2 uses
          done = mbar_wait(&bars.kfree[b], last) && done;
          for (int g = 0; g < G; ++g) done = mbar_wait(&bars.sfull[g][b], last) && mbar_wait(&bars.pvdone[g][b], last) && done;
        }
      }
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
    const bool in = lr < nr;
    float inv = 0.f;
    // 16 dims of the row from dim c: to the output, or into the part
    auto emit = [&](int c, const float (&o)[16]) {
      if (nsplit == 1) {
        if (in) {
#pragma unroll
          for (int e = 0; e < 16; e += 4) store_out<D>(a, q0, h, row, c + e, make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]), inv);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4 *>(part + (c + e) * R + 4 * lr) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      }
    };
    auto finish = [&]() {
      if (nsplit == 1) {
        if (in) store_lse(a, q0, h, row, m, l);
      } else {
        part[D * R + lr] = m;
        part[D * R + R + lr] = l;
      }
    };
    if constexpr (SPLIT) {
      // The groups are joined: each gives the other half its dims through shared memory, in the place of the tiles, and
      // writes the other half.  (The second has no tile where the part has one.)
      __shared__ float s_ml[2][2][kTcRows];
      float4 *other = reinterpret_cast<float4 *>(kring);  // [four dims][row]
      const bool some = nt > grp, others = nt > 1 - grp;
      if (warp < kSoft * G) {
        if (some) {
#pragma unroll 1
          for (int c = (1 - grp) * (D / 2); c < (2 - grp) * (D / 2); c += 16) {
            uint32_t o[16];
            tmem_ld16_async(otm + c, o);
            tmem_wait_ld16(o);
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              other[(c + e) / 4 * kTcRows + lr] = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                                              __uint_as_float(o[e + 3]));
          }
        }
        s_ml[grp][0][lr] = m;
        s_ml[grp][1][lr] = l;
      }
      __syncthreads();
      if (warp < kSoft * G) {
        const float m0 = s_ml[0][0][lr], m1 = s_ml[1][0][lr], top = fmaxf(m0, m1), ref = top == ninf ? 0.f : top;
        const float f0 = ex2(m0 - ref), f1 = ex2(m1 - ref);
        const float f_own = grp == 0 ? f0 : f1, f_other = grp == 0 ? f1 : f0;
        l = lost ? qnan : fmaf(s_ml[0][1][lr], f0, s_ml[1][1][lr] * f1);
        m = top;
        inv = l == 0.f ? 0.f : (1.f / kPScale) / l;
#pragma unroll 1
        for (int c = grp * (D / 2); c < (grp + 1) * (D / 2); c += 16) {
          uint32_t o[16];
          float v[16];
          if (some) {
            tmem_ld16_async(otm + c, o);
            tmem_wait_ld16(o);
          }
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 x = others ? other[(c + e) / 4 * kTcRows + lr] : make_float4(0.f, 0.f, 0.f, 0.f);
            v[e] = fmaf(some ? __uint_as_float(o[e]) : 0.f, f_own, x.x * f_other);
            v[e + 1] = fmaf(some ? __uint_as_float(o[e + 1]) : 0.f, f_own, x.y * f_other);
            v[e + 2] = fmaf(some ? __uint_as_float(o[e + 2]) : 0.f, f_own, x.z * f_other);
            v[e + 3] = fmaf(some ? __uint_as_float(o[e + 3]) : 0.f, f_own, x.w * f_other);
          }
          emit(c, v);
        }
        if (grp == 0) finish();
      }
    } else if (warp < kSoft * G) {
      if (lost) l = qnan;
      inv = l == 0.f ? 0.f : (1.f / kPScale) / l;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        float v[16];
        if (nt > 0) {
          tmem_ld16_async(otm + c, o);
          tmem_wait_ld16(o);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(o[e]);
        emit(c, v);
      }
      finish();
    }
    tc_fence_before();
    // (a tree's parts are joined by another kernel)
    if (!TREE && nsplit > 1) {
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

// A tree's parts, joined in order: a CTA takes 16 dims of a unit's rows (one CTA for all of them took 50 us for 38 parts
// of 128 rows of 128).  The line of work is found as the CTAs of the attention found it.
template <int D>
__global__ void __launch_bounds__(kTcRows) attn_tree_join_kernel(const AttnArgs a) {
  __shared__ long long s_sum[2][kTcRows / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kSlices = D / 16, kPart = kTcRows * (D + 2);
  const float ninf = __int_as_float(0xff800000);
  const int slice = blockIdx.x % kSlices, unit = blockIdx.x / kSlices, h = unit % a.c.n_kv, e = unit / a.c.n_kv;
  pdl_launch_dependents();
  pdl_wait();
  const int n_entries = a.n_seqs * a.tiles;
  long long before = 0, total = 0;
  for (int i = tid; i < n_entries; i += kTcRows) {
    const int tiles = tc_entry<true>(a, i, kTcRows).tiles;
    const int line = tiles ? tiles + kTcPartCost : 0;
    total += line;
    if (i < e) before += line;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (lane == 0) {
    s_sum[0][warp] = before;
    s_sum[1][warp] = total;
  }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int w = 0; w < kTcRows / 32; ++w) {
    before += s_sum[0][w];
    total += s_sum[1][w];
  }
  before *= a.c.n_kv;
  total *= a.c.n_kv;
  const TcEntry en = tc_entry<true>(a, e, kTcRows);
  if (en.tiles == 0) return;
  const int shares = int(min((long long)a.splits, max(1ll, total / kMinShare)));
  auto owner = [&](long long g) { return int(((g + 1) * shares - 1) / total); };
  const long long first = before + (long long)h * (en.tiles + kTcPartCost);
  const int c_lo = owner(first + kTcPartCost), nsplit = owner(first + kTcPartCost + en.tiles - 1) - c_lo + 1;
  if (nsplit == 1 || tid >= en.nr) return;
  if (!QDQ_GUARD(2 * (int64_t(c_lo) + nsplit) * kPart <= a.room, QDQ_CHECK_OUT)) return;
  const bool another = first > total * c_lo / shares;
  const float4 *p = reinterpret_cast<const float4 *>(a.partial + 2 * int64_t(c_lo) * kPart) + (4 * slice) * kTcRows + tid;
  const float *q = a.partial + 2 * int64_t(c_lo) * kPart + D * kTcRows + tid;
  if (another) {  // the unit's first part is its CTA's second
    p += kPart / 4;
    q += kPart;
  }
  float M = ninf, L = 0.f;
  float4 v[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < nsplit; ++k) {
    const float mk = __ldcg(q), lk = __ldcg(q + kTcRows);
    float4 x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = __ldcg(p + c * kTcRows);
    const int64_t step = 2 * int64_t(kPart) - (k == 0 && another ? kPart : 0);
    p += step / 4;
    q += step;
    const float top = fmaxf(M, mk), ref = top == ninf ? 0.f : top, f = ex2(M - ref), w = ex2(mk - ref);
    M = top;
    L = fmaf(lk, w, L * f);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      v[c] = make_float4(fmaf(x[c].x, w, v[c].x * f), fmaf(x[c].y, w, v[c].y * f), fmaf(x[c].z, w, v[c].z * f), fmaf(x[c].w, w, v[c].w * f));
  }
  const float inv = L == 0.f ? 0.f : (1.f / kPScale) / L;
  const int64_t to = out_at<D>(a, en.q0, h, en.r0 + tid) + 16 * slice;
#pragma unroll
  for (int c = 0; c < 4; ++c) store_at(a, to + 4 * c, v[c], inv);
  if (slice == 0) store_lse(a, en.q0, h, en.r0 + tid, M, L);
}

template <bool TREE, int D, int PARTS, int G>
cudaError_t run(const AttnArgs &a, cudaStream_t s) {
  using C = Cfg<D, PARTS, G, TREE && G == 2>;
  const auto kernel = a.softcap > 0.f || a.slopes ? attn_tc_kernel<D, PARTS, G, true, TREE> : attn_tc_kernel<D, PARTS, G, false, TREE>;
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), int(C::kSmem));
  if (e != cudaSuccess) return e;
  e = launch(kernel, dim3(a.splits), dim3(C::kThreads), C::kSmem, s, a);
  if constexpr (TREE) {
    if (e == cudaSuccess) e = launch(attn_tree_join_kernel<D>, dim3(unsigned(a.units * (D / 16))), dim3(kTcRows), 0, s, a);
  }
  return e;
}
template <bool TREE, int D, int PARTS>
cudaError_t run(const AttnArgs &a, int groups, cudaStream_t s) {
  if constexpr (TREE) return run<true, D, PARTS, D <= 128 ? 2 : 1>(a, s);
  if constexpr (!TREE && D <= 128) {
    if (groups == 2) return run<false, D, PARTS, 2>(a, s);
  }
  if constexpr (!TREE) return run<false, D, PARTS, 1>(a, s);
}
template <bool TREE>
cudaError_t run_attn_tc(const AttnArgs &a, int head_dim, int parts, int groups, cudaStream_t s) {
  switch (head_dim) {
    case 64: return parts == 2 ? run<TREE, 64, 2>(a, groups, s) : run<TREE, 64, 1>(a, groups, s);
    case 128: return parts == 2 ? run<TREE, 128, 2>(a, groups, s) : run<TREE, 128, 1>(a, groups, s);
    case 192: return parts == 2 ? run<TREE, 192, 2>(a, groups, s) : run<TREE, 192, 1>(a, groups, s);
    default: return parts == 1 ? run<TREE, 256, 1>(a, groups, s) : cudaErrorInvalidValue;
  }
}

int read_timeouts() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_tc_timeouts, sizeof(v)) != cudaSuccess) return -1;
  if (v && cudaMemcpyToSymbol(g_attn_tc_timeouts, &zero, sizeof(zero)) != cudaSuccess) return -1;
  return int(v);
}

}  // namespace

}  // namespace qdq
