// Attention of many query rows over the paged 8-bit cache on the 5th-generation tensor cores
// (prompt chunks; the formulas are those of qdq_kv_attn.cu).
//
// A CTA takes 128 rows (query token, head of the group) of one key/value head and walks tiles of
// 64 tokens of its split:
//   S = Q K^T (128 x 64, f32 in TMEM), P = 2^(S - reference) in f16 written over S in TMEM,
//   O += P V (128 x D, f32 in TMEM).
// Codes are exact in f16, so K and V tiles are converted in registers, without their scales, into
// the 128-byte-swizzled layout the tensor core reads (V transposed on the way, four by four bytes); a
// block's key scale multiplies its 16 columns of S, its value scale the probabilities.
//   one part (16-bit activations): the queries are exact in f16 but for elements 2^-25 below the
//     row's largest, the probabilities are rounded to f16 (2^-11 relative, as the output is);
//   two parts (f32): queries and probabilities in two f16 parts each, twice the products.
//
// Warp roles (288 threads):
//   warps 0-3  softmax: one row per thread (a TMEM lane), so its maximum and sum need no
//              exchange; O is rescaled only when a reference has grown by 2^kLazy;
//   warps 4-7  convert the codes (two tiles of K and of V in shared memory, loads one tile ahead);
//   warp 8     allocates TMEM and issues the products: S of tile i + 1 before P V of tile i, so
//              that the tensor core works while the softmax of a tile runs.
// With one part and D <= 128 two CTAs share an SM (256 columns of TMEM each) and fill each
// other's waits.  Every wait is bounded; one that runs out makes the tile's rows NaN and counts in
// qdq_pipeline_timeouts.
#include "qdq_kv_attn.cuh"

namespace qdq {

__device__ unsigned int g_attn_tc_timeouts = 0;

namespace {

constexpr int BN = 64;  // tokens per tile
constexpr int kSoft = 4, kConv = 4;
constexpr int kThreads = 32 * (kSoft + kConv + 1);

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
// K-major operand tile, rows of 128 bytes, 128-byte swizzle (16-byte chunk c of row r at c ^ (r % 8)).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
// kind::f16 with f16 operands (format 0), f32 accumulator, both K-major.
constexpr uint32_t idesc_f16(int m, int n) { return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24); }

template <int D, int PARTS>
struct Cfg {
  static constexpr int kSub = D / 64;                       // 64-dim sub-tiles
  static constexpr uint32_t kQPart = kSub * kTcRows * 128;  // bytes
  static constexpr uint32_t kK = kSub * BN * 128, kV = D * 128;
  static constexpr uint32_t kRing = PARTS * kQPart + 2 * (kK + kV);
  static constexpr uint32_t kOCol = 2 * BN;  // S0 | S1 | O
  static constexpr uint32_t kCols = kOCol + D <= 256 ? 256 : 512;
  static constexpr uint32_t kBytes = 1024 + kRing + kTcSplitBlocks * uint32_t(sizeof(BlockAt));
  // an SM's 512 columns of TMEM hold two CTAs at most: no third one may fit its shared memory
  static constexpr uint32_t kSmem = kBytes > 80 * 1024 ? kBytes : 80 * 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static constexpr int kPerSm = kCols == 256 && kSmem <= 112 * 1024 ? 2 : 1;
};

struct Bars {
  uint64_t kfull[2], vfull[2], sfull[2], pready[2], pvdone[2], drain;
  uint32_t tmem;
  int abort, last;
};

template <int D, int PARTS>
__global__ void __launch_bounds__(kThreads, Cfg<D, PARTS>::kPerSm) attn_tc_kernel(const AttnArgs a) {
  using C = Cfg<D, PARTS>;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t *kring = smem + PARTS * C::kQPart, *vring = kring + 2 * C::kK;
  BlockAt *s_blk = reinterpret_cast<BlockAt *>(smem + C::kRing);
  __shared__ Bars bars;
  const float ninf = __int_as_float(0xff800000), qnan = __int_as_float(0x7fffffff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x % a.splits;
  const int unit = blockIdx.x / a.splits;
  // tiles of a sequence and head in reverse: with a causal mask the last see the most tokens
  const int tile = a.tiles - 1 - unit % a.tiles, h = unit / a.tiles % a.c.n_kv, s = unit / a.tiles / a.c.n_kv;
  pdl_launch_dependents();
  pdl_wait();

  const int q0 = a.cu_q ? int(ld_u1(a.cu_q + s)) : s;
  const int nq = a.cu_q ? int(ld_u1(a.cu_q + s + 1)) - q0 : 1;
  const int len = int(ld_u1(a.kv_len + s));
  const int rows = nq * a.group, r0 = tile * kTcRows;
  if (r0 >= rows) return;
  const int nr = min(kTcRows, rows - r0);
  const bool bad = len < 0 || len > a.max_kv_len || (len + a.c.page_tokens - 1) / a.c.page_tokens > a.c.table_stride;
  const int pos_lo = len - nq + r0 / a.group, pos_hi = len - nq + (r0 + nr - 1) / a.group;
  const int b_lo = a.window > 0 ? max(0, pos_lo - a.window + 1) / kKvBlock : 0;
  const int b_hi = bad ? 0 : (pos_hi + kKvBlock) / kKvBlock;
  const int nb = max(0, b_hi - b_lo);
  const int nsplit = max(1, (nb + a.split_blocks - 1) / a.split_blocks);
  if (split >= nsplit) return;
  const int c0 = b_lo + split * a.split_blocks, cn = max(0, min(a.split_blocks, b_hi - c0));
  const int nt = (cn + 3) / 4;  // tiles of 64 tokens

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.kfull[i], kConv);
      mbar_init(&bars.vfull[i], kConv);
      mbar_init(&bars.sfull[i], 1);
      mbar_init(&bars.pready[i], kSoft);
      mbar_init(&bars.pvdone[i], 1);
    }
    mbar_init(&bars.drain, 1);
    bars.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kSoft + kConv) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem)),
                 "r"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // the split's blocks: places and scales (past the last one: zeros, hidden from every row)
  const int64_t rec = kv_record_bytes(a.c.page_tokens, D);
  const int64_t vplane = int64_t(a.c.page_tokens) * D;
  for (int i = tid; i < 4 * nt; i += kThreads) {
    BlockAt e{-1, 0.f, 0.f, 0.f};
    if (i < cn) {
      const int blk = c0 + i, b = blk % (a.c.page_tokens / kKvBlock);
      const int64_t at = kv_record_of(a.c, s, blk, h, rec);
      if (at >= 0) {
        const uint8_t *sc = a.c.pages + at + 2 * vplane + 4 * b;
        const float ks = __uint_as_float(ld_u1(sc)), vs = __uint_as_float(ld_u1(sc + 4 * (a.c.page_tokens / kKvBlock)));
        e = BlockAt{at + int64_t(b) * kKvBlock * D, ks, vs * kPScale, log2f(fmaxf(vs, kMinScale))};
      } else {
        e.ks = qnan;  // no page: its codes count as 0, its scores are NaN
      }
    }
    s_blk[i] = e;
  }

  // softmax threads: their row's queries, scaled by a power of two, into f16 parts
  const int row = r0 + tid;  // tid < 128
  float qs = 0.f;
  if (warp < kSoft) {
    const bool in = tid < nr;
    const int64_t base = in ? int64_t(q0 + row / a.group) * a.q_stride + int64_t(h * a.group + row % a.group) * D : 0;
    auto load8 = [&](int d, float (&v)[8]) {  // dims d .. d + 7
      if (!in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
      } else if (a.type == QDQ_TYPE_F32) {
        const float4 x = load4(static_cast<const float *>(a.q) + base + d), y = load4(static_cast<const float *>(a.q) + base + d + 4);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
      } else {
        const uint4 u = ld_u4(static_cast<const uint16_t *>(a.q) + base + d);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = a.type == QDQ_TYPE_F16 ? unpack2(w[i], __half{}) : unpack2(w[i], __nv_bfloat16{});
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        }
      }
    };
    float m = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 8) {
      float v[8];
      load8(d, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max_abs_bits(m, v[i]);
    }
    const bool finite = m < __int_as_float(0x7f800000);
    int ex = 13 - (int(__float_as_uint(m) >> 23) - 127);
    ex = max(-120, min(120, ex));
    // the scale's sign goes into the queries, so that a larger product is a larger score
    float up = finite ? __uint_as_float(uint32_t(ex + 127) << 23) : 0.f;
    qs = (finite ? __uint_as_float(uint32_t(127 - ex) << 23) : qnan) * fabsf(a.scale);
    if (a.scale < 0.f) up = -up;
    if (!(a.softcap > 0.f)) qs *= kLog2e;
#pragma unroll 4
    for (int d = 0; d < D; d += 8) {
      float v[8];
      load8(d, v);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = finite ? v[2 * i] * up : 0.f, y = finite ? v[2 * i + 1] * up : 0.f;
        hi[i] = pack2(x, y, __half{});
        const float2 b = unpack2(hi[i], __half{});
        lo[i] = pack2(x - b.x, y - b.y, __half{});
      }
      uint8_t *dst = smem + (d / 64) * (kTcRows * 128) + tid * 128 + (((d % 64 / 8) ^ (tid & 7)) << 4);
      *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if (PARTS == 2) *reinterpret_cast<uint4 *>(dst + C::kQPart) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
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

  float m = ninf, l = 0.f;  // softmax threads: their row's reference and sum
  if (warp < kSoft) {
    const int pos = len - nq + row / a.group;
    const int lo_pos = a.window > 0 ? pos - a.window + 1 : 0;
    const float slope = a.slopes && tid < nr ? __ldg(a.slopes + h * a.group + row % a.group) * kLog2e : 0.f;
    // tokens that every row of the tile sees
    const int all_lo = a.window > 0 ? max(0, pos_hi - a.window + 1) : 0, all_hi = pos_lo + 1;
    const uint32_t lanes = uint32_t(warp * 32) << 16;
    for (int i = 0; i < nt; ++i) {
      const int b = i & 1;
      const uint32_t sp = tmem + lanes + uint32_t(b * BN);
      if (!wait(&bars.sfull[b], i >> 1)) break;
      tc_fence_after();
      uint32_t r[BN];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld16_async(sp + 16 * c, r + 16 * c);
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_wait_ld16(r + 16 * c);
      const int j0 = (c0 + 4 * i) * kKvBlock;
      const bool whole = j0 >= all_lo && j0 + BN <= all_hi;
      float f[4], mx = ninf;
      if (whole && !(a.softcap > 0.f) && !a.slopes) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float bm = __uint_as_float(r[16 * c]);
#pragma unroll
          for (int e = 1; e < 16; ++e) bm = fmaxf(bm, __uint_as_float(r[16 * c + e]));
          f[c] = qs * s_blk[4 * i + c].ks;
          mx = fmaxf(mx, fmaf(bm, f[c], s_blk[4 * i + c].lv));
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float fc = qs * s_blk[4 * i + c].ks;
          float bm = ninf;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int j = j0 + 16 * c + e;
            float x = __uint_as_float(r[16 * c + e]) * fc;
            if (a.softcap > 0.f) x = a.softcap * kLog2e * tanhf(x / a.softcap);
            if (a.slopes) x = fmaf(-slope, float(pos - j), x);
            if (j > pos || j < lo_pos) x = ninf;
            bm = fmaxf(bm, x);
            r[16 * c + e] = __float_as_uint(x);
          }
          mx = fmaxf(mx, bm + s_blk[4 * i + c].lv);
          f[c] = 1.f;
        }
      }
      // the reference is the row's largest score plus log2 of its value scale (see qdq_kv_attn.cu)
      const bool grow = mx > m + (m == ninf ? 0.f : kLazy);
      if (__any_sync(0xffffffffu, grow)) {
        const float m_new = fmaxf(m, mx);
        const float corr = m_new > m ? ex2(m - m_new) : 1.f;
        l *= corr;
        m = m_new;
        if (i > 0) {
          if (!wait(&bars.pvdone[(i - 1) & 1], (i - 1) >> 1)) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld16_async(tmem + lanes + C::kOCol + c, o);
            tmem_wait_ld16(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
            tmem_st16(tmem + lanes + C::kOCol + c, o);
          }
        }
      }
      const float mref = m == ninf ? 0.f : m;
      float2 l2 = f2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float vs = s_blk[4 * i + c].vs;
        const float2 ff = f2(f[c], f[c]), mm = f2(-mref, -mref), vv = f2(vs, vs);
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 x = __ffma2_rn(f2_bits(r[16 * c + 2 * e], r[16 * c + 2 * e + 1]), ff, mm);
          const float2 p = f2(ex2(x.x), ex2(x.y));
          l2 = __fadd2_rn(l2, p);
          float2 pv = __fmul2_rn(p, vv);
          if (!whole) {  // a hidden token's scale may be NaN
            if (x.x == ninf) pv.x = 0.f;
            if (x.y == ninf) pv.y = 0.f;
          }
          hi[e] = pack2(pv.x, pv.y, __half{});
          if (PARTS == 2) {
            const float2 back = unpack2(hi[e], __half{});
            lo[e] = pack2(pv.x - back.x, pv.y - back.y, __half{});
          }
        }
        tmem_st8(sp + 8 * c, hi);
        if (PARTS == 2) tmem_st8(sp + BN / 2 + 8 * c, lo);
      }
      l += l2.x + l2.y;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.pready[b]);
    }
  } else if (warp < kSoft + kConv) {
    // ---------------- codes to f16 tiles ----------------
    const int w = warp - kSoft;
    constexpr int KL = D / 32;          // 16-byte loads of keys per thread: tokens 16 w .. 16 w + 15 of the tile
    constexpr int VG = (D / 32 + 3) / 4;  // groups of 32 dims of the values per warp
    uint4 kq[KL];
    uint2 vq[VG][8];
    const int ktok = lane & 7, kch = lane >> 3;  // row and 16-dim chunk of a load
    const int vtc = lane & 7, vd = lane >> 3;    // 8-token chunk, 8-dim part of the group
    auto load_k = [&](int i) {
      const int64_t at = s_blk[4 * i + w].k;
      const uint8_t *p = a.c.pages + at + ktok * D + kch * 16;
#pragma unroll
      for (int j = 0; j < KL; ++j)  // rows + 8 (j & 1), chunks + 4 (j >> 1)
        kq[j] = at < 0 ? make_uint4(0, 0, 0, 0) : ld_u4(p + (j & 1) * 8 * D + (j >> 1) * 64);
    };
    auto load_v = [&](int i) {
      const int64_t at = s_blk[4 * i + vtc / 2].k;
      const uint8_t *p = a.c.pages + at + vplane + (vtc & 1) * 8 * D + vd * 8;
#pragma unroll
      for (int g = 0; g < VG; ++g)
        if (w + 4 * g < D / 32) {
#pragma unroll
          for (int t = 0; t < 8; ++t) vq[g][t] = at < 0 ? make_uint2(0, 0) : ld_u2(p + t * D + (w + 4 * g) * 32);
        }
    };
    if (nt > 0) {
      load_k(0);
      load_v(0);
    }
    for (int i = 0; i < nt; ++i) {
      const int b = i & 1;
      if (i >= 2 && !wait(&bars.sfull[b], (i - 2) >> 1)) break;  // S of tile i - 2 is done: its keys' tile is free
      uint8_t *kt = kring + b * C::kK;
#pragma unroll
      for (int j = 0; j < KL; ++j) {
        const int rr = 16 * w + 8 * (j & 1) + ktok, ch = kch + 4 * (j >> 1);
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
      if (i + 1 < nt) load_k(i + 1);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.kfull[b]);
      if (i >= 2 && !wait(&bars.pvdone[b], (i - 2) >> 1)) break;  // P V of tile i - 2: its values' tile is free
      uint8_t *vt = vring + b * C::kV;
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
      if (i + 1 < nt) load_v(i + 1);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.vfull[b]);
    }
  } else {
    // ---------------- products ----------------
    const uint32_t leader = elect_lane();
    const uint32_t q_base = smem_u32(smem), k_base = smem_u32(kring), v_base = smem_u32(vring);
    auto scores = [&](int i) {  // S of tile i
      const int b = i & 1;
#pragma unroll
      for (int part = 0; part < PARTS; ++part)
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(leader, tmem + uint32_t(b * BN), desc_sw128(q_base + part * C::kQPart + (k / 4) * (kTcRows * 128) + (k % 4) * 32),
                 desc_sw128(k_base + b * C::kK + (k / 4) * (BN * 128) + (k % 4) * 32), idesc_f16(kTcRows, BN), (part | k) != 0);
      mma_commit(leader, &bars.sfull[b]);
    };
    bool ok = true;
    if (nt > 0) {
      ok = wait(&bars.kfull[0], 0);
      if (ok) {
        tc_fence_after();
        scores(0);
      }
    }
    for (int i = 0; i < nt && ok; ++i) {
      const int b = i & 1;
      if (i + 1 < nt) {
        ok = wait(&bars.kfull[b ^ 1], (i + 1) >> 1);
        // the other S holds the probabilities of tile i - 1 until its products are done
        if (ok && i >= 1) ok = wait(&bars.pvdone[b ^ 1], (i - 1) >> 1);
        if (!ok) break;
        tc_fence_after();
        scores(i + 1);
      }
      ok = wait(&bars.pready[b], i >> 1) && wait(&bars.vfull[b], i >> 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int part = 0; part < PARTS; ++part)
#pragma unroll
        for (int k = 0; k < BN / 16; ++k)
          mma_ts(leader, tmem + C::kOCol, tmem + uint32_t(b * BN + part * (BN / 2) + 8 * k),
                 desc_sw128(v_base + b * C::kV + k * 32), idesc_f16(kTcRows, D), (i | part | k) != 0);
      mma_commit(leader, &bars.pvdone[b]);
    }
    mma_commit(leader, &bars.drain);
  }

  // ---------------- output ----------------
  __syncwarp();
  // every product has completed before the accumulators are read and TMEM is freed
  if (!wait(&bars.drain, 0) && lane == 0) atomicAdd(&g_attn_tc_timeouts, 1u);
  tc_fence_after();
  __syncthreads();
  const bool lost = bad || *reinterpret_cast<volatile int *>(&bars.abort) != 0;
  if (tid == 0 && bars.abort) atomicAdd(&g_attn_tc_timeouts, 1u);
  constexpr int kPart = kTcRows * (D + 2);
  float *part = a.partial + (int64_t(unit) * a.splits + split) * kPart;  // [dim][row], maxima, sums
  if (warp < kSoft) {
    if (lost) l = qnan;
    const float inv = l == 0.f ? 0.f : (1.f / kPScale) / l;
    const bool in = tid < nr;
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      uint32_t o[16];
      if (nt > 0) {
        tmem_ld16_async(tmem + (uint32_t(warp * 32) << 16) + C::kOCol + c, o);
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
        for (int e = 0; e < 16; ++e) part[(c + e) * kTcRows + tid] = __uint_as_float(o[e]);
      }
    }
    if (nsplit == 1) {
      if (in) store_lse(a, q0, h, row, m, l);
    } else {
      part[D * kTcRows + tid] = m;
      part[D * kTcRows + kTcRows + tid] = l;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoft + kConv) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
  }
  if (nsplit == 1) return;

  // the CTA that finishes last joins the splits, in split order
  __threadfence();
  __syncthreads();
  if (tid == 0) bars.last = atomicInc(a.tickets + unit, nsplit - 1) == uint32_t(nsplit - 1);
  __syncthreads();
  if (!bars.last) return;
  __threadfence();
  if (tid >= 2 * kTcRows) return;
  const float *all = a.partial + int64_t(unit) * a.splits * kPart;
  const int jr = tid & (kTcRows - 1), half = tid / kTcRows;  // row, half of the dims
  if (jr >= nr) return;
  float M = ninf, L = 0.f;
  for (int k = 0; k < nsplit; ++k) M = fmaxf(M, __ldcg(all + int64_t(k) * kPart + D * kTcRows + jr));
  const float ref = M == ninf ? 0.f : M;
  for (int k = 0; k < nsplit; ++k)
    L = fmaf(__ldcg(all + int64_t(k) * kPart + (D + 1) * kTcRows + jr), ex2(__ldcg(all + int64_t(k) * kPart + D * kTcRows + jr) - ref), L);
  const float inv = L == 0.f ? 0.f : (1.f / kPScale) / L;
#pragma unroll 1
  for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 16) {
    float v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 0.f;
    for (int k = 0; k < nsplit; ++k) {
      const float f = ex2(__ldcg(all + int64_t(k) * kPart + D * kTcRows + jr) - ref);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = fmaf(__ldcg(all + int64_t(k) * kPart + (d + e) * kTcRows + jr), f, v[e]);
    }
#pragma unroll
    for (int e = 0; e < 16; e += 4) store_out<D>(a, q0, h, r0 + jr, d + e, make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]), inv);
  }
  if (half == 0) store_lse(a, q0, h, r0 + jr, M, L);
}

template <int D, int PARTS>
cudaError_t run(const AttnArgs &a, cudaStream_t s) {
  const auto kernel = attn_tc_kernel<D, PARTS>;
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), int(Cfg<D, PARTS>::kSmem));
  if (e != cudaSuccess) return e;
  const int64_t grid = int64_t(a.n_seqs) * a.c.n_kv * a.tiles * a.splits;
  return launch(kernel, dim3(unsigned(grid)), dim3(kThreads), Cfg<D, PARTS>::kSmem, s, a);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs &a, int head_dim, int parts, cudaStream_t s) {
  switch (head_dim) {
    case 64: return parts == 2 ? run<64, 2>(a, s) : run<64, 1>(a, s);
    case 128: return parts == 2 ? run<128, 2>(a, s) : run<128, 1>(a, s);
    case 192: return parts == 2 ? run<192, 2>(a, s) : run<192, 1>(a, s);
    default: return parts == 1 ? run<256, 1>(a, s) : cudaErrorInvalidValue;
  }
}

int read_attn_tc_timeouts() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_tc_timeouts, sizeof(v)) != cudaSuccess) return -1;
  if (v && cudaMemcpyToSymbol(g_attn_tc_timeouts, &zero, sizeof(zero)) != cudaSuccess) return -1;
  return int(v);
}

}  // namespace qdq
