// Attention of query tokens over the paged 8-bit cache.
//
//   s[j] = scale * q . (kc[j] * ks[j / 16])        (kc, vc: int8 codes; ks, vs: a block's scales)
//   s[j] = cap * tanh(s[j] / cap)                   when cap > 0
//   s[j] -= slope * (pos - j)                       when slopes are given
//   o    = sum_j e^(s[j] - m) vc[j] vs[j / 16] / sum_j e^(s[j] - m)  over the visible j
//
// Rows are (query token, head of the group) pairs that share a key/value head, eight to a tile.
// A warp walks blocks of 16 tokens: the codes go from global memory straight into the operand
// registers of 16-bit matrix instructions (a code is exact in f16), with the next block's loads
// in flight meanwhile.  The instruction has 16 rows: rows 0-7 hold the high f16 part of the eight
// queries (scaled to a power of two below 2^14 per row), rows 8-15 the rest in f16, so the products are exact
// and a score has f32 precision; probabilities are split the same way.  The running maximum,
// the sum and the accumulators are f32.  The four warps of a CTA take every fourth block of
// their split of the tokens and are joined through shared memory; splits of one tile are joined
// by the CTA that finishes last, in split order.
#include <cuda_fp16.h>

#include "qdq_types.cuh"

namespace qdq {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 8;         // rows per tile
constexpr int kMaxSplitBlocks = 128;
constexpr float kPScale = 16384.f;  // probabilities are split into f16 parts at this scale
constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
  KvPool c;
  const int *kv_len, *cu_q;
  const void *q;
  void *out;
  float *lse;
  const float *slopes;
  uint32_t *tickets;
  float *partial;
  int64_t q_stride, out_stride;
  int n_seqs, max_kv_len, n_heads, group, tiles, splits, split_blocks, window, type;
  float scale, softcap;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Bytes 0, 1 (lo) or 2, 3 (hi) of four excess-128 codes as two exact f16: the byte under the
// exponent of 1024, then 1024 + 128 taken off.
template <int SEL>
__device__ __forceinline__ uint32_t codes_f16(uint32_t u) {
  const uint32_t w = __byte_perm(u, 0x64646464u, SEL);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&w), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t *>(&r);
}

template <int N>
struct Words {
  uint32_t w[N];
};
template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *w) {
  if constexpr (BYTES == 16) {
    const uint4 v = ld_u4(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if constexpr (BYTES == 8) {
    const uint2 v = ld_u2(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = ld_u1(p);
  }
}

template <int D>
struct Shape {
  static constexpr int kKB = D % 64 == 0 ? 16 : 8;   // bytes of a key row per lane and load
  static constexpr int kKL = D / (4 * kKB);          // loads per key row
  static constexpr int kKSteps = D / 16;
  static constexpr int kVB = D % 128 == 0 ? 16 : D % 64 == 0 ? 8 : 4;  // of a value row
  static constexpr int kVL = D / (8 * kVB);
  static constexpr int kWords = 2 * D / 16;          // words per lane of a block's keys (and of its values): 2 D / 16
  static constexpr int kNT = D / 8;                  // accumulator tiles of 8 dims
};

// dim of accumulator column n (0..7) of tile j
template <int D>
__device__ __forceinline__ int dim_of(int j, int n) {
  constexpr int VB = Shape<D>::kVB;
  return (j / VB) * 8 * VB + n * VB + j % VB;
}

struct BlockAt {
  int64_t k;  // byte offset of the block's first key code, -1 when it has no page
  float ks, vs;
  float lv;   // log2 of the value scale, at least -95 (a block of zeros has scale 0)
};

// One warp per block of 16 tokens at a time.
template <int D>
__global__ void __launch_bounds__(kWarps * 32, D <= 128 ? 3 : 1) kv_attn_kernel(const AttnArgs a) {
  using S = Shape<D>;
  extern __shared__ uint8_t smem[];
  uint4 *qf = reinterpret_cast<uint4 *>(smem);                           // [k step][lane] A fragments
  float *s_acc = reinterpret_cast<float *>(smem + S::kKSteps * 512);     // [warp][row][D]
  BlockAt *s_blk = reinterpret_cast<BlockAt *>(s_acc + kWarps * kRows * D);
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows], s_w[kWarps][kRows], s_inv[kRows], s_qs[kRows];
  __shared__ int s_last;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x % a.splits;
  const int unit = blockIdx.x / a.splits;  // (sequence, kv head, tile)
  const int tile = unit % a.tiles, h = unit / a.tiles % a.c.n_kv, s = unit / a.tiles / a.c.n_kv;
  pdl_launch_dependents();
  pdl_wait();

  const int q0 = a.cu_q ? int(ld_u1(a.cu_q + s)) : s;
  const int nq = a.cu_q ? int(ld_u1(a.cu_q + s + 1)) - q0 : 1;
  const int len = int(ld_u1(a.kv_len + s));
  const int rows = nq * a.group, r0 = tile * kRows;
  if (r0 >= rows) return;
  const int nr = min(kRows, rows - r0);
  const bool bad = len < 0 || len > a.max_kv_len || (len + a.c.page_tokens - 1) / a.c.page_tokens > a.c.table_stride;
  const int pos_lo = len - nq + r0 / a.group, pos_hi = len - nq + (r0 + nr - 1) / a.group;
  const int b_lo = a.window > 0 ? max(0, pos_lo - a.window + 1) / kKvBlock : 0;
  const int b_hi = bad ? 0 : (pos_hi + kKvBlock) / kKvBlock;  // pos_hi >= -nq: 0 or negative when nothing is visible
  const int nb = max(0, b_hi - b_lo);
  const int nsplit = max(1, (nb + a.split_blocks - 1) / a.split_blocks);
  if (split >= nsplit) return;
  const int c0 = b_lo + split * a.split_blocks, cn = min(a.split_blocks, b_hi - c0);

  // the blocks of this split: where they are and their scales
  const int64_t rec = kv_record_bytes(a.c.page_tokens, D);
  const int64_t vplane = int64_t(a.c.page_tokens) * D;
  for (int i = threadIdx.x; i < cn; i += kWarps * 32) {
    const int blk = c0 + i, t0 = blk * kKvBlock % a.c.page_tokens;
    const int64_t at = kv_record_of(a.c, s, blk, h, rec);
    BlockAt e;
    e.k = at < 0 ? -1 : at + int64_t(t0) * D;
    const uint8_t *sc = a.c.pages + (at < 0 ? 0 : at) + 2 * vplane + 4 * (t0 / kKvBlock);
    e.ks = at < 0 ? __int_as_float(0x7fffffff) : __uint_as_float(ld_u1(sc));
    const float vs = at < 0 ? 1.f : __uint_as_float(ld_u1(sc + 4 * (a.c.page_tokens / kKvBlock)));
    e.lv = log2f(fmaxf(vs, 2.5243549e-29f));  // a NaN scale gives -95 here and stays NaN in vs
    e.vs = vs * kPScale;
    if (e.k < 0) e.k = 0;
    s_blk[i] = e;
  }
  // the tile's queries: scaled by a power of two per row, then split into two f16 parts
  for (int r = warp; r < kRows; r += kWarps) {
    const int row = r0 + r;
    const bool in = r < nr;
    const int64_t base = in ? int64_t(q0 + row / a.group) * a.q_stride + int64_t(h * a.group + row % a.group) * D : 0;
    float v[D / 32];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      v[i] = 0.f;
      if (in) {
        const int64_t e = base + lane + 32 * i;
        v[i] = a.type == QDQ_TYPE_F32   ? load1(static_cast<const float *>(a.q) + e)
               : a.type == QDQ_TYPE_F16 ? load1(static_cast<const __half *>(a.q) + e)
                                        : load1(static_cast<const __nv_bfloat16 *>(a.q) + e);
      }
      m = max_abs_bits(m, v[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_abs_bits(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool finite = m < __int_as_float(0x7f800000);
    // exponent so that the largest element lies in [2^13, 2^14)
    int ex = 13 - (int(__float_as_uint(m) >> 23) - 127);
    ex = max(-120, min(120, ex));
    const float up = finite ? __uint_as_float(uint32_t(ex + 127) << 23) : 0.f;
    if (lane == 0) s_qs[r] = finite ? __uint_as_float(uint32_t(127 - ex) << 23) : __int_as_float(0x7fffffff);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int d = lane + 32 * i;
      const float f = finite ? v[i] * up : 0.f;
      const __half hi = __float2half_rn(f), lo = __float2half_rn(f - __half2float(hi));
      // dim d is element (d % kKB) of lane t = d / kKB % 4 in load d / (4 kKB)
      const int ld = d / (4 * S::kKB), tt = d / S::kKB % 4, e = d % S::kKB;
      const int ks = ld * (S::kKB / 4) + e / 4, el = e % 4;
      __half *f16 = reinterpret_cast<__half *>(qf + ks * 32 + r * 4 + tt);
      f16[(el >> 1) * 4 + (el & 1)] = hi;      // registers 0, 2: rows 0-7
      f16[(el >> 1) * 4 + 2 + (el & 1)] = lo;  // registers 1, 3: rows 8-15
    }
  }
  __syncthreads();

  const int row = r0 + g;  // this lane's row
  const int pos = len - nq + row / a.group;
  const float qs = s_qs[g] * a.scale;
  const float slope = a.slopes && g < nr ? __ldg(a.slopes + h * a.group + row % a.group) * kLog2e : 0.f;
  const int lo_pos = a.window > 0 ? pos - a.window + 1 : 0;

  float acc[S::kNT][4];
#pragma unroll
  for (int j = 0; j < S::kNT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
  float m = -__int_as_float(0x7f800000), l = 0.f;

  uint32_t kw[S::kWords], vw[S::kWords];
  auto load_k = [&](int i) {
    const uint8_t *p = a.c.pages + s_blk[i].k + int64_t(g) * D + t * S::kKB;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < S::kKL; ++c)
        load_words<S::kKB>(p + j * 8 * D + c * 4 * S::kKB, kw + (j * S::kKL + c) * (S::kKB / 4));
  };
  auto load_v = [&](int i) {
    const uint8_t *p = a.c.pages + s_blk[i].k + vplane + int64_t(2 * t) * D + g * S::kVB;
#pragma unroll
    for (int r = 0; r < 4; ++r)  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int c = 0; c < S::kVL; ++c)
        load_words<S::kVB>(p + ((r & 1) + 8 * (r >> 1)) * D + c * 8 * S::kVB, vw + (r * S::kVL + c) * (S::kVB / 4));
  };
  if (warp < cn) {
    load_k(warp);
    load_v(warp);
  }
  for (int i = warp; i < cn; i += kWarps) {
    const float ks = s_blk[i].ks, vs = s_blk[i].vs, lv = s_blk[i].lv;
    // scores: two tiles of 8 tokens
    float sc[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[j][e] = 0.f;
#pragma unroll
      for (int k = 0; k < S::kKSteps; ++k) {
        const uint32_t u = kw[j * S::kKSteps + k] ^ 0x80808080u;
        mma_f16(sc[j], qf[k * 32 + lane], codes_f16<0x4140>(u), codes_f16<0x4342>(u));
      }
    }
    if (i + kWarps < cn) load_k(i + kWarps);
    float p[4];  // tokens 2t, 2t + 1, 2t + 8, 2t + 9 of the block
    const float f = qs * ks;
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = (sc[e >> 1][e & 1] + sc[e >> 1][2 + (e & 1)]) * f;
    if (a.softcap > 0.f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = a.softcap * tanhf(p[e] / a.softcap);
    }
    const int j0 = (c0 + i) * kKvBlock + 2 * t;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = j0 + (e & 1) + 8 * (e >> 1);
      p[e] *= kLog2e;
      if (a.slopes) p[e] = fmaf(-slope, float(pos - j), p[e]);
      if (j > pos || j < lo_pos) p[e] = -__int_as_float(0x7f800000);
    }
    float mx = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // the reference is the row's largest score plus log2 of its value scale: then p * vs is at
    // most 1, so its f16 parts keep their precision however far the blocks' scales lie apart
    const float m_new = fmaxf(m, mx + lv);
    const bool grow = m_new > m;
    if (__any_sync(0xffffffffu, grow)) {
      const float corr = grow ? exp2f(m - m_new) : 1.f;  // 0 from -inf
      l *= corr;
      m = m_new;
#pragma unroll
      for (int j = 0; j < S::kNT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] *= corr;
    }
    const float mref = m == -__int_as_float(0x7f800000) ? 0.f : m;
    float pv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool seen = p[e] != -__int_as_float(0x7f800000);
      p[e] = exp2f(p[e] - mref);
      l += p[e];
      pv[e] = seen ? p[e] * vs : 0.f;  // a hidden token's scale may be NaN
    }
    uint4 pa;
    {
      const __half2 h01 = __floats2half2_rn(pv[0], pv[1]), h23 = __floats2half2_rn(pv[2], pv[3]);
      const float2 f01 = __half22float2(h01), f23 = __half22float2(h23);
      const __half2 l01 = __floats2half2_rn(pv[0] - f01.x, pv[1] - f01.y), l23 = __floats2half2_rn(pv[2] - f23.x, pv[3] - f23.y);
      pa.x = *reinterpret_cast<const uint32_t *>(&h01);
      pa.y = *reinterpret_cast<const uint32_t *>(&l01);
      pa.z = *reinterpret_cast<const uint32_t *>(&h23);
      pa.w = *reinterpret_cast<const uint32_t *>(&l23);
    }
    // values: words of 4 dims of the four tokens, re-paired by token
    constexpr int VW = S::kVL * (S::kVB / 4);  // words per token
#pragma unroll
    for (int c = 0; c < VW; ++c) {
      const uint32_t u0 = vw[c] ^ 0x80808080u, u1 = vw[VW + c] ^ 0x80808080u;
      const uint32_t u2 = vw[2 * VW + c] ^ 0x80808080u, u3 = vw[3 * VW + c] ^ 0x80808080u;
      const uint32_t a01 = __byte_perm(u0, u1, 0x5140), b01 = __byte_perm(u0, u1, 0x7362);
      const uint32_t a23 = __byte_perm(u2, u3, 0x5140), b23 = __byte_perm(u2, u3, 0x7362);
      mma_f16(acc[4 * c + 0], pa, codes_f16<0x4140>(a01), codes_f16<0x4140>(a23));
      mma_f16(acc[4 * c + 1], pa, codes_f16<0x4342>(a01), codes_f16<0x4342>(a23));
      mma_f16(acc[4 * c + 2], pa, codes_f16<0x4140>(b01), codes_f16<0x4140>(b23));
      mma_f16(acc[4 * c + 3], pa, codes_f16<0x4342>(b01), codes_f16<0x4342>(b23));
    }
    if (i + kWarps < cn) load_v(i + kWarps);
  }

  // join the four warps
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (t == 0) {
    s_m[warp][g] = m;
    s_l[warp][g] = l;
  }
  float *mine = s_acc + (warp * kRows + g) * D;
#pragma unroll
  for (int j = 0; j < S::kNT; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) mine[dim_of<D>(j, 2 * t + e)] = acc[j][e] + acc[j][e + 2];
  __syncthreads();
  if (threadIdx.x < kRows) {
    const int r = threadIdx.x;
    float M = -__int_as_float(0x7f800000), L = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
    const float ref = M == -__int_as_float(0x7f800000) ? 0.f : M;
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(s_m[w][r] - ref);
      L = fmaf(s_l[w][r], f, L);
      s_w[w][r] = f / kPScale;
    }
    if (bad) L = __int_as_float(0x7fffffff);
    s_m[0][r] = M;
    s_l[0][r] = L;
  }
  __syncthreads();

  auto finish = [&](int r, int d, float4 v, float inv) {  // four dims of one row
    const int rw = r0 + r;
    const int64_t e = int64_t(q0 + rw / a.group) * a.out_stride + int64_t(h * a.group + rw % a.group) * D + d;
    v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    if (a.type == QDQ_TYPE_F32)
      store4(static_cast<float *>(a.out) + e, v);
    else if (a.type == QDQ_TYPE_F16)
      store4(static_cast<__half *>(a.out) + e, v);
    else
      store4(static_cast<__nv_bfloat16 *>(a.out) + e, v);
  };
  auto write_lse = [&](int r, float M, float L) {
    const int rw = r0 + r;
    if (a.lse)
      a.lse[int64_t(q0 + rw / a.group) * a.n_heads + h * a.group + rw % a.group] =
          L == 0.f ? -__int_as_float(0x7f800000) : (M + log2f(L)) * 0.6931471805599453f;
  };

  float *part = a.partial + (int64_t(unit) * a.splits + split) * (kRows * (D + 2));
  for (int i = threadIdx.x; i < nr * (D / 4); i += kWarps * 32) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 x = *reinterpret_cast<const float4 *>(s_acc + (w * kRows + r) * D + d);
      const float f = s_w[w][r];
      v = make_float4(fmaf(x.x, f, v.x), fmaf(x.y, f, v.y), fmaf(x.z, f, v.z), fmaf(x.w, f, v.w));
    }
    if (nsplit == 1) {
      const float L = s_l[0][r];
      finish(r, d, v, L == 0.f ? 0.f : 1.f / L);
    } else {
      *reinterpret_cast<float4 *>(part + r * D + d) = v;
    }
  }
  if (nsplit == 1) {
    if (threadIdx.x < nr) write_lse(threadIdx.x, s_m[0][threadIdx.x], s_l[0][threadIdx.x]);
    return;
  }
  if (threadIdx.x < nr) {
    part[kRows * D + threadIdx.x] = s_m[0][threadIdx.x];
    part[kRows * D + kRows + threadIdx.x] = s_l[0][threadIdx.x];
  }
  // the CTA that finishes last joins the splits, in split order; the ticket wraps to 0 for the next call
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicInc(a.tickets + unit, nsplit - 1) == uint32_t(nsplit - 1);
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const float *all = a.partial + int64_t(unit) * a.splits * (kRows * (D + 2));
  const int step = kRows * (D + 2);
  if (threadIdx.x < nr) {
    const int r = threadIdx.x;
    float M = -__int_as_float(0x7f800000), L = 0.f;
    for (int i = 0; i < nsplit; ++i) M = fmaxf(M, __ldcg(all + i * step + kRows * D + r));
    const float ref = M == -__int_as_float(0x7f800000) ? 0.f : M;
    for (int i = 0; i < nsplit; ++i)
      L = fmaf(__ldcg(all + i * step + kRows * D + kRows + r), exp2f(__ldcg(all + i * step + kRows * D + r) - ref), L);
    s_m[0][r] = ref;
    s_inv[r] = L == 0.f ? 0.f : 1.f / L;
    write_lse(r, M, L);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nr * (D / 4); i += kWarps * 32) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < nsplit; ++k) {
      const float4 x = __ldcg(reinterpret_cast<const float4 *>(all + k * step + r * D + d));
      const float f = exp2f(__ldcg(all + k * step + kRows * D + r) - s_m[0][r]);
      v = make_float4(fmaf(x.x, f, v.x), fmaf(x.y, f, v.y), fmaf(x.z, f, v.z), fmaf(x.w, f, v.w));
    }
    finish(r, d, v, s_inv[r]);
  }
}

template <int D>
size_t attn_smem() {
  return Shape<D>::kKSteps * 512 + size_t(kWarps) * kRows * D * 4 + size_t(kMaxSplitBlocks) * sizeof(BlockAt);
}

template <typename F>
int with_dim(int d, F &&f) {
  switch (d) {
    case 64: return f(std::integral_constant<int, 64>{});
    case 96: return f(std::integral_constant<int, 96>{});
    case 128: return f(std::integral_constant<int, 128>{});
    case 192: return f(std::integral_constant<int, 192>{});
    default: return f(std::integral_constant<int, 256>{});
  }
}

struct Plan {
  int tiles, splits, split_blocks;
  int64_t units;
  size_t ticket_bytes, bytes;
};

Plan plan(const DeviceInfo &di, int n_seqs, int max_q, int max_kv_len, int n_heads, int n_kv, int head_dim) {
  Plan p{};
  p.tiles = int((int64_t(max_q) * (n_heads / n_kv) + kRows - 1) / kRows);
  p.units = int64_t(n_seqs) * n_kv * p.tiles;
  const int64_t blocks = (int64_t(max_kv_len) + kKvBlock - 1) / kKvBlock;
  // enough CTAs for a few waves of three per SM, but no fewer than two blocks per warp and split
  const int64_t want = int64_t(di.sm_count) * 3 * 2;
  int64_t per = blocks * p.units / (want > 0 ? want : 1);
  if (per < 2 * kWarps) per = 2 * kWarps;
  if (per > kMaxSplitBlocks) per = kMaxSplitBlocks;
  p.split_blocks = int(per);
  p.splits = int((blocks + per - 1) / per);
  if (p.splits < 1) p.splits = 1;
  p.ticket_bytes = (size_t(p.units) * 4 + 255) / 256 * 256;
  p.bytes = p.ticket_bytes + (p.splits > 1 ? size_t(p.units) * p.splits * kRows * (head_dim + 2) * 4 : 0);
  return p;
}

}  // namespace

size_t kv_attention_workspace_bytes(int n_seqs, int max_q, int max_kv_len, int n_heads, int n_kv, int head_dim) {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return 0;
  return plan(di, n_seqs, max_q, max_kv_len, n_heads, n_kv, head_dim).bytes;
}

int launch_kv_attention(const KvPool &c, int head_dim, const int *kv_len, const int *cu_q, int n_seqs, int max_q,
                        int max_kv_len, int n_heads, const void *q, int64_t q_stride, void *out, int64_t out_stride,
                        float *lse, const float *slopes, float scale, float softcap, int window, int type,
                        void *workspace, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return fail_cuda(e);
  const Plan p = plan(di, n_seqs, max_q, max_kv_len, n_heads, c.n_kv, head_dim);
  if (p.units * p.splits > 0x7fffffff) return QDQ_ERR_UNSUPPORTED;
  AttnArgs a{};
  a.c = c;
  a.kv_len = kv_len;
  a.cu_q = cu_q;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.slopes = slopes;
  a.tickets = static_cast<uint32_t *>(workspace);
  a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + p.ticket_bytes);
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.n_seqs = n_seqs;
  a.max_kv_len = max_kv_len;
  a.n_heads = n_heads;
  a.group = n_heads / c.n_kv;
  a.tiles = p.tiles;
  a.splits = p.splits;
  a.split_blocks = p.split_blocks;
  a.window = window;
  a.type = type;
  a.scale = scale;
  a.softcap = softcap;
  e = cudaError_t(with_dim(head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    const size_t sm = attn_smem<D>();
    const cudaError_t r = allow_dynamic_smem(reinterpret_cast<const void *>(kv_attn_kernel<D>), int(sm));
    if (r != cudaSuccess) return int(r);
    return int(launch(kv_attn_kernel<D>, dim3(unsigned(p.units * p.splits)), dim3(kWarps * 32), sm, s, a));
  }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

}  // namespace qdq
