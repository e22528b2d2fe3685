// Attention of query tokens over the paged 8-bit cache.
//
//   s[j] = scale * q . (kc[j] * ks[j / 16])        (kc, vc: int8 codes; ks, vs: a block's scales)
//   s[j] = cap * tanh(s[j] / cap)                   when cap > 0
//   s[j] -= slope * (pos - j)                       when slopes are given
//   o    = sum_j e^(s[j] - m) vc[j] vs[j / 16] / sum_j e^(s[j] - m)  over the visible j
//
// Rows are (query token, head of the group) pairs that share a key/value head.  A warp walks
// blocks of 16 tokens: their codes come through a ring of asynchronous copies in its own part of
// shared memory (16-byte chunks exchanged by row so that the fragment loads below meet no bank
// conflict) and become the operands of 16-row matrix instructions with 16-bit operands (a code
// is exact in f16).  A query row is scaled by a power of two to below 2^14 first.
//   two parts (f32 activations; a tile is 8 rows): instruction rows 0-7 hold the high f16 part
//     of the queries, rows 8-15 the rest in f16, so the products are exact and a score has f32
//     precision; the probabilities are split the same way.
//   one part (16-bit activations with more than 8 rows per head; a tile is 16 rows): the queries
//     are exact in f16 but for elements 2^-25 below the row's largest, the
//     probabilities are rounded to f16 (2^-11 relative, as the output is).
// The running maximum, the sum and the accumulators are f32.  The warps of a CTA (4, or 16 or 8
// where there are few tiles) take blocks of their split of the tokens in turn and are joined through
// shared memory; splits of one tile are joined by the CTA that finishes last, in split order.
// Bound: memory for many or long sequences (a code is read once for all rows of its head); for a short one the
// chain of a launch, length, page, codes, joins.  Measured (8 heads of 128 in the cache): one sequence of
// 777 tokens, 24 heads f32 9.0 us; 48 of 1 to 8191 78.5 us (5.2 TB/s, 76 % of a plain copy's rate); one of 131071
// tokens, 32 heads bf16 50.6 us (5.3 TB/s, 78 %).
#include <algorithm>

#include "qdq_kv_attn.cuh"

namespace qdq {

std::atomic<int> g_opt_attn_kernel{0};

namespace {

constexpr int kStages = 3;       // blocks in a warp's ring
constexpr int kMaxEntries = 128;  // sequences times tiles up to which the splits' length is chosen on the device
// Blocks of 16 tokens in a split from which on its length is chosen on the device: the choice costs 1.6 us (8
// sequences of 8000 tokens bf16, heads of 64: 20.6 -> 22.2 us), but sequences of different lengths share the SMs evenly (4
// of 2000 to 20000 f32: 33.9 -> 24.0 us; 8 of 100 to 8000: 29.4 -> 23.6 us).  Small CTAs even out by themselves
// (48 of 1 to 8191: 79 us, with the choice 94 us).
constexpr int kEvenBlocks = 192;
constexpr int kMinBlocks = 4;     // of a split, per warp: a split costs its join (about 3 us)
// Splits of one tile (the joining CTA keeps their maxima and sums in shared memory), and blocks
// of 16 tokens in one split.
constexpr int max_splits(int warps) { return warps > 4 ? 512 : 64; }
constexpr int max_split_blocks(int warps) { return warps > 4 ? 512 : 128; }
static_assert(int64_t(max_splits(8)) * max_split_blocks(8) * kKvBlock == QDQ_MAX_KV_LEN, "the longest cache");

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

template <int BYTES>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t *w) {
  if constexpr (BYTES == 16) {
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  } else if constexpr (BYTES == 8) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  }
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int D>
struct Shape {
  static constexpr int kKB = D % 64 == 0 ? 16 : 8;   // bytes of a key row per lane and load
  static constexpr int kKL = D / (4 * kKB);          // loads per key row
  static constexpr int kKSteps = D / 16;
  static constexpr int kVB = D % 128 == 0 ? 16 : D % 64 == 0 ? 8 : 4;  // of a value row
  static constexpr int kVL = D / (8 * kVB);
  static constexpr int kNT = D / 8;                  // accumulator tiles of 8 dims
  static constexpr int kPlane = kKvBlock * D;        // bytes of a block's keys (and of its values)
  static constexpr int kRing = kStages * 2 * kPlane;
};

// First dim of lane t's load `ld` of a key row: neighbouring lanes' loads lie kKL loads apart
// where rows are whole 128-byte lines, so that even and odd rows meet in different banks.
template <int D>
__device__ __forceinline__ int key_dim(int t, int ld) {
  constexpr int KB = Shape<D>::kKB;
  if constexpr (D == 128 || D == 256) return (ld / 2) * 128 + (2 * t + ld % 2) * KB;
  return (4 * ld + t) * KB;
}
// Byte offset of 16-byte chunk c of row r within a block's plane in shared memory.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (D == 128 || D == 256) return uint32_t(r * D + ((c ^ (r & 7)) * 16));
  if constexpr (D == 64) {  // two rows to a 128-byte line
    const int l = r >> 1, p = (r & 1) * 4 + c;
    return uint32_t(l * 128 + ((p ^ ((l & 3) * 2)) * 16));
  }
  return uint32_t(r * D + c * 16);
}

// dim of accumulator column n (0..7) of tile j
template <int D>
__device__ __forceinline__ int dim_of(int j, int n) {
  constexpr int VB = Shape<D>::kVB;
  return (j / VB) * 8 * VB + n * VB + j % VB;
}

// Bytes of the rings, which the warps' accumulators and the join of the splits use afterwards
// (a maximum and a sum per split and row, and a float4 per thread).
template <int D, int PARTS, int W>
constexpr int body_bytes() {
  constexpr int ring = W * Shape<D>::kRing, acc = W * (16 / PARTS) * D * 4;
  constexpr int join = 2 * max_splits(W) * (16 / PARTS) * 4 + W * 32 * 16;
  constexpr int most = ring > acc ? ring : acc;
  return most > join ? most : join;
}

// Place of four dims (quad c) in a row of accumulators in shared memory: exchanged so that the
// lanes of one store, which hold dims 32 or 16 apart of rows a whole number of lines apart, meet
// in different banks (unexchanged, a one-token call took 1.5 us longer).
__device__ __forceinline__ int quad_at(int row, int c) { return c ^ (((c >> 3) & 3) | ((row & 1) << 2)); }

// PARTS = 2: 8 rows per tile in two f16 parts; 1: 16 rows.  W warps.  EVEN: the splits' length follows all
// sequences' lengths, else it is at most a.split_blocks.
template <int D, int PARTS, int W, bool EVEN>
__global__ void __launch_bounds__(W * 32, (D <= 128 ? 16 : 8) / W) kv_attn_kernel(const AttnArgs a) {
  constexpr int kThreads = W * 32;
  using S = Shape<D>;
  constexpr int R = 16 / PARTS;  // rows of a tile
  constexpr int NR = 2 / PARTS;  // rows per lane: g, and g + 8 with one part
  extern __shared__ __align__(128) uint8_t smem[];
  uint4 *qf = reinterpret_cast<uint4 *>(smem);                         // [k step][lane] query fragments
  uint8_t *ring = smem + S::kKSteps * 512;                             // [warp][stage] keys, values
  float *s_acc = reinterpret_cast<float *>(ring);                      // at the end: [warp][row][D]
  constexpr int kBody = body_bytes<D, PARTS, W>();
  BlockAt *s_blk = reinterpret_cast<BlockAt *>(ring + kBody);
  __shared__ float s_m[W][R], s_l[W][R], s_w[W][R], s_inv[R], s_qs[R];
  __shared__ int s_last;
  const float ninf = __int_as_float(0xff800000), qnan = __int_as_float(0x7fffffff);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_launch_dependents();
  pdl_wait();

  // rows and blocks of one tile of a sequence
  struct Tile {
    int q0, nq, len, nr, b_lo, nb;
    bool bad;
  };
  auto tile_of = [&](int s, int tile) {
    Tile x;
    x.q0 = a.cu_q ? int(ld_u1(a.cu_q + s)) : s;
    x.nq = a.cu_q ? int(ld_u1(a.cu_q + s + 1)) - x.q0 : 1;
    x.len = int(ld_u1(a.kv_len + s));
    const int r0 = tile * R, rows = x.nq * a.group;
    x.nr = min(min(R, a.max_rows - r0), rows - r0);
    x.bad = x.len < 0 || x.len > a.max_kv_len || (x.len + a.c.page_tokens - 1) / a.c.page_tokens > a.c.table_stride;
    const int pos_lo = x.len - x.nq + int(a.query_of(r0)), pos_hi = x.len - x.nq + int(a.query_of(r0 + max(x.nr, 1) - 1));
    x.b_lo = a.window > 0 ? max(0, pos_lo - a.window + 1) / kKvBlock : 0;
    // pos_hi >= -nq: 0 or negative when nothing is visible
    x.nb = x.bad ? 0 : max(0, (pos_hi + kKvBlock) / kKvBlock - x.b_lo);
    return x;
  };
  int s, h, tile, split, nsplit, per;  // this CTA's: blocks of a split
  int64_t first;                       // its unit's first part
  Tile me;
  if constexpr (!EVEN) {
    split = blockIdx.x % a.splits;
    const int u = blockIdx.x / a.splits;  // (sequence, kv head, tile)
    tile = u % a.tiles;
    h = u / a.tiles % a.c.n_kv;
    s = u / a.tiles / a.c.n_kv;
    me = tile_of(s, tile);
    // in large CTAs a sequence far below max_kv_len is cut into as many splits as one at it (one of 4000
    // tokens under a bound of 131072: 24.0 us in one split)
    per = W > 4 ? min(a.split_blocks, max(kMinBlocks * W, int(float(me.nb) * a.inv_splits) + 1)) : a.split_blocks;
    nsplit = max(1, (me.nb + per - 1) / per);
    if (me.nr <= 0 || split >= nsplit) return;
    first = int64_t(u) * a.splits;
  } else {
    // Every warp by itself: the shortest splits of which there are no more than CTAs (their length grows by the
    // excess until that holds), then the entry (sequence, tile) of this CTA, and its head and split.
    constexpr int kPer = kMaxEntries / 32;
    int blocks[kPer];  // of entry 32 j + lane; -1: no rows
    int total = 0, most = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = 32 * j + lane;
      blocks[j] = -1;
      if (e < a.entries) {
        const Tile x = tile_of(e / a.tiles, e % a.tiles);
        if (x.nr > 0) blocks[j] = x.nb;
        total += max(blocks[j], 0);
        most = max(most, blocks[j]);
      }
    }
    total = __reduce_add_sync(0xffffffffu, total);
    most = __reduce_max_sync(0xffffffffu, most);
    const int ctas = gridDim.x / a.c.n_kv;  // for one head
    per = max(max(kMinBlocks * W, (most + max_splits(W) - 1) / max_splits(W)), (total + ctas - 1) / ctas);
    int n[kPer];
    for (;;) {
      per = min(per, max_split_blocks(W));
      int sum = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        n[j] = blocks[j] < 0 ? 0 : max(1, (blocks[j] + per - 1) / per);
        sum += n[j];
      }
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (sum <= ctas || per == max_split_blocks(W)) break;
      per += (per * (sum - ctas) + ctas - 1) / ctas;
    }
    int off = 0, found = -1, cnt = 0, at = 0;  // off: parts (of all heads) before entry 32 j
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (32 * j >= a.entries) break;
      const int mine = n[j] * a.c.n_kv;
      int up = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += x;
      }
      const uint32_t who = __ballot_sync(0xffffffffu, int(blockIdx.x) >= off + up - mine && int(blockIdx.x) < off + up);
      if (who) {
        const int l = __ffs(who) - 1;
        found = 32 * j + l;
        cnt = __shfl_sync(0xffffffffu, n[j], l);
        at = off + __shfl_sync(0xffffffffu, up - mine, l);
        break;
      }
      off += __shfl_sync(0xffffffffu, up, 31);
    }
    if (found < 0) return;  // more CTAs than parts
    s = found / a.tiles;
    tile = found % a.tiles;
    nsplit = cnt;
    h = (int(blockIdx.x) - at) / cnt;
    split = (int(blockIdx.x) - at) % cnt;
    first = at + int64_t(h) * cnt;
    me = tile_of(s, tile);
    per = max(1, (me.nb + cnt - 1) / cnt);  // the unit's splits alike
  }
  const int unit = (s * a.c.n_kv + h) * a.tiles + tile;
  const int q0 = me.q0, nq = me.nq, len = me.len, nr = me.nr, r0 = tile * R;
  const bool bad = me.bad;
  const int b_lo = me.b_lo, b_hi = me.b_lo + me.nb;
  const int c0 = b_lo + split * per, cn = max(0, min(per, b_hi - c0));
  if (!QDQ_GUARD(cn <= max_split_blocks(W) && nsplit <= max_splits(W), QDQ_CHECK_SMEM)) return;
  if (nsplit > 1 && !QDQ_GUARD((first + nsplit) * (R * (D + 2)) <= a.room && unit < a.units, QDQ_CHECK_OUT)) return;

  // where the blocks of this split are
  const int64_t rec = kv_record_bytes(a.c.page_tokens, D);
  const int64_t vplane = int64_t(a.c.page_tokens) * D;
  for (int i = threadIdx.x; i < cn; i += kThreads) {
    const int blk = c0 + i, t0 = blk % (a.c.page_tokens / kKvBlock) * kKvBlock;
    const int64_t at = kv_record_of(a.c, s, blk, h, rec);
    s_blk[i].k = (at < 0 ? 0 : at) + int64_t(t0) * D;
    s_blk[i].ks = at < 0 ? qnan : 0.f;  // without a page: any valid place, and marked
  }
  __syncthreads();

  const uint32_t my_ring = smem_u32(ring) + warp * S::kRing;
  auto fetch = [&](int i, int stage) {  // this warp's copies of block i
    if (i < cn) {
      const uint8_t *k = a.c.pages + s_blk[i].k;
      const uint32_t dst = my_ring + stage * 2 * S::kPlane;
      constexpr int CR = D / 16;  // chunks per row
#pragma unroll
      for (int j = 0; j < CR / 2; ++j) {  // 16 rows x CR chunks over 32 lanes
        const int e = lane + 32 * j, r = e / CR, c = e % CR;
        copy16(dst + chunk_at<D>(r, c), k + e * 16);
        copy16(dst + S::kPlane + chunk_at<D>(r, c), k + vplane + e * 16);
      }
    }
    copies_commit();
  };
  // the queries' and the scales' loads first, all in flight together: behind the ring's copies
  // they would come microseconds later
  constexpr int QR = (R + W - 1) / W;  // rows per warp
  float qv[QR][D / 32];
#pragma unroll
  for (int i = 0; i < QR; ++i) {
    const int r = warp + i * W, row = r0 + r;
    const bool in = r < nr;
    const int qi = int(a.query_of(row));
    const int64_t base = in ? int64_t(q0 + qi) * a.q_stride + int64_t(h * a.group + row - qi * a.group) * D + lane : 0;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      qv[i][j] = 0.f;
      if (in)
        qv[i][j] = a.type == QDQ_TYPE_F32   ? load1(static_cast<const float *>(a.q) + base + 32 * j)
                   : a.type == QDQ_TYPE_F16 ? load1(static_cast<const __half *>(a.q) + base + 32 * j)
                                            : load1(static_cast<const __nv_bfloat16 *>(a.q) + base + 32 * j);
    }
  }
  auto scales = [&](int i, float &ks, float &vs) {
    const int b = (c0 + i) % (a.c.page_tokens / kKvBlock);  // of its page
    const uint8_t *sc = a.c.pages + (s_blk[i].k - int64_t(b) * S::kPlane + 2 * vplane + 4 * b);
    ks = __uint_as_float(ld_u1(sc));
    vs = __uint_as_float(ld_u1(sc + 4 * (a.c.page_tokens / kKvBlock)));
  };
  auto keep = [&](int i, float ks, float vs) {
    const bool none = s_blk[i].ks != 0.f;  // no page: NaN scores
    s_blk[i].lv = log2f(fmaxf(none ? 1.f : vs, kMinScale));  // a NaN scale gives -95 here and stays NaN in vs
    s_blk[i].vs = none ? 1.f : vs * kPScale;
    if (!none) s_blk[i].ks = ks;
  };
  float ks0 = 0.f, vs0 = 0.f;
  if (int(threadIdx.x) < cn) scales(threadIdx.x, ks0, vs0);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(warp + i * W, i);
  if (int(threadIdx.x) < cn) keep(threadIdx.x, ks0, vs0);
  for (int i = threadIdx.x + kThreads; i < cn; i += kThreads) {
    scales(i, ks0, vs0);
    keep(i, ks0, vs0);
  }
  // the tile's queries: scaled by a power of two per row, then f16 parts
#pragma unroll
  for (int qi = 0; qi < QR; ++qi) {
    const int r = warp + qi * W;
    if (r >= R) break;
    const float(&v)[D / 32] = qv[qi];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) m = max_abs_bits(m, v[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_abs_bits(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool finite = m < __int_as_float(0x7f800000);
    // exponent so that the largest element lies in [2^13, 2^14)
    int ex = 13 - (int(__float_as_uint(m) >> 23) - 127);
    ex = max(-120, min(120, ex));
    const float up = finite ? __uint_as_float(uint32_t(ex + 127) << 23) : 0.f;
    if (lane == 0) s_qs[r] = finite ? __uint_as_float(uint32_t(127 - ex) << 23) : qnan;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int d = lane + 32 * i;
      const float f = finite ? v[i] * up : 0.f;
      const __half hi = __float2half_rn(f);
      int ld, tt;  // the load and the lane that bring dim d
      if constexpr (D == 128 || D == 256) {
        const int c = d / 16;
        ld = (c / 8) * 2 + (c & 1);
        tt = (c % 8) / 2;
      } else {
        ld = d / (4 * S::kKB);
        tt = d / S::kKB % 4;
      }
      const int e = d % S::kKB, ks = ld * (S::kKB / 4) + e / 4, el = e % 4;
      __half *f16 = reinterpret_cast<__half *>(qf + ks * 32 + (r & 7) * 4 + tt) + (el >> 1) * 4 + (el & 1);
      if constexpr (PARTS == 2) {
        f16[0] = hi;                                       // registers 0, 2: rows 0-7
        f16[2] = __float2half_rn(f - __half2float(hi));  // registers 1, 3: rows 8-15
      } else {
        f16[r >= 8 ? 2 : 0] = hi;
      }
    }
  }
  __syncthreads();

  int pos[NR], lo_pos[NR];
  float qs[NR], slope[NR], m[NR], l[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int lr = g + 8 * r, row = r0 + lr;
    const int qi = int(a.query_of(row));
    pos[r] = len - nq + qi;
    lo_pos[r] = a.window > 0 ? pos[r] - a.window + 1 : 0;
    qs[r] = s_qs[lr] * a.scale * (a.softcap > 0.f ? 1.f : kLog2e);
    slope[r] = a.slopes && lr < nr ? __ldg(a.slopes + h * a.group + row - qi * a.group) * kLog2e : 0.f;
    m[r] = ninf;
    l[r] = 0.f;
  }
  // blocks in [full_lo, full_hi) are visible to every row of the tile
  const int pos_lo = len - nq + int(a.query_of(r0)), pos_hi = len - nq + int(a.query_of(r0 + nr - 1));
  const int full_lo = a.window > 0 ? max(0, pos_hi - a.window + 1 + kKvBlock - 1) / kKvBlock : 0;
  const int full_hi = (pos_lo + 1) / kKvBlock;

  float acc[S::kNT][4];
#pragma unroll
  for (int j = 0; j < S::kNT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

  // fragment addresses within a stage
  uint32_t ka[S::kKL], va[4];  // a row's 8 rows down and the other chunks are fixed distances where nothing is exchanged
#pragma unroll
  for (int c = 0; c < S::kKL; ++c) {
    const int d = key_dim<D>(t, c);
    ka[c] = my_ring + chunk_at<D>(g, d / 16) + d % 16;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int d = g * S::kVB;
    va[r] = my_ring + S::kPlane + chunk_at<D>(2 * t + (r & 1) + 8 * (r >> 1), d / 16) + d % 16;
  }

  int stage = 0;
  for (int i = warp; i < cn; i += W) {
    copies_wait<kStages - 2>();
    __syncwarp();  // every lane's copies of this block are in, and the stage refilled next is free
    fetch(i + (kStages - 1) * W, stage == 0 ? kStages - 1 : stage - 1);
    const uint32_t so = stage * 2 * S::kPlane;
    stage = stage == kStages - 1 ? 0 : stage + 1;
    // scores: two tiles of 8 tokens
    float sc[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[j][e] = 0.f;
#pragma unroll
    for (int c = 0; c < S::kKL; ++c) {
      uint32_t w[2][4];
      lds_words<S::kKB>(ka[c] + so, w[0]);
      lds_words<S::kKB>(ka[c] + so + 8 * D, w[1]);
#pragma unroll
      for (int k = 0; k < S::kKB / 4; ++k) {
        const uint4 q = qf[(c * (S::kKB / 4) + k) * 32 + lane];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t u = w[j][k] ^ 0x80808080u;
          mma_f16(sc[j], q, codes_f16<0x4140>(u), codes_f16<0x4342>(u));
        }
      }
    }
    const float ks = s_blk[i].ks, vs = s_blk[i].vs, lv = s_blk[i].lv;
    const int blk = c0 + i;
    const bool whole = blk >= full_lo && blk < full_hi;
    float p[NR][4];  // tokens 2t, 2t + 1, 2t + 8, 2t + 9 of the block
    float mx[NR];
    bool grow = false;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float f = qs[r] * ks;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        p[r][e] = (PARTS == 2 ? sc[e >> 1][e & 1] + sc[e >> 1][2 + (e & 1)] : sc[e >> 1][2 * r + (e & 1)]) * f;
      if (a.softcap > 0.f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) p[r][e] = a.softcap * kLog2e * tanh_of<PARTS == 2>(p[r][e] * a.inv_cap);
      }
      const int j0 = blk * kKvBlock + 2 * t;
      if (a.slopes) {
#pragma unroll
        for (int e = 0; e < 4; ++e) p[r][e] = fmaf(-slope[r], float(pos[r] - (j0 + (e & 1) + 8 * (e >> 1))), p[r][e]);
      }
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + (e & 1) + 8 * (e >> 1);
          if (j > pos[r] || j < lo_pos[r]) p[r][e] = ninf;
        }
      }
      mx[r] = fmaxf(fmaxf(p[r][0], p[r][1]), fmaxf(p[r][2], p[r][3]));
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      // the reference is the row's largest score plus log2 of its value scale: then p * vs is at
      // most 1 (2^kLazy while the reference is behind), so its f16 parts keep their precision
      // however far the blocks' scales lie apart
      mx[r] += lv;
      grow |= mx[r] > m[r] + (m[r] == ninf ? 0.f : kLazy);
    }
    if (__any_sync(0xffffffffu, grow)) {
      float corr[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float m_new = fmaxf(m[r], mx[r]);
        corr[r] = m_new > m[r] ? ex2(m[r] - m_new) : 1.f;  // 0 from -inf
        l[r] *= corr[r];
        m[r] = m_new;
      }
#pragma unroll
      for (int j = 0; j < S::kNT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] *= corr[PARTS == 2 ? 0 : e >> 1];
    }
    uint4 pa;
    {
      float pv[NR][4];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float mref = m[r] == ninf ? 0.f : m[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = ex2(p[r][e] - mref);
          l[r] += x;
          pv[r][e] = x * vs;
        }
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (p[r][e] == ninf) pv[r][e] = 0.f;  // a hidden token's scale may be NaN
        }
      }
      const __half2 h01 = __floats2half2_rn(pv[0][0], pv[0][1]), h23 = __floats2half2_rn(pv[0][2], pv[0][3]);
      __half2 l01, l23;
      if constexpr (PARTS == 2) {
        const float2 f01 = __half22float2(h01), f23 = __half22float2(h23);
        l01 = __floats2half2_rn(pv[0][0] - f01.x, pv[0][1] - f01.y);
        l23 = __floats2half2_rn(pv[0][2] - f23.x, pv[0][3] - f23.y);
      } else {
        l01 = __floats2half2_rn(pv[NR - 1][0], pv[NR - 1][1]);
        l23 = __floats2half2_rn(pv[NR - 1][2], pv[NR - 1][3]);
      }
      pa.x = *reinterpret_cast<const uint32_t *>(&h01);
      pa.y = *reinterpret_cast<const uint32_t *>(&l01);
      pa.z = *reinterpret_cast<const uint32_t *>(&h23);
      pa.w = *reinterpret_cast<const uint32_t *>(&l23);
    }
    // values: words of 4 dims of the four tokens, re-paired by token
#pragma unroll
    for (int c = 0; c < S::kVL; ++c) {
      uint32_t w[4][S::kVB / 4];
#pragma unroll
      for (int r = 0; r < 4; ++r) lds_words<S::kVB>(va[r] + so + c * 8 * S::kVB, w[r]);
#pragma unroll
      for (int k = 0; k < S::kVB / 4; ++k) {
        const uint32_t u0 = w[0][k] ^ 0x80808080u, u1 = w[1][k] ^ 0x80808080u;
        const uint32_t u2 = w[2][k] ^ 0x80808080u, u3 = w[3][k] ^ 0x80808080u;
        const uint32_t a01 = __byte_perm(u0, u1, 0x5140), b01 = __byte_perm(u0, u1, 0x7362);
        const uint32_t a23 = __byte_perm(u2, u3, 0x5140), b23 = __byte_perm(u2, u3, 0x7362);
        float(*o)[4] = acc + c * S::kVB + 4 * k;
        mma_f16(o[0], pa, codes_f16<0x4140>(a01), codes_f16<0x4140>(a23));
        mma_f16(o[1], pa, codes_f16<0x4342>(a01), codes_f16<0x4342>(a23));
        mma_f16(o[2], pa, codes_f16<0x4140>(b01), codes_f16<0x4140>(b23));
        mma_f16(o[3], pa, codes_f16<0x4342>(b01), codes_f16<0x4342>(b23));
      }
    }
  }
  copies_wait<0>();
  __syncthreads();  // every warp is done with its ring, which becomes s_acc

  // join the warps
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    if (t == 0) {
      s_m[warp][g + 8 * r] = m[r];
      s_l[warp][g + 8 * r] = l[r];
    }
    float4 *mine = reinterpret_cast<float4 *>(s_acc + (warp * R + g + 8 * r) * D);
#pragma unroll
    for (int j = 0; j < S::kNT; j += 4)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        auto v = [&](int i) { return PARTS == 2 ? acc[j + i][e] + acc[j + i][e + 2] : acc[j + i][2 * r + e]; };
        mine[quad_at(g, dim_of<D>(j, 2 * t + e) / 4)] = make_float4(v(0), v(1), v(2), v(3));
      }
  }
  __syncthreads();
  if (threadIdx.x < R) {
    const int r = threadIdx.x;
    float M = ninf, L = 0.f;
    for (int w = 0; w < W; ++w) M = fmaxf(M, s_m[w][r]);
    const float ref = M == ninf ? 0.f : M;
    for (int w = 0; w < W; ++w) {
      const float f = ex2(s_m[w][r] - ref);
      L = fmaf(s_l[w][r], f, L);
      s_w[w][r] = f / kPScale;
    }
    if (bad) L = qnan;
    s_m[0][r] = M;
    s_l[0][r] = L;
  }
  __syncthreads();

  float *part = a.partial + (first + split) * (R * (D + 2));
  for (int i = threadIdx.x; i < nr * (D / 4); i += kThreads) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float4 x = reinterpret_cast<const float4 *>(s_acc + (w * R + r) * D)[quad_at(r, d / 4)];
      const float f = s_w[w][r];
      v = make_float4(fmaf(x.x, f, v.x), fmaf(x.y, f, v.y), fmaf(x.z, f, v.z), fmaf(x.w, f, v.w));
    }
    if (nsplit == 1) {
      const float L = s_l[0][r];
      store_out<D>(a, q0, h, r0 + r, d, v, L == 0.f ? 0.f : 1.f / L);
    } else {
      *reinterpret_cast<float4 *>(part + r * D + d) = v;
    }
  }
  if (nsplit == 1) {
    if (int(threadIdx.x) < nr) store_lse(a, q0, h, r0 + threadIdx.x, s_m[0][threadIdx.x], s_l[0][threadIdx.x]);
    return;
  }
  if (int(threadIdx.x) < nr) {
    part[R * D + threadIdx.x] = s_m[0][threadIdx.x];
    part[R * D + R + threadIdx.x] = s_l[0][threadIdx.x];
  }
  // the CTA that finishes last joins the splits, in split order; the ticket wraps to 0 for the next call
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicInc(a.tickets + unit, nsplit - 1) == uint32_t(nsplit - 1);
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // maxima and sums into shared memory, weights from them, then the accumulators: thread
  // (k, item) adds every KG-th split's four dims of one row, the KG sums are added in order
  const int step = R * (D + 2);
  const float *all = a.partial + first * step;
  float *w_m = s_acc, *w_l = s_acc + nsplit * R;
  for (int i = threadIdx.x; i < nsplit * R; i += kThreads) {
    const float *p = all + int64_t(i / R) * step + R * D + i % R;
    w_m[i] = __ldcg(p);
    w_l[i] = __ldcg(p + R);
  }
  __syncthreads();
  for (int r = warp; r < nr; r += W) {
    float M = ninf, L = 0.f;
    for (int i = lane; i < nsplit; i += 32) M = fmaxf(M, w_m[i * R + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == ninf ? 0.f : M;
    for (int i = lane; i < nsplit; i += 32) {
      const float f = ex2(w_m[i * R + r] - ref);
      w_m[i * R + r] = f;
      L = fmaf(w_l[i * R + r], f, L);
    }
    L = warp_sum(L);
    if (lane == 0) {
      s_inv[r] = L == 0.f ? 0.f : 1.f / L;
      store_lse(a, q0, h, r0 + r, M, L);
    }
  }
  __syncthreads();
  float4 *s_sum = reinterpret_cast<float4 *>(s_acc + (2 * nsplit * R + 3) / 4 * 4);  // [k][item]
  const int items = nr * (D / 4);
  const int KG = items >= kThreads ? 1 : min(8, kThreads / items);
  for (int i = threadIdx.x; i < items * KG; i += kThreads) {
    const int kg = i / items, it = i % items, r = it / (D / 4), d = it % (D / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = kg; k < nsplit; k += KG) {
      const float4 x = __ldcg(reinterpret_cast<const float4 *>(all + int64_t(k) * step + r * D + d));
      const float f = w_m[k * R + r];
      v = make_float4(fmaf(x.x, f, v.x), fmaf(x.y, f, v.y), fmaf(x.z, f, v.z), fmaf(x.w, f, v.w));
    }
    if (KG == 1)
      store_out<D>(a, q0, h, r0 + r, d, v, s_inv[r]);
    else
      s_sum[i] = v;
  }
  if (KG == 1) return;
  __syncthreads();
  for (int it = threadIdx.x; it < items; it += kThreads) {
    float4 v = s_sum[it];
    for (int kg = 1; kg < KG; ++kg) {
      const float4 x = s_sum[kg * items + it];
      v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
    }
    const int r = it / (D / 4);
    store_out<D>(a, q0, h, r0 + r, it % (D / 4) * 4, v, s_inv[r]);
  }
}

template <int D, int PARTS, int W>
size_t attn_smem() {
  return Shape<D>::kKSteps * 512 + body_bytes<D, PARTS, W>() + size_t(max_split_blocks(W)) * sizeof(BlockAt);
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

// Query rows per key/value head from which on the tensor-core kernel runs.  This file's kernel is kept all the same
// where its tiles do not outnumber the SMs (each is then an SM's, split over idle ones) and a CTA's context is at
// most kTcMinTokens, and where all rows' tokens times dims are at most kTcMinWork.  Us here and there, 24 / 8 heads
// of 128: 8 sequences of up to 6000 tokens, 8 queries bf16 39 52, 16 71 52, 64 146 67; 48 of up to 3000, 16
// queries bf16 123 157, 22 176 158; one of 4000, 64 queries bf16 28 42, 128 84 45, 43 queries f32 25 46; 30 queries
// f32 over 16000 90 57; a prompt of 100 queries over 1000 f32 31 42, 4 of 64 over 1000 bf16 50 37; 8 / 8 heads,
// 300 queries over 600 f32 21 43; heads of 64, 512 queries over themselves f32 20 34, bf16 29 30.
constexpr int kTcMinRows = 64, kTcMinTokens = 6000;
constexpr int64_t kTcMinWork = 340'000'000;

struct Plan {
  bool tc;  // the tensor-core kernel of qdq_kv_attn_tc.cu
  int parts, groups, warps, tiles, splits, split_blocks, entries, ctas;
  int64_t units;
  size_t bytes;  // of the workspace, for any window
};

Plan plan(const DeviceInfo &di, int n_seqs, int max_q, int max_kv_len, int n_heads, int n_kv, int head_dim, int window,
          int type) {
  Plan p{};
  const int64_t rows = int64_t(max_q) * (n_heads / n_kv);
  p.parts = type != QDQ_TYPE_F32 && rows > 8 ? 1 : 2;
  const int64_t small = int64_t(n_seqs) * n_kv * ((rows * p.parts + 15) / 16);  // tiles of the other kernel
  const bool few = small <= di.sm_count && max_kv_len / (di.sm_count / small) <= kTcMinTokens;
  // Blocks without a window.  A window's are never more, or its plan could want a larger workspace.
  const int64_t all_blocks = (int64_t(max_kv_len) + kKvBlock - 1) / kKvBlock;
  const int64_t tokens_seen = std::max<int64_t>(1, int64_t(max_kv_len) - max_q / 2);
  const bool light = int64_t(n_seqs) * n_kv * rows * head_dim <= kTcMinWork / tokens_seen;
  const int forced = g_opt_attn_kernel.load(std::memory_order_relaxed);
  p.tc = (forced == 2 || (forced == 0 && rows > kTcMinRows && !few && !light)) && (type == QDQ_TYPE_F32 || p.parts == 1) &&
         attn_tc_supported(head_dim, p.parts);
  if (p.tc) {
    p.groups = rows > kTcRows && head_dim <= 128 ? 2 : 1;
    const int R = kTcRows * p.groups;
    p.tiles = int((rows + R - 1) / R);
    p.units = int64_t(n_seqs) * n_kv * p.tiles;
    int64_t tokens = max_kv_len;
    if (window > 0 && tokens > int64_t(window) + R) tokens = int64_t(window) + R;
    const int64_t blocks = std::min(all_blocks, (tokens + kKvBlock - 1) / kKvBlock + (window > 0));
    // whole waves of CTAs (one per SM), each with at most kTcSplitBlocks of the blocks there can be
    const int64_t most = p.units * ((blocks + 4) / 4 + kTcPartCost);  // tiles of 64 tokens and parts' costs
    const int64_t wave = int64_t(di.sm_count) * (kTcSplitBlocks / 4);
    const int64_t ctas = di.sm_count * ((most + wave - 1) / wave);
    p.splits = int(ctas < 0x7fffffff ? ctas : 0);
    p.bytes = workspace_for(size_t(p.units), 2 * size_t(ctas) * attn_tc_part_bytes(head_dim, p.groups));
    return p;
  }
  const int R = 16 / p.parts;
  p.tiles = int((rows + R - 1) / R);
  p.units = small;
  // blocks a tile can see: its rows span at most R queries
  int64_t tokens = max_kv_len;
  if (window > 0 && tokens > int64_t(window) + R) tokens = int64_t(window) + R;
  const int64_t blocks = std::min(all_blocks, (tokens + kKvBlock - 1) / kKvBlock + (window > 0));
  const int resident = head_dim <= 128 ? 16 : 8;  // warps per SM
  // Few tiles: CTAs that fill an SM, so that a tile is cut into few splits; many: small CTAs,
  // whose starts and ends overlap with their neighbours' work.
  p.warps = p.units <= di.sm_count || blocks > int64_t(max_splits(4)) * max_split_blocks(4) ? resident : 4;
  const int64_t per_wave = int64_t(di.sm_count) * (resident / p.warps);
  // small CTAs: four waves of them, so that sequences of different lengths even out (48 sequences
  // of up to 8K tokens, 24 / 8 heads of 128: 78 us; two waves 87 us, eight 89 us)
  int64_t splits = p.warps == 4 ? 4 * per_wave / p.units : per_wave / p.units;
  if (splits < 1) splits = 1;
  if (splits > max_splits(p.warps)) splits = max_splits(p.warps);
  int64_t per = (blocks + splits - 1) / splits;
  if (per < kMinBlocks * p.warps) per = kMinBlocks * p.warps;
  if (per > max_split_blocks(p.warps)) per = max_split_blocks(p.warps);
  p.split_blocks = int(per);
  p.splits = int((blocks + per - 1) / per);
  if (p.splits < 1) p.splits = 1;
  p.ctas = p.units * p.splits <= 0x7fffffff ? int(p.units * p.splits) : 0;
  // sequences of their own lengths: splits whose length the device chooses (above), as many as CTAs are aimed at
  const int64_t aim = p.warps == 4 ? 4 * per_wave : per_wave, entries = int64_t(n_seqs) * p.tiles;
  if (entries <= kMaxEntries && p.warps > 4 && n_seqs > 1 && per >= kEvenBlocks) {
    const int64_t least = entries * ((blocks + max_split_blocks(p.warps) - 1) / max_split_blocks(p.warps));
    const int64_t per_head = std::max(std::max(aim / n_kv, entries), least);
    p.entries = int(entries);
    p.ctas = per_head * n_kv <= 0x7fffffff ? int(per_head * n_kv) : 0;
  }
  // Parts there can be, with any window: another one can want either size of CTA.  More CTAs than units cut a unit;
  // as many do where the device chooses the splits, since a sequence without queries leaves its CTAs to the others.
  const bool chosen = n_seqs > 1 && entries <= kMaxEntries && p.units <= di.sm_count;
  int64_t slots = chosen ? p.units : 0;
  for (int warps : {4, resident})
    if (warps == resident || p.units > di.sm_count) {
      const int64_t to = (warps == 4 ? 4 : 1) * int64_t(di.sm_count) * (resident / warps);
      const int64_t forced = p.units * ((all_blocks + max_split_blocks(warps) - 1) / max_split_blocks(warps));
      for (int64_t n : {to, forced})
        if (n > p.units && n > slots) slots = n;
    }
  p.bytes = workspace_for(size_t(p.units), size_t(slots) * R * (head_dim + 2) * 4);
  return p;
}

}  // namespace

size_t kv_attention_workspace_bytes(int n_seqs, int max_q, int max_kv_len, int n_heads, int n_kv, int head_dim) {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return 0;
  size_t most = 0;  // enough for every element type
  for (int type : {QDQ_TYPE_F32, QDQ_TYPE_BF16}) {
    const size_t b = plan(di, n_seqs, max_q, max_kv_len, n_heads, n_kv, head_dim, 0, type).bytes;
    if (b > most) most = b;
  }
  return most;
}

int launch_kv_attention(const KvPool &c, int head_dim, const int *kv_len, const int *cu_q, int n_seqs, int max_q,
                        int max_kv_len, int n_heads, const void *q, int64_t q_stride, void *out, int64_t out_stride,
                        float *lse, const float *slopes, float scale, float softcap, int window, int type,
                        void *workspace, size_t workspace_bytes, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return fail_cuda(e);
  // a window that hides nothing is none, and a position less a smaller one stays within 32 bits
  if (window >= max_kv_len) window = 0;
  const Plan p = plan(di, n_seqs, max_q, max_kv_len, n_heads, c.n_kv, head_dim, window, type);
  if (p.splits < 1 || p.units > 0x7fffffff || (!p.tc && p.ctas < 1)) return QDQ_ERR_UNSUPPORTED;
  AttnArgs a{};
  a.c = c;
  a.kv_len = kv_len;
  a.cu_q = cu_q;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.slopes = slopes;
  a.tickets = static_cast<uint32_t *>(workspace);
  a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + workspace_tickets(workspace_bytes));
  a.room = int64_t((workspace_bytes - workspace_tickets(workspace_bytes)) / 4);
  a.units = p.units;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.n_seqs = n_seqs;
  a.max_q = max_q;
  a.max_rows = max_q * (n_heads / c.n_kv);
  a.max_kv_len = max_kv_len;
  a.n_heads = n_heads;
  a.group = n_heads / c.n_kv;
  a.group_mul = ((uint64_t(1) << 40) + uint64_t(a.group) - 1) / uint64_t(a.group);
  a.tiles = p.tiles;
  a.splits = p.splits;
  a.split_blocks = p.split_blocks;
  a.inv_splits = 1.f / float(p.splits);
  a.entries = p.entries;
  a.window = window;
  a.type = type;
  a.scale = scale;
  a.softcap = softcap;
  a.inv_cap = softcap > 0.f ? 1.f / softcap : 0.f;
  if (p.tc) {
    e = launch_attn_tc(a, head_dim, p.parts, p.groups, s);
    return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
  }
  e = cudaError_t(with_dim(head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    constexpr int W = D <= 128 ? 16 : 8;
    auto run = [&](auto kernel, size_t sm) {
      const cudaError_t r = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), int(sm));
      if (r != cudaSuccess) return int(r);
      return int(launch(kernel, dim3(unsigned(p.ctas)), dim3(p.warps * 32), sm, s, a));
    };
    if (p.warps == 4)
      return p.parts == 2 ? run(kv_attn_kernel<D, 2, 4, false>, attn_smem<D, 2, 4>()) : run(kv_attn_kernel<D, 1, 4, false>, attn_smem<D, 1, 4>());
    if (p.entries > 0)
      return p.parts == 2 ? run(kv_attn_kernel<D, 2, W, true>, attn_smem<D, 2, W>())
                          : run(kv_attn_kernel<D, 1, W, true>, attn_smem<D, 1, W>());
    return p.parts == 2 ? run(kv_attn_kernel<D, 2, W, false>, attn_smem<D, 2, W>())
                        : run(kv_attn_kernel<D, 1, W, false>, attn_smem<D, 1, W>());
  }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

QDQ_CHECK_READER(read_checks_attn)

}  // namespace qdq
