// Log probabilities of given tokens, the entropy and the top alternatives of each row of
// logits, in one pass over the logits.
//
//   lse = log sum_i e^x_i,  logprob = x_t - lse,  entropy = lse - sum_i e^(x_i - lse) x_i
//   top: the k first of the order of qdq_topk_rows, with their log probabilities
//
// A row is cut into segments (one CTA each) of tiles of 4096 logits.  Each thread brings its own
// 16 logits of the next tiles by asynchronous copies into shared memory (no barrier: it alone reads
// them; in registers the compiler moved such loads behind the arithmetic).  A thread keeps its own running maximum M, l = sum 2^y and
// u = sum 2^y y with y = (x - M) log2(e) (the difference first: a mask of the type's lowest value
// must not turn into an infinity), so the tiles need no barrier for the sums; the threads'
// triples are joined at the end.  The top k: the k-th largest of 64 maxima (each over the
// same number of logits), taken after 1, 2, 4, ... tiles, is a lower bound of the row's k-th best, so only the few
// logits at or above it become 64-bit keys, in a list per warp; a list that fills is cut to its best 64 by
// the warp.  What the lists hold at the end is ranked by counting the larger keys (all threads
// at once; sorting networks of one warp took three times as long) or, where they are many, folded
// by sorting networks.  Segments of one row are joined by the CTA that finishes last: the k-th
// largest of the segments' first few keys bounds what has to be ranked.
// Bound: memory for many rows, with the arithmetic close behind (5 instructions and one exponential per
// logit); for one row the chain of a launch, two loads, the joins.  Measured: 300 rows of 128256 f32 with 5
// alternatives 32.9 us (4.7 TB/s, without alternatives 28.6 us), one row with 20 9.2 us.
#include <type_traits>

#include "qdq_types.cuh"

namespace qdq {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;                     // logits per thread and tile
constexpr int kTile = kThreads * kPer;
constexpr int kTop = QDQ_MAX_TOPK;
constexpr int kWarps = kThreads / 32;
constexpr int kList = 64 + 32;              // a warp's keys: 64 kept and one more of each lane
constexpr int kStages = 3;                  // tiles in flight or in work
constexpr int kBuf = 2048;                  // keys of other segments sorted at a time
constexpr int kRank = 256;                  // keys that are ranked by counting
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kBehind = 16.f;             // natural units
constexpr float kLn2 = 0.6931471805599453f;

struct LpArgs {
  const void *logits;
  int64_t stride;
  const int *tokens;
  float *logprob, *entropy, *top_logprob;
  int *top_index;
  uint32_t *tickets;
  uint8_t *partial;  // [row][segment] { float M, l, u, pad; uint64 keys[k] }
  int n, k, segs, seg_tiles;
  int64_t room, rows;  // bytes of the workspace's parts, rows (read by the debug build's guards)
};

// Bytes of a segment's partial result, a multiple of 16.
__host__ __device__ constexpr size_t part_bytes(int k) { return 16 + size_t(k + 1) / 2 * 16; }

struct Stat {
  float m, l, u;  // the reference M, sum 2^y, sum 2^y y
};
// The larger reference; NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Exponent that moves sums from reference `from` to `to` (a NaN passes; 2^-1000 is 0 and
// its product with any finite sum finite).
__device__ __forceinline__ float shift_of(float from, float to) { return max_nan((from - to) * kLog2e, -1000.f); }
__device__ __forceinline__ Stat join(const Stat &a, const Stat &b) {
  Stat r;
  r.m = max_nan(a.m, b.m);
  const float da = a.l == 0.f ? 0.f : shift_of(a.m, r.m), db = b.l == 0.f ? 0.f : shift_of(b.m, r.m);
  const float ea = exp2f(da), eb = exp2f(db);
  r.l = a.l * ea + b.l * eb;
  r.u = ea * fmaf(a.l, da, a.u) + eb * fmaf(b.l, db, b.u);
  return r;
}
__device__ __forceinline__ Stat shfl_stat(const Stat &a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.l, o), __shfl_xor_sync(0xffffffffu, a.u, o)};
}

__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

struct Shared {
  union {
    uint4 tile[kStages][kPer / 4][kThreads];  // (16-bit logits use half)
    struct {  // after the tiles
      uint64_t buf[kBuf], rank[kRank], list[kWarps / 2][64];
    };
  };
  uint64_t lists[kWarps][kList];  // the warps' keys
  uint64_t top[kTop];             // best so far, descending, 0 past the end
  uint32_t group[128];
  Stat stat[kWarps];
  int fill[kWarps];              // keys in each warp's list
  int count;
  uint64_t bound;                // keys at or below it are not among the k best
  int last;
};

__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = uint32_t(key >> 32);
  return o == 0xFFFFFFFFu ? __int_as_float(0x7fffffff) : __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// The best of the n <= kRank keys of sh.rank, sorted, into sh.top (0 past the n-th); keys that are
// not 0 are distinct.  All threads call it; sh.rank is written before a barrier.
__device__ void rank_keys(Shared &sh, int n) {
  const int tid = threadIdx.x;
  int share = 1;  // threads per key
  while (share < 8 && 2 * share * n <= kThreads) share *= 2;
  if (tid < kTop) sh.top[tid] = 0;
  __syncthreads();
  const int i = tid / share, part = tid % share;
  const uint64_t mine = i < n ? sh.rank[i] : 0ull;
  int r = 0;
#pragma unroll 8
  for (int j = part; j < n; j += share) r += sh.rank[j] > mine;
  for (int o = 1; o < share; o *= 2) r += __shfl_xor_sync(0xffffffffu, r, o);
  if (part == 0 && i < n && mine != 0 && r < kTop) sh.top[r] = mine;
  __syncthreads();
}

// The best 64 of `count` keys (not among sh.list), sorted, into sh.top.  All threads call it; count
// is the same for all, the keys are written before a barrier.
__device__ void sort_keys(Shared &sh, const uint64_t *keys, int count) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t a = 0, b = 0;
  for (int base = 64 * warp; base < count; base += 64 * kWarps) {
    uint64_t c = base + lane < count ? keys[base + lane] : 0ull;
    uint64_t d = base + 32 + lane < count ? keys[base + 32 + lane] : 0ull;
    warp_sort64_desc(c, d, lane);
    if (base == 64 * warp) {
      a = c;
      b = d;
    } else {
      warp_top64_merge(a, b, c, d, lane);
    }
  }
  for (int half = kWarps / 2; half >= 1; half >>= 1) {
    if (warp >= half && warp < 2 * half) {
      sh.list[warp - half][lane] = a;
      sh.list[warp - half][lane + 32] = b;
    }
    __syncthreads();
    if (warp < half) warp_top64_merge(a, b, sh.list[warp][lane], sh.list[warp][lane + 32], lane);
    __syncthreads();
  }
  if (warp == 0) {
    sh.top[lane] = a;
    sh.top[lane + 32] = b;
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LpArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared &sh = *reinterpret_cast<Shared *>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = blockIdx.x % a.segs, row = blockIdx.x / a.segs;
  const int k = a.k;
  constexpr int V = 16 / int(sizeof(T));  // elements per 16-byte load
  pdl_launch_dependents();
  pdl_wait();
  const T *x = static_cast<const T *>(a.logits) + int64_t(row) * a.stride;
  // elements are counted from the 16-byte boundary at or below the row's start
  const int shift = int((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const T *x0 = x - shift;
  const int lo = shift, hi = shift + a.n;  // valid elements of x0
  if (tid < kWarps) sh.fill[tid] = 0;
  if (tid == 0) sh.count = 0;
  const float ninf = __int_as_float(0xff800000);
  Stat st{ninf, 0.f, 0.f};
  const int e0 = seg * a.seg_tiles * kTile;  // below 2^30 + a tile, as hi is
  const int e1 = min(hi, e0 + a.seg_tiles * kTile);

  // this thread's logits of the tile at `base` into stage n, -inf outside the row
  const uint32_t mine = smem_u32(&sh.tile[0][0][tid]);
  constexpr uint32_t kStageBytes = sizeof(sh.tile[0]);
  auto fetch = [&](int base, int n) {
    if (base < e1) {
      const T *p = x0 + base + tid * V;
      const uint32_t dst = mine + uint32_t(n) * kStageBytes;
      if (base >= lo && base + kTile <= hi) {  // inside the row
#pragma unroll
        for (int i = 0; i < kPer / V; ++i)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * (kThreads * 16)), "l"(p + i * (kThreads * V)) : "memory");
      } else {
#pragma unroll 1
        for (int i = 0; i < kPer / V; ++i) {
          const int e = base + (i * kThreads + tid) * V;
          if (e >= lo && e + V <= hi) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * (kThreads * 16)), "l"(x0 + e) : "memory");
          } else {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if constexpr (sizeof(T) == 4) {
                w[j] = e + j >= lo && e + j < hi ? ld_u1(x0 + e + j) : 0xff800000u;
              } else {
                const uint32_t pad = std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
                const uint32_t p0 = e + 2 * j >= lo && e + 2 * j < hi ? ld_h1(x0 + e + 2 * j) : pad;
                const uint32_t p1 = e + 2 * j + 1 >= lo && e + 2 * j + 1 < hi ? ld_h1(x0 + e + 2 * j + 1) : pad;
                w[j] = p0 | (p1 << 16);
              }
            }
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + i * (kThreads * 16)), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  uint64_t *list = sh.lists[warp];
  uint64_t bound = 0;        // this warp's: keys at or below it are not among the k best
  float bound_v = ninf, rm = ninf;  // rm: the largest of this thread's logits
  int done = 0;              // tiles
  const bool many = k > 48;
  // tiles after which no new bound is taken: fewer than about 40 keys would be saved (300 rows of 128256 f32,
  // k = 5: one bound 37.4 us, this 32.9; bf16, k = 40: 68.6 and 46.9; 2000 rows of 32000 bf16, k = 5, always 50.7, this 46.8)
  const int until = max(1, k > 0 ? a.seg_tiles - 40 / k : 0);
#pragma unroll
  for (int t = 0; t < kStages - 1; ++t) fetch(e0 + t * kTile, t);
  __syncthreads();
  for (int n = 0, base = e0; base < e1; base += kTile) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer / V; ++i) {
      uint4 held;
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(held.x), "=r"(held.y), "=r"(held.z), "=r"(held.w)
                   : "r"(mine + uint32_t(n) * kStageBytes + i * (kThreads * 16))
                   : "memory");
      const uint32_t ww[4] = {held.x, held.y, held.z, held.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          v[4 * i + j] = __uint_as_float(ww[j]);
        } else {
          const float2 f = unpack2(ww[j], T{});
          v[V * i + 2 * j] = f.x;
          v[V * i + 2 * j + 1] = f.y;
        }
      }
    }
    fetch(base + (kStages - 1) * kTile, n == 0 ? kStages - 1 : n - 1);
    n = n == kStages - 1 ? 0 : n + 1;
    float tm = v[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) tm = max_nan(tm, v[i]);
    // the reference moves only when it has fallen kBehind behind (2^(kBehind log2 e) is far from the
    // largest f32), which is rare; a NaN becomes the reference and stays it
    if (!(tm <= st.m + kBehind)) {
      const float m2 = max_nan(st.m, tm);
      const float d = st.l == 0.f ? 0.f : shift_of(st.m, m2), e = exp2f(d);
      st.u = e * fmaf(st.l, d, st.u);
      st.l *= e;
      st.m = m2;
    }
    const float ref = st.m == ninf ? 0.f : st.m;
    float2 tl = f2(0.f, 0.f), tu = f2(0.f, 0.f);
    const float yref = ref * kLog2e;
    const float2 nref = f2(-yref, -yref), log2e = f2(kLog2e, kLog2e);
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      const float2 d = __ffma2_rn(f2(v[i], v[i + 1]), log2e, nref);
      const float2 e = f2(ex2_approx(d.x), ex2_approx(d.y));
      tl = __fadd2_rn(tl, e);
      tu = __ffma2_rn(e, d, tu);
    }
    float l = tl.x + tl.y, u = tu.x + tu.y;
    // the exponents above are all too large by rho = ref log2(e) - yref, a rounding: first-order corrections
    const float rho = fmaf(ref, kLog2e, -yref);
    u = fmaf(-rho * kLn2, u, fmaf(-rho, l, u));
    l = fmaf(-rho * kLn2, l, l);
    // 0 * -inf of a masked logit, a NaN (it stays one in l), or a reference so large that rho is not
    // small: once more, the difference first and the exponent limited
    if (u != u || fabsf(ref) > 1024.f) {
      l = u = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float d = shift_of(v[i], ref), e = ex2_approx(d);
        l += e;
        u = fmaf(e, d, u);
      }
    }
    st.l += l;
    st.u += u;
    if (k > 0) {
      // A bound, after 1, 2, 4, ... tiles: the k-th largest of 64 groups' maxima so far (128 from 49 up: of
      // 64 groups' maxima the 64th lets some 300 logits of a tile by, of 128 some 90: 406 rows of 21944 f32, k = 64, 136
      // and 31 us; bf16 rows of 128256, k = 40, 47 and 51 us).  (With the first
      // tile's alone every tile has about k logits above it, and half the warps have one.)
      rm = max_nan(rm, tm);
      if (done < until && (done & (done + 1)) == 0) {
        float gm = max_nan(rm, __shfl_xor_sync(0xffffffffu, rm, 1));
        if (!many) gm = max_nan(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
        const uint32_t mine = uint32_t(topk_key(gm, 0u) >> 32);  // its order; NaN the largest
        const int size = many ? 2 : 4, i = tid / size, part = tid % size;
        if (part == 0) sh.group[i] = mine;
        __syncthreads();
        int r = 0;
#pragma unroll 4
        for (int j = part; j < kThreads / size; j += size) r += sh.group[j] > mine || (sh.group[j] == mine && j < i);
        r += __shfl_xor_sync(0xffffffffu, r, 1);
        if (!many) r += __shfl_xor_sync(0xffffffffu, r, 2);
        if (part == 0 && r == k - 1) sh.bound = uint64_t(mine) << 32;  // below every key of this value
        __syncthreads();
        const uint64_t b = sh.bound;
        if (b > bound && key_value(b) > ninf) {  // not padding alone, nor NaN
          bound = b;
          bound_v = key_value(b);
        }
      }
      ++done;
      uint32_t which = 0;  // of this thread's logits, those that may be among the best: rarely any
      if (!(tm < bound_v)) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) which |= v[i] < bound_v ? 0u : 1u << i;
      }
      while (__any_sync(0xffffffffu, which != 0)) {  // one more of each lane
        if (which) {
          const int i = __ffs(which) - 1;
          which &= which - 1;
          float x = v[0];
#pragma unroll
          for (int j = 1; j < kPer; ++j) x = i == j ? v[j] : x;
          const int e = base + ((i / V) * kThreads + tid) * V + i % V;
          const uint64_t key = topk_key(x, uint32_t(e - shift));
          if (e >= lo && e < hi && key > bound) {
            const int at = atomicAdd(&sh.fill[warp], 1);
            if (QDQ_GUARD(at < kList, QDQ_CHECK_SMEM)) list[at] = key;
          }
        }
        __syncwarp();
        const int fill = *reinterpret_cast<volatile int *>(&sh.fill[warp]);
        if (fill > 64) {  // the next 32 may not fit: the warp keeps its best k
          uint64_t p = list[lane], q = list[lane + 32];
          uint64_t c = 64 + lane < fill ? list[64 + lane] : 0ull, d = 0ull;
          warp_sort64_desc(p, q, lane);
          warp_sort64_desc(c, d, lane);
          warp_top64_merge(p, q, c, d, lane);
          __syncwarp();
          list[lane] = p;
          list[lane + 32] = q;
          const uint64_t pk = __shfl_sync(0xffffffffu, p, (k - 1) & 31), qk = __shfl_sync(0xffffffffu, q, (k - 1) & 31);
          bound = k <= 32 ? pk : qk;
          bound_v = key_value(bound);
          if (lane == 0) sh.fill[warp] = k;
        }
        __syncwarp();
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (k > 0) {  // the warps' lists into one, and its best k
    __syncthreads();  // from here the tiles' space is used for keys
    int at[kWarps], count = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      at[w] = count;
      count += sh.fill[w];
    }
    if (count > kRank) {  // many: without those that a later bound has passed
      const uint64_t low = sh.bound;
      for (int i = lane; i < sh.fill[warp]; i += 32)
        if (list[i] > low) {
          const int to = atomicAdd(&sh.count, 1);
          if (to < kRank) sh.rank[to] = list[i];
        }
      __syncthreads();
      count = sh.count;
      __syncthreads();
      if (tid == 0) sh.count = 0;
    } else {
      for (int i = lane; i < sh.fill[warp]; i += 32) sh.rank[at[warp] + i] = list[i];
      __syncthreads();
    }
    if (count <= kRank) {
      rank_keys(sh, count);
    } else {  // many: sorted, in the lists' places
      for (int i = lane; i < kList; i += 32)
        if (i >= sh.fill[warp]) list[i] = 0;
      __syncthreads();
      sort_keys(sh, sh.lists[0], kWarps * kList);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) st = join(st, shfl_stat(st, o));
  if (lane == 0) sh.stat[warp] = st;
  __syncthreads();
  if (warp == 0) {
    st = lane < kWarps ? sh.stat[lane] : Stat{ninf, 0.f, 0.f};
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) st = join(st, shfl_stat(st, o));
    if (lane == 0) sh.stat[0] = st;
  }
  __syncthreads();

  if (a.segs > 1) {
    const size_t part = part_bytes(k);
    if (!QDQ_GUARD(int64_t((size_t(row) + 1) * a.segs * part) <= a.room && row < a.rows, QDQ_CHECK_OUT)) return;
    uint8_t *mine = a.partial + (size_t(row) * a.segs + seg) * part;
    if (tid == 0) {
      float *f = reinterpret_cast<float *>(mine);
      f[0] = sh.stat[0].m;
      f[1] = sh.stat[0].l;
      f[2] = sh.stat[0].u;
    }
    if (tid < k) reinterpret_cast<uint64_t *>(mine + 16)[tid] = sh.top[tid];
    __threadfence();
    __syncthreads();
    if (tid == 0) sh.last = atomicInc(a.tickets + row, a.segs - 1) == uint32_t(a.segs - 1);
    __syncthreads();
    if (!sh.last) return;
    __threadfence();
    const uint8_t *all = a.partial + size_t(row) * a.segs * part;
    Stat t{ninf, 0.f, 0.f};
    for (int i = tid; i < a.segs; i += kThreads) {
      const float4 f = __ldcg(reinterpret_cast<const float4 *>(all + i * part));
      t = join(t, Stat{f.x, f.y, f.z});
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t = join(t, shfl_stat(t, o));
    if (lane == 0) sh.stat[warp] = t;
    if (k > 0) {
      auto key_of = [&](int i, int j) {  // j-th key of segment i
        return __ldcg(reinterpret_cast<const unsigned long long *>(all + size_t(i) * part + 16) + j);
      };
      // the k-th largest of every segment's first `few` keys bounds the k-th best of all
      const int few = (k + a.segs - 1) / a.segs, n0 = few * a.segs;
      uint64_t low = 0;
      if (n0 <= kRank) {
        for (int i = tid; i < n0; i += kThreads) sh.rank[i] = key_of(i / few, i % few);
        if (tid == 0) sh.count = 0;
        rank_keys(sh, n0);
        low = sh.top[k - 1];
        __syncthreads();
      }
      const int total = a.segs * k;
      for (int i = tid; i < total; i += kThreads) {
        const uint64_t key = key_of(i / k, i % k);
        if (key >= low && key != 0) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kRank) sh.rank[at] = key;
        }
      }
      __syncthreads();
      const int count = sh.count;
      __syncthreads();
      if (count <= kRank) {
        rank_keys(sh, count);
      } else {  // many equal bounds: all keys, as many as fit at a time, with the best of those before
        int have = 0;
        for (int base = 0; base < total; base += kBuf - kTop) {
          const int m = min(kBuf - kTop, total - base);
          for (int i = tid; i < m; i += kThreads) sh.buf[have + i] = key_of((base + i) / k, (base + i) % k);
          __syncthreads();
          sort_keys(sh, sh.buf, have + m);
          have = kTop;
          if (tid < kTop) sh.buf[tid] = sh.top[tid];
          __syncthreads();
        }
      }
    }
    __syncthreads();
    if (tid == 0) {
      Stat r = sh.stat[0];
      for (int i = 1; i < kWarps; ++i) r = join(r, sh.stat[i]);
      sh.stat[0] = r;
    }
    __syncthreads();
  }
  // a row without a finite logit has no distribution: NaN
  st = sh.stat[0];
  const float ll = log2f(st.l);
  auto lp = [&](float xv) { return st.l > 0.f ? (xv - st.m) - ll * kLn2 : __int_as_float(0x7fffffff); };
  if (tid == 0) {
    if (a.logprob) {
      const int t = int(ld_u1(a.tokens + row));
      a.logprob[row] = t >= 0 && t < a.n ? lp(load1(x + t)) : __int_as_float(0x7fffffff);
    }
    if (a.entropy) a.entropy[row] = st.l > 0.f ? (ll - st.u / st.l) * kLn2 : __int_as_float(0x7fffffff);
  }
  if (tid < k) {
    const uint64_t key = sh.top[tid];
    const uint32_t id = ~uint32_t(key);
    a.top_index[int64_t(row) * k + tid] = int(id);
    a.top_logprob[int64_t(row) * k + tid] = lp(key_value(key));
  }
}

struct Plan {
  int segs, seg_tiles;
  size_t bytes;
};
Plan plan(const DeviceInfo &di, int rows, int n, int k) {
  Plan p{};
  const int tiles = int((int64_t(n) + 7 + kTile - 1) / kTile);  // a row may start up to 7 elements past a boundary
  // the number of segments with the least time by a simple count: waves of resident CTAs (4 per SM)
  // times a segment's tiles and about 3 tiles' time for its start and end
  const int64_t slots = int64_t(di.sm_count) * 4;
  int64_t best = -1;
  for (int segs = 1; segs <= tiles && segs <= 512; ++segs) {
    const int per = (tiles + segs - 1) / segs;
    if (segs > 1 && per == (tiles + segs - 2) / (segs - 1)) continue;  // no shorter than with one segment less
    const int64_t cost = (int64_t(rows) * segs + slots - 1) / slots * (per + 3);
    if (best < 0 || cost < best) {
      best = cost;
      p.seg_tiles = per;
    }
  }
  p.segs = (tiles + p.seg_tiles - 1) / p.seg_tiles;
  p.bytes = workspace_for(size_t(rows), p.segs > 1 ? size_t(rows) * p.segs * part_bytes(k) : 0);
  return p;
}

}  // namespace

static_assert(sizeof(Shared) <= 57344, "four CTAs per SM");

size_t token_logprobs_workspace_bytes(int rows, int n, int k) {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return 0;
  return plan(di, rows, n, k).bytes;
}

int launch_token_logprobs(const void *logits, int64_t stride, int type, const int *tokens, int rows, int n, int k,
                          void *workspace, size_t workspace_bytes, float *logprob, float *entropy, int *top_index,
                          float *top_logprob, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return fail_cuda(e);
  const Plan p = plan(di, rows, n, k);
  if (int64_t(rows) * p.segs > 0x7fffffff) return QDQ_ERR_UNSUPPORTED;
  const LpArgs a{logits, stride, tokens, logprob, entropy, top_logprob, top_index, static_cast<uint32_t *>(workspace),
                 static_cast<uint8_t *>(workspace) + workspace_tickets(workspace_bytes), n, k, p.segs, p.seg_tiles,
                 int64_t(workspace_bytes - workspace_tickets(workspace_bytes)), rows};
  e = cudaError_t(with_type(type, [&](auto t) {
    const auto kernel = logprobs_kernel<decltype(t)>;
    const cudaError_t r = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), int(sizeof(Shared)));
    if (r != cudaSuccess) return int(r);
    return int(launch(kernel, dim3(unsigned(rows * p.segs)), dim3(kThreads), sizeof(Shared), s, a));
  }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

QDQ_CHECK_READER(read_checks_logprobs)

}  // namespace qdq
