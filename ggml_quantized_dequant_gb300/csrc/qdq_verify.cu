// Drafted tokens against the target's probabilities, with given random numbers.
//
// A sequence's rows are a tree: row 0 its last token, the others drafted tokens, each with its parent.  From the root on,
// with w the target's probabilities p at the present node (a softmax of its logits over the temperature) and q the
// probabilities that its children were drawn from, the children in order:
//   child x with number u is accepted when u q(x) < w(x), and is the present node then;
//   else w <- max(w - q, 0), scaled to a sum of 1 (as it was where nothing is left).
// When no child is left the next token is drawn from w: the first i with w_0 + ... + w_i > u_0 (w_0 + ... + w_n-1).
// So the tokens have the target's distribution whatever the drafts are.  Drafts without probabilities count as
// drawn with certainty (q = 1 at the child): w loses the child.  Temperature 0: a child is accepted when it is the
// target's best token (the smallest of equals), which is also the next one.
//
// w is always max(p - b q, 0) / S with two numbers b and S, first 0 and 1: a rejection adds S to b, and S is then the sum of
// max(p - b q, 0).  So a rejection is one pass over a row of logits and a row of q, nothing is stored or divided, and
// the comparison is u q S < max(p - b q, 0).
//
// A row's softmax comes from its chunks of 1024, one warp each: the largest logit and the sum of exponentials relative to it
// (at temperature 0 the best key).  Either a kernel of its own reads every row, and the walk, one CTA or cluster
// per sequence, joins their chunks (few rows: all of them at once are sooner there than one after the other); or the
// walk's cluster reads each node's row when it gets there (many rows: those of drafts that are not reached are not
// read), its warps' sums exchanged through one another's shared memory.  Then every child's p and q at once, and the
// comparisons; a rejection's pass is shared by the cluster, too.  The drawn token's chunk is found from the
// chunks' sums, and the token in it by a warp.
// Sums within a chunk are f32, without its likeliest token, which is taken as a pair of f32 like the sums over chunks (48 bits; f64
// adds have a 64th of f32's rate here and were most of the walk's time).  A child's p, b, S and what lost tokens leave are pairs,
// too: they are compared with near numbers where a draft has nearly all of the probability, or nearly the target's.
// A kernel's code runs once here, so that its length is time too (fetched from the L2): the draw is two tokens to a thread, not
// 32 to a lane of one warp, which took 4 us more.
// Measured (in a graph, with the results read back): one chain of 6, 128256 tokens, f32, with probabilities 11.8 us; 48 chains of 2
// to 8, bf16 36.5 us; 16 trees of 9 to 40, f32, without probabilities 25.4 us; one row 7.4 us.  (All in f32: 9.9, 28, 19 and 6.3, but of
// 9600 drawn tokens 8 were a neighbour of the exact one, now 1.)  Draft probabilities brought into the L2 before they are needed
// cost more than they save: one chain 12.8 us, 8 chains 18.4 (17.2 without), 48 chains 39.5.
// Bound: memory for many rows, the chain of loads and joins for few.
#include <cmath>

#include "qdq_types.cuh"

namespace qdq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;  // of the first kernel
constexpr int kWalk = 512, kWalkWarps = kWalk / 32;    // of the walk
constexpr int kPer = 32;             // logits per lane
constexpr int kChunk = 32 * kPer;    // ... and warp
constexpr int kCluster = 8;          // CTAs of a sequence at most
// Of logits, from which on the walk reads the rows it reaches (its steps take 3 to 4 us each).  Measured, of 128256 tokens:
// 16 trees of 9 to 40, f32 (328 MB at most) 25 us, by all rows 53; 100 of 9 to 40, bf16 (1026 MB) 61, 162; 48 chains of 2 to 8, bf16
// (98 MB) 60, 36.5; near the bound 48 trees of 6 with probabilities, f32 (148 MB) 54, 50; 200 of 4 of 50000, bf16 (80 MB) 50, 44.
constexpr int64_t kLazyBytes = int64_t(128) << 20;
constexpr float kBig = 1.f / 512.f;  // a probability from which on a token's weight is taken as a pair where the next token is drawn
constexpr float kFar = -1e30f;       // stands for -inf, whose product with 0 would be NaN

struct VerifyArgs {
  const void *logits;
  int64_t stride, draft_stride;
  const int *tokens, *cu, *parent;
  const float *draft, *uniform;
  int *accepted, *path, *next;
  float2 *stats;  // [sequence][row][chunk]: largest logit, the others' sum of 2^((x - largest) c); temperature 0: a 64-bit key
  float2 *sums;   // [sequence][chunk]: of a rejection's pass, as pairs
  int n_seqs, max_rows, n, chunks, groups;  // chunks: of a row, at most
  float c_hi, c_lo;                         // log2(e) / temperature in two parts
};

// 16 bytes of elements as f32.
template <typename T>
__device__ __forceinline__ void unpack(const uint4 &u, float *x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      const float2 f = unpack2(w[i], T{});
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// A row from the 16-byte boundary at or below its start: its elements are lo .. hi - 1.
template <typename T>
struct Row {
  const T *x;
  int lo, hi;
  __device__ __forceinline__ Row(const VerifyArgs &a, int64_t row) {
    const T *p = static_cast<const T *>(a.logits) + row * a.stride;
    lo = int((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    x = p - lo;
    hi = lo + a.n;
  }
  __device__ __forceinline__ int chunks() const { return (hi + kChunk - 1) / kChunk; }
};

// This lane's value i of a run of 32 N elements (neighbouring lanes' vectors beside one another): its place in the run.
template <typename T>
__device__ __forceinline__ int element(int i, int lane) {
  constexpr int V = 16 / int(sizeof(T));
  return (i / V * 32 + lane) * V + i % V;
}

// A run's logits, -inf outside the row.
template <typename T, int N>
__device__ __forceinline__ void load_run(const Row<T> &r, int base, int lane, float (&x)[N]) {
  constexpr int V = 16 / int(sizeof(T));
  if (base >= r.lo && base + 32 * N <= r.hi) {
    uint4 u[N / V];
#pragma unroll
    for (int j = 0; j < N / V; ++j) u[j] = ld_u4(r.x + base + element<T>(j * V, lane));
#pragma unroll
    for (int j = 0; j < N / V; ++j) unpack<T>(u[j], x + j * V);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = base + element<T>(i, lane);
      x[i] = e >= r.lo && e < r.hi ? load1(r.x + e) : __int_as_float(0xff800000);
    }
  }
}

// The same elements of a row of draft probabilities (0 outside the row).
template <typename T, int N>
__device__ __forceinline__ void load_draft(const float *q, const Row<T> &r, int base, int lane, float (&x)[N]) {
  const float *p = q - r.lo;  // element e of the row's count is p[e]
  if (base >= r.lo && base + 32 * N <= r.hi && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    uint4 u[N / 4];
#pragma unroll
    for (int j = 0; j < N / 4; ++j) u[j] = ld_u4(p + base + element<T>(4 * j, lane));
#pragma unroll
    for (int j = 0; j < N / 4; ++j) unpack<float>(u[j], x + 4 * j);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = base + element<T>(i, lane);
      x[i] = e >= r.lo && e < r.hi ? load1(p + e) : 0.f;
    }
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 2^((x - m) c): the factor in two parts, or its rounding would act as another temperature
__device__ __forceinline__ float weight(const VerifyArgs &a, float x, float m) {
  const float y = fmaxf(x - m, kFar);
  return ex2(fmaf(y, a.c_hi, y * a.c_lo));
}

// A sum as hi + lo, with the roundings of hi in lo.
struct Pair {
  float hi, lo;
  __device__ __forceinline__ float value() const { return hi + lo; }
};
__device__ __forceinline__ Pair operator+(const Pair &a, const Pair &b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  return {s, a.lo + b.lo + ((a.hi - (s - t)) + (b.hi - t))};
}
__device__ __forceinline__ Pair operator*(float f, const Pair &a) {
  const float h = f * a.hi;
  return {h, fmaf(f, a.lo, fmaf(f, a.hi, -h))};
}
__device__ __forceinline__ float operator-(const Pair &a, const Pair &b) { return (a.hi - b.hi) + (a.lo - b.lo); }
__device__ __forceinline__ Pair warp_sum_pair(Pair v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = v + Pair{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)};
  return v;
}
// The sum of this lane's and lower lanes' (the warp's all in lane 31).
__device__ __forceinline__ Pair warp_scan(Pair v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair u = {__shfl_up_sync(0xffffffffu, v.hi, o), __shfl_up_sync(0xffffffffu, v.lo, o)};
    if (lane >= o) v = u + v;
  }
  return v;
}
__device__ __forceinline__ float warp_max_nan(float m) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
__device__ __forceinline__ uint64_t warp_max_key(uint64_t key) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t other = shfl_xor_key(key, o);
    key = other > key ? other : key;
  }
  return key;
}
__device__ __forceinline__ Pair operator*(const Pair &a, const Pair &b) {
  const float h = a.hi * b.hi;
  return {h, fmaf(a.hi, b.hi, -h) + fmaf(a.hi, b.lo, a.lo * b.hi)};
}
// weight() to 2^-30: the difference and its product with the factor as pairs, 2^i times the series of e^g, |g| <= ln(2) / 2.
__device__ __forceinline__ Pair weight_pair(const VerifyArgs &a, float x, float m) {
  const float y = x - m, back = y - x, rest = (x - (y - back)) - (m + back);
  const float h = y * a.c_hi;
  if (!(h > -100.f)) return {0.f, 0.f};
  const float i = rintf(h), f = h - i, l = fmaf(y, a.c_hi, -h) + fmaf(y, a.c_lo, rest * a.c_hi);
  const float g = f * 0.693147182464599609375f;  // ln 2 and what is left of it
  const Pair e = {g, fmaf(f, 0.693147182464599609375f, -g) + fmaf(f, -1.904654323148236e-9f, l * 0.693147182464599609375f)};
  float r = 1.f / 362880.f;
  r = fmaf(r, g, 1.f / 40320.f);
  r = fmaf(r, g, 1.f / 5040.f);
  r = fmaf(r, g, 1.f / 720.f);
  r = fmaf(r, g, 1.f / 120.f);
  r = fmaf(r, g, 1.f / 24.f);
  r = fmaf(r, g, 1.f / 6.f);
  const Pair v = Pair{1.f, 0.f} + e + 0.5f * (e * e) + Pair{r * g * g * g, 0.f};
  return __int_as_float((127 + int(i)) << 23) * v;
}
// As weight_pair, which is 0 below 2^-100; to 2^-16 there.
__device__ __forceinline__ Pair weight_any(const VerifyArgs &a, float x, float m) {
  const Pair v = weight_pair(a, x, m);
  return v.hi > 0.f ? v : Pair{weight(a, x, m), 0.f};
}
__device__ __forceinline__ Pair reciprocal(const Pair &z) {
  const float i = 1.f / z.value();
  return {i, i * (fmaf(-i, z.hi, 1.f) - i * z.lo)};
}
// max(p - b q, 0) of a weight e (1 / inverse: the row's sum), as a pair.
__device__ __forceinline__ Pair share(const Pair &inverse, const Pair &e, const Pair &b, float q) {
  const float t = b.hi * q;
  const Pair w = inverse * e + Pair{-t, -fmaf(b.lo, q, fmaf(b.hi, q, -t))};
  return w.value() > 0.f ? w : Pair{0.f, 0.f};
}
// A chunk of 1024 elements of size B at p, less what the row does not have, into the L2.
__device__ __forceinline__ void prefetch(const void *p, int bytes, int lane) {
  for (int o = lane * 128; o < bytes; o += 32 * 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(p) + o));
}

// What is kept of a chunk: its largest logit and the sum of the others' exponentials relative to it, or its best key.  (The largest is
// 1 by itself: beside it the others would lose what lies below its last place.)
template <typename T, bool GREEDY>
__device__ __forceinline__ uint2 chunk_stats(const VerifyArgs &a, const Row<T> &r, int c, int lane, const float (&x)[kPer]) {
  float m = x[0];
#pragma unroll
  for (int k = 1; k < kPer; ++k) m = max_nan(m, x[k]);
  m = warp_max_nan(m);
  if constexpr (GREEDY) {
    // the first that equals it (a row whose largest is NaN or -inf has no best token, so that any will do there)
    int at = 0x7fffffff;
#pragma unroll
    for (int k = kPer - 1; k >= 0; --k)
      if (x[k] == m) at = c * kChunk + element<T>(k, lane);
    at = __reduce_min_sync(0xffffffffu, at);
    const uint64_t key = topk_key(m, uint32_t(at - r.lo));
    return make_uint2(uint32_t(key), uint32_t(key >> 32));
  } else {
    const float ref = m == __int_as_float(0xff800000) ? 0.f : m;
    const Two off(-ref, -ref), hi(a.c_hi, a.c_hi), lo(a.c_lo, a.c_lo);
    Two l(0.f, 0.f), ones(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kPer; k += 2) {
      float u, v, p, q;
      const Two y = Two(x[k], x[k + 1]) + off;
      y.to(p, q);
      const Two one(p == 0.f ? -1.f : 0.f, q == 0.f ? -1.f : 0.f);
      fma(y, hi, y * lo).to(u, v);
      l = l + (Two(ex2(u), ex2(v)) + one);
      ones = ones + one;
    }
    float u, v, p, q;
    l.to(u, v);
    ones.to(p, q);
    const float more = __reduce_add_sync(0xffffffffu, int(-(p + q))) - 1;  // of equal largest ones
    return make_uint2(__float_as_uint(m), __float_as_uint(warp_sum(u + v) + (m == ref ? more : 0.f)));
  }
}

template <typename T, bool GREEDY>
__global__ void __launch_bounds__(kThreads, 5) verify_stats_kernel(const VerifyArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.x % a.groups, at = blockIdx.x / a.groups, s = at / a.max_rows, i = at % a.max_rows;
  pdl_launch_dependents();
  pdl_wait();
  const int first = a.cu ? int(ld_u1(a.cu + s)) : s, n = a.cu ? int(ld_u1(a.cu + s + 1)) - first : 1;
  if (i >= n) return;
  const Row<T> r(a, int64_t(first) + i);
  const int chunks = r.chunks();
  for (int c = g * kWarps + warp; c < chunks; c += a.groups * kWarps) {
    float x[kPer];
    load_run<T>(r, c * kChunk, lane, x);
    const uint2 v = chunk_stats<T, GREEDY>(a, r, c, lane, x);
    if (lane == 0 && QDQ_GUARD(c < a.chunks, QDQ_CHECK_OUT)) *reinterpret_cast<uint2 *>(a.stats + int64_t(at) * a.chunks + c) = v;
  }
}

template <int CTAS>
__device__ __forceinline__ void all_ctas() {  // barrier, with global writes before it visible behind it
  if constexpr (CTAS == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

struct WalkShared {
  uint4 parts[2][kCluster * kWalkWarps];  // every warp's part of a sum or a maximum, of the cluster; two exchanges in turn
  Pair z[QDQ_MAX_TREE];               // a row's sum of weights relative to its largest logit
  float m[QDQ_MAX_TREE];              // its largest logit
  int best[QDQ_MAX_TREE];             // temperature 0: its best token
  int bad[QDQ_MAX_TREE];              // a NaN or +inf, or nothing above -inf
  int parent[QDQ_MAX_TREE], token[QDQ_MAX_TREE], path[QDQ_MAX_TREE];
  Pair e[QDQ_MAX_TREE];               // of a child: its weight at its parent, relative to the largest logit there
  float q[QDQ_MAX_TREE], u[QDQ_MAX_TREE];  // ... its draft probability, its number
  int lost[QDQ_MAX_TREE];             // rejected drafts without probabilities, at the present node
  Pair rest[QDQ_MAX_TREE];            // their chunks' sums without them
  uint32_t mask[kWalkWarps][kChunk / 32];  // a chunk's lost tokens
  Pair part[kWalkWarps];
  Pair left;
  int chunk, next;
};

// Every warp's part to every CTA of the cluster; what the warps wrote to global memory before is visible behind it.
template <int CTAS>
__device__ __forceinline__ void exchange(WalkShared &sh, int turn, uint4 mine, int rank, int warp, int lane) {
  uint4 *to = &sh.parts[turn][rank * kWalkWarps + warp];
  if constexpr (CTAS == 1) {
    if (lane == 0) *to = mine;
    __syncthreads();
  } else {
    if (lane < CTAS) {
      uint32_t at = uint32_t(__cvta_generic_to_shared(to));
      asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(lane));
      asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(mine.x), "r"(mine.y), "r"(mine.z), "r"(mine.w) : "memory");
    }
    __syncwarp();
    all_ctas<CTAS>();
  }
}

// What decides over a draft: whether it is the row's best token, its probability alone, or that and its draft probability.  A kernel
// for each: one for the last two spilled registers (one chain 13.3 us, 16 trees 29, apart 11.9 and 25.5).
enum Kind { kBest, kCertain, kDrawn };

template <typename T, Kind KIND, int CTAS, bool LAZY>
__global__ void __launch_bounds__(kWalk, CTAS > 1 ? 2 : 1) verify_walk_kernel(const VerifyArgs a) {
  constexpr bool GREEDY = KIND == kBest, DRAFT = KIND == kDrawn;
  __shared__ WalkShared sh;
  constexpr int kParts = CTAS * kWalkWarps;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = blockIdx.x / CTAS, rank = blockIdx.x % CTAS;
  const float ninf = __int_as_float(0xff800000);
  pdl_launch_dependents();
  if constexpr (CTAS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  const int first = a.cu ? int(ld_u1(a.cu + s)) : s;
  const int n = min(a.cu ? int(ld_u1(a.cu + s + 1)) - first : 1, a.max_rows);
  int *path = a.path + int64_t(s) * a.max_rows;
  if constexpr (CTAS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA runs
  if (n <= 0) {  // (the whole cluster leaves)
    if (rank == 0) {
      for (int i = tid; i < a.max_rows; i += kWalk) path[i] = -1;
      if (tid == 0) a.accepted[s] = a.next[s] = -1;
    }
    return;
  }
  float2 *stats = a.stats + int64_t(s) * a.max_rows * a.chunks;
  int turn = 0;
  // a warp's share of a row's chunks, into the L2
  auto row_ahead = [&](int node) {
    const Row<T> r(a, int64_t(first) + node);
    for (int c = rank * kWalkWarps + warp; c < r.chunks(); c += kParts) prefetch(r.x + c * kChunk, min(kChunk, r.hi - c * kChunk) * int(sizeof(T)), lane);
  };
  if constexpr (LAZY) row_ahead(0);
  float cx = ninf, cq = 1.f;  // of a thread's row, as a child: its logit at its parent, its draft probability
  if (tid < n) {
    const int up = tid == 0 ? -1 : a.parent ? int(ld_u1(a.parent + first + tid)) : tid - 1;
    sh.parent[tid] = up >= 0 && up < tid ? up : -1;  // without a parent: never reached
    const int x = tid == 0 ? -1 : int(ld_u1(a.tokens + first + tid));
    sh.token[tid] = x;
    // (numbers outside [0, 1) count as the nearest inside)
    if constexpr (!GREEDY) {
      sh.u[tid] = fminf(fmaxf(__uint_as_float(ld_u1(a.uniform + first + tid)), 0.f), 0.99999994f);
      if (up >= 0 && up < tid && x >= 0 && x < a.n) {
        const int64_t row = int64_t(first) + up;
        cx = load1(static_cast<const T *>(a.logits) + row * a.stride + x);
        if constexpr (DRAFT) cq = load1(a.draft + row * a.draft_stride + x);
      }
    }
  }
  auto row_key = [&](int i, uint64_t key) {
    const uint32_t hi = uint32_t(key >> 32);  // +inf and NaN from 0xFF800000 on, -inf 0x007FFFFF
    sh.bad[i] = hi >= 0xFF800000u || hi <= 0x007FFFFFu;
    sh.best[i] = int(~uint32_t(key));
  };
  // a row's largest logit, and its sum from lanes' sums relative to it
  auto row_sum = [&](int i, float most, Pair z) {
    z = warp_sum_pair(z);
    if (lane == 0) {
      sh.bad[i] = !(most > ninf && most < -ninf);
      sh.m[i] = most;
      sh.z[i] = z;
    }
  };
  // a chunk's sum relative to a row's largest logit
  auto chunk_part = [&](const uint2 &v, float most) {
    return weight_pair(a, __uint_as_float(v.x), most) * (Pair{1.f, 0.f} + Pair{__uint_as_float(v.y), 0.f});
  };
  auto chunk_of = [&](int node, int c) { return ld_u2(stats + int64_t(node) * a.chunks + c); };
  if constexpr (!LAZY) {
    // every row's sums
    for (int i = warp; i < n; i += kWalkWarps) {
      const Row<T> r(a, int64_t(first) + i);
      const int chunks = r.chunks();
      if constexpr (GREEDY) {
        uint64_t key = 0;
        for (int c = lane; c < chunks; c += 32) {
          const uint2 k = chunk_of(i, c);
          const uint64_t mine = (uint64_t(k.y) << 32) | k.x;
          key = mine > key ? mine : key;
        }
        key = warp_max_key(key);
        if (lane == 0) row_key(i, key);
      } else {
        uint2 v[4];  // (all at up to 128 chunks)
        float m = ninf;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = lane + 32 * k < chunks ? chunk_of(i, lane + 32 * k) : make_uint2(0xff800000u, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) m = max_nan(m, __uint_as_float(v[k].x));
        for (int c = lane + 128; c < chunks; c += 32) m = max_nan(m, __uint_as_float(chunk_of(i, c).x));
        m = warp_max_nan(m);
        Pair z = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 4; ++k) z = z + chunk_part(v[k], m);
        for (int c = lane + 128; c < chunks; c += 32) z = z + chunk_part(chunk_of(i, c), m);
        row_sum(i, m, z);
      }
    }
  }
  __syncthreads();
  if constexpr (!LAZY && !GREEDY) {
    if (tid < n && sh.parent[tid] >= 0) {
      const int up = sh.parent[tid];
      sh.e[tid] = weight_any(a, cx, sh.m[up]);
      sh.q[tid] = cq;
    }
    __syncthreads();
  }

  int cur = 0, count = 0, lost = 0;
  Pair wb = {0.f, 0.f}, ws = {1.f, 0.f};  // w = max(p - wb q, 0) / ws
  Pair kept = {0.f, 0.f};     // what rejected drafts without probabilities have left, relative to the largest logit
  float known = 0.f;          // ... when it was summed last
  bool summed = false;        // a.sums holds the chunks' sums of max(p - wb q, 0)
  // the chunks' sums of max(p - b q, 0) at the present node, and their sum
  auto pass = [&](const Pair &b) {
    const Row<T> r(a, int64_t(first) + cur);
    const float *q = a.draft + (int64_t(first) + cur) * a.draft_stride;
    const float m = sh.m[cur];
    const Pair inverse = reciprocal(sh.z[cur]);
    const float inv = inverse.hi, big = kBig * sh.z[cur].value();
    const int chunks = r.chunks();
    float2 *sums = a.sums + int64_t(s) * a.chunks;
    Pair z = {0.f, 0.f};
    for (int c = rank * kWalkWarps + warp; c < chunks; c += kParts) {
      // likely tokens' shares as pairs, the others' in f32: token for token what the draw takes, or a chunk whose sum is above 0
      // could have no token there
      uint32_t likes = 0;
      float l[2] = {0.f, 0.f};
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float x[kPer / 2], y[kPer / 2];
        load_run<T>(r, c * kChunk + h * (kChunk / 2), lane, x);
        load_draft<T>(q, r, c * kChunk + h * (kChunk / 2), lane, y);
#pragma unroll
        for (int k = 0; k < kPer / 2; ++k) {
          const float w = weight(a, x[k], m);
          if (w > big)
            likes |= 1u << (h * (kPer / 2) + k);
          else
            l[k & 1] += fmaxf(fmaf(inv, w, -b.hi * y[k]), 0.f);
        }
      }
      Pair sum = {l[0] + l[1], 0.f};
      for (; likes; likes &= likes - 1) {
        const int j = __ffs(likes) - 1, e = c * kChunk + j / (kPer / 2) * (kChunk / 2) + element<T>(j % (kPer / 2), lane);
        sum = sum + share(inverse, weight_pair(a, load1(r.x + e), m), b, load1(q + e - r.lo));
      }
      __syncwarp();
      sum = warp_sum_pair(sum);
      if (lane == 0 && QDQ_GUARD(c < a.chunks, QDQ_CHECK_OUT)) sums[c] = make_float2(sum.hi, sum.lo);
      z = z + sum;
    }
    exchange<CTAS>(sh, turn, make_uint4(__float_as_uint(z.hi), __float_as_uint(z.lo), 0, 0), rank, warp, lane);
    z = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < (kParts + 31) / 32; ++k) {
      const uint4 v = lane + 32 * k < kParts ? sh.parts[turn][lane + 32 * k] : make_uint4(0, 0, 0, 0);
      z = z + Pair{__uint_as_float(v.x), __uint_as_float(v.y)};
    }
    turn ^= 1;
    return warp_sum_pair(z);
  };
  // the lost tokens of a chunk as bits
  auto mask_of = [&](const Row<T> &r, uint32_t *mask, int c, int from, int step) {
    for (int o = from; o < lost; o += step) {
      const int at = sh.lost[o] + r.lo - c * kChunk;
      if (at >= 0 && at < kChunk) atomicOr(mask + at / 32, 1u << (at % 32));
    }
  };
  // the sums of the chunks that hold lost tokens, without these
  auto rests = [&](const Row<T> &r) {
    const float m = sh.m[cur], big = kBig * sh.z[cur].value();
    for (int k = warp; k < lost; k += kWalkWarps) {
      const int c = (sh.lost[k] + r.lo) / kChunk;
      uint32_t *mask = sh.mask[warp];
      __syncwarp();
      mask[lane] = 0;
      __syncwarp();
      mask_of(r, mask, c, lane, 32);
      __syncwarp();
      uint32_t likes = 0;  // this lane's likely tokens
      float l[2] = {0.f, 0.f};
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        float x[kPer / 2];
        load_run<T>(r, c * kChunk + h * (kChunk / 2), lane, x);
#pragma unroll
        for (int j = 0; j < kPer / 2; ++j) {
          const int at = h * (kChunk / 2) + element<T>(j, lane);
          const float w = x[j] > ninf && !((mask[at / 32] >> (at % 32)) & 1) ? weight(a, x[j], m) : 0.f;
          if (w > big)
            likes |= 1u << (h * (kPer / 2) + j);
          else
            l[j & 1] += w;
        }
      }
      Pair sum = {l[0] + l[1], 0.f};
      for (; likes; likes &= likes - 1) {
        const int j = __ffs(likes) - 1;
        sum = sum + weight_pair(a, load1(r.x + c * kChunk + j / (kPer / 2) * (kChunk / 2) + element<T>(j % (kPer / 2), lane)), m);
      }
      __syncwarp();
      sum = warp_sum_pair(sum);
      if (lane == 0) sh.rest[k] = sum;
    }
    __syncthreads();
  };
  // a chunk's sum without lost tokens, whose chunks have been summed by rests()
  auto chunk_left = [&](const Row<T> &r, int c) {
    for (int k = 0; k < lost; ++k)
      if ((sh.lost[k] + r.lo) / kChunk == c) return sh.rest[k];
    return chunk_part(chunk_of(cur, c), sh.m[cur]);
  };

  for (;;) {  // at the present node (every thread of every CTA alike)
    // its children, in order, as bits
    const uint64_t low = __ballot_sync(0xffffffffu, lane < n && sh.parent[lane] == cur);
    const uint64_t high = __ballot_sync(0xffffffffu, lane + 32 < n && sh.parent[lane + 32] == cur);
    uint64_t children = low | (high << 32);
    if constexpr (LAZY) {
      const Row<T> r(a, int64_t(first) + cur);
      const int chunks = r.chunks();
      float m = ninf;
      Pair l = {0.f, 0.f};
      uint64_t key = 0;
      for (int c = rank * kWalkWarps + warp; c < chunks; c += kParts) {
        float x[kPer];
        load_run<T>(r, c * kChunk, lane, x);
        if (c < kParts && children) row_ahead(__ffsll((long long)children) - 1);  // the likeliest to come next
        const uint2 v = chunk_stats<T, GREEDY>(a, r, c, lane, x);
        if constexpr (GREEDY) {
          const uint64_t mine = (uint64_t(v.y) << 32) | v.x;
          key = mine > key ? mine : key;
        } else {
          if (lane == 0 && QDQ_GUARD(c < a.chunks && cur < a.max_rows, QDQ_CHECK_OUT)) *reinterpret_cast<uint2 *>(stats + int64_t(cur) * a.chunks + c) = v;
          const float mine = __uint_as_float(v.x), most = max_nan(m, mine);
          const Pair part = Pair{1.f, 0.f} + Pair{__uint_as_float(v.y), 0.f};
          if (m == ninf)
            l = part;
          else if (most > ninf)
            l = weight_pair(a, m, most) * l + weight_pair(a, mine, most) * part;
          m = most;
        }
      }
      exchange<CTAS>(sh, turn, GREEDY ? make_uint4(uint32_t(key), uint32_t(key >> 32), 0, 0)
                                        : make_uint4(__float_as_uint(m), __float_as_uint(l.hi), __float_as_uint(l.lo), 0), rank, warp, lane);
      if (warp == 0) {
        if constexpr (GREEDY) {
          key = 0;
#pragma unroll
          for (int k = 0; k < (kParts + 31) / 32; ++k) {
            const uint4 v = sh.parts[turn][lane + 32 * k];
            const uint64_t mine = (uint64_t(v.y) << 32) | v.x;
            key = mine > key ? mine : key;
          }
          key = warp_max_key(key);
          if (lane == 0) row_key(cur, key);
        } else {
          float most = ninf;
#pragma unroll
          for (int k = 0; k < kParts / 32; ++k) most = max_nan(most, __uint_as_float(sh.parts[turn][lane + 32 * k].x));
          most = warp_max_nan(most);
          Pair z = {0.f, 0.f};
#pragma unroll
          for (int k = 0; k < kParts / 32; ++k) {
            const uint4 v = sh.parts[turn][lane + 32 * k];
            z = z + weight_pair(a, __uint_as_float(v.x), most) * Pair{__uint_as_float(v.y), __uint_as_float(v.z)};
          }
          row_sum(cur, most, z);
        }
      }
      turn ^= 1;
      __syncthreads();
    }
    if (sh.bad[cur]) children = 0;
    if constexpr (!GREEDY) {
      if (LAZY && children) {
        if (tid < n && sh.parent[tid] == cur) {
          sh.e[tid] = weight_any(a, cx, sh.m[cur]);
          sh.q[tid] = cq;
        }
        __syncthreads();
      }
    }
    int went = -1;
    if constexpr (!GREEDY) {
      kept = sh.z[cur];
      known = kept.value();
    }
    while (children) {
      const int i = __ffsll((long long)children) - 1;
      children &= children - 1;
      const int x = sh.token[i];
      if constexpr (GREEDY) {
        if (x == sh.best[cur]) went = i;
      } else if (x < 0 || x >= a.n) {
        continue;
      } else if constexpr (DRAFT) {
        // (near numbers where the draft's probabilities are nearly the target's)
        if (sh.u[i] * sh.q[i] * ws - share(reciprocal(sh.z[cur]), sh.e[i], wb, sh.q[i]) < 0.f) {
          went = i;
        } else {
          const Pair b = wb + ws, z = pass(b);
          summed = z.value() > 0.f;
          if (summed) {
            wb = b;
            ws = z;
          }
        }
      } else {
        bool again = false;  // lost already
        for (int k = 0; k < lost; ++k) again |= sh.lost[k] == x;
        if (!again) {
          const Pair e = sh.e[i];
          if (sh.u[i] * kept - e < 0.f) {
            went = i;
          } else {
            kept = kept + Pair{-e.hi, -e.lo};
            __syncthreads();
            if (tid == 0 && QDQ_GUARD(lost < QDQ_MAX_TREE, QDQ_CHECK_SMEM)) sh.lost[lost] = x;
            ++lost;
            __syncthreads();
            // Less than half of what was summed: that sum's error is now twice as large a share, so the tokens that are left are
            // summed by themselves (by every CTA for itself; a likely token that is refused is rare).
            if (!(kept.value() >= 0.5f * known)) {
              const Row<T> r(a, int64_t(first) + cur);
              rests(r);
              Pair z = {0.f, 0.f};
              for (int c = tid; c < r.chunks(); c += kWalk) z = z + chunk_left(r, c);
              z = warp_sum_pair(z);
              if (lane == 0) sh.part[warp] = z;
              __syncthreads();
              kept = {0.f, 0.f};
#pragma unroll 1
              for (int w = 0; w < kWalkWarps; ++w) kept = kept + sh.part[w];
              known = kept.value();
            }
          }
        }
      }
      if (went >= 0) break;
    }
    if (went < 0) break;
    cur = went;
    if (tid == 0 && QDQ_GUARD(count < QDQ_MAX_TREE, QDQ_CHECK_SMEM)) sh.path[count] = went;
    ++count;
    wb = {0.f, 0.f};
    ws = {1.f, 0.f};
    summed = false;
    lost = 0;
  }
  // w as the last pass summed it, where a later one found nothing left
  if constexpr (DRAFT) {
    if (wb.hi > 0.f && !summed) pass(wb);
  }
  if (rank != 0) return;
  __syncthreads();
  if (tid == 0) a.accepted[s] = count;
  for (int i = tid; i < a.max_rows; i += kWalk) path[i] = i == 0 ? 0 : i <= count ? sh.path[i - 1] : -1;
  if constexpr (GREEDY) {
    if (tid == 0) a.next[s] = sh.bad[cur] ? -1 : sh.best[cur];
    return;
  }
  if (sh.bad[cur]) {
    if (tid == 0) a.next[s] = -1;
    return;
  }

  // The next token, drawn from w.  A drawn number is often next to the border of two tokens where most of the vocabulary
  // shares little of the probability (128256 tokens with 1 %: 8e-8 each), so what lies before it is summed with likely tokens
  // by weight_pair, and the others, whose roundings are a share of little, in f32.
  const Row<T> r(a, int64_t(first) + cur);
  const int chunks = r.chunks();
  const float2 *sums = a.sums + int64_t(s) * a.chunks;
  const float *q = DRAFT ? a.draft + (int64_t(first) + cur) * a.draft_stride : nullptr;
  const bool left = DRAFT && wb.hi > 0.f;  // w by the pass's sums, else the target's without the lost tokens
  const float m = sh.m[cur], big = kBig * sh.z[cur].value();
  const Pair inverse = reciprocal(sh.z[cur]);
  const float inv = inverse.hi;
  bool with_lost = false;  // nothing else is left: the lost tokens count again
  if (lost) rests(r);
  auto chunk_sum = [&](int c) {
    if (c >= chunks) return Pair{0.f, 0.f};
    if (left) {
      const float2 v = __ldcg(sums + c);
      return Pair{v.x, v.y};
    }
    return with_lost ? chunk_part(chunk_of(cur, c), m) : chunk_left(r, c);
  };
  // each thread's chunks one after the other; where the sums pass the drawn number
  const int per = (chunks + kWalk - 1) / kWalk, c0 = tid * per;
  Pair before, all, v0;
  for (int again = 0; again < 2; ++again) {
    Pair mine = {0.f, 0.f};
    for (int k = 0; k < per; ++k) {
      const Pair v = chunk_sum(c0 + k);
      if (k == 0) v0 = v;
      mine = mine + v;
    }
    const Pair up = warp_scan(mine, lane);
    if (lane == 31) sh.part[warp] = up;
    if (tid == 0) sh.chunk = sh.next = -1;
    __syncthreads();
    before = up + Pair{-mine.hi, -mine.lo};
    all = {0.f, 0.f};
#pragma unroll 1
    for (int w = 0; w < kWalkWarps; ++w) {
      const Pair v = sh.part[w];
      if (w < warp) before = v + before;
      all = all + v;
    }
    __syncthreads();
    if (all.value() > 0.f || lost == 0) break;
    with_lost = true;
  }
  const Pair drawn = sh.u[0] * all;
  {
    // the last chunk with a sum above 0 whose tokens begin at or below the drawn number
    Pair at = before;
    int found = -1;
    Pair rest = {0.f, 0.f};
    for (int k = 0; k < per; ++k) {
      const Pair v = k == 0 ? v0 : chunk_sum(c0 + k);
      const Pair over = drawn + Pair{-at.hi, -at.lo};
      if (v.value() > 0.f && over.value() >= 0.f) {
        found = c0 + k;
        rest = over;
      }
      at = at + v;
    }
    if (found >= 0) atomicMax(&sh.chunk, found);
    __syncthreads();
    if (found >= 0 && sh.chunk == found) sh.left = rest;
  }
  // the last token of that chunk with a weight whose range begins at or below the drawn number, each thread's beside one another
  const int c = sh.chunk;
  if (c < 0) {  // no sum above 0: draft probabilities that are no numbers
    if (tid == 0) a.next[s] = -1;
    return;
  }
  if (tid < kChunk / 32) sh.mask[0][tid] = 0;
  __syncthreads();
  if (!with_lost) mask_of(r, sh.mask[0], c, tid, kWalk);
  __syncthreads();
  constexpr int kOwn = kChunk / kWalk;
  Pair mine[kOwn], own = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    const int at = tid * kOwn + k, e = c * kChunk + at;
    const bool in = e >= r.lo && e < r.hi && !((sh.mask[0][at / 32] >> (at % 32)) & 1);
    const float x = in ? load1(r.x + e) : ninf, prob = in && left ? load1(q + e - r.lo) : 0.f;
    const float w = x > ninf ? weight(a, x, m) : 0.f;
    if (w > big)
      mine[k] = left ? share(inverse, weight_pair(a, x, m), wb, prob) : weight_pair(a, x, m);
    else
      mine[k] = Pair{left ? fmaxf(fmaf(inv, w, -wb.hi * prob), 0.f) : w, 0.f};
    own = own + mine[k];
  }
  const Pair up = warp_scan(own, lane);
  if (lane == 31) sh.part[warp] = up;
  __syncthreads();
  Pair at = {__shfl_up_sync(0xffffffffu, up.hi, 1), __shfl_up_sync(0xffffffffu, up.lo, 1)};
  if (lane == 0) at = {0.f, 0.f};
  Pair below = {0.f, 0.f};
#pragma unroll 1
  for (int w = 0; w < warp; ++w) below = below + sh.part[w];
  at = below + at;
  const Pair to = sh.left;
  int token = -1;
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    if (mine[k].value() > 0.f && to - at >= 0.f) token = c * kChunk + tid * kOwn + k - r.lo;
    at = at + mine[k];
  }
  token = __reduce_max_sync(0xffffffffu, token);
  if (lane == 0 && token >= 0) atomicMax(&sh.next, token);
  __syncthreads();
  if (tid == 0) a.next[s] = sh.next;
}

// Chunks of a row, whatever its alignment.
int64_t row_chunks(int n) { return (int64_t(n) + 7 + kChunk - 1) / kChunk; }

template <int CTAS, typename Kernel>
cudaError_t launch_walk(Kernel kernel, const VerifyArgs &a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.n_seqs) * CTAS);
  cfg.blockDim = dim3(kWalk);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = opt_pdl() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CTAS > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

size_t verify_drafts_workspace_bytes(int n_seqs, int max_rows, int n) {
  const size_t chunks = size_t(row_chunks(n));
  return workspace_for(0, size_t(n_seqs) * chunks * (size_t(max_rows) * 8 + 8));
}

int launch_verify_drafts(const void *logits, int64_t stride, int type, const int *tokens, const int *cu, const int *parent,
                         int n_seqs, int max_rows, int n, const float *draft_probs, int64_t draft_stride, const float *uniform,
                         float temperature, int *accepted, int *path, int *next_token, void *workspace,
                         size_t workspace_bytes, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return fail_cuda(e);
  const bool greedy = temperature == 0.f;
  VerifyArgs a{};
  a.logits = logits;
  a.stride = stride;
  a.draft = greedy ? nullptr : draft_probs;
  a.draft_stride = draft_stride;
  a.tokens = tokens;
  a.cu = cu;
  a.parent = parent;
  a.uniform = uniform;
  a.accepted = accepted;
  a.path = path;
  a.next = next_token;
  a.n_seqs = n_seqs;
  a.max_rows = max_rows;
  a.n = n;
  a.chunks = int(row_chunks(n));
  const double c = greedy ? 0.0 : 1.4426950408889634074 / double(temperature);
  a.c_hi = float(c);
  if (!greedy && double(a.c_hi) >= c) a.c_hi = std::nextafterf(a.c_hi, 0.f);
  a.c_lo = float(c - double(a.c_hi));  // above 0, so that -inf times both is -inf
  const int64_t rows = int64_t(n_seqs) * max_rows;
  a.stats = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) + workspace_tickets(workspace_bytes));
  a.sums = a.stats + rows * a.chunks;
  const int most = (a.chunks + kWarps - 1) / kWarps;  // CTAs of a row with a chunk for each warp
  // many rows: two chunks for each warp (48 chains 36.5 us, with four 37.2, with one 38.2); few: one (one chain 11.8 us, with two 12.5)
  a.groups = rows * most <= 8 * di.sm_count ? most : (most + 1) / 2;
  if (rows * a.groups > 0x7fffffff || int64_t(n_seqs) * kCluster > 0x7fffffff) return QDQ_ERR_UNSUPPORTED;
  // 8 CTAs to a sequence while all are resident together, else 4: 48 chains of 128256 36.5 us, with 8 39.3; 8 chains 21.5, with 8 18.4
  const bool wide = a.chunks > 2 * kWarps, few = int64_t(n_seqs) * kCluster <= 2 * di.sm_count;
  e = cudaError_t(with_type(type, [&](auto t) {
    using T = decltype(t);
    auto lazy = [&](auto kind) {
      constexpr Kind K = decltype(kind)::value;
      return int(few ? launch_walk<kCluster>(verify_walk_kernel<T, K, kCluster, true>, a, s)
                     : launch_walk<kCluster / 2>(verify_walk_kernel<T, K, kCluster / 2, true>, a, s));
    };
    constexpr std::integral_constant<Kind, kBest> best{};
    constexpr std::integral_constant<Kind, kCertain> certain{};
    constexpr std::integral_constant<Kind, kDrawn> drawn{};
    if (wide && max_rows > 1 && rows * n * int64_t(sizeof(T)) > kLazyBytes) return greedy ? lazy(best) : a.draft ? lazy(drawn) : lazy(certain);
    const dim3 grid(unsigned(rows * a.groups));
    const cudaError_t r = greedy ? launch(verify_stats_kernel<T, true>, grid, dim3(kThreads), 0, s, a)
                                 : launch(verify_stats_kernel<T, false>, grid, dim3(kThreads), 0, s, a);
    if (r != cudaSuccess) return int(r);
    if (greedy) return int(launch_walk<1>(verify_walk_kernel<T, kBest, 1, false>, a, s));
    if (!a.draft) return int(launch_walk<1>(verify_walk_kernel<T, kCertain, 1, false>, a, s));
    if (!wide) return int(launch_walk<1>(verify_walk_kernel<T, kDrawn, 1, false>, a, s));
    return int(few ? launch_walk<kCluster>(verify_walk_kernel<T, kDrawn, kCluster, false>, a, s)
                   : launch_walk<kCluster / 2>(verify_walk_kernel<T, kDrawn, kCluster / 2, false>, a, s));
  }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

QDQ_CHECK_READER(read_checks_verify)

}  // namespace qdq
