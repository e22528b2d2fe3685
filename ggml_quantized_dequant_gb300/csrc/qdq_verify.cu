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
// w is always max(a p - b q, 0) with two numbers a and b: a rejection turns them into a / Z and (b + 1) / Z, Z the sum
// of max(a p - (b + 1) q, 0).  So a rejection is one pass over a row of logits and a row of q, and nothing is stored.
//
// First kernel: every row of logits, in chunks of 1024, one warp each: the largest logit and the sum of exponentials relative
// to it (at temperature 0 the best key).  Second kernel, one CTA or cluster per sequence: the rows' sums from their
// chunks, every child's p and q at once, then the walk; a rejection's pass is shared by the CTAs of the cluster, its
// chunks' sums go through the workspace; the drawn token's chunk is found from the chunks' sums, and the token in it by
// a warp.  Sums over chunks, a, b and Z are f64, within a chunk f32.
// Bound: memory in the first kernel, the chain of loads and joins in the second.
#include "qdq_types.cuh"

namespace qdq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = 32;             // logits per lane
constexpr int kChunk = 32 * kPer;    // ... and warp
constexpr int kCluster = 8;          // CTAs that share a rejection's pass
constexpr float kFar = -1e30f;       // stands for -inf, whose product with 0 would be NaN

struct VerifyArgs {
  const void *logits;
  int64_t stride, draft_stride;
  const int *tokens, *cu, *parent;
  const float *draft, *uniform;
  int *accepted, *path, *next;
  float2 *stats;  // [sequence][row][chunk]: largest logit, sum of 2^((x - largest) c); temperature 0: a 64-bit key
  float *sums;    // [sequence][chunk]: of a rejection's pass
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

// Element of this lane's value i of a chunk: neighbouring lanes' vectors beside one another, or each lane's values.
template <typename T, bool OWN>
__device__ __forceinline__ int element(int i, int lane) {
  constexpr int V = 16 / int(sizeof(T)), G = kPer / V;
  return ((OWN ? lane * G + i / V : i / V * 32 + lane)) * V + i % V;
}

// A chunk's logits, -inf outside the row.
template <typename T, bool OWN>
__device__ __forceinline__ void load_chunk(const Row<T> &r, int base, int lane, float (&x)[kPer]) {
  constexpr int V = 16 / int(sizeof(T)), G = kPer / V;
  if (base >= r.lo && base + kChunk <= r.hi) {
    uint4 u[G];
#pragma unroll
    for (int j = 0; j < G; ++j) u[j] = ld_u4(r.x + base + element<T, OWN>(j * V, lane));
#pragma unroll
    for (int j = 0; j < G; ++j) unpack<T>(u[j], x + j * V);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = base + element<T, OWN>(i, lane);
      x[i] = e >= r.lo && e < r.hi ? load1(r.x + e) : __int_as_float(0xff800000);
    }
  }
}

// The same elements of a row of draft probabilities (0 outside the row).
template <typename T, bool OWN>
__device__ __forceinline__ void load_draft(const float *q, const Row<T> &r, int base, int lane, float (&x)[kPer]) {
  const float *p = q - r.lo;  // element e of the row's count is p[e]
  if (base >= r.lo && base + kChunk <= r.hi && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    uint4 u[kPer / 4];
#pragma unroll
    for (int j = 0; j < kPer / 4; ++j) u[j] = ld_u4(p + base + element<T, OWN>(4 * j, lane));
#pragma unroll
    for (int j = 0; j < kPer / 4; ++j) unpack<float>(u[j], x + 4 * j);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = base + element<T, OWN>(i, lane);
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
__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T, bool GREEDY>
__global__ void __launch_bounds__(kThreads) verify_stats_kernel(const VerifyArgs a) {
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
    load_chunk<T, false>(r, c * kChunk, lane, x);
    float2 *to = a.stats + int64_t(at) * a.chunks + c;
    if constexpr (GREEDY) {
      uint64_t key = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int e = c * kChunk + element<T, false>(k, lane);
        const uint64_t mine = e >= r.lo && e < r.hi ? topk_key(x[k], uint32_t(e - r.lo)) : 0;
        key = mine > key ? mine : key;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t other = shfl_xor_key(key, o);
        key = other > key ? other : key;
      }
      if (lane == 0) *reinterpret_cast<uint64_t *>(to) = key;
    } else {
      float m = x[0];
#pragma unroll
      for (int k = 1; k < kPer; ++k) m = max_nan(m, x[k]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float ref = m == __int_as_float(0xff800000) ? 0.f : m;
      float l[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kPer; ++k) l[k & 3] += weight(a, x[k], ref);
      const float sum = warp_sum((l[0] + l[1]) + (l[2] + l[3]));
      if (lane == 0) *to = make_float2(m, sum);
    }
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
  double z[QDQ_MAX_TREE];            // a row's sum of weights relative to its largest logit
  float m[QDQ_MAX_TREE];             // its largest logit
  int best[QDQ_MAX_TREE];            // temperature 0: its best token
  int bad[QDQ_MAX_TREE];             // a NaN or +inf, or nothing above -inf
  int parent[QDQ_MAX_TREE], token[QDQ_MAX_TREE], path[QDQ_MAX_TREE];
  float p[QDQ_MAX_TREE], q[QDQ_MAX_TREE], u[QDQ_MAX_TREE];  // of a child: its probabilities at its parent, its number
  int lost[QDQ_MAX_TREE];            // rejected drafts without probabilities, at the present node
  float rest[QDQ_MAX_TREE];          // their chunks' sums without them
  double part[kWarps], left;
  int chunk;
};

template <typename T, bool GREEDY, int CTAS>
__global__ void __launch_bounds__(kThreads) verify_walk_kernel(const VerifyArgs a) {
  __shared__ WalkShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = blockIdx.x / CTAS, rank = blockIdx.x % CTAS;
  const float ninf = __int_as_float(0xff800000);
  pdl_launch_dependents();
  pdl_wait();
  const int first = a.cu ? int(ld_u1(a.cu + s)) : s;
  const int n = min(a.cu ? int(ld_u1(a.cu + s + 1)) - first : 1, a.max_rows);
  int *path = a.path + int64_t(s) * a.max_rows;
  if (n <= 0) {  // (the whole cluster leaves)
    if (rank == 0) {
      for (int i = tid; i < a.max_rows; i += kThreads) path[i] = -1;
      if (tid == 0) a.accepted[s] = a.next[s] = -1;
    }
    return;
  }
  const float2 *stats = a.stats + int64_t(s) * a.max_rows * a.chunks;
  // every row's sums; a child's token, parent and number
  for (int i = warp; i < n; i += kWarps) {
    const Row<T> r(a, int64_t(first) + i);
    const int chunks = r.chunks();
    const float2 *st = stats + int64_t(i) * a.chunks;
    if constexpr (GREEDY) {
      uint64_t key = 0;
      for (int c = lane; c < chunks; c += 32) {
        const uint2 k = ld_u2(st + c);
        const uint64_t mine = (uint64_t(k.y) << 32) | k.x;
        key = mine > key ? mine : key;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t other = shfl_xor_key(key, o);
        key = other > key ? other : key;
      }
      if (lane == 0) {
        const uint32_t hi = uint32_t(key >> 32);  // +inf and NaN from 0xFF800000 on, -inf 0x007FFFFF
        sh.bad[i] = hi >= 0xFF800000u || hi <= 0x007FFFFFu;
        sh.best[i] = int(~uint32_t(key));
      }
    } else {
      float m = ninf;
      for (int c = lane; c < chunks; c += 32) m = max_nan(m, __uint_as_float(ld_u1(&st[c].x)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      const bool bad = !(m > ninf && m < -ninf);
      double z = 0.0;
      if (!bad)
        for (int c = lane; c < chunks; c += 32) {
          const uint2 v = ld_u2(st + c);
          z += double(__uint_as_float(v.y) * weight(a, __uint_as_float(v.x), m));
        }
      z = warp_sum_f64(z);
      if (lane == 0) {
        sh.bad[i] = bad;
        sh.m[i] = m;
        sh.z[i] = z;
      }
    }
  }
  if (tid < n) {
    const int up = tid == 0 ? -1 : a.parent ? int(ld_u1(a.parent + first + tid)) : tid - 1;
    sh.parent[tid] = up >= 0 && up < tid ? up : -1;  // without a parent: never reached
    sh.token[tid] = tid == 0 ? -1 : int(ld_u1(a.tokens + first + tid));
    // (numbers outside [0, 1) count as the nearest inside)
    if constexpr (!GREEDY) sh.u[tid] = fminf(fmaxf(__uint_as_float(ld_u1(a.uniform + first + tid)), 0.f), 0.99999994f);
  }
  __syncthreads();
  if constexpr (!GREEDY) {
    if (tid < n && sh.parent[tid] >= 0) {
      const int up = sh.parent[tid], x = sh.token[tid];
      float p = 0.f, q = 1.f;
      if (x >= 0 && x < a.n && !sh.bad[up]) {
        const int64_t row = int64_t(first) + up;
        p = float(double(weight(a, load1(static_cast<const T *>(a.logits) + row * a.stride + x), sh.m[up])) / sh.z[up]);
        if (a.draft) q = load1(a.draft + row * a.draft_stride + x);
      }
      sh.p[tid] = p;
      sh.q[tid] = q;
    }
    __syncthreads();
  }

  int cur = 0, count = 0, lost = 0;
  double wa = 1.0, wb = 0.0, gone = 0.0;  // w = max(wa p - wb q, 0); what rejected drafts without probabilities had
  double sa = 1.0, sb = 0.0;              // a.sums holds the chunks' sums of max(sa p - sb q, 0), a multiple of w
  bool summed = false;                    // ... where this is set
  // the chunks' sums of max(ka p - kb q, 0) at the present node, and their sum
  auto pass = [&](double ka, double kb) {
    const Row<T> r(a, int64_t(first) + cur);
    const float *q = a.draft + (int64_t(first) + cur) * a.draft_stride;
    const float fa = float(ka / sh.z[cur]), fb = float(kb), m = sh.m[cur];
    const int chunks = r.chunks();
    float *sums = a.sums + int64_t(s) * a.chunks;
    for (int c = rank * kWarps + warp; c < chunks; c += CTAS * kWarps) {
      float x[kPer], y[kPer];
      load_chunk<T, false>(r, c * kChunk, lane, x);
      load_draft<T, false>(q, r, c * kChunk, lane, y);
      float l[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kPer; ++k) l[k & 3] += fmaxf(fmaf(fa, weight(a, x[k], m), -fb * y[k]), 0.f);
      const float sum = warp_sum((l[0] + l[1]) + (l[2] + l[3]));
      if (lane == 0) sums[c] = sum;
    }
    __syncwarp();
    all_ctas<CTAS>();
    double z = 0.0;
    for (int c = tid; c < chunks; c += kThreads) z += double(__ldcg(sums + c));
    z = warp_sum_f64(z);
    if (lane == 0) sh.part[warp] = z;
    __syncthreads();
    z = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) z += sh.part[w];
    all_ctas<CTAS>();  // everyone has read the sums (and the parts) before the next pass writes them
    return z;
  };

  for (;;) {  // at the present node (every thread of every CTA alike)
    // its children, in order, as bits
    const uint64_t low = __ballot_sync(0xffffffffu, lane < n && sh.parent[lane] == cur);
    const uint64_t high = __ballot_sync(0xffffffffu, lane + 32 < n && sh.parent[lane + 32] == cur);
    uint64_t children = sh.bad[cur] ? 0 : low | (high << 32);
    int went = -1;
    while (children) {
      const int i = __ffsll((long long)children) - 1;
      children &= children - 1;
      const int x = sh.token[i];
      if constexpr (GREEDY) {
        if (x == sh.best[cur]) went = i;
      } else if (a.draft) {
        const double w = fmax(wa * double(sh.p[i]) - wb * double(sh.q[i]), 0.0);
        if (double(sh.u[i]) * double(sh.q[i]) < w) {
          went = i;
        } else if (x >= 0 && x < a.n) {
          const double z = pass(wa, wb + 1.0);
          summed = z > 0.0;
          if (summed) {
            sa = wa;
            sb = wb + 1.0;
            wa = sa / z;
            wb = sb / z;
          }
        }
      } else {
        bool again = x < 0 || x >= a.n;  // no token, or one that is lost already
        for (int k = 0; k < lost; ++k) again |= sh.lost[k] == x;
        if (!again) {
          if (double(sh.u[i]) * fmax(1.0 - gone, 0.0) < double(sh.p[i])) {
            went = i;
          } else {
            gone += double(sh.p[i]);
            __syncthreads();
            if (tid == 0) sh.lost[lost] = x;
            ++lost;
            __syncthreads();
          }
        }
      }
      if (went >= 0) break;
    }
    if (went < 0) break;
    cur = went;
    if (tid == 0) sh.path[count] = went;
    ++count;
    wa = 1.0;
    wb = gone = 0.0;
    lost = 0;
    summed = false;
  }
  // w as the last pass summed it, where a later one found nothing left
  if constexpr (!GREEDY) {
    if (a.draft && wb > 0.0 && !summed) {
      sa = wa;
      sb = wb;
      pass(sa, sb);
    }
  }
  if (rank != 0) return;
  __syncthreads();
  if (tid == 0) a.accepted[s] = count;
  for (int i = tid; i < a.max_rows; i += kThreads) path[i] = i == 0 ? 0 : i <= count ? sh.path[i - 1] : -1;
  if constexpr (GREEDY) {
    if (tid == 0) a.next[s] = sh.bad[cur] ? -1 : sh.best[cur];
    return;
  }
  if (sh.bad[cur]) {
    if (tid == 0) a.next[s] = -1;
    return;
  }

  // the next token, drawn from w
  const Row<T> r(a, int64_t(first) + cur);
  const int chunks = r.chunks();
  const float2 *st = stats + int64_t(cur) * a.chunks;
  const float *sums = a.sums + int64_t(s) * a.chunks;
  const bool left = a.draft && wb > 0.0;  // w from the pass's sums, else the target's without the lost tokens
  const float m = sh.m[cur];
  for (int k = warp; k < lost; k += kWarps) {  // sums of the chunks that hold lost tokens
    const int c = (sh.lost[k] + r.lo) / kChunk;
    float x[kPer];
    load_chunk<T, false>(r, c * kChunk, lane, x);
    const float ref = __uint_as_float(ld_u1(&st[c].x));
    float l = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = c * kChunk + element<T, false>(j, lane) - r.lo;
      bool out = !(ref > ninf);
      for (int o = 0; o < lost; ++o) out |= sh.lost[o] == e;
      l += out ? 0.f : weight(a, x[j], ref);
    }
    l = warp_sum(l);
    if (lane == 0) sh.rest[k] = l;
  }
  __syncthreads();
  bool with_lost = false;  // nothing else is left: the lost tokens count again
  auto chunk_sum = [&](int c) {
    if (left) return double(__ldcg(sums + c));
    const uint2 v = ld_u2(st + c);
    float l = __uint_as_float(v.y);
    if (!with_lost)
      for (int k = 0; k < lost; ++k)
        if ((sh.lost[k] + r.lo) / kChunk == c) l = sh.rest[k];
    return double(l * weight(a, __uint_as_float(v.x), m));
  };
  // each thread's chunks one after the other; where the sums pass the drawn number
  const int per = (chunks + kThreads - 1) / kThreads, c0 = min(chunks, tid * per), c1 = min(chunks, c0 + per);
  double mine = 0.0, before = 0.0, all = 0.0;
  for (int turn = 0; turn < 2; ++turn) {
    mine = 0.0;
    for (int c = c0; c < c1; ++c) mine += chunk_sum(c);
    double up = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    __syncthreads();
    if (lane == 31) sh.part[warp] = up;
    if (tid == 0) sh.chunk = -1;
    __syncthreads();
    before = up - mine;
    all = 0.0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.part[w];
      all += sh.part[w];
    }
    if (all > 0.0 || lost == 0) break;
    with_lost = true;
  }
  const double drawn = double(sh.u[0]) * all;
  {
    // the last chunk with a sum above 0 whose tokens begin at or below the drawn number
    double at = before;
    int found = -1;
    double rest = 0.0;
    for (int c = c0; c < c1; ++c) {
      const double v = chunk_sum(c);
      if (v > 0.0 && at <= drawn) {
        found = c;
        rest = drawn - at;
      }
      at += v;
    }
    if (found >= 0) atomicMax(&sh.chunk, found);
    __syncthreads();
    if (found >= 0 && sh.chunk == found) sh.left = rest;
    __syncthreads();
  }
  if (warp != 0) return;
  const int c = sh.chunk;
  if (c < 0) {  // no sum above 0: draft probabilities that are no numbers
    if (lane == 0) a.next[s] = -1;
    return;
  }
  float x[kPer], y[kPer];
  load_chunk<T, true>(r, c * kChunk, lane, x);
  double to = sh.left;
  const float ref = left ? m : __uint_as_float(ld_u1(&st[c].x));
  if (left) {
    load_draft<T, true>(a.draft + (int64_t(first) + cur) * a.draft_stride, r, c * kChunk, lane, y);
  } else {
    to /= double(weight(a, ref, m));  // in the chunk's own units
  }
  const float fa = float(sa / sh.z[cur]), fb = float(sb);
  double own = 0.0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int e = c * kChunk + element<T, true>(k, lane) - r.lo;
    float w;
    if (left) {
      w = fmaxf(fmaf(fa, weight(a, x[k], m), -fb * y[k]), 0.f);
    } else {
      bool out = !(x[k] > ninf);
      if (!with_lost)
        for (int o = 0; o < lost; ++o) out |= sh.lost[o] == e;
      w = out ? 0.f : weight(a, x[k], ref);
    }
    x[k] = w;
    own += double(w);
  }
  double up = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double v = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += v;
  }
  // the last token with a weight whose range begins at or below the drawn number
  double at = up - own;
  int token = -1;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (x[k] > 0.f && at <= to) token = c * kChunk + element<T, true>(k, lane) - r.lo;
    at += double(x[k]);
  }
  token = __reduce_max_sync(0xffffffffu, token);
  if (lane == 0) a.next[s] = token;
}

// Chunks of a row, whatever its alignment.
int64_t row_chunks(int n) { return (int64_t(n) + 7 + kChunk - 1) / kChunk; }

template <int CTAS, typename Kernel>
cudaError_t launch_walk(Kernel kernel, const VerifyArgs &a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.n_seqs) * CTAS);
  cfg.blockDim = dim3(kThreads);
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
  return workspace_for(0, size_t(n_seqs) * chunks * (size_t(max_rows) * 8 + 4));
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
  a.c_lo = float(c - double(a.c_hi));
  const int64_t rows = int64_t(n_seqs) * max_rows;
  a.stats = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) + workspace_tickets(workspace_bytes));
  a.sums = reinterpret_cast<float *>(a.stats + rows * a.chunks);
  const int most = (a.chunks + kWarps - 1) / kWarps;  // CTAs of a row with a chunk for each warp
  a.groups = rows * most <= 8 * di.sm_count ? most : (most + 3) / 4;
  if (rows * a.groups > 0x7fffffff || int64_t(n_seqs) * kCluster > 0x7fffffff) return QDQ_ERR_UNSUPPORTED;
  e = cudaError_t(with_type(type, [&](auto t) {
    using T = decltype(t);
    const dim3 grid(unsigned(rows * a.groups));
    const cudaError_t r = greedy ? launch(verify_stats_kernel<T, true>, grid, dim3(kThreads), 0, s, a)
                                 : launch(verify_stats_kernel<T, false>, grid, dim3(kThreads), 0, s, a);
    if (r != cudaSuccess) return int(r);
    if (greedy) return int(launch_walk<1>(verify_walk_kernel<T, true, 1>, a, s));
    if (a.draft && a.chunks > 2 * kWarps) return int(launch_walk<kCluster>(verify_walk_kernel<T, false, kCluster>, a, s));
    return int(launch_walk<1>(verify_walk_kernel<T, false, 1>, a, s));
  }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

QDQ_CHECK_READER(read_checks_verify)

}  // namespace qdq
