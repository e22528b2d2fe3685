// Log probabilities of given tokens, the entropy and the top alternatives of each row of
// logits, in one pass over the logits.
//
//   lse = log sum_i e^x_i,  logprob = x_t - lse,  entropy = lse - sum_i e^(x_i - lse) x_i
//   top: the k first of the order of qdq_topk_rows, with their log probabilities
//
// A row is cut into segments (one CTA each) of tiles of 4096 logits.  A thread keeps its own
// running maximum M, l = sum 2^y and u = sum 2^y y with y = (x - M) log2(e) (the difference
// first: a mask of the type's lowest value must not turn into an infinity), so the
// tiles need no barrier for the sums; the threads' triples are joined at the end.  The top k:
// the k-th largest of 64 maxima of the first tile (each over the same number of logits) is a
// lower bound of the row's k-th best, so only the few logits at or above it become 64-bit keys
// in shared memory; they are sorted 64 at a time by warps and folded into the best 64 so far,
// whose k-th then is the bound.  Segments of one row are joined by the CTA that finishes last.
#include "qdq_types.cuh"

namespace qdq {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;                     // logits per thread and tile
constexpr int kTile = kThreads * kPer;
constexpr int kTop = QDQ_MAX_TOPK;
constexpr int kBuf = kTile + 256;            // candidate keys: a full tile and what waits
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
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

struct Shared {
  uint64_t buf[kBuf];
  uint64_t top[kTop];            // best 64 so far, descending, 0 past the end
  uint64_t list[kWarps / 2][64];
  float group[64];
  Stat stat[kWarps];
  int count;
  uint64_t bound;                // keys at or below it are not among the k best
  float bound_v;                 // its value
  int last;
};

__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = uint32_t(key >> 32);
  return o == 0xFFFFFFFFu ? __int_as_float(0x7fffffff) : __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// Folds the `count` keys of sh.buf into sh.top and raises the bound.  All threads call it.
__device__ void fold_candidates(Shared &sh, int count, int k) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t a = 0, b = 0;
  bool any = false;
  for (int base = 64 * warp; base < count; base += 64 * kWarps) {
    uint64_t c = base + lane < count ? sh.buf[base + lane] : 0ull;
    uint64_t d = base + 32 + lane < count ? sh.buf[base + 32 + lane] : 0ull;
    warp_sort64_desc(c, d, lane);
    if (!any) {
      a = c;
      b = d;
      any = true;
    } else {
      warp_top64_merge(a, b, c, d, lane);
    }
  }
  if (warp == 0) warp_top64_merge(a, b, sh.top[lane], sh.top[lane + 32], lane);
  for (int half = kWarps / 2; half >= 1; half >>= 1) {
    if (count <= 64 * half) continue;  // warps past the keys have nothing
    if (warp >= half && warp < 2 * half) {
      sh.list[warp - half][lane] = a;
      sh.list[warp - half][lane + 32] = b;
    }
    __syncthreads();
    if (warp < half) warp_top64_merge(a, b, sh.list[warp][lane], sh.list[warp][lane + 32], lane);
    __syncthreads();
  }
  __syncthreads();
  if (warp == 0) {
    sh.top[lane] = a;
    sh.top[lane + 32] = b;
    const uint64_t ka = __shfl_sync(0xffffffffu, a, (k - 1) & 31), kb = __shfl_sync(0xffffffffu, b, (k - 1) & 31);
    const uint64_t kk = k <= 32 ? ka : kb;
    if (lane == 0) {
      if (kk > sh.bound) {
        sh.bound = kk;
        sh.bound_v = key_value(kk);
      }
      sh.count = 0;
    }
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LpArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared &sh = *reinterpret_cast<Shared *>(raw);
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
  if (tid < kTop) sh.top[tid] = 0;
  if (tid == 0) {
    sh.count = 0;
    sh.bound = 0;
    sh.bound_v = __int_as_float(0xff800000);
  }
  __syncthreads();
  const float ninf = __int_as_float(0xff800000);
  Stat st{ninf, 0.f, 0.f};
  const int64_t e0 = int64_t(seg) * a.seg_tiles * kTile;
  const int64_t e1 = min(int64_t(hi), e0 + int64_t(a.seg_tiles) * kTile);

  float v[kPer];
  auto load = [&](int64_t base) {
#pragma unroll
    for (int i = 0; i < kPer / V; ++i) {
      const int64_t e = base + (int64_t(i) * kThreads + tid) * V;
      if (e >= lo && e + V <= hi) {
        const uint4 w = ld_u4(x0 + e);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
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
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[V * i + j] = e + j >= lo && e + j < hi ? load1(x0 + e + j) : ninf;
      }
    }
  };
  bool first = true;
  for (int64_t base = e0; base < e1; base += kTile) {
    load(base);
    float tm = v[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) tm = max_nan(tm, v[i]);
    const float m2 = max_nan(st.m, tm);
    if (m2 != st.m) {  // also for NaN
      const float d = st.l == 0.f ? 0.f : shift_of(st.m, m2), e = exp2f(d);
      st.u = e * fmaf(st.l, d, st.u);
      st.l *= e;
      st.m = m2;
    }
    const float ref = st.m == ninf ? 0.f : st.m;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float d = shift_of(v[i], ref);
      const float e = exp2f(d);
      st.l += e;
      st.u = fmaf(e, d, st.u);
    }
    if (k > 0) {
      if (first) {  // a first bound: the k-th largest of 64 groups' maxima
        first = false;
        float gm = max_nan(tm, __shfl_xor_sync(0xffffffffu, tm, 1));
        gm = max_nan(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
        if ((tid & 3) == 0) sh.group[tid >> 2] = gm;
        __syncthreads();
        if (warp == 0) {
          // a group of padding alone gives -inf: no bound
          uint64_t p = topk_key(sh.group[lane], 0xFFFFFFFFu), q = topk_key(sh.group[lane + 32], 0xFFFFFFFFu);
          warp_sort64_desc(p, q, lane);
          const uint64_t pk = __shfl_sync(0xffffffffu, p, (k - 1) & 31), qk = __shfl_sync(0xffffffffu, q, (k - 1) & 31);
          const uint64_t kk = k <= 32 ? pk : qk;
          const float kv = key_value(kk);
          if (lane == 0 && kv > ninf) {  // not for NaN: those are few or the row is lost anyway
            sh.bound = kk;
            sh.bound_v = kv;
          }
        }
        __syncthreads();
      }
      const float bv = sh.bound_v;
      const uint64_t bk = sh.bound;
      if (!(tm < bv)) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int64_t e = base + (int64_t(i / V) * kThreads + tid) * V + i % V;
          if (!(v[i] < bv) && e >= lo && e < hi) {
            const uint64_t key = topk_key(v[i], uint32_t(e - shift));
            if (key > bk) sh.buf[atomicAdd(&sh.count, 1)] = key;
          }
        }
      }
      __syncthreads();
      const int count = sh.count;
      if (count > kBuf - kTile) fold_candidates(sh, count, k);
      else __syncthreads();  // nobody adds before everyone has read the count
    }
  }
  if (k > 0) {
    const int count = sh.count;
    __syncthreads();
    if (count > 0) fold_candidates(sh, count, k);
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
    if (k > 0) {  // all segments' keys, folded in batches that fit the buffer
      if (tid < kTop) sh.top[tid] = 0;
      if (tid == 0) sh.bound = 0;
      const int total = a.segs * k;
      for (int base = 0; base < total; base += kBuf) {
        const int m = min(kBuf, total - base);
        __syncthreads();
        for (int i = tid; i < m; i += kThreads)
          sh.buf[i] = __ldcg(reinterpret_cast<const unsigned long long *>(all + size_t((base + i) / k) * part + 16) + (base + i) % k);
        __syncthreads();
        fold_candidates(sh, m, k);
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
  size_t ticket_bytes, bytes;
};
Plan plan(const DeviceInfo &di, int rows, int n, int k) {
  Plan p{};
  const int tiles = int((int64_t(n) + 7 + kTile - 1) / kTile);  // a row may start up to 7 elements past a boundary
  const int64_t want = int64_t(di.sm_count) * 8;
  int64_t segs = (want + rows - 1) / rows;
  if (segs > tiles) segs = tiles;
  if (segs < 1) segs = 1;
  p.seg_tiles = int((tiles + segs - 1) / segs);
  p.segs = (tiles + p.seg_tiles - 1) / p.seg_tiles;
  p.ticket_bytes = (size_t(rows) * 4 + 255) / 256 * 256;
  p.bytes = p.ticket_bytes + (p.segs > 1 ? size_t(rows) * p.segs * part_bytes(k) : 0);
  return p;
}

}  // namespace

size_t token_logprobs_workspace_bytes(int rows, int n, int k) {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return 0;
  return plan(di, rows, n, k).bytes;
}

int launch_token_logprobs(const void *logits, int64_t stride, int type, const int *tokens, int rows, int n, int k,
                          void *workspace, float *logprob, float *entropy, int *top_index, float *top_logprob,
                          cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return fail_cuda(e);
  const Plan p = plan(di, rows, n, k);
  if (int64_t(rows) * p.segs > 0x7fffffff) return QDQ_ERR_UNSUPPORTED;
  const LpArgs a{logits, stride, tokens, logprob, entropy, top_logprob, top_index, static_cast<uint32_t *>(workspace),
                 static_cast<uint8_t *>(workspace) + p.ticket_bytes, n, k, p.segs, p.seg_tiles};
  e = cudaError_t(with_type(type, [&](auto t) {
    const auto kernel = logprobs_kernel<decltype(t)>;
    const cudaError_t r = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), int(sizeof(Shared)));
    if (r != cudaSuccess) return int(r);
    return int(launch(kernel, dim3(unsigned(rows * p.segs)), dim3(kThreads), sizeof(Shared), s, a));
  }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

}  // namespace qdq
