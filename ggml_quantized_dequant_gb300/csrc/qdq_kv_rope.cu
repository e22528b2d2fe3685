// New tokens' queries and keys normed for each head and turned by their positions, keys and values quantised
// into the paged 8-bit cache, in one pass.
//
//   y = x / sqrt(mean x^2 + eps) * w            per head of D elements, where weights are given
//   (a, b) -> (a cos - b sin, b cos + a sin)    pairs of the first n_rot elements, angle = position * freq
//   cache: the definition in qdq_kv.cu, from the turned keys in f32 (no rounding to the type in between)
//
// The angle as a fraction of a turn is position * F in 64-bit integers that wrap at a whole turn, F = 2^64 frac(freq /
// 2 pi): no digits are lost at far positions (in f32 the angle of position 4,000,000 is off by a tenth of
// a radian), and cos and sin get the fraction between -1/2 and 1/2.
//
// A CTA takes the new tokens of one block of 16 (which share a key scale) and a share of the heads.  Its threads compute
// the tokens' cosines and sines once into shared memory, while the first loads are on their way; then 4 to 8 lanes
// take a token's head, in couples of four elements and the four that they are paired with, so that a rotation needs no other
// lane and the sum of squares two or three shuffles (32 lanes to a head: 9 shuffles each, 136 us for the prompts below).  A
// warp holds a head's 16 keys (a block's maximum comes from its registers), or 16 queries of any heads and tokens.  Every
// input is read once, every output written once.
// Bound: memory for prompts, with the arithmetic close behind; for single tokens the chain of launch, length, page and scale.
#include "qdq_types.cuh"

namespace qdq {
namespace {

constexpr int kWarps = 4;

struct RopeArgs {
  KvPool c;
  const int *kv_len, *cu, *parent;  // cu NULL: one token each; parent NULL: one after the other
  const void *q, *k, *v;
  void *q_out;
  const float *q_weight, *k_weight, *freqs;
  int64_t q_stride, q_out_stride, k_stride, v_stride;
  int n_seqs, n_blocks, max_new, n_heads, n_rot;
  int q_iters;  // of GT queries in a warp's item
  float eps;
};

// LPT lanes to a token's head, GT heads at a time, C couples of four elements and four others per lane; NI times GT
// tokens are a block's.
template <int D>
struct Lanes {
  static constexpr int C = D == 64 ? 1 : D == 128 ? 2 : D == 256 ? 4 : 3;
  static constexpr int LPT = D / 8 / C, GT = 32 / LPT, NI = kKvBlock / GT;
};

// Four elements as loaded.
template <typename T>
struct Raw {
  uint32_t w[sizeof(T)];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (sizeof(T) == 4) {
      const uint4 v = ld_u4(p);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else {
      const uint2 v = ld_u2(p);
      w[0] = v.x;
      w[1] = v.y;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (uint32_t &x : w) x = 0;
  }
  __device__ __forceinline__ void values(float *x) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(w[e]);
    } else {
      const float2 a = unpack2(w[0], T{}), b = unpack2(w[1], T{});
      x[0] = a.x;
      x[1] = a.y;
      x[2] = b.x;
      x[3] = b.y;
    }
  }
};

// First element of a couple's two quads: of pairs that lie n_rot / 2 apart, or beside one another.
template <bool ADJACENT>
struct Couple {
  int a, b;
  __device__ __forceinline__ Couple(const RopeArgs &r, int j) {
    const bool apart = !ADJACENT && j < r.n_rot / 8;
    a = apart ? 4 * j : 8 * j;
    b = apart ? 4 * j + r.n_rot / 2 : 8 * j + 4;
  }
};

// Norm (weight: of the lane's elements) and rotation of a token's head.
template <int D, bool ADJACENT>
__device__ __forceinline__ void norm_turn(const RopeArgs &a, float (&x)[Lanes<D>::C][8], bool norm, const float (&weight)[Lanes<D>::C][8],
                                          const float *cs, const float *sn, int sub) {
  using L = Lanes<D>;
  if (norm) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < L::C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(x[c][e], x[c][e], s);
#pragma unroll
    for (int o = L::LPT / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float inv = rsqrtf(s * (1.f / D) + a.eps);
#pragma unroll
    for (int c = 0; c < L::C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[c][e] *= inv * weight[c][e];
  }
#pragma unroll
  for (int c = 0; c < L::C; ++c) {
    const int j = sub + L::LPT * c;
    if (j < a.n_rot / 8) {
      const float4 co = *reinterpret_cast<const float4 *>(cs + 4 * j), si = *reinterpret_cast<const float4 *>(sn + 4 * j);
      const float cw[4] = {co.x, co.y, co.z, co.w}, sw[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float &u = x[c][ADJACENT ? 2 * e : e], &v = x[c][ADJACENT ? 2 * e + 1 : 4 + e];
        const float p = u, q = v;
        u = p * cw[e] - q * sw[e];
        v = q * cw[e] + p * sw[e];
      }
    }
  }
}

// The larger magnitude; NaN wins.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// The block's codes and scale from its new tokens held .. end - 1 in x, whose largest magnitude is m (definition in qdq_kv.cu).
// A product with 1 / s is at most 127 and some roundings, so that 1.5 2^23 added and its bits' low byte are rint and its code.
template <int D, bool ADJACENT>
__device__ __forceinline__ void quantise(const RopeArgs &a, uint8_t *record, int which, int t0, int held, int end, float s_old, float m,
                                         const float (&x)[Lanes<D>::NI][Lanes<D>::C][8], int lane) {
  using L = Lanes<D>;
  const int sub = lane % L::LPT, page_tokens = a.c.page_tokens;
  int8_t *codes = reinterpret_cast<int8_t *>(record) + (int64_t(which) * page_tokens + t0) * D;
  float s_new = __fdiv_rn(m, 127.f);
  if (s_new < 1.17549435e-38f) s_new = 0.f;
  if (!(m < __int_as_float(0x7f800000))) s_new = __int_as_float(0x7fffffff);
  const float sc = max_abs_bits(s_old, s_new);  // NaN wins
  const float inv = sc > 0.f ? __frcp_rn(sc) : 0.f;
  const bool grown = held && sc != s_old;
  const float again = grown && sc > 0.f ? __fdiv_rn(s_old, sc) : 0.f;
#pragma unroll
  for (int i = 0; i < L::NI; ++i) {
    const int t = i * L::GT + lane / L::LPT;
#pragma unroll
    for (int c = 0; c < L::C; ++c) {
      const Couple<ADJACENT> at(a, sub + L::LPT * c);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t *p = reinterpret_cast<uint32_t *>(codes + t * D + (which ? 8 * (sub + L::LPT * c) + 4 * q : q ? at.b : at.a));
        if (grown && t < held) {  // a larger scale: what the block held, rounded to it
          const uint32_t w = ld_u1(p);
          uint32_t r = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) r |= uint32_t(__float2int_rn(float(int8_t(w >> (8 * j))) * again) & 0xFF) << (8 * j);
          *p = r;
        }
        if (t >= held && t < end) {
          const float *v = &x[i][c][4 * q];
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(__fadd_rn(__fmul_rn(v[e], inv), 12582912.f));
          const uint32_t r = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
          *p = sc == sc ? r : 0u;
        }
      }
    }
  }
  if (lane == 0 && (held == 0 || sc != s_old))
    *(reinterpret_cast<float *>(record + int64_t(2) * page_tokens * D) + which * (page_tokens / kKvBlock) + t0 / kKvBlock) = sc;
}

template <typename T, int D, bool ADJACENT>
__global__ void __launch_bounds__(kWarps * 32, D <= 128 ? 3 : 2) kv_append_rope_kernel(const RopeArgs a) {
  using L = Lanes<D>;
  constexpr int kThreads = kWarps * 32;
  __shared__ unsigned long long s_turn[D / 2];  // 2^64 frac(freq / 2 pi)
  __shared__ __align__(16) float s_cos[kKvBlock][D / 2], s_sin[kKvBlock][D / 2];
  __shared__ int s_parent[QDQ_MAX_TREE], s_pos[kKvBlock];
  __shared__ bool s_bad[kKvBlock];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane % L::LPT, grp = lane / L::LPT;
  const float qnan = __int_as_float(0x7fffffff);
  pdl_launch_dependents();
  const int pairs = a.n_rot / 2;
  for (int i = tid; i < pairs; i += kThreads) {  // (frequencies and weights count as weights: read ahead of the wait)
    const float f = __ldg(a.freqs + i);
    const double turns = double(f) * 0.15915494309189533577;  // 1 / (2 pi)
    s_turn[i] = isfinite(f) ? (unsigned long long)((turns - floor(turns)) * 18446744073709551616.0) : 0ull;
  }
  pdl_wait();
  const int64_t rec = kv_record_bytes(a.c.page_tokens, D);
  for (int s = blockIdx.z; s < a.n_seqs; s += gridDim.z)
    for (int b = blockIdx.y; b < a.n_blocks; b += gridDim.y) {
      const int first = a.cu ? int(ld_u1(a.cu + s)) : s;
      const int n_new = a.cu ? int(ld_u1(a.cu + s + 1)) - first : 1;
      const int all = int(ld_u1(a.kv_len + s));
      if (n_new <= 0) break;
      const bool bad = all < n_new;  // more new tokens than there are: nothing is appended, their queries are NaN
      const int old = bad ? 0 : all - n_new, n = min(n_new, a.max_new), len = old + n;
      const int blk = old / kKvBlock + b, p0 = blk * kKvBlock;
      if (p0 >= len) break;
      const int held = max(old - p0, 0), end = min(len - p0, kKvBlock), fresh = end - held;
      const int64_t row0 = int64_t(first) + p0 - old;  // the row of the block's token 0 (a negative part is never read)
      // items: keys and values of a head, then q_iters times GT queries (head, token) one after the other
      const uint32_t by_fresh = uint32_t(((uint64_t(1) << 32) + fresh - 1) / fresh);  // (2^32 for 1 is 0)
      auto head_of = [&](int u) { return fresh == 1 ? u : int(__umulhi(uint32_t(u), by_fresh)); };  // u / fresh: u is below 2^28
      const int q_all = a.n_heads * fresh, q_item = a.q_iters * L::GT, items = 2 * a.c.n_kv + (q_all + q_item - 1) / q_item;
      Raw<T> raw[L::NI][L::C][2];
      int64_t at = -1;   // of a key or value item: its record
      float s_old = 0.f;
      auto load = [&](int item) {
        const bool kv = item < 2 * a.c.n_kv;
        const int which = item & 1, h = item >> 1;
        const T *x = kv ? static_cast<const T *>(which ? a.v : a.k) + row0 * (which ? a.v_stride : a.k_stride) + h * D
                        : static_cast<const T *>(a.q) + row0 * a.q_stride;
        const int64_t stride = !kv ? a.q_stride : which ? a.v_stride : a.k_stride;
#pragma unroll
        for (int i = 0; i < L::NI; ++i) {
          const int u = (item - 2 * a.c.n_kv) * q_item + i * L::GT + grp, hq = kv ? 0 : head_of(u);  // the query, its head
          const int t = kv ? i * L::GT + grp : held + u - hq * fresh;
          const bool in = kv ? t >= held && t < end && !bad : i < a.q_iters && u < q_all;
          const T *p = x + t * stride + hq * D;
#pragma unroll
          for (int c = 0; c < L::C; ++c) {
            const int j = sub + L::LPT * c;
            const Couple<ADJACENT> cp(a, j);
            raw[i][c][0].clear();
            raw[i][c][1].clear();
            if (in) {
              raw[i][c][0].load(p + (kv && which ? 8 * j : cp.a));
              raw[i][c][1].load(p + (kv && which ? 8 * j + 4 : cp.b));
            }
          }
        }
        if (kv && !bad) {
          at = kv_record_of(a.c, s, blk, h, rec);
          const int t0 = p0 % a.c.page_tokens;
          s_old = held && at >= 0 ? __uint_as_float(ld_u1(a.c.pages + at + int64_t(2) * a.c.page_tokens * D +
                                                           4 * (which * (a.c.page_tokens / kKvBlock) + t0 / kKvBlock)))
                                  : 0.f;
        }
      };
      int item = blockIdx.x * kWarps + warp;
      if (item < items) load(item);  // in flight beside the tables
      __syncthreads();               // the tables of the block before have been read
      if (a.parent) {
        if (tid < min(n, QDQ_MAX_TREE)) s_parent[tid] = int(ld_u1(a.parent + first + tid));
        __syncthreads();
      }
      if (tid < kKvBlock) {
        const int i = p0 + tid - old;  // the token among the new ones
        int pos = p0 + tid;
        bool wrong = bad;
        if (a.parent && i >= 0 && i < n) {
          pos = old;
          for (int node = i;;) {  // up to the root (to ever smaller numbers, so it ends)
            const int up = s_parent[node];
            wrong |= up < -1 || up >= node;
            if (up < 0 || up >= node) break;
            node = up;
            ++pos;
          }
        }
        s_pos[tid] = pos;
        s_bad[tid] = wrong;
      }
      __syncthreads();
      for (int i = tid; i < fresh * pairs; i += kThreads) {
        const int t = held + i / pairs, p = i % pairs;
        const long long turn = (long long)((unsigned long long)(long long)s_pos[t] * s_turn[p]);
        float sn, cs;
        sincospif(float(turn) * 1.0842021724855044e-19f, &sn, &cs);  // 2^-63: half turns
        const bool wrong = s_bad[t] || !isfinite(__ldg(a.freqs + p));
        s_cos[t][p] = wrong ? qnan : cs;
        s_sin[t][p] = wrong ? qnan : sn;
      }
      __syncthreads();
      while (item < items) {
        const bool kv = item < 2 * a.c.n_kv;
        const int which = item & 1;
        const float *wp = kv ? (which ? nullptr : a.k_weight) : a.q_weight;
        float w[L::C][8];
        if (wp) {
#pragma unroll
          for (int c = 0; c < L::C; ++c) {
            const Couple<ADJACENT> cp(a, sub + L::LPT * c);
            const float4 u = __ldg(reinterpret_cast<const float4 *>(wp + cp.a)), v = __ldg(reinterpret_cast<const float4 *>(wp + cp.b));
            w[c][0] = u.x;
            w[c][1] = u.y;
            w[c][2] = u.z;
            w[c][3] = u.w;
            w[c][4] = v.x;
            w[c][5] = v.y;
            w[c][6] = v.z;
            w[c][7] = v.w;
          }
        }
        if (kv) {
          if (!bad && at >= 0) {  // (no page for these tokens: they are dropped)
            float x[L::NI][L::C][8], m = 0.f;
#pragma unroll
            for (int i = 0; i < L::NI; ++i) {
              const int t = i * L::GT + grp;
#pragma unroll
              for (int c = 0; c < L::C; ++c) {
                raw[i][c][0].values(x[i][c]);
                raw[i][c][1].values(x[i][c] + 4);
              }
              if (which == 0 && (i + 1) * L::GT > held && i * L::GT < end) {
                const int tt = min(max(t, held), end - 1);  // (a lane whose token is no new one: zeros by any angle)
                norm_turn<D, ADJACENT>(a, x[i], wp != nullptr, w, s_cos[tt], s_sin[tt], sub);
                if (t == tt && s_bad[tt]) m = qnan;
              }
              // (tokens that are not new: their zeros stay zeros, unless an angle is NaN)
              if (t >= held && t < end)
#pragma unroll
                for (int c = 0; c < L::C; ++c)
#pragma unroll
                  for (int e = 0; e < 8; ++e) m = max_abs(m, x[i][c][e]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
            quantise<D, ADJACENT>(a, a.c.pages + at, which, p0 % a.c.page_tokens, held, end, s_old, m, x, lane);
          }
        } else {
          const int u0 = (item - 2 * a.c.n_kv) * q_item;
#pragma unroll
          for (int i = 0; i < L::NI; ++i) {
            if (i < a.q_iters && u0 + i * L::GT < q_all) {
              // (past the last query: any token's angles)
              const int u = u0 + i * L::GT + grp, hq = head_of(u), t = held + u - hq * fresh;
              float x[L::C][8];
#pragma unroll
              for (int c = 0; c < L::C; ++c) {
                raw[i][c][0].values(x[c]);
                raw[i][c][1].values(x[c] + 4);
              }
              norm_turn<D, ADJACENT>(a, x, wp != nullptr, w, s_cos[t], s_sin[t], sub);
              T *o = static_cast<T *>(a.q_out) + (row0 + t) * a.q_out_stride + hq * D;
              const bool wrong = s_bad[t];
              if (u < q_all) {
#pragma unroll
                for (int c = 0; c < L::C; ++c) {
                  const Couple<ADJACENT> cp(a, sub + L::LPT * c);
                  if (wrong)
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[c][e] = qnan;
                  store4(o + cp.a, make_float4(x[c][0], x[c][1], x[c][2], x[c][3]));
                  store4(o + cp.b, make_float4(x[c][4], x[c][5], x[c][6], x[c][7]));
                }
              }
            }
          }
        }
        item += gridDim.x * kWarps;
        if (item < items) load(item);
      }
    }
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

}  // namespace

int launch_kv_append_rope(const KvPool &c, int head_dim, const int *kv_len, const int *cu, const int *parent, int n_seqs,
                          int max_new, int n_heads, const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride,
                          const void *k, int64_t k_stride, const void *v, int64_t v_stride, const float *q_weight,
                          const float *k_weight, float eps, const float *freqs, int n_rot, int adjacent, int type, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return fail_cuda(e);
  RopeArgs a{c, kv_len, cu, parent, q, k, v, q_out, q_weight, k_weight, freqs, q_stride, q_out_stride, k_stride, v_stride,
             n_seqs, kv_blocks_touched(max_new), max_new, n_heads, freqs ? n_rot : 0, 1, eps};
  const int gt = with_dim(head_dim, [](auto d) { return Lanes<decltype(d)::value>::GT; });
  const int tokens = max_new < kKvBlock ? max_new : kKvBlock;  // of a block
  const int64_t blocks = int64_t(a.n_blocks) * n_seqs, queries = int64_t(n_heads) * tokens;
  // few queries: a warp for every GT of them; many: 16 to a warp, whose loads are in flight together
  a.q_iters = queries * blocks > 64 * int64_t(di.sm_count) * gt ? kKvBlock / gt : 1;
  const int64_t items = 2 * c.n_kv + (queries + a.q_iters * gt - 1) / (a.q_iters * gt), groups = (items + kWarps - 1) / kWarps;
  const int64_t want = blocks < 4 * di.sm_count ? (4 * di.sm_count + blocks - 1) / blocks : 1;
  const dim3 grid(unsigned(groups < want ? groups : want), a.n_blocks < 65535 ? a.n_blocks : 65535, n_seqs < 65535 ? n_seqs : 65535);
  e = cudaError_t(with_type(type, [&](auto t) {
    return with_dim(head_dim, [&](auto d) {
      constexpr int D = decltype(d)::value;
      return int(adjacent ? launch(kv_append_rope_kernel<decltype(t), D, true>, grid, dim3(kWarps * 32), 0, s, a)
                          : launch(kv_append_rope_kernel<decltype(t), D, false>, grid, dim3(kWarps * 32), 0, s, a));
    });
  }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

}  // namespace qdq
