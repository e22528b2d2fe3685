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
// A CTA takes the new tokens of one block of 16 (which share a key scale) and a share of the heads: their cosines
// and sines once into shared memory, then a warp at a time one head's 16 tokens: all loads before the first use, a token's
// elements in 16 or 32 lanes (its sum of squares is folded by shuffles, the other element of a pair lies in another
// lane or in the same four elements), a key block's maximum from registers.  Every input is read once, every output written once.
// Bound: memory for prompts, for single tokens the chain of launch, length, page and scale.
#include "qdq_types.cuh"

namespace qdq {
namespace {

constexpr int kWarps = 8;

struct RopeArgs {
  KvPool c;
  const int *kv_len, *cu, *parent;  // cu NULL: one token each; parent NULL: one after the other
  const void *q, *k, *v;
  void *q_out;
  const float *q_weight, *k_weight, *freqs;
  int64_t q_stride, q_out_stride, k_stride, v_stride;
  int n_seqs, n_blocks, max_new, n_heads, n_rot, adjacent;
  float eps;
};

// Where a lane's elements lie: LPT lanes to a token, TPI tokens at a time, CPT times four elements 128 apart.
template <int D>
struct Lanes {
  static constexpr int LPT = D == 64 ? 16 : 32, TPI = 32 / LPT, NI = kKvBlock / TPI, CPT = (D + 127) / 128;
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
  __device__ __forceinline__ void values(float (&x)[4]) const {
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

// One head's new tokens of a block: tokens lo to hi - 1 of the 16; x: element 0 of token 0's head.
template <typename T, int D>
__device__ __forceinline__ void load_head(const T *x, int64_t stride, int lo, int hi, int lane,
                                          float (&f)[Lanes<D>::NI][Lanes<D>::CPT][4]) {
  using L = Lanes<D>;
  Raw<T> r[L::NI][L::CPT];
  const int sub = lane % L::LPT;
#pragma unroll
  for (int i = 0; i < L::NI; ++i) {
    const int t = i * L::TPI + lane / L::LPT;
#pragma unroll
    for (int c = 0; c < L::CPT; ++c) {
      const int d = 4 * sub + 128 * c;
#pragma unroll
      for (uint32_t &w : r[i][c].w) w = 0;
      if (t >= lo && t < hi && d < D) r[i][c].load(x + t * stride + d);
    }
  }
#pragma unroll
  for (int i = 0; i < L::NI; ++i)
#pragma unroll
    for (int c = 0; c < L::CPT; ++c) r[i][c].values(f[i][c]);
}

// Norm and rotation of iteration i's tokens.
template <int D>
__device__ __forceinline__ void norm_turn(const RopeArgs &a, float (&x)[Lanes<D>::CPT][4], const float *weight, const float *cs,
                                          const float *sn, int lane) {
  using L = Lanes<D>;
  const int sub = lane % L::LPT;
  if (weight) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < L::CPT; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) s = fmaf(x[c][e], x[c][e], s);
#pragma unroll
    for (int o = L::LPT / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float inv = rsqrtf(s * (1.f / D) + a.eps);
#pragma unroll
    for (int c = 0; c < L::CPT; ++c) {
      const int d = 4 * sub + 128 * c;
      const float4 w = d < D ? __ldg(reinterpret_cast<const float4 *>(weight + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[c][0] *= inv * w.x;
      x[c][1] *= inv * w.y;
      x[c][2] *= inv * w.z;
      x[c][3] *= inv * w.w;
    }
  }
  if (a.n_rot == 0) return;
  if (a.adjacent) {
#pragma unroll
    for (int c = 0; c < L::CPT; ++c) {
      const int d = 4 * sub + 128 * c;
      if (d < a.n_rot) {
        const float2 co = *reinterpret_cast<const float2 *>(cs + d / 2), si = *reinterpret_cast<const float2 *>(sn + d / 2);
        const float x0 = x[c][0], x2 = x[c][2];
        x[c][0] = x0 * co.x - x[c][1] * si.x;
        x[c][1] = x[c][1] * co.x + x0 * si.x;
        x[c][2] = x2 * co.y - x[c][3] * si.y;
        x[c][3] = x[c][3] * co.y + x2 * si.y;
      }
    }
    return;
  }
  const int h = a.n_rot / 2;
  float y[L::CPT][4];
#pragma unroll
  for (int c = 0; c < L::CPT; ++c) {
    const int d = 4 * sub + 128 * c;
    const bool turned = d < a.n_rot, low = d < h;
    const int other = turned ? (low ? d + h : d - h) : d;  // where the other elements of the pairs are
    const int from = lane / L::LPT * L::LPT + other / 4 % L::LPT;
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[e] = __shfl_sync(0xffffffffu, x[0][e], from);
      if constexpr (L::CPT == 2) {
        const float far = __shfl_sync(0xffffffffu, x[1][e], from);
        p[e] = other >= 128 ? far : p[e];
      }
    }
    if (turned) {
      const int i = low ? d : d - h;
      const float4 co = *reinterpret_cast<const float4 *>(cs + i), si = *reinterpret_cast<const float4 *>(sn + i);
      const float g = low ? -1.f : 1.f;
      y[c][0] = x[c][0] * co.x + g * p[0] * si.x;
      y[c][1] = x[c][1] * co.y + g * p[1] * si.y;
      y[c][2] = x[c][2] * co.z + g * p[2] * si.z;
      y[c][3] = x[c][3] * co.w + g * p[3] * si.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[c][e] = x[c][e];
    }
  }
#pragma unroll
  for (int c = 0; c < L::CPT; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[c][e] = y[c][e];
}

// The block's codes and scale from its new tokens held..end - 1 in x (definition in qdq_kv.cu).
template <int D>
__device__ __forceinline__ void quantise(uint8_t *record, int page_tokens, int which, int t0, int held, int end,
                                         const float (&x)[Lanes<D>::NI][Lanes<D>::CPT][4], int lane) {
  using L = Lanes<D>;
  const int sub = lane % L::LPT;
  int8_t *codes = reinterpret_cast<int8_t *>(record) + (int64_t(which) * page_tokens + t0) * D;
  float *scale = reinterpret_cast<float *>(record + int64_t(2) * page_tokens * D) + which * (page_tokens / kKvBlock) + t0 / kKvBlock;
  const float s_old = held ? __uint_as_float(ld_u1(scale)) : 0.f;
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < L::NI; ++i)
#pragma unroll
    for (int c = 0; c < L::CPT; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max_abs_bits(m, x[i][c][e]);  // 0 where there is no new token
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_abs_bits(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s_new = __fdiv_rn(m, 127.f);
  if (s_new < 1.17549435e-38f) s_new = 0.f;
  if (!(m < __int_as_float(0x7f800000))) s_new = __int_as_float(0x7fffffff);
  const float sc = max_abs_bits(s_old, s_new);  // NaN wins
  const float inv = sc > 0.f ? __frcp_rn(sc) : 0.f;
  const bool grown = held && sc != s_old;
  const float again = grown && sc > 0.f ? __fdiv_rn(s_old, sc) : 0.f;
#pragma unroll
  for (int i = 0; i < L::NI; ++i) {
    const int t = i * L::TPI + lane / L::LPT;
#pragma unroll
    for (int c = 0; c < L::CPT; ++c) {
      const int d = 4 * sub + 128 * c;
      if (d >= D) continue;
      uint32_t *p = reinterpret_cast<uint32_t *>(codes + t * D + d);
      if (grown && t < held) {  // a larger scale: what the block held, rounded to it
        const uint32_t w = ld_u1(p);
        uint32_t r = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) r |= uint32_t(__float2int_rn(float(int8_t(w >> (8 * j))) * again) & 0xFF) << (8 * j);
        *p = r;
      }
      if (t >= held && t < end) {
        auto code = [&](float f) { return uint32_t(__float2int_rn(fminf(fmaxf(f * inv, -127.f), 127.f)) & 0xFF); };
        *p = code(x[i][c][0]) | (code(x[i][c][1]) << 8) | (code(x[i][c][2]) << 16) | (code(x[i][c][3]) << 24);
      }
    }
  }
  if (lane == 0 && (held == 0 || sc != s_old)) *scale = sc;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, D <= 128 ? 2 : 1) kv_append_rope_kernel(const RopeArgs a) {
  using L = Lanes<D>;
  constexpr int kThreads = kWarps * 32;
  __shared__ unsigned long long s_turn[D / 2];  // 2^64 frac(freq / 2 pi)
  __shared__ __align__(16) float s_cos[kKvBlock][D / 2], s_sin[kKvBlock][D / 2];
  __shared__ int s_parent[QDQ_MAX_TREE], s_pos[kKvBlock];
  __shared__ bool s_bad[kKvBlock];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float qnan = __int_as_float(0x7fffffff);
  pdl_launch_dependents();
  const int pairs = a.n_rot / 2;
  for (int i = tid; i < pairs; i += kThreads) {  // (frequencies and weights count as weights: read ahead of the wait)
    const double turns = double(__ldg(a.freqs + i)) * 0.15915494309189533577;  // 1 / (2 pi)
    s_turn[i] = (unsigned long long)((turns - floor(turns)) * 18446744073709551616.0);
  }
  pdl_wait();
  const int items = 2 * a.c.n_kv + a.n_heads;
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
      const int held = max(old - p0, 0), end = min(len - p0, kKvBlock);
      __syncthreads();  // the tables of the block before have been read
      if (a.parent && tid < min(n, QDQ_MAX_TREE)) s_parent[tid] = int(ld_u1(a.parent + first + tid));
      __syncthreads();
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
      for (int i = tid; i < (end - held) * pairs; i += kThreads) {
        const int t = held + i / pairs, p = i % pairs;
        const long long turn = (long long)((unsigned long long)(long long)s_pos[t] * s_turn[p]);
        float sn, cs;
        sincospif(float(turn) * 1.0842021724855044e-19f, &sn, &cs);  // 2^-63: half turns
        const bool wrong = s_bad[t] || !isfinite(__ldg(a.freqs + p));
        s_cos[t][p] = wrong ? qnan : cs;
        s_sin[t][p] = wrong ? qnan : sn;
      }
      __syncthreads();
      for (int item = blockIdx.x * kWarps + warp; item < items; item += gridDim.x * kWarps) {
        float x[L::NI][L::CPT][4];
        const int64_t row0 = int64_t(first) + p0 - old;  // the row of the block's token 0 (a negative part is never read)
        if (item < 2 * a.c.n_kv) {
          const int h = item >> 1, which = item & 1;
          if (bad) continue;
          const T *p = static_cast<const T *>(which ? a.v : a.k) + row0 * (which ? a.v_stride : a.k_stride) + h * D;
          load_head<T, D>(p, which ? a.v_stride : a.k_stride, held, end, lane, x);
          const int64_t at = kv_record_of(a.c, s, blk, h, rec);
          if (at < 0) continue;  // no page for these tokens: they are dropped
          if (which == 0) {
#pragma unroll
            for (int i = 0; i < L::NI; ++i) {
              const int t = i * L::TPI + lane / L::LPT;
              if (i * L::TPI + L::TPI > held && i * L::TPI < end) {
                const int at_t = min(max(t, held), end - 1);  // (a lane whose token is no new one: zeros by any angle)
                norm_turn<D>(a, x[i], a.k_weight, s_cos[at_t], s_sin[at_t], lane);
                if (t < held || t >= end) {
#pragma unroll
                  for (int c = 0; c < L::CPT; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[i][c][e] = 0.f;
                } else if (s_bad[t]) {  // also where nothing is turned
#pragma unroll
                  for (int c = 0; c < L::CPT; ++c) x[i][c][0] = qnan;
                }
              }
            }
          }
          quantise<D>(a.c.pages + at, a.c.page_tokens, which, p0 % a.c.page_tokens, held, end, x, lane);
        } else {
          const int h = item - 2 * a.c.n_kv;
          load_head<T, D>(static_cast<const T *>(a.q) + row0 * a.q_stride + h * D, a.q_stride, held, end, lane, x);
          T *o = static_cast<T *>(a.q_out) + row0 * a.q_out_stride + h * D;
#pragma unroll
          for (int i = 0; i < L::NI; ++i) {
            const int t = i * L::TPI + lane / L::LPT;
            if (i * L::TPI + L::TPI > held && i * L::TPI < end) {
              const int at_t = min(max(t, held), end - 1);
              norm_turn<D>(a, x[i], a.q_weight, s_cos[at_t], s_sin[at_t], lane);
              const bool wrong = s_bad[at_t];
#pragma unroll
              for (int c = 0; c < L::CPT; ++c) {
                const int d = 4 * (lane % L::LPT) + 128 * c;
                if (t >= held && t < end && d < D)
                  store4(o + t * a.q_out_stride + d, wrong ? make_float4(qnan, qnan, qnan, qnan)
                                                            : make_float4(x[i][c][0], x[i][c][1], x[i][c][2], x[i][c][3]));
              }
            }
          }
        }
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
  const RopeArgs a{c, kv_len, cu, parent, q, k, v, q_out, q_weight, k_weight, freqs, q_stride, q_out_stride, k_stride, v_stride,
                   n_seqs, kv_blocks_touched(max_new), max_new, n_heads, freqs ? n_rot : 0, adjacent, eps};
  const int groups = (2 * c.n_kv + n_heads + kWarps - 1) / kWarps;
  const int64_t blocks = int64_t(a.n_blocks) * n_seqs;
  const int want = int(blocks < 4 * di.sm_count ? (4 * di.sm_count + blocks - 1) / blocks : 1);
  const dim3 grid(groups < want ? groups : want, a.n_blocks < 65535 ? a.n_blocks : 65535, n_seqs < 65535 ? n_seqs : 65535);
  e = cudaError_t(with_type(type, [&](auto t) {
    return with_dim(head_dim, [&](auto d) {
      return int(launch(kv_append_rope_kernel<decltype(t), decltype(d)::value>, grid, dim3(kWarps * 32), 0, s, a));
    });
  }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

}  // namespace qdq
