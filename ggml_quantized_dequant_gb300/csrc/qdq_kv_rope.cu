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
// A CTA takes the new tokens of one block of 16 (which share a key scale) and a share of the heads.  4 to 8 lanes take a
// token's head, in couples of four elements and the four that they are paired with, so that a rotation needs no other
// lane and the sum of squares two or three shuffles (32 lanes to a head: 9 shuffles each, 136 us for the prompts below).
// Every input is read once, every output written once.  Two kernels:
//   items (few new tokens): the CTA's threads compute the tokens' cosines and sines once into shared memory, while the first
//   loads are on their way; a warp holds a head's 16 keys (a block's maximum comes from its registers), or 16 queries of any
//   heads and tokens, so that a single token's heads spread over all warps.
//   rows (many): a warp keeps 4 or 8 tokens and goes through the heads with them.
// Measured (alone, in a graph): one token, 24 / 8 heads of 128, f32 5.3 us; 48 trees of 5 to 26 tokens, 32 / 8 heads of 128,
// bf16 9.7 us (items 13.9); 6 prompts of 900 to 3000 tokens, 24 / 8 heads of 128, bf16 53 us, 4.2 TB/s (items 85).
// Bound: for prompts the loads that 16 warps to an SM have in flight and the instructions' issue (half its rate) together; for
// single tokens the chain of launch, length, page and scale.
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

template <typename Couple>
__device__ __forceinline__ void load_weight(const float *p, const Couple &cp, float (&w)[8]) {
  const float4 u = __ldg(reinterpret_cast<const float4 *>(p + cp.a)), v = __ldg(reinterpret_cast<const float4 *>(p + cp.b));
  w[0] = u.x;
  w[1] = u.y;
  w[2] = u.z;
  w[3] = u.w;
  w[4] = v.x;
  w[5] = v.y;
  w[6] = v.z;
  w[7] = v.w;
}

// Norm (weight: of the lane's elements) and rotation of a token's head, all times `factor`; cosines and sines by couples, the
// lane's or the token's.  Each product and sum is rounded by itself in either kernel and kind of pairs, so that they agree:
// ((a w_a) cos - (b w_b) sin) / rms, ((b w_b) cos + [(a w_a) sin]) / rms, with one rounding for what is in brackets.
template <int D, bool ADJACENT, bool IN_LANE>
__device__ __forceinline__ void norm_turn(const RopeArgs &a, float (&x)[Lanes<D>::C][8], bool norm, const float (&weight)[Lanes<D>::C][8],
                                          const float4 *cs, const float4 *sn, int sub, float factor) {
  using L = Lanes<D>;
  if (norm) {
    Two s(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < L::C; ++c)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const Two v(x[c][e], x[c][e + 1]);
        s = fma(v, v, s);
        (v * Two(weight[c][e], weight[c][e + 1])).to(x[c][e], x[c][e + 1]);
      }
    float s0, s1;
    s.to(s0, s1);
    s0 += s1;
#pragma unroll
    for (int o = L::LPT / 2; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    factor *= rsqrtf(s0 * (1.f / D) + a.eps);
  }
  const Two minus(-1.f, -1.f), times(factor, factor);
#pragma unroll
  for (int c = 0; c < L::C; ++c) {
    const int j = sub + L::LPT * c;
    if (j < a.n_rot / 8) {
      const float4 co = cs[IN_LANE ? c : j], si = sn[IN_LANE ? c : j];
      if constexpr (ADJACENT) {
        const float cw[4] = {co.x, co.y, co.z, co.w}, sw[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = x[c][2 * e], q = x[c][2 * e + 1];
          x[c][2 * e] = __fmaf_rn(__fmul_rn(q, sw[e]), -1.f, __fmul_rn(p, cw[e]));
          x[c][2 * e + 1] = __fmaf_rn(p, sw[e], __fmul_rn(q, cw[e]));
        }
      } else {
        const Two cw[2] = {Two(co.x, co.y), Two(co.z, co.w)}, sw[2] = {Two(si.x, si.y), Two(si.z, si.w)};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const Two p(x[c][2 * e], x[c][2 * e + 1]), q(x[c][4 + 2 * e], x[c][5 + 2 * e]);
          fma(q * sw[e], minus, p * cw[e]).to(x[c][2 * e], x[c][2 * e + 1]);
          fma(p, sw[e], q * cw[e]).to(x[c][4 + 2 * e], x[c][5 + 2 * e]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; e += 2) (Two(x[c][e], x[c][e + 1]) * times).to(x[c][e], x[c][e + 1]);
  }
}

// The larger magnitude; NaN wins.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// What a block's codes are made by (definition in qdq_kv.cu).
struct Scale {
  float old, now, inv, again;
  __device__ __forceinline__ Scale(float s_old, float m) : old(s_old) {  // m: the new tokens' largest magnitude
    float s_new = __fdiv_rn(m, 127.f);
    if (s_new < 1.17549435e-38f) s_new = 0.f;
    if (!(m < __int_as_float(0x7f800000))) s_new = __int_as_float(0x7fffffff);
    now = max_abs_bits(s_old, s_new);  // NaN wins
    inv = now > 0.f ? __frcp_rn(now) : 0.f;
    again = now > 0.f ? __fdiv_rn(s_old, now) : 0.f;
  }
};
// Four new codes.  A product with 1 / s is at most 127 and some roundings, so that 1.5 2^23 added and its bits' low byte
// are rint and its code.
__device__ __forceinline__ uint32_t new_codes(const float *v, const Scale &sc) {
  uint32_t w[4];  // (a product and a sum of two f32 at once come out as one rounding here, which is not the definition)
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(__fadd_rn(__fmul_rn(v[e], sc.inv), 12582912.f));
  const uint32_t r = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
  return sc.now == sc.now ? r : 0u;
}
// Four codes that a block held, rounded to a larger scale.
__device__ __forceinline__ void old_codes(uint32_t *p, const Scale &sc) {
  const uint32_t w = ld_u1(p);
  uint32_t r = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) r |= uint32_t(__float2int_rn(float(int8_t(w >> (8 * j))) * sc.again) & 0xFF) << (8 * j);
  *p = r;
}

// The block's codes and scale from its new tokens held .. end - 1 in x, whose largest magnitude is m.
template <int D, bool ADJACENT>
__device__ __forceinline__ void quantise(const RopeArgs &a, uint8_t *record, int which, int t0, int held, int end, float s_old, float m,
                                         const float (&x)[Lanes<D>::NI][Lanes<D>::C][8], int lane) {
  using L = Lanes<D>;
  const int sub = lane % L::LPT, page_tokens = a.c.page_tokens;
  if (!QDQ_GUARD(t0 + kKvBlock <= page_tokens && record >= a.c.pages &&
                     record + kv_record_bytes(page_tokens, D) <= a.c.pages + int64_t(a.c.n_pages) * a.c.n_kv * kv_record_bytes(page_tokens, D),
                 QDQ_CHECK_OUT))
    return;
  int8_t *codes = reinterpret_cast<int8_t *>(record) + (int64_t(which) * page_tokens + t0) * D;
  const Scale sc(s_old, m);
  const bool grown = held && sc.now != sc.old;
#pragma unroll
  for (int i = 0; i < L::NI; ++i) {
    const int t = i * L::GT + lane / L::LPT;
#pragma unroll
    for (int c = 0; c < L::C; ++c) {
      const int j = sub + L::LPT * c;
      const Couple<ADJACENT> at(a, j);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t *p = reinterpret_cast<uint32_t *>(codes + t * D + (which ? 8 * j + 4 * q : q ? at.b : at.a));
        if (grown && t < held) old_codes(p, sc);
        if (t >= held && t < end) *p = new_codes(&x[i][c][4 * q], sc);
      }
    }
  }
  if (lane == 0 && (held == 0 || grown))
    *(reinterpret_cast<float *>(record + int64_t(2) * page_tokens * D) + which * (page_tokens / kKvBlock) + t0 / kKvBlock) = sc.now;
}

// 2^64 frac(freq / 2 pi), a turn's fraction per position
__device__ __forceinline__ unsigned long long turn_of(float f) {
  const double turns = double(f) * 0.15915494309189533577;  // 1 / (2 pi)
  return isfinite(f) ? (unsigned long long)((turns - floor(turns)) * 18446744073709551616.0) : 0ull;
}
__device__ __forceinline__ void angle(int pos, unsigned long long turn, float *sn, float *cs) {
  // the product's upper 32 bits: a turn to 2^-32, where an angle's f32 has 2^-25
  const int half = int(((unsigned long long)(long long)pos * turn + 0x80000000ull) >> 32);
  sincospif(float(half) * 4.656612873077393e-10f, sn, cs);  // 2^-31: half turns
}
// Position of node i of a tree whose first node is at `old`; `wrong` where it or an ancestor has no valid parent.
__device__ __forceinline__ int tree_position(const int *parent, int i, int old, bool &wrong) {
  int pos = old;
  for (int node = i;;) {  // up to the root (to ever smaller numbers, so it ends)
    const int up = parent[node];
    wrong |= up < -1 || up >= node;
    if (up < 0 || up >= node) return pos;
    node = up;
    ++pos;
  }
}

template <typename T, int D, bool ADJACENT>
__global__ void __launch_bounds__(kWarps * 32, D <= 128 ? 3 : 2) kv_append_rope_kernel(const RopeArgs a) {
  using L = Lanes<D>;
  constexpr int kThreads = kWarps * 32;
  __shared__ unsigned long long s_turn[D / 2];
  __shared__ __align__(16) float s_cos[kKvBlock][D / 2], s_sin[kKvBlock][D / 2];
  __shared__ int s_parent[QDQ_MAX_TREE], s_pos[kKvBlock];
  __shared__ bool s_bad[kKvBlock];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane % L::LPT, grp = lane / L::LPT;
  const float qnan = __int_as_float(0x7fffffff);
  pdl_launch_dependents();
  const int pairs = a.n_rot / 2;
  for (int i = tid; i < pairs; i += kThreads) {  // (frequencies and weights count as weights: read ahead of the wait)
    s_turn[i] = turn_of(__ldg(a.freqs + i));
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
        if (a.parent && i >= 0 && i < n) pos = tree_position(s_parent, i, old, wrong);
        s_pos[tid] = pos;
        s_bad[tid] = wrong;
      }
      __syncthreads();
      for (int i = tid; i < fresh * pairs; i += kThreads) {
        const int t = held + i / pairs, p = i % pairs;
        float sn, cs;
        angle(s_pos[t], s_turn[p], &sn, &cs);
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
          for (int c = 0; c < L::C; ++c) load_weight(wp, Couple<ADJACENT>(a, sub + L::LPT * c), w[c]);
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
                norm_turn<D, ADJACENT, false>(a, x[i], wp != nullptr, w, reinterpret_cast<const float4 *>(s_cos[tt]),
                                              reinterpret_cast<const float4 *>(s_sin[tt]), sub, 1.f);
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
              norm_turn<D, ADJACENT, false>(a, x, wp != nullptr, w, reinterpret_cast<const float4 *>(s_cos[t]),
                                            reinterpret_cast<const float4 *>(s_sin[t]), sub, s_bad[t] ? qnan : 1.f);
              T *o = static_cast<T *>(a.q_out) + (row0 + t) * a.q_out_stride + hq * D;
              if (u < q_all) {
#pragma unroll
                for (int c = 0; c < L::C; ++c) {
                  const Couple<ADJACENT> cp(a, sub + L::LPT * c);
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

template <typename T, int D>
constexpr int kRowsCtas = D == 64 ? 5 - (sizeof(T) == 4) : D == 128 ? (sizeof(T) == 2 ? 4 : 3) : 2;  // resident per SM
// Prompts: a warp keeps GT tokens of the block and goes through the heads with them, their cosines and sines in
// registers (no tables, and a quarter of the registers that a whole block's keys take).  The NI warps that share a block
// exchange the largest magnitudes of a head's keys and values; the next head's elements are on the way meanwhile.
// A CTA for 8 heads: for 6 the prompts take 61 us, for 8 53, for 12 54; three heads of queries on their way: with two 56, with
// four 52.5, but heads of 256 in f32 38 instead of 37.
template <typename T, int D, bool ADJACENT>
__global__ void __launch_bounds__(kWarps * 32, kRowsCtas<T, D>) kv_append_rope_rows_kernel(const RopeArgs a) {
  using L = Lanes<D>;
  constexpr int kThreads = kWarps * 32, kGroups = kWarps / L::NI;  // groups of warps, each with heads of its own
  __shared__ unsigned long long s_turn[D / 2];
  __shared__ float s_max[2][kWarps][2];
  __shared__ int s_parent[QDQ_MAX_TREE];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane % L::LPT, grp = lane / L::LPT;
  const int slice = warp % L::NI, group = warp / L::NI;
  const float qnan = __int_as_float(0x7fffffff);
  pdl_launch_dependents();
  const int pairs = a.n_rot / 2;
  for (int i = tid; i < pairs; i += kThreads) s_turn[i] = turn_of(__ldg(a.freqs + i));
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
      const int blk = old / kKvBlock + b, p0 = blk * kKvBlock, t0 = p0 % a.c.page_tokens;
      if (p0 >= len) break;
      const int held = max(old - p0, 0), end = min(len - p0, kKvBlock);
      const int t = slice * L::GT + grp, i = p0 + t - old;  // the lane's token in the block, and among the new ones
      const bool in = t >= held && t < end;
      const int64_t row = int64_t(first) + (in ? i : 0);
      const int stride = gridDim.x * kGroups, h0 = blockIdx.x * kGroups + group;
      __syncthreads();  // (s_turn is written; the block before is done with s_parent and s_max)
      if (a.parent) {
        if (tid < min(n, QDQ_MAX_TREE)) s_parent[tid] = int(ld_u1(a.parent + first + tid));
        __syncthreads();
      }
      int pos = p0 + t;
      bool wrong = bad;
      if (a.parent && in) pos = tree_position(s_parent, i, old, wrong);
      float4 cs[L::C], sn[L::C];
#pragma unroll
      for (int c = 0; c < L::C; ++c) {
        const int j = sub + L::LPT * c;
        float x[4], y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = 1.f;
          y[e] = 0.f;
          if (j < a.n_rot / 8) {
            angle(pos, s_turn[4 * j + e], &y[e], &x[e]);
            if (wrong || !isfinite(__ldg(a.freqs + 4 * j + e))) x[e] = y[e] = qnan;
          }
        }
        cs[c] = make_float4(x[0], x[1], x[2], x[3]);
        sn[c] = make_float4(y[0], y[1], y[2], y[3]);
      }
      // (lanes without a token read the first one's elements and write nothing)
      auto load = [&](Raw<T> (&r)[L::C][2], const T *p, bool plain) {
#pragma unroll
        for (int c = 0; c < L::C; ++c) {
          const int j = sub + L::LPT * c;
          const Couple<ADJACENT> cp(a, j);
          r[c][0].load(p + (plain ? 8 * j : cp.a));
          r[c][1].load(p + (plain ? 8 * j + 4 : cp.b));
        }
      };
      // keys and values, head by head (every warp of the CTA goes through the same number of them)
      if (!bad) {
        const T *kp = static_cast<const T *>(a.k) + row * a.k_stride, *vp = static_cast<const T *>(a.v) + row * a.v_stride;
        const int rounds = (a.c.n_kv - int(blockIdx.x) * kGroups + stride - 1) / stride;
        float w[L::C][8];
        if (a.k_weight)
#pragma unroll
          for (int c = 0; c < L::C; ++c) load_weight(a.k_weight, Couple<ADJACENT>(a, sub + L::LPT * c), w[c]);
        Raw<T> rk[L::C][2], rv[L::C][2];
        load(rk, kp + min(h0, a.c.n_kv - 1) * D, false);
        load(rv, vp + min(h0, a.c.n_kv - 1) * D, true);
        const int64_t at0 = kv_record_of(a.c, s, blk, 0, rec);  // without a page the tokens are dropped
        uint8_t *const records = a.c.pages + (at0 < 0 ? 0 : at0);
        for (int r = 0; r < rounds; ++r) {
          const int h = h0 + r * stride;
          const bool there = at0 >= 0 && h < a.c.n_kv;
          int8_t *const record = reinterpret_cast<int8_t *>(records + (there ? h * rec : 0));
          float *scales = reinterpret_cast<float *>(record + 2 * a.c.page_tokens * D) + t0 / kKvBlock, *v_scale = scales + a.c.page_tokens / kKvBlock;
          float k_old = 0.f, v_old = 0.f;
          if (held && there) {
            k_old = __uint_as_float(ld_u1(scales));
            v_old = __uint_as_float(ld_u1(v_scale));
          }
          float xk[L::C][8], xv[L::C][8], mk = 0.f, mv = 0.f;
#pragma unroll
          for (int c = 0; c < L::C; ++c) {
            rk[c][0].values(xk[c]);
            rk[c][1].values(xk[c] + 4);
            rv[c][0].values(xv[c]);
            rv[c][1].values(xv[c] + 4);
          }
          if (h + stride < a.c.n_kv) {
            load(rk, kp + (h + stride) * D, false);
            load(rv, vp + (h + stride) * D, true);
          }
          norm_turn<D, ADJACENT, true>(a, xk, a.k_weight != nullptr, w, cs, sn, sub, 1.f);
          if (in) {
#pragma unroll
            for (int c = 0; c < L::C; ++c)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                mk = max_abs(mk, xk[c][e]);
                mv = max_abs(mv, xv[c][e]);
              }
            if (wrong) mk = qnan;
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            mk = max_abs(mk, __shfl_xor_sync(0xffffffffu, mk, o));
            mv = max_abs(mv, __shfl_xor_sync(0xffffffffu, mv, o));
          }
          if (lane == 0) {
            s_max[r & 1][warp][0] = mk;
            s_max[r & 1][warp][1] = mv;
          }
          __syncthreads();
          if (!there || !QDQ_GUARD(t0 + kKvBlock <= a.c.page_tokens && at0 + (h + 1) * rec <= int64_t(a.c.n_pages) * a.c.n_kv * rec, QDQ_CHECK_OUT)) continue;
#pragma unroll
          for (int y = 0; y < L::NI; ++y) {
            mk = max_abs(mk, s_max[r & 1][group * L::NI + y][0]);
            mv = max_abs(mv, s_max[r & 1][group * L::NI + y][1]);
          }
          const Scale sk(k_old, mk), sv(v_old, mv);
          int8_t *codes = record + (t0 + t) * D, *v_codes = codes + a.c.page_tokens * D;
#pragma unroll
          for (int c = 0; c < L::C; ++c) {
            const int j = sub + L::LPT * c;
            const Couple<ADJACENT> cp(a, j);
            if (in) {
              *reinterpret_cast<uint32_t *>(codes + cp.a) = new_codes(xk[c], sk);
              *reinterpret_cast<uint32_t *>(codes + cp.b) = new_codes(xk[c] + 4, sk);
              *reinterpret_cast<uint2 *>(v_codes + 8 * j) = make_uint2(new_codes(xv[c], sv), new_codes(xv[c] + 4, sv));
            } else if (t < held) {  // a larger scale: what the block held, rounded to it
              if (sk.now != sk.old) {
                old_codes(reinterpret_cast<uint32_t *>(codes + cp.a), sk);
                old_codes(reinterpret_cast<uint32_t *>(codes + cp.b), sk);
              }
              if (sv.now != sv.old) {
                old_codes(reinterpret_cast<uint32_t *>(v_codes + 8 * j), sv);
                old_codes(reinterpret_cast<uint32_t *>(v_codes + 8 * j + 4), sv);
              }
            }
          }
          if (lane == 0 && slice == 0) {
            if (held == 0 || sk.now != sk.old) *scales = sk.now;
            if (held == 0 || sv.now != sv.old) *v_scale = sv.now;
          }
        }
      }
      // queries
      if (a.n_heads > 0) {
        const T *qp = static_cast<const T *>(a.q) + row * a.q_stride;
        T *op = static_cast<T *>(a.q_out) + row * a.q_out_stride;
        float w[L::C][8];
        if (a.q_weight)
#pragma unroll
          for (int c = 0; c < L::C; ++c) load_weight(a.q_weight, Couple<ADJACENT>(a, sub + L::LPT * c), w[c]);
        constexpr int kAhead = 3;  // heads whose elements are on the way
        Raw<T> r[kAhead][L::C][2];
#pragma unroll
        for (int y = 0; y < kAhead; ++y)
          load(r[y], qp + min(h0 + y * stride, a.n_heads - 1) * D, false);
        for (int h = h0; h < a.n_heads; h += kAhead * stride) {
#pragma unroll
          for (int y = 0; y < kAhead; ++y) {
            const int hh = h + y * stride;
            if (hh >= a.n_heads) break;
            float x[L::C][8];
#pragma unroll
            for (int c = 0; c < L::C; ++c) {
              r[y][c][0].values(x[c]);
              r[y][c][1].values(x[c] + 4);
            }
            if (hh + kAhead * stride < a.n_heads) load(r[y], qp + (hh + kAhead * stride) * D, false);
            norm_turn<D, ADJACENT, true>(a, x, a.q_weight != nullptr, w, cs, sn, sub, wrong ? qnan : 1.f);
            if (in && QDQ_GUARD(i >= 0 && i < n && hh < a.n_heads, QDQ_CHECK_OUT)) {
#pragma unroll
              for (int c = 0; c < L::C; ++c) {
                const Couple<ADJACENT> cp(a, sub + L::LPT * c);
                store4(op + hh * D + cp.a, make_float4(x[c][0], x[c][1], x[c][2], x[c][3]));
                store4(op + hh * D + cp.b, make_float4(x[c][4], x[c][5], x[c][6], x[c][7]));
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
  RopeArgs a{c, kv_len, cu, parent, q, k, v, q_out, q_weight, k_weight, freqs, q_stride, q_out_stride, k_stride, v_stride,
             n_seqs, kv_blocks_touched(max_new), max_new, n_heads, freqs ? n_rot : 0, 1, eps};
  const int gt = with_dim(head_dim, [](auto d) { return Lanes<decltype(d)::value>::GT; });
  const int tokens = max_new < kKvBlock ? max_new : kKvBlock;  // of a block
  const int64_t blocks = int64_t(a.n_blocks) * n_seqs, queries = int64_t(n_heads) * tokens;
  // few queries: a warp for every GT of them; many: 16 to a warp, whose loads are in flight together
  a.q_iters = queries * blocks > 64 * int64_t(di.sm_count) * gt ? kKvBlock / gt : 1;
  // A warp that keeps its tokens pays for their angles by itself and takes an idle share of a block with few of them:
  // 1 sequence of 5 tokens, 32 / 8 heads of 128, bf16: 5.5 us items, 7.6 rows; 64 of 5: 10.7, 11.2; 64 of 8: 13.4, 11.4;
  // 16 of 8: 8.3, 8.7; 16 of 12: 9.7, 8.7; 1 of 64: 7.6, 8.2; 1 of 4096: 39.8, 27.5.
  const bool rows = max_new >= 6 && int64_t(n_seqs) * max_new >= 160;
  const int64_t items = 2 * c.n_kv + (queries + a.q_iters * gt - 1) / (a.q_iters * gt);
  const int64_t heads = n_heads > c.n_kv ? n_heads : c.n_kv;
  const int64_t groups = rows ? (heads + 7) / 8 : (items + kWarps - 1) / kWarps;
  const int64_t want = rows ? groups : blocks < 4 * di.sm_count ? (4 * di.sm_count + blocks - 1) / blocks : 1;
  const dim3 grid(unsigned(groups < want ? groups : want), a.n_blocks < 65535 ? a.n_blocks : 65535, n_seqs < 65535 ? n_seqs : 65535);
  e = cudaError_t(with_type(type, [&](auto t) {
    return with_dim(head_dim, [&](auto d) {
      constexpr int D = decltype(d)::value;
      if (rows)
        return int(adjacent ? launch(kv_append_rope_rows_kernel<decltype(t), D, true>, grid, dim3(kWarps * 32), 0, s, a)
                            : launch(kv_append_rope_rows_kernel<decltype(t), D, false>, grid, dim3(kWarps * 32), 0, s, a));
      return int(adjacent ? launch(kv_append_rope_kernel<decltype(t), D, true>, grid, dim3(kWarps * 32), 0, s, a)
                          : launch(kv_append_rope_kernel<decltype(t), D, false>, grid, dim3(kWarps * 32), 0, s, a));
    });
  }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

QDQ_CHECK_READER(read_checks_rope)

}  // namespace qdq
