// The paged 8-bit key/value cache: appending tokens (quantisation) and reading tokens back.
//
// A block is 16 consecutive tokens of one sequence and head; its keys share one f32 scale and
// its values another:
//   s = max(s_old, max |x| / 127)  over the new tokens x of the block (s_old: its scale before,
//       0 when it held no token; a scale below the smallest normal f32 counts as 0),
//   code = rint(x * (1 / s)) for new tokens,  rint(code * (s_old / s)) for those it held,
// every quotient, product and maximum in f32.  So a scale never shrinks while a block fills,
// and appending the same tokens twice changes nothing.  A new token that is not finite makes
// the block's scale NaN, and with it every value of the block.
//
// One warp per (sequence, block, head, keys or values): the block's new elements stay in
// registers between the maximum and the rounding, so each is read once.
// Bound: memory for a prompt's tokens, for single tokens the chain of launch, length, page and scale.
// Measured (8 heads of 128): append 48 single tokens 3.1 us; append 6 sequences of 500 to 900 bf16 tokens
// 16.2 us (17 MB in and out with the codes), read 3001 tokens of them back 14.8 us; the two
// one after the other 27.9 us, 80 % of a plain copy's rate.
#include "qdq_types.cuh"

namespace qdq {
namespace {

constexpr int kWarps = 4;

struct AppendArgs {
  KvPool c;
  const int *kv_len, *cu;  // tokens after the append; new tokens before each sequence (NULL: one each)
  const void *k, *v;
  int64_t k_stride, v_stride;
  int n_seqs, n_blocks;  // blocks per sequence that the grid covers
  int max_new;           // tokens of a sequence past it are dropped
};

// Four elements as loaded: half the registers for the 16-bit types, and a maximum in half the steps
// (their magnitudes' order is that of their bits, a NaN the largest).
template <typename T>
struct Quad {
  uint32_t w[sizeof(T)];  // 4 sizeof(T) bytes
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
  __device__ __forceinline__ uint32_t raise(uint32_t bits) const {  // the larger magnitudes' bits
#pragma unroll
    for (uint32_t x : w) {
      if constexpr (sizeof(T) == 4)
        bits = max(bits, x & 0x7FFFFFFFu);
      else
        bits = __vmaxu2(bits, x & 0x7FFF7FFFu);
    }
    return bits;
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) return max(a, b);
    return __vmaxu2(a, b);
  }
  static __device__ __forceinline__ float magnitude(uint32_t bits) {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(bits);
    } else {
      const uint32_t b = max(bits & 0xFFFFu, bits >> 16);
      return unpack2(b, T{}).x;
    }
  }
  __device__ __forceinline__ float4 values() const {
    if constexpr (sizeof(T) == 4) {
      return make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
      const float2 a = unpack2(w[0], T{}), b = unpack2(w[1], T{});
      return make_float4(a.x, a.y, b.x, b.y);
    }
  }
};

// Block `blk` of sequence s, keys or values of head h.
template <typename T, int D>
__device__ __forceinline__ void append_block(const AppendArgs &a, int64_t rec, int s, int h, int which, int blk, int old, int len,
                                             int first, int lane) {
  constexpr int C = D / 8;   // 4-element chunks per lane: 16 * D / 4 chunks over 32 lanes
  constexpr int PT = D / 4;  // chunks per token
  const int p0 = blk * kKvBlock;
  const int held = old > p0 ? old - p0 : 0;                    // tokens the block held
  const int end = len - p0 < kKvBlock ? len - p0 : kKvBlock;  // tokens it holds now
  const T *x = static_cast<const T *>(which ? a.v : a.k) + int64_t(h) * D;
  const int64_t stride = which ? a.v_stride : a.k_stride;
  const int64_t x0 = int64_t(first) + p0 - old;  // row of the block's token 0 (negative part never read)

  // the new elements' loads first: they need no page
  // chunk i of this lane: token i / (D / 128) or (128 / D) i + lane / PT of the block
  constexpr bool kEven = 32 % PT == 0 || PT % 32 == 0;
  const T *x_lane = x + x0 * stride + (kEven && PT <= 32 ? (lane / PT) * stride + 4 * (lane % PT) : 4 * lane);
  Quad<T> q[C];
  if (kEven && held == 0 && end == kKvBlock) {  // a whole block
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if constexpr (PT <= 32)
        q[i].load(x_lane + (i * (32 / PT)) * stride);
      else
        q[i].load(x_lane + (i / (PT / 32)) * stride + 128 * (i % (PT / 32)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int ch = lane + 32 * i, t = ch / PT;
      q[i].clear();
      if (t >= held && t < end) q[i].load(x + (x0 + t) * stride + 4 * (ch % PT));
    }
  }
  const int64_t at = kv_record_of(a.c, s, blk, h, rec);
  if (at < 0) return;  // no page for these tokens: they are dropped
  const int t0 = p0 % a.c.page_tokens;
  int8_t *codes = reinterpret_cast<int8_t *>(a.c.pages + at) + (int64_t(which) * a.c.page_tokens + t0) * D;
  float *scale = reinterpret_cast<float *>(a.c.pages + at + int64_t(2) * a.c.page_tokens * D) +
                 which * (a.c.page_tokens / kKvBlock) + t0 / kKvBlock;
  const float s_old = held ? __uint_as_float(ld_u1(scale)) : 0.f;
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < C; ++i) bits = q[i].raise(bits);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) bits = Quad<T>::larger(bits, __shfl_xor_sync(0xffffffffu, bits, o));
  const float m = Quad<T>::magnitude(bits);
  float s_new = __fdiv_rn(m, 127.f);
  if (s_new < 1.17549435e-38f) s_new = 0.f;
  if (!(m < __int_as_float(0x7f800000))) s_new = __int_as_float(0x7fffffff);
  const float sc = max_abs_bits(s_old, s_new);  // NaN wins
  const float inv = sc > 0.f ? __frcp_rn(sc) : 0.f;
  if (held && sc != s_old) {  // a larger scale: what the block held, rounded to it
    const float again = sc > 0.f ? __fdiv_rn(s_old, sc) : 0.f;
#pragma unroll 4
    for (int i = 0; i < C; ++i) {
      const int ch = lane + 32 * i, t = ch / PT;
      if (t < held) {
        uint32_t *p = reinterpret_cast<uint32_t *>(codes + int64_t(t) * D + 4 * (ch % PT));
        const uint32_t w = ld_u1(p);
        uint32_t r = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          r |= uint32_t(__float2int_rn(float(int8_t(w >> (8 * j))) * again) & 0xFF) << (8 * j);
        *p = r;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int ch = lane + 32 * i, t = ch / PT;
    if (t >= held && t < end) {
      const float4 v = q[i].values();
      auto code = [&](float f) { return uint32_t(__float2int_rn(fminf(fmaxf(f * inv, -127.f), 127.f)) & 0xFF); };
      *reinterpret_cast<uint32_t *>(codes + int64_t(t) * D + 4 * (ch % PT)) =
          code(v.x) | (code(v.y) << 8) | (code(v.z) << 16) | (code(v.w) << 24);
    }
  }
  if (lane == 0 && (held == 0 || sc != s_old)) *scale = sc;
}

// (fewer registers for more warps: the loads' latency is what a block waits for)
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, D <= 128 ? (sizeof(T) == 2 ? 8 : 5) : 3) kv_append_kernel(const AppendArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int hw = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (hw >= 2 * a.c.n_kv) return;
  const int h = hw >> 1, which = hw & 1;
  const int64_t rec = kv_record_bytes(a.c.page_tokens, D);
  for (int s = blockIdx.z; s < a.n_seqs; s += gridDim.z)
    for (int b = blockIdx.y; b < a.n_blocks; b += gridDim.y) {
      const int first = a.cu ? int(ld_u1(a.cu + s)) : s;
      const int n_new = a.cu ? int(ld_u1(a.cu + s + 1)) - first : 1;
      const int all = int(ld_u1(a.kv_len + s)), old = all - n_new;
      if (n_new <= 0 || old < 0) break;
      const int len = n_new > a.max_new ? old + a.max_new : all;
      const int blk = old / kKvBlock + b, p0 = blk * kKvBlock;
      if (p0 >= len) break;
      append_block<T, D>(a, rec, s, h, which, blk, old, len, first, lane);
    }
}

struct ReadArgs {
  KvPool c;
  const int *start, *cu;  // first token of each sequence's range (NULL: 0); range sizes, summed
  void *k, *v;
  int64_t k_stride, v_stride;
  int n_seqs, n_blocks, max_tokens;
};

// One warp per (sequence, block, head, keys or values), as above; a token without a valid page
// reads as NaN.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) kv_read_kernel(const ReadArgs a) {
  constexpr int C = D / 8, PT = D / 4;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int hw = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (hw >= 2 * a.c.n_kv) return;
  const int h = hw >> 1, which = hw & 1;
  const int64_t rec = kv_record_bytes(a.c.page_tokens, D);
  T *o = static_cast<T *>(which ? a.v : a.k) + int64_t(h) * D;
  const int64_t stride = which ? a.v_stride : a.k_stride;
  for (int s = blockIdx.z; s < a.n_seqs; s += gridDim.z)
    for (int b = blockIdx.y; b < a.n_blocks; b += gridDim.y) {
      const int row0 = int(ld_u1(a.cu + s)), n = min(int(ld_u1(a.cu + s + 1)) - row0, a.max_tokens);
      const int start = a.start ? int(ld_u1(a.start + s)) : 0;
      if (n <= 0 || start < 0) break;
      const int blk = start / kKvBlock + b, p0 = blk * kKvBlock;
      if (int64_t(p0) >= int64_t(start) + n) break;
      const int64_t at = kv_record_of(a.c, s, blk, h, rec);
      const int t0 = p0 % a.c.page_tokens;
      const int64_t off = at < 0 ? 0 : at;
      const uint8_t *codes = a.c.pages + off + (int64_t(which) * a.c.page_tokens + t0) * D;
      const float *scale = reinterpret_cast<const float *>(a.c.pages + off + int64_t(2) * a.c.page_tokens * D) +
                           which * (a.c.page_tokens / kKvBlock) + t0 / kKvBlock;
      const float sc = at < 0 ? __int_as_float(0x7fffffff) : __uint_as_float(ld_u1(scale));
      uint32_t w[C];  // all of the block's codes in flight (any block of a page can be read whole)
#pragma unroll
      for (int i = 0; i < C; ++i) w[i] = ld_u1(codes + 4 * (lane + 32 * i));
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int ch = lane + 32 * i, t = ch / PT;
        const int64_t r = int64_t(p0) + t - start;
        if (r >= 0 && r < n)
          store4(o + (row0 + r) * stride + 4 * (ch % PT),
                 at < 0 ? make_float4(sc, sc, sc, sc)
                        : make_float4(float(int8_t(w[i])) * sc, float(int8_t(w[i] >> 8)) * sc, float(int8_t(w[i] >> 16)) * sc,
                                      float(int8_t(w[i] >> 24)) * sc));
      }
    }
}

struct KeepArgs {
  KvPool c;
  const int *kv_len, *cu, *path, *accepted;  // path: path_stride per sequence, of which accepted + 1 count
  int n_seqs, path_stride;
};

// The tokens of an accepted path, moved to the places behind the old ones.  One warp per (sequence, head, keys or
// values) goes over the blocks that change, in order: a token only moves to an earlier place, so
// a block's sources lie in it or behind it, where nothing has been written yet.  Block by block: lanes 0-15 find their
// tokens' sources and scales, then all codes are loaded before any is written.
// Measured: one path 3.7 us, 48 paths of up to 60 nodes, 8 heads of 128 6.1 us.  Bound: the chain of lengths, path, pages, scales,
// codes.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv_keep_kernel(const KeepArgs a) {
  constexpr int PT = D / 4, CPT = (PT + 31) / 32;  // words of a token, words per lane
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int hw = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (hw >= 2 * a.c.n_kv) return;
  const int h = hw >> 1, which = hw & 1;
  const int64_t rec = kv_record_bytes(a.c.page_tokens, D);
  const int64_t plane = int64_t(which) * a.c.page_tokens * D;
  const float qnan = __int_as_float(0x7fffffff);
  for (int s = blockIdx.y; s < a.n_seqs; s += gridDim.y) {
    const int n = int(ld_u1(a.cu + s + 1)) - int(ld_u1(a.cu + s)), len = int(ld_u1(a.kv_len + s));
    const int most = int(ld_u1(a.accepted + s));
    if (n <= 0 || len < n || most < 0) continue;
    const int old = len - n;
    const int m = min(min(most, a.path_stride - 1), n - 1) + 1;
    int last = -1;  // the node before this block's first
    for (int blk = old / kKvBlock; blk <= (old + m - 1) / kKvBlock; ++blk) {  // (a count of places would pass 32 bits near 2^31)
      const int p0 = blk * kKvBlock;
      // lane t (and t + 16): the block's token t
      const int t = lane & 15, i = p0 + t - old;
      const int node = i >= 0 && i < m ? int(ld_u1(a.path + int64_t(s) * a.path_stride + i)) : -1;
      int before = __shfl_up_sync(0xffffffffu, node, 1, 16);
      if (t == 0 || i == 0) before = last;
      // nodes in ever larger numbers: at the first that is not one the path ends
      const uint32_t wrong = __ballot_sync(0xffffffffu, i >= 0 && i < m && (node <= before || node >= n)) & 0xFFFFu;
      const int cut = wrong ? __ffs(wrong) - 1 : kKvBlock;
      const bool mine = i < m && t < cut;
      const int src = !mine ? p0 : i < 0 ? p0 + t : old + node;
      if (__any_sync(0xffffffffu, mine && src != p0 + t)) {
        const int64_t to = kv_record_of(a.c, s, blk, h, rec);
        const int64_t from = mine ? kv_record_of(a.c, s, src / kKvBlock, h, rec) : -1;
        const int sb = src % a.c.page_tokens;
        float sc = 0.f;
        if (mine)
          sc = from < 0 ? qnan  // a token without a page
                        : __uint_as_float(ld_u1(a.c.pages + from + int64_t(2) * a.c.page_tokens * D +
                                                4 * (which * (a.c.page_tokens / kKvBlock) + sb / kKvBlock)));
        float top = sc;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max_abs_bits(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float ratio = top > 0.f ? __fdiv_rn(sc, top) : 0.f;
        const int64_t off = (from < 0 ? 0 : from) + plane + int64_t(sb) * D;  // without a page: any valid place
        uint32_t w[kKvBlock][CPT];
#pragma unroll
        for (int j = 0; j < kKvBlock; ++j) {
          const int64_t at = __shfl_sync(0xffffffffu, (long long)off, j);
#pragma unroll
          for (int c = 0; c < CPT; ++c)
            if (lane + 32 * c < PT) w[j][c] = ld_u1(a.c.pages + at + 4 * (lane + 32 * c));
        }
        if (to >= 0) {
          uint8_t *codes = a.c.pages + to + plane + int64_t(p0 % a.c.page_tokens) * D;
#pragma unroll
          for (int j = 0; j < kKvBlock; ++j) {
            const float r = __shfl_sync(0xffffffffu, ratio, j);
            const bool moved = __shfl_sync(0xffffffffu, int(mine && (src != p0 + t || r != 1.f)), j);
            if (!moved) continue;
#pragma unroll
            for (int c = 0; c < CPT; ++c)
              if (lane + 32 * c < PT) {
                uint32_t v = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) v |= uint32_t(__float2int_rn(float(int8_t(w[j][c] >> (8 * e))) * r) & 0xFF) << (8 * e);
                *reinterpret_cast<uint32_t *>(codes + j * D + 4 * (lane + 32 * c)) = v;
              }
          }
          if (lane == 0)
            *reinterpret_cast<float *>(a.c.pages + to + int64_t(2) * a.c.page_tokens * D +
                                       4 * (which * (a.c.page_tokens / kKvBlock) + p0 % a.c.page_tokens / kKvBlock)) = top;
        }
      }
      if (wrong) break;
      last = __shfl_sync(0xffffffffu, node, 15);
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

// (keys and values of the heads, blocks, sequences); the kernels step over what exceeds the grid.
dim3 grid_of(const KvPool &c, int n_seqs, int n_blocks) {
  return dim3((2 * c.n_kv + kWarps - 1) / kWarps, n_blocks < 65535 ? n_blocks : 65535, n_seqs < 65535 ? n_seqs : 65535);
}

}  // namespace

int launch_kv_append(const KvPool &c, int head_dim, const int *kv_len, const int *cu, int n_seqs, int max_new,
                     const void *k, const void *v, int64_t k_stride, int64_t v_stride, int type, cudaStream_t s) {
  const AppendArgs a{c, kv_len, cu, k, v, k_stride, v_stride, n_seqs, kv_blocks_touched(max_new), max_new};
  const dim3 grid = grid_of(c, n_seqs, a.n_blocks);
  const cudaError_t e = cudaError_t(with_type(type, [&](auto t) {
    return with_dim(head_dim, [&](auto d) {
      return int(launch(kv_append_kernel<decltype(t), decltype(d)::value>, grid, dim3(kWarps * 32), 0, s, a));
    });
  }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

int launch_kv_read(const KvPool &c, int head_dim, const int *start, const int *cu, int n_seqs, int max_tokens, void *k,
                   void *v, int64_t k_stride, int64_t v_stride, int type, cudaStream_t s) {
  const ReadArgs a{c, start, cu, k, v, k_stride, v_stride, n_seqs, kv_blocks_touched(max_tokens), max_tokens};
  const dim3 grid = grid_of(c, n_seqs, a.n_blocks);
  const cudaError_t e = cudaError_t(with_type(type, [&](auto t) {
    return with_dim(head_dim, [&](auto d) {
      return int(launch(kv_read_kernel<decltype(t), decltype(d)::value>, grid, dim3(kWarps * 32), 0, s, a));
    });
  }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

int launch_kv_keep(const KvPool &c, int head_dim, const int *kv_len, const int *cu, int n_seqs, const int *path, int path_stride,
                   const int *accepted, cudaStream_t s) {
  const KeepArgs a{c, kv_len, cu, path, accepted, n_seqs, path_stride};
  const dim3 grid((2 * c.n_kv + kWarps - 1) / kWarps, n_seqs < 65535 ? n_seqs : 65535);
  const cudaError_t e = cudaError_t(
      with_dim(head_dim, [&](auto d) { return int(launch(kv_keep_kernel<decltype(d)::value>, grid, dim3(kWarps * 32), 0, s, a)); }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

}  // namespace qdq
