// What the two attention kernels over the paged 8-bit cache share: the arguments, the blocks of a
// split, the codes' conversion and the outputs' stores.
#pragma once

#include <cuda_fp16.h>

#include "qdq_types.cuh"

namespace qdq {

constexpr float kLazy = 5.5f;    // accumulators are rescaled once a maximum has grown by 2^kLazy
constexpr float kPScale = 1024.f;  // probabilities become f16 at this scale: at most 2^15.5 (f16: below 2^16)
constexpr float kLog2PScale = 10.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinScale = 2.5243549e-29f;  // 2^-95: a smaller value scale counts as this in the reference

struct AttnArgs {
  KvPool c;
  const int *kv_len, *cu_q;
  const int *parent;  // of each query row in its sequence's tree (the tree kernels)
  const void *q;
  void *out;
  float *lse;
  const float *slopes;
  uint32_t *tickets;
  float *partial;
  int64_t q_stride, out_stride;
  int64_t room, units;  // floats of the workspace's parts, tickets that are used (read by the debug build's guards)
  int n_seqs, max_q, max_rows;  // max_rows: the rows of max_q queries of one cache head
  int max_kv_len, n_heads, group, tiles, splits, split_blocks, window, type;
  int entries;  // decode kernel: sequences times tiles where the splits' length is chosen on the device, else 0
  float scale, softcap, inv_cap, inv_splits;  // 1 / softcap, 1 / splits
  uint64_t group_mul;  // ceil(2^40 / group)
  // row / group, exact while row * group < 2^40 (rows are at most 2^30, the group of a row's heads below 2^10)
  __device__ __forceinline__ uint32_t query_of(int row) const { return uint32_t((uint64_t(uint32_t(row)) * group_mul) >> 40); }
};

// Bytes 0, 1 (lo) or 2, 3 (hi) of four excess-128 codes as two exact f16: the byte under the
// exponent of 1024, then 1024 + 128 taken off.
template <int SEL>
__device__ __forceinline__ uint32_t codes_f16(uint32_t u) {
  const uint32_t w = __byte_perm(u, 0x64646464u, SEL);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&w), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// 2^x, 0 for -inf (one instruction; a result below the normal numbers is 0)
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// tanh(x) = 1 - 2 / (1 + e^2x), off by 2^-21 at most; with kSmall (f32 activations) also to a few 1e-7
// relative near 0: below 1/4 the Taylor series (its next term is 1e-8 of the value there).  (tanhf took twice
// the instructions, a third of a capped call.)
template <bool kSmall>
__device__ __forceinline__ float tanh_of(float x) {
  const float e = ex2(x * (2.f * kLog2e));  // 0 or infinity at the ends: -1 and 1
  const float large = 1.f - __fdividef(2.f, 1.f + e);
  if constexpr (!kSmall) return large;
  const float t = x * x;
  const float small = x * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
  return fabsf(x) < 0.25f ? small : large;
}

// A block of the split.
struct BlockAt {
  int64_t k;  // byte offset of its first key code
  float ks, vs;
  float lv;   // log2 of the value scale, at least -95 (a block of zeros has scale 0)
  float inv;  // tensor-core kernel: 1 / vs, 0 where the scale is below 2^-95 or not finite
};

// Element of dim 0 of a row's output; four dims at element e, times inv, in the output's type.
template <int D>
__device__ __forceinline__ int64_t out_at(const AttnArgs &a, int q0, int h, int row) {
  const int qi = int(a.query_of(row));
  return int64_t(q0 + qi) * a.out_stride + int64_t(h * a.group + row - qi * a.group) * D;
}
__device__ __forceinline__ void store_at(const AttnArgs &a, int64_t e, float4 v, float inv) {
  v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  if (a.type == QDQ_TYPE_F32)
    store4(static_cast<float *>(a.out) + e, v);
  else if (a.type == QDQ_TYPE_F16)
    store4(static_cast<__half *>(a.out) + e, v);
  else
    store4(static_cast<__nv_bfloat16 *>(a.out) + e, v);
}
template <int D>
__device__ __forceinline__ void store_out(const AttnArgs &a, int q0, int h, int row, int d, float4 v, float inv) {
  store_at(a, out_at<D>(a, q0, h, row) + d, v, inv);
}
// M: the reference (log2 units), L: the sum of 2^(score - M)
__device__ __forceinline__ void store_lse(const AttnArgs &a, int q0, int h, int row, float M, float L) {
  const int qi = int(a.query_of(row));
  if (a.lse)
    a.lse[int64_t(q0 + qi) * a.n_heads + h * a.group + row - qi * a.group] =
        L == 0.f ? -__int_as_float(0x7f800000) : (M + log2f(L)) * 0.6931471805599453f;
}

// A sequence's tree of drafted tokens in shared memory: each node's depth, and itself and its ancestors as bits.  Node i is
// the i-th of the sequence's last tokens; its position is that of the first of them plus its depth.
template <bool TREE>
struct TreeNodes {  // no tree: nothing of it is called
  __device__ __forceinline__ int depth_of(int) const { return 0; }
  __device__ __forceinline__ bool wrong(int) const { return false; }
};
template <>
struct TreeNodes<true> {
  uint64_t seen[QDQ_MAX_TREE];
  int parent[QDQ_MAX_TREE], depth[QDQ_MAX_TREE];
  // threads 0, 1, ... (64 at least) of a block; a barrier between the two, and one behind them
  __device__ __forceinline__ void load(const int *p, int n, int tid) {
    if (tid < n) parent[tid] = int(ld_u1(p + tid));
  }
  __device__ __forceinline__ void walk(int n, int window, int tid) {
    if (tid >= n) {  // rows past the tree's last are computed, and share votes with its rows: the same ones in every call
      if (tid < QDQ_MAX_TREE) {
        seen[tid] = 0;
        depth[tid] = 0;
      }
      return;
    }
    uint64_t bits = 0;
    int steps = 0;
    for (int node = tid;;) {  // up to the root (to ever smaller numbers, so it ends)
      if (window <= 0 || steps < window) bits |= uint64_t(1) << node;
      const int up = parent[node];
      if (up == -1) break;
      if (up < 0 || up >= node) {  // no tree: the row is NaN
        steps = -1;
        break;
      }
      node = up;
      ++steps;
    }
    seen[tid] = bits;
    depth[tid] = steps;
  }
  // (rows and keys past 64: the last node's, they are hidden or not written)
  __device__ __forceinline__ int depth_of(int node) const { return depth[min(node, QDQ_MAX_TREE - 1)]; }
  __device__ __forceinline__ uint64_t seen_of(int node) const { return seen[min(node, QDQ_MAX_TREE - 1)]; }
  __device__ __forceinline__ bool wrong(int node) const { return depth_of(node) < 0; }
};
// Bit e: whether a row sees token at + e, e < 16: tokens from lo up to base, and of those from base on the ones in `seen`.
__device__ __forceinline__ uint32_t tree_sees(uint64_t seen, int base, int lo, int at) {
  const int old = min(max(base - at, 0), 16), skip = min(max(lo - at, 0), 16), off = at - base;
  const uint32_t cached = ((1u << old) - 1u) & ~((1u << skip) - 1u);
  const uint32_t drafted = off >= 0 ? (off < 64 ? uint32_t(seen >> off) : 0u) : (off > -16 ? uint32_t(seen) << -off : 0u);
  return (cached | drafted) & 0xFFFFu;
}

// The tensor-core kernel (qdq_kv_attn_tc.cu): one or two groups of 128 rows to a tile, head dims that are whole 64s
// (256 in two parts does not fit shared memory).
constexpr int kTcRows = 128;
// What a unit costs besides its tiles of 64 tokens, in tiles: a part costs 11 us, a tile 1.2 us, a join 8 us.  (4
// sequences of 300 queries over 300 to 2500 tokens, 32 / 8 heads of 128, f16: 9 75.2 us, 12 70.4, 15 70.2, 18 70.6; 48 trees of 22
// nodes behind 300 to 3000: 8 127, 11 121, 15 118, 20 123.)
constexpr int kTcPartCost = 15;
constexpr int kTcSplitBlocks = 256;  // blocks of 16 tokens in one part, at most
constexpr int kTcTreeBlocks = 768;  // ... of a tree's
inline bool attn_tc_supported(int head_dim, int parts) { return head_dim % 64 == 0 && head_dim * parts <= 384; }
// Bytes of one part's result (two per CTA).
inline size_t attn_tc_part_bytes(int head_dim, int groups) { return size_t(kTcRows) * groups * (head_dim + 2) * 4; }
// Launches a.splits CTAs, of which each has at most kTcSplitBlocks blocks; parts: f16 parts of the queries and
// probabilities; groups: of 128 rows to a tile (2 up to head_dim 128).
cudaError_t launch_attn_tc(const AttnArgs &a, int head_dim, int parts, int groups, cudaStream_t s);
int read_attn_tc_timeouts();

// The same two kernels for trees of drafted tokens (qdq_kv_tree.cu, qdq_kv_tree_tc.cu).
cudaError_t launch_attn_tree(const AttnArgs &a, int head_dim, int parts, int warps, int ctas, cudaStream_t s);
cudaError_t launch_attn_tree_tc(const AttnArgs &a, int head_dim, int parts, int groups, cudaStream_t s);
int read_attn_tree_tc_timeouts();

}  // namespace qdq
