// Activation element types of the decode-step operators (QDQ_TYPE_* in qdq.h): coherent
// loads of consecutive elements as f32, stores with one rounding, the
// int8 cache's page geometry, and the operators' launchers.
#pragma once

#include <atomic>

#include <cuda_bf16.h>

#include "qdq_internal.cuh"

namespace qdq {

inline int type_bytes(int type) { return type == QDQ_TYPE_F32 ? 4 : 2; }
inline bool type_ok(int type) { return type == QDQ_TYPE_F32 || type == QDQ_TYPE_F16 || type == QDQ_TYPE_BF16; }

// Runs `f` with a value of the element type as its argument.
template <typename F>
inline int with_type(int type, F &&f) {
  switch (type) {
    case QDQ_TYPE_F32: return f(float{});
    case QDQ_TYPE_F16: return f(__half{});
    default: return f(__nv_bfloat16{});
  }
}

// Loads of data an earlier kernel wrote: volatile, so that they stay behind griddepcontrol.wait.
__device__ __forceinline__ uint4 ld_u4(const void *p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_u2(const void *p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_u1(const void *p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t ld_h1(const void *p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ float2 unpack2(uint32_t w, __half) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {  // bf16 is the high half of an f32
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float load1(const float *p) { return __uint_as_float(ld_u1(p)); }
__device__ __forceinline__ float load1(const __half *p) { return __half2float(__ushort_as_half(ld_h1(p))); }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) { return __uint_as_float(uint32_t(ld_h1(p)) << 16); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(__half *p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Four consecutive elements (16- or 8-byte aligned).
__device__ __forceinline__ float4 load4(const float *p) {
  const uint4 v = ld_u4(p);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
template <typename T>
__device__ __forceinline__ float4 load4(const T *p) {
  const uint2 v = ld_u2(p);
  const float2 a = unpack2(v.x, T{}), b = unpack2(v.y, T{});
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(v.x, v.y, T{}), pack2(v.z, v.w, T{}));
}

// Larger of two non-negative floats with a NaN counted as the largest (the order of their bits).
__device__ __forceinline__ float max_abs_bits(float a, float b) {
  const uint32_t x = __float_as_uint(a) & 0x7FFFFFFFu, y = __float_as_uint(b) & 0x7FFFFFFFu;
  return __uint_as_float(x > y ? x : y);
}

// ---- the int8 cache (layout in qdq.h) ---------------------------------------------
constexpr int kKvBlock = QDQ_KV_BLOCK;

__host__ __device__ __forceinline__ int64_t kv_record_bytes(int page_tokens, int head_dim) {
  return (int64_t(2) * page_tokens * head_dim + 8 * (page_tokens / kKvBlock) + 127) / 128 * 128;
}

struct KvPool {
  uint8_t *pages;
  const int *table;  // n_seqs rows of table_stride page ids
  int n_pages, page_tokens, n_kv, table_stride;
};

// Byte offset in the pool of head h's record of the page that holds block `blk` (16 tokens) of
// sequence s, or -1 when the table has no valid page for it.
__device__ __forceinline__ int64_t kv_record_of(const KvPool &c, int s, int blk, int h, int64_t rec) {
  const int pg = blk / (c.page_tokens / kKvBlock);
  if (pg >= c.table_stride) return -1;
  const int id = int(ld_u1(c.table + int64_t(s) * c.table_stride + pg));
  if (id < 0 || id >= c.n_pages) return -1;
  return (int64_t(id) * c.n_kv + h) * rec;
}

// Decode-step operators (qdq_norm.cu, qdq_kv.cu, qdq_kv_attn.cu, qdq_logprobs.cu); arguments as in qdq.h.
int launch_rms_norm(const void *x, const void *residual, const float *weight, void *sum_out, void *out, void *q8,
                    int type, int rows, int n, int64_t x_stride, int64_t residual_stride, int64_t sum_stride,
                    int64_t out_stride, float eps, cudaStream_t s);
int launch_kv_append(const KvPool &c, int head_dim, const int *kv_len, const int *cu, int n_seqs, int max_new,
                     const void *k, const void *v, int64_t k_stride, int64_t v_stride, int type, cudaStream_t s);
int launch_kv_read(const KvPool &c, int head_dim, const int *start, const int *cu, int n_seqs, int max_tokens, void *k,
                   void *v, int64_t k_stride, int64_t v_stride, int type, cudaStream_t s);
// A workspace holds the tickets (zero between calls) in its first eighth and the parts in the rest.  The
// border follows from the workspace's size alone, so that no call of another shape or operator on the
// same workspace writes where this one's tickets are.
inline size_t workspace_tickets(size_t bytes) { return bytes / 8 / 256 * 256; }
inline size_t workspace_for(size_t tickets, size_t part_bytes) {  // its bytes for that many 4-byte tickets
  const size_t t = (tickets * 4 + 255) / 256 * 2048, p = (part_bytes + 6) / 7 * 8;
  return ((t > p ? t : p) + 2047) / 2048 * 2048;
}
extern std::atomic<int> g_opt_attn_kernel;  // QDQ_OPT_ATTN_KERNEL
size_t kv_attention_workspace_bytes(int n_seqs, int max_q, int max_kv_len, int n_heads, int n_kv, int head_dim);
int launch_kv_attention(const KvPool &c, int head_dim, const int *kv_len, const int *cu_q, int n_seqs, int max_q,
                        int max_kv_len, int n_heads, const void *q, int64_t q_stride, void *out, int64_t out_stride,
                        float *lse, const float *slopes, float scale, float softcap, int window, int type,
                        void *workspace, size_t workspace_bytes, cudaStream_t s);
size_t token_logprobs_workspace_bytes(int rows, int n, int k);
int launch_token_logprobs(const void *logits, int64_t stride, int type, const int *tokens, int rows, int n, int k,
                          void *workspace, size_t workspace_bytes, float *logprob, float *entropy, int *top_index,
                          float *top_logprob, cudaStream_t s);

}  // namespace qdq
