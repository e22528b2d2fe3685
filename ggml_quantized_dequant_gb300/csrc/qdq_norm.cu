// Root-mean-square norm of activation rows, with the residual's addition in front and the
// result in the input's type, as a packed Q8_0 matrix, or both.
//
//   h = x + r,   y = h / sqrt(mean(h^2) + eps) * w
//   Q8_0: d = f16(max |y| / 127) over 32 consecutive y, code = rint(y * (1 / d)) within +-127
//
// Bound: memory (4 elements moved per element with residual and sum), for one row latency.  A row
// is read once into registers (8 to 32 elements per thread, all loads before the first use), its sum of
// squares is folded over the warps through shared memory in a fixed order, and every output is
// written from the registers: x and r are read once and each output written once, which is the floor.
// One CTA per row, or, for many wide or many short rows, CTAs that take row after row through a ring
// (the rule stands at the launch).  Sums are f32.
// Measured: one row of 3072 f32 1.8 us; 4096 rows of 8192 bf16 with residual 43 us (6.2 TB/s, 92 % of a
// plain copy's rate); 1500 rows of 3072 f32 with residual to f32 and Q8_0 14.7 us (5.3 TB/s, its inputs partly in L2), to Q8_0
// alone 12.8 us (4.7 TB/s: by their 41 registers three of the CTAs of 384 threads fit an SM, and 1500 rows are 3.3 rounds
// of them).  Rows that are not aligned go element by element (4096 rows of 8193 bf16 273 us, above 8192 elements with spills).
#include "qdq_types.cuh"

namespace qdq {
namespace {

struct NormArgs {
  const void *x, *residual;
  const float *weight;
  void *sum_out, *out;
  uint8_t *q8;
  int rows, n;
  int64_t x_stride, residual_stride, sum_stride, out_stride;
  float eps;
};

template <int V, typename T>
__device__ __forceinline__ void load_v(const T *p, float (&v)[V]) {
  if constexpr (V == 8) {
    const uint4 u = ld_u4(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2(w[i], T{});
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else if constexpr (V == 4) {
    const float4 f = load4(p);
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
  } else {
    v[0] = load1(p);
  }
}
// 16 bytes of shared memory as elements.
template <typename T, int V>
__device__ __forceinline__ void load_s(const T *p, float (&v)[V]) {
  const uint4 u = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (V == 8) {
      const float2 f = unpack2(w[i], T{});
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    } else {
      v[i] = __uint_as_float(w[i]);
    }
  }
}
template <int V, typename T>
__device__ __forceinline__ void store_v(T *p, const float (&v)[V]) {
  if constexpr (V == 8) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(v[0], v[1], T{}), pack2(v[2], v[3], T{}), pack2(v[4], v[5], T{}),
                                               pack2(v[6], v[7], T{}));
  } else if constexpr (V == 4) {
    store4(p, make_float4(v[0], v[1], v[2], v[3]));
  } else {
    store1(p, v[0]);
  }
}

template <int V>
__device__ __forceinline__ void load_weight(const float *p, float (&w)[V]) {
  if constexpr (V == 8) {
    const float4 w0 = __ldg(reinterpret_cast<const float4 *>(p)), w1 = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
    w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
  } else if constexpr (V == 4) {
    const float4 w0 = __ldg(reinterpret_cast<const float4 *>(p));
    w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
  } else {
    w[0] = __ldg(p);
  }
}

// V elements per load (16 or 8 bytes, or 1 element where the rows are not aligned), E elements
// per thread; element (i * blockDim + thread) * V + j of the row is the thread's i-th group.

// The row's norm and outputs from its elements in registers; weight(i, w) gives group i's weights.
template <typename T, int V, int E, typename W>
__device__ __forceinline__ void norm_row(const NormArgs &a, int row, const float (&h)[E / V][V], float *part, W &&weight) {
  constexpr int G = E / V;
  const int n = a.n;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) s = fmaf(h[i][j], h[i][j], s);
  s = warp_sum(s);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) part[warp] = s;
  __syncthreads();
  s = warp_sum(lane < int(blockDim.x >> 5) ? part[lane] : 0.f);
  const float inv = rsqrtf(s / float(n) + a.eps);
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int e = (i * int(blockDim.x) + int(threadIdx.x)) * V;
    const bool in = e < n;
    if (in && a.sum_out) store_v<V>(static_cast<T *>(a.sum_out) + row * a.sum_stride + e, h[i]);
    float y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = h[i][j] * inv;
    if (in && a.weight) {
      float w[V];
      weight(i, w);
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] *= w[j];
    }
    if (in && a.out) store_v<V>(static_cast<T *>(a.out) + row * a.out_stride + e, y);
    if (a.q8) {  // n % 32 == 0: a block of 32 lies in 32 / V neighbouring lanes, all in or all past the row
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) m = max_abs_bits(m, y[j]);
#pragma unroll
      for (int o = 16 / V; o > 0; o >>= 1) m = max_abs_bits(m, __shfl_xor_sync(0xffffffffu, m, o));
      const __half d = __float2half_rn(__fdiv_rn(m, 127.f));
      const float df = __half2float(d);
      const float id = df > 0.f ? __frcp_rn(df) : 0.f;
      if (in) {
        int8_t q[V];
#pragma unroll
        for (int j = 0; j < V; ++j) q[j] = int8_t(__float2int_rn(fminf(fmaxf(y[j] * id, -127.f), 127.f)));
        int8_t *qp = reinterpret_cast<int8_t *>(a.q8) + int64_t(row) * n + e;
        if constexpr (V == 8)
          *reinterpret_cast<uint2 *>(qp) = *reinterpret_cast<const uint2 *>(q);
        else if constexpr (V == 4)
          *reinterpret_cast<uint32_t *>(qp) = *reinterpret_cast<const uint32_t *>(q);
        else
          *qp = q[0];
        if ((e & 31) == 0)
          reinterpret_cast<__half *>(a.q8 + int64_t(a.rows) * n)[int64_t(row) * (n / 32) + e / 32] = d;
      }
    }
  }
}

// The next kernel on the stream may start early, unless a Q8_0 matrix is written: a projection reads its
// weights ahead of its wait.
__device__ __forceinline__ void start_next(const NormArgs &a) {
  // (a predicate: a branch here cost rows of single elements 5 % in spills)
  asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u64 p, %0, 0;\n\t@p griddepcontrol.launch_dependents;\n\t}" ::"l"(a.q8) : "memory");
}

template <typename T, int V, int E>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormArgs a) {
  constexpr int G = E / V;
  __shared__ float part[32];
  const int row = blockIdx.x, n = a.n;
  start_next(a);
  pdl_wait();
  const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
  const T *r = a.residual ? static_cast<const T *>(a.residual) + row * a.residual_stride : nullptr;
  float h[G][V];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int e = (i * int(blockDim.x) + int(threadIdx.x)) * V;
    if (e < n) {
      load_v<V>(x + e, h[i]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) h[i][j] = 0.f;
    }
  }
  if (r) {
    float b[G][V];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int e = (i * int(blockDim.x) + int(threadIdx.x)) * V;
      if (e < n) load_v<V>(r + e, b[i]);
    }
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int e = (i * int(blockDim.x) + int(threadIdx.x)) * V;
      if (e < n) {
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] += b[i][j];
      }
    }
  }
  if constexpr (E <= 16) {  // the weights' latency beside the sum's
    float w[G][V];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int e = (i * int(blockDim.x) + int(threadIdx.x)) * V;
      if (a.weight && e < n) load_weight<V>(a.weight + e, w[i]);
    }
    norm_row<T, V, E>(a, row, h, part, [&](int i, float (&v)[V]) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = w[i][j];
    });
  } else {  // no registers for them
    norm_row<T, V, E>(a, row, h, part, [&](int i, float (&w)[V]) {
      load_weight<V>(a.weight + (i * int(blockDim.x) + int(threadIdx.x)) * V, w);
    });
  }
}

// Many rows: as many CTAs as fit, each takes every gridDim-th row.  A thread copies its own elements of
// the next rows into shared memory (no barrier: it alone reads them) while a row is summed and written.
constexpr int kStages = 3;
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <typename T, int E>
__global__ void __launch_bounds__(1024) rms_norm_rows_kernel(const NormArgs a) {
  constexpr int V = 16 / sizeof(T), G = E / V;
  extern __shared__ uint8_t ring[];
  __shared__ float part[2][32];
  const int n = a.n, tid = threadIdx.x, threads = blockDim.x;
  start_next(a);
  pdl_wait();
  const uint32_t mine = smem_u32(ring) + 16 * tid, group = 16 * threads, slot = (a.residual ? 2 : 1) * G * group;
  auto fetch = [&](int64_t row, int st) {
    if (row < a.rows) {
      const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
      const T *r = static_cast<const T *>(a.residual) + row * a.residual_stride;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int e = (i * threads + tid) * V;
        if (e < n) {
          copy16(mine + st * slot + i * group, x + e);
          if (a.residual) copy16(mine + st * slot + (G + i) * group, r + e);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float w[G][V];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int e = (i * threads + tid) * V;
    if (a.weight && e < n) load_weight<V>(a.weight + e, w[i]);
  }
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(blockIdx.x + int64_t(i) * gridDim.x, i);
  int st = 0, k = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, k ^= 1) {
    fetch(row + int64_t(kStages - 1) * gridDim.x, st == 0 ? kStages - 1 : st - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    float h[G][V];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const uint8_t *at = ring + 16 * tid + st * slot + i * group;
      const bool in = (i * threads + tid) * V < n;
      if (in) {
        load_s(reinterpret_cast<const T *>(at), h[i]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] = 0.f;
      }
      if (in && a.residual) {
        float b[V];
        load_s(reinterpret_cast<const T *>(at + G * group), b);
#pragma unroll
        for (int j = 0; j < V; ++j) h[i][j] += b[j];
      }
    }
    norm_row<T, V, E>(a, int(row), h, part[k], [&](int i, float (&v)[V]) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = w[i][j];
    });
    if (++st == kStages) st = 0;
  }
}

template <typename T, int E>
cudaError_t run_rows(const NormArgs &a, int ctas, int threads, cudaStream_t s) {
  const auto kernel = rms_norm_rows_kernel<T, E>;
  const int bytes = kStages * (a.residual ? 2 : 1) * E * int(sizeof(T)) * threads;
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), bytes);
  return e != cudaSuccess ? e : launch(kernel, dim3(ctas), dim3(threads), bytes, s, a);
}

template <typename T, int V, int E>
cudaError_t run_norm(const NormArgs &a, cudaStream_t s) {
  const int groups = (a.n + V - 1) / V, per = E / V;
  const int threads = ((groups + per - 1) / per + 31) / 32 * 32;
  return launch(rms_norm_kernel<T, V, E>, dim3(a.rows), dim3(threads), 0, s, a);
}

}  // namespace

int launch_rms_norm(const void *x, const void *residual, const float *weight, void *sum_out, void *out, void *q8,
                    int type, int rows, int n, int64_t x_stride, int64_t residual_stride, int64_t sum_stride,
                    int64_t out_stride, float eps, cudaStream_t s) {
  const NormArgs a{x, residual, weight, sum_out, out, static_cast<uint8_t *>(q8), rows, n, x_stride, residual_stride,
                   sum_stride, out_stride, eps};
  const int eb = type_bytes(type);
  DeviceInfo di;
  const cudaError_t de = device_info(&di);
  if (de != cudaSuccess) return fail_cuda(de);
  // vector loads where every row of every operand starts on a vector boundary
  auto fits = [&](int v) {
    const uintptr_t b = uintptr_t(v) * eb;
    auto ok = [&](const void *p, int64_t st) {
      return !p || (reinterpret_cast<uintptr_t>(p) % b == 0 && (rows == 1 || (st * eb) % int64_t(b) == 0));
    };
    return n % v == 0 && ok(x, x_stride) && ok(residual, residual_stride) && ok(sum_out, sum_stride) &&
           ok(out, out_stride) && (!weight || reinterpret_cast<uintptr_t>(weight) % 16 == 0);
  };
  const cudaError_t e = cudaError_t(with_type(type, [&](auto t) {
    using T = decltype(t);
    auto pick = [&](auto v) {
      constexpr int V = decltype(v)::value;
      // the fewest elements per thread that a CTA can hold: at 4096 rows of 8192 (bf16, residual, a CTA
      // each) 8, 16 and 32 per thread took 47.4, 52.8 and 55.2 us, one row of 3072 1.9, 2.1 and 3.6 us
      if constexpr (V * sizeof(T) == 16) {
        // Rows through a ring where by their threads only two CTAs of one row each fit an SM (they wait on barriers and
        // memory by turns; 4096 rows of 8192 bf16 with residual 47.2 -> 43.0 us, f32 without 48.2 -> 42.9 us; of the
        // ring's CTAs of 1024 threads at 50 to 57 registers one is on an SM at a time, so they come in two rounds) and
        // shared memory has room for two as well (f32 with residual: one, 78 -> 89 us), or where a row is
        // moved in less time than a CTA is started (60000 rows of 256 bf16: 60.6 -> 21.3 us, 30000 of 512
        // 30.6 -> 20.1 us).  Between, small CTAs hide each other's barriers (8192 rows of 4096 bf16: 41.4, ring 44.0 us).
        const int threads = ((n + 7) / 8 + 31) / 32 * 32, fit = 2048 / threads;
        if (n <= 8192 && (fit <= 2 || n * eb <= 1536)) {
          const int smem = kStages * (residual ? 2 : 1) * 8 * eb * threads, room = 220 * 1024 / (smem + 1280);
          const int most = fit < 32 ? fit : 32, ctas = di.sm_count * (most < room ? most : room);
          if (room >= 2 && rows > 2 * ctas) return run_rows<T, 8>(a, ctas, threads, s);
        }
      }
      if (n <= 8192) return run_norm<T, V, 8>(a, s);
      if (n <= 16384) return run_norm<T, V, 16>(a, s);
      return run_norm<T, V, 32>(a, s);
    };
    if constexpr (sizeof(T) == 2) {
      if (fits(8)) return int(pick(std::integral_constant<int, 8>{}));
    }
    if (fits(4)) return int(pick(std::integral_constant<int, 4>{}));
    return int(pick(std::integral_constant<int, 1>{}));
  }));
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

}  // namespace qdq
