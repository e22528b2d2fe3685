// C-ABI boundary of the qdq library: argument validation, status codes and
// dispatch to the kernel launchers.  Nothing here touches tensor data; every
// arithmetic step runs in the CUDA kernels.
#include <atomic>
#include <mutex>
#include <vector>

#include "qdq_internal.cuh"
#include "qdq_types.cuh"

namespace qdq {

// Argmax over each of `batch` rows of n floats (csrc/qdq_argmax.cu).
int launch_argmax_rows(const float *logits, int n, int batch, int *index, float *value, cudaStream_t s);

namespace {
__global__ void noop_kernel() {}

thread_local int g_last_cuda_error = 0;
std::atomic<int> g_opt_pdl{1};
std::atomic<int> g_opt_l2_prefetch{0};
std::atomic<int> g_opt_ctas_per_sm{0};
std::atomic<int> g_opt_xs_groups{0};
std::atomic<int> g_opt_xs_stages{0};
std::atomic<int> g_opt_xs_float_x{1};
std::atomic<int> g_opt_batch1_kernel{0};

constexpr int kMaxDevices = 64;
std::once_flag g_dev_once[kMaxDevices];
DeviceInfo g_dev_info[kMaxDevices];
cudaError_t g_dev_err[kMaxDevices];

std::mutex g_smem_mu;
struct SmemEntry {
  const void *func;
  int device;
  int bytes;
};
std::vector<SmemEntry> g_smem;
}  // namespace

int opt_pdl() { return g_opt_pdl.load(std::memory_order_relaxed); }
int opt_l2_prefetch() { return g_opt_l2_prefetch.load(std::memory_order_relaxed); }
int opt_ctas_per_sm() { return g_opt_ctas_per_sm.load(std::memory_order_relaxed); }
int opt_xs_groups() { return g_opt_xs_groups.load(std::memory_order_relaxed); }
int opt_xs_stages() { return g_opt_xs_stages.load(std::memory_order_relaxed); }
int opt_xs_float_x() { return g_opt_xs_float_x.load(std::memory_order_relaxed); }
int opt_batch1_kernel() { return g_opt_batch1_kernel.load(std::memory_order_relaxed); }

int fail_cuda(cudaError_t e) {
  g_last_cuda_error = int(e);
  return QDQ_ERR_CUDA;
}

cudaError_t device_info(DeviceInfo *out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(g_dev_once[dev], [dev]() {
    DeviceInfo di{};
    cudaError_t err = cudaDeviceGetAttribute(&di.sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (err == cudaSuccess)
      err = cudaDeviceGetAttribute(&di.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (err == cudaSuccess)
      err = cudaDeviceGetAttribute(&di.smem_per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
    if (err == cudaSuccess)
      err = cudaDeviceGetAttribute(&di.reserved_smem_per_block, cudaDevAttrReservedSharedMemoryPerBlock, dev);
    if (err == cudaSuccess)
      err = cudaDeviceGetAttribute(&di.regs_per_sm, cudaDevAttrMaxRegistersPerMultiprocessor, dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&di.l2_bytes, cudaDevAttrL2CacheSize, dev);
    g_dev_info[dev] = di;
    g_dev_err[dev] = err;
  });
  *out = g_dev_info[dev];
  return g_dev_err[dev];
}

size_t gemv_smem_bytes(const DeviceInfo &di, size_t need) {
  if (!opt_pdl()) return need;
  const int per_sm = ctas_per_sm_or(1) + 1;  // this kernel's CTAs + one of the next kernel
  long cap = long(di.smem_per_sm) / per_sm - di.reserved_smem_per_block;
  if (cap > di.max_smem_optin) cap = di.max_smem_optin;
  return size_t(cap) > need ? size_t(cap) : need;
}

cudaError_t allow_dynamic_smem(const void *func, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_smem_mu);
  for (SmemEntry &s : g_smem) {
    if (s.func == func && s.device == dev) {
      if (s.bytes >= bytes) return cudaSuccess;
      e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (e == cudaSuccess) s.bytes = bytes;
      return e;
    }
  }
  e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  // the largest shared-memory carve-out, so that a CTA of the next kernel fits beside one of this kernel
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(func, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess) g_smem.push_back({func, dev, bytes});
  return e;
}

namespace {
bool dims_q4k_(int n_out, int n_in) { return n_out > 0 && n_in > 0 && (n_in % 256) == 0; }
size_t q4k_bytes_(int n_out, int n_in) { return size_t(n_out) * size_t(n_in / 256) * 144; }
}  // namespace

int check_ffn_residual(const void *Wg, const void *Wu, const void *Wd, const float *x, const float *residual,
                       const float *out, const float *mid, int n_embd, int n_ff, int batch) {
  if (!Wg || !Wu || !Wd || !x || !residual || !out) return QDQ_ERR_NULL;
  if (!dims_q4k_(n_ff, n_embd) || !dims_q4k_(n_embd, n_ff)) return QDQ_ERR_DIMS;
  if (batch < 1 || batch > QDQ_MAX_GEMV_BATCH) return QDQ_ERR_DIMS;
  if (n_embd > QDQ_MAX_GEMV_N_IN || n_ff > QDQ_MAX_GEMV_N_IN) return QDQ_ERR_UNSUPPORTED;
  if (!aligned(Wg, 16) || !aligned(Wu, 16) || !aligned(Wd, 16) || !aligned(x, 16) || !aligned(residual, 4) ||
      !aligned(out, 4) || (mid && !aligned(mid, 16)))
    return QDQ_ERR_ALIGN;
  const size_t wgb = q4k_bytes_(n_ff, n_embd), wdb = q4k_bytes_(n_embd, n_ff);
  const size_t eb = size_t(batch) * n_embd * 4, fb = size_t(batch) * n_ff * 4;
  // mid may overlap nothing; out may only coincide exactly with residual
  if (mid && (overlaps(mid, fb, Wg, wgb) || overlaps(mid, fb, Wu, wgb) || overlaps(mid, fb, Wd, wdb) ||
              overlaps(mid, fb, x, eb) || overlaps(mid, fb, residual, eb) || overlaps(mid, fb, out, eb)))
    return QDQ_ERR_ALIAS;
  if (overlaps(out, eb, Wg, wgb) || overlaps(out, eb, Wu, wgb) || overlaps(out, eb, Wd, wdb) ||
      overlaps(out, eb, x, eb))
    return QDQ_ERR_ALIAS;
  if (out != residual && overlaps(out, eb, residual, eb)) return QDQ_ERR_ALIAS;
  return QDQ_OK;
}

}  // namespace qdq

using namespace qdq;

namespace {

bool dims_q8(int n_out, int n_in) { return n_out > 0 && n_in > 0 && (n_in % 32) == 0; }
bool dims_q4k(int n_out, int n_in) { return n_out > 0 && n_in > 0 && (n_in % 256) == 0; }

size_t q8_bytes(int n_out, int n_in) { return size_t(n_out) * size_t(n_in / 32) * 34; }
size_t q4k_bytes(int n_out, int n_in) { return size_t(n_out) * size_t(n_in / 256) * 144; }
size_t q6k_ggml_bytes(int n_out, int n_in) { return size_t(n_out) * size_t(n_in / 256) * 210; }
size_t q6k_bytes(int n_out, int n_in) { return size_t(n_out) * size_t(q6k_row_bytes(n_in)); }

// Arguments of a top-k over `batch` rows of n logits (qdq_topk_rows).
int check_topk(const float *logits, int n, int batch, int k, const void *ws, const int *index, const float *value) {
  if (!logits || !ws || !index || !value) return QDQ_ERR_NULL;
  if (n < 1 || batch < 1 || k < 1 || k > n) return QDQ_ERR_DIMS;
  if (k > QDQ_MAX_TOPK) return QDQ_ERR_UNSUPPORTED;
  if (!aligned(logits, 4) || !aligned(ws, 16) || !aligned(index, 4) || !aligned(value, 4)) return QDQ_ERR_ALIGN;
  const size_t lb = size_t(batch) * n * 4, wb = topk_workspace_bytes(n, batch, k), rb = size_t(batch) * k * 4;
  if (overlaps(ws, wb, logits, lb) || overlaps(index, rb, logits, lb) || overlaps(value, rb, logits, lb) ||
      overlaps(index, rb, ws, wb) || overlaps(value, rb, ws, wb) || overlaps(index, rb, value, rb))
    return QDQ_ERR_ALIAS;
  return QDQ_OK;
}

int check_gemv_common(const void *W, const float *x, const float *y, int n_out, int n_in, int batch,
                      size_t w_bytes) {
  if (!W || !x || !y) return QDQ_ERR_NULL;
  if (batch < 1 || batch > QDQ_MAX_GEMV_BATCH) return QDQ_ERR_DIMS;
  if (n_in > QDQ_MAX_GEMV_N_IN) return QDQ_ERR_UNSUPPORTED;
  if (!aligned(W, 16) || !aligned(x, 16) || !aligned(y, 4)) return QDQ_ERR_ALIGN;
  const size_t yb = size_t(batch) * n_out * 4, xb = size_t(batch) * n_in * 4;
  if (overlaps(y, yb, W, w_bytes) || overlaps(y, yb, x, xb)) return QDQ_ERR_ALIAS;
  return QDQ_OK;
}

}  // namespace

extern "C" {

const char *qdq_status_string(int status) {
  switch (status) {
    case QDQ_OK: return "QDQ_OK";
    case QDQ_ERR_NULL: return "QDQ_ERR_NULL: a required pointer is NULL";
    case QDQ_ERR_DIMS: return "QDQ_ERR_DIMS: bad dimension";
    case QDQ_ERR_ALIGN: return "QDQ_ERR_ALIGN: pointer misaligned";
    case QDQ_ERR_UNSUPPORTED: return "QDQ_ERR_UNSUPPORTED: shape not handled by this build";
    case QDQ_ERR_CUDA: return "QDQ_ERR_CUDA: CUDA runtime error (see qdq_last_cuda_error)";
    case QDQ_ERR_ALIAS: return "QDQ_ERR_ALIAS: output overlaps an input";
    case QDQ_ERR_SCRATCH: return "QDQ_ERR_SCRATCH: request exceeds the fixed scratch array (batch * n_ff) or the given workspace";
    default: return "unknown qdq status";
  }
}

int qdq_last_cuda_error(void) { return g_last_cuda_error; }

const char *qdq_version(void) { return "qdq 0.1 sm_103a"; }

int qdq_set_option(int key, int value) {
  switch (key) {
    case QDQ_OPT_PDL:
      if (value != 0 && value != 1) return QDQ_ERR_DIMS;
      return g_opt_pdl.exchange(value);
    case QDQ_OPT_L2_PREFETCH:
      if (value < 0 || value > 3) return QDQ_ERR_DIMS;
      return g_opt_l2_prefetch.exchange(value);
    case QDQ_OPT_CTAS_PER_SM:
      if (value < 0 || value > 4) return QDQ_ERR_DIMS;
      return g_opt_ctas_per_sm.exchange(value);
    case QDQ_OPT_XS_GROUPS:
      if (value < 0 || value > 16) return QDQ_ERR_DIMS;
      return g_opt_xs_groups.exchange(value);
    case QDQ_OPT_XS_STAGES:
      if (value < 0 || value > 16) return QDQ_ERR_DIMS;
      return g_opt_xs_stages.exchange(value);
    case QDQ_OPT_XS_FLOAT_X:
      if (value != 0 && value != 1) return QDQ_ERR_DIMS;
      return g_opt_xs_float_x.exchange(value);
    case QDQ_OPT_BATCH1_KERNEL:
      if (value != 0 && value != 1) return QDQ_ERR_DIMS;
      return g_opt_batch1_kernel.exchange(value);
    case QDQ_OPT_ATTN_KERNEL:
      if (value < 0 || value > 2) return QDQ_ERR_DIMS;
      return qdq::g_opt_attn_kernel.exchange(value);
    default: return QDQ_ERR_DIMS;
  }
}

size_t qdq_q8_0_packed_bytes(int n_out, int n_in) { return dims_q8(n_out, n_in) ? q8_bytes(n_out, n_in) : 0; }
size_t qdq_q4k_packed_bytes(int n_out, int n_in) { return dims_q4k(n_out, n_in) ? q4k_bytes(n_out, n_in) : 0; }

int qdq_q8_0_pack(const void *ggml, void *packed, int n_out, int n_in, cudaStream_t stream) {
  if (!ggml || !packed) return QDQ_ERR_NULL;
  if (!dims_q8(n_out, n_in)) return QDQ_ERR_DIMS;
  if (!aligned(packed, 16)) return QDQ_ERR_ALIGN;
  const size_t n = q8_bytes(n_out, n_in);
  if (overlaps(ggml, n, packed, n)) return QDQ_ERR_ALIAS;
  return launch_q8_0_pack(ggml, packed, n_out, n_in, stream);
}

int qdq_q4k_pack(const void *ggml, void *packed, int n_out, int n_in, cudaStream_t stream) {
  if (!ggml || !packed) return QDQ_ERR_NULL;
  if (!dims_q4k(n_out, n_in)) return QDQ_ERR_DIMS;
  if (!aligned(packed, 16)) return QDQ_ERR_ALIGN;
  const size_t n = q4k_bytes(n_out, n_in);
  if (overlaps(ggml, n, packed, n)) return QDQ_ERR_ALIAS;
  return launch_q4k_pack(ggml, packed, n_out, n_in, stream);
}

int qdq_q8_0_dequant(const void *W, float *out, int n_out, int n_in, cudaStream_t stream) {
  if (!W || !out) return QDQ_ERR_NULL;
  if (!dims_q8(n_out, n_in)) return QDQ_ERR_DIMS;
  if (!aligned(W, 16) || !aligned(out, 4)) return QDQ_ERR_ALIGN;
  if (overlaps(out, size_t(n_out) * n_in * 4, W, q8_bytes(n_out, n_in))) return QDQ_ERR_ALIAS;
  return launch_q8_0_dequant(W, out, n_out, n_in, stream);
}

int qdq_q4k_dequant(const void *W, float *out, int n_out, int n_in, cudaStream_t stream) {
  if (!W || !out) return QDQ_ERR_NULL;
  if (!dims_q4k(n_out, n_in)) return QDQ_ERR_DIMS;
  if (!aligned(W, 16) || !aligned(out, 4)) return QDQ_ERR_ALIGN;
  if (overlaps(out, size_t(n_out) * n_in * 4, W, q4k_bytes(n_out, n_in))) return QDQ_ERR_ALIAS;
  return launch_q4k_dequant(W, out, n_out, n_in, stream);
}

int qdq_q8_0_gemv(const void *W, const float *x, float *y, int n_out, int n_in, int batch,
                  cudaStream_t stream) {
  if (!dims_q8(n_out, n_in)) return (!W || !x || !y) ? QDQ_ERR_NULL : QDQ_ERR_DIMS;
  const int rc = check_gemv_common(W, x, y, n_out, n_in, batch, q8_bytes(n_out, n_in));
  if (rc != QDQ_OK) return rc;
  return launch_q8_0_gemv(W, x, y, n_out, n_in, batch, stream);
}

int qdq_q4k_gemv(const void *W, const float *x, float *y, int n_out, int n_in, int batch,
                 cudaStream_t stream) {
  if (!dims_q4k(n_out, n_in)) return (!W || !x || !y) ? QDQ_ERR_NULL : QDQ_ERR_DIMS;
  const int rc = check_gemv_common(W, x, y, n_out, n_in, batch, q4k_bytes(n_out, n_in));
  if (rc != QDQ_OK) return rc;
  return launch_q4k_gemv(0, W, nullptr, x, nullptr, y, n_out, n_in, batch, stream);
}

int qdq_q4k_swiglu(const void *Wg, const void *Wu, const float *x, float *mid, int n_ff, int n_embd,
                   int batch, cudaStream_t stream) {
  if (!Wg || !Wu || !x || !mid) return QDQ_ERR_NULL;
  if (!dims_q4k(n_ff, n_embd)) return QDQ_ERR_DIMS;
  int rc = check_gemv_common(Wg, x, mid, n_ff, n_embd, batch, q4k_bytes(n_ff, n_embd));
  if (rc != QDQ_OK) return rc;
  if (!aligned(Wu, 16)) return QDQ_ERR_ALIGN;
  if (overlaps(mid, size_t(batch) * n_ff * 4, Wu, q4k_bytes(n_ff, n_embd))) return QDQ_ERR_ALIAS;
  return launch_q4k_gemv(1, Wg, Wu, x, nullptr, mid, n_ff, n_embd, batch, stream);
}

int qdq_q4k_ffn_residual(const void *Wg, const void *Wu, const void *Wd, const float *x,
                         const float *residual, float *out, float *mid, int n_embd, int n_ff, int batch,
                         cudaStream_t stream) {
  if (!mid) return QDQ_ERR_NULL;
  int rc = check_ffn_residual(Wg, Wu, Wd, x, residual, out, mid, n_embd, n_ff, batch);
  if (rc != QDQ_OK) return rc;
  rc = launch_q4k_gemv(1, Wg, Wu, x, nullptr, mid, n_ff, n_embd, batch, stream);
  if (rc != QDQ_OK) return rc;
  return launch_q4k_gemv(2, Wd, nullptr, mid, residual, out, n_embd, n_ff, batch, stream);
}

int qdq_q8_0_logits_argmax(const void *W, const float *x, float *logits, int *index, float *value, int n_vocab,
                           int n_in, int batch, cudaStream_t stream) {
  if (!W || !x || !logits || !index || !value) return QDQ_ERR_NULL;
  if (!dims_q8(n_vocab, n_in)) return QDQ_ERR_DIMS;
  const int rc = check_gemv_common(W, x, logits, n_vocab, n_in, batch, q8_bytes(n_vocab, n_in));
  if (rc != QDQ_OK) return rc;
  if (!aligned(index, 4) || !aligned(value, 4)) return QDQ_ERR_ALIGN;
  const size_t lb = size_t(batch) * n_vocab * 4, rb = size_t(batch) * 4;
  const void *others[3] = {W, x, logits};
  const size_t ob[3] = {q8_bytes(n_vocab, n_in), size_t(batch) * n_in * 4, lb};
  for (int i = 0; i < 3; ++i)
    if (overlaps(index, rb, others[i], ob[i]) || overlaps(value, rb, others[i], ob[i])) return QDQ_ERR_ALIAS;
  if (overlaps(index, rb, value, rb)) return QDQ_ERR_ALIAS;
  const int r = launch_q8_0_gemv(W, x, logits, n_vocab, n_in, batch, stream);
  if (r != QDQ_OK) return r;
  return launch_argmax_rows(logits, n_vocab, batch, index, value, stream);
}

size_t qdq_q6k_packed_bytes(int n_out, int n_in) { return dims_q4k(n_out, n_in) ? q6k_bytes(n_out, n_in) : 0; }

int qdq_q6k_pack(const void *ggml, void *packed, int n_out, int n_in, cudaStream_t stream) {
  if (!ggml || !packed) return QDQ_ERR_NULL;
  if (!dims_q4k(n_out, n_in)) return QDQ_ERR_DIMS;
  if (!aligned(packed, 16)) return QDQ_ERR_ALIGN;
  if (overlaps(ggml, q6k_ggml_bytes(n_out, n_in), packed, q6k_bytes(n_out, n_in))) return QDQ_ERR_ALIAS;
  return launch_q6k_pack(ggml, packed, n_out, n_in, stream);
}

int qdq_q6k_dequant(const void *W, float *out, int n_out, int n_in, cudaStream_t stream) {
  if (!W || !out) return QDQ_ERR_NULL;
  if (!dims_q4k(n_out, n_in)) return QDQ_ERR_DIMS;
  if (!aligned(W, 16) || !aligned(out, 4)) return QDQ_ERR_ALIGN;
  if (overlaps(out, size_t(n_out) * n_in * 4, W, q6k_bytes(n_out, n_in))) return QDQ_ERR_ALIAS;
  return launch_q6k_dequant(W, out, n_out, n_in, stream);
}

int qdq_q6k_gemv(const void *W, const float *x, float *y, int n_out, int n_in, int batch, cudaStream_t stream) {
  if (!dims_q4k(n_out, n_in)) return (!W || !x || !y) ? QDQ_ERR_NULL : QDQ_ERR_DIMS;
  const int rc = check_gemv_common(W, x, y, n_out, n_in, batch, q6k_bytes(n_out, n_in));
  if (rc != QDQ_OK) return rc;
  return launch_q6k_gemv(W, x, y, n_out, n_in, batch, stream);
}

int qdq_q6k_get_rows(const void *W, const int *ids, float *out, int n_ids, int n_rows, int n_in, cudaStream_t stream) {
  if (!W || !ids || !out) return QDQ_ERR_NULL;
  if (n_ids < 0 || !dims_q4k(n_rows, n_in)) return QDQ_ERR_DIMS;
  if (!aligned(W, 16) || !aligned(ids, 4) || !aligned(out, 4)) return QDQ_ERR_ALIGN;
  const size_t ob = size_t(n_ids) * n_in * 4;
  if (overlaps(out, ob, W, q6k_bytes(n_rows, n_in)) || overlaps(out, ob, ids, size_t(n_ids) * 4)) return QDQ_ERR_ALIAS;
  if (n_ids == 0) return QDQ_OK;  // nothing to look up
  return launch_q6k_get_rows(W, ids, out, n_ids, n_rows, n_in, stream);
}

size_t qdq_topk_workspace_bytes(int n, int batch, int k) {
  if (n < 1 || batch < 1 || k < 1 || k > n || k > QDQ_MAX_TOPK) return 0;
  return topk_workspace_bytes(n, batch, k);
}

int qdq_topk_rows(const float *logits, int n, int batch, int k, void *workspace, int *index, float *value,
                  cudaStream_t stream) {
  const int rc = check_topk(logits, n, batch, k, workspace, index, value);
  if (rc != QDQ_OK) return rc;
  // k = 1 is the argmax (the same order: NaN first, then larger, then smaller index)
  if (k == 1) return launch_argmax_rows(logits, n, batch, index, value, stream);
  return launch_topk_rows(logits, n, batch, k, workspace, index, value, stream);
}

int qdq_q8_0_logits_topk(const void *W, const float *x, float *logits, void *workspace, int *index, float *value,
                         int n_vocab, int n_in, int batch, int k, cudaStream_t stream) {
  if (!W || !x || !logits || !workspace || !index || !value) return QDQ_ERR_NULL;
  if (!dims_q8(n_vocab, n_in)) return QDQ_ERR_DIMS;
  int rc = check_gemv_common(W, x, logits, n_vocab, n_in, batch, q8_bytes(n_vocab, n_in));
  if (rc != QDQ_OK) return rc;
  rc = check_topk(logits, n_vocab, batch, k, workspace, index, value);
  if (rc != QDQ_OK) return rc;
  const size_t wb = q8_bytes(n_vocab, n_in), xb = size_t(batch) * n_in * 4, rb = size_t(batch) * k * 4;
  const size_t sb = topk_workspace_bytes(n_vocab, batch, k);
  if (overlaps(workspace, sb, W, wb) || overlaps(workspace, sb, x, xb) || overlaps(index, rb, W, wb) ||
      overlaps(index, rb, x, xb) || overlaps(value, rb, W, wb) || overlaps(value, rb, x, xb))
    return QDQ_ERR_ALIAS;
  if (k == 1) {  // the argmax epilogue (the same order)
    rc = launch_q8_0_gemv(W, x, logits, n_vocab, n_in, batch, stream);
    if (rc != QDQ_OK) return rc;
    return launch_argmax_rows(logits, n_vocab, batch, index, value, stream);
  }
  if (batch == 1 && gemv_xs_supported(n_in, 1, 0) && opt_batch1_kernel() == 0 && opt_xs_float_x()) {
    // batch 1: the projection's CTAs write their rows' k best keys as they finish, so the
    // logits are not read back for the first selection; then the merge rounds
    int n_cand = 0;
    rc = launch_gemv_dl_topk(W, x, logits, n_vocab, n_in, static_cast<uint64_t *>(workspace), k, &n_cand, stream);
    if (rc != QDQ_OK) return rc;
    return launch_topk_merge(n_cand, k, workspace, logits, n_vocab, index, value, stream);
  }
  rc = launch_q8_0_gemv(W, x, logits, n_vocab, n_in, batch, stream);
  if (rc != QDQ_OK) return rc;
  return launch_topk_rows(logits, n_vocab, batch, k, workspace, index, value, stream);
}

int qdq_q4k_qkv(const void *Wq, const void *Wk, const void *Wv, const float *x, float *q, float *k, float *v,
                int n_q, int n_kv, int n_embd, int batch, cudaStream_t stream) {
  if (!Wq || !Wk || !Wv || !x || !q || !k || !v) return QDQ_ERR_NULL;
  if (!dims_q4k(n_q, n_embd) || !dims_q4k(n_kv, n_embd) || n_kv > n_q) return QDQ_ERR_DIMS;
  if (batch < 1 || batch > QDQ_MAX_GEMV_BATCH) return QDQ_ERR_DIMS;
  if (n_embd > QDQ_MAX_GEMV_N_IN) return QDQ_ERR_UNSUPPORTED;
  if (int64_t(n_q) + 2 * int64_t(n_kv) > int64_t(1 << 30)) return QDQ_ERR_UNSUPPORTED;  // one row range
  if (!aligned(Wq, 16) || !aligned(Wk, 16) || !aligned(Wv, 16) || !aligned(x, 16) || !aligned(q, 4) ||
      !aligned(k, 4) || !aligned(v, 4))
    return QDQ_ERR_ALIGN;
  const size_t wqb = q4k_bytes(n_q, n_embd), wkb = q4k_bytes(n_kv, n_embd), xb = size_t(batch) * n_embd * 4;
  const size_t qb = size_t(batch) * n_q * 4, kb = size_t(batch) * n_kv * 4;
  const void *ins[4] = {Wq, Wk, Wv, x};
  const size_t inb[4] = {wqb, wkb, wkb, xb};
  const void *outs[3] = {q, k, v};
  const size_t outb[3] = {qb, kb, kb};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 4; ++i)
      if (overlaps(outs[o], outb[o], ins[i], inb[i])) return QDQ_ERR_ALIAS;
    for (int p = o + 1; p < 3; ++p)
      if (overlaps(outs[o], outb[o], outs[p], outb[p])) return QDQ_ERR_ALIAS;
  }
  if (gemv_xs_supported(n_embd, batch, 1)) return launch_gemv_xs_qkv(Wq, Wk, Wv, x, q, k, v, n_q, n_kv, n_embd, stream);
  // batch 2..8 (or rows wider than the batch-1 pipeline takes): three GEMV launches
  int rc = launch_q4k_gemv(0, Wq, nullptr, x, nullptr, q, n_q, n_embd, batch, stream);
  if (rc == QDQ_OK) rc = launch_q4k_gemv(0, Wk, nullptr, x, nullptr, k, n_kv, n_embd, batch, stream);
  if (rc == QDQ_OK) rc = launch_q4k_gemv(0, Wv, nullptr, x, nullptr, v, n_kv, n_embd, batch, stream);
  return rc;
}

size_t qdq_gemm_batch_workspace_bytes(int M, int n_out, int n_in) {
  if (M < 1 || n_out < 1 || n_in < 1) return 0;
  return gemm_workspace_bytes(M, n_out, n_in, 1);
}

size_t qdq_q4k_swiglu_batch_workspace_bytes(int M, int n_ff, int n_embd) {
  if (M < 1 || n_ff < 1 || n_embd < 1) return 0;
  return gemm_workspace_bytes(M, n_ff, n_embd, 2);
}

namespace {
// Shared checks of the tensor-core batch GEMMs: W (and W2 when non-NULL) packed
// n_out x n_in of w_bytes each, X M x n_in, Y M x n_out, workspace of ws_bytes.
int check_gemm_batch(const void *W, const void *W2, const float *X, const float *Y, const void *ws, int n_out,
                     int n_in, int M, size_t w_bytes) {
  if (!W || !X || !Y || !ws) return QDQ_ERR_NULL;
  if ((n_in % 64) != 0 || (n_out % 128) != 0) return QDQ_ERR_UNSUPPORTED;
  if (!aligned(W, 16) || (W2 && !aligned(W2, 16)) || !aligned(X, 16) || !aligned(Y, 16) || !aligned(ws, 256))
    return QDQ_ERR_ALIGN;
  const size_t xb = size_t(M) * n_in * 4, yb = size_t(M) * n_out * 4;
  // the workspace bytes the call uses: the bf16 activations above 64 tokens, else none (256 reserved)
  const size_t wsb = M > 64 ? size_t(M) * n_in * 2 : 256;
  if (overlaps(Y, yb, W, w_bytes) || (W2 && overlaps(Y, yb, W2, w_bytes)) || overlaps(Y, yb, X, xb) ||
      overlaps(Y, yb, ws, wsb) || overlaps(ws, wsb, W, w_bytes) || (W2 && overlaps(ws, wsb, W2, w_bytes)) ||
      overlaps(ws, wsb, X, xb))
    return QDQ_ERR_ALIAS;
  return QDQ_OK;
}
}  // namespace

int qdq_q8_0_gemm_batch(const void *W, const float *X, float *Y, void *workspace, int n_out, int n_in,
                        int M, cudaStream_t stream) {
  if (!W || !X || !Y || !workspace) return QDQ_ERR_NULL;
  if (!dims_q8(n_out, n_in) || M < 1) return QDQ_ERR_DIMS;
  const int rc = check_gemm_batch(W, nullptr, X, Y, workspace, n_out, n_in, M, q8_bytes(n_out, n_in));
  if (rc != QDQ_OK) return rc;
  return launch_q8_0_gemm_batch(W, X, Y, workspace, n_out, n_in, M, stream);
}

int qdq_q4k_gemm_batch(const void *W, const float *X, float *Y, void *workspace, int n_out, int n_in,
                       int M, cudaStream_t stream) {
  if (!W || !X || !Y || !workspace) return QDQ_ERR_NULL;
  if (!dims_q4k(n_out, n_in) || M < 1) return QDQ_ERR_DIMS;
  const int rc = check_gemm_batch(W, nullptr, X, Y, workspace, n_out, n_in, M, q4k_bytes(n_out, n_in));
  if (rc != QDQ_OK) return rc;
  return launch_q4k_gemm_batch(W, X, Y, workspace, n_out, n_in, M, stream);
}

int qdq_q4k_swiglu_batch(const void *Wg, const void *Wu, const float *X, float *mid, void *workspace, int n_ff,
                         int n_embd, int M, cudaStream_t stream) {
  if (!Wg || !Wu || !X || !mid || !workspace) return QDQ_ERR_NULL;
  if (!dims_q4k(n_ff, n_embd) || M < 1) return QDQ_ERR_DIMS;
  const int rc = check_gemm_batch(Wg, Wu, X, mid, workspace, n_ff, n_embd, M, q4k_bytes(n_ff, n_embd));
  if (rc != QDQ_OK) return rc;
  return launch_q4k_swiglu_batch(Wg, Wu, X, mid, workspace, n_ff, n_embd, M, stream);
}

int qdq_checks_enabled(void) {
#ifdef QDQ_CHECKS
  return 1;
#else
  return 0;
#endif
}

int qdq_check_status(void) {
  if (qdq_checks_enabled() && cudaDeviceSynchronize() != cudaSuccess) return -1;
  const int r[] = {read_checks_dl(), read_checks_xs(), read_checks_gemm(), read_checks_topk(), read_checks_q6k(),
                   read_checks_attn(), read_checks_attn_tc(), read_checks_logprobs()};
  int v = 0;
  for (int x : r) {
    if (x < 0) return -1;
    v |= x;
  }
  return v;
}

int qdq_noop(cudaStream_t stream) {
  noop_kernel<<<1, 1, 0, stream>>>();
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? QDQ_OK : fail_cuda(e);
}

}  // extern "C"
