// qg_api.cu -- the C ABI of libqgemm: argument checks on the host, then
// dispatch to the kernels on the caller's stream. Nothing here allocates.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <atomic>
#include <cmath>
#include <map>
#include <mutex>
#include <tuple>
#include <unordered_map>
#include <utility>

#include "qg_internal.h"
#include "qg_kv.cuh"
#include "qgemm.h"

namespace qg {

int device_sm_count() {
  static std::mutex mu;
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lk(mu);
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cache[dev] = n;
  }
  return cache[dev];
}

// Kernel preparation, cached per device. The dynamic shared-memory limit of a
// kernel is only ever raised (to the largest size any call has needed), so a
// launch on one host thread never finds the limit lowered by another thread
// between its check and its launch.
namespace {
std::mutex g_kmu;
std::map<std::pair<int, const void*>, size_t> g_smem_limit;          // (device, kernel)
std::map<std::tuple<int, const void*, int, size_t>, int> g_occupancy;  // (device, kernel, threads, smem)
}  // namespace

cudaError_t prepare_kernel(const void* kern, size_t smem, bool nonportable_cluster) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(g_kmu);
  auto it = g_smem_limit.find({dev, kern});
  if (it == g_smem_limit.end()) {
    if (nonportable_cluster &&
        (e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
      return e;
    it = g_smem_limit.emplace(std::make_pair(dev, kern), (size_t)0).first;
  }
  if (smem > it->second) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
        cudaSuccess)
      return e;
    it->second = smem;
  }
  return cudaSuccess;
}

cudaError_t kernel_occupancy(const void* kern, int threads, size_t smem, int* occ) {
  cudaError_t e = prepare_kernel(kern, smem, false);
  if (e != cudaSuccess) return e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(g_kmu);
  const auto key = std::make_tuple(dev, kern, threads, smem);
  auto it = g_occupancy.find(key);
  if (it == g_occupancy.end()) {
    int n = 0;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem)) != cudaSuccess)
      return e;
    it = g_occupancy.emplace(key, n < 1 ? 1 : n).first;
  }
  *occ = it->second;
  return cudaSuccess;
}

// The CUDA error behind the latest QG_ERR_CUDA returned on this host thread.
static thread_local cudaError_t t_last_cuda = cudaSuccess;
void note_cuda_error(cudaError_t e) { t_last_cuda = e; }
cudaError_t last_cuda_error() { return t_last_cuda; }

static std::atomic<uint64_t> g_launches{0};
void note_launch(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }

qg_status moe_check_shape(int t, int n_expert, int ffn, int hidden, int ncols, int topk) {
  if (t != QG_Q4_0 && t != QG_Q8_0) return QG_ERR_TYPE;
  if (n_expert < 1 || n_expert > QG_MOE_MAX_EXPERTS || ffn <= 0 || hidden <= 0 || (ffn % 32) ||
      (hidden % 32) || ncols < 1 || ncols > 16 || topk < 1 || topk > 16 ||
      !moe_shape_supported(ffn, hidden, ncols, topk))
    return QG_ERR_SHAPE;
  return QG_OK;
}

bool pdl_allowed(cudaStream_t s, LaunchClass cls) {
  static std::mutex mu;
  static std::unordered_map<cudaStream_t, int> last;  // class of the latest launch per stream
  std::lock_guard<std::mutex> lk(mu);
  auto it = last.find(s);
  const int prev = it == last.end() ? -1 : it->second;
  if (it == last.end()) {
    if (last.size() > 4096) last.clear();  // streams come and go; forget stale handles
    last.emplace(s, (int)cls);
  } else {
    it->second = (int)cls;
  }
  return !(cls == LC_FULL || (cls == LC_L1 && prev > LC_L1));
}

}  // namespace qg

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool valid_type(int t) { return t == QG_Q4_0 || t == QG_Q8_0; }

// Partial overlap of two byte ranges (identical start is allowed by the caller).
bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + nb && pb < pa + na;
}

qg_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return QG_OK;
  qg::note_cuda_error(e);
  return QG_ERR_CUDA;
}

// Common checks of a (rows x k) matrix product with ncols input columns.
qg_status check_matmul(int t, const void* q, const uint16_t* scl, int rows, int k,
                       const uint16_t* x, int ncols, int max_cols, const float* y0,
                       const void* out, size_t out_elem) {
  if (!valid_type(t)) return QG_ERR_TYPE;
  if (rows < 0 || k <= 0 || (k % 32) != 0 || ncols < 1 || ncols > max_cols) return QG_ERR_SHAPE;
  if (rows == 0) return QG_OK;
  if (!q || !scl || !x || !out) return QG_ERR_NULL;
  if (!aligned(q, 16) || !aligned(scl, 16) || !aligned(x, 16) || !aligned(out, out_elem) ||
      (y0 && !aligned(y0, 4)))
    return QG_ERR_ALIGN;
  if (y0 && y0 != out) {
    const size_t n = (size_t)ncols * rows * sizeof(float);
    if (overlaps(y0, n, out, n)) return QG_ERR_ALIAS;
  }
  return QG_OK;
}

// Token rows of the rotary and cache calls: ntok rows of `row` elements, `stride` apart.
bool float_type(int t) { return t == QG_F32 || t == QG_F16; }
bool rows_ok(int ntok, int64_t row, int64_t stride) {
  return ntok <= 1 || (stride >= row && stride <= ((int64_t)1 << 40) / ntok);
}
size_t rows_bytes(int ntok, int64_t row, int64_t stride, int t) {
  return ((size_t)(ntok - 1) * (ntok > 1 ? stride : 0) + row) * (t == QG_F32 ? 4 : 2);
}
bool plan_ok(const qg_rope* p) {
  return p->rot_dim >= 2 && p->rot_dim <= QG_ROPE_MAX_DIM && (p->rot_dim & 1) == 0;
}
qg_status kv_shape(int type, int n_kv_heads, int head_dim, int page_size) {
  if (type != QG_F16 && type != QG_Q8_0) return QG_ERR_TYPE;
  if (n_kv_heads < 1 || n_kv_heads > 256 || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return QG_ERR_SHAPE;
  return QG_OK;
}
qg_status check_cache(const qg_kvcache* c) {
  if (!c) return QG_ERR_NULL;
  const qg_status st = kv_shape(c->type, c->n_kv_heads, c->head_dim, c->page_size);
  if (st != QG_OK) return st;
  if (c->n_pages < 1 || c->n_seq < 1 || c->n_seq > QG_KV_MAX_SEQ || c->max_pages < 1 ||
      (int64_t)c->max_pages * c->page_size >= ((int64_t)1 << 31))
    return QG_ERR_SHAPE;
  if (!c->pool || !c->page_table) return QG_ERR_NULL;
  if (!aligned(c->pool, 16) || !aligned(c->page_table, 4)) return QG_ERR_ALIGN;
  return QG_OK;
}

// Device readiness (a device must be present and current).
qg_status check_device() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return from_cuda(e);
  // A host thread's first runtime calls need not bind the device's primary
  // context, and the tensor-core path calls the driver (tensor-map encoding)
  // before its first launch: on a fresh thread that failed with invalid value.
  // Make the context current once per thread and device.
  static thread_local int bound = -1;
  if (bound != dev) {
    if ((e = cudaSetDevice(dev)) != cudaSuccess) return from_cuda(e);
    bound = dev;
  }
  return qg::device_sm_count() > 0 ? QG_OK : from_cuda(cudaErrorNoDevice);
}

qg_status gemv_any(int t, const void* q, const uint16_t* scl, int rows, int k,
                   const uint16_t* x, int ncols, const float* y0, float* y, cudaStream_t s,
                   int max_cols) {
  qg_status st = check_matmul(t, q, scl, rows, k, x, ncols, max_cols, y0, y, 4);
  if (st != QG_OK || rows == 0) return st;
  if ((st = check_device()) != QG_OK) return st;
  if (qg::tc_supported(t, ncols, false, rows, k))
    return from_cuda(qg::tc_gemm(t, q, scl, nullptr, nullptr, rows, k, x, ncols, y0, y, nullptr, s));
  // CUDA-core path, at most 8 columns per launch
  for (int c0 = 0; c0 < ncols; c0 += 8) {
    const int nc = ncols - c0 < 8 ? ncols - c0 : 8;
    cudaError_t e = qg::cc_gemv(t, q, scl, rows, k, x + (size_t)c0 * k, nc,
                                y0 ? y0 + (size_t)c0 * rows : nullptr, y + (size_t)c0 * rows, s);
    if (e != cudaSuccess) return from_cuda(e);
  }
  return QG_OK;
}

}  // namespace

extern "C" {

int qg_last_cuda_error(void) { return (int)qg::last_cuda_error(); }

const char* qg_last_cuda_error_string(void) {
  static thread_local char buf[256];
  const cudaError_t e = qg::last_cuda_error();
  snprintf(buf, sizeof(buf), "%s: %s", cudaGetErrorName(e), cudaGetErrorString(e));
  return buf;
}

const char* qg_status_str(qg_status s) {
  switch (s) {
    case QG_OK: return "ok";
    case QG_ERR_NULL: return "a required pointer is NULL";
    case QG_ERR_SHAPE: return "invalid shape (k must be a positive multiple of 32; rows >= 0; ncols/topk/n_expert in range)";
    case QG_ERR_ALIGN: return "misaligned pointer or stride (quants, scales, x: 16 bytes; y, y0: 4 bytes; h: 2 bytes)";
    case QG_ERR_TYPE: return "a type the call does not take (weights: Q4_0=2 or Q8_0=8)";
    case QG_ERR_WORKSPACE: return "workspace missing or smaller than the call's workspace_bytes()";
    case QG_ERR_CUDA: return "CUDA runtime error";
    case QG_ERR_ALIAS: return "an input partially overlaps the output (such as y0 and y)";
  }
  return "unknown status";
}

qg_status qgemv_q4_0(const uint8_t* nib, const uint16_t* scl, int rows, int k,
                     const uint16_t* x, int ncols, const float* y0, float* y,
                     cudaStream_t stream) {
  return gemv_any(QG_Q4_0, nib, scl, rows, k, x, ncols, y0, y, stream, 8);
}

qg_status qgemv_q8_0(const int8_t* qs, const uint16_t* scl, int rows, int k,
                     const uint16_t* x, int ncols, const float* y0, float* y,
                     cudaStream_t stream) {
  return gemv_any(QG_Q8_0, qs, scl, rows, k, x, ncols, y0, y, stream, 8);
}

qg_status qgemm_cols(qg_type t, const void* q, const uint16_t* scl, int rows, int k,
                     const uint16_t* x, int ncols, const float* y0, float* y,
                     cudaStream_t stream) {
  return gemv_any((int)t, q, scl, rows, k, x, ncols, y0, y, stream, 16);
}

qg_status qffn_gate_up_silu(qg_type t, const void* qg, const uint16_t* sg, const void* qu,
                            const uint16_t* su, int rows, int k, const uint16_t* x,
                            int ncols, uint16_t* h, cudaStream_t stream) {
  qg_status st = check_matmul((int)t, qg, sg, rows, k, x, ncols, 16, nullptr, h, 2);
  if (st != QG_OK || rows == 0) return st;
  if (!qu || !su) return QG_ERR_NULL;
  if (!aligned(qu, 16) || !aligned(su, 16)) return QG_ERR_ALIGN;
  if ((st = check_device()) != QG_OK) return st;
  if (qg::tc_supported((int)t, ncols, true, rows, k))
    return from_cuda(qg::tc_gemm((int)t, qg, sg, qu, su, rows, k, x, ncols, nullptr, nullptr, h, stream));
  for (int c0 = 0; c0 < ncols; c0 += 8) {
    const int nc = ncols - c0 < 8 ? ncols - c0 : 8;
    cudaError_t e = qg::cc_gate_up_silu((int)t, qg, sg, qu, su, rows, k, x + (size_t)c0 * k, nc,
                                        h + (size_t)c0 * rows, stream);
    if (e != cudaSuccess) return from_cuda(e);
  }
  return QG_OK;
}

size_t qmoe_workspace_bytes(int n_expert, int ffn, int hidden, int ncols, int topk) {
  if (qg::moe_check_shape(QG_Q8_0, n_expert, ffn, hidden, ncols, topk) != QG_OK) return 0;
  return qg::moe_ws_bytes(n_expert, ffn, hidden, ncols, topk);
}

qg_status qmoe_experts(qg_type t, const void* qg, const uint16_t* sg, const void* qu,
                       const uint16_t* su, const void* qd, const uint16_t* sd,
                       int n_expert, int ffn, int hidden, const int32_t* ids,
                       const float* rw, int topk, const qg_expert* shared,
                       const uint16_t* x, int ncols, const float* y0, float* y,
                       void* ws, size_t ws_bytes, int32_t* err_flag,
                       int32_t* uniq_ids_out, cudaStream_t stream) {
  qg_status st0 = qg::moe_check_shape((int)t, n_expert, ffn, hidden, ncols, topk);
  if (st0 != QG_OK) return st0;
  if (!qg || !sg || !qu || !su || !qd || !sd || !ids || !rw || !x || !y) return QG_ERR_NULL;
  const void* p16[] = {qg, sg, qu, su, qd, sd, x};
  for (const void* p : p16)
    if (!aligned(p, 16)) return QG_ERR_ALIGN;
  if (!aligned(ids, 4) || !aligned(rw, 4) || !aligned(y, 4) || (y0 && !aligned(y0, 4)) ||
      (err_flag && !aligned(err_flag, 4)) || (uniq_ids_out && !aligned(uniq_ids_out, 4)))
    return QG_ERR_ALIGN;
  if (shared) {
    if (!shared->qg || !shared->sg || !shared->qu || !shared->su || !shared->qd || !shared->sd)
      return QG_ERR_NULL;
    const void* s16[] = {shared->qg, shared->sg, shared->qu, shared->su, shared->qd, shared->sd};
    for (const void* p : s16)
      if (!aligned(p, 16)) return QG_ERR_ALIGN;
  }
  if (y0 && y0 != y) {
    const size_t n = (size_t)ncols * hidden * sizeof(float);
    if (overlaps(y0, n, y, n)) return QG_ERR_ALIAS;
  }
  const size_t need = qg::moe_ws_bytes(n_expert, ffn, hidden, ncols, topk);
  if (!ws || ws_bytes < need) return QG_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return QG_ERR_ALIGN;
  qg_status st = check_device();
  if (st != QG_OK) return st;
  qg::MoeArgs a{};
  a.qt = (int)t;
  a.qg = qg; a.qu = qu; a.qd = qd; a.sg = sg; a.su = su; a.sd = sd;
  a.n_expert = n_expert; a.ffn = ffn; a.hidden = hidden;
  a.ids = ids; a.rw = rw; a.topk = topk;
  a.has_shared = shared != nullptr;
  if (shared) {
    a.sqg = shared->qg; a.squ = shared->qu; a.sqd = shared->qd;
    a.ssg = shared->sg; a.ssu = shared->su; a.ssd = shared->sd;
  }
  a.x = x; a.ncols = ncols; a.y0 = y0; a.y = y;
  a.ws = ws; a.err_flag = err_flag; a.uniq_out = uniq_ids_out;
  return from_cuda(qg::moe_forward(a, stream));
}

qg_status qmoe_router(const float* w_router, const uint16_t* x, int n_expert, int hidden,
                      int ncols, int topk, float* logits_out, int32_t* ids_out, float* rw_out,
                      cudaStream_t stream) {
  if (!qg::router_shape_ok(n_expert, hidden, ncols, topk)) return QG_ERR_SHAPE;
  if (!w_router || !x || !ids_out || !rw_out) return QG_ERR_NULL;
  if (!aligned(w_router, 16) || !aligned(x, 2) || !aligned(ids_out, 4) || !aligned(rw_out, 4) ||
      (logits_out && !aligned(logits_out, 4)))
    return QG_ERR_ALIGN;
  qg_status st = check_device();
  if (st != QG_OK) return st;
  return from_cuda(qg::router_launch(w_router, x, n_expert, hidden, ncols, topk, logits_out,
                                     ids_out, rw_out, stream));
}

qg_status qargmax_f32(const float* x, int n, int ncols, int32_t* idx_out, float* val_out,
                      cudaStream_t stream) {
  if (n < 1 || ncols < 1 || ncols > 64) return QG_ERR_SHAPE;
  if (!x || !idx_out) return QG_ERR_NULL;
  if (!aligned(x, 4) || !aligned(idx_out, 4) || (val_out && !aligned(val_out, 4))) return QG_ERR_ALIGN;
  qg_status st = check_device();
  if (st != QG_OK) return st;
  return from_cuda(qg::argmax_launch(x, n, ncols, idx_out, val_out, stream));
}

qg_status qtopk_f32(const float* x, int n, int ncols, int k, int32_t* idx_out, float* val_out,
                    cudaStream_t stream) {
  if (n < 1 || ncols < 1 || ncols > 64 || k < 1 || k > 256 || k > n) return QG_ERR_SHAPE;
  if (!x || !idx_out) return QG_ERR_NULL;
  if (!aligned(x, 4) || !aligned(idx_out, 4) || (val_out && !aligned(val_out, 4))) return QG_ERR_ALIGN;
  qg_status st = check_device();
  if (st != QG_OK) return st;
  return from_cuda(qg::topk_launch(x, n, ncols, k, idx_out, val_out, stream));
}

qg_status qrepack(qg_type t, const void* gguf, int rows, int k, void* q_out,
                  uint16_t* scl_out, cudaStream_t stream) {
  if (!valid_type((int)t)) return QG_ERR_TYPE;
  if (rows < 0 || k <= 0 || (k % 32) != 0) return QG_ERR_SHAPE;
  if (rows == 0) return QG_OK;
  if (!gguf || !q_out || !scl_out) return QG_ERR_NULL;
  if (!aligned(gguf, 2) || !aligned(q_out, 16) || !aligned(scl_out, 16)) return QG_ERR_ALIGN;
  qg_status st = check_device();
  if (st != QG_OK) return st;
  return from_cuda(qg::repack_launch((int)t, gguf, rows, k, q_out, scl_out, stream));
}

qg_status qrope_plan(qg_rope* plan, int rot_dim, int interleaved, double base, double factor,
                     int orig_ctx, double low_turns, double high_turns, double mscale) {
  if (!plan) return QG_ERR_NULL;
  const double pi2 = 6.283185307179586476925;
  if (rot_dim < 2 || rot_dim > QG_ROPE_MAX_DIM || (rot_dim & 1) || !(base > 0) || !std::isfinite(base) ||
      !(factor > 0) || !std::isfinite(factor) || orig_ctx < 0 || !std::isfinite(mscale) ||
      !std::isfinite((double)(float)mscale))
    return QG_ERR_SHAPE;
  if (orig_ctx > 0 &&
      (!std::isfinite(low_turns) || !std::isfinite(high_turns) || !(high_turns > low_turns)))
    return QG_ERR_SHAPE;
  qg_rope p{};
  p.rot_dim = rot_dim;
  p.interleaved = interleaved != 0;
  p.mscale = (float)mscale;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double theta = std::pow(base, -2.0 * i / rot_dim);
    if (factor != 1.0) {
      double keep = 0.0;
      if (orig_ctx > 0) {
        keep = (orig_ctx * theta / pi2 - low_turns) / (high_turns - low_turns);
        keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      }
      theta = theta * keep + theta / factor * (1 - keep);
    }
    double turns = theta / pi2;
    // its rounding errors (a few 2^-53 of it) would exceed those of the f32 angle, 2^-26 turns
    if (!(turns < 67108864.0)) return QG_ERR_SHAPE;
    turns -= std::floor(turns);  // whole turns do nothing
    if (turns >= 1.0) turns = 0.0;
    p.step[i] = (uint64_t)std::ldexp(turns, 64);
  }
  *plan = p;
  return QG_OK;
}

qg_status qrope(const qg_rope* plan, qg_type xt, const void* x, int64_t x_stride,
                const int32_t* pos, int ntok, int n_heads, int head_dim, qg_type yt, void* y,
                int64_t y_stride, cudaStream_t stream) {
  if (!float_type((int)xt) || !float_type((int)yt)) return QG_ERR_TYPE;
  if (!plan) return QG_ERR_NULL;
  if (!plan_ok(plan) || ntok < 0 || n_heads < 1 || n_heads > (1 << 20) || head_dim < 8 ||
      head_dim > 256 || (head_dim % 8) || plan->rot_dim > head_dim)
    return QG_ERR_SHAPE;
  if (ntok == 0) return QG_OK;
  const int64_t row = (int64_t)n_heads * head_dim;
  if (!rows_ok(ntok, row, x_stride) || !rows_ok(ntok, row, y_stride)) return QG_ERR_SHAPE;
  if (!x || !y || !pos) return QG_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(pos, 4) || (ntok > 1 && (x_stride % 8 || y_stride % 8)))
    return QG_ERR_ALIGN;
  const size_t xb = rows_bytes(ntok, row, x_stride, (int)xt), yb = rows_bytes(ntok, row, y_stride, (int)yt);
  const bool in_place = x == y && xt == yt && (ntok == 1 || x_stride == y_stride);
  if ((!in_place && overlaps(x, xb, y, yb)) || overlaps(pos, (size_t)ntok * 4, y, yb)) return QG_ERR_ALIAS;
  qg_status st = check_device();
  if (st != QG_OK) return st;
  return from_cuda(qg::rope_launch(*plan, (int)xt, x, x_stride, pos, ntok, n_heads, head_dim, (int)yt, y,
                                   y_stride, stream));
}

size_t qkv_page_bytes(qg_type type, int n_kv_heads, int head_dim, int page_size) {
  if (kv_shape((int)type, n_kv_heads, head_dim, page_size) != QG_OK) return 0;
  return qg::kv_page_bytes((int)type, n_kv_heads, head_dim, page_size);
}

qg_status qkv_append(const qg_kvcache* cache, const qg_rope* rope, qg_type xt, const void* k,
                     int64_t k_stride, const void* v, int64_t v_stride, const void* q,
                     int64_t q_stride, int n_q_heads, uint16_t* q_out, const int32_t* seq,
                     const int32_t* pos, int ntok, int32_t* err_flag, cudaStream_t stream) {
  qg_status st = check_cache(cache);
  if (st != QG_OK) return st;
  if (!float_type((int)xt)) return QG_ERR_TYPE;
  if (ntok < 0 || (rope && (!plan_ok(rope) || rope->rot_dim > cache->head_dim)) ||
      (q && (n_q_heads < 1 || n_q_heads > (1 << 20))) || (!seq && ntok % cache->n_seq))
    return QG_ERR_SHAPE;
  if (ntok == 0) return QG_OK;
  const int64_t row = (int64_t)cache->n_kv_heads * cache->head_dim;
  const int64_t qrow = q ? (int64_t)n_q_heads * cache->head_dim : 0;
  if (!rows_ok(ntok, row, k_stride) || !rows_ok(ntok, row, v_stride) || (q && !rows_ok(ntok, qrow, q_stride)))
    return QG_ERR_SHAPE;
  if (!k || !v || !pos || (q && !q_out)) return QG_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(pos, 4) || !aligned(seq, 4) || !aligned(err_flag, 4) ||
      (q && (!aligned(q, 16) || !aligned(q_out, 16))) ||
      (ntok > 1 && (k_stride % 8 || v_stride % 8 || (q && q_stride % 8))))
    return QG_ERR_ALIGN;
  // what is written (q_out, the pool) must not be read: queries, keys, values, positions, table
  struct Range { const void* p; size_t n; };
  const Range in[] = {{k, rows_bytes(ntok, row, k_stride, (int)xt)},
                      {v, rows_bytes(ntok, row, v_stride, (int)xt)},
                      {q, q ? rows_bytes(ntok, qrow, q_stride, (int)xt) : 0},
                      {pos, (size_t)ntok * 4},
                      {seq, seq ? (size_t)ntok * 4 : 0},
                      {cache->page_table, (size_t)cache->n_seq * cache->max_pages * 4}};
  const Range out[] = {{q ? q_out : nullptr, q ? (size_t)ntok * qrow * 2 : 0},
                       {cache->pool, (size_t)cache->n_pages * qg::kv_page_bytes(cache->type, cache->n_kv_heads,
                                                                                cache->head_dim, cache->page_size)}};
  for (const Range& o : out)
    for (const Range& i : in)
      if (o.n && i.n && overlaps(o.p, o.n, i.p, i.n)) return QG_ERR_ALIAS;
  if (out[0].n && overlaps(out[0].p, out[0].n, out[1].p, out[1].n)) return QG_ERR_ALIAS;
  if ((st = check_device()) != QG_OK) return st;
  qg::KvAppendArgs a{};
  a.c = *cache;
  a.rope = rope;
  a.xt = (int)xt;
  a.q = q; a.k = k; a.v = v;
  a.qs = q_stride; a.ks = k_stride; a.vs = v_stride;
  a.n_q = q ? n_q_heads : 0;
  a.q_out = q_out;
  a.seq = seq; a.pos = pos; a.ntok = ntok;
  a.err = err_flag;
  return from_cuda(qg::kv_append_launch(a, stream));
}

qg_status qkv_read(const qg_kvcache* cache, const int32_t* seq, const int32_t* pos, int ntok,
                   qg_type yt, void* k_out, void* v_out, int32_t* err_flag, cudaStream_t stream) {
  qg_status st = check_cache(cache);
  if (st != QG_OK) return st;
  if (!float_type((int)yt)) return QG_ERR_TYPE;
  if (ntok < 0 || (!seq && ntok % cache->n_seq)) return QG_ERR_SHAPE;
  if (ntok == 0 || (!k_out && !v_out)) return QG_OK;
  if (!pos) return QG_ERR_NULL;
  if (!aligned(pos, 4) || !aligned(seq, 4) || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(err_flag, 4))
    return QG_ERR_ALIGN;
  const size_t nb = rows_bytes(ntok, (int64_t)cache->n_kv_heads * cache->head_dim,
                               (int64_t)cache->n_kv_heads * cache->head_dim, (int)yt);
  const size_t pool = (size_t)cache->n_pages *
                      qg::kv_page_bytes(cache->type, cache->n_kv_heads, cache->head_dim, cache->page_size);
  const size_t table = (size_t)cache->n_seq * cache->max_pages * 4;
  if (k_out && v_out && overlaps(k_out, nb, v_out, nb)) return QG_ERR_ALIAS;
  for (const void* o : {(const void*)k_out, (const void*)v_out})
    if (o && (overlaps(o, nb, cache->pool, pool) || overlaps(o, nb, pos, (size_t)ntok * 4) ||
              (seq && overlaps(o, nb, seq, (size_t)ntok * 4)) || overlaps(o, nb, cache->page_table, table)))
      return QG_ERR_ALIAS;
  if ((st = check_device()) != QG_OK) return st;
  return from_cuda(qg::kv_read_launch(*cache, seq, pos, ntok, (int)yt, k_out, v_out, err_flag, stream));
}

size_t qattn_workspace_bytes(int n_seq, int n_heads, int n_kv_heads, int head_dim, int ncols) {
  if (!qg::attn_shape_ok(n_seq, n_heads, n_kv_heads, head_dim, ncols)) return 0;
  return qg::attn_ws_bytes(n_seq, n_heads, n_kv_heads, head_dim, ncols);
}

qg_status qattn_paged(const qg_kvcache* cache, const uint16_t* q, int n_heads, int ncols,
                      const int32_t* lens, int window, float scale, uint16_t* y, void* ws,
                      size_t ws_bytes, int32_t* err_flag, cudaStream_t stream) {
  qg_status st = check_cache(cache);
  if (st != QG_OK) return st;
  if (!qg::attn_shape_ok(cache->n_seq, n_heads, cache->n_kv_heads, cache->head_dim, ncols) || window < 0 ||
      !std::isfinite(scale) || !qg::attn_size_ok(*cache, n_heads, ncols))
    return QG_ERR_SHAPE;
  if (!q || !lens || !y) return QG_ERR_NULL;
  if (!aligned(q, 16) || !aligned(y, 16) || !aligned(lens, 4) || !aligned(err_flag, 4)) return QG_ERR_ALIGN;
  const size_t need = qg::attn_ws_bytes(cache->n_seq, n_heads, cache->n_kv_heads, cache->head_dim, ncols);
  if (!ws || ws_bytes < need) return QG_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return QG_ERR_ALIGN;
  const size_t nq = (size_t)cache->n_seq * ncols * n_heads * cache->head_dim * 2;
  const size_t pool = (size_t)cache->n_pages *
                      qg::kv_page_bytes(cache->type, cache->n_kv_heads, cache->head_dim, cache->page_size);
  const size_t nl = (size_t)cache->n_seq * 4, table = nl * cache->max_pages;
  struct Range { const void* p; size_t n; };
  const Range in[] = {{q, nq}, {lens, nl}, {cache->pool, pool}, {cache->page_table, table}};
  if (overlaps(ws, need, y, nq)) return QG_ERR_ALIAS;
  for (const Range& r : in)
    if (overlaps(r.p, r.n, y, nq) || overlaps(r.p, r.n, ws, need)) return QG_ERR_ALIAS;
  if ((st = check_device()) != QG_OK) return st;
  qg::AttnArgs a{};
  a.c = *cache;
  a.q = q;
  a.n_heads = n_heads; a.ncols = ncols;
  a.lens = lens;
  a.window = window;
  a.scale = scale;
  a.y = y;
  a.ws = ws;
  a.err = err_flag;
  return from_cuda(qg::attn_launch(a, stream));
}

uint64_t qg_kernel_launches(void) { return qg::g_launches.load(std::memory_order_relaxed); }

}  // extern "C"
