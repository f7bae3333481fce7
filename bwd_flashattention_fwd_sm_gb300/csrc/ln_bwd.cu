// Backward pass of dropout + residual add + LayerNorm: the entry, and the join of the columns'
// partial sums.  ln_bwd.cuh has the kernels.
#include "ln_bwd.cuh"

#include "overlap.h"

namespace gbattn {
void set_last_error_text(const char* text);
attn_status_t device_status(int** status, int* sms, unsigned long long* wait_ns);

extern template cudaError_t launch_ln_bwd<__nv_bfloat16>(const BwdLnArgs&, bool, int*, int*, unsigned long long,
                                                         cudaStream_t);
extern template cudaError_t launch_ln_bwd<float>(const BwdLnArgs&, bool, int*, int*, unsigned long long, cudaStream_t);

namespace {

// Adds the blocks' rows: sixteen warps each a stretch of them, in order, then the sixteen in order.
// A warp's loads are all in flight at once, ten at a time: the join waits for memory twice at most.
constexpr int kJoinWarps = 16, kJoinAtOnce = 10;

__global__ void __launch_bounds__(32 * kJoinWarps) k_ln_bwd_join(const float* part, int parts, int64_t cols,
                                                                 float* dgamma, float* dbeta) {
  __shared__ float sum[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const int each = (parts + kJoinWarps - 1) / kJoinWarps;
  const int end = min(parts, (warp + 1) * each);
  const int64_t step = 2 * cols;
  part += (blockIdx.y ? cols : 0) + c + warp * each * step;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
  float s = 0.f;
  if (c < cols) {
    for (int i = warp * each; i < end; i += kJoinAtOnce, part += kJoinAtOnce * step) {
      float v[kJoinAtOnce];
#pragma unroll
      for (int k = 0; k < kJoinAtOnce; ++k) v[k] = i + k < end ? part[k * step] : 0.f;
#pragma unroll
      for (int k = 0; k < kJoinAtOnce; ++k) s += v[k];
    }
  }
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) s += sum[w][lane];
    out[c] = s;
  }
}

// The join may be set up while the first kernel runs.
cudaError_t launch_join(const BwdLnArgs& a, int parts, float* dgamma, float* dbeta, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((a.p.cols + 31) / 32), 2);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_ln_bwd_join, (const float*)a.part, parts, a.p.cols, dgamma, dbeta);
}

attn_status_t bfail(attn_status_t s, const char* msg) {
  set_last_error_text(msg);
  return s;
}

attn_status_t check_params(const ln_bwd_params_t* p) {
  if (!p) return bfail(ATTN_ERR_INVALID_ARG, "ln_residual_bwd: params is NULL");
  if (p->dtype != ATTN_BF16 && p->dtype != ATTN_F32)
    return bfail(ATTN_ERR_INVALID_ARG, "ln_residual_bwd: dtype is not ATTN_F32 or ATTN_BF16");
  if (p->rows < 0 || p->cols < 1) return bfail(ATTN_ERR_INVALID_ARG, "ln_residual_bwd: rows < 0 or cols < 1");
  if (p->cols > 16384) return bfail(ATTN_ERR_UNSUPPORTED, "ln_residual_bwd: cols above 16384");
  return ATTN_OK;
}

// Whether something that the call writes shares memory with something else of it: the outputs dx and dr in place of
// dy or dh are allowed, and one in place of the other where they are equal (drops is false).
bool outputs_meet(const BwdLnArgs& a, bool drops, float* dgamma, float* dbeta, const void* workspace, size_t need) {
  const int64_t size = a.p.dtype == ATTN_BF16 ? 2 : 4, width = a.p.cols * size, rows = a.p.rows;
  auto line = [](const void* at, int64_t bytes) { return RowSpan{at, 1, bytes, bytes}; };
  const int64_t stats = rows * 4, columns = a.p.cols * 4;
  const RowSpan written[5] = {{a.dx, rows, a.p.dx_stride * size, width}, {a.dr, rows, a.p.dr_stride * size, width},
                              line(dgamma, columns), line(dbeta, columns), line(workspace, (int64_t)need)};
  const RowSpan read[6] = {{a.dy, rows, a.p.dy_stride * size, width}, {a.dh, rows, a.p.dh_stride * size, width},
                           {a.h, rows, a.p.h_stride * size, width}, line(a.mean, stats), line(a.rstd, stats),
                           line(a.gamma, columns)};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 6; ++j)
      if (rows_meet(written[i], read[j]) && !(i < 2 && j < 2 && same_rows(written[i], read[j]))) return true;
    for (int j = 0; j < i; ++j)
      if (rows_meet(written[i], written[j]) && !(i == 1 && j == 0 && !drops && same_rows(written[i], written[j])))
        return true;
  }
  return false;
}

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" {

size_t ln_residual_bwd_workspace_size(const ln_bwd_params_t* p) {
  if (check_params(p) != ATTN_OK) return SIZE_MAX;
  if (ln_bwd_joins(*p)) return 0;
  return (size_t)std::min<int64_t>(p->rows, kLnMaxParts) * 2 * (size_t)p->cols * sizeof(float);
}

attn_status_t ln_residual_bwd(const ln_bwd_params_t* p, const ln_dropout_t* d, const void* dy, const void* dh,
                              const void* h, const float* mean, const float* rstd, const float* gamma, void* dx,
                              void* dr, float* dgamma, float* dbeta, void* workspace, size_t workspace_bytes,
                              void* stream) {
  attn_status_t s = check_params(p);
  if (s != ATTN_OK) return s;
  BwdLnArgs a{*p, dy, dh, h, mean, rstd, gamma, dx, dr, nullptr, nullptr, nullptr, false, 0, 1, {}};
  bool drops = false;
  if (const char* wrong = resolve_dropout(d, &a.drop, &drops)) return bfail(ATTN_ERR_INVALID_ARG, wrong);
  if (drops && p->rows >= (int64_t)1 << 32)
    return bfail(ATTN_ERR_UNSUPPORTED, "ln_residual_bwd: dropout of 2^32 rows or more");
  const void* tensors[5] = {dy, dh, h, dx, dr};
  const int64_t strides[5] = {p->dy_stride, p->dh_stride, p->h_stride, p->dx_stride, p->dr_stride};
  const uintptr_t esize = p->dtype == ATTN_BF16 ? 2 : 4;
  uintptr_t at = 0;
  for (int i = 0; i < 5; ++i) {
    if (!tensors[i]) continue;
    if (((reinterpret_cast<uintptr_t>(tensors[i]) ^ reinterpret_cast<uintptr_t>(dy)) & 15) || strides[i] != p->dy_stride)
      a.alike = 0;
    if (strides[i] < p->cols) return bfail(ATTN_ERR_INVALID_ARG, "ln_residual_bwd: a row stride is below cols");
    at |= reinterpret_cast<uintptr_t>(tensors[i]) | (uintptr_t)strides[i] * esize;
  }
  auto floats = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 3) != 0; };
  if ((at & (esize - 1)) || floats(mean) || floats(rstd) || floats(gamma) || floats(dgamma) || floats(dbeta))
    return bfail(ATTN_ERR_INVALID_ARG, "ln_residual_bwd: a pointer is not aligned to its element size");
  const bool weights = dgamma || dbeta;
  if (p->rows == 0 && !weights) return ATTN_OK;
  if (p->rows > 0 && (!dy || !h || !mean || !rstd))
    return bfail(ATTN_ERR_INVALID_ARG, "ln_residual_bwd: dy, h, mean or rstd is NULL");
  const size_t need = weights ? ln_residual_bwd_workspace_size(p) : 0;
  if (need && !workspace) return bfail(ATTN_ERR_WORKSPACE, "ln_residual_bwd: workspace is NULL");
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return bfail(ATTN_ERR_WORKSPACE, "ln_residual_bwd: workspace is not 256-byte aligned");
  if (workspace_bytes < need) return bfail(ATTN_ERR_WORKSPACE, "ln_residual_bwd: workspace is too small");
  int* status = nullptr;
  int sms = 0;
  unsigned long long wait_ns = 0;
  if ((s = device_status(&status, &sms, &wait_ns))) return s;
  if (outputs_meet(a, drops, dgamma, dbeta, workspace, need))
    return bfail(ATTN_ERR_INVALID_ARG, "ln_residual_bwd: an output or the workspace overlaps another argument");
  a.vec = ((at | reinterpret_cast<uintptr_t>(gamma)) & 15) == 0;
  if (weights && p->rows > 0) {
    if (ln_bwd_joins(*p))
      a.join = true, a.dgamma = dgamma, a.dbeta = dbeta;
    else
      a.part = static_cast<float*>(workspace);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int blocks = 0;
  cudaError_t e = cudaSuccess;
  if (p->rows > 0)
    e = p->dtype == ATTN_BF16 ? launch_ln_bwd<__nv_bfloat16>(a, drops, &blocks, status, wait_ns, st)
                              : launch_ln_bwd<float>(a, drops, &blocks, status, wait_ns, st);
  if (e == cudaSuccess && weights && !a.join) e = launch_join(a, blocks, dgamma, dbeta, st);
  if (e != cudaSuccess) return bfail(ATTN_ERR_CUDA, "ln_residual_bwd: launch failed");
  return ATTN_OK;
}

}  // extern "C"
