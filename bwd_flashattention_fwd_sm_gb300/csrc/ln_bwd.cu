// Backward pass of dropout + residual add + LayerNorm (include/gbln.h has the formulas).
//
// Two sums of a row (of g and of g xh) decide its dr, and two sums of a column (of dy
// xh and of dy) are dgamma and dbeta.  A row belongs to a warp (short rows) or to a
// block; a thread keeps the same columns in every row, so that its parts of the columns'
// sums stay in registers from its block's first row to its last.  Each block leaves one
// row of partial sums; k_ln_bwd_join adds them in a fixed order.
// Bound by device memory: dy, h and dh are read once and dr and dx written once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gbln.h"
#include "common.cuh"
#include "dropout.cuh"
#include "rowvec.cuh"

namespace gbattn {
void set_last_error_text(const char* text);
attn_status_t device_status(int** status, int* sms, unsigned long long* wait_ns);

namespace {

// Rows of partial sums at most: two blocks on each of 152 SMs.  A constant, so that
// the size of the workspace and the order of the sums are the same everywhere.
constexpr int kMaxParts = 304;

struct BwdLnArgs {
  ln_bwd_params_t p;
  const void* dy;
  const void* dh;
  const void* h;
  const float* mean;
  const float* rstd;
  const float* gamma;
  void* dx;
  void* dr;
  float* part;  // [blocks][2][cols]: sums of dy xh, and of dy; NULL: not wanted
  int vec;      // every pointer 16-byte aligned and every stride a whole number of vectors
  DropArgs drop;
};

// The widened vector at column c0 of a row; 0 behind the row's end.
template <class T>
__device__ __forceinline__ void load_cols(const T* row, int64_t c0, int64_t cols, bool vec, float (&v)[Vec<T>::E]) {
  if (vec && c0 + Vec<T>::E <= cols) {
    Vec<T>::load(row + c0, v);
  } else {
#pragma unroll
    for (int e = 0; e < Vec<T>::E; ++e) v[e] = c0 + e < cols ? Vec<T>::load1(row + c0 + e) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void store_cols(T* row, int64_t c0, int64_t cols, bool vec, const float (&v)[Vec<T>::E]) {
  if (vec && c0 + Vec<T>::E <= cols) {
    Vec<T>::store(row + c0, v);
  } else {
#pragma unroll
    for (int e = 0; e < Vec<T>::E; ++e)
      if (c0 + e < cols) Vec<T>::store1(row + c0 + e, v[e]);
  }
}

// kThreads threads a block, kRow of them (a warp or all) on a row, kVpt vectors of a row each.
template <class T, int kThreads, int kRow, int kVpt, bool kDrop>
__global__ void __launch_bounds__(kThreads) k_ln_bwd(const BwdLnArgs a) {
  constexpr int E = Vec<T>::E, kRows = kThreads / kRow, kWarps = kRow / 32;
  static_assert(kRow == 32 || kRow == kThreads, "a warp or a block");
  __shared__ float2 warp_sum[2][kWarps];
  extern __shared__ float column[];  // [cols] twice, where a block has several rows
  const int tid = threadIdx.x % kRow, lane = threadIdx.x & 31, warp = tid >> 5;
  const int64_t cols = a.p.cols;
  const float inv = 1.f / (float)cols;
  DropKey key{};
  if constexpr (kDrop) key = drop_key(a.drop);
  float sg[kVpt][E], sb[kVpt][E];
#pragma unroll
  for (int j = 0; j < kVpt; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) sg[j][e] = sb[j][e] = 0.f;
  int phase = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kRow; row < a.p.rows;
       row += (int64_t)gridDim.x * kRows, phase ^= 1) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.p.dy_stride;
    const T* h = static_cast<const T*>(a.h) + row * a.p.h_stride;
    const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.p.dh_stride : nullptr;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float g[kVpt][E], xh[kVpt][E], in[kVpt][E];
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      const int64_t c0 = (int64_t)(tid + j * kRow) * E;
      if (c0 >= cols) continue;
      load_cols<T>(dy, c0, cols, a.vec, g[j]);
      load_cols<T>(h, c0, cols, a.vec, xh[j]);
      if (dh) load_cols<T>(dh, c0, cols, a.vec, in[j]);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (!dh) in[j][e] = 0.f;
        if (c0 + e < cols) {  // a row's end inside a vector
          xh[j][e] = (xh[j][e] - mean) * rstd;
          sg[j][e] += g[j][e] * xh[j][e];
          sb[j][e] += g[j][e];
          if (a.gamma) g[j][e] *= __ldg(a.gamma + c0 + e);
          s0 += g[j][e];
          s1 += g[j][e] * xh[j][e];
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, o);
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    }
    if constexpr (kWarps > 1) {
      if (lane == 0) warp_sum[phase][warp] = make_float2(s0, s1);
      __syncthreads();  // the other phase's sums are read before the next barrier, and written after it
      s0 = s1 = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 t = warp_sum[phase][w];
        s0 += t.x;
        s1 += t.y;
      }
    }
    s0 *= inv;
    s1 *= inv;
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      const int64_t c0 = (int64_t)(tid + j * kRow) * E;
      if (c0 >= cols) continue;
      float d[E];
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = in[j][e] + rstd * (g[j][e] - s0 - xh[j][e] * s1);
      if (a.dr) store_cols<T>(static_cast<T*>(a.dr) + row * a.p.dr_stride, c0, cols, a.vec, d);
      if (a.dx) {
        if constexpr (kDrop) drop_vector<E>(a.drop, key, c0, row, d);
        store_cols<T>(static_cast<T*>(a.dx) + row * a.p.dx_stride, c0, cols, a.vec, d);
      }
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * cols;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int j = 0; j < kVpt; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int64_t c = (int64_t)(tid + j * kRow) * E + e;
        if (c < cols) part[c] = sg[j][e], part[cols + c] = sb[j][e];
      }
  } else {  // the block's warps one after the other
    for (int w = 0; w < kRows; ++w) {
      if ((int)threadIdx.x / kRow == w) {
#pragma unroll
        for (int j = 0; j < kVpt; ++j)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int c = (tid + j * kRow) * E + e;
            if (c < cols) {
              column[c] = (w ? column[c] : 0.f) + sg[j][e];
              column[cols + c] = (w ? column[cols + c] : 0.f) + sb[j][e];
            }
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * cols; c += kThreads) part[c] = column[c];
  }
}

// Adds the blocks' rows: eight warps each a stretch of them, in order, then the eight in order.
__global__ void __launch_bounds__(256) k_ln_bwd_join(const float* part, int parts, int64_t cols, float* dgamma,
                                                     float* dbeta) {
  __shared__ float sum[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  part += (blockIdx.y ? cols : 0) + c;
  const int each = (parts + 7) / 8;
  float s = 0.f;
  if (c < cols)
    for (int i = warp * each; i < min(parts, (warp + 1) * each); ++i) s += part[(int64_t)i * 2 * cols];
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
    for (int w = 1; w < 8; ++w) s += sum[w][lane];
    out[c] = s;
  }
}

int rows_a_block(int64_t cols, int e) { return (cols + e - 1) / e <= 128 ? 8 : 1; }

int parts_of(const ln_bwd_params_t& p) {
  const int each = rows_a_block(p.cols, p.dtype == ATTN_BF16 ? 8 : 4);
  return (int)std::min<int64_t>((p.rows + each - 1) / each, kMaxParts);
}

template <class T, int kThreads, int kRow, int kVpt>
void launch_rows(const BwdLnArgs& a, bool drops, int blocks, cudaStream_t st) {
  const size_t smem = kRow == kThreads || !a.part ? 0 : 2 * a.p.cols * sizeof(float);
  if (drops)
    k_ln_bwd<T, kThreads, kRow, kVpt, true><<<blocks, kThreads, smem, st>>>(a);
  else
    k_ln_bwd<T, kThreads, kRow, kVpt, false><<<blocks, kThreads, smem, st>>>(a);
}

template <class T>
void launch_bwd(const BwdLnArgs& a, bool drops, cudaStream_t st) {
  const int64_t n = (a.p.cols + Vec<T>::E - 1) / Vec<T>::E;
  const int blocks = parts_of(a.p);
  if (n <= 32) return launch_rows<T, 256, 32, 1>(a, drops, blocks, st);
  if (n <= 64) return launch_rows<T, 256, 32, 2>(a, drops, blocks, st);
  if (n <= 128) return launch_rows<T, 256, 32, 4>(a, drops, blocks, st);
  if (n <= 256) return launch_rows<T, 256, 256, 1>(a, drops, blocks, st);
  if (n <= 512) return launch_rows<T, 256, 256, 2>(a, drops, blocks, st);
  if (n <= 1024) return launch_rows<T, 512, 512, 2>(a, drops, blocks, st);
  if (n <= 2048) return launch_rows<T, 512, 512, 4>(a, drops, blocks, st);
  if constexpr (Vec<T>::E == 4) launch_rows<T, 512, 512, 8>(a, drops, blocks, st);
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

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" {

size_t ln_residual_bwd_workspace_size(const ln_bwd_params_t* p) {
  if (check_params(p) != ATTN_OK) return SIZE_MAX;
  return (size_t)parts_of(*p) * 2 * (size_t)p->cols * sizeof(float);
}

attn_status_t ln_residual_bwd(const ln_bwd_params_t* p, const ln_dropout_t* d, const void* dy, const void* dh,
                              const void* h, const float* mean, const float* rstd, const float* gamma, void* dx,
                              void* dr, float* dgamma, float* dbeta, void* workspace, size_t workspace_bytes,
                              void* stream) {
  attn_status_t s = check_params(p);
  if (s != ATTN_OK) return s;
  BwdLnArgs a{*p, dy, dh, h, mean, rstd, gamma, dx, dr, nullptr, 0, {}};
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
  a.vec = (at & 15) == 0;
  a.part = weights ? static_cast<float*>(workspace) : nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p->rows > 0) {
    if (p->dtype == ATTN_BF16)
      launch_bwd<__nv_bfloat16>(a, drops, st);
    else
      launch_bwd<float>(a, drops, st);
  }
  if (weights) {
    const dim3 grid((unsigned)((p->cols + 31) / 32), 2);
    k_ln_bwd_join<<<grid, 256, 0, st>>>(a.part, parts_of(*p), p->cols, dgamma, dbeta);
  }
  if (cudaGetLastError() != cudaSuccess) return bfail(ATTN_ERR_CUDA, "ln_residual_bwd: launch failed");
  return ATTN_OK;
}

}  // extern "C"
