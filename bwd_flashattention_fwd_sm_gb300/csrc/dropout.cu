// Dropout of a [rows, cols] tensor, and of its gradient (include/gbln.h has the definition).
//
// Bound by device memory: an element is read and written once, the mask is computed
// (dropout.cuh).  A thread takes groups of eight columns, the unit of the mask, two at
// a time so that its loads overlap.
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

constexpr int kThreads = 256;
constexpr int kAtOnce = 2;  // groups of a thread in flight

struct DropoutArgs {
  const void* x;
  void* y;
  int64_t rows, cols, groups;  // groups of eight columns in a row
  int64_t x_stride, y_stride;
  int64_t row_step, group_step;  // kThreads * blocks groups on, as rows and groups of a row
  int vec;
  DropArgs drop;
};

template <class T>
__global__ void __launch_bounds__(kThreads) k_dropout(const DropoutArgs a) {
  constexpr int V = 8 / Vec<T>::E;  // 16-byte vectors of a group
  const DropKey key = drop_key(a.drop);
  const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  int64_t row = first / a.groups, group = first % a.groups;
  const T* X = static_cast<const T*>(a.x);
  T* Y = static_cast<T*>(a.y);
  while (row < a.rows) {
    int64_t rows[kAtOnce], groups[kAtOnce];
    float v[kAtOnce][8];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      rows[i] = row, groups[i] = group;
      if (row < a.rows) {
        const T* x = X + row * a.x_stride + group * 8;
        if (a.vec && group * 8 + 8 <= a.cols) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            float w[Vec<T>::E];
            Vec<T>::load(x + j * Vec<T>::E, w);
#pragma unroll
            for (int e = 0; e < Vec<T>::E; ++e) v[i][j * Vec<T>::E + e] = w[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = group * 8 + e < a.cols ? Vec<T>::load1(x + e) : 0.f;
        }
      }
      row += a.row_step, group += a.group_step;
      if (group >= a.groups) group -= a.groups, ++row;
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (rows[i] >= a.rows) continue;
      drop_vector<8>(a.drop, key, groups[i] * 8, rows[i], v[i]);
      T* y = Y + rows[i] * a.y_stride + groups[i] * 8;
      if (a.vec && groups[i] * 8 + 8 <= a.cols) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float w[Vec<T>::E];
#pragma unroll
          for (int e = 0; e < Vec<T>::E; ++e) w[e] = v[i][j * Vec<T>::E + e];
          Vec<T>::store(y + j * Vec<T>::E, w);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (groups[i] * 8 + e < a.cols) Vec<T>::store1(y + e, v[i][e]);
      }
    }
  }
}

attn_status_t dfail(attn_status_t s, const char* msg) {
  set_last_error_text(msg);
  return s;
}

}  // namespace
}  // namespace gbattn

extern "C" attn_status_t ln_dropout(const ln_params_t* p, const ln_dropout_t* d, const void* x, void* y, void* stream) {
  using namespace gbattn;
  if (!p || !d) return dfail(ATTN_ERR_INVALID_ARG, "ln_dropout: params or dropout is NULL");
  if (p->dtype != ATTN_BF16 && p->dtype != ATTN_F32)
    return dfail(ATTN_ERR_INVALID_ARG, "ln_dropout: dtype is not ATTN_F32 or ATTN_BF16");
  if (p->rows < 0 || p->cols < 0) return dfail(ATTN_ERR_INVALID_ARG, "ln_dropout: rows < 0 or cols < 0");
  const int64_t most = (int64_t)1 << 32;
  if (p->rows >= most || p->cols >= most) return dfail(ATTN_ERR_UNSUPPORTED, "ln_dropout: 2^32 rows or columns or more");
  DropoutArgs a{};
  bool drops = false;
  if (const char* wrong = resolve_dropout(d, &a.drop, &drops)) return dfail(ATTN_ERR_INVALID_ARG, wrong);
  if (p->rows == 0 || p->cols == 0) return ATTN_OK;
  if (p->x_stride < p->cols || p->y_stride < p->cols)
    return dfail(ATTN_ERR_INVALID_ARG, "ln_dropout: a row stride is below cols");
  if (!x || !y) return dfail(ATTN_ERR_INVALID_ARG, "ln_dropout: x or y is NULL");
  const uintptr_t esize = p->dtype == ATTN_BF16 ? 2 : 4;
  const uintptr_t at = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y);
  if (at & (esize - 1)) return dfail(ATTN_ERR_INVALID_ARG, "ln_dropout: a pointer is not aligned to its element size");
  a.vec = ((at | (uintptr_t)p->x_stride * esize | (uintptr_t)p->y_stride * esize) & 15) == 0;
  a.x = x, a.y = y;
  a.rows = p->rows, a.cols = p->cols, a.groups = (p->cols + 7) / 8;
  a.x_stride = p->x_stride, a.y_stride = p->y_stride;
  int* status = nullptr;
  int sms = 0;
  unsigned long long wait_ns = 0;
  attn_status_t ds = device_status(&status, &sms, &wait_ns);
  if (ds != ATTN_OK) return ds;
  // rows * groups passes 63 bits at the extreme sizes: count blocks in floating point there
  const double total = (double)a.rows * (double)a.groups;
  const int64_t want = total > 1e12 ? INT64_MAX : (a.rows * a.groups + kThreads - 1) / kThreads;
  const int64_t blocks = std::min<int64_t>(want, (int64_t)sms * 8);
  const int64_t step = blocks * kThreads;
  a.row_step = step / a.groups, a.group_step = step % a.groups;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p->dtype == ATTN_BF16)
    k_dropout<__nv_bfloat16><<<(int)blocks, kThreads, 0, st>>>(a);
  else
    k_dropout<float><<<(int)blocks, kThreads, 0, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return dfail(ATTN_ERR_CUDA, "ln_dropout: launch failed");
  return ATTN_OK;
}
