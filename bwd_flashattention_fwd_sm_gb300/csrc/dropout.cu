// Dropout of a [rows, cols] tensor, and of its gradient (include/gbln.h has the definition).
//
// Bound by device memory: an element is read and written once, the mask is computed
// (dropout.cuh).  The mask's unit is a group of eight columns.  Rows of whole groups at aligned
// addresses: a thread takes a few groups at a time as 16-byte vectors.  Others: a warp takes
// 32 groups of a row, each lane makes the mask of one and then deals with every 32nd element, so
// that loads and stores stay in line; the masks change hands through shared memory.
// Short rows of that kind: a thread takes a group alone, element by element.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gbln.h"
#include "common.cuh"
#include "dropout.cuh"
#include "overlap.h"
#include "rowvec.cuh"

namespace gbattn {
void set_last_error_text(const char* text);
attn_status_t device_status(int** status, int* sms, unsigned long long* wait_ns);

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct DropoutArgs {
  const void* x;
  void* y;
  int64_t rows, cols;
  int64_t x_stride, y_stride;
  uint32_t units;                // of a row: groups, or pieces of 32 groups
  uint32_t row_step, unit_step;  // all units that the grid takes at once, as rows and units of a row
  DropArgs drop;
};

// A place among rows * units places, and the place a fixed number of them on.
struct Place {
  uint64_t row;
  uint32_t unit;
  __device__ Place(const DropoutArgs& a, uint64_t first) : row(first / a.units), unit((uint32_t)(first % a.units)) {}
  __device__ void advance(const DropoutArgs& a) {
    row += a.row_step;
    unit += a.unit_step;
    if (unit >= a.units) unit -= a.units, ++row;
  }
};

// Whole groups, kAtOnce of a thread in flight.
template <class T, int kAtOnce>
__global__ void __launch_bounds__(kThreads) k_dropout(const DropoutArgs a) {
  constexpr int E = Vec<T>::E, P = E / 2, V = 8 / E;  // V vectors of a group
  const DropKey key = drop_key(a.drop);
  const DropRate rate = drop_rate(a.drop);
  const float2 factor = make_float2(rate.factor, rate.factor);
  const uint4* X = static_cast<const uint4*>(a.x);
  uint4* Y = static_cast<uint4*>(a.y);
  const int64_t xs = a.x_stride / E, ys = a.y_stride / E;
  Place at(a, (uint64_t)blockIdx.x * kThreads + threadIdx.x);
  while (at.row < (uint64_t)a.rows) {
    uint4 v[kAtOnce][V];
    Place from = at;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (at.row < (uint64_t)a.rows) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = X[at.row * xs + (uint64_t)at.unit * V + j];
      }
      at.advance(a);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (from.row < (uint64_t)a.rows) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float2 w[P];
          Vec<T>::pairs(drop_mask<T>(v[i][j], from.unit * 8 + j * E, (uint32_t)from.row, key, rate), w);
#pragma unroll
          for (int e = 0; e < P; ++e) w[e] = pair_mul(w[e], factor);
          Y[from.row * ys + (uint64_t)from.unit * V + j] = Vec<T>::pack(w);
        }
      }
      from.advance(a);
    }
  }
}

__device__ __forceinline__ uint4 compared(const DropoutArgs& a, uint64_t group, uint64_t row, const DropKey& key,
                                          const DropRate& rate) {
  const uint4 b = drop_bits(key, (uint32_t)group, (uint32_t)row);
  return make_uint4(drop_compare(b.x, rate), drop_compare(b.y, rate), drop_compare(b.z, rate), drop_compare(b.w, rate));
}

// Any rows: a warp takes 32 groups of a row.
template <class T>
__global__ void __launch_bounds__(kThreads) k_dropout_any(const DropoutArgs a) {
  __shared__ uint4 mask[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const DropKey key = drop_key(a.drop);
  const DropRate rate = drop_rate(a.drop);
  const uint16_t* bit = reinterpret_cast<const uint16_t*>(mask[warp]);
  for (Place at(a, (uint64_t)blockIdx.x * kWarps + warp); at.row < (uint64_t)a.rows; at.advance(a)) {
    const int64_t c0 = (int64_t)at.unit * 256 + lane;
    const T* x = static_cast<const T*>(a.x) + at.row * a.x_stride + c0;
    T* y = static_cast<T*>(a.y) + at.row * a.y_stride + c0;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c0 + 32 * i < a.cols ? Vec<T>::load1(x + 32 * i) : 0.f;
    mask[warp][lane] = compared(a, (uint64_t)at.unit * 32 + lane, at.row, key, rate);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + 32 * i < a.cols) Vec<T>::store1(y + 32 * i, bit[32 * i + lane] >> 15 ? v[i] * rate.factor : 0.f);
    __syncwarp();
  }
}

// Short rows: a thread takes a group.
template <class T>
__global__ void __launch_bounds__(kThreads) k_dropout_short(const DropoutArgs a) {
  const DropKey key = drop_key(a.drop);
  const DropRate rate = drop_rate(a.drop);
  for (Place at(a, (uint64_t)blockIdx.x * kThreads + threadIdx.x); at.row < (uint64_t)a.rows; at.advance(a)) {
    const int left = (int)a.cols - (int)at.unit * 8;
    const T* x = static_cast<const T*>(a.x) + at.row * a.x_stride + at.unit * 8;
    T* y = static_cast<T*>(a.y) + at.row * a.y_stride + at.unit * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? Vec<T>::load1(x + e) : 0.f;
    const uint4 c = compared(a, at.unit, at.row, key, rate);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) Vec<T>::store1(y + e, (w[e / 2] << (e & 1 ? 0 : 16)) >> 31 ? v[e] * rate.factor : 0.f);
  }
}

// Rows of fewer groups go to k_dropout_short where they are no whole vectors.
constexpr int64_t kShort = 16;

// One wave of blocks at most, each taking `a_block` places at a time.
template <class K>
cudaError_t launch_places(K kernel, DropoutArgs a, int a_block, int sms, cudaStream_t st) {
  int per_sm = 1;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, 0);
  if (e != cudaSuccess) return e;
  // rows * units may pass 63 bits: any grid is small beside such a number
  const double all = (double)a.rows * a.units;
  const int64_t want = all > 1e12 ? INT64_MAX : (a.rows * a.units + a_block - 1) / a_block;
  const int64_t blocks = std::min<int64_t>(want, (int64_t)sms * std::max(per_sm, 1));
  a.row_step = (uint32_t)(blocks * a_block / a.units), a.unit_step = (uint32_t)(blocks * a_block % a.units);
  kernel<<<(unsigned)blocks, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <class T>
cudaError_t launch_dropout(DropoutArgs a, bool whole, int sms, cudaStream_t st) {
  const int64_t groups = (a.cols + 7) / 8;
  a.units = (uint32_t)groups;
  if (whole) return launch_places(k_dropout<T, 4 * (int)sizeof(__nv_bfloat16) / (int)sizeof(T)>, a, kThreads, sms, st);
  if (groups < kShort) return launch_places(k_dropout_short<T>, a, kThreads, sms, st);
  a.units = (uint32_t)((groups + 31) / 32);
  return launch_places(k_dropout_any<T>, a, kWarps, sms, st);
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
  const int64_t width = p->cols * (int64_t)esize;
  const RowSpan from{x, p->rows, p->x_stride * (int64_t)esize, width}, to{y, p->rows, p->y_stride * (int64_t)esize, width};
  if (rows_meet(from, to) && !same_rows(from, to))
    return dfail(ATTN_ERR_INVALID_ARG, "ln_dropout: x and y overlap and are not the same rows");
  const bool whole =
      p->cols % 8 == 0 && ((at | (uintptr_t)p->x_stride * esize | (uintptr_t)p->y_stride * esize) & 15) == 0;
  a.x = x, a.y = y;
  a.rows = p->rows, a.cols = p->cols;
  a.x_stride = p->x_stride, a.y_stride = p->y_stride;
  int* status = nullptr;
  int sms = 0;
  unsigned long long wait_ns = 0;
  attn_status_t ds = device_status(&status, &sms, &wait_ns);
  if (ds != ATTN_OK) return ds;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p->dtype == ATTN_BF16 ? launch_dropout<__nv_bfloat16>(a, whole, sms, st)
                                              : launch_dropout<float>(a, whole, sms, st);
  return e == cudaSuccess ? ATTN_OK : dfail(ATTN_ERR_CUDA, "ln_dropout: launch failed");
}
