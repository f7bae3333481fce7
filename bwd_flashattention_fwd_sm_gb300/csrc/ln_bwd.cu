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
#include "ptx.cuh"
#include "rowvec.cuh"

namespace gbattn {
void set_last_error_text(const char* text);
attn_status_t device_status(int** status, int* sms, unsigned long long* wait_ns);

namespace {

// Rows of partial sums at most, blocks on each of 152 SMs.  Constants, so that the size of
// the workspace and the order of the sums are the same everywhere.
constexpr int kSms = 152;
constexpr int kMaxParts = 4 * kSms;

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

// A longer row that is no whole vectors, or not at aligned addresses, or too long for the
// ring: a block, kVpt vectors a thread.  Where the registers do not hold a row it is read again
// (from the caches) once its sums are known.
template <class T, int kThreads, int kVpt, bool kDrop>
__global__ void __launch_bounds__(kThreads) k_ln_bwd(const BwdLnArgs a) {
  constexpr int E = Vec<T>::E, kWarps = kThreads / 32;
  constexpr bool kHold = kVpt * E <= 16;
  constexpr int H = kHold ? kVpt : 1;
  __shared__ float2 warp_sum[2][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t cols = a.p.cols;
  const float inv = 1.f / (float)cols;
  DropKey key{};
  DropRate rate{};
  if constexpr (kDrop) key = drop_key(a.drop), rate = drop_rate(a.drop);
  float sg[kVpt][E], sb[kVpt][E];
#pragma unroll
  for (int j = 0; j < kVpt; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) sg[j][e] = sb[j][e] = 0.f;
  int phase = 0;
  for (int64_t row = blockIdx.x; row < a.p.rows; row += gridDim.x, phase ^= 1) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.p.dy_stride;
    const T* h = static_cast<const T*>(a.h) + row * a.p.h_stride;
    const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.p.dh_stride : nullptr;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float g[H][E], xh[H][E], in[H][E];
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      const int64_t c0 = (int64_t)(tid + j * kThreads) * E;
      if (c0 >= cols) continue;
      float (&gj)[E] = g[kHold ? j : 0], (&xj)[E] = xh[kHold ? j : 0];
      load_cols<T>(dy, c0, cols, a.vec, gj);
      load_cols<T>(h, c0, cols, a.vec, xj);
      if (kHold) {
        if (dh) load_cols<T>(dh, c0, cols, a.vec, in[kHold ? j : 0]);
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!dh) in[kHold ? j : 0][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (c0 + e < cols) {  // a row's end inside a vector
          xj[e] = (xj[e] - mean) * rstd;
          sg[j][e] += gj[e] * xj[e];
          sb[j][e] += gj[e];
          if (a.gamma) gj[e] *= __ldg(a.gamma + c0 + e);
          s0 += gj[e];
          s1 += gj[e] * xj[e];
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, o);
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    }
    if (lane == 0) warp_sum[phase][warp] = make_float2(s0, s1);
    __syncthreads();  // the other phase's sums are read before the next barrier, and written after it
    s0 = s1 = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 t = warp_sum[phase][w];
      s0 += t.x;
      s1 += t.y;
    }
    s0 *= inv;
    s1 *= inv;
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      const int64_t c0 = (int64_t)(tid + j * kThreads) * E;
      if (c0 >= cols) continue;
      float (&gj)[E] = g[kHold ? j : 0], (&xj)[E] = xh[kHold ? j : 0], (&ij)[E] = in[kHold ? j : 0];
      if (!kHold) {
        load_cols<T>(dy, c0, cols, a.vec, gj);
        load_cols<T>(h, c0, cols, a.vec, xj);
        if (dh) load_cols<T>(dh, c0, cols, a.vec, ij);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (!dh) ij[e] = 0.f;
          xj[e] = (xj[e] - mean) * rstd;
          if (a.gamma && c0 + e < cols) gj[e] *= __ldg(a.gamma + c0 + e);
        }
      }
      float d[E];
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = ij[e] + rstd * (gj[e] - s0 - xj[e] * s1);
      if (a.dr) store_cols<T>(static_cast<T*>(a.dr) + row * a.p.dr_stride, c0, cols, a.vec, d);
      if (a.dx) {
        if constexpr (kDrop) {
#pragma unroll
          for (int e = 0; e < E; ++e) d[e] *= rate.factor;
          Vec<T>::unpack(drop_mask<T>(Vec<T>::pack(d), (uint32_t)c0, (uint32_t)row, key, rate), d);
        }
        store_cols<T>(static_cast<T*>(a.dx) + row * a.p.dx_stride, c0, cols, a.vec, d);
      }
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
  for (int j = 0; j < kVpt; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t c = (int64_t)(tid + j * kThreads) * E + e;
      if (c < cols) part[c] = sg[j][e], part[cols + c] = sb[j][e];
    }
}

// A short row: kRow lanes of a warp, kVpt vectors each.  The next row's vectors come in while
// this one's sums are joined.  kWhole: rows are whole vectors at aligned addresses.
template <class T, int kRow, int kVpt, bool kDrop, bool kWhole>
__global__ void __launch_bounds__(512) k_ln_bwd_warp(const BwdLnArgs a) {
  constexpr int E = Vec<T>::E, P = E / 2;
  extern __shared__ float column[];  // [2][cols]
  const int lane = threadIdx.x % kRow, groups = blockDim.x / kRow;
  const int cols = (int)a.p.cols;
  const float inv = 1.f / (float)cols;
  DropKey key{};
  DropRate rate{};
  if constexpr (kDrop) key = drop_key(a.drop), rate = drop_rate(a.drop);
  float2 sg[kVpt][P], sb[kVpt][P], gamma[kVpt][P];
#pragma unroll
  for (int j = 0; j < kVpt; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) {
      sg[j][i] = sb[j][i] = make_float2(0.f, 0.f);
      const int c = (lane + j * kRow) * E + 2 * i;
      gamma[j][i] = make_float2(a.gamma && c < cols ? a.gamma[c] : 1.f, a.gamma && c + 1 < cols ? a.gamma[c + 1] : 1.f);
    }
  const T* DY = static_cast<const T*>(a.dy);
  const T* H = static_cast<const T*>(a.h);
  const T* DH = static_cast<const T*>(a.dh);
  const int64_t step = (int64_t)gridDim.x * groups;
  // every lane of a warp takes the same number of turns: a row behind the last is one of zeros
  const int64_t first = (int64_t)blockIdx.x * groups + threadIdx.x / kRow;
  const int64_t turns = (a.p.rows - ((int64_t)blockIdx.x * groups + (threadIdx.x & ~31) / kRow) + step - 1) / step;
  uint4 dy[kVpt], h[kVpt], dh[kVpt];
  float mean = 0.f, rstd = 0.f;
  auto vector = [&](const T* row, int c0) -> uint4 {
    if (kWhole || (a.vec && c0 + E <= cols)) return *reinterpret_cast<const uint4*>(row + c0);
    float2 v[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      v[i].x = c0 + 2 * i < cols ? Vec<T>::load1(row + c0 + 2 * i) : 0.f;
      v[i].y = c0 + 2 * i + 1 < cols ? Vec<T>::load1(row + c0 + 2 * i + 1) : 0.f;
    }
    return Vec<T>::pack(v);
  };
  auto fetch = [&](int64_t row) {
    const bool there = row < a.p.rows;
    mean = there ? a.mean[row] : 0.f, rstd = there ? a.rstd[row] : 0.f;
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      const int c0 = (lane + j * kRow) * E;
      dy[j] = h[j] = dh[j] = make_uint4(0u, 0u, 0u, 0u);
      if (there && c0 < cols) {
        dy[j] = vector(DY + row * a.p.dy_stride, c0);
        h[j] = vector(H + row * a.p.h_stride, c0);
        if (DH) dh[j] = vector(DH + row * a.p.dh_stride, c0);
      }
    }
  };
  fetch(first);
  int64_t row = first;
  for (int64_t t = 0; t < turns; ++t, row += step) {
    float2 g[kVpt][P], xh[kVpt][P];
    uint4 in[kVpt];
    float2 s0 = make_float2(0.f, 0.f), s1 = s0;
    const float scale = rstd;
    const float2 shift2 = make_float2(-mean, -mean), scale2 = make_float2(rstd, rstd);
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      const int c0 = (lane + j * kRow) * E;
      Vec<T>::pairs(dy[j], g[j]);
      Vec<T>::pairs(h[j], xh[j]);
      in[j] = dh[j];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        xh[j][i] = pair_mul(pair_add(xh[j][i], shift2), scale2);
        if (!kWhole) {  // behind the row's end: dy is 0 there, but h - mean is not
          if (c0 + 2 * i >= cols) xh[j][i].x = 0.f;
          if (c0 + 2 * i + 1 >= cols) xh[j][i].y = 0.f;
        }
        sg[j][i] = pair_fma(g[j][i], xh[j][i], sg[j][i]);
        sb[j][i] = pair_add(g[j][i], sb[j][i]);
        g[j][i] = pair_mul(g[j][i], gamma[j][i]);
        s0 = pair_add(g[j][i], s0);
        s1 = pair_fma(g[j][i], xh[j][i], s1);
      }
    }
    fetch(t + 1 < turns ? row + step : a.p.rows);
    float m0 = s0.x + s0.y, m1 = s1.x + s1.y;
#pragma unroll
    for (int o = kRow / 2; o > 0; o >>= 1) {
      m0 += __shfl_xor_sync(0xffffffffu, m0, o);
      m1 += __shfl_xor_sync(0xffffffffu, m1, o);
    }
    if (row >= a.p.rows) continue;
    const float2 n0 = make_float2(-m0 * inv, -m0 * inv), n1 = make_float2(-m1 * inv, -m1 * inv);
    const float2 r2 = make_float2(scale, scale);
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      const int c0 = (lane + j * kRow) * E;
      if (c0 >= cols) continue;
      float2 d[P];
      Vec<T>::pairs(in[j], d);
#pragma unroll
      for (int i = 0; i < P; ++i) d[i] = pair_fma(pair_fma(xh[j][i], n1, pair_add(g[j][i], n0)), r2, d[i]);
      auto store = [&](void* base, int64_t stride, uint4 v) {
        T* out = static_cast<T*>(base) + row * stride + c0;
        if (kWhole || (a.vec && c0 + E <= cols)) {
          *reinterpret_cast<uint4*>(out) = v;
        } else {
          Vec<T>::pairs(v, d);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            if (c0 + 2 * i < cols) Vec<T>::store1(out + 2 * i, d[i].x);
            if (c0 + 2 * i + 1 < cols) Vec<T>::store1(out + 2 * i + 1, d[i].y);
          }
        }
      };
      uint4 dx = Vec<T>::pack(d);
      const uint4 dr = dx;
      if constexpr (kDrop) {  // of the unrounded dr
#pragma unroll
        for (int i = 0; i < P; ++i) d[i] = pair_mul(d[i], make_float2(rate.factor, rate.factor));
        dx = drop_mask<T>(Vec<T>::pack(d), (uint32_t)c0, (uint32_t)row, key, rate);
      }
      if (a.dr) store(a.dr, a.p.dr_stride, dr);
      if (a.dx) store(a.dx, a.p.dx_stride, dx);
    }
  }
  if (!a.part) return;
  // the groups of lanes that share a warp, then the block's warps one after the other
  if constexpr (kRow < 32) {
#pragma unroll
    for (int j = 0; j < kVpt; ++j)
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int o = kRow; o < 32; o <<= 1) {
          sg[j][i].x += __shfl_xor_sync(0xffffffffu, sg[j][i].x, o);
          sg[j][i].y += __shfl_xor_sync(0xffffffffu, sg[j][i].y, o);
          sb[j][i].x += __shfl_xor_sync(0xffffffffu, sb[j][i].x, o);
          sb[j][i].y += __shfl_xor_sync(0xffffffffu, sb[j][i].y, o);
        }
  }
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int w = 0; w < warps; ++w) {
    if (warp == w && (threadIdx.x & 31) < kRow) {
#pragma unroll
      for (int j = 0; j < kVpt; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int c = (lane + j * kRow) * E + 2 * i;
          if (c < cols) {
            column[c] = (w ? column[c] : 0.f) + sg[j][i].x;
            column[cols + c] = (w ? column[cols + c] : 0.f) + sb[j][i].x;
          }
          if (c + 1 < cols) {
            column[c + 1] = (w ? column[c + 1] : 0.f) + sg[j][i].y;
            column[cols + c + 1] = (w ? column[cols + c + 1] : 0.f) + sb[j][i].y;
          }
        }
    }
    __syncthreads();
  }
  float* part = a.part + (int64_t)blockIdx.x * 2 * cols;
  for (int c = threadIdx.x; c < 2 * cols; c += blockDim.x) part[c] = column[c];
}

// A longer row of whole vectors: a block, kVpt vectors a thread.  Rows stream through a ring of
// stages in shared memory that bulk copies fill some rows ahead, so that the block's one
// barrier a row does not stop the loads.  A stage is read twice (for the sums, then for
// dr), which leaves the registers to the columns' sums.  Waits are bounded: a block that gives up
// records ATTN_ERR_DEVICE_TIMEOUT, waits (bounded) for its own copies and returns.
constexpr int kMaxStages = 8;

template <class T, int kThreads, int kVpt, int kBlocks, bool kDrop>
__global__ void __launch_bounds__(kThreads, kBlocks)
    k_ln_bwd_ring(const BwdLnArgs a, int stages, int* status, unsigned long long wait_ns) {
  constexpr int E = Vec<T>::E, P = E / 2, kWarps = kThreads / 32;
  constexpr bool kKeepGamma = kVpt * E <= 16;  // registers allow it
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxStages];
  __shared__ float warp_sum[2][2][kWarps];
  __shared__ ptx::Abort abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cols = (int)a.p.cols, n = cols / E;
  const float inv = 1.f / (float)cols;
  const uint32_t row_bytes = (uint32_t)cols * sizeof(T);
  const bool has_dh = a.dh != nullptr;
  const uint32_t stage_bytes = row_bytes * (has_dh ? 3 : 2);
  const T* DY = static_cast<const T*>(a.dy);
  const T* H = static_cast<const T*>(a.h);
  const T* DH = static_cast<const T*>(a.dh);
  auto issue = [&](int s, int64_t row) {  // thread 0 only
    uint8_t* to = ring + (size_t)s * stage_bytes;
    ptx::mbar_arrive_expect_tx(&full[s], stage_bytes);
    ptx::bulk_load(to, DY + row * a.p.dy_stride, row_bytes, &full[s]);
    ptx::bulk_load(to + row_bytes, H + row * a.p.h_stride, row_bytes, &full[s]);
    if (has_dh) ptx::bulk_load(to + 2 * row_bytes, DH + row * a.p.dh_stride, row_bytes, &full[s]);
  };
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) ptx::mbar_init(&full[s], 1);
    abort.flag = 0;
    ptx::fence_mbar_init();
    for (int s = 0; s < stages; ++s) {
      const int64_t row = blockIdx.x + (int64_t)s * gridDim.x;
      if (row < a.p.rows) issue(s, row);
    }
  }
  DropKey key{};
  DropRate rate{};
  if constexpr (kDrop) key = drop_key(a.drop), rate = drop_rate(a.drop);
  float2 sg[kVpt][P], sb[kVpt][P], keep[kKeepGamma ? kVpt : 1][P];
  auto gamma_at = [&](int j, float2 (&g)[P]) {
    const int c0 = (tid + j * kThreads) * E;
#pragma unroll
    for (int i = 0; i < P; i += 2) {
      const float4 v = a.gamma ? __ldg(reinterpret_cast<const float4*>(a.gamma + c0 + 2 * i))
                               : make_float4(1.f, 1.f, 1.f, 1.f);
      g[i] = make_float2(v.x, v.y), g[i + 1] = make_float2(v.z, v.w);
    }
  };
#pragma unroll
  for (int j = 0; j < kVpt; ++j) {
#pragma unroll
    for (int i = 0; i < P; ++i) sg[j][i] = sb[j][i] = make_float2(0.f, 0.f);
    if (kKeepGamma && tid + j * kThreads < n) gamma_at(j, keep[j]);
  }
  float mean = 0.f, rstd = 0.f;
  if (blockIdx.x < a.p.rows) mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
  __syncthreads();
  int64_t it = 0;
  int s = 0, last = 0;        // this row's stage, and the one before
  uint32_t phase = 0;
  bool ok = true;
  for (int64_t row = blockIdx.x; row < a.p.rows; row += gridDim.x, ++it) {
    const bool mine = ptx::mbar_wait(&full[s], phase, &abort, status, wait_ns);
    const uint4* dy = reinterpret_cast<const uint4*>(ring + (size_t)s * stage_bytes);
    const uint4* h = reinterpret_cast<const uint4*>(ring + (size_t)s * stage_bytes + row_bytes);
    const uint4* dh = reinterpret_cast<const uint4*>(ring + (size_t)s * stage_bytes + 2 * row_bytes);
    const float2 shift2 = make_float2(-mean, -mean), scale2 = make_float2(rstd, rstd);
    const int64_t next = row + gridDim.x;
    if (next < a.p.rows) mean = a.mean[next], rstd = a.rstd[next];
    float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      if (tid + j * kThreads >= n) continue;
      float2 g[P], xh[P], w[P];
      Vec<T>::pairs(dy[tid + j * kThreads], g);
      Vec<T>::pairs(h[tid + j * kThreads], xh);
      if (!kKeepGamma) gamma_at(j, w);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        xh[i] = pair_mul(pair_add(xh[i], shift2), scale2);
        sg[j][i] = pair_fma(g[i], xh[i], sg[j][i]);
        sb[j][i] = pair_add(g[i], sb[j][i]);
        g[i] = pair_mul(g[i], kKeepGamma ? keep[kKeepGamma ? j : 0][i] : w[i]);
        s0 = pair_add(g[i], s0);
        s1 = pair_fma(g[i], xh[i], s1);
      }
    }
    // both sums at once: the lower half of the warp joins the first, the upper the second
    const float x0 = s0.x + s0.y, x1 = s1.x + s1.y;
    float m = lane < 16 ? x0 : x1;
    m += __shfl_xor_sync(0xffffffffu, lane < 16 ? x1 : x0, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    if ((lane & 15) == 0) warp_sum[it & 1][lane >> 4][warp] = m;
    // the barrier also says that every warp is done with the last row's stage
    if (__syncthreads_or(!mine)) { ok = false; break; }
    if (tid == 0 && it > 0) {
      const int64_t ahead = row + (int64_t)(stages - 1) * gridDim.x;
      if (ahead < a.p.rows) issue(last, ahead);
    }
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m0 += warp_sum[it & 1][0][w], m1 += warp_sum[it & 1][1][w];
    const float2 n0 = make_float2(-m0 * inv, -m0 * inv), n1 = make_float2(-m1 * inv, -m1 * inv);
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      if (tid + j * kThreads >= n) continue;
      const int c0 = (tid + j * kThreads) * E;
      float2 g[P], xh[P], d[P], w[P];
      Vec<T>::pairs(dy[tid + j * kThreads], g);
      Vec<T>::pairs(h[tid + j * kThreads], xh);
      if (has_dh) {
        Vec<T>::pairs(dh[tid + j * kThreads], d);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) d[i] = make_float2(0.f, 0.f);
      }
      if (!kKeepGamma) gamma_at(j, w);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        xh[i] = pair_mul(pair_add(xh[i], shift2), scale2);
        g[i] = pair_fma(g[i], kKeepGamma ? keep[kKeepGamma ? j : 0][i] : w[i], n0);
        d[i] = pair_fma(pair_fma(xh[i], n1, g[i]), scale2, d[i]);
      }
      uint4 dx = Vec<T>::pack(d);
      if (a.dr) *reinterpret_cast<uint4*>(static_cast<T*>(a.dr) + row * a.p.dr_stride + c0) = dx;
      if (a.dx) {
        if constexpr (kDrop) {  // of the unrounded dr
#pragma unroll
          for (int i = 0; i < P; ++i) d[i] = pair_mul(d[i], make_float2(rate.factor, rate.factor));
          dx = drop_mask<T>(Vec<T>::pack(d), (uint32_t)c0, (uint32_t)row, key, rate);
        }
        *reinterpret_cast<uint4*>(static_cast<T*>(a.dx) + row * a.p.dx_stride + c0) = dx;
      }
    }
    last = s;
    if (++s == stages) s = 0, phase ^= 1;
  }
  if (!ok) {
    if (tid == 0) {  // copies that this block issued and did not wait for
      ptx::Abort none;
      none.flag = 0;
      for (int64_t j = it; j < it + stages - (it > 0 ? 1 : 0); ++j) {
        if (blockIdx.x + j * gridDim.x >= a.p.rows) break;
        ptx::mbar_wait(&full[j % stages], (uint32_t)((j / stages) & 1), &none, status, wait_ns);
      }
    }
    return;
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
  for (int j = 0; j < kVpt; ++j) {
    if (tid + j * kThreads >= n) continue;
    const int c0 = (tid + j * kThreads) * E;
#pragma unroll
    for (int i = 0; i < P; i += 2) {
      *reinterpret_cast<float4*>(part + c0 + 2 * i) =
          make_float4(sg[j][i].x, sg[j][i].y, sg[j][i + 1].x, sg[j][i + 1].y);
      *reinterpret_cast<float4*>(part + cols + c0 + 2 * i) =
          make_float4(sb[j][i].x, sb[j][i].y, sb[j][i + 1].x, sb[j][i + 1].y);
    }
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
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
  part += (blockIdx.y ? cols : 0) + c;
  const int each = (parts + 7) / 8;
  const int end = min(parts, (warp + 1) * each);
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int i = warp * each; i < end; ++i) s += part[(int64_t)i * 2 * cols];
  }
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
    for (int w = 1; w < 8; ++w) s += sum[w][lane];
    out[c] = s;
  }
}

// How a call is shared out: by sizes, types and alignment alone.
struct Plan {
  int threads, blocks;
};

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Rows of up to 64 vectors: a warp or eight lanes each.  As many warps a block as leave every
// SM a block, 16 at most.
Plan warp_plan(int64_t rows, int lanes) {
  int warps = 1;
  const int a_warp = 32 / lanes;
  while (warps < 16 && div_up(rows, (int64_t)warps * a_warp) > kSms) warps *= 2;
  return Plan{32 * warps, (int)std::min<int64_t>(div_up(rows, (int64_t)warps * a_warp), 2 * kSms)};
}

template <class T, int kRow, int kVpt>
cudaError_t launch_warp(const BwdLnArgs& a, bool drops, int* blocks, cudaStream_t st) {
  const Plan plan = warp_plan(a.p.rows, kRow);
  *blocks = plan.blocks;
  const size_t smem = a.part ? 2 * a.p.cols * sizeof(float) : 0;
  const bool whole = a.vec && a.p.cols % Vec<T>::E == 0;
  auto kernel = drops ? (whole ? k_ln_bwd_warp<T, kRow, kVpt, true, true> : k_ln_bwd_warp<T, kRow, kVpt, true, false>)
                      : (whole ? k_ln_bwd_warp<T, kRow, kVpt, false, true> : k_ln_bwd_warp<T, kRow, kVpt, false, false>);
  kernel<<<plan.blocks, plan.threads, smem, st>>>(a);
  return cudaGetLastError();
}

template <class T, int kThreads, int kVpt, int kBlocks>
cudaError_t launch_ring(const BwdLnArgs& a, bool drops, int stages, int* blocks, int* status,
                        unsigned long long wait_ns, cudaStream_t st) {
  *blocks = (int)std::min<int64_t>(a.p.rows, kBlocks * kSms);
  const size_t smem = (size_t)stages * a.p.cols * sizeof(T) * (a.dh ? 3 : 2);
  auto kernel = drops ? k_ln_bwd_ring<T, kThreads, kVpt, kBlocks, true> : k_ln_bwd_ring<T, kThreads, kVpt, kBlocks, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<*blocks, kThreads, smem, st>>>(a, stages, status, wait_ns);
  return cudaGetLastError();
}

template <class T, int kThreads, int kVpt>
cudaError_t launch_rows(const BwdLnArgs& a, bool drops, int* blocks, cudaStream_t st) {
  *blocks = (int)std::min<int64_t>(a.p.rows, 2 * kSms);
  if (drops)
    k_ln_bwd<T, kThreads, kVpt, true><<<*blocks, kThreads, 0, st>>>(a);
  else
    k_ln_bwd<T, kThreads, kVpt, false><<<*blocks, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <class T>
cudaError_t launch_bwd(const BwdLnArgs& a, bool drops, int* blocks, int* status, unsigned long long wait_ns,
                       cudaStream_t st) {
  const int64_t n = div_up(a.p.cols, Vec<T>::E);
  if (n <= 8) return launch_warp<T, 8, 1>(a, drops, blocks, st);
  if (n <= 32) return launch_warp<T, 32, 1>(a, drops, blocks, st);
  if (n <= 64) return launch_warp<T, 32, 2>(a, drops, blocks, st);
  if (a.vec && a.p.cols % Vec<T>::E == 0) {
    const int64_t stage = a.p.cols * sizeof(T) * (a.dh ? 3 : 2);
    // an SM's shared memory over its blocks, less what they hold beside the ring
    auto stages = [&](int per_sm) { return (int)std::min<int64_t>(kMaxStages, (224 * 1024 / per_sm - 1536) / stage); };
    if (n <= 128) return launch_ring<T, 128, 1, 4>(a, drops, stages(4), blocks, status, wait_ns, st);
    if (n <= 256) return launch_ring<T, 128, 2, 4>(a, drops, stages(4), blocks, status, wait_ns, st);
    if (n <= 512) return launch_ring<T, 256, 2, 2>(a, drops, stages(2), blocks, status, wait_ns, st);
    if (n <= 1024) return launch_ring<T, 512, 2, 1>(a, drops, stages(1), blocks, status, wait_ns, st);
    if (n <= 2048 && stages(1) >= 2)
      return launch_ring<T, 512, 4, 1>(a, drops, stages(1), blocks, status, wait_ns, st);
  }
  if (n <= 256) return launch_rows<T, 256, 1>(a, drops, blocks, st);
  if (n <= 512) return launch_rows<T, 256, 2>(a, drops, blocks, st);
  if (n <= 1024) return launch_rows<T, 512, 2>(a, drops, blocks, st);
  if (n <= 2048) return launch_rows<T, 512, 4>(a, drops, blocks, st);
  if constexpr (Vec<T>::E == 4) return launch_rows<T, 512, 8>(a, drops, blocks, st);
  return cudaErrorInvalidValue;
}

// The join may be set up while the first kernel runs.
cudaError_t launch_join(const BwdLnArgs& a, int parts, float* dgamma, float* dbeta, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)div_up(a.p.cols, 32), 2);
  cfg.blockDim = dim3(256);
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

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" {

size_t ln_residual_bwd_workspace_size(const ln_bwd_params_t* p) {
  if (check_params(p) != ATTN_OK) return SIZE_MAX;
  return (size_t)std::min<int64_t>(p->rows, kMaxParts) * 2 * (size_t)p->cols * sizeof(float);
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
  a.vec = ((at | reinterpret_cast<uintptr_t>(gamma)) & 15) == 0;
  a.part = weights ? static_cast<float*>(workspace) : nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int blocks = 0;
  cudaError_t e = cudaSuccess;
  if (p->rows > 0)
    e = p->dtype == ATTN_BF16 ? launch_bwd<__nv_bfloat16>(a, drops, &blocks, status, wait_ns, st)
                              : launch_bwd<float>(a, drops, &blocks, status, wait_ns, st);
  if (e == cudaSuccess && weights) e = launch_join(a, blocks, dgamma, dbeta, st);
  if (e != cudaSuccess) return bfail(ATTN_ERR_CUDA, "ln_residual_bwd: launch failed");
  return ATTN_OK;
}

}  // extern "C"
