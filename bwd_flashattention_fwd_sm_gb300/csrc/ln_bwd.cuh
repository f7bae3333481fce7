// Kernels of LayerNorm's backward pass (include/gbln.h has the formulas) and the rule that chooses
// among them, for one element type; ln_bwd.cu has the entry.
//
// Two sums of a row (of g and of g xh) decide its dr, and two sums of a column (of dy
// xh and of dy) are dgamma and dbeta.  A thread keeps the same columns in every row that it
// meets, so that its parts of the columns' sums stay in registers from the first row to
// the last.  Each block leaves one row of partial sums, and k_ln_bwd_join adds those in
// a fixed order.  Bound by device memory: dy, h and dh are read once and dr and dx
// written once.
//
// Rows that are no whole vectors.  Where the rows of all tensors begin at the same place
// within 16 bytes, a row is still moved as aligned vectors: with `shift` elements between
// the 16-byte boundary and the row's first element, vector v holds the columns v E - shift
// .. v E - shift + E - 1.  The shift depends on the row modulo 8 alone, so blocks whose
// rows are a multiple of 8 apart keep theirs, and with it their columns.  Only the vectors at a row's
// two ends are read and written by elements.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gbln.h"
#include "common.cuh"
#include "dropout.cuh"
#include "ptx.cuh"
#include "row_group.cuh"
#include "rowvec.cuh"

namespace gbattn {

// Rows of partial sums at most: two blocks on each of 152 SMs.  Constants, so that the size of the
// workspace and the order of the sums are the same everywhere.
constexpr int kLnSms = 152;
constexpr int kLnMaxParts = 2 * kLnSms;
constexpr int kLnCluster = 8;             // blocks of the cluster that does little work alone
constexpr int64_t kLnFewBytes = 1 << 16;  // of one tensor

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
  float* part;  // [blocks][2][cols]: sums of dy xh, and of dy; NULL: not wanted, or joined at once
  float* dgamma;  // where the grid is one cluster, which joins its blocks' sums itself; else NULL
  float* dbeta;
  bool join;
  int vec;      // every pointer 16-byte aligned and every stride a whole number of vectors
  int alike;    // every tensor's pointer the same modulo 16 bytes, and every stride the same
  DropArgs drop;
};

// So little work that one cluster does it and joins its blocks' sums over shared memory: one launch and
// no workspace.  [32, 1024] bf16 takes the GPU 7.0 us this way and 4.6 with k_ln_bwd_join, but the host
// issues a call in 25 us instead of 32, and calls of this size wait for the host.  By sizes alone,
// because the workspace's size says so too.
inline bool ln_bwd_joins(const ln_bwd_params_t& p) {
  return p.rows <= kLnFewBytes / (p.cols * (p.dtype == ATTN_BF16 ? 2 : 4));
}

// Launches the kernel for a.p's rows; *parts: how many rows of partial sums it leaves.
template <class T>
cudaError_t launch_ln_bwd(const BwdLnArgs& a, bool drops, int* parts, int* status, unsigned long long wait_ns,
                          cudaStream_t st);

namespace {

// dgamma and dbeta from the blocks' columns [2][cols] in shared memory, the blocks in order.  All threads of all
// blocks of the cluster come here; good: this block's columns hold sums.
__device__ __forceinline__ void join_columns(const float* column, int cols, float* dgamma, float* dbeta, bool good) {
  uint32_t blocks;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(blocks));
  __syncthreads();
  cluster_barrier();
  if (good) {
    for (int c = cluster_rank() * blockDim.x + threadIdx.x; c < 2 * cols; c += blocks * blockDim.x) {
      float v[kLnCluster], s = 0.f;
#pragma unroll
      for (uint32_t r = 0; r < kLnCluster; ++r) {
        uint32_t from;
        v[r] = 0.f;
        if (r < blocks) {
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(ptx::smem_u32(column + c)), "r"(r));
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[r]) : "r"(from) : "memory");
        }
      }
#pragma unroll
      for (uint32_t r = 0; r < kLnCluster; ++r) s += v[r];
      float* to = c < cols ? dgamma : dbeta;
      if (to) to[c < cols ? c : c - cols] = s;
    }
    __syncwarp();
  }
  cluster_barrier();  // no block leaves while another reads its columns
}

// The sums of a block's groups, each group's [2][cols] at its place in shared memory (`apart` floats on), in
// order: to `part`, or (NULL) to the first group's place.
__device__ __forceinline__ void add_groups(float* column, int groups, int apart, int cols, float* part) {
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * cols; c += blockDim.x) {
    float s = column[c];
#pragma unroll 8
    for (int g = 1; g < groups; ++g) s += column[g * apart + c];
    (part ? part : column)[c] = s;
  }
}

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
  extern __shared__ float column[];  // [2][cols], where the cluster joins
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
  if (!a.part && !a.join) return;
  float* part = a.join ? column : a.part + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
  for (int j = 0; j < kVpt; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t c = (int64_t)(tid + j * kThreads) * E + e;
      if (c < cols) part[c] = sg[j][e], part[cols + c] = sb[j][e];
    }
  if (a.join) join_columns(column, (int)cols, a.dgamma, a.dbeta, true);
}

// A short row: kRow lanes of a warp, a vector each, kRows rows of a lane at a time with all their
// loads in flight.  kRagged: see above.
template <class T, int kRow, int kRows, bool kDrop, bool kRagged>
__global__ void __launch_bounds__(512, 2) k_ln_bwd_warp(const BwdLnArgs a) {
  constexpr int E = Vec<T>::E, P = E / 2;
  extern __shared__ float column[];  // [groups][2][cols]
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x % kRow, groups = blockDim.x / kRow;
  const int cols = (int)a.p.cols;
  const float inv = 1.f / (float)cols;
  DropKey key{};
  DropRate rate{};
  if constexpr (kDrop) key = drop_key(a.drop), rate = drop_rate(a.drop);
  const T* DY = static_cast<const T*>(a.dy);
  const T* H = static_cast<const T*>(a.h);
  const T* DH = static_cast<const T*>(a.dh);
  const int64_t step = (int64_t)gridDim.x * groups;
  const int64_t first = (int64_t)blockIdx.x * groups + threadIdx.x / kRow;
  int shift = 0;
  if constexpr (kRagged) shift = (int)(reinterpret_cast<uintptr_t>(DY + first * a.p.dy_stride) & 15) / (int)sizeof(T);
  const int c0 = lane * E - shift;
  const bool mine = c0 < cols, inside = !kRagged || (c0 >= 0 && c0 + E <= cols);
  float2 sg[P], sb[P], gamma[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    sg[i] = sb[i] = make_float2(0.f, 0.f);
    const int c = c0 + 2 * i;
    gamma[i] = make_float2(a.gamma && c >= 0 && c < cols ? a.gamma[c] : 1.f,
                           a.gamma && c + 1 >= 0 && c + 1 < cols ? a.gamma[c + 1] : 1.f);
  }
  // Places that are no columns get 0 in dy and a column's value in h (`fill`), so that they add
  // nothing to any sum.
  auto fetch = [&](const T* row, bool fill) -> uint4 {
    if constexpr (kRagged) {
      if (!inside) {
        float2 v[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int c = c0 + 2 * i;
          v[i].x = fill || (c >= 0 && c < cols) ? Vec<T>::load1(row + min(max(c, 0), cols - 1)) : 0.f;
          v[i].y = fill || (c + 1 >= 0 && c + 1 < cols) ? Vec<T>::load1(row + min(max(c + 1, 0), cols - 1)) : 0.f;
        }
        return Vec<T>::pack(v);
      }
    }
    return *reinterpret_cast<const uint4*>(row + c0);
  };
  auto store = [&](void* base, int64_t stride, int64_t row, uint4 v) {
    T* out = static_cast<T*>(base) + row * stride;
    if (inside) {
      *reinterpret_cast<uint4*>(out + c0) = v;
    } else {
      float2 d[P];
      Vec<T>::pairs(v, d);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = c0 + 2 * i;
        if (c >= 0 && c < cols) Vec<T>::store1(out + c, d[i].x);
        if (c + 1 >= 0 && c + 1 < cols) Vec<T>::store1(out + c + 1, d[i].y);
      }
    }
  };
  // every lane of a warp takes the same number of turns: a row behind the last is one of zeros
  const int64_t warp_first = (int64_t)blockIdx.x * groups + (threadIdx.x & ~31) / kRow;
  for (int64_t turn = warp_first, row = first; turn < a.p.rows; turn += kRows * step, row += kRows * step) {
    uint4 dy[kRows], h[kRows], dh[kRows];
    float mean[kRows], rstd[kRows], m0[kRows], m1[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t r = row + u * step;
      dy[u] = h[u] = dh[u] = make_uint4(0u, 0u, 0u, 0u);
      mean[u] = rstd[u] = 0.f;
      if (r < a.p.rows && mine) {
        mean[u] = a.mean[r], rstd[u] = a.rstd[r];
        dy[u] = fetch(DY + r * a.p.dy_stride, false);
        h[u] = fetch(H + r * a.p.h_stride, true);
        if (DH) dh[u] = fetch(DH + r * a.p.dh_stride, false);
      }
    }
    auto normalised = [&](int u, float2 (&xh)[P]) {
      Vec<T>::pairs(h[u], xh);
#pragma unroll
      for (int i = 0; i < P; ++i)
        xh[i] = pair_mul(pair_add(xh[i], make_float2(-mean[u], -mean[u])), make_float2(rstd[u], rstd[u]));
    };
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      float2 g[P], xh[P];
      float2 s0 = make_float2(0.f, 0.f), s1 = s0;
      Vec<T>::pairs(dy[u], g);
      normalised(u, xh);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        sg[i] = pair_fma(g[i], xh[i], sg[i]);
        sb[i] = pair_add(g[i], sb[i]);
        g[i] = pair_mul(g[i], gamma[i]);
        s0 = pair_add(g[i], s0);
        s1 = pair_fma(g[i], xh[i], s1);
      }
      m0[u] = s0.x + s0.y, m1[u] = s1.x + s1.y;
    }
#pragma unroll
    for (int o = kRow / 2; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        m0[u] += __shfl_xor_sync(0xffffffffu, m0[u], o);
        m1[u] += __shfl_xor_sync(0xffffffffu, m1[u], o);
      }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t r = row + u * step;
      if (r >= a.p.rows || !mine) continue;
      float2 g[P], xh[P], d[P];
      Vec<T>::pairs(dy[u], g);
      normalised(u, xh);
      Vec<T>::pairs(dh[u], d);
      const float2 n0 = make_float2(-m0[u] * inv, -m0[u] * inv), n1 = make_float2(-m1[u] * inv, -m1[u] * inv);
#pragma unroll
      for (int i = 0; i < P; ++i)
        d[i] = pair_fma(pair_fma(xh[i], n1, pair_fma(g[i], gamma[i], n0)), make_float2(rstd[u], rstd[u]), d[i]);
      uint4 dx = Vec<T>::pack(d);
      if (a.dr) store(a.dr, a.p.dr_stride, r, dx);
      if (a.dx) {
        if constexpr (kDrop) {  // of the unrounded dr
#pragma unroll
          for (int i = 0; i < P; ++i) d[i] = pair_mul(d[i], make_float2(rate.factor, rate.factor));
          dx = drop_mask_at<T, kRagged>(Vec<T>::pack(d), c0, (uint32_t)r, key, rate);
        }
        store(a.dx, a.p.dx_stride, r, dx);
      }
    }
  }
  if (!a.part && !a.join) return;
  float* own = column + (threadIdx.x / kRow) * 2 * cols;
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = c0 + 2 * i + k;
      if (c >= 0 && c < cols) own[c] = k ? sg[i].y : sg[i].x, own[cols + c] = k ? sb[i].y : sb[i].x;
    }
  add_groups(column, groups, 2 * cols, cols, a.join ? nullptr : a.part + (int64_t)blockIdx.x * 2 * cols);
  if (a.join) join_columns(column, cols, a.dgamma, a.dbeta, true);
}

// A longer row: kRow threads, kVpt vectors each.  A block holds kGroups such rows side by side;
// kCluster blocks share one row (its sums then meet over the cluster's shared memory).
// Rows stream through a ring of stages in shared memory that bulk copies fill some rows ahead,
// so that the one barrier a row does not stop the loads.  A stage is read twice (for the sums,
// then for dr), which leaves the registers to the columns' sums.  Waits are bounded: a
// group that gives up records ATTN_ERR_DEVICE_TIMEOUT, waits (bounded) for its own copies and
// stops, and its block leaves no partial sums.
template <class T, int kRow, int kGroups, int kVpt, int kBlocks, int kCluster, bool kDrop, bool kRagged>
__global__ void __launch_bounds__(kRow* kGroups, kBlocks)
    k_ln_bwd_ring(const BwdLnArgs a, int stages, int slots, int* status, unsigned long long wait_ns) {
  constexpr int E = Vec<T>::E, P = E / 2, kWarps = kRow / 32, kParts = kCluster * kWarps;
  constexpr bool kKeepGamma = kVpt * E <= 16;       // registers allow it
  constexpr int kEdge = (6 * E + kRow - 1) / kRow;  // elements at a row's ends, of one thread
  static_assert(kCluster == 1 || kGroups == 1, "one row of a cluster");
  // of the longest rows, with dh; two: float32 rows of more than 6308 columns of a block, or 12620 of two
  constexpr int kLeastStages = ring_stages(kBlocks, kGroups, kRow * kVpt * 16 * 3);
  static_assert(kLeastStages >= 2, "a stage is read while another is filled");
  extern __shared__ __align__(128) uint8_t ring[];  // [groups][stages][2 or 3][slots] vectors
  __shared__ uint64_t full_all[kGroups][kMaxStages];
  __shared__ uint64_t met[2];  // the other block's sums have come, by the row's parity
  __shared__ __align__(16) float sums_all[kGroups][2][2][kParts];
  __shared__ ptx::Abort abort;
  const int group = threadIdx.x / kRow, tid = threadIdx.x % kRow, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int groups = blockDim.x / kRow;  // kGroups, or fewer where there are few rows
  uint64_t* full = full_all[group];
  const uint32_t rank = kCluster > 1 ? cluster_rank() : 0;
  const int64_t unit = blockIdx.x / kCluster;
  const int64_t first = unit * groups + group, step = (int64_t)(gridDim.x / kCluster) * groups;
  const int turns = first < a.p.rows ? (int)((a.p.rows - first + step - 1) / step) : 0;
  const int cols = (int)a.p.cols;
  const float inv = 1.f / (float)cols;
  const bool has_dh = a.dh != nullptr;
  const int tensors = has_dh ? 3 : 2;
  const T* in[3] = {static_cast<const T*>(a.dy) + first * a.p.dy_stride, static_cast<const T*>(a.h) + first * a.p.h_stride,
                    static_cast<const T*>(a.dh) + (has_dh ? first * a.p.dh_stride : 0)};
  const int64_t ahead[3] = {step * a.p.dy_stride, step * a.p.h_stride, step * a.p.dh_stride};
  int shift = 0;
  if constexpr (kRagged) shift = (int)(reinterpret_cast<uintptr_t>(in[0]) & 15) / (int)sizeof(T);
  const int vectors = (shift + cols + E - 1) / E;
  const int each = (vectors + kCluster - 1) / kCluster;           // <= slots
  const int v0 = (int)rank * each, v1 = min(vectors, v0 + each);  // this block's
  const int whole0 = max(v0, shift > 0 ? 1 : 0), whole1 = min(v1, (shift + cols) / E);
  const uint32_t slot_bytes = (uint32_t)slots * 16, copy_bytes = whole1 > whole0 ? (uint32_t)(whole1 - whole0) * 16 : 0;
  const uint32_t stage_bytes = slot_bytes * tensors;
  uint8_t* stage0 = ring + (size_t)group * stages * stage_bytes;
  auto issue = [&](int s, int turn) {  // thread 0 only
    uint8_t* to = stage0 + (size_t)s * stage_bytes + (whole0 - v0) * 16;
    ptx::mbar_arrive_expect_tx(&full[s], copy_bytes * tensors);
    if (copy_bytes) {
      const int c = whole0 * E - shift;
      ptx::bulk_load(to, in[0] + turn * ahead[0] + c, copy_bytes, &full[s]);
      ptx::bulk_load(to + slot_bytes, in[1] + turn * ahead[1] + c, copy_bytes, &full[s]);
      if (has_dh) ptx::bulk_load(to + 2 * slot_bytes, in[2] + turn * ahead[2] + c, copy_bytes, &full[s]);
    }
  };
  // The vectors at the two ends, by elements: of which element this thread moves, the address in the
  // first row and the place in a stage (negative: none).  Places that are no columns get 0 in dy
  // (address NULL) and a column's value in h, so that they add nothing to any sum.
  const T* edge_from[kEdge] = {};
  int edge_to[kEdge] = {};
  if constexpr (kRagged) {
#pragma unroll
    for (int k = 0; k < kEdge; ++k) {
      const int i = tid + k * kRow, t = i / (2 * E), e = i % E;
      const bool right = (i / E) & 1;
      const int v = right ? (shift + cols) / E : 0, c = v * E - shift + e;
      const bool there = i < 2 * E * tensors && (right ? (shift + cols) % E != 0 : shift > 0) && v >= v0 && v < v1;
      edge_to[k] = there ? (int)(t * slot_bytes) + ((v - v0) * E + e) * (int)sizeof(T) : -1;
      edge_from[k] = t == 1 ? in[1] + min(max(c, 0), cols - 1)
                            : there && c >= 0 && c < cols ? (t == 0 ? in[0] : in[2]) + c : nullptr;
    }
  }
  auto edge_load = [&](int k, int turn) {
    return edge_to[k] >= 0 && edge_from[k] ? edge_from[k][turn * ahead[0]] : from_f32<T>(0.f);
  };
  auto edge_store = [&](int k, int s, T x) {
    if (edge_to[k] >= 0) *reinterpret_cast<T*>(stage0 + (size_t)s * stage_bytes + edge_to[k]) = x;
  };
  int issued = 0;  // thread 0: turns whose copies are on their way
  if (threadIdx.x == 0) {
    abort.flag = 0;
    if constexpr (kCluster > 1)
      for (int i = 0; i < 2; ++i) ptx::mbar_init(&met[i], 1);
  }
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) ptx::mbar_init(&full[s], 1);
    ptx::fence_mbar_init();
    for (; issued < stages && issued < turns; ++issued) issue(issued, issued);
    if constexpr (kCluster > 1)
      for (int i = 0; i < 2; ++i) ptx::mbar_arrive_expect_tx(&met[i], 2 * kWarps * sizeof(float));
  }
  if constexpr (kRagged) {
    for (int s = 0; s < stages && s < turns; ++s)
#pragma unroll
      for (int k = 0; k < kEdge; ++k) edge_store(k, s, edge_load(k, s));
  }
  DropKey key{};
  DropRate rate{};
  if constexpr (kDrop) key = drop_key(a.drop), rate = drop_rate(a.drop);
  float2 sg[kVpt][P], sb[kVpt][P], keep[kKeepGamma ? kVpt : 1][P];
  auto gamma_at = [&](int c0, float2 (&g)[P]) {
    if (!kRagged) {
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        const float4 v = a.gamma ? __ldg(reinterpret_cast<const float4*>(a.gamma + c0 + 2 * i))
                                 : make_float4(1.f, 1.f, 1.f, 1.f);
        g[i] = make_float2(v.x, v.y), g[i + 1] = make_float2(v.z, v.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = c0 + 2 * i;
        g[i].x = a.gamma && c >= 0 && c < cols ? __ldg(a.gamma + c) : 1.f;
        g[i].y = a.gamma && c + 1 >= 0 && c + 1 < cols ? __ldg(a.gamma + c + 1) : 1.f;
      }
    }
  };
#pragma unroll
  for (int j = 0; j < kVpt; ++j) {
#pragma unroll
    for (int i = 0; i < P; ++i) sg[j][i] = sb[j][i] = make_float2(0.f, 0.f);
    if (kKeepGamma && v0 + tid + j * kRow < v1) gamma_at((v0 + tid + j * kRow) * E - shift, keep[j]);
  }
  const float* mean_at = a.mean + first;
  const float* rstd_at = a.rstd + first;
  float mean = 0.f, rstd = 0.f;
  if (turns > 0) mean = *mean_at, rstd = *rstd_at;
  // where this thread's first vector of the row goes
  const int c_first = (v0 + tid) * E - shift;
  T* dr = a.dr ? static_cast<T*>(a.dr) + first * a.p.dr_stride + c_first : nullptr;
  T* dx = a.dx ? static_cast<T*>(a.dx) + first * a.p.dx_stride + c_first : nullptr;
  const int64_t dr_step = step * a.p.dr_stride, dx_step = step * a.p.dx_stride;
  uint32_t row = (uint32_t)first;  // for the mask, which takes 32 bits of it
  if constexpr (kCluster > 1) {
    __syncwarp();
    cluster_barrier();  // the other block's barriers are there too
  } else {
    __syncthreads();
  }
  int s = 0, last = 0;  // this row's stage, and the one before
  uint32_t phase = 0;
  int turn = 0;
  bool ok = true, late = false;
  for (; turn < turns; ++turn) {
    const bool mine = ptx::mbar_wait(&full[s], phase, &abort, status, wait_ns);
    const uint4* dy = reinterpret_cast<const uint4*>(stage0 + (size_t)s * stage_bytes) + tid;
    const uint4* h = dy + slots;
    const uint4* dh = h + slots;
    float* sums = &sums_all[group][turn & 1][0][0];  // [2][kParts]
    const float2 shift2 = make_float2(-mean, -mean), scale2 = make_float2(rstd, rstd);
    mean_at += step, rstd_at += step;
    if (turn + 1 < turns) mean = *mean_at, rstd = *rstd_at;
    auto normalised = [&](int j, float2 (&xh)[P]) {
      Vec<T>::pairs(h[j * kRow], xh);
#pragma unroll
      for (int i = 0; i < P; ++i) xh[i] = pair_mul(pair_add(xh[i], shift2), scale2);
    };
    float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      if (v0 + tid + j * kRow >= v1) continue;
      float2 g[P], xh[P], w[P];
      Vec<T>::pairs(dy[j * kRow], g);
      normalised(j, xh);
      if (!kKeepGamma) gamma_at(c_first + j * kRow * E, w);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        sg[j][i] = pair_fma(g[i], xh[i], sg[j][i]);
        sb[j][i] = pair_add(g[i], sb[j][i]);
        g[i] = pair_mul(g[i], kKeepGamma ? keep[kKeepGamma ? j : 0][i] : w[i]);
        s0 = pair_add(g[i], s0);
        s1 = pair_fma(g[i], xh[i], s1);
      }
    }
    // both sums at once: the lower half of the warp joins the first, the upper the second
    auto both = [&](float x0, float x1) {
      float m = lane < 16 ? x0 : x1;
      m += __shfl_xor_sync(0xffffffffu, lane < 16 ? x1 : x0, 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
      return m;
    };
    float m = both(s0.x + s0.y, s1.x + s1.y), m0, m1;
    if constexpr (kRow > 32) {
      if ((lane & 15) == 0) {
        float* to = sums + (lane >> 4) * kParts + rank * kWarps + warp;
        *to = m;
        if constexpr (kCluster > 1) cluster_send(to, &met[turn & 1], rank ^ 1, m);
      }
    }
    if (group_any<kRow, kGroups>(group, !mine || late)) { ok = false; break; }
    // the barrier also said that every warp is done with the last row's stage
    const bool refill = turn > 0 && turn + stages - 1 < turns;
    if (tid == 0 && refill) issue(last, issued++);
    if constexpr (kCluster > 1) {
      // a thread that gives up here goes on with what there is and says so at the next barrier
      late = !ptx::mbar_wait<true>(&met[turn & 1], (uint32_t)(turn >> 1) & 1, &abort, status, wait_ns);
      if (tid == 0) ptx::mbar_arrive_expect_tx(&met[turn & 1], 2 * kWarps * sizeof(float));
    }
    if constexpr (kParts == 1) {
      m0 = __shfl_sync(0xffffffffu, m, 0);
      m1 = __shfl_sync(0xffffffffu, m, 16);
    } else if constexpr (kParts <= 16) {
      m0 = m1 = 0.f;
#pragma unroll
      for (int w = 0; w < kParts; ++w) m0 += sums[w], m1 += sums[kParts + w];
    } else {  // a thread's own additions would be as many as a vector's
      m = both(sums[lane], sums[32 + lane]);
      m0 = __shfl_sync(0xffffffffu, m, 0);
      m1 = __shfl_sync(0xffffffffu, m, 16);
    }
    T edge[kEdge];
    if constexpr (kRagged) {
      if (refill)
#pragma unroll
        for (int k = 0; k < kEdge; ++k) edge[k] = edge_load(k, turn + stages - 1);
    }
    const float2 n0 = make_float2(-m0 * inv, -m0 * inv), n1 = make_float2(-m1 * inv, -m1 * inv);
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      if (v0 + tid + j * kRow >= v1) continue;
      const int c0 = c_first + j * kRow * E;
      float2 g[P], xh[P], d[P], w[P];
      Vec<T>::pairs(dy[j * kRow], g);
      normalised(j, xh);
      Vec<T>::pairs(has_dh ? dh[j * kRow] : make_uint4(0u, 0u, 0u, 0u), d);
      if (!kKeepGamma) gamma_at(c0, w);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        g[i] = pair_fma(g[i], kKeepGamma ? keep[kKeepGamma ? j : 0][i] : w[i], n0);
        d[i] = pair_fma(pair_fma(xh[i], n1, g[i]), scale2, d[i]);
      }
      auto store = [&](T* out, uint4 v) {
        if (!kRagged || (c0 >= 0 && c0 + E <= cols)) {
          *reinterpret_cast<uint4*>(out) = v;
        } else {
          float2 o[P];
          Vec<T>::pairs(v, o);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const int c = c0 + 2 * i;
            if (c >= 0 && c < cols) Vec<T>::store1(out + 2 * i, o[i].x);
            if (c + 1 >= 0 && c + 1 < cols) Vec<T>::store1(out + 2 * i + 1, o[i].y);
          }
        }
      };
      uint4 out = Vec<T>::pack(d);
      if (dr) store(dr + j * kRow * E, out);
      if (dx) {
        if constexpr (kDrop) {  // of the unrounded dr
#pragma unroll
          for (int i = 0; i < P; ++i) d[i] = pair_mul(d[i], make_float2(rate.factor, rate.factor));
          out = drop_mask_at<T, kRagged>(Vec<T>::pack(d), c0, row, key, rate);
        }
        store(dx + j * kRow * E, out);
      }
    }
    if constexpr (kRagged) {
      if (refill) {
#pragma unroll
        for (int k = 0; k < kEdge; ++k) edge_store(k, last, edge[k]);
        // Other threads read these elements.  The next turn's barrier stands between where the stage is that of a
        // later turn; of two stages it is the next turn's, which is read in front of that barrier.
        if constexpr (kLeastStages < 3)
          if (stages < 3) group_any<kRow, kGroups>(group, false);
      }
    }
    if (dr) dr += dr_step;
    if (dx) dx += dx_step;
    row += (uint32_t)step;
    last = s;
    if (++s == stages) s = 0, phase ^= 1;
  }
  if constexpr (kCluster > 1) ok = !__syncthreads_or(late) && ok;
  if (!ok && tid == 0) {  // copies that this group issued and did not wait for
    ptx::Abort none;
    none.flag = 0;
    for (int j = turn; j < issued; ++j)
      ptx::mbar_wait(&full[j % stages], (uint32_t)((j / stages) & 1), &none, status, wait_ns);
  }
  if constexpr (kCluster > 1) {  // the other block may still send its sums here
    __syncwarp();
    cluster_barrier();
  }
  if (!a.part && !a.join) return;
  float* part = a.part + unit * 2 * cols;
  if (!a.join && groups == 1) {
    if (!ok) return;
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      if (v0 + tid + j * kRow >= v1) continue;
      const int c0 = c_first + j * kRow * E;
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        if (!kRagged) {
          *reinterpret_cast<float4*>(part + c0 + 2 * i) =
              make_float4(sg[j][i].x, sg[j][i].y, sg[j][i + 1].x, sg[j][i + 1].y);
          *reinterpret_cast<float4*>(part + cols + c0 + 2 * i) =
              make_float4(sb[j][i].x, sb[j][i].y, sb[j][i + 1].x, sb[j][i + 1].y);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int c = c0 + 2 * i + k;
            if (c < 0 || c >= cols) continue;
            part[c] = k & 1 ? sg[j][i + k / 2].y : sg[j][i + k / 2].x;
            part[cols + c] = k & 1 ? sb[j][i + k / 2].y : sb[j][i + k / 2].x;
          }
        }
      }
    }
  } else {
    const bool good = __syncthreads_and(ok);  // and the ring is free: every copy has been waited for
    if (good) {  // a group's own stages hold its sums
      float* own = reinterpret_cast<float*>(stage0);
#pragma unroll
      for (int j = 0; j < kVpt; ++j) {
        if (v0 + tid + j * kRow >= v1) continue;
        const int c0 = c_first + j * kRow * E;
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int c = c0 + 2 * i + k;
            if (kRagged && (c < 0 || c >= cols)) continue;
            own[c] = k ? sg[j][i].y : sg[j][i].x, own[cols + c] = k ? sb[j][i].y : sb[j][i].x;
          }
      }
      add_groups(reinterpret_cast<float*>(ring), groups, stages * (int)stage_bytes / 4, cols, a.join ? nullptr : part);
    }
    if constexpr (kCluster == 1)
      if (a.join) join_columns(reinterpret_cast<float*>(ring), cols, a.dgamma, a.dbeta, good);
  }
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class K, class... A>
cudaError_t launch_cluster(K kernel, int blocks, int threads, size_t smem, int cluster, cudaStream_t st, A... args) {
  const cudaError_t e = allow_shared(kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)cluster, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A kernel's variants: with and without dropout, whole vectors and ragged rows.
template <class T, int kRow, int kRows>
cudaError_t launch_warp(const BwdLnArgs& a, bool drops, bool ragged, int* parts, cudaStream_t st) {
  // as many warps a block as leave every SM (of the cluster, if one does it all) a block, 16 at most
  const int a_warp = 32 / kRow;
  int warps = 1;
  while (warps < 16 && div_up(a.p.rows, (int64_t)warps * a_warp) > (a.join ? kLnCluster : kLnSms)) warps *= 2;
  const int blocks =
      (int)std::min<int64_t>(div_up(a.p.rows, (int64_t)warps * a_warp), a.join ? kLnCluster : kLnMaxParts);
  *parts = blocks;
  const size_t smem = a.part || a.join ? (size_t)warps * a_warp * 2 * a.p.cols * sizeof(float) : 0;  // 32 KB at most
  auto kernel =
      ragged ? (drops ? k_ln_bwd_warp<T, kRow, kRows, true, true> : k_ln_bwd_warp<T, kRow, kRows, false, true>)
             : (drops ? k_ln_bwd_warp<T, kRow, kRows, true, false> : k_ln_bwd_warp<T, kRow, kRows, false, false>);
  return launch_cluster(kernel, blocks, 32 * warps, smem, a.join ? blocks : 1, st, a);
}

template <class T, int kRow, int kGroups, int kVpt, int kBlocks, int kCluster>
cudaError_t launch_ring(const BwdLnArgs& a, bool drops, bool ragged, int* parts, int* status,
                        unsigned long long wait_ns, cudaStream_t st) {
  // A grid's rows are a multiple of 8 apart wherever a group has more than one, for the ragged
  // form: 304 or 152 blocks, 76 clusters of two (period 4 of the 4-byte type) or 72.
  int most = kBlocks * kLnSms / kCluster;
  if (ragged && kGroups * most % (int)(16 / sizeof(T)) != 0) most = most / 8 * 8;
  // where rows are few, on as many SMs as there are (the cluster has, if one does it all)
  const bool join = kCluster == 1 && a.join;
  if (join) most = kLnCluster;
  int groups = 1;
  while (groups < kGroups && div_up(a.p.rows, groups) > (join ? kLnCluster : kLnSms)) groups *= 2;
  *parts = (int)std::min<int64_t>(div_up(a.p.rows, groups), most);
  const int slots = (int)div_up(div_up(a.p.cols, Vec<T>::E) + (ragged ? 1 : 0), kCluster);
  const int stage = slots * 16 * (a.dh ? 3 : 2);
  const int stages = ring_stages(kBlocks, kGroups, stage);
  const size_t smem = (size_t)groups * stages * stage;
  auto kernel = ragged ? (drops ? k_ln_bwd_ring<T, kRow, kGroups, kVpt, kBlocks, kCluster, true, true>
                                : k_ln_bwd_ring<T, kRow, kGroups, kVpt, kBlocks, kCluster, false, true>)
                       : (drops ? k_ln_bwd_ring<T, kRow, kGroups, kVpt, kBlocks, kCluster, true, false>
                                : k_ln_bwd_ring<T, kRow, kGroups, kVpt, kBlocks, kCluster, false, false>);
  return launch_cluster(kernel, *parts * kCluster, kRow * groups, smem, join ? *parts : kCluster, st, a, stages, slots,
                        status, wait_ns);
}

template <class T, int kThreads, int kVpt>
cudaError_t launch_rows(const BwdLnArgs& a, bool drops, int* parts, cudaStream_t st) {
  *parts = (int)std::min<int64_t>(a.p.rows, a.join ? kLnCluster : kLnMaxParts);
  const size_t smem = a.join ? 2 * a.p.cols * sizeof(float) : 0;
  return launch_cluster(drops ? k_ln_bwd<T, kThreads, kVpt, true> : k_ln_bwd<T, kThreads, kVpt, false>, *parts, kThreads,
                        smem, a.join ? *parts : 1, st, a);
}

}  // namespace

template <class T>
cudaError_t launch_ln_bwd(const BwdLnArgs& a, bool drops, int* parts, int* status, unsigned long long wait_ns,
                          cudaStream_t st) {
  constexpr int E = Vec<T>::E;
  const bool ragged = !(a.vec && a.p.cols % E == 0);
  const int64_t n = div_up(a.p.cols, E), m = n + (ragged ? 1 : 0);  // vectors of a row, at most
  if (!ragged || a.alike) {
    // Rows of a lane in flight.  64 registers hold them in the plain form; dropping and ragged forms spill 24 to 168 bytes.
    // bf16: [262144, 128] 49 us, 72 with two.  float32: [131072, 128] 44, 47 with one and 70 with four; dropping 62, 57 and
    // 95; ragged [166000, 101] 68, 58 and 133.
    constexpr int kRows = E == 8 ? 1 : 2;
    if (m <= 8) return launch_warp<T, 8, kRows>(a, drops, ragged, parts, st);
    if (m <= 16) return launch_warp<T, 16, kRows>(a, drops, ragged, parts, st);
    if (m <= 32) return launch_warp<T, 32, kRows>(a, drops, ragged, parts, st);
    if (m <= 64) return launch_ring<T, 32, 8, 2, 2, 1>(a, drops, ragged, parts, status, wait_ns, st);
    if (m <= 128) return launch_ring<T, 64, 4, 2, 2, 1>(a, drops, ragged, parts, status, wait_ns, st);
    if (m <= 256) return launch_ring<T, 128, 2, 2, 2, 1>(a, drops, ragged, parts, status, wait_ns, st);
    if (m <= 512) return launch_ring<T, 256, 1, 2, 2, 1>(a, drops, ragged, parts, status, wait_ns, st);
    if (m <= 1024) return launch_ring<T, 512, 1, 2, 1, 1>(a, drops, ragged, parts, status, wait_ns, st);
    if constexpr (E == 8) {
      if (m <= 2048 && !a.join) return launch_ring<T, 512, 1, 2, 1, 2>(a, drops, ragged, parts, status, wait_ns, st);
    } else {
      if (m <= 2048) return launch_ring<T, 512, 1, 4, 1, 1>(a, drops, ragged, parts, status, wait_ns, st);
      if (m <= 4096 && !a.join) return launch_ring<T, 512, 1, 4, 1, 2>(a, drops, ragged, parts, status, wait_ns, st);
    }
  }
  if (n <= 256) return launch_rows<T, 256, 1>(a, drops, parts, st);
  if (n <= 512) return launch_rows<T, 256, 2>(a, drops, parts, st);
  if (n <= 1024) return launch_rows<T, 512, 2>(a, drops, parts, st);
  if (n <= 2048) return launch_rows<T, 512, 4>(a, drops, parts, st);
  if constexpr (E == 4) return launch_rows<T, 512, 8>(a, drops, parts, st);
  return cudaErrorInvalidValue;
}

}  // namespace gbattn
