// Dropout, residual add and LayerNorm in one pass (include/gbln.h has the formulas), for one element
// type; ln.cu has the entry, and the form without dropout.
//
// A row belongs to a group of kRow threads, kVpt vectors each, and a block holds kGroups such
// groups (rows of up to 32 vectors: some lanes of a warp, without the ring).  Rows stream through a
// ring of stages in shared memory that bulk copies fill some rows ahead.  h is made once and stays in registers; its mean and then the sum of its squared
// distances from that mean are two sums over the group, so nothing cancels.  Bound by device memory
// at long rows; the mask (some 60 instructions for eight elements) and the two barriers a row are next.
// Rows of more than 8192 columns: two blocks of a cluster, which send each other their warps' sums.
// Rows that are no whole vectors are moved as shifted aligned vectors, as in the backward pass
// (ln_bwd.cuh), where the rows of all tensors begin at the same place within 16 bytes.
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

struct LnDropArgs {
  ln_params_t p;
  const void* x;
  const void* r;
  const float* gamma;
  const float* beta;
  void* y;
  void* h;
  float* mean;
  float* rstd;
  DropArgs drop;
};

// Launches the kernel; false: it does not take rows of this length (nothing was launched).
template <class T>
bool launch_ln_drop(const LnDropArgs& a, bool ragged, int* status, unsigned long long wait_ns, cudaStream_t st,
                    cudaError_t* error);

namespace {

template <class T, int kRow, int kGroups, int kVpt, int kBlocks, int kCluster, bool kRagged>
__global__ void __launch_bounds__(kRow* kGroups, kBlocks)
    k_ln_drop(const LnDropArgs a, int stages, int slots, int* status, unsigned long long wait_ns) {
  constexpr int E = Vec<T>::E, P = E / 2, kWarps = kRow / 32, kParts = kCluster * kWarps;
  static_assert(kCluster == 1 || kGroups == 1, "one row of a cluster");
  constexpr bool kKeep = kVpt * E <= 16;            // gamma and beta in registers
  constexpr int kEdge = (4 * E + kRow - 1) / kRow;  // elements at a row's ends, of one thread
  extern __shared__ __align__(128) uint8_t ring[];  // [groups][stages][1 or 2][slots] vectors
  __shared__ uint64_t full_all[kGroups][kMaxStages];
  __shared__ float sums_all[kGroups][2][kParts];
  __shared__ uint64_t met[2];  // the other block's sums have come: of h, of its squares
  __shared__ ptx::Abort abort;
  const int group = threadIdx.x / kRow, tid = threadIdx.x % kRow, lane = tid & 31, warp = tid >> 5;
  const int groups = blockDim.x / kRow;  // kGroups, or fewer where there are few rows
  uint64_t* full = full_all[group];
  float (&sums)[2][kParts] = sums_all[group];
  const uint32_t rank = kCluster > 1 ? cluster_rank() : 0;
  const int64_t first = (int64_t)(blockIdx.x / kCluster) * groups + group, step = (int64_t)(gridDim.x / kCluster) * groups;
  const int turns = first < a.p.rows ? (int)((a.p.rows - first + step - 1) / step) : 0;
  const int cols = (int)a.p.cols;
  const float inv = 1.f / (float)cols;
  const bool has_r = a.r != nullptr;
  const int tensors = has_r ? 2 : 1;
  const T* in[2] = {static_cast<const T*>(a.x) + first * a.p.x_stride,
                    static_cast<const T*>(a.r) + (has_r ? first * a.p.r_stride : 0)};
  const int64_t ahead[2] = {step * a.p.x_stride, step * a.p.r_stride};
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
      if (has_r) ptx::bulk_load(to + slot_bytes, in[1] + turn * ahead[1] + c, copy_bytes, &full[s]);
    }
  };
  // The vectors at the two ends, by elements: the address in the first row (NULL: no column, 0) and
  // the place in a stage (negative: none) of those that this thread moves.
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
      edge_from[k] = there && c >= 0 && c < cols ? (t == 0 ? in[0] : in[1]) + c : nullptr;
    }
  }
  auto edge_load = [&](int k, int turn) {
    return edge_from[k] ? edge_from[k][turn * ahead[0]] : from_f32<T>(0.f);
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
      for (int i = 0; i < 2; ++i) ptx::mbar_arrive_expect_tx(&met[i], kWarps * sizeof(float));
  }
  if constexpr (kRagged) {
    for (int s = 0; s < stages && s < turns; ++s)
#pragma unroll
      for (int k = 0; k < kEdge; ++k) edge_store(k, s, edge_load(k, s));
  }
  const DropKey key = drop_key(a.drop);
  const DropRate rate = drop_rate(a.drop);
  const float2 factor = make_float2(rate.factor, rate.factor);
  const int c_first = (v0 + tid) * E - shift;
  auto columns = [&](const float* from, float other, int c0, float2 (&g)[P]) {  // of gamma or beta
    if (!kRagged) {
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        const float4 v = from ? __ldg(reinterpret_cast<const float4*>(from + c0 + 2 * i))
                              : make_float4(other, other, other, other);
        g[i] = make_float2(v.x, v.y), g[i + 1] = make_float2(v.z, v.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = c0 + 2 * i;
        g[i].x = from && c >= 0 && c < cols ? __ldg(from + c) : other;
        g[i].y = from && c + 1 >= 0 && c + 1 < cols ? __ldg(from + c + 1) : other;
      }
    }
  };
  float2 gamma[kKeep ? kVpt : 1][P], beta[kKeep ? kVpt : 1][P];
  if constexpr (kKeep) {
#pragma unroll
    for (int j = 0; j < kVpt; ++j)
      if (v0 + tid + j * kRow < v1) {
        columns(a.gamma, 1.f, c_first + j * kRow * E, gamma[j]);
        columns(a.beta, 0.f, c_first + j * kRow * E, beta[j]);
      }
  }
  T* y = static_cast<T*>(a.y) + first * a.p.y_stride + c_first;
  T* h_to = a.h ? static_cast<T*>(a.h) + first * a.p.h_stride + c_first : nullptr;
  const int64_t y_step = step * a.p.y_stride, h_step = step * a.p.h_stride;
  if constexpr (kCluster > 1) {
    __syncwarp();
    cluster_barrier();  // the other block's barriers are there too
  } else {
    __syncthreads();
  }
  int s = 0;
  uint32_t phase = 0, row = (uint32_t)first;
  int turn = 0;
  bool ok = true, late = false;
  for (; turn < turns; ++turn) {
    const bool mine = ptx::mbar_wait(&full[s], phase, &abort, status, wait_ns);
    const uint4* x = reinterpret_cast<const uint4*>(stage0 + (size_t)s * stage_bytes) + tid;
    const uint4* r = x + slots;
    auto store = [&](T* out, int c0, uint4 v) {
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
    float2 h[kVpt][P], sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      if (v0 + tid + j * kRow >= v1) continue;
      const int c0 = c_first + j * kRow * E;
      float2 w[P];
      Vec<T>::pairs(drop_mask_at<T, kRagged>(x[j * kRow], c0, row, key, rate), h[j]);
      Vec<T>::pairs(has_r ? r[j * kRow] : make_uint4(0u, 0u, 0u, 0u), w);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        h[j][i] = pair_fma(h[j][i], factor, w[i]);
        sum = pair_add(h[j][i], sum);
      }
    }
    auto total = [&](float m, int kind) {  // over the group; the barrier is the caller's
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
      if (kRow > 32 && lane == 0) {
        sums[kind][rank * kWarps + warp] = m;
        if constexpr (kCluster > 1) cluster_send(&sums[kind][rank * kWarps + warp], &met[kind], rank ^ 1, m);
      }
      return m;
    };
    auto joined = [&](float m, int kind) {
      if constexpr (kRow == 32) return m;
      if constexpr (kCluster > 1) {
        // a thread that gives up here goes on with what there is and says so at the next barrier
        late = !ptx::mbar_wait<true>(&met[kind], (uint32_t)turn & 1, &abort, status, wait_ns) || late;
        if (tid == 0) ptx::mbar_arrive_expect_tx(&met[kind], kWarps * sizeof(float));
      }
      m = 0.f;
#pragma unroll
      for (int w = 0; w < kParts; ++w) m += sums[kind][w];
      return m;
    };
    float m = total(sum.x + sum.y, 0);
    // the barrier also says that every warp is done with the stage
    if (group_any<kRow, kGroups>(group, !mine || late)) { ok = false; break; }
    const bool refill = turn + stages < turns;
    if (tid == 0 && refill) issue(s, issued++);
    T edge[kEdge];
    if constexpr (kRagged) {
      if (refill)
#pragma unroll
        for (int k = 0; k < kEdge; ++k) edge[k] = edge_load(k, turn + stages);
    }
    const float mean = joined(m, 0) * inv;
    const float2 shift2 = make_float2(-mean, -mean);
    sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      if (v0 + tid + j * kRow >= v1) continue;
      const int c0 = c_first + j * kRow * E;
      if (h_to) {
        store(h_to + j * kRow * E, c0, Vec<T>::pack(h[j]));
      }
#pragma unroll
      for (int i = 0; i < P; ++i) h[j][i] = pair_add(h[j][i], shift2);
      if (kRagged && (c0 < 0 || c0 + E > cols)) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int c = c0 + 2 * i;
          if (c < 0 || c >= cols) h[j][i].x = 0.f;
          if (c + 1 < 0 || c + 1 >= cols) h[j][i].y = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < P; ++i) sum = pair_fma(h[j][i], h[j][i], sum);
    }
    m = total(sum.x + sum.y, 1);
    group_any<kRow, kGroups>(group, false);
    const float rstd = 1.f / sqrtf(joined(m, 1) * inv + a.p.eps);
    const float2 scale2 = make_float2(rstd, rstd);
    if (tid == 0 && rank == 0) {
      if (a.mean) a.mean[first + turn * step] = mean;
      if (a.rstd) a.rstd[first + turn * step] = rstd;
    }
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      if (v0 + tid + j * kRow >= v1) continue;
      const int c0 = c_first + j * kRow * E;
      float2 g[P], b[P];
      if constexpr (!kKeep) {
        columns(a.gamma, 1.f, c0, g);
        columns(a.beta, 0.f, c0, b);
      }
#pragma unroll
      for (int i = 0; i < P; ++i)
        h[j][i] = pair_fma(pair_mul(h[j][i], scale2), kKeep ? gamma[kKeep ? j : 0][i] : g[i],
                           kKeep ? beta[kKeep ? j : 0][i] : b[i]);
      store(y + j * kRow * E, c0, Vec<T>::pack(h[j]));
    }
    if constexpr (kRagged) {  // read only after the next barriers
      if (refill)
#pragma unroll
        for (int k = 0; k < kEdge; ++k) edge_store(k, s, edge[k]);
    }
    y += y_step;
    if (h_to) h_to += h_step;
    row += (uint32_t)step;
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
}

// A short row: kRow lanes of a warp, a vector each, kRows rows of a lane at a time, loaded straight to registers.
template <class T, int kRow, int kRows, bool kRagged>
__global__ void __launch_bounds__(512, 2) k_ln_drop_warp(const LnDropArgs a) {
  constexpr int E = Vec<T>::E, P = E / 2;
  const int lane = threadIdx.x % kRow, groups = blockDim.x / kRow;
  const int cols = (int)a.p.cols;
  const float inv = 1.f / (float)cols;
  const DropKey key = drop_key(a.drop);
  const DropRate rate = drop_rate(a.drop);
  const float2 factor = make_float2(rate.factor, rate.factor);
  const int64_t step = (int64_t)gridDim.x * groups;
  const int64_t first = (int64_t)blockIdx.x * groups + threadIdx.x / kRow;
  const T* X = static_cast<const T*>(a.x);
  const T* R = static_cast<const T*>(a.r);
  int shift = 0;
  if constexpr (kRagged) shift = (int)(reinterpret_cast<uintptr_t>(X + first * a.p.x_stride) & 15) / (int)sizeof(T);
  const int c0 = lane * E - shift;
  const bool mine = c0 < cols, inside = c0 >= 0 && c0 + E <= cols;
  float2 gamma[P], beta[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = c0 + 2 * i;
    const bool x = c >= 0 && c < cols, y = c + 1 >= 0 && c + 1 < cols;
    gamma[i] = make_float2(a.gamma && x ? a.gamma[c] : 1.f, a.gamma && y ? a.gamma[c + 1] : 1.f);
    beta[i] = make_float2(a.beta && x ? a.beta[c] : 0.f, a.beta && y ? a.beta[c + 1] : 0.f);
  }
  auto fetch = [&](const T* row) -> uint4 {  // 0 where there is no column
    if constexpr (kRagged) {
      if (!inside) {
        float2 v[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int c = c0 + 2 * i;
          v[i].x = c >= 0 && c < cols ? Vec<T>::load1(row + c) : 0.f;
          v[i].y = c + 1 >= 0 && c + 1 < cols ? Vec<T>::load1(row + c + 1) : 0.f;
        }
        return Vec<T>::pack(v);
      }
    }
    return *reinterpret_cast<const uint4*>(row + c0);
  };
  auto store = [&](void* base, int64_t stride, int64_t row, uint4 v) {
    T* out = static_cast<T*>(base) + row * stride;
    if (!kRagged || inside) {
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
  // every lane of a warp takes the same number of turns
  const int64_t warp_first = (int64_t)blockIdx.x * groups + (threadIdx.x & ~31) / kRow;
  for (int64_t turn = warp_first, row = first; turn < a.p.rows; turn += kRows * step, row += kRows * step) {
    uint4 x[kRows], r[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t at = row + u * step;
      x[u] = r[u] = make_uint4(0u, 0u, 0u, 0u);
      if (at < a.p.rows && mine) {
        x[u] = fetch(X + at * a.p.x_stride);
        if (R) r[u] = fetch(R + at * a.p.r_stride);
      }
    }
    float2 h[kRows][P];
    float m[kRows], mean[kRows];
    auto total = [&] {
#pragma unroll
      for (int o = kRow / 2; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < kRows; ++u) m[u] += __shfl_xor_sync(0xffffffffu, m[u], o);
    };
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      float2 w[P], sum = make_float2(0.f, 0.f);
      Vec<T>::pairs(drop_mask_at<T, kRagged>(x[u], c0, (uint32_t)(row + u * step), key, rate), h[u]);
      Vec<T>::pairs(r[u], w);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        h[u][i] = pair_fma(h[u][i], factor, w[i]);
        sum = pair_add(h[u][i], sum);
      }
      m[u] = sum.x + sum.y;
    }
    total();
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t at = row + u * step;
      if (a.h && at < a.p.rows && mine) store(a.h, a.p.h_stride, at, Vec<T>::pack(h[u]));
      mean[u] = m[u] * inv;
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        h[u][i] = pair_add(h[u][i], make_float2(-mean[u], -mean[u]));
        if (!inside) {
          const int c = c0 + 2 * i;
          if (c < 0 || c >= cols) h[u][i].x = 0.f;
          if (c + 1 < 0 || c + 1 >= cols) h[u][i].y = 0.f;
        }
        sum = pair_fma(h[u][i], h[u][i], sum);
      }
      m[u] = sum.x + sum.y;
    }
    total();
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t at = row + u * step;
      if (at >= a.p.rows || !mine) continue;
      const float rstd = 1.f / sqrtf(m[u] * inv + a.p.eps);
      if (lane == 0) {
        if (a.mean) a.mean[at] = mean[u];
        if (a.rstd) a.rstd[at] = rstd;
      }
#pragma unroll
      for (int i = 0; i < P; ++i) h[u][i] = pair_fma(pair_mul(h[u][i], make_float2(rstd, rstd)), gamma[i], beta[i]);
      store(a.y, a.p.y_stride, at, Vec<T>::pack(h[u]));
    }
  }
}

template <class T, int kRow, int kRows>
void launch_drop_warp(const LnDropArgs& a, bool ragged, cudaStream_t st, cudaError_t* error) {
  constexpr int kSms = 152, kGroup = 32 / kRow;
  // as many warps a block as leave every SM a block, 16 at most; rows of a lane are a multiple of 8 apart
  int warps = 1;
  while (warps < 16 && (a.p.rows + warps * kGroup - 1) / (warps * kGroup) > kSms) warps *= 2;
  const int blocks = (int)std::min<int64_t>((a.p.rows + warps * kGroup - 1) / (warps * kGroup), 2 * kSms);
  if (ragged)
    k_ln_drop_warp<T, kRow, kRows, true><<<blocks, 32 * warps, 0, st>>>(a);
  else
    k_ln_drop_warp<T, kRow, kRows, false><<<blocks, 32 * warps, 0, st>>>(a);
  *error = cudaGetLastError();
}

template <class T, int kRow, int kGroups, int kVpt, int kBlocks, int kCluster>
void launch_drop(const LnDropArgs& a, bool ragged, int* status, unsigned long long wait_ns, cudaStream_t st,
                 cudaError_t* error) {
  constexpr int kSms = 152;
  static_assert(ring_stages(kBlocks, kGroups, kRow * kVpt * 16 * 2) >= 2, "a stage is read while another is filled");
  const int vectors = (int)((a.p.cols + Vec<T>::E - 1) / Vec<T>::E) + (ragged ? 1 : 0);
  const int slots = (vectors + kCluster - 1) / kCluster;
  const int stage = slots * 16 * (a.r ? 2 : 1);
  const int stages = ring_stages(kBlocks, kGroups, stage);
  int groups = 1;  // where rows are few, on as many SMs as there are
  while (groups < kGroups && (a.p.rows + groups - 1) / groups > kSms) groups *= 2;
  // rows of a group are a multiple of 8 apart (4 of the 4-byte type) wherever it has more than one: 304 or 152
  // blocks, 76 clusters or 72
  int most = kBlocks * kSms / kCluster;
  if (ragged && most % (int)(16 / sizeof(T)) != 0) most = most / 8 * 8;
  const int units = (int)std::min<int64_t>((a.p.rows + groups - 1) / groups, most);
  const size_t smem = (size_t)groups * stages * stage;
  auto kernel = ragged ? k_ln_drop<T, kRow, kGroups, kVpt, kBlocks, kCluster, true>
                       : k_ln_drop<T, kRow, kGroups, kVpt, kBlocks, kCluster, false>;
  *error = allow_shared(kernel, smem);
  if (*error != cudaSuccess) return;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)units * kCluster);
  cfg.blockDim = dim3(kRow * groups);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = kCluster, cluster.val.clusterDim.y = 1, cluster.val.clusterDim.z = 1;
  cfg.attrs = &cluster;
  cfg.numAttrs = kCluster > 1 ? 1 : 0;
  *error = cudaLaunchKernelEx(&cfg, kernel, a, stages, slots, status, wait_ns);
}

}  // namespace

template <class T>
bool launch_ln_drop(const LnDropArgs& a, bool ragged, int* status, unsigned long long wait_ns, cudaStream_t st,
                    cudaError_t* error) {
  const int64_t m = (a.p.cols + Vec<T>::E - 1) / Vec<T>::E + (ragged ? 1 : 0);  // vectors of a row, at most
  // Rows of a lane in flight.  64 registers do not hold them: all but one form spill, 36 to 140 bytes.  Against half as
  // many: [131072, 256] bf16 48 us and 53, but [262144, 128] 65 and 53, float32 [131072, 128] 49 and 45; twice as many
  // bf16 rows 58 and 71, float32 ones 49 with one row.
  constexpr int kRows = Vec<T>::E == 8 ? 2 : 4;
  if (m <= 8) return launch_drop_warp<T, 8, kRows>(a, ragged, st, error), true;
  if (m <= 16) return launch_drop_warp<T, 16, kRows>(a, ragged, st, error), true;
  if (m <= 32) return launch_drop_warp<T, 32, kRows>(a, ragged, st, error), true;
  if (m <= 64) return launch_drop<T, 32, 8, 2, 2, 1>(a, ragged, status, wait_ns, st, error), true;
  if (m <= 128) return launch_drop<T, 64, 4, 2, 2, 1>(a, ragged, status, wait_ns, st, error), true;
  if (m <= 256) return launch_drop<T, 128, 2, 2, 2, 1>(a, ragged, status, wait_ns, st, error), true;
  if (m <= 512) return launch_drop<T, 256, 1, 2, 2, 1>(a, ragged, status, wait_ns, st, error), true;
  if (m <= 1024) return launch_drop<T, 512, 1, 2, 1, 1>(a, ragged, status, wait_ns, st, error), true;
  if constexpr (Vec<T>::E == 8) {
    if (m <= 2048) return launch_drop<T, 512, 1, 2, 1, 2>(a, ragged, status, wait_ns, st, error), true;
  } else {
    if (m <= 2048) return launch_drop<T, 512, 1, 4, 1, 1>(a, ragged, status, wait_ns, st, error), true;
    if (m <= 4096) return launch_drop<T, 512, 1, 4, 1, 2>(a, ragged, status, wait_ns, st, error), true;
  }
  return false;
}

}  // namespace gbattn
