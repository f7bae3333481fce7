// The 4-bit key/value cache: argument checks of its three operators, and the
// kernels that quantise rows as they are written and read them back.
//
// Both kernels give a thread one 32-bit code word, 8 values: 16 (bf16) or 32
// (float32) bytes of a row on one side and 4 on the other, so that a warp's loads
// and stores cover whole rows.  They are bound by device memory: 2 D bytes in and
// D / 2 + D / 16 out for a bf16 row of D values, or the other way round.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/gbkv4.h"
#include "kv4.h"
#include "ptx.cuh"

namespace gbattn {
void set_last_error_text(const char* text);
attn_status_t device_status(int** status, int* sms, unsigned long long* wait_ns);

namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerThread = 4;  // rows whose loads a thread issues before it uses the first

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(ptx::pack_bf16x2(v[0], v[1]), ptx::pack_bf16x2(v[2], v[3]),
                                            ptx::pack_bf16x2(v[4], v[5]), ptx::pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Row r of a sequence, counted along memory: position-major heads when packed
// ([tokens, heads, D]), head-major otherwise ([heads, seqlen, D]).
__device__ __forceinline__ void split_row(const Kv4Args& a, const Kv4Seq& s, int r, int* h, int* i) {
  if (a.cu) {
    *i = r / a.heads_kv;
    *h = r - *i * a.heads_kv;
  } else {
    *h = r / s.n;
    *i = r - *h * s.n;
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads) k_kv4_write(const __grid_constant__ Kv4Args a, int blocks_per_seq) {
  constexpr int L = D / 8;             // threads of a row
  constexpr int R = kThreads / L;      // rows of the block at a time
  constexpr int G = D / kKv4Group;
  const int b = blockIdx.x / blocks_per_seq;
  const Kv4Seq s = kv4_seq(a, b);
  const int rows = s.n * a.heads_kv;
  const int r0 = (blockIdx.x - b * blocks_per_seq) * (R * kRowsPerThread) + threadIdx.x / L;
  const int e = threadIdx.x % L;  // values 8 e .. 8 e + 7: word i = e % 8 of group g = e / 8
  const bool is_v = blockIdx.y != 0;
  const T* src = static_cast<const T*>(is_v ? a.y : a.x);
  const long long sb = is_v ? a.y_sb : a.x_sb, sh = is_v ? a.y_sh : a.x_sh, ss = is_v ? a.y_ss : a.x_ss;
  uint8_t* codes = is_v ? a.vc : a.kc;
  uint32_t* scale = is_v ? a.vs : a.ks;

  float x[kRowsPerThread][8];
  long long row[kRowsPerThread];
#pragma unroll
  for (int j = 0; j < kRowsPerThread; ++j) {
    const int r = r0 + j * R;
    row[j] = -1;
#pragma unroll
    for (int k = 0; k < 8; ++k) x[j][k] = 0.f;
    if (r < rows) {
      int h, i;
      split_row(a, s, r, &h, &i);
      const int pos = s.len - s.n + i;
      if (pos >= 0) {
        load8(src + (a.cu ? (s.row0 + i) * ss : b * sb + i * ss) + h * sh + e * 8, x[j]);
        row[j] = kv4_row(a, b, h, pos);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kRowsPerThread; ++j) {
    float lo = x[j][0], hi = x[j][0];
#pragma unroll
    for (int k = 1; k < 8; ++k) lo = fminf(lo, x[j][k]), hi = fmaxf(hi, x[j][k]);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {  // the group's 8 threads
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    float st = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f)));
    if (st < 1.1754943508222875e-38f) st = 0.f;  // 2^-126: its reciprocal would not be finite
    const float ce = __bfloat162float(__float2bfloat16_rn(__fadd_rn(lo, 8.f * st)));
    const float inv = st > 0.f ? __fdiv_rn(1.f, st) : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float u = fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(x[j][k], ce), inv)) + 8.f, 0.f), 15.f);
      w |= (uint32_t)u << (4 * k);
    }
    if (row[j] >= 0) {
      *reinterpret_cast<uint32_t*>(codes + row[j] * (D / 2) + ((e & 7) * G + (e >> 3)) * 4) = w;
      if ((e & 7) == 0) scale[row[j] * G + (e >> 3)] = (__float_as_uint(st) >> 16) | (__float_as_uint(ce) & 0xFFFF0000u);
    }
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads) k_kv4_read(const __grid_constant__ Kv4Args a, int blocks_per_seq) {
  constexpr int L = D / 8, R = kThreads / L, G = D / kKv4Group;
  const int b = blockIdx.x / blocks_per_seq;
  const Kv4Seq s = kv4_seq(a, b);
  const int rows = s.n * a.heads_kv;
  const int r0 = (blockIdx.x - b * blocks_per_seq) * (R * kRowsPerThread) + threadIdx.x / L;
  const int e = threadIdx.x % L;  // stored word e: word i = e / G of group g = e % G
  const int g = e % G, d0 = g * kKv4Group + e / G * 8;
  const bool is_v = blockIdx.y != 0;
  T* dst = static_cast<T*>(is_v ? a.y : a.x);
  const long long sb = is_v ? a.y_sb : a.x_sb, sh = is_v ? a.y_sh : a.x_sh, ss = is_v ? a.y_ss : a.x_ss;
  const uint8_t* codes = is_v ? a.vc : a.kc;
  const uint32_t* scale = is_v ? a.vs : a.ks;

  uint32_t w[kRowsPerThread], sc[kRowsPerThread];
  T* out[kRowsPerThread];
#pragma unroll
  for (int j = 0; j < kRowsPerThread; ++j) {
    const int r = r0 + j * R;
    w[j] = sc[j] = 0;
    out[j] = nullptr;
    if (r < rows) {
      int h, i;
      split_row(a, s, r, &h, &i);
      const int pos = s.len - s.n + i;
      out[j] = dst + (a.cu ? (s.row0 + i) * ss : b * sb + i * ss) + h * sh + d0;
      const long long row = pos >= 0 ? kv4_row(a, b, h, pos) : -1;
      if (row >= 0) {
        w[j] = *reinterpret_cast<const uint32_t*>(codes + row * (D / 2) + e * 4);
        sc[j] = scale[row * G + g];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kRowsPerThread; ++j) {
    if (!out[j]) continue;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = fmaf(bf16_lo(sc[j]), (float)(int)((w[j] >> (4 * k)) & 15u) - 8.f, bf16_hi(sc[j]));
    store8(out[j], v);
  }
}

template <class F>
cudaError_t launch_rows(const Kv4Args& a, int head_dim, F&& kernel, cudaStream_t st) {
  const int per_block = kThreads / (head_dim / 8) * kRowsPerThread;
  const long long rows = (long long)a.seqlen * a.heads_kv, per_seq = (rows + per_block - 1) / per_block;
  const long long blocks = per_seq * a.batch;
  if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  kernel<<<dim3((unsigned)blocks, 2), kThreads, 0, st>>>(a, (int)per_seq);
  return cudaGetLastError();
}

attn_status_t kfail(attn_status_t s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
attn_status_t kfail(attn_status_t s, const char* fmt, ...) {
  char buf[320];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error_text(buf);
  return s;
}

// Checks everything about the parameters that no data pointer is needed for and
// fills the kernels' arguments; *empty: there is no row to deal with.
attn_status_t resolve(const attn_kv4_params_t* p, bool attention, Kv4Args* a, bool* empty) {
  std::memset(a, 0, sizeof(*a));
  set_last_error_text("");
  if (!p) return kfail(ATTN_ERR_INVALID_ARG, "params is NULL");
  if (p->dtype != ATTN_F32 && p->dtype != ATTN_BF16)
    return kfail(ATTN_ERR_INVALID_ARG, "dtype %d is not ATTN_F32 or ATTN_BF16", (int)p->dtype);
  if (p->heads_kv <= 0 || (attention && p->heads_q <= 0))
    return kfail(ATTN_ERR_INVALID_ARG, "heads_q=%d and heads_kv=%d must be positive", p->heads_q, p->heads_kv);
  if (attention && p->heads_q % p->heads_kv)
    return kfail(ATTN_ERR_INVALID_ARG, "heads_q=%d is not a multiple of heads_kv=%d", p->heads_q, p->heads_kv);
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256)
    return kfail(ATTN_ERR_UNSUPPORTED, "head_dim=%d: only 64, 128 and 256 are implemented", p->head_dim);
  if (p->page_size <= 0 || p->page_size % 16)
    return kfail(ATTN_ERR_INVALID_ARG, "page_size=%d must be a positive multiple of 16", p->page_size);
  if (p->batch < 0 || p->seqlen < 0 || p->n_pages < 0 || p->max_pages < 0)
    return kfail(ATTN_ERR_INVALID_ARG, "batch=%d, seqlen=%d, n_pages=%d or max_pages=%d is negative", p->batch, p->seqlen,
                 p->n_pages, p->max_pages);
  if (attention && !std::isfinite(p->scale)) return kfail(ATTN_ERR_INVALID_ARG, "scale is not finite");
  long long total = (long long)p->batch * p->seqlen;
  if (p->cu_seqlens) {
    if (!p->cu_seqlens_host) return kfail(ATTN_ERR_INVALID_ARG, "cu_seqlens_host is required with cu_seqlens");
    if (p->cu_seqlens_host[0] != 0)
      return kfail(ATTN_ERR_INVALID_ARG, "cu_seqlens[0]=%d must be 0", p->cu_seqlens_host[0]);
    for (int n = 0; n < p->batch; ++n) {
      const long long t = (long long)p->cu_seqlens_host[n + 1] - p->cu_seqlens_host[n];
      if (t < 0) return kfail(ATTN_ERR_INVALID_ARG, "cu_seqlens decreases at %d", n);
      if (t > p->seqlen)
        return kfail(ATTN_ERR_INVALID_ARG, "sequence %d has %lld rows > seqlen %d", n, t, p->seqlen);
    }
    total = p->cu_seqlens_host[p->batch];
  }
  *empty = total == 0;
  if (*empty) return ATTN_OK;  // nothing is read or written
  const int heads = attention ? p->heads_q : p->heads_kv;
  if (total * heads >= (1ll << 31) || (long long)p->seqlen * heads * p->batch >= (1ll << 31))
    return kfail(ATTN_ERR_UNSUPPORTED, "%lld rows over all heads: at most 2^31 - 1 are supported",
                 std::max(total, (long long)p->seqlen * p->batch) * heads);
  if (!p->lens) return kfail(ATTN_ERR_INVALID_ARG, "lens is NULL");
  if (p->max_pages > 0 && !p->block_table) return kfail(ATTN_ERR_INVALID_ARG, "block_table is NULL");
  if (p->table_stride < p->max_pages && p->batch > 1)
    return kfail(ATTN_ERR_INVALID_ARG, "table_stride=%lld is smaller than max_pages=%d", (long long)p->table_stride,
                 p->max_pages);
  const int align = p->dtype == ATTN_BF16 ? 8 : 4;
  const long long strides[6] = {p->x_stride_b, p->x_stride_h, p->x_stride_s, p->y_stride_b, p->y_stride_h, p->y_stride_s};
  const char* names[6] = {"x_stride_b", "x_stride_h", "x_stride_s", "y_stride_b", "y_stride_h", "y_stride_s"};
  for (int i = 0; i < 6; ++i) {
    if (p->cu_seqlens && i % 3 == 0) continue;
    if (strides[i] < 0 || strides[i] % align)
      return kfail(ATTN_ERR_INVALID_ARG, "%s=%lld must be a non-negative multiple of %d elements", names[i], strides[i],
                   align);
  }
  a->table = p->block_table;
  a->table_stride = p->table_stride;
  a->lens = p->lens;
  a->cu = p->cu_seqlens;
  a->total = total;
  a->batch = p->batch;
  a->heads_q = p->heads_q;
  a->heads_kv = p->heads_kv;
  a->group = attention ? p->heads_q / p->heads_kv : 1;
  a->seqlen = p->seqlen;
  a->page = p->page_size;
  a->n_pages = p->n_pages;
  a->max_pages = p->max_pages;
  a->x_sb = p->x_stride_b, a->x_sh = p->x_stride_h, a->x_ss = p->x_stride_s;
  a->y_sb = p->y_stride_b, a->y_sh = p->y_stride_h, a->y_ss = p->y_stride_s;
  a->scale_log2 = (float)((double)p->scale * 1.4426950408889634);
  a->causal = p->causal ? 1 : 0;
  return ATTN_OK;
}

// Data pointers of one call; the cache's arrays may be NULL only if it has no page.
attn_status_t check_pointers(const attn_kv4_params_t* p, const void* x, const void* y, const void* kc, const void* ks,
                             const void* vc, const void* vs) {
  const void* ptr[6] = {x, y, kc, ks, vc, vs};
  const char* names[6] = {"x", "y", "k_codes", "k_scale", "v_codes", "v_scale"};
  for (int i = 0; i < 6; ++i) {
    if (!ptr[i] && (i < 2 || p->n_pages > 0)) return kfail(ATTN_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (reinterpret_cast<uintptr_t>(ptr[i]) & 15u)
      return kfail(ATTN_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  return ATTN_OK;
}

attn_status_t launch_status(cudaError_t e, const char* what) {
  return e == cudaSuccess ? ATTN_OK : kfail(ATTN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4Args& a, int head_dim, bool bf16, cudaStream_t st) {
  if (bf16) {
    if (head_dim == 64) return launch_rows(a, 64, k_kv4_write<__nv_bfloat16, 64>, st);
    if (head_dim == 128) return launch_rows(a, 128, k_kv4_write<__nv_bfloat16, 128>, st);
    return launch_rows(a, 256, k_kv4_write<__nv_bfloat16, 256>, st);
  }
  if (head_dim == 64) return launch_rows(a, 64, k_kv4_write<float, 64>, st);
  if (head_dim == 128) return launch_rows(a, 128, k_kv4_write<float, 128>, st);
  return launch_rows(a, 256, k_kv4_write<float, 256>, st);
}

cudaError_t launch_kv4_read(const Kv4Args& a, int head_dim, bool bf16, cudaStream_t st) {
  if (bf16) {
    if (head_dim == 64) return launch_rows(a, 64, k_kv4_read<__nv_bfloat16, 64>, st);
    if (head_dim == 128) return launch_rows(a, 128, k_kv4_read<__nv_bfloat16, 128>, st);
    return launch_rows(a, 256, k_kv4_read<__nv_bfloat16, 256>, st);
  }
  if (head_dim == 64) return launch_rows(a, 64, k_kv4_read<float, 64>, st);
  if (head_dim == 128) return launch_rows(a, 128, k_kv4_read<float, 128>, st);
  return launch_rows(a, 256, k_kv4_read<float, 256>, st);
}

}  // namespace gbattn

using namespace gbattn;

extern "C" {

attn_status_t attn_kv4_write(const attn_kv4_params_t* p, const void* x, const void* y, void* k_codes, void* k_scale,
                             void* v_codes, void* v_scale, void* stream) {
  Kv4Args a;
  bool empty = false;
  attn_status_t s = resolve(p, false, &a, &empty);
  if (s != ATTN_OK || empty) return s;
  if ((s = check_pointers(p, x, y, k_codes, k_scale, v_codes, v_scale))) return s;
  int sms = 0;
  unsigned long long wait_ns = 0;
  if ((s = device_status(&a.status, &sms, &wait_ns))) return s;
  a.x = const_cast<void*>(x);
  a.y = const_cast<void*>(y);
  a.kc = static_cast<uint8_t*>(k_codes);
  a.ks = static_cast<uint32_t*>(k_scale);
  a.vc = static_cast<uint8_t*>(v_codes);
  a.vs = static_cast<uint32_t*>(v_scale);
  return launch_status(launch_kv4_write(a, p->head_dim, p->dtype == ATTN_BF16, static_cast<cudaStream_t>(stream)),
                       "cache write launch");
}

attn_status_t attn_kv4_read(const attn_kv4_params_t* p, const void* k_codes, const void* k_scale, const void* v_codes,
                            const void* v_scale, void* x, void* y, void* stream) {
  Kv4Args a;
  bool empty = false;
  attn_status_t s = resolve(p, false, &a, &empty);
  if (s != ATTN_OK || empty) return s;
  if ((s = check_pointers(p, x, y, k_codes, k_scale, v_codes, v_scale))) return s;
  int sms = 0;
  unsigned long long wait_ns = 0;
  if ((s = device_status(&a.status, &sms, &wait_ns))) return s;
  a.x = x;
  a.y = y;
  a.kc = static_cast<uint8_t*>(const_cast<void*>(k_codes));
  a.ks = static_cast<uint32_t*>(const_cast<void*>(k_scale));
  a.vc = static_cast<uint8_t*>(const_cast<void*>(v_codes));
  a.vs = static_cast<uint32_t*>(const_cast<void*>(v_scale));
  return launch_status(launch_kv4_read(a, p->head_dim, p->dtype == ATTN_BF16, static_cast<cudaStream_t>(stream)),
                       "cache read launch");
}

size_t attn_kv4_workspace_size(const attn_kv4_params_t* p) {
  Kv4Args a;
  bool empty = false;
  if (resolve(p, true, &a, &empty) != ATTN_OK) return SIZE_MAX;
  return empty ? 0 : kv4_attn_workspace(a, p->head_dim, p->dtype == ATTN_BF16);
}

attn_status_t attn_fwd_kv4(const attn_kv4_params_t* p, const void* x, const void* k_codes, const void* k_scale,
                           const void* v_codes, const void* v_scale, void* y, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  Kv4Args a;
  bool empty = false;
  attn_status_t s = resolve(p, true, &a, &empty);
  if (s != ATTN_OK || empty) return s;
  if ((s = check_pointers(p, x, y, k_codes, k_scale, v_codes, v_scale))) return s;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return kfail(ATTN_ERR_INVALID_ARG, "lse is NULL or not 4-byte aligned");
  const bool bf16 = p->dtype == ATTN_BF16;
  const size_t need = kv4_attn_workspace(a, p->head_dim, bf16);
  if (need && !workspace) return kfail(ATTN_ERR_WORKSPACE, "workspace is NULL but %zu bytes are needed", need);
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return kfail(ATTN_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (workspace_bytes < need)
    return kfail(ATTN_ERR_WORKSPACE, "workspace has %zu bytes, %zu are needed", workspace_bytes, need);
  int sms = 0;
  unsigned long long wait_ns = 0;
  if ((s = device_status(&a.status, &sms, &wait_ns))) return s;
  a.x = const_cast<void*>(x);
  a.y = y;
  a.lse = lse;
  a.kc = static_cast<uint8_t*>(const_cast<void*>(k_codes));
  a.ks = static_cast<uint32_t*>(const_cast<void*>(k_scale));
  a.vc = static_cast<uint8_t*>(const_cast<void*>(v_codes));
  a.vs = static_cast<uint32_t*>(const_cast<void*>(v_scale));
  return launch_status(launch_kv4_attn(a, p->head_dim, bf16, workspace, static_cast<cudaStream_t>(stream)),
                       "cache attention launch");
}

}  // extern "C"
