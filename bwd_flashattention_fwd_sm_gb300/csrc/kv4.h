// The 4-bit key/value cache: what its kernels share.  Internal to the library
// (the public interface is include/gbkv4.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace gbattn {

constexpr int kKv4Group = 64;  // values that share one (s, b) pair

// n / d for 0 <= n < 2^31: (n * mul) >> shift with mul = floor(2^shift / d) + 1.
struct FastDiv {
  uint32_t mul, shift;
};
inline FastDiv fast_div(int d) {
  int l = 0;
  while ((1ll << l) < d) ++l;
  return {(uint32_t)((1ull << (31 + l)) / (uint32_t)d + 1), (uint32_t)(31 + l)};
}
__device__ __forceinline__ int div_by(int n, FastDiv d) {
  return (int)(((unsigned long long)(uint32_t)n * d.mul) >> d.shift);
}

// Everything a kernel needs, resolved on the host.  Strides in elements.
struct Kv4Args {
  uint8_t* kc;   // codes [n_pages, heads_kv, page, D / 2]
  uint8_t* vc;
  uint32_t* ks;  // (s, b) pairs [n_pages, heads_kv, page, D / 64], s in the low half
  uint32_t* vs;
  const int* table;
  long long table_stride;
  const int* lens;
  const int* cu;         // NULL: fixed length
  long long total;       // packed rows
  int batch, heads_q, heads_kv, group, seqlen, page, n_pages, max_pages;
  FastDiv by_group;  // group, as a divisor
  void* x;
  void* y;
  float* lse;
  long long x_sb, x_sh, x_ss, y_sb, y_sh, y_ss;
  float scale_log2;  // scale * log2(e)
  int causal;
  int* status;
};

// One sequence's rows in x and y and its length in the cache.
struct Kv4Seq {
  int n;           // rows; row i sits at position len - n + i
  int len;         // positions, cut to what the page list can hold
  long long row0;  // packed: first row
};

// What only the device knows is checked by the two functions below: *bad is set,
// and the sequence has no rows, or the row is -1.
__host__ __device__ inline Kv4Seq kv4_seq_of(const Kv4Args& a, int b, bool* bad) {
  Kv4Seq s;
  s.n = a.seqlen;
  s.row0 = 0;
  if (a.cu) {
    const int r0 = a.cu[b], r1 = a.cu[b + 1];
    const bool ok = r0 >= 0 && r1 >= r0 && r1 <= a.total && r1 - r0 <= a.seqlen;
    if (!ok) *bad = true;
    s.n = ok ? r1 - r0 : 0;
    s.row0 = r0;
  }
  const long long room = (long long)a.max_pages * a.page, most = room < 0x7FFFFFFF ? room : 0x7FFFFFFF;
  const int len = a.lens[b];
  if (len < 0 || len > most) *bad = true;
  s.len = len < 0 ? 0 : (len > most ? (int)most : len);
  return s;
}

// Row of position `pos` (below the sequence's length) and head h in the cache, as
// an index over [n_pages, heads_kv, page].
__host__ __device__ inline long long kv4_row_index(const Kv4Args& a, int b, int h, int pos, bool* bad) {
  const int pid = a.table[b * a.table_stride + pos / a.page];
  if (pid < 0 || pid >= a.n_pages) {
    *bad = true;
    return -1;
  }
  return ((long long)pid * a.heads_kv + h) * a.page + pos % a.page;
}

__device__ __forceinline__ Kv4Seq kv4_seq(const Kv4Args& a, int b) {
  bool bad = false;
  const Kv4Seq s = kv4_seq_of(a, b, &bad);
  if (bad) set_status(a.status, kStatusBounds);
  return s;
}

__device__ __forceinline__ long long kv4_row(const Kv4Args& a, int b, int h, int pos) {
  bool bad = false;
  const long long row = kv4_row_index(a, b, h, pos, &bad);
  if (bad) set_status(a.status, kStatusBounds);
  return row;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Whether both bf16 numbers of a pair are finite.
__device__ __forceinline__ bool finite2(uint32_t w) {
  return (((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u) == 0;  // an exponent of ones carries
}

// Two float32 numbers at a time.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float x, float y) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 apart(Two x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ Two fma2(Two x, Two y, Two z) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ Two mul2(Two x, Two y) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ Two add2(Two x, Two y) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

cudaError_t launch_kv4_write(const Kv4Args& a, int head_dim, bool bf16, cudaStream_t st);
cudaError_t launch_kv4_read(const Kv4Args& a, int head_dim, bool bf16, cudaStream_t st);

// Attention over the cache: device scratch for these shapes, and the launch.  Few query
// rows on a KV head: any type and head dim.  Many: bf16, head dim 64 or 128.
size_t kv4_attn_workspace(const Kv4Args& a, int head_dim, bool bf16);
cudaError_t launch_kv4_attn(const Kv4Args& a, int head_dim, bool bf16, void* workspace, cudaStream_t st);
size_t kv4_rows_workspace(const Kv4Args& a, int head_dim);
cudaError_t launch_kv4_rows(const Kv4Args& a, int head_dim, void* workspace, unsigned long long wait_ns, cudaStream_t st);

// Which of the two: the tcgen05 kernel from 25 rows on.  Measured with 16 sequences of up to
// 4096 positions (32 query heads on 8, head dim 128; us): 24 rows 49 against 48, 32 rows
// 77 against 47, 128 rows 172 against 55.
inline bool kv4_many_rows(const Kv4Args& a, int head_dim, bool bf16) {
  return bf16 && head_dim <= 128 && (long long)a.seqlen * a.group > 24;
}

}  // namespace gbattn
