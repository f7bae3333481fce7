// The 4-bit key/value cache: argument checks of its three operators, and the
// kernels that quantise rows as they are written and read them back.
//
// Both kernels give a block 16 positions of a few heads, 8 lanes a row: a lane has word i
// of every group, 8 values each, so that rows are read and written in whole lines, a
// position's page is looked up once, and neighbouring positions' (s, b) pairs fill
// their 32-byte sectors.  They are bound by device memory: 2 D bytes in and D / 2 + D / 16
// out for a bf16 row of D values, or the other way round.  Measured: 16 packed prompts of up
// to 8192, 32 heads of 128, written and read back 473 us (5.9 TB/s); 16 of 4096 written 217 us (6.3
// TB/s; with single sums 224: issue slots 75% busy, the arithmetic is next); 131072 tokens of 8 heads
// read 104 us (6.6 TB/s).
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

constexpr int kThreads = 128, kSlots = kThreads / 8;  // positions of a block
constexpr int kWords = 8;                             // code words of a thread: 8 / (D / 64) heads

__device__ __forceinline__ uint32_t min_bf16(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t add_bf16(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16(uint32_t x, uint32_t y, uint32_t z) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
  return r;
}

// Eight values of a row, and the least and largest of them as a pair (low, -high) that
// lanes can join by minima.
template <class T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  using Pair = uint32_t;  // two bf16
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void clear() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ Pair range() const {
    const uint32_t lo = min_bf16(min_bf16(u.x, u.y), min_bf16(u.z, u.w));
    const uint32_t hi = max_bf16(max_bf16(u.x, u.y), max_bf16(u.z, u.w)) ^ 0x80008000u;
    return min_bf16(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
  }
  __device__ static __forceinline__ Pair join(Pair a, Pair b) { return min_bf16(a, b); }
  __device__ static __forceinline__ Pair shuffle(Pair a, int o) { return __shfl_xor_sync(0xffffffffu, a, o); }
  __device__ static __forceinline__ float low(Pair a) { return bf16_lo(a); }
  __device__ static __forceinline__ float high(Pair a) { return -bf16_hi(a); }
  __device__ __forceinline__ float operator[](int i) const {
    const uint32_t w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
    return (i & 1) ? bf16_hi(w) : bf16_lo(w);
  }
};
template <>
struct Eight<float> {
  using Pair = float2;
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p + 4));
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ Pair range() const {
    return make_float2(fminf(fminf(fminf(a.x, a.y), fminf(a.z, a.w)), fminf(fminf(b.x, b.y), fminf(b.z, b.w))),
                       -fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w))));
  }
  __device__ static __forceinline__ Pair join(Pair a, Pair b) { return make_float2(fminf(a.x, b.x), fminf(a.y, b.y)); }
  __device__ static __forceinline__ Pair shuffle(Pair a, int o) {
    return make_float2(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o));
  }
  __device__ static __forceinline__ float low(Pair a) { return a.x; }
  __device__ static __forceinline__ float high(Pair a) { return -a.y; }
  __device__ __forceinline__ float operator[](int i) const {
    const float4& v = i < 4 ? a : b;
    return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
  }
};

// round((x - b) / s) + 8 of eight values in the places of a code word.  The sum with
// 1.5 2^23 + 8 rounds to a whole number, halves to even, and leaves it in the last bits;
// the sums' first bits are taken off together.
template <bool kClamp, class T>
__device__ __forceinline__ uint32_t code_word(const Eight<T>& x, float b, float inv) {
  uint32_t w = 0;
  const Two minus_b = two(-b, -b), last = two(12582920.f, 12582920.f);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    // the products one by one: packed ones would be joined with the sums that follow
    const float2 v = apart(add2(two(x[k], x[k + 1]), minus_b));
    float m0 = __fmul_rn(v.x, inv), m1 = __fmul_rn(v.y, inv);
    if (kClamp) m0 = fminf(fmaxf(m0, -8.f), 7.f), m1 = fminf(fmaxf(m1, -8.f), 7.f);
    const float2 u = apart(add2(two(m0, m1), last));
    w += (__float_as_uint(u.x) << (4 * k)) + (__float_as_uint(u.y) << (4 * k + 4));
  }
  return w - (0x4B400000u + (0x4B400000u << 4) + (0x4B400000u << 8));
}

// Where a thread's rows lie: position slot of the block, heads h0 .. h0 + heads - 1.
struct Place {
  int i, pos, h0, heads;
  long long x0;   // first element of head h0's row in x (or y)
  long long row;  // head h0's row in the cache; -1: none
};
template <int kHeads>
__device__ __forceinline__ Place place_of(const Kv4Args& a, const Kv4Seq& s, int b, int c, long long sb, long long sh,
                                          long long ss) {
  const int head_blocks = (a.heads_kv + kHeads - 1) / kHeads, tile = c / head_blocks;
  Place p;
  p.h0 = (c - tile * head_blocks) * kHeads;
  p.i = tile * kSlots + threadIdx.x / 8;
  p.heads = p.i < s.n ? min(kHeads, a.heads_kv - p.h0) : 0;
  p.pos = s.len - s.n + p.i;
  p.x0 = (a.cu ? (s.row0 + p.i) * ss : b * sb + p.i * ss) + p.h0 * sh;
  p.row = p.heads && p.pos >= 0 ? kv4_row(a, b, p.h0, p.pos) : -1;
  return p;
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads) k_kv4_write(const __grid_constant__ Kv4Args a, int blocks_per_seq) {
  constexpr int G = D / kKv4Group, H = kWords / G;
  using E = Eight<T>;
  const int b = blockIdx.x / blocks_per_seq, lane = threadIdx.x & 31, e = lane & 7;
  const Kv4Seq s = kv4_seq(a, b);
  const bool is_v = blockIdx.y != 0;
  const long long sh = is_v ? a.y_sh : a.x_sh;
  const Place p = place_of<H>(a, s, b, blockIdx.x - b * blocks_per_seq, is_v ? a.y_sb : a.x_sb, sh, is_v ? a.y_ss : a.x_ss);
  if (p.i - (int)threadIdx.x / 8 >= s.n) return;  // the sequence ends before the block
  const T* src = static_cast<const T*>(is_v ? a.y : a.x) + p.x0 + e * 8;
  uint8_t* codes = is_v ? a.vc : a.kc;
  uint32_t* scale = is_v ? a.vs : a.ks;

  E x[kWords];  // word e of group k % G of head h0 + k / G
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    x[k].clear();
    if (p.row >= 0 && k / G < p.heads) x[k].load(src + k / G * sh + k % G * kKv4Group);
  }
  // The groups' ranges: each exchange of lanes halves the groups a lane still joins, so that
  // lane e ends with group e's, and works out its step and offset for all eight.
  typename E::Pair r[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) r[k] = x[k].range();
#pragma unroll
  for (int o = 4; o; o >>= 1)
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const typename E::Pair other = E::shuffle((e & o) ? r[k] : r[k + o], o);
      r[k] = E::join((e & o) ? r[k + o] : r[k], other);
    }
  const float lo = E::low(r[0]), hi = E::high(r[0]);
  float st = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f)));
  if (st < 1.1754943508222875e-38f) st = 0.f;  // 2^-126: its reciprocal would not be finite
  const float ce = __bfloat162float(__float2bfloat16_rn(__fadd_rn(lo, 8.f * st)));
  const float inv = st > 0.f ? __frcp_rn(st) : 0.f;
  const uint32_t sb = (__float_as_uint(st) >> 16) | (__float_as_uint(ce) & 0xFFFF0000u);
  if (p.row >= 0 && e / G < p.heads) scale[(p.row + (long long)(e / G) * a.page) * G + e % G] = sb;
  // b's rounding may have moved the ends past the codes: then every value is held to them
  const bool inside = __fmul_rn(__fsub_rn(lo, ce), inv) >= -8.5f && __fmul_rn(__fsub_rn(hi, ce), inv) < 7.5f;
  const bool clamp = !__all_sync(0xffffffffu, inside);
  uint32_t w[kWords];
  float bk[kWords], ik[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) bk[k] = __shfl_sync(0xffffffffu, ce, k, 8), ik[k] = __shfl_sync(0xffffffffu, inv, k, 8);
  if (clamp) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = code_word<true>(x[k], bk[k], ik[k]);
  } else {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = code_word<false>(x[k], bk[k], ik[k]);
  }
#pragma unroll
  for (int u = 0; u < H; ++u)
    if (p.row >= 0 && u < p.heads) {
      uint8_t* to = codes + (p.row + (long long)u * a.page) * (D / 2) + e * (4 * G);
      if constexpr (G == 1) *reinterpret_cast<uint32_t*>(to) = w[u];
      if constexpr (G == 2) *reinterpret_cast<uint2*>(to) = make_uint2(w[2 * u], w[2 * u + 1]);
      if constexpr (G == 4)
        *reinterpret_cast<uint4*>(to) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
    }
}

// A code word's eight values.
__device__ __forceinline__ void store_values(__nv_bfloat16* p, uint32_t w, uint32_t sb) {
  // 0x4300 is 128 in bf16, its last bit 1: codes by bit operations, minus 136, both exact; the
  // product's sum with b is rounded once
  const uint32_t s2 = __byte_perm(sb, sb, 0x1010), b2 = __byte_perm(sb, sb, 0x3232);
  uint32_t v[4];  // values k and k + 4
#pragma unroll
  for (int k = 0; k < 4; ++k)
    v[k] = fma_bf16(s2, add_bf16(((w >> (4 * k)) & 0x000F000Fu) | 0x43004300u, 0xC308C308u), b2);
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                                                 __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632)));
}
__device__ __forceinline__ void store_values(float* p, uint32_t w, uint32_t sb) {
  const float s = bf16_lo(sb), b = bf16_hi(sb);
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)  // 2^23 + u by bit operations, minus 2^23 + 8
    v[k] = fmaf(s, __uint_as_float(((w >> (4 * k)) & 15u) | 0x4B000000u) - 8388616.f, b);
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(p + 4), make_float4(v[4], v[5], v[6], v[7]));
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads) k_kv4_read(const __grid_constant__ Kv4Args a, int blocks_per_seq) {
  constexpr int G = D / kKv4Group, H = kWords / G;
  const int b = blockIdx.x / blocks_per_seq, e = threadIdx.x & 7;
  const Kv4Seq s = kv4_seq(a, b);
  const bool is_v = blockIdx.y != 0;
  const long long sh = is_v ? a.y_sh : a.x_sh;
  const Place p = place_of<H>(a, s, b, blockIdx.x - b * blocks_per_seq, is_v ? a.y_sb : a.x_sb, sh, is_v ? a.y_ss : a.x_ss);
  if (p.i - (int)threadIdx.x / 8 >= s.n) return;  // the sequence ends before the block
  T* dst = static_cast<T*>(is_v ? a.y : a.x) + p.x0 + e * 8;
  const uint8_t* codes = is_v ? a.vc : a.kc;
  const uint32_t* scale = is_v ? a.vs : a.ks;

  uint32_t w[kWords], sb[kWords];
#pragma unroll
  for (int u = 0; u < H; ++u) {
#pragma unroll
    for (int g = 0; g < G; ++g) w[u * G + g] = sb[u * G + g] = 0;  // padding: values 0
    if (p.row >= 0 && u < p.heads) {
      const long long row = p.row + (long long)u * a.page;
      const uint8_t* from = codes + row * (D / 2) + e * (4 * G);
      if constexpr (G == 1) {
        w[u] = __ldcs(reinterpret_cast<const uint32_t*>(from));
        sb[u] = __ldg(scale + row);
      }
      if constexpr (G == 2) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(from)), t = __ldg(reinterpret_cast<const uint2*>(scale + row * 2));
        w[2 * u] = v.x, w[2 * u + 1] = v.y, sb[2 * u] = t.x, sb[2 * u + 1] = t.y;
      }
      if constexpr (G == 4) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(from)), t = __ldg(reinterpret_cast<const uint4*>(scale + row * 4));
        w[4 * u] = v.x, w[4 * u + 1] = v.y, w[4 * u + 2] = v.z, w[4 * u + 3] = v.w;
        sb[4 * u] = t.x, sb[4 * u + 1] = t.y, sb[4 * u + 2] = t.z, sb[4 * u + 3] = t.w;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kWords; ++k)
    if (k / G < p.heads) store_values(dst + k / G * sh + k % G * kKv4Group, w[k], sb[k]);
}

long long blocks_per_seq(int seqlen, int heads_kv, int head_dim) {
  const int heads = kWords / (head_dim / kKv4Group);
  return ((long long)seqlen + kSlots - 1) / kSlots * (((long long)heads_kv + heads - 1) / heads);
}

template <class F>
cudaError_t launch_rows(const Kv4Args& a, int head_dim, F&& kernel, cudaStream_t st) {
  const long long per_seq = blocks_per_seq(a.seqlen, a.heads_kv, head_dim);
  kernel<<<dim3((unsigned)(per_seq * a.batch), 2), kThreads, 0, st>>>(a, (int)per_seq);
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

enum class Op { kWrite, kRead, kAttend };

// Checks everything about the parameters that no data pointer is needed for and
// fills the kernels' arguments; *empty: there is no row to deal with.
attn_status_t resolve(const attn_kv4_params_t* p, Op op, Kv4Args* a, bool* empty) {
  const bool attention = op == Op::kAttend;
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
  // Quotients: a product of three counts may not fit 64 bits.
  if (total > 0x7FFFFFFFll / heads)
    return kfail(ATTN_ERR_UNSUPPORTED, "%lld rows of %d heads: at most 2^31 - 1 over all heads are supported", total, heads);
  const int seqlen = (int)std::min<long long>(p->seqlen, total);  // a packed sequence has no more rows than all
  if (!attention && p->batch > 0x7FFFFFFFll / blocks_per_seq(seqlen, heads, p->head_dim))
    return kfail(ATTN_ERR_UNSUPPORTED, "%d packed sequences of up to %d rows: too many blocks of 16 rows", p->batch, seqlen);
  if (attention) {  // the attention counts its rows, positions and the cache's rows in 32 bits
    if (total > (1ll << 30) / heads)
      return kfail(ATTN_ERR_UNSUPPORTED, "%lld query rows of %d heads: at most 2^30 over all heads are supported", total,
                   heads);
    if ((long long)p->max_pages * p->page_size > (1ll << 30))
      return kfail(ATTN_ERR_UNSUPPORTED, "max_pages * page_size = %lld: at most 2^30 positions of a sequence are supported",
                   (long long)p->max_pages * p->page_size);
    if ((long long)p->n_pages * p->page_size > 0xFFFFFFFFll / p->heads_kv)
      return kfail(ATTN_ERR_UNSUPPORTED, "n_pages=%d times heads_kv=%d times page_size=%d: fewer than 2^32 rows are supported",
                   p->n_pages, p->heads_kv, p->page_size);
  }
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
    const long long entries = i % 3 == 0 ? p->batch : i % 3 == 1 ? heads : p->cu_seqlens ? total : p->seqlen;
    const bool output = op == Op::kRead || (op == Op::kAttend && i >= 3);
    if (output && entries > 1 && strides[i] < p->head_dim)
      return kfail(ATTN_ERR_INVALID_ARG, "%s=%lld over %lld entries: rows of an output must not overlap", names[i],
                   strides[i], entries);
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
  a->by_group = fast_div(a->group);
  a->seqlen = seqlen;
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

size_t attention_workspace(const Kv4Args& a, int head_dim, bool bf16) {
  return kv4_many_rows(a, head_dim, bf16) ? kv4_rows_workspace(a, head_dim) : kv4_attn_workspace(a, head_dim, bf16);
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
  attn_status_t s = resolve(p, Op::kWrite, &a, &empty);
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
  attn_status_t s = resolve(p, Op::kRead, &a, &empty);
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
  if (resolve(p, Op::kAttend, &a, &empty) != ATTN_OK) return SIZE_MAX;
  return empty ? 0 : attention_workspace(a, p->head_dim, p->dtype == ATTN_BF16);
}

attn_status_t attn_fwd_kv4(const attn_kv4_params_t* p, const void* x, const void* k_codes, const void* k_scale,
                           const void* v_codes, const void* v_scale, void* y, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  Kv4Args a;
  bool empty = false;
  attn_status_t s = resolve(p, Op::kAttend, &a, &empty);
  if (s != ATTN_OK || empty) return s;
  if ((s = check_pointers(p, x, y, k_codes, k_scale, v_codes, v_scale))) return s;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return kfail(ATTN_ERR_INVALID_ARG, "lse is NULL or not 4-byte aligned");
  const bool bf16 = p->dtype == ATTN_BF16;
  const size_t need = attention_workspace(a, p->head_dim, bf16);
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_status(kv4_many_rows(a, p->head_dim, bf16) ? launch_kv4_rows(a, p->head_dim, workspace, wait_ns, st)
                                                           : launch_kv4_attn(a, p->head_dim, bf16, workspace, st),
                       "cache attention launch");
}

}  // extern "C"
