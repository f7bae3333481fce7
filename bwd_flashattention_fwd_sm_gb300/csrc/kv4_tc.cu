// Attention over the 4-bit key/value cache for many query rows: a prompt's chunk, or
// a few proposed tokens of a large group of heads.
//
// Here the products bound, not the cache's bytes, and unpacking a key must not be
// repeated for every few queries: 128 query rows of a KV head meet 128 keys on tcgen05
// instructions, with the row sums in tensor memory.  Four warps unpack each tile once
// into shared memory (128-byte rows of 64 values, swizzled, one box for each group
// of 64):
//   K: pairs of codes as float16 subnormals, u 2^-24 from a word's even values and
//      u 2^-20 from the odd ones, five operations for eight codes.  Q is float16 in
//      each row's own power of two, in the same order, its odd values scaled by 1/16.
//   V: codes as bfloat16 integers -8 .. 7.
// Each group has its own score product, so that a key's step and offset are applied to
// float32 sums: x = sum_g s_g C_g + (b_g - 8 s_g) sum(q_g), exact but for float32
// roundings.  The weights p s_g are rounded once to bfloat16 (2^-8 of themselves at
// most) and multiply V group by group; the offsets' part sum(p b_g) and the row sums
// stay in float32.
//
// Sixteen warps do the softmax, four for each 32 rows with a quarter of the keys each;
// the scores of tile t + 1 are computed while they work on tile t.  The running maximum
// is raised only when a score is above it by more than 2^8; the four warps of a row
// agree on that with one barrier a tile.  What bounds it: about 14 instructions an element
// in the softmax warps, against 4 D of a product's operations.  Blocks share the work
// by equal stretches of one line of tiles, as for few rows (kv4_attn.cu).
#include <algorithm>
#include <atomic>

#include "kv4_line.cuh"
#include "ptx.cuh"

namespace gbattn {

namespace {

constexpr int kRows = 128, kKeys = 128, kSpare = 2;  // kSpare: what a row tile costs beside its keys, in tiles
constexpr int kParts = 4, kPart = kKeys / kParts;  // warps of a row, and the keys of each
// four warps of each 32 rows, four that unpack, and four of which one issues the products
constexpr int kSoftWarps = 4 * kParts, kUnpackWarps = 4, kWarps = kSoftWarps + kUnpackWarps + 4;
constexpr int kThreads = kWarps * 32;
// Registers: 80 a thread at launch; what the issuing warps give up the softmax warps take
// (512 * 88 + 128 * 72 + 128 * 56 = 768 * 80).
constexpr int kSoftRegs = 88, kUnpackRegs = 72, kIssueRegs = 56;

template <int D>
struct Smem {
  static constexpr int G = D / kKv4Group;
  uint8_t q[G][kRows * 128];  // float16, 128-byte rows, 128-byte swizzle
  uint8_t k[2][G][kKeys * 128];
  uint8_t v[2][G][kKeys * 128];
  float4 ksz[2][G][kKeys / 2];  // s and b - 8 s of two neighbouring keys' groups: (s, s, z, z)
  float4 vsb[2][G][kKeys / 2];  // (s, s, b, b)
  uint8_t dead[2][kKeys];   // the key has no page
  uint32_t bad[2];          // a byte for each unpacking warp: it has a dead key
  float top[kParts][kRows];  // row maxima over the parts of the keys
  float sums[kParts][kRows][1 + G];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], q_full, s_full, s_free, p_full, pv_done, drain;
  ptx::Abort abort;
  uint32_t tmem;
};

// Tensor memory, in 32-bit columns: the groups' scores, the weights, O.
template <int D>
struct Tmem {
  static constexpr int G = D / kKv4Group;
  static constexpr uint32_t S = 0, P = G * 128, O = P + G * 64, N = O + D;
  static constexpr uint32_t kCols = N <= 256 ? 256 : 512;
};

using TcLine = Line<kRows, kKeys, kSpare, kWarps>;

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {  // float16 operands, K-major, float32 sums
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Tiles of a piece that any of its rows sees.
__device__ __forceinline__ int piece_end(const TcLine::Piece& p) { return min(p.t1, (p.klen + kKeys - 1) / kKeys); }

// Whether any lane of the four warps that share 32 rows says so (a barrier of all four).
__device__ __forceinline__ bool rows_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}
// A warp that gives up does not leave the others waiting: their barrier ends, and they see
// the flag.
__device__ __forceinline__ void rows_leave(int id) { asm volatile("barrier.cta.arrive %0, 128;" ::"r"(id) : "memory"); }

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

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void fetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ---------------------------------------------------------------- unpacking
template <int D>
__device__ __forceinline__ bool unpack_role(const AttnArgs& args, Smem<D>& sm, TcLine line, int warp, int lane) {
  constexpr int G = D / kKv4Group, W = 8 * G;  // code words of a row
  const Kv4Args& a = args.a;
  const int key = warp * 32 + lane;
  uint32_t n = 0;
  TcLine::Piece p;
  while (line.next(a, &p)) {
    const int te = piece_end(p);
    const int* table = a.table + p.b * a.table_stride;
    uint4 kw[W / 4], vw[W / 4];
    uint32_t ks[G], vs[G];
    auto id_of = [&](int t) {
      const int pos = t * kKeys + key;
      return t < te && pos < p.s.len ? table[div_by(pos, args.page_div)] : -2;
    };
    // This thread's key of a tile: its row of the cache, none for what is no position or has no page.
    constexpr unsigned long long kNone = ~0ull;
    auto row_of = [&](int t, int id) {
      const int pos = t * kKeys + key, pg = div_by(pos, args.page_div);
      const bool ok = (unsigned)id < (unsigned)a.n_pages;
      if (!ok && id != -2) set_status(a.status, kStatusBounds);
      return ok ? ((unsigned long long)id * a.heads_kv + p.h) * a.page + (pos - pg * a.page) : kNone;
    };
    auto load = [&](const uint8_t* codes, const uint32_t* scale, unsigned long long row, uint4 (&w)[W / 4], uint32_t (&sc)[G]) {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) w[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int g = 0; g < G; ++g) sc[g] = 0;
      if (row != kNone) {
        const uint4* from = reinterpret_cast<const uint4*>(codes + row * (D / 2));
#pragma unroll
        for (int i = 0; i < W / 4; ++i) w[i] = __ldg(from + i);
#pragma unroll
        for (int g = 0; g < G; ++g) sc[g] = __ldg(scale + row * G + g);
      }
    };
    unsigned long long row = kNone, next_row = kNone;
    if (p.t0 < te) {
      const int id0 = id_of(p.t0);
      int id1 = id_of(p.t0 + 1);
      row = row_of(p.t0, id0);
      load(a.kc, a.ks, row, kw, ks);
      load(a.vc, a.vs, row, vw, vs);
      next_row = row_of(p.t0 + 1, id1);
    }
    int id = id_of(p.t0 + 2);
    for (int t = p.t0; t < te; ++t, ++n) {
      const uint32_t st = n & 1, ph = (n >> 1) & 1;
      const bool none = row == kNone;
      const uint32_t any_none = __ballot_sync(0xffffffffu, none);
      row = next_row;  // the next tile's
      if (t + 2 < te) {
        next_row = row_of(t + 2, id);
        if (next_row != kNone) {  // on its way to L2
          fetch_l2(a.kc + next_row * (D / 2));
          fetch_l2(a.vc + next_row * (D / 2));
        }
        id = id_of(t + 3);
      }
      if (n >= 2 && !__all_sync(0xffffffffu, ptx::mbar_wait(&sm.k_empty[st], ph ^ 1, &sm.abort, a.status, args.wait_ns)))
        return false;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(kw);  // word (i, g) at i * G + g
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint8_t* row = sm.k[st][g] + key * 128;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t x = w[i * G + g], y = x >> 8;
          *reinterpret_cast<uint4*>(row + ((i ^ (key & 7)) << 4)) =
              make_uint4(x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u);
        }
        const float s = bf16_lo(ks[g]);
        float* sz = reinterpret_cast<float*>(&sm.ksz[st][g][key >> 1]) + (key & 1);
        sz[0] = s, sz[2] = fmaf(-8.f, s, bf16_hi(ks[g]));
      }
      sm.dead[st][key] = none ? 1 : 0;
      if (lane == 0) reinterpret_cast<uint8_t*>(&sm.bad[st])[warp] = any_none ? 1 : 0;
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.k_full[st]);
      if (t + 1 < te) load(a.kc, a.ks, row, kw, ks);

      if (n >= 2 && !__all_sync(0xffffffffu, ptx::mbar_wait(&sm.v_empty[st], ph ^ 1, &sm.abort, a.status, args.wait_ns)))
        return false;
      w = reinterpret_cast<const uint32_t*>(vw);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint8_t* row = sm.v[st][g] + key * 128;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t x = w[i * G + g];
          uint32_t u[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 128 + u by bit operations, minus 136: exact
            u[k] = add_bf16x2(((x >> (4 * k)) & 0x000F000Fu) | 0x43004300u, 0xC308C308u);
          *reinterpret_cast<uint4*>(row + ((i ^ (key & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
        }
        float* sb = reinterpret_cast<float*>(&sm.vsb[st][g][key >> 1]) + (key & 1);
        sb[0] = bf16_lo(vs[g]), sb[2] = bf16_hi(vs[g]);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.v_full[st]);
      if (t + 1 < te) load(a.vc, a.vs, row, vw, vs);
    }
  }
  return true;
}

// ---------------------------------------------------------------- products
template <int D>
__device__ __forceinline__ bool product_role(const AttnArgs& args, Smem<D>& sm, TcLine line, uint32_t tmem) {
  constexpr int G = D / kKv4Group;
  const Kv4Args& a = args.a;
  constexpr uint32_t kS = idesc_f16(kRows, kKeys), kPV = ptx::idesc_bf16(kRows, kKv4Group, false, true);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return (bool)__all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, &sm.abort, a.status, args.wait_ns));
  };
  const uint64_t q_desc = ptx::sdesc_sw128(ptx::smem_u32(sm.q[0]), 16, 1024), k_desc = ptx::sdesc_sw128(ptx::smem_u32(sm.k[0][0]), 16, 1024);
  const uint64_t v_desc = ptx::sdesc_sw128(ptx::smem_u32(sm.v[0][0]), 16384, 1024);
  auto scores = [&](uint32_t st) {
    ptx::tc_fence_after();
    if (ptx::elect_one()) {
      const uint64_t kd = k_desc + st * (G * 1024);
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          ptx::mma_ss(tmem + Tmem<D>::S + g * 128, q_desc + g * 1024 + kk * 2, kd + g * 1024 + kk * 2, kS, kk > 0 ? 1u : 0u);
      ptx::mma_commit(&sm.s_full);
      ptx::mma_commit(&sm.k_empty[st]);
    }
    __syncwarp();
  };
  uint32_t n = 0, pieces = 0;
  TcLine::Piece p;
  while (line.next(a, &p)) {
    const int te = piece_end(p);
    if (p.t0 >= te) continue;
    if (!wait(&sm.q_full, pieces & 1)) return false;
    ++pieces;
    if (!wait(&sm.k_full[n & 1], (n >> 1) & 1)) return false;
    if (n > 0 && !wait(&sm.s_free, (n - 1) & 1)) return false;
    scores(n & 1);
    for (int t = p.t0; t < te; ++t, ++n) {
      const uint32_t st = n & 1;
      if (t + 1 < te) {
        if (!wait(&sm.k_full[(n + 1) & 1], ((n + 1) >> 1) & 1) || !wait(&sm.s_free, n & 1)) return false;
        scores((n + 1) & 1);
      }
      if (!wait(&sm.v_full[st], (n >> 1) & 1) || !wait(&sm.p_full, n & 1)) return false;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            ptx::mma_ts(tmem + Tmem<D>::O + g * 64, tmem + Tmem<D>::P + g * 64 + kk * 8,
                        v_desc + st * (G * 1024) + g * 1024 + kk * 128, kPV,
                        t > p.t0 || kk > 0 ? 1u : 0u);
        ptx::mma_commit(&sm.pv_done);
        ptx::mma_commit(&sm.v_empty[st]);
      }
      __syncwarp();
    }
  }
  return true;
}

// ---------------------------------------------------------------- softmax
template <int D>
__device__ __forceinline__ bool softmax_role(const AttnArgs& args, Smem<D>& sm, TcLine line, uint32_t tmem, int warp,
                                             int lane) {
  constexpr int G = D / kKv4Group, NV = D / kParts;  // NV: a thread's values of its row, and its columns of O
  const Kv4Args& a = args.a;
  const int part = warp >> 2, row = (warp & 3) * 32 + lane, id = 1 + (warp & 3);
  const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes of tensor memory
  const float q_sign = a.scale_log2 > 0.f ? 1.f : a.scale_log2 < 0.f ? -1.f : 0.f;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, &sm.abort, a.status, args.wait_ns))) return true;
    rows_leave(id);
    return false;
  };
  auto gone = [&]() {
    if (!__any_sync(0xffffffffu, sm.abort.flag != 0)) return false;
    rows_leave(id);
    return true;
  };
  auto arrive = [&](uint64_t* bar) {
    if (lane == 0) ptx::mbar_arrive(bar);
  };
  uint32_t n = 0;
  TcLine::Piece p;
  while (line.next(a, &p)) {
    const int te = piece_end(p), b = p.b;
    const int grow = p.r0 + row;  // of the (sequence, KV head)
    const RowPlace pl = row_place(a, p.h, min(grow, p.rows - 1));
    const int pos = p.s.len - p.s.n + pl.token;
    const int lim = grow >= p.rows ? kNoRow : pos < 0 ? 0 : a.causal ? pos + 1 : p.s.len;
    if (p.r0 + (warp & 3) * 32 >= p.rows) {
      // No query in this warp's rows: what stands in their lanes is never read.  It keeps
      // step with the others: a tile's arrivals come after the end of the last one's.
      if (p.t0 < te) arrive(&sm.q_full);
      for (int t = p.t0; t < te; ++t, ++n) {
        const uint32_t st = n & 1;
        if (!wait(&sm.s_full, n & 1)) return false;
        arrive(&sm.s_free);
        arrive(&sm.k_empty[st]);
        if (n > 0 && !wait(&sm.pv_done, (n - 1) & 1)) return false;
        arrive(&sm.p_full);
        arrive(&sm.v_empty[st]);
      }
      continue;
    }
    float rf = 1.f, rz[G], mu = 0.f, bar = -INFINITY;
    Two l = 0, off[G];  // sums over even and odd keys
#pragma unroll
    for (int g = 0; g < G; ++g) rz[g] = 0.f, off[g] = 0;

    if (p.t0 < te) {
      // Q: a quarter of this thread's row into its operand
      uint4 raw[NV / 8];
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.x) + x_row(a, p.s, b, pl) + part * NV;
      float big = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV / 8; ++i) {
        raw[i] = grow < p.rows ? *reinterpret_cast<const uint4*>(src + i * 8) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = bf16_lo(w[e]) * q_sign, y = bf16_hi(w[e]) * q_sign;
          big = fmaxf(big, fmaxf(fabsf(x), fabsf(y)));
          sum += x + y;
        }
      }
      sm.top[part][row] = big;
      sm.sums[part][row][0] = sum;
      rows_any(id, false);
      if (gone()) return false;
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        big = fmaxf(big, sm.top[i][row]);
        rz[i * G / kParts] += sm.sums[i][row][0];
      }
      int ex = 0;  // |q| < 2^ex: scaled below 2^14
      if (big > 0.f && big < INFINITY) frexpf(big, &ex);
      ex -= 14;
#pragma unroll
      for (int g = 0; g < G; ++g) rz[g] = ldexpf(rz[g], -(24 + ex));
      // at least 2^-126, at most the largest float32: scores of 0 times it stay 0
      rf = a.scale_log2 != 0.f ? fminf(fmaxf(ldexpf(fabsf(a.scale_log2), 24 + ex), 1.17549435e-38f), 3.40282347e38f) : 1.f;
      const float up = pow2(-ex / 2) * q_sign, up2 = pow2(-ex - -ex / 2);
#pragma unroll
      for (int i = 0; i < NV / 8; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = bf16_lo(w[e]) * up * up2;
          v[2 * e + 1] = bf16_hi(w[e]) * up * up2 * 0.0625f;
        }
        const int word = part * (NV / 8) + i, g = word / 8, slot = word % 8;
        *reinterpret_cast<uint4*>(sm.q[g] + row * 128 + ((slot ^ (row & 7)) << 4)) =
            make_uint4(pack_f16x2(v[0], v[4]), pack_f16x2(v[1], v[5]), pack_f16x2(v[2], v[6]), pack_f16x2(v[3], v[7]));
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      arrive(&sm.q_full);
    }

    for (int t = p.t0; t < te; ++t, ++n) {
      const uint32_t st = n & 1, ph = (n >> 1) & 1;
      if (!wait(&sm.s_full, n & 1) || !wait(&sm.k_full[st], ph)) return false;
      ptx::tc_fence_after();
      Two x[kPart / 2];  // of two neighbouring keys
#pragma unroll
      for (int c = 0; c < kPart; c += 16) {
        uint32_t s0[16], s1[G == 2 ? 16 : 1];
        ptx::tmem_ld16(lanes + Tmem<D>::S + part * kPart + c, s0);
        if constexpr (G == 2) ptx::tmem_ld16(lanes + Tmem<D>::S + 128 + part * kPart + c, s1);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const ulonglong2 z = *reinterpret_cast<const ulonglong2*>(&sm.ksz[st][0][(part * kPart + c + j) / 2]);
          Two v = fma2(z.x, two(__uint_as_float(s0[j]), __uint_as_float(s0[j + 1])), mul2(z.y, two(rz[0], rz[0])));
          if constexpr (G == 2) {
            const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(&sm.ksz[st][G - 1][(part * kPart + c + j) / 2]);
            v = fma2(y.x, two(__uint_as_float(s1[j]), __uint_as_float(s1[j + 1])), fma2(y.y, two(rz[G - 1], rz[G - 1]), v));
          }
          x[(c + j) / 2] = v;
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      arrive(&sm.s_free);
      const uint32_t dead = sm.bad[st];
      const int k0 = t * kKeys + part * kPart;
      if (k0 + kPart > p.all_see || dead) {  // keys that not all rows see
#pragma unroll
        for (int j = 0; j < kPart; j += 2) {
          float2 v = apart(x[j / 2]);
          if (k0 + j >= lim || sm.dead[st][part * kPart + j]) v.x = -INFINITY;
          if (k0 + j + 1 >= lim || sm.dead[st][part * kPart + j + 1]) v.y = -INFINITY;
          x[j / 2] = two(v.x, v.y);
        }
      }
      __syncwarp();
      arrive(&sm.k_empty[st]);
      float high = -INFINITY;
#pragma unroll
      for (int j = 0; j < kPart / 2; ++j) {
        const float2 v = apart(x[j]);
        high = fmax3f(high, v.x, v.y);
      }
      const bool raise = rows_any(id, high > bar);
      if (gone()) return false;
      if (raise) {
        sm.top[part][row] = high;
        rows_any(id, false);
        if (gone()) return false;
#pragma unroll
        for (int i = 0; i < kParts; ++i) high = fmaxf(high, sm.top[i][row]);
        float f = 1.f;
        if (high > -INFINITY) {
          high *= rf;
          if (bar > -INFINITY) {
            high = fmaxf(high, mu);
            f = fast_exp2(mu - high);
          }
          mu = high;
          bar = (high + 8.f) / rf;
        }
        l = mul2(l, two(f, f));
#pragma unroll
        for (int g = 0; g < G; ++g) off[g] = mul2(off[g], two(f, f));
        if (t > p.t0 && __any_sync(0xffffffffu, f != 1.f)) {
          if (!wait(&sm.pv_done, (n - 1) & 1)) return false;
          ptx::tc_fence_after();
#pragma unroll
          for (int c = 0; c < NV; c += 16) {
            uint32_t o[16];
            ptx::tmem_ld16(lanes + Tmem<D>::O + part * NV + c, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            ptx::tmem_st16(lanes + Tmem<D>::O + part * NV + c, o);
          }
          ptx::tmem_st_wait();
        }
      }
      if (!wait(&sm.v_full[st], ph) || (n > 0 && !wait(&sm.pv_done, (n - 1) & 1))) return false;
      ptx::tc_fence_after();
      uint32_t w[G][kPart / 2];  // weights
#pragma unroll
      for (int j = 0; j < kPart / 2; ++j) {
        const float2 v = apart(fma2(x[j], two(rf, rf), two(-mu, -mu)));
        const Two pr = two(fast_exp2(v.x), fast_exp2(v.y));
        l = add2(l, pr);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const ulonglong2 z = *reinterpret_cast<const ulonglong2*>(&sm.vsb[st][g][part * kPart / 2 + j]);
          const float2 u = apart(mul2(pr, z.x));
          w[g][j] = ptx::pack_bf16x2(u.x, u.y);
          off[g] = fma2(pr, z.y, off[g]);
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) ptx::tmem_st16(lanes + Tmem<D>::P + g * 64 + part * (kPart / 2), w[g]);
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      arrive(&sm.p_full);
      arrive(&sm.v_empty[st]);
    }

    // ---- the row's sums over all keys, and its result
    sm.sums[part][row][0] = apart(l).x + apart(l).y;
#pragma unroll
    for (int g = 0; g < G; ++g) sm.sums[part][row][1 + g] = apart(off[g]).x + apart(off[g]).y;
    rows_any(id, false);
    if (gone()) return false;
    float sum = 0.f, add = 0.f;  // of p; of p b for this thread's columns
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      sum += sm.sums[i][row][0];
      add += sm.sums[i][row][1 + part * G / kParts];
    }
    if (p.t0 < te) {
      if (!wait(&sm.pv_done, (n - 1) & 1)) return false;
      ptx::tc_fence_after();
    }
    const float m = bar == -INFINITY ? -INFINITY : mu;
    const long long slot = (long long)blockIdx.x * 2 + (p.t0 == 0 ? 1 : 0);
    const float inv = p.whole ? (sum != 0.f ? 1.f / sum : 0.f) : 1.f;
#pragma unroll
    for (int c = 0; c < NV; c += 16) {
      uint32_t o[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = 0;
      if (p.t0 < te) {
        ptx::tmem_ld16(lanes + Tmem<D>::O + part * NV + c, o);
        ptx::tmem_ld_wait();
      }
      if (grow < p.rows) {
#pragma unroll
        for (int j = 0; j < 16; j += 8) {  // a word's values stand as 0, 4, 1, 5, 2, 6, 3, 7
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = (__uint_as_float(o[j + 2 * e]) + add) * inv;
            v[e + 4] = (__uint_as_float(o[j + 2 * e + 1]) + add) * inv;
          }
          const int d = part * NV + c + j;
          if (p.whole) {
            __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + y_row(a, p.s, b, pl) + d;
            *reinterpret_cast<uint4*>(y) = make_uint4(ptx::pack_bf16x2(v[0], v[1]), ptx::pack_bf16x2(v[2], v[3]),
                                                      ptx::pack_bf16x2(v[4], v[5]), ptx::pack_bf16x2(v[6], v[7]));
          } else {
            float* y = args.part_o + (slot * kRows + row) * D + d;
            *reinterpret_cast<float4*>(y) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(y + 4) = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
      }
    }
    ptx::tc_fence_before();
    if (part == 0 && grow < p.rows) {
      if (p.whole) {
        a.lse[lse_row(a, p.s, b, pl)] = row_lse(m, sum);
      } else {
        args.part_ml[(slot * kRows + row) * 2] = m;
        args.part_ml[(slot * kRows + row) * 2 + 1] = sum;
      }
    }
    if (warp == 0 && lane == 0 && p.t0 == 0 && !p.whole)
      args.shared[blockIdx.x] = make_int4(b, p.h, p.r0 / kRows, line.owner(p.last, line.total, line.n));
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_kv4_rows(const __grid_constant__ AttnArgs args) {
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  TcLine line;
  const bool any = line.begin(args.a);
  if (threadIdx.x == 0) args.shared[blockIdx.x] = make_int4(0, 0, 0, -1);
  if (!any) return;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.k_full[i], kUnpackWarps);
      ptx::mbar_init(&sm.v_full[i], kUnpackWarps);
      ptx::mbar_init(&sm.k_empty[i], kSoftWarps + 1);  // the scales are read, the score product is done
      ptx::mbar_init(&sm.v_empty[i], kSoftWarps + 1);
    }
    ptx::mbar_init(&sm.q_full, kSoftWarps);
    ptx::mbar_init(&sm.s_full, 1);
    ptx::mbar_init(&sm.s_free, kSoftWarps);
    ptx::mbar_init(&sm.p_full, kSoftWarps);
    ptx::mbar_init(&sm.pv_done, 1);
    ptx::mbar_init(&sm.drain, 1);
    sm.abort.flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kWarps - 1) {
    ptx::tmem_alloc(&sm.tmem, Tmem<D>::kCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sm.tmem;
  if (warp < kSoftWarps) {
    ptx::regs_increase<kSoftRegs>();
    softmax_role<D>(args, sm, line, tmem, warp, lane);
  } else if (warp < kSoftWarps + kUnpackWarps) {
    ptx::regs_decrease<kUnpackRegs>();
    unpack_role<D>(args, sm, line, warp - kSoftWarps, lane);
  } else {
    ptx::regs_decrease<kIssueRegs>();
  }
  if (warp == kWarps - 1) {
    product_role<D>(args, sm, line, tmem);
    // every product that was issued ends before the tensor memory is given back
    if (ptx::elect_one()) ptx::mma_commit(&sm.drain);
    __syncwarp();
    ptx::Abort none;
    none.flag = 0;
    ptx::mbar_wait(&sm.drain, 0, &none, args.a.status, args.wait_ns);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kWarps - 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, Tmem<D>::kCols);
  }
}

// Joins the parts of row tiles whose keys several blocks shared, in the blocks' order:
// a thread for eight values of a row.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) k_kv4_rows_join(const __grid_constant__ AttnArgs args) {
  const Kv4Args& a = args.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
  const int4 tile = __ldcg(&args.shared[blockIdx.x]);
  const int b = tile.x, h = tile.y, i0 = blockIdx.x, i1 = tile.w;
  if (i1 < 0) return;
  const Kv4Seq s = kv4_seq(a, b);
  const int row = blockIdx.y * (kJoinThreads * 8 / D) + threadIdx.x / (D / 8), d = threadIdx.x % (D / 8) * 8;
  const int grow = tile.z * kRows + row;
  if (grow >= s.n * a.group) return;
  float o[8] = {}, m = -INFINITY, l = 0.f;
  for (int i = i0; i <= i1; ++i) {
    const long long slot = (long long)i * 2 + (i == i0 ? 1 : 0);
    const float4* from = reinterpret_cast<const float4*>(args.part_o + (slot * kRows + row) * D + d);
    const float4 x = __ldcg(from), y = __ldcg(from + 1);
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(args.part_ml + (slot * kRows + row) * 2));
    const float top = fmaxf(m, ml.x), u = top == -INFINITY ? 0.f : top;
    const float f = m == -INFINITY ? 1.f : fast_exp2(m - u), fp = ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - u);
    m = top;
    l = l * f + ml.y * fp;
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = o[e] * f + v[e] * fp;
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const RowPlace pl = row_place(a, h, grow);
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + y_row(a, s, b, pl) + d;
  *reinterpret_cast<uint4*>(y) =
      make_uint4(ptx::pack_bf16x2(o[0] * inv, o[1] * inv), ptx::pack_bf16x2(o[2] * inv, o[3] * inv),
                 ptx::pack_bf16x2(o[4] * inv, o[5] * inv), ptx::pack_bf16x2(o[6] * inv, o[7] * inv));
  if (d == 0) a.lse[lse_row(a, s, b, pl)] = row_lse(m, l);
}

template <int D>
struct Launch {
  static int grid(const Kv4Args& a) {
    const long long row_tiles = ((long long)a.seqlen * a.group + kRows - 1) / kRows;
    const long long key_tiles = std::max(1ll, ((long long)a.max_pages * a.page + kKeys - 1) / kKeys);
    const long long most = (long long)a.batch * a.heads_kv * row_tiles;
    return (int)(most >= kSms ? kSms : std::min<long long>(kSms, most * std::min(key_tiles, (long long)kSms)));
  }
  static size_t o_bytes(const Kv4Args& a) { return (size_t)grid(a) * 2 * kRows * D * 4; }
  static size_t ml_bytes(const Kv4Args& a) { return (size_t)grid(a) * 2 * kRows * 8; }
  static size_t workspace(const Kv4Args& a) { return o_bytes(a) + ml_bytes(a) + (size_t)grid(a) * sizeof(int4); }
  static cudaError_t run(const Kv4Args& a, void* ws, unsigned long long wait_ns, cudaStream_t st) {
    AttnArgs args = {};
    args.a = a;
    args.page_div = fast_div(a.page);
    args.part_o = static_cast<float*>(ws);
    args.part_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + o_bytes(a));
    args.shared = reinterpret_cast<int4*>(static_cast<char*>(ws) + o_bytes(a) + ml_bytes(a));
    args.wait_ns = wait_ns;
    static std::atomic<unsigned long long> raised{0};  // the shared-memory limit, once a device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(k_kv4_rows<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<D>));
      if (e != cudaSuccess) return e;
      raised.fetch_or(bit, std::memory_order_relaxed);
    }
    const int n = grid(a);
    k_kv4_rows<D><<<n, kThreads, sizeof(Smem<D>), st>>>(args);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((long long)a.max_pages * a.page <= kKeys) return cudaSuccess;  // a row tile has one tile of keys
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n, kRows * D / 8 / kJoinThreads);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_kv4_rows_join<D>, args);
  }
};

}  // namespace

size_t kv4_rows_workspace(const Kv4Args& a, int head_dim) {
  return head_dim == 64 ? Launch<64>::workspace(a) : Launch<128>::workspace(a);
}

cudaError_t launch_kv4_rows(const Kv4Args& a, int head_dim, void* workspace, unsigned long long wait_ns, cudaStream_t st) {
  return head_dim == 64 ? Launch<64>::run(a, workspace, wait_ns, st) : Launch<128>::run(a, workspace, wait_ns, st);
}

}  // namespace gbattn
