// Attention over the 4-bit key/value cache for many query rows: a prompt's chunk, or
// a few proposed tokens of a large group of heads.
//
// Here the work per score bounds, not the cache's bytes: 128 query rows of a KV head meet
// 128 keys on tcgen05 instructions, with scores, weights and sums in tensor memory, and
// what an unpacked key costs is shared by the rows.  So everything that belongs to a key
// goes into its operands, and a score needs no more than a masked maximum, one
// multiplication and addition, exp2 and a rounding:
//   - A step has 8 significant bits and u - 8 three, so s (u - 8) is a float16 number,
//     exactly, once the tile's largest step is brought below 2^12 (steps 2^-25 of that
//     and less lose bits).  Four warps write these, K's and V's, into 128-byte rows of 64
//     values, swizzled, one box for each group of 64.
//   - The offsets are operands too: sum_g b_g sum(q_g) is one more step of 16 of Q K^T
//     (sum(q_g) in three float16 parts), and sum(p b_g) one more product of 16 columns.
//   - K's power of two, a tile's, goes into the factor that takes scores to log2 units; V's
//     is the largest since the first tile, and where it grows the sums are scaled.
// Q is float16 in each row's own power of two.  The weights p are rounded once to
// float16, with 2^7 at the running maximum and at most 2^15 (it is raised only when a score
// is above it by more than 2^8): 11 bits, 2^-32 of the maximum at least.
//
// Sixteen warps do the softmax, four for each 32 rows with a quarter of the keys each;
// they agree on the maximum with one barrier a tile.  Scores have two places, so that the
// next tile's are computed meanwhile.
// Blocks share the work by equal stretches of one line of tiles, as for few rows
// (kv4_attn.cu).
//
// Measured: 2 sequences of up to 8192, 512 new tokens, 32 heads on 8 of 128: 119 us, 467 TFLOP/s
// of products; issue slots 48% busy, tensor pipe 24%, memory 2%.  What bounds it is the length of a
// tile's chain (unpack, scores, softmax, weights), about 4500 cycles between two tiles: with
// an eighth of the unpacking 40 us less, without exp2 or most of the products nothing.
// Two quarters of the keys a warp instead of one: 132 us; warps of their own for K and V: 123
// (118 then).  80 registers a thread leave 344 bytes of spills at head dim 128.
#include <algorithm>
#include <atomic>

#include "kv4_line.cuh"
#include "ptx.cuh"

namespace gbattn {

namespace {

// kSpare: what a row tile costs beside its keys, in tiles (1, 2, 3, 5: 60, 55, 52, 53 us with 16
// sequences of up to 4096 and 32 tokens each, 80, 81, 81, 85 us with 16 of 4096).
constexpr int kRows = 128, kKeys = 128, kSpare = 2;
constexpr int kParts = 4, kPart = kKeys / kParts;  // warps of a row, and the keys of each
// four warps of each 32 rows, four that unpack, and four of which one issues the products and one
// finds the pieces of work
constexpr int kSoftWarps = 4 * kParts, kUnpackWarps = 4, kWarps = kSoftWarps + kUnpackWarps + 4;
constexpr int kThreads = kWarps * 32;
// Registers: 80 a thread at launch; what the issuing warps give up the others take
// ((512 + 128) * 88 + 128 * 40 = 768 * 80).
constexpr int kSoftRegs = 88, kUnpackRegs = 88, kIssueRegs = 40;

using TcLine = Line<kRows, kKeys, kSpare, kWarps>;

// A piece of the block's stretch as one warp finds it, ahead of the others.
struct Work {
  TcLine::Piece p;
  int owner;  // the block whose stretch has the row tile's last keys
  bool any;   // false: the stretch's end
  int odd[2];  // the first position of the piece's keys whose value is not finite, by groups
};

template <int D>
struct Smem {
  static constexpr int G = D / kKv4Group;
  uint8_t q[G][kRows * 128];  // float16, 128-byte rows, 128-byte swizzle
  uint8_t qx[kRows * 128];    // three parts of each group's sum(q), in the first 16 columns
  uint8_t k[2][G][kKeys * 128];
  uint8_t kx[2][kKeys * 128];  // offsets, to qx's columns
  uint8_t v[2][G][kKeys * 128];
  uint8_t vx[2][2][16 * 128];  // V's offsets: a group a row, 64 keys a box
  uint8_t dead[2][kKeys];      // the key has no page
  uint32_t bad[2];             // a byte for each unpacking warp: it has a dead key
  int2 exps[2][kUnpackWarps];  // the unpacking warps' powers of two (K's, V's)
  int2 unit[2];                // and the tile's
  float top[kParts][kRows];  // row maxima over the parts of the keys
  float sums[kParts][kRows];  // of Q's groups
  // of the weights, at a piece's end, by the piece's parity: a warp that is ahead writes the next
  // piece's while others still read this one's, and the barrier of that piece's end lies
  // before this place is written again
  float last[2][kParts][kRows];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], s_free[2], p_full[2], pv_done[2], work_full[2], work_free[2], q_full, drain;
  Work work[2];
  ptx::Abort abort;
  uint32_t tmem;
};

// Tensor memory, in 32-bit columns: two tiles' scores, the weights, O and the offsets' sums.
template <int D>
struct Tmem {
  static constexpr uint32_t S = 0, P = 256, O = 320, X = O + D, kCols = 512;
};


// float16 operands, float32 sums; A K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Tiles of a piece that any of its rows sees.
__device__ __forceinline__ int piece_end(const TcLine::Piece& p) { return min(p.t1, (p.klen + kKeys - 1) / kKeys); }

// Whether any lane of four warps says so (a barrier of all four: those that share 32 rows,
// or those that unpack).
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

__device__ __forceinline__ uint32_t add_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void fetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ---------------------------------------------------------------- unpacking
// |x| < 2^size_of(x), kNotFinite for what is not finite; that counts for nothing in exp_of.
constexpr int kNotFinite = 129;
__device__ __forceinline__ int size_of(float x) { return (int)((__float_as_uint(x) >> 23) & 255) - 126; }
__device__ __forceinline__ int exp_of(float x) {
  const int e = size_of(x);
  return e == kNotFinite ? -126 : e;
}
// s (u - 8) of a code word's values (0, 4), (1, 5), (2, 6), (3, 7); step: s twice, step16: s / 16.
// 1024 + u and 1024 + 16 u by bit operations; minus 1032 or 1152, exact.
__device__ __forceinline__ uint4 eight_values(uint32_t x, uint32_t step, uint32_t step16) {
  const uint32_t y = x >> 8;
  return make_uint4(mul_f16x2(add_f16x2((x & 0x000F000Fu) | 0x64006400u, 0xE408E408u), step),
                    mul_f16x2(add_f16x2((x & 0x00F000F0u) | 0x64006400u, 0xE480E480u), step16),
                    mul_f16x2(add_f16x2((y & 0x000F000Fu) | 0x64006400u, 0xE408E408u), step),
                    mul_f16x2(add_f16x2((y & 0x00F000F0u) | 0x64006400u, 0xE480E480u), step16));
}

template <int D>
__device__ __forceinline__ bool unpack_role(const AttnArgs& args, Smem<D>& sm, int warp, int lane) {
  constexpr int G = D / kKv4Group, W = 8 * G;  // code words of a row
  const Kv4Args& a = args.a;
  const int key = warp * 32 + lane, id = 1 + kSoftWarps / kParts;  // id: their barrier
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, &sm.abort, a.status, args.wait_ns))) return true;
    rows_leave(id);
    return false;
  };
  auto meet = [&]() {  // the barrier of these warps; false: one of them has given up
    rows_any(id, false);
    if (!__any_sync(0xffffffffu, sm.abort.flag != 0)) return true;
    rows_leave(id);
    return false;
  };
  // A group's values into a box's row.
  auto unpack = [&](uint8_t* box, const uint32_t (&w)[W], int g, float s) {
    const uint32_t step = pack_f16x2(s, s), step16 = pack_f16x2(s * 0.0625f, s * 0.0625f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<uint4*>(box + key * 128 + ((i ^ (key & 7)) << 4)) = eight_values(w[i * G + g], step, step16);
  };
  uint32_t n = 0;
  for (uint32_t m = 0;; ++m) {
    if (!wait(&sm.work_full[m & 1], (m >> 1) & 1)) return false;
    if (!sm.work[m & 1].any) return true;
    const TcLine::Piece& p = sm.work[m & 1].p;
    const int t0 = p.t0, te = piece_end(p), len = p.s.len, h = p.h;
    const int* table = a.table + p.b * a.table_stride;
    // This thread's key of a tile: its row of the cache, none for what is no position or has no page.
    constexpr uint32_t kNone = 0xFFFFFFFFu;
    auto held = [&](int t) { return t < te && t * kKeys + key < len; };
    auto page_of = [&](int t) { return held(t) ? table[div_by(t * kKeys + key, args.page_div)] : -1; };
    auto row_of = [&](int t, int page) {
      const int pos = t * kKeys + key, pg = div_by(pos, args.page_div);
      const bool ok = (unsigned)page < (unsigned)a.n_pages;
      if (!ok && held(t)) set_status(a.status, kStatusBounds);
      return ok ? ((uint32_t)page * a.heads_kv + h) * a.page + (pos - pg * a.page) : kNone;
    };
    uint32_t kw[W], vw[W], ks[G], vs[G];
    auto load = [&](const uint8_t* codes, const uint32_t* scale, uint32_t row, uint32_t (&w)[W], uint32_t (&sc)[G]) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = 0;
#pragma unroll
      for (int g = 0; g < G; ++g) sc[g] = 0;
      if (row != kNone) {
        const uint4* from = reinterpret_cast<const uint4*>(codes + (unsigned long long)row * (D / 2));
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          const uint4 v = __ldg(from + i);
          w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int g = 0; g < G; ++g) sc[g] = __ldg(scale + (unsigned long long)row * G + g);
      }
    };
    uint32_t row = kNone, next_row = kNone;
    int page = -1, unit_v = -119;
    if (t0 < te) {
      const int page0 = page_of(t0), page1 = page_of(t0 + 1);
      page = page_of(t0 + 2);
      row = row_of(t0, page0);
      load(a.kc, a.ks, row, kw, ks);
      load(a.vc, a.vs, row, vw, vs);
      next_row = row_of(t0 + 1, page1);
    }
    for (int t = t0; t < te; ++t, ++n) {
      const uint32_t st = n & 1, ph = (n >> 1) & 1;
      const bool none = row == kNone;
      row = next_row;  // the next tile's
      if (t + 2 < te) {
        next_row = row_of(t + 2, page);
        if (next_row != kNone) {  // on its way to L2
          fetch_l2(a.kc + (unsigned long long)next_row * (D / 2));
          fetch_l2(a.vc + (unsigned long long)next_row * (D / 2));
        }
        page = page_of(t + 3);
      }
      // The tile's powers of two: steps below 2^12, offsets below 2^9 (V's 2^15).
      int ek = -119, ev = unit_v;
      auto powers = [&]() {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          ek = max(ek, max(exp_of(bf16_lo(ks[g])) - 12, exp_of(bf16_hi(ks[g])) - 9));
          ev = max(ev, max(size_of(bf16_lo(vs[g])) - 12, size_of(bf16_hi(vs[g])) - 15));
        }
        ek = __reduce_max_sync(0xffffffffu, ek), ev = __reduce_max_sync(0xffffffffu, ev);
        if (lane == 0) sm.exps[st][warp] = make_int2(ek, ev);
        if (!meet()) return false;
#pragma unroll
        for (int i = 0; i < kUnpackWarps; ++i) {
          const int2 e = sm.exps[st][i];
          ek = max(ek, e.x), ev = max(ev, e.y);
        }
        return true;
      };
      if (!powers()) return false;
      if (ev >= kNotFinite - 15) {
        // There may be a value that is not finite: it stays out of the product (0 times it is not 0),
        // the rows that see it learn of it beside the product.
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (!finite2(vs[g])) {
            atomicMin(&sm.work[m & 1].odd[g], t * kKeys + key);
            vs[g] = 0;
          }
        ev = unit_v;
        if (!meet() || !powers()) return false;  // the others have read
      }
      unit_v = ev;
      if (n >= 2 && !wait(&sm.k_empty[st], ph ^ 1)) return false;
      const float up_k = pow2(-ek), up_v = pow2(-ev);
      uint32_t o[2];  // offsets of the groups, float16
#pragma unroll
      for (int g = 0; g < G; ++g) {
        unpack(sm.k[st][g], kw, g, bf16_lo(ks[g]) * up_k);
        const float x = bf16_hi(ks[g]) * up_k * 64.f;  // sum(q) in qx is divided by that
        o[g] = pack_f16x2(x, x);
      }
      *reinterpret_cast<uint4*>(sm.kx[st] + key * 128 + ((key & 7) << 4)) =
          G == 2 ? make_uint4(o[0], __byte_perm(o[0], o[G - 1], 0x5410), o[G - 1], 0) : make_uint4(o[0], o[0] & 0xFFFFu, 0, 0);
      sm.dead[st][key] = none ? 1 : 0;
      const bool any_none = __any_sync(0xffffffffu, none);
      if (lane == 0) reinterpret_cast<uint8_t*>(&sm.bad[st])[warp] = any_none ? 1 : 0;
      if (key == 0) sm.unit[st] = make_int2(ek, ev);
      if (t + 1 < te) load(a.kc, a.ks, row, kw, ks);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.k_full[st]);

      if (n >= 2 && !wait(&sm.v_empty[st], ph ^ 1)) return false;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        unpack(sm.v[st][g], vw, g, bf16_lo(vs[g]) * up_v);
        *reinterpret_cast<__half*>(sm.vx[st][key / 64] + g * 128 + (((key % 64 / 8) ^ g) << 4) + key % 8 * 2) =
            __float2half_rn(bf16_hi(vs[g]) * up_v);
      }
      if (t + 1 < te) load(a.vc, a.vs, row, vw, vs);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.v_full[st]);
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&sm.work_free[m & 1]);
  }
}

// ---------------------------------------------------------------- pieces
template <int D>
__device__ __forceinline__ bool work_role(const AttnArgs& args, Smem<D>& sm, TcLine line, int lane) {
  for (uint32_t m = 0;; ++m) {
    TcLine::Piece p = {};
    const bool any = line.next(args.a, &p);
    if (m >= 2 && !__all_sync(0xffffffffu, ptx::mbar_wait(&sm.work_free[m & 1], (m >> 1 & 1) ^ 1, &sm.abort, args.a.status, args.wait_ns)))
      return false;
    if (lane == 0) {
      sm.work[m & 1].p = p;
      sm.work[m & 1].owner = any ? TcLine::owner(p.last, line.total, line.n) : 0;
      sm.work[m & 1].any = any;
      sm.work[m & 1].odd[0] = sm.work[m & 1].odd[1] = kNoRow;
      ptx::mbar_arrive(&sm.work_full[m & 1]);
    }
    __syncwarp();
    if (!any) return true;
  }
}

// ---------------------------------------------------------------- products
template <int D>
__device__ __forceinline__ bool product_role(const AttnArgs& args, Smem<D>& sm, uint32_t tmem, int lane) {
  constexpr int G = D / kKv4Group;
  const Kv4Args& a = args.a;
  constexpr uint32_t kS = idesc_f16(kRows, kKeys, false), kPV = idesc_f16(kRows, D, true), kPX = idesc_f16(kRows, 16, false);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return (bool)__all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, &sm.abort, a.status, args.wait_ns));
  };
  const uint64_t q_desc = ptx::sdesc_sw128(ptx::smem_u32(sm.q[0]), 16, 1024), k_desc = ptx::sdesc_sw128(ptx::smem_u32(sm.k[0][0]), 16, 1024);
  const uint64_t qx_desc = ptx::sdesc_sw128(ptx::smem_u32(sm.qx), 16, 1024), kx_desc = ptx::sdesc_sw128(ptx::smem_u32(sm.kx[0]), 16, 1024);
  const uint64_t v_desc = ptx::sdesc_sw128(ptx::smem_u32(sm.v[0][0]), 16384, 1024), vx_desc = ptx::sdesc_sw128(ptx::smem_u32(sm.vx[0][0]), 16, 1024);
  auto scores = [&](uint32_t st) {
    ptx::tc_fence_after();
    if (ptx::elect_one()) {
      const uint64_t kd = k_desc + st * (G * 1024);
#pragma unroll
      for (int kk = 0; kk < 4 * G; ++kk)
        ptx::mma_ss(tmem + Tmem<D>::S + st * 128, q_desc + (kk >> 2) * 1024 + (kk & 3) * 2,
                    kd + (kk >> 2) * 1024 + (kk & 3) * 2, kS, kk > 0 ? 1u : 0u);
      ptx::mma_ss(tmem + Tmem<D>::S + st * 128, qx_desc, kx_desc + st * 1024, kS, 1u);
      ptx::mma_commit(&sm.s_full[st]);
      ptx::mma_commit(&sm.k_empty[st]);
    }
    __syncwarp();
  };
  // A tile's scores take the place of those two tiles before.  A row tile's first ones
  // follow Q, which is written when the last row tile's products are done.
  uint32_t n = 0, pieces = 0;
  for (uint32_t m = 0;; ++m) {
    if (!wait(&sm.work_full[m & 1], (m >> 1) & 1)) return false;
    if (!sm.work[m & 1].any) return true;
    const int t0 = sm.work[m & 1].p.t0, te = piece_end(sm.work[m & 1].p);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&sm.work_free[m & 1]);
    if (t0 >= te) continue;
    if (!wait(&sm.q_full, pieces & 1)) return false;
    ++pieces;
    if (!wait(&sm.k_full[n & 1], (n >> 1) & 1)) return false;
    scores(n & 1);
    for (int t = t0; t < te; ++t, ++n) {
      const uint32_t st = n & 1, ph = (n >> 1) & 1;
      if (t + 1 < te) {
        if (!wait(&sm.k_full[st ^ 1], ((n + 1) >> 1) & 1)) return false;
        if (n > 0 && !wait(&sm.s_free[st ^ 1], ((n - 1) >> 1) & 1)) return false;
        scores(st ^ 1);
      }
      if (!wait(&sm.v_full[st], ph) || !wait(&sm.p_full[st], ph)) return false;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t from = tmem + Tmem<D>::P + kk * 8;
          const uint32_t acc = t > t0 || kk > 0 ? 1u : 0u;
          ptx::mma_ts(tmem + Tmem<D>::O, from, v_desc + st * (G * 1024) + kk * 128, kPV, acc);
          ptx::mma_ts(tmem + Tmem<D>::X, from, vx_desc + st * 256 + (kk >> 2) * 128 + (kk & 3) * 2, kPX, acc);
        }
        ptx::mma_commit(&sm.pv_done[st]);
        ptx::mma_commit(&sm.v_empty[st]);
      }
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------- softmax
template <int D>
__device__ __forceinline__ bool softmax_role(const AttnArgs& args, Smem<D>& sm, uint32_t tmem, int warp, int lane) {
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
  auto limit = [&](const TcLine::Piece& p, int row) {  // the keys that a row sees
    if (p.r0 + row >= p.rows) return kNoRow;
    const int pos = p.s.len - p.s.n + div_by(p.r0 + row, a.by_group);
    return pos < 0 ? 0 : a.causal ? pos + 1 : p.s.len;
  };
  uint32_t n = 0;
  for (uint32_t m = 0;; ++m) {
    if (!wait(&sm.work_full[m & 1], (m >> 1) & 1)) return false;
    if (!sm.work[m & 1].any) return true;
    const TcLine::Piece& p = sm.work[m & 1].p;
    const int t0 = p.t0, te = piece_end(p), all_see = p.all_see;
    const int grow = p.r0 + row;  // of the (sequence, KV head)
    const int lim = limit(p, row);
    if (p.r0 + (warp & 3) * 32 >= p.rows) {
      // No query in this warp's rows: what stands in their lanes is never read.  It keeps
      // step with the others: a tile's scores come after the arrivals of two tiles before.
      if (t0 < te) arrive(&sm.q_full);
      for (int t = t0; t < te; ++t, ++n) {
        const uint32_t st = n & 1;
        if (!wait(&sm.s_full[st], (n >> 1) & 1)) return false;
        arrive(&sm.s_free[st]);
        arrive(&sm.k_empty[st]);
        arrive(&sm.p_full[st]);
      }
      __syncwarp();
      arrive(&sm.work_free[m & 1]);
      continue;
    }
    float rf = 1.f, top = 0.f, bar = -INFINITY;
    int unit_v = 0;
    Two l = 0;  // sums over even and odd keys

    if (t0 < te) {
      // Q: a quarter of this thread's row into its operand
      uint4 raw[NV / 8];
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.x) + x_row(a, p.s, p.b, row_place(a, p.h, min(grow, p.rows - 1))) + part * NV;
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
      sm.sums[part][row] = sum;
      rows_any(id, false);
      if (gone()) return false;
      float rz[G] = {};
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        big = fmaxf(big, sm.top[i][row]);
        rz[i * G / kParts] += sm.sums[i][row];
      }
      int ex = 0;  // |q| < 2^ex: scaled below 2^14
      if (big > 0.f && big < INFINITY) frexpf(big, &ex);
      ex -= 14;
      // at least 2^-126, at most the largest float32: scores of 0 times it stay 0
      rf = a.scale_log2 != 0.f ? fminf(fmaxf(ldexpf(fabsf(a.scale_log2), ex), 1.17549435e-38f), 3.40282347e38f) : 1.f;
      const float up = pow2(-ex / 2) * q_sign, up2 = pow2(-ex - -ex / 2);
#pragma unroll
      for (int i = 0; i < NV / 8; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = bf16_lo(w[e]) * up * up2;
          v[2 * e + 1] = bf16_hi(w[e]) * up * up2;
        }
        const int word = part * (NV / 8) + i, g = word / 8, slot = word % 8;
        *reinterpret_cast<uint4*>(sm.q[g] + row * 128 + ((slot ^ (row & 7)) << 4)) =
            make_uint4(pack_f16x2(v[0], v[4]), pack_f16x2(v[1], v[5]), pack_f16x2(v[2], v[6]), pack_f16x2(v[3], v[7]));
      }
      if (part == 0) {  // the groups' sums in units of 2^(ex + 6), below 2^14
        uint32_t x[2] = {0, 0}, y[2] = {0, 0};  // a group's first two parts; its third
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float z = ldexpf(rz[g], -(ex + 6));
          const float h = __half2float(__float2half_rn(z));
          z -= h;
          const float m = __half2float(__float2half_rn(z));
          x[g] = pack_f16x2(h, m), y[g] = pack_f16x2(z - m, 0.f);
        }
        *reinterpret_cast<uint4*>(sm.qx + row * 128 + ((row & 7) << 4)) =
            make_uint4(x[0], (y[0] & 0xFFFFu) | (x[1] << 16), (x[1] >> 16) | (y[1] << 16), 0);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      arrive(&sm.q_full);
    }

    for (int t = t0; t < te; ++t, ++n) {
      const uint32_t st = n & 1, ph = (n >> 1) & 1;
      if (!wait(&sm.s_full[st], ph) || !wait(&sm.k_full[st], ph)) return false;
      ptx::tc_fence_after();
      uint32_t x[kPart];
      ptx::tmem_ld32(lanes + Tmem<D>::S + st * 128 + part * kPart, x);
      ptx::tmem_ld_wait();
      ptx::tc_fence_before();
      __syncwarp();
      arrive(&sm.s_free[st]);
      const int2 unit = sm.unit[st];
      const uint32_t dead = sm.bad[st];
      const int k0 = t * kKeys + part * kPart;
      if (k0 + kPart > all_see || dead) {  // keys that not all rows see
#pragma unroll
        for (int j = 0; j < kPart; ++j)
          if (k0 + j >= lim || sm.dead[st][part * kPart + j]) x[j] = 0xFF800000u;  // minus infinity
      }
      __syncwarp();
      arrive(&sm.k_empty[st]);
      float high = -INFINITY;
#pragma unroll
      for (int j = 0; j < kPart; j += 2) high = fmax3f(high, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
      const float of_tile = pow2(unit.x);
      high *= of_tile;
      const bool raise = rows_any(id, high > bar);
      if (gone()) return false;
      float f = 1.f;
      if (raise) {
        sm.top[part][row] = high;
        rows_any(id, false);
        if (gone()) return false;
#pragma unroll
        for (int i = 0; i < kParts; ++i) high = fmaxf(high, sm.top[i][row]);
        if (high > -INFINITY) {
          high *= rf;
          if (bar > -INFINITY) {
            high = fmaxf(high, top);
            f = fast_exp2(top - high);
          }
          top = high;
          bar = (high + 8.f) / rf;
        }
        l = mul2(l, two(f, f));
      }
      if (t > t0) {
        if (unit.y != unit_v) f *= unit_v - unit.y < -126 ? 0.f : pow2(unit_v - unit.y);
        if ((raise || unit.y != unit_v) && __any_sync(0xffffffffu, f != 1.f)) {
          if (!wait(&sm.pv_done[st ^ 1], ((n - 1) >> 1) & 1)) return false;  // (and once more below)
          ptx::tc_fence_after();
          auto scale = [&](uint32_t at) {
            uint32_t o[16];
            ptx::tmem_ld16(lanes + at, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            ptx::tmem_st16(lanes + at, o);
          };
#pragma unroll
          for (int c = 0; c < NV; c += 16) scale(Tmem<D>::O + part * NV + c);
          if (part == 0) scale(Tmem<D>::X);
          ptx::tmem_st_wait();
        }
      }
      unit_v = unit.y;
      // rf as for rf itself
      const float r = fminf(fmaxf(rf * of_tile, 1.17549435e-38f), 3.40282347e38f), shift = 7.f - top;
      uint32_t w[kPart / 2];  // weights
#pragma unroll
      for (int j = 0; j < kPart; j += 2) {
        const float2 v = apart(fma2(two(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), two(r, r), two(shift, shift)));
        const float p0 = fast_exp2(v.x), p1 = fast_exp2(v.y);
        l = add2(l, two(p0, p1));
        w[j / 2] = pack_f16x2(p0, p1);
      }
      if (n > 0 && !wait(&sm.pv_done[st ^ 1], ((n - 1) >> 1) & 1)) return false;
      ptx::tc_fence_after();
      ptx::tmem_st16(lanes + Tmem<D>::P + part * (kPart / 2), w);
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      arrive(&sm.p_full[st]);
    }

    // ---- the row's sums over all keys, and its result
    sm.last[m & 1][part][row] = apart(l).x + apart(l).y;
    rows_any(id, false);
    if (gone()) return false;
    float sum = 0.f, add = 0.f;  // of p; of p b for this thread's columns
#pragma unroll
    for (int i = 0; i < kParts; ++i) sum += sm.last[m & 1][i][row];
    if (t0 < te) {
      if (!wait(&sm.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) return false;
      ptx::tc_fence_after();
      uint32_t o[16];
      ptx::tmem_ld16(lanes + Tmem<D>::X, o);
      ptx::tmem_ld_wait();
      const int g = G == 2 && part >= kParts / 2 ? 1 : 0;  // of this thread's columns
      add = limit(p, row) > sm.work[m & 1].odd[g] ? NAN : __uint_as_float(g ? o[1] : o[0]);
    }
    const RowPlace pl = row_place(a, p.h, min(grow, p.rows - 1));
    const int b = p.b;
    const float high = bar == -INFINITY ? -INFINITY : top - 7.f;
    const long long slot = (long long)blockIdx.x * 2 + (p.t0 == 0 ? 1 : 0);
    const float inv = pow2(unit_v) * (p.whole ? (sum != 0.f ? 1.f / sum : 0.f) : 1.f);
#pragma unroll
    for (int c = 0; c < NV; c += 16) {
      uint32_t o[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = 0;
      if (t0 < te) {
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
          } else {  // four values of all rows side by side
            float4* y = reinterpret_cast<float4*>(args.part_o) + (slot * (D / 4) + d / 4) * kRows + row;
            y[0] = make_float4(v[0], v[1], v[2], v[3]);
            y[kRows] = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
      }
    }
    ptx::tc_fence_before();
    if (part == 0 && grow < p.rows) {
      if (p.whole) {
        a.lse[lse_row(a, p.s, b, pl)] = row_lse(high, sum);
      } else {
        args.part_ml[(slot * kRows + row) * 2] = high;
        args.part_ml[(slot * kRows + row) * 2 + 1] = sum;
      }
    }
    if (warp == 0 && lane == 0 && p.t0 == 0 && !p.whole)
      args.shared[blockIdx.x] = make_int4(b, p.h, p.r0 / kRows, sm.work[m & 1].owner);
    __syncwarp();
    arrive(&sm.work_free[m & 1]);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_kv4_rows(const __grid_constant__ AttnArgs args) {
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.k_full[i], kUnpackWarps);
      ptx::mbar_init(&sm.v_full[i], kUnpackWarps);
      ptx::mbar_init(&sm.k_empty[i], kSoftWarps + 1);  // the units and dead keys are read, the score product is done
      ptx::mbar_init(&sm.v_empty[i], 1);
      ptx::mbar_init(&sm.s_full[i], 1);
      ptx::mbar_init(&sm.s_free[i], kSoftWarps);
      ptx::mbar_init(&sm.p_full[i], kSoftWarps);
      ptx::mbar_init(&sm.pv_done[i], 1);
      ptx::mbar_init(&sm.work_full[i], 1);
      ptx::mbar_init(&sm.work_free[i], kSoftWarps + kUnpackWarps + 1);
    }
    ptx::mbar_init(&sm.q_full, kSoftWarps);
    ptx::mbar_init(&sm.drain, 1);
    sm.abort.flag = 0;
    ptx::fence_mbar_init();
    args.shared[blockIdx.x] = make_int4(0, 0, 0, -1);
  }
  // columns and rows that no group fills
  auto clear = [&](uint8_t* to, int bytes) {
    for (int i = threadIdx.x * 16; i < bytes; i += kThreads * 16) *reinterpret_cast<uint4*>(to + i) = make_uint4(0, 0, 0, 0);
  };
  clear(sm.qx, sizeof(sm.qx));
  clear(sm.kx[0], sizeof(sm.kx));
  clear(sm.vx[0][0], sizeof(sm.vx));
  ptx::fence_proxy_async_smem();
  if (warp == kWarps - 1) {
    ptx::tmem_alloc(&sm.tmem, Tmem<D>::kCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  TcLine line;
  const bool any = line.begin(args.a);  // with barriers of the block
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sm.tmem;
  if (!any) {
    if (warp == kWarps - 1) ptx::tmem_dealloc(tmem, Tmem<D>::kCols);
    return;
  }
  if (warp < kSoftWarps) {
    ptx::regs_increase<kSoftRegs>();
    softmax_role<D>(args, sm, tmem, warp, lane);
  } else if (warp < kSoftWarps + kUnpackWarps) {
    ptx::regs_increase<kUnpackRegs>();
    unpack_role<D>(args, sm, warp - kSoftWarps, lane);
  } else {
    ptx::regs_decrease<kIssueRegs>();
  }
  if (warp == kWarps - 2) work_role<D>(args, sm, line, lane);
  if (warp == kWarps - 1) {
    product_role<D>(args, sm, tmem, lane);
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
  const int row = threadIdx.x % kRows, d = (blockIdx.y * (kJoinThreads / kRows) + threadIdx.x / kRows) * 8;
  const int grow = tile.z * kRows + row;
  if (grow >= s.n * a.group) return;
  float o[8] = {}, m = -INFINITY, l = 0.f;
  for (int i = i0; i <= i1; ++i) {
    const long long slot = (long long)i * 2 + (i == i0 ? 1 : 0);
    const float4* from = reinterpret_cast<const float4*>(args.part_o) + (slot * (D / 4) + d / 4) * kRows + row;
    const float4 x = __ldcg(from), y = __ldcg(from + kRows);
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
