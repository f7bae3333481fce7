// The dropout mask of include/gbln.h, computed where it is used and never stored.
//
// An element's bits depend on (seed, offset, row, col) alone: Philox4x32 (Salmon,
// Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", 2011), a bijection
// of the 128-bit counter (col / 8, row, offset) under the 64-bit key seed.  One
// evaluation gives the 16 bits of eight neighbouring elements, one 16-byte vector of
// bfloat16.  Seven rounds: the fewest that the paper reports to pass BigCrush.  A round is
// two 32 x 32 -> 64 bit products; ten rounds would bring the products of a bfloat16
// dropout near the time of its bytes.
// 16 bits an element: the rate is a multiple of 2^-16, and the factor of what stays
// is made from that rate, so the mean is kept exactly.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gbln.h"

namespace gbattn {

// As the host hands it to a kernel.
struct DropArgs {
  uint32_t below;        // t = round(65536 p): elements whose bits are below it are dropped
  float factor;          // 65536 / (65536 - t); 0 if t = 65536
  uint64_t seed, offset;
  const uint64_t* rng;   // device pair added to both, or NULL
};

// What a thread works with: the key, and the half of the counter that a call fixes.
struct DropKey {
  uint32_t k0, k1, c2, c3;
};

__device__ __forceinline__ DropKey drop_key(const DropArgs& d) {
  uint64_t seed = d.seed, offset = d.offset;
  if (d.rng) {
    seed += d.rng[0];
    offset += d.rng[1];
  }
  return DropKey{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
}

// 128 bits for the eight elements 8 group .. 8 group + 7 of a row: element 8 group + e
// has the low (e even) or high (e odd) half of word e / 2.
__device__ __forceinline__ uint4 drop_bits(const DropKey& key, uint32_t group, uint32_t row) {
  uint32_t c0 = group, c1 = row, c2 = key.c2, c3 = key.c3, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ bool drop_keeps(const uint4& bits, int e, uint32_t below) {
  const uint32_t w = e < 2 ? bits.x : e < 4 ? bits.y : e < 6 ? bits.z : bits.w;
  return (e & 1 ? w >> 16 : w & 0xFFFFu) >= below;
}

// The E elements (4 or 8, at a column that is a multiple of E) v of one row, through the dropout.
template <int E>
__device__ __forceinline__ void drop_vector(const DropArgs& d, const DropKey& key, int64_t c0, int64_t row,
                                            float (&v)[E]) {
  static_assert(E == 4 || E == 8, "half a group or a whole one");
  uint4 bits = drop_bits(key, (uint32_t)(c0 >> 3), (uint32_t)row);
  if (E == 4 && (c0 & 4)) bits.x = bits.z, bits.y = bits.w;
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = drop_keeps(bits, e, d.below) ? v[e] * d.factor : 0.f;
}

// The same for pairs.
template <int P>
__device__ __forceinline__ void drop_pairs(const DropArgs& d, const DropKey& key, uint32_t c0, uint32_t row,
                                           float2 (&v)[P]) {
  static_assert(P == 2 || P == 4, "half a group or a whole one");
  uint4 bits = drop_bits(key, c0 >> 3, row);
  if (P == 2 && (c0 & 4)) bits.x = bits.z, bits.y = bits.w;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    v[i].x = drop_keeps(bits, 2 * i, d.below) ? v[i].x * d.factor : 0.f;
    v[i].y = drop_keeps(bits, 2 * i + 1, d.below) ? v[i].y * d.factor : 0.f;
  }
}

// Checks d and fills a: dropped stays false where nothing is dropped (d is NULL or t is 0).
// Returns what is wrong, or NULL.
inline const char* resolve_dropout(const ln_dropout_t* d, DropArgs* a, bool* drops) {
  *drops = false;
  if (!d) return nullptr;
  if (!(d->p >= 0.0 && d->p <= 1.0)) return "dropout: p must be between 0 and 1";
  if (reinterpret_cast<uintptr_t>(d->rng) & 7u) return "dropout: rng is not 8-byte aligned";
  a->below = (uint32_t)(65536.0 * d->p + 0.5);
  a->factor = a->below < 65536u ? (float)(65536.0 / (65536.0 - a->below)) : 0.f;
  a->seed = d->seed;
  a->offset = d->offset;
  a->rng = d->rng;
  *drops = a->below > 0;
  return nullptr;
}

}  // namespace gbattn
