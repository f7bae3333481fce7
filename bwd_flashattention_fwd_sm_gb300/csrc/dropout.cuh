// The dropout mask of include/gbln.h, computed where it is used and never stored.
//
// An element's bits depend on (seed, offset, row, col) alone: Philox4x32 (Salmon,
// Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", 2011), a bijection
// of the 128-bit counter (col / 8, row, offset) under the 64-bit key seed.  One
// evaluation gives the 16 bits of eight neighbouring elements, one 16-byte vector of
// bfloat16.  Seven rounds: the fewest that the paper reports to pass BigCrush; a round is two 32 x 32 -> 64
// bit products, two exclusive ors and two additions, seven are a third of the 116 instructions that
// eight elements of a bfloat16 dropout take (61% of the issue slots at 94% of the copy rate).
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

// What a thread compares with: t in both halves of a word, its top bits and the rest apart.
struct DropRate {
  uint32_t whole, low, none;  // none: 0 if everything is dropped (t is 65536), else all ones
  float factor;
};

__device__ __forceinline__ DropRate drop_rate(const DropArgs& d) {
  const uint32_t t = (d.below & 0xFFFFu) * 0x10001u;
  return DropRate{t, t & 0x7FFF7FFFu, d.below > 0xFFFFu ? 0u : 0xFFFFFFFFu, d.factor};
}

// Both halves u of a word against t at once: their top bits are set where u >= t.  Without the
// top bits (u | top) - t cannot borrow from the other half; with them u >= t is u's bit if
// the two differ and that difference's bit if not.
__device__ __forceinline__ uint32_t drop_compare(uint32_t word, const DropRate& r) {
  const uint32_t d = (word | 0x80008000u) - r.low;
  return ((word & ~r.whole) | (~(word ^ r.whole) & d)) & r.none;
}

// Masks for what drop_compare gives, its top bits spread: of two 16-bit elements, of the lower
// and of the upper 32-bit element.
template <int kBytes>
__device__ __forceinline__ uint32_t drop_spread(uint32_t c) {
  uint32_t m;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(m) : "r"(c), "n"(kBytes));
  return m;
}
__device__ __forceinline__ uint32_t drop_mask_pair(uint32_t c) { return drop_spread<0xBB99>(c); }
__device__ __forceinline__ uint32_t drop_mask_low(uint32_t c) { return drop_spread<0x9999>(c); }
__device__ __forceinline__ uint32_t drop_mask_high(uint32_t c) { return drop_spread<0xBBBB>(c); }

// A 16-byte vector of T (at column c0 of its row) with 0 in the place of what is dropped; the
// factor is the caller's to apply.
template <class T>
__device__ __forceinline__ uint4 drop_mask(uint4 v, uint32_t c0, uint32_t row, const DropKey& key, const DropRate& r) {
  uint4 bits = drop_bits(key, c0 >> 3, row);
  if constexpr (sizeof(T) == 2) {
    v.x &= drop_mask_pair(drop_compare(bits.x, r));
    v.y &= drop_mask_pair(drop_compare(bits.y, r));
    v.z &= drop_mask_pair(drop_compare(bits.z, r));
    v.w &= drop_mask_pair(drop_compare(bits.w, r));
  } else {
    const bool upper = c0 & 4;
    const uint32_t a = drop_compare(upper ? bits.z : bits.x, r), b = drop_compare(upper ? bits.w : bits.y, r);
    v.x &= drop_mask_low(a);
    v.y &= drop_mask_high(a);
    v.z &= drop_mask_low(b);
    v.w &= drop_mask_high(b);
  }
  return v;
}

// The same at any column c0, where kAny says so: the vector's elements may belong to two groups (of
// a group in front of the row only elements that are no column).
template <class T, bool kAny>
__device__ __forceinline__ uint4 drop_mask_at(uint4 v, int c0, uint32_t row, const DropKey& key, const DropRate& r) {
  if constexpr (!kAny) {
    return drop_mask<T>(v, (uint32_t)c0, row, key, r);
  } else {
    const uint4 a = drop_bits(key, (uint32_t)(c0 >> 3), row), b = drop_bits(key, (uint32_t)(c0 >> 3) + 1, row);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    // the vector's 16-bit numbers to the front: by four, by two, by one
    if (c0 & 4)
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    if (c0 & 2)
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (c0 & 1) * 16);
    if constexpr (sizeof(T) == 2) {
      v.x &= drop_mask_pair(drop_compare(w[0], r));
      v.y &= drop_mask_pair(drop_compare(w[1], r));
      v.z &= drop_mask_pair(drop_compare(w[2], r));
      v.w &= drop_mask_pair(drop_compare(w[3], r));
    } else {
      const uint32_t x = drop_compare(w[0], r), y = drop_compare(w[1], r);
      v.x &= drop_mask_low(x);
      v.y &= drop_mask_high(x);
      v.z &= drop_mask_low(y);
      v.w &= drop_mask_high(y);
    }
    return v;
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
