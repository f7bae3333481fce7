// Attention over the 4-bit key/value cache.
//
// Few query rows meet many keys: the kernel is bound by the cache's bytes, and next
// by the instructions that turn codes into operands.  So keys take the place of the
// rows of a matrix product and the queries of one KV head (its group's heads times
// the new tokens) that of the columns: S^T = K Q^T and O^T = V^T P^T on
// m16n8k16 instructions, 16 keys (16 values of the head) by 8 queries.  A lane then
// needs whole code words of a key, in the order in which the cache holds them, and
// every operand is unpacked once however many columns there are.
//
//   K: word & 0x000F000F is a pair of codes u 2^-24 as float16 subnormals, word &
//      0x00F000F0 a pair u 2^-20: no conversion at all.  Q is held in float16, each
//      row scaled by its own power of two, those of
//      the second kind of pair by 1/16 more.  With s, b a key's step and offset of a
//      group, its part of the score is s sum(q u) + (b - 8 s) sum(q), in float32.
//   V: the same pairs, two keys side by side.  The weights p s are float16 too, each row's and
//      group's in units of a power of two of its own that follows the largest p s it has met, so
//      that this is 2^4 at least and 2^15 at most: 11 bits down to 2^-18 of it, off by at most
//      2^-29 of it below.  Units of the largest step would lose the sums of a row whose weight
//      lies on a position with small steps, such as a first token that all look at.
//      Sums of u instead of u - 8 would cancel against 8 sum(p s) over long contexts, so
//      a ninth product counts -8 sum(p s) beside them and is folded in every 128 keys;
//      the offsets' part sum(p b) stays in float32.
//   float32: the instruction cuts its sums off where it should round them, a bias that
//      grows with the context (3e-5 of O at 65536 keys).  So Q is three parts, multiples
//      of 2^4, 2^-6 and 2^-16, and the weights two, of 2^5 and 2^-6, each part of at most
//      11 bits: over 64 values or 16 keys, its products with u - 8 (exact in float16) add
//      up to less than 2^24 of its grid, nothing is cut off, and float32 additions join
//      the parts and the keys.  What is left of a weight, below 2^-7, is two more parts
//      in units of 2^-12, off by 2^-37 in the end, 2^-41 of the row's largest p s.
//
// Work.  A tile is the keys that a block's warps take at a time; the tiles of all
// sequences, KV heads and row tiles stand in one line that is cut into equal
// stretches, one a block, whatever the lengths are: the blocks read the lengths
// themselves.  A stretch that ends inside a row tile's keys leaves its partial
// result, which a second kernel joins in order, so results do not vary.
//
// Measured (bf16, 32 heads on 8 of 128): 64 sequences of up to 8192, one token each, 77 us, 60% of
// the rate of a copy; a sequence of 131072 38 us, 58%; one of 777 9.4 us with both kernels.  No pipe
// bounds it (issue slots 50% busy, ALU 46%, tensor pipe 25%, DRAM 57%), and hardly a warp waits for memory:
// two warps a scheduler, each with one chain of products, exp2 and products again, wait for their own
// results.  Without the arithmetic the same copies run at the rate of memory.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "kv4_line.cuh"
#include "ptx.cuh"

namespace gbattn {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;  // each warp joins and stores a quarter of a row tile's sums

// Scores may be 2^kSlack above the running maximum, steps 2^kRoom in the weights' units; together
// they stay at 2^15.  A weight that is found too large is brought below 2^kSet, so that steps
// of four times its size still have room.
constexpr int kSlack = 8, kRoom = 15 - kSlack, kSet = kRoom - 2;
constexpr int kFinest = 126;  // the weights' largest power of two: it and its reciprocal are normal numbers

// What a row tile costs beside its keys (queries into operands, the warps' results
// joined), in tiles: the line has that many empty places before a row tile's keys.  2, 6 and
// 12 with 64 sequences of up to 8192: 88, 76, 78 us; 16 of up to 4100 at head dim 256: 61, 52, 58.
constexpr int kEmpty = 6;

template <int D, int NT, bool F32>
struct Shape {
  static constexpr int G = D / kKv4Group;
  static constexpr int R = 8 * NT;                      // query rows of a row tile
  static constexpr int CH = (D == 256 || NT >= 3) ? 1 : 2;  // 16-key chunks of a warp at a time
  static constexpr int KT = kWarps * CH * 16;           // keys of a tile
  static constexpr int QP = F32 ? 3 : 1;                // float16 parts of Q
  static constexpr int PP = F32 ? 4 : 1;                // float16 parts of the weights
  static constexpr int FOLD = 8 / CH;                   // tiles between two folds: 128 keys of a warp
  static constexpr int ACC = G * 4 * NT * 4;            // accumulators of a lane
  // Blocks of an SM: 1, 2 and 3 (fewer registers) with 64 sequences of up to 8192 103, 76, 82 us, a
  // sequence of 131072 48, 38, 42.  Tiles in a warp's ring: 2, 3 and 4 75.8, 76.2 and 75.4 us, 37.8,
  // 38.3 and 37.8: the next block's warps cover what one waits for.
  static constexpr int BLOCKS = 2;
  static constexpr int STAGES = 2;
  static constexpr int CHUNK_BYTES = 16 * (D + 8 * G);  // K codes, V codes, K scales, V scales of 16 keys
  static constexpr int STAGE_BYTES = CH * CHUNK_BYTES;
  // Sums of u beside a count of -8 sum(p s): cheaper than subtracting 8 from each
  // code while there are few columns and registers for the count.
  static constexpr bool COUNT = NT == 1 && !F32;
  // The weights' units: a lane's own, or a warp's in shared memory where registers are short (16
  // sequences of up to 4100, bf16: head dim 256, 16 rows 41.3 and 40.3 us, 128, 20 rows 47.5 and 47.0).
  static constexpr bool UP_SMEM = G * NT > 4;
  static constexpr int GRID = kSms * BLOCKS;
  static constexpr size_t Q_BYTES = (size_t)G * 4 * NT * QP * 32 * 8;
  static constexpr size_t MERGE_BYTES = (size_t)kWarps * ACC * 32 * 4, RING_BYTES = (size_t)kWarps * STAGES * STAGE_BYTES;
  // The joined sums have a place of their own where two blocks of an SM have room for it, else
  // the rings'.
  static constexpr bool OVER = BLOCKS * (Q_BYTES + MERGE_BYTES + RING_BYTES + 4096) > 227 * 1024;
  static constexpr size_t SMEM =
      Q_BYTES + (!OVER ? MERGE_BYTES + RING_BYTES : MERGE_BYTES > RING_BYTES ? MERGE_BYTES : RING_BYTES);
};

__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, "
      "%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8x8 matrix of 16-bit elements (lane l holds row l / 4, columns 2 (l % 4) and + 1) transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// x to the nearest multiple of 2^k, for |x| < 2^(k + 22).
template <int k>
__device__ __forceinline__ float on_grid(float x) {
  constexpr float kBig = k >= 0 ? 12582912.f * (1 << (k >= 0 ? k : 0)) : 12582912.f / (1 << (k < 0 ? -k : 0));
  return __fsub_rn(__fadd_rn(x, kBig), kBig);
}
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }  // x > 0, normal
__device__ __forceinline__ uint32_t max_u16(uint32_t x, uint32_t y) {  // of both halves
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t add_f16(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// N values of a query row.
template <int N>
__device__ __forceinline__ void load_q(float (&q)[N], const float* p) {
  if constexpr (N == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    q[0] = v.x, q[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      q[i] = v.x, q[i + 1] = v.y, q[i + 2] = v.z, q[i + 3] = v.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void load_q(float (&q)[N], const __nv_bfloat16* p) {
  uint32_t w[N / 2];
  if constexpr (N == 2) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) q[2 * i] = bf16_lo(w[i]), q[2 * i + 1] = bf16_hi(w[i]);
}

// N words from shared memory.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], const uint8_t* p) {
  static_assert(N == 1 || N == 2 || N % 4 == 0, "vector loads");
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  }
}
// 16 bytes from global to shared memory, asynchronously; groups complete in order.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void store2(__nv_bfloat16* p, float x, float y) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16(x, y);
}
__device__ __forceinline__ void store2(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }

// Stores a 16 by 8 tile of a row tile's accumulators: accumulator e of tile j = (g, mt, nt) stands for row nt * 8 + 2 t + e % 2 and
// value 64 g + 8 (lane / 4) + 2 mt + e / 2 of the head.
template <class T, int NT>
__device__ __forceinline__ void store_tile(const Kv4Args& a, const Kv4Seq& s, int b, int h, int r0, int rows, int j,
                                           const float (&acc)[4], const float (&l)[2], int lane) {
  const int nt = j % NT, mt = j / NT % 4, g = j / NT / 4;
  const int d = g * kKv4Group + (lane >> 2) * 8 + 2 * mt;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = r0 + nt * 8 + 2 * (lane & 3) + e;
    if (row < rows) {
      const float inv = l[e] != 0.f ? 1.f / l[e] : 0.f;
      T* y = static_cast<T*>(a.y) + y_row(a, s, b, row_place(a, h, row)) + d;
      store2(y, acc[e] * inv, acc[2 + e] * inv);
    }
  }
}

template <class T, int D, int NT>
__global__ void __launch_bounds__(kThreads, (Shape<D, NT, sizeof(T) == 4>::BLOCKS))
    k_kv4_attn(const __grid_constant__ AttnArgs args) {
  constexpr bool F32 = sizeof(T) == 4;
  using S = Shape<D, NT, F32>;
  constexpr int G = S::G, R = S::R, CH = S::CH, KT = S::KT, QP = S::QP, PP = S::PP, ST = S::STAGES;
  const Kv4Args& a = args.a;
  extern __shared__ __align__(128) uint8_t smem[];
  uint2* qfrag = reinterpret_cast<uint2*>(smem);  // [g][s][part][nt][lane] (b0, b1)
  float* merge = reinterpret_cast<float*>(smem + S::Q_BYTES + (S::OVER ? 0 : S::RING_BYTES));
  __shared__ __align__(16) float row_f[R], row_z[G][R];  // read in pairs
  __shared__ int row_lim[R];
  __shared__ float warp_m[kWarps][R], warp_l[kWarps][R];
  __shared__ __align__(16) float warp_up[S::UP_SMEM ? kWarps : 1][S::UP_SMEM ? G : 1][R];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, t4 = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Line<R, KT, kEmpty, kWarps> line;
  const bool any = line.begin(a);
  if (threadIdx.x == 0) args.shared[blockIdx.x] = make_int4(0, 0, 0, -1);
  if (!any) return;
  const float q_sign = a.scale_log2 > 0.f ? 1.f : a.scale_log2 < 0.f ? -1.f : 0.f;

  // Copies into a warp's ring, 16 bytes a lane: codes in order, and the scales of a tile by
  // one copy (chunk lane / 8 G, K's in the first half of the 8 G lanes, V's in the second).
  uint8_t* ring = smem + S::Q_BYTES + warp * (ST * S::STAGE_BYTES);
  const uint8_t* k_from = a.kc + lane * 16;
  const uint8_t* v_from = a.vc + lane * 16;
  const uint8_t* s_from =
      reinterpret_cast<const uint8_t*>((lane / (4 * G) & 1) ? a.vs : a.ks) + lane % (4 * G) * 16;
  const uint32_t to = ptx::smem_u32(ring) + lane * 16;
  const uint32_t s_to = ptx::smem_u32(ring) + lane / (8 * G) * S::CHUNK_BYTES + 16 * D + lane % (8 * G) * 16;
  // Row r of eight keys is key r ^ (r >> 1 & 1): neighbours in K's reads and every second
  // row in V's then lie in both halves of the shared-memory banks.
  const int key8 = g8 ^ (g8 >> 1 & 1);
  const uint32_t k_lane = key8 * (D / 2) + t4 * (8 * G), s_lane = 16 * D + key8 * (4 * G);
  const uint32_t v_lane0 = 8 * D + ((2 * t4) ^ (t4 & 1)) * (D / 2) + g8 * (4 * G);
  const uint32_t v_lane1 = 8 * D + ((2 * t4 + 1) ^ (t4 & 1)) * (D / 2) + g8 * (4 * G);

  // ---- a piece's keys: where they lie, and the first copies; and its queries
  constexpr int kBatch = 8 / CH;  // tiles
  constexpr int E = D / 32;
  typename Line<R, KT, kEmpty, kWarps>::Piece next;
  bool more = line.next(a, &next);
  int t0 = 0, te = 0, klen = 0, h = 0, ids = 0;
  const int* table = nullptr;
  uint32_t rows_now = 0;
  bool bad = false;  // a chunk's page was none
  float q[R / kWarps][E];
  // Chunks of 16 keys, each in one page, in batches of 8: lane 4 x knows chunk x's row of
  // the cache.  Where the page is none, or no row sees the chunk, a row that does exist
  // is copied in its place, and masked.
  const int my_step = (lane >> 2) / CH, my_chunk = (lane >> 2) % CH;
  auto key_of = [&](int t) { return min((t + my_step) * KT + (warp * CH + my_chunk) * 16, (klen - 1) & ~15); };
  auto id_of = [&](int t) { return table[div_by(key_of(t), args.page_div)]; };
  auto rows_of = [&](int t, int id) {
    const int k0 = key_of(t), pg = div_by(k0, args.page_div);
    const bool ok = (unsigned)id < (unsigned)a.n_pages;
    if (!__all_sync(0xffffffffu, ok)) {
      bad = true;
      set_status(a.status, kStatusBounds);
    }
    return ((uint32_t)(ok ? id : 0) * a.heads_kv + h) * a.page + (k0 - pg * a.page);
  };
  auto issue = [&](int t) {  // tile t into its stage; tiles in order
    const int x = (t - t0) % kBatch;
    if (x == 0) {
      rows_now = rows_of(t, ids);
      ids = id_of(t + kBatch);
    }
    const uint32_t stage = (uint32_t)((t - t0) % ST) * S::STAGE_BYTES;
    uint32_t row[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      row[c] = __shfl_sync(0xffffffffu, rows_now, (x * CH + c) * 4);
      const uint8_t* k = k_from + (unsigned long long)row[c] * (D / 2);
      const uint8_t* v = v_from + (unsigned long long)row[c] * (D / 2);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        copy16(to + stage + c * S::CHUNK_BYTES + i * 512, k + i * 512);
        copy16(to + stage + c * S::CHUNK_BYTES + 8 * D + i * 512, v + i * 512);
      }
    }
    if (CH * 8 * G >= 32 || lane < CH * 8 * G)
      copy16(s_to + stage, s_from + (unsigned long long)(CH == 2 && lane >= 8 * G ? row[CH - 1] : row[0]) * (4 * G));
  };
  auto begin = [&]() {
    h = next.h, t0 = next.t0, klen = next.klen, bad = false;
    // This warp's tiles end where no row sees its keys.
    te = klen > warp * CH * 16 ? min(next.t1, (klen - warp * CH * 16 + KT - 1) / KT) : 0;
    table = a.table + next.b * a.table_stride;
#pragma unroll
    for (int y = 0; y < R / kWarps; ++y) {
#pragma unroll
      for (int e = 0; e < E; ++e) q[y][e] = 0.f;
      const int row = next.r0 + y * kWarps + warp;
      if (row < next.rows)
        load_q(q[y], static_cast<const T*>(a.x) + x_row(a, next.s, next.b, row_place(a, h, row)) + lane * E);
    }
    if (t0 < te) ids = id_of(t0);
#pragma unroll
    for (int x = 0; x < ST; ++x) {
      if (t0 + x < te) issue(t0 + x);
      copy_commit();
    }
  };
  if (more) begin();

  while (more) {
    const typename Line<R, KT, kEmpty, kWarps>::Piece p = next;
    const int b = p.b, r0 = p.r0, rows = p.rows, all_see = p.all_see;

    // ---- Q: each row's power of two, group sums and operands
    __syncthreads();  // nobody still reads the last row tile's
#pragma unroll
    for (int y = 0; y < R / kWarps; ++y) {
      const int r = y * kWarps + warp;
      float big = 0.f, sum = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        q[y][e] *= q_sign;
        big = fmaxf(big, fabsf(q[y][e])), sum += q[y][e];
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
#pragma unroll
      for (int o = 32 / G / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      // |q| < 2^(ex + 14), by the exponent's bits: scaled below 2^14
      const int ex = (big < INFINITY ? (int)(__float_as_uint(big) >> 23) - 126 : 0) - 14;
      // 2^-ex in two factors that are float32 numbers for every ex
      const float up = pow2(-ex / 2), up2 = pow2(-ex - -ex / 2);
      if (lane % (32 / G) == 0) row_z[lane / (32 / G)][r] = sum * up * up2 * 0x1p-24f;
      if (lane == 0) {
        // at least 2^-126, at most the largest float32: scores of 0 times it stay 0
        const float f = fabsf(a.scale_log2) * pow2(ex / 2 + 12) * pow2(ex - ex / 2 + 12);
        row_f[r] = a.scale_log2 != 0.f ? fminf(fmaxf(f, 1.17549435e-38f), 3.40282347e38f) : 1.f;
        const int pos = p.s.len - p.s.n + div_by(r0 + r, a.by_group);
        row_lim[r] = r0 + r >= rows ? kNoRow : pos < 0 ? 0 : a.causal ? pos + 1 : p.s.len;
      }
      __half* qh = reinterpret_cast<__half*>(qfrag);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int d = lane * E + e, g = d / 64, i = d % 64 / 8, n8 = d % 8;
        const int st = (i & 1) * 2 + (n8 & 3) / 2, reg = n8 & 1, half = n8 >> 2;
        float v = q[y][e] * up * up2;
#pragma unroll
        for (int part = 0; part < QP; ++part) {
          // parts of at most 11 bits: multiples of 2^4, 2^-6 and 2^-16
          const float t = !F32 ? v : part == 0 ? on_grid<4>(v) : part == 1 ? on_grid<-6>(v) : on_grid<-16>(v);
          const __half hv = __float2half_rn(reg ? t * 0.0625f : t);
          v -= t;
          qh[(((((g * 4 + st) * QP + part) * NT + r / 8) * 32 + (r & 7) * 4 + i / 2) * 2 + reg) * 2 + half] = hv;
        }
      }
    }
    __syncthreads();

    // up: the power of two that two rows' weights of a group are multiplied by; cap: steps that it leaves room
    // for.  acc: sums of those weights and u, in units of 2^-24 (values 0, 2, 4, 6 of a word) and
    // 2^-20 (1, 3, 5, 7).  minus: -8 sum(p s) since it was last folded in.
    float acc[G][4][NT][4], minus[S::COUNT ? G : 1][NT][4], accb[G][NT][2], bar[NT][2], mu[NT][2], l[NT][2];
    float cap[G];
    float2 own_up[S::UP_SMEM ? 1 : G][S::UP_SMEM ? 1 : NT];
    auto up = [&](int g, int nt) -> float2& {
      return S::UP_SMEM ? *reinterpret_cast<float2*>(&warp_up[S::UP_SMEM ? warp : 0][S::UP_SMEM ? g : 0][nt * 8 + 2 * t4])
                        : own_up[S::UP_SMEM ? 0 : g][S::UP_SMEM ? 0 : nt];
    };
#pragma unroll
    for (int g = 0; g < G; ++g) {
      cap[g] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        up(g, nt) = make_float2(pow2(kFinest), pow2(kFinest));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (S::COUNT) minus[g][nt][e] = 0.f;
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) acc[g][mt][nt][e] = 0.f;
        }
        accb[g][nt][0] = accb[g][nt][1] = 0.f;
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) bar[nt][e] = -INFINITY, mu[nt][e] = l[nt][e] = 0.f;
    // A row's sums of a group times f.
    auto rescale = [&](int g, int nt, int e, float f) {
      if constexpr (S::COUNT) minus[g][nt][e] *= f;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) acc[g][mt][nt][e] *= f, acc[g][mt][nt][2 + e] *= f;
    };
    auto fold = [&]() {
      if constexpr (S::COUNT) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int mt = 0; mt < 4; ++mt) {
                acc[g][mt][nt][e] += minus[g][nt][e];
                acc[g][mt][nt][2 + e] = fmaf(16.f, minus[g][nt][e], acc[g][mt][nt][2 + e]);
              }
#pragma unroll
            for (int e = 0; e < 4; ++e) minus[g][nt][e] = 0.f;
          }
      }
    };

    for (int t = t0; t < te; ++t) {
      const int k0 = t * KT + warp * CH * 16;
      const uint8_t* stage = ring + (uint32_t)((t - t0) % ST) * S::STAGE_BYTES;
      copy_wait<ST - 1>();
      __syncwarp();
      // S^T, in units of 1 / rf
      float x[CH][NT][4];
      {
        uint32_t kw[CH][2][2 * G];
        float sc[G][CH][NT][4];
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int y = 0; y < 2; ++y) lds_words(kw[c][y], stage + c * S::CHUNK_BYTES + k_lane + y * (4 * D));
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float low[F32 ? 2 : 1][F32 ? CH : 1][F32 ? NT : 1][4];  // Q's other parts: sums of their own
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            uint2 bq[QP][NT];
#pragma unroll
            for (int part = 0; part < QP; ++part)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                bq[part][nt] = qfrag[(((g * 4 + st) * QP + part) * NT + nt) * 32 + lane];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              const uint32_t wa = kw[c][0][(st >> 1) * G + g] >> (8 * (st & 1));
              const uint32_t wb = kw[c][1][(st >> 1) * G + g] >> (8 * (st & 1));
              uint32_t ak[4] = {wa & 0x000F000Fu, wb & 0x000F000Fu, wa & 0x00F000F0u, wb & 0x00F000F0u};
              if constexpr (F32) {
#pragma unroll
                for (int e = 0; e < 4; ++e) ak[e] = add_f16(ak[e], e < 2 ? 0x80088008u : 0x80808080u);  // -8: exact
              }
#pragma unroll
              for (int part = 0; part < QP; ++part)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float(&to)[4] = part == 0 ? sc[g][c][nt] : low[F32 ? part - 1 : 0][F32 ? c : 0][F32 ? nt : 0];
                  if (st == 0) mma_f16_first(to, ak, bq[part][nt].x, bq[part][nt].y);
                  else mma_f16(to, ak, bq[part][nt].x, bq[part][nt].y);
                }
            }
          }
#pragma unroll
          for (int c = 0; c < (F32 ? CH : 0); ++c)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[g][c][nt][e] += low[0][c][nt][e] + low[F32 ? 1 : 0][c][nt][e];
        }
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t ksw[G];
            lds_words(ksw, stage + c * S::CHUNK_BYTES + s_lane + y * (32 * G));
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const float st = bf16_lo(ksw[g]), z = F32 ? bf16_hi(ksw[g]) : fmaf(-8.f, st, bf16_hi(ksw[g]));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const float2 sum = *reinterpret_cast<const float2*>(&row_z[g][nt * 8 + 2 * t4]);
                const float p0 = g ? fmaf(z, sum.x, x[c][nt][2 * y]) : z * sum.x;
                const float p1 = g ? fmaf(z, sum.y, x[c][nt][2 * y + 1]) : z * sum.y;
                x[c][nt][2 * y] = fmaf(st, sc[g][c][nt][2 * y], p0);
                x[c][nt][2 * y + 1] = fmaf(st, sc[g][c][nt][2 * y + 1], p1);
              }
            }
          }
      }
      uint32_t vw[CH][4][G], vsw[CH][2][G];
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          lds_words(vw[c][2 * y], stage + c * S::CHUNK_BYTES + v_lane0 + y * (4 * D));
          lds_words(vw[c][2 * y + 1], stage + c * S::CHUNK_BYTES + v_lane1 + y * (4 * D));
          lds_words(vsw[c][y], stage + c * S::CHUNK_BYTES + s_lane + 64 * G + y * (32 * G));
        }
      __syncwarp();  // the stage is read: the tile ST ahead may come
      if (t + ST < te) issue(t + ST);
      copy_commit();

      // keys that not all rows see: by their places
      if (k0 + CH * 16 > all_see || bad) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int kc0 = min(k0 + c * 16, (klen - 1) & ~15);
          const bool dead = k0 + c * 16 >= klen || (bad && (unsigned)table[div_by(kc0, args.page_div)] >= (unsigned)a.n_pages);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int key = k0 + c * 16 + y * 8 + key8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (dead || key >= row_lim[nt * 8 + 2 * t4 + e]) x[c][nt][2 * y + e] = -INFINITY;
            if (dead || key >= p.s.len) {  // what no position holds may be anything: not into the sums
#pragma unroll
              for (int g = 0; g < G; ++g) vsw[c][y][g] = 0;
            }
#pragma unroll
            for (int g = 0; g < G; ++g)
              if (!finite2(vsw[c][y][g])) {  // to the rows that see it alone: 0 times it is not 0
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    if (key < row_lim[nt * 8 + 2 * t4 + e]) accb[g][nt][e] = NAN;
                vsw[c][y][g] = 0;
              }
          }
        }
      }
      // The running maximum is raised only when a score is above it by more than 2^kSlack, the weights
      // are looked at only then or when a step is above what their units have room for and may have
      // the weight to need it (where a position with small steps holds a row's weight, most steps are:
      // 64 sequences of up to 8192 76 us, so 80, and 97 if all of those were looked at).
      float high[NT][2], step[G];
      bool over = false, wide = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = fmaxf(x[0][nt][e], x[0][nt][2 + e]);
#pragma unroll
          for (int c = 1; c < CH; ++c) v = fmax3f(v, x[c][nt][e], x[c][nt][2 + e]);
          high[nt][e] = v;
          over |= v > bar[nt][e];
        }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float v = fmaxf(bf16_lo(vsw[0][0][g]), bf16_lo(vsw[0][1][g]));
#pragma unroll
        for (int c = 1; c < CH; ++c) v = fmax3f(v, bf16_lo(vsw[c][0][g]), bf16_lo(vsw[c][1][g]));
        step[g] = v;
        wide |= v > cap[g];
      }
      if (__any_sync(0xffffffffu, over || wide)) {
        over = __any_sync(0xffffffffu, over);
        if (!over) {
          // a lane's largest step with its largest weight
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 rf = *reinterpret_cast<const float2*>(&row_f[nt * 8 + 2 * t4]);
            const float p0 = fast_exp2(fmaf(high[nt][0], rf.x, -mu[nt][0]));
            const float p1 = fast_exp2(fmaf(high[nt][1], rf.y, -mu[nt][1]));
#pragma unroll
            for (int g = 0; g < G; ++g) over |= fmaxf(p0 * step[g] * up(g, nt).x, p1 * step[g] * up(g, nt).y) > 0x1p15f;
          }
          over = __any_sync(0xffffffffu, over);
        }
      }
      float fall[NT][2];  // what the weights so far are multiplied by, if over
      if (over) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = high[nt][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
            float f = 1.f;
            if (v > -INFINITY) {
              const float r = row_f[nt * 8 + 2 * t4 + e];
              v *= r;
              if (bar[nt][e] > -INFINITY) {
                v = fmaxf(v, mu[nt][e]);
                f = fast_exp2(mu[nt][e] - v);
              }
              mu[nt][e] = v;
              bar[nt][e] = (v + (float)kSlack) / r;
            }
            l[nt][e] *= f;
#pragma unroll
            for (int g = 0; g < G; ++g) accb[g][nt][e] *= f;
            fall[nt][e] = f;
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 rf = *reinterpret_cast<const float2*>(&row_f[nt * 8 + 2 * t4]);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[c][nt][e] = fast_exp2(fmaf(x[c][nt][e], (e & 1) ? rf.y : rf.x, -mu[nt][e & 1]));
            l[nt][e & 1] += x[c][nt][e];
          }
      }
      if (over) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          int most = -kFinest;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float v[2] = {0.f, 0.f};  // the rows' largest weights here
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                v[e] = fmax3f(v[e], x[c][nt][e] * bf16_lo(vsw[c][0][g]), x[c][nt][2 + e] * bf16_lo(vsw[c][1][g]));
            uint32_t both = __byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x7632);  // their first 16 bits
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) both = max_u16(both, __shfl_xor_sync(0xffffffffu, both, o));
            const float2 u = up(g, nt);
            if constexpr (S::UP_SMEM) __syncwarp();  // read by all lanes
            float to[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int size = (int)(both >> (e ? 23 : 7) & 255u) - 127;  // 2^size <= v < 2^(size + 1)
              // the sums' factor f: its power of two goes into the units, what is left of it is 1 to 2
              const float f = fall[nt][e];
              const int was = exponent(e ? u.y : u.x), less = f > 0.f ? -exponent(f) : 2 * kFinest;
              int now = min(was + less, kFinest);
              if (size + now >= kSet) now = kSet - 1 - size;
              const int by = now - was - less;
              rescale(g, nt, e, f > 0.f && by >= -126 ? f * pow2(less) * pow2(by) : 0.f);
              most = max(most, now);
              to[e] = pow2(now);
            }
            up(g, nt) = make_float2(to[0], to[1]);
          }
          cap[g] = pow2(min(kRoom - most, 127));
        }
      }

      // O^T += V^T (p s), and the offsets' sums
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int g = 0; g < G; ++g) {
          uint32_t pb[PP][NT][2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float st = bf16_lo(vsw[c][y][g]), o = bf16_hi(vsw[c][y][g]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              // p s first: it is finite where s times the units may not be
              const float2 u = up(g, nt);
              const Two ps = mul2(two(x[c][nt][2 * y], x[c][nt][2 * y + 1]), two(st, st));
              float p0 = apart(mul2(ps, two(u.x, u.y))).x, p1 = apart(mul2(ps, two(u.x, u.y))).y;
              accb[g][nt][0] = fmaf(x[c][nt][2 * y], o, accb[g][nt][0]);
              accb[g][nt][1] = fmaf(x[c][nt][2 * y + 1], o, accb[g][nt][1]);
#pragma unroll
              for (int part = 0; part < PP; ++part) {
                // two parts of at most 11 bits, multiples of 2^5 and 2^-6, and what is left, twice rounded
                float t0 = p0, t1 = p1;
                if (F32 && part == 0) t0 = on_grid<5>(p0), t1 = on_grid<5>(p1);
                if (F32 && part == 1) t0 = on_grid<-6>(p0), t1 = on_grid<-6>(p1);
                const uint32_t v = pack_f16(t0, t1);
                pb[part][nt][y] = transpose8(v);
                if (part + 1 < PP) p0 -= half_lo(v), p1 -= half_hi(v);
                if (F32 && part == 1) p0 *= 0x1p12f, p1 *= 0x1p12f;
              }
            }
          }
          // keys 2 t and 2 t + 1 (2 t + 8 and + 9) side by side, values 0 .. 3 and 4 .. 7 of the word
          uint32_t va[2][2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            va[y][0] = __byte_perm(vw[c][2 * y][g], vw[c][2 * y + 1][g], 0x5410);
            va[y][1] = __byte_perm(vw[c][2 * y][g], vw[c][2 * y + 1][g], 0x7632);
          }
          if constexpr (S::COUNT) {
            const uint32_t eight[4] = {0x80088008u, 0x80088008u, 0x80088008u, 0x80088008u};  // -8 2^-24
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(minus[g][nt], eight, pb[0][nt][0], pb[0][nt][1]);
          }
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            const uint32_t a0 = va[0][mt >> 1] >> (8 * (mt & 1)), a1 = va[1][mt >> 1] >> (8 * (mt & 1));
            uint32_t av[4] = {a0 & 0x000F000Fu, a0 & 0x00F000F0u, a1 & 0x000F000Fu, a1 & 0x00F000F0u};
            if constexpr (!S::COUNT) {
#pragma unroll
              for (int e = 0; e < 4; ++e) av[e] = add_f16(av[e], (e & 1) ? 0x80808080u : 0x80088008u);  // -8: exact
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (F32) {
                float sum[3][4];
#pragma unroll
                for (int part = 0; part < PP; ++part) {
                  if (part < 3) mma_f16_first(sum[part], av, pb[part][nt][0], pb[part][nt][1]);
                  else mma_f16(sum[2], av, pb[part][nt][0], pb[part][nt][1]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[g][mt][nt][e] += sum[0][e] + fmaf(sum[2][e], 0x1p-12f, sum[1][e]);
              } else {
                mma_f16(acc[g][mt][nt], av, pb[0][nt][0], pb[0][nt][1]);
              }
            }
          }
        }
      if ((t - t0) % S::FOLD == S::FOLD - 1) fold();
    }
    fold();
    // The next piece's first copies come in while this one's sums are joined.
    more = line.next(a, &next);
    if (!S::OVER && more) begin();
    // to the values' own units, the offsets' part added
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) accb[g][nt][e] += __shfl_xor_sync(0xffffffffu, accb[g][nt][e], o);
          const float down = pow2(-exponent(e ? up(g, nt).y : up(g, nt).x));
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            acc[g][mt][nt][e] = fmaf(acc[g][mt][nt][e] * 0x1p24f, down, accb[g][nt][e]);
            acc[g][mt][nt][2 + e] = fmaf(acc[g][mt][nt][2 + e] * 0x1p20f, down, accb[g][nt][e]);
          }
        }

    // ---- the warps' results joined
    float m[NT][2];  // in log2 units
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = bar[nt][e] == -INFINITY ? -INFINITY : mu[nt][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], o);
        if (g8 == 0) {
          warp_m[warp][nt * 8 + 2 * t4 + e] = m[nt][e];
          warp_l[warp][nt * 8 + 2 * t4 + e] = l[nt][e];
        }
      }
    __syncthreads();
    float rm[NT][2], rl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * t4 + e;
        float v = warp_m[0][r];
#pragma unroll
        for (int y = 1; y < kWarps; ++y) v = fmaxf(v, warp_m[y][r]);
        rm[nt][e] = v;
        const float u = v == -INFINITY ? 0.f : v;
        rl[nt][e] = 0.f;
#pragma unroll
        for (int y = 0; y < kWarps; ++y)
          rl[nt][e] += warp_m[y][r] == -INFINITY ? warp_l[y][r] : warp_l[y][r] * fast_exp2(warp_m[y][r] - u);
        const float f = m[nt][e] == -INFINITY ? 1.f : fast_exp2(m[nt][e] - u);
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) acc[g][mt][nt][e] *= f, acc[g][mt][nt][2 + e] *= f;
      }
#pragma unroll
    for (int j = 0; j < G * 4 * NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        merge[(warp * S::ACC + j * 4 + e) * 32 + lane] = acc[j / NT / 4][j / NT % 4][j % NT][e];
    __syncthreads();
    const bool whole = p.whole;
    if (p.t0 == 0 && !whole && threadIdx.x == 0)
      args.shared[blockIdx.x] = make_int4(b, p.h, r0 / R, line.owner(p.last, line.total, line.n));
    const long long slot = blockIdx.x * 2 + (p.t0 == 0 ? 1 : 0);
#pragma unroll
    for (int jj = 0; jj < G * NT; ++jj) {
      const int j = warp * G * NT + jj;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = 0.f;
#pragma unroll
        for (int y = 0; y < kWarps; ++y) v[e] += merge[(y * S::ACC + j * 4 + e) * 32 + lane];
      }
      if (whole) {
        store_tile<T, NT>(a, p.s, b, p.h, r0, rows, j, v, rl[j % NT], lane);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) args.part_o[(slot * S::ACC + j * 4 + e) * 32 + lane] = v[e];
      }
    }
    if (warp == 0 && g8 == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nt * 8 + 2 * t4 + e;
          if (whole) {
            if (r0 + r < rows) a.lse[lse_row(a, p.s, b, row_place(a, p.h, r0 + r))] = row_lse(rm[nt][e], rl[nt][e]);
          } else {
            args.part_ml[(slot * R + r) * 2] = rm[nt][e];
            args.part_ml[(slot * R + r) * 2 + 1] = rl[nt][e];
          }
        }
    }
    if (S::OVER && more) {
      __syncthreads();  // the joined sums are read: the rings may take their place
      begin();
    }
  }
}

// Joins the parts of row tiles whose keys several blocks shared, in a fixed order: a
// block for each 16 by 8 tile of a row tile's accumulators, a warp for every eighth
// part, four parts' loads at a time.
constexpr int kJoinWarps = 8;
template <class T, int D, int NT>
__global__ void __launch_bounds__(kJoinWarps * 32) k_kv4_join(const __grid_constant__ AttnArgs args) {
  using S = Shape<D, NT, sizeof(T) == 4>;
  constexpr int R = S::R, kAhead = 4;
  const Kv4Args& a = args.a;
  __shared__ float sm[kJoinWarps][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t4 = lane & 3;
  const int i0 = blockIdx.x, j = blockIdx.y, nt = j % NT;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
  const int4 tile = __ldcg(&args.shared[i0]);
  const int b = tile.x, h = tile.y, rt = tile.z, i1 = tile.w;
  if (i1 < 0) return;
  const Kv4Seq seq = kv4_seq(a, b);

  float acc[4] = {0.f, 0.f, 0.f, 0.f}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  auto add = [&](const float (&v)[4], const float (&pm)[2], const float (&pl)[2]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float top = fmaxf(m[e], pm[e]), u = top == -INFINITY ? 0.f : top;
      const float f = m[e] == -INFINITY ? 1.f : fast_exp2(m[e] - u);
      const float fp = pm[e] == -INFINITY ? 1.f : fast_exp2(pm[e] - u);
      m[e] = top;
      l[e] = l[e] * f + pl[e] * fp;
      acc[e] = acc[e] * f + v[e] * fp;
      acc[2 + e] = acc[2 + e] * f + v[2 + e] * fp;
    }
  };
  for (int i = i0 + warp; i <= i1; i += kJoinWarps * kAhead) {
    float v[kAhead][4], pm[kAhead][2], pl[kAhead][2];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int part = i + k * kJoinWarps;
      if (part <= i1) {
        const long long slot = (long long)part * 2 + (part == i0 ? 1 : 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = __ldcg(&args.part_o[(slot * S::ACC + j * 4 + e) * 32 + lane]);
        const float4 ml = __ldcg(reinterpret_cast<const float4*>(args.part_ml + (slot * R + nt * 8 + 2 * t4) * 2));
        pm[k][0] = ml.x, pl[k][0] = ml.y, pm[k][1] = ml.z, pl[k][1] = ml.w;
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k * kJoinWarps <= i1) add(v[k], pm[k], pl[k]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sm[warp][e][lane] = acc[e];
#pragma unroll
  for (int e = 0; e < 2; ++e) sm[warp][4 + e][lane] = m[e], sm[warp][6 + e][lane] = l[e];
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int y = 1; y < kJoinWarps; ++y) {
    const float v[4] = {sm[y][0][lane], sm[y][1][lane], sm[y][2][lane], sm[y][3][lane]};
    const float pm[2] = {sm[y][4][lane], sm[y][5][lane]}, pl[2] = {sm[y][6][lane], sm[y][7][lane]};
    add(v, pm, pl);
  }
  const int rows = seq.n * a.group, r0 = rt * R;
  store_tile<T, NT>(a, seq, b, h, r0, rows, j, acc, l, lane);
  if (j < NT && lane < 4) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = r0 + nt * 8 + 2 * t4 + e;
      if (row < rows) a.lse[lse_row(a, seq, b, row_place(a, h, row))] = row_lse(m[e], l[e]);
    }
  }
}

template <class T, int D, int NT>
struct Launch {
  using S = Shape<D, NT, sizeof(T) == 4>;
  // Blocks: no more than there can be tiles.
  static int grid(const Kv4Args& a) {
    const long long row_tiles = ((long long)a.seqlen * a.group + S::R - 1) / S::R;
    const long long key_tiles = std::max(1ll, ((long long)a.max_pages * a.page + S::KT - 1) / S::KT);
    const long long most = (long long)a.batch * a.heads_kv * row_tiles;
    return (int)(most >= S::GRID ? S::GRID : std::min<long long>(S::GRID, most * std::min(key_tiles, (long long)S::GRID)));
  }
  static size_t o_bytes(const Kv4Args& a) { return (size_t)grid(a) * 2 * S::ACC * 32 * 4; }
  static size_t ml_bytes(const Kv4Args& a) { return (size_t)grid(a) * 2 * S::R * 8; }
  static size_t workspace(const Kv4Args& a) { return o_bytes(a) + ml_bytes(a) + (size_t)grid(a) * sizeof(int4); }
  static cudaError_t run(const Kv4Args& a, void* ws, cudaStream_t st) {
    AttnArgs args = {};
    args.a = a;
    args.page_div = fast_div(a.page);
    args.part_o = static_cast<float*>(ws);
    args.part_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + o_bytes(a));
    args.shared = reinterpret_cast<int4*>(static_cast<char*>(ws) + o_bytes(a) + ml_bytes(a));
    // the kernel's shared-memory limit, once a device
    static std::atomic<unsigned long long> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(k_kv4_attn<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::SMEM);
      if (e != cudaSuccess) return e;
      raised.fetch_or(bit, std::memory_order_relaxed);
    }
    const int n = grid(a);
    k_kv4_attn<T, D, NT><<<n, kThreads, S::SMEM, st>>>(args);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((long long)a.max_pages * a.page <= S::KT) return cudaSuccess;  // a row tile has one tile of keys
    // The join may be set up while the first kernel still runs: its blocks wait for that
    // kernel's end themselves.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n, S::ACC / 4);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_kv4_join<T, D, NT>, args);
  }
};

// Row tiles of 8, 16 or 24 queries: the least that hold all of a KV head's, else the
// widest that the registers hold (accumulators: D / 16 * 4 a lane and 8 queries).
// Sequences of 8192 tokens, 32 heads on 8, 4 / 16 new tokens each, us, 16 rows against 8:
// float32 head dim 64 (8 sequences) 39 / 125 against 42 / 139, 128 72 / 238 against 71 / 241,
// 256 160 / 531 against 139 / 498; bf16 256 84 / 235 against 78 / 262.
// More bf16 rows than 24 at head dim 64 and 128 are the tcgen05 kernel's.
template <class T, int D, class F>
auto with_width(const Kv4Args& a, F&& f) {
  constexpr int kWide = sizeof(T) == 2 ? (D <= 128 ? 3 : 2) : (D == 64 ? 2 : 1);
  const long long rows = (long long)a.seqlen * a.group;
  if (rows <= 8 || kWide == 1) return f(Launch<T, D, 1>());
  if (rows <= 16 || kWide == 2) return f(Launch<T, D, kWide < 2 ? 1 : 2>());
  return f(Launch<T, D, kWide>());
}
template <class F>
auto with_shape(const Kv4Args& a, int head_dim, bool bf16, F&& f) {
  if (bf16) {
    if (head_dim == 64) return with_width<__nv_bfloat16, 64>(a, f);
    if (head_dim == 128) return with_width<__nv_bfloat16, 128>(a, f);
    return with_width<__nv_bfloat16, 256>(a, f);
  }
  if (head_dim == 64) return with_width<float, 64>(a, f);
  if (head_dim == 128) return with_width<float, 128>(a, f);
  return with_width<float, 256>(a, f);
}

}  // namespace

size_t kv4_attn_workspace(const Kv4Args& a, int head_dim, bool bf16) {
  return with_shape(a, head_dim, bf16, [&](auto k) { return decltype(k)::workspace(a); });
}

cudaError_t launch_kv4_attn(const Kv4Args& a, int head_dim, bool bf16, void* workspace, cudaStream_t st) {
  return with_shape(a, head_dim, bf16, [&](auto k) { return decltype(k)::run(a, workspace, st); });
}

}  // namespace gbattn
