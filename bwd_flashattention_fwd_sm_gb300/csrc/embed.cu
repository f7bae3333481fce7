// Embedding table: lookup with scaling, and the table's gradient by sorted tokens
// (include/gbembed.h has the formulas).
//
// Lookup.  Bound by device memory; every thread has several vectors in flight, because a
// row's address waits for its id.
//
// Gradient.  One launch sorts the tokens' places by id (a stable radix sort by one cluster of
// blocks, all in shared memory but the hand-over between passes) while its other blocks write
// zeros over the table.  The sorted places are cut in pieces of 16 to 64, and each block adds the rows of
// one piece over a stretch of columns: equal work however often a word comes.  A word
// that lies inside one piece is written to the table at once; of one that
// several pieces share each piece leaves a partial sum, and k_embed_join adds those in order.
// No atomics on sums: their order follows from the ids, the sizes and the types.
// Up to kFewTokens tokens take one launch and no workspace (k_embed_few): each block finds its word's places
// by reading all ids.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <type_traits>

#include "../../include/gbembed.h"
#include "common.cuh"
#include "overlap.h"

namespace gbattn {
void set_last_error_text(const char* text);
attn_status_t device_status(int** status, int* sms, unsigned long long* wait_ns);

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;     // lookup, fill
template <class T, int N>
constexpr int kAtOnce = sizeof(T) * N >= 8 ? 4 : 8;  // accesses of a thread in flight
constexpr int kMostPiece = 64;    // sorted places of one block of the gradient's sums (a.piece), at most
constexpr int kSumThreads = 128;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBits = 10;      // of one pass's digit: a thread a digit
constexpr int kHeld = 8;          // places of a lane that stay in shared memory
constexpr int kMaxCluster = 8;
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinCols = 128;    // columns taken together: four each lane
constexpr int kFew = 16;          // partial sums (after a word's first) that one warp adds
// Tokens that go without sorting.  300 tokens of a table [1000, 256] take 4.5 us this way and 14 sorted;
// a word that comes 512 times is added by one block a stretch of columns, 20 us.
constexpr int kFewTokens = 512;
constexpr int kFewThreads = 512;
constexpr int kFewParts = kFewThreads / kSumThreads;  // of a word's places, added side by side
constexpr int kFillRows = 8192;   // rows of the table whose words a block notes at once
constexpr int64_t kMaxDim = 1 << 20;

// N neighbouring elements of T as one load or store, widened to float32.
template <class T, int N>
struct Elems {
  static_assert(sizeof(T) * N == 16 || sizeof(T) * N == 8 || sizeof(T) * N == 4 || sizeof(T) * N == 2, "one access");
  union U {
    T t[N];
    uint4 w16;
    uint2 w8;
    uint32_t w4;
    __device__ U() {}
  };
  __device__ static U raw(const T* p) {
    U u;
    if constexpr (sizeof(T) * N == 16) u.w16 = *reinterpret_cast<const uint4*>(p);
    else if constexpr (sizeof(T) * N == 8) u.w8 = *reinterpret_cast<const uint2*>(p);
    else if constexpr (sizeof(T) * N == 4) u.w4 = *reinterpret_cast<const uint32_t*>(p);
    else u.w4 = *reinterpret_cast<const uint16_t*>(p);  // in a register of its own: packed, each load waits for the last
    return u;
  }
  __device__ static U zero() {
    U u;
    u.w4 = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if constexpr (sizeof(T) * N > 4) u.t[i] = from_f32<T>(0.f);
    return u;
  }
  __device__ static void widen(const U& u, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if constexpr (sizeof(T) * N == 2) v[i] = __uint_as_float(u.w4 << 16);  // bfloat16
      else v[i] = to_f32(u.t[i]);
  }
  __device__ static void load(const T* p, float (&v)[N]) { widen(raw(p), v); }
  __device__ static void store(T* p, const float (&v)[N]) {
    U u;
#pragma unroll
    for (int i = 0; i < N; ++i) u.t[i] = from_f32<T>(v[i]);
    if constexpr (sizeof(T) * N == 16) *reinterpret_cast<uint4*>(p) = u.w16;
    else if constexpr (sizeof(T) * N == 8) *reinterpret_cast<uint2*>(p) = u.w8;
    else if constexpr (sizeof(T) * N == 4) *reinterpret_cast<uint32_t*>(p) = u.w4;
    else *p = u.t[0];
  }
};

struct EmbedArgs {
  const void* ids;
  const void* x;        // weight, or dy
  void* y;              // y, or dweight
  int64_t tokens, vocab, dim;
  int64_t x_stride, y_stride;
  int64_t padding;
  uint32_t row_step, unit_step;  // fill: all threads' vectors on, as rows and vectors of a row
  float scale;
  int ids_64, accumulate;
  uint2* pairs[2];      // gradient: ids and places, before and after a pass of the sort
  float* part;          // [pieces][2][dim]: sums of words that began before the piece, that go on after it
  // Words that several pieces share: how many of few partial sums and of many, and the pieces in which they
  // begin (in any order): the few from the front of [pieces] numbers, the many from the back.
  uint32_t* shared;
  int passes, bits, piece;
  int* status;
};

__device__ __forceinline__ int64_t id_at(const EmbedArgs& a, int64_t i) {
  return a.ids_64 ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
}

// `lanes` threads (a power of two) on a row; each has up to kAtOnce accesses of it in flight.
template <class T, int N>
__global__ void __launch_bounds__(kThreads, 6) k_embed(const EmbedArgs a, int lanes_log) {
  constexpr int kAt = kAtOnce<T, N>;
  const int lanes = 1 << lanes_log;
  const int64_t row = (int64_t)blockIdx.x * (kThreads >> lanes_log) + (threadIdx.x >> lanes_log);
  if (row >= a.tokens) return;
  const int64_t id = id_at(a, row);
  const bool there = id >= 0 && id < a.vocab;
  if (!there) set_status(a.status, kStatusBounds);
  const int units = (int)(a.dim / N);  // N divides dim
  const T* w = static_cast<const T*>(a.x) + (there ? id : 0) * a.x_stride;
  T* y = static_cast<T*>(a.y) + row * a.y_stride;
  for (int u = threadIdx.x & (lanes - 1); u < units; u += kAt * lanes) {
    typename Elems<T, N>::U v[kAt];
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      v[i] = Elems<T, N>::zero();
      if (there && u + i * lanes < units) v[i] = Elems<T, N>::raw(w + (u + i * lanes) * N);
    }
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      if (u + i * lanes >= units) continue;
      float x[N];
      Elems<T, N>::widen(v[i], x);
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] *= a.scale;
      Elems<T, N>::store(y + (u + i * lanes) * N, x);
    }
  }
}

// Zeros over the whole table, by `blocks` blocks of which this one is number `block`.
template <class W, int N>
__device__ __forceinline__ void fill_table(const EmbedArgs& a, int64_t block, int64_t blocks) {
  const uint32_t units = (uint32_t)a.dim / N, at = (uint32_t)(block * blockDim.x + threadIdx.x);  // grids are small
  uint32_t unit = at % units;
  int64_t row = at / units;
  const float zero[N] = {};
  while (row < a.vocab) {
    Elems<W, N>::store(static_cast<W*>(a.y) + row * a.y_stride + (int64_t)unit * N, zero);
    row += a.row_step, unit += a.unit_step;
    if (unit >= units) unit -= units, ++row;
  }
}

// The sort key of place i: its id; `vocab`, behind all others, if its row of dy goes nowhere.
__device__ __forceinline__ uint32_t key_at(const EmbedArgs& a, int64_t i) {
  const int64_t id = id_at(a, i);
  if (id < 0 || id >= a.vocab) {
    set_status(a.status, kStatusBounds);
    return (uint32_t)a.vocab;
  }
  return id == a.padding ? (uint32_t)a.vocab : (uint32_t)id;
}

// Stable sort of (id, place) by id: `passes` passes over digits of `bits` bits, least
// significant first.  Every warp of the cluster owns a stretch of the input.  It counts its
// digits; the counts of all warps in front of it and of all lower digits say where its
// first of each digit goes; then it takes its stretch in order, 32 at a time, and those
// with equal digits find their order by votes.  Ends in buffer passes % 2.  A warp's first kHeld * 32
// places (65536 tokens of the cluster) stay in shared memory between the two; later ones are read twice.
// Bound by the latency of its steps and by fetching its instructions, which run once or a
// few times: loops stay rolled (unrolled over a thread's places most of a pass was fetches).  16384 tokens of
// a table of 50000 (two passes): 30,000 cycles, half of them votes; 40001 of 1000 (one): 22,000.
__device__ void sort_places(const EmbedArgs& a, uint32_t* count) {
  __shared__ uint32_t total[1 << kMaxBits];   // of the block, for the cluster
  __shared__ uint32_t start[1 << kMaxBits];   // where the block's first of a digit goes
  __shared__ uint32_t warp_total[kSortWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster.block_rank(), blocks = cluster.num_blocks();
  const uint32_t digits = 1u << a.bits, tokens = (uint32_t)a.tokens;  // below 2^31
  const uint32_t each = (tokens / (blocks * kSortWarps) / 32 + 1) * 32;
  const uint32_t begin = min(tokens, (rank * kSortWarps + warp) * each), end = min(tokens, begin + each);
  uint32_t* mine = count + warp * digits;
  uint2* held = reinterpret_cast<uint2*>(count + kSortWarps * digits) + warp * kHeld * 32;
  if (rank == 0 && threadIdx.x < 2) a.shared[threadIdx.x] = 0;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    const uint2* pairs = a.pairs[pass & 1];
    uint2* pairs_to = a.pairs[(pass + 1) & 1];
    auto pair_at = [&](uint32_t i) { return pass == 0 ? make_uint2(key_at(a, i), i) : __ldcg(pairs + i); };
    for (uint32_t d = 4 * lane; d < digits; d += 128) *reinterpret_cast<uint4*>(mine + d) = make_uint4(0u, 0u, 0u, 0u);
    __syncwarp();
#pragma unroll 4
    for (uint32_t i = begin + lane; i < end; i += 32) {
      const uint2 p = pair_at(i);
      atomicAdd(&mine[(p.x >> shift) & (digits - 1)], 1u);
      if (i - begin < kHeld * 32) held[i - begin] = p;
    }
    __syncthreads();
    uint32_t sum = 0;  // of this thread's digit; counts become those of the warps in front
    if (threadIdx.x < digits) {
#pragma unroll 1
      for (int w0 = 0; w0 < kSortWarps; w0 += 16) {
        uint32_t* at = count + w0 * digits + threadIdx.x;
        uint32_t n[16];
#pragma unroll
        for (int w = 0; w < 16; ++w) n[w] = at[w * digits];
#pragma unroll
        for (int w = 0; w < 16; ++w) {
          at[w * digits] = sum;
          sum += n[w];
        }
      }
      total[threadIdx.x] = sum;
    }
    if (blocks > 1) cluster.sync();
    uint32_t all = sum, before = 0;
    if (blocks > 1 && threadIdx.x < digits) {
      uint32_t n[kMaxCluster];
#pragma unroll
      for (uint32_t r = 0; r < kMaxCluster; ++r) n[r] = r < blocks ? cluster.map_shared_rank(total, r)[threadIdx.x] : 0;
      all = 0;
#pragma unroll
      for (uint32_t r = 0; r < kMaxCluster; ++r) {
        all += n[r];
        if (r < rank) before += n[r];
      }
    }
    uint32_t upto = all;  // inclusive over the digits of a warp, then of the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t n = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += n;
    }
    if (lane == 31) warp_total[warp] = upto;
    __syncthreads();
    uint32_t in_front = lane < warp ? warp_total[lane] : 0;
    in_front = __reduce_add_sync(0xffffffffu, in_front);
    if (threadIdx.x < digits) start[threadIdx.x] = in_front + before + upto - all;
    __syncthreads();
#pragma unroll 1
    for (uint32_t i0 = begin; i0 < end; i0 += 32) {
      const uint32_t i = i0 + lane, at = i - begin;
      const bool there = i < end;
      uint2 p = make_uint2(0u, 0u);
      if (there) p = at < kHeld * 32 ? held[at] : pair_at(i);
      const uint32_t d = (p.x >> shift) & (digits - 1);
      // which lanes have the same digit: a vote for each bit (1700 cycles for 32 warps; __match_any_sync 2600)
      unsigned same = __ballot_sync(0xffffffffu, there);
#pragma unroll
      for (int b = 0; b < kMaxBits; ++b) {
        const bool one = d >> b & 1;
        const unsigned ones = __ballot_sync(0xffffffffu, one);
        same &= one ? ones : ~ones;
      }
      const uint32_t first = mine[d], to = start[d] + first + __popc(same & ((1u << lane) - 1));
      if (there && bounds_ok(to < tokens, a.status)) pairs_to[to] = p;
      __syncwarp();
      if (there && lane == __ffs(same) - 1) mine[d] = first + __popc(same);
      __syncwarp();
    }
    if (blocks > 1)
      cluster.sync();  // the next pass reads what all blocks wrote; `total` may be written again
    else
      __syncthreads();
  }
}

// The first cluster sorts, the other blocks write zeros.
template <class W, int N>
__global__ void __launch_bounds__(kSortThreads) k_embed_sort(const EmbedArgs a) {
  extern __shared__ __align__(16) uint32_t count[];  // [kSortWarps][digits], and pairs [kSortWarps][kHeld * 32]
  const unsigned sorting = cg::this_cluster().num_blocks();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x < sorting)
    sort_places(a, count);
  else
    fill_table<W, N>(a, blockIdx.x - sorting, gridDim.x - sorting);
}

template <class W, int N>
__global__ void __launch_bounds__(kThreads) k_embed_fill(const EmbedArgs a) {
  fill_table<W, N>(a, blockIdx.x, gridDim.x);
}

// The sums of one piece of sorted places over kSumThreads * N * kLoads columns: kLoads accesses of N
// columns a thread, kRows rows of dy in flight.
template <class T, class W, int N, int kLoads, int kRows>
__global__ void __launch_bounds__(kSumThreads) k_embed_sum(const EmbedArgs a) {
  __shared__ uint32_t key[kMostPiece + 2];  // with the neighbours on both sides
  __shared__ uint32_t place[kMostPiece];
  const uint32_t piece = a.piece, begin = blockIdx.x * piece, tokens = (uint32_t)a.tokens;
  const int n = (int)min(tokens - begin, piece);
  const uint2* pairs = a.pairs[a.passes & 1];
  const uint32_t none = (uint32_t)a.vocab;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // sorted, and zeros written
  if ((int)threadIdx.x < n + 2) {
    const uint32_t at = begin + threadIdx.x - 1;  // wraps in front of the first
    const uint2 p = at < tokens ? pairs[at] : make_uint2(none, 0);
    key[threadIdx.x] = p.x;
    if (threadIdx.x >= 1 && (int)threadIdx.x <= n) place[threadIdx.x - 1] = p.y;
  }
  __syncthreads();
  if (blockIdx.y == 0 && threadIdx.x == 0) {  // a word that begins here and goes on
    const uint32_t k = key[n];
    if (k < none && key[n + 1] == k && (key[1] != k || key[0] != k)) {
      const uint64_t far = (uint64_t)begin + (kFew + 1) * piece;
      const bool many = far < tokens && pairs[far].x == k;
      const uint32_t at = atomicAdd(a.shared + many, 1u);
      a.shared[2 + (many ? gridDim.x - 1 - at : at)] = blockIdx.x;
    }
  }
  constexpr int kApart = kSumThreads * N;  // columns between a thread's accesses
  const int dim = (int)a.dim, c0 = blockIdx.y * kApart * kLoads + threadIdx.x * N;
  if (c0 >= dim) return;
  const T* DY = static_cast<const T*>(a.x) + c0;
  float sum[kLoads][N];
#pragma unroll
  for (int l = 0; l < kLoads; ++l)
#pragma unroll
    for (int e = 0; e < N; ++e) sum[l][e] = 0.f;
  bool from_before = key[0] == key[1];
#pragma unroll 1
  for (int i0 = 1; i0 <= n; i0 += kRows) {
    if (key[i0] >= none) break;  // sorted behind all words
    typename Elems<T, N>::U v[kRows][kLoads];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int i = i0 + u;
      const bool there = i <= n && key[i] < none && bounds_ok(place[i - 1] < (uint64_t)a.tokens, a.status);
      const T* row = DY + (there ? (int64_t)place[i - 1] * a.x_stride : 0);
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        v[u][l] = Elems<T, N>::zero();
        if (there && c0 + l * kApart < dim) v[u][l] = Elems<T, N>::raw(row + l * kApart);
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int i = i0 + u;
      const uint32_t k = i <= n ? key[i] : none;
      if (k >= none) continue;
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        float w[N];
        Elems<T, N>::widen(v[u][l], w);
#pragma unroll
        for (int e = 0; e < N; ++e) sum[l][e] += w[e];
      }
      const bool goes_on = key[i + 1] == k;
      if (goes_on && i < n) continue;
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        if (c0 + l * kApart >= dim) continue;
        if (from_before || goes_on) {
          float* part = a.part + (2 * (int64_t)blockIdx.x + (from_before ? 0 : 1)) * dim + c0 + l * kApart;
#pragma unroll
          for (int e = 0; e < N; ++e) part[e] = sum[l][e];
        } else {
          W* to = static_cast<W*>(a.y) + (int64_t)k * a.y_stride + c0 + l * kApart;
          float old[N];
          if (a.accumulate) Elems<W, N>::load(to, old);
#pragma unroll
          for (int e = 0; e < N; ++e) sum[l][e] = a.accumulate ? old[e] + a.scale * sum[l][e] : a.scale * sum[l][e];
          Elems<W, N>::store(to, sum[l]);
        }
#pragma unroll
        for (int e = 0; e < N; ++e) sum[l][e] = 0.f;
      }
      from_before = false;
    }
  }
}

// Words that several pieces share: the partial sums of the piece in which a word begins, and of those
// after it.  Few: a warp adds kJoinCols columns of them in order.  Many: a block does, each warp a
// stretch of them, and then the warps' sums in order.
template <class W>
__global__ void __launch_bounds__(kJoinThreads) k_embed_join(const EmbedArgs a) {
  __shared__ float sums[kJoinWarps][kJoinCols];
  const uint2* pairs = a.pairs[a.passes & 1];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tokens = (uint32_t)a.tokens;
  const uint32_t dim = (uint32_t)a.dim, groups = (dim + kJoinCols - 1) / kJoinCols;
  const uint32_t piece = a.piece, pieces = (tokens + piece - 1) / piece;
  // partial sums `from` .. `to` - 1 after the first of the word that begins in piece `first`
  auto add = [&](uint32_t first, uint32_t from, uint32_t to, uint32_t col, float (&s)[4]) {
    const float* p = a.part + 2 * (int64_t)(first + 1 + from) * dim + col;
#pragma unroll 1
    for (uint32_t i = from; i < to; i += 4, p += 8 * (int64_t)dim) {
      float v[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[u][e] = i + u < to && col + 32 * e < dim ? p[2 * u * (int64_t)dim + 32 * e] : 0.f;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += v[u][e];
    }
  };
  auto begin = [&](uint32_t first, uint32_t col, float (&s)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = col + 32 * e < dim ? a.part[(2 * (int64_t)first + 1) * dim + col + 32 * e] : 0.f;
  };
  auto finish = [&](uint32_t k, uint32_t col, const float (&s)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (col + 32 * e >= dim) continue;
      W* out = static_cast<W*>(a.y) + (int64_t)k * a.y_stride + col + 32 * e;
      *out = from_f32<W>(a.accumulate ? to_f32(*out) + a.scale * s[e] : a.scale * s[e]);
    }
  };
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums are there
  const uint64_t few = (uint64_t)a.shared[0] * groups, many = (uint64_t)a.shared[1] * groups;
#pragma unroll 1
  for (uint64_t i = (uint64_t)blockIdx.x * kJoinWarps + warp; i < few; i += (uint64_t)gridDim.x * kJoinWarps) {
    const uint32_t first = a.shared[2 + i / groups], col = (uint32_t)(i % groups) * kJoinCols + lane;
    const uint32_t at = (first + 1 + lane) * piece;  // below 2^32: tokens is below 2^31
    float s[4];
    begin(first, col, s);
    const uint32_t k = pairs[(first + 1) * piece].x;
    // sorted: the pieces that begin with this word are the next ones
    const uint32_t n = __popc(__ballot_sync(0xffffffffu, at < tokens && pairs[at].x == k));
    add(first, 0, n, col, s);
    finish(k, col, s);
  }
#pragma unroll 1
  for (uint64_t i = blockIdx.x; i < many; i += gridDim.x) {
    const uint32_t first = a.shared[2 + pieces - 1 - i / groups], col = (uint32_t)(i % groups) * kJoinCols + lane;
    const uint32_t k = pairs[(first + 1) * piece].x;
    uint32_t n = 0, found;
    do {
      const uint64_t at = ((uint64_t)first + 1 + n + threadIdx.x) * piece;
      found = __syncthreads_count(at < tokens && pairs[at].x == k);
      n += found;
    } while (found == kJoinThreads);
    const uint32_t each = (n + kJoinWarps - 1) / kJoinWarps, from = min(n, warp * each);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (warp == 0) begin(first, col, s);
    add(first, from, min(n, from + each), col, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[warp][lane + 32 * e] = s[e];
    __syncthreads();
    if (warp == 0) {
#pragma unroll 1
      for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += sums[w][lane + 32 * e];
      finish(k, col, s);
    }
    __syncthreads();  // sums may be written again
  }
}

// Few tokens, in one launch.  The first `stretches` * tokens blocks: one for each place and stretch of
// columns; that of a word's first place adds its rows, kFewParts stretches of its places side by side and
// these in order, and writes the word's row.  The others write zeros over the rows of words that
// do not come.
template <class T, class W, int N, int kLoads>
__global__ void __launch_bounds__(kFewThreads) k_embed_few(const EmbedArgs a, int stretches) {
  constexpr int kApart = kSumThreads * N, kRows = kLoads == 1 ? 8 : 4;
  __shared__ uint32_t key[kFewTokens];
  __shared__ uint16_t match[kFewTokens];
  __shared__ uint32_t warp_count[kFewThreads / 32];
  __shared__ uint32_t noted[kFillRows / 32];
  __shared__ float sums[kFewParts - 1][kLoads][kSumThreads][N];
  const uint32_t tokens = (uint32_t)a.tokens, none = (uint32_t)a.vocab;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dim = (int)a.dim;
  if (threadIdx.x < tokens) key[threadIdx.x] = key_at(a, threadIdx.x);
  __syncthreads();
  if (blockIdx.x >= tokens * stretches) {  // zeros
    const int64_t block = blockIdx.x - tokens * stretches, blocks = gridDim.x - tokens * stretches;
    const int64_t each = (a.vocab + blocks - 1) / blocks, end = min(a.vocab, (block + 1) * each);
    constexpr int Z = 16 / (int)sizeof(W);
    const bool wide = a.dim % Z == 0 && a.y_stride % Z == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
    const uint32_t units = wide ? dim / Z : dim;
    for (int64_t r0 = block * each; r0 < end; r0 += kFillRows) {
      const uint32_t rows = (uint32_t)min((int64_t)kFillRows, end - r0);
      for (uint32_t i = threadIdx.x; i < (rows + 31) / 32; i += kFewThreads) noted[i] = 0;
      __syncthreads();
      if (threadIdx.x < tokens) {
        const int64_t r = (int64_t)key[threadIdx.x] - r0;
        if (r >= 0 && r < rows) atomicOr(&noted[r >> 5], 1u << (r & 31));
      }
      __syncthreads();
      uint32_t row = threadIdx.x / units, unit = threadIdx.x % units;
      const uint32_t row_step = kFewThreads / units, unit_step = kFewThreads % units;
      while (row < rows) {
        if (!(noted[row >> 5] >> (row & 31) & 1)) {
          W* to = static_cast<W*>(a.y) + (r0 + row) * a.y_stride;
          if (wide) reinterpret_cast<uint4*>(to)[unit] = make_uint4(0u, 0u, 0u, 0u);
          else to[unit] = from_f32<W>(0.f);
        }
        row += row_step, unit += unit_step;
        if (unit >= units) unit -= units, ++row;
      }
      __syncthreads();
    }
    return;
  }
  const uint32_t place = blockIdx.x / stretches, k = key[place];
  if (k >= none) return;
  // the word's places, in order; this block's is the first, or another block deals with the word
  const bool same = threadIdx.x < tokens && key[threadIdx.x] == k;
  const unsigned vote = __ballot_sync(0xffffffffu, same);
  if (lane == 0) warp_count[warp] = __popc(vote);
  if (__syncthreads_or(same && threadIdx.x < place)) return;
  uint32_t n = 0, before = 0;
  for (int w = 0; w < kFewThreads / 32; ++w) {
    if (w < warp) before += warp_count[w];
    n += warp_count[w];
  }
  if (same) match[before + __popc(vote & ((1u << lane) - 1))] = (uint16_t)threadIdx.x;
  __syncthreads();
  const int part = threadIdx.x / kSumThreads, tid = threadIdx.x % kSumThreads;
  const int c0 = (blockIdx.x % stretches) * kApart * kLoads + tid * N;
  const uint32_t each = (n + kFewParts - 1) / kFewParts, from = min(n, part * each), to = min(n, from + each);
  float sum[kLoads][N];
#pragma unroll
  for (int l = 0; l < kLoads; ++l)
#pragma unroll
    for (int e = 0; e < N; ++e) sum[l][e] = 0.f;
  for (uint32_t i0 = from; i0 < to; i0 += kRows) {
    typename Elems<T, N>::U v[kRows][kLoads];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const T* row = static_cast<const T*>(a.x) + (i0 + u < to ? match[i0 + u] : 0) * a.x_stride + c0;
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        v[u][l] = Elems<T, N>::zero();
        if (i0 + u < to && c0 + l * kApart < dim) v[u][l] = Elems<T, N>::raw(row + l * kApart);
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u)
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        float w[N];
        Elems<T, N>::widen(v[u][l], w);
#pragma unroll
        for (int e = 0; e < N; ++e) sum[l][e] += w[e];
      }
  }
  if (n > 1) {
    if (part > 0) {
#pragma unroll
      for (int l = 0; l < kLoads; ++l)
#pragma unroll
        for (int e = 0; e < N; ++e) sums[part - 1][l][tid][e] = sum[l][e];
    }
    __syncthreads();
  }
  if (part > 0) return;
#pragma unroll
  for (int l = 0; l < kLoads; ++l) {
    if (c0 + l * kApart >= dim) continue;
    if (n > 1)
      for (int p = 0; p < kFewParts - 1; ++p)
#pragma unroll
        for (int e = 0; e < N; ++e) sum[l][e] += sums[p][l][tid][e];
    W* out = static_cast<W*>(a.y) + (int64_t)k * a.y_stride + c0 + l * kApart;
    float old[N];
    if (a.accumulate) Elems<W, N>::load(out, old);
#pragma unroll
    for (int e = 0; e < N; ++e) sum[l][e] = a.accumulate ? old[e] + a.scale * sum[l][e] : a.scale * sum[l][e];
    Elems<W, N>::store(out, sum[l]);
  }
}

attn_status_t efail(attn_status_t s, const char* msg) {
  char buf[200];
  snprintf(buf, sizeof(buf), "embedding: %s", msg);
  set_last_error_text(buf);
  return s;
}

attn_status_t check_params(const attn_embedding_params_t* p, bool backward) {
  if (!p) return efail(ATTN_ERR_INVALID_ARG, "params is NULL");
  if ((p->dtype != ATTN_BF16 && p->dtype != ATTN_F32) ||
      (backward && p->w_dtype != ATTN_BF16 && p->w_dtype != ATTN_F32))
    return efail(ATTN_ERR_INVALID_ARG, "a dtype is not ATTN_F32 or ATTN_BF16");
  if (p->tokens < 0 || p->vocab < 0 || p->dim < 0) return efail(ATTN_ERR_INVALID_ARG, "a size is negative");
  const int64_t most = INT32_MAX;
  if (p->tokens >= most || p->vocab >= most || p->dim > kMaxDim)
    return efail(ATTN_ERR_UNSUPPORTED, "tokens or vocab of 2^31 - 1 or more, or dim above 2^20");
  if (p->x_stride < p->dim || p->w_stride < p->dim) return efail(ATTN_ERR_INVALID_ARG, "a row stride is below dim");
  if (!(p->scale - p->scale == 0.f)) return efail(ATTN_ERR_INVALID_ARG, "scale is not finite");
  return ATTN_OK;
}

// Whether rows `to`, which a call writes, share memory with the ids or with the rows `x` that it reads.
bool meets_inputs(const attn_embedding_params_t& p, const RowSpan& to, const RowSpan& x, const void* ids) {
  const int64_t bytes = p.tokens * (p.ids_64 ? 8 : 4);
  return rows_meet(to, x) || rows_meet(to, RowSpan{ids, 1, bytes, bytes});
}

// Sorted places of a block: as many as leave some 1000 blocks (2000, where accesses are narrower and a place costs
// more).  16384 tokens of [50000, 4096] bf16 take 105, 104 and 101 us with 16, 32 and 64; 20000 of [5000, 777] 32, 38 and
// 50.  By sizes and types alone, because the workspace's size follows it.
int piece_of(const attn_embedding_params_t* p) {
  const bool bf16 = p->dtype == ATTN_BF16, same = p->dtype == p->w_dtype;
  int64_t n = p->dim % 4 == 0 ? 4 : bf16 && same && p->dim % 2 == 0 ? 2 : 1;
  if (bf16 && same && p->dim % 8 == 0) n = 8;
  const int64_t bytes = n * (bf16 ? 2 : 4), cols = kSumThreads * n * (bytes >= 8 ? 1 : 4);
  const int64_t rows = p->tokens * ((p->dim + cols - 1) / cols), blocks = bytes == 16 ? 1000 : 2000;
  return rows >= 64 * blocks ? 64 : rows >= 32 * blocks ? 32 : 16;
}

struct Layout {
  size_t pairs[2], part, shared, total;
};

Layout layout_of(const attn_embedding_params_t* p) {
  Layout l{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t n = (size_t)p->tokens;
  for (int i = 0; i < 2; ++i) l.pairs[i] = take(8 * n);
  const size_t piece = piece_of(p), pieces = (n + piece - 1) / piece;
  l.part = take(pieces * 2 * (size_t)p->dim * 4);
  l.shared = take((2 + pieces) * 4);
  l.total = at;
  return l;
}

constexpr int kSms = 152;

// The steps of a fill by `blocks` blocks of `threads`.
void fill_steps(EmbedArgs* a, int64_t units, int64_t blocks, int threads) {
  a->row_step = (uint32_t)(blocks * threads / units), a->unit_step = (uint32_t)(blocks * threads % units);
}

template <class T, int N>
void launch_lookup(const EmbedArgs& a, cudaStream_t st) {
  int lanes_log = 0;
  while ((1 << lanes_log) < kThreads && ((int64_t)kAtOnce<T, N> << lanes_log) < a.dim / N) ++lanes_log;
  const int rows = kThreads >> lanes_log;
  k_embed<T, N><<<(unsigned)((a.tokens + rows - 1) / rows), kThreads, 0, st>>>(a, lanes_log);
}

template <class W, int N>
void launch_fill(EmbedArgs a, cudaStream_t st) {
  const int64_t units = a.dim / N;
  const int64_t blocks = std::min<int64_t>((a.vocab * units + kThreads - 1) / kThreads, kSms * 8);  // below 2^51
  fill_steps(&a, units, blocks, kThreads);
  k_embed_fill<W, N><<<(unsigned)blocks, kThreads, 0, st>>>(a);
}

// A kernel that may be set up while the one before it runs.
template <class K>
cudaError_t launch_after(K kernel, dim3 grid, int threads, const EmbedArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <class T, class W, int N>
cudaError_t launch_sums(const EmbedArgs& a, cudaStream_t st) {
  // narrow accesses: several a thread, which share the work of finding a word's end
  constexpr int kLoads = sizeof(T) * N >= 8 ? 1 : 4, kRows = kLoads == 1 ? 8 : 4;
  if (a.tokens <= kFewTokens) {
    const int stretches = (int)((a.dim + kSumThreads * N * kLoads - 1) / (kSumThreads * N * kLoads));
    // zeros: four vectors a thread at least
    const int64_t bytes = a.vocab * a.dim * (int64_t)sizeof(W);  // below 2^53
    const int64_t most = a.accumulate ? 0 : 4 * kSms;
    const int64_t filling = std::min<int64_t>((bytes + 64 * kFewThreads - 1) / (64 * kFewThreads), most);
    k_embed_few<T, W, N, kLoads><<<(unsigned)(a.tokens * stretches + filling), kFewThreads, 0, st>>>(a, stretches);
    return cudaGetLastError();
  }
  const unsigned pieces = (unsigned)((a.tokens + a.piece - 1) / a.piece);
  const unsigned stretches = (unsigned)((a.dim + kSumThreads * N * kLoads - 1) / (kSumThreads * N * kLoads));
  const cudaError_t e = launch_after(k_embed_sum<T, W, N, kLoads, kRows>, dim3(pieces, stretches), kSumThreads, a, st);
  if (e != cudaSuccess || pieces == 1) return e;
  // what there is to join only the device knows: at most a word in every second piece
  const int64_t warps = (int64_t)((pieces + 1) / 2) * ((a.dim + kJoinCols - 1) / kJoinCols);
  const unsigned blocks = (unsigned)std::min<int64_t>((warps + kJoinWarps - 1) / kJoinWarps, 4 * kSms);
  return launch_after(k_embed_join<W>, dim3(blocks), kJoinThreads, a, st);
}

template <class W, int N>
cudaError_t launch_sort(EmbedArgs a, cudaStream_t st) {
  int sorting = 1;
  while (sorting < kMaxCluster && (int64_t)sorting * kSortThreads < a.tokens) sorting *= 2;
  auto shared_bytes = [](int bits) { return kSortWarps * sizeof(uint32_t) * ((1u << bits) + 2 * kHeld * 32); };
  const size_t smem = shared_bytes(a.bits);
  cudaError_t e = cudaFuncSetAttribute(k_embed_sort<W, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)shared_bytes(kMaxBits));
  if (e != cudaSuccess) return e;
  int64_t filling = 0;  // blocks, in whole clusters
  if (!a.accumulate) {
    const int64_t units = a.dim / N;
    // many, because whole clusters do not fit on all SMs at once
    filling = std::min<int64_t>((a.vocab * units + 4 * kSortThreads - 1) / (4 * kSortThreads), 8 * kSms);
    filling = (filling + sorting - 1) / sorting * sorting;
    fill_steps(&a, units, filling, kSortThreads);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(sorting + filling));
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = sorting, cluster.val.clusterDim.y = 1, cluster.val.clusterDim.z = 1;
  cfg.attrs = &cluster;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_embed_sort<W, N>, a);
}

// launch(W{}, N) for the table's element type and its widest access.
template <class F>
cudaError_t for_table(bool bf16, int n, F launch) {
  using std::integral_constant;
  if (bf16) {
    if (n == 8) return launch(__nv_bfloat16(), integral_constant<int, 8>());
    if (n >= 2) return launch(__nv_bfloat16(), integral_constant<int, 2>());
    return launch(__nv_bfloat16(), integral_constant<int, 1>());
  }
  if (n == 4) return launch(float(), integral_constant<int, 4>());
  return launch(float(), integral_constant<int, 1>());
}

// Elements of one access: whole 16-byte vectors of the 2-byte type (8) or of the 4-byte type
// (4) where every address allows it, else pairs or single elements.
int width(uintptr_t at, int64_t dim, size_t small) {
  for (int n = small == 2 ? 8 : 4; n > 1; n /= 2)
    if ((at & (n * small - 1)) == 0 && dim % n == 0) return n;
  return 1;
}

}  // namespace
}  // namespace gbattn

using namespace gbattn;

extern "C" {

attn_status_t attn_embedding_fwd(const attn_embedding_params_t* p, const void* weight, const void* ids, void* y,
                                 void* stream) {
  attn_status_t s = check_params(p, false);
  if (s != ATTN_OK) return s;
  if (p->tokens == 0 || p->dim == 0) return ATTN_OK;
  const uintptr_t esize = p->dtype == ATTN_BF16 ? 2 : 4;
  if ((!weight && p->vocab > 0) || !ids || !y) return efail(ATTN_ERR_INVALID_ARG, "weight, ids or y is NULL");
  const uintptr_t at = reinterpret_cast<uintptr_t>(weight) | reinterpret_cast<uintptr_t>(y) |
                       (uintptr_t)p->x_stride * esize | (uintptr_t)p->w_stride * esize;
  if ((at & (esize - 1)) || (reinterpret_cast<uintptr_t>(ids) & (p->ids_64 ? 7u : 3u)))
    return efail(ATTN_ERR_INVALID_ARG, "a pointer is not aligned to its element size");
  EmbedArgs a{};
  int sms = 0;
  unsigned long long wait_ns = 0;
  if ((s = device_status(&a.status, &sms, &wait_ns))) return s;
  const int64_t width_y = p->dim * (int64_t)esize;
  if (meets_inputs(*p, RowSpan{y, p->tokens, p->x_stride * (int64_t)esize, width_y},
                   RowSpan{weight, p->vocab, p->w_stride * (int64_t)esize, width_y}, ids))
    return efail(ATTN_ERR_INVALID_ARG, "y overlaps weight or ids");
  a.ids = ids, a.x = weight, a.y = y;
  a.tokens = p->tokens, a.vocab = p->vocab, a.dim = p->dim;
  a.x_stride = p->w_stride, a.y_stride = p->x_stride;
  a.scale = p->scale, a.ids_64 = p->ids_64;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int n = width(at, p->dim, esize);
  if (p->dtype == ATTN_BF16) {
    if (n == 8) launch_lookup<__nv_bfloat16, 8>(a, st);
    else if (n >= 2) launch_lookup<__nv_bfloat16, 2>(a, st);
    else launch_lookup<__nv_bfloat16, 1>(a, st);
  } else {
    if (n == 4) launch_lookup<float, 4>(a, st);
    else launch_lookup<float, 1>(a, st);
  }
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : efail(ATTN_ERR_CUDA, "launch failed");
}

size_t attn_embedding_bwd_workspace_size(const attn_embedding_params_t* p) {
  if (check_params(p, true) != ATTN_OK) return SIZE_MAX;
  if (p->tokens <= kFewTokens || p->vocab == 0 || p->dim == 0) return 0;
  return layout_of(p).total;
}

attn_status_t attn_embedding_bwd(const attn_embedding_params_t* p, const void* dy, const void* ids, void* dweight,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  attn_status_t s = check_params(p, true);
  if (s != ATTN_OK) return s;
  if (p->vocab == 0 || p->dim == 0 || (p->tokens == 0 && p->accumulate)) return ATTN_OK;
  const uintptr_t esize = p->dtype == ATTN_BF16 ? 2 : 4, wsize = p->w_dtype == ATTN_BF16 ? 2 : 4;
  if (!dweight || (p->tokens > 0 && (!dy || !ids))) return efail(ATTN_ERR_INVALID_ARG, "dy, ids or dweight is NULL");
  const uintptr_t at_x = reinterpret_cast<uintptr_t>(dy) | (uintptr_t)p->x_stride * esize;
  const uintptr_t at_w = reinterpret_cast<uintptr_t>(dweight) | (uintptr_t)p->w_stride * wsize;
  if ((at_x & (esize - 1)) || (at_w & (wsize - 1)) || (reinterpret_cast<uintptr_t>(ids) & (p->ids_64 ? 7u : 3u)))
    return efail(ATTN_ERR_INVALID_ARG, "a pointer is not aligned to its element size");
  const size_t need = attn_embedding_bwd_workspace_size(p);
  if (need && !workspace) return efail(ATTN_ERR_WORKSPACE, "workspace is NULL");
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return efail(ATTN_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (workspace_bytes < need) return efail(ATTN_ERR_WORKSPACE, "workspace is too small");
  EmbedArgs a{};
  int sms = 0;
  unsigned long long wait_ns = 0;
  if ((s = device_status(&a.status, &sms, &wait_ns))) return s;
  const RowSpan dy_rows{dy, p->tokens, p->x_stride * (int64_t)esize, p->dim * (int64_t)esize};
  const RowSpan dw_rows{dweight, p->vocab, p->w_stride * (int64_t)wsize, p->dim * (int64_t)wsize};
  const RowSpan scratch{workspace, 1, (int64_t)need, (int64_t)need};
  if (meets_inputs(*p, dw_rows, dy_rows, ids)) return efail(ATTN_ERR_INVALID_ARG, "dweight overlaps dy or ids");
  if (meets_inputs(*p, scratch, dy_rows, ids) || rows_meet(scratch, dw_rows))
    return efail(ATTN_ERR_WORKSPACE, "workspace overlaps another argument");
  a.ids = ids, a.x = dy, a.y = dweight;
  a.tokens = p->tokens, a.vocab = p->vocab, a.dim = p->dim;
  a.x_stride = p->x_stride, a.y_stride = p->w_stride;
  a.scale = p->scale, a.ids_64 = p->ids_64, a.accumulate = p->accumulate != 0;
  a.padding = p->padding_id < 0 ? -1 : p->padding_id;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  const int n_w = width(at_w, p->dim, wsize);
  if (p->tokens == 0) {
    e = for_table(wsize == 2, n_w, [&](auto w, auto n) {
      launch_fill<decltype(w), decltype(n)::value>(a, st);
      return cudaGetLastError();
    });
  } else {
    if (p->tokens > kFewTokens) {
      const Layout l = layout_of(p);
      char* ws = static_cast<char*>(workspace);
      for (int i = 0; i < 2; ++i) a.pairs[i] = reinterpret_cast<uint2*>(ws + l.pairs[i]);
      a.piece = piece_of(p);
      a.part = reinterpret_cast<float*>(ws + l.part);
      a.shared = reinterpret_cast<uint32_t*>(ws + l.shared);
      int bits = 1;  // of the largest key, vocab
      while (p->vocab >> bits) ++bits;
      a.passes = (bits + kMaxBits - 1) / kMaxBits;
      a.bits = std::max((bits + a.passes - 1) / a.passes, 7);  // 128 counts: a vector a lane
      e = for_table(wsize == 2, n_w,
                    [&](auto w, auto n) { return launch_sort<decltype(w), decltype(n)::value>(a, st); });
      if (e != cudaSuccess) return efail(ATTN_ERR_CUDA, "sort launch failed");
    }
    // one width for dy's elements and the table's: both addresses have to allow it
    const int n = std::min(width(at_x, p->dim, esize), n_w);
    if (esize == 2 && wsize == 2) {
      if (n == 8) e = launch_sums<__nv_bfloat16, __nv_bfloat16, 8>(a, st);
      else if (n >= 2) e = launch_sums<__nv_bfloat16, __nv_bfloat16, 2>(a, st);
      else e = launch_sums<__nv_bfloat16, __nv_bfloat16, 1>(a, st);
    } else if (esize == 2) {
      e = n == 4 ? launch_sums<__nv_bfloat16, float, 4>(a, st) : launch_sums<__nv_bfloat16, float, 1>(a, st);
    } else if (wsize == 2) {
      e = n == 4 ? launch_sums<float, __nv_bfloat16, 4>(a, st) : launch_sums<float, __nv_bfloat16, 1>(a, st);
    } else {
      e = n == 4 ? launch_sums<float, float, 4>(a, st) : launch_sums<float, float, 1>(a, st);
    }
  }
  return e == cudaSuccess ? ATTN_OK : efail(ATTN_ERR_CUDA, "launch failed");
}

}  // extern "C"
