// How the attention over the 4-bit cache is shared out between blocks: the tiles of all
// sequences, KV heads and row tiles in one line, cut into equal stretches.  Used by
// both of its kernels.
#pragma once

#include <cuda_fp16.h>

#include "kv4.h"

namespace gbattn {
namespace {

constexpr int kSms = 152;  // a fixed count, so that the workspace size needs no device query

// The line of a kernel whose row tiles are kRows queries high, whose tiles are kKeys
// keys long and whose blocks have kWarps warps.  A row tile has kEmpty places before
// its keys' tiles: what it costs beside them (queries into operands, results joined),
// in tiles.  It has one tile at least, so that rows that see nothing are written too.
// With `causal` too all of a sequence's tiles are counted, seen or not: even shares while the new tokens
// are few beside the context (one of 512 in 8192 is 1.03 of the mean), up to twice the mean where they
// are all of it (a prompt of 4096 over itself 465 us, 459 without `causal`).
template <int kRows, int kKeys, int kEmpty, int kWarps>
struct Line {
  struct SeqWork {
    Kv4Seq s;
    int row_tiles, key_tiles;
    __device__ __forceinline__ int places() const { return key_tiles + kEmpty; }  // of a row tile
  };
  static __device__ __forceinline__ SeqWork seq_work(const Kv4Args& a, int b) {
    SeqWork w;
    w.s = kv4_seq(a, b);
    w.row_tiles = (int)(((long long)w.s.n * a.group + kRows - 1) / kRows);
    w.key_tiles = max(1, (w.s.len + (kKeys - 1)) / kKeys);
    return w;
  }
  static __device__ __forceinline__ long long places_of(const Kv4Args& a, int b) {
    const SeqWork w = seq_work(a, b);
    return (long long)a.heads_kv * w.row_tiles * w.places();
  }
  // The block whose stretch holds place x of `total` cut over n <= total blocks (block i:
  // i * total / n up to (i + 1) * total / n).
  static __device__ __forceinline__ int owner(long long x, long long total, long long n) {
    return (int)(((x + 1) * n - 1) / total);
  }

  // A row tile's keys as far as they lie in the stretch: tiles t0 .. t1 - 1.
  struct Piece {
    int b, h, r0, rows;  // rows: of the (sequence, KV head); the tile's first is r0
    int t0, t1;
    int klen, all_see;   // keys that any of the tile's rows sees, and that all of them see
    Kv4Seq s;
    bool whole;          // the stretch has all the row tile's keys
    long long last;      // the row tile's last place
  };
  int b;
  long long tile, tile_end, total, first, n;
  SeqWork w;

  // Block-wide.  False for a block without a stretch: there are as many stretches as
  // blocks, or places where those are fewer, and none is empty.
  __device__ __forceinline__ bool begin(const Kv4Args& a) {
    __shared__ long long warp_sums[kWarps];
    __shared__ long long found_first;
    __shared__ int found_seq;
    constexpr int kThreads = kWarps * 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto scan = [&](long long v, long long* sum) {  // inclusive prefix sums over the block
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      __syncthreads();
      if (lane == 31) warp_sums[warp] = v;
      __syncthreads();
      long long before = 0, all = 0;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        if (x < warp) before += warp_sums[x];
        all += warp_sums[x];
      }
      *sum = all;
      return v + before;
    };
    if (threadIdx.x == 0) found_seq = 0, found_first = 0;  // lengths that change under the kernel may hide the place
    total = 0;
    long long mine = 0, incl = 0, sum;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
      mine = b0 + (int)threadIdx.x < a.batch ? places_of(a, b0 + threadIdx.x) : 0;
      incl = scan(mine, &sum);
      total += sum;
    }
    n = min(total, (long long)gridDim.x);
    if (blockIdx.x >= n) return false;
    // 64-bit divisions only where the numbers need them: they take longer than the rest here
    const bool small = total < (1 << 22);  // kSms * 2 blocks at most
    tile = small ? (uint32_t)blockIdx.x * (uint32_t)total / (uint32_t)n : blockIdx.x * total / n;
    tile_end = small ? (uint32_t)(blockIdx.x + 1) * (uint32_t)total / (uint32_t)n : (blockIdx.x + 1) * total / n;
    long long before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
      const int x = b0 + threadIdx.x;
      if (a.batch > kThreads) {
        mine = x < a.batch ? places_of(a, x) : 0;
        incl = scan(mine, &sum) + before;
        before += sum;
      }
      if (x < a.batch && tile < incl && tile >= incl - mine) {
        found_seq = x;
        found_first = incl - mine;
      }
    }
    __syncthreads();
    b = found_seq;
    first = found_first;
    w = seq_work(a, b);
    return true;
  }

  // The next piece of the stretch; false at its end.
  __device__ __forceinline__ bool next(const Kv4Args& a, Piece* p) {
    if (tile >= tile_end) return false;
    while (tile - first >= (long long)a.heads_kv * w.row_tiles * w.places()) {
      if (b + 1 >= a.batch) return false;  // lengths that changed under the kernel
      first += (long long)a.heads_kv * w.row_tiles * w.places();
      w = seq_work(a, ++b);
    }
    const long long in = tile - first;
    const int in_seq = in < 0x7FFFFFFF ? (int)in / w.places() : (int)(in / w.places());  // (head, row tile)
    const int at = (int)(tile - first - (long long)in_seq * w.places());
    p->b = b;
    p->s = w.s;
    p->t0 = max(at - kEmpty, 0);
    p->t1 = (int)min((long long)w.key_tiles, at - kEmpty + (tile_end - tile));
    p->h = in_seq / w.row_tiles;
    p->r0 = (in_seq - p->h * w.row_tiles) * kRows;
    p->rows = w.s.n * a.group;
    p->whole = p->t0 == 0 && p->t1 == w.key_tiles;
    p->last = first + (long long)(in_seq + 1) * w.places() - 1;
    tile += w.places() - at;
    if (p->t1 <= 0) return false;  // the stretch ends before the row tile's keys
    const int low = w.s.len - w.s.n + div_by(p->r0, a.by_group);
    const int high = w.s.len - w.s.n + div_by(min(p->r0 + kRows, p->rows) - 1, a.by_group);
    p->klen = high < 0 ? 0 : a.causal ? high + 1 : w.s.len;
    p->all_see = low < 0 ? 0 : a.causal ? low + 1 : w.s.len;
    if (a.n_pages == 0 && p->klen > 0) {  // a cache without a page
      set_status(a.status, kStatusBounds);
      p->klen = 0;
    }
    return true;
  }
};

// Where a row tile's query rows lie: row r of the tile is query row r0 + r of the
// (sequence, KV head), token (r0 + r) / group, head h * group + (r0 + r) % group.
struct RowPlace {
  int token, head;
};
__device__ __forceinline__ RowPlace row_place(const Kv4Args& a, int h, int row) {
  RowPlace p;
  p.token = div_by(row, a.by_group);
  p.head = h * a.group + (row - p.token * a.group);
  return p;
}
__device__ __forceinline__ long long x_row(const Kv4Args& a, const Kv4Seq& s, int b, RowPlace p) {
  return (a.cu ? (s.row0 + p.token) * a.x_ss : b * a.x_sb + p.token * a.x_ss) + p.head * a.x_sh;
}
__device__ __forceinline__ long long y_row(const Kv4Args& a, const Kv4Seq& s, int b, RowPlace p) {
  return (a.cu ? (s.row0 + p.token) * a.y_ss : b * a.y_sb + p.token * a.y_ss) + p.head * a.y_sh;
}
__device__ __forceinline__ long long lse_row(const Kv4Args& a, const Kv4Seq& s, int b, RowPlace p) {
  return a.cu ? (long long)p.head * a.total + s.row0 + p.token
              : ((long long)b * a.heads_q + p.head) * a.seqlen + p.token;
}
// One row's log of the sum: m in log2 units.  A row that saw nothing has l = 0.
__device__ __forceinline__ float row_lse(float m, float l) {
  return l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127
__device__ __forceinline__ float half_lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)w)); }
__device__ __forceinline__ float half_hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }

constexpr int kNoRow = 0x7FFFFFFF;  // the limit of a column without a query: it masks nothing

// Where a stretch's partial results go.
struct AttnArgs {
  Kv4Args a;
  FastDiv page_div;
  float* part_o;   // [blocks][2][row tile's sums]
  float* part_ml;  // [blocks][2][rows][2]: row maximum (log2 units) and sum
  // [blocks]: the row tile whose keys begin in the block's stretch and end in block
  // w's: (sequence, KV head, row tile, w); w = -1: there is none
  int4* shared;
  unsigned long long wait_ns;  // limit of a wait on the device
};

}  // namespace
}  // namespace gbattn
