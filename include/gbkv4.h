/*
 * gbkv4.h - C ABI of the 4-bit key/value cache for GB300 (sm_103a): quantising
 * keys and values as they are written, reading them back, and attention over
 * the cache.
 *
 * The source pages stop at the forward and backward of whole sequences; their
 * closing section on precision (smzdm contest article) says why fewer bits pay:
 * every transfer carries more numbers while sums stay in a wider format.  A
 * model that answers token by token reads all its keys and values for each
 * token, so those bytes are its time.
 *
 * Format.  A row (one position of one KV head, head_dim values) is cut into
 * groups of 64 values.  With lo and hi the least and largest value of a group,
 *     s = bf16((hi - lo) / 15), stored as 0 if below 2^-126;   b = bf16(lo + 8 s);
 *     u = clamp(round((x - b) * (1 / s)) + 8, 0, 15)           (8 if s is 0),
 * every difference, sum, quotient and product rounded to float32 and round()
 * taking halves to the even number.  Code u stands for the value s (u - 8) + b.
 * Inputs must be finite, with hi - lo finite in float32; a group that breaks
 * this holds unspecified values, other groups are not touched by it.
 *
 * Memory of a cache of n_pages pages of page_size positions (contiguous):
 *     k_codes, v_codes  [n_pages, heads_kv, page_size, head_dim / 2] bytes;
 *     k_scale, v_scale  [n_pages, heads_kv, page_size, head_dim / 64, 2] bf16, (s, b).
 * A row's codes are 32-bit words [8][head_dim / 64]: word (i, g) holds the
 * values 8 i .. 8 i + 7 of group g, value 8 i + n in bits 4 n .. 4 n + 3.  The
 * groups alternate word by word so that one wide load of a lane brings words of
 * every group.
 *
 * Sequences.  Position p of sequence n is row p % page_size of page
 * block_table[n * table_stride + p / page_size].  lens[n] is the number of
 * positions sequence n holds, those that the call itself deals with included.
 * All three operators deal with each sequence's newest tokens: the t rows of
 * sequence n are its positions lens[n] - t .. lens[n] - 1.
 *     fixed length    t = seqlen for each sequence; a row whose position is
 *                     negative is padding;
 *     variable length (cu_seqlens != NULL) t = cu_seqlens[n + 1] - cu_seqlens[n],
 *                     rows of all sequences packed one after the other.
 * block_table, lens and cu_seqlens are device memory that the kernels read when
 * they run, so that a captured graph follows new lengths and page lists.
 *
 * Layouts of the tensors x (k of a write or read, q of the attention) and y (v,
 * o): rows of head_dim contiguous elements (dtype), [batch, heads, seqlen, head_dim]
 * by x_stride_b/h/s and y_stride_b/h/s, or [total_tokens, heads, head_dim] by
 * x_stride_s and x_stride_h when cu_seqlens is given (x_stride_b ignored).
 *
 * Constraints.  head_dim 64, 128 or 256; page_size a positive multiple of 16;
 * heads_q % heads_kv == 0; x and y and the code arrays 16-byte aligned, scale
 * arrays 16-byte aligned too; strides multiples of 16 bytes, not negative; rows of an
 * output must not overlap (refused where one stride alone makes them: one below head_dim over
 * more than one entry); fewer than 2^31 rows over all heads in one call, packed ones counted
 * as they are (a packed write or read: and batch * ceil(seqlen / 16) * heads_kv below 2^31).
 * Offsets into the cache are 64-bit.  The attention takes up to 2^30 query rows over all heads,
 * up to 2^30 positions in a page list
 * and fewer than 2^32 rows (n_pages * heads_kv * page_size) in the cache.
 *
 * Errors and asynchrony are as for gbattn.h.  What only the device knows is
 * checked there, in every build: a page outside [0, n_pages), a length below 0 or
 * above max_pages * page_size, or a packed row outside the tensor is recorded as
 * ATTN_ERR_DEVICE_BOUNDS (attn_get_status()) and nothing of it is read or
 * written: a write skips the row, a read gives zeros, the attention leaves the
 * page's positions out; a length is cut to the range.
 */
#ifndef GBKV4_H
#define GBKV4_H

#include <stddef.h>
#include <stdint.h>

#include "gbattn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t batch;      /* sequences */
  int32_t heads_q;    /* attention only: query heads; query head h reads KV head h / (heads_q / heads_kv) */
  int32_t heads_kv;
  int32_t head_dim;
  int32_t page_size;
  int32_t n_pages;    /* pages of the cache */
  int32_t max_pages;  /* entries of one block_table row */
  int32_t seqlen;     /* fixed length: rows of each sequence; variable: at least the most of any */
  const int32_t* block_table;     /* device, [batch] rows of max_pages, table_stride apart */
  int64_t table_stride;
  const int32_t* lens;            /* device, [batch] */
  const int32_t* cu_seqlens;      /* device [batch + 1] row starts, or NULL */
  const int32_t* cu_seqlens_host; /* host copy, required when cu_seqlens != NULL */
  int64_t x_stride_b, x_stride_h, x_stride_s; /* k or q (elements) */
  int64_t y_stride_b, y_stride_h, y_stride_s; /* v or o (elements) */
  float scale;        /* attention: score scale, usually 1/sqrt(head_dim) */
  attn_dtype_t dtype; /* element type of x and y */
  int32_t causal;     /* attention: 1: a row sees the positions up to its own; 0: all lens[n] */
} attn_kv4_params_t;

/*
 * Quantises the newest tokens' keys x and values y and stores them in the cache.
 * Rows of padding are skipped; no other position is touched.  Pages that two
 * sequences share must not be written through both: positions that two rows of
 * one call name hold either row's groups.  Bound by device-memory bandwidth: 2
 * (bf16) bytes in and 9/16 out per value.
 */
attn_status_t attn_kv4_write(const attn_kv4_params_t* p, const void* x, const void* y, void* k_codes, void* k_scale,
                             void* v_codes, void* v_scale, void* stream);

/*
 * Reads the newest tokens' keys and values back: x and y get s (u - 8) + b,
 * rounded once to dtype.  Rows of padding get zeros; no other memory is touched.
 */
attn_status_t attn_kv4_read(const attn_kv4_params_t* p, const void* k_codes, const void* k_scale, const void* v_codes,
                            const void* v_scale, void* x, void* y, void* stream);

/*
 * Attention of the newest tokens' queries x over the cache.  With k_j and v_j
 * the values the cache stands for (never rounded to fewer bits as a whole row)
 * and the row of position i of sequence n,
 *     s_ij = scale <q_i, k_j> for j < lens[n] and, with causal, j <= i;
 *     LSE_i = ln sum_j exp(s_ij);   O_i = sum_j exp(s_ij - LSE_i) v_j.
 * A row that sees nothing (padding, an empty sequence) gets O = 0 and LSE = -inf.  A cached group
 * that is not finite reaches the rows that see its position and no other.
 * Sums are float32.  Roundings to fewer bits, beside that of O:
 *   float32 rows  none but at the far end: queries to 2^-30 of a row's largest element, the weights
 *     p_j s_j (p_j = exp(s_ij - LSE_i), s_j a group's step) to 2^-41 of the row's largest;
 *   bf16 rows     the weights p_j s_j, to 11 bits, or to 2^-29 of the row's largest where that is
 *     more; query elements 2^26 times smaller than a row's largest lose bits.
 * bf16 calls with head_dim 64 or 128 and more than 24 query rows on a KV head (seqlen * heads_q /
 * heads_kv) round the weights p_j instead, to 11 bits, or to 2^-32 of the row's largest, and hold the
 * cache's values of 128 keys (V: of all keys so far) in units of the largest step and offset among
 * them: steps that are 2^25 times smaller than the largest step, or than the largest offset 2^22 (keys)
 * or 2^28 (values) times, lose bits.
 * Cached values beyond 2^96 in size may overflow the sums.
 * y: O; lse: contiguous float32 [batch, heads_q, seqlen], packed [heads_q,
 * total_tokens].  The result is bit-identical from run to run.  workspace: device
 * scratch, 256-byte aligned, >= attn_kv4_workspace_size(p) bytes (SIZE_MAX if the
 * parameters are invalid); it keeps nothing from one call to the next, and calls
 * that may overlap need one each.
 */
size_t attn_kv4_workspace_size(const attn_kv4_params_t* p);
attn_status_t attn_fwd_kv4(const attn_kv4_params_t* p, const void* x, const void* k_codes, const void* k_scale,
                           const void* v_codes, const void* v_scale, void* y, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GBKV4_H */
