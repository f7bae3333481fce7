/*
 * gbembed.h - embedding table for GB300 (sm_103a): lookup with scaling, and the
 * table's gradient by sorted tokens.  C ABI.
 *
 * The source pages begin after the embedding; a model that trains on attn_fwd and
 * attn_bwd takes the first rows of its residual stream from such a table, and
 * gives its last gradient back to it.
 *
 *     y_i = scale W[id_i];      dW[v] = scale sum over i with id_i = v of dy_i.
 *
 * Layout.  W is [vocab, dim], its row v at weight + v * w_stride (elements); y and dy
 * are [tokens, dim] with rows x_stride apart; dim is contiguous.  ids: device, [tokens],
 * int32 or int64.  Rows move as 16-byte vectors where every pointer is 16-byte
 * aligned and every stride and dim whole vectors, else as 4-byte words or elements.
 *
 * Constraints.  tokens and vocab below 2^31 - 1, dim at most 2^20; strides >= dim; scale
 * finite; pointers aligned to their elements; outputs and workspace must not overlap inputs or
 * one another (refused; rows that lie between another tensor's rows do not overlap).  Offsets
 * are 64-bit.  Errors and asynchrony are as for gbattn.h.  An id outside [0, vocab) is
 * recorded as ATTN_ERR_DEVICE_BOUNDS (attn_get_status()) and nothing is read or written
 * for it: its row of y is 0, and no row of dW gets its dy.  Where nothing is to be written (dim 0, dW of
 * vocab 0) no id is looked at.
 */
#ifndef GBEMBED_H
#define GBEMBED_H

#include <stddef.h>
#include <stdint.h>

#include "gbattn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t tokens, vocab, dim;
  int64_t x_stride;     /* y or dy: elements between tokens */
  int64_t w_stride;     /* weight or dweight: elements between rows of the table */
  float scale;
  attn_dtype_t dtype;   /* element type of weight and y; of dy */
  attn_dtype_t w_dtype; /* element type of dweight (backward only) */
  int32_t ids_64;       /* 1: ids are int64; 0: int32 */
  int32_t accumulate;   /* backward: 1: dweight += the gradient; 0: dweight = the gradient */
  int64_t padding_id;   /* backward: a token that gives no gradient; negative: none */
} attn_embedding_params_t;

/* y_i = scale W[id_i], in float32 and rounded once. */
attn_status_t attn_embedding_fwd(const attn_embedding_params_t* p, const void* weight, const void* ids, void* y,
                                 void* stream);

/*
 * dweight of the lookup.  Without accumulate every row is written, 0 where no token
 * names it; with it only rows that a token names are read and written, one rounding
 * per call.  A row's tokens are added in float32 in a fixed order that ids, sizes and types
 * decide: the result is bit-identical from run to run.  workspace: device scratch, 256-byte
 * aligned, >= attn_embedding_bwd_workspace_size(p) bytes (SIZE_MAX if the parameters
 * are invalid; 0 for few tokens); it keeps nothing from one call to the next, and calls that
 * may overlap need one each.
 */
size_t attn_embedding_bwd_workspace_size(const attn_embedding_params_t* p);
attn_status_t attn_embedding_bwd(const attn_embedding_params_t* p, const void* dy, const void* ids, void* dweight,
                                 void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GBEMBED_H */
