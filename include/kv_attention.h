/*
 * Operators over a page-major KV-cache pool (kv_pool.h): append with position
 * rotation, attention of new tokens over the pages, and a gather that applies
 * the scales of an 8-bit pool.
 *
 * Batch. A kv_batch names this step's tokens: sequence s holds seq_len[s]
 * tokens through its row of the block table, and tokens j in
 * [seq_start[s], seq_len[s]) are the step's, row cu[s] + j - seq_start[s] of
 * every [n_rows, heads, dim] tensor. It is the gather's metadata
 * (kv_gather_layer), so one batch serves append, attention and gather.
 * Rows of no token (cu spans longer than the tokens) are not written; they
 * may be read (append copies rows while it looks up whose they are), and
 * their contents do not matter. A sequence whose metadata is inconsistent (seq_start < 0,
 * seq_len > max_pages * page_size, a cu span that is negative, shorter than
 * its tokens, or outside [0, n_rows]) takes no part and sets
 * KV_DEV_ERR_TABLE (a batch of no rows is not looked at). Page 0 is the pool's sink and holds no tokens: a
 * table entry that is negative or names page 0 is a tombstone, whose tokens
 * are not stored, not visible to attention, and gathered as zeros. An entry
 * past the pool sets KV_DEV_ERR_ROW, one off the kernel-facing grid
 * KV_DEV_ERR_FORM; both then count as tombstones.
 *
 * 8-bit pools. In a pool of itemsize 1 these calls hold e4m3 codes with one
 * float scale for each page, layer, K or V, and head, in the caller's buffer
 * scales[num_pages][L][2][H] (kv_scale_bytes): value = code * scale. Calls
 * that move bytes (kv_move, kv_store_layer) do not know of scales: move
 * whole pages together with their scales, or append anew.
 *
 * Like the calls of kv_pool.h these are asynchronous on the stream, allocate
 * nothing, capture into CUDA graphs, need the pool's device current and
 * report data errors in the pool's error word. MLA pools are refused
 * (KV_ERR_INVALID). Calls that overlap on the GPU must not append to the
 * same page, nor append to a page that another reads.
 */
#ifndef GATHER_TRANSLATE_KV_GB300_KV_ATTENTION_H
#define GATHER_TRANSLATE_KV_GB300_KV_ATTENTION_H

#include "kv_pool.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the tensors beside the pool. */
enum { KV_TYPE_BF16 = 1, KV_TYPE_F16 = 2, KV_TYPE_F32 = 3 };

/* A further bit of the device error word (kv_pool_last_error). */
#define KV_DEV_ERR_POSITION 32 /* append: a position outside the rotation's table; the row's rotated
                                  heads (queries and keys) and its value are not written */

typedef struct {
  const int32_t* table_dev;     /* [n_seqs, max_pages] physical pages, or kernel-facing entries phys * 2L */
  const int32_t* seq_start_dev; /* [n_seqs] first of this step's tokens, or NULL for 0 */
  const int32_t* seq_len_dev;   /* [n_seqs] one past the last token */
  const int64_t* cu_dev;        /* [n_seqs + 1] first row of each sequence, non-decreasing */
  int64_t n_rows;               /* rows of the tensors; cu[n_seqs] <= n_rows */
  int32_t n_seqs;
  int32_t max_pages;            /* n_seqs * max_pages < 2^31, max_pages * page_size < 2^31 */
  int32_t kernel_facing;        /* 1: the table of kv_translate_block_table */
  int32_t reserved;             /* must be 0 */
} kv_batch;

/* Position rotation. Pair f of a head's first rotary_dim elements turns by
 * the angle whose cosine and sine are cos_sin[p][f] and
 * cos_sin[p][rotary_dim / 2 + f], (x1, x2) -> (x1 c - x2 s, x2 c + x1 s) in
 * 32 bits without fused products, rounded once; p is the token's position on
 * the axis that pair f belongs to. The first axis_pairs[0] pairs belong to
 * axis 0, the next axis_pairs[1] to axis 1, and so on (time, height and width
 * of image and video tokens, for example). */
typedef struct {
  const float* cos_sin_dev;     /* [n_positions, rotary_dim] */
  const int32_t* positions_dev; /* [n_axes, n_rows], or NULL: a token's index in its sequence on every axis */
  int64_t n_positions;
  int32_t rotary_dim;           /* even, 0 <= rotary_dim <= head_dim */
  int32_t interleaved;          /* 0: pair f is elements f and f + rotary_dim / 2; 1: 2f and 2f + 1 */
  int32_t n_axes;               /* 1 to 4 */
  int32_t axis_pairs[4];        /* sum over the axes: rotary_dim / 2 */
  int32_t reserved;             /* must be 0 */
} kv_rotary;

/* Size in bytes of an 8-bit pool's scale buffer, 4 * num_pages * L * 2 * H
 * (host only; KV_ERR_INVALID for other pools). */
int kv_scale_bytes(const kv_pool_t* pool, int64_t* bytes);

/* Append one layer's new keys and values through the block table, keys
 * rotated on the way, and write the rotated queries (in one launch; two that
 * overlap for an 8-bit pool with queries).
 *  type      KV_TYPE_* of k, v, q and q_out. A pool of itemsize 2 or 4 stores
 *            that type (itemsize 2: BF16 or F16; 4: F32); an 8-bit pool
 *            takes any of the three.
 *  k_dev, v_dev, q_dev  rows of [H, D] ([q_heads, D]) contiguous elements,
 *            *_stride elements from row to row (a fused projection's slices
 *            can be passed as they are), aligned to their elements; loads are
 *            widest when rows start on 16 bytes and D and rotary_dim are
 *            multiples of 16.
 *  q_dev may be NULL (q_heads = 0); q_out_dev is [n_rows, q_heads, D]
 *            contiguous and may be q_dev itself when that is contiguous too.
 *  rotary    NULL: nothing is rotated.
 *  scales_dev  8-bit pools only (else NULL). For each (page, head), K and V
 *            apart, with new tokens of the call: base is the page's scale if
 *            it holds earlier tokens of the sequence, else 0 (0 too when it
 *            is not finite and positive); amax the largest finite magnitude
 *            of the new values; the new scale S = max(base, 2^e), e the least
 *            integer >= -60 with amax <= 448 * 2^e. Earlier tokens' codes
 *            become rne(code * (base / S)), new ones rne(x * (1 / S)); a
 *            value that is not finite becomes the NaN code. With power-of-two
 *            scales the earlier codes lose nothing but subnormal bits.
 * Pages are a sequence's own: two sequences of one batch that append to the
 * same page race (bytes and scale unspecified, nothing out of bounds). */
int kv_append_layer(const kv_pool_t* pool, int32_t layer, const kv_batch* batch, int32_t type, const void* k_dev,
                    int64_t k_stride, const void* v_dev, int64_t v_stride, const kv_rotary* rotary, const void* q_dev,
                    int64_t q_stride, int32_t q_heads, void* q_out_dev, float* scales_dev, kv_stream_t stream);

/* Attention of the batch's rows over one layer's cache. Row r of sequence s,
 * the token at position i = seq_start[s] + r - cu[s], sees the tokens
 *   j <= i  with  window == 0, or i - j < window, or j < sinks
 * that are not tombstones (its own token among them: append first), and query head h reads
 * KV head h / (q_heads / H):
 *   out[r][h] = sum_j softmax_j(scale * q[r][h] . k_j) v_j,
 *   lse[r][h] = log sum_j exp(scale * q[r][h] . k_j).
 * A row that sees nothing gives 0 and -infinity. What a row does not see
 * does not change it, infinities and NaN included. Pages that no row of the
 * batch sees are not read.
 *  type      KV_TYPE_BF16 or KV_TYPE_F16 of q and out; a 16-bit pool holds
 *            the same type, an 8-bit pool takes either.
 *  q_dev     rows of [q_heads, D], q_stride elements from row to row
 *  out_dev   [n_rows, q_heads, D] contiguous, apart from q_dev (rows may be done again from q)
 *  lse_dev   [n_rows, q_heads] float, or NULL
 *  scales_dev  the 8-bit pool's scales (positive; any value, not only powers of two), else NULL
 *  workspace_dev  kv_attend_workspace_bytes() bytes, 16-byte aligned, contents
 *            arbitrary; calls that overlap on the GPU need one each (its size goes by the
 *            device and head_dim alone: 81 MB for 128 on 152 SMs)
 * Should a wait inside the kernel for many rows a sequence run out (about a second; not
 * expected on a healthy GPU), the call sets KV_DEV_ERR_TIMEOUT, ends, and leaves the rows
 * of sequences with many new tokens unspecified.
 * Sums, maxima and the softmax statistics are held in 32 bits. head_dim is
 * at most 256; 64 and 128 run on the tensor cores. */
int kv_attend_workspace_bytes(const kv_pool_t* pool, int32_t q_heads, int32_t n_seqs, int64_t n_rows,
                              int64_t* bytes);
int kv_attend_layer(const kv_pool_t* pool, int32_t layer, const kv_batch* batch, int32_t type, const void* q_dev,
                    int64_t q_stride, int32_t q_heads, void* out_dev, float* lse_dev, float scale, int32_t window,
                    int32_t sinks, const float* scales_dev, void* workspace_dev, int64_t workspace_bytes,
                    kv_stream_t stream);

/* Gather of an 8-bit pool's values: out[row] = code * scale of the batch's
 * tokens, one layer's K and V as [n_rows, H, D] of `type` (rounded to nearest
 * even; BF16 holds every product with a power-of-two scale exactly, up to its
 * range), 16-byte aligned. */
int kv_gather_layer_scaled(const kv_pool_t* pool, int32_t layer, const kv_batch* batch, const float* scales_dev,
                           int32_t type, void* out_k_dev, void* out_v_dev, kv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GATHER_TRANSLATE_KV_GB300_KV_ATTENTION_H */
