/*
 * mqa_kv_fp4.h -- C ABI of libmqa_fp4.so (gfx950): attention over a paged
 * key-value cache held in 4 bits.
 *
 * The cache is in the indexer's own number format (OCP MXFP4): E2M1 codes, two
 * to a byte with the even dim in the low half, and one UE8M0 byte for 32
 * neighbouring dims of a head; a number is code * 2^(byte - 127), and a scale
 * byte of 255 makes its 32 numbers NaN. mqa_kv_append_fp4 (mqa_kv_append.h)
 * writes such pages.
 *
 * Queries, tables, windows, lists, outputs, workspaces, failing rows, status
 * bits, streams and overlaps are those of mqa_kv_attention_decode and
 * mqa_kv_attention_selected in mqa_kv_cache.h, and so is the arithmetic. The
 * numbers are taken in the queries' type: exact in bfloat16 up to a scale byte
 * of 252, in float16 for scale bytes 104 to 140; beyond, those that float16
 * cannot hold become infinite, or are rounded to its subnormal numbers.
 */
#ifndef MQA_KV_FP4_H
#define MQA_KV_FP4_H

#include "mqa_kv_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A paged key-value cache in 4 bits (host memory, read during the call only).
 * Codes are tensors [P_phys, 64, Hkv, D / 2] and scales [P_phys, 64, Hkv, D / 32]
 * of bytes, given by a base and the strides in BYTES of page, position and head;
 * the bytes of one head are contiguous. Bases and strides of codes must be
 * multiples of 16, of scales of D / 32; strides not negative and below 2^36 (of
 * scales 2^32), and one page must span less than 2 GiB; the page stride of one page
 * and the head stride of one head are not looked at. A page that a window touches
 * is read in tiles of 32 positions; what it holds outside the window does not
 * matter. Nothing of other pages is read.
 * mqa_kv_compact moves such a cache as four arrays, one row of all heads to a position where
 * those are contiguous; with D = 64 the scales need an even Hkv for that (whole words). */
typedef struct mqa_kv_cache_fp4 {
  void* k;                        /* codes of keys and values (an attention only reads them) */
  void* v;
  void* k_scale;                  /* and their scales */
  void* v_scale;
  int64_t k_stride[3];            /* page, position, head, in bytes */
  int64_t v_stride[3];
  int64_t k_scale_stride[3];
  int64_t v_scale_stride[3];
  int64_t num_phys_pages;         /* P_phys >= 0, 64 * P_phys <= INT32_MAX */
  int32_t num_kv_heads;           /* Hkv >= 1 */
  int32_t head_dim;               /* D: 64, 128 or 256 */
} mqa_kv_cache_fp4;

/* mqa_kv_attention_decode over a cache in 4 bits (the same workspace:
 * mqa_kv_attention_decode_workspace_bytes). Its contents need not outlive the call,
 * but calls that may run at the same time (on two streams, or in two captured
 * graphs that are replayed side by side) need one each. */
int32_t mqa_kv_attention_decode_fp4(const mqa_kv_query* q, const mqa_kv_cache_fp4* cache, const int32_t* block_table,
                                    int64_t num_seqs, int64_t max_pages, const int32_t* seq_of_row,
                                    const int32_t* row_start, const int32_t* row_end, void* out, float* lse,
                                    void* workspace, int64_t workspace_bytes, void* stream);

/* mqa_kv_attention_selected over a cache in 4 bits (the same workspace:
 * mqa_kv_attention_selected_workspace_bytes). */
int32_t mqa_kv_attention_selected_fp4(const mqa_kv_query* q, const mqa_kv_cache_fp4* cache, const int32_t* slots,
                                      const int32_t* count, int64_t K, void* out, float* lse, void* workspace,
                                      int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MQA_KV_FP4_H */
