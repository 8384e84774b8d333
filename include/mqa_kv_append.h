/*
 * mqa_kv_append.h -- C ABI of libmqa_fp4.so (gfx950): what fills a paged
 * key-value cache. New queries and keys are normed and rotated by their
 * position; new keys and values go to their positions of the cache in 16, 8 or
 * 4 bits.
 *
 * Return codes, status bits, streams and devices are those of mqa_fp4_topk.h,
 * pages, tables and caches those of mqa_kv_cache.h and mqa_kv_fp4.h. All tensor
 * pointers are DEVICE pointers on one gfx950 device, owned by the caller. No
 * call needs a workspace, allocates or synchronises; every one accepts a
 * capturing stream.
 *
 * Norm. A head's D numbers x become x / sqrt(mean(x^2) + eps) * (weight +
 * weight_offset); the squares are added in 32 bits (numbers beyond 1e18 count
 * as infinite). Without a weight there is no norm.
 *
 * Rotation. Dims [rotary_offset, rotary_offset + rotary_dim) of a head turn in
 * pairs, pair i (below rotary_dim / 2) by the angle position * inv_freq[i],
 * which is taken in 64 bits:
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * Pair i is dims i and i + rotary_dim / 2 of the range, or with `interleaved`
 * 2 i and 2 i + 1. The norm comes first. Everything between the 16-bit inputs
 * and the one rounding at the end is held in 32 bits.
 */
#ifndef MQA_KV_APPEND_H
#define MQA_KV_APPEND_H

#include "mqa_kv_fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of new heads (host memory, read during the call only): x [num_rows,
 * num_heads, D] with a row stride (elements; a multiple of 16 bytes, num_heads *
 * D .. 2^32 unless num_rows <= 1), the heads of one row contiguous, so that a
 * slice of a fused projection's output fits; 16-byte aligned. */
typedef struct mqa_kv_rows {
  const void* x;
  int64_t row_stride;
  void* out;                /* where normed and rotated rows go: as x, with its own row stride; may be x itself with x's stride. Unused for appended keys and values */
  int64_t out_stride;
  const void* weight;       /* [D] of the rows' type, or NULL: no norm */
  float weight_offset;      /* added to every weight (finite) */
  int32_t num_heads;        /* 1 .. 65,536 */
} mqa_kv_rows;

/* The rotation, and what norms share. Without inv_freq only eps is looked at. */
typedef struct mqa_kv_turn {
  const float* inv_freq;    /* [rotary_dim / 2], or NULL: no rotation */
  const int32_t* position;  /* [num_rows] any number; NULL (appending only): the rows' positions in the cache */
  int32_t rotary_dim;       /* a multiple of 16, 16 .. D - rotary_offset */
  int32_t rotary_offset;    /* a multiple of 8 */
  int32_t interleaved;      /* 0 or 1 */
  float eps;                /* not negative, finite */
} mqa_kv_turn;

/*
 * Norms and rotates queries and, in the same launch, keys (k may be NULL):
 * out = rotate(norm(x)), of type (MQA_KV_BF16 or MQA_KV_FP16), D = head_dim
 * (64, 128 or 256). num_rows: 0 .. 2^24 - 256. Overlaps of an output with
 * anything but its own x in place are refused (MQA_ERR_OVERLAP).
 */
int32_t mqa_kv_norm_rotate(const mqa_kv_rows* q, const mqa_kv_rows* k, const mqa_kv_turn* turn, int64_t num_rows,
                           int32_t head_dim, int32_t type, void* stream);

/* The rows that a call appends. */
typedef struct mqa_kv_new {
  mqa_kv_rows k;                /* k.num_heads and v.num_heads: the cache's Hkv */
  mqa_kv_rows v;                /* v.x NULL: keys only. v is never normed or rotated */
  int64_t num_rows;             /* 0 .. 2^24 - 256 */
  int32_t type;                 /* MQA_KV_BF16 or MQA_KV_FP16 */
  const int32_t* block_table;   /* [num_seqs, max_pages] */
  int64_t num_seqs;
  int64_t max_pages;
  const int32_t* seq_of_row;    /* [num_rows] */
  const int32_t* position;      /* [num_rows] in the cache */
  mqa_kv_turn turn;
} mqa_kv_new;

/*
 * Appends keys and values: row r goes to position p = position[r] of sequence
 * s = seq_of_row[r], in physical page block_table[s * max_pages + p / 64], all
 * Hkv heads. Keys are normed (k.weight) and rotated (turn) on the way; queries q, if
 * any, are normed and rotated in the same launch. Nothing else of the cache's k and v is touched.
 *   the rows' type  rounded once to nearest even (values are copied bit by bit, and so are keys
 *                   without norm and rotation); k_scale and v_scale must be 1
 *   MQA_KV_E4M3     x / k_scale (v_scale), which must be positive, rounded to nearest even, saturating at 448; NaN
 *                   stays NaN
 * A row with position -1 is padding: it writes nothing to the cache and sets no status. A row
 * with a sequence outside [0, num_seqs) or a position outside [0, 64 *
 * max_pages) is not written (MQA_STATUS_BAD_WINDOW), nor is one whose page
 * maps outside [0, P_phys) (MQA_STATUS_BAD_PAGE). The queries of such rows are
 * turned all the same. Rows must go to distinct slots: of two that share one,
 * what it holds afterwards is unspecified (no access leaves the cache).
 * Overlaps of the queries' output are refused as above; the cache must lie apart
 * from every other tensor, which is not looked at.
 */
int32_t mqa_kv_append(const mqa_kv_new* rows, const mqa_kv_rows* q, const mqa_kv_cache* cache, void* stream);

/*
 * The same into a cache in 4 bits, by the rule of mqa_fp4_quantize: a block's
 * scale is 2^(floor(log2 of its largest magnitude) - 2), byte clamped to [0,
 * 254]; every number is divided by it and rounded to the nearest E2M1 number,
 * ties to the even code, saturating at 6; a block of zeros gets byte 0, one
 * with a NaN or an infinity byte 255 and zero codes. With one key head of 128
 * dims, keys only, these are the indexer's own pages.
 */
int32_t mqa_kv_append_fp4(const mqa_kv_new* rows, const mqa_kv_rows* q, const mqa_kv_cache_fp4* cache, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MQA_KV_APPEND_H */
