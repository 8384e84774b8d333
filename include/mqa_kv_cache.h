/*
 * mqa_kv_cache.h -- C ABI of the key-value cache operators of libmqa_fp4.so
 * (gfx950): attention of new tokens over a paged key-value cache, attention
 * over the slots that the FP4 indexer selected, and eviction from that cache
 * by accumulated attention weight.
 *
 * The cache is paged like the indexer's own (pages of 64 positions, int32
 * tables of physical pages), and the operators share its conventions: return
 * codes, per-row failure, sticky status bits (mqa_fp4_status), streams and
 * devices are those of mqa_fp4_topk.h, with the additions below. All tensor
 * pointers are DEVICE pointers on one gfx950 device, owned by the caller.
 * Every call allocates nothing, never synchronises and accepts a capturing
 * stream. Two calls that share a workspace or an output must be ordered (one
 * stream, or replays of graphs that do not overlap); a workspace needs no
 * initialisation and holds nothing from one call to the next.
 *
 * Outputs and workspaces must not overlap each other or anything that the call
 * reads. Two may take an input's place: an attention's out its queries' (where
 * those lie contiguous), and an eviction's kept the lengths. Overlaps with
 * tensors other than caches and paged arrays are refused with MQA_ERR_OVERLAP.
 *
 * The cache. Keys and values are tensors [P_phys, 64, Hkv, D] given by a base
 * pointer and the strides, in ELEMENTS, of page, position and head; the D
 * elements of one head are contiguous. So [P, 64, Hkv, D] and [P, Hkv, 64, D]
 * memory, or keys and values interleaved in one pool, all fit. Bases and
 * strides must be multiples of 16 bytes, strides not negative and below 2^35
 * elements, and one page must span less than 2 GiB; the page stride of one page and the
 * head stride of one head are not looked at. Everything behind a page, position or head that
 * a call does not address is never read.
 *
 * Types. MQA_KV_BF16 and MQA_KV_FP16 caches go with queries and outputs of the
 * same type; an MQA_KV_E4M3 cache (OCP e4m3, largest value 448) with either.
 * An 8-bit cache holds keys and values divided by one scale each: k_scale and
 * v_scale (1 for the other types, or any finite number) multiply them back.
 *
 * Heads. H query heads share Hkv key heads, H a multiple of Hkv: query head h
 * reads key head h / (H / Hkv). D is 64, 128 or 256.
 *
 * Arithmetic. Products of the query with the keys, the scores, the softmax's
 * maximum and sum and the weighted sums of the values are held in 32 bits; the
 * weights are rounded to the query's type before they multiply the values, and
 * the output is rounded once. Up to 16 heads per key head the largest weight is a
 * power of two, which that rounding leaves alone; with more heads the running maximum
 * follows the scores by up to 2^8, and the largest weight is rounded as the others
 * are, by half a step of the type. The order of the sums depends on the sizes and,
 * for the decode form, on the windows of the whole batch, and on nothing else:
 * the same call gives the same bits.
 */
#ifndef MQA_KV_CACHE_H
#define MQA_KV_CACHE_H

#include "mqa_fp4_topk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MQA_KV_BF16 0
#define MQA_KV_FP16 1
#define MQA_KV_E4M3 2

/* A paged key-value cache (host memory, read during the call only). */
typedef struct mqa_kv_cache {
  const void* k;            /* keys; values (v and its strides may be 0 where a call reads keys only) */
  const void* v;
  int64_t k_stride[3];      /* page, position, head, in elements */
  int64_t v_stride[3];
  int64_t num_phys_pages;   /* P_phys >= 0, 64 * P_phys <= INT32_MAX */
  int32_t num_kv_heads;     /* Hkv >= 1 */
  int32_t head_dim;         /* D: 64, 128 or 256 */
  int32_t type;             /* MQA_KV_* */
  float k_scale;
  float v_scale;
} mqa_kv_cache;

/* The queries: [num_rows, H, D] with a row stride (elements; a multiple of 16
 * bytes, H * D .. 2^32 unless num_rows <= 1), the heads of one row contiguous, so that a
 * slice of a fused projection's output fits. 16-byte aligned. */
typedef struct mqa_kv_query {
  const void* q;
  int64_t row_stride;
  int64_t num_rows;         /* num_rows * H <= 2^24 - 256 */
  int32_t num_heads;        /* H, 1 .. 65,536 */
  int32_t type;             /* MQA_KV_BF16 or MQA_KV_FP16 */
  float scale;              /* multiplies every product of a query and a key (finite) */
} mqa_kv_query;

/*
 * Attention of new tokens over a paged cache. Row r of the queries belongs to
 * sequence seq_of_row[r] and attends to that sequence's positions
 * [row_start[r], row_end[r]), position p in physical page
 * block_table[seq * max_pages + p / 64]:
 *   s_p = scale * k_scale * q . k_p,   lse = log sum_p exp(s_p),
 *   out = sum_p exp(s_p - lse) * v_scale * v_p
 *   out  [num_rows, H, D] of the queries' type, contiguous, 16-byte aligned
 *   lse  float [num_rows, H], optional (NULL)
 *   block_table, seq_of_row, row_start, row_end: as in mqa_fp4_topk_decode
 * A row whose window is empty gets out = 0 and lse = -infinity. A row with a
 * sequence outside [0, num_seqs) or a window outside [0, 64 * max_pages) or
 * end < start, and one whose window touches a page that maps outside [0,
 * P_phys), fails closed: out and lse are NaN and MQA_STATUS_BAD_WINDOW or
 * MQA_STATUS_BAD_PAGE is set. Nothing outside the windows is read, so NaN or
 * infinities there do not matter; inside they take part by IEEE rules: a NaN or
 * +infinite score, or nothing but -infinite ones, make that head's out NaN; a
 * -infinite score beside others drops out.
 * workspace: mqa_kv_attention_decode_workspace_bytes() bytes, 256-byte aligned.
 * The work is cut into equal shares over the whole batch's pages, whatever the
 * lengths are, so max_pages may be any capacity.
 */
int32_t mqa_kv_attention_decode(const mqa_kv_query* q, const mqa_kv_cache* cache, const int32_t* block_table,
                                int64_t num_seqs, int64_t max_pages, const int32_t* seq_of_row,
                                const int32_t* row_start, const int32_t* row_end, void* out, float* lse,
                                void* workspace, int64_t workspace_bytes, void* stream);
int64_t mqa_kv_attention_decode_workspace_bytes(int64_t num_rows, int32_t num_heads, int32_t num_kv_heads,
                                                int32_t head_dim);

/*
 * Attention over a list of cache slots per row: the consumer of the indexer's
 * out_slot and out_count, for decode rows and prefill chunks alike. Row r
 * attends to slots[r * K .. r * K + count[r]), slot = page * 64 + position in
 * the page; every key head reads the same slots. A slot listed twice counts
 * twice. Formulas, out and lse as above.
 *   slots  int32 [num_rows, K], 0 <= K <= INT32_MAX; entries from count[r] on
 *          are not read
 *   count  int32 [num_rows]
 * count 0 gives out = 0 and lse = -infinity. A negative count (a row that the
 * indexer failed closed), a count above K (sets MQA_STATUS_BAD_WINDOW) and a
 * slot outside [0, 64 * P_phys) (sets MQA_STATUS_BAD_PAGE) give NaN.
 * workspace: mqa_kv_attention_selected_workspace_bytes() bytes (may be 0, and
 * the workspace then NULL), 256-byte aligned.
 */
int32_t mqa_kv_attention_selected(const mqa_kv_query* q, const mqa_kv_cache* cache, const int32_t* slots,
                                  const int32_t* count, int64_t K, void* out, float* lse, void* workspace,
                                  int64_t workspace_bytes, void* stream);
int64_t mqa_kv_attention_selected_workspace_bytes(int64_t num_rows, int64_t K, int32_t num_heads,
                                                  int32_t num_kv_heads, int32_t head_dim);

/*
 * Accumulated attention weight, the measure that eviction goes by:
 *   acc[seq, p] += sum over the sequence's rows r whose window holds p, and all heads h, of
 *                  exp(scale * k_scale * q[r, h] . k_p - lse[r, h])
 * with lse as the attention above returned it for the same rows (rows may also
 * be a whole prompt's). A position's keys are read once for every row whose window
 * holds it and every 64 query heads of a key head (32 where D = 256). The order of the
 * additions is fixed (by rows within a key head), without atomics: the same call gives the same
 * bits. Positions outside every window keep their bits. A head whose lse is not finite
 * (an empty or failed row) adds nothing, nor does a row with a bad sequence or
 * window (MQA_STATUS_BAD_WINDOW) or a position whose page maps outside
 * [0, P_phys) (MQA_STATUS_BAD_PAGE).
 *   acc  float [num_seqs, acc_stride], in logical positions; 64 * max_pages <= acc_stride
 */
int32_t mqa_kv_weights_accumulate(const mqa_kv_query* q, const float* lse, const mqa_kv_cache* cache,
                                  const int32_t* block_table, int64_t num_seqs, int64_t max_pages,
                                  const int32_t* seq_of_row, const int32_t* row_start, const int32_t* row_end,
                                  float* acc, int64_t acc_stride, void* stream);

/*
 * Chooses what a budget keeps. Of sequence s's positions [0, seq_len[s]) the
 * last `recent` are kept and, of those before them, the budget - recent with
 * the largest acc, in the indexer's total order (value descending, position
 * ascending; NaN below every number, +0 above -0); all of them where seq_len
 * <= budget.
 *   acc      float [num_seqs, acc_stride]
 *   seq_len  int32 [num_seqs]; one outside [0, max_len] fails closed: keep all
 *            -1, kept -1, kept_acc 0, MQA_STATUS_BAD_WINDOW
 *   max_len  at most acc_stride and INT32_MAX - 512
 *   budget   0 .. INT32_MAX;  0 <= recent <= budget
 *   keep     int32 [num_seqs, budget]   kept positions, rising, padded with -1
 *   kept     int32 [num_seqs]           how many
 *   kept_acc float [num_seqs, budget]   optional: their acc, padded with 0. To go on after mqa_kv_compact,
 *            the caller copies it to the first `budget` sums of each sequence and clears those behind
 *            (mqa_kv_weights_accumulate wants 64 * max_pages of them)
 * kept may be seq_len itself: the new lengths take the old ones' place. Any other overlap of keep, kept,
 * kept_acc or the workspace with each other, acc or seq_len is refused (MQA_ERR_OVERLAP).
 * workspace: mqa_kv_evict_workspace_bytes() bytes, 256-byte aligned: 0 (and the
 * workspace then NULL) up to a max_len of 16,384, at most 6.3 MB per sequence.
 * num_seqs: at most 16,383 whatever max_len is, 4,194,240 up to a max_len of 16,384.
 */
int32_t mqa_kv_evict_select(const float* acc, int64_t acc_stride, const int32_t* seq_len, int64_t num_seqs,
                            int64_t max_len, int64_t budget, int64_t recent, int32_t* keep, int32_t* kept,
                            float* kept_acc, void* workspace, int64_t workspace_bytes, void* stream);
int64_t mqa_kv_evict_workspace_bytes(int64_t num_seqs, int64_t max_len);

/* One paged array to compact: rows_per_position pieces of row_bytes bytes per
 * position (2^24 bytes together at most), at byte strides of page, position and
 * piece, 0 .. 2^32. Bases, strides and row_bytes must be multiples of 4 bytes; the
 * page stride of a pool of one page and the piece stride of one piece are not looked at.
 * src and dst may be one pool. */
typedef struct mqa_kv_array {
  const void* src;
  void* dst;
  int64_t src_stride[3];
  int64_t dst_stride[3];
  int64_t row_bytes;
  int64_t rows_per_position;
} mqa_kv_array;
#define MQA_KV_MAX_ARRAYS 8

/*
 * Moves what was kept into other pages: for every array, sequence s and
 * j < kept[s], position keep[s, j] of src_table's pages goes to position j of
 * dst_table's. Works for keys, values, the indexer's codes and scales, or any
 * other paged array of whole 4-byte words.
 *   keep, kept  int32 [num_seqs, budget], [num_seqs] as mqa_kv_evict_select gives them
 *   src_table   int32 [num_seqs, src_max_pages], dst_table int32 [num_seqs, dst_max_pages]
 * Destination pages must be distinct and none of the source pages that the call reads: otherwise
 * what they hold afterwards is unspecified (no access leaves the arrays).
 * Positions behind kept[s] in the last destination page, and pages that no
 * kept position maps to, are left as they were. A sequence whose kept is
 * negative is left alone; one whose kept exceeds budget or 64 * dst_max_pages
 * is too, and sets MQA_STATUS_BAD_WINDOW; a keep entry outside [0, 64 *
 * src_max_pages) is not moved (MQA_STATUS_BAD_WINDOW), nor is one whose source
 * or destination page is outside its pool (MQA_STATUS_BAD_PAGE).
 */
int32_t mqa_kv_compact(const int32_t* keep, const int32_t* kept, int64_t num_seqs, int64_t budget,
                       const int32_t* src_table, int64_t src_max_pages, int64_t num_src_phys_pages,
                       const int32_t* dst_table, int64_t dst_max_pages, int64_t num_dst_phys_pages,
                       const mqa_kv_array* arrays, int32_t num_arrays, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MQA_KV_CACHE_H */
