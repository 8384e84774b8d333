// Internal declarations of the key-value cache operators: what the host side
// (mqa_kv_api.hip) hands to the kernels' launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mqa {

// One call of an attention over the cache. Strides in bytes.
struct KvAttnArgs {
  const char* q;
  int64_t q_row;
  int64_t Q;
  const char* k;
  const char* v;
  int64_t k_page, k_pos, k_head;
  int64_t v_page, v_pos, v_head;
  int64_t P_phys;
  int32_t H, Hkv, D;
  int32_t G;                 // query heads per key head
  int32_t q_type, kv_type;   // MQA_KV_*
  float c;                   // |scale * k_scale| * log2(e), or 1 where that is 0
  uint32_t q_keep;           // 0 where scale * k_scale is 0 (the queries count as 0), else all bits
  uint32_t q_flip;           // 0x80008000 where scale * k_scale is negative, else 0
  float score_scale;         // scale * k_scale (weights)
  float v_scale;
  void* out;
  float* lse;
  // windows (decode, weights)
  const int32_t* table;
  int64_t n_seq, max_pages;
  const int32_t *seq_of_row, *row_start, *row_end;
  // lists (selected)
  const int32_t *slots, *count;
  int64_t K;
  int32_t splits;
  uint32_t join_cost;        // of one more part, in pages (16 bits behind the point; decode)
  // workspace
  int64_t* prefix;           // [Q + 1] window pages of the rows before each row (decode)
  float* part_o;             // [slots of partial sums, heads, D]
  float2* part_ml;           // [slots of partial sums, heads] maximum (log2 domain) and sum
  int32_t* status;
};

// Query heads that a workgroup carries for one row, in tiles of 16: as many as the
// group has, up to four tiles (two where D = 256, whose sums need twice the registers).
constexpr int kv_tiles(int D, int G) { return G <= 16 ? 1 : G <= 32 || D == 256 ? 2 : 4; }
constexpr int kv_head_groups(int D, int G) { return (G + 16 * kv_tiles(D, G) - 1) / (16 * kv_tiles(D, G)); }
constexpr int kv_group_rows(int D, int G) { return G < 16 * kv_tiles(D, G) ? G : 16 * kv_tiles(D, G); }

// Workgroups of the decode form: two for each of 256 compute units, which is what LDS leaves the staged kernels room for,
// and registers the others with D = 128 in 16 bits and D = 256. D = 64 would have room for four, 8 bits with fewer dims for three.
constexpr int kKvDecodeGroups = 512;
constexpr int kKvPlanRows = 1024;     // rows up to which every workgroup plans for itself
constexpr int kKvSelBlock = 1024;     // slots of a list in LDS at once (selected form)

int32_t kv_selected_splits(int64_t Q, int64_t K, int D, int G, int Hkv);

hipError_t launch_kv_decode(const KvAttnArgs& a, hipStream_t st);
hipError_t launch_kv_selected(const KvAttnArgs& a, hipStream_t st);

// acc[seq * acc_stride + p] += the rows' weights (a.lse is read, out unused).
hipError_t launch_kv_weights(const KvAttnArgs& a, const float* lse, float* acc, int64_t acc_stride, hipStream_t st);

struct KvEvictArgs {
  const float* acc;
  int64_t acc_stride;
  const int32_t* seq_len;
  int64_t n_seq, max_len, budget, recent;
  int32_t* keep;
  int32_t* kept;
  float* kept_acc;
  int32_t* status;
  // workspace of long sequences
  uint32_t* counts;   // [n_seq, chunks, 3, 2048] counts of each chunk's digits
  uint32_t* state;    // [n_seq, 8] prefix and need behind the first two digits, and the length
};
// Sequences of up to 16,384 positions (the capacity's bound, as the host knows no lengths) take one
// workgroup; longer ones one per chunk, of which there are at most 256.
constexpr int kKvEvictPiece = 8192, kKvEvictChunks = 256;
// Chunks that a launch and its workspace have room for.
constexpr int64_t kv_evict_chunks(int64_t max_len) {
  if (max_len <= 16384) return 1;
  const int64_t pieces = (max_len + kKvEvictPiece - 1) / kKvEvictPiece;
  return pieces < kKvEvictChunks ? pieces : kKvEvictChunks;
}
hipError_t launch_kv_evict_select(const KvEvictArgs& a, hipStream_t st);

constexpr int kKvMaxArrays = 8;
struct KvCompactArray {
  const char* src;
  char* dst;
  int64_t src_page, src_pos, src_row, dst_page, dst_pos, dst_row;   // byte strides
  int64_t units;       // pieces of 16 (or 4) bytes per row
  int64_t rows;        // rows per position
  int32_t wide;        // 16-byte pieces
};
struct KvCompactArgs {
  const int32_t *keep, *kept;
  int64_t n_seq, budget;
  const int32_t* src_table;
  int64_t src_pages, P_src;
  const int32_t* dst_table;
  int64_t dst_pages, P_dst;
  int32_t n_arrays;
  KvCompactArray arrays[kKvMaxArrays];
  int32_t* status;
};
hipError_t launch_kv_compact(const KvCompactArgs& a, hipStream_t st);

// A cache in 4 bits: the codes are KvAttnArgs' k and v, these their scales. Strides in bytes.
struct KvFp4Args : KvAttnArgs {
  const char* ks;
  const char* vs;
  int64_t ks_page, ks_pos, ks_head;
  int64_t vs_page, vs_pos, vs_head;
};
hipError_t launch_kv_decode_fp4(const KvFp4Args& a, hipStream_t st);
hipError_t launch_kv_selected_fp4(const KvFp4Args& a, hipStream_t st);

// New heads: norm, rotation, appending. Strides in bytes.
struct KvHeads {
  const char* x;
  int64_t x_row;
  char* out;
  int64_t out_row;
  const uint16_t* weight;    // null: no norm
  float offset;
  int32_t n;                 // 0: none
};
struct KvPages {
  char* p;
  int64_t page, pos, head;
};
enum KvStore : int32_t { kKvStoreRows, kKvStoreSame, kKvStoreE4m3, kKvStoreFp4 };
struct KvWriteArgs {
  KvHeads q, k, v;           // out of k and v: kKvStoreRows
  int64_t T;
  int32_t D, type;           // MQA_KV_*
  int32_t store;             // KvStore
  const float* inv_freq;     // null: no rotation
  const int32_t* turn_pos;   // null: pos
  int32_t half, offset, interleaved;   // pairs of dims, the first dim
  float eps;
  const int32_t* table;
  int64_t n_seq, max_pages;
  const int32_t *seq, *pos;
  int64_t P_phys;
  KvPages kc, vc, ks, vs;    // codes or numbers, and the scales of 4 bits
  float k_scale, v_scale;    // of 8 bits
  int32_t* status;
};
hipError_t launch_kv_write(const KvWriteArgs& a, hipStream_t st);

}  // namespace mqa
