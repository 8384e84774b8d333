// Host side of the C ABI declared in include/mqa_kv_cache.h and include/mqa_kv_fp4.h: argument checks,
// strides in bytes, workspace layout. Nothing here allocates or synchronises.
#include "mqa_fp4_topk.h"
#include "mqa_host.h"
#include "mqa_kv.h"
#include "mqa_kv_cache.h"
#include "mqa_kv_fp4.h"
#include "mqa_kv_host.h"
#include "mqa_launch.h"

#include <hip/hip_runtime.h>

#include <cmath>

namespace {

using namespace mqa::host;
using mqa::KvAttnArgs;

// Checks queries over a cache's heads and pages and fills the kernels' arguments.
int32_t query_args(const mqa_kv_query* q, int32_t Hkv, int32_t D, int64_t P_phys, float k_scale, float v_scale,
                   KvAttnArgs* a) {
  const int32_t rc = check_heads(q->num_rows, q->num_heads, Hkv, D);
  if (rc != MQA_OK) return rc;
  if (P_phys < 0 || P_phys > kMaxPages) return MQA_ERR_BAD_SIZE;
  if (!std::isfinite(q->scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale)) return MQA_ERR_BAD_SIZE;
  const float scale = q->scale * k_scale;
  const float log2e = 1.44269504088896340736f;
  if (!std::isfinite(scale * log2e)) return MQA_ERR_BAD_SIZE;
  const int64_t row = static_cast<int64_t>(q->num_heads) * D;
  if (q->num_rows > 1 && (q->row_stride < row || q->row_stride > (1ll << 32))) return MQA_ERR_BAD_SIZE;
  if (q->num_rows > 1 && q->row_stride * 2 % 16) return MQA_ERR_MISALIGNED;
  a->q = static_cast<const char*>(q->q);
  a->q_row = q->num_rows > 1 ? q->row_stride * 2 : 0;
  a->Q = q->num_rows;
  a->P_phys = P_phys;
  a->H = q->num_heads;
  a->Hkv = Hkv;
  a->G = a->H / a->Hkv;
  a->D = D;
  a->q_type = q->type;
  // the running maximum is taken before the scale, which therefore must not be
  // negative: a negative one changes the queries' signs instead
  // and a zero one, so that -infinity times it stays that, clears the queries
  a->c = std::fabs(scale) * log2e;
  a->q_keep = a->c > 0.0f ? ~0u : 0u;
  if (!(a->c > 0.0f)) a->c = 1.0f;
  a->q_flip = std::signbit(scale) ? 0x80008000u : 0u;
  a->score_scale = scale;
  a->v_scale = v_scale;
  return MQA_OK;
}

// Checks queries and cache and fills the kernels' arguments; `values`: the call reads values too.
int32_t attn_args(const mqa_kv_query* q, const mqa_kv_cache* c, bool values, KvAttnArgs* a) {
  if (q == nullptr || c == nullptr) return MQA_ERR_NULL_POINTER;
  if (q->type != MQA_KV_BF16 && q->type != MQA_KV_FP16) return MQA_ERR_UNSUPPORTED;
  if (c->type != q->type && c->type != MQA_KV_E4M3) return MQA_ERR_UNSUPPORTED;
  *a = KvAttnArgs{};
  int32_t rc = query_args(q, c->num_kv_heads, c->head_dim, c->num_phys_pages, c->k_scale, c->v_scale, a);
  if (rc == MQA_OK) rc = cache_strides(c->k_stride, *c, &a->k_page, &a->k_pos, &a->k_head);
  if (rc == MQA_OK && values) rc = cache_strides(c->v_stride, *c, &a->v_page, &a->v_pos, &a->v_head);
  if (rc != MQA_OK) return rc;
  a->k = static_cast<const char*>(c->k);
  a->v = static_cast<const char*>(c->v);
  a->kv_type = c->type;
  return MQA_OK;
}

// The same over a cache in 4 bits.
int32_t fp4_args(const mqa_kv_query* q, const mqa_kv_cache_fp4* c, mqa::KvFp4Args* a) {
  if (q == nullptr || c == nullptr) return MQA_ERR_NULL_POINTER;
  if (q->type != MQA_KV_BF16 && q->type != MQA_KV_FP16) return MQA_ERR_UNSUPPORTED;
  *a = mqa::KvFp4Args{};
  int32_t rc = query_args(q, c->num_kv_heads, c->head_dim, c->num_phys_pages, 1.0f, 1.0f, a);
  const int64_t codes = c->head_dim / 2, scales = c->head_dim / 32;
  if (rc == MQA_OK) rc = fp4_strides(c->k_stride, *c, codes, 16, &a->k_page, &a->k_pos, &a->k_head);
  if (rc == MQA_OK) rc = fp4_strides(c->v_stride, *c, codes, 16, &a->v_page, &a->v_pos, &a->v_head);
  if (rc == MQA_OK) rc = fp4_strides(c->k_scale_stride, *c, scales, scales, &a->ks_page, &a->ks_pos, &a->ks_head);
  if (rc == MQA_OK) rc = fp4_strides(c->v_scale_stride, *c, scales, scales, &a->vs_page, &a->vs_pos, &a->vs_head);
  if (rc != MQA_OK) return rc;
  a->k = static_cast<const char*>(c->k);
  a->v = static_cast<const char*>(c->v);
  a->ks = static_cast<const char*>(c->k_scale);
  a->vs = static_cast<const char*>(c->v_scale);
  return MQA_OK;
}

int32_t window_args(KvAttnArgs* a, const int32_t* table, int64_t n_seq, int64_t max_pages, const int32_t* seq_of_row,
                    const int32_t* row_start, const int32_t* row_end) {
  if (n_seq < 0 || max_pages < 0 || n_seq > 0x7FFFFFFFll || max_pages > kMaxLogical) return MQA_ERR_BAD_SIZE;
  if (max_pages > 0 && n_seq > 0x7FFFFFFFll / max_pages) return MQA_ERR_BAD_SIZE;
  a->table = table;
  a->n_seq = n_seq;
  a->max_pages = max_pages;
  a->seq_of_row = seq_of_row;
  a->row_start = row_start;
  a->row_end = row_end;
  return MQA_OK;
}

struct PartialLayout {
  int64_t prefix, ml, o, total;
};

// Workspace: page prefix of the rows, then (maximum, sum) and weighted values of `slots` partial results.
PartialLayout partial_layout(int64_t prefix_rows, int64_t slots, int32_t D, int32_t group_rows) {
  const int64_t heads = slots * group_rows;
  PartialLayout l;
  l.prefix = 0;
  l.ml = align_up(prefix_rows * static_cast<int64_t>(sizeof(int64_t)));
  l.o = l.ml + align_up(heads * static_cast<int64_t>(sizeof(float2)));
  l.total = l.o + align_up(heads * D * static_cast<int64_t>(sizeof(float)));
  return l;
}

PartialLayout decode_layout(int64_t Q, int32_t D, int32_t G) {
  return partial_layout(Q + 1, 2 * mqa::kKvDecodeGroups, D, mqa::kv_group_rows(D, G));
}

PartialLayout selected_layout(int64_t Q, int32_t D, int32_t G, int32_t Hkv, int32_t splits) {
  return partial_layout(0, splits > 1 ? Q * Hkv * mqa::kv_head_groups(D, G) * splits : 0, D, mqa::kv_group_rows(D, G));
}

// The outputs of an attention lie apart from each other and from what it reads besides the cache, but for out in
// the queries' place: a workgroup that writes a head's row is the only one that reads it, or its launch comes later.
int32_t check_attn_apart(const KvAttnArgs& a, const void* out, const float* lse, const void* workspace, int64_t bytes,
                         const Span* ints, int n_ints) {
  const int64_t row = static_cast<int64_t>(a.H) * a.D * 2;
  const Span outs[] = {{out, 1, 0, a.Q * row}, {lse, 1, 0, a.Q * a.H * 4}, {workspace, 1, 0, bytes}};
  const bool in_place = out == a.q && (a.Q <= 1 || a.q_row == row);
  const Span q = {a.q, a.Q, a.q_row, row};
  int32_t rc = check_apart(outs, 3, ints, n_ints);
  if (rc == MQA_OK) rc = check_apart(outs + (in_place ? 1 : 0), in_place ? 2 : 3, &q, 1);
  return rc;
}

void place(KvAttnArgs* a, const PartialLayout& l, void* workspace) {
  char* base = static_cast<char*>(workspace);
  a->prefix = reinterpret_cast<int64_t*>(base + l.prefix);
  a->part_ml = reinterpret_cast<float2*>(base + l.ml);
  a->part_o = reinterpret_cast<float*>(base + l.o);
}

}  // namespace

extern "C" {

int64_t mqa_kv_attention_decode_workspace_bytes(int64_t num_rows, int32_t num_heads, int32_t num_kv_heads,
                                                int32_t head_dim) {
  const int32_t rc = check_heads(num_rows, num_heads, num_kv_heads, head_dim);
  if (rc != MQA_OK) return rc;
  return decode_layout(num_rows, head_dim, num_heads / num_kv_heads).total;
}

int32_t mqa_kv_attention_decode(const mqa_kv_query* q, const mqa_kv_cache* cache, const int32_t* block_table,
                                int64_t num_seqs, int64_t max_pages, const int32_t* seq_of_row,
                                const int32_t* row_start, const int32_t* row_end, void* out, float* lse,
                                void* workspace, int64_t workspace_bytes, void* stream) {
  KvAttnArgs a;
  int32_t rc = attn_args(q, cache, true, &a);
  if (rc == MQA_OK) rc = window_args(&a, block_table, num_seqs, max_pages, seq_of_row, row_start, row_end);
  if (rc != MQA_OK) return rc;
  const bool rows = a.Q > 0, pages = a.P_phys > 0;
  const PartialLayout lay = decode_layout(a.Q, a.D, a.G);
  if (rows && workspace_bytes < lay.total) return MQA_ERR_BAD_SIZE;
  const PtrSpec specs[] = {
      {a.q, rows, 16},        {a.k, pages, 16},    {a.v, pages, 16},   {block_table, num_seqs > 0 && max_pages > 0, 4},
      {seq_of_row, rows, 4},  {row_start, rows, 4}, {row_end, rows, 4}, {out, rows, 16},
      {lse, false, 4},        {workspace, rows, 256},
  };
  rc = check_ptrs_host(specs, sizeof(specs) / sizeof(specs[0]));
  if (rc != MQA_OK) return rc;
  const Span ints[] = {{block_table, 1, 0, num_seqs * max_pages * 4}, {seq_of_row, 1, 0, a.Q * 4},
                       {row_start, 1, 0, a.Q * 4}, {row_end, 1, 0, a.Q * 4}};
  rc = check_attn_apart(a, out, lse, workspace, lay.total, ints, 4);
  if (rc != MQA_OK) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  DeviceGuard guard;
  DeviceInfo info;
  rc = enter(st, specs, sizeof(specs) / sizeof(specs[0]), guard, &info, /*allow_capture=*/true);
  if (rc != MQA_OK || !rows) return rc;
  a.out = out;
  a.lse = lse;
  a.status = mqa::status_word();
  if (a.status == nullptr) return MQA_ERR_HIP;
  place(&a, lay, workspace);
  return hip_rc(mqa::launch_kv_decode(a, st));
}

int64_t mqa_kv_attention_selected_workspace_bytes(int64_t num_rows, int64_t K, int32_t num_heads,
                                                  int32_t num_kv_heads, int32_t head_dim) {
  const int32_t rc = check_heads(num_rows, num_heads, num_kv_heads, head_dim);
  if (rc != MQA_OK) return rc;
  if (K < 0 || K > 0x7FFFFFFFll) return MQA_ERR_BAD_SIZE;
  const int32_t G = num_heads / num_kv_heads;
  return selected_layout(num_rows, head_dim, G, num_kv_heads,
                         mqa::kv_selected_splits(num_rows, K, head_dim, G, num_kv_heads)).total;
}

int32_t mqa_kv_attention_selected(const mqa_kv_query* q, const mqa_kv_cache* cache, const int32_t* slots,
                                  const int32_t* count, int64_t K, void* out, float* lse, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  KvAttnArgs a;
  int32_t rc = attn_args(q, cache, true, &a);
  if (rc != MQA_OK) return rc;
  if (K < 0 || K > 0x7FFFFFFFll) return MQA_ERR_BAD_SIZE;
  const bool rows = a.Q > 0, pages = a.P_phys > 0;
  a.splits = mqa::kv_selected_splits(a.Q, K, a.D, a.G, a.Hkv);
  const PartialLayout lay = selected_layout(a.Q, a.D, a.G, a.Hkv, a.splits);
  if (rows && workspace_bytes < lay.total) return MQA_ERR_BAD_SIZE;
  const PtrSpec specs[] = {
      {a.q, rows, 16},  {a.k, pages, 16},  {a.v, pages, 16},    {slots, rows && K > 0, 4},
      {count, rows, 4}, {out, rows, 16},   {lse, false, 4},     {workspace, rows && lay.total > 0, 256},
  };
  rc = check_ptrs_host(specs, sizeof(specs) / sizeof(specs[0]));
  if (rc != MQA_OK) return rc;
  const Span ints[] = {{slots, 1, 0, a.Q * K * 4}, {count, 1, 0, a.Q * 4}};
  rc = check_attn_apart(a, out, lse, workspace, lay.total, ints, 2);
  if (rc != MQA_OK) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  DeviceGuard guard;
  DeviceInfo info;
  rc = enter(st, specs, sizeof(specs) / sizeof(specs[0]), guard, &info, /*allow_capture=*/true);
  if (rc != MQA_OK || !rows) return rc;
  a.slots = slots;
  a.count = count;
  a.K = K;
  a.out = out;
  a.lse = lse;
  a.status = mqa::status_word();
  if (a.status == nullptr) return MQA_ERR_HIP;
  place(&a, lay, workspace);
  return hip_rc(mqa::launch_kv_selected(a, st));
}

int32_t mqa_kv_attention_decode_fp4(const mqa_kv_query* q, const mqa_kv_cache_fp4* cache, const int32_t* block_table,
                                    int64_t num_seqs, int64_t max_pages, const int32_t* seq_of_row,
                                    const int32_t* row_start, const int32_t* row_end, void* out, float* lse,
                                    void* workspace, int64_t workspace_bytes, void* stream) {
  mqa::KvFp4Args a;
  int32_t rc = fp4_args(q, cache, &a);
  if (rc == MQA_OK) rc = window_args(&a, block_table, num_seqs, max_pages, seq_of_row, row_start, row_end);
  if (rc != MQA_OK) return rc;
  const bool rows = a.Q > 0, pages = a.P_phys > 0;
  const uintptr_t unit = a.D / 32;
  const PartialLayout lay = decode_layout(a.Q, a.D, a.G);
  if (rows && workspace_bytes < lay.total) return MQA_ERR_BAD_SIZE;
  const PtrSpec specs[] = {
      {a.q, rows, 16},        {a.k, pages, 16},    {a.v, pages, 16},   {block_table, num_seqs > 0 && max_pages > 0, 4},
      {a.ks, pages, unit},    {a.vs, pages, unit},
      {seq_of_row, rows, 4},  {row_start, rows, 4}, {row_end, rows, 4}, {out, rows, 16},
      {lse, false, 4},        {workspace, rows, 256},
  };
  rc = check_ptrs_host(specs, sizeof(specs) / sizeof(specs[0]));
  if (rc != MQA_OK) return rc;
  const Span ints[] = {{block_table, 1, 0, num_seqs * max_pages * 4}, {seq_of_row, 1, 0, a.Q * 4},
                       {row_start, 1, 0, a.Q * 4}, {row_end, 1, 0, a.Q * 4}};
  rc = check_attn_apart(a, out, lse, workspace, lay.total, ints, 4);
  if (rc != MQA_OK) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  DeviceGuard guard;
  DeviceInfo info;
  rc = enter(st, specs, sizeof(specs) / sizeof(specs[0]), guard, &info, /*allow_capture=*/true);
  if (rc != MQA_OK || !rows) return rc;
  a.out = out;
  a.lse = lse;
  a.status = mqa::status_word();
  if (a.status == nullptr) return MQA_ERR_HIP;
  place(&a, lay, workspace);
  return hip_rc(mqa::launch_kv_decode_fp4(a, st));
}

int32_t mqa_kv_attention_selected_fp4(const mqa_kv_query* q, const mqa_kv_cache_fp4* cache, const int32_t* slots,
                                      const int32_t* count, int64_t K, void* out, float* lse, void* workspace,
                                      int64_t workspace_bytes, void* stream) {
  mqa::KvFp4Args a;
  int32_t rc = fp4_args(q, cache, &a);
  if (rc != MQA_OK) return rc;
  if (K < 0 || K > 0x7FFFFFFFll) return MQA_ERR_BAD_SIZE;
  const bool rows = a.Q > 0, pages = a.P_phys > 0;
  const uintptr_t unit = a.D / 32;
  a.splits = mqa::kv_selected_splits(a.Q, K, a.D, a.G, a.Hkv);
  const PartialLayout lay = selected_layout(a.Q, a.D, a.G, a.Hkv, a.splits);
  if (rows && workspace_bytes < lay.total) return MQA_ERR_BAD_SIZE;
  const PtrSpec specs[] = {
      {a.q, rows, 16},      {a.k, pages, 16},    {a.v, pages, 16}, {a.ks, pages, unit}, {a.vs, pages, unit},
      {slots, rows && K > 0, 4}, {count, rows, 4}, {out, rows, 16},  {lse, false, 4},
      {workspace, rows && lay.total > 0, 256},
  };
  rc = check_ptrs_host(specs, sizeof(specs) / sizeof(specs[0]));
  if (rc != MQA_OK) return rc;
  const Span ints[] = {{slots, 1, 0, a.Q * K * 4}, {count, 1, 0, a.Q * 4}};
  rc = check_attn_apart(a, out, lse, workspace, lay.total, ints, 2);
  if (rc != MQA_OK) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  DeviceGuard guard;
  DeviceInfo info;
  rc = enter(st, specs, sizeof(specs) / sizeof(specs[0]), guard, &info, /*allow_capture=*/true);
  if (rc != MQA_OK || !rows) return rc;
  a.slots = slots;
  a.count = count;
  a.K = K;
  a.out = out;
  a.lse = lse;
  a.status = mqa::status_word();
  if (a.status == nullptr) return MQA_ERR_HIP;
  place(&a, lay, workspace);
  return hip_rc(mqa::launch_kv_selected_fp4(a, st));
}

int32_t mqa_kv_weights_accumulate(const mqa_kv_query* q, const float* lse, const mqa_kv_cache* cache,
                                  const int32_t* block_table, int64_t num_seqs, int64_t max_pages,
                                  const int32_t* seq_of_row, const int32_t* row_start, const int32_t* row_end,
                                  float* acc, int64_t acc_stride, void* stream) {
  KvAttnArgs a;
  int32_t rc = attn_args(q, cache, false, &a);
  if (rc == MQA_OK) rc = window_args(&a, block_table, num_seqs, max_pages, seq_of_row, row_start, row_end);
  if (rc != MQA_OK) return rc;
  if (acc_stride < 64 * max_pages || acc_stride > (1ll << 32)) return MQA_ERR_BAD_SIZE;
  const bool rows = a.Q > 0, pages = a.P_phys > 0, sums = num_seqs > 0 && max_pages > 0;
  const PtrSpec specs[] = {
      {a.q, rows, 16},        {lse, rows, 4},       {a.k, pages, 16},   {block_table, sums, 4},
      {seq_of_row, rows, 4},  {row_start, rows, 4}, {row_end, rows, 4}, {acc, sums, 4},
  };
  rc = check_ptrs_host(specs, sizeof(specs) / sizeof(specs[0]));
  if (rc != MQA_OK) return rc;
  const Span out = {acc, num_seqs, acc_stride * 4, 64 * max_pages * 4};
  const Span ins[] = {{a.q, a.Q, a.q_row, static_cast<int64_t>(a.H) * a.D * 2}, {lse, 1, 0, a.Q * a.H * 4},
                      {block_table, 1, 0, num_seqs * max_pages * 4}, {seq_of_row, 1, 0, a.Q * 4},
                      {row_start, 1, 0, a.Q * 4}, {row_end, 1, 0, a.Q * 4}};
  rc = check_apart(&out, 1, ins, 6);
  if (rc != MQA_OK) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  DeviceGuard guard;
  DeviceInfo info;
  rc = enter(st, specs, sizeof(specs) / sizeof(specs[0]), guard, &info, /*allow_capture=*/true);
  if (rc != MQA_OK || !rows) return rc;
  a.status = mqa::status_word();
  if (a.status == nullptr) return MQA_ERR_HIP;
  return hip_rc(mqa::launch_kv_weights(a, lse, acc, acc_stride, st));
}

int64_t mqa_kv_evict_workspace_bytes(int64_t num_seqs, int64_t max_len) {
  // workgroups of 1,024 threads, counted in 32 bits
  if (num_seqs < 0 || max_len < 0 || max_len > 0x7FFFFFFFll - 512) return MQA_ERR_BAD_SIZE;
  const int64_t chunks = mqa::kv_evict_chunks(max_len);
  if (num_seqs > kMaxItems / 4 / chunks) return MQA_ERR_BAD_SIZE;
  return chunks == 1 ? 0 : align_up(num_seqs * 8 * 4) + align_up(num_seqs * chunks * 3 * 2048 * 4);
}

int32_t mqa_kv_evict_select(const float* acc, int64_t acc_stride, const int32_t* seq_len, int64_t num_seqs,
                            int64_t max_len, int64_t budget, int64_t recent, int32_t* keep, int32_t* kept,
                            float* kept_acc, void* workspace, int64_t workspace_bytes, void* stream) {
  const int64_t need = mqa_kv_evict_workspace_bytes(num_seqs, max_len);
  if (need < 0) return static_cast<int32_t>(need);
  if (acc_stride < max_len || acc_stride > (1ll << 32)) return MQA_ERR_BAD_SIZE;
  if (budget < 0 || budget > 0x7FFFFFFFll || recent < 0 || recent > budget) return MQA_ERR_BAD_SIZE;
  const bool rows = num_seqs > 0;
  if (rows && workspace_bytes < need) return MQA_ERR_BAD_SIZE;
  const PtrSpec specs[] = {
      {acc, rows && max_len > 0, 4}, {seq_len, rows, 4},  {keep, rows && budget > 0, 4},
      {kept, rows, 4},               {kept_acc, false, 4}, {workspace, rows && need > 0, 256},
  };
  int32_t rc = check_ptrs_host(specs, sizeof(specs) / sizeof(specs[0]));
  if (rc != MQA_OK) return rc;
  const Span outs[] = {{keep, 1, 0, num_seqs * budget * 4},
                       {kept, 1, 0, num_seqs * 4},
                       {kept_acc, 1, 0, num_seqs * budget * 4},
                       {workspace, 1, 0, need}};
  // the kernels read every length before its kept is written, so that kept may take the lengths' place
  const Span ins[] = {{acc, num_seqs, acc_stride * 4, max_len * 4}, {kept == seq_len ? nullptr : seq_len, 1, 0, num_seqs * 4}};
  rc = check_apart(outs, 4, ins, 2);
  if (rc != MQA_OK) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  DeviceGuard guard;
  DeviceInfo info;
  rc = enter(st, specs, sizeof(specs) / sizeof(specs[0]), guard, &info, /*allow_capture=*/true);
  if (rc != MQA_OK || !rows) return rc;
  mqa::KvEvictArgs a{acc, acc_stride, seq_len, num_seqs, max_len, budget, recent, keep, kept, kept_acc,
                     mqa::status_word(), nullptr, nullptr};
  if (a.status == nullptr) return MQA_ERR_HIP;
  a.state = static_cast<uint32_t*>(workspace);
  a.counts = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + align_up(num_seqs * 8 * 4));
  return hip_rc(mqa::launch_kv_evict_select(a, st));
}

int32_t mqa_kv_compact(const int32_t* keep, const int32_t* kept, int64_t num_seqs, int64_t budget,
                       const int32_t* src_table, int64_t src_max_pages, int64_t num_src_phys_pages,
                       const int32_t* dst_table, int64_t dst_max_pages, int64_t num_dst_phys_pages,
                       const mqa_kv_array* arrays, int32_t num_arrays, void* stream) {
  if (num_seqs < 0 || num_seqs > 0x7FFFFFFFll || budget < 0 || budget > 0x7FFFFFFFll) return MQA_ERR_BAD_SIZE;
  if (src_max_pages < 0 || src_max_pages > kMaxLogical || dst_max_pages < 0 || dst_max_pages > kMaxLogical)
    return MQA_ERR_BAD_SIZE;
  if (num_src_phys_pages < 0 || num_src_phys_pages > kMaxPages || num_dst_phys_pages < 0 ||
      num_dst_phys_pages > kMaxPages)
    return MQA_ERR_BAD_SIZE;
  if (num_arrays < 0 || num_arrays > MQA_KV_MAX_ARRAYS) return MQA_ERR_BAD_SIZE;
  if (num_arrays > 0 && arrays == nullptr) return MQA_ERR_NULL_POINTER;
  const bool rows = num_seqs > 0 && budget > 0 && num_arrays > 0;
  mqa::KvCompactArgs a{};
  PtrSpec specs[4 + 2 * MQA_KV_MAX_ARRAYS];
  int n = 0;
  specs[n++] = {keep, rows, 4};
  specs[n++] = {kept, rows, 4};
  specs[n++] = {src_table, rows && src_max_pages > 0, 4};
  specs[n++] = {dst_table, rows && dst_max_pages > 0, 4};
  for (int i = 0; i < num_arrays; ++i) {
    const mqa_kv_array& x = arrays[i];
    mqa::KvCompactArray& y = a.arrays[i];
    if (x.row_bytes < 1 || x.row_bytes > (1ll << 24) || x.rows_per_position < 1 ||
        x.rows_per_position > (1ll << 24) / x.row_bytes)
      return MQA_ERR_BAD_SIZE;
    bool wide = x.row_bytes % 16 == 0 && reinterpret_cast<uintptr_t>(x.src) % 16 == 0 &&
                reinterpret_cast<uintptr_t>(x.dst) % 16 == 0;
    if (x.row_bytes % 4) return MQA_ERR_MISALIGNED;
    int64_t strides[2][3];   // of source and destination; those of one page or one piece, never taken, as 0
    for (int d = 0; d < 2; ++d)
      for (int k = 0; k < 3; ++k) {
        const bool taken = k == 1 || (k == 2 ? x.rows_per_position : d == 0 ? num_src_phys_pages : num_dst_phys_pages) > 1;
        const int64_t stride = strides[d][k] = taken ? (d == 0 ? x.src_stride : x.dst_stride)[k] : 0;
        if (stride < 0 || stride > (1ll << 32)) return MQA_ERR_BAD_SIZE;
        if (stride % 4) return MQA_ERR_MISALIGNED;
        wide = wide && stride % 16 == 0;
      }
    y.src = static_cast<const char*>(x.src);
    y.dst = static_cast<char*>(x.dst);
    y.src_page = strides[0][0];
    y.src_pos = strides[0][1];
    y.src_row = strides[0][2];
    y.dst_page = strides[1][0];
    y.dst_pos = strides[1][1];
    y.dst_row = strides[1][2];
    y.wide = wide;
    y.rows = x.rows_per_position;
    y.units = x.row_bytes / (wide ? 16 : 4);
    // pieces that lie end to end on both sides are one
    if (y.rows == 1 || (x.src_stride[2] == x.row_bytes && x.dst_stride[2] == x.row_bytes)) {
      y.units *= y.rows;
      y.rows = 1;
    }
    specs[n++] = {x.src, rows && num_src_phys_pages > 0, 4};
    specs[n++] = {x.dst, rows && num_dst_phys_pages > 0, 4};
  }
  const hipStream_t st = static_cast<hipStream_t>(stream);
  DeviceGuard guard;
  DeviceInfo info;
  int32_t rc = enter(st, specs, n, guard, &info, /*allow_capture=*/true);
  if (rc != MQA_OK || !rows) return rc;
  a.keep = keep;
  a.kept = kept;
  a.n_seq = num_seqs;
  a.budget = budget;
  a.src_table = src_table;
  a.src_pages = src_max_pages;
  a.P_src = num_src_phys_pages;
  a.dst_table = dst_table;
  a.dst_pages = dst_max_pages;
  a.P_dst = num_dst_phys_pages;
  a.n_arrays = num_arrays;
  a.status = mqa::status_word();
  if (a.status == nullptr) return MQA_ERR_HIP;
  return hip_rc(mqa::launch_kv_compact(a, st));
}

}  // extern "C"
