// Host side of the C ABI declared in include/mqa_kv_append.h: argument checks and
// strides in bytes. Nothing here allocates or synchronises.
#include "mqa_fp4_topk.h"
#include "mqa_host.h"
#include "mqa_kv.h"
#include "mqa_kv_append.h"
#include "mqa_kv_host.h"
#include "mqa_launch.h"

#include <hip/hip_runtime.h>

#include <cmath>

namespace {

using namespace mqa::host;
using mqa::KvHeads;
using mqa::KvWriteArgs;

// Rows of heads; `out`: the call writes them to x.out.
int32_t heads_args(const mqa_kv_rows& x, int64_t num_rows, int32_t D, bool out, KvHeads* h) {
  if (x.num_heads < 1 || x.num_heads > 65536 || !std::isfinite(x.weight_offset)) return MQA_ERR_BAD_SIZE;
  const int64_t row = static_cast<int64_t>(x.num_heads) * D;
  const int64_t strides[2] = {x.row_stride, x.out_stride};
  for (int i = 0; i < (out ? 2 : 1); ++i) {
    if (num_rows > 1 && (strides[i] < row || strides[i] > (1ll << 32))) return MQA_ERR_BAD_SIZE;
    if (num_rows > 1 && strides[i] * 2 % 16) return MQA_ERR_MISALIGNED;
  }
  h->x = static_cast<const char*>(x.x);
  h->x_row = num_rows > 1 ? x.row_stride * 2 : 0;
  h->out = out ? static_cast<char*>(x.out) : nullptr;
  h->out_row = out && num_rows > 1 ? x.out_stride * 2 : 0;
  h->weight = static_cast<const uint16_t*>(x.weight);
  h->offset = x.weight_offset;
  h->n = x.num_heads;
  return MQA_OK;
}

int32_t turn_args(const mqa_kv_turn& t, int32_t D, KvWriteArgs* a) {
  if (!std::isfinite(t.eps) || t.eps < 0.0f) return MQA_ERR_BAD_SIZE;
  a->eps = t.eps;
  if (t.inv_freq == nullptr) return MQA_OK;
  if (t.rotary_dim < 16 || t.rotary_dim % 16 || t.rotary_offset < 0 || t.rotary_offset % 8 ||
      t.rotary_offset > D - t.rotary_dim || t.interleaved < 0 || t.interleaved > 1)
    return MQA_ERR_BAD_SIZE;
  a->inv_freq = t.inv_freq;
  a->turn_pos = t.position;
  a->half = t.rotary_dim / 2;
  a->offset = t.rotary_offset;
  a->interleaved = t.interleaved;
  return MQA_OK;
}

int32_t check_kind(int64_t num_rows, int32_t D, int32_t type) {
  if (type != MQA_KV_BF16 && type != MQA_KV_FP16) return MQA_ERR_UNSUPPORTED;
  if (D != 64 && D != 128 && D != 256) return MQA_ERR_UNSUPPORTED;
  return num_rows < 0 || num_rows > kMaxItems ? MQA_ERR_BAD_SIZE : MQA_OK;
}

Span rows_span(const void* p, int64_t row, const KvHeads& h, const KvWriteArgs& a) {
  return Span(p, h.n > 0 ? a.T : 0, row, static_cast<int64_t>(h.n) * a.D * 2);
}

// check_apart of two; rows of different strides count as one piece from the first to the last.
int32_t check_two_apart(Span x, Span y) {
  if (x.rows > 1 && y.rows > 1 && x.stride != y.stride) {
    x = Span(x.p, 1, 0, (x.rows - 1) * x.stride + x.bytes);
    y = Span(y.p, 1, 0, (y.rows - 1) * y.stride + y.bytes);
  }
  return overlap(x, y) ? MQA_ERR_OVERLAP : MQA_OK;
}

// Outputs of queries and keys lie apart from each other and from what the call reads, but for one in its own
// x's place: the lanes that write a head are the only ones that read it, and have read it before.
int32_t check_rows_apart(const KvWriteArgs& a, const Span* more, int n_more) {
  const KvHeads* heads[3] = {&a.q, &a.k, &a.v};
  const Span small[] = {{a.q.weight, 1, 0, a.D * 2}, {a.k.weight, 1, 0, a.D * 2}, {a.inv_freq, 1, 0, a.half * 4},
                        {a.turn_pos, 1, 0, a.T * 4}};
  const Span outs[] = {rows_span(a.q.out, a.q.out_row, a.q, a), rows_span(a.k.out, a.k.out_row, a.k, a)};
  int32_t rc = check_two_apart(outs[0], outs[1]);
  for (int o = 0; o < 2 && rc == MQA_OK; ++o) {
    rc = check_apart(&outs[o], 1, small, 4);
    if (rc == MQA_OK) rc = check_apart(&outs[o], 1, more, n_more);
  }
  for (int o = 0; o < 2 && rc == MQA_OK; ++o)
    for (int i = 0; i < 3 && rc == MQA_OK; ++i) {
      const bool in_place = o == i && heads[i]->x == heads[o]->out && heads[i]->x_row == heads[o]->out_row;
      const Span in = rows_span(heads[i]->x, heads[i]->x_row, *heads[i], a);
      if (!in_place) rc = check_two_apart(outs[o], in);
    }
  return rc;
}

constexpr int kMaxSpecs = 20;

void rows_specs(const KvWriteArgs& a, const KvHeads& h, bool out, PtrSpec* specs, int* n) {
  const bool any = a.T > 0 && h.n > 0;
  specs[(*n)++] = {h.x, any, 16};
  specs[(*n)++] = {h.weight, false, 16};
  if (out) specs[(*n)++] = {h.out, any, 16};
}

// Checks the pointers, enters the device and launches.
int32_t launch(KvWriteArgs* a, const PtrSpec* specs, int n, const Span* more, int n_more, void* stream) {
  int32_t rc = check_ptrs_host(specs, n);
  if (rc == MQA_OK) rc = check_rows_apart(*a, more, n_more);
  if (rc != MQA_OK) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  DeviceGuard guard;
  DeviceInfo info;
  rc = enter(st, specs, n, guard, &info, /*allow_capture=*/true);
  if (rc != MQA_OK || a->T == 0) return rc;
  a->status = mqa::status_word();
  if (a->status == nullptr) return MQA_ERR_HIP;
  return hip_rc(mqa::launch_kv_write(*a, st));
}

// What both appending calls check alike; the cache's tensors are in `a` already.
int32_t append(const mqa_kv_new* x, const mqa_kv_rows* q, int32_t Hkv, uintptr_t align, uintptr_t scale_align, KvWriteArgs* a,
               void* stream) {
  const bool values = x->v.x != nullptr;
  if (x->k.num_heads != Hkv || (values && x->v.num_heads != Hkv)) return MQA_ERR_BAD_SIZE;
  int32_t rc = heads_args(x->k, x->num_rows, a->D, false, &a->k);
  if (rc == MQA_OK && values) rc = heads_args(x->v, x->num_rows, a->D, false, &a->v);
  if (rc == MQA_OK && q != nullptr) rc = heads_args(*q, x->num_rows, a->D, true, &a->q);
  if (rc == MQA_OK) rc = turn_args(x->turn, a->D, a);
  if (rc != MQA_OK) return rc;
  a->v.weight = nullptr;
  if (x->num_seqs < 0 || x->max_pages < 0 || x->num_seqs > 0x7FFFFFFFll || x->max_pages > kMaxLogical) return MQA_ERR_BAD_SIZE;
  if (x->max_pages > 0 && x->num_seqs > 0x7FFFFFFFll / x->max_pages) return MQA_ERR_BAD_SIZE;
  a->T = x->num_rows;
  a->type = x->type;
  a->table = x->block_table;
  a->n_seq = x->num_seqs;
  a->max_pages = x->max_pages;
  a->seq = x->seq_of_row;
  a->pos = x->position;
  const bool rows = a->T > 0, pages = a->P_phys > 0, fp4 = a->store == mqa::kKvStoreFp4;
  PtrSpec specs[kMaxSpecs];
  int n = 0;
  rows_specs(*a, a->q, true, specs, &n);
  rows_specs(*a, a->k, false, specs, &n);
  rows_specs(*a, a->v, false, specs, &n);
  specs[n++] = {a->table, a->n_seq > 0 && a->max_pages > 0, 4};
  specs[n++] = {a->seq, rows, 4};
  specs[n++] = {a->pos, rows, 4};
  specs[n++] = {a->inv_freq, false, 4};
  specs[n++] = {a->turn_pos, false, 4};
  specs[n++] = {a->kc.p, pages, align};
  if (values) specs[n++] = {a->vc.p, pages, align};
  if (fp4) specs[n++] = {a->ks.p, pages, scale_align};
  if (fp4 && values) specs[n++] = {a->vs.p, pages, scale_align};
  const Span more[] = {{a->table, 1, 0, a->n_seq * a->max_pages * 4}, {a->seq, 1, 0, a->T * 4}, {a->pos, 1, 0, a->T * 4}};
  return launch(a, specs, n, more, 3, stream);
}

}  // namespace

extern "C" {

int32_t mqa_kv_norm_rotate(const mqa_kv_rows* q, const mqa_kv_rows* k, const mqa_kv_turn* turn, int64_t num_rows,
                           int32_t head_dim, int32_t type, void* stream) {
  if (q == nullptr || turn == nullptr) return MQA_ERR_NULL_POINTER;
  int32_t rc = check_kind(num_rows, head_dim, type);
  KvWriteArgs a{};
  if (rc == MQA_OK) rc = heads_args(*q, num_rows, head_dim, true, &a.q);
  if (rc == MQA_OK && k != nullptr) rc = heads_args(*k, num_rows, head_dim, true, &a.k);
  if (rc == MQA_OK) rc = turn_args(*turn, head_dim, &a);
  if (rc != MQA_OK) return rc;
  a.T = num_rows;
  a.D = head_dim;
  a.type = type;
  a.store = mqa::kKvStoreRows;
  PtrSpec specs[kMaxSpecs];
  int n = 0;
  rows_specs(a, a.q, true, specs, &n);
  rows_specs(a, a.k, true, specs, &n);
  specs[n++] = {a.inv_freq, false, 4};
  specs[n++] = {a.turn_pos, num_rows > 0 && a.inv_freq != nullptr, 4};
  return launch(&a, specs, n, nullptr, 0, stream);
}

int32_t mqa_kv_append(const mqa_kv_new* rows, const mqa_kv_rows* q, const mqa_kv_cache* cache, void* stream) {
  if (rows == nullptr || cache == nullptr) return MQA_ERR_NULL_POINTER;
  const mqa_kv_cache& c = *cache;
  int32_t rc = check_kind(rows->num_rows, c.head_dim, rows->type);
  if (rc != MQA_OK) return rc;
  const bool e4m3 = c.type == MQA_KV_E4M3, values = rows->v.x != nullptr;
  if (!e4m3 && c.type != rows->type) return MQA_ERR_UNSUPPORTED;
  if (c.num_kv_heads < 1 || c.num_phys_pages < 0 || c.num_phys_pages > kMaxPages) return MQA_ERR_BAD_SIZE;
  const float scales[2] = {c.k_scale, values ? c.v_scale : 1.0f};
  for (float s : scales)
    if (e4m3 ? !std::isfinite(s) || s <= 0.0f : s != 1.0f) return MQA_ERR_BAD_SIZE;
  KvWriteArgs a{};
  a.D = c.head_dim;
  a.store = e4m3 ? mqa::kKvStoreE4m3 : mqa::kKvStoreSame;
  a.P_phys = c.num_phys_pages;
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.kc.p = static_cast<char*>(const_cast<void*>(c.k));
  a.vc.p = static_cast<char*>(const_cast<void*>(c.v));
  rc = cache_strides(c.k_stride, c, &a.kc.page, &a.kc.pos, &a.kc.head);
  if (rc == MQA_OK && values) rc = cache_strides(c.v_stride, c, &a.vc.page, &a.vc.pos, &a.vc.head);
  if (rc != MQA_OK) return rc;
  return append(rows, q, c.num_kv_heads, 16, 0, &a, stream);
}

int32_t mqa_kv_append_fp4(const mqa_kv_new* rows, const mqa_kv_rows* q, const mqa_kv_cache_fp4* cache, void* stream) {
  if (rows == nullptr || cache == nullptr) return MQA_ERR_NULL_POINTER;
  const mqa_kv_cache_fp4& c = *cache;
  int32_t rc = check_kind(rows->num_rows, c.head_dim, rows->type);
  if (rc != MQA_OK) return rc;
  const bool values = rows->v.x != nullptr;
  if (c.num_kv_heads < 1 || c.num_phys_pages < 0 || c.num_phys_pages > kMaxPages) return MQA_ERR_BAD_SIZE;
  const int64_t codes = c.head_dim / 2, scales = c.head_dim / 32;
  KvWriteArgs a{};
  a.D = c.head_dim;
  a.store = mqa::kKvStoreFp4;
  a.P_phys = c.num_phys_pages;
  a.kc.p = static_cast<char*>(c.k);
  a.vc.p = static_cast<char*>(c.v);
  a.ks.p = static_cast<char*>(c.k_scale);
  a.vs.p = static_cast<char*>(c.v_scale);
  rc = fp4_strides(c.k_stride, c, codes, 16, &a.kc.page, &a.kc.pos, &a.kc.head);
  if (rc == MQA_OK) rc = fp4_strides(c.k_scale_stride, c, scales, scales, &a.ks.page, &a.ks.pos, &a.ks.head);
  if (rc == MQA_OK && values) rc = fp4_strides(c.v_stride, c, codes, 16, &a.vc.page, &a.vc.pos, &a.vc.head);
  if (rc == MQA_OK && values) rc = fp4_strides(c.v_scale_stride, c, scales, scales, &a.vs.page, &a.vs.pos, &a.vs.head);
  if (rc != MQA_OK) return rc;
  return append(rows, q, c.num_kv_heads, 16, static_cast<uintptr_t>(scales), &a, stream);
}

}  // extern "C"
