// New heads on their way into use (gfx950): norm and rotation of queries and keys,
// keys and values into the paged cache in 16, 8 or 4 bits.
//
// Mathematics. y = x / sqrt(mean(x^2) + eps) * (w + offset); pair (a, b) of dims turns by
// t = position * inv_freq: (a cos t - b sin t, b cos t + a sin t). t is taken in 64 bits as
// turns of a circle, of which the fraction alone goes on in 32: a position of a million
// times a frequency of one has lost 0.06 rad in 32 bits, here 2^-31.
//
// Bound by memory: a head's numbers are read and written once. A lane holds 8 neighbouring
// dims of a head (16 bytes), D / 8 lanes a head; sums go over them by lane permutes, and a
// pair's other half comes from the lane that has it. A workgroup takes some rows with all
// their heads (or, where rows are few, a part of the heads), so that a row's cosines and
// sines are made once, by one thread each, and lie in LDS.
#include "mqa_fp4_topk.h"
#include "mqa_kv.h"
#include "mqa_kv_cache.h"
#include "mqa_device.h"
#include "mqa_launch.h"

namespace mqa {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kWriteThreads = 256;
constexpr int kWriteRows = 16;        // rows of a workgroup at most
constexpr int kMaxHalf = 128;

template <class PAIR>
struct Pairs {
  static __device__ __forceinline__ void unpack(uint32_t w, float* x) {
    const v2f f = __builtin_convertvector(__builtin_bit_cast(PAIR, w), v2f);
    x[0] = f.x;
    x[1] = f.y;
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {   // round to nearest even
    const v2f f = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, PAIR));
  }
};

// A lane-permuted copy of x (inside a row of 16 lanes).
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(dpp_take<CTRL, 0xF>(0u, __float_as_uint(x)));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) { return dpp_take<CTRL, 0xF>(0u, x); }
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

// Sum over the L lanes of a head, in every one of them and in one order.
template <int L>
__device__ __forceinline__ float head_sum(float x) {
  x += dpp<kQuadXor1>(x);
  x += dpp<kQuadXor2>(x);
  x += dpp<kHalfMirror>(x);
  if constexpr (L >= 16) x += dpp<kMirror>(x);
  if constexpr (L >= 32) {
    const uint32_t b = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return x;
}

__device__ __forceinline__ uint32_t to_e4m3(float x, float y) {   // saturating; NaN stays
  x = x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x;
  y = y > 448.0f ? 448.0f : y < -448.0f ? -448.0f : y;
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(x, y, 0, false)) & 0xFFFFu;
}

// Eight E2M1 codes of y, and the scale byte of the 32 numbers that this lane's quad holds. The
// conversion rounds to nearest, ties to the even code, saturating, for every scale.
__device__ __forceinline__ uint32_t to_fp4(const float (&y)[8], uint32_t* byte) {
  uint32_t m = 0;   // magnitudes by their bits: infinities and NaN above every number
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(y[e]) & 0x7FFFFFFFu);
  m = max(m, dpp<kQuadXor1>(m));
  m = max(m, dpp<kQuadXor2>(m));
  const bool bad = m >= 0x7F800000u;
  const uint32_t by = (m >> 23) > 2 ? (m >> 23) - 2 : 0u;   // exponent of the maximum less two, at least 0
  const float scale = __uint_as_float(by << 23);
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, y[0], y[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], scale, 3);
  *byte = bad ? 0xFFu : by;
  return bad ? 0u : w;
}

// One lane's cosines and sines of its 8 dims, the sines with the sign of their term.
struct Turn {
  float c[8], s[8];
  // at: this lane's first pair; `second`: its dims are the pairs' second halves (not interleaved)
  __device__ __forceinline__ void load(const float* cos, const float* sin, int at, bool interleaved, bool second) {
    if (interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[2 * e] = c[2 * e + 1] = cos[at + e];
        s[2 * e] = -sin[at + e];
        s[2 * e + 1] = sin[at + e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = cos[at + e];
        s[e] = second ? sin[at + e] : -sin[at + e];
      }
    }
  }
};

template <class P, int D, int STORE>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(KvWriteArgs a, int rows_of_group, int splits) {
  constexpr int L = D / 8, kAtOnce = kWriteThreads / L;   // lanes of a head, heads at once
  __shared__ float cosines[kWriteRows * kMaxHalf], sines[kWriteRows * kMaxHalf];
  __shared__ int slots[kWriteRows];
  const int split = blockIdx.x % splits;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / splits) * rows_of_group;
  const int rows = static_cast<int>(a.T - t0 < rows_of_group ? a.T - t0 : rows_of_group);
  const int n = a.q.n + a.k.n + a.v.n, items = rows * n;
  const int at = threadIdx.x % L, group = threadIdx.x / L;
  const bool turns = a.inv_freq != nullptr;

  // item i: head i % n of row i / n, queries before keys before values
  auto row_of = [&](int i) { return rows_of_group == 1 ? 0 : i / n; };
  auto source = [&](int i) {
    const int r = row_of(i);
    int h = i - r * n;
    const KvHeads* x = &a.q;
    if (h >= a.q.n) {
      h -= a.q.n;
      x = &a.k;
      if (h >= a.k.n) {
        h -= a.k.n;
        x = &a.v;
      }
    }
    return *reinterpret_cast<const v4u*>(x->x + (t0 + r) * x->x_row + static_cast<int64_t>(h) * (2 * D) + 16 * at);
  };
  const int step = splits * kAtOnce;
  int i = split * kAtOnce + group;
  v4u next = source(min(i, items - 1));

  float wq[8], wk[8];
  if (a.q.n > 0 && a.q.weight != nullptr) {
    const v4u w = reinterpret_cast<const v4u*>(a.q.weight)[at];
#pragma unroll
    for (int e = 0; e < 4; ++e) P::unpack(w[e], &wq[2 * e]);
#pragma unroll
    for (int e = 0; e < 8; ++e) wq[e] += a.q.offset;
  }
  if (a.k.n > 0 && a.k.weight != nullptr) {
    const v4u w = reinterpret_cast<const v4u*>(a.k.weight)[at];
#pragma unroll
    for (int e = 0; e < 4; ++e) P::unpack(w[e], &wk[2 * e]);
#pragma unroll
    for (int e = 0; e < 8; ++e) wk[e] += a.k.offset;
  }
  if (turns)
    for (int e = threadIdx.x; e < rows * a.half; e += kWriteThreads) {
      const int r = e / a.half;
      const int p = (a.turn_pos != nullptr ? a.turn_pos : a.pos)[t0 + r];
      const double whole = static_cast<double>(p) * static_cast<double>(a.inv_freq[e - r * a.half]) * 0.15915494309189533577;
      sincospif(2.0f * static_cast<float>(whole - __builtin_rint(whole)), &sines[e], &cosines[e]);
    }
  if (STORE != kKvStoreRows && threadIdx.x < rows) {
    const int64_t t = t0 + threadIdx.x;
    const int seq = a.seq[t], p = a.pos[t];
    int slot = -1, code = 0;
    if (p != -1) {
      if (seq < 0 || seq >= a.n_seq || p < 0 || p >= kPage * a.max_pages) {
        code = kStBadWindow;
      } else {
        const int page = a.table[seq * a.max_pages + p / kPage];
        if (page < 0 || page >= a.P_phys) code = kStBadPage;
        else slot = page * kPage + p % kPage;
      }
    }
    slots[threadIdx.x] = slot;
    if (code != 0 && split == 0) atomicOr(a.status, code);
  }
  __syncthreads();

  // this lane's place in the rotated range
  const int dim = 8 * at - a.offset;
  const bool turned = turns && dim >= 0 && dim < 2 * a.half;
  const bool second = !a.interleaved && dim >= a.half;
  const int pair = !turned ? 0 : a.interleaved ? dim / 2 : second ? dim - a.half : dim;
  const int other = 4 * ((threadIdx.x & 63) + (!turned || a.interleaved ? 0 : second ? -(a.half / 8) : a.half / 8));
  Turn turn;
  if (turns && rows_of_group == 1) turn.load(cosines, sines, pair, a.interleaved, second);

  for (int i0 = split * kAtOnce; i0 < items; i0 += step, i += step) {   // the same for every lane
    const v4u x = next;
    if (i0 + step < items) next = source(min(i + step, items - 1));
    const bool live = i < items;
    const int mine = min(i, items - 1), r = row_of(mine);
    int h = mine - r * n, kind = 0;
    if (h >= a.q.n) {
      h -= a.q.n;
      kind = 1;
      if (h >= a.k.n) {
        h -= a.k.n;
        kind = 2;
      }
    }
    float y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) P::unpack(x[e], &y[2 * e]);
    if (a.q.weight != nullptr || a.k.weight != nullptr) {
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(y[e], y[e], sum);
      sum = head_sum<L>(sum);
      const float by = 1.0f / __builtin_sqrtf(sum * (1.0f / D) + a.eps);
      if (kind == 0 && a.q.weight != nullptr)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] * by * wq[e];
      if (kind == 1 && a.k.weight != nullptr)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] * by * wk[e];
    }
    if (turns) {
      float z[8];
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = y[e ^ 1];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          z[e] = __int_as_float(__builtin_amdgcn_ds_bpermute(other, __float_as_int(y[e])));
      }
      if (turned && kind < 2) {
        if (rows_of_group > 1) turn.load(cosines + r * a.half, sines + r * a.half, pair, a.interleaved, second);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(y[e], turn.c[e], z[e] * turn.s[e]);
      }
    }
    const bool same = kind == 2 || (kind == 1 && !turns && a.k.weight == nullptr);   // copied bit by bit
    uint32_t codes = 0, byte = 0;
    if constexpr (STORE == kKvStoreFp4) codes = to_fp4(y, &byte);
    if (!live) continue;
    const v4u packed = {P::pack(y[0], y[1]), P::pack(y[2], y[3]), P::pack(y[4], y[5]), P::pack(y[6], y[7])};
    if (kind == 0 || STORE == kKvStoreRows) {
      const KvHeads& to = kind == 0 ? a.q : a.k;
      *reinterpret_cast<v4u*>(to.out + (t0 + r) * to.out_row + static_cast<int64_t>(h) * (2 * D) + 16 * at) = packed;
      continue;
    }
    if constexpr (STORE != kKvStoreRows) {
      const int slot = slots[r];
      if (slot < 0) continue;
      const int64_t page = slot / kPage, pos = slot % kPage;
      const KvPages& to = kind == 1 ? a.kc : a.vc;
      char* base = to.p + page * to.page + pos * to.pos + h * to.head;
      if constexpr (STORE == kKvStoreSame) {
        *reinterpret_cast<v4u*>(base + 16 * at) = same ? x : packed;
      } else if constexpr (STORE == kKvStoreE4m3) {
        const float by = kind == 1 ? a.k_scale : a.v_scale;
        *reinterpret_cast<v2u*>(base + 8 * at) = v2u{to_e4m3(y[0] / by, y[1] / by) | to_e4m3(y[2] / by, y[3] / by) << 16,
                                                     to_e4m3(y[4] / by, y[5] / by) | to_e4m3(y[6] / by, y[7] / by) << 16};
      } else {
        *reinterpret_cast<uint32_t*>(base + 4 * at) = codes;
        const KvPages& scale = kind == 1 ? a.ks : a.vs;
        if (at % 4 == 0) scale.p[page * scale.page + pos * scale.pos + h * scale.head + at / 4] = static_cast<char>(byte);
      }
    }
  }
}

template <class P, int D, int STORE>
void write_on(const KvWriteArgs& a, hipStream_t st) {
  constexpr int kAtOnce = kWriteThreads / (D / 8);
  const int64_t n = static_cast<int64_t>(a.q.n) + a.k.n + a.v.n;
  // few heads: several rows to a workgroup, as long as there are workgroups for every compute unit twice
  int64_t rows = n < kAtOnce ? (2 * kAtOnce + n - 1) / n : 1;
  if (rows > kWriteRows) rows = kWriteRows;
  if (rows > (a.T + 511) / 512) rows = (a.T + 511) / 512;
  // few rows: a row's heads over several workgroups
  const int64_t passes = (rows * n + kAtOnce - 1) / kAtOnce, groups = (a.T + rows - 1) / rows;
  int64_t splits = (2048 + groups - 1) / groups;
  if (splits > passes) splits = passes;
  kv_write_kernel<P, D, STORE><<<dim3(static_cast<unsigned>(groups * splits)), dim3(kWriteThreads), 0, st>>>(
      a, static_cast<int>(rows), static_cast<int>(splits));
}

template <class P, int D>
void by_store(const KvWriteArgs& a, hipStream_t st) {
  if (a.store == kKvStoreRows) write_on<P, D, kKvStoreRows>(a, st);
  else if (a.store == kKvStoreSame) write_on<P, D, kKvStoreSame>(a, st);
  else if (a.store == kKvStoreE4m3) write_on<P, D, kKvStoreE4m3>(a, st);
  else write_on<P, D, kKvStoreFp4>(a, st);
}

template <class P>
void by_dim(const KvWriteArgs& a, hipStream_t st) {
  if (a.D == 64) by_store<P, 64>(a, st);
  else if (a.D == 128) by_store<P, 128>(a, st);
  else by_store<P, 256>(a, st);
}

}  // namespace

hipError_t launch_kv_write(const KvWriteArgs& a, hipStream_t st) {
  if (a.type == MQA_KV_BF16) by_dim<Pairs<bf16x2>>(a, st);
  else by_dim<Pairs<f16x2>>(a, st);
  return hipGetLastError();
}

}  // namespace mqa
