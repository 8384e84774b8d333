// New heads on their way into use (gfx950): norm and rotation of queries and keys,
// keys and values into the paged cache in 16, 8 or 4 bits.
//
// Mathematics. y = x / sqrt(mean(x^2) + eps) * (w + offset); pair (a, b) of dims turns by
// t = position * inv_freq: (a cos t - b sin t, b cos t + a sin t). t is taken in 64 bits as
// turns of a circle, of which the fraction alone, 1/2 at most, goes on in 32: its rounding
// is an angle of pi 2^-25 at most, and the product's own 2^-51 of t. (In 32 bits throughout, an
// angle of a million has neighbours 0.06 rad away and is off by half of that.)
//
// Bound by memory: a head's numbers are read and written once. A lane holds 8 neighbouring
// dims of a head (16 bytes), D / 8 lanes a head; sums go over them by lane permutes, and a
// pair's other half comes from the lane that has it. A wave takes 512 / D heads of one kind
// (queries, keys or values) at a time, so that what depends on the kind is scalar, with the
// next ones on their way. A workgroup takes some rows with all their heads (or, where rows
// are few, a part of the heads), so that a row's cosines and sines, and its place in the
// cache, are found once, by one thread each, and lie in LDS. 64 registers, so that a compute
// unit holds 32 waves: 8192 rows of 40 + 8 heads of 128 dims take 43 us (201 MB, 4.7 TB/s; a
// large copy does 4.9), with 80 registers 46 us, and two blocks ahead instead of one 45 us.
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
typedef float v4f __attribute__((ext_vector_type(4)));
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

// y / by to within what 8 bits can tell (`by` between 2^-100 and 2^100, one_by its reciprocal): one step of
// Newton's division behind the product, whose remainder is exact. Far out the quotient is held at 1024 first, so
// that an infinity saturates too; NaN stays, and a zero's sign.
__device__ __forceinline__ float divide(float y, float by, float one_by) {
  const float q = __builtin_amdgcn_fmed3f(y * one_by, -1024.0f, 1024.0f);
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, by, y), one_by, q), y);
}

// 1 / sqrt(m): one instruction (to an ulp), but for the numbers that it takes for zero.
__device__ __forceinline__ float one_by_root(float m) {
  return m >= 0x1p-126f ? __builtin_amdgcn_rsqf(m) : 1.0f / __builtin_sqrtf(m);
}

template <class P, int D, int STORE>
__global__ void __launch_bounds__(kWriteThreads, 8) kv_write_kernel(KvWriteArgs a, int rows_of_group, int splits) {
  constexpr int L = D / 8, G = 64 / L;   // lanes of a head, heads of a block
  __shared__ v4f cosines[kWriteRows * kMaxHalf / 4], sines[kWriteRows * kMaxHalf / 4];
  __shared__ int64_t places[4][kWriteRows];   // of a row's keys and values and of their scales, in bytes; -1: padding
  const int split = blockIdx.x % splits;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / splits) * rows_of_group;
  const int rows = static_cast<int>(a.T - t0 < rows_of_group ? a.T - t0 : rows_of_group);
  const bool one_row = rows_of_group == 1;
  const int lane = threadIdx.x & 63, at = lane % L;
  const bool turns = a.inv_freq != nullptr;

  // Blocks: G heads of one kind each, queries before keys before values, of the rows together.
  const int end_q = (rows * a.q.n + G - 1) / G, end_k = end_q + (rows * a.k.n + G - 1) / G;
  const int blocks = end_k + (rows * a.v.n + G - 1) / G, step = splits * (kWriteThreads / 64);
  struct Head {
    int r, h;
    bool live;
  };
  auto kind_of = [&](int b) { return b < end_q ? 0 : b < end_k ? 1 : 2; };
  auto head_of = [&](int b, int kind) -> Head {
    const int n = kind == 0 ? a.q.n : kind == 1 ? a.k.n : a.v.n;
    const int i = (b - (kind == 0 ? 0 : kind == 1 ? end_q : end_k)) * G + lane / L, all = rows * n;
    const int j = min(i, all - 1);   // a lane behind the last head reads that one and writes nothing
    // j < 2^20: (j + 1/2) / n is 2^-17 or more away from the next whole number, 32 bits err by less than 2^-18
    const int r = one_row ? 0 : static_cast<int>((static_cast<float>(j) + 0.5f) * __builtin_amdgcn_rcpf(static_cast<float>(n)));
    return {r, j - r * n, i < all};
  };
  auto load = [&](int b) {
    const int kind = kind_of(b);
    const Head x = head_of(b, kind);
    const KvHeads& from = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const uint32_t off = static_cast<uint32_t>(x.r) * static_cast<uint32_t>(from.x_row) + x.h * (2 * D) + 16 * at;
    return *reinterpret_cast<const v4u*>(from.x + t0 * from.x_row + off);
  };
  int b = split * (kWriteThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  v4u next = {};
  if (b < blocks) next = load(b);

  v4u wq = {}, wk = {};
  if (a.q.n > 0 && a.q.weight != nullptr) wq = reinterpret_cast<const v4u*>(a.q.weight)[at];
  if (a.k.n > 0 && a.k.weight != nullptr) wk = reinterpret_cast<const v4u*>(a.k.weight)[at];
  if (turns)
    for (int e = threadIdx.x; e < rows * a.half; e += kWriteThreads) {
      const int r = e / a.half;
      const int p = (a.turn_pos != nullptr ? a.turn_pos : a.pos)[t0 + r];
      const double whole = static_cast<double>(p) * static_cast<double>(a.inv_freq[e - r * a.half]) * 0.15915494309189533577;
      sincospif(2.0f * static_cast<float>(whole - __builtin_rint(whole)), reinterpret_cast<float*>(sines) + e,
                reinterpret_cast<float*>(cosines) + e);
    }
  if (STORE != kKvStoreRows && threadIdx.x < rows) {
    const int64_t t = t0 + threadIdx.x;
    const int seq = a.seq[t], p = a.pos[t];
    int64_t page = -1, pos = 0;
    int code = 0;
    if (p != -1) {
      if (seq < 0 || seq >= a.n_seq || p < 0 || p >= kPage * a.max_pages) {
        code = kStBadWindow;
      } else {
        page = a.table[seq * a.max_pages + p / kPage];
        pos = p % kPage;
        if (page < 0 || page >= a.P_phys) {
          code = kStBadPage;
          page = -1;
        }
      }
    }
    places[0][threadIdx.x] = page < 0 ? -1 : page * a.kc.page + pos * a.kc.pos;
    places[1][threadIdx.x] = page < 0 ? -1 : page * a.vc.page + pos * a.vc.pos;
    if constexpr (STORE == kKvStoreFp4) {
      places[2][threadIdx.x] = page * a.ks.page + pos * a.ks.pos;
      places[3][threadIdx.x] = page * a.vs.page + pos * a.vs.pos;
    }
    if (code != 0 && split == 0) atomicOr(a.status, code);
  }
  __syncthreads();

  // this lane's place in the rotated range
  const int dim = 8 * at - a.offset;
  const bool turned = turns && dim >= 0 && dim < 2 * a.half;
  const bool second = !a.interleaved && dim >= a.half;   // its dims are the pairs' second halves
  const int pair = !turned ? 0 : a.interleaved ? dim / 2 : second ? dim - a.half : dim;
  const int other = 4 * (lane + (!turned || a.interleaved ? 0 : second ? -(a.half / 8) : a.half / 8));
  v4f c0, c1, s0, s1;
  auto take_turn = [&](int r) {
    const int i = (r * a.half + pair) / 4, j = a.interleaved ? i : i + 1;
    c0 = cosines[i];
    c1 = cosines[j];
    s0 = sines[i];
    s1 = sines[j];
    if (second) {
      s0 = -s0;
      s1 = -s1;
    }
  };
  const bool by_one = a.k_scale >= 0x1p-100f && a.k_scale <= 0x1p100f && a.v_scale >= 0x1p-100f && a.v_scale <= 0x1p100f;

  for (; b < blocks; b += step) {
    const v4u x = next;
    if (b + step < blocks) next = load(b + step);
    const int kind = kind_of(b);
    const Head to = head_of(b, kind);
    float y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) P::unpack(x[e], &y[2 * e]);
    const bool norm = kind == 0 ? a.q.weight != nullptr : kind == 1 && a.k.weight != nullptr;
    if (norm) {
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(y[e], y[e], sum);
      const float by = one_by_root(head_sum<L>(sum) * (1.0f / D) + a.eps);
      const v4u weight = kind == 0 ? wq : wk;
      const float offset = kind == 0 ? a.q.offset : a.k.offset;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float w[2];
        P::unpack(weight[e / 2], w);
        y[e] = y[e] * by * (w[0] + offset);
        y[e + 1] = y[e + 1] * by * (w[1] + offset);
      }
    }
    if (turns && kind < 2) {
      float z[8];
      if (!a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          z[e] = __int_as_float(__builtin_amdgcn_ds_bpermute(other, __float_as_int(y[e])));
      }
      if (turned) {
        take_turn(to.r);
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = y[2 * e], v = y[2 * e + 1];
            y[2 * e] = __builtin_fmaf(u, c0[e], -(v * s0[e]));
            y[2 * e + 1] = __builtin_fmaf(v, c0[e], u * s0[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] = __builtin_fmaf(y[e], c0[e], -(z[e] * s0[e]));
            y[4 + e] = __builtin_fmaf(y[4 + e], c1[e], -(z[4 + e] * s1[e]));
          }
        }
      }
    }
    uint32_t codes = 0, byte = 0;
    if constexpr (STORE == kKvStoreFp4) codes = to_fp4(y, &byte);
    if (!to.live) continue;
    const v4u packed = {P::pack(y[0], y[1]), P::pack(y[2], y[3]), P::pack(y[4], y[5]), P::pack(y[6], y[7])};
    if (kind == 0 || STORE == kKvStoreRows) {
      const KvHeads& out = kind == 0 ? a.q : a.k;
      const uint32_t off = static_cast<uint32_t>(to.r) * static_cast<uint32_t>(out.out_row) + to.h * (2 * D) + 16 * at;
      *reinterpret_cast<v4u*>(out.out + t0 * out.out_row + off) = packed;
      continue;
    }
    if constexpr (STORE != kKvStoreRows) {
      const KvPages& pages = kind == 1 ? a.kc : a.vc;
      const int64_t place = places[kind - 1][to.r];
      if (place < 0) continue;
      char* base = pages.p + place + to.h * pages.head;
      if constexpr (STORE == kKvStoreSame) {
        const bool same = kind == 2 || (!turns && !norm);   // copied bit by bit
        *reinterpret_cast<v4u*>(base + 16 * at) = same ? x : packed;
      } else if constexpr (STORE == kKvStoreE4m3) {
        const float by = kind == 1 ? a.k_scale : a.v_scale;
        if (by_one) {
          const float one_by = 1.0f / by;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = divide(y[e], by, one_by);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = y[e] / by;
        }
        *reinterpret_cast<v2u*>(base + 8 * at) =
            v2u{to_e4m3(y[0], y[1]) | to_e4m3(y[2], y[3]) << 16, to_e4m3(y[4], y[5]) | to_e4m3(y[6], y[7]) << 16};
      } else {
        *reinterpret_cast<uint32_t*>(base + 4 * at) = codes;
        const KvPages& scale = kind == 1 ? a.ks : a.vs;
        if (at % 4 == 0) scale.p[places[kind + 1][to.r] + to.h * scale.head + at / 4] = static_cast<char>(byte);
      }
    }
  }
}

template <class P, int D, int STORE>
void write_on(const KvWriteArgs& a, hipStream_t st) {
  constexpr int G = 512 / D, kWaves = kWriteThreads / 64;
  const auto blocks_of = [&](int64_t rows) {
    return (rows * a.q.n + G - 1) / G + (rows * a.k.n + G - 1) / G + (rows * a.v.n + G - 1) / G;
  };
  // Two rows to a workgroup, or more until each wave has two blocks, as long as every compute unit keeps a workgroup:
  // what comes before the first block (position, angles, block table) is then paid once for them (8192 rows of 48
  // heads: 47.5 us by one row, 46.3 by two, 50.2 by four, whose workgroups end too unevenly).
  int64_t rows = 1;
  while (rows < kWriteRows && a.T >= 512 * rows && (rows < 2 || blocks_of(rows) < 2 * kWaves)) rows *= 2;
  // The kernel's offsets inside a group are held in 32 bits. Managed memory may be larger than the card's, and rows of it farther apart.
  int64_t widest = 0;
  for (const int64_t row : {a.q.x_row, a.q.out_row, a.k.x_row, a.k.out_row, a.v.x_row}) widest = row > widest ? row : widest;
  while (rows > 1 && rows * widest > 0x7FFFFFFF) rows /= 2;
  // few rows: their heads over several workgroups, four to a compute unit (1001 rows of 18 heads of 256 dims: 8.1 us,
  // 9.9 with eight: workgroups start at about one in a nanosecond)
  const int64_t passes = (blocks_of(rows) + kWaves - 1) / kWaves, groups = (a.T + rows - 1) / rows;
  int64_t splits = (1024 + groups - 1) / groups;
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
