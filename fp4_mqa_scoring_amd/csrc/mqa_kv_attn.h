// What the attention kernels over the paged key-value cache share (gfx950): matrix operands and a wave's running
// sums, the joining of partial results, the plan that cuts a batch into shares. The mathematics
// stands at the head of mqa_kv_attn.hip (16- and 8-bit caches); mqa_kv_fp4.hip has the caches in 4 bits.
#pragma once

#include "mqa_fp4_topk.h"
#include "mqa_kv.h"
#include "mqa_kv_cache.h"
#include "mqa_device.h"

namespace mqa {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

template <bool FIRST, class A, class B>
struct Pick { typedef A type; };
template <class A, class B>
struct Pick<false, A, B> { typedef B type; };

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kTilePos = 32;
constexpr float kLn2 = 0.69314718055994530942f;

// kTop: the largest weight is kept at 2^kTop. bf16's range is that of 32 bits, so 1 will do. fp16's normal numbers
// end at 2^-14, and where one position outweighs many others the weights of these, which count together, would be lost to
// its subnormal ones (4,096 of 2^-24.7 each: outputs wrong by 13 %); below 2^15 they lie at 2^-29 and less.
struct Bf16 {
  static constexpr int kTop = 0;
  static __device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
  }
  static __device__ __forceinline__ v4f mfma(v2u a, v2u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, a), __builtin_bit_cast(s16x4, b), c, 0,
                                                     0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {   // round to nearest even
    const v2f f = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
  }
  template <bool HI>
  static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {    // exact
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  }
};

struct Fp16 {
  static constexpr int kTop = 15;
  static __device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                  0, 0);
  }
  static __device__ __forceinline__ v4f mfma(v2u a, v2u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(f16x4, a), __builtin_bit_cast(f16x4, b), c, 0, 0,
                                                 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const v2f f = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
  }
  template <bool HI>
  static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {    // exact
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
  }
};

// Maxima by hand: fmaxf quiets either operand first, an instruction each. A NaN gives way to a number here too.
__device__ __forceinline__ float max2(float x, float y) {
  float r;
  __asm__("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(x), "v"(y));
  return r;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  __asm__("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
  return r;
}

// Maximum / sum over the four lane groups of 16 (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float groups_max(float x) {
  const uint32_t b = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t y = __float_as_uint(max2(__uint_as_float(r[0]), __uint_as_float(r[1])));
  const auto s = __builtin_amdgcn_permlane16_swap(y, y, false, false);
  return max2(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

__device__ __forceinline__ float groups_sum(float x) {
  const uint32_t b = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t y = __float_as_uint(__uint_as_float(r[0]) + __uint_as_float(r[1]));
  const auto s = __builtin_amdgcn_permlane16_swap(y, y, false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// log of a sum of weights held under the running maximum m (log2 domain). kTop, which m lacks and the sum has too
// much, goes from one to the other first: the logarithm of a sum near one is small, and so is its rounding.
template <class T>
__device__ __forceinline__ float lse_of(float m, float sum) {
  if constexpr (T::kTop == 0) return (m + __builtin_amdgcn_logf(sum)) * kLn2;
  constexpr float kBy = 1.0f / (1 << T::kTop);
  return ((m + static_cast<float>(T::kTop)) + __builtin_amdgcn_logf(sum * kBy)) * kLn2;
}

// Passes matrix results on once they can be read, which a 16x16x32 product's can after
// eight wait states. Ordinary code waits for them by itself, but behind a branch that
// overwrites a part of them under a mask (the edge of a window) this compiler has left out
// the wait for the other parts, and a maximum was taken of what the registers held before.
template <int N>
__device__ __forceinline__ void settle(v4f (&s)[N][1]) {
  static_assert(N == 1, "one tile of 16 positions goes with one of queries");
  __asm__ __volatile__("s_nop 7" : "+v"(s[0][0]));
}
template <int N>
__device__ __forceinline__ void settle(v4f (&s)[N][2]) {
  if constexpr (N == 1) {
    __asm__ __volatile__("s_nop 7" : "+v"(s[0][0]), "+v"(s[0][1]));
  } else if constexpr (N == 2) {
    __asm__ __volatile__("s_nop 7" : "+v"(s[0][0]), "+v"(s[0][1]), "+v"(s[1][0]), "+v"(s[1][1]));
  } else {
    static_assert(N == 4, "one, two or four");
    __asm__ __volatile__("s_nop 7"
                         : "+v"(s[0][0]), "+v"(s[0][1]), "+v"(s[1][0]), "+v"(s[1][1]), "+v"(s[2][0]), "+v"(s[2][1]),
                           "+v"(s[3][0]), "+v"(s[3][1]));
  }
}

// The registers and steps of one wave: NQ tiles of 16 query heads of one row and
// key head, POS (16 or 32) positions at a time.
//
// The running maximum m is the largest score seen less kBias (log2 domain), so that the largest weight is 2^kTop at most
// (bf16 with SLACK 8: 2^8), and moves when it is passed by more than SLACK. 0: the largest weight is a power of two (to
// 2^-20), which the rounding of the weights to 16 bits leaves alone, and where few weights count that is most of the
// rounding's error (bf16: relative error of the output 0.0018, of its own rounding alone 0.0017, with SLACK 8 0.0022). 8:
// the relative rounding is the same, and the sums are multiplied once or twice instead of in nearly every one of the first tiles.
template <class T, bool E4M3, int D, int NQ, int POS = 32, bool QL = false, int SLACK = 0>
struct Wave {
  static constexpr int kPositions = POS;
  static constexpr int kBytes = E4M3 ? 1 : 2;
  static constexpr int kChunks = D / 32;                 // matrix steps over the dims
  static constexpr int kLoads = D * kBytes / 64;         // 16-byte key loads per lane and position
  static constexpr int kDims = D / 16;                   // dims of a position that a lane's values hold
  static constexpr int kWords = kDims * kBytes / 4;      // and their registers
  static constexpr int kTiles = POS / 16;                // matrix tiles of positions
  static constexpr int kMine = POS / 4;                  // positions whose weights and values this lane holds
  static constexpr bool kShared = QL;                    // the queries lie in LDS
  static constexpr int kBias = T::kTop == 0 ? 0 : T::kTop - SLACK;
  typedef typename Pick<POS == 32, v4u, v2u>::type P;    // weights of kMine positions, packed

  v4u q[kShared ? 1 : NQ][kShared ? 1 : kChunks];
  const v4u* q_lds;
  v4u k[kTiles][kLoads];
  uint32_t v[kMine][kWords];
  v4f o[NQ][kDims];
  float m[NQ];   // running maximum in the log2 domain, equal in the four lane groups
  float l[NQ];   // this lane's part of the sum
  int lane, col, grp;

  __device__ __forceinline__ void init() {
    lane = threadIdx.x & 63;
    col = lane & 15;
    grp = lane >> 4;
  }

  __device__ __forceinline__ void start() {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      m[n] = -__builtin_inff();
      l[n] = 0.0f;
#pragma unroll
      for (int t = 0; t < kDims; ++t) o[n][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }

  // Which of the POS positions this lane's j-th one is.
  __device__ __forceinline__ int mine(int j) const { return 16 * (j >> 2) + 4 * grp + (j & 3); }

  // This lane's part of step c of query tile n: of heads [0, rows) at `p`, one after
  // another, the dims that the keys' pieces hold there.
  __device__ __forceinline__ v4u query(const char* p, int n, int c, int rows, uint32_t keep, uint32_t flip) const {
    const int h = 16 * n + col;
    const int dim = E4M3 ? 64 * (c >> 1) + 16 * grp + 8 * (c & 1) : 32 * c + 8 * grp;
    v4u x = {0, 0, 0, 0};
    if (h < rows) x = *reinterpret_cast<const v4u*>(p + (static_cast<int64_t>(h) * D + dim) * 2);
    return (x & v4u{keep, keep, keep, keep}) ^ v4u{flip, flip, flip, flip};
  }

  // Loads the queries: into registers, or by the whole workgroup into `lds`
  // (NQ * kChunks * 64 of it; a barrier must follow, and one precede).
  __device__ __forceinline__ void load_q(const char* p, int rows, uint32_t keep, uint32_t flip, v4u* lds) {
    if constexpr (kShared) {
      q_lds = lds + lane;
      for (int x = threadIdx.x >> 6; x < NQ * kChunks; x += blockDim.x >> 6)
        lds[64 * x + lane] = query(p, x / kChunks, x % kChunks, rows, keep, flip);
    } else {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < kChunks; ++c) q[n][c] = query(p, n, c, rows, keep, flip);
    }
  }

  // Position a * 16 + col is at `p`.
  __device__ __forceinline__ void load_k(int a, const char* p) {
#pragma unroll
    for (int c = 0; c < kLoads; ++c) k[a][c] = *reinterpret_cast<const v4u*>(p + 64 * c + 16 * grp);
  }

  // Position mine(j) is at `p`.
  __device__ __forceinline__ void load_v(int j, const char* p) {
    const char* at = p + col * (kWords * 4);
    if constexpr (kWords == 1) {
      v[j][0] = *reinterpret_cast<const uint32_t*>(at);
    } else if constexpr (kWords == 2) {
      const v2u x = *reinterpret_cast<const v2u*>(at);
      v[j][0] = x.x;
      v[j][1] = x.y;
    } else {
#pragma unroll
      for (int e = 0; e < kWords; e += 4) {
        const v4u x = *reinterpret_cast<const v4u*>(at + 4 * e);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][e + i] = x[i];
      }
    }
  }

  __device__ __forceinline__ void scores(v4f (&s)[NQ][kTiles]) {
    const v4u* queries = q_lds;
    if constexpr (kShared) __asm__ __volatile__("" : "+v"(queries));   // read anew for every tile, not kept in registers
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int a = 0; a < kTiles; ++a) s[n][a] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      v4u x[kTiles];
#pragma unroll
      for (int a = 0; a < kTiles; ++a) {
        if constexpr (E4M3) {
          const uint32_t w0 = k[a][c >> 1][2 * (c & 1)], w1 = k[a][c >> 1][2 * (c & 1) + 1];
          x[a] = v4u{T::template from_e4m3<false>(w0), T::template from_e4m3<true>(w0),
                     T::template from_e4m3<false>(w1), T::template from_e4m3<true>(w1)};
        } else {
          x[a] = k[a][c];
        }
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        v4u y;
        if constexpr (kShared) y = queries[(n * kChunks + c) * 64];
        else y = q[n][c];
#pragma unroll
        for (int a = 0; a < kTiles; ++a) s[n][a] = T::mfma(x[a], y, s[n][a]);
      }
    }
    settle(s);
  }

  // The same bits, known only where this stands: what is made of them stays behind the branch around it.
  static __device__ __forceinline__ uint32_t here(uint32_t inside) {
    __asm__ __volatile__("" : "+v"(inside));
    return inside;
  }

  // Scores to weights; `inside` bit j says whether this lane's j-th position counts
  // (looked at where `edge`). Returns the weights packed as the second product's operand.
  __device__ __forceinline__ void weights(v4f (&s)[NQ][kTiles], float c, bool edge, uint32_t inside, P (&p)[NQ]) {
    float top[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      if (edge) {   // a score of -infinity is a weight of 0, as c > 0
        const uint32_t in = here(inside);
#pragma unroll
        for (int j = 0; j < kMine; ++j) s[n][j >> 2][j & 3] = (in >> j & 1) ? s[n][j >> 2][j & 3] : -__builtin_inff();
      }
      float x = max2(max3(s[n][0][0], s[n][0][1], s[n][0][2]), s[n][0][3]);
#pragma unroll
      for (int a = 1; a < kTiles; ++a) x = max3(max3(x, s[n][a][0], s[n][a][1]), s[n][a][2], s[n][a][3]);
      top[n] = x;
    }
    bool rise = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      top[n] = kBias == 0 ? groups_max(top[n]) * c : __builtin_fmaf(groups_max(top[n]), c, static_cast<float>(-kBias));
      rise |= top[n] > m[n] + static_cast<float>(SLACK);
    }
    if (__any(rise)) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float to = fmaxf(m[n], top[n]);
        const float f = to == m[n] ? 1.0f : __builtin_amdgcn_exp2f(m[n] - to);
        m[n] = to;
        l[n] *= f;
#pragma unroll
        for (int t = 0; t < kDims; ++t) o[n][t] *= f;
      }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const float ref = m[n] == -__builtin_inff() ? 0.0f : m[n];
      float w[kMine];
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][j >> 2][j & 3], c, -ref));
      }
      float sum = (w[0] + w[1]) + (w[2] + w[3]);
      if constexpr (POS == 32) sum += (w[4] + w[5]) + (w[6] + w[7]);
      l[n] += sum;
#pragma unroll
      for (int j = 0; j < kMine / 2; ++j) p[n][j] = T::pack(w[2 * j], w[2 * j + 1]);
    }
  }

  // Dims 2 e and 2 e + 1 of this lane's position j, in the query's type.
  __device__ __forceinline__ uint32_t dims_pair(int j, int e) {
    if constexpr (E4M3) {
      return (e & 1) ? T::template from_e4m3<true>(v[j][e >> 1]) : T::template from_e4m3<false>(v[j][e >> 1]);
    } else {
      return v[j][e];
    }
  }

  // Values outside the window are whatever the cache holds there, NaN perhaps.
  __device__ __forceinline__ void clear_outside(uint32_t inside) {
    inside = here(inside);
#pragma unroll
    for (int j = 0; j < kMine; ++j)
#pragma unroll
      for (int e = 0; e < kWords; ++e) v[j][e] = (inside >> j & 1) ? v[j][e] : 0u;
  }

  __device__ __forceinline__ void add_values(const P (&p)[NQ]) {
#pragma unroll
    for (int e = 0; e < kDims / 2; ++e) {
      uint32_t w[kMine];
#pragma unroll
      for (int j = 0; j < kMine; ++j) w[j] = dims_pair(j, e);
      P even, odd;
#pragma unroll
      for (int jj = 0; jj < kMine / 2; ++jj) {
        even[jj] = __builtin_amdgcn_perm(w[2 * jj + 1], w[2 * jj], 0x05040100u);   // low halves
        odd[jj] = __builtin_amdgcn_perm(w[2 * jj + 1], w[2 * jj], 0x07060302u);    // high halves
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        o[n][2 * e] = T::mfma(even, p[n], o[n][2 * e]);
        o[n][2 * e + 1] = T::mfma(odd, p[n], o[n][2 * e + 1]);
      }
    }
  }
};

// A barrier for what lies in LDS alone: loads from memory and stores to it that are on their way stay so.
__device__ __forceinline__ void lds_barrier() { __asm__ __volatile__("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Offset of a slot in units of 16 bytes, of which the strides are multiples. A page's is below 2^36 bytes, 63
// positions' below 2^31: one 32-bit multiplication and one of 24 bits.
__device__ __forceinline__ uint64_t slot_offset(int slot, uint32_t page, uint32_t pos) {
  const uint32_t s = static_cast<uint32_t>(slot);
  return static_cast<uint64_t>(s >> 6) * page + __umul24(s & 63, pos);
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p));
}

// --- decode form --------------------------------------------------------------

// Pages that row r's window touches; 0 for an empty one; code < 0 where the row
// is invalid (0 pages then).
__device__ __forceinline__ int row_pages(const KvAttnArgs& a, int64_t r, int* code) {
  const int seq = a.seq_of_row[r], start = a.row_start[r], end = a.row_end[r];
  *code = 0;
  if (seq < 0 || seq >= a.n_seq || start < 0 || end < start || end > 64 * a.max_pages) {
    *code = kCodeBadWindow;
    return 0;
  }
  if (start == end) return 0;
  if (a.P_phys == 0) {
    *code = kCodeBadPage;
    return 0;
  }
  return (end + 63) / 64 - start / 64;
}

__device__ __forceinline__ void report(const KvAttnArgs& a, int code) {
  if (code == kCodeBadWindow) atomicOr(a.status, kStBadWindow);
  if (code == kCodeBadPage) atomicOr(a.status, kStBadPage);
}

// Inclusive sum over the workgroup's threads; `total` gets the sum of all.
template <int WAVES>
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* wave_sums, int64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(static_cast<long long>(x), d, 64);
    if (lane >= d) x += y;
  }
  if (lane == 63) wave_sums[wave] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    if (i < wave) before += wave_sums[i];
    all += wave_sums[i];
  }
  *total = all;
  return x + before;
}

// prefix[r] = pages of the rows before r, for batches of more than kKvPlanRows rows.
__global__ void __launch_bounds__(1024) kv_plan_kernel(KvAttnArgs a) {
  __shared__ int64_t sums[16];
  int64_t base = 0;
  for (int64_t r0 = 0; r0 < a.Q; r0 += 1024) {
    const int64_t r = r0 + threadIdx.x;
    int code = 0;
    const int64_t n = r < a.Q ? row_pages(a, r, &code) : 0;
    report(a, code);
    int64_t total;
    const int64_t upto = base + block_scan<16>(n, sums, &total);
    if (r < a.Q) a.prefix[r] = upto - n;
    base += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) a.prefix[a.Q] = base;
}

// Pages of one (row, head group) are its units of work; a workgroup takes a share of consecutive units of all
// (row, head group) pairs laid end to end: an equal one, or where that would make many short parts the power of two
// nearest to sqrt(units * join_cost), at which the parts and their joining take the least together (decode_on() has the
// figures). In whole numbers: the launches of one call must agree on it.
__device__ __forceinline__ int64_t unit_share(const KvAttnArgs& a, int64_t units, int64_t groups) {
  const int64_t equal = (units + groups - 1) / groups;
  const uint32_t some = static_cast<uint32_t>(units < 1 << 24 ? units : 1 << 24);
  // At most 2^24 times a cost of 2^23 at most (4 bits, many key heads): x is at most 2^31, and s at most 2^15.
  const uint32_t x = static_cast<uint32_t>(static_cast<uint64_t>(some) * a.join_cost >> 16);
  const int64_t s = x < 2 ? 1 : 1 << ((32 - __builtin_clz(x - 1)) >> 1);   // the least with 2 s^2 >= x
  return equal > s ? equal : s;
}

// Integers that no kernel of this launch writes, read through the scalar cache.
typedef const __attribute__((address_space(4))) int32_t* ScalarInts;
__device__ __forceinline__ ScalarInts scalar_ints(const int32_t* p) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32));
  return reinterpret_cast<ScalarInts>(static_cast<uintptr_t>(static_cast<uint64_t>(hi) << 32 | lo));
}

// The plan of a decode launch, the same in every workgroup: pages before each row.
template <int WAVES>
struct Plan {
  int64_t prefix_lds[kKvPlanRows + 1];
  int64_t sums[WAVES];

  // Returns the prefix (in LDS, or the one that kv_plan_kernel left in the workspace).
  __device__ __forceinline__ const int64_t* make(const KvAttnArgs& a) {
    if (a.Q > kKvPlanRows) return a.prefix;
    // A thread's rows one after another, two trips to memory each, the sequence and then the window: two where the batch
    // has one row, up to eight with four waves and four rows or more. (One short sequence: 4,400 clocks with what follows here.)
    constexpr int kPer = kKvPlanRows / (64 * WAVES);
    const bool first = blockIdx.x == 0;
    int64_t n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t r = kPer * threadIdx.x + i;
      int code = 0;
      n[i] = r < a.Q ? row_pages(a, r, &code) : 0;
      if (first) report(a, code);
      sum += n[i];
    }
    int64_t total;
    int64_t at = block_scan<WAVES>(sum, sums, &total) - sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t r = kPer * threadIdx.x + i;
      if (r <= a.Q) {
        prefix_lds[r] = at;
        if (first) a.prefix[r] = at;
      }
      at += n[i];
    }
    if (threadIdx.x == 0) {
      prefix_lds[a.Q] = total;
      if (first) a.prefix[a.Q] = total;
    }
    __syncthreads();
    return prefix_lds;
  }
};

// A workgroup's run of units, one (row, head group) at a time.
struct Segment {
  int64_t r;        // row
  int g;            // head group
  int pa, pb;       // pages [pa, pb) of the row's n
  int64_t n;
  int seq, start, end;

  // The segment at unit `cur`, which it advances.
  template <class ARGS>
  __device__ __forceinline__ void take(ARGS& a, const int64_t* prefix, int64_t gh, int64_t* cur, int64_t stop) {
    // the row that the unit belongs to: the last one whose prefix is not above it
    int64_t lo = 0, hi = a.Q;
    const int64_t page_unit = *cur / gh;
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (prefix[mid] <= page_unit) lo = mid;
      else hi = mid;
    }
    r = __builtin_amdgcn_readfirstlane(static_cast<int>(lo));   // Q < 2^24
    n = prefix[r + 1] - prefix[r];
    const int64_t in_row = *cur - prefix[r] * gh;
    g = __builtin_amdgcn_readfirstlane(static_cast<int>(gh == 1 ? 0 : in_row / n));
    pa = __builtin_amdgcn_readfirstlane(static_cast<int>(in_row - g * n));
    const int64_t left = stop - *cur;
    pb = __builtin_amdgcn_readfirstlane(static_cast<int>(n - pa < left ? n : pa + left));
    *cur += pb - pa;
    seq = scalar_ints(a.seq_of_row)[r];
    start = scalar_ints(a.row_start)[r];
    end = scalar_ints(a.row_end)[r];
  }
};

// --- joining partial sums -----------------------------------------------------

// Writes one head's row as a constant (0 for an empty window, NaN for a failed one).
template <class T, int D>
__device__ __forceinline__ void fill_row(const KvAttnArgs& a, int64_t head, bool failed, int tid, int threads) {
  const float x = failed ? __builtin_nanf("") : 0.0f;
  const uint32_t y = T::pack(x, x);
  for (int i = tid; i < D / 2; i += threads) reinterpret_cast<uint32_t*>(a.out)[head * (D / 2) + i] = y;
  if (tid == 0 && a.lse != nullptr) a.lse[head] = failed ? x : -__builtin_inff();
}

// Joins the partial sums of one (row, head): partial i < n is in slot slot0 + i * step
// (the first one in slot first_slot). WAVES waves (of the whole workgroup: 4) take the partials in turn, eight at
// a time, as the positions were taken before: with a running maximum, so that sums and maxima
// are loaded together.
template <class T, int D, int WAVES>
__device__ __forceinline__ void join_row(const KvAttnArgs& a, int64_t head, int in_group, int group_rows, int64_t n,
                                         int64_t first_slot, int64_t slot0, int64_t step) {
  constexpr int kPer = D / 64, kBatch = 8;
  const int lane = threadIdx.x & 63, wave = WAVES == 1 ? 0 : threadIdx.x >> 6;
  float m = -__builtin_inff(), sum = 0.0f, acc[kPer] = {};
  for (int64_t i0 = wave; i0 < n; i0 += kBatch * WAVES) {
    float2 ml[kBatch];
    float o[kBatch][kPer];
    float top = m;
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int64_t i = i0 + x * WAVES;
      ml[x] = make_float2(-__builtin_inff(), 0.0f);
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[x][e] = 0.0f;
      if (i < n) {
        const int64_t s = (i == 0 ? first_slot : slot0 + i * step) * group_rows + in_group;
        ml[x] = a.part_ml[s];
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[x][e] = a.part_o[s * D + kPer * lane + e];
      }
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) top = fmaxf(top, ml[x].x);
    const float ref = top == -__builtin_inff() ? 0.0f : top;
    const float by = __builtin_amdgcn_exp2f(m - ref);
    m = top;
    sum *= by;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= by;
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const float f = __builtin_amdgcn_exp2f(ml[x].x - ref);
      sum += ml[x].y * f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] += o[x][e] * f;
    }
  }
  if constexpr (WAVES > 1) {
    __shared__ float2 ml_lds[WAVES];
    __shared__ float acc_lds[WAVES][D];
    if (lane == 0) ml_lds[wave] = make_float2(m, sum);
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc_lds[wave][kPer * lane + e] = acc[e];
    __syncthreads();
    if (wave > 0) return;
    float top = m;
#pragma unroll
    for (int i = 1; i < WAVES; ++i) top = fmaxf(top, ml_lds[i].x);
    const float ref = top == -__builtin_inff() ? 0.0f : top;
    const float by = __builtin_amdgcn_exp2f(m - ref);
    m = top;
    sum *= by;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= by;
#pragma unroll
    for (int i = 1; i < WAVES; ++i) {
      const float f = __builtin_amdgcn_exp2f(ml_lds[i].x - ref);
      sum += ml_lds[i].y * f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] += acc_lds[i][kPer * lane + e] * f;
    }
  }
  const float inv = a.v_scale / sum;
  uint16_t* out = static_cast<uint16_t*>(a.out) + head * D + kPer * lane;
  if constexpr (kPer == 1) {
    *out = static_cast<uint16_t>(T::pack(acc[0] * inv, 0.0f));
  } else {
#pragma unroll
    for (int e = 0; e < kPer; e += 2)
      *reinterpret_cast<uint32_t*>(out + e) = T::pack(acc[e] * inv, acc[e + 1] * inv);
  }
  if (lane == 0 && a.lse != nullptr) a.lse[head] = lse_of<T>(m, sum);
}

// Head of a join launch: one per workgroup, or (WAVES 1) one per wave; -1 behind the last.
template <int WAVES>
__device__ __forceinline__ int64_t join_head(const KvAttnArgs& a) {
  if (WAVES > 1) return blockIdx.x;
  const int64_t head = static_cast<int64_t>(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  return head < a.Q * a.H ? head : -1;
}

// --- selected form ------------------------------------------------------------

// Slots of one split of a row with n of them: whole tiles, the same for every split.
__device__ __forceinline__ int64_t split_share(int64_t n, int splits) {
  const int64_t tiles = (n + kTilePos - 1) / kTilePos;
  return (tiles + splits - 1) / splits * kTilePos;
}

// One workgroup's part of a selected launch.
struct ListPart {
  int64_t r, item;
  int g, split;
  int64_t n, from, to;   // slots [from, to) of the row's n

  // False where there is nothing to attend to; a row that is empty or invalid is `fill`ed by split 0.
  __device__ __forceinline__ bool take(const KvAttnArgs& a, int64_t gh, bool* fill) {
    // Workgroups go to the eight dies in turn: each die gets a run of neighbouring
    // rows, whose lists share most of their slots, so that its L2 holds them.
    const int64_t per_die = gridDim.x / 8;
    item = (blockIdx.x & 7) * per_die + (blockIdx.x >> 3);
    *fill = false;
    if (item >= a.Q * gh * a.splits) return false;
    r = item / (gh * a.splits);
    const int64_t rest = item - r * gh * a.splits;
    g = static_cast<int>(rest / a.splits);
    split = static_cast<int>(rest - static_cast<int64_t>(g) * a.splits);
    n = a.count[r];
    if (n > a.K && rest == 0 && threadIdx.x == 0) atomicOr(a.status, kStBadWindow);
    if (n <= 0 || n > a.K) {
      *fill = split == 0;
      return false;
    }
    const int64_t share = split_share(n, a.splits);
    from = split * share;
    to = from + share < n ? from + share : n;
    return from < to;
  }
};

// Heads up to which a whole workgroup joins one (a long sequence has hundreds of parts); beyond, there are
// few parts each and a wave does.
constexpr int64_t kJoinHeads = 512;

}  // namespace
}  // namespace mqa
