// Attention over the paged key-value cache (gfx950): new tokens over their
// sequence's window (decode form) and rows over a list of slots (selected form).
//
// Mathematics. For one row and head: s_p = scale q.k_p, out = sum_p e^(s_p - m) v_p
// / sum_p e^(s_p - m) for any m; m runs with the largest score seen, and sums
// taken under an older m are multiplied by e^(m_old - m_new). Partial results
// (m, sum, weighted values) of parts of the window join the same way. All
// exponentials are taken to base 2 with log2(e) folded into the scale.
//
// One wave works on 32 positions at a time with 16x16x32 matrix instructions,
// both products transposed so that nothing moves between lanes or through LDS:
//   S^T[position, query] = K Q^T   A = K: lane l holds position l % 16, 8 dims of group l / 16
//                                  result: query l % 16, positions 4 (l / 16) + 0..3
//   O^T[dim, query] = V^T P^T      B = P^T: query l % 16, 8 positions of group l / 16
// The order of positions inside the second product is free, so its 8 positions
// of a lane group are the 2 x 4 that the first product left in that lane: the
// weights are packed in place. A = V^T needs 8 positions of one dim in a lane: a lane
// loads D/16 neighbouring dims of its 8 positions (16 lanes read one position's
// row), and a byte permute per register pairs them; the dims of matrix tile t
// are t, t + D/16, t + 2 D/16, ...
//
// What bounds it: decode reads every key and value once for at most 64 query
// heads and is bound by memory (MI355X, whose large copies run at 4.9 TB/s: 64
// sequences of 32K to 131K positions under 64 heads 5.6 to 5.8 TB/s, 32 of 2K to
// 16K under 32 heads over 8 key heads 5.2). Lists of slots that rows share are read
// from the L2 caches (2,048 rows of 1,024 slots, 64 heads: 130 us, 8.3 TB/s and
// 530 TFLOP/s). Up to 16 heads per key head go through registers, more through LDS,
// both below with the reasons.
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

// --- up to 16 heads: keys and values in registers ---------------------------------
//
// The four waves of a workgroup take every fourth tile of 32 positions. The next
// tile's keys are loaded into the registers that the first product has just read,
// its values into those that the second has.

// Joins the four waves' results in LDS and writes the heads' outputs, or their partial
// sums where part_o is not null. `bad`: an invalid page or slot was met.
template <class T, int D>
struct Merge {
  static constexpr int kPart = D < 128 ? D : 128;   // dims of a head at a time, so that LDS holds two workgroups or more
  static constexpr int kPitch = kPart + 4;
  float o[kWaves][16][kPitch];
  float2 ml[kWaves][16];
  float2 fin[16];

  template <class W>
  __device__ __forceinline__ void run(W& w, bool bad, int rows, float v_scale, char* out, float* lse, float* part_o,
                                      float2* part_ml) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();   // the previous use of this memory is over
    const float mine = groups_sum(w.l[0]);
    if (w.grp == 0) ml[wave][w.col] = make_float2(w.m[0], bad ? __builtin_nanf("") : mine);
    __syncthreads();
    float2 x[kWaves];
    float top = -__builtin_inff(), total = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      x[i] = ml[i][w.col];
      top = fmaxf(top, x[i].x);
    }
    const float ref = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) total += x[i].y * __builtin_amdgcn_exp2f(x[i].x - ref);
    const float f = __builtin_amdgcn_exp2f(w.m[0] - ref);
    if (wave == 0 && w.grp == 0) fin[w.col] = make_float2(top, total);
    constexpr int kT = kPart / 16;   // matrix tiles of a part
#pragma unroll
    for (int t0 = 0; t0 < W::kDims; t0 += kT) {
      if (t0 > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < kT; t += 4)
          *reinterpret_cast<v4f*>(&o[wave][w.col][(4 * w.grp + i) * kT + t]) =
              v4f{w.o[0][t0 + t][i] * f, w.o[0][t0 + t + 1][i] * f, w.o[0][t0 + t + 2][i] * f,
                  w.o[0][t0 + t + 3][i] * f};
      __syncthreads();
      for (int e = threadIdx.x; e < 16 * kPart / 4; e += kThreads) {
        const int head = e / (kPart / 4), at = 4 * (e % (kPart / 4));
        const int d = at / kT * W::kDims + t0 + at % kT;
        if (head >= rows) continue;
        v4f sum = *reinterpret_cast<const v4f*>(&o[0][head][at]);
#pragma unroll
        for (int i = 1; i < kWaves; ++i) sum += *reinterpret_cast<const v4f*>(&o[i][head][at]);
        const float2 e2 = fin[head];
        if (part_o != nullptr) {
          *reinterpret_cast<v4f*>(part_o + static_cast<int64_t>(head) * D + d) = sum;
          if (d == 0) part_ml[head] = e2;
        } else {
          const float inv = v_scale / e2.y;
          const v2u y = {T::pack(sum[0] * inv, sum[1] * inv), T::pack(sum[2] * inv, sum[3] * inv)};
          *reinterpret_cast<v2u*>(out + (static_cast<int64_t>(head) * D + d) * 2) = y;
          if (d == 0 && lse != nullptr) lse[head] = lse_of<T>(e2.x, e2.y);
        }
      }
    }
  }
};

// This wave's tiles t, t + kWaves, ... below t_hi; range(t, &lo, &hi) gives the positions of a tile that count.
template <class W, class KEYS, class VALUES, class RANGE>
__device__ __forceinline__ void run_tiles(W& w, int t, int t_hi, float c, KEYS&& load_keys, VALUES&& load_values,
                                          RANGE&& range) {
  if (t >= t_hi) return;
  load_keys(t);
  load_values(t);
  while (true) {
    const int tn = t + kWaves;
    const bool more = tn < t_hi;
    int lo, hi;
    range(t, &lo, &hi);
    const bool edge = lo > 0 || hi < W::kPositions;
    uint32_t inside = 0xFFu;
    if (edge) {
      inside = 0;
#pragma unroll
      for (int j = 0; j < W::kMine; ++j) inside |= (w.mine(j) >= lo && w.mine(j) < hi ? 1u : 0u) << j;
    }
    v4f s[1][W::kTiles];
    typename W::P p[1];
    w.scores(s);
    if (more) load_keys(tn);
    w.weights(s, c, edge, inside, p);
    if (edge) w.clear_outside(inside);
    w.add_values(p);
    if (!more) break;
    load_values(tn);
    t = tn;
  }
}

// Positions of a register tile: 32, or 16 where D = 256 in 16 bits would need more registers than
// two waves per SIMD leave.
constexpr int register_tile(int D, bool e4m3) { return D == 256 && !e4m3 ? 16 : 32; }

// Offset of a slot in units of 16 bytes, of which the strides are multiples. A page's is below 2^36 bytes, 63
// positions' below 2^31: one 32-bit multiplication and one of 24 bits.
__device__ __forceinline__ uint64_t slot_offset(int slot, uint32_t page, uint32_t pos) {
  const uint32_t s = static_cast<uint32_t>(slot);
  return static_cast<uint64_t>(s >> 6) * page + __umul24(s & 63, pos);
}

// --- more heads: positions staged in LDS ------------------------------------------
//
// Two waves (a half) carry the first heads, two the others; each takes half of a stage
// of kStagePos positions (a page, or half of one). Asynchronous copies (memory to LDS, no
// registers) write the stages, kStages in turn, so that every byte crosses from the caches
// once, in whole rows, whatever the number of heads.
//
// The compiler would wait for every copy in flight before an LDS read that it
// cannot prove apart from them; the reads are inline assembly for that reason, each
// block with its own wait, and the copies are waited for by count before the
// barrier that hands a stage over. Keys lie with the 16-byte pieces of a row permuted by
// its position (piece ^ swizzle), which the copies' source addresses do, so that
// the rows that one read takes fall on different banks.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p));
}

template <int OFF>
__device__ __forceinline__ void read4(uint32_t at, uint32_t at2, v4u& a, v4u& b, v4u& c, v4u& d) {
  __asm__ __volatile__(
      "ds_read_b128 %0, %4 offset:%6\n\tds_read_b128 %1, %5 offset:%6\n\t"
      "ds_read_b128 %2, %4 offset:%7\n\tds_read_b128 %3, %5 offset:%7\n\ts_waitcnt lgkmcnt(0)"
      : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)
      : "v"(at), "v"(at2), "n"(OFF), "n"(OFF + 128)
      : "memory");
}

template <class T, bool E4M3, int D, int NQ>
struct Ring {
  static constexpr int kParts = 2;
  static constexpr int kPos = D < 256 ? 32 : 16;             // positions of a wave
  // SLACK 8: where the bytes come from the L2 caches or are half as many, the vector unit is what a stage waits for most.
  // us with 8 and with 0, 64 heads over one key head, D = 128: 2,048 lists of 1,024 slots 130, 140; 64 sequences of
  // 16,384 positions in 8 bits 76.5, 83.6; 200 rows of one sequence of 8,192 in bf16 102.6, 109.8. From memory in bf16
  // (64 of 32K to 131K) it makes no difference: 487.7, 488.6.
  typedef Wave<T, E4M3, D, NQ, kPos, false, 8> W;
  static constexpr int kStagePos = kParts * kPos;
  static constexpr int kRow = D * W::kBytes;                 // bytes of one position
  static constexpr int kImage = kStagePos * kRow;            // of a stage's keys, or values
  static constexpr int kStages = kImage >= 16384 ? 2 : 4;
  static constexpr int kCopies = kImage / 1024 / kWaves;     // 1 KiB copies per wave, of keys and of values each
  static constexpr int kCopyRows = 1024 / kRow;
  static constexpr int kPieces = kRow / 16;
  static constexpr int kHeads = 2 * 16 * NQ;
  char stage[kStages][2][kImage];
  float2 ml[2][kParts][16 * NQ];

  static __device__ __forceinline__ int swizzle(int row) { return kRow >= 128 ? row & 7 : row >> 1 & 3; }

  // Position of the stage that this lane fetches in copy c of its wave.
  static __device__ __forceinline__ int copy_row(int wave, int c, int lane) {
    return (wave * kCopies + c) * kCopyRows + lane / kPieces;
  }

  __device__ __forceinline__ void copy(int s, int kv, int wave, int c, const char* src) {
    __builtin_amdgcn_global_load_lds(src, &stage[s][kv][(wave * kCopies + c) * 1024], 16, 0, 0);
  }

  // Waits until at most `left` (0, 1 or 2) later stages of this wave's copies are in flight, then for the
  // other waves.
  static __device__ __forceinline__ void hand_over(int left) {
    constexpr int kPer = 2 * kCopies;
    if (kStages > 2 && left >= 2) __asm__ __volatile__("s_waitcnt vmcnt(%0)" ::"n"(2 * kPer) : "memory");
    else if (kStages > 2 && left == 1) __asm__ __volatile__("s_waitcnt vmcnt(%0)" ::"n"(kPer) : "memory");
    else __asm__ __volatile__("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __asm__ __volatile__("" ::: "memory");
  }

  // This lane's slots of stage i of the list at LDS address `list`, by hand as the stages' reads are.
  static __device__ __forceinline__ void read_slots(int (&slot)[kCopies], int i, int wave, int lane, uint32_t list) {
    const uint32_t at = list + 4 * (kStagePos * i + copy_row(wave, 0, lane));
    if constexpr (kCopies == 4) {
      __asm__ __volatile__(
          "ds_read_b32 %0, %4\n\tds_read_b32 %1, %4 offset:%5\n\t"
          "ds_read_b32 %2, %4 offset:%6\n\tds_read_b32 %3, %4 offset:%7\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(slot[0]), "=&v"(slot[1]), "=&v"(slot[2]), "=&v"(slot[3])
          : "v"(at), "n"(4 * kCopyRows), "n"(8 * kCopyRows), "n"(12 * kCopyRows)
          : "memory");
    } else if constexpr (kCopies == 2) {
      __asm__ __volatile__("ds_read_b32 %0, %2\n\tds_read_b32 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
                           : "=&v"(slot[0]), "=&v"(slot[1])
                           : "v"(at), "n"(4 * kCopyRows)
                           : "memory");
    } else {
      static_assert(kCopies == 1, "one, two or four");
      __asm__ __volatile__("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(slot[0]) : "v"(at) : "memory");
    }
  }

  // The piece of a row that a lane fetches for its place in LDS.
  static __device__ __forceinline__ int source_piece(int kv, int row, int lane) {
    return kv == 0 ? lane % kPieces ^ swizzle(row) : lane % kPieces;
  }

  // This wave's copies of stage i: positions from `base` on of the page whose keys are at kp and
  // values at vp; [lo, hi) of the page are inside the window, the lanes of others read the nearest one inside.
  __device__ __forceinline__ void copy_page(const KvAttnArgs& a, const char* kp, const char* vp, int i, int wave,
                                            int lane, int base, int lo, int hi) {
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int row = copy_row(wave, c, lane);
      const int pos = min(max(base + row, lo), hi - 1);
      copy(i % kStages, 0, wave, c,
           kp + static_cast<uint32_t>(pos * static_cast<int>(a.k_pos)) + 16 * source_piece(0, row, lane));
      copy(i % kStages, 1, wave, c,
           vp + static_cast<uint32_t>(pos * static_cast<int>(a.v_pos)) + 16 * source_piece(1, row, lane));
    }
  }

  // The same of stage i of a list of slots in LDS, filled up to whole stages.
  __device__ __forceinline__ void copy_list(const KvAttnArgs& a, const char* kb, const char* vb, int i, int wave,
                                            int lane, uint32_t list) {
    const uint32_t k_page = static_cast<uint32_t>(a.k_page >> 4), v_page = static_cast<uint32_t>(a.v_page >> 4);
    const uint32_t k_pos = static_cast<uint32_t>(a.k_pos >> 4), v_pos = static_cast<uint32_t>(a.v_pos >> 4);
    int slot[kCopies];
    read_slots(slot, i, wave, lane, list);
    uint64_t off[kCopies];
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      off[c] = slot_offset(slot[c], k_page, k_pos);
      copy(i % kStages, 0, wave, c, kb + (off[c] << 4) + 16 * source_piece(0, copy_row(wave, c, lane), lane));
    }
    if (k_page != v_page || k_pos != v_pos)
#pragma unroll
      for (int c = 0; c < kCopies; ++c) off[c] = slot_offset(slot[c], v_page, v_pos);
#pragma unroll
    for (int c = 0; c < kCopies; ++c)
      copy(i % kStages, 1, wave, c, vb + (off[c] << 4) + 16 * source_piece(1, copy_row(wave, c, lane), lane));
  }

  // Keys of positions kPos part + 16 a + col into w.k.
  __device__ __forceinline__ void read_keys(W& w, int s, int part) {
    const int z = swizzle(w.col);
    const uint32_t row = lds_address(&stage[s][0][0]) + (kPos * part + w.col) * kRow + 16 * (w.grp ^ (z & 3));
    const uint32_t even = row + 64 * (z >> 2), odd = row + 64 * (1 - (z >> 2));
    if constexpr (kRow == 512) {
      static_assert(W::kTiles == 1, "16 positions per wave");
      read4<0>(even, odd, w.k[0][0], w.k[0][1], w.k[0][2], w.k[0][3]);
      read4<256>(even, odd, w.k[0][4], w.k[0][5], w.k[0][6], w.k[0][7]);
    } else if constexpr (kRow == 256) {
      if constexpr (W::kTiles == 1) {
        read4<0>(even, odd, w.k[0][0], w.k[0][1], w.k[0][2], w.k[0][3]);
      } else {
        __asm__ __volatile__(
            "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\t"
            "ds_read_b128 %2, %8 offset:128\n\tds_read_b128 %3, %9 offset:128\n\t"
            "ds_read_b128 %4, %8 offset:4096\n\tds_read_b128 %5, %9 offset:4096\n\t"
            "ds_read_b128 %6, %8 offset:4224\n\tds_read_b128 %7, %9 offset:4224\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(w.k[0][0]), "=&v"(w.k[0][1]), "=&v"(w.k[0][2]), "=&v"(w.k[0][3]), "=&v"(w.k[1][0]),
              "=&v"(w.k[1][1]), "=&v"(w.k[1][2]), "=&v"(w.k[1][3])
            : "v"(even), "v"(odd)
            : "memory");
      }
    } else if constexpr (kRow == 128) {
      static_assert(W::kTiles == 2, "D < 256");
      __asm__ __volatile__(
          "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\t"
          "ds_read_b128 %2, %4 offset:2048\n\tds_read_b128 %3, %5 offset:2048\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(w.k[0][0]), "=&v"(w.k[0][1]), "=&v"(w.k[1][0]), "=&v"(w.k[1][1])
          : "v"(even), "v"(odd)
          : "memory");
    } else {
      __asm__ __volatile__("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:1024\n\ts_waitcnt lgkmcnt(0)"
                           : "=&v"(w.k[0][0]), "=&v"(w.k[1][0])
                           : "v"(row)
                           : "memory");
    }
  }

  // Values of this lane's positions into w.v.
  __device__ __forceinline__ void read_values(W& w, int s, int part) {
    const uint32_t at = lds_address(&stage[s][1][0]) + (kPos * part + 4 * w.grp) * kRow + w.col * (kRow / 16);
    if constexpr (kRow == 512) {
      v4u x[8];
      __asm__ __volatile__(
          "ds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:16\n\t"
          "ds_read_b128 %2, %8 offset:512\n\tds_read_b128 %3, %8 offset:528\n\t"
          "ds_read_b128 %4, %8 offset:1024\n\tds_read_b128 %5, %8 offset:1040\n\t"
          "ds_read_b128 %6, %8 offset:1536\n\tds_read_b128 %7, %8 offset:1552\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
          : "v"(at)
          : "memory");
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) w.v[j / 2][4 * (j & 1) + e] = x[j][e];
    } else if constexpr (kRow == 256 && W::kTiles == 1) {
      v4u x[4];
      __asm__ __volatile__(
          "ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:256\n\t"
          "ds_read_b128 %2, %4 offset:512\n\tds_read_b128 %3, %4 offset:768\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
          : "v"(at)
          : "memory");
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) w.v[j][e] = x[j][e];
    } else if constexpr (kRow == 256) {
      v4u x[8];
      __asm__ __volatile__(
          "ds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:256\n\t"
          "ds_read_b128 %2, %8 offset:512\n\tds_read_b128 %3, %8 offset:768\n\t"
          "ds_read_b128 %4, %8 offset:4096\n\tds_read_b128 %5, %8 offset:4352\n\t"
          "ds_read_b128 %6, %8 offset:4608\n\tds_read_b128 %7, %8 offset:4864\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
          : "v"(at)
          : "memory");
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) w.v[j][e] = x[j][e];
    } else if constexpr (kRow == 128) {
      v2u x[8];
      __asm__ __volatile__(
          "ds_read_b64 %0, %8\n\tds_read_b64 %1, %8 offset:128\n\t"
          "ds_read_b64 %2, %8 offset:256\n\tds_read_b64 %3, %8 offset:384\n\t"
          "ds_read_b64 %4, %8 offset:2048\n\tds_read_b64 %5, %8 offset:2176\n\t"
          "ds_read_b64 %6, %8 offset:2304\n\tds_read_b64 %7, %8 offset:2432\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
          : "v"(at)
          : "memory");
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) w.v[j][e] = x[j][e];
    } else {
      static_assert(kRow == 64 && W::kTiles == 2, "D = 64 in 8 bits");
      __asm__ __volatile__(
          "ds_read_b32 %0, %8\n\tds_read_b32 %1, %8 offset:64\n\t"
          "ds_read_b32 %2, %8 offset:128\n\tds_read_b32 %3, %8 offset:192\n\t"
          "ds_read_b32 %4, %8 offset:1024\n\tds_read_b32 %5, %8 offset:1088\n\t"
          "ds_read_b32 %6, %8 offset:1152\n\tds_read_b32 %7, %8 offset:1216\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(w.v[0][0]), "=&v"(w.v[1][0]), "=&v"(w.v[2][0]), "=&v"(w.v[3][0]), "=&v"(w.v[4][0]),
            "=&v"(w.v[5][0]), "=&v"(w.v[6][0]), "=&v"(w.v[7][0])
          : "v"(at)
          : "memory");
    }
  }

  // Runs the n stages of one segment or list. fetch(i) issues this wave's copies of
  // stage i; range(i, &lo, &hi) gives the positions of the stage that count.
  template <class FETCH, class RANGE>
  __device__ __forceinline__ void run(W& w, int n, int part, float c, FETCH&& fetch, RANGE&& range) {
    // no other load or store of this wave is in flight when the copies are counted
    __asm__ __volatile__("s_waitcnt vmcnt(0)" ::: "memory");
    constexpr int kAhead = kStages - 1;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i < n) {
        fetch(i);
        __asm__ __volatile__("" ::: "memory");   // a stage's copies are counted before the next one's
      }
    for (int i = 0; i < n; ++i) {
      hand_over(min(n - 1 - i, kAhead - 1));
      if (i + kAhead < n) {
        fetch(i + kAhead);
        __asm__ __volatile__("" ::: "memory");
      }
      int lo, hi;
      range(i, &lo, &hi);
      lo -= kPos * part;
      hi -= kPos * part;
      if (lo >= kPos || hi <= 0) continue;
      const bool edge = lo > 0 || hi < kPos;
      uint32_t inside = 0xFFu;
      if (edge) {
        inside = 0;
#pragma unroll
        for (int j = 0; j < W::kMine; ++j) inside |= (w.mine(j) >= lo && w.mine(j) < hi ? 1u : 0u) << j;
      }
      v4f x[NQ][W::kTiles];
      typename W::P p[NQ];
      read_keys(w, i % kStages, part);
      w.scores(x);
      w.weights(x, c, edge, inside, p);
      read_values(w, i % kStages, part);
      if (edge) w.clear_outside(inside);
      w.add_values(p);
    }
  }

  // Joins a half's waves and writes its heads' outputs, or their partial sums where
  // part_o is not null. `bad`: an invalid page or slot was met. The stages' memory
  // carries the sums; either wave adds and writes half of them.
  __device__ __forceinline__ void finish(W& w, int half, int part, bool bad, int rows, float v_scale, char* out,
                                         float* lse, float* part_o, float2* part_ml) {
    constexpr int kShare = NQ * W::kDims / kParts;   // dim tiles that each wave joins
    v4f* space = reinterpret_cast<v4f*>(&stage[0][0][0]) + half * kParts * (NQ * W::kDims) * 64 + w.lane;
    static_assert(sizeof(stage) >= sizeof(v4f) * 2 * kParts * NQ * W::kDims * 64, "the stages hold all sums");
    __syncthreads();   // every read of the stages is over
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const float sum = groups_sum(w.l[n]);
      if (w.grp == 0) ml[half][part][16 * n + w.col] = make_float2(w.m[n], bad ? __builtin_nanf("") : sum);
    }
    __syncthreads();
    float f[NQ], top[NQ], sum[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float2 x[kParts];
      top[n] = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        x[i] = ml[half][i][16 * n + w.col];
        top[n] = fmaxf(top[n], x[i].x);
      }
      const float ref = top[n] == -__builtin_inff() ? 0.0f : top[n];
      sum[n] = 0.0f;
#pragma unroll
      for (int i = 0; i < kParts; ++i) sum[n] += x[i].y * __builtin_amdgcn_exp2f(x[i].x - ref);
      f[n] = __builtin_amdgcn_exp2f(w.m[n] - ref);
    }
#pragma unroll
    for (int x = 0; x < NQ * W::kDims; ++x) space[(part * NQ * W::kDims + x) * 64] = w.o[x / W::kDims][x % W::kDims] * f[x / W::kDims];
    __syncthreads();
    v4f got[kShare];   // tiles part * kShare .. of (query tile, dim tile) pairs: one query tile, neighbouring dims
#pragma unroll
    for (int x = 0; x < kShare; ++x) {
      got[x] = space[(part * kShare + x) * 64];
#pragma unroll
      for (int i = 1; i < kParts; ++i) got[x] += space[(i * NQ * W::kDims + part * kShare + x) * 64];
    }
    const int n = part * kShare / W::kDims, t0 = part * kShare % W::kDims, head = 16 * n + w.col;
    float inv = 0.0f, my_top = 0.0f, my_sum = 0.0f;
#pragma unroll
    for (int x = 0; x < NQ; ++x)
      if (x == n) {
        my_top = top[x];
        my_sum = sum[x];
      }
    inv = v_scale / my_sum;
    if (head < rows) {
      const int64_t at = static_cast<int64_t>(head) * D + 4 * w.grp * W::kDims + t0;
      if (part_o != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          store_dims<float>(part_o + at + i * W::kDims, got, i, 1.0f);
        if (w.grp == 0 && t0 == 0) part_ml[head] = make_float2(my_top, my_sum);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) store_dims<T>(reinterpret_cast<uint16_t*>(out) + at + i * W::kDims, got, i, inv);
        if (w.grp == 0 && t0 == 0 && lse != nullptr) lse[head] = lse_of<T>(my_top, my_sum);
      }
    }
    __syncthreads();   // the stages may be filled again
  }

  // Element i of each of the tiles, neighbouring dims, to `to`.
  template <class OUT, class PTR>
  static __device__ __forceinline__ void store_dims(PTR* to, const v4f (&x)[NQ * W::kDims / kParts], int i, float by) {
    constexpr int kShare = NQ * W::kDims / kParts;
    if constexpr (sizeof(PTR) == 4) {
      if constexpr (kShare >= 4) {
#pragma unroll
        for (int t = 0; t < kShare; t += 4)
          *reinterpret_cast<v4f*>(to + t) = v4f{x[t][i], x[t + 1][i], x[t + 2][i], x[t + 3][i]};
      } else {
#pragma unroll
        for (int t = 0; t < kShare; ++t) to[t] = x[t][i];
      }
    } else if constexpr (kShare >= 4) {
#pragma unroll
      for (int t = 0; t < kShare; t += 4)
        *reinterpret_cast<v2u*>(to + t) = v2u{OUT::pack(x[t][i] * by, x[t + 1][i] * by),
                                              OUT::pack(x[t + 2][i] * by, x[t + 3][i] * by)};
    } else if constexpr (kShare == 2) {
      *reinterpret_cast<uint32_t*>(to) = OUT::pack(x[0][i] * by, x[1][i] * by);
    } else {
      *to = static_cast<PTR>(OUT::pack(x[0][i] * by, 0.0f));
    }
  }
};

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
  const uint32_t x = static_cast<uint32_t>(static_cast<uint64_t>(some) * a.join_cost >> 16);   // below 2^23
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
    // one round trip to memory, less than another launch
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
  __device__ __forceinline__ void take(const KvAttnArgs& a, const int64_t* prefix, int64_t gh, int64_t* cur,
                                       int64_t stop) {
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
    g = __builtin_amdgcn_readfirstlane(static_cast<int>(in_row / n));
    pa = __builtin_amdgcn_readfirstlane(static_cast<int>(in_row - g * n));
    const int64_t left = stop - *cur;
    pb = __builtin_amdgcn_readfirstlane(static_cast<int>(n - pa < left ? n : pa + left));
    *cur += pb - pa;
    seq = scalar_ints(a.seq_of_row)[r];
    start = scalar_ints(a.row_start)[r];
    end = scalar_ints(a.row_end)[r];
  }
};

template <class T, bool E4M3, int D>
__global__ void __launch_bounds__(kThreads, 2) kv_decode_kernel(KvAttnArgs a) {
  constexpr int kTile = register_tile(D, E4M3), kPer = 64 / kTile;   // tiles of a page
  typedef Wave<T, E4M3, D, 1, kTile> W;
  __shared__ Plan<kWaves> plan;
  __shared__ Merge<T, D> merge;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t* prefix = plan.make(a);
  const int64_t units = prefix[a.Q] * a.Hkv;
  const int64_t share = unit_share(a, units, gridDim.x);
  int64_t cur = blockIdx.x * share;
  const int64_t stop = cur + share < units ? cur + share : units;
  W w;
  w.init();
  while (cur < stop) {
    Segment sg;
    sg.take(a, prefix, a.Hkv, &cur, stop);
    const int64_t r = sg.r;
    const int kvh = sg.g;
    const int start = sg.start, end = sg.end;
    const int32_t* table = a.table + static_cast<int64_t>(sg.seq) * a.max_pages;
    const int p0 = start >> 6;
    const int t_lo = max(kPer * (p0 + sg.pa), start / kTile);
    const int t_hi = min(kPer * (p0 + sg.pb), (end + kTile - 1) / kTile);
    const char* kb = a.k + kvh * a.k_head;
    const char* vb = a.v + kvh * a.v_head;
    const int64_t head0 = r * a.H + static_cast<int64_t>(kvh) * a.G;
    w.start();
    w.load_q(a.q + r * a.q_row + static_cast<int64_t>(kvh) * a.G * D * 2, a.G, a.q_keep, a.q_flip, nullptr);

    bool bad = false;
    int next = t_lo + wave < t_hi ? table[(t_lo + wave) / kPer] : 0;   // entry of the next tile's page, read early
    int64_t page = 0;
    // positions outside the window are not read: their lanes read the nearest one inside
    auto clamp = [&](int pos) { return min(max(pos, start), end - 1) & 63; };
    run_tiles(
        w, t_lo + wave, t_hi, a.c,
        [&](int t) {
          page = next;
          if (t + kWaves < t_hi) next = table[(t + kWaves) / kPer];
          if (page < 0 || page >= a.P_phys) {   // nothing of it is read; page 0 stands in
            bad = true;
            page = 0;
          }
          const char* base = kb + page * a.k_page;
#pragma unroll
          for (int b = 0; b < W::kTiles; ++b)
            w.load_k(b, base + static_cast<uint32_t>(clamp(kTile * t + 16 * b + w.col) * static_cast<int>(a.k_pos)));
        },
        [&](int t) {
          const char* base = vb + page * a.v_page;
#pragma unroll
          for (int j = 0; j < W::kMine; ++j)
            w.load_v(j, base + static_cast<uint32_t>(clamp(kTile * t + w.mine(j)) * static_cast<int>(a.v_pos)));
        },
        [&](int t, int* lo, int* hi) {
          *lo = start - kTile * t;
          *hi = end - kTile * t;
        });
    if (bad && w.lane == 0) atomicOr(a.status, kStBadPage);
    const bool whole = sg.pa == 0 && sg.pb == sg.n;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (sg.pa == 0 ? 1 : 0);
    merge.run(w, bad, a.G, a.v_scale, static_cast<char*>(a.out) + head0 * D * 2,
              a.lse == nullptr ? nullptr : a.lse + head0, whole ? nullptr : a.part_o + slot * a.G * D,
              a.part_ml + slot * a.G);
  }
}

template <class T, bool E4M3, int D, int NQ>
__global__ void __launch_bounds__(kThreads, 2) kv_decode_staged_kernel(KvAttnArgs a) {
  typedef Ring<T, E4M3, D, NQ> R;
  constexpr int kHeads = R::kHeads, kPer = 64 / R::kStagePos;   // stages of a page
  __shared__ Plan<kWaves> plan;
  __shared__ __align__(16) R ring;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = wave / R::kParts, part = wave % R::kParts;
  const int64_t* prefix = plan.make(a);
  const int qg = (a.G + kHeads - 1) / kHeads;
  const int64_t gh = static_cast<int64_t>(a.Hkv) * qg;
  const int64_t units = prefix[a.Q] * gh;
  const int64_t share = unit_share(a, units, gridDim.x);
  int64_t cur = blockIdx.x * share;
  const int64_t stop = cur + share < units ? cur + share : units;
  const int group_rows = a.G < kHeads ? a.G : kHeads;
  typename R::W w;
  w.init();
  while (cur < stop) {
    Segment s;
    s.take(a, prefix, gh, &cur, stop);
    const int kvh = s.g / qg, at = half * 16 * NQ, first = (s.g % qg) * kHeads + at;
    const int rows = a.G - first < 16 * NQ ? a.G - first : 16 * NQ;   // of this half; none perhaps
    // Two stages: every wait is for all copies anyway, and a table entry may be loaded as they are. More:
    // it goes through the scalar cache, whose loads are counted apart.
    const int32_t* table_at = a.table + static_cast<int64_t>(s.seq) * a.max_pages;
    typename Pick<R::kStages == 2, const int32_t*, ScalarInts>::type table;
    if constexpr (R::kStages == 2) table = table_at;
    else table = scalar_ints(table_at);
    const int p0 = (s.start >> 6) + s.pa, n = (s.pb - s.pa) * kPer;
    const char* kb = a.k + kvh * a.k_head;
    const char* vb = a.v + kvh * a.v_head;
    const int64_t head0 = s.r * a.H + static_cast<int64_t>(kvh) * a.G + first;
    w.start();
    w.load_q(a.q + s.r * a.q_row + (static_cast<int64_t>(kvh) * a.G + first) * D * 2, rows, a.q_keep, a.q_flip, nullptr);
    bool bad = false;
    int next = table[p0];   // the entry of the page to be fetched next, read early
    int64_t page = 0;
    ring.run(
        w, n, part, a.c,
        [&](int i) {
          if (i % kPer == 0) {
            page = next;
            if (i + kPer < n) next = table[p0 + i / kPer + 1];
            if (page < 0 || page >= a.P_phys) {   // nothing of it is read; page 0 stands in
              bad = true;
              page = 0;
            }
          }
          const int at = 64 * (p0 + i / kPer);
          ring.copy_page(a, kb + page * a.k_page, vb + page * a.v_page, i, wave, w.lane, i % kPer * R::kStagePos,
                         s.start - at, min(s.end - at, 64));
        },
        [&](int i, int* lo, int* hi) {
          const int at = 64 * (p0 + i / kPer) + i % kPer * R::kStagePos;
          *lo = s.start - at;
          *hi = s.end - at;
        });
    if (bad && threadIdx.x == 0) atomicOr(a.status, kStBadPage);
    const bool whole = s.pa == 0 && s.pb == s.n;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (s.pa == 0 ? 1 : 0);
    ring.finish(w, half, part, bad, rows, a.v_scale, static_cast<char*>(a.out) + head0 * D * 2,
                a.lse == nullptr ? nullptr : a.lse + head0,
                whole ? nullptr : a.part_o + (slot * group_rows + at) * D, a.part_ml + slot * group_rows + at);
  }
}

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

template <class T, int D, int WAVES>
__global__ void __launch_bounds__(kThreads) kv_decode_join_kernel(KvAttnArgs a, int per, int groups) {
  const int64_t head = join_head<WAVES>(a);
  if (head < 0) return;
  const int64_t r = head / a.H;
  const int h = static_cast<int>(head - r * a.H);
  const int64_t before = a.prefix[r], n = a.prefix[r + 1] - before, all = a.prefix[a.Q];
  if (n == 0) {
    int code;
    row_pages(a, r, &code);
    fill_row<T, D>(a, head, code != 0, WAVES > 1 ? threadIdx.x : threadIdx.x & 63, 64 * WAVES);
    return;
  }
  const int qg = (a.G + per - 1) / per;
  const int64_t gh = static_cast<int64_t>(a.Hkv) * qg;
  const int64_t share = unit_share(a, all * gh, groups);
  const int kvh = h / a.G, in_kv = h - kvh * a.G;
  const int64_t from = before * gh + (static_cast<int64_t>(kvh) * qg + in_kv / per) * n;
  const int64_t w0 = from / share, w1 = (from + n - 1) / share;
  if (w0 == w1) return;   // one workgroup had all of it and wrote the output
  // the first part is its workgroup's last one (slot 2 w + 1), the others are first ones (slot 2 w)
  join_row<T, D, WAVES>(a, head, in_kv % per, a.G < per ? a.G : per, w1 - w0 + 1, 2 * w0 + 1, 2 * w0, 2);
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

template <class T, bool E4M3, int D>
__global__ void __launch_bounds__(kThreads, 2) kv_selected_kernel(KvAttnArgs a) {
  constexpr int kTile = register_tile(D, E4M3);
  typedef Wave<T, E4M3, D, 1, kTile> W;
  __shared__ int list[kKvSelBlock];
  __shared__ Merge<T, D> merge;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  ListPart p;
  bool fill;
  const bool any = p.take(a, a.Hkv, &fill);
  if (!any && !fill) return;
  const int64_t head0 = p.r * a.H + static_cast<int64_t>(p.g) * a.G;
  if (!any) {
    for (int h = 0; h < a.G; ++h) fill_row<T, D>(a, head0 + h, p.n != 0, threadIdx.x, kThreads);
    return;
  }
  W w;
  w.init();
  w.start();
  w.load_q(a.q + p.r * a.q_row + static_cast<int64_t>(p.g) * a.G * D * 2, a.G, a.q_keep, a.q_flip, nullptr);
  const char* kb = a.k + p.g * a.k_head;
  const char* vb = a.v + p.g * a.v_head;
  const uint32_t k_page = static_cast<uint32_t>(a.k_page >> 4), v_page = static_cast<uint32_t>(a.v_page >> 4);
  const uint32_t k_pos = static_cast<uint32_t>(a.k_pos >> 4), v_pos = static_cast<uint32_t>(a.v_pos >> 4);
  bool bad = false;
  for (int64_t b0 = p.from; b0 < p.to; b0 += kKvSelBlock) {
    const int len = static_cast<int>(p.to - b0 < kKvSelBlock ? p.to - b0 : kKvSelBlock);
    if (b0 != p.from) __syncthreads();
    bool mine = false;
    for (int i = threadIdx.x; i < len; i += kThreads) {
      const int s = a.slots[p.r * a.K + b0 + i];
      list[i] = s;
      mine |= s < 0 || s >= 64 * a.P_phys;
    }
    if (__syncthreads_or(mine)) {   // nothing of the list is read
      bad = true;
      break;
    }
    run_tiles(
        w, wave, (len + kTile - 1) / kTile, a.c,
        [&](int t) {
#pragma unroll
          for (int b = 0; b < W::kTiles; ++b)
            w.load_k(b, kb + (slot_offset(list[min(kTile * t + 16 * b + w.col, len - 1)], k_page, k_pos) << 4));
        },
        [&](int t) {
#pragma unroll
          for (int j = 0; j < W::kMine; ++j)
            w.load_v(j, vb + (slot_offset(list[min(kTile * t + w.mine(j), len - 1)], v_page, v_pos) << 4));
        },
        [&](int t, int* lo, int* hi) {
          *lo = 0;
          *hi = len - kTile * t;
        });
  }
  if (bad && threadIdx.x == 0) atomicOr(a.status, kStBadPage);
  merge.run(w, bad, a.G, a.v_scale, static_cast<char*>(a.out) + head0 * D * 2, a.lse == nullptr ? nullptr : a.lse + head0,
            a.splits == 1 ? nullptr : a.part_o + p.item * a.G * D, a.part_ml + p.item * a.G);
}

template <class T, bool E4M3, int D, int NQ>
__global__ void __launch_bounds__(kThreads, 2) kv_selected_staged_kernel(KvAttnArgs a) {
  typedef Ring<T, E4M3, D, NQ> R;
  constexpr int kHeads = R::kHeads;
  __shared__ __align__(16) R ring;
  __shared__ int list[kKvSelBlock];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = wave / R::kParts, part = wave % R::kParts;
  const int qg = (a.G + kHeads - 1) / kHeads;
  ListPart p;
  bool fill;
  const bool any = p.take(a, static_cast<int64_t>(a.Hkv) * qg, &fill);
  if (!any && !fill) return;
  const int kvh = p.g / qg, at = half * 16 * NQ, first = (p.g % qg) * kHeads + at;
  const int rows = a.G - first < 16 * NQ ? a.G - first : 16 * NQ;   // of this half; none perhaps
  const int64_t head0 = p.r * a.H + static_cast<int64_t>(kvh) * a.G + first;
  if (!any) {
    for (int h = 0; h < rows; ++h) fill_row<T, D>(a, head0 + h, p.n != 0, threadIdx.x % (64 * R::kParts), 64 * R::kParts);
    return;
  }
  typename R::W w;
  w.init();
  w.start();
  w.load_q(a.q + p.r * a.q_row + (static_cast<int64_t>(kvh) * a.G + first) * D * 2, rows, a.q_keep, a.q_flip, nullptr);
  const char* kb = a.k + kvh * a.k_head;
  const char* vb = a.v + kvh * a.v_head;
  bool bad = false;
  for (int64_t b0 = p.from; b0 < p.to; b0 += kKvSelBlock) {
    const int len = static_cast<int>(p.to - b0 < kKvSelBlock ? p.to - b0 : kKvSelBlock);
    if (b0 != p.from) __syncthreads();
    bool mine = false;
    const int n = (len + R::kStagePos - 1) / R::kStagePos;
    for (int i = threadIdx.x; i < n * R::kStagePos; i += kThreads) {
      const int s = a.slots[p.r * a.K + b0 + min(i, len - 1)];   // the last one again behind the end
      list[i] = s;
      mine |= s < 0 || s >= 64 * a.P_phys;
    }
    if (__syncthreads_or(mine)) {   // nothing of the list is read
      bad = true;
      break;
    }
    const uint32_t list_at = lds_address(list);
    ring.run(
        w, n, part, a.c, [&](int i) { ring.copy_list(a, kb, vb, i, wave, w.lane, list_at); },
        [&](int i, int* lo, int* hi) {
          *lo = 0;
          *hi = len - R::kStagePos * i;
        });
  }
  if (bad && threadIdx.x == 0) atomicOr(a.status, kStBadPage);
  const int group_rows = a.G < kHeads ? a.G : kHeads;
  const bool whole = a.splits == 1;
  ring.finish(w, half, part, bad, rows, a.v_scale, static_cast<char*>(a.out) + head0 * D * 2,
              a.lse == nullptr ? nullptr : a.lse + head0,
              whole ? nullptr : a.part_o + (p.item * group_rows + at) * D, a.part_ml + p.item * group_rows + at);
}

template <class T, int D, int WAVES>
__global__ void __launch_bounds__(kThreads) kv_selected_join_kernel(KvAttnArgs a, int per) {
  const int64_t head = join_head<WAVES>(a);
  if (head < 0) return;
  const int64_t r = head / a.H;
  const int h = static_cast<int>(head - r * a.H);
  const int64_t n = a.count[r];
  if (n <= 0 || n > a.K) return;   // written already
  const int qg = (a.G + per - 1) / per;
  const int kvh = h / a.G, in_kv = h - kvh * a.G;
  const int64_t share = split_share(n, a.splits);
  const int64_t slot = ((r * a.Hkv + kvh) * qg + in_kv / per) * a.splits;
  join_row<T, D, WAVES>(a, head, in_kv % per, a.G < per ? a.G : per, (n + share - 1) / share, slot, slot, 1);
}

// --- accumulated weights ------------------------------------------------------

constexpr int kWeightSeqs = 1024;     // sequences planned at once
constexpr int kWeightTiles = 32;      // tiles of a workgroup's sums in LDS

// Sum over the 16 lanes of a row of lanes, in every one of them.
__device__ __forceinline__ float row_sum(float x) {
  x += __uint_as_float(dpp_take<0x128, 0xF>(0u, __float_as_uint(x)));   // row_ror:8
  x += __uint_as_float(dpp_take<0x124, 0xF>(0u, __float_as_uint(x)));
  x += __uint_as_float(dpp_take<0x122, 0xF>(0u, __float_as_uint(x)));
  x += __uint_as_float(dpp_take<0x121, 0xF>(0u, __float_as_uint(x)));
  return x;
}

// acc[seq, p] += sum over rows and heads of exp(s_p - lse). The unit of work is one
// page of one sequence with all of its rows and heads, so that a position's sum
// has one owner and one order. Bound by the keys' bytes.
//
// Up to 16 heads per key head: eight waves, of which `hg` (a power of two) take the key
// heads in turn and 8 / hg the tiles of 32 positions; each of the former sums for itself in LDS and
// the sums are added in order at the end. More heads: four waves take tiles, the queries lie in LDS.
// The next tile's keys are loaded into the registers that the product has just read.
constexpr int weight_waves(int nq) { return nq == 1 ? 8 : 4; }

template <class T, bool E4M3, int D, int NQ>
__global__ void __launch_bounds__(64 * weight_waves(NQ), D == 256 ? 2 : NQ == 1 ? 4 : 3)
    kv_weights_kernel(KvAttnArgs a, const float* __restrict__ lse, float* __restrict__ acc, int64_t acc_stride, int hg) {
  typedef Wave<T, E4M3, D, NQ, 32, (NQ > 1)> W;
  constexpr int kBlock = kWeightTiles * kTilePos, kWeightWaves = weight_waves(NQ), kWeightThreads = 64 * kWeightWaves;
  __shared__ int seq_lo[kWeightSeqs], seq_hi[kWeightSeqs];
  __shared__ int64_t prefix[kWeightSeqs + 1];
  __shared__ int64_t sums[kWeightWaves];
  __shared__ v4u q_lds[W::kShared ? NQ * W::kChunks * 64 : 1];
  __shared__ float part[(NQ > 1 ? 1 : kWeightWaves) * kBlock];
  __shared__ int covered[kBlock];
  __shared__ int next_seq;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int head_at = wave % hg, tile_at = wave / hg, tile_step = kWeightWaves / hg;
  const int64_t me = blockIdx.x;
  const int qg = (a.G + 16 * NQ - 1) / (16 * NQ);
  W w;
  w.init();
  // kWeightSeqs sequences at a time, from the first that a row behind the ones before belongs to
  int64_t s0 = 0;
  do {
    // the positions that any row of each sequence looks at
    __syncthreads();
    if (threadIdx.x == 0) next_seq = 0x7FFFFFFF;
    for (int i = threadIdx.x; i < kWeightSeqs; i += kWeightThreads) {
      seq_lo[i] = 0x7FFFFFFF;
      seq_hi[i] = 0;
    }
    __syncthreads();
    for (int64_t r = threadIdx.x; r < a.Q; r += kWeightThreads) {
      int code = 0;
      const int n = row_pages(a, r, &code);
      if (me == 0 && s0 == 0) report(a, code);
      const int64_t i = a.seq_of_row[r] - s0;
      if (n > 0 && i >= 0 && i < kWeightSeqs) {
        atomicMin(&seq_lo[i], a.row_start[r]);
        atomicMax(&seq_hi[i], a.row_end[r]);
      } else if (n > 0 && i >= kWeightSeqs) {
        atomicMin(&next_seq, a.seq_of_row[r]);
      }
    }
    __syncthreads();
    constexpr int kPer = kWeightSeqs / kWeightThreads;
    int64_t n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = kPer * threadIdx.x + i;
      n[i] = seq_hi[x] > 0 ? (seq_hi[x] + 63) / 64 - seq_lo[x] / 64 : 0;
      sum += n[i];
    }
    int64_t units;
    int64_t at = block_scan<kWeightWaves>(sum, sums, &units) - sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      prefix[kPer * threadIdx.x + i] = at;
      at += n[i];
    }
    if (threadIdx.x == 0) prefix[kWeightSeqs] = units;
    __syncthreads();
    const int64_t after = next_seq;

    const int64_t share = (units + gridDim.x - 1) / gridDim.x;
    int64_t cur = me * share;
    const int64_t stop = cur + share < units ? cur + share : units;
    while (cur < stop) {
      int lo = 0, hi = kWeightSeqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= cur) lo = mid;
        else hi = mid;
      }
      const int si = __builtin_amdgcn_readfirstlane(lo);
      const int64_t seq = s0 + si;
      const int pages = static_cast<int>(prefix[si + 1] - prefix[si]);
      const int pa = __builtin_amdgcn_readfirstlane(static_cast<int>(cur - prefix[si]));
      int64_t pn = stop - cur;
      if (pn > pages - pa) pn = pages - pa;
      if (pn > kWeightTiles / 2) pn = kWeightTiles / 2;
      cur += pn;
      const int t_lo = 2 * ((seq_lo[si] >> 6) + pa), t_hi = t_lo + 2 * static_cast<int>(pn);
      const int32_t* table = a.table + seq * a.max_pages;
      __syncthreads();   // the sums of the run before are written
      for (int i = threadIdx.x; i < hg * kBlock; i += kWeightThreads) part[i] = 0.0f;
      for (int i = threadIdx.x; i < kBlock; i += kWeightThreads) covered[i] = 0;
      __syncthreads();
      for (int64_t r0 = 0; r0 < a.Q; r0 += 64) {
        const int64_t rl = r0 + w.lane;
        bool mine = false;
        if (rl < a.Q && a.seq_of_row[rl] == seq) {
          int code;
          mine = row_pages(a, rl, &code) > 0 && a.row_start[rl] < 32 * t_hi && a.row_end[rl] > 32 * t_lo;
        }
        uint64_t todo = __ballot(mine);   // the same in every wave
        while (todo) {
          const int64_t r = r0 + __builtin_ctzll(todo);
          todo &= todo - 1;
          const int start = a.row_start[r], end = a.row_end[r];
          // this wave's tiles of the row's window
          const int first_t = max(t_lo, start >> 5), last_t = min(t_hi, (end + 31) >> 5);
          const int from = first_t + (tile_at - (first_t - t_lo) % tile_step + tile_step) % tile_step;
          for (int g = head_at; g < a.Hkv * qg; g += hg) {
            const int kvh = g / qg, first = (g % qg) * 16 * NQ;
            const int rows = a.G - first < 16 * NQ ? a.G - first : 16 * NQ;
            const int64_t head0 = r * a.H + static_cast<int64_t>(kvh) * a.G + first;
            const char* kb = a.k + kvh * a.k_head;
            bool good = false, next_good = false;
            // positions outside the window are not read: their lanes read the nearest one inside
            auto load_keys = [&](int t) {
              int64_t page = table[t >> 1];
              next_good = page >= 0 && page < a.P_phys;
              if (!next_good) page = 0;
              const char* base = kb + page * a.k_page;
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const int pos = min(max(32 * t + 16 * b + w.col, start), end - 1) & 63;
                w.load_k(b, base + static_cast<uint32_t>(pos * static_cast<int>(a.k_pos)));
              }
            };
            if (from < last_t) load_keys(from);
            if (W::kShared) __syncthreads();
            w.load_q(a.q + r * a.q_row + (static_cast<int64_t>(kvh) * a.G + first) * D * 2, rows, ~0u, 0u, q_lds);
            float sub[NQ];
            bool counts[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              const int h = 16 * n + w.col;
              sub[n] = h < rows ? lse[head0 + h] : __builtin_inff();
              counts[n] = __builtin_fabsf(sub[n]) < __builtin_inff();
            }
            if (W::kShared) __syncthreads();
            for (int t = from; t < last_t; t += tile_step) {
              v4f s[NQ][2];
              w.scores(s);
              good = next_good;
              if (t + tile_step < last_t) load_keys(t + tile_step);
              float x[8] = {};
#pragma unroll
              for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  // the difference first, in full: it is small where the weight is not
                  const float d = __builtin_fmaf(s[n][j >> 2][j & 3], a.score_scale, -sub[n]);
                  const float p = __builtin_amdgcn_exp2f(d * 1.44269504088896340736f);
                  x[j] += counts[n] ? p : 0.0f;
                }
              float y = 0.0f;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float z = row_sum(x[j]);
                y = w.col == j ? z : y;
              }
              if (!good) {
                if (w.lane == 0) atomicOr(a.status, kStBadPage);
              } else if (w.col < 8) {
                const int pos = 32 * t + w.mine(w.col);
                if (pos >= start && pos < end) {
                  part[head_at * kBlock + pos - 32 * t_lo] += y;
                  covered[pos - 32 * t_lo] = 1;
                }
              }
            }
          }
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 32 * (t_hi - t_lo); i += kWeightThreads)
        if (covered[i]) {
          float total = part[i];
          for (int h = 1; h < hg; ++h) total += part[h * kBlock + i];
          acc[seq * acc_stride + 32 * t_lo + i] += total;
        }
    }
    s0 = after;
  } while (s0 < a.n_seq);
}

// --- dispatch -----------------------------------------------------------------

// Heads up to which a whole workgroup joins one (a long sequence has hundreds of parts); beyond, there are
// few parts each and a wave does.
constexpr int64_t kJoinHeads = 512;

// Device us with shares of at least 1, 2, 4 and 8 pages, D = 128. 64 heads over 1 key head, 1 row: 512 positions 11.8, 12.8,
// 15.0, 17.8; 8,192 16.8, 14.9, 15.6, 19.7; 32,768 37.2, 24.6, 20.3, 21.7; 131,072 -, -, 40.2, 31.0; 16 rows of 2,048 26.6,
// 20.3, 18.8, 21.0. 32 over 8, 1 row: 64 7.9, 10.6, 16.2, 27.0; 2,048 9.8, 10.0, 11.3, 13.8; 8,192 13.9, 13.9, 13.0, 16.2.
template <class T, bool E4M3, int D, int TILES>
void decode_on(KvAttnArgs a, hipStream_t st) {
  const int groups = kKvDecodeGroups;
  // what one more part costs (its sums' bytes, its turn in the joining of its heads) by what a page takes, both in ns
  const double page_ns = TILES > 1 ? (D == 256 ? 1600 : 1000) : 100 + 2.75 * D;
  const double sums_ns = kv_group_rows(D, a.G) * D * 4 * 0.8e-3, turn_ns = a.Q * a.H <= kJoinHeads ? 20 : 80;
  const double pairs = static_cast<double>(a.Q) * a.Hkv * kv_head_groups(D, a.G);
  a.join_cost = static_cast<uint32_t>((sums_ns + turn_ns / pairs) / page_ns * 65536.0);
  if (a.Q > kKvPlanRows) kv_plan_kernel<<<dim3(1), dim3(1024), 0, st>>>(a);
  if constexpr (TILES == 1) kv_decode_kernel<T, E4M3, D><<<dim3(groups), dim3(kThreads), 0, st>>>(a);
  else kv_decode_staged_kernel<T, E4M3, D, TILES / 2><<<dim3(groups), dim3(kThreads), 0, st>>>(a);
  const int64_t heads = a.Q * a.H;
  if (heads <= kJoinHeads)
    kv_decode_join_kernel<T, D, kWaves><<<dim3(static_cast<unsigned>(heads)), dim3(kThreads), 0, st>>>(a, 16 * TILES, groups);
  else
    kv_decode_join_kernel<T, D, 1>
        <<<dim3(static_cast<unsigned>((heads + kWaves - 1) / kWaves)), dim3(kThreads), 0, st>>>(a, 16 * TILES, groups);
}

template <class T, bool E4M3, int D, int TILES>
void selected_on(const KvAttnArgs& a, hipStream_t st) {
  const int64_t items = a.Q * a.Hkv * kv_head_groups(D, a.G) * a.splits;
  const unsigned grid = static_cast<unsigned>((items + 7) / 8 * 8);
  if constexpr (TILES == 1) kv_selected_kernel<T, E4M3, D><<<dim3(grid), dim3(kThreads), 0, st>>>(a);
  else kv_selected_staged_kernel<T, E4M3, D, TILES / 2><<<dim3(grid), dim3(kThreads), 0, st>>>(a);
  if (a.splits > 1)
    kv_selected_join_kernel<T, D, 1>
        <<<dim3(static_cast<unsigned>((a.Q * a.H + kWaves - 1) / kWaves)), dim3(kThreads), 0, st>>>(a, 16 * TILES);
}

template <class T, bool E4M3, int D, int NQ>
void weights_on(const KvAttnArgs& a, const float* lse, float* acc, int64_t acc_stride, hipStream_t st) {
  // as many workgroups as 256 compute units hold: two of eight waves, three of four (32 sequences of 4K to 32K
  // under 64 heads 44 us; twice as many 50, as every workgroup plans for itself)
  int hg = 1;   // key heads at once
  if (NQ == 1)
    while (hg < weight_waves(NQ) && 2 * hg <= a.Hkv) hg *= 2;
  kv_weights_kernel<T, E4M3, D, NQ><<<dim3(NQ == 1 ? 512 : 768), dim3(64 * weight_waves(NQ)), 0, st>>>(a, lse, acc, acc_stride, hg);
}

// Calls f<type, 8-bit cache, dim, query tiles>() for the call's types and sizes.
template <class T, bool E4M3, class F>
void by_size(const KvAttnArgs& a, int nq, F&& f) {
  if (a.D == 64) {
    if (nq == 1) f.template operator()<T, E4M3, 64, 1>();
    else if (nq == 2) f.template operator()<T, E4M3, 64, 2>();
    else f.template operator()<T, E4M3, 64, 4>();
  } else if (a.D == 128) {
    if (nq == 1) f.template operator()<T, E4M3, 128, 1>();
    else if (nq == 2) f.template operator()<T, E4M3, 128, 2>();
    else f.template operator()<T, E4M3, 128, 4>();
  } else {
    if (nq == 1) f.template operator()<T, E4M3, 256, 1>();
    else f.template operator()<T, E4M3, 256, 2>();
  }
}

template <class F>
hipError_t by_type(const KvAttnArgs& a, int nq, F&& f) {
  const bool e4m3 = a.kv_type == MQA_KV_E4M3;
  if (a.q_type == MQA_KV_BF16) {
    if (e4m3) by_size<Bf16, true>(a, nq, f);
    else by_size<Bf16, false>(a, nq, f);
  } else {
    if (e4m3) by_size<Fp16, true>(a, nq, f);
    else by_size<Fp16, false>(a, nq, f);
  }
  return hipGetLastError();
}

struct DecodeOn {
  const KvAttnArgs& a;
  hipStream_t st;
  template <class T, bool E4M3, int D, int NQ>
  void operator()() const { decode_on<T, E4M3, D, NQ>(a, st); }
};
struct SelectedOn {
  const KvAttnArgs& a;
  hipStream_t st;
  template <class T, bool E4M3, int D, int NQ>
  void operator()() const { selected_on<T, E4M3, D, NQ>(a, st); }
};
struct WeightsOn {
  const KvAttnArgs& a;
  const float* lse;
  float* acc;
  int64_t acc_stride;
  hipStream_t st;
  template <class T, bool E4M3, int D, int NQ>
  void operator()() const { weights_on<T, E4M3, D, NQ>(a, lse, acc, acc_stride, st); }
};

}  // namespace

// Splits of the selected form, a power of two with no more workgroups than the device holds: the least sum of what a
// row's longest part takes (ns per 32 positions of a workgroup that runs alone, which takes one to four of them at
// once) and, where there are several parts, the launch that joins them, its trips to memory and the sums' bytes.
// Measured, us with 1, 2, 4, 8 and 16 splits under 64 heads, D = 128: 1 row of 512 slots 13.5, 13.0, 11.0, -, 11.3; 64
// rows of 512 14.5, 16.9, 18.2; 64 of 1,024 -, 21.6, 19.5, 23.3; 200 of 1,024 24.8, 33.3; 16 of 2,048 -, -, 18.7, 16.1, 18.3.
int32_t kv_selected_splits(int64_t Q, int64_t K, int D, int G, int Hkv) {
  const int64_t items = Q * Hkv * kv_head_groups(D, G), tiles = (K + kTilePos - 1) / kTilePos;
  const int64_t at_once = (G > 16 ? 2 : 4) / (D == 256 ? 2 : 1), tile_ns = (G > 16 ? 490 : 310) * (D == 256 ? 3 : 2) / 2;
  const int64_t join_ns = 2700;
  const int64_t part_ns = 80 + Q * Hkv * G * D * 4 / 1250;   // 0.8 ns per 1,000 bytes of sums
  int64_t best = 1, least = tiles * tile_ns;
  for (int64_t s = 2; s * items <= kKvDecodeGroups && s <= tiles; s *= 2) {
    const int64_t longest = ((tiles + s - 1) / s + at_once - 1) / at_once * at_once;
    const int64_t ns = longest * tile_ns + join_ns + s * part_ns;
    if (ns < least) {
      least = ns;
      best = s;
    }
  }
  return static_cast<int32_t>(best);
}

hipError_t launch_kv_decode(const KvAttnArgs& a, hipStream_t st) {
  return by_type(a, kv_tiles(a.D, a.G), DecodeOn{a, st});
}
hipError_t launch_kv_selected(const KvAttnArgs& a, hipStream_t st) {
  return by_type(a, kv_tiles(a.D, a.G), SelectedOn{a, st});
}
hipError_t launch_kv_weights(const KvAttnArgs& a, const float* lse, float* acc, int64_t acc_stride, hipStream_t st) {
  return by_type(a, kv_tiles(a.D, a.G), WeightsOn{a, lse, acc, acc_stride, st});
}

}  // namespace mqa
