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
// heads and is bound by memory. The four waves of a workgroup take every fourth
// 32-position tile; the next tile's keys are loaded into the registers that the
// first product has just read, its values into those that the second has.
#include "mqa_fp4_topk.h"
#include "mqa_kv.h"
#include "mqa_kv_cache.h"
#include "mqa_device.h"

namespace mqa {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kTilePos = 32;
constexpr float kLn2 = 0.69314718055994530942f;

struct Bf16 {
  static __device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
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
  static __device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                  0, 0);
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

// Maximum / sum over the four lane groups of 16 (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float groups_max(float x) {
  const uint32_t b = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t y = __float_as_uint(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
  const auto s = __builtin_amdgcn_permlane16_swap(y, y, false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

__device__ __forceinline__ float groups_sum(float x) {
  const uint32_t b = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t y = __float_as_uint(__uint_as_float(r[0]) + __uint_as_float(r[1]));
  const auto s = __builtin_amdgcn_permlane16_swap(y, y, false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// The registers and steps of one wave: NQ tiles of 16 query heads of one row and
// key head, 32 positions at a time.
template <class T, bool E4M3, int D, int NQ>
struct Wave {
  static constexpr int kBytes = E4M3 ? 1 : 2;
  static constexpr int kChunks = D / 32;                 // matrix steps over the dims
  static constexpr int kLoads = D * kBytes / 64;         // 16-byte key loads per lane and position
  static constexpr int kDims = D / 16;                   // dims of a position that a lane's values hold
  static constexpr int kWords = kDims * kBytes / 4;      // and their registers

  v4u q[NQ][kChunks];
  v4u k[2][kLoads];
  uint32_t v[8][kWords];
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

  // Query heads [0, rows) at `p`, one after another; the dims of a step are those
  // that the key loads put there.
  __device__ __forceinline__ void load_q(const char* p, int rows, uint32_t flip) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int h = 16 * n + col;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int dim = E4M3 ? 64 * (c >> 1) + 16 * grp + 8 * (c & 1) : 32 * c + 8 * grp;
        v4u x = {0, 0, 0, 0};
        if (h < rows) x = *reinterpret_cast<const v4u*>(p + (static_cast<int64_t>(h) * D + dim) * 2);
        q[n][c] = x ^ v4u{flip, flip, flip, flip};
      }
    }
  }

  // Position a * 16 + col of the tile is at `p`.
  __device__ __forceinline__ void load_k(int a, const char* p) {
#pragma unroll
    for (int c = 0; c < kLoads; ++c) k[a][c] = *reinterpret_cast<const v4u*>(p + 64 * c + 16 * grp);
  }

  // Position 16 (j / 4) + 4 grp + j % 4 of the tile is at `p`.
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
        v[j][e] = x.x;
        v[j][e + 1] = x.y;
        v[j][e + 2] = x.z;
        v[j][e + 3] = x.w;
      }
    }
  }

  __device__ __forceinline__ void scores(v4f (&s)[NQ][2]) {
#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) s[n][a] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        v4u x;
        if constexpr (E4M3) {
          const uint32_t w0 = k[a][c >> 1][2 * (c & 1)], w1 = k[a][c >> 1][2 * (c & 1) + 1];
          x = v4u{T::template from_e4m3<false>(w0), T::template from_e4m3<true>(w0),
                  T::template from_e4m3<false>(w1), T::template from_e4m3<true>(w1)};
        } else {
          x = k[a][c];
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) s[n][a] = T::mfma(x, q[n][c], s[n][a]);
      }
    }
  }

  // Scores to weights; `inside` bit j says whether this lane's j-th position counts
  // (all ones: every one). Returns the weights packed as the second product's operand.
  __device__ __forceinline__ void weights(v4f (&s)[NQ][2], float c, bool edge, uint32_t inside, v4u (&p)[NQ]) {
    float top[NQ];
    bool rise = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      if (edge) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!(inside >> j & 1)) s[n][j >> 2][j & 3] = -__builtin_inff();
      }
      float x = fmaxf(fmaxf(fmaxf(s[n][0][0], s[n][0][1]), fmaxf(s[n][0][2], s[n][0][3])),
                      fmaxf(fmaxf(s[n][1][0], s[n][1][1]), fmaxf(s[n][1][2], s[n][1][3])));
      top[n] = groups_max(x) * c;
      rise |= top[n] > m[n];
    }
    if (__any(rise)) {   // rare after the first tiles
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
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][j >> 2][j & 3], c, -ref));
        if (edge) w[j] = (inside >> j & 1) ? w[j] : 0.0f;
      }
      l[n] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
      p[n] = v4u{T::pack(w[0], w[1]), T::pack(w[2], w[3]), T::pack(w[4], w[5]), T::pack(w[6], w[7])};
    }
  }

  // Register e of dims pair e of position j, in the query's type.
  __device__ __forceinline__ uint32_t dims_pair(int j, int e) {
    if constexpr (E4M3) {
      return (e & 1) ? T::template from_e4m3<true>(v[j][e >> 1]) : T::template from_e4m3<false>(v[j][e >> 1]);
    } else {
      return v[j][e];
    }
  }

  // Values outside the window are whatever the cache holds there, NaN perhaps.
  __device__ __forceinline__ void clear_outside(uint32_t inside) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < kWords; ++e) v[j][e] = (inside >> j & 1) ? v[j][e] : 0u;
  }

  __device__ __forceinline__ void add_values(const v4u (&p)[NQ]) {
#pragma unroll
    for (int e = 0; e < kDims / 2; ++e) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = dims_pair(j, e);
      v4u even, odd;
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
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

// Joins the four waves' results in LDS and writes the heads' outputs, or their
// partial sums where part_o is not null. `bad`: this wave met an invalid page.
template <class T, int D, int NQ>
struct Merge {
  static constexpr int kPitch = D + 4;
  float o[kWaves][16][kPitch];
  float2 ml[kWaves][NQ * 16];
  float2 fin[NQ * 16];

  template <class W>
  __device__ __forceinline__ void run(W& w, bool bad, int rows, float v_scale, char* out, float* lse, float* part_o,
                                      float2* part_ml) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();   // the previous use of this memory is over
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const float sum = groups_sum(w.l[n]);
      if (w.grp == 0) ml[wave][16 * n + w.col] = make_float2(w.m[n], bad ? __builtin_nanf("") : sum);
    }
    __syncthreads();
    float f[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float2 x[kWaves];
      float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        x[i] = ml[i][16 * n + w.col];
        top = fmaxf(top, x[i].x);
      }
      const float ref = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) sum += x[i].y * __builtin_amdgcn_exp2f(x[i].x - ref);
      f[n] = __builtin_amdgcn_exp2f(w.m[n] - ref);
      if (wave == 0 && w.grp == 0) fin[16 * n + w.col] = make_float2(top, sum);
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      if (n > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < W::kDims; t += 4) {
          float* at = &o[wave][w.col][(4 * w.grp + i) * W::kDims + t];
          *reinterpret_cast<v4f*>(at) = v4f{w.o[n][t][i] * f[n], w.o[n][t + 1][i] * f[n], w.o[n][t + 2][i] * f[n],
                                            w.o[n][t + 3][i] * f[n]};
        }
      __syncthreads();
      for (int x = threadIdx.x; x < 16 * D / 4; x += kThreads) {
        const int h = x / (D / 4), d = 4 * (x % (D / 4)), head = 16 * n + h;
        if (head >= rows) continue;
        v4f sum = *reinterpret_cast<const v4f*>(&o[0][h][d]);
#pragma unroll
        for (int i = 1; i < kWaves; ++i) sum += *reinterpret_cast<const v4f*>(&o[i][h][d]);
        const float2 e = fin[head];
        if (part_o != nullptr) {
          *reinterpret_cast<v4f*>(part_o + static_cast<int64_t>(head) * D + d) = sum;
          if (d == 0) part_ml[head] = e;
        } else {
          const float inv = v_scale / e.y;
          const v2u y = {T::pack(sum[0] * inv, sum[1] * inv), T::pack(sum[2] * inv, sum[3] * inv)};
          *reinterpret_cast<v2u*>(out + (static_cast<int64_t>(head) * D + d) * 2) = y;
          if (d == 0 && lse != nullptr) lse[head] = (e.x + __builtin_amdgcn_logf(e.y)) * kLn2;
        }
      }
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

// Pages of one (row, head group) are its units of work; a workgroup takes
// `share` consecutive units of all (row, head group) pairs laid end to end, at least two pages.
__device__ __forceinline__ int64_t unit_share(int64_t units, int64_t groups) {
  const int64_t s = (units + groups - 1) / groups;
  return s < 2 ? 2 : s;
}

template <class T, bool E4M3, int D, int NQ>
__global__ void __launch_bounds__(kThreads, NQ == 1 && D < 256 ? 3 : 1) kv_decode_kernel(KvAttnArgs a) {
  typedef Wave<T, E4M3, D, NQ> W;
  __shared__ int64_t prefix_lds[kKvPlanRows + 1];
  __shared__ int64_t sums[kWaves];
  __shared__ Merge<T, D, NQ> merge;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t me = blockIdx.x;
  const int64_t* prefix = a.prefix;
  const int qg = (a.G + 16 * NQ - 1) / (16 * NQ);
  const int64_t gh = static_cast<int64_t>(a.Hkv) * qg;
  if (a.Q <= kKvPlanRows) {   // one round trip to memory, less than another launch
    constexpr int kPer = kKvPlanRows / kThreads;
    int64_t n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t r = kPer * threadIdx.x + i;
      int code = 0;
      n[i] = r < a.Q ? row_pages(a, r, &code) : 0;
      if (me == 0) report(a, code);
      sum += n[i];
    }
    int64_t total;
    int64_t at = block_scan<kWaves>(sum, sums, &total) - sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t r = kPer * threadIdx.x + i;
      if (r <= a.Q) {
        prefix_lds[r] = at;
        if (me == 0) a.prefix[r] = at;
      }
      at += n[i];
    }
    if (threadIdx.x == 0) {
      prefix_lds[a.Q] = total;
      if (me == 0) a.prefix[a.Q] = total;
    }
    __syncthreads();
    prefix = prefix_lds;
  }
  const int64_t units = prefix[a.Q] * gh;
  const int64_t share = unit_share(units, gridDim.x);
  int64_t cur = me * share;
  const int64_t stop = cur + share < units ? cur + share : units;
  const int group_rows = a.G < 16 * NQ ? a.G : 16 * NQ;

  W w;
  w.init();
  while (cur < stop) {
    // the row that unit `cur` belongs to: the last one whose prefix is not above it
    int64_t lo = 0, hi = a.Q;
    const int64_t page_unit = cur / gh;
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (prefix[mid] <= page_unit) lo = mid;
      else hi = mid;
    }
    const int64_t r = (static_cast<int64_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(lo >> 32))) << 32) |
                      static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(lo)));
    const int64_t n = prefix[r + 1] - prefix[r];
    const int64_t in_row = cur - prefix[r] * gh;
    const int g = __builtin_amdgcn_readfirstlane(static_cast<int>(in_row / n));
    const int pa = __builtin_amdgcn_readfirstlane(static_cast<int>(in_row - g * n));
    const int64_t left = stop - cur;
    const int pb = __builtin_amdgcn_readfirstlane(static_cast<int>(n - pa < left ? n : pa + left));
    cur += pb - pa;

    const int kvh = g / qg, first = (g % qg) * 16 * NQ;
    const int rows = a.G - first < 16 * NQ ? a.G - first : 16 * NQ;
    const int seq = a.seq_of_row[r], start = a.row_start[r], end = a.row_end[r];
    const int32_t* table = a.table + static_cast<int64_t>(seq) * a.max_pages;
    const int p0 = start >> 6;
    const int t_lo = 2 * (p0 + pa) > (start >> 5) ? 2 * (p0 + pa) : (start >> 5);
    const int t_hi = 2 * (p0 + pb) < ((end + 31) >> 5) ? 2 * (p0 + pb) : ((end + 31) >> 5);
    const char* kb = a.k + kvh * a.k_head;
    const char* vb = a.v + kvh * a.v_head;
    const int64_t head0 = r * a.H + static_cast<int64_t>(kvh) * a.G + first;
    w.start();
    w.load_q(a.q + r * a.q_row + (static_cast<int64_t>(kvh) * a.G + first) * D * 2, rows, a.q_flip);

    bool bad = false;
    auto page_of = [&](int t) {
      int p = table[t >> 1];
      if (p < 0 || p >= a.P_phys) {   // nothing of it is read; page 0 stands in
        bad = true;
        p = 0;
      }
      return p;
    };
    // positions outside the window are not read: their lanes read the nearest one inside
    auto clamp = [&](int pos) { return min(max(pos, start), end - 1) & 63; };
    auto load_keys = [&](int t, int page) {
      const char* base = kb + page * a.k_page;
#pragma unroll
      for (int b = 0; b < 2; ++b)
        w.load_k(b, base + static_cast<uint32_t>(clamp(32 * t + 16 * b + w.col) * static_cast<int>(a.k_pos)));
    };
    auto load_values = [&](int t, int page) {
      const char* base = vb + page * a.v_page;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w.load_v(j, base + static_cast<uint32_t>(clamp(32 * t + 16 * (j >> 2) + 4 * w.grp + (j & 3)) *
                                                 static_cast<int>(a.v_pos)));
    };
    int t = t_lo + wave;
    if (t < t_hi) {
      int page = page_of(t);
      load_keys(t, page);
      load_values(t, page);
      int next_page = t + kWaves < t_hi ? page_of(t + kWaves) : 0;
      while (true) {
        const int tn = t + kWaves;
        const bool more = tn < t_hi;
        const bool edge = 32 * t < start || 32 * t + 32 > end;
        uint32_t inside = 0xFFu;
        if (edge) {
          inside = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int pos = 32 * t + 16 * (j >> 2) + 4 * w.grp + (j & 3);
            inside |= (pos >= start && pos < end ? 1u : 0u) << j;
          }
        }
        v4f s[NQ][2];
        v4u p[NQ];
        w.scores(s);
        if (more) load_keys(tn, next_page);
        w.weights(s, a.c, edge, inside, p);
        if (edge) w.clear_outside(inside);
        w.add_values(p);
        if (!more) break;
        load_values(tn, next_page);
        if (tn + kWaves < t_hi) next_page = page_of(tn + kWaves);
        t = tn;
      }
    }
    if (bad && w.lane == 0) atomicOr(a.status, kStBadPage);
    const bool whole = pa == 0 && pb == n;
    const int64_t slot = 2 * me + (pa == 0 ? 1 : 0);
    merge.run(w, bad, rows, a.v_scale, static_cast<char*>(a.out) + head0 * D * 2,
              a.lse == nullptr ? nullptr : a.lse + head0, whole ? nullptr : a.part_o + slot * group_rows * D,
              a.part_ml + slot * group_rows);
  }
}

// --- joining partial sums -----------------------------------------------------

// Writes one head's row as a constant (0 for an empty window, NaN for a failed one).
template <class T, int D>
__device__ __forceinline__ void fill_row(const KvAttnArgs& a, int64_t head, bool failed) {
  const float x = failed ? __builtin_nanf("") : 0.0f;
  const uint32_t y = T::pack(x, x);
  for (int i = threadIdx.x; i < D / 2; i += kThreads) reinterpret_cast<uint32_t*>(a.out)[head * (D / 2) + i] = y;
  if (threadIdx.x == 0 && a.lse != nullptr) a.lse[head] = failed ? x : -__builtin_inff();
}

// One workgroup joins the partial sums of one (row, head): partial i < n is in
// slot slot0 + i * step (the first one in slot first_slot).
template <class T, int D>
__device__ __forceinline__ void join_row(const KvAttnArgs& a, int64_t head, int in_group, int group_rows, int64_t n,
                                         int64_t first_slot, int64_t slot0, int64_t step) {
  __shared__ float tops[kWaves];
  __shared__ float sums[kWaves];
  __shared__ float acc_lds[kWaves][D];
  constexpr int kPer = D / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto slot_of = [&](int64_t i) { return i == 0 ? first_slot : slot0 + i * step; };
  float top = -__builtin_inff();
  for (int64_t i = threadIdx.x; i < n; i += kThreads)
    top = fmaxf(top, a.part_ml[slot_of(i) * group_rows + in_group].x);
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  if (lane == 0) tops[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  const float ref = top == -__builtin_inff() ? 0.0f : top;
  float acc[kPer] = {}, sum = 0.0f;
#pragma unroll 8
  for (int64_t i = wave; i < n; i += kWaves) {
    const int64_t s = slot_of(i) * group_rows + in_group;
    const float2 ml = a.part_ml[s];
    const float f = __builtin_amdgcn_exp2f(ml.x - ref);
    sum += ml.y * f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] += f * a.part_o[s * D + lane + 64 * e];
  }
  if (lane == 0) sums[wave] = sum;
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc_lds[wave][lane + 64 * e] = acc[e];
  __syncthreads();
  sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  const float inv = a.v_scale / sum;
  for (int i = threadIdx.x; i < D / 2; i += kThreads) {
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      x[e] = ((acc_lds[0][2 * i + e] + acc_lds[1][2 * i + e]) + (acc_lds[2][2 * i + e] + acc_lds[3][2 * i + e])) * inv;
    reinterpret_cast<uint32_t*>(a.out)[head * (D / 2) + i] = T::pack(x[0], x[1]);
  }
  if (threadIdx.x == 0 && a.lse != nullptr) a.lse[head] = (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads) kv_decode_join_kernel(KvAttnArgs a, int nq, int groups) {
  const int64_t head = blockIdx.x;
  const int64_t r = head / a.H;
  const int h = static_cast<int>(head - r * a.H);
  const int64_t n = a.prefix[r + 1] - a.prefix[r];
  if (n == 0) {
    int code;
    row_pages(a, r, &code);
    fill_row<T, D>(a, head, code != 0);
    return;
  }
  const int qg = (a.G + 16 * nq - 1) / (16 * nq);
  const int64_t gh = static_cast<int64_t>(a.Hkv) * qg;
  const int64_t share = unit_share(a.prefix[a.Q] * gh, groups);
  const int kvh = h / a.G, in_kv = h - kvh * a.G;
  const int64_t from = a.prefix[r] * gh + (static_cast<int64_t>(kvh) * qg + in_kv / (16 * nq)) * n;
  const int64_t w0 = from / share, w1 = (from + n - 1) / share;
  if (w0 == w1) return;   // one workgroup had all of it and wrote the output
  // the first part is its workgroup's last one (slot 2 w + 1), the others are first ones (slot 2 w)
  join_row<T, D>(a, head, in_kv % (16 * nq), a.G < 16 * nq ? a.G : 16 * nq, w1 - w0 + 1, 2 * w0 + 1, 2 * w0, 2);
}

// --- selected form ------------------------------------------------------------

// Slots of one split of a row with n of them: whole tiles, the same for every split.
__device__ __forceinline__ int64_t split_share(int64_t n, int splits) {
  const int64_t tiles = (n + kTilePos - 1) / kTilePos;
  return (tiles + splits - 1) / splits * kTilePos;
}

template <class T, bool E4M3, int D, int NQ>
__global__ void __launch_bounds__(kThreads, NQ == 1 && D < 256 ? 3 : 1) kv_selected_kernel(KvAttnArgs a) {
  typedef Wave<T, E4M3, D, NQ> W;
  __shared__ int64_t k_off[kKvSelBlock];
  __shared__ int64_t v_off[kKvSelBlock];
  __shared__ Merge<T, D, NQ> merge;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int qg = (a.G + 16 * NQ - 1) / (16 * NQ);
  const int64_t gh = static_cast<int64_t>(a.Hkv) * qg;
  // Workgroups go to the eight dies in turn: each die gets a run of neighbouring
  // rows, whose lists share most of their slots, so that its L2 holds them.
  const int64_t per_die = (gridDim.x + 7) / 8;
  const int64_t item = (blockIdx.x & 7) * per_die + (blockIdx.x >> 3);
  if (item >= a.Q * gh * a.splits) return;
  const int64_t r = item / (gh * a.splits);
  const int64_t rest = item - r * gh * a.splits;
  const int g = static_cast<int>(rest / a.splits), split = static_cast<int>(rest - static_cast<int64_t>(g) * a.splits);
  const int kvh = g / qg, first = (g % qg) * 16 * NQ;
  const int rows = a.G - first < 16 * NQ ? a.G - first : 16 * NQ;
  const int64_t head0 = r * a.H + static_cast<int64_t>(kvh) * a.G + first;
  const int64_t n = a.count[r];
  if (n > a.K && rest == 0 && threadIdx.x == 0) atomicOr(a.status, kStBadWindow);
  if (n <= 0 || n > a.K) {
    if (split == 0)
      for (int h = 0; h < rows; ++h) fill_row<T, D>(a, head0 + h, n != 0);
    return;
  }
  const int64_t share = split_share(n, a.splits);
  const int64_t from = split * share;
  const int64_t to = from + share < n ? from + share : n;
  if (from >= to) return;

  W w;
  w.init();
  w.start();
  w.load_q(a.q + r * a.q_row + (static_cast<int64_t>(kvh) * a.G + first) * D * 2, rows, a.q_flip);
  const char* kb = a.k + kvh * a.k_head;
  const char* vb = a.v + kvh * a.v_head;
  const int32_t* list = a.slots + r * a.K;
  bool bad = false;
  for (int64_t b0 = from; b0 < to; b0 += kKvSelBlock) {
    const int len = static_cast<int>(to - b0 < kKvSelBlock ? to - b0 : kKvSelBlock);
    if (b0 != from) __syncthreads();
    bool mine = false;
    for (int i = threadIdx.x; i < len; i += kThreads) {
      const int s = list[b0 + i];
      const bool ok = s >= 0 && s < 64 * a.P_phys;
      mine |= !ok;
      const int page = s >> 6, pos = s & 63;
      k_off[i] = page * a.k_page + pos * a.k_pos;
      v_off[i] = page * a.v_page + pos * a.v_pos;
    }
    if (__syncthreads_or(mine)) {   // nothing of the list is read
      bad = true;
      break;
    }
    auto load_keys = [&](int t) {
#pragma unroll
      for (int b = 0; b < 2; ++b) w.load_k(b, kb + k_off[min(32 * t + 16 * b + w.col, len - 1)]);
    };
    auto load_values = [&](int t) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w.load_v(j, vb + v_off[min(32 * t + 16 * (j >> 2) + 4 * w.grp + (j & 3), len - 1)]);
    };
    const int tiles = (len + kTilePos - 1) / kTilePos;
    int t = wave;
    if (t < tiles) {
      load_keys(t);
      load_values(t);
      while (true) {
        const int tn = t + kWaves;
        const bool more = tn < tiles;
        const bool edge = 32 * t + 32 > len;
        uint32_t inside = 0xFFu;
        if (edge) {
          inside = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) inside |= (32 * t + 16 * (j >> 2) + 4 * w.grp + (j & 3) < len ? 1u : 0u) << j;
        }
        v4f s[NQ][2];
        v4u p[NQ];
        w.scores(s);
        if (more) load_keys(tn);
        w.weights(s, a.c, edge, inside, p);
        if (edge) w.clear_outside(inside);
        w.add_values(p);
        if (!more) break;
        load_values(tn);
        t = tn;
      }
    }
  }
  if (bad && threadIdx.x == 0) atomicOr(a.status, kStBadPage);
  const int group_rows = a.G < 16 * NQ ? a.G : 16 * NQ;
  const bool whole = a.splits == 1;
  merge.run(w, bad, rows, a.v_scale, static_cast<char*>(a.out) + head0 * D * 2,
            a.lse == nullptr ? nullptr : a.lse + head0, whole ? nullptr : a.part_o + item * group_rows * D,
            a.part_ml + item * group_rows);
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads) kv_selected_join_kernel(KvAttnArgs a, int nq) {
  const int64_t head = blockIdx.x;
  const int64_t r = head / a.H;
  const int h = static_cast<int>(head - r * a.H);
  const int64_t n = a.count[r];
  if (n <= 0 || n > a.K) return;   // written already
  const int qg = (a.G + 16 * nq - 1) / (16 * nq);
  const int kvh = h / a.G, in_kv = h - kvh * a.G;
  const int64_t share = split_share(n, a.splits);
  const int64_t slot = ((r * a.Hkv + kvh) * qg + in_kv / (16 * nq)) * a.splits;
  join_row<T, D>(a, head, in_kv % (16 * nq), a.G < 16 * nq ? a.G : 16 * nq, (n + share - 1) / share, slot, slot, 1);
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
template <class T, bool E4M3, int D, int NQ>
__global__ void __launch_bounds__(kThreads, NQ == 1 && D < 256 ? 4 : 2)
    kv_weights_kernel(KvAttnArgs a, const float* __restrict__ lse, float* __restrict__ acc, int64_t acc_stride) {
  typedef Wave<T, E4M3, D, NQ> W;
  __shared__ int seq_lo[kWeightSeqs], seq_hi[kWeightSeqs];
  __shared__ int64_t prefix[kWeightSeqs + 1];
  __shared__ int64_t sums[kWaves];
  __shared__ float part[kWeightTiles * kTilePos];
  __shared__ int covered[kWeightTiles * kTilePos];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t me = blockIdx.x;
  const int qg = (a.G + 16 * NQ - 1) / (16 * NQ);
  W w;
  w.init();
  for (int64_t s0 = 0; s0 < a.n_seq; s0 += kWeightSeqs) {
    // the positions that any row of each sequence looks at
    __syncthreads();
    for (int i = threadIdx.x; i < kWeightSeqs; i += kThreads) {
      seq_lo[i] = 0x7FFFFFFF;
      seq_hi[i] = 0;
    }
    __syncthreads();
    for (int64_t r = threadIdx.x; r < a.Q; r += kThreads) {
      int code = 0;
      const int n = row_pages(a, r, &code);
      if (me == 0 && s0 == 0) report(a, code);
      const int64_t i = a.seq_of_row[r] - s0;
      if (n > 0 && i >= 0 && i < kWeightSeqs) {
        atomicMin(&seq_lo[i], a.row_start[r]);
        atomicMax(&seq_hi[i], a.row_end[r]);
      }
    }
    __syncthreads();
    constexpr int kPer = kWeightSeqs / kThreads;
    int64_t n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = kPer * threadIdx.x + i;
      n[i] = seq_hi[x] > 0 ? (seq_hi[x] + 63) / 64 - seq_lo[x] / 64 : 0;
      sum += n[i];
    }
    int64_t units;
    int64_t at = block_scan<kWaves>(sum, sums, &units) - sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      prefix[kPer * threadIdx.x + i] = at;
      at += n[i];
    }
    if (threadIdx.x == 0) prefix[kWeightSeqs] = units;
    __syncthreads();

    const int64_t share = unit_share(units, gridDim.x);
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
      __syncthreads();
      for (int i = threadIdx.x; i < kWeightTiles * kTilePos; i += kThreads) {
        part[i] = 0.0f;
        covered[i] = 0;
      }
      __syncthreads();
      for (int64_t r0 = 0; r0 < a.Q; r0 += 64) {
        const int64_t rl = r0 + w.lane;
        bool mine = false;
        if (rl < a.Q && a.seq_of_row[rl] == seq) {
          int code;
          mine = row_pages(a, rl, &code) > 0 && a.row_start[rl] < 32 * t_hi && a.row_end[rl] > 32 * t_lo;
        }
        uint64_t todo = __ballot(mine);
        while (todo) {
          const int64_t r = r0 + __builtin_ctzll(todo);
          todo &= todo - 1;
          const int start = a.row_start[r], end = a.row_end[r];
          for (int g = 0; g < a.Hkv * qg; ++g) {
            const int kvh = g / qg, first = (g % qg) * 16 * NQ;
            const int rows = a.G - first < 16 * NQ ? a.G - first : 16 * NQ;
            const int64_t head0 = r * a.H + static_cast<int64_t>(kvh) * a.G + first;
            w.load_q(a.q + r * a.q_row + (static_cast<int64_t>(kvh) * a.G + first) * D * 2, rows, 0u);
            float sub[NQ];
            bool counts[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              const int h = 16 * n + w.col;
              sub[n] = h < rows ? lse[head0 + h] : __builtin_inff();
              counts[n] = __builtin_fabsf(sub[n]) < __builtin_inff();
            }
            for (int t = t_lo + wave; t < t_hi; t += kWaves) {
              if (32 * t + 32 <= start || 32 * t >= end) continue;
              const int page = table[t >> 1];
              if (page < 0 || page >= a.P_phys) {
                if (w.lane == 0) atomicOr(a.status, kStBadPage);
                continue;
              }
              const char* base = a.k + kvh * a.k_head + page * a.k_page;
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const int pos = min(max(32 * t + 16 * b + w.col, start), end - 1) & 63;
                w.load_k(b, base + static_cast<uint32_t>(pos * static_cast<int>(a.k_pos)));
              }
              v4f s[NQ][2];
              w.scores(s);
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
              if (w.col < 8) {
                const int pos = 32 * t + 16 * (w.col >> 2) + 4 * w.grp + (w.col & 3);
                if (pos >= start && pos < end) {
                  part[pos - 32 * t_lo] += y;
                  covered[pos - 32 * t_lo] = 1;
                }
              }
            }
          }
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 32 * (t_hi - t_lo); i += kThreads)
        if (covered[i]) acc[seq * acc_stride + 32 * t_lo + i] += part[i];
    }
  }
}

// --- dispatch -----------------------------------------------------------------

template <class T, bool E4M3, int D, int NQ>
void decode_on(const KvAttnArgs& a, hipStream_t st) {
  const int groups = kv_decode_groups(D, a.G);
  if (a.Q > kKvPlanRows) kv_plan_kernel<<<dim3(1), dim3(1024), 0, st>>>(a);
  kv_decode_kernel<T, E4M3, D, NQ><<<dim3(groups), dim3(kThreads), 0, st>>>(a);
  kv_decode_join_kernel<T, D><<<dim3(static_cast<unsigned>(a.Q * a.H)), dim3(kThreads), 0, st>>>(a, NQ, groups);
}

template <class T, bool E4M3, int D, int NQ>
void selected_on(const KvAttnArgs& a, hipStream_t st) {
  const int64_t items = a.Q * a.Hkv * kv_q_groups(D, a.G) * a.splits;
  const unsigned grid = static_cast<unsigned>((items + 7) / 8 * 8);
  kv_selected_kernel<T, E4M3, D, NQ><<<dim3(grid), dim3(kThreads), 0, st>>>(a);
  if (a.splits > 1)
    kv_selected_join_kernel<T, D><<<dim3(static_cast<unsigned>(a.Q * a.H)), dim3(kThreads), 0, st>>>(a, NQ);
}

template <class T, bool E4M3, int D, int NQ>
void weights_on(const KvAttnArgs& a, const float* lse, float* acc, int64_t acc_stride, hipStream_t st) {
  kv_weights_kernel<T, E4M3, D, NQ><<<dim3(kKvWeightGroups), dim3(kThreads), 0, st>>>(a, lse, acc, acc_stride);
}

// Calls f<type, 8-bit cache, dim, query tiles>() for the call's types and sizes.
template <class T, bool E4M3, class F>
void by_size(const KvAttnArgs& a, F&& f) {
  const int nq = kv_q_tiles(a.D, a.G);
  if (a.D == 64) {
    if (nq == 1) f.template operator()<T, E4M3, 64, 1>();
    else f.template operator()<T, E4M3, 64, 4>();
  } else if (a.D == 128) {
    if (nq == 1) f.template operator()<T, E4M3, 128, 1>();
    else f.template operator()<T, E4M3, 128, 4>();
  } else {
    if (nq == 1) f.template operator()<T, E4M3, 256, 1>();
    else f.template operator()<T, E4M3, 256, 2>();
  }
}

template <class F>
hipError_t by_type(const KvAttnArgs& a, F&& f) {
  const bool e4m3 = a.kv_type == MQA_KV_E4M3;
  if (a.q_type == MQA_KV_BF16) {
    if (e4m3) by_size<Bf16, true>(a, f);
    else by_size<Bf16, false>(a, f);
  } else {
    if (e4m3) by_size<Fp16, true>(a, f);
    else by_size<Fp16, false>(a, f);
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

// Splits of the selected form: one workgroup per (row, head group) once they
// fill the device, else enough splits of at least four tiles each.
int32_t kv_selected_splits(int64_t Q, int64_t K, int D, int G, int Hkv) {
  const int64_t items = Q * Hkv * kv_q_groups(D, G);
  const int64_t room = kv_decode_groups(D, G);
  int64_t s = items <= 0 ? 1 : room / items;
  const int64_t most = (K + 4 * kTilePos - 1) / (4 * kTilePos);
  if (s > most) s = most;
  return static_cast<int32_t>(s < 1 ? 1 : s);
}

hipError_t launch_kv_decode(const KvAttnArgs& a, hipStream_t st) { return by_type(a, DecodeOn{a, st}); }
hipError_t launch_kv_selected(const KvAttnArgs& a, hipStream_t st) { return by_type(a, SelectedOn{a, st}); }
hipError_t launch_kv_weights(const KvAttnArgs& a, const float* lse, float* acc, int64_t acc_stride, hipStream_t st) {
  return by_type(a, WeightsOn{a, lse, acc, acc_stride, st});
}

}  // namespace mqa
