// Attention over a paged key-value cache in 4 bits (gfx950). Formulas, tiles and the
// operands' layout are those of mqa_kv_attn.hip; keys and values are made 16-bit numbers in
// registers, exactly, right before their product: one instruction makes two numbers of a
// byte and their block's power of two.
//
// Every wave streams its own tiles of 32 positions through LDS: asynchronous copies (memory to
// LDS, no registers) fill a ring of kDepth tiles, keys and values apart, and as soon as a
// tile's keys (values) are in registers the copies of the tile kDepth further go into their
// place. Nothing is shared between waves, so there are no barriers, only a count of
// copies to wait for. The reads are inline assembly, each block with its own wait: the
// compiler would wait for every copy in flight before an LDS read that it cannot prove apart.
//
// Few heads on a key head are bound by memory (32 sequences of 2K-16K positions, 32 heads on 8 of 128 dims: 82 us, 4.0
// TB/s of codes and scales), 64 by the vector and matrix units, which hardly run beside each other (64 sequences of
// 32K-131K on one key head: 227 us, 54 and 38 % of the clocks; 2,048 lists of 1,024 slots 106 us, 53 and 27 %), short sequences by code that runs
// once from a cold instruction cache (1,500 positions: 10.6 us, and 4.0 for the joining launch).
#include "mqa_kv_attn.h"

namespace mqa {
namespace {

template <int SEL>
__device__ __forceinline__ uint32_t pair_of(Bf16, uint32_t w, uint32_t scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, __uint_as_float(scale), SEL));
}
template <int SEL>
__device__ __forceinline__ uint32_t pair_of(Fp16, uint32_t w, uint32_t scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, __uint_as_float(scale), SEL));
}

// A word of scale bytes turned so that the wanted one lies at a 32-bit number's exponent, which is
// all that the conversions look at. shift: 8 * byte + 9.
__device__ __forceinline__ uint32_t scale_of(uint32_t word, uint32_t shift) { return __builtin_amdgcn_alignbit(word, word, shift); }

// A wave's tile of 32 positions over a cache in 4 bits. Lane (col, grp) holds, of keys 16 a + col, the codes of
// D / 4 dims, 32 of a block at most, and of values mine(j) those of D / 16 neighbouring ones.
//
// More than 16 heads: the running maximum may lag by 2^8.
template <class T, int D, int NQ>
struct Wave4 : Wave<T, false, D, NQ, 32, true, (NQ > 1 ? 8 : 0)> {
  typedef Wave<T, false, D, NQ, 32, true, (NQ > 1 ? 8 : 0)> Base;   // (queries and loads are this one's own)
  using Base::kChunks;
  using Base::kDims;
  using Base::kMine;
  using Base::kTiles;
  using Base::col;
  using Base::grp;
  typedef typename Base::P P;
  static constexpr int kKeyBlocks = D == 256 ? 2 : 1;    // scales of a lane's key
  static constexpr int kKeyWords = D / 32;               // words of 8 codes of a lane's key
  // Tiles of 16 heads whose queries stay in registers, as many as there is room for (64 heads, D = 128: 1, 2 and 3 of the four
  // 238, 277 and 350 us, from the second on with spills); those of the others lie in LDS.
  static constexpr int kHeld = D == 64 || NQ == 1 || (D == 128 && NQ == 2) ? NQ : D == 128 ? 1 : 0;
  static constexpr int kInLds = NQ - kHeld;
  static constexpr int kWords4 = D == 256 ? 2 : 1;       // words of a lane's value (half of one with D = 64)

  v4u q[kHeld > 0 ? kHeld : 1][kChunks];
  const v4u* q_lane;                                     // those in LDS, from this lane's on
  uint32_t kc[kTiles][kKeyWords], kb[kTiles][kKeyBlocks];
  uint32_t vc[kMine][kWords4], vb[kMine];

  // First dim of matrix step c in this lane's keys.
  __device__ __forceinline__ int step_dim(int c) const {
    return D == 64 ? 16 * grp + 8 * c : 128 * (c >> 2) + 32 * grp + 8 * (c & 3);
  }

  // This lane's part of step c of query tile n, of heads [0, rows) at `p`.
  __device__ __forceinline__ v4u query(const char* p, int n, int c, int rows) const {
    const int h = 16 * n + col;
    v4u x = {0, 0, 0, 0};
    if (h < rows) x = *reinterpret_cast<const v4u*>(p + (static_cast<int64_t>(h) * D + step_dim(c)) * 2);
    return x;
  }

  // Asks for the queries that stay in registers, and loads the others, by the whole workgroup, into `lds` (kInLds *
  // kChunks * 64 of it, which nobody reads any more).
  template <int WAVES>
  __device__ __forceinline__ void load_q(const char* p, int rows, uint32_t keep, uint32_t flip, v4u* lds) {
#pragma unroll
    for (int n = 0; n < kHeld; ++n)
#pragma unroll
      for (int c = 0; c < kChunks; ++c) q[n][c] = query(p, n, c, rows);
    if constexpr (kInLds > 0) {
      q_lane = lds + this->lane;
      constexpr int kPer = (kInLds * kChunks + WAVES - 1) / WAVES;
      v4u x[kPer];   // all asked for before the first is waited for
      const int first = threadIdx.x >> 6;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = first + WAVES * i;
        x[i] = query(p, kHeld + at / kChunks, at % kChunks, at < kInLds * kChunks ? rows : 0);
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = first + WAVES * i;
        if (at < kInLds * kChunks) lds[64 * at + this->lane] = (x[i] & v4u{keep, keep, keep, keep}) ^ v4u{flip, flip, flip, flip};
      }
      lds_barrier();
    }
  }

  // Takes those in registers, once their tiles' first copies are on their way.
  __device__ __forceinline__ void take_q(uint32_t keep, uint32_t flip) {
#pragma unroll
    for (int n = 0; n < kHeld; ++n)
#pragma unroll
      for (int c = 0; c < kChunks; ++c) q[n][c] = (q[n][c] & v4u{keep, keep, keep, keep}) ^ v4u{flip, flip, flip, flip};
  }

  __device__ __forceinline__ void keys_of(int c, v4u (&x)[kTiles]) const {
#pragma unroll
    for (int a = 0; a < kTiles; ++a) {
      const uint32_t w = kc[a][c], by = kb[a][D == 256 ? c >> 2 : 0];
      x[a] = v4u{pair_of<0>(T{}, w, by), pair_of<1>(T{}, w, by), pair_of<2>(T{}, w, by), pair_of<3>(T{}, w, by)};
    }
  }

  // Scores of the tile that lies in kc and kb: 32 dims of every key at a time, under all queries.
  __device__ __forceinline__ void scores(v4f (&s)[NQ][kTiles]) const {
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int a = 0; a < kTiles; ++a) s[n][a] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      v4u x[kTiles];
      keys_of(c, x);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        v4u y;
        if (n < kHeld) y = q[n < kHeld ? n : 0][c];
        else y = q_lane[((n - kHeld) * kChunks + c) * 64];
#pragma unroll
        for (int a = 0; a < kTiles; ++a) s[n][a] = T::mfma(x[a], y, s[n][a]);
      }
    }
    settle(s);
  }

  // First half of Wave::weights: the mask of a window's edge, and the running maximum.
  __device__ __forceinline__ void follow_maximum(v4f (&s)[NQ][kTiles], float c, bool edge, uint32_t inside) {
    if (edge) {   // a score of -infinity is a weight of 0, as c > 0
      const uint32_t in = Base::here(inside);
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int j = 0; j < kMine; ++j) s[n][j >> 2][j & 3] = (in >> j & 1) ? s[n][j >> 2][j & 3] : -__builtin_inff();
    }
    // A lane's own scores tell whether the maximum moves; the other lanes' are asked for only if it does.
    float top[NQ];
    bool rise = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      top[n] = max3(max3(max3(s[n][0][0], s[n][0][1], s[n][0][2]), s[n][0][3], s[n][1][0]), s[n][1][1], max2(s[n][1][2], s[n][1][3]));
      const float least = static_cast<float>(Base::kBias + (NQ > 1 ? 8 : 0));
      rise |= (least == 0.0f ? top[n] * c : __builtin_fmaf(top[n], c, -least)) > this->m[n];
    }
    if (__any(rise)) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float mine = groups_max(top[n]);
        const float to = fmaxf(this->m[n], Base::kBias == 0 ? mine * c : __builtin_fmaf(mine, c, static_cast<float>(-Base::kBias)));
        const float f = to == this->m[n] ? 1.0f : __builtin_amdgcn_exp2f(this->m[n] - to);
        this->m[n] = to;
        this->l[n] *= f;
#pragma unroll
        for (int t = 0; t < kDims; ++t) this->o[n][t] *= f;
      }
    }
  }

  // The running maximum begins at the least number: a score of -infinity under it weighs 0.
  __device__ __forceinline__ void start() {
    Base::start();
#pragma unroll
    for (int n = 0; n < NQ; ++n) this->m[n] = -3.402823466e38f;
  }

  // Second half: weights, their sums and the weighted values.
  __device__ __forceinline__ void add_weighted(const v4f (&s)[NQ][kTiles], float c) {
    P p[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float w[kMine];
#pragma unroll
      for (int j = 0; j < kMine; ++j) w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][j >> 2][j & 3], c, -this->m[n]));
      this->l[n] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
#pragma unroll
      for (int j = 0; j < kMine / 2; ++j) p[n][j] = T::pack(w[2 * j], w[2 * j + 1]);
    }
    add_values(p);
  }

  // Values outside the window: every code is a number, so a scale of nearly 0 will do.
  __device__ __forceinline__ void clear_outside(uint32_t inside) {
    inside = Base::here(inside);
#pragma unroll
    for (int j = 0; j < kMine; ++j) vb[j] = (inside >> j & 1) ? vb[j] : 0u;
  }

  template <int E>
  __device__ __forceinline__ void add_pair(const P (&p)[NQ]) {
    uint32_t w[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) w[j] = pair_of<(E & 3)>(T{}, vc[j][E >> 2], vb[j]);
    P even, odd;
#pragma unroll
    for (int jj = 0; jj < kMine / 2; ++jj) {
      even[jj] = __builtin_amdgcn_perm(w[2 * jj + 1], w[2 * jj], 0x05040100u);   // low halves
      odd[jj] = __builtin_amdgcn_perm(w[2 * jj + 1], w[2 * jj], 0x07060302u);    // high halves
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      this->o[n][2 * E] = T::mfma(even, p[n], this->o[n][2 * E]);
      this->o[n][2 * E + 1] = T::mfma(odd, p[n], this->o[n][2 * E + 1]);
    }
  }

  __device__ __forceinline__ void add_values(const P (&p)[NQ]) {
    add_pair<0>(p);
    add_pair<1>(p);
    if constexpr (D >= 128) {
      add_pair<2>(p);
      add_pair<3>(p);
    }
    if constexpr (D >= 256) {
      add_pair<4>(p);
      add_pair<5>(p);
      add_pair<6>(p);
      add_pair<7>(p);
    }
  }
};

// --- a wave's stream of tiles ---------------------------------------------------

// Waves of a workgroup of NH key heads, and workgroups of a launch: four waves of it to a SIMD where registers and LDS
// leave room for them, two otherwise.
constexpr int ring_waves(int D, int NQ, int NH) { return NH > 1 || (NQ == 1 && D <= 128) ? 8 : 4; }
constexpr int ring_groups(int NH) { return kKvDecodeGroups / NH; }
constexpr int ring_waves_per_simd(int D, int NQ, int NH) { return NQ == 1 && NH == 1 && D <= 128 ? 4 : 2; }

// LDS of the waves' rings. A piece is the keys or values of a tile under NH neighbouring key heads: 32 rows of NH * D / 2
// bytes of codes, one after another, and their scales, head by head, one word a row (two with D = 256; with D = 64 the
// upper half is empty).
//
// kDepth: as many tiles as LDS holds for all workgroups of a compute unit.
template <class T, int D, int NQ, int NH>
struct Ring4 {
  typedef Wave4<T, D, NQ> W;
  static constexpr int kHeadRow = D / 2, kRow = NH * kHeadRow, kCodes = 32 * kRow, kScaleWords = D == 256 ? 2 : 1;
  static constexpr int kHeadScales = 32 * 4 * kScaleWords, kPiece = kCodes + NH * kHeadScales;
  static constexpr int kWaves = ring_waves(D, NQ, NH);
  static constexpr int kDepth = NH > 1 ? (D == 64 ? 3 : 2) : D == 64 ? (NQ == 1 ? 3 : 4) : D == 128 ? (NQ == 1 ? 2 : 3) : (NQ == 1 ? 2 : 1);
  static constexpr int kParts = kRow / 16;                   // 16-byte parts of a row, and lanes that copy one
  static constexpr int kCopyRows = 64 / kParts;              // rows of one copy of 1 KiB
  static constexpr int kCodeCopies = kCodes / 1024, kCopies = kCodeCopies + 1;   // per piece
  static_assert(NH * kHeadScales <= 256, "one copy takes all scales of a piece");
  char piece[kWaves][kDepth][2][kPiece];

  // Keys lie with the parts of a row permuted by its number, so that the rows that one read takes fall on
  // different banks. The same for every copy of a piece.
  static __device__ __forceinline__ int swizzle(int row) { return kParts == 2 ? row >> 3 & 1 : kParts == 4 ? row >> 1 & 3 : row & 7; }

  // What this lane copies: its row in the first copy of a piece, its head and its bytes of that head's row.
  static __device__ __forceinline__ int code_row(int lane) { return lane / kParts; }
  static __device__ __forceinline__ int code_part(int kv, int lane) { return kv == 0 ? lane % kParts ^ swizzle(code_row(lane)) : lane % kParts; }
  static __device__ __forceinline__ int code_head(int kv, int lane) { return code_part(kv, lane) / (kHeadRow / 16); }
  static __device__ __forceinline__ int code_byte(int kv, int lane) { return 16 * (code_part(kv, lane) % (kHeadRow / 16)); }
  static __device__ __forceinline__ int scale_row(int lane) { return D == 256 ? lane >> 1 : lane & 31; }
  static __device__ __forceinline__ int scale_head(int lane) { return NH > 1 ? lane >> 5 : 0; }
  static __device__ __forceinline__ int scale_byte(int lane) { return D == 256 ? 4 * (lane & 1) : 0; }

  // Copy i of a piece's codes, and of its scales.
  __device__ __forceinline__ void copy(int wave, int stage, int kv, int i, const char* src) {
    __builtin_amdgcn_global_load_lds(src, &piece[wave][stage][kv][1024 * i], 16, 0, 0);
  }
  __device__ __forceinline__ void copy_scales(int wave, int stage, int kv, int lane, const char* src) {
    if (NH * kHeadScales == 256 || lane < 32) __builtin_amdgcn_global_load_lds(src, &piece[wave][stage][kv][kCodes], D == 64 ? 2 : 4, 0, 0);
  }

  // The same from a scalar base, `off` bytes and a lane's own offset behind it (all together below 2^31).
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t page_at(const char* base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, 0x7FFFFFFF, 0x00027000);
  }
  __device__ __forceinline__ void copy(int wave, int stage, int kv, int i, __amdgpu_buffer_rsrc_t page, int off, uint32_t lane_at) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(page, &piece[wave][stage][kv][1024 * i], 16, lane_at, off, 0, 0);
  }
  __device__ __forceinline__ void copy_scales(int wave, int stage, int kv, int lane, __amdgpu_buffer_rsrc_t page, int off, uint32_t lane_at) {
    if (NH * kHeadScales == 256 || lane < 32)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(page, &piece[wave][stage][kv][kCodes], D == 64 ? 2 : 4, lane_at, off, 0, 0);
  }

  // Waits until the oldest piece in flight is there: `more` younger ones at least are on their way.
  static __device__ __forceinline__ void arrived(int more) {
    constexpr int kYounger = 2 * kDepth - 1;
    if (more >= kYounger) __asm__ __volatile__("s_waitcnt vmcnt(%0)" ::"n"(kYounger * kCopies) : "memory");
    else __asm__ __volatile__("s_waitcnt vmcnt(0)" ::: "memory");
  }

  // Keys 16 a + col of head h of a piece into w.kc and w.kb.
  static __device__ __forceinline__ void read_keys(W& w, uint32_t at, int h, uint32_t shift) {
    const uint32_t row = at + w.col * kRow, scales = at + kCodes + h * kHeadScales + 4 * kScaleWords * w.col;
    const int z = swizzle(w.col);
    if constexpr (D == 64) {
      const uint32_t codes = row + 16 * ((2 * h + (w.grp >> 1)) ^ z) + 8 * (w.grp & 1);
      v2u x, y;
      uint32_t sx, sy;
      __asm__ __volatile__(
          "ds_read_b64 %0, %4\n\tds_read_b64 %1, %4 offset:%6\n\t"
          "ds_read_b32 %2, %5\n\tds_read_b32 %3, %5 offset:64\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x), "=&v"(y), "=&v"(sx), "=&v"(sy)
          : "v"(codes), "v"(scales), "n"(16 * kRow)
          : "memory");
      w.kc[0][0] = x.x;
      w.kc[0][1] = x.y;
      w.kc[1][0] = y.x;
      w.kc[1][1] = y.y;
      w.kb[0][0] = scale_of(sx, shift);
      w.kb[1][0] = scale_of(sy, shift);
    } else if constexpr (D == 128) {
      const uint32_t codes = row + 16 * ((4 * h + w.grp) ^ z);
      v4u x, y;
      uint32_t sx, sy;
      __asm__ __volatile__(
          "ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:%6\n\t"
          "ds_read_b32 %2, %5\n\tds_read_b32 %3, %5 offset:64\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x), "=&v"(y), "=&v"(sx), "=&v"(sy)
          : "v"(codes), "v"(scales), "n"(16 * kRow)
          : "memory");
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w.kc[0][e] = x[e];
        w.kc[1][e] = y[e];
      }
      w.kb[0][0] = scale_of(sx, shift);
      w.kb[1][0] = scale_of(sy, shift);
    } else {
      const uint32_t codes = row + 16 * (w.grp ^ z), other = row + 16 * (w.grp ^ z ^ 4);
      v4u x[4];
      v2u s[2];
      __asm__ __volatile__(
          "ds_read_b128 %0, %6\n\tds_read_b128 %1, %7\n\t"
          "ds_read_b128 %2, %6 offset:2048\n\tds_read_b128 %3, %7 offset:2048\n\t"
          "ds_read_b64 %4, %8\n\tds_read_b64 %5, %8 offset:128\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(s[0]), "=&v"(s[1])
          : "v"(codes), "v"(other), "v"(scales)
          : "memory");
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w.kc[a][4 * i + e] = x[2 * a + i][e];
          w.kb[a][i] = scale_of(s[a][i], shift);
        }
    }
  }

  // Values mine(j) of head h of a piece into w.vc and w.vb.
  static __device__ __forceinline__ void read_values(W& w, uint32_t at, int h, uint32_t shift) {
    const uint32_t codes = at + 4 * w.grp * kRow + h * kHeadRow + w.col * (D / 32);
    const uint32_t scales = at + kCodes + h * kHeadScales + 16 * kScaleWords * w.grp + (D == 256 ? 4 * (w.col >> 3) : 0);
    if constexpr (D == 256) {
      v2u x[8], s[4];
      __asm__ __volatile__(
          "ds_read_b64 %0, %12\n\tds_read_b64 %1, %12 offset:128\n\t"
          "ds_read_b64 %2, %12 offset:256\n\tds_read_b64 %3, %12 offset:384\n\t"
          "ds_read_b64 %4, %12 offset:2048\n\tds_read_b64 %5, %12 offset:2176\n\t"
          "ds_read_b64 %6, %12 offset:2304\n\tds_read_b64 %7, %12 offset:2432\n\t"
          "ds_read2_b32 %8, %13 offset0:0 offset1:2\n\tds_read2_b32 %9, %13 offset0:4 offset1:6\n\t"
          "ds_read2_b32 %10, %13 offset0:32 offset1:34\n\tds_read2_b32 %11, %13 offset0:36 offset1:38\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7]),
            "=&v"(s[0]), "=&v"(s[1]), "=&v"(s[2]), "=&v"(s[3])
          : "v"(codes), "v"(scales)
          : "memory");
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w.vc[j][0] = x[j].x;
        w.vc[j][1] = x[j].y;
        w.vb[j] = scale_of(s[j / 2][j & 1], shift);
      }
    } else {
      v4u s[2];
      if constexpr (D == 128) {
        __asm__ __volatile__(
            "ds_read_b32 %0, %10\n\tds_read_b32 %1, %10 offset:%12\n\t"
            "ds_read_b32 %2, %10 offset:%13\n\tds_read_b32 %3, %10 offset:%14\n\t"
            "ds_read_b32 %4, %10 offset:%15\n\tds_read_b32 %5, %10 offset:%16\n\t"
            "ds_read_b32 %6, %10 offset:%17\n\tds_read_b32 %7, %10 offset:%18\n\t"
            "ds_read_b128 %8, %11\n\tds_read_b128 %9, %11 offset:64\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(w.vc[0][0]), "=&v"(w.vc[1][0]), "=&v"(w.vc[2][0]), "=&v"(w.vc[3][0]), "=&v"(w.vc[4][0]),
              "=&v"(w.vc[5][0]), "=&v"(w.vc[6][0]), "=&v"(w.vc[7][0]), "=&v"(s[0]), "=&v"(s[1])
            : "v"(codes), "v"(scales), "n"(kRow), "n"(2 * kRow), "n"(3 * kRow), "n"(16 * kRow), "n"(17 * kRow), "n"(18 * kRow),
              "n"(19 * kRow)
            : "memory");
      } else {
        __asm__ __volatile__(
            "ds_read_u16 %0, %10\n\tds_read_u16 %1, %10 offset:%12\n\t"
            "ds_read_u16 %2, %10 offset:%13\n\tds_read_u16 %3, %10 offset:%14\n\t"
            "ds_read_u16 %4, %10 offset:%15\n\tds_read_u16 %5, %10 offset:%16\n\t"
            "ds_read_u16 %6, %10 offset:%17\n\tds_read_u16 %7, %10 offset:%18\n\t"
            "ds_read_b128 %8, %11\n\tds_read_b128 %9, %11 offset:64\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(w.vc[0][0]), "=&v"(w.vc[1][0]), "=&v"(w.vc[2][0]), "=&v"(w.vc[3][0]), "=&v"(w.vc[4][0]),
              "=&v"(w.vc[5][0]), "=&v"(w.vc[6][0]), "=&v"(w.vc[7][0]), "=&v"(s[0]), "=&v"(s[1])
            : "v"(codes), "v"(scales), "n"(kRow), "n"(2 * kRow), "n"(3 * kRow), "n"(16 * kRow), "n"(17 * kRow), "n"(18 * kRow),
              "n"(19 * kRow)
            : "memory");
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) w.vb[j] = scale_of(s[j / 4][j & 3], shift);
    }
  }

  // This lane's slots of a tile: of the rows that it copies codes of, and scales.
  static __device__ __forceinline__ void read_slots(int (&slot)[kCodeCopies], int* scale_slot, uint32_t codes, uint32_t scales) {
    if constexpr (kCodeCopies == 4) {
      __asm__ __volatile__(
          "ds_read_b32 %0, %5\n\tds_read_b32 %1, %5 offset:%7\n\tds_read_b32 %2, %5 offset:%8\n\t"
          "ds_read_b32 %3, %5 offset:%9\n\tds_read_b32 %4, %6\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(slot[0]), "=&v"(slot[1]), "=&v"(slot[2]), "=&v"(slot[3]), "=&v"(*scale_slot)
          : "v"(codes), "v"(scales), "n"(4 * kCopyRows), "n"(8 * kCopyRows), "n"(12 * kCopyRows)
          : "memory");
    } else if constexpr (kCodeCopies == 2) {
      __asm__ __volatile__("ds_read_b32 %0, %3\n\tds_read_b32 %1, %3 offset:%5\n\tds_read_b32 %2, %4\n\ts_waitcnt lgkmcnt(0)"
                           : "=&v"(slot[0]), "=&v"(slot[1]), "=&v"(*scale_slot)
                           : "v"(codes), "v"(scales), "n"(4 * kCopyRows)
                           : "memory");
    } else {
      static_assert(kCodeCopies == 1, "one, two or four");
      __asm__ __volatile__("ds_read_b32 %0, %2\n\tds_read_b32 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                           : "=&v"(slot[0]), "=&v"(*scale_slot)
                           : "v"(codes), "v"(scales)
                           : "memory");
    }
  }

  // This wave's tiles t, t + kWaves, ... below t_hi. keys(t, stage) and values(t, stage) issue the copies of one
  // piece, values those of the tile that keys was last called for; range(t, &lo, &hi) gives the positions that count.
  // ready() is called by every wave once its first copies are on their way. Other loads and stores may be in flight
  // when the copies are counted: loads arrive in order, so one more of either only makes a wait longer.
  template <class KEYS, class VALUES, class RANGE, class READY>
  __device__ __forceinline__ void run(W (&w)[NH], int wave, int t, int t_hi, float c, KEYS&& keys, VALUES&& values, RANGE&& range,
                                      READY&& ready) {
    const uint32_t ring = lds_address(&piece[wave][0][0][0]);
    // byte of the word that holds the scale of this lane's keys, and of its values
    const int col = w[0].col, grp = w[0].grp;
    const uint32_t k_shift = 8 * (D == 64 ? grp >> 1 : grp) + 9;
    const uint32_t v_shift = 8 * (D == 64 ? col >> 3 : D == 128 ? col >> 2 : col >> 1 & 3) + 9;
    const int tiles = t < t_hi ? (t_hi - t + kWaves - 1) / kWaves : 0;
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
      if (i < tiles) {
        keys(t + kWaves * i, i);
        __asm__ __volatile__("" ::: "memory");   // a piece's copies are counted before the next one's
        values(t + kWaves * i, i);
        __asm__ __volatile__("" ::: "memory");
      }
    ready();
    int stage = 0;
    for (int i = 0; i < tiles; ++i, t += kWaves) {
      int lo, hi;
      range(t, &lo, &hi);
      const bool edge = lo > 0 || hi < 32;
      uint32_t inside = 0xFFu;
      if (edge) {
        inside = 0;
#pragma unroll
        for (int j = 0; j < W::kMine; ++j) inside |= (w[0].mine(j) >= lo && w[0].mine(j) < hi ? 1u : 0u) << j;
      }
      const bool more = i + kDepth < tiles;   // tiles to ask for
      const uint32_t at = ring + 2 * kPiece * stage;
      v4f s[NH][NQ][2];
      arrived(2 * (tiles - i) - 1);           // pieces behind this one
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        read_keys(w[h], at, h, k_shift);
        if (h == NH - 1 && more) {
          keys(t + kWaves * kDepth, stage);
          __asm__ __volatile__("" ::: "memory");
        }
        w[h].scores(s[h]);
        w[h].follow_maximum(s[h], c, edge, inside);
      }
      arrived(more ? 2 * kDepth : 0);         // the keys that were just asked for are younger too
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        read_values(w[h], at + kPiece, h, v_shift);
        if (h == NH - 1 && more) {
          values(t + kWaves * kDepth, stage);
          __asm__ __volatile__("" ::: "memory");
        }
        if (edge) w[h].clear_outside(inside);
        w[h].add_weighted(s[h], c);
      }
      stage = stage + 1 < kDepth ? stage + 1 : 0;
    }
  }
};

// Query heads of one row and key head that a workgroup carries.
template <int NQ>
__device__ __forceinline__ int group_of(const KvFp4Args& a) { return a.G < 16 * NQ ? a.G : 16 * NQ; }

// Joins a workgroup's waves' results in LDS and writes the heads' outputs, or their partial sums where part_o is not
// null. Each wave ends up with 16 heads, or where there are more waves than tiles of 16 heads with some dims of them,
// and adds up what all of them have of those: a lane reads what the same lane of each wave has written, so that the
// numbers cross LDS in the order of the registers. All tiles at once, in up to four rounds. (One tile of 16 heads after
// another, every thread adding up four dims and a wait for the stores between them, took 64 heads 15,000 of a short
// sequence's 35,000 cycles; so 7,400. One sequence of 1,500 positions 18.0 -> 15.4 us, 8 of 16,000 36 -> 31 us; up to 16
// heads the same but for 0.2 us more for one short sequence.)
template <class T, int D, int NQ, int NH>
struct Merge4 {
  typedef Wave4<T, D, NQ> W;
  static constexpr int kWaves = ring_waves(D, NQ, NH), kSets = NQ * NH, kDims = D / 16;
  // waves of a tile of 16 heads: four matrix tiles of dims each at least, so that 16 bytes are stored at a time
  static constexpr int kShares = kWaves / kSets < kDims / 4 ? kWaves / kSets : kDims / 4;
  static constexpr int kOwn = kDims / kShares;            // matrix tiles of dims of a wave
  // of which a round takes so many: less beside queries in LDS, which have to lie apart from everything that copies write
  static constexpr int kStep = W::kInLds > 0 ? 2 : 4;
  static_assert(kShares >= 1 && kOwn * kShares == kDims && kOwn % kStep == 0, "every tile has its wave");
  v4f part[kSets * kShares][kStep][kWaves][64];
  float2 ml[kWaves][kSets][16];

  // The largest of the waves' maxima of a tile's head, and the sum that goes with it.
  __device__ __forceinline__ float top_of(int set, int col) const {
    float top = ml[0][set][col].x;
#pragma unroll
    for (int i = 1; i < kWaves; ++i) top = fmaxf(top, ml[i][set][col].x);
    return top;
  }

  // out, lse, part_o, part_ml: of the first head; those of the next key head lie `heads` and `parts` rows behind.
  __device__ __forceinline__ void run(W (&w)[NH], int wave, bool bad, int rows, int64_t heads, int64_t parts, char* out, float* lse,
                                      float* part_o, float2* part_ml) {
    const int col = w[0].col, grp = w[0].grp, lane = w[0].lane;
    lds_barrier();   // every wave has its tiles behind it
#pragma unroll
    for (int set = 0; set < kSets; ++set) {
      const float l = groups_sum(w[set / NQ].l[set % NQ]);
      if (grp == 0) ml[wave][set][col] = make_float2(w[set / NQ].m[set % NQ], bad ? __builtin_nanf("") : l);
    }
    lds_barrier();
    float f[kSets];
#pragma unroll
    for (int set = 0; set < kSets; ++set) f[set] = __builtin_amdgcn_exp2f(w[set / NQ].m[set % NQ] - top_of(set, col));
    const int mine = wave / kShares, piece = wave % kShares;   // this wave's tile of heads, its dims
    const bool owner = mine < kSets && 16 * (mine % NQ) < rows;
    v4f sum[kOwn];
#pragma unroll
    for (int at = 0; at < kOwn; at += kStep) {
      if (at > 0) lds_barrier();
#pragma unroll
      for (int set = 0; set < kSets; ++set)
        if (16 * (set % NQ) < rows) {
#pragma unroll
          for (int s = 0; s < kShares; ++s)
#pragma unroll
            for (int j = 0; j < kStep; ++j) part[set * kShares + s][j][wave][lane] = w[set / NQ].o[set % NQ][s * kOwn + at + j] * f[set];
        }
      lds_barrier();
      if (owner) {
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
          sum[at + j] = part[wave][j][0][lane];
#pragma unroll
          for (int i = 1; i < kWaves; ++i) sum[at + j] += part[wave][j][i][lane];
        }
      }
    }
    const int row = 16 * (mine % NQ) + col;
    if (!owner || row >= rows) return;
    const float top = top_of(mine, col);
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) total += ml[i][mine][col].y * __builtin_amdgcn_exp2f(ml[i][mine][col].x - top);
    const int dim = 4 * grp * kDims + piece * kOwn;   // of sum[t][i]: dim + i * kDims + t
    if (part_o != nullptr) {
      const int64_t to = (mine / NQ) * parts + row;
      if (piece == 0 && grp == 0) part_ml[to] = make_float2(top, total);
      float* p = part_o + to * D + dim;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int t = 0; t < kOwn; t += 4)
          *reinterpret_cast<v4f*>(p + i * kDims + t) = v4f{sum[t][i], sum[t + 1][i], sum[t + 2][i], sum[t + 3][i]};
      }
      return;
    }
    const int64_t to = (mine / NQ) * heads + row;
    if (piece == 0 && grp == 0 && lse != nullptr) lse[to] = lse_of<T>(top, total);
    const float by = 1.0f / total;
    char* p = out + (to * D + dim) * 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int t = 0; t < kOwn; t += 4)
        *reinterpret_cast<v2u*>(p + 2 * (i * kDims + t)) =
            v2u{T::pack(sum[t][i] * by, sum[t + 1][i] * by), T::pack(sum[t + 2][i] * by, sum[t + 3][i] * by)};
    }
  }
};

// A workgroup's LDS: the rings, and when the last tile is done the memory that joins the waves.
template <class T, int D, int NQ, int NH>
union Space {
  Ring4<T, D, NQ, NH> ring;
  Merge4<T, D, NQ, NH> merge;
};

// --- decode form --------------------------------------------------------------

// A row's pages lie end to end with the others' and are cut into shares, and a workgroup takes one share of one of the `sets`
// of NH key heads and 16 NQ query heads of each. All sets of a share go to one die, next to each other in the launch: what one
// workgroup leaves of a cache line that it reads a part of, the others find in the die's L2. `groups` workgroups at most; more sets
// than that leave one share only.
__device__ __forceinline__ int decode_shares(uint32_t sets, uint32_t groups) {
  if (sets <= groups / 8) return groups / (8 * sets) * 8;
  return sets < groups ? groups / sets : 1;
}

// x, which every lane holds, as a scalar: what hangs on it (pages' addresses) is then computed once for the wave.
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(static_cast<uint64_t>(x) >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// The kernel's arguments, read from memory anew: kept in scalar registers over a segment, those that only its beginning
// and end need push the streaming loop's own out of them.
typedef const __attribute__((address_space(4))) KvFp4Args ArgsInMemory;
__device__ __forceinline__ ArgsInMemory& fresh_args() {
  auto p = (ArgsInMemory*)__builtin_amdgcn_kernarg_segment_ptr();
  __asm__ __volatile__("" : "+s"(p));
  return *p;
}

template <class T, int D, int NQ, int NH>
__global__ void __launch_bounds__(64 * ring_waves(D, NQ, NH), ring_waves_per_simd(D, NQ, NH)) kv_decode_fp4_kernel(KvFp4Args a) {
  typedef Wave4<T, D, NQ> W;
  typedef Ring4<T, D, NQ, NH> R;
  constexpr int kGroups = ring_groups(NH);
  __shared__ Plan<R::kWaves> plan;
  __shared__ __align__(16) Space<T, D, NQ, NH> lds;
  __shared__ v4u q_lds[W::kInLds > 0 ? W::kInLds * W::kChunks * 64 : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t* prefix = plan.make(a);
  const int group = group_of<NQ>(a), qg = (a.G + 16 * NQ - 1) / (16 * NQ);
  const int sets = a.Hkv / NH * qg, shares = decode_shares(sets, kGroups), at = blockIdx.x;
  int set = sets < kGroups ? at % sets : at, which = sets < kGroups ? at / sets : 0;
  if (shares >= 8) {
    set = (at >> 3) % sets;
    which = (at >> 3) / sets * 8 + (at & 7);
  }
  if (which >= shares) return;
  const int64_t units = uniform(prefix[a.Q]);
  const int64_t share = unit_share(a, units, shares);
  const int64_t stop = which * share + share < units ? which * share + share : units;
  W w[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h) w[h].init();
  const int lane = w[0].lane;
  // strides inside a page, whose extent is below 2^31, and what a lane adds to a piece's address
  const int k_pos = static_cast<int>(a.k_pos), v_pos = static_cast<int>(a.v_pos), ks_pos = static_cast<int>(a.ks_pos), vs_pos = static_cast<int>(a.vs_pos);
  const uint32_t k_at = R::code_row(lane) * k_pos + R::code_head(0, lane) * static_cast<int>(a.k_head) + R::code_byte(0, lane);
  const uint32_t v_at = R::code_row(lane) * v_pos + R::code_head(1, lane) * static_cast<int>(a.v_head) + R::code_byte(1, lane);
  const uint32_t ks_at = R::scale_row(lane) * ks_pos + R::scale_head(lane) * static_cast<int>(a.ks_head) + R::scale_byte(lane);
  const uint32_t vs_at = R::scale_row(lane) * vs_pos + R::scale_head(lane) * static_cast<int>(a.vs_head) + R::scale_byte(lane);
  // (with more sets than workgroups there is one share only)
  for (int64_t cur = which * share; cur < stop || set + kGroups < sets;) {
    if (cur >= stop) {
      set += kGroups;
      cur = which * share;
      continue;
    }
    ArgsInMemory& m = fresh_args();
    Segment sg;
    sg.take(m, prefix, 1, &cur, stop);
    const int64_t r = sg.r;
    const int kvh = set / qg * NH, first = (set % qg) * 16 * NQ, rows = m.G - first < 16 * NQ ? m.G - first : 16 * NQ;
    const int start = sg.start, end = sg.end;
    const ScalarInts table = scalar_ints(m.table + static_cast<int64_t>(sg.seq) * m.max_pages);
    const int p0 = start >> 6;
    const int t_lo = max(2 * (p0 + sg.pa), start / 32);
    const int t_hi = min(2 * (p0 + sg.pb), (end + 31) / 32);
    const char *kb = m.k + kvh * m.k_head, *vb = m.v + kvh * m.v_head;
    const char *ksb = m.ks + kvh * m.ks_head, *vsb = m.vs + kvh * m.vs_head;
    const int64_t head0 = r * m.H + static_cast<int64_t>(kvh) * m.G + first;
    int next = t_lo + wave < t_hi ? table[(t_lo + wave) / 2] : 0;   // entry of the next tile's page, read early
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      w[h].start();
      w[h].template load_q<R::kWaves>(m.q + r * m.q_row + (static_cast<int64_t>(kvh + h) * m.G + first) * D * 2, rows, m.q_keep, m.q_flip, q_lds);
    }

    const int64_t k_page = m.k_page, v_page = m.v_page, ks_page = m.ks_page, vs_page = m.vs_page;
    const int pages = static_cast<int>(m.P_phys);
    bool bad = false;
    int64_t page = 0;
    // whole tiles are read: what a page holds outside the window is masked
    lds.ring.run(
        w, wave, t_lo + wave, t_hi, m.c,
        [&](int t, int stage) {
          page = next;
          if (t + R::kWaves < t_hi) next = table[(t + R::kWaves) / 2];
          if (page < 0 || page >= pages) {   // nothing of it is read; page 0 stands in
            bad = true;
            page = 0;
          }
          const int first_pos = 32 * (t & 1);
          const auto codes = R::page_at(kb + page * k_page), scales = R::page_at(ksb + page * ks_page);
#pragma unroll
          for (int i = 0; i < R::kCodeCopies; ++i) lds.ring.copy(wave, stage, 0, i, codes, (first_pos + i * R::kCopyRows) * k_pos, k_at);
          lds.ring.copy_scales(wave, stage, 0, lane, scales, first_pos * ks_pos, ks_at);
        },
        [&](int t, int stage) {
          const int first_pos = 32 * (t & 1);
          const auto codes = R::page_at(vb + page * v_page), scales = R::page_at(vsb + page * vs_page);
#pragma unroll
          for (int i = 0; i < R::kCodeCopies; ++i) lds.ring.copy(wave, stage, 1, i, codes, (first_pos + i * R::kCopyRows) * v_pos, v_at);
          lds.ring.copy_scales(wave, stage, 1, lane, scales, first_pos * vs_pos, vs_at);
        },
        [&](int t, int* lo, int* hi) {
          *lo = start - 32 * t;
          *hi = end - 32 * t;
        },
        [&]() {
#pragma unroll
          for (int h = 0; h < NH; ++h) w[h].take_q(m.q_keep, m.q_flip);
        });
    ArgsInMemory& e = fresh_args();
    if (bad && lane == 0) atomicOr(e.status, kStBadPage);
    const bool whole = sg.pa == 0 && sg.pb == sg.n;
    const int64_t slot = 2 * (static_cast<int64_t>(set) * shares + which) + (sg.pa == 0 ? 1 : 0);
    const int64_t part = slot * NH * group;
    lds.merge.run(w, wave, bad, rows, e.G, group, static_cast<char*>(e.out) + head0 * D * 2, e.lse == nullptr ? nullptr : e.lse + head0,
                  whole ? nullptr : e.part_o + part * D, e.part_ml + part);
    lds_barrier();   // the rings may be filled again
  }
}

// Joins the parts of rows that several shares have a part of, and writes the rows that have no pages.
template <class T, int D, int NQ, int NH, int WAVES>
__global__ void __launch_bounds__(kThreads) kv_decode_fp4_join_kernel(KvFp4Args a) {
  const int64_t head = join_head<WAVES>(a);
  if (head < 0) return;
  const int64_t r = head / a.H;
  const int h = static_cast<int>(head - r * a.H);
  const int64_t before = a.prefix[r], n = a.prefix[r + 1] - before;
  if (n == 0) {
    int code;
    row_pages(a, r, &code);
    fill_row<T, D>(a, head, code != 0, WAVES > 1 ? threadIdx.x : threadIdx.x & 63, 64 * WAVES);
    return;
  }
  const int qg = (a.G + 16 * NQ - 1) / (16 * NQ), shares = decode_shares(a.Hkv / NH * qg, ring_groups(NH));
  const int64_t share = unit_share(a, a.prefix[a.Q], shares);
  const int64_t w0 = before / share, w1 = (before + n - 1) / share;
  if (w0 == w1) return;   // one workgroup had all of it and wrote the output
  const int kvh = h / a.G, in_kv = h - kvh * a.G, group = group_of<NQ>(a);
  const int64_t slot = 2 * ((static_cast<int64_t>(kvh / NH) * qg + in_kv / (16 * NQ)) * shares + w0);
  // the first part is its workgroup's last one (slot + 1), the others are first ones
  join_row<T, D, WAVES>(a, head, kvh % NH * group + in_kv % (16 * NQ), NH * group, w1 - w0 + 1, slot + 1, slot, 2);
}

// --- selected form ------------------------------------------------------------

// Offset of a slot's scales: a page's stride is below 2^32.
__device__ __forceinline__ uint64_t scale_offset(int slot, int64_t page, int64_t pos) {
  const uint32_t s = slot;
  return static_cast<uint64_t>(s >> 6) * static_cast<uint32_t>(page) + static_cast<uint64_t>((s & 63) * static_cast<uint32_t>(pos));
}

// The tiles of a list of slots in LDS, filled up to whole tiles.
template <class R>
struct ListTiles {
  const KvFp4Args& a;
  const char *k, *v, *ks, *vs;
  uint32_t k_page, v_page, k_pos, v_pos;   // in units of 16 bytes
  bool alike;                              // keys and values lie at the same offsets
  uint32_t codes, scales;                  // LDS addresses of this lane's slots
  int wave, lane, len;
  int slot[R::kCodeCopies], scale_slot;    // of the tile that keys() was last called for
  uint64_t off[R::kCodeCopies], scale_off;

  __device__ __forceinline__ ListTiles(const KvFp4Args& a_, int kvh, int wave_, int lane_, uint32_t list)
      : a(a_), wave(wave_), lane(lane_), len(0), scale_slot(0), scale_off(0) {
    k = a.k + (kvh + R::code_head(0, lane)) * a.k_head + R::code_byte(0, lane);
    v = a.v + (kvh + R::code_head(1, lane)) * a.v_head + R::code_byte(1, lane);
    ks = a.ks + (kvh + R::scale_head(lane)) * a.ks_head + R::scale_byte(lane);
    vs = a.vs + (kvh + R::scale_head(lane)) * a.vs_head + R::scale_byte(lane);
    k_page = static_cast<uint32_t>(a.k_page >> 4);
    v_page = static_cast<uint32_t>(a.v_page >> 4);
    k_pos = static_cast<uint32_t>(a.k_pos >> 4);
    v_pos = static_cast<uint32_t>(a.v_pos >> 4);
    alike = k_page == v_page && k_pos == v_pos && a.ks_page == a.vs_page && a.ks_pos == a.vs_pos;
    codes = list + 4 * R::code_row(lane);
    scales = list + 4 * R::scale_row(lane);
  }

  __device__ __forceinline__ void keys(R& ring, int t, int stage) {
    R::read_slots(slot, &scale_slot, codes + 128 * t, scales + 128 * t);
#pragma unroll
    for (int i = 0; i < R::kCodeCopies; ++i) {
      off[i] = slot_offset(slot[i], k_page, k_pos);
      ring.copy(wave, stage, 0, i, k + (off[i] << 4));
    }
    scale_off = scale_offset(scale_slot, a.ks_page, a.ks_pos);
    ring.copy_scales(wave, stage, 0, lane, ks + scale_off);
  }

  __device__ __forceinline__ void values(R& ring, int, int stage) {
    if (!alike) {
#pragma unroll
      for (int i = 0; i < R::kCodeCopies; ++i) off[i] = slot_offset(slot[i], v_page, v_pos);
      scale_off = scale_offset(scale_slot, a.vs_page, a.vs_pos);
    }
#pragma unroll
    for (int i = 0; i < R::kCodeCopies; ++i) ring.copy(wave, stage, 1, i, v + (off[i] << 4));
    ring.copy_scales(wave, stage, 1, lane, vs + scale_off);
  }
};

template <class T, int D, int NQ, int NH>
__global__ void __launch_bounds__(64 * ring_waves(D, NQ, NH), ring_waves_per_simd(D, NQ, NH)) kv_selected_fp4_kernel(KvFp4Args a) {
  typedef Wave4<T, D, NQ> W;
  typedef Ring4<T, D, NQ, NH> R;
  __shared__ int list[kKvSelBlock];
  __shared__ __align__(16) Space<T, D, NQ, NH> lds;
  __shared__ v4u q_lds[W::kInLds > 0 ? W::kInLds * W::kChunks * 64 : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int qg = (a.G + 16 * NQ - 1) / (16 * NQ);
  ListPart p;
  bool fill;
  const bool any = p.take(a, static_cast<int64_t>(a.Hkv / NH) * qg, &fill);
  if (!any && !fill) return;
  const int kvh = p.g / qg * NH, first = (p.g % qg) * 16 * NQ, rows = a.G - first < 16 * NQ ? a.G - first : 16 * NQ;
  const int64_t head0 = p.r * a.H + static_cast<int64_t>(kvh) * a.G + first;
  if (!any) {
    for (int h = 0; h < NH * rows; ++h)
      fill_row<T, D>(a, head0 + h / rows * a.G + h % rows, p.n != 0, threadIdx.x, 64 * R::kWaves);
    return;
  }
  W w[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    w[h].init();
    w[h].start();
    w[h].template load_q<R::kWaves>(a.q + p.r * a.q_row + (static_cast<int64_t>(kvh + h) * a.G + first) * D * 2, rows, a.q_keep, a.q_flip, q_lds);
  }
  ListTiles<R> tiles_of(a, kvh, wave, w[0].lane, lds_address(list));
  bool bad = false;
  for (int64_t b0 = p.from; b0 < p.to; b0 += kKvSelBlock) {
    const int len = static_cast<int>(p.to - b0 < kKvSelBlock ? p.to - b0 : kKvSelBlock);
    if (b0 != p.from) __syncthreads();
    bool mine = false;
    const int tiles = (len + 31) / 32;
    for (int i = threadIdx.x; i < 32 * tiles; i += 64 * R::kWaves) {
      const int s = a.slots[p.r * a.K + b0 + min(i, len - 1)];   // the last one again behind the end
      list[i] = s;
      mine |= s < 0 || s >= 64 * a.P_phys;
    }
    if (__syncthreads_or(mine)) {   // nothing of the list is read
      bad = true;
      break;
    }
    tiles_of.len = len;
    lds.ring.run(w, wave, wave, tiles, a.c, [&](int t, int stage) { tiles_of.keys(lds.ring, t, stage); },
                 [&](int t, int stage) { tiles_of.values(lds.ring, t, stage); },
                 [&](int t, int* lo, int* hi) {
                   *lo = 0;
                   *hi = tiles_of.len - 32 * t;
                 },
                 [&]() {
                   if (b0 != p.from) return;
#pragma unroll
                   for (int h = 0; h < NH; ++h) w[h].take_q(a.q_keep, a.q_flip);
                 });
  }
  if (bad && threadIdx.x == 0) atomicOr(a.status, kStBadPage);
  const int group = group_of<NQ>(a);
  const int64_t part = p.item * NH * group;
  lds.merge.run(w, wave, bad, rows, a.G, group, static_cast<char*>(a.out) + head0 * D * 2, a.lse == nullptr ? nullptr : a.lse + head0,
                a.splits == 1 ? nullptr : a.part_o + part * D, a.part_ml + part);
}

template <class T, int D, int NQ, int NH, int WAVES>
__global__ void __launch_bounds__(kThreads) kv_selected_fp4_join_kernel(KvFp4Args a) {
  const int64_t head = join_head<WAVES>(a);
  if (head < 0) return;
  const int64_t r = head / a.H;
  const int h = static_cast<int>(head - r * a.H);
  const int64_t n = a.count[r];
  if (n <= 0 || n > a.K) return;   // written already
  const int qg = (a.G + 16 * NQ - 1) / (16 * NQ), kvh = h / a.G, in_kv = h - kvh * a.G, group = group_of<NQ>(a);
  const int64_t share = split_share(n, a.splits);
  const int64_t slot = ((r * (a.Hkv / NH) + kvh / NH) * qg + in_kv / (16 * NQ)) * a.splits;
  join_row<T, D, WAVES>(a, head, kvh % NH * group + in_kv % (16 * NQ), NH * group, (n + share - 1) / share, slot, slot, 1);
}

// --- dispatch -----------------------------------------------------------------

template <class T, int D, int NQ, int NH>
void decode_on(KvFp4Args a, hipStream_t st) {
  // What one more part costs (its sums' bytes, its turn in the joining of its heads) by what a page takes, both in ns, as
  // for pages of 16 bits: over 15 batches of one to 16 rows, 300 to 128,000 positions and four head layouts, 0.6 to 1.7 times
  // this cost took the same times, 0.15 and 6 times up to 25 % longer ones.
  const double page_ns = NQ > 1 ? 1000 : 100 + 2.75 * D;
  const double pairs = static_cast<double>(a.Hkv) * kv_head_groups(D, a.G);
  const double sums_ns = kv_group_rows(D, a.G) * D * 4 * 0.8e-3, turn_ns = a.Q * a.H <= kJoinHeads ? 20 : 80;
  const double cost = (sums_ns * pairs + turn_ns / static_cast<double>(a.Q)) / page_ns * 65536.0;
  a.join_cost = cost < 8388608.0 ? static_cast<uint32_t>(cost) : 8388608u;
  if (a.Q > kKvPlanRows) kv_plan_kernel<<<dim3(1), dim3(1024), 0, st>>>(a);
  kv_decode_fp4_kernel<T, D, NQ, NH><<<dim3(ring_groups(NH)), dim3(64 * ring_waves(D, NQ, NH)), 0, st>>>(a);
  const int64_t heads = a.Q * a.H;
  if (heads <= kJoinHeads)
    kv_decode_fp4_join_kernel<T, D, NQ, NH, kWaves><<<dim3(static_cast<unsigned>(heads)), dim3(kThreads), 0, st>>>(a);
  else
    kv_decode_fp4_join_kernel<T, D, NQ, NH, 1>
        <<<dim3(static_cast<unsigned>((heads + kWaves - 1) / kWaves)), dim3(kThreads), 0, st>>>(a);
}

template <class T, int D, int NQ, int NH>
void selected_on(const KvFp4Args& a, hipStream_t st) {
  // A launch's threads are counted in 32 bits, and workgroups have up to 512: where one query head has a key head to itself, rows
  // beyond 2^23 go in a second launch. (Lists in several parts have 512 workgroups in all, and one launch.)
  constexpr int kGroupThreads = 64 * ring_waves(D, NQ, NH);
  const int64_t of_row = static_cast<int64_t>(a.Hkv / NH) * kv_head_groups(D, a.G) * a.splits;
  const int64_t most = 0xFFFFFFFFll / kGroupThreads / 8 * 8 / of_row;
  KvFp4Args part = a;
  for (int64_t at = 0; at < a.Q; at += most) {
    part.Q = a.Q - at < most ? a.Q - at : most;
    part.q = a.q + at * a.q_row;
    part.slots = a.K == 0 ? a.slots : a.slots + at * a.K;
    part.count = a.count + at;
    part.out = static_cast<char*>(a.out) + at * a.H * D * 2;
    part.lse = a.lse == nullptr ? nullptr : a.lse + at * a.H;
    const unsigned grid = static_cast<unsigned>((part.Q * of_row + 7) / 8 * 8);
    kv_selected_fp4_kernel<T, D, NQ, NH><<<dim3(grid), dim3(kGroupThreads), 0, st>>>(part);
  }
  if (a.splits > 1)
    kv_selected_fp4_join_kernel<T, D, NQ, NH, 1>
        <<<dim3(static_cast<unsigned>((a.Q * a.H + kWaves - 1) / kWaves)), dim3(kThreads), 0, st>>>(a);
}

struct DecodeOn {
  const KvFp4Args& a;
  hipStream_t st;
  template <class T, int D, int NQ, int NH>
  void operator()() const { decode_on<T, D, NQ, NH>(a, st); }
};
struct SelectedOn {
  const KvFp4Args& a;
  hipStream_t st;
  template <class T, int D, int NQ, int NH>
  void operator()() const { selected_on<T, D, NQ, NH>(a, st); }
};

// Calls f<type, dim, query tiles, key heads at once>() for the call's type and sizes. Two key heads at once, where there
// are two and a head's row is less than a cache line of 128 bytes.
template <class T, class F>
void by_size(const KvFp4Args& a, F&& f) {
  const int nq = kv_tiles(a.D, a.G);
  const bool two = a.Hkv % 2 == 0;
  if (a.D == 64) {
    if (nq == 1 && two) f.template operator()<T, 64, 1, 2>();
    else if (nq == 1) f.template operator()<T, 64, 1, 1>();
    else if (nq == 2) f.template operator()<T, 64, 2, 1>();
    else f.template operator()<T, 64, 4, 1>();
  } else if (a.D == 128) {
    if (nq == 1 && two) f.template operator()<T, 128, 1, 2>();
    else if (nq == 1) f.template operator()<T, 128, 1, 1>();
    else if (nq == 2) f.template operator()<T, 128, 2, 1>();
    else f.template operator()<T, 128, 4, 1>();
  } else {
    if (nq == 1) f.template operator()<T, 256, 1, 1>();
    else f.template operator()<T, 256, 2, 1>();
  }
}

template <class F>
hipError_t by_type(const KvFp4Args& a, F&& f) {
  if (a.q_type == MQA_KV_BF16) by_size<Bf16>(a, f);
  else by_size<Fp16>(a, f);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_decode_fp4(const KvFp4Args& a, hipStream_t st) { return by_type(a, DecodeOn{a, st}); }
hipError_t launch_kv_selected_fp4(const KvFp4Args& a, hipStream_t st) { return by_type(a, SelectedOn{a, st}); }

}  // namespace mqa
