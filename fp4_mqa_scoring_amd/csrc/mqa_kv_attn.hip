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
#include "mqa_kv_attn.h"

namespace mqa {
namespace {

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
