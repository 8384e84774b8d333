// Eviction from the key-value cache by accumulated attention weight (gfx950):
// the choice of what a budget keeps, and the move of what was kept into other
// pages.
//
// Choice. The m = budget - recent largest sums of a sequence are those above the
// m-th largest, and as many of its equals, lowest positions first, as are
// missing. A sum's bits map to an unsigned key whose order is the total order
// (order_bits); counts of its upper, middle and lower bits (digits) fix the m-th
// key. A pass over the keys costs a compute unit about a nanosecond each, so that sequences
// of up to 16,384 positions take one workgroup and one launch, longer ones a
// workgroup per 8,192 positions and four: three that leave their counts of one digit in the
// workspace, the next one adding them up, and one that writes. A position's
// place follows from the same counts, so nothing is counted twice and no order of atomics
// matters. One sequence of 16,000 positions takes 18 us (one workgroup), one of 32,000 35 us with
// one workgroup and 24 with chunks, of 131,072 157 and 31; 64 of 131,072 205 and 109.
//
// Move. A copy, bound by memory: every kept byte is read and written once, 16
// bytes a lane where alignment allows, four pieces in flight.
#include "mqa_fp4_topk.h"
#include "mqa_kv.h"
#include "mqa_device.h"

namespace mqa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;

struct SelectMemory {
  uint32_t hist[4096];   // of the first digit four copies, of the others two: lanes often share their upper digits
  uint32_t wave_sums[kSelWaves];
  uint32_t digit, need;
  int above[kSelWaves], equal[kSelWaves];
};

// Inclusive sum over the workgroup's threads.
__device__ __forceinline__ uint32_t select_scan(uint32_t x, SelectMemory& lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  x = wave_prefix_sum_dpp(x);
  if (lane == 63) lds.wave_sums[wave] = x;
  __syncthreads();
  uint32_t before = 0;
#pragma unroll
  for (int i = 0; i < kSelWaves; ++i)
    if (i < wave) before += lds.wave_sums[i];
  return x + before;
}

// One digit of the m-th key: counts the keys whose upper bits equal `prefix`'s (those in
// `above_mask`) by BITS bits from `shift` on, and finds the digit at which the count
// from the top reaches `need`. key(it, &valid): this lane's key of step it.
template <int BITS, int STEPS, class KEY>
__device__ __forceinline__ void select_digit(SelectMemory& lds, int steps, int shift, uint32_t above_mask,
                                             uint32_t* prefix, uint32_t* need, KEY&& key) {
  constexpr int kBins = 1 << BITS, kWords = 4096, kCopies = kWords / kBins, kPer = kBins / kSelThreads;
  const int lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < kWords / 4; i += kSelThreads) reinterpret_cast<uint4*>(lds.hist)[i] = uint4{0, 0, 0, 0};
  __syncthreads();
  auto count = [&](int it) {
    bool valid;
    const uint32_t k = key(it, &valid);
    const bool in = valid && ((k ^ *prefix) & above_mask) == 0;
    const uint64_t all = __ballot(in);
    if (all == 0) return;
    const uint32_t digit = k >> shift & (kBins - 1);
    // one addition for the lanes with the first one's digit
    const uint32_t first = __builtin_amdgcn_readlane(static_cast<int>(digit), __builtin_ctzll(all));
    const uint64_t same = __ballot(in && digit == first);
    if (in && (digit != first || lane == __builtin_ctzll(all)))
      atomicAdd(&lds.hist[digit * kCopies + lane % kCopies], digit == first ? __popcll(same) : 1u);
  };
#pragma unroll
  for (int it = 0; it < STEPS; ++it)
    if (it < steps) count(it);
  __syncthreads();
  // thread t: bins from the top, kPer of them
  uint32_t c[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint32_t bin = kBins - 1 - (kPer * threadIdx.x + i);
    c[i] = 0;
#pragma unroll
    for (int x = 0; x < kCopies; x += 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(&lds.hist[bin * kCopies + x]);
      c[i] += v.x + v.y;
    }
    sum += c[i];
  }
  uint32_t before = select_scan(sum, lds) - sum;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (before < *need && before + c[i] >= *need) {   // in one thread, once
      lds.digit = kBins - 1 - (kPer * threadIdx.x + i);
      lds.need = *need - before;
    }
    before += c[i];
  }
  __syncthreads();
  *prefix |= lds.digit << shift;
  *need = lds.need;
}

// Keeps m of the first `old` positions and writes them, in order. STEPS: 64-position
// steps of a wave at most.
template <int STEPS>
__device__ __forceinline__ void select_old(const float* acc, int32_t* keep, float* kept_acc, int old, int m,
                                           SelectMemory& lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = ((old + kSelWaves - 1) / kSelWaves + 63) / 64 * 64;   // a wave's run
  const int from = wave * per < old ? wave * per : old, to = from + per < old ? from + per : old;
  const int steps = (to - from + 63) / 64;
  float x[STEPS];
#pragma unroll
  for (int it = 0; it < STEPS; ++it) {
    const int i = from + 64 * it + lane;
    x[it] = i < to ? acc[i] : 0.0f;
  }
  auto value = [&](int it, bool* valid) {
    const int i = from + 64 * it + lane;
    *valid = i < to;
    return x[it];
  };
  auto key = [&](int it, bool* valid) { return order_bits(value(it, valid)); };
  const bool all = m == old;
  uint32_t prefix = 0, need = static_cast<uint32_t>(m);
  if (m == 0) prefix = ~0u;   // no key is above, no equal is kept
  if (m > 0 && !all) {
    select_digit<10, STEPS>(lds, steps, 22, 0u, &prefix, &need, key);
    select_digit<11, STEPS>(lds, steps, 11, ~0u << 22, &prefix, &need, key);
    select_digit<11, STEPS>(lds, steps, 0, ~0u << 11, &prefix, &need, key);
  }
  int above = 0, equal = 0;   // of the wave's run
  auto count = [&](int it) {
    bool valid;
    const uint32_t k = key(it, &valid);
    above += __popcll(__ballot(valid && (all || k > prefix)));
    equal += __popcll(__ballot(valid && !all && k == prefix));
  };
#pragma unroll
  for (int it = 0; it < STEPS; ++it)
    if (it < steps) count(it);
  if (lane == 0) {
    lds.above[wave] = above;
    lds.equal[wave] = equal;
  }
  __syncthreads();
  int at = 0, equals = 0;
  for (int i = 0; i < wave; ++i) {
    at += lds.above[i];
    equals += lds.equal[i];
  }
  const int want = all ? 0 : static_cast<int>(need);   // equals that are kept
  at += equals < want ? equals : want;
  auto emit = [&](int it) {
    bool valid;
    const float v = value(it, &valid);
    const uint32_t k = order_bits(v);
    const bool eq = valid && !all && k == prefix;
    const uint64_t eqs = __ballot(eq);
    const bool take = (valid && (all || k > prefix)) || (eq && equals + mbcnt64(eqs) < want);
    const uint64_t taken = __ballot(take);
    if (take) {
      const int j = at + mbcnt64(taken);
      keep[j] = from + 64 * it + lane;
      if (kept_acc != nullptr) kept_acc[j] = v;
    }
    at += __popcll(taken);
    equals += __popcll(eqs);
  };
#pragma unroll
  for (int it = 0; it < STEPS; ++it)
    if (it < steps) emit(it);
}

// What is to be done for one sequence.
struct SelectRow {
  const float* acc;
  int32_t* keep;
  float* kept_acc;
  int64_t len, n_kept;
  bool bad;
  int old, m;   // positions that compete, and how many of them are kept

  // seq_len: of the sequence. What reads it in memory that is also a.kept does so before write_rest() writes there.
  __device__ __forceinline__ SelectRow(const KvEvictArgs& a, int64_t s, int32_t seq_len) {
    acc = a.acc + s * a.acc_stride;
    keep = a.keep + s * a.budget;
    kept_acc = a.kept_acc == nullptr ? nullptr : a.kept_acc + s * a.budget;
    len = seq_len;
    bad = len < 0 || len > a.max_len;
    n_kept = bad ? 0 : len < a.budget ? len : a.budget;
    old = static_cast<int>(n_kept == 0 ? 0 : len <= a.budget ? len : len - a.recent);
    m = static_cast<int>(n_kept == 0 ? 0 : len <= a.budget ? len : a.budget - a.recent);
  }

  // Everything but the kept ones of the first `old`, by thread `t` of `threads`.
  __device__ __forceinline__ void write_rest(const KvEvictArgs& a, int64_t s, int64_t t, int64_t threads) const {
    if (t == 0) {
      a.kept[s] = bad ? kCodeBadWindow : static_cast<int32_t>(n_kept);
      if (bad) atomicOr(a.status, kStBadWindow);
    }
    for (int64_t i = n_kept + t; i < a.budget; i += threads) {
      keep[i] = -1;
      if (kept_acc != nullptr) kept_acc[i] = 0.0f;
    }
    if (n_kept == 0) return;
    for (int64_t i = old + t; i < len; i += threads) {   // the recent ones
      keep[m + (i - old)] = static_cast<int32_t>(i);
      if (kept_acc != nullptr) kept_acc[m + (i - old)] = acc[i];
    }
  }
};

__global__ void __launch_bounds__(kSelThreads) kv_evict_select_kernel(KvEvictArgs a) {
  __shared__ __align__(16) SelectMemory lds;
  const int64_t s = blockIdx.x;
  const SelectRow row(a, s, a.seq_len[s]);
  __syncthreads();   // every wave has read the length
  row.write_rest(a, s, threadIdx.x, kSelThreads);
  if (row.old == 0) return;
  if (row.old <= 4 * kSelThreads) select_old<4>(row.acc, row.keep, row.kept_acc, row.old, row.m, lds);
  else select_old<16>(row.acc, row.keep, row.kept_acc, row.old, row.m, lds);   // no more than that by the launch's rule
}

// --- long sequences: one workgroup per chunk -----------------------------------

// A chunk is one piece of 8,192 positions where up to 2,097,152 compete, else several, one in registers at a time:
// every workgroup adds up all chunks' counts, which would come to outweigh the rest (5,000,000 positions: 150 us, with
// chunks of one piece 975).
constexpr int kChunkSteps = kKvEvictPiece / kSelThreads;   // 64-position steps of a wave
constexpr int kDigitBins = 2048;                           // digits of 11, 11 and 10 bits
__device__ __forceinline__ int digit_shift(int stage) { return stage == 0 ? 21 : stage == 1 ? 10 : 0; }
__device__ __forceinline__ uint32_t digit_of(uint32_t key, int stage) {
  return key >> digit_shift(stage) & (stage == 2 ? 1023u : 2047u);
}

// One piece: this thread's positions and their sums.
struct Piece {
  float v[kChunkSteps];
  int base;

  __device__ __forceinline__ int position(int it) const {
    return base + (threadIdx.x >> 6) * (64 * kChunkSteps) + 64 * it + (threadIdx.x & 63);
  }
  __device__ __forceinline__ void load(const SelectRow& row, int at) {
    base = at;
#pragma unroll
    for (int it = 0; it < kChunkSteps; ++it) v[it] = position(it) < row.old ? row.acc[position(it)] : 0.0f;
  }
};

// The chunks of a row of which `old` >= 1 positions compete: 2^shift pieces each, as few as make no more than
// kKvEvictChunks of them. LONG false: capacities where that is one piece (choosing in the kernel costs 0.3 us a launch).
template <bool LONG>
struct Chunks {
  int pieces, shift, n;

  __device__ __forceinline__ explicit Chunks(int old) {
    pieces = (old - 1) / kKvEvictPiece + 1;
    const uint32_t over = static_cast<uint32_t>(pieces - 1) / kKvEvictChunks;
    shift = !LONG || over == 0 ? 0 : 32 - __builtin_clz(over);
    n = ((pieces - 1) >> shift) + 1;
  }
  __device__ __forceinline__ int first(int c) const { return (c << shift) * kKvEvictPiece; }   // position
  __device__ __forceinline__ int pieces_of(int c) const {
    if (!LONG) return 1;
    const int left = pieces - (c << shift);
    return left < 1 << shift ? left : 1 << shift;
  }
};

struct ChunkMemory {
  uint32_t hist[2 * kDigitBins];   // two copies
  uint32_t wave_sums[kSelWaves];
  uint32_t digit, need;
  uint32_t above[kSelWaves], equal[kSelWaves];
};

__device__ __forceinline__ uint32_t chunk_scan(uint32_t x, ChunkMemory& lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  x = wave_prefix_sum_dpp(x);
  if (lane == 63) lds.wave_sums[wave] = x;
  __syncthreads();
  uint32_t before = 0;
#pragma unroll
  for (int i = 0; i < kSelWaves; ++i)
    if (i < wave) before += lds.wave_sums[i];
  return x + before;
}

// Adds up the chunks' counts of digit `stage` and finds the digit at which the count from the top reaches
// `need`; *prefix and *need go on to the next digit.
__device__ __forceinline__ void chunk_digit(const uint32_t* counts, int chunks, int stage, ChunkMemory& lds,
                                            uint32_t* prefix, uint32_t* need) {
  const uint32_t bin = kDigitBins - 2 - 2 * threadIdx.x;   // this thread's bins: bin + 1, then bin
  uint2 c = {0, 0};
#pragma unroll 8
  for (int i = 0; i < chunks; ++i) {
    const uint2 x = *reinterpret_cast<const uint2*>(counts + (static_cast<int64_t>(i) * 3 + stage) * kDigitBins + bin);
    c.x += x.x;
    c.y += x.y;
  }
  const uint32_t before = chunk_scan(c.x + c.y, lds) - (c.x + c.y);
  if (before < *need && before + c.y >= *need) {
    lds.digit = bin + 1;
    lds.need = *need - before;
  } else if (before + c.y < *need && before + c.y + c.x >= *need) {
    lds.digit = bin;
    lds.need = *need - before - c.y;
  }
  __syncthreads();
  *prefix |= lds.digit << digit_shift(stage);
  *need = lds.need;
}

// Counts one digit of a chunk's keys whose upper digits are the m-th key's. state[s * 8 + 2 d, + 1]:
// prefix and need behind digit d (d < 2); state[s * 8 + 4]: the length, for the last launch, in which
// kept is written and may lie over the lengths.
template <bool LONG>
__global__ void __launch_bounds__(kSelThreads) kv_evict_count_kernel(KvEvictArgs a, int chunks, int stage) {
  __shared__ __align__(16) ChunkMemory lds;
  const int64_t s = blockIdx.x / chunks;
  const int c = static_cast<int>(blockIdx.x - s * chunks);
  const SelectRow row(a, s, a.seq_len[s]);
  uint32_t* state = a.state + 8 * s;
  if (stage == 0 && c == 0 && threadIdx.x == 0) state[4] = static_cast<uint32_t>(row.len);
  if (row.m == 0 || row.m == row.old) return;
  const Chunks<LONG> of(row.old);
  if (c >= of.n) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Piece x;
  x.load(row, of.first(c));
  uint32_t* counts = a.counts + s * chunks * 3 * kDigitBins;
  uint32_t prefix = 0, need = static_cast<uint32_t>(row.m);
  if (stage > 0) {
    if (stage == 2) {
      prefix = state[0];
      need = state[1];
    }
    chunk_digit(counts, of.n, stage - 1, lds, &prefix, &need);
    if (c == 0 && threadIdx.x == 0) {
      state[2 * (stage - 1)] = prefix;
      state[2 * (stage - 1) + 1] = need;
    }
  }
  for (int i = threadIdx.x; i < 2 * kDigitBins; i += kSelThreads) lds.hist[i] = 0;
  __syncthreads();
  const uint32_t mask = stage == 0 ? 0u : ~0u << digit_shift(stage - 1);
  for (int left = of.pieces_of(c);;) {
#pragma unroll
    for (int it = 0; it < kChunkSteps; ++it) {
      const uint32_t k = order_bits(x.v[it]);
      const bool in = x.position(it) < row.old && ((k ^ prefix) & mask) == 0;
      const uint64_t all = __ballot(in);
      if (all == 0) continue;
      const uint32_t digit = digit_of(k, stage);
      // one addition for the lanes with the first one's digit
      const int leader = __builtin_ctzll(all);
      const uint32_t first = __builtin_amdgcn_readlane(static_cast<int>(digit), leader);
      const uint64_t same = __ballot(in && digit == first);
      if (in && (digit != first || lane == leader))
        atomicAdd(&lds.hist[2 * digit + (lane & 1)], digit == first ? __popcll(same) : 1u);
    }
    if (--left == 0) break;
    x.load(row, x.base + kKvEvictPiece);
  }
  __syncthreads();
  uint32_t* mine = counts + (static_cast<int64_t>(c) * 3 + stage) * kDigitBins;
  for (int i = threadIdx.x; i < kDigitBins; i += kSelThreads) mine[i] = lds.hist[2 * i] + lds.hist[2 * i + 1];
}

// Writes a chunk's kept positions where the counts say.
template <bool LONG>
__global__ void __launch_bounds__(kSelThreads) kv_evict_write_kernel(KvEvictArgs a, int chunks) {
  __shared__ __align__(16) ChunkMemory lds;
  const int64_t s = blockIdx.x / chunks;
  const int c = static_cast<int>(blockIdx.x - s * chunks);
  const SelectRow row(a, s, static_cast<int32_t>(a.state[8 * s + 4]));
  row.write_rest(a, s, c * kSelThreads + threadIdx.x, static_cast<int64_t>(chunks) * kSelThreads);
  if (row.m == 0) return;
  const Chunks<LONG> of(row.old);
  if (c >= of.n) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Piece x;
  x.load(row, of.first(c));
  const bool all = row.m == row.old;
  uint32_t prefix = 0, need = 0;
  int aboves = of.first(c), equals = 0;   // positions before the piece above the m-th key (every one where all are kept), equal to it
  if (!all) {
    const uint32_t* counts = a.counts + s * chunks * 3 * kDigitBins;
    prefix = a.state[8 * s + 2];
    need = a.state[8 * s + 3];
    chunk_digit(counts, of.n, 2, lds, &prefix, &need);
    // keys above the m-th one in earlier chunks: by the digit at which they differ
    uint32_t above = 0, equal = 0;
    const uint32_t bin = 2 * threadIdx.x;
#pragma unroll 4
    for (int i = 0; i < c; ++i)
#pragma unroll
      for (int st = 0; st < 3; ++st) {
        const uint32_t digit = digit_of(prefix, st);
        const uint2 n =
            *reinterpret_cast<const uint2*>(counts + (static_cast<int64_t>(i) * 3 + st) * kDigitBins + bin);
        above += (bin > digit ? n.x : 0u) + (bin + 1 > digit ? n.y : 0u);
        if (st == 2) equal += bin == digit ? n.x : bin + 1 == digit ? n.y : 0u;
      }
    __syncthreads();
    above = lane63(wave_prefix_sum_dpp(above));
    equal = lane63(wave_prefix_sum_dpp(equal));
    if (lane == 0) {
      lds.above[wave] = above;
      lds.equal[wave] = equal;
    }
    __syncthreads();
    aboves = 0;
    for (int i = 0; i < kSelWaves; ++i) {
      aboves += static_cast<int>(lds.above[i]);
      equals += static_cast<int>(lds.equal[i]);
    }
    __syncthreads();
  }
  const int want = static_cast<int>(need);
  for (int left = of.pieces_of(c);;) {
    int above = 0, equal = 0;
#pragma unroll
    for (int it = 0; it < kChunkSteps; ++it) {
      const bool valid = x.position(it) < row.old;
      const uint32_t k = order_bits(x.v[it]);
      above += __popcll(__ballot(valid && (all || k > prefix)));
      equal += __popcll(__ballot(valid && !all && k == prefix));
    }
    if (lane == 0) {
      lds.above[wave] = above;
      lds.equal[wave] = equal;
    }
    __syncthreads();
    // the waves before this one
    int at = aboves, eq_at = equals;
    for (int i = 0; i < wave; ++i) {
      at += static_cast<int>(lds.above[i]);
      eq_at += static_cast<int>(lds.equal[i]);
    }
    at += eq_at < want ? eq_at : want;
#pragma unroll
    for (int it = 0; it < kChunkSteps; ++it) {
      const bool valid = x.position(it) < row.old;
      const uint32_t k = order_bits(x.v[it]);
      const bool eq = valid && !all && k == prefix;
      const uint64_t eqs = __ballot(eq);
      const bool take = (valid && (all || k > prefix)) || (eq && eq_at + mbcnt64(eqs) < want);
      const uint64_t taken = __ballot(take);
      if (take) {
        const int j = at + mbcnt64(taken);
        row.keep[j] = x.position(it);
        if (row.kept_acc != nullptr) row.kept_acc[j] = x.v[it];
      }
      at += __popcll(taken);
      eq_at += __popcll(eqs);
    }
    if (--left == 0) break;
    for (int i = 0; i < kSelWaves; ++i) {
      aboves += static_cast<int>(lds.above[i]);
      equals += static_cast<int>(lds.equal[i]);
    }
    x.load(row, x.base + kKvEvictPiece);
    __syncthreads();   // the counts are read
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;      // kept positions per piece of work
constexpr int kMoveAhead = 4;      // pieces of a thread in flight
typedef uint32_t move16 __attribute__((ext_vector_type(4)));

template <class V>
__device__ __forceinline__ void move_rows(const KvCompactArray& x, const int64_t* src, const int64_t* dst, int n) {
  const uint32_t per = static_cast<uint32_t>(x.units * x.rows), units = static_cast<uint32_t>(x.units);   // < 2^24
  const uint32_t all = static_cast<uint32_t>(n) * per;
  for (uint32_t e0 = threadIdx.x; e0 < all; e0 += kMoveAhead * kMoveThreads) {
    V v[kMoveAhead];
    char* to[kMoveAhead];
#pragma unroll
    for (int i = 0; i < kMoveAhead; ++i) {
      const uint32_t e = e0 + i * kMoveThreads;
      to[i] = nullptr;
      if (e >= all) continue;
      const uint32_t j = e / per, rest = e - j * per;
      const uint32_t row = rest / units, u = rest - row * units;
      const int64_t s = src[j], d = dst[j];
      if (s < 0) continue;
      to[i] = x.dst + (d >> 6) * x.dst_page + (d & 63) * x.dst_pos + row * x.dst_row + u * sizeof(V);
      v[i] = *reinterpret_cast<const V*>(x.src + (s >> 6) * x.src_page + (s & 63) * x.src_pos + row * x.src_row +
                                         u * sizeof(V));
    }
#pragma unroll
    for (int i = 0; i < kMoveAhead; ++i)
      if (to[i] != nullptr) *reinterpret_cast<V*>(to[i]) = v[i];
  }
}

__global__ void __launch_bounds__(kMoveThreads) kv_compact_kernel(KvCompactArgs a, int64_t blocks, int64_t items) {
  __shared__ int64_t src[kMoveRows], dst[kMoveRows];
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t x = item % a.n_arrays, rest = item / a.n_arrays;
    const int64_t s = rest / blocks, j0 = (rest - s * blocks) * kMoveRows;
    const int64_t n = a.kept[s];
    if (n > a.budget || n > 64 * a.dst_pages) {
      if (x == 0 && j0 == 0 && threadIdx.x == 0) atomicOr(a.status, kStBadWindow);
      continue;
    }
    if (j0 >= n) continue;
    const int len = static_cast<int>(n - j0 < kMoveRows ? n - j0 : kMoveRows);
    __syncthreads();
    if (threadIdx.x < len) {
      const int64_t j = j0 + threadIdx.x;
      const int32_t p = a.keep[s * a.budget + j];
      int64_t from = -1, to = -1;
      if (p < 0 || p >= 64 * a.src_pages) {
        atomicOr(a.status, kStBadWindow);
      } else {
        const int32_t sp = a.src_table[s * a.src_pages + (p >> 6)], dp = a.dst_table[s * a.dst_pages + (j >> 6)];
        if (sp < 0 || sp >= a.P_src || dp < 0 || dp >= a.P_dst) {
          atomicOr(a.status, kStBadPage);
        } else {
          from = 64 * static_cast<int64_t>(sp) + (p & 63);
          to = 64 * static_cast<int64_t>(dp) + (j & 63);
        }
      }
      src[threadIdx.x] = from;
      dst[threadIdx.x] = to;
    }
    __syncthreads();
    if (a.arrays[x].wide) move_rows<move16>(a.arrays[x], src, dst, len);
    else move_rows<uint32_t>(a.arrays[x], src, dst, len);
  }
}

}  // namespace

hipError_t launch_kv_evict_select(const KvEvictArgs& a, hipStream_t st) {
  const int64_t chunks = kv_evict_chunks(a.max_len);
  const dim3 grid(static_cast<unsigned>(a.n_seq * chunks)), block(kSelThreads);
  if (chunks == 1) {
    kv_evict_select_kernel<<<grid, block, 0, st>>>(a);
  } else {
    const int n = static_cast<int>(chunks);
    const bool several = a.max_len > kKvEvictPiece * kKvEvictChunks;
    const auto count = several ? kv_evict_count_kernel<true> : kv_evict_count_kernel<false>;
    const auto write = several ? kv_evict_write_kernel<true> : kv_evict_write_kernel<false>;
    for (int stage = 0; stage < 3; ++stage) count<<<grid, block, 0, st>>>(a, n, stage);
    write<<<grid, block, 0, st>>>(a, n);
  }
  return hipGetLastError();
}

hipError_t launch_kv_compact(const KvCompactArgs& a, hipStream_t st) {
  const int64_t blocks = (a.budget + kMoveRows - 1) / kMoveRows;
  const int64_t items = blocks * a.n_seq * a.n_arrays;
  const int64_t grid = items < 16384 ? items : 16384;
  kv_compact_kernel<<<dim3(static_cast<unsigned>(grid)), dim3(kMoveThreads), 0, st>>>(a, blocks, items);
  return hipGetLastError();
}

}  // namespace mqa
