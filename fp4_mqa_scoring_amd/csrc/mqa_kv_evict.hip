// Eviction from the key-value cache by accumulated attention weight (gfx950):
// the choice of what a budget keeps, and the move of what was kept into other
// pages.
//
// Choice. The m = budget - recent largest sums of a sequence are those above the
// m-th largest, and as many of its equals, lowest positions first, as are
// missing. A sum's bits map to an unsigned key whose order is the total order
// (order_bits); four histograms of eight bits each, from the top, fix the m-th
// key. One workgroup per sequence: its sums stay in L2 from pass to pass.
//
// Move. A copy, bound by memory: every kept byte is read and written once, 16
// bytes a lane where alignment allows.
#include "mqa_fp4_topk.h"
#include "mqa_kv.h"
#include "mqa_device.h"

namespace mqa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;

__global__ void __launch_bounds__(kSelThreads) kv_evict_select_kernel(KvEvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t digit_lds, need_lds;
  __shared__ int wave_above[kSelWaves], wave_equal[kSelWaves];
  const int64_t s = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float* acc = a.acc + s * a.acc_stride;
  int32_t* keep = a.keep + s * a.budget;
  float* kept_acc = a.kept_acc == nullptr ? nullptr : a.kept_acc + s * a.budget;
  const int64_t len = a.seq_len[s];
  const bool bad = len < 0 || len > a.max_len;
  const int64_t n_kept = bad ? 0 : len < a.budget ? len : a.budget;
  if (threadIdx.x == 0) {
    a.kept[s] = bad ? kCodeBadWindow : static_cast<int32_t>(n_kept);
    if (bad) atomicOr(a.status, kStBadWindow);
  }
  for (int64_t i = n_kept + threadIdx.x; i < a.budget; i += kSelThreads) {
    keep[i] = -1;
    if (kept_acc != nullptr) kept_acc[i] = 0.0f;
  }
  if (n_kept == 0) return;
  const int old = static_cast<int>(len <= a.budget ? len : len - a.recent);       // positions that compete
  const int m = static_cast<int>(len <= a.budget ? len : a.budget - a.recent);    // and how many are kept
  uint32_t prefix = 0, need = static_cast<uint32_t>(m);
  if (m > 0 && m < old) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (threadIdx.x < 256) hist[threadIdx.x] = 0;
      __syncthreads();
      const uint32_t above_mask = shift == 24 ? 0u : ~0u << (shift + 8);
      for (int i = threadIdx.x; i < old; i += kSelThreads) {
        const uint32_t key = order_bits(acc[i]);
        if (((key ^ prefix) & above_mask) == 0) atomicAdd(&hist[key >> shift & 0xFF], 1u);
      }
      __syncthreads();
      if (wave == 0) {   // lane l: digits 255 - 4 l down to 252 - 4 l
        uint32_t h[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[i] = hist[255 - 4 * lane - i];
          sum += h[i];
        }
        uint32_t before = wave_prefix_sum_dpp(sum) - sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (before < need && before + h[i] >= need) {
            digit_lds = static_cast<uint32_t>(255 - 4 * lane - i);
            need_lds = need - before;
          }
          before += h[i];
        }
      }
      __syncthreads();
      prefix |= digit_lds << shift;
      need = need_lds;   // how many equals of the digits so far are kept
    }
  } else if (m == 0) {
    prefix = ~0u;        // no key is above, no equal is kept
    need = 0;
  }                      // m == old: key 0 and below: every one is kept
  const bool all = m == old;
  // each wave emits a run of positions; two counts per run place them
  const int per = ((old + kSelWaves - 1) / kSelWaves + 63) / 64 * 64;
  const int from = wave * per < old ? wave * per : old, to = from + per < old ? from + per : old;
  int above = 0, equal = 0;
  for (int i0 = from; i0 < to; i0 += 64) {
    const int i = i0 + lane;
    const uint32_t key = i < to ? order_bits(acc[i]) : 0u;
    above += __popcll(__ballot(i < to && (all || key > prefix)));
    equal += __popcll(__ballot(i < to && !all && key == prefix));
  }
  if (lane == 0) {
    wave_above[wave] = above;
    wave_equal[wave] = equal;
  }
  __syncthreads();
  int at = 0, equals = 0;
  for (int i = 0; i < wave; ++i) {
    at += wave_above[i];
    equals += wave_equal[i];
  }
  at += equals < static_cast<int>(need) ? equals : static_cast<int>(need);
  if (all) equals = 0;
  for (int i0 = from; i0 < to; i0 += 64) {
    const int i = i0 + lane;
    const float x = i < to ? acc[i] : 0.0f;
    const uint32_t key = order_bits(x);
    const bool eq = i < to && !all && key == prefix;
    const uint64_t eqs = __ballot(eq);
    const bool take = (i < to && (all || key > prefix)) || (eq && equals + mbcnt64(eqs) < static_cast<int>(need));
    const uint64_t taken = __ballot(take);
    if (take) {
      const int j = at + mbcnt64(taken);
      keep[j] = i;
      if (kept_acc != nullptr) kept_acc[j] = x;
    }
    at += __popcll(taken);
    equals += __popcll(eqs);
  }
  for (int64_t i = old + threadIdx.x; i < len; i += kSelThreads) {   // the recent ones
    keep[m + (i - old)] = static_cast<int32_t>(i);
    if (kept_acc != nullptr) kept_acc[m + (i - old)] = acc[i];
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;      // kept positions per piece of work

template <class V>
__device__ __forceinline__ void move_rows(const KvCompactArray& x, const int64_t* src, const int64_t* dst, int n) {
  const int64_t per = x.units * x.rows;
  for (int64_t e = threadIdx.x; e < n * per; e += kMoveThreads) {
    const int i = static_cast<int>(e / per);
    const int64_t rest = e - i * per;
    const int64_t row = rest / x.units, u = rest - row * x.units;
    if (src[i] < 0) continue;
    const int64_t from = (src[i] >> 6) * x.src_page + (src[i] & 63) * x.src_pos + row * x.src_row;
    const int64_t to = (dst[i] >> 6) * x.dst_page + (dst[i] & 63) * x.dst_pos + row * x.dst_row;
    *reinterpret_cast<V*>(x.dst + to + u * sizeof(V)) = *reinterpret_cast<const V*>(x.src + from + u * sizeof(V));
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
    if (a.arrays[x].wide) move_rows<uint4>(a.arrays[x], src, dst, len);
    else move_rows<uint32_t>(a.arrays[x], src, dst, len);
  }
}

}  // namespace

hipError_t launch_kv_evict_select(const KvEvictArgs& a, hipStream_t st) {
  kv_evict_select_kernel<<<dim3(static_cast<unsigned>(a.n_seq)), dim3(kSelThreads), 0, st>>>(a);
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
