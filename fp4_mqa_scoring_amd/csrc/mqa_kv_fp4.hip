// Attention over a paged key-value cache in 4 bits (gfx950). Formulas, tiles and the
// operands' layout are those of mqa_kv_attn.hip; keys and values are made 16-bit numbers in
// registers, exactly, right before their product: one instruction makes two numbers of a
// byte and their block's power of two.
#include "mqa_kv_attn.h"

namespace mqa {
namespace {

template <int SEL>
__device__ __forceinline__ uint32_t pair_of(Bf16, uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
}
template <int SEL>
__device__ __forceinline__ uint32_t pair_of(Fp16, uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, SEL));
}

// 2^(byte - 127) as the conversions take it: they look at the exponent alone.
__device__ __forceinline__ float power_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Reads of one page: a scalar base, and 32-bit offsets of the lane and of what is read.
struct PageReads {
  __amdgpu_buffer_rsrc_t page;
  uint32_t lane;
  int at;   // added to the offsets below

  __device__ __forceinline__ PageReads(const char* base, uint32_t lane_) : lane(lane_), at(0) {
    page = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, 0x7FFFFFFF, 0x00027000);
  }
  __device__ __forceinline__ PageReads& from(int at_) {
    at = at_;
    return *this;
  }
  __device__ __forceinline__ void operator()(int off, v4u& x) const { x = __builtin_amdgcn_raw_buffer_load_b128(page, lane + off, at, 0); }
  __device__ __forceinline__ void operator()(int off, v2u& x) const { x = __builtin_amdgcn_raw_buffer_load_b64(page, lane + off, at, 0); }
  __device__ __forceinline__ void operator()(int off, uint32_t& x) const { x = __builtin_amdgcn_raw_buffer_load_b32(page, lane + off, at, 0); }
  __device__ __forceinline__ void operator()(int off, uint16_t& x) const { x = __builtin_amdgcn_raw_buffer_load_b16(page, lane + off, at, 0); }
  __device__ __forceinline__ void operator()(int off, uint8_t& x) const { x = __builtin_amdgcn_raw_buffer_load_b8(page, lane + off, at, 0); }
};

// Reads behind a lane's own address.
struct LaneReads {
  const char* p;
  template <class X>
  __device__ __forceinline__ void operator()(int off, X& x) const { x = *reinterpret_cast<const X*>(p + off); }
};

// A wave's tile of 32 positions over a cache in 4 bits. Lane (col, grp) holds, of keys 16 a + col, the codes of
// kKeyDims neighbouring dims (one block's, or a half of one with D = 64), and of values mine(j) those of D / 16.
//
// More than 16 heads: the queries lie in LDS, and the running maximum may lag by 2^8.
template <class T, int D, int NQ>
struct Wave4 : Wave<T, false, D, NQ, 32, (NQ > 1), (NQ > 1 ? 8 : 0)> {
  typedef Wave<T, false, D, NQ, 32, (NQ > 1), (NQ > 1 ? 8 : 0)> Base;
  using Base::kChunks;
  using Base::kDims;
  using Base::kMine;
  using Base::kShared;
  using Base::kTiles;
  using Base::col;
  using Base::grp;
  using Base::q;
  typedef typename Base::P P;
  static constexpr int kKeyBlocks = D == 256 ? 2 : 1;    // scales of a lane's key
  static constexpr int kKeyWords = D / 32;               // words of 8 codes of a lane's key
  static constexpr int kWords4 = D == 256 ? 2 : 1;       // words of a lane's value (half of one with D = 64)

  const __attribute__((address_space(3))) v4u* ql;       // the queries in LDS, from this lane's on
  uint32_t kc[kTiles][kKeyWords], kb[kTiles][kKeyBlocks];
  uint32_t vc[kMine][kWords4], vb[kMine];

  // First dim of matrix step c in this lane's keys.
  __device__ __forceinline__ int step_dim(int c) const {
    return D == 64 ? 16 * grp + 8 * c : 128 * (c >> 2) + 32 * grp + 8 * (c & 3);
  }

  // This lane's part of step c of query tile n, of heads [0, rows) at `p`.
  __device__ __forceinline__ v4u query(const char* p, int n, int c, int rows, uint32_t keep, uint32_t flip) const {
    const int h = 16 * n + col;
    v4u x = {0, 0, 0, 0};
    if (h < rows) x = *reinterpret_cast<const v4u*>(p + (static_cast<int64_t>(h) * D + step_dim(c)) * 2);
    return (x & v4u{keep, keep, keep, keep}) ^ v4u{flip, flip, flip, flip};
  }

  // Loads the queries: into registers, or by the whole workgroup into `lds` (NQ * kChunks * 64 of it), between barriers.
  __device__ __forceinline__ void load_q(const char* p, int rows, uint32_t keep, uint32_t flip, v4u* lds) {
    if constexpr (kShared) {
      ql = (const __attribute__((address_space(3))) v4u*)lds + this->lane;
      __syncthreads();
      for (int x = threadIdx.x >> 6; x < NQ * kChunks; x += kWaves)
        lds[64 * x + this->lane] = query(p, x / kChunks, x % kChunks, rows, keep, flip);
      __syncthreads();
    } else {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < kChunks; ++c) q[n][c] = query(p, n, c, rows, keep, flip);
    }
  }

  // What a lane adds to the address of its key: of the codes and scales of position 16 a.
  __device__ __forceinline__ uint32_t key_at() const { return D == 64 ? 8 * grp : 16 * grp; }
  __device__ __forceinline__ uint32_t key_scale_at() const { return D == 64 ? grp >> 1 : grp; }
  // And of its values.
  __device__ __forceinline__ uint32_t value_at() const { return col * (D / 32); }
  __device__ __forceinline__ uint32_t value_scale_at() const { return col * kDims / 32; }

  // This lane's codes and scale of position 16 a + col; get(offset, x) reads x at that offset behind their place.
  template <class CODES, class SCALES>
  __device__ __forceinline__ void load_k(int a, CODES&& codes, SCALES&& scales) {
    if constexpr (D == 64) {
      v2u x;
      codes(0, x);
      kc[a][0] = x.x;
      kc[a][1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        v4u x;
        codes(64 * i, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) kc[a][4 * i + e] = x[e];
      }
    }
#pragma unroll
    for (int i = 0; i < kKeyBlocks; ++i) {
      uint8_t x;
      scales(4 * i, x);
      kb[a][i] = x;
    }
  }

  // Of position mine(j).
  template <class CODES, class SCALES>
  __device__ __forceinline__ void load_v(int j, CODES&& codes, SCALES&& scales) {
    if constexpr (D == 64) {
      uint16_t x;
      codes(0, x);
      vc[j][0] = x;
    } else if constexpr (D == 128) {
      codes(0, vc[j][0]);
    } else {
      v2u x;
      codes(0, x);
      vc[j][0] = x.x;
      vc[j][1] = x.y;
    }
    uint8_t x;
    scales(0, x);
    vb[j] = x;
  }

  __device__ __forceinline__ void scores(v4f (&s)[NQ][kTiles]) {
    auto queries = ql;
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
        const uint32_t w = kc[a][c];
        const float by = power_of(kb[a][D == 256 ? c >> 2 : 0]);
        x[a] = v4u{pair_of<0>(T{}, w, by), pair_of<1>(T{}, w, by), pair_of<2>(T{}, w, by), pair_of<3>(T{}, w, by)};
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

  // Values outside the window: every code is a number, so a scale of nearly 0 will do.
  __device__ __forceinline__ void clear_outside(uint32_t inside) {
    inside = Base::here(inside);
#pragma unroll
    for (int j = 0; j < kMine; ++j) vb[j] = (inside >> j & 1) ? vb[j] : 0u;
  }

  template <int E>
  __device__ __forceinline__ uint32_t dims_pair(int j) const {
    return pair_of<(E & 3)>(T{}, vc[j][E >> 2], power_of(vb[j]));
  }

  template <int E>
  __device__ __forceinline__ void add_pair(const P (&p)[NQ]) {
    uint32_t w[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) w[j] = dims_pair<E>(j);
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

// Heads of one row and key head that a workgroup carries.
template <int NQ>
__device__ __forceinline__ int group_of(const KvFp4Args& a) { return a.G < 16 * NQ ? a.G : 16 * NQ; }

// Joins the waves' results, 16 heads at a time.
template <int N, class T, int D, class W>
__device__ __forceinline__ void join_waves(Merge<T, D>& merge, W& w, bool bad, int rows, char* out, float* lse, float* part_o,
                                           float2* part_ml) {
  if constexpr (N < W::kQueries) {
    if (16 * N >= rows) return;
    constexpr int64_t at = 16 * N;
    merge.template run<N>(w, bad, rows - 16 * N < 16 ? rows - 16 * N : 16, 1.0f, out + at * D * 2, lse == nullptr ? nullptr : lse + at,
                          part_o == nullptr ? nullptr : part_o + at * D, part_ml + at);
    join_waves<N + 1, T, D>(merge, w, bad, rows, out, lse, part_o, part_ml);
  }
}

// --- decode form --------------------------------------------------------------

template <class T, int D, int NQ>
__global__ void __launch_bounds__(kThreads, 2) kv_decode_fp4_kernel(KvFp4Args a) {
  typedef Wave4<T, D, NQ> W;
  __shared__ Plan<kWaves> plan;
  __shared__ Merge<T, D> merge;
  __shared__ v4u q_lds[W::kShared ? NQ * W::kChunks * 64 : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t* prefix = plan.make(a);
  const int group = group_of<NQ>(a), qg = (a.G + 16 * NQ - 1) / (16 * NQ);
  const int64_t gh = static_cast<int64_t>(a.Hkv) * qg;
  const int64_t units = prefix[a.Q] * gh;
  const int64_t share = unit_share(a, units, gridDim.x);
  int64_t cur = blockIdx.x * share;
  const int64_t stop = cur + share < units ? cur + share : units;
  W w;
  w.init();
  // strides inside a page, whose extent is below 2^31
  const int k_pos = static_cast<int>(a.k_pos), v_pos = static_cast<int>(a.v_pos), ks_pos = static_cast<int>(a.ks_pos), vs_pos = static_cast<int>(a.vs_pos);
  const uint32_t k_at = w.col * k_pos + w.key_at(), ks_at = w.col * ks_pos + w.key_scale_at();
  const uint32_t v_at = 4 * w.grp * v_pos + w.value_at(), vs_at = 4 * w.grp * vs_pos + w.value_scale_at();
  while (cur < stop) {
    Segment sg;
    sg.take(a, prefix, gh, &cur, stop);
    const int64_t r = sg.r;
    const int kvh = sg.g / qg, first = (sg.g % qg) * 16 * NQ, rows = a.G - first < 16 * NQ ? a.G - first : 16 * NQ;
    const int start = sg.start, end = sg.end;
    const int32_t* table = a.table + static_cast<int64_t>(sg.seq) * a.max_pages;
    const int p0 = start >> 6;
    const int t_lo = max(2 * (p0 + sg.pa), start / 32);
    const int t_hi = min(2 * (p0 + sg.pb), (end + 31) / 32);
    const char *kb = a.k + kvh * a.k_head, *vb = a.v + kvh * a.v_head;
    const char *ksb = a.ks + kvh * a.ks_head, *vsb = a.vs + kvh * a.vs_head;
    const int64_t head0 = r * a.H + static_cast<int64_t>(kvh) * a.G + first;
    w.start();
    w.load_q(a.q + r * a.q_row + (static_cast<int64_t>(kvh) * a.G + first) * D * 2, rows, a.q_keep, a.q_flip, q_lds);

    bool bad = false;
    int next = t_lo + wave < t_hi ? table[(t_lo + wave) / 2] : 0;   // entry of the next tile's page, read early
    int page = 0;
    // Whole tiles are read: what a page holds outside the window is masked. A tile's page is the same for the wave, so
    // that addresses are a scalar base and a lane's offset, which never changes.
    run_tiles(
        w, t_lo + wave, t_hi, a.c,
        [&](int t) {
          page = __builtin_amdgcn_readfirstlane(next);
          if (t + kWaves < t_hi) next = table[(t + kWaves) / 2];
          if (page < 0 || page >= a.P_phys) {   // nothing of it is read; page 0 stands in
            bad = true;
            page = 0;
          }
          const int first = 32 * (t & 1);
          PageReads codes(kb + page * a.k_page, k_at), scales(ksb + page * a.ks_page, ks_at);
#pragma unroll
          for (int b = 0; b < W::kTiles; ++b) w.load_k(b, codes.from((first + 16 * b) * k_pos), scales.from((first + 16 * b) * ks_pos));
        },
        [&](int t) {
          const int first = 32 * (t & 1);
          PageReads codes(vb + page * a.v_page, v_at), scales(vsb + page * a.vs_page, vs_at);
#pragma unroll
          for (int j = 0; j < W::kMine; ++j) {
            const int pos = first + 16 * (j >> 2) + (j & 3);
            w.load_v(j, codes.from(pos * v_pos), scales.from(pos * vs_pos));
          }
        },
        [&](int t, int* lo, int* hi) {
          *lo = start - 32 * t;
          *hi = end - 32 * t;
        });
    if (bad && w.lane == 0) atomicOr(a.status, kStBadPage);
    const bool whole = sg.pa == 0 && sg.pb == sg.n;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (sg.pa == 0 ? 1 : 0);
    join_waves<0, T, D>(merge, w, bad, rows, static_cast<char*>(a.out) + head0 * D * 2, a.lse == nullptr ? nullptr : a.lse + head0,
                        whole ? nullptr : a.part_o + slot * group * D, a.part_ml + slot * group);
  }
}

// --- selected form ------------------------------------------------------------

// Where a slot's codes and scales lie. A page's strides are below 2^36 (codes, multiples of 16) and 2^32.
struct SlotAt {
  uint64_t codes, scales;
};
__device__ __forceinline__ SlotAt slot_at(int slot, int64_t page, int64_t pos, int64_t s_page, int64_t s_pos) {
  const uint32_t in = slot & 63;
  return {slot_offset(slot, static_cast<uint32_t>(page >> 4), static_cast<uint32_t>(pos >> 4)) << 4,
          static_cast<uint64_t>(static_cast<uint32_t>(slot) >> 6) * static_cast<uint32_t>(s_page) + in * static_cast<uint32_t>(s_pos)};
}

template <class T, int D, int NQ>
__global__ void __launch_bounds__(kThreads, 2) kv_selected_fp4_kernel(KvFp4Args a) {
  typedef Wave4<T, D, NQ> W;
  __shared__ union {
    SlotAt list[2][kKvSelBlock];   // of keys and values: made once by one lane, not by each that reads there
    Merge<T, D> merge;
  } lds;
  __shared__ v4u q_lds[W::kShared ? NQ * W::kChunks * 64 : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int qg = (a.G + 16 * NQ - 1) / (16 * NQ);
  ListPart p;
  bool fill;
  const bool any = p.take(a, static_cast<int64_t>(a.Hkv) * qg, &fill);
  if (!any && !fill) return;
  const int kvh = p.g / qg, first = (p.g % qg) * 16 * NQ, rows = a.G - first < 16 * NQ ? a.G - first : 16 * NQ;
  const int64_t head0 = p.r * a.H + static_cast<int64_t>(kvh) * a.G + first;
  if (!any) {
    for (int h = 0; h < rows; ++h) fill_row<T, D>(a, head0 + h, p.n != 0, threadIdx.x, kThreads);
    return;
  }
  W w;
  w.init();
  w.start();
  w.load_q(a.q + p.r * a.q_row + (static_cast<int64_t>(kvh) * a.G + first) * D * 2, rows, a.q_keep, a.q_flip, q_lds);
  const char *kb = a.k + kvh * a.k_head + w.key_at(), *vb = a.v + kvh * a.v_head + w.value_at();
  const char *ksb = a.ks + kvh * a.ks_head + w.key_scale_at(), *vsb = a.vs + kvh * a.vs_head + w.value_scale_at();
  bool bad = false;
  for (int64_t b0 = p.from; b0 < p.to; b0 += kKvSelBlock) {
    const int len = static_cast<int>(p.to - b0 < kKvSelBlock ? p.to - b0 : kKvSelBlock);
    if (b0 != p.from) __syncthreads();
    bool mine = false;
    for (int i = threadIdx.x; i < len; i += kThreads) {
      const int s = a.slots[p.r * a.K + b0 + i];
      lds.list[0][i] = slot_at(s, a.k_page, a.k_pos, a.ks_page, a.ks_pos);
      lds.list[1][i] = slot_at(s, a.v_page, a.v_pos, a.vs_page, a.vs_pos);
      mine |= s < 0 || s >= 64 * a.P_phys;
    }
    if (__syncthreads_or(mine)) {   // nothing of the list is read
      bad = true;
      break;
    }
    run_tiles(
        w, wave, (len + 31) / 32, a.c,
        [&](int t) {
#pragma unroll
          for (int b = 0; b < W::kTiles; ++b) {
            const SlotAt at = lds.list[0][min(32 * t + 16 * b + w.col, len - 1)];
            w.load_k(b, LaneReads{kb + at.codes}, LaneReads{ksb + at.scales});
          }
        },
        [&](int t) {
#pragma unroll
          for (int j = 0; j < W::kMine; ++j) {
            const SlotAt at = lds.list[1][min(32 * t + w.mine(j), len - 1)];
            w.load_v(j, LaneReads{vb + at.codes}, LaneReads{vsb + at.scales});
          }
        },
        [&](int t, int* lo, int* hi) {
          *lo = 0;
          *hi = len - 32 * t;
        });
  }
  if (bad && threadIdx.x == 0) atomicOr(a.status, kStBadPage);
  const int64_t part = p.item * group_of<NQ>(a);
  join_waves<0, T, D>(lds.merge, w, bad, rows, static_cast<char*>(a.out) + head0 * D * 2, a.lse == nullptr ? nullptr : a.lse + head0,
                      a.splits == 1 ? nullptr : a.part_o + part * D, a.part_ml + part);
}

// --- dispatch -----------------------------------------------------------------

template <class T, int D, int NQ>
void decode_on(KvFp4Args a, hipStream_t st) {
  const int groups = kKvDecodeGroups;
  const double page_ns = NQ > 1 ? 1000 : 100 + 2.75 * D;
  const double sums_ns = kv_group_rows(D, a.G) * D * 4 * 0.8e-3, turn_ns = a.Q * a.H <= kJoinHeads ? 20 : 80;
  const double pairs = static_cast<double>(a.Q) * a.Hkv * kv_head_groups(D, a.G);
  a.join_cost = static_cast<uint32_t>((sums_ns + turn_ns / pairs) / page_ns * 65536.0);
  if (a.Q > kKvPlanRows) kv_plan_kernel<<<dim3(1), dim3(1024), 0, st>>>(a);
  kv_decode_fp4_kernel<T, D, NQ><<<dim3(groups), dim3(kThreads), 0, st>>>(a);
  const int64_t heads = a.Q * a.H;
  if (heads <= kJoinHeads)
    kv_decode_join_kernel<T, D, kWaves><<<dim3(static_cast<unsigned>(heads)), dim3(kThreads), 0, st>>>(a, 16 * NQ, groups);
  else
    kv_decode_join_kernel<T, D, 1>
        <<<dim3(static_cast<unsigned>((heads + kWaves - 1) / kWaves)), dim3(kThreads), 0, st>>>(a, 16 * NQ, groups);
}

template <class T, int D, int NQ>
void selected_on(const KvFp4Args& a, hipStream_t st) {
  const int64_t items = a.Q * a.Hkv * kv_head_groups(D, a.G) * a.splits;
  const unsigned grid = static_cast<unsigned>((items + 7) / 8 * 8);
  kv_selected_fp4_kernel<T, D, NQ><<<dim3(grid), dim3(kThreads), 0, st>>>(a);
  if (a.splits > 1)
    kv_selected_join_kernel<T, D, 1>
        <<<dim3(static_cast<unsigned>((a.Q * a.H + kWaves - 1) / kWaves)), dim3(kThreads), 0, st>>>(a, 16 * NQ);
}

struct DecodeOn {
  const KvFp4Args& a;
  hipStream_t st;
  template <class T, int D, int NQ>
  void operator()() const { decode_on<T, D, NQ>(a, st); }
};
struct SelectedOn {
  const KvFp4Args& a;
  hipStream_t st;
  template <class T, int D, int NQ>
  void operator()() const { selected_on<T, D, NQ>(a, st); }
};

// Calls f<type, dim, query tiles>() for the call's type and sizes.
template <class T, class F>
void by_size(const KvFp4Args& a, F&& f) {
  const int nq = kv_tiles(a.D, a.G);
  if (a.D == 64) {
    if (nq == 1) f.template operator()<T, 64, 1>();
    else if (nq == 2) f.template operator()<T, 64, 2>();
    else f.template operator()<T, 64, 4>();
  } else if (a.D == 128) {
    if (nq == 1) f.template operator()<T, 128, 1>();
    else if (nq == 2) f.template operator()<T, 128, 2>();
    else f.template operator()<T, 128, 4>();
  } else {
    if (nq == 1) f.template operator()<T, 256, 1>();
    else f.template operator()<T, 256, 2>();
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
