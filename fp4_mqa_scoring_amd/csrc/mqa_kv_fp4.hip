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

// A wave's tile of 32 positions over a cache in 4 bits. Lane (col, grp) holds, of keys 16 a + col, the codes of
// kKeyDims neighbouring dims (one block's, or a half of one with D = 64), and of values mine(j) those of D / 16.
template <class T, int D, int NQ, int SLACK = 0>
struct Wave4 : Wave<T, false, D, NQ, 32, false, SLACK> {
  typedef Wave<T, false, D, NQ, 32, false, SLACK> Base;
  using Base::kChunks;
  using Base::kDims;
  using Base::kMine;
  using Base::kTiles;
  using Base::col;
  using Base::grp;
  using Base::q;
  typedef typename Base::P P;
  static constexpr int kKeyBlocks = D == 256 ? 2 : 1;    // scales of a lane's key
  static constexpr int kKeyWords = D / 32;               // words of 8 codes of a lane's key
  static constexpr int kWords4 = D == 256 ? 2 : 1;       // words of a lane's value (half of one with D = 64)

  uint32_t kc[kTiles][kKeyWords], kb[kTiles][kKeyBlocks];
  uint32_t vc[kMine][kWords4], vb[kMine];

  // First dim of matrix step c in this lane's keys.
  __device__ __forceinline__ int step_dim(int c) const {
    return D == 64 ? 16 * grp + 8 * c : 128 * (c >> 2) + 32 * grp + 8 * (c & 3);
  }

  __device__ __forceinline__ void load_q(const char* p, int rows, uint32_t keep, uint32_t flip) {
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int h = 16 * n + col;
        v4u x = {0, 0, 0, 0};
        if (h < rows) x = *reinterpret_cast<const v4u*>(p + (static_cast<int64_t>(h) * D + step_dim(c)) * 2);
        q[n][c] = (x & v4u{keep, keep, keep, keep}) ^ v4u{flip, flip, flip, flip};
      }
  }

  // Position 16 a + col has its codes at `p` and its scales at `s`.
  __device__ __forceinline__ void load_k(int a, const char* p, const char* s) {
    if constexpr (D == 64) {
      const v2u x = *reinterpret_cast<const v2u*>(p + 8 * grp);
      kc[a][0] = x.x;
      kc[a][1] = x.y;
      kb[a][0] = static_cast<uint8_t>(s[grp >> 1]);
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const v4u x = *reinterpret_cast<const v4u*>(p + 64 * i + 16 * grp);
#pragma unroll
        for (int e = 0; e < 4; ++e) kc[a][4 * i + e] = x[e];
        kb[a][i] = static_cast<uint8_t>(s[4 * i + grp]);
      }
    }
  }

  // Position mine(j) has its codes at `p` and its scales at `s`.
  __device__ __forceinline__ void load_v(int j, const char* p, const char* s) {
    const char* at = p + col * (D / 32);
    if constexpr (D == 64) {
      vc[j][0] = *reinterpret_cast<const uint16_t*>(at);
    } else if constexpr (D == 128) {
      vc[j][0] = *reinterpret_cast<const uint32_t*>(at);
    } else {
      const v2u x = *reinterpret_cast<const v2u*>(at);
      vc[j][0] = x.x;
      vc[j][1] = x.y;
    }
    vb[j] = static_cast<uint8_t>(s[col * kDims / 32]);
  }

  __device__ __forceinline__ void scores(v4f (&s)[NQ][kTiles]) {
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
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int a = 0; a < kTiles; ++a) s[n][a] = T::mfma(x[a], q[n][c], s[n][a]);
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

// --- decode form --------------------------------------------------------------

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 2) kv_decode_fp4_kernel(KvFp4Args a) {
  typedef Wave4<T, D, 1> W;
  __shared__ Plan<kWaves> plan;
  __shared__ Merge<T, D> merge;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t* prefix = plan.make(a);
  const int qg = (a.G + 15) / 16;
  const int64_t gh = static_cast<int64_t>(a.Hkv) * qg;
  const int64_t units = prefix[a.Q] * gh;
  const int64_t share = unit_share(a, units, gridDim.x);
  int64_t cur = blockIdx.x * share;
  const int64_t stop = cur + share < units ? cur + share : units;
  const int group_rows = a.G < 16 ? a.G : 16;
  W w;
  w.init();
  while (cur < stop) {
    Segment sg;
    sg.take(a, prefix, gh, &cur, stop);
    const int64_t r = sg.r;
    const int kvh = sg.g / qg, first = (sg.g % qg) * 16, rows = a.G - first < 16 ? a.G - first : 16;
    const int start = sg.start, end = sg.end;
    const int32_t* table = a.table + static_cast<int64_t>(sg.seq) * a.max_pages;
    const int p0 = start >> 6;
    const int t_lo = max(2 * (p0 + sg.pa), start / 32);
    const int t_hi = min(2 * (p0 + sg.pb), (end + 31) / 32);
    const char *kb = a.k + kvh * a.k_head, *vb = a.v + kvh * a.v_head;
    const char *ksb = a.ks + kvh * a.ks_head, *vsb = a.vs + kvh * a.vs_head;
    const int64_t head0 = r * a.H + static_cast<int64_t>(kvh) * a.G + first;
    w.start();
    w.load_q(a.q + r * a.q_row + (static_cast<int64_t>(kvh) * a.G + first) * D * 2, rows, a.q_keep, a.q_flip);

    bool bad = false;
    int next = t_lo + wave < t_hi ? table[(t_lo + wave) / 2] : 0;   // entry of the next tile's page, read early
    int64_t page = 0;
    // positions outside the window are not read: their lanes read the nearest one inside
    auto clamp = [&](int pos) { return min(max(pos, start), end - 1) & 63; };
    run_tiles(
        w, t_lo + wave, t_hi, a.c,
        [&](int t) {
          page = next;
          if (t + kWaves < t_hi) next = table[(t + kWaves) / 2];
          if (page < 0 || page >= a.P_phys) {   // nothing of it is read; page 0 stands in
            bad = true;
            page = 0;
          }
          const char *codes = kb + page * a.k_page, *scales = ksb + page * a.ks_page;
#pragma unroll
          for (int b = 0; b < W::kTiles; ++b) {
            const int pos = clamp(32 * t + 16 * b + w.col);
            w.load_k(b, codes + static_cast<uint32_t>(pos * static_cast<int>(a.k_pos)),
                     scales + static_cast<uint32_t>(pos * static_cast<int>(a.ks_pos)));
          }
        },
        [&](int t) {
          const char *codes = vb + page * a.v_page, *scales = vsb + page * a.vs_page;
#pragma unroll
          for (int j = 0; j < W::kMine; ++j) {
            const int pos = clamp(32 * t + w.mine(j));
            w.load_v(j, codes + static_cast<uint32_t>(pos * static_cast<int>(a.v_pos)),
                     scales + static_cast<uint32_t>(pos * static_cast<int>(a.vs_pos)));
          }
        },
        [&](int t, int* lo, int* hi) {
          *lo = start - 32 * t;
          *hi = end - 32 * t;
        });
    if (bad && w.lane == 0) atomicOr(a.status, kStBadPage);
    const bool whole = sg.pa == 0 && sg.pb == sg.n;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (sg.pa == 0 ? 1 : 0);
    merge.run(w, bad, rows, 1.0f, static_cast<char*>(a.out) + head0 * D * 2, a.lse == nullptr ? nullptr : a.lse + head0,
              whole ? nullptr : a.part_o + slot * group_rows * D, a.part_ml + slot * group_rows);
  }
}

// --- selected form ------------------------------------------------------------

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 2) kv_selected_fp4_kernel(KvFp4Args a) {
  typedef Wave4<T, D, 1> W;
  __shared__ int list[kKvSelBlock];
  __shared__ Merge<T, D> merge;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int qg = (a.G + 15) / 16;
  ListPart p;
  bool fill;
  const bool any = p.take(a, static_cast<int64_t>(a.Hkv) * qg, &fill);
  if (!any && !fill) return;
  const int kvh = p.g / qg, first = (p.g % qg) * 16, rows = a.G - first < 16 ? a.G - first : 16;
  const int64_t head0 = p.r * a.H + static_cast<int64_t>(kvh) * a.G + first;
  if (!any) {
    for (int h = 0; h < rows; ++h) fill_row<T, D>(a, head0 + h, p.n != 0, threadIdx.x, kThreads);
    return;
  }
  W w;
  w.init();
  w.start();
  w.load_q(a.q + p.r * a.q_row + (static_cast<int64_t>(kvh) * a.G + first) * D * 2, rows, a.q_keep, a.q_flip);
  const char *kb = a.k + kvh * a.k_head, *vb = a.v + kvh * a.v_head;
  const char *ksb = a.ks + kvh * a.ks_head, *vsb = a.vs + kvh * a.vs_head;
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
        w, wave, (len + 31) / 32, a.c,
        [&](int t) {
#pragma unroll
          for (int b = 0; b < W::kTiles; ++b) {
            const int64_t s = list[min(32 * t + 16 * b + w.col, len - 1)], page = s >> 6, pos = s & 63;
            w.load_k(b, kb + page * a.k_page + pos * a.k_pos, ksb + page * a.ks_page + pos * a.ks_pos);
          }
        },
        [&](int t) {
#pragma unroll
          for (int j = 0; j < W::kMine; ++j) {
            const int64_t s = list[min(32 * t + w.mine(j), len - 1)], page = s >> 6, pos = s & 63;
            w.load_v(j, vb + page * a.v_page + pos * a.v_pos, vsb + page * a.vs_page + pos * a.vs_pos);
          }
        },
        [&](int t, int* lo, int* hi) {
          *lo = 0;
          *hi = len - 32 * t;
        });
  }
  if (bad && threadIdx.x == 0) atomicOr(a.status, kStBadPage);
  // all heads of a key head count as one group in the workspace
  const int64_t part = ((p.r * a.Hkv + kvh) * a.splits + p.split) * a.G + first;
  merge.run(w, bad, rows, 1.0f, static_cast<char*>(a.out) + head0 * D * 2, a.lse == nullptr ? nullptr : a.lse + head0,
            a.splits == 1 ? nullptr : a.part_o + part * D, a.part_ml + part);
}

// --- dispatch -----------------------------------------------------------------

template <class T, int D>
void decode_on(KvFp4Args a, hipStream_t st) {
  const int groups = kKvDecodeGroups;
  const double page_ns = 100 + 2.75 * D;
  const int qg = (a.G + 15) / 16;
  const double sums_ns = (a.G < 16 ? a.G : 16) * D * 4 * 0.8e-3, turn_ns = a.Q * a.H <= kJoinHeads ? 20 : 80;
  const double pairs = static_cast<double>(a.Q) * a.Hkv * qg;
  a.join_cost = static_cast<uint32_t>((sums_ns + turn_ns / pairs) / page_ns * 65536.0);
  if (a.Q > kKvPlanRows) kv_plan_kernel<<<dim3(1), dim3(1024), 0, st>>>(a);
  kv_decode_fp4_kernel<T, D><<<dim3(groups), dim3(kThreads), 0, st>>>(a);
  const int64_t heads = a.Q * a.H;
  if (heads <= kJoinHeads)
    kv_decode_join_kernel<T, D, kWaves><<<dim3(static_cast<unsigned>(heads)), dim3(kThreads), 0, st>>>(a, 16, groups);
  else
    kv_decode_join_kernel<T, D, 1>
        <<<dim3(static_cast<unsigned>((heads + kWaves - 1) / kWaves)), dim3(kThreads), 0, st>>>(a, 16, groups);
}

template <class T, int D>
void selected_on(const KvFp4Args& a, hipStream_t st) {
  const int64_t items = a.Q * a.Hkv * ((a.G + 15) / 16) * a.splits;
  const unsigned grid = static_cast<unsigned>((items + 7) / 8 * 8);
  kv_selected_fp4_kernel<T, D><<<dim3(grid), dim3(kThreads), 0, st>>>(a);
  if (a.splits > 1)
    kv_selected_join_kernel<T, D, 1>
        <<<dim3(static_cast<unsigned>((a.Q * a.H + kWaves - 1) / kWaves)), dim3(kThreads), 0, st>>>(a, a.G);
}

struct DecodeOn {
  const KvFp4Args& a;
  hipStream_t st;
  template <class T, int D>
  void operator()() const { decode_on<T, D>(a, st); }
};
struct SelectedOn {
  const KvFp4Args& a;
  hipStream_t st;
  template <class T, int D>
  void operator()() const { selected_on<T, D>(a, st); }
};

// Calls f<type, dim>() for the call's type and size.
template <class F>
hipError_t by_type(const KvFp4Args& a, F&& f) {
  if (a.q_type == MQA_KV_BF16) {
    if (a.D == 64) f.template operator()<Bf16, 64>();
    else if (a.D == 128) f.template operator()<Bf16, 128>();
    else f.template operator()<Bf16, 256>();
  } else {
    if (a.D == 64) f.template operator()<Fp16, 64>();
    else if (a.D == 128) f.template operator()<Fp16, 128>();
    else f.template operator()<Fp16, 256>();
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_decode_fp4(const KvFp4Args& a, hipStream_t st) { return by_type(a, DecodeOn{a, st}); }
hipError_t launch_kv_selected_fp4(const KvFp4Args& a, hipStream_t st) { return by_type(a, SelectedOn{a, st}); }

}  // namespace mqa
