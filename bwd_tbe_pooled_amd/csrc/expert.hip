// Tokens sorted by expert and back: the plan (a stable split of the N*K
// assignments by expert), dispatch and combine, and their gradients.
//
// Every row kernel gives a wave a segment of one token's row (U vectors of 16
// bytes per lane) and walks the token's K places with it, so that the row the
// K assignments share is read or written once and the K other rows move at
// full vector width. They are bound by HBM: no row is read twice. 16384 tokens
// with 8 assignments, 2048 bf16 (604 MB either way): dispatch 120 us, 5.0 TB/s
// (it writes 4 KB rows in no order), combine 100 us, 6.0; the gradients of 8192
// with 4, 4096 bf16: 99 us for 604 MB and 46 us for 336 MB. One or four vectors
// a lane in place of two, and more or fewer rows in flight, are within 4%.
#include "lm_split.h"

namespace tbe {

namespace {

struct ExpertOf {
  using type = int32_t;
  const void* ids;
  int32_t idx64, E;
  __device__ __forceinline__ type none() const { return E; }
  __device__ __forceinline__ type load(int64_t j) const {
    const int64_t v = load_id(ids, idx64, j);
    return v >= 0 && v < E ? (int32_t)v : E;  // dropped: the last bin
  }
  __device__ __forceinline__ int32_t bin(type v) const { return v; }
};

__global__ __launch_bounds__(kSplitThreads) void expert_count_kernel(
    ExpertOf of, int64_t M, SplitShape sh, int32_t stride, int32_t* __restrict__ counts) {
  split_count(M, sh, of.E + 1, stride, counts, of);
}

__global__ __launch_bounds__(kSplitThreads) void expert_plan_kernel(
    ExpertOf of, int64_t M, SplitShape sh, int bits, int32_t stride,
    const int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
    int32_t* __restrict__ order, int32_t* __restrict__ slots) {
  __shared__ SplitLds s;
  const int32_t E = of.E;
  split_tile(M, sh, E + 1, bits, stride, counts, s, of, [&](int64_t j, int32_t, int32_t bin, int32_t p) {
    order[p] = (int32_t)j;
    slots[j] = bin == E ? ~p : p;
  });
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= E; i += kSplitThreads) offsets[i] = s.start[i];
}

// Place of an assignment and whether it is kept; a slot outside [-M, M) has
// no place.
struct Slot {
  int32_t place;
  bool kept, has;
  __device__ __forceinline__ Slot(int32_t slot, int32_t M) {
    place = slot >= 0 ? slot : ~slot;
    has = place < M;
    kept = has && slot >= 0;
  }
};

// The token's K slots (and weights), one per lane, from one load: as scalars
// each would be waited for before its row.
struct TokenSlots {
  int32_t slot;
  float w;
  __device__ __forceinline__ TokenSlots(const int32_t* __restrict__ slots,
                                        const float* __restrict__ weights, int64_t n, int32_t K) {
    const int lane = lane_id();
    slot = lane < K ? slots[n * K + lane] : INT32_MIN;
    w = lane < K && weights ? weights[n * K + lane] : 1.f;
  }
  __device__ __forceinline__ Slot at(int32_t k, int32_t M) const {
    return Slot(__builtin_amdgcn_readlane(slot, k), M);
  }
  __device__ __forceinline__ float weight(int32_t k) const {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), k));
  }
};

template <typename T, int VE, int U>
__global__ __launch_bounds__(256) void expert_dispatch_kernel(
    const T* __restrict__ x, int64_t ldx, const int32_t* __restrict__ slots, int32_t K, int32_t M,
    int32_t D, T* __restrict__ xs, int64_t ldxs, Units units) {
  using R = typename Pack<T, VE>::raw;
  const int32_t nv = (D + VE - 1) / VE;
  for (UnitWalk u(units, blockIdx.x * 4 + wave_index()); u.valid(units); u.next(units)) {
    const T* row = x + u.row * ldx;
    const int32_t i0 = u.seg * (U * kWave) + lane_id();
    const TokenSlots sl(slots, nullptr, u.row, K);
    R v[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i0 + i * kWave < nv) v[i] = load_pack_once<T, VE>(row + pack_column<VE>(i0 + i * kWave, D));
    for (int32_t k = 0; k < K; ++k) {
      const Slot s = sl.at(k, M);
      if (!s.has) continue;
      T* to = xs + (int64_t)s.place * ldxs;
      R zero;
      zero_raw(zero);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (i0 + i * kWave < nv)
          store_pack_once<T, VE>(to + pack_column<VE>(i0 + i * kWave, D), s.kept ? v[i] : zero);
    }
  }
}

// out[n] = sum of the kept places' rows, weighted unless w is null.
template <typename T, int VE, int U>
__global__ __launch_bounds__(256) void expert_combine_kernel(
    const T* __restrict__ ys, int64_t ldys, const int32_t* __restrict__ slots,
    const float* __restrict__ w, int32_t K, int32_t M, int32_t D, T* __restrict__ out, int64_t ldo,
    Units units) {
  using R = typename Pack<T, VE>::raw;
  const int32_t nv = (D + VE - 1) / VE;
  for (UnitWalk u(units, blockIdx.x * 4 + wave_index()); u.valid(units); u.next(units)) {
    const int32_t i0 = u.seg * (U * kWave) + lane_id();
    float acc[U][VE];
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[i][e] = 0.f;
    const TokenSlots sl(slots, w, u.row, K);
    constexpr int KU = 4;  // rows in flight
    for (int32_t k0 = 0; k0 < K; k0 += KU) {
      R v[KU][U];
      float wk[KU];
#pragma unroll
      for (int q = 0; q < KU; ++q) {
        const int32_t k = k0 + q < K ? k0 + q : K - 1;
        const Slot s = sl.at(k, M);
        const bool use = k0 + q < K && s.kept;
        wk[q] = use ? sl.weight(k) : 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          zero_raw(v[q][i]);
          if (use && i0 + i * kWave < nv)
            v[q][i] = load_pack_once<T, VE>(ys + (int64_t)s.place * ldys +
                                            pack_column<VE>(i0 + i * kWave, D));
        }
      }
#pragma unroll
      for (int q = 0; q < KU; ++q)
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float f[VE];
          widen<T, VE>(v[q][i], f);
#pragma unroll
          for (int e = 0; e < VE; ++e) acc[i][e] = fmaf(wk[q], f[e], acc[i][e]);
        }
    }
    T* to = out + u.row * ldo;
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i0 + i * kWave < nv)
        store_pack_once<T, VE>(to + pack_column<VE>(i0 + i * kWave, D), narrow<T, VE>(acc[i]));
  }
}

// dys[place] = w * dout[n], dw[n,k] = <dout[n], ys[place]>. WPT waves share a
// token; each keeps up to U vectors per lane of dout in registers over the K
// places, and wider rows go panel by panel with the partial dots in LDS.
// dys may be ys: a lane reads its vector of ys before it stores there. A row's
// last vector overlaps the one before it, which another wave may have: the
// columns it reads twice are left out of its dot, and with IN_PLACE it stores
// the others alone, element by element. So a column is stored only by the lane
// whose dot takes it, and no order among the lanes matters. (Whole vectors and
// single elements after them, in place or not, took 164 us in place of 137 at
// 20000 x 4 rows of 1029 bf16: a load and a store more per place. Asked at run
// time instead of by IN_PLACE it cost calls of a few hundred tokens 2 to 4%.)
template <typename T, int VE, int U, int WPT, bool IN_PLACE>
__global__ __launch_bounds__(256) void expert_combine_backward_kernel(
    const T* __restrict__ dout, int64_t lddo, const T* ys, int64_t ldys,
    const int32_t* __restrict__ slots, const float* __restrict__ w, int64_t N, int32_t K,
    int32_t M, int32_t D, T* dys, int64_t lddys, float* __restrict__ dw) {
  using R = typename Pack<T, VE>::raw;
  constexpr int TPB = 4 / WPT;  // tokens of a workgroup
  __shared__ float dots[4][64];
  const int wave = wave_index();
  const int lane = lane_id();
  const int part = wave % WPT;
  const int32_t nv = (D + VE - 1) / VE;
  for (int64_t n0 = (int64_t)blockIdx.x * TPB; n0 < N; n0 += (int64_t)gridDim.x * TPB) {
    const int64_t n = n0 + wave / WPT;
    const bool live = n < N;
    if (lane < K) dots[wave][lane] = 0.f;
    wave_lds_sync();
    if (live) {
      const TokenSlots sl(slots, w, n, K);
      for (int32_t p0 = part * kWave + lane; p0 - lane < nv; p0 += U * WPT * kWave) {
        float d[U][VE];
        int32_t col[U], skip[U];
        bool in[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int32_t at = p0 + i * (WPT * kWave);
          in[i] = at < nv;
          col[i] = in[i] ? pack_column<VE>(at, D) : 0;
          skip[i] = in[i] ? pack_overlap<VE>(at, D) : VE;
          R r;
          zero_raw(r);
          if (in[i]) r = load_pack<T, VE>(dout + n * lddo + col[i]);
          widen<T, VE>(r, d[i]);
        }
        constexpr int KU = 2;  // places in flight
        for (int32_t k0 = 0; k0 < K; k0 += KU) {
          R v[KU][U];
          int32_t place[KU];
          bool kept[KU], has[KU];
#pragma unroll
          for (int q = 0; q < KU; ++q) {
            const Slot s = sl.at(k0 + q < K ? k0 + q : K - 1, M);
            place[q] = s.place;
            kept[q] = k0 + q < K && s.kept;
            has[q] = k0 + q < K && s.has;
#pragma unroll
            for (int i = 0; i < U; ++i) {
              zero_raw(v[q][i]);
              if (kept[q] && in[i])
                v[q][i] = load_pack_once<T, VE>(ys + (int64_t)place[q] * ldys + col[i]);
            }
          }
#pragma unroll
          for (int q = 0; q < KU; ++q) {
            if (!has[q]) continue;
            const float wk = kept[q] ? sl.weight(k0 + q) : 0.f;
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < U; ++i) {
              float f[VE], o[VE];
              widen<T, VE>(v[q][i], f);
#pragma unroll
              for (int e = 0; e < VE; ++e) {
                const float t = fmaf(d[i][e], f[e], dot);
                dot = e >= skip[i] ? t : dot;
                o[e] = kept[q] ? wk * d[i][e] : 0.f;
              }
              if (!in[i]) continue;
              T* to = dys + (int64_t)place[q] * lddys + col[i];
              const R r = narrow<T, VE>(o);
              if (IN_PLACE && skip[i] > 0) {
                const T* own = reinterpret_cast<const T*>(&r);
#pragma unroll
                for (int e = 0; e < VE; ++e)
                  if (e >= skip[i]) to[e] = own[e];
              } else {
                store_pack_once<T, VE>(to, r);
              }
            }
            dot = wave_sum(dot);
            if (kept[q] && lane == 0) dots[wave][k0 + q] += dot;
          }
        }
      }
    }
    if constexpr (WPT > 1) __syncthreads(); else wave_lds_sync();
    if (live && part == 0 && lane < K) {
      float t = 0.f;
#pragma unroll
      for (int q = 0; q < WPT; ++q) t += dots[wave + q][lane];
      dw[n * K + lane] = t;
    }
    if constexpr (WPT > 1) __syncthreads(); else wave_lds_sync();
  }
}

// Vector width of a row kernel: 16 bytes, single elements for rows narrower
// than that.
template <typename T, typename F>
hipError_t with_width(int32_t D, F f) {
  constexpr int VE = pack_elems<T>();
  if (D >= VE) return f(std::integral_constant<int, VE>{});
  return f(std::integral_constant<int, 1>{});
}

}  // namespace

SplitShape split_shape(int64_t n, int32_t bins) {
  // one workgroup alone: 4096 keys in 6.1 us (64 bins; 512 bins 7.2), where two
  // launches take 7.4 (8.9); 8192 keys in 9.1 (10.7)
  if (n <= 4096) return SplitShape{1, n > 0 ? (int32_t)((n + 1023) / 1024 * 1024) : 1024};
  // every tile reads all tiles' counts (about 80 bytes a ns) and places 1024
  // keys a round (about 1.4 us): the sum is least at this number of tiles.
  // 262144 keys in 1001 bins: 12.4 us with 86 tiles, 13.0 with 43, 19.4 with 256.
  int64_t tiles = 1;
  while (tiles < 256 && tiles * tiles * bins < n * 28) ++tiles;
  const int64_t len = ((n + tiles - 1) / tiles + 1023) / 1024 * 1024;
  return SplitShape{(int32_t)((n + len - 1) / len), (int32_t)len};
}

int32_t split_stride(int32_t bins) { return (bins + 3) / 4 * 4; }

static int bits_for(int32_t bins) {
  int b = 0;
  while ((1 << b) < bins) ++b;
  return b;
}

hipError_t launch_expert_plan(const tbe_expert_desc& d, const void* ids, int32_t* offsets,
                              int32_t* order, int32_t* slots, int32_t* counts, hipStream_t s) {
  const int64_t M = d.N * d.K;
  const SplitShape sh = split_shape(M, d.E + 1);
  const int32_t stride = split_stride(d.E + 1);
  const ExpertOf of{ids, d.idx64, d.E};
  if (sh.tiles > 1) {
    hipLaunchKernelGGL(expert_count_kernel, dim3(sh.tiles), dim3(kSplitThreads), 0, s, of, M, sh,
                       stride, counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(expert_plan_kernel, dim3(sh.tiles), dim3(kSplitThreads), 0, s, of, M, sh,
                     bits_for(d.E + 1), stride, counts, offsets, order, slots);
  return hipGetLastError();
}

hipError_t launch_expert_dispatch(const tbe_expert_desc& d, const void* x, int64_t ldx,
                                  const int32_t* slots, void* xs, int64_t ldxs, hipStream_t s) {
  return with_type(d.dtype, [&](auto t) {
    using T = decltype(t);
    return with_width<T>(d.D, [&](auto ve) {
      constexpr int VE = decltype(ve)::value;
      constexpr int U = 2;
      unsigned blocks;
      const Units u = make_units(d.N, (d.D + U * kWave * VE - 1) / (U * kWave * VE), &blocks);
      hipLaunchKernelGGL((expert_dispatch_kernel<T, VE, U>), dim3(blocks), dim3(256), 0, s,
                         static_cast<const T*>(x), ldx, slots, d.K, (int32_t)(d.N * d.K), d.D,
                         static_cast<T*>(xs), ldxs, u);
      return hipGetLastError();
    });
  });
}

hipError_t launch_expert_combine(const tbe_expert_desc& d, const void* ys, int64_t ldys,
                                 const int32_t* slots, const float* w, void* out, int64_t ldo,
                                 hipStream_t s) {
  return with_type(d.dtype, [&](auto t) {
    using T = decltype(t);
    return with_width<T>(d.D, [&](auto ve) {
      constexpr int VE = decltype(ve)::value;
      constexpr int U = 2;
      unsigned blocks;
      const Units u = make_units(d.N, (d.D + U * kWave * VE - 1) / (U * kWave * VE), &blocks);
      hipLaunchKernelGGL((expert_combine_kernel<T, VE, U>), dim3(blocks), dim3(256), 0, s,
                         static_cast<const T*>(ys), ldys, slots, w, d.K, (int32_t)(d.N * d.K), d.D,
                         static_cast<T*>(out), ldo, u);
      return hipGetLastError();
    });
  });
}

hipError_t launch_expert_combine_backward(const tbe_expert_desc& d, const void* dout, int64_t lddo,
                                          const void* ys, int64_t ldys, const int32_t* slots,
                                          const float* w, void* dys, int64_t lddys, float* dw,
                                          hipStream_t s) {
  return with_type(d.dtype, [&](auto t) {
    using T = decltype(t);
    return with_width<T>(d.D, [&](auto ve) {
      constexpr int VE = decltype(ve)::value;
      constexpr int U = 2;
      auto go = [&](auto wpt, auto in_place) {
        constexpr int WPT = decltype(wpt)::value;
        constexpr bool IN_PLACE = decltype(in_place)::value;
        const int64_t need = (d.N * WPT + 3) / 4;
        const unsigned blocks = (unsigned)(need < (1 << 20) ? need : (1 << 20));
        hipLaunchKernelGGL((expert_combine_backward_kernel<T, VE, U, WPT, IN_PLACE>), dim3(blocks),
                           dim3(256), 0, s, static_cast<const T*>(dout), lddo,
                           static_cast<const T*>(ys), ldys, slots, w, d.N, d.K,
                           (int32_t)(d.N * d.K), d.D, static_cast<T*>(dys), lddys, dw);
        return hipGetLastError();
      };
      // one wave holds U vectors per lane of a row; wider rows take four
      auto with_waves = [&](auto in_place) {
        if ((d.D + VE - 1) / VE <= U * kWave) return go(std::integral_constant<int, 1>{}, in_place);
        return go(std::integral_constant<int, 4>{}, in_place);
      };
      if constexpr (VE > 1)
        if (dys == ys && d.D % VE) return with_waves(std::true_type{});
      return with_waves(std::false_type{});
    });
  });
}

}  // namespace tbe
