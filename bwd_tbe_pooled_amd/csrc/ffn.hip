// The experts' gated feed-forward products and their gradients.
//
//   forward   h = act(xs gate^T) * (xs up^T)      one kernel: a tile holds the same
//                                                 columns of both products
//             ys = h down^T
//   backward  dh = dys down, from which the same kernel forms the gradients of the
//                            two products, and h again, from the kept products
//             dxs = dg gate + du up               one sum over 2 F
//             dgate = dg^T xs, dup = du^T xs, ddown = dys^T h       one kernel
//
// A workgroup finds its expert and rows from the offsets by itself, so nothing
// waits for the host; workgroups beyond the last tile end at once. A tile's rows
// are one expert's: rows behind its end repeat its last row and are not stored.
#include <algorithm>
#include <type_traits>

#include "ffn_tile.h"

namespace tbe {
namespace {

enum Product { Up, Down, Dh, Dx, Dw };

struct Args {
  const int32_t* offsets;
  int32_t M, E, D, F;
  int32_t act;
  int32_t nt;                      // blocks of columns (Dw: unused)
  int64_t tiles;
  const void* a; int64_t lda;      // rows: xs, h, dys, or the gradients of g and u
  tbe_stack b0, b1;                // matrices: gate and up, or down
  const void* pre; int64_t ldpre;  // Dh: the kept products
  void* c; int64_t ldc;            // rows written: h, ys, dxs
  void* c2; int64_t ldc2;          // Up: pre or NULL; Dh: the gradients of g and u
  int64_t half;                    // columns from g's gradient to u's
  // Dw: dys, xs and the three results
  const void* dys; int64_t lddys;
  const void* xs; int64_t ldxs;
  const void* h; int64_t ldh;
  tbe_stack o0, o1, o2;
};

// exp(-g^2 / 2) and the normal distribution up to g. Far below zero 1 + erf cancels: the
// complement is formed there. 16 bits: it is the exponential times a polynomial in
// t = 1 / (1 + 0.46 |g| / sqrt(2)), the one of 8 terms with the least largest relative
// error, 2^-20; 2^-17 at -13 with the exponent's rounding.
template <typename T>
__device__ __forceinline__ void normal(float g, float& e, float& cdf) {
  if constexpr (sizeof(T) == 4) {
    e = expf(-0.5f * g * g);
    cdf = 0.5f * erfcf(g * -0.70710678f);
  } else {
    e = __builtin_amdgcn_exp2f(g * g * -0.72134752f);
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(g), 0.325052302f, 1.f));
    constexpr float k[8] = {0.129676998f, 0.129694268f, 0.115500562f, 0.0936133787f,
                            0.0257740766f, 0.085640423f, -0.113822207f, 0.0339228176f};
    float p = k[7];
#pragma unroll
    for (int i = 6; i >= 0; --i) p = fmaf(p, t, k[i]);
    p *= t * e;
    cdf = g < 0.f ? p : 1.f - p;
  }
}

// The activation and its derivative.
template <typename T>
__device__ __forceinline__ void activate(int32_t act, float g, float& a, float& da) {
  if (act == TBE_ACT_SILU) {
    // (16 bits: the hardware's power of two and reciprocal, 1 ulp each)
    const float s = sizeof(T) == 4 ? 1.f / (1.f + expf(-g))
                                   : __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * g));
    a = g * s;
    da = s * fmaf(g, 1.f - s, 1.f);
  } else {
    float e, cdf;
    normal<T>(g, e, cdf);
    a = g * cdf;
    da = fmaf(g * 0.39894228f, e, cdf);
  }
}

// Up to eight neighbouring elements of a row.
template <typename T>
__device__ __forceinline__ void store8(T* p, int32_t n, const float (&f)[8]) {
  if (n >= 8) {
    store_pack<T, 8>(p, narrow<T, 8>(f));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = round_to<T>(f[j]);
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, int32_t n, const float (&f)[4]) {
  if (n >= 4) {
    store_pack<T, 4>(p, narrow<T, 4>(f));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[j] = round_to<T>(f[j]);
  }
}
template <typename T>
__device__ __forceinline__ typename Pack<T, 8>::raw load8(const T* p, int32_t n) {
  typename Pack<T, 8>::raw r{};
  if (n >= 8) {
    r = load_pack<T, 8>(p);
  } else if (n > 0) {
    T e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = j < n ? p[j] : T{};
    r = __builtin_bit_cast(typename Pack<T, 8>::raw, e);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ const T* matrix(const tbe_stack& m, int32_t e) {
  return static_cast<const T*>(m.data) + (int64_t)e * m.stride;
}

// Where a tile lies.
struct Tile {
  int32_t e;
  int32_t m0, n0;          // first row (Dw: of the matrix) and column
  int32_t rows, cols;      // behind the last
  int32_t K;
  int32_t first;           // Dw: the expert's first row
  int32_t which;           // Dw: gate's, up's or down's gradient
};

// Workgroups stay, and take tiles by XCD: each XCD has a run of neighbouring tiles,
// its workgroups neighbours in it at any time.
// Large batches are bound by the feeding of the matrix cores: a step of a 256 x 256 tile
// takes 3060 to 3400 clocks, its products 2048. 131072 rows of 128 experts, 2048 x 768
// bf16: Up 1044 TFLOP/s, Down 872, Dh 713 (its epilogue reads two values an element and
// writes three), Dx 1067, Dw 988; 16384 rows of one expert, 4096 x 8192: 1189, 1251, 967,
// 1303, 1305.
template <typename T, Product P, class S, bool DIRECT>
__global__ __launch_bounds__(S::NT, 2) void ffn_kernel(Args g) {
  __shared__ __attribute__((aligned(kLdsUnit))) char lds[2 * S::AREA];
  constexpr int BK = kStepBytes / (int)sizeof(T);
  // columns of a tile: of Up's two products half each
  constexpr int BN = P == Up ? S::BN / 2 : S::BN, HALF = S::NF / 2, COLS = P == Up ? HALF : S::NF;
  static_assert(COLS % 2 == 0, "fragments in pairs");
  __shared__ Spans spans;
  const int64_t x = blockIdx.x % kXcds;
  int32_t begin, end;   // this XCD's tiles
  if constexpr (P == Dw) {
    // an expert's tiles take as long as its rows: an XCD's experts have as many as
    // another's (a tile's stores and first loads count as 6 steps of 64 rows)
    spans.fill(g.offsets, g.E, g.M, [](int32_t rows) { return (rows + 63) / 64 + 6; });
    const int64_t one = g.tiles / g.E, all = spans.upto[g.E - 1];
    auto bound = [&](int64_t x) {
      if (x == kXcds) return (int32_t)g.tiles;
      const int32_t e = spans.expert_of((int32_t)(x * all / kXcds), g.E);
      const int32_t before = e ? spans.upto[e - 1] : 0;
      return __builtin_amdgcn_readfirstlane(
          (int32_t)(e * one + (x * all - (int64_t)kXcds * before) * one /
                                  ((int64_t)kXcds * (spans.upto[e] - before))));
    };
    begin = bound(x);
    end = bound(x + 1);
  } else {
    spans.fill(g.offsets, g.E, g.M, [](int32_t rows) { return (rows + S::BM - 1) / S::BM; });
    const int32_t all = __builtin_amdgcn_readfirstlane(spans.upto[g.E - 1]) * g.nt;
    const int32_t per = (all + kXcds - 1) / kXcds;
    begin = (int32_t)x * per;
    end = min(begin + per, all);
  }
  int32_t at = begin + (int32_t)(blockIdx.x / kXcds);
  const int32_t stride = (int32_t)(gridDim.x / kXcds);

  auto locate = [&](int32_t tile) {
    Tile t;
    if constexpr (P == Dw) {
      // tiles of one expert: gate's, up's, down's
      const int32_t ft = (g.F + S::BM - 1) / S::BM, dt = (g.D + S::BN - 1) / S::BN;
      const int32_t dt2 = (g.D + S::BM - 1) / S::BM, ft2 = (g.F + S::BN - 1) / S::BN;
      const int32_t each = ft * dt, one = 2 * each + dt2 * ft2;
      t.e = tile / one;
      const int32_t in = tile % one;
      t.which = in < each ? 0 : in < 2 * each ? 1 : 2;
      const int32_t across = t.which == 2 ? ft2 : dt, place = in - t.which * each;
      t.m0 = place / across * S::BM;
      t.n0 = place % across * S::BN;
      t.rows = t.which == 2 ? g.D : g.F;
      t.cols = t.which == 2 ? g.F : g.D;
      t.first = __builtin_amdgcn_readfirstlane(spans.first[t.e]);
      t.K = __builtin_amdgcn_readfirstlane(spans.first[t.e + 1]) - t.first;
    } else {
      t.e = __builtin_amdgcn_readfirstlane(spans.expert_of(tile / g.nt, g.E));
      t.first = __builtin_amdgcn_readfirstlane(spans.first[t.e]);
      t.rows = __builtin_amdgcn_readfirstlane(spans.first[t.e + 1]);
      const int32_t blocks = (t.rows - t.first + S::BM - 1) / S::BM;
      const int32_t place = tile - (__builtin_amdgcn_readfirstlane(spans.upto[t.e]) - blocks) * g.nt;
      // an expert's tiles in groups of 8 blocks of rows, in a group the rows first: the
      // 32 tiles that an XCD works on share rows and matrices in its L2
      constexpr int GROUP = 8;
      const int32_t group = place / (GROUP * g.nt) * GROUP;
      const int32_t high = min(GROUP, blocks - group), in = place - group * g.nt;
      t.m0 = t.first + (group + in % high) * S::BM;
      t.n0 = in / high * BN;
      t.cols = P == Up || P == Dh ? g.F : g.D;
      t.K = P == Up || P == Dh ? g.D : g.F;
      t.which = 0;
    }
    return t;
  };
  using OA = Operand<T, P == Dw ? Across : Along, S::BM, S::NT, DIRECT>;
  using OB = Operand<T, P == Up || P == Down ? Along : Across, S::BN, S::NT, DIRECT, P == Up>;
  Walk<T, S, DIRECT, OA, OB> w;
  w.lds = lds;
  // Sets the operands to a tile; part 1 of Dx is up's.
  auto set = [&](const Tile& t, int part) {
    if constexpr (P == Dw) {
      const bool down = t.which == 2;
      const int64_t lda = down ? g.lddys : g.lda, ldb = down ? g.ldh : g.ldxs;
      const T* a = static_cast<const T*>(down ? g.dys : g.a) + (t.which == 1 ? g.half : 0) + t.first * lda + t.m0;
      const T* b = static_cast<const T*>(down ? g.h : g.xs) + t.first * ldb + t.n0;
      w.a.start(t.rows - t.m0, lda, t.K, [&](int) { return a; }, a);
      w.b.start(t.cols - t.n0, ldb, t.K, [&](int) { return b; }, b);
    } else {
      const T* a = static_cast<const T*>(g.a) + (int64_t)t.m0 * g.lda + (part ? g.half : 0);
      const int32_t last = t.rows - 1 - t.m0, right = t.cols - 1 - t.n0;
      w.a.start(S::BM, g.lda, t.K, [&](int r) { return a + (int64_t)min(r, last) * g.lda; }, a);
      const tbe_stack& m = part ? g.b1 : g.b0;
      if constexpr (P == Up) {   // rows of up behind those of gate
        const T *b0 = matrix<T>(g.b0, t.e) + t.n0 * g.b0.ld, *b1 = matrix<T>(g.b1, t.e) + t.n0 * g.b1.ld;
        w.b.start(S::BN, 0, t.K, [&](int r) {
          return r < BN ? b0 + min(r, right) * g.b0.ld : b1 + min(r - BN, right) * g.b1.ld;
        }, b0, b1);
      } else if constexpr (P == Down) {
        const T* b = matrix<T>(m, t.e) + t.n0 * m.ld;
        w.b.start(S::BN, 0, t.K, [&](int r) { return b + min(r, right) * m.ld; }, b);
      } else {
        const T* b = matrix<T>(m, t.e) + t.n0;
        w.b.start(t.cols - t.n0, m.ld, t.K, [&](int) { return b; }, b);
      }
    }
  };
  auto steps = [](int32_t k) { return (k + BK - 1) / BK; };
  auto row_b = [&](int j) {
    const int wn = wave_index() % S::WN;
    if constexpr (P == Up) return j < HALF ? (wn * HALF + j) * 16 : BN + (wn * HALF + j - HALF) * 16;
    else return (wn * S::NF + j) * 16;
  };

  if (at >= end) return;
  Tile t = locate(at);
  set(t, 0);
  if (t.K > 0) w.fetch();
  for (; at < end; at += stride) {
    f32x4 acc[S::MF][S::NF];
#pragma unroll
    for (int i = 0; i < S::MF; ++i)
#pragma unroll
      for (int j = 0; j < S::NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const Tile now = t;
    // Dh's rows of `pre`, AHEAD at a time: a group is loaded before the stores of the group
    // before it, the first one before the next tile's first step
    constexpr int AHEAD = P == Dh ? 1 : S::MF, GROUPS = S::MF / AHEAD;
    static_assert(S::MF % AHEAD == 0, "whole groups");
    typedef typename Pack<T, 8>::raw Raw;
    [[maybe_unused]] Raw kept[P == Dh ? 2 : 1][AHEAD][COLS / 2][2];
    const bool whole = now.m0 + S::BM <= now.rows && now.n0 + BN <= now.cols;
    auto load_kept = [&](int group) {
      if constexpr (P == Dh) {
        const int thread = thread_again(), lane = thread % kWave;
        const int wave = __builtin_amdgcn_readfirstlane(thread / kWave), wm = wave / S::WN, wn = wave % S::WN;
        const int32_t nw = now.n0 + wn * COLS * 16 + eight_at(lane);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const int32_t m = now.m0 + (wm * S::MF + group * AHEAD + i) * 16 + lane % 16;
          const T* pre = static_cast<const T*>(g.pre) + m * g.ldpre + nw;
#pragma unroll
          for (int j = 0; j < COLS; j += 2) {
            Raw(&r)[2] = kept[group & 1][i][j / 2];
            if (whole) {
              r[0] = load_pack<T, 8>(pre + j * 16);
              r[1] = load_pack<T, 8>(pre + now.cols + j * 16);
            } else {
              const int32_t n = m < now.rows ? now.cols - nw - j * 16 : 0;
              r[0] = load8<T>(pre + j * 16, n);
              r[1] = load8<T>(pre + now.cols + j * 16, n);
            }
          }
        }
      }
    };
    w.multiply(acc, steps(now.K), P == Dx ? steps(now.K) : 0, row_b, [&] { set(now, 1); }, [&] {
      load_kept(0);
      if (at + stride < end) {
        t = locate(at + stride);
        set(t, 0);
        if (t.K > 0) w.fetch();
      }
      asm volatile("" ::: "memory");   // the stores stay behind the fetch
    });

    // eight columns of a row at a time
    auto finish = [&](auto is_whole) {
      constexpr bool WHOLE = decltype(is_whole)::value;
      const int thread = thread_again(), lane = thread % kWave;
      const int wave = __builtin_amdgcn_readfirstlane(thread / kWave), wm = wave / S::WN, wn = wave % S::WN;
      const int32_t N = now.cols, nw = now.n0 + wn * COLS * 16 + eight_at(lane);
      auto put = [&](T* p, int32_t n, const float(&f)[8]) {
        if constexpr (WHOLE) store_pack<T, 8>(p, narrow<T, 8>(f));
        else store8<T>(p, n, f);
      };
#pragma unroll
      for (int group = 0; group < GROUPS; ++group) {
        if (group + 1 < GROUPS) load_kept(group + 1);
#pragma unroll
        for (int i = group * AHEAD; i < (group + 1) * AHEAD; ++i) {
          const int32_t m = now.m0 + (wm * S::MF + i) * 16 + lane % 16;
          const bool in = WHOLE || m < now.rows;
          T *c, *c2 = nullptr;
          if constexpr (P == Dw) {
            const tbe_stack& o = now.which == 0 ? g.o0 : now.which == 1 ? g.o1 : g.o2;
            c = static_cast<T*>(o.data) + now.e * o.stride + m * o.ld;
          } else {
            c = static_cast<T*>(g.c) + m * g.ldc;
            c2 = static_cast<T*>(g.c2) + m * g.ldc2;
          }
#pragma unroll
          for (int j = 0; j < COLS; j += 2) {
            const int32_t n = nw + j * 16;
            float f[8];
            eight(acc[i][j], acc[i][j + 1], f);   // (all lanes)
            [[maybe_unused]] float u[8], v[8];
            if constexpr (P == Up) eight(acc[i][j + HALF], acc[i][j + HALF + 1], u);
            if (!WHOLE && (!in || n >= N)) continue;
            if constexpr (P == Up) {
              if (g.c2) {
                put(c2 + n, N - n, f);
                put(c2 + N + n, N - n, u);
              }
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                float x, da;
                activate<T>(g.act, f[q], x, da);
                f[q] = x * u[q];
              }
            } else if constexpr (P == Dh) {
              widen<T, 8>(kept[group & 1][i - group * AHEAD][j / 2][0], u);
              widen<T, 8>(kept[group & 1][i - group * AHEAD][j / 2][1], v);
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const float dh = f[q];
                float x, da;
                activate<T>(g.act, u[q], x, da);
                f[q] = x * v[q];
                u[q] = dh * v[q] * da;
                v[q] = dh * x;
              }
              put(c2 + n, N - n, u);
              put(c2 + g.half + n, N - n, v);
            }
            put(c + n, N - n, f);
          }
        }
        if constexpr (P == Dh) asm volatile("" ::: "memory");   // this group's stores before the next loads
      }
    };
    // stores of 16 bytes, of which a whole tile makes as many in every wave
    constexpr int STORES = S::MF * COLS / 2 * (sizeof(T) == 4 ? 2 : 1);
    if (whole) finish(std::true_type{});
    else finish(std::false_type{});
    w.later = !whole ? 0 : P == Dh || (P == Up && g.c2) ? 3 * STORES : STORES;
  }
}

// Few rows an expert (decoding): what counts is that the weights are read once, at
// memory's rate. A workgroup has 16 columns of an expert's products (NB = 2: of Up both
// products', of Down 32) and up to 16 MB of its rows at a time; its waves share k. A
// lane's pieces of a matrix row go straight to registers, and the waves' sums meet in
// LDS. WAVES: 4, or 16 where the workgroups are too few to fill the card. 32 rows of 64
// experts, 2048 x 768 bf16: Up 33 us for 167 MB of weights, 5.1 TB/s.
template <typename T, Product P, int MB, int NB, int WAVES>
__global__ __launch_bounds__(WAVES * kWave) void ffn_few_kernel(Args g) {
  constexpr int VE = 16 / (int)sizeof(T);
  constexpr int BK = 8 * VE;   // of k in one turn of a wave: a line of 128 bytes, in two halves
  constexpr int COLS = P == Up ? 16 : NB * 16;
  static_assert(P == Down || NB == 2, "both products of Up");
  __shared__ f32x4 meet[WAVES][MB][NB][kWave];
  const int wave = wave_index(), lane = lane_id();
  const int32_t e = blockIdx.x / g.nt, n0 = (int32_t)(blockIdx.x % g.nt) * COLS;
  const int32_t first = first_row(g.offsets, e, g.M);
  const int32_t end = max(first, min(max(g.offsets[e + 1], 0), g.M));
  const int32_t K = P == Up ? g.D : g.F, N = P == Up ? g.F : g.D;
  const int kl = lane / 16 * VE;   // of k, in half a line: this lane's
  const T* rows_b[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const tbe_stack& m = P == Up && j ? g.b1 : g.b0;
    const int32_t n = n0 + lane % 16 + (P == Up ? 0 : j * 16);
    rows_b[j] = matrix<T>(m, e) + min(n, N - 1) * m.ld + kl;
  }
  for (int32_t m0 = first; m0 < end; m0 += 16 * MB) {
    const T* rows_a[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
      rows_a[i] = static_cast<const T*>(g.a) + (int64_t)min(m0 + i * 16 + lane % 16, end - 1) * g.lda + kl;
    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // COUNT turns from k, their loads in flight together; WHOLE: all of them in the rows
    auto turns = [&](int32_t k, auto count, auto is_whole) {
      constexpr int COUNT = decltype(count)::value;
      auto piece = [&](const T* row, int32_t at) {   // 16 bytes, zeros behind K
        if constexpr (decltype(is_whole)::value) return __builtin_bit_cast(uint4, load_pack<T, VE>(row + at));
        const int32_t n = K - at - kl;
        uint4 r = make_uint4(0, 0, 0, 0);
        if (n >= VE) {
          r = __builtin_bit_cast(uint4, load_pack<T, VE>(row + at));
        } else if (n > 0) {
          T x[VE];
#pragma unroll
          for (int j = 0; j < VE; ++j) x[j] = j < n ? row[at + j] : T{};
          r = __builtin_bit_cast(uint4, x);
        }
        return r;
      };
      uint4 a[COUNT][MB][2], b[COUNT][NB][2];
#pragma unroll
      for (int t = 0; t < COUNT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int32_t at = k + t * WAVES * BK + h * BK / 2;
#pragma unroll
          for (int j = 0; j < NB; ++j) b[t][j][h] = piece(rows_b[j], at);
#pragma unroll
          for (int i = 0; i < MB; ++i) a[t][i][h] = piece(rows_a[i], at);
        }
#pragma unroll
      for (int t = 0; t < COUNT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = Mma<T>::mul(b[t][j][h], a[t][i][h], acc[i][j]);
    };
    int32_t k = wave * BK;
    constexpr int TURNS = MB == 1 ? 4 : 2;
    for (; k + ((TURNS - 1) * WAVES + 1) * BK <= K; k += TURNS * WAVES * BK)
      turns(k, std::integral_constant<int, TURNS>{}, std::true_type{});
    for (; k < K; k += WAVES * BK) turns(k, std::integral_constant<int, 1>{}, std::false_type{});
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) meet[wave][i][j][lane] = acc[i][j];
    __syncthreads();
    for (int i = wave; i < MB; i += WAVES) {   // a block of 16 rows' sums
      f32x4 s[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        s[j] = meet[0][i][j][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s[j] += meet[w][i][j][lane];
      }
      const int32_t m = m0 + i * 16 + lane % 16;
      if (m >= end) continue;
      T* c = static_cast<T*>(g.c) + m * g.ldc;
      if constexpr (P == Up) {
        const int32_t n = n0 + lane / 16 * 4;
        float f[4], u[4], h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float da;
          f[q] = s[0][q];
          u[q] = s[1][q];
          activate<T>(g.act, f[q], h[q], da);
          h[q] *= u[q];
        }
        if (g.c2) {
          T* c2 = static_cast<T*>(g.c2) + m * g.ldc2;
          store4<T>(c2 + n, N - n, f);
          store4<T>(c2 + N + n, N - n, u);
        }
        store4<T>(c + n, N - n, h);
      } else {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int32_t n = n0 + j * 16 + lane / 16 * 4;
          const float f[4] = {s[j][0], s[j][1], s[j][2], s[j][3]};
          store4<T>(c + n, N - n, f);
        }
      }
    }
    __syncthreads();
  }
}

int64_t blocks_of(int64_t n, int64_t b) { return (n + b - 1) / b; }

// Tiles of shape S that have work, at least.
template <Product P, class S>
int64_t tiles_of(const Args& g) {
  if (P == Dw)
    return (int64_t)g.E * (2 * blocks_of(g.F, S::BM) * blocks_of(g.D, S::BN) + blocks_of(g.D, S::BM) * blocks_of(g.F, S::BN));
  return std::max<int64_t>(std::min(g.E, g.M), blocks_of(g.M, S::BM)) *
         blocks_of(P == Up || P == Dh ? g.F : g.D, P == Up ? S::BN / 2 : S::BN);
}

// Launches one product with tiles of shape S.
template <typename T, Product P, class S>
hipError_t launch(Args g, bool direct, hipStream_t s) {
  if constexpr (P == Dw) {
    g.tiles = tiles_of<P, S>(g);
  } else {
    constexpr int BN = P == Up ? S::BN / 2 : S::BN;
    g.nt = (int32_t)blocks_of(P == Up || P == Dh ? g.F : g.D, BN);
    // every expert may end in a part of a block
    g.tiles = (g.M / S::BM + std::min(g.E, g.M)) * (int64_t)g.nt;
  }
  // as many workgroups as find room at once, a multiple of the XCDs
  constexpr int64_t kRoom = 256 * (S::BM * S::BN >= 65536 ? 1 : S::BM * S::BN >= 16384 ? 2 : 4);
  const unsigned grid = (unsigned)std::min(xcd_grid(g.tiles), kRoom);
  if (direct) ffn_kernel<T, P, S, true><<<grid, S::NT, 0, s>>>(g);
  else if constexpr (S::NT == 256) ffn_kernel<T, P, S, false><<<grid, S::NT, 0, s>>>(g);
  return hipGetLastError();
}

// Whether all pieces of 16 bytes lie whole and aligned in their matrices, and a tile's
// rows within the 2 GiB that a direct load's offsets reach.
struct Aligned {
  size_t size;
  bool ok = true;
  void rows(const void* p, int64_t ld) {
    ok = ok && reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0 && ld < (1 << 20);
  }
  void stack(const tbe_stack& m) {
    rows(m.data, m.ld);
    ok = ok && m.stride * size % 16 == 0;
  }
};

using Small = Shape<4, 1, 1, 4>;    // 64 x 64, four workgroups on a CU
using Middle = Shape<2, 2, 4, 4>;   // 128 x 128, two
using Large = Shape<2, 4, 8, 4>;    // 256 x 256, one

template <typename T, Product P, int MB>
hipError_t launch_few(Args g, hipStream_t s) {
  // workgroups that have work, at most: 512 give every CU eight waves
  constexpr int WIDE = P == Up ? 16 : 32;
  const int32_t cols = P == Up ? g.F : g.D;
  if (std::min(g.E, g.M) * blocks_of(cols, WIDE) >= 512) {
    g.nt = (int32_t)blocks_of(cols, WIDE);
    ffn_few_kernel<T, P, MB, 2, 4><<<(unsigned)(g.E * g.nt), 4 * kWave, 0, s>>>(g);
  } else {
    constexpr int WAVES = 16 / MB;
    g.nt = (int32_t)blocks_of(cols, 16);
    ffn_few_kernel<T, P, MB, P == Up ? 2 : 1, WAVES><<<(unsigned)(g.E * g.nt), WAVES * kWave, 0, s>>>(g);
  }
  return hipGetLastError();
}

// Launches one product with the tiles that suit it: the largest of which every CU has
// one, and an expert's rows fill most of (256 rows an expert and 64 experts of 2048 x
// 768: Large 217 us forward, Middle 209 for 192). With less than one Middle tile a CU
// Small is faster (one expert of 4096 x 8192, 192 rows: 153 against 171 us). Few rows
// are bound by the weights: where Middle has few tiles, ffn_few has more workgroups
// (the same, 1 row: 47 against 144 us; 63 rows: 101 against 144; eight experts of 4096
// x 1536: 62 against 87 for 1 row, 85 against 88 for 31, 127 against 89 for 63), else
// Middle's tiles read them as fast (64 experts: 131 and 131 us for 1 row, 160 and 127
// for 15).
template <typename T, Product P>
hipError_t launch_product(const Args& g, bool direct, hipStream_t s) {
  const int64_t rows = g.M / g.E, tiles = tiles_of<P, Middle>(g);
  if constexpr (P == Up || P == Down) {
    if (tiles < 512) {
      if (rows < 16) return launch_few<T, P, 1>(g, s);
      if (rows < 32) return launch_few<T, P, 2>(g, s);
      if (rows < 64 && tiles <= 128) return launch_few<T, P, 4>(g, s);
    }
  }
  if (tiles < 256) return launch<T, P, Small>(g, direct, s);
  if constexpr (sizeof(T) == 2)
    if (direct && rows >= 256 && tiles_of<P, Large>(g) >= 256) return launch<T, P, Large>(g, direct, s);
  return launch<T, P, Middle>(g, direct, s);
}

}  // namespace

FfnLayout ffn_layout(const tbe_ffn_desc& d) {
  const size_t size = d.dtype == TBE_F32 ? 4 : 2;
  auto pad = [](size_t n) { return (n + 255) / 256 * 256; };
  FfnLayout L;
  L.ld = (d.F + 7) / 8 * 8;
  L.h = 0;
  L.dgu = pad((size_t)d.M * L.ld * size);
  L.total = L.dgu + pad((size_t)d.M * 2 * L.ld * size) + 256;
  return L;
}

hipError_t launch_ffn_forward(const tbe_ffn_desc& d, const FfnForward& a, hipStream_t s) {
  const FfnLayout L = ffn_layout(d);
  return with_type(d.dtype, [&](auto t) {
    using T = decltype(t);
    Aligned al{sizeof(T)};
    al.rows(a.xs, a.ldxs);
    al.rows(nullptr, d.D);
    al.rows(nullptr, d.F);
    for (const tbe_stack* m : {&a.gate, &a.up, &a.down}) al.stack(*m);
    Args g = {};
    g.offsets = a.offsets;
    g.M = (int32_t)d.M; g.E = d.E; g.D = d.D; g.F = d.F; g.act = d.act;
    g.a = a.xs; g.lda = a.ldxs;
    g.b0 = a.gate; g.b1 = a.up;
    g.c = a.ws + L.h; g.ldc = L.ld;
    g.c2 = a.pre; g.ldc2 = a.ldpre;
    hipError_t e = launch_product<T, Up>(g, al.ok, s);
    if (e != hipSuccess) return e;
    g.a = a.ws + L.h; g.lda = L.ld;
    g.b0 = a.down;
    g.c = a.ys; g.ldc = a.ldys;
    return launch_product<T, Down>(g, al.ok, s);
  });
}

hipError_t launch_ffn_backward(const tbe_ffn_desc& d, const FfnBackward& a, hipStream_t s) {
  const FfnLayout L = ffn_layout(d);
  return with_type(d.dtype, [&](auto t) {
    using T = decltype(t);
    Aligned al{sizeof(T)};
    al.rows(a.xs, a.ldxs);
    al.rows(a.dys, a.lddys);
    al.rows(nullptr, d.D);
    al.rows(nullptr, d.F);
    for (const tbe_stack* m : {&a.gate, &a.up, &a.down}) al.stack(*m);
    Args g = {};
    g.offsets = a.offsets;
    g.M = (int32_t)d.M; g.E = d.E; g.D = d.D; g.F = d.F; g.act = d.act;
    g.half = L.ld;
    if (d.M > 0) {
      g.a = a.dys; g.lda = a.lddys;
      g.b0 = a.down;
      g.pre = a.pre; g.ldpre = a.ldpre;
      g.c = a.ws + L.h; g.ldc = L.ld;
      g.c2 = a.ws + L.dgu; g.ldc2 = 2 * L.ld;
      hipError_t e = launch_product<T, Dh>(g, al.ok, s);
      if (e != hipSuccess) return e;
      g.a = a.ws + L.dgu; g.lda = 2 * L.ld;
      g.b0 = a.gate; g.b1 = a.up;
      g.c = a.dxs; g.ldc = a.lddxs;
      e = launch_product<T, Dx>(g, al.ok, s);
      if (e != hipSuccess) return e;
    }
    g.a = a.ws + L.dgu; g.lda = 2 * L.ld;
    g.dys = a.dys; g.lddys = a.lddys;
    g.xs = a.xs; g.ldxs = a.ldxs;
    g.h = a.ws + L.h; g.ldh = L.ld;
    g.o0 = a.dgate; g.o1 = a.dup; g.o2 = a.ddown;
    return launch_product<T, Dw>(g, al.ok, s);
  });
}

}  // namespace tbe
