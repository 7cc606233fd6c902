// Layer norm of rows and its gradients.
//
// A row is cut into vectors of 16 bytes and lies in the registers of LPR lanes,
// NV vectors each, from its load to its store: memory is read once and written
// once, which bounds every case but the smallest. Mean and variance take two
// reductions, the second over x - mean: it also gives what the first mean lost
// by rounding, so a row far from zero keeps its deviation's precision. The
// backward needs one reduction of three sums: the third is again the sum of
// x - mean, as the mean in `stats` is rounded to float32.
//
// w and b, and in the backward the columns' sums of dw and db, stay in the
// registers of the lanes that own the columns while a workgroup walks over its
// rows. Workgroups leave a partial row of dw and db each; norm_join_kernel adds
// them in a fixed order. Rows wider than 2048 vectors are read again for each
// pass (norm_wide_*).
//
// Medians of many launches: 16384 rows of 4096 bf16, forward 54 us, 5.0 TB/s, backward 85,
// 4.8, and the join of 256 partial rows 5; 262144 rows of 1024, backward 272 us, 5.9 TB/s
// (the least of them 50, 73 and 261). Launches 8 to 50 after a pause of the card take up to
// a third more, on any buffers, and then as long as the first; a copy's do not. Not found why.
#include <algorithm>
#include <type_traits>

#include "lm.h"
#include "lm_device.h"

namespace tbe {
namespace {

constexpr int kThreads = 1024;      // of the backward's and the wide rows' workgroups
constexpr int kMaxParts = 256;      // workgroups of the backward: one per CU
constexpr int kMaxVectors = 2048;   // vectors of a row that stays in registers

// VE elements of a vector whose type is known at run time (the weights').
template <int VE>
__device__ __forceinline__ void load_as(const void* p, int32_t type, int64_t at, float (&f)[VE]) {
  if (type == TBE_F32) {
    const float* q = static_cast<const float*>(p) + at;
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = q[i];
  } else if (type == TBE_F16) {
    widen<f16_t, VE>(load_pack<f16_t, VE>(static_cast<const f16_t*>(p) + at), f);
  } else {
    widen<bf16_t, VE>(load_pack<bf16_t, VE>(static_cast<const bf16_t*>(p) + at), f);
  }
}

// Sums over the LPR lanes of a row, in each of them. Rows of more than a wave
// meet in LDS; `turn` alternates between two areas, so one barrier is enough.
template <int LPR, int NS>
__device__ __forceinline__ void row_sums(float (&s)[NS], float (*lds)[kThreads / kWave][NS],
                                         int& turn) {
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    s[i] = row16_sum(s[i]);
    if constexpr (LPR >= 32) s[i] += __shfl_xor(s[i], 16);
    if constexpr (LPR >= 64) s[i] += __shfl_xor(s[i], 32);
  }
  if constexpr (LPR > kWave) {
    constexpr int kWaves = LPR / kWave;
    const int wave = wave_index();
    if (lane_id() == 0) {
#pragma unroll
      for (int i = 0; i < NS; ++i) lds[turn][wave][i] = s[i];
    }
    __syncthreads();
    const int first = wave / kWaves * kWaves;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) s[i] += lds[turn][first + w][i];
    }
    turn ^= 1;
  }
}

struct ForwardArgs {
  const void* x; int64_t ldx;
  const void *w, *b;
  void* y; int64_t ldy;
  float* stats;
  int64_t N;
  int32_t D, wtype;
  float eps, inv_d;
};

// A lane's columns: vector i begins at col[i]; its first skip[i] columns belong
// to the vector before it (a row's last vector is moved back to end at D).
template <int VE, int LPR, int NV>
struct Columns {
  int32_t col[NV];
  int32_t skip[NV];
  __device__ __forceinline__ Columns(int32_t D) {
    const int32_t lane = threadIdx.x % LPR;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t v = lane + i * LPR;
      const bool in = (int64_t)v * VE < D;
      col[i] = in ? pack_column<VE>(v, D) : -1;
      skip[i] = in ? pack_overlap<VE>(v, D) : VE;
    }
  }
};

template <typename T, int VE, int LPR, int NV, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_forward_kernel(ForwardArgs a) {
  __shared__ float lds[2][kThreads / kWave][2];
  int turn = 0;
  const Columns<VE, LPR, NV> c(a.D);
  float w[NV][VE], b[NV][VE];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < VE; ++j) w[i][j] = 1.f, b[i][j] = 0.f;
    if (c.col[i] >= 0) {
      if (a.w) load_as<VE>(a.w, a.wtype, c.col[i], w[i]);
      if (a.b) load_as<VE>(a.b, a.wtype, c.col[i], b[i]);
    }
  }
  constexpr int kRows = THREADS / LPR;
  const int64_t step = (int64_t)gridDim.x * kRows;
  const int slot = threadIdx.x / LPR;
  typename Pack<T, VE>::raw raw[NV];
  auto load = [&](int64_t n) {
    const T* x = static_cast<const T*>(a.x) + n * a.ldx;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (c.col[i] >= 0) raw[i] = load_pack_once<T, VE>(x + c.col[i]);
  };
  // every lane walks the same number of rounds: the reductions need them all
  int64_t n = (int64_t)blockIdx.x * kRows + slot;
  if (n < a.N) load(n);
  for (int64_t n0 = (int64_t)blockIdx.x * kRows; n0 < a.N; n0 += step, n += step) {
    const bool live = n < a.N;
    float x[NV][VE];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (live && c.col[i] >= 0) widen<T, VE>(raw[i], x[i]);
      else
#pragma unroll
        for (int j = 0; j < VE; ++j) x[i][j] = 0.f;
    }
    if (n + step < a.N) load(n + step);   // in flight while this row is reduced
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VE; ++j) s[0] += j >= c.skip[i] ? x[i][j] : 0.f;
    row_sums<LPR, 2>(s, lds, turn);
    const float mean = s[0] * a.inv_d;
    s[0] = s[1] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        x[i][j] -= mean;
        const float v = j >= c.skip[i] ? x[i][j] : 0.f;
        s[0] += v;
        s[1] = fmaf(v, v, s[1]);
      }
    row_sums<LPR, 2>(s, lds, turn);
    const float lost = s[0] * a.inv_d;            // of the mean, by its rounding
    const float var = fmaxf(fmaf(-lost, lost, s[1] * a.inv_d), 0.f);
    const float r = 1.f / sqrtf(var + a.eps);
    if (live) {
      T* y = static_cast<T*>(a.y) + n * a.ldy;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (c.col[i] < 0) continue;
        float o[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) o[j] = fmaf((x[i][j] - lost) * r, w[i][j], b[i][j]);
        store_pack_once<T, VE>(y + c.col[i], narrow<T, VE>(o));
      }
      if (threadIdx.x % LPR == 0)
        *reinterpret_cast<float2*>(a.stats + 2 * n) = make_float2(mean + lost, r);
    }
  }
}

struct BackwardArgs {
  const void* dy; int64_t lddy;
  const void* x; int64_t ldx;
  const void* w;
  const float* stats;
  void* dx; int64_t lddx;
  float* parts;      // [workgroups][2][D]
  int64_t N;
  int32_t D, wtype;
  float inv_d;
  bool sums;         // whether dw or db is wanted
};

template <typename T, int VE, int LPR, int NV>
__global__ __launch_bounds__(kThreads) void norm_backward_kernel(BackwardArgs a) {
  __shared__ float lds[2][kThreads / kWave][3];
  int turn = 0;
  const Columns<VE, LPR, NV> c(a.D);
  float w[NV][VE], dw[NV][VE], db[NV][VE];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < VE; ++j) w[i][j] = 1.f, dw[i][j] = db[i][j] = 0.f;
    if (a.w && c.col[i] >= 0) load_as<VE>(a.w, a.wtype, c.col[i], w[i]);
  }
  constexpr int kRows = kThreads / LPR;
  const int64_t step = (int64_t)gridDim.x * kRows;
  const int slot = threadIdx.x / LPR;
  typename Pack<T, VE>::raw rx[NV], rg[NV];
  float2 st;
  auto load = [&](int64_t n) {
    const T* x = static_cast<const T*>(a.x) + n * a.ldx;
    const T* g = static_cast<const T*>(a.dy) + n * a.lddy;
    st = *reinterpret_cast<const float2*>(a.stats + 2 * n);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (c.col[i] >= 0) {
        rx[i] = load_pack_once<T, VE>(x + c.col[i]);
        rg[i] = load_pack_once<T, VE>(g + c.col[i]);
      }
  };
  int64_t n = (int64_t)blockIdx.x * kRows + slot;
  if (n < a.N) load(n);
  for (int64_t n0 = (int64_t)blockIdx.x * kRows; n0 < a.N; n0 += step, n += step) {
    const bool live = n < a.N;
    // the row stays as it was loaded: widened twice, it takes half the registers
    typename Pack<T, VE>::raw x[NV], g[NV];
    const float mean = live ? st.x : 0.f;
    const float r = live ? st.y : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = rx[i];
      g[i] = rg[i];
      if (!live || c.col[i] < 0) zero_raw(x[i]), zero_raw(g[i]);
    }
    if (n + step < a.N) load(n + step);
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float fx[VE], fg[VE];
      widen<T, VE>(x[i], fx);
      widen<T, VE>(g[i], fg);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const bool own = j >= c.skip[i];   // (none of a vector that does not exist)
        const float u = own ? fx[j] - mean : 0.f;
        const float v = own ? fg[j] * w[i][j] : 0.f;
        s[0] += v;
        s[1] = fmaf(v, u, s[1]);
        s[2] += u;
      }
    }
    row_sums<LPR, 3>(s, lds, turn);
    const float lost = s[2] * a.inv_d;
    const float m0 = s[0] * a.inv_d;
    const float m1 = fmaf(-lost, s[0], s[1]) * r * a.inv_d;
    if constexpr (NV > 1 && VE == 8) {   // (the compiler would keep the widened row)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t p = x[i][k], q = g[i][k];
          asm volatile("" : "+v"(p), "+v"(q));
          x[i][k] = p;
          g[i][k] = q;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float fx[VE], fg[VE], o[VE];
      widen<T, VE>(x[i], fx);
      widen<T, VE>(g[i], fg);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float xh = (fx[j] - mean - lost) * r;
        o[j] = r * (fmaf(fg[j], w[i][j], -m0) - xh * m1);
        dw[i][j] = fmaf(fg[j], xh, dw[i][j]);
        db[i][j] += fg[j];
      }
      if (live && c.col[i] >= 0)
        store_pack_once<T, VE>(static_cast<T*>(a.dx) + n * a.lddx + c.col[i], narrow<T, VE>(o));
    }
  }
  if (!a.sums) return;
  // the slots' columns meet in LDS, one vector at a time
  __shared__ float meet[kRows > 1 ? kThreads * VE : 1];
  float* out = a.parts + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
  for (int which = 0; which < 2; ++which, out += a.D) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float(&sum)[VE] = which ? db[i] : dw[i];
      if constexpr (kRows > 1) {
#pragma unroll
        for (int j = 0; j < VE; ++j) meet[j * kThreads + threadIdx.x] = sum[j];
        __syncthreads();
        if (slot == 0) {
#pragma unroll
          for (int j = 0; j < VE; ++j)
            for (int q = 1; q < kRows; ++q) sum[j] += meet[j * kThreads + q * LPR + threadIdx.x];
        }
        __syncthreads();
      }
      if (slot == 0 && c.col[i] >= 0) {
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (j >= c.skip[i]) out[c.col[i] + j] = sum[j];
      }
    }
  }
}

// Rows wider than the registers hold: a workgroup reads its row for each pass, vector
// by vector. f(column, first of its own elements) for each vector of the lane.
template <int VE, typename F>
__device__ __forceinline__ void each_vector(int32_t D, F f) {
  const int32_t vectors = (int32_t)(((int64_t)D + VE - 1) / VE);
  for (int32_t v = threadIdx.x; v < vectors; v += kThreads) f(pack_column<VE>(v, D), pack_overlap<VE>(v, D));
}
template <int VE>
__device__ __forceinline__ void load_or(const void* p, int32_t type, int32_t at, float other, float (&f)[VE]) {
  if (p) {
    load_as<VE>(p, type, at, f);
  } else {
#pragma unroll
    for (int j = 0; j < VE; ++j) f[j] = other;
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void norm_wide_forward_kernel(ForwardArgs a) {
  constexpr int VE = pack_elems<T>();
  __shared__ float lds[2][kThreads / kWave][2];
  int turn = 0;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + n * a.ldx;
    T* y = static_cast<T*>(a.y) + n * a.ldy;
    float s[2] = {0.f, 0.f};
    each_vector<VE>(a.D, [&](int32_t at, int32_t own) {
      float f[VE];
      widen<T, VE>(load_pack<T, VE>(x + at), f);
#pragma unroll
      for (int j = 0; j < VE; ++j) s[0] += j >= own ? f[j] : 0.f;
    });
    row_sums<kThreads, 2>(s, lds, turn);
    const float mean = s[0] * a.inv_d;
    s[0] = s[1] = 0.f;
    each_vector<VE>(a.D, [&](int32_t at, int32_t own) {
      float f[VE];
      widen<T, VE>(load_pack<T, VE>(x + at), f);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float v = j >= own ? f[j] - mean : 0.f;
        s[0] += v;
        s[1] = fmaf(v, v, s[1]);
      }
    });
    row_sums<kThreads, 2>(s, lds, turn);
    const float lost = s[0] * a.inv_d;
    const float r = 1.f / sqrtf(fmaxf(fmaf(-lost, lost, s[1] * a.inv_d), 0.f) + a.eps);
    each_vector<VE>(a.D, [&](int32_t at, int32_t) {
      float f[VE], w[VE], b[VE];
      widen<T, VE>(load_pack<T, VE>(x + at), f);
      load_or<VE>(a.w, a.wtype, at, 1.f, w);
      load_or<VE>(a.b, a.wtype, at, 0.f, b);
#pragma unroll
      for (int j = 0; j < VE; ++j) f[j] = fmaf((f[j] - mean - lost) * r, w[j], b[j]);
      store_pack_once<T, VE>(y + at, narrow<T, VE>(f));
    });
    if (threadIdx.x == 0) {
      a.stats[2 * n] = mean + lost;
      a.stats[2 * n + 1] = r;
    }
  }
}

// A workgroup's partial rows are in memory; a column is always its lane's.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_wide_backward_kernel(BackwardArgs a) {
  constexpr int VE = pack_elems<T>();
  __shared__ float lds[2][kThreads / kWave][3];
  int turn = 0;
  float* dw = a.parts + (int64_t)blockIdx.x * 2 * a.D;
  float* db = dw + a.D;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + n * a.ldx;
    const T* g = static_cast<const T*>(a.dy) + n * a.lddy;
    T* dx = static_cast<T*>(a.dx) + n * a.lddx;
    const float mean = a.stats[2 * n], r = a.stats[2 * n + 1];
    float s[3] = {0.f, 0.f, 0.f};
    each_vector<VE>(a.D, [&](int32_t at, int32_t own) {
      float fx[VE], fg[VE], w[VE];
      widen<T, VE>(load_pack<T, VE>(x + at), fx);
      widen<T, VE>(load_pack<T, VE>(g + at), fg);
      load_or<VE>(a.w, a.wtype, at, 1.f, w);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float u = j >= own ? fx[j] - mean : 0.f, v = j >= own ? fg[j] * w[j] : 0.f;
        s[0] += v;
        s[1] = fmaf(v, u, s[1]);
        s[2] += u;
      }
    });
    row_sums<kThreads, 3>(s, lds, turn);
    const float lost = s[2] * a.inv_d;
    const float m0 = s[0] * a.inv_d;
    const float m1 = fmaf(-lost, s[0], s[1]) * r * a.inv_d;
    each_vector<VE>(a.D, [&](int32_t at, int32_t own) {
      float fx[VE], fg[VE], w[VE], o[VE];
      widen<T, VE>(load_pack<T, VE>(x + at), fx);
      widen<T, VE>(load_pack<T, VE>(g + at), fg);
      load_or<VE>(a.w, a.wtype, at, 1.f, w);
      const bool first = n == blockIdx.x;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float xh = (fx[j] - mean - lost) * r;
        o[j] = r * (fmaf(fg[j], w[j], -m0) - xh * m1);
        fx[j] = xh;
      }
      store_pack_once<T, VE>(dx + at, narrow<T, VE>(o));
      if (!a.sums) return;
      if (own == 0) {
        float pw[VE], pb[VE];
        if (first) {
#pragma unroll
          for (int j = 0; j < VE; ++j) pw[j] = pb[j] = 0.f;
        } else {
          widen<float, VE>(load_pack<float, VE>(dw + at), pw);
          widen<float, VE>(load_pack<float, VE>(db + at), pb);
        }
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          pw[j] = fmaf(fg[j], fx[j], pw[j]);
          pb[j] += fg[j];
        }
        store_pack<float, VE>(dw + at, narrow<float, VE>(pw));
        store_pack<float, VE>(db + at, narrow<float, VE>(pb));
        return;
      }
#pragma unroll
      for (int j = 0; j < VE; ++j) {   // the row's last vector: its own columns
        if (j < own) continue;
        dw[at + j] = fmaf(fg[j], fx[j], first ? 0.f : dw[at + j]);
        db[at + j] = fg[j] + (first ? 0.f : db[at + j]);
      }
    });
  }
}

// dw[d], db[d]: the partials of column d added by 64 lanes, then by a fixed tree.
// A workgroup takes 16 columns at a time: 64-byte pieces of the partial rows, and enough
// workgroups for the narrowest rows.
constexpr int64_t kJoinBlocks = 1 << 16;   // at most: a launch has less than 2^32 threads
__global__ __launch_bounds__(kThreads) void norm_join_kernel(const float* parts, int32_t P,
                                                             int32_t D, int32_t wtype, void* dw,
                                                             void* db) {
  __shared__ float meet[64][17];
  const int32_t col = threadIdx.x % 16, lane = threadIdx.x / 16;
  const int64_t columns = 2 * (int64_t)D;   // dw's, then db's
  for (int64_t i0 = (int64_t)blockIdx.x * 16; i0 < columns; i0 += (int64_t)gridDim.x * 16) {
    const int64_t i = i0 + col;
    float s = 0.f;
    if (i < columns) {
#pragma unroll 4
      for (int32_t p = lane; p < P; p += 64) s += parts[(int64_t)p * columns + i];
    }
    meet[lane][col] = s;
    __syncthreads();
    for (int half = 32; half > 0; half /= 2) {
      if (lane < half) meet[lane][col] += meet[lane + half][col];
      __syncthreads();
    }
    void* out = i < D ? dw : db;
    if (lane == 0 && i < columns && out) {
      const int64_t d = i < D ? i : i - D;
      const float v = meet[0][col];   // (the next columns' are written to it by this lane)
      if (wtype == TBE_F32) static_cast<float*>(out)[d] = v;
      else if (wtype == TBE_F16) static_cast<f16_t*>(out)[d] = round_to<f16_t>(v);
      else static_cast<bf16_t*>(out)[d] = round_to<bf16_t>(v);
    }
  }
}

// Calls f(VE, LPR, NV) with the shape for rows of D columns: one vector a lane as long
// as 1024 lanes hold the row. (Two vectors on half the lanes hold fewer waves on a CU:
// 16384 rows of 4096 bf16, forward and backward, 131 us against 126.)
template <typename T, typename F>
bool with_shape(int32_t D, F f) {
  constexpr int VE = pack_elems<T>();
  const int64_t v = ((int64_t)D + VE - 1) / VE;
  auto shape = [&](auto ve, auto lpr, auto nv) { f(ve, lpr, nv); };
#define TBE_SHAPE(VE, LPR, NV)                                                           \
  shape(std::integral_constant<int, VE>{}, std::integral_constant<int, LPR>{},           \
        std::integral_constant<int, NV>{})
  if (D < VE) TBE_SHAPE(1, 16, 1);
  else if (v <= 16) TBE_SHAPE(VE, 16, 1);
  else if (v <= 32) TBE_SHAPE(VE, 32, 1);
  else if (v <= 64) TBE_SHAPE(VE, 64, 1);
  else if (v <= 128) TBE_SHAPE(VE, 128, 1);
  else if (v <= 256) TBE_SHAPE(VE, 256, 1);
  else if (v <= 512) TBE_SHAPE(VE, 512, 1);
  else if (v <= 1024) TBE_SHAPE(VE, 1024, 1);
  else if (v <= kMaxVectors) TBE_SHAPE(VE, 1024, 2);
  else return false;
#undef TBE_SHAPE
  return true;
}

}  // namespace

int32_t norm_partials(const tbe_norm_desc& d) {
  // one per workgroup: no more than rows, and of wide rows no more than 1 GiB together
  const int64_t room = (int64_t(1) << 27) / d.D;
  const int64_t p = std::min<int64_t>(kMaxParts, std::min<int64_t>(d.N, room < 1 ? 1 : room));
  return p < 1 ? 1 : (int32_t)p;
}

hipError_t launch_norm_forward(const tbe_norm_desc& d, const void* x, int64_t ldx, const void* w,
                               const void* b, void* y, int64_t ldy, float* stats, hipStream_t s) {
  const ForwardArgs a = {x, ldx, w, b, y, ldy, stats, d.N, d.D, (int32_t)d.wdtype, d.eps,
                         (float)(1.0 / d.D)};
  return with_type(d.dtype, [&](auto t) {
    using T = decltype(t);
    const bool done = with_shape<T>(d.D, [&](auto ve, auto lpr, auto nv) {
      constexpr int LPR = decltype(lpr)::value;
      constexpr int THREADS = LPR > 256 ? LPR : 256;
      const int64_t rows = THREADS / LPR;
      // as many as find room at once, eight waves on a SIMD
      const int64_t blocks = std::min<int64_t>((d.N + rows - 1) / rows, 2048 / (THREADS / 256));
      norm_forward_kernel<T, decltype(ve)::value, LPR, decltype(nv)::value, THREADS>
          <<<(unsigned)blocks, THREADS, 0, s>>>(a);
    });
    if (!done)
      norm_wide_forward_kernel<T><<<(unsigned)std::min<int64_t>(d.N, 1024), kThreads, 0, s>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_norm_backward(const tbe_norm_desc& d, const void* dy, int64_t lddy, const void* x,
                                int64_t ldx, const void* w, const float* stats, void* dx,
                                int64_t lddx, void* dw, void* db, float* parts, hipStream_t s) {
  const bool sums = dw || db;
  const BackwardArgs a = {dy, lddy, x, ldx, w, stats, dx, lddx, parts, d.N, d.D,
                          (int32_t)d.wdtype, (float)(1.0 / d.D), sums};
  int32_t P = 0;
  hipError_t e = hipSuccess;
  if (d.N > 0) {
    e = with_type(d.dtype, [&](auto t) {
      using T = decltype(t);
      const bool done = with_shape<T>(d.D, [&](auto ve, auto lpr, auto nv) {
        constexpr int LPR = decltype(lpr)::value;
        const int64_t rows = kThreads / LPR;
        P = (int32_t)std::min<int64_t>(norm_partials(d), (d.N + rows - 1) / rows);
        norm_backward_kernel<T, decltype(ve)::value, LPR, decltype(nv)::value>
            <<<(unsigned)P, kThreads, 0, s>>>(a);
      });
      if (!done) {
        P = norm_partials(d);
        norm_wide_backward_kernel<T><<<(unsigned)P, kThreads, 0, s>>>(a);
      }
      return hipGetLastError();
    });
  }
  if (e != hipSuccess || !sums) return e;
  const int64_t joins = std::min<int64_t>((2 * (int64_t)d.D + 15) / 16, kJoinBlocks);
  norm_join_kernel<<<(unsigned)joins, kThreads, 0, s>>>(parts, P, d.D, (int32_t)d.wdtype,
                                                        dw, db);
  return hipGetLastError();
}

}  // namespace tbe
