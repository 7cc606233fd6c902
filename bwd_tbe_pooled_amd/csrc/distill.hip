// Distillation loss of a student's logits against a teacher's top logits, and
// its gradient:
//   p = softmax(t / tau) over the teacher's entries, q = softmax(x / tau) over
//   the vocabulary, loss = tau^2 sum p (log p - log q at their places),
//   gx = gl tau (q - p scattered to its places).
//
// One pass over the logits keeps a running maximum and sum per lane (s is
// rescaled when the maximum grows); only differences x - max are scaled, so
// rows of the type's lowest value stay exact. A row without a teacher is not
// read. The gradient's dense part writes c * q everywhere; after a barrier
// the lanes that hold the teacher's entries overwrite those places with
// c * (q - p), where p is the sum over equal places.
#include "lm.h"
#include "lm_device.h"

namespace tbe {

namespace {

constexpr int kTeacherMax = 1024;

// Running maximum and sum of exp(a (x - maximum)) in base 2.
struct MaxSum {
  float m, s;
};

// The shift of a maximum that may be -inf (nothing seen, or only -inf): with
// 0 in its place exp2(a (x - 0)) of such logits is 0.
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ float exp2_scaled(float x, float m, float a) {
  return __builtin_amdgcn_exp2f((x - m) * a);
}

template <int VE>
__device__ __forceinline__ void add_logits(MaxSum& r, const float (&x)[VE], float a) {
  float m = r.m;
#pragma unroll
  for (int e = 0; e < VE; ++e) m = fmaxf(m, x[e]);
  const float sh = shift_of(m);
  float s = r.s * exp2_scaled(r.m, sh, a);
#pragma unroll
  for (int e = 0; e < VE; ++e) s += exp2_scaled(x[e], sh, a);
  r.m = m;
  r.s = s;
}

__device__ __forceinline__ MaxSum merge(MaxSum p, MaxSum q, float a) {
  MaxSum r;
  r.m = fmaxf(p.m, q.m);
  const float sh = shift_of(r.m);
  r.s = p.s * exp2_scaled(p.m, sh, a) + q.s * exp2_scaled(q.m, sh, a);
  return r;
}

__device__ __forceinline__ MaxSum wave_merge(MaxSum r, float a) {
  const float m = wave_max(r.m);
  const float s = wave_sum(r.s * exp2_scaled(r.m, shift_of(m), a));
  return MaxSum{m, s};
}

// The teacher's side of one row in LDS.
struct Teacher {
  int32_t id[kTeacherMax];   // place, or -1
  float p[kTeacherMax];      // probability
};

template <int BS>
struct Block {
  static constexpr int kWaves = BS / kWave;
  float red[4][kWaves];

  // Every thread receives the result; one barrier before the first use of
  // `slot` again is the caller's.
  __device__ __forceinline__ float sum(float x, int slot) {
    x = wave_sum(x);
    if (lane_id() == 0) red[slot][threadIdx.x / kWave] = x;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) t += red[slot][w];
    return t;
  }
  __device__ __forceinline__ float max(float x, int slot) {
    x = wave_max(x);
    if (lane_id() == 0) red[slot][threadIdx.x / kWave] = x;
    __syncthreads();
    float t = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) t = fmaxf(t, red[slot][w]);
    return t;
  }
};

struct Args {
  const void *ids, *t;
  int32_t idx64, K;
  int64_t N, V;
  float tau, a;  // a = log2(e) / tau
};

// Loads a row's teacher. Returns whether any entry takes part; then id, p and
// (per thread, for the entries tid + i BS) logp = log p. Two barriers at
// least; the LDS is valid in every thread afterwards.
template <typename TT, int BS>
__device__ __forceinline__ bool load_teacher(const Args& g, int64_t n, Teacher& T, Block<BS>& B,
                                             float (&logp)[(kTeacherMax + BS - 1) / BS]) {
  constexpr int KP = (kTeacherMax + BS - 1) / BS;
  float t[KP];
  bool ok[KP];
  float m = -INFINITY;
  bool any = false;
#pragma unroll
  for (int i = 0; i < KP; ++i) {
    const int32_t k = threadIdx.x + i * BS;
    ok[i] = false;
    t[i] = 0.f;
    if (k < g.K) {
      const int64_t id = load_id(g.ids, g.idx64, n * g.K + k);
      t[i] = to_float(static_cast<const TT*>(g.t)[n * g.K + k]);
      ok[i] = id >= 0 && id < g.V && t[i] != -INFINITY;
      T.id[k] = ok[i] ? (int32_t)id : -1;
      if (ok[i]) m = fmaxf(m, t[i]);
      any |= ok[i];
    }
  }
  // a NaN drops out of the maximum, so what takes part is counted apart
  any = __syncthreads_or(any);
  if (!any) return false;
  m = B.max(m, 0);
  float s = 0.f;
  const float inv_tau = 1.f / g.tau;
#pragma unroll
  for (int i = 0; i < KP; ++i)
    if (ok[i]) s += expf((t[i] - m) * inv_tau);
  s = B.sum(s, 1);
  const float logs = logf(s);
#pragma unroll
  for (int i = 0; i < KP; ++i) {
    const int32_t k = threadIdx.x + i * BS;
    logp[i] = (t[i] - m) * inv_tau - logs;
    if (k < g.K) T.p[k] = ok[i] ? expf(logp[i]) : 0.f;
  }
  __syncthreads();
  return true;
}

// Sum of p over the entries with the place of entry k, in the entries' order.
__device__ __forceinline__ float p_at(const Teacher& T, int32_t K, int32_t id) {
  float p = 0.f;
  for (int32_t j = 0; j < K; ++j) p += T.id[j] == id ? T.p[j] : 0.f;
  return p;
}

// Maximum and sum over a row by the whole workgroup.
template <typename XT, int BS, int U>
__device__ __forceinline__ MaxSum row_stats(const XT* __restrict__ x, int64_t V, float a,
                                            Block<BS>& B) {
  constexpr int VE = pack_elems<XT>();
  using R = typename Pack<XT, VE>::raw;
  const int64_t nv = V / VE;
  MaxSum r{-INFINITY, 0.f};
  int64_t i = threadIdx.x;
  for (; i + (U - 1) * BS < nv; i += U * BS) {
    R v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = load_pack<XT, VE>(x + (i + u * BS) * VE);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[VE];
      widen<XT, VE>(v[u], f);
      add_logits<VE>(r, f, a);
    }
  }
  for (; i < nv; i += BS) {
    float f[VE];
    widen<XT, VE>(load_pack<XT, VE>(x + i * VE), f);
    add_logits<VE>(r, f, a);
  }
  const int64_t rest = nv * VE + threadIdx.x;
  if (rest < V) {
    const float f[1] = {to_float(x[rest])};
    add_logits<1>(r, f, a);
  }
  r = wave_merge(r, a);
  if (lane_id() == 0) {
    B.red[2][threadIdx.x / kWave] = r.m;
    B.red[3][threadIdx.x / kWave] = r.s;
  }
  __syncthreads();
  r = MaxSum{B.red[2][0], B.red[3][0]};
#pragma unroll
  for (int w = 1; w < Block<BS>::kWaves; ++w) r = merge(r, MaxSum{B.red[2][w], B.red[3][w]}, a);
  return r;
}

// The row's loss, in every thread; xk: the logits at the entries' places.
template <int BS>
__device__ __forceinline__ float row_loss(const Args& g, const Teacher& T, Block<BS>& B, MaxSum r,
                                          const float (&logp)[(kTeacherMax + BS - 1) / BS],
                                          const float (&xk)[(kTeacherMax + BS - 1) / BS]) {
  constexpr int KP = (kTeacherMax + BS - 1) / BS;
  const float inv_tau = 1.f / g.tau;
  const float logs = logf(r.s);
  float loss = 0.f;
#pragma unroll
  for (int i = 0; i < KP; ++i) {
    const int32_t k = threadIdx.x + i * BS;
    if (k >= g.K) continue;
    const float p = T.p[k];
    if (p != 0.f) loss += p * (logp[i] - ((xk[i] - r.m) * inv_tau - logs));
  }
  return g.tau * g.tau * B.sum(loss, 0);
}

template <typename XT, int BS>
__device__ __forceinline__ void load_places(const XT* __restrict__ x, const Teacher& T, int32_t K,
                                            float (&xk)[(kTeacherMax + BS - 1) / BS]) {
#pragma unroll
  for (int i = 0; i < (kTeacherMax + BS - 1) / BS; ++i) {
    const int32_t k = threadIdx.x + i * BS;
    xk[i] = k < K && T.id[k] >= 0 ? to_float(x[T.id[k]]) : 0.f;
  }
}

template <typename XT, typename TT, int BS>
__global__ __launch_bounds__(BS) void distill_forward_kernel(const XT* __restrict__ x, int64_t ldx,
                                                             Args g, float* __restrict__ loss,
                                                             float* __restrict__ stats) {
  __shared__ Teacher T;
  __shared__ Block<BS> B;
  for (int64_t n = blockIdx.x; n < g.N; n += gridDim.x) {
    float logp[(kTeacherMax + BS - 1) / BS], xk[(kTeacherMax + BS - 1) / BS];
    float l = 0.f;
    MaxSum r{0.f, 1.f};
    __syncthreads();  // the row before is done with the LDS
    if (load_teacher<TT, BS>(g, n, T, B, logp)) {
      const XT* row = x + n * ldx;
      load_places<XT, BS>(row, T, g.K, xk);
      r = row_stats<XT, BS, 4>(row, g.V, g.a, B);
      l = row_loss<BS>(g, T, B, r, logp, xk);
    }
    if (threadIdx.x == 0) {
      loss[n] = l;
      stats[2 * n] = r.m;
      stats[2 * n + 1] = r.s;
    }
  }
}

// gx[v] = c q[v] for the vectors [i0, i1) of a row and, if `tail`, the
// elements after its whole vectors. x may be gx.
template <typename XT, int BS, int U>
__device__ __forceinline__ void write_gradient(const XT* x, XT* gx, int64_t V, int64_t i0,
                                               int64_t i1, bool tail, float m, float c, float a) {
  constexpr int VE = pack_elems<XT>();
  using R = typename Pack<XT, VE>::raw;
  int64_t i = i0 + threadIdx.x;
  for (; i + (U - 1) * BS < i1; i += U * BS) {
    R v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = load_pack<XT, VE>(x + (i + u * BS) * VE);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[VE];
      widen<XT, VE>(v[u], f);
#pragma unroll
      for (int e = 0; e < VE; ++e) f[e] = c * exp2_scaled(f[e], m, a);
      store_pack_once<XT, VE>(gx + (i + u * BS) * VE, narrow<XT, VE>(f));
    }
  }
  for (; i < i1; i += BS) {
    float f[VE];
    widen<XT, VE>(load_pack<XT, VE>(x + i * VE), f);
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = c * exp2_scaled(f[e], m, a);
    store_pack_once<XT, VE>(gx + i * VE, narrow<XT, VE>(f));
  }
  const int64_t rest = V / VE * VE + threadIdx.x;
  if (tail && rest < V) gx[rest] = round_to<XT>(c * exp2_scaled(to_float(x[rest]), m, a));
}

template <typename XT, int BS>
__device__ __forceinline__ void write_zeros(XT* gx, int64_t V, int64_t i0, int64_t i1, bool tail) {
  constexpr int VE = pack_elems<XT>();
  typename Pack<XT, VE>::raw z;
  zero_raw(z);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += BS) store_pack_once<XT, VE>(gx + i * VE, z);
  const int64_t rest = V / VE * VE + threadIdx.x;
  if (tail && rest < V) gx[rest] = round_to<XT>(0.f);
}

// The teacher's places in [v0, v1) after the dense part (a barrier between).
template <typename XT, int BS>
__device__ __forceinline__ void write_places(XT* gx, const Teacher& T, int32_t K, int64_t v0,
                                             int64_t v1, float m, float c, float inv_s_c, float a,
                                             const float (&xk)[(kTeacherMax + BS - 1) / BS]) {
#pragma unroll
  for (int i = 0; i < (kTeacherMax + BS - 1) / BS; ++i) {
    const int32_t k = threadIdx.x + i * BS;
    if (k >= K) continue;
    const int32_t id = T.id[k];
    if (id < v0 || id >= v1 || id < 0) continue;
    gx[id] = round_to<XT>(inv_s_c * exp2_scaled(xk[i], m, a) - c * p_at(T, K, id));
  }
}

constexpr int kPieceVectors = 2048;  // vectors of a row one workgroup of the backward takes

template <typename XT, typename TT, int BS>
__global__ __launch_bounds__(BS) void distill_backward_kernel(const XT* x, int64_t ldx, Args g,
                                                              const float* __restrict__ stats,
                                                              const float* __restrict__ gl, XT* gx,
                                                              int64_t ldgx, int32_t pieces) {
  __shared__ Teacher T;
  __shared__ Block<BS> B;
  constexpr int VE = pack_elems<XT>();
  const int64_t nv = g.V / VE;
  for (int64_t w = blockIdx.x; w < g.N * pieces; w += gridDim.x) {
    const int64_t n = w / pieces;
    const int32_t piece = (int32_t)(w % pieces);
    const int64_t i0 = (int64_t)piece * kPieceVectors;
    const bool last = piece == pieces - 1;
    const int64_t i1 = last ? nv : i0 + kPieceVectors;
    const int64_t v1 = last ? g.V : i1 * VE;
    const XT* row = x + n * ldx;
    XT* to = gx + n * ldgx;
    float logp[(kTeacherMax + BS - 1) / BS], xk[(kTeacherMax + BS - 1) / BS];
    __syncthreads();  // the piece before is done with the LDS
    if (!load_teacher<TT, BS>(g, n, T, B, logp)) {
      write_zeros<XT, BS>(to, g.V, i0, i1, last);
      continue;
    }
#pragma unroll
    for (int i = 0; i < (kTeacherMax + BS - 1) / BS; ++i) {
      const int32_t k = threadIdx.x + i * BS;
      xk[i] = k < g.K && T.id[k] >= i0 * VE && T.id[k] < v1 ? to_float(row[T.id[k]]) : 0.f;
    }
    __syncthreads();  // gx may be x: the places are read before they are written
    const float m = stats[2 * n];
    const float c = gl[n] * g.tau;
    const float cs = c / stats[2 * n + 1];
    write_gradient<XT, BS, 4>(row, to, g.V, i0, i1, last, m, cs, g.a);
    __syncthreads();
    write_places<XT, BS>(to, T, g.K, i0 * VE, v1, m, c, cs, g.a, xk);
  }
}

// Both passes over a row by one workgroup; the second reads the row again.
template <typename XT, typename TT, int BS>
__global__ __launch_bounds__(BS) void distill_step_kernel(const XT* x, int64_t ldx, Args g,
                                                          const float* __restrict__ gl,
                                                          float* __restrict__ loss, XT* gx,
                                                          int64_t ldgx) {
  __shared__ Teacher T;
  __shared__ Block<BS> B;
  constexpr int VE = pack_elems<XT>();
  const int64_t nv = g.V / VE;
  for (int64_t n = blockIdx.x; n < g.N; n += gridDim.x) {
    const XT* row = x + n * ldx;
    XT* to = gx + n * ldgx;
    float logp[(kTeacherMax + BS - 1) / BS], xk[(kTeacherMax + BS - 1) / BS];
    __syncthreads();
    if (!load_teacher<TT, BS>(g, n, T, B, logp)) {
      if (threadIdx.x == 0) loss[n] = 0.f;
      write_zeros<XT, BS>(to, g.V, 0, nv, true);
      continue;
    }
    load_places<XT, BS>(row, T, g.K, xk);
    const MaxSum r = row_stats<XT, BS, 4>(row, g.V, g.a, B);
    const float l = row_loss<BS>(g, T, B, r, logp, xk);
    if (threadIdx.x == 0) loss[n] = l;
    const float c = gl[n] * g.tau;
    const float cs = c / r.s;
    write_gradient<XT, BS, 4>(row, to, g.V, 0, nv, true, r.m, cs, g.a);
    __syncthreads();
    write_places<XT, BS>(to, T, g.K, 0, g.V, r.m, c, cs, g.a, xk);
  }
}

Args make_args(const tbe_distill_desc& d, const void* ids, const void* t) {
  Args g;
  g.ids = ids;
  g.t = t;
  g.idx64 = d.idx64;
  g.K = d.K;
  g.N = d.N;
  g.V = d.V;
  g.tau = d.temperature;
  g.a = (float)(1.4426950408889634 / (double)d.temperature);
  return g;
}

unsigned grid_for(int64_t n) { return (unsigned)(n < (1 << 20) ? n : (1 << 20)); }

}  // namespace

size_t distill_workspace(const tbe_distill_desc&) { return 256; }

hipError_t launch_distill_forward(const tbe_distill_desc& d, const void* x, int64_t ldx,
                                  const void* ids, const void* t, float* loss, float* stats,
                                  void*, hipStream_t s) {
  const Args g = make_args(d, ids, t);
  return with_type(d.dtype, [&](auto xt) {
    using XT = decltype(xt);
    return with_type(d.tdtype, [&](auto tt) {
      using TT = decltype(tt);
      constexpr int BS = 1024;
      hipLaunchKernelGGL((distill_forward_kernel<XT, TT, BS>), dim3(grid_for(d.N)), dim3(BS), 0, s,
                         static_cast<const XT*>(x), ldx, g, loss, stats);
      return hipGetLastError();
    });
  });
}

hipError_t launch_distill_backward(const tbe_distill_desc& d, const void* x, int64_t ldx,
                                   const void* ids, const void* t, const float* stats,
                                   const float* gl, void* gx, int64_t ldgx, hipStream_t s) {
  const Args g = make_args(d, ids, t);
  return with_type(d.dtype, [&](auto xt) {
    using XT = decltype(xt);
    return with_type(d.tdtype, [&](auto tt) {
      using TT = decltype(tt);
      constexpr int BS = 256;
      const int64_t per = (int64_t)kPieceVectors * pack_elems<XT>();
      const int32_t pieces = (int32_t)((d.V + per - 1) / per);
      hipLaunchKernelGGL((distill_backward_kernel<XT, TT, BS>), dim3(grid_for(d.N * pieces)),
                         dim3(BS), 0, s, static_cast<const XT*>(x), ldx, g, stats, gl,
                         static_cast<XT*>(gx), ldgx, pieces);
      return hipGetLastError();
    });
  });
}

hipError_t launch_distill_step(const tbe_distill_desc& d, const void* x, int64_t ldx,
                               const void* ids, const void* t, const float* gl, float* loss,
                               void* gx, int64_t ldgx, void*, hipStream_t s) {
  const Args g = make_args(d, ids, t);
  return with_type(d.dtype, [&](auto xt) {
    using XT = decltype(xt);
    return with_type(d.tdtype, [&](auto tt) {
      using TT = decltype(tt);
      constexpr int BS = 1024;
      hipLaunchKernelGGL((distill_step_kernel<XT, TT, BS>), dim3(grid_for(d.N)), dim3(BS), 0, s,
                         static_cast<const XT*>(x), ldx, g, gl, loss, static_cast<XT*>(gx), ldgx);
      return hipGetLastError();
    });
  });
}

}  // namespace tbe
