// Distillation loss of a student's logits against a teacher's top logits, and
// its gradient:
//   p = softmax(t / tau) over the teacher's entries, q = softmax(x / tau) over
//   the vocabulary, loss = tau^2 sum p (log p - log q at their places),
//   gx = gl tau (q - p scattered to its places).
//
// Exponentials are in base 2 with a = log2(e) / tau: q[v] = 2^(a x - c) / s with
// the shift c = round(a max x) and s the sum of these powers. a x - c is one
// fma, and whatever c was rounded to divides out, as s has the same c. Beyond
// |a max x| = 2^23 that rounding could itself overflow the power: such "far"
// rows (the type's lowest value everywhere, say) are read again, element by
// element, with the power of (x - max x) a.
//
// A row without a teacher is not read. The gradient's dense part writes gl tau
// q everywhere; after a barrier the threads that hold the teacher's entries
// write gl tau (q - p) to their places, with p the sum over equal places.
#include "lm.h"
#include "lm_device.h"

#include <type_traits>

namespace tbe {

namespace {

// |a max x| above which a thread's own sum counts for nothing, and above which
// a row is far: so a far thread is 2^23 below the maximum of a row that is not.
constexpr float kFar = 16777216.f;
constexpr float kFarRow = kFar / 2;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_of(float x) { return __builtin_amdgcn_logf(x); }

// The powers' argument for a maximum m (that may be -inf: nothing seen, or only
// -inf, whose powers are 0 with any finite shift).
struct Shift {
  float m, c;
  bool far;
  __device__ __forceinline__ Shift(float max, float a, float limit = kFar) {
    // c is the rounded product wherever it is used: no fma takes its factors
#pragma clang fp contract(off)
    m = max == -INFINITY ? 0.f : max;
    c = m * a;
    far = !(fabsf(c) <= limit);
  }
  __device__ __forceinline__ float of(float x, float a) const {
    return far ? (x - m) * a : fmaf(x, a, -c);
  }
  // The power of the maximum: 1 but for c's rounding, by which every power of
  // the row is off. (The statistics are given without it: they are the sum of
  // exp((x - max) / tau) for any reader, not for this shift alone.)
  __device__ __forceinline__ float of_max(float a) const {
    return far ? 1.f : exp2_of(fmaf(m, a, -c));
  }
};

// Factor from the powers' sum with maximum m to that with the maximum of `to`.
__device__ __forceinline__ float rescale(float m, const Shift& to, float a) {
  const Shift from(m, a);
  if (m == -INFINITY) return 0.f;
  return exp2_of(from.far || to.far ? (m - to.m) * a : from.c - to.c);
}

struct Args {
  const void *ids, *t;
  int32_t idx64, K;
  tbe_dtype tdtype;
  int64_t N, V;
  float tau, a;  // a = log2(e) / tau
};

// The teacher's entries k0 + q step (q < KU) of row n below K: their places (-1
// if they take no part) and logits. All loads are in flight together; the
// types are looked at once, not per entry.
template <int KU>
__device__ __forceinline__ void load_entries(const Args& g, int64_t n, int32_t k0, int32_t step,
                                             int32_t (&id)[KU], float (&t)[KU]) {
  const int64_t row = n * g.K;
  uint32_t bits[KU];
  int64_t v[KU];
  if (g.tdtype == TBE_F32) {
    const uint32_t* p = static_cast<const uint32_t*>(g.t) + row;
#pragma unroll
    for (int q = 0; q < KU; ++q) bits[q] = k0 + q * step < g.K ? p[k0 + q * step] : 0;
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(g.t) + row;
#pragma unroll
    for (int q = 0; q < KU; ++q) bits[q] = k0 + q * step < g.K ? p[k0 + q * step] : 0;
  }
  if (g.idx64) {
    const int64_t* p = static_cast<const int64_t*>(g.ids) + row;
#pragma unroll
    for (int q = 0; q < KU; ++q) v[q] = k0 + q * step < g.K ? p[k0 + q * step] : -1;
  } else {
    const int32_t* p = static_cast<const int32_t*>(g.ids) + row;
#pragma unroll
    for (int q = 0; q < KU; ++q) v[q] = k0 + q * step < g.K ? p[k0 + q * step] : -1;
  }
#pragma unroll
  for (int q = 0; q < KU; ++q) {
    t[q] = __uint_as_float(g.tdtype == TBE_BF16 ? bits[q] << 16 : bits[q]);
    if (g.tdtype == TBE_F16) t[q] = to_float(f16_t{(uint16_t)bits[q]});
    id[q] = v[q] >= 0 && v[q] < g.V && t[q] != -INFINITY ? (int32_t)v[q] : -1;
  }
}

// Whether any entry of the row takes part, found by each wave for itself.
__device__ __forceinline__ bool has_teacher(const Args& g, int64_t n) {
  for (int32_t k0 = 0; k0 < g.K; k0 += kWave) {
    int32_t id[1];
    float t[1];
    load_entries<1>(g, n, k0 + lane_id(), 0, id, t);
    if (__ballot(id[0] >= 0)) return true;
  }
  return false;
}

// The teacher's entries of one row in LDS, K rounded up to whole int4s each.
struct Teacher {
  int32_t* id;
  float *p, *x;  // probability (its logit at first), student's logit
  __device__ __forceinline__ Teacher(void* lds, int32_t K) {
    const int32_t k4 = (K + 3) / 4 * 4;
    id = static_cast<int32_t*>(lds);
    p = reinterpret_cast<float*>(id + k4);
    x = p + k4;
  }
  static size_t bytes(int32_t K) { return 3 * sizeof(int32_t) * (size_t)((K + 3) / 4 * 4); }

  // Sum of p over the entries with this place, in the entries' order. (The
  // entries past K that make whole int4s have the place -1.) All K entries are
  // looked at for each of K: 1001 x 50021 f16 rows take 44 us a step at K = 128
  // and 127 at K = 1024, and forward and backward 67 and 234, as the backward
  // also reads the list in each piece of a row.
  __device__ __forceinline__ float p_at(int32_t K, int32_t place) const {
    float s = 0.f;
#pragma unroll 2
    for (int32_t j = 0; j < K; j += 4) {
      const int4 i = *reinterpret_cast<const int4*>(id + j);
      const float4 f = *reinterpret_cast<const float4*>(p + j);
      s += i.x == place ? f.x : 0.f;
      s += i.y == place ? f.y : 0.f;
      s += i.z == place ? f.z : 0.f;
      s += i.w == place ? f.w : 0.f;
    }
    return s;
  }
};

template <int BS>
__device__ __forceinline__ void group_sync() {
  if constexpr (BS == kWave) wave_lds_sync(); else __syncthreads();
}

// A thread's part of a row: the vectors gt + BS i (i < NV) below `left` from
// some base. All NV are loaded, those past the end as the last one again (from
// the caches), and left out of sums and stores: a load under a condition would
// cost the compiler a second set of the registers. What is one address for the
// wave and what is the lane's own stays apart, so that NV vectors take no NV
// addresses. NV is 0 for rows without a whole vector.
template <typename XT, int BS, int NV>
struct Part {
  static constexpr int VE = pack_elems<XT>();
  using Raw = typename Pack<XT, VE>::raw;
  Raw v[NV > 0 ? NV : 1];
  int32_t left;
  uint32_t last;  // byte offset of the last vector
  int used;       // of the NV, how many any lane of the wave has

  __device__ __forceinline__ void shape(int64_t vectors, int wave) {
    left = vectors < BS * NV ? (int32_t)vectors : BS * NV;
    last = left > 0 ? (uint32_t)(left - 1) * 16u : 0u;
    const int32_t l = left - wave * kWave;
    used = l <= 0 ? 0 : (l + BS - 1) / BS;
  }
  static __device__ __forceinline__ uint32_t offset(int i, uint32_t gt) {
    uint32_t o = gt * 16u;
    asm volatile("" : "+v"(o));  // one offset and an addition, not NV offsets kept
    return o + (uint32_t)(i * BS) * 16u;
  }
  // Whether the lane has vector i, asked where it is needed: as masks kept for
  // all vectors it took the scalar registers of the loop over rows.
  template <bool FULL>
  __device__ __forceinline__ bool below_end(int i, uint32_t gt) const {
    if constexpr (FULL) return true;
    int32_t o = (int32_t)gt;
    asm volatile("" : "+v"(o));
    return o + i * BS < left;
  }
  __device__ __forceinline__ bool full() const { return left == BS * NV; }

  template <bool ONCE, bool FULL>
  __device__ __forceinline__ void load_all(const XT* base, uint32_t gt) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t o = offset(i, gt);
      if (!FULL) o = o < last ? o : last;
      const XT* p = reinterpret_cast<const XT*>(reinterpret_cast<const char*>(base) + o);
      v[i] = ONCE ? load_pack_once<XT, VE>(p) : load_pack<XT, VE>(p);
    }
  }
  template <bool ONCE>
  __device__ __forceinline__ void load(const XT* base, uint32_t gt) {
    if (full()) load_all<ONCE, true>(base, gt);
    else load_all<ONCE, false>(base, gt);
  }

  // For the compiler: the vectors may have changed. Without it the elements
  // widened for the maximum would be kept for the sum, in twice the registers.
  __device__ __forceinline__ void touch() {
#pragma unroll
    for (int i = 0; i < NV; ++i) asm volatile("" : "+v"(v[i]));
  }

  // The largest of m and the elements. As whole numbers the patterns of floats
  // have the floats' order unless all are negative (and a positive NaN above
  // all): half an instruction per element, against one and a half to widen it
  // and take the float maximum.
  __device__ __forceinline__ float max(float m) const {
    typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
    int32_t top;
    if constexpr (sizeof(XT) == 4) {
      top = INT32_MIN;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i < used) {
          const int32_t p = (int32_t)v[i][0] > (int32_t)v[i][1] ? (int32_t)v[i][0] : (int32_t)v[i][1];
          const int32_t q = (int32_t)v[i][2] > (int32_t)v[i][3] ? (int32_t)v[i][2] : (int32_t)v[i][3];
          const int32_t r = p > q ? p : q;
          top = r > top ? r : top;
        }
    } else {
      i16x2 t = {INT16_MIN, INT16_MIN};
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i < used) {
          const i16x2 p = __builtin_elementwise_max(__builtin_bit_cast(i16x2, (uint32_t)v[i][0]),
                                                    __builtin_bit_cast(i16x2, (uint32_t)v[i][1]));
          const i16x2 q = __builtin_elementwise_max(__builtin_bit_cast(i16x2, (uint32_t)v[i][2]),
                                                    __builtin_bit_cast(i16x2, (uint32_t)v[i][3]));
          t = __builtin_elementwise_max(t, __builtin_elementwise_max(p, q));
        }
      top = t.x > t.y ? t.x : t.y;
    }
    if (__builtin_expect(!__any(top < 0), 1)) {
      if constexpr (sizeof(XT) == 4) return fmaxf(m, __int_as_float(top));
      else return fmaxf(m, to_float(XT{(uint16_t)top}));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i < used) {
        float f[VE];
        widen<XT, VE>(v[i], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) m = fmaxf(m, f[e]);
      }
    return m;
  }

  // Sum of the powers.
  template <bool FULL>
  __device__ __forceinline__ float sum_all(const Shift& sh, uint32_t gt, float s, float a) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (FULL || i < used) {
        float f[VE];
        widen<XT, VE>(v[i], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = exp2_of(fmaf(f[e], a, -sh.c));
        float t = 0.f;
        if constexpr (VE == 8) t = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        else t = (f[0] + f[1]) + (f[2] + f[3]);
        s += below_end<FULL>(i, gt) ? t : 0.f;
      }
    return s;
  }
  // That and the power of `rest`. Of a far maximum only whether there is a NaN:
  // the sum counts for nothing beside a near one, and is formed again if there
  // is none.
  __device__ __forceinline__ float sum(const Shift& sh, uint32_t gt, float rest, float a) {
    touch();
    float s = exp2_of(fmaf(rest, a, -sh.c));
    s = full() ? sum_all<true>(sh, gt, s, a) : sum_all<false>(sh, gt, s, a);
    if (__builtin_expect(__any(sh.far), 0)) {
      touch();
      bool n = rest != rest;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i < used) {
          float f[VE];
          widen<XT, VE>(v[i], f);
#pragma unroll
          for (int e = 0; e < VE; ++e) n |= f[e] != f[e];
        }
      if (sh.far) return n ? NAN : 1.f;
    }
    return s;
  }

  // The gradient cs 2^(a x - c).
  template <bool FULL>
  __device__ __forceinline__ void store_all(XT* base, uint32_t gt, float a, float c, float cs) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (FULL || i < used) {
        float f[VE];
        widen<XT, VE>(v[i], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = cs * exp2_of(fmaf(f[e], a, -c));
        const Raw r = narrow<XT, VE>(f);
        if (below_end<FULL>(i, gt))
          store_pack_once<XT, VE>(
              reinterpret_cast<XT*>(reinterpret_cast<char*>(base) + offset(i, gt)), r);
      }
  }
  __device__ __forceinline__ void store(XT* base, uint32_t gt, float a, float c, float cs) {
    touch();
    if (full()) store_all<true>(base, gt, a, c, cs);
    else store_all<false>(base, gt, a, c, cs);
  }
};

// The sum and the gradient of a far row, element by element, by BS threads.
template <typename XT, int BS>
__device__ float far_sum(const XT* row, int64_t V, uint32_t gt, float m,
                                                   float a) {
  float s = 0.f;
#pragma unroll 1
  for (int64_t v = gt; v < V; v += BS) s += exp2_of((to_float(row[v]) - m) * a);
  return wave_sum(s);
}
template <typename XT, int BS>
__device__ void far_gradient(const XT* row, XT* to, int64_t v0, int64_t v1,
                                                       uint32_t gt, float m, float a, float cs) {
#pragma unroll 1
  for (int64_t v = v0 + gt; v < v1; v += BS)
    to[v] = round_to<XT>(cs * exp2_of((to_float(row[v]) - m) * a));
}

// How a row is cut: `head` elements up to the next 16 bytes, nv vectors, and the
// elements after them. 16-bit vectors at odd elements cost a fifth of the
// forward's and the step's time (1001 x 50021 f16: 26 and 54 us against 21 and
// 43). Rows below 64 vectors keep their first element in a vector, so that a row
// with a vector at all has one.
template <typename XT>
struct Cut {
  static constexpr int VE = pack_elems<XT>();
  int64_t V, nv;
  uint32_t head;
  __device__ __forceinline__ Cut(const XT* row, int64_t v) : V(v) {
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(row) % 16);
    head = v >= 64 * VE && off ? (16 - off) / (uint32_t)sizeof(XT) : 0;
    nv = (v - head) / VE;
  }
  // The element outside the vectors that thread gt has, of `others`.
  __device__ __forceinline__ int64_t others() const { return V - nv * VE; }
  __device__ __forceinline__ int64_t other(uint32_t gt) const {
    return gt < head ? (int64_t)gt : nv * VE + gt;
  }
};

// Zeros for vectors [i0, i1) of a row by a group of BS threads.
template <typename XT, int BS>
__device__ __forceinline__ void write_zeros(XT* gx, const Cut<XT>& cut, int64_t i0, int64_t i1,
                                            uint32_t gt) {
  constexpr int VE = pack_elems<XT>();
  typename Pack<XT, VE>::raw z;
  zero_raw(z);
  for (int64_t i = i0 + gt; i < i1; i += BS) store_pack_once<XT, VE>(gx + cut.head + i * VE, z);
}

// The teacher's maximum and sum of powers over a thread's entries gt + BS j, for
// its wave; a NaN entry makes the sum NaN.
template <int BS>
__device__ __forceinline__ void teacher_sum(const Args& g, const Teacher& T, uint32_t gt, float& tm,
                                            float& ts) {
  tm = -INFINITY;
  float tn = 0.f;
#pragma unroll 1
  for (int32_t k = (int32_t)gt; k < g.K; k += BS)
    if (T.id[k] >= 0) {
      tm = fmaxf(tm, T.p[k]);
      tn += T.p[k] - T.p[k];
    }
  tm = wave_max(tm);
#pragma unroll 1
  for (int32_t k = (int32_t)gt; k < g.K; k += BS)
    if (T.id[k] >= 0) tn += exp2_of((T.p[k] - tm) * g.a);
  ts = wave_sum(tn);
}

// The statistics of a row and its teacher, from those of the group's waves.
struct RowStats {
  float m, s, tm, ts;
  // red[0..3][wave]: maximum, sum, the teacher's maximum and sum
  template <int WAVES>
  __device__ __forceinline__ void join(const float (*red)[WAVES], float a) {
    if constexpr (WAVES == 1) {
      m = red[0][0];
      s = red[1][0];
      tm = red[2][0];
      ts = red[3][0];
    } else {
      const int lane = lane_id(), w = lane % WAVES;
      const float wm = red[0][w], wt = red[2][w];
      m = wave_max(wm);
      tm = wave_max(wt);
      s = wave_sum(lane < WAVES ? red[1][w] * rescale(wm, Shift(m, a), a) : 0.f);
      ts = wave_sum(lane < WAVES ? red[3][w] * (wt == -INFINITY ? 1.f : exp2_of((wt - tm) * a)) : 0.f);
    }
  }
};

// The thread's entries' probabilities into T.p, and its wave's sum of
// tau p (log p - log q). It is in the logits' own units, so that a place with a
// logit of the type's lowest value has a finite loss wherever float32 holds it.
template <int BS>
__device__ __forceinline__ float entries_loss(const Args& g, const Teacher& T, uint32_t gt,
                                              const RowStats& r, const Shift& sh) {
  const float ls = log2_of(r.s), lt = log2_of(r.ts);
  float l = 0.f;
#pragma unroll 1
  for (int32_t k = (int32_t)gt; k < g.K; k += BS) {
    if (T.id[k] < 0) continue;
    const float lp = (T.p[k] - r.tm) * g.a - lt;
    const float p = exp2_of(lp);
    T.p[k] = p;
    if (p == 0.f) continue;
    const float x = T.x[k], scale = g.tau * kLn2;
    const float u = sh.far || !(fabsf(x * g.a) <= kFar) ? x - sh.m : scale * fmaf(x, g.a, -sh.c);
    l += p * (scale * (lp + ls) - u);
  }
  return wave_sum(l);
}

// The places in [v0, v1) of the teacher's entries, after the dense part.
template <typename XT, int BS>
__device__ __forceinline__ void write_places(const Args& g, const Teacher& T, XT* to, uint32_t gt,
                                             int64_t v0, int64_t v1, const Shift& sh, float c,
                                             float cs) {
#pragma unroll 1
  for (int32_t k = (int32_t)gt; k < g.K; k += BS) {
    const int32_t e = T.id[k];
    if (e >= v0 && e < v1 && e >= 0)
      to[e] = round_to<XT>(cs * exp2_of(sh.of(T.x[k], g.a)) - c * T.p_at(g.K, e));
  }
}

// A group of BS threads per row, part by part of NV vectors a thread; the last
// part stays in registers between the sum and the gradient, which reads the
// others again. Each thread takes the powers' sum with the maximum of its own
// elements, so that one barrier joins maxima and sums, the teacher's too.
//
// Bound by memory, with the powers close behind: an element of the gradient
// takes two quarter-rate exponentials and about ten other instructions, 60% of
// the time of 4096 x 131072 bf16 rows. 1024 threads hold those in registers, but
// for two a lane (12 bytes of scratch, and about 50 scalars in other lanes'
// registers), and read them once: 387 us, 5.3 TB/s (a copy of as much: 330 us);
// with two passes over memory in their place 462 us. Rows that leave a quarter of the
// 1024 x 16 vectors empty do better as parts of 512 x 8, two workgroups a CU:
// 294 us against 309 at 4878 x 67572 f16. The forward alone wants more, smaller
// workgroups: 256 x 4. With few rows a row's time counts: 1024 threads.
//   loss, stats [N, 2], gx: each may be null.
//   again: the logits are read again soon and may stay in the caches: the parts
//   of a long row, or all logits by the backward.
template <typename XT, int BS, int NV>
__global__ __launch_bounds__(BS < 256 ? 256 : BS) void distill_row_kernel(
    const XT* x, int64_t ldx, Args g, float* __restrict__ loss, float* __restrict__ stats,
    const float* __restrict__ gl, XT* gx, int64_t ldgx, bool again) {
  constexpr int VE = pack_elems<XT>();
  constexpr int kRows = (BS < 256 ? 256 : BS) / BS;  // rows of a workgroup
  constexpr int kWaves = BS / kWave;
  __shared__ float red[kRows][6][kWaves];
  extern __shared__ __align__(16) char lds[];
  const int group = kRows > 1 ? wave_index() : 0;
  const uint32_t gt = kRows > 1 ? lane_id() : threadIdx.x;
  const int wave = kRows > 1 ? 0 : wave_index();
  const int lane = lane_id();
  const int32_t k4 = (g.K + 3) / 4 * 4;
  const Teacher T(lds + group * 3 * sizeof(int32_t) * k4, g.K);
  for (int64_t n = (int64_t)blockIdx.x * kRows + group; n < g.N; n += (int64_t)gridDim.x * kRows) {
    const XT* row = x + n * ldx;
    XT* to = gx + n * ldgx;
    const Cut<XT> cut(gx ? to : row, g.V);
    const int64_t nv = cut.nv, at = cut.other(gt);
    const bool mine = gt < cut.others();
    const int32_t parts = NV ? (int32_t)((nv + BS * NV - 1) / (BS * (NV ? NV : 1))) : 1;
    if (!has_teacher(g, n)) {
      if (gt == 0) {
        if (loss) loss[n] = 0.f;
        if (stats) stats[2 * n] = 0.f, stats[2 * n + 1] = 0.f;
      }
      if (gx) {
        write_zeros<XT, BS>(to, cut, 0, nv, gt);
        if (mine) to[at] = round_to<XT>(0.f);
      }
      continue;
    }
    // the teacher's entries, and the student's logits at their places
    constexpr int KU = BS >= 1024 ? 1 : 4;  // entries a thread has in flight
    for (int32_t k0 = (int32_t)gt; k0 < k4; k0 += KU * BS) {
      int32_t id[KU];
      float t[KU], xk[KU];
      load_entries<KU>(g, n, k0, BS, id, t);
#pragma unroll
      for (int q = 0; q < KU; ++q) xk[q] = id[q] >= 0 ? to_float(row[id[q]]) : 0.f;
#pragma unroll
      for (int q = 0; q < KU; ++q) {
        const int32_t k = k0 + q * BS;
        if (k < k4) {
          T.id[k] = id[q];
          T.p[k] = t[q];
          T.x[k] = xk[q];
        }
      }
    }

    Part<XT, BS, NV> p;
    float m = -INFINITY, s = 0.f, rest = -INFINITY;
    for (int32_t i = 0; i < parts; ++i) {
      const int64_t base = (int64_t)i * (BS * NV);
      p.shape(nv - base, wave);
      const XT* from = row + cut.head + base * VE;
      if (again) p.template load<false>(from, gt);
      else p.template load<true>(from, gt);
      if (i == parts - 1 && mine) rest = to_float(row[at]);
      const float before = m;
      m = p.max(fmaxf(m, rest));
      const Shift sh(m, g.a);
      const float add = p.sum(sh, gt, rest, g.a);
      s = sh.far && s == s ? add : s * rescale(before, sh, g.a) + add;
    }
    {
      const float wm = wave_max(m);
      const float ws = wave_sum(s * rescale(m, Shift(wm, g.a), g.a));
      float tm, ts;
      teacher_sum<BS>(g, T, gt, tm, ts);
      if (lane == 0) {
        red[group][0][wave] = wm;
        red[group][1][wave] = ws;
        red[group][2][wave] = tm;
        red[group][3][wave] = ts;
      }
    }
    group_sync<BS>();
    RowStats r;
    r.join<kWaves>(red[group], g.a);
    const Shift sh(r.m, g.a, kFarRow);
    if (__builtin_expect(sh.far, 0)) {
      const float ws = far_sum<XT, BS>(row, g.V, gt, r.m, g.a);
      if (lane == 0) red[group][4][wave] = ws;
      group_sync<BS>();
      r.s = 0.f;
      for (int w = 0; w < kWaves; ++w) r.s += red[group][4][w];
    }
    const float l = entries_loss<BS>(g, T, gt, r, sh);
    if (lane == 0) red[group][5][wave] = l;

    const float c = gx ? gl[n] * g.tau : 0.f;
    const float cs = c / r.s;
    if (gx) {
      if (__builtin_expect(sh.far, 0)) {
        far_gradient<XT, BS>(row, to, 0, g.V, gt, r.m, g.a, cs);
      } else {
        for (int32_t i = parts - 1; i >= 0; --i) {
          const int64_t base = (int64_t)i * (BS * NV);
          if (i != parts - 1) {
            p.shape(nv - base, wave);
            p.template load<true>(row + cut.head + base * VE, gt);
          }
          p.store(to + cut.head + base * VE, gt, g.a, sh.c, cs);
        }
        if (mine) to[at] = round_to<XT>(cs * exp2_of(sh.of(rest, g.a)));
      }
    }
    group_sync<BS>();
    if (gt == 0) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) sum += red[group][5][w];
      if (loss) loss[n] = g.tau * sum;
      if (stats) stats[2 * n] = r.m, stats[2 * n + 1] = r.s / sh.of_max(g.a);
    }
    if (gx) write_places<XT, BS>(g, T, to, gt, 0, g.V, sh, c, cs);
    group_sync<BS>();  // the next row takes the LDS
  }
}

// The gradient from the forward's statistics: a workgroup per piece of at most
// NV vectors a thread of a row, or a wave per row where that holds it. The
// first wave finds the teacher's maximum and sum again, while the piece is on
// the way; the others need only the statistics. Bound by memory: with 16 KB a
// piece 44 us at 1001 x 50021 f16 (190 MB, the logits from the Infinity
// Cache), with 32 KB 47, with 8 KB 54.
template <typename XT, int BS, int NV>
__global__ __launch_bounds__(256) void distill_backward_kernel(
    const XT* x, int64_t ldx, Args g, const float* __restrict__ stats,
    const float* __restrict__ gl, XT* gx, int64_t ldgx, int32_t pieces, int64_t per) {
  constexpr int VE = pack_elems<XT>();
  constexpr int kRows = 256 / BS;
  __shared__ bool places[kRows];
  extern __shared__ __align__(16) char lds[];
  const int group = kRows > 1 ? wave_index() : 0;
  const uint32_t gt = kRows > 1 ? lane_id() : threadIdx.x;
  const int wave = kRows > 1 ? 0 : wave_index();
  const int lane = lane_id();
  const int32_t k4 = (g.K + 3) / 4 * 4;
  const Teacher T(lds + group * 3 * sizeof(int32_t) * k4, g.K);
  const int64_t items = g.N * pieces;
  for (int64_t w = (int64_t)blockIdx.x * kRows + group; w < items; w += (int64_t)gridDim.x * kRows) {
    const int64_t n = pieces == 1 ? w : w / pieces;
    const int32_t piece = (int32_t)(w - n * pieces);
    const bool last = piece == pieces - 1;
    const XT* row = x + n * ldx;
    XT* to = gx + n * ldgx;
    const Cut<XT> cut(to, g.V);
    // vectors [i0, i1), none in the last piece of some rows; the first piece has
    // the elements before them, the last one those after
    const int64_t i0 = piece * per, i1 = last ? cut.nv : i0 + per;
    const int64_t v0 = piece == 0 ? 0 : cut.head + i0 * VE, v1 = last ? g.V : cut.head + i1 * VE;
    const int64_t at = cut.other(gt);
    const bool other = gt < cut.others() && (gt < cut.head ? piece == 0 : last);
    const float m = stats[2 * n], s = stats[2 * n + 1];
    if (m == 0.f && s == 0.f) {  // no teacher
      write_zeros<XT, BS>(to, cut, i0, i1, gt);
      if (other) to[at] = round_to<XT>(0.f);
      continue;
    }
    constexpr int KU = 4;  // entries a lane has in flight
    int32_t id[KU] = {};
    float t[KU] = {};
    if (wave == 0) load_entries<KU>(g, n, lane, kWave, id, t);
    Part<XT, BS, NV> p;
    p.shape(i1 - i0, wave);
    p.template load<true>(row + cut.head + (i1 > i0 ? i0 * VE : 0), gt);
    float rest = 0.f;
    if (other) rest = to_float(row[at]);
    if (wave == 0) {
      bool here = false;
      for (int32_t k0 = lane; k0 < k4; k0 += KU * kWave) {
        if (k0 != lane) load_entries<KU>(g, n, k0, kWave, id, t);
        float xk[KU];
#pragma unroll
        for (int q = 0; q < KU; ++q) {
          const bool mine = id[q] >= v0 && id[q] < v1;
          xk[q] = mine ? to_float(row[id[q]]) : 0.f;
          here |= mine;
        }
#pragma unroll
        for (int q = 0; q < KU; ++q) {
          const int32_t k = k0 + q * kWave;
          if (k < k4) {
            T.id[k] = id[q];
            T.p[k] = t[q];
            T.x[k] = xk[q];
          }
        }
      }
      here = __any(here);
      if (here) {  // p, where this piece has an entry
        float tm, ts;
        teacher_sum<kWave>(g, T, lane, tm, ts);
        const float lt = log2_of(ts);
#pragma unroll 1
        for (int32_t k = lane; k < g.K; k += kWave)
          if (T.id[k] >= 0) T.p[k] = exp2_of((T.p[k] - tm) * g.a - lt);
      }
      if (lane == 0) places[group] = here;
    }
    const Shift sh(m, g.a, kFarRow);
    const float c = gl[n] * g.tau;
    const float cs = c / (s * sh.of_max(g.a));
    if (x == gx) group_sync<BS>();  // the places are read before they are written
    if (__builtin_expect(sh.far, 0)) {
      far_gradient<XT, BS>(row, to, v0, v1, gt, m, g.a, cs);
    } else {
      p.store(to + cut.head + i0 * VE, gt, g.a, sh.c, cs);
      if (other) to[at] = round_to<XT>(cs * exp2_of(sh.of(rest, g.a)));
    }
    group_sync<BS>();
    if (places[group]) write_places<XT, BS>(g, T, to, gt, v0, v1, sh, c, cs);
    group_sync<BS>();  // the next piece takes the LDS
  }
}

Args make_args(const tbe_distill_desc& d, const void* ids, const void* t) {
  Args g;
  g.ids = ids;
  g.t = t;
  g.idx64 = d.idx64;
  g.K = d.K;
  g.tdtype = d.tdtype;
  g.N = d.N;
  g.V = d.V;
  g.tau = d.temperature;
  g.a = distill_factor(d.temperature);
  return g;
}

unsigned grid_for(int64_t n) { return (unsigned)(n < (1 << 20) ? n : (1 << 20)); }

constexpr int64_t kFewRows = 256;             // a row per CU
// The Infinity Cache: logits of up to its size stay there for the backward if
// the forward's loads are ordinary ones (1001 x 50021 f16: with nontemporal ones
// both calls together took a tenth longer).
constexpr int64_t kCacheBytes = 256 << 20;

hipError_t launch_rows(const tbe_distill_desc& d, const void* x, int64_t ldx, const void* ids,
                       const void* t, float* loss, float* stats, const float* gl, void* gx,
                       int64_t ldgx, hipStream_t s) {
  const Args g = make_args(d, ids, t);
  return with_type(d.dtype, [&](auto xt) {
    using XT = decltype(xt);
    const int64_t nv = d.V / pack_elems<XT>();
    auto go = [&](auto bs, auto vectors) {
      constexpr int BS = decltype(bs)::value, NV = decltype(vectors)::value;
      constexpr int kRows = BS < 256 ? 256 / BS : 1;
      const bool again = (gx && nv > BS * NV) ||
                         (!gx && d.N * d.V * (int64_t)sizeof(XT) <= kCacheBytes);
      hipLaunchKernelGGL((distill_row_kernel<XT, BS, NV>), dim3(grid_for((d.N + kRows - 1) / kRows)),
                         dim3(BS < 256 ? 256 : BS), kRows * Teacher::bytes(d.K), s,
                         static_cast<const XT*>(x), ldx, g, loss, stats, gl, static_cast<XT*>(gx),
                         ldgx, again);
      return hipGetLastError();
    };
    using std::integral_constant;
    if (nv == 0) return go(integral_constant<int, 64>{}, integral_constant<int, 0>{});
    if (nv <= 64 * 2) return go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (nv <= 64 * 8) return go(integral_constant<int, 64>{}, integral_constant<int, 8>{});
    if (nv <= 256 * 8) {
      if (gx || d.N <= kFewRows) return go(integral_constant<int, 256>{}, integral_constant<int, 8>{});
    } else if (d.N <= kFewRows) {
      return go(integral_constant<int, 1024>{}, integral_constant<int, 8>{});
    }
    if (!gx) return go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
    if (nv <= 1024 * 12 || nv > 1024 * 16)
      return go(integral_constant<int, 512>{}, integral_constant<int, 8>{});
    return go(integral_constant<int, 1024>{}, integral_constant<int, 16>{});
  });
}

}  // namespace

// The kernels need no scratch memory. The calls take a workspace, as the other
// operators' do, of one alignment unit.
size_t distill_workspace(const tbe_distill_desc&) { return 256; }

hipError_t launch_distill_forward(const tbe_distill_desc& d, const void* x, int64_t ldx,
                                  const void* ids, const void* t, float* loss, float* stats,
                                  void*, hipStream_t s) {
  return launch_rows(d, x, ldx, ids, t, loss, stats, nullptr, nullptr, 0, s);
}

hipError_t launch_distill_backward(const tbe_distill_desc& d, const void* x, int64_t ldx,
                                   const void* ids, const void* t, const float* stats,
                                   const float* gl, void* gx, int64_t ldgx, hipStream_t s) {
  const Args g = make_args(d, ids, t);
  return with_type(d.dtype, [&](auto xt) {
    using XT = decltype(xt);
    const int64_t nv = d.V / pack_elems<XT>();
    auto go = [&](auto bs, auto vectors) {
      constexpr int BS = decltype(bs)::value, NV = decltype(vectors)::value;
      constexpr int kRows = 256 / BS;
      // pieces of one size, whole rounds of a wave
      int64_t pieces = 1, per = nv;
      if (nv > BS * NV) {
        pieces = (nv + BS * NV - 1) / (BS * (NV ? NV : 1));
        per = ((nv + pieces - 1) / pieces + 63) / 64 * 64;
        pieces = (nv + per - 1) / per;
      }
      hipLaunchKernelGGL((distill_backward_kernel<XT, BS, NV>),
                         dim3(grid_for((d.N * pieces + kRows - 1) / kRows)), dim3(256),
                         kRows * Teacher::bytes(d.K), s, static_cast<const XT*>(x), ldx, g, stats,
                         gl, static_cast<XT*>(gx), ldgx, (int32_t)pieces, per);
      return hipGetLastError();
    };
    using std::integral_constant;
    if (nv == 0) return go(integral_constant<int, 64>{}, integral_constant<int, 0>{});
    if (nv <= 64 * 2) return go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (nv <= 64 * 8) return go(integral_constant<int, 64>{}, integral_constant<int, 8>{});
    return go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  });
}

hipError_t launch_distill_step(const tbe_distill_desc& d, const void* x, int64_t ldx,
                               const void* ids, const void* t, const float* gl, float* loss,
                               void* gx, int64_t ldgx, void*, hipStream_t s) {
  return launch_rows(d, x, ldx, ids, t, loss, nullptr, gl, gx, ldgx, s);
}

}  // namespace tbe
