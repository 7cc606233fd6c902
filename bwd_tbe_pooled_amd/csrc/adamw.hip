// One AdamW step over many tensors.
//
// A launch takes up to kTensors tensors, whose addresses stand in the kernel's
// arguments (no table in memory to keep or to copy), and a workgroup one chunk
// of one tensor. Memory bounds it: each element of parameter, gradient and
// moments is read once and written once, 28 bytes for float32 parameters with a
// 16-bit gradient and copy, 10 for 16-bit parameters with 8-bit moments. A
// thread loads all its vectors before it computes. 357 million of the former
// take 1.73 to 1.75 ms, 5.8 TB/s; 738 million of the latter 1.29 to 1.30, 5.7.
// (The latter's 57 vector instructions an element take 1.06 ms to issue: exact
// roots and quotients are paid for by what one wave works out for four.)
//
// An 8-bit moment's block of 256 elements lies in neighbouring lanes (64 of 4
// elements or 32 of 8), so its scale takes one reduction and no memory.
#include <algorithm>
#include <type_traits>

#include "lm.h"
#include "lm_device.h"

namespace tbe {
namespace {

constexpr int kThreads = 256;
constexpr int kTensors = 52;      // of a launch: the arguments stay within 4 KiB

struct Args {
  const int64_t* step;
  const float *lr, *scale;
  double beta1, beta2;
  float eps, decay;
  int32_t count;
  int32_t end[kTensors];          // first chunk behind each tensor
  tbe_adamw_tensor t[kTensors];
};
static_assert(sizeof(Args) <= 4096 - 64, "kernel arguments");

// b^t for t >= 1 by squaring.
__device__ __forceinline__ double power(double b, uint64_t t) {
  double r = 1.0;
  for (; t; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

// a * b + c, the product rounded before the sum. 8-bit moments have their codes at the
// float32 formulas' borders, to the last bit: what is fused is rounded once less, and a
// code in some millions falls to the other side.
__device__ __forceinline__ float apart(float a, float b, float c) {
#pragma clang fp contract(off)
  const float p = a * b;
  return p + c;
}

// Roots of numbers >= 0, rounded to nearest. The hardware's root is off by one step now
// and then, and takes subnormal numbers for zeros; a fused residual and one correction put
// it right (as sqrtf does, compared for all mantissas) where no part of it is subnormal.
template <int V>
__device__ __forceinline__ void roots(const float (&v)[V], float (&r)[V]) {
  uint32_t low = ~0u, high = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    low = min(low, __float_as_uint(v[j]));
    high = max(high, __float_as_uint(v[j]));
  }
  if (low >= __float_as_uint(0x1p-96f) && high <= __float_as_uint(0x1p96f)) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float y = __builtin_amdgcn_rsqf(v[j]), s = v[j] * y;
      r[j] = fmaf(fmaf(-s, s, v[j]), 0.5f * y, s);
    }
  } else {   // (zeros among them)
#pragma unroll
    for (int j = 0; j < V; ++j) r[j] = sqrtf(v[j]);
  }
}

// Largest over the LANES neighbouring lanes that hold a block, all of them active.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, false);
}
template <int LANES>
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
  x = max(x, dpp_u32<0xB1>(x));
  x = max(x, dpp_u32<0x4E>(x));
  x = max(x, dpp_u32<0x141>(x));
  x = max(x, dpp_u32<0x140>(x));
  x = max(x, (uint32_t)__shfl_xor((int)x, 16));
  if constexpr (LANES == 64) x = max(x, (uint32_t)__shfl_xor((int)x, 32));
  return x;
}

// 4 or 8 e4m3 numbers in one or two words.
template <int V>
struct Codes {
  uint32_t w[V / 4];
};
template <int V>
__device__ __forceinline__ void decode(const Codes<V>& q, float scale, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.w[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.w[i], true);
    f[4 * i] = lo[0] * scale;
    f[4 * i + 1] = lo[1] * scale;
    f[4 * i + 2] = hi[0] * scale;
    f[4 * i + 3] = hi[1] * scale;
  }
}

// Codes of f / scale, inv = 1 / scale; LEAST holds what is above zero at 2^-9, the smallest
// code, at least. What is not finite becomes NaN (only asked of blocks that hold such a
// value). The quotient is rounded to nearest: times the reciprocal it is off by a step or
// two, which one residual puts right (as a division does, compared for 2^32 pairs); a code
// at the border of two would fall to the wrong one otherwise.
template <int V, bool LEAST, bool FINITE>
__device__ __forceinline__ Codes<V> codes_of(const float (&f)[V], float scale, float inv) {
  float q[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    q[j] = f[j] * inv;
    q[j] = fmaf(fmaf(-q[j], scale, f[j]), inv, q[j]);
    if (LEAST) q[j] = f[j] > 0.f && inv > 0.f ? fmaxf(q[j], 0x1p-9f) : q[j];
    if (!FINITE) q[j] = fabsf(f[j]) < __builtin_inff() ? q[j] : __builtin_nanf("");
  }
  Codes<V> r;
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
    r.w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], w, true);
  }
  return r;
}

// f as codes and their block's scale. A code is the nearest to its value by the scale as it
// is stored, ties to even: at most half a step (2^-4 of the value) off. Elements that do not
// exist are zeros. The largest magnitude is found on the bit patterns, where infinities and
// NaN are above all numbers: then it is looked for again among the finite ones.
template <int V, bool LEAST>
__device__ __forceinline__ Codes<V> encode(const float (&f)[V], float* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
  top = block_max<kAdamBlock / V>(top);
  const bool finite = top < 0x7f800000u;
  if (!finite) {
    top = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t u = __float_as_uint(f[j]) & 0x7fffffffu;
      top = max(top, u < 0x7f800000u ? u : 0u);
    }
    top = block_max<kAdamBlock / V>(top);
  }
  const float t = __uint_as_float(top);
  const bool some = t >= 0x1p-100f;
  const float by = some ? t * (1.f / 448.f) : 0.f;
  const float inv = some ? 1.f / by : 0.f;
  *scale = by;
  return finite ? codes_of<V, LEAST, true>(f, by, inv) : codes_of<V, LEAST, false>(f, by, inv);
}

// V elements from p + at, of which n exist (all of them in whole vectors).
template <typename T, int V>
__device__ __forceinline__ void load_some(const T* p, int n, float (&f)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = j < n ? to_float(p[j]) : 0.f;
}
template <typename T, int V>
__device__ __forceinline__ void store_some(T* p, int n, const float (&f)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (j < n) p[j] = round_to<T>(f[j]);
}

// Elements of a thread's vector, and vectors of a thread where there is much to do: what
// is in flight covers memory's latency (357 million float32 parameters: 1759 us with 4
// vectors of 4, 1806 with 2; 738 million of 16 bits with 8-bit moments: 1339 with 2
// vectors of 8, 1299 with 1). With little to do more workgroups are faster, and one
// vector is taken.
template <typename P>
constexpr int vector_of() { return sizeof(P) == 4 ? 4 : 8; }
template <typename P, int BITS>
constexpr int most_vectors() { return (BITS == 32 ? 16 : 8) / vector_of<P>(); }
constexpr int64_t kMuch = int64_t(1) << 22;   // elements

// P, G, C: types of parameters, gradients and copies (C = void: none). U: vectors of a
// thread.
template <typename P, typename G, typename C, int BITS, int U>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Args a) {
  constexpr bool kCopy = !__is_same(C, void);
  using CT = std::conditional_t<kCopy, C, bf16_t>;
  constexpr int V = vector_of<P>();
  constexpr int kChunk = kThreads * V * U;
  static_assert(kChunk % kAdamBlock == 0, "chunks of whole blocks");
  const int64_t step = *a.step;
  const float lr = *a.lr;
  const float scale = a.scale ? *a.scale : 1.f;
  // the tensor: the first whose end is behind this chunk; a lane looks at each end
  const int lane = lane_id();
  const int lo = __popcll(__ballot(lane < a.count && a.end[lane < kTensors ? lane : 0] <= (int)blockIdx.x));
  const tbe_adamw_tensor& t = a.t[lo];
  const int64_t base = (int64_t)((int)blockIdx.x - (lo ? a.end[lo - 1] : 0)) * kChunk;
  P* const p = static_cast<P*>(t.p) + base;
  const G* const g = static_cast<const G*>(t.g) + base;
  CT* const c = kCopy ? static_cast<CT*>(t.c) + base : nullptr;
  const int64_t left64 = t.n - base;
  const int left = left64 < kChunk ? (int)left64 : kChunk;

  auto at = [&](int u) { return (u * kThreads + (int)threadIdx.x) * V; };
  float x[U][V], gr[U][V], m[U][V], v[U][V];
  typename Pack<P, V>::raw rp[U];
  typename Pack<G, V>::raw rg[U];
  typename Pack<float, V>::raw rm[U], rv[U];
  Codes<V> qm[U], qv[U];
  float sm[U], sv[U];
  uint8_t* const m8 = static_cast<uint8_t*>(t.m) + base;
  uint8_t* const v8 = static_cast<uint8_t*>(t.v) + base;
  float* const m32 = static_cast<float*>(t.m) + base;
  float* const v32 = static_cast<float*>(t.v) + base;
  const int64_t block0 = base / kAdamBlock;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = at(u);
    if (i + V > left) continue;
    rp[u] = load_pack_once<P, V>(p + i);
    rg[u] = load_pack_once<G, V>(g + i);
    if constexpr (BITS == 32) {
      rm[u] = load_pack_once<float, V>(m32 + i);
      rv[u] = load_pack_once<float, V>(v32 + i);
    } else {
      qm[u] = *reinterpret_cast<const Codes<V>*>(m8 + i);
      qv[u] = *reinterpret_cast<const Codes<V>*>(v8 + i);
      sm[u] = t.mscale[block0 + i / kAdamBlock];
      sv[u] = t.vscale[block0 + i / kAdamBlock];
    }
  }
  const uint64_t n_step = step < 1 ? 1 : (uint64_t)step;
  const float b1 = (float)a.beta1, b2 = (float)a.beta2;
  const float g1 = (float)(1.0 - a.beta1), g2 = (float)(1.0 - a.beta2);
  // The corrections of the bias, by one wave for all: in 64 bits, where 1 - beta^t keeps its
  // digits, they cost a wave as much as 150 instructions in 32. Even lanes lr / (1 - beta1^t),
  // odd ones 1 / sqrt(1 - beta2^t).
  __shared__ float shared[2];
  if (wave_index() == 0) {
    const bool second = lane & 1;
    const double c = 1.0 - power(second ? a.beta2 : a.beta1, n_step);
    const float f = (float)((second ? 1.0 : (double)lr) / (second ? sqrt(c) : c));
    if (lane < 2) shared[lane] = f;
  }
  __syncthreads();
  const float move = shared[0], unbias = shared[1];
  const float keep = (float)(1.0 - (double)lr * (double)a.decay);

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = at(u);
    const int n = left - i < V ? left - i : V;
    if (n == V) {
      widen<P, V>(rp[u], x[u]);
      widen<G, V>(rg[u], gr[u]);
      if constexpr (BITS == 32) {
        widen<float, V>(rm[u], m[u]);
        widen<float, V>(rv[u], v[u]);
      } else {
        decode<V>(qm[u], sm[u], m[u]);
        decode<V>(qv[u], sv[u], v[u]);
      }
    } else {   // the tensor's last vector, and none behind it
      load_some<P, V>(p + i, n, x[u]);
      load_some<G, V>(g + i, n, gr[u]);
      if constexpr (BITS == 32) {
        load_some<float, V>(m32 + i, n, m[u]);
        load_some<float, V>(v32 + i, n, v[u]);
      } else {
        float ms = 0.f, vs = 0.f;
        if (n > 0) {
          ms = t.mscale[block0 + i / kAdamBlock];
          vs = t.vscale[block0 + i / kAdamBlock];
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
          m[u][j] = j < n ? __builtin_amdgcn_cvt_f32_fp8((int)m8[i + j], 0) * ms : 0.f;
          v[u][j] = j < n ? __builtin_amdgcn_cvt_f32_fp8((int)v8[i + j], 0) * vs : 0.f;
        }
      }
    }
    float root[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float gj = gr[u][j] * scale;
      if constexpr (BITS == 32) {
        m[u][j] = fmaf(b1, m[u][j], g1 * gj);
        v[u][j] = fmaf(b2, v[u][j], g2 * gj * gj);
      } else {
        m[u][j] = apart(b1, m[u][j], g1 * gj);
        v[u][j] = apart(b2, v[u][j] * v[u][j], g2 * gj * gj);
      }
    }
    roots<V>(v[u], root);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (BITS == 8) v[u][j] = root[j];
      // (the hardware's reciprocal is within 1 ulp)
      x[u][j] = fmaf(-(move * m[u][j]), __builtin_amdgcn_rcpf(fmaf(root[j], unbias, a.eps)), keep * x[u][j]);
    }
    if (n == V) {
      store_pack_once<P, V>(p + i, narrow<P, V>(x[u]));
      if constexpr (kCopy) store_pack_once<CT, V>(c + i, narrow<CT, V>(x[u]));
      if constexpr (BITS == 32) {
        store_pack_once<float, V>(m32 + i, narrow<float, V>(m[u]));
        store_pack_once<float, V>(v32 + i, narrow<float, V>(v[u]));
      }
    } else if (n > 0) {
      store_some<P, V>(p + i, n, x[u]);
      if constexpr (kCopy) store_some<CT, V>(c + i, n, x[u]);
      if constexpr (BITS == 32) {
        store_some<float, V>(m32 + i, n, m[u]);
        store_some<float, V>(v32 + i, n, v[u]);
      }
    }
    if constexpr (BITS == 8) {   // every lane of a block takes part in its reduction
      float ms, vs;
      const Codes<V> em = encode<V, false>(m[u], &ms), ev = encode<V, true>(v[u], &vs);
      if (n == V) {
        *reinterpret_cast<Codes<V>*>(m8 + i) = em;
        *reinterpret_cast<Codes<V>*>(v8 + i) = ev;
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (j >= n) continue;
          m8[i + j] = (uint8_t)(em.w[j / 4] >> (8 * (j % 4)));
          v8[i + j] = (uint8_t)(ev.w[j / 4] >> (8 * (j % 4)));
        }
      }
      if (n > 0 && i % kAdamBlock == 0) {
        t.mscale[block0 + i / kAdamBlock] = ms;
        t.vscale[block0 + i / kAdamBlock] = vs;
      }
    }
  }
}

template <typename F>
hipError_t with_types(const tbe_adamw_desc& d, F f) {
  return with_type(d.pdtype, [&](auto p) {
    using P = decltype(p);
    return with_type(d.gdtype, [&](auto g) {
      using G = decltype(g);
      if constexpr (sizeof(P) == 4) {
        if (d.cdtype == TBE_F16) return f((P*)nullptr, (G*)nullptr, (f16_t*)nullptr);
        if (d.cdtype == TBE_BF16) return f((P*)nullptr, (G*)nullptr, (bf16_t*)nullptr);
      }
      return f((P*)nullptr, (G*)nullptr, (void*)nullptr);
    });
  });
}

}  // namespace

hipError_t launch_adamw(const tbe_adamw_desc& d, const tbe_adamw_tensor* tensors, int64_t count,
                        const int64_t* step, const float* lr, const float* scale, hipStream_t s) {
  constexpr int64_t kMaxBlocks = int64_t(1) << 23;   // of a launch: 2^31 threads
  const int64_t esize[3] = {d.pdtype == TBE_F32 ? 4 : 2, d.gdtype == TBE_F32 ? 4 : 2,
                            d.bits == 32 ? 4 : 1};
  Args a;
  a.step = step;
  a.lr = lr;
  a.scale = scale;
  a.beta1 = d.beta1;
  a.beta2 = d.beta2;
  a.eps = (float)d.eps;
  a.decay = (float)d.weight_decay;
  a.count = 0;
  int64_t blocks = 0;
  int64_t elements = 0;
  for (int64_t i = 0; i < count; ++i) elements += tensors[i].n;
  const bool much = elements >= kMuch;
  const int vector = d.pdtype == TBE_F32 ? 4 : 8, most = (d.bits == 32 ? 16 : 8) / vector;
  const int64_t chunk = (int64_t)kThreads * vector * (much ? most : 1);
  auto flush = [&]() -> hipError_t {
    if (a.count == 0) return hipSuccess;
    const hipError_t e = with_types(d, [&](auto* p, auto* g, auto* c) {
      using P = std::remove_pointer_t<decltype(p)>;
      using G = std::remove_pointer_t<decltype(g)>;
      using C = std::remove_pointer_t<decltype(c)>;
      auto run = [&](auto bits) {
        constexpr int BITS = decltype(bits)::value, MOST = most_vectors<P, BITS>();
        if (much) adamw_kernel<P, G, C, BITS, MOST><<<(unsigned)blocks, kThreads, 0, s>>>(a);
        else adamw_kernel<P, G, C, BITS, 1><<<(unsigned)blocks, kThreads, 0, s>>>(a);
      };
      if (d.bits == 32) run(std::integral_constant<int, 32>{});
      else run(std::integral_constant<int, 8>{});
      return hipGetLastError();
    });
    a.count = 0;
    blocks = 0;
    return e;
  };
  for (int64_t i = 0; i < count; ++i) {
    tbe_adamw_tensor t = tensors[i];
    while (t.n > 0) {   // a tensor of more workgroups than a launch has left is cut
      const int64_t need = (t.n + chunk - 1) / chunk;
      const int64_t take = std::min(need, kMaxBlocks - blocks);
      const int64_t elems = std::min(t.n, take * chunk);
      tbe_adamw_tensor part = t;
      part.n = elems;
      a.t[a.count] = part;
      blocks += take;
      a.end[a.count++] = (int32_t)blocks;
      t.n -= elems;
      t.p = static_cast<char*>(t.p) + elems * esize[0];
      t.g = static_cast<const char*>(t.g) + elems * esize[1];
      t.m = static_cast<char*>(t.m) + elems * esize[2];
      t.v = static_cast<char*>(t.v) + elems * esize[2];
      if (t.mscale) t.mscale += elems / kAdamBlock;
      if (t.vscale) t.vscale += elems / kAdamBlock;
      if (t.c) t.c = static_cast<char*>(t.c) + elems * 2;
      if (a.count == kTensors || blocks == kMaxBlocks) {
        const hipError_t e = flush();
        if (e != hipSuccess) return e;
      }
    }
  }
  return flush();
}

}  // namespace tbe
