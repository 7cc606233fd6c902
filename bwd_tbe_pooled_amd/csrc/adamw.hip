// One AdamW step over many tensors.
//
// A launch takes up to kTensors tensors, whose addresses stand in the kernel's
// arguments (no table in memory to keep or to copy), and a workgroup one chunk
// of one tensor. Memory bounds it: each element of parameter, gradient and
// moments is read once and written once, 28 bytes for float32 parameters with a
// 16-bit gradient and copy, 10 for 16-bit parameters with 8-bit moments. A
// thread loads all its vectors before it computes.
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
constexpr int kChunk = 4096;      // elements of a workgroup: whole blocks of the 8-bit moments
constexpr int kTensors = 52;      // of a launch: the arguments stay within 4 KiB
static_assert(kChunk % kAdamBlock == 0, "chunks of whole blocks");

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

// Largest over the lanes that hold a block.
template <int LANES>
__device__ __forceinline__ float block_max(float x) {
  x = fmaxf(x, dpp_f32<0xB1>(x));
  x = fmaxf(x, dpp_f32<0x4E>(x));
  x = fmaxf(x, dpp_f32<0x141>(x));
  x = fmaxf(x, dpp_f32<0x140>(x));
  x = fmaxf(x, __shfl_xor(x, 16));
  if constexpr (LANES == 64) x = fmaxf(x, __shfl_xor(x, 32));
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

// f as codes and their block's scale. Rounded to nearest even, at most half a
// step (2^-4 of the value) off; LEAST holds what is above zero at 2^-9, the
// smallest code, at least. Elements from `n` on are none.
template <int V, bool LEAST>
__device__ __forceinline__ Codes<V> encode(float (&f)[V], int n, float* scale) {
  constexpr float kInf = __builtin_inff();
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float a = fabsf(f[j]);
    top = fmaxf(top, j < n && a < kInf ? a : 0.f);
  }
  top = block_max<kAdamBlock / V>(top);
  const bool some = top >= 0x1p-100f;
  const float inv = some ? 448.f / top : 0.f;
  *scale = some ? top * (1.f / 448.f) : 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float q = f[j] * inv;
    if (LEAST) q = f[j] > 0.f && some ? fmaxf(q, 0x1p-9f) : q;
    f[j] = fabsf(f[j]) < kInf ? q : __builtin_nanf("");
  }
  Codes<V> r;
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], 0, false);
    r.w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], w, true);
  }
  return r;
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

// P, G, C: types of parameters, gradients and copies (C = void: none).
template <typename P, typename G, typename C, int BITS>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Args a) {
  constexpr bool kCopy = !__is_same(C, void);
  using CT = std::conditional_t<kCopy, C, bf16_t>;
  constexpr int V = sizeof(P) == 4 ? 4 : 8;
  constexpr int U = kChunk / (kThreads * V);   // vectors of a thread
  // the tensor: the first whose end is behind this chunk
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if ((int)blockIdx.x < a.end[mid]) hi = mid;
    else lo = mid + 1;
  }
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
  const int64_t step = *a.step;
  const uint64_t n_step = step < 1 ? 1 : (uint64_t)step;
  const float lr = *a.lr;
  const float scale = a.scale ? *a.scale : 1.f;
  const float b1 = (float)a.beta1, b2 = (float)a.beta2;
  const float g1 = (float)(1.0 - a.beta1), g2 = (float)(1.0 - a.beta2);
  const float move = (float)((double)lr / (1.0 - power(a.beta1, n_step)));
  const float unbias = (float)(1.0 / sqrt(1.0 - power(a.beta2, n_step)));
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
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float gj = gr[u][j] * scale;
      m[u][j] = fmaf(b1, m[u][j], g1 * gj);
      const float old = BITS == 32 ? v[u][j] : v[u][j] * v[u][j];
      const float vn = fmaf(b2, old, g2 * gj * gj);
      const float root = sqrtf(vn);
      v[u][j] = BITS == 32 ? vn : root;
      x[u][j] = fmaf(keep, x[u][j], -(move * m[u][j]) / fmaf(root, unbias, a.eps));
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
      const Codes<V> em = encode<V, false>(m[u], n, &ms), ev = encode<V, true>(v[u], n, &vs);
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
  auto flush = [&]() -> hipError_t {
    if (a.count == 0) return hipSuccess;
    const hipError_t e = with_types(d, [&](auto* p, auto* g, auto* c) {
      using P = std::remove_pointer_t<decltype(p)>;
      using G = std::remove_pointer_t<decltype(g)>;
      using C = std::remove_pointer_t<decltype(c)>;
      if (d.bits == 32) adamw_kernel<P, G, C, 32><<<(unsigned)blocks, kThreads, 0, s>>>(a);
      else adamw_kernel<P, G, C, 8><<<(unsigned)blocks, kThreads, 0, s>>>(a);
      return hipGetLastError();
    });
    a.count = 0;
    blocks = 0;
    return e;
  };
  for (int64_t i = 0; i < count; ++i) {
    tbe_adamw_tensor t = tensors[i];
    while (t.n > 0) {   // a tensor of more workgroups than a launch has left is cut
      const int64_t need = (t.n + kChunk - 1) / kChunk;
      const int64_t take = std::min(need, kMaxBlocks - blocks);
      const int64_t elems = std::min(t.n, take * kChunk);
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
