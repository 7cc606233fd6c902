// Device-side helpers of the language-model kernels: vectors of up to 16
// bytes at any element alignment, float packing, and how waves share rows.
#pragma once

#include "device.h"

namespace tbe {

// VE consecutive elements as they are in memory. The vector types carry the
// element's alignment only: gfx950 loads and stores 16 bytes at any such
// address, so rows of odd width take the same instructions as aligned ones.
template <typename T, int VE> struct Pack;
#define TBE_PACK(T, VE, N, A)                                              \
  template <> struct Pack<T, VE> {                                         \
    typedef uint32_t raw __attribute__((ext_vector_type(N)));              \
    typedef uint32_t mem __attribute__((ext_vector_type(N), aligned(A)));  \
  };
TBE_PACK(float, 4, 4, 4)
TBE_PACK(f16_t, 8, 4, 2)
TBE_PACK(f16_t, 4, 2, 2)
TBE_PACK(bf16_t, 8, 4, 2)
TBE_PACK(bf16_t, 4, 2, 2)
#undef TBE_PACK
template <> struct Pack<float, 8> {  // two 16-byte halves
  struct raw { Pack<float, 4>::raw h[2]; };
};
template <typename T> struct Pack<T, 1> { typedef T raw; };

template <typename T, int VE>
__device__ __forceinline__ typename Pack<T, VE>::raw load_pack(const T* p) {
  if constexpr (VE == 1) {
    return *p;
  } else if constexpr (VE == 8 && sizeof(T) == 4) {
    typename Pack<T, 8>::raw r;
    r.h[0] = load_pack<T, 4>(p);
    r.h[1] = load_pack<T, 4>(p + 4);
    return r;
  } else {
    return *reinterpret_cast<const typename Pack<T, VE>::mem*>(p);
  }
}

// Nontemporal load: data this call reads once.
template <typename T, int VE>
__device__ __forceinline__ typename Pack<T, VE>::raw load_pack_once(const T* p) {
  if constexpr (VE == 1) {
    return *p;
  } else if constexpr (VE == 8 && sizeof(T) == 4) {
    typename Pack<T, 8>::raw r;
    r.h[0] = load_pack_once<T, 4>(p);
    r.h[1] = load_pack_once<T, 4>(p + 4);
    return r;
  } else {
    return __builtin_nontemporal_load(reinterpret_cast<const typename Pack<T, VE>::mem*>(p));
  }
}

template <typename T, int VE>
__device__ __forceinline__ void store_pack(T* p, const typename Pack<T, VE>::raw& v) {
  if constexpr (VE == 1) {
    *p = v;
  } else if constexpr (VE == 8 && sizeof(T) == 4) {
    store_pack<T, 4>(p, v.h[0]);
    store_pack<T, 4>(p + 4, v.h[1]);
  } else {
    *reinterpret_cast<typename Pack<T, VE>::mem*>(p) = v;
  }
}

// Nontemporal store: results this call does not read again.
template <typename T, int VE>
__device__ __forceinline__ void store_pack_once(T* p, const typename Pack<T, VE>::raw& v) {
  if constexpr (VE == 1) {
    *p = v;
  } else if constexpr (VE == 8 && sizeof(T) == 4) {
    store_pack_once<T, 4>(p, v.h[0]);
    store_pack_once<T, 4>(p + 4, v.h[1]);
  } else {
    __builtin_nontemporal_store(v, reinterpret_cast<typename Pack<T, VE>::mem*>(p));
  }
}

template <typename T>
__device__ __forceinline__ void zero_raw(T& r) {
  r = T{};
}

template <typename T, int VE>
__device__ __forceinline__ void widen(const typename Pack<T, VE>::raw& r, float (&f)[VE]) {
  if constexpr (VE == 1) {
    f[0] = to_float(r);
  } else if constexpr (sizeof(T) == 4) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = __uint_as_float(u[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
      const uint32_t u = r[i];
      T lo, hi;
      lo.bits = (uint16_t)u;
      hi.bits = (uint16_t)(u >> 16);
      f[2 * i] = to_float(lo);
      f[2 * i + 1] = to_float(hi);
    }
  }
}

// One rounding to nearest even for 16-bit types (the hardware conversions;
// bf16 in pairs), none for float.
template <typename T>
__device__ __forceinline__ uint32_t round_pair(float a, float b) {
  if constexpr (__is_same(T, bf16_t)) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const f2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
  } else {
    return (uint32_t)f32_to_f16_bits(a) | ((uint32_t)f32_to_f16_bits(b) << 16);
  }
}

template <typename T>
__device__ __forceinline__ T round_to(float a) {
  if constexpr (sizeof(T) == 4) {
    return a;
  } else {
    T r;
    r.bits = (uint16_t)round_pair<T>(a, 0.f);
    return r;
  }
}

template <typename T, int VE>
__device__ __forceinline__ typename Pack<T, VE>::raw narrow(const float (&f)[VE]) {
  if constexpr (VE == 1) {
    return round_to<T>(f[0]);
  } else {
    typename Pack<T, VE>::raw r;
    if constexpr (sizeof(T) == 4) {
      uint32_t* u = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
      for (int i = 0; i < VE; ++i) u[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VE / 2; ++i) r[i] = round_pair<T>(f[2 * i], f[2 * i + 1]);
    }
    return r;
  }
}

// Elements per 16-byte vector, of the wider of two types.
template <typename A, typename B = A>
constexpr int pack_elems() {
  return 16 / (int)(sizeof(A) > sizeof(B) ? sizeof(A) : sizeof(B));
}

// First column of a lane's vector i (in vectors of VE columns from column 0).
// The last vector of a row is moved back to end at D, so it is whole and
// stores columns of its neighbour again, with the same values; where the output
// is also an input it must not. Needs D >= VE.
template <int VE>
__device__ __forceinline__ int32_t pack_column(int32_t i, int32_t D) {
  const int64_t c = (int64_t)i * VE;
  return (int32_t)(c + VE <= D ? c : D - VE);
}
// Columns of that vector that belong to the vector before it.
template <int VE>
__device__ __forceinline__ int32_t pack_overlap(int32_t i, int32_t D) {
  const int64_t c = (int64_t)i * VE;
  return (int32_t)(c + VE <= D ? 0 : c + VE - D);
}

__device__ __forceinline__ int wave_index() {
  return __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
}

__device__ __forceinline__ int64_t load_id(const void* ids, int idx64, int64_t i) {
  return idx64 ? static_cast<const int64_t*>(ids)[i]
               : (int64_t) static_cast<const int32_t*>(ids)[i];
}

// Work units (row, segment of the row) of a grid of waves: unit u is segment
// u % segs of row u / segs, and a wave strides over the units by the whole
// grid. The steps are formed on the host, so the loop divides nothing.
struct Units {
  int64_t rows;
  int32_t segs;
  int64_t step_rows;
  int32_t step_segs;
};

struct UnitWalk {
  int64_t row;
  int32_t seg;
  __device__ __forceinline__ UnitWalk(const Units& u, uint32_t first) {
    row = first / (uint32_t)u.segs;
    seg = (int32_t)(first % (uint32_t)u.segs);
  }
  __device__ __forceinline__ bool valid(const Units& u) const { return row < u.rows; }
  __device__ __forceinline__ void next(const Units& u) {
    row += u.step_rows;
    seg += u.step_segs;
    if (seg >= u.segs) {
      seg -= u.segs;
      ++row;
    }
  }
};

// Waves of a 256-thread workgroup grid over (rows x segs) units: at most 2^20
// workgroups (a launch may have 2^32 - 1 threads), the rest by striding.
inline Units make_units(int64_t rows, int32_t segs, unsigned* blocks, int waves_per_block = 4) {
  const int64_t cap = int64_t(1) << 20;
  const int64_t need = rows > cap * waves_per_block ? cap
                       : (rows * segs + waves_per_block - 1) / waves_per_block;
  const int64_t b = need < 1 ? 1 : (need > cap ? cap : need);
  *blocks = (unsigned)b;
  Units u;
  u.rows = rows;
  u.segs = segs;
  u.step_rows = b * waves_per_block / segs;
  u.step_segs = (int32_t)(b * waves_per_block % segs);
  return u;
}

// Sum over the 64 lanes of a wave, in every lane.
__device__ __forceinline__ float wave_sum(float x) {
  x = row16_sum(x);
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, dpp_f32<0xB1>(x));
  x = fmaxf(x, dpp_f32<0x4E>(x));
  x = fmaxf(x, dpp_f32<0x141>(x));
  x = fmaxf(x, dpp_f32<0x140>(x));
  x = fmaxf(x, __shfl_xor(x, 16));
  x = fmaxf(x, __shfl_xor(x, 32));
  return x;
}

// Calls f with a value of the element type `t` stands for.
template <typename F>
hipError_t with_type(tbe_dtype t, F f) {
  switch (t) {
    case TBE_F32: return f(float{});
    case TBE_F16: return f(f16_t{});
    default: return f(bf16_t{});
  }
}

}  // namespace tbe
