// Tiles of the experts' matrix products on the matrix cores.
//
// A product is C[m, n] = sum over k of A[m, k] B[n, k]. Its operands come in two
// layouts: rows with k along them (Along), or k as the row (Across: the matrix
// is read as it lies and transposed on the way from LDS to the registers). A
// workgroup owns a tile of C and walks over k in steps of 128 bytes (64 elements
// of 16 bits, 32 of float32); two areas of LDS take turns, so one barrier a step
// is enough and the next step's loads are in flight during a step's products.
//
// In LDS a 16-byte piece stands at a place permuted by its row, so that the
// lanes of one read meet different banks. The wave multiplies B by A: a lane
// then holds four neighbouring columns of one row of C.
#pragma once

#include "lm.h"
#include "lm_device.h"

namespace tbe {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStepBytes = 128;   // of k in one step

template <typename T> struct Mma;
template <> struct Mma<bf16_t> {
  typedef __bf16 frag __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ f32x4 mul(uint4 b, uint4 a, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(frag, b),
                                                   __builtin_bit_cast(frag, a), c, 0, 0, 0);
  }
};
template <> struct Mma<f16_t> {
  typedef _Float16 frag __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ f32x4 mul(uint4 b, uint4 a, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag, b),
                                                  __builtin_bit_cast(frag, a), c, 0, 0, 0);
  }
};
template <> struct Mma<float> {   // a lane's four elements of k: one product each
  static __device__ __forceinline__ f32x4 mul(uint4 b, uint4 a, f32x4 c) {
    const f32x4 fb = __builtin_bit_cast(f32x4, b), fa = __builtin_bit_cast(f32x4, a);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(fb[j], fa[j], c, 0, 0, 0);
    return c;
  }
};

enum Layout { Along, Across };

// Byte offset of a piece in LDS. Along: row r, piece c of 8.
__device__ __forceinline__ uint32_t along_at(int r, int c) {
  return (uint32_t)(r * kStepBytes + ((c ^ (r & 7)) << 4));
}
// Across: row k, byte b of BYTES; 32-byte units are permuted: by k mod 4 and k / 8
// for 16 bits, whose transposing reads take four rows and two rows 8 apart at a
// time; in pairs by k / 4 for float32, where the four rows of one read are 4 apart.
template <typename T, int BYTES>
__device__ __forceinline__ uint32_t across_at(int k, int b) {
  const int f = sizeof(T) == 2 ? (k & 3) | ((k >> 1) & 4) : ((k >> 2) & 3) << 1;
  return (uint32_t)(k * BYTES + ((((b >> 5) ^ f) & (BYTES / 32 - 1)) << 5) + (b & 31));
}

// One operand's pieces of a step, from memory through registers to LDS. ROWS: of
// the tile, NT: threads; VEC: pieces lie in the matrix whole or not at all.
template <typename T, Layout L, int ROWS, int NT, bool VEC>
struct Operand {
  static constexpr int VE = 16 / (int)sizeof(T);
  static constexpr int BK = kStepBytes / (int)sizeof(T);
  static constexpr int BYTES = ROWS * (int)sizeof(T);        // of a row of Across
  static constexpr int PIECES = ROWS * (kStepBytes / 16) / NT;
  static_assert(PIECES * NT * 16 == ROWS * kStepBytes, "whole pieces per thread");
  const T* p[PIECES];
  int64_t step;      // elements from one step to the next
  int32_t limit;     // Across: columns behind p's tile start
  uint4 r[PIECES];

  // row(i): address of row i of the tile. Along, rows from `rows` on repeat the
  // last one (their products are not stored); Across, the tile has `rows` columns.
  template <typename Row>
  __device__ __forceinline__ void start(int32_t rows, int64_t ld, Row row) {
    limit = rows;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int at = (int)threadIdx.x + i * NT;
      if constexpr (L == Along) {
        const int q = at / 8;
        p[i] = row(q) + (at % 8) * VE;
      } else {
        constexpr int PER = BYTES / 16;
        p[i] = row(0) + (int64_t)(at / PER) * ld + (at % PER) * VE;
      }
    }
    step = L == Along ? BK : BK * ld;
  }

  // Loads the pieces of the step at k of K; zeros outside.
  __device__ __forceinline__ void load(int32_t k, int32_t K) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int at = (int)threadIdx.x + i * NT;
      int n;   // elements of the piece that exist
      if constexpr (L == Along) {
        n = K - k - (at % 8) * VE;
      } else {
        constexpr int PER = BYTES / 16;
        n = k + at / PER < K ? limit - (at % PER) * VE : 0;
      }
      r[i] = make_uint4(0, 0, 0, 0);
      if (n >= VE) {
        r[i] = __builtin_bit_cast(uint4, load_pack<T, VE>(p[i]));
      } else if (!VEC && n > 0) {
        T e[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) e[j] = j < n ? p[i][j] : T{};
        r[i] = __builtin_bit_cast(uint4, e);
      }
      p[i] += step;
    }
  }

  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int at = (int)threadIdx.x + i * NT;
      uint32_t to;
      if constexpr (L == Along) {
        to = along_at(at / 8, at % 8);
      } else {
        constexpr int PER = BYTES / 16;
        to = across_at<T, BYTES>(at / PER, (at % PER) * 16);
      }
      *reinterpret_cast<uint4*>(lds + to) = r[i];
    }
  }

  // A lane's part of 16 rows of the tile from `row`: row + lane % 16, and of half
  // step s (64 bytes of k) the quarter lane / 16.
  static __device__ __forceinline__ uint4 frag(const char* lds, int row, int s) {
    const int lane = lane_id();
    if constexpr (L == Along) {
      return *reinterpret_cast<const uint4*>(lds + along_at(row + lane % 16, s * 4 + lane / 16));
    } else if constexpr (sizeof(T) == 2) {
      // of 16 lanes, lane i asks for row i / 4, columns i % 4 * 4 on; it gets column i
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      const int k = s * 32 + lane / 16 * 8 + lane % 16 / 4;
      const int b = (row + lane % 4 * 4) * 2;
      union { s16x4 h[2]; uint4 u; } v;
      v.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(lds + across_at<T, BYTES>(k, b)));
      v.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(lds + across_at<T, BYTES>(k + 4, b)));
      return v.u;
    } else {
      uint32_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = *reinterpret_cast<const uint32_t*>(
            lds + across_at<T, BYTES>(s * 16 + lane / 16 * 4 + j, (row + lane % 16) * 4));
      return make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
};

// Shape of a tile: WM x WN waves of (16 MF) x (16 NF) each.
template <int WM_, int WN_, int MF_, int NF_>
struct Shape {
  static constexpr int WM = WM_, WN = WN_, MF = MF_, NF = NF_;
  static constexpr int BM = WM * MF * 16, BN = WN * NF * 16, NT = WM * WN * kWave;
  static constexpr int AREA = (BM + BN) * kStepBytes;   // of LDS for one step
};

// acc += the product over K. `row_b(nf)`: first of the 16 rows of B's tile that
// fragment nf of this wave takes.
template <typename T, class S, class A, class B, typename RowB>
__device__ __forceinline__ void multiply(f32x4 (&acc)[S::MF][S::NF], A& a, B& b, int32_t K,
                                         char* lds, RowB row_b) {
  constexpr int BK = kStepBytes / (int)sizeof(T);
  const int steps = (K + BK - 1) / BK;
  if (steps == 0) return;
  const int wm = wave_index() / S::WN;
  a.load(0, K);
  b.load(0, K);
  __syncthreads();   // the areas' last readers are done
  a.store(lds);
  b.store(lds + S::BM * kStepBytes);
  __syncthreads();
  for (int i = 0; i < steps; ++i) {
    const char* now = lds + (i & 1) * S::AREA;
    if (i + 1 < steps) {
      a.load((i + 1) * BK, K);
      b.load((i + 1) * BK, K);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint4 fa[S::MF], fb[S::NF];
#pragma unroll
      for (int i = 0; i < S::MF; ++i) fa[i] = A::frag(now, (wm * S::MF + i) * 16, s);
#pragma unroll
      for (int j = 0; j < S::NF; ++j) fb[j] = B::frag(now + S::BM * kStepBytes, row_b(j), s);
#pragma unroll
      for (int i = 0; i < S::MF; ++i)
#pragma unroll
        for (int j = 0; j < S::NF; ++j) acc[i][j] = Mma<T>::mul(fb[j], fa[i], acc[i][j]);
    }
    if (i + 1 < steps) {
      char* next = lds + (~i & 1) * S::AREA;
      a.store(next);
      b.store(next + S::BM * kStepBytes);
    }
    __syncthreads();
  }
}

// The experts' rows, from the offsets: each is at least its predecessor and in
// [0, M], whatever the memory holds. Uniform over the wave.
struct Span {
  int32_t e, first, end;   // expert, its rows
  int32_t place;           // find: which of the expert's `tiles` blocks of rows times `nt`
  int32_t tiles;
};

__device__ __forceinline__ int32_t wave_scan_max(int32_t x) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int32_t y = __shfl_up(x, d);
    if (lane_id() >= d) x = max(x, y);
  }
  return x;
}
__device__ __forceinline__ int32_t wave_scan_sum(int32_t x) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int32_t y = __shfl_up(x, d);
    if (lane_id() >= d) x += y;
  }
  return x;
}

// Block `tile` of the experts' rows in blocks of BM, nt of them side by side: an
// expert's blocks are neighbours. False behind the last.
template <int BM>
__device__ __forceinline__ bool find_block(const int32_t* __restrict__ offsets, int32_t E, int32_t M,
                                           int32_t nt, int32_t tile, Span& s) {
  const int32_t want = tile / nt;
  int32_t before = 0, low = 0;
  for (int32_t e0 = 0; e0 < E; e0 += kWave) {
    const int32_t e = e0 + lane_id();
    int32_t a = e <= E ? min(max(offsets[min(e, E)], 0), M) : 0;
    int32_t z = e < E ? min(max(offsets[e + 1], 0), M) : 0;
    a = max(wave_scan_max(a), low);
    z = max(a, z);
    const int32_t tiles = e < E ? (z - a + BM - 1) / BM : 0;
    const int32_t upto = before + wave_scan_sum(tiles);
    const uint64_t hit = __ballot(upto > want);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      s.e = e0 + l;
      s.first = __builtin_amdgcn_readlane(a, l);
      s.end = __builtin_amdgcn_readlane(z, l);
      s.tiles = __builtin_amdgcn_readlane(tiles, l);
      s.place = tile - (__builtin_amdgcn_readlane(upto, l) - s.tiles) * nt;
      return true;
    }
    before = __builtin_amdgcn_readlane(upto, kWave - 1);
    low = __builtin_amdgcn_readlane(z, kWave - 1);
  }
  return false;
}

// Rows of expert e.
__device__ __forceinline__ void expert_rows(const int32_t* __restrict__ offsets, int32_t e, int32_t M,
                                            Span& s) {
  int32_t low = 0;
  for (int32_t e0 = 0; e0 <= e; e0 += kWave) {
    const int32_t i = e0 + lane_id();
    low = max(low, i <= e ? min(max(offsets[i], 0), M) : 0);
  }
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) low = max(low, __shfl_xor(low, d));
  s.e = e;
  s.first = __builtin_amdgcn_readfirstlane(low);
  s.end = max(s.first, min(max(offsets[e + 1], 0), M));
}

}  // namespace tbe
