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
// then holds four neighbouring columns of one row of C from each fragment; lanes
// exchange half of two fragments' for eight neighbouring ones (eight()).
#pragma once

#include "lm.h"
#include "lm_device.h"

namespace tbe {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStepBytes = 128;   // of k in one step
// Every operand's area in LDS begins at a multiple of the longest row of Across: frag()
// finds columns by exclusive or with whole addresses.
constexpr int kLdsUnit = 512;

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

// The thread's index, unknown to the compiler from here on: what is formed from it is
// formed here, and holds no registers through the products before.
__device__ __forceinline__ int thread_again() {
  int t = (int)threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// Byte offset of a piece in LDS. Along: row r, piece c of 8.
__device__ __forceinline__ uint32_t along_at(int r, int c) {
  return (uint32_t)(r * kStepBytes + ((c ^ ((r >> 1) & 7)) << 4));
}
// Across: row k, byte b of BYTES; 32-byte units are permuted: by k mod 4 and k / 8
// for 16 bits, whose transposing reads take four rows and the four 8 further on at
// a time; in pairs by k / 4 for float32, where the four rows of one read are 4 apart.
template <typename T, int BYTES>
__device__ __forceinline__ uint32_t across_at(int k, int b) {
  const int f = sizeof(T) == 2 ? (k & 3) | ((k >> 1) & 4) : ((k >> 2) & 3) << 1;
  return (uint32_t)(k * BYTES + ((((b >> 5) ^ f) & (BYTES / 32 - 1)) << 5) + (b & 31));
}

// Eight neighbouring columns of a row of C from two fragments of 16 columns: lanes of
// even sixteens take the first fragment's, the others the second's, of the 16 columns
// the half that (lane / 32) says.
__device__ __forceinline__ void eight(const f32x4& p, const f32x4& q, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(p[j]), __float_as_uint(q[j]), false, false);
    f[j] = __uint_as_float(r[0]);
    f[j + 4] = __uint_as_float(r[1]);
  }
}
__device__ __forceinline__ int eight_at(int lane) { return (lane & 16) + (lane & 32) / 4; }

// One operand's pieces of a step, from memory to LDS. ROWS: of the tile, NT:
// threads. DIRECT: every piece lies in its matrix whole and aligned, and goes to
// LDS without a register in between; otherwise it passes through registers, where
// elements outside become zeros one by one. SPLIT: the second half of the rows is
// another matrix's.
template <typename T, Layout L, int ROWS, int NT, bool DIRECT, bool SPLIT = false>
struct Operand {
  static constexpr int VE = 16 / (int)sizeof(T);
  static constexpr int BK = kStepBytes / (int)sizeof(T);
  static constexpr int BYTES = ROWS * (int)sizeof(T);        // of a row of Across
  static constexpr int PER = BYTES / 16;                     // its pieces
  static constexpr int PIECES = ROWS * (kStepBytes / 16) / NT;
  static constexpr int READS = L == Along ? 1 : sizeof(T) == 2 ? 2 : 4;   // of LDS, for a fragment
  static_assert(PIECES * NT * 16 == ROWS * kStepBytes, "whole pieces per thread");
  static_assert(L == Along || (kLdsUnit % BYTES == 0 && (ROWS * kStepBytes) % kLdsUnit == 0), "areas of whole rows");
  int32_t limit;     // Across: columns behind the tile's start
  int32_t left;      // elements of k not loaded yet
  int64_t step;      // elements from one step to the next
  // through registers
  const T* p[DIRECT ? 1 : PIECES];
  uint4 r[DIRECT ? 1 : PIECES];
  // direct
  const T* base[1 + SPLIT];
  uint32_t off[DIRECT ? PIECES : 1];

  // Piece i of this thread: row (of the tile, or of k) and column in pieces. Direct
  // pieces are written in the order of threads, so it is the source that is permuted.
  static __device__ __forceinline__ void place(int thread, int i, int& row, int& col) {
    const int at = thread + i * NT;
    if constexpr (L == Along) {
      row = at / 8;
      col = DIRECT ? (at % 8) ^ ((row >> 1) & 7) : at % 8;
    } else {
      row = at / PER;
      col = at % PER;
      if (DIRECT) col = (int)(across_at<T, BYTES>(row, col * 16) % BYTES) / 16;
    }
  }

  // row(i): address of row i of the tile. Along, rows from `rows` on repeat the
  // last one (their products are not stored); Across, the tile has `rows` columns.
  // first: an address at or before every piece's; second: of the second matrix's.
  template <typename Row>
  __device__ __forceinline__ void start(int32_t rows, int64_t ld, int32_t K, Row row, const T* first,
                                        const T* second = nullptr) {
    limit = rows;
    left = K;
    base[0] = first;
    if constexpr (SPLIT) base[1] = second;
    step = L == Along ? BK : BK * ld;
    const int thread = thread_again();
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      int q, c;
      place(thread, i, q, c);
      const T* from = L == Along ? row(q) + c * VE : row(0) + (int64_t)q * ld + c * VE;
      if constexpr (DIRECT) {
        off[i] = (uint32_t)((from - (SPLIT && i >= PIECES / 2 ? second : first)) * (int64_t)sizeof(T));
        if (L == Across && c * VE >= rows) off[i] = kOutside;
      } else {
        p[i] = from;
      }
    }
  }

  // Direct: the next step's pieces on their way to `lds`, zeros outside. No register
  // is written, so the compiler needs no part in waiting for them: multiply does.
  static constexpr uint32_t kOutside = 0x80000000u;
  __device__ __forceinline__ void fetch(uint32_t lds) {
    typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
    i32x4 rsrc[1 + SPLIT];
#pragma unroll
    for (int j = 0; j <= SPLIT; ++j) {
      const uint64_t at = reinterpret_cast<uint64_t>(base[j]);
      rsrc[j] = {__builtin_amdgcn_readfirstlane((int)at), __builtin_amdgcn_readfirstlane((int)(at >> 32) & 0xffff),
                 (int)kOutside, 0x00020000};
      base[j] += step;
    }
    const uint32_t to = __builtin_amdgcn_readfirstlane(lds + wave_index() * (kWave * 16));
    auto one = [&](int i, uint32_t from) {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // m0 is reserved: the compiler keeps nothing in it
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                   :: "s"(to + i * (NT * 16)), "v"(from), "s"(rsrc[SPLIT && i >= PIECES / 2 ? 1 : 0]) : "m0");
#pragma clang diagnostic pop
    };
    if (left >= BK) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) one(i, off[i]);
    } else {
      const int thread = thread_again();
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        int q, c;
        place(thread, i, q, c);
        one(i, (L == Along ? c * VE : q) >= left ? kOutside : off[i]);
      }
    }
    left -= BK;
  }

  // Through registers: loads the next step's pieces; zeros outside.
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      int q, c;
      place((int)threadIdx.x, i, q, c);
      // elements of the piece that exist
      const int n = L == Along ? left - c * VE : q < left ? limit - c * VE : 0;
      r[i] = make_uint4(0, 0, 0, 0);
      if (n >= VE) {
        r[i] = __builtin_bit_cast(uint4, load_pack<T, VE>(p[i]));
      } else if (n > 0) {
        T e[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) e[j] = j < n ? p[i][j] : T{};
        r[i] = __builtin_bit_cast(uint4, e);
      }
      p[i] += step;
    }
    left -= BK;
  }
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      int q, c;
      place((int)threadIdx.x, i, q, c);
      *reinterpret_cast<uint4*>(lds + (L == Along ? along_at(q, c) : across_at<T, BYTES>(q, c * 16))) = r[i];
    }
  }

  // Where a lane reads its part of rows: of row lane % 16, and of half step s (64
  // bytes of k) the quarter lane / 16; other rows differ by a known number. (Unknown
  // to the compiler, which would otherwise keep an address for each fragment in
  // registers that the products need.)
  typedef __attribute__((address_space(3))) const char* lds_ptr;
  static __device__ __forceinline__ uint32_t lane_at(const char* lds, int s) {
    const int lane = lane_id();
    uint32_t at;
    if constexpr (L == Along) at = along_at(lane % 16, s * 4 + lane / 16);
    else if constexpr (sizeof(T) == 2)   // of 16 lanes, lane i asks for row i / 4, columns i % 4 * 4 on; it gets column i
      at = across_at<T, BYTES>(s * 32 + lane / 16 * 8 + lane % 16 / 4, lane % 4 * 8);
    else at = across_at<T, BYTES>(s * 16 + lane / 16 * 4, lane % 16 * 4);
    at += (uint32_t)(uintptr_t)(lds_ptr)lds;
    if constexpr (L == Across) asm volatile("" : "+v"(at));
    return at;
  }
  // A lane's part of the 16 rows from `row`.
  static __device__ __forceinline__ uint4 frag(uint32_t at, int row) {
    if constexpr (L == Along) {
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) const u32x4* ptr;
      return __builtin_bit_cast(uint4, *(ptr)(uintptr_t)(at + row * kStepBytes));
    } else {
      at ^= row * (int)sizeof(T);   // (units are permuted by the same pattern in all columns; kLdsUnit)
      if constexpr (sizeof(T) == 2) {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4* ptr;
        union { s16x4 h[2]; uint4 u; } v;
        v.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(uintptr_t)at);
        v.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(uintptr_t)(at + 4 * BYTES));
        return v.u;
      } else {
        typedef __attribute__((address_space(3))) const uint32_t* ptr;
        const ptr p = (ptr)(uintptr_t)at;
        return make_uint4(p[0], p[BYTES / 4], p[BYTES / 2], p[3 * BYTES / 4]);
      }
    }
  }
};

// Shape of a tile: WM x WN waves of (16 MF) x (16 NF) each.
template <int WM_, int WN_, int MF_, int NF_>
struct Shape {
  static constexpr int WM = WM_, WN = WN_, MF = MF_, NF = NF_;
  static constexpr int BM = WM * MF * 16, BN = WN * NF * 16, NT = WM * WN * kWave;
  static constexpr int AREA = (BM + BN) * kStepBytes;   // of LDS for one step
  static_assert(BM * kStepBytes % kLdsUnit == 0 && AREA % kLdsUnit == 0, "operands' areas at whole units");
};

// A wave's fragments of half a step.
template <class S>
struct Frags {
  uint4 a[S::MF], b[S::NF];
  template <class A, class B, typename RowB>
  __device__ __forceinline__ void read(const char* lds, int s, RowB row_b) {
    const int wm = wave_index() / S::WN;
    const uint32_t at_a = A::lane_at(lds, s), at_b = B::lane_at(lds + S::BM * kStepBytes, s);
#pragma unroll
    for (int j = 0; j < S::NF; ++j) b[j] = B::frag(at_b, row_b(j));
#pragma unroll
    for (int i = 0; i < S::MF; ++i) a[i] = A::frag(at_a, (wm * S::MF + i) * 16);
  }
  template <typename T>
  __device__ __forceinline__ void mul(f32x4 (&acc)[S::MF][S::NF]) const {
#pragma unroll
    for (int i = 0; i < S::MF; ++i)
#pragma unroll
      for (int j = 0; j < S::NF; ++j) acc[i][j] = Mma<T>::mul(b[j], a[i], acc[i][j]);
  }
};

// Asks the scheduler for READS reads of LDS spread over PRODUCTS products.
template <int READS, int PRODUCTS>
__device__ __forceinline__ void interleave() {
  constexpr int EACH = PRODUCTS / READS;
#pragma unroll
  for (int i = 0; i < READS; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, EACH, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, PRODUCTS - READS * EACH, 0);
}

// The products of a workgroup's tiles, one after the other.
//
// Direct: behind the barrier of step i its data are in one area of LDS and no wave
// reads the other any more, so step i + 1 is asked of memory into that. A wave then
// multiplies the second half of step i - 1, which it has in registers, while it reads
// the first half of step i, and so on: loads, reads of LDS and products always have
// each other to run beside. What is done with a tile's result runs while the next
// tile's first step is on its way (`next`).
template <typename T, class S, bool DIRECT, class A, class B>
struct Walk {
  char* lds;
  uint32_t area = 0;   // of the next step
  int later = 0;       // loads and stores this wave is sure to have made after the fetch of a tile's first step
  A a;
  B b;

  // All but the LATER last loads and stores of every wave have been made, and its reads
  // of LDS. (They are counted in the order in which they were issued.)
  template <int LATER>
  __device__ __forceinline__ void arrived() const {
    typedef __attribute__((address_space(3))) char* lds_ptr;
    asm volatile("s_waitcnt vmcnt(%1) lgkmcnt(0)\n\ts_barrier"
                 :: "s"((uint32_t)(uintptr_t)(lds_ptr)lds), "n"(LATER) : "memory");
  }
  // The same for a tile's first step, behind which the stores of the tile before stand.
  __device__ __forceinline__ void first_arrived() const {
    if (later >= 48) arrived<48>();
    else if (later >= 24) arrived<24>();
    else if (later >= 16) arrived<16>();
    else if (later >= 8) arrived<8>();
    else arrived<0>();
  }
  __device__ __forceinline__ void fetch() {
    if constexpr (DIRECT) {
      typedef __attribute__((address_space(3))) char* lds_ptr;
      const uint32_t to = (uint32_t)(uintptr_t)(lds_ptr)lds + area;
      a.fetch(to);
      b.fetch(to + S::BM * kStepBytes);
      area ^= S::AREA;
    }
  }

  // acc += the product over `steps` steps of the operands as they are and `more` after
  // turn(). row_b(nf): first of the 16 rows of B's tile that fragment nf of this wave
  // takes. next(): sets the operands to the next tile and fetches its first step.
  // The first step of this tile has been fetched.
  template <typename RowB, typename Turn, typename Next>
  __device__ __forceinline__ void multiply(f32x4 (&acc)[S::MF][S::NF], int steps, int more, RowB row_b,
                                           Turn turn, Next next) {
    const int all = steps + more;
    if constexpr (DIRECT) {
      constexpr int kReads = S::MF * A::READS + S::NF * B::READS;
      constexpr int kProducts = S::MF * S::NF * (sizeof(T) == 4 ? 4 : 1);
      if (all == 0) return next();
      Frags<S> even, odd;
      const char* now = lds + (area ^ S::AREA);
      first_arrived();
      if (1 == steps && more > 0) turn();
      if (all > 1) fetch();
      even.template read<A, B>(now, 0, row_b);
      odd.template read<A, B>(now, 1, row_b);
      even.template mul<T>(acc);
      for (int i = 1; i < all; ++i) {
        now = lds + (area ^ S::AREA);
        arrived<0>();
        if (i + 1 == steps && more > 0) turn();
        if (i + 1 < all) fetch();
        even.template read<A, B>(now, 0, row_b);
        odd.template mul<T>(acc);
        interleave<kReads, kProducts>();
        odd.template read<A, B>(now, 1, row_b);
        even.template mul<T>(acc);
        interleave<kReads, kProducts>();
      }
      odd.template mul<T>(acc);
      next();
    } else {
      auto load = [&](int i) {
        if (i == steps && more > 0) turn();
        a.load();
        b.load();
      };
      if (all > 0) {
        load(0);
        __syncthreads();   // the last tile's readers are done
        a.store(lds);
        b.store(lds + S::BM * kStepBytes);
        __syncthreads();
      }
      for (int i = 0; i < all; ++i) {
        const char* now = lds + (i & 1) * S::AREA;
        if (i + 1 < all) load(i + 1);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          Frags<S> f;
          f.template read<A, B>(now, s, row_b);
          f.template mul<T>(acc);
        }
        if (i + 1 < all) {
          char* then = lds + (~i & 1) * S::AREA;
          a.store(then);
          b.store(then + S::BM * kStepBytes);
        }
        __syncthreads();
      }
      next();
    }
  }
};

// The experts' rows, from the offsets: each is at least its predecessor and in
// [0, M], whatever the memory holds. In LDS, once a workgroup.
struct Spans {
  static constexpr int kMost = 1024;
  int32_t first[kMost];   // of expert e; behind the last expert's
  int32_t upto[kMost];    // blocks of rows (or another number) of the experts up to e

  // By every thread of the workgroup. number(rows): of an expert, >= 0.
  template <typename Number>
  __device__ __forceinline__ void fill(const int32_t* __restrict__ offsets, int32_t E, int32_t M, Number number) {
    if (wave_index() == 0) {
      int32_t low = 0, blocks = 0;
      for (int32_t e0 = 0; e0 <= E; e0 += kWave) {
        const int32_t e = e0 + lane_id();
        int32_t a = e <= E ? min(max(offsets[e], 0), M) : 0;
        int32_t z = e < E ? min(max(offsets[e + 1], 0), M) : 0;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
          const int32_t y = __shfl_up(a, d);
          if (lane_id() >= d) a = max(a, y);
        }
        a = max(a, low);
        z = max(a, z);
        int32_t n = e < E ? number(z - a) : 0;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
          const int32_t y = __shfl_up(n, d);
          if (lane_id() >= d) n += y;
        }
        n += blocks;
        if (e <= E) {
          first[e] = a;
          upto[e] = n;
        }
        low = __builtin_amdgcn_readlane(z, kWave - 1);
        blocks = __builtin_amdgcn_readlane(n, kWave - 1);
      }
    }
    __syncthreads();
  }

  // The expert of number `want` of all experts': the first whose numbers reach behind it.
  // Found by 64 lanes in two looks. Uniform over the wave; there is one.
  __device__ __forceinline__ int32_t expert_of(int32_t want, int32_t E) const {
    const int32_t step = (E + kWave - 1) / kWave;
    const int32_t i = min((lane_id() + 1) * step, E) - 1;
    const int32_t e0 = (__ffsll((unsigned long long)__ballot(upto[i] > want)) - 1) * step;
    const int32_t j = min(e0 + lane_id(), E - 1);
    return e0 + __ffsll((unsigned long long)__ballot(upto[j] > want)) - 1;
  }
};

// First row of expert e, as Spans has it, by one wave.
__device__ __forceinline__ int32_t first_row(const int32_t* __restrict__ offsets, int32_t e, int32_t M) {
  int32_t x = 0;
  for (int32_t i = lane_id(); i <= e; i += kWave) x = max(x, offsets[i]);
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) x = max(x, __shfl_xor(x, d));
  return min(__builtin_amdgcn_readfirstlane(x), M);
}

}  // namespace tbe
