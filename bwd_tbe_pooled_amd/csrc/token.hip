// Token table: lookup with a scale, and its dense gradient.
//
// gW[v] = scale * sum of the gradient rows of v's tokens, all V rows written.
// The tokens are sorted by id so that no sum depends on the order in which
// workgroups run:
//   split    a stable split of the tokens by the upper part of their id into
//            up to 1023 buckets (lm_split.h)
//   bucket   a workgroup per bucket sorts it by the lower part and writes the
//            first place of every id of the table; with few tokens the
//            workgroup picks its bucket out of all ids itself, and the split
//            is not launched
//   sum      waves add up the rows of `chunk` sorted places each, a segment
//            of columns per wave; other workgroups of the launch write the
//            zero rows meanwhile
//   join     adds the partial sums of the ids with more than `chunk` tokens
// A run (one id's places) of at most `chunk` tokens is summed whole by the
// wave whose chunk it starts in, so a wave sums under 2 * chunk rows whatever
// the distribution of ids; longer runs are cut at chunk borders.
#include "block_scan.h"
#include "lm_split.h"

namespace tbe {

namespace {

// A wave per token and segment of 4 vectors a lane: 16 bytes per lane and load,
// 4 loads in flight. Bound by memory; rows that several tokens share come from
// the caches, which the nontemporal stores leave to them: 16381 of 131072 rows
// of 4096 bf16 (184 MB) in 31 us, 5.9 TB/s; with ordinary stores 43 us.
template <typename WT, typename XT, int VE, int U>
__global__ __launch_bounds__(256) void token_forward_kernel(
    const WT* __restrict__ W, int64_t ldw, const void* __restrict__ ids, int32_t idx64, int64_t V,
    int32_t D, float scale, XT* __restrict__ out, int64_t ldo, Units units) {
  using RW = typename Pack<WT, VE>::raw;
  const int32_t nv = (D + VE - 1) / VE;
  for (UnitWalk u(units, blockIdx.x * 4 + wave_index()); u.valid(units); u.next(units)) {
    const int64_t id = load_id(ids, idx64, u.row);
    const bool ok = id >= 0 && id < V;
    const WT* from = W + (ok ? id : 0) * ldw;
    XT* to = out + u.row * ldo;
    const int32_t i0 = u.seg * (U * kWave) + lane_id();
    RW v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      zero_raw(v[i]);
      if (ok && i0 + i * kWave < nv)
        v[i] = load_pack<WT, VE>(from + pack_column<VE>(i0 + i * kWave, D));
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i0 + i * kWave < nv) {
        float f[VE];
        widen<WT, VE>(v[i], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = ok ? f[e] * scale : 0.f;
        store_pack_once<XT, VE>(to + pack_column<VE>(i0 + i * kWave, D), narrow<XT, VE>(f));
      }
  }
}

// --- sort -----------------------------------------------------------------------
struct BucketOf {
  using type = int32_t;
  const void* ids;
  int32_t idx64, shift, buckets;
  int32_t V;
  __device__ __forceinline__ type none() const { return -1; }
  __device__ __forceinline__ type load(int64_t j) const {  // -1: padding
    const int64_t v = load_id(ids, idx64, j);
    return v >= 0 && v < V ? (int32_t)v : -1;
  }
  __device__ __forceinline__ int32_t bin(type v) const {
    return v >= 0 ? v >> shift : buckets;  // padding: the last bin
  }
};

__global__ __launch_bounds__(kSplitThreads) void token_count_kernel(
    BucketOf of, int64_t N, SplitShape sh, int32_t stride, int32_t* __restrict__ counts) {
  split_count(N, sh, of.buckets + 1, stride, counts, of);
}

__global__ __launch_bounds__(kSplitThreads) void token_split_kernel(
    BucketOf of, int64_t N, SplitShape sh, int bits, int32_t stride,
    const int32_t* __restrict__ counts, int32_t* __restrict__ bstart, int2* __restrict__ split) {
  __shared__ SplitLds s;
  const int32_t low = (1 << of.shift) - 1;
  split_tile(N, sh, of.buckets + 1, bits, stride, counts, s, of,
             [&](int64_t j, int32_t v, int32_t bin, int32_t p) {
               if (bin == of.buckets) return;
               split[p] = make_int2((int32_t)j, v & low);
             });
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= of.buckets; i += kSplitThreads) bstart[i] = s.start[i];
}

// Tokens a workgroup filters by itself: 4096 in 24 us (D 512) against 30 with the
// split's launches; 8192 would take as long as those.
constexpr int kFilterTokens = 4096;
constexpr int kFilterRounds = kFilterTokens / 512;
constexpr int kRounds = 8;               // rounds of 64 places a wave has in flight

// Sorts one bucket by the lower part of the id: (token, id) at the sorted
// places, the id's top bit marking runs longer than `chunk`, and off[v] of the
// bucket's ids.
// FILTER: the bucket's tokens are picked out of all ids into LDS first.
// Bound by latency: 5 us for 16 tokens a bucket; the bucket of a frequent id
// takes longest, 20 us for 11000 of 262144 tokens in one (with 8 rounds of 8
// waves in flight; 16 waves 19.6, 4 waves 33).
template <int THREADS, bool FILTER>
__global__ __launch_bounds__(THREADS) void token_bucket_kernel(
    BucketOf of, int32_t N, int32_t chunk, const int32_t* __restrict__ bstart,
    const int2* __restrict__ split, int32_t* __restrict__ off, int2* __restrict__ sorted,
    int32_t* __restrict__ listed) {
  constexpr int kWaves = THREADS / kWave;
  extern __shared__ int32_t lds[];
  int32_t* const next = lds;  // [wave][low]: counts, then the next place
  const int shift = of.shift;
  const int32_t width = 1 << shift;
  uint32_t* const is_long = reinterpret_cast<uint32_t*>(lds + (kWaves << shift));  // [low]
  int32_t* const list = lds + ((kWaves + 1) << shift);  // FILTER: token | low << 12
  __shared__ int32_t sums[2 * kWaves];
  const int tid = threadIdx.x;
  const int wave = wave_index();
  const int lane = lane_id();
  const int32_t b = blockIdx.x;
  const uint64_t below = lanes_below();
  int32_t base = 0, n = 0;
  if (b == 0 && tid < 2) listed[tid] = 0;  // the sum's lists of long runs

  if constexpr (FILTER) {
    // the wave's span of tokens: those of this bucket and of lower ones
    static_assert(THREADS == 512 || !FILTER, "a span is kFilterRounds rounds");
    const int32_t span = ((N + THREADS - 1) / THREADS) * kWave;
    const int32_t wa = wave * span;
    const int32_t we = wa + span < N ? wa + span : N;
    int32_t id[kFilterRounds];
#pragma unroll
    for (int q = 0; q < kFilterRounds; ++q) {
      const int32_t j = wa + q * kWave + lane;
      id[q] = j < we ? of.load(j) : of.none();
    }
    int32_t mine = 0, lower = 0;
#pragma unroll
    for (int q = 0; q < kFilterRounds; ++q) {
      const int32_t bin = of.bin(id[q]);
      mine += __popcll(__ballot(bin == b));
      lower += __popcll(__ballot(bin < b));
    }
    if (lane == 0) {
      sums[wave] = mine;
      sums[kWaves + wave] = lower;
    }
    __syncthreads();
    int32_t at = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      at += w < wave ? sums[w] : 0;
      n += sums[w];
      base += sums[kWaves + w];
    }
    if (mine) {
#pragma unroll
      for (int q = 0; q < kFilterRounds; ++q) {
        const bool ok = of.bin(id[q]) == b;
        const uint64_t m = __ballot(ok);
        if (ok)
          list[at + __popcll(m & below)] =
              (wa + q * kWave + lane) | ((id[q] & (width - 1)) << 12);
        at += __popcll(m);
      }
    }
  } else {
    base = bstart[b];
    n = bstart[b + 1] - base;
  }
  auto token_of = [&](int32_t i) {
    return FILTER ? make_int2(list[i] & (kFilterTokens - 1), list[i] >> 12) : split[base + i];
  };

  for (int i = tid; i < (kWaves << shift); i += THREADS) next[i] = 0;
  __syncthreads();
  const int32_t span = ((n + THREADS - 1) / THREADS) * kWave;
  const int32_t wa = wave * span;
  const int32_t we = wa + span < n ? wa + span : n;
  int2 tok[kRounds];  // (token, low) of the batch in hand, low -1 past the end
  auto load_batch = [&](int32_t i0) {
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
      const int32_t i = i0 + q * kWave + lane;
      tok[q] = i < we ? token_of(i) : make_int2(0, -1);
    }
  };
  for (int32_t i0 = wa; i0 < we; i0 += kRounds * kWave) {
    load_batch(i0);
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
      // one lane adds for all lanes of its id: a frequent id would take the
      // counter 64 times a round
      if (i0 + q * kWave >= we) break;
      const bool ok = tok[q].y >= 0;
      const uint64_t m = same_bin((uint32_t)tok[q].y, ok, shift);
      if (ok && (m & below) == 0)
        __hip_atomic_fetch_add(&next[(wave << shift) + tok[q].y], __popcll(m), __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_WORKGROUP);
    }
  }
  __syncthreads();

  // exclusive scan over the ids of the bucket; each thread has `per` of them
  const int32_t per = (width + THREADS - 1) / THREADS;
  int32_t mine = 0;
  for (int32_t q = 0; q < per; ++q) {
    const int32_t l = tid * per + q;
    if (l < width) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mine += next[(w << shift) + l];
    }
  }
  const int32_t inc = wave_inclusive_scan(mine);
  if (lane == kWave - 1) sums[wave] = inc;
  __syncthreads();
  int32_t run = base + inc - mine;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) run += w < wave ? sums[w] : 0;
  for (int32_t q = 0; q < per; ++q) {
    const int32_t l = tid * per + q;
    if (l >= width) break;
    const int32_t v = (b << shift) + l;
    if (v <= of.V) off[v] = run;
    const int32_t first = run;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int32_t c = next[(w << shift) + l];
      next[(w << shift) + l] = run;
      run += c;
    }
    is_long[l] = run - first > chunk ? 0x80000000u : 0u;
  }
  // the table's end, where it is the end of a bucket
  if (b == of.buckets - 1 && tid == 0 && (of.buckets << shift) == of.V) off[of.V] = base + n;
  __syncthreads();

  for (int32_t i0 = wa; i0 < we; i0 += kRounds * kWave) {
    if (span > kRounds * kWave) load_batch(i0);
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
      if (i0 + q * kWave >= we) break;
      const bool ok = tok[q].y >= 0;
      const int32_t l = ok ? tok[q].y : 0;
      const uint64_t m = same_bin((uint32_t)l, ok, shift);
      if (ok) {
        const int32_t p = next[(wave << shift) + l] + __popcll(m & below);
        sorted[p] = make_int2(tok[q].x, (int32_t)((uint32_t)((b << shift) + l) | is_long[l]));
      }
      wave_lds_sync();
      if (ok && (m & below) == 0) next[(wave << shift) + l] += __popcll(m);
      wave_lds_sync();
    }
  }
}

// --- sum -----------------------------------------------------------------------
constexpr int kMaxChunk = 32;      // a wave's places and the window around them fit its lanes
constexpr int kZeroVectors = 4;    // vectors of zeros per thread
constexpr int kWavePieces = 32;    // pieces of a run one wave joins alone, at most

// Runs longer than a chunk, (id, first chunk, pieces) in any order: each is joined by
// itself. list[0..capacity): up to kWavePieces pieces, list[capacity..): more.
struct LongRuns {
  int32_t* count;  // [2]
  int4* list;
  int32_t capacity;
};

// Zeros of the table's empty rows, in spans of 1024 vectors (a row taken as nz
// of them), one per workgroup: stores in the order of addresses from many short
// workgroups fill memory fastest here (1 GiB at 6.0 TB/s; with 64 KB per
// workgroup 5.5, from a grid that strides over the table 4.4). It has to stay
// short: with whole lines of a dense table instead, and the test of a vector's
// second row that this takes, the sum kernel's 1.2 GB went from 6.0 to 4.7 TB/s.
template <typename WT, int VZ>
struct EmptySpans {
  WT* gW;
  int64_t ldgw;
  int32_t V, D;

  EmptySpans(void* table, int64_t ld, const tbe_token_desc& d)
      : gW(static_cast<WT*>(table)), ldgw(ld), V((int32_t)d.V), D(d.D) {}
  unsigned blocks() const {
    const int64_t vectors = (int64_t)V * ((D + VZ - 1) / VZ);
    return (unsigned)((vectors + kSpan - 1) / kSpan);
  }
  static constexpr int kSpan = 256 * kZeroVectors;
  static constexpr int kRows = kSpan + 1;  // rows a span touches, at most

  // First row of a span, and which of its vectors the span starts with.
  __device__ __forceinline__ int64_t first_row(uint32_t block, uint32_t* rem) const {
    const uint32_t nz = (uint32_t)((D + VZ - 1) / VZ);
    const uint64_t first = (uint64_t)block * kSpan;
    const int64_t row = first >> 32 ? (int64_t)(first / nz) : (int64_t)((uint32_t)first / nz);
    *rem = (uint32_t)(first - (uint64_t)row * nz);
    return row;
  }

  // has(r): whether row row0 + r has tokens.
  template <typename Has>
  __device__ __forceinline__ void write(int64_t row0, uint32_t rem, Has has) const {
    const uint32_t nz = (uint32_t)((D + VZ - 1) / VZ);
    typename Pack<WT, VZ>::raw zero;
    zero_raw(zero);
    bool empty[kZeroVectors];
    WT* to[kZeroVectors];
#pragma unroll
    for (int i = 0; i < kZeroVectors; ++i) {
      const uint32_t o = rem + i * 256 + threadIdx.x;
      const uint32_t r = o / nz;
      const bool in = row0 + r < V;
      empty[i] = !has(in ? r : 0) && in;
      to[i] = gW + (row0 + r) * ldgw + pack_column<VZ>((int32_t)(o - r * nz), D);
    }
#pragma unroll
    for (int i = 0; i < kZeroVectors; ++i)
      if (empty[i]) store_pack<WT, VZ>(to[i], zero);
  }
};

// A wave has `chunk` (at most 32) sorted places and 64 lanes of columns. It loads
// the (token, id) of those places and of 32 after them at once, finds the
// borders of runs with ballots, and keeps 8 rows in flight; it needs nothing
// else from memory before the rows. Bound by memory: 16384 tokens into 131072 x
// 4096 bf16 (1.2 GB, most of it zeros) 198 us, 6.1 TB/s; 262144 tokens into
// 32000 x 1024 f32 (616 MB and 15% of partial rows) 122 us. With 64 places a
// wave the longest waves ended late (170 us), with 16 the partial rows grew.
//
// VE: columns per lane of the sums (16 bytes of g), VZ: of the zero rows.
template <typename WT, typename XT, int VE, int VZ>
__global__ __launch_bounds__(256) void token_sum_kernel(
    const XT* __restrict__ g, int64_t ldg, const int32_t* __restrict__ off,
    const int2* __restrict__ sorted, int32_t V, int32_t D,
    float scale, WT* __restrict__ gW, int64_t ldgw, LongRuns runs,
    float* __restrict__ parts, int64_t part_ld, int32_t chunk, Units units, uint32_t sum_blocks,
    EmptySpans<WT, VZ> empty) {
  using RX = typename Pack<XT, VE>::raw;
  if (blockIdx.x >= sum_blocks) {
    uint32_t rem;
    const int64_t row0 = empty.first_row(blockIdx.x - sum_blocks, &rem);
    empty.write(row0, rem, [&](uint32_t r) { return off[row0 + r] != off[row0 + r + 1]; });
    return;
  }
  const int lane = lane_id();
  const int32_t nv = (D + VE - 1) / VE;
  const int32_t kept = off[V];
  for (UnitWalk u(units, blockIdx.x * 4 + wave_index()); u.valid(units); u.next(units)) {
    const int64_t b64 = u.row * chunk;
    if (b64 >= kept) continue;
    const int32_t b = (int32_t)b64;
    const int32_t n = kept - b > chunk ? chunk : kept - b;
    const int32_t i = u.seg * kWave + lane;
    const bool in = i < nv;
    const int32_t col = in ? pack_column<VE>(i, D) : 0;
    const XT* gc = g + col;
    float* part = parts + (u.row * 2) * part_ld + col;

    // lane l has place b - 1 + l
    const int32_t k = b - 1 + lane;
    const bool there = k >= 0 && k < kept;
    const int32_t at = there ? k : b;
    const int32_t w = sorted[at].y, p = sorted[at].x;
    const int32_t before = __shfl_up(w, 1);
    // first places of runs among lanes 1.. (lane 0 only tells where lane 1's run began)
    const uint64_t firsts =
        __ballot(there && lane > 0 && (k == 0 || before != w)) |
        (kept - b + 1 < kWave ? uint64_t(1) << (kept - b + 1) : 0);  // the end of all places
    const uint64_t longs = __ballot(there && w < 0);
    const uint64_t mine = (uint64_t(2) << n) - 2;      // lanes 1..n
    int32_t s0 = 1, s1 = n + 1;
    bool head = false, tail = false;
    if (!(firsts & 2)) {
      if (longs & 2) head = true;                      // a piece of a long run
      else s0 = __builtin_ctzll(firsts);               // a short run: its start's chunk sums it
    }
    if (firsts & mine) {
      const int last = 63 - __builtin_clzll(firsts & mine);
      if ((longs >> last) & 1) {
        tail = true;                                   // goes on in the next chunk
      } else {
        const uint64_t after = firsts & ~((uint64_t(2) << last) - 1);
        s1 = after ? __builtin_ctzll(after) : kWave;
      }
    } else if (!head) {
      s0 = s1;
    }
    if (tail && u.seg == 0 && lane == 0) {
      // a long run starts here: into the list for one wave, or for 16, to join
      const int32_t v = sorted[b + n - 1].y & 0x7fffffff;
      const int32_t pieces = (off[v + 1] - 1) / chunk - (int32_t)u.row + 1;
      const int hot = pieces > kWavePieces;
      runs.list[hot * runs.capacity + atomicAdd(runs.count + hot, 1)] =
          make_int4(v, (int32_t)u.row, pieces, 0);
    }

    float acc[VE];
#pragma unroll
    for (int q = 0; q < VE; ++q) acc[q] = 0.f;
    constexpr int KU = 8;  // rows in flight
    for (int32_t k0 = s0; k0 < s1; k0 += KU) {
      RX r[KU];
#pragma unroll
      for (int q = 0; q < KU; ++q) {
        zero_raw(r[q]);
        if (k0 + q < s1) {
          const int32_t row = __builtin_amdgcn_readlane(p, k0 + q);
          if (in) r[q] = load_pack_once<XT, VE>(gc + (int64_t)row * ldg);
        }
      }
#pragma unroll
      for (int q = 0; q < KU; ++q) {
        if (k0 + q >= s1) break;
        float f[VE];
        widen<XT, VE>(r[q], f);
#pragma unroll
        for (int j = 0; j < VE; ++j) acc[j] += f[j];
        const bool last = k0 + q + 1 == s1;
        if (!last && !((firsts >> (k0 + q + 1)) & 1)) continue;
        // the run ends here: a whole one goes to the table, a piece of a
        // long one to this chunk's partial rows
        if (in) {
          if (head || (last && tail)) {
            store_pack<float, VE>(part + (head ? 0 : part_ld), narrow<float, VE>(acc));
          } else {
            const int32_t v = __builtin_amdgcn_readlane(w, k0 + q);
            float o[VE];
#pragma unroll
            for (int j = 0; j < VE; ++j) o[j] = acc[j] * scale;
            store_pack<WT, VE>(gW + (int64_t)v * ldgw + col, narrow<WT, VE>(o));
          }
        }
        head = false;
#pragma unroll
        for (int j = 0; j < VE; ++j) acc[j] = 0.f;
      }
    }
  }
}

// The sum of a long run's pieces p = p0, p0 + step, ... in 4 columns from d:
// its first piece is in the second partial row of chunk c, the others in the
// first rows of the chunks after it. (Partial rows are padded to float4s.)
__device__ __forceinline__ float4 sum_pieces(const float* __restrict__ parts, int64_t part_ld,
                                             int64_t c, int32_t p0, int32_t step, int32_t pieces,
                                             int64_t d) {
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int32_t p = p0; p < pieces; p += step) {
    const float4 f = *reinterpret_cast<const float4*>(
        parts + ((c + p) * 2 + (p == 0 ? 1 : 0)) * part_ld + d);
    a.x += f.x; a.y += f.y; a.z += f.z; a.w += f.w;
  }
  return a;
}

// Joins the long runs, 256 columns at a time: a wave per run of few pieces, a
// workgroup's 16 waves together on one of many. Bound by latency: 8 us for 60
// runs of up to 21 pieces of 4096 columns, 10 us for 1100 of up to 350 pieces of
// 1024 columns (a workgroup per 16 chunks, without the list: 13 and 30 us).
constexpr int kJoinWaves = 16;
constexpr int kJoinBlocks = 512;

template <typename WT>
__global__ __launch_bounds__(kJoinWaves * kWave) void token_join_kernel(
    LongRuns runs, int32_t D, float scale, WT* __restrict__ gW, int64_t ldgw,
    const float* __restrict__ parts, int64_t part_ld) {
  __shared__ float4 red[kJoinWaves][kWave];
  const int wave = wave_index();
  const int lane = lane_id();
  const int32_t panels = (D + 255) / 256;
  const int64_t few = (int64_t)runs.count[0] * panels, many = (int64_t)runs.count[1] * panels;
  for (int64_t i = blockIdx.x; i < many; i += gridDim.x) {
    const int4 run = runs.list[runs.capacity + i / panels];
    const int64_t d = (i % panels) * 256 + lane * 4;
    red[wave][lane] = d < D ? sum_pieces(parts, part_ld, run.y, wave, kJoinWaves, run.z, d)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    const int64_t col = (i % panels) * 256 + threadIdx.x;
    if (threadIdx.x < 256 && col < D) {
      float t = 0.f;
#pragma unroll
      for (int q = 0; q < kJoinWaves; ++q) t += reinterpret_cast<const float*>(red[q])[threadIdx.x];
      gW[run.x * ldgw + col] = round_to<WT>(t * scale);
    }
    __syncthreads();
  }
  // neighbouring waves in different workgroups: few units go to all CUs
  for (int64_t i = (int64_t)wave * gridDim.x + blockIdx.x; i < few; i += gridDim.x * kJoinWaves) {
    const int4 run = runs.list[i / panels];
    const int64_t d = (i % panels) * 256 + lane * 4;
    if (d >= D) continue;
    const float4 a = sum_pieces(parts, part_ld, run.y, 0, 1, run.z, d);
    const float o[4] = {a.x, a.y, a.z, a.w};
    WT* row = gW + run.x * ldgw;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (d + q < D) row[d + q] = round_to<WT>(o[q] * scale);
  }
}

// --- few tokens --------------------------------------------------------------------
// One launch without a sort. A workgroup of the first kind has one token and a
// segment of columns; the first token of an id sums the rows of all tokens of
// that id, a quarter of them per wave, the others leave. One of the second
// kind writes zeros over 1024 vectors of the table, but for rows that have a
// token. Each finds its tokens by looking at all ids: that is cheaper than the
// launches of the sort, 30 us against 40 for 777 tokens and a table of 132 MB, 6
// against 20 for 1024 tokens and 8 MB. A workgroup costs about 0.7 + 0.9 N / 1024
// ns of the whole card, the sort's launches about 17 us: both are equal where
// N (tokens) segments (768 + N) is 18 M. And a frequent id's rows are summed by
// one workgroup per segment, at 24 rows a us, which 2048 tokens bound. At 8000
// rows of 512 bf16, 2048 tokens take 9.2 us (2049, by the sort, 20.8); where all
// have one id 87 (2049: 18.8), and 512 of one id 24. The ids are on the device,
// so the host cannot choose by them.
constexpr int kFewTokens = 2048;

// IDS: ids per thread
template <typename WT, typename XT, int VE, int VZ, int IDS>
__global__ __launch_bounds__(256) void token_few_kernel(
    const XT* __restrict__ g, int64_t ldg, BucketOf of, int32_t N, int32_t D, float scale,
    WT* __restrict__ gW, int64_t ldgw, int32_t segs, uint32_t sum_blocks,
    EmptySpans<WT, VZ> empty) {
  using RX = typename Pack<XT, VE>::raw;
  constexpr int kUsedWords = (EmptySpans<WT, VZ>::kRows + 31) / 32;  // a bit per row
  __shared__ union {
    struct {
      float part[3][kWave][VE];
      int32_t token[IDS * 256];
      int32_t count[IDS * 4];
    } s;
    uint32_t used[kUsedWords];
  } l;
  const int tid = threadIdx.x, lane = lane_id(), wave = wave_index();
  int32_t id[IDS];  // of token q * 256 + tid
#pragma unroll
  for (int q = 0; q < IDS; ++q) id[q] = q * 256 + tid < N ? of.load(q * 256 + tid) : of.none();

  if (blockIdx.x >= sum_blocks) {
    uint32_t rem;
    const int64_t row0 = empty.first_row(blockIdx.x - sum_blocks, &rem);
    if (tid < kUsedWords) l.used[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < IDS; ++q) {
      const int64_t r = id[q] - row0;
      if (id[q] >= 0 && r >= 0 && r < 32 * kUsedWords) atomicOr(&l.used[r / 32], 1u << (r % 32));
    }
    __syncthreads();
    empty.write(row0, rem, [&](uint32_t r) { return (l.used[r / 32] >> (r % 32)) & 1; });
    return;
  }

  const int32_t n = (int32_t)(blockIdx.x / (uint32_t)segs), seg = (int32_t)(blockIdx.x % (uint32_t)segs);
  const int32_t v = of.load(n);
  if (v < 0) return;
  bool earlier = false;
  uint64_t mine[IDS];
#pragma unroll
  for (int q = 0; q < IDS; ++q) {
    earlier |= id[q] == v && q * 256 + tid < n;
    mine[q] = __ballot(id[q] == v);
    if (lane == 0) l.s.count[q * 4 + wave] = __popcll(mine[q]);
  }
  if (__syncthreads_or(earlier)) return;
  int32_t m = 0, at[IDS];
#pragma unroll
  for (int i = 0; i < IDS * 4; ++i) {
    if (i % 4 == wave) at[i / 4] = m;
    m += l.s.count[i];
  }
#pragma unroll
  for (int q = 0; q < IDS; ++q)
    if (id[q] == v) l.s.token[at[q] + __popcll(mine[q] & lanes_below())] = q * 256 + tid;
  __syncthreads();

  const int32_t i = seg * kWave + lane;
  const bool in = i < (D + VE - 1) / VE;
  const int32_t col = in ? pack_column<VE>(i, D) : 0;
  const int32_t each = (m + 3) / 4;
  const int32_t k1 = (wave + 1) * each < m ? (wave + 1) * each : m;
  float acc[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) acc[e] = 0.f;
  constexpr int KU = 8;  // rows in flight
  for (int32_t k0 = wave * each; k0 < k1; k0 += KU) {
    RX r[KU];
#pragma unroll
    for (int q = 0; q < KU; ++q) {
      zero_raw(r[q]);
      if (k0 + q < k1 && in) r[q] = load_pack_once<XT, VE>(g + l.s.token[k0 + q] * ldg + col);
    }
#pragma unroll
    for (int q = 0; q < KU; ++q) {
      float f[VE];
      widen<XT, VE>(r[q], f);
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[e] += f[e];
    }
  }
  if (m > 1) {
    if (wave)
#pragma unroll
      for (int e = 0; e < VE; ++e) l.s.part[wave - 1][lane][e] = acc[e];
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int w = 0; w < 3; ++w)
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[e] += l.s.part[w][lane][e];
  }
  if (wave || !in) return;
#pragma unroll
  for (int e = 0; e < VE; ++e) acc[e] *= scale;
  store_pack<WT, VE>(gW + v * ldgw + col, narrow<WT, VE>(acc));
}

template <typename WT, typename XT, typename F>
hipError_t with_width(int32_t D, F f) {
  constexpr int VE = pack_elems<WT, XT>();
  if (D >= VE) return f(std::integral_constant<int, VE>{});
  return f(std::integral_constant<int, 1>{});
}

// f(element of gW, element of g, columns per lane of the sums, of the zeros)
template <typename F>
hipError_t with_gradient_types(const tbe_token_desc& d, F f) {
  return with_type(d.wdtype, [&](auto wt) {
    return with_type(d.xdtype, [&](auto xt) {
      using std::integral_constant;
      if (d.D >= 8)
        return f(wt, xt, integral_constant<int, pack_elems<decltype(xt)>()>{},
                 integral_constant<int, pack_elems<decltype(wt)>()>{});
      return f(wt, xt, integral_constant<int, 1>{}, integral_constant<int, 1>{});
    });
  });
}

int bits_for(int32_t bins) {
  int b = 0;
  while ((1 << b) < bins) ++b;
  return b;
}

}  // namespace

TokenLayout token_layout(const tbe_token_desc& d) {
  TokenLayout L{};
  L.shift = 0;
  while (((d.V - 1) >> L.shift) + 1 > kSplitBins - 1) ++L.shift;
  L.buckets = (int32_t)(((d.V - 1) >> L.shift) + 1);
  L.filtered = d.N <= kFilterTokens;
  // 32 sorted places a wave, 16 where that leaves the chip without waves
  const int32_t vec = d.xdtype == TBE_F32 ? 4 : 8;
  const int64_t segs = (d.D + 64 * vec - 1) / (64 * vec);
  L.few = d.N <= kFewTokens && d.N * segs * (768 + d.N) <= (18 << 20);
  L.chunk = d.N * segs >= kMaxChunk * 2048 ? kMaxChunk : 16;
  L.chunks = (d.N + L.chunk - 1) / L.chunk;
  L.part_ld = ((int64_t)d.D + 3) / 4 * 4;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += (bytes + 255) & ~size_t(255);
    return a;
  };
  const size_t n8 = sizeof(int2) * (size_t)d.N;
  L.off = take(sizeof(int32_t) * ((size_t)d.V + 1));
  L.sorted = take(n8);
  if (!L.filtered) {
    L.split = take(n8);
    L.bstart = take(sizeof(int32_t) * ((size_t)L.buckets + 1));
    L.counts = take(sizeof(int32_t) * (size_t)split_shape(d.N, L.buckets + 1).tiles * split_stride(L.buckets + 1));
  }
  L.listed = take(sizeof(int4) * (1 + 2 * (size_t)L.chunks));
  L.parts = take(sizeof(float) * 2 * (size_t)L.chunks * (size_t)L.part_ld);
  L.total = at;
  return L;
}

hipError_t launch_token_forward(const tbe_token_desc& d, const void* W, int64_t ldw,
                                const void* ids, void* out, int64_t ldo, hipStream_t s) {
  return with_type(d.wdtype, [&](auto wt) {
    using WT = decltype(wt);
    return with_type(d.xdtype, [&](auto xt) {
      using XT = decltype(xt);
      return with_width<WT, XT>(d.D, [&](auto ve) {
        constexpr int VE = decltype(ve)::value;
        constexpr int U = 4;
        unsigned blocks;
        const Units u = make_units(d.N, (d.D + U * kWave * VE - 1) / (U * kWave * VE), &blocks);
        hipLaunchKernelGGL((token_forward_kernel<WT, XT, VE, U>), dim3(blocks), dim3(256), 0, s,
                           static_cast<const WT*>(W), ldw, ids, d.idx64, d.V, d.D, d.scale,
                           static_cast<XT*>(out), ldo, u);
        return hipGetLastError();
      });
    });
  });
}

hipError_t launch_token_backward(const tbe_token_desc& d, const TokenLayout& L, const void* g,
                                 int64_t ldg, const void* ids, void* gW, int64_t ldgw, void* ws,
                                 hipStream_t s) {
  char* base = static_cast<char*>(ws);
  auto at = [&](size_t o) { return reinterpret_cast<int32_t*>(base + o); };
  int32_t *off = at(L.off), *listed = at(L.listed);
  int2 *sorted = reinterpret_cast<int2*>(base + L.sorted), *split = reinterpret_cast<int2*>(base + L.split);
  const LongRuns runs{listed, reinterpret_cast<int4*>(listed + 4), (int32_t)L.chunks};
  float* parts = reinterpret_cast<float*>(base + L.parts);
  const BucketOf of{ids, d.idx64, L.shift, L.buckets, (int32_t)d.V};
  if (L.few) {
    return with_gradient_types(d, [&](auto wt, auto xt, auto ve, auto vz) {
      using WT = decltype(wt);
      using XT = decltype(xt);
      constexpr int VE = decltype(ve)::value, VZ = decltype(vz)::value;
      const int32_t segs = (d.D + kWave * VE - 1) / (kWave * VE);
      const unsigned sum_blocks = (unsigned)(d.N * segs);
      const EmptySpans<WT, VZ> empty(gW, ldgw, d);
      auto go = [&](auto ids_per_thread) {
        hipLaunchKernelGGL((token_few_kernel<WT, XT, VE, VZ, decltype(ids_per_thread)::value>),
                           dim3(sum_blocks + empty.blocks()), dim3(256), 0, s,
                           static_cast<const XT*>(g), ldg, of, (int32_t)d.N, d.D, d.scale,
                           static_cast<WT*>(gW), ldgw, segs, sum_blocks, empty);
        return hipGetLastError();
      };
      if (d.N <= 512) return go(std::integral_constant<int, 2>{});
      if (d.N <= 1024) return go(std::integral_constant<int, 4>{});
      return go(std::integral_constant<int, kFewTokens / 256>{});
    });
  }
  hipError_t e;
  if (!L.filtered) {
    const SplitShape sh = split_shape(d.N, L.buckets + 1);
    const int32_t stride = split_stride(L.buckets + 1);
    hipLaunchKernelGGL(token_count_kernel, dim3(sh.tiles), dim3(kSplitThreads), 0, s, of, d.N, sh,
                       stride, at(L.counts));
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(token_split_kernel, dim3(sh.tiles), dim3(kSplitThreads), 0, s, of, d.N, sh,
                       bits_for(L.buckets + 1), stride, at(L.counts), at(L.bstart), split);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  auto sort_buckets = [&](auto threads, auto filter) {
    constexpr int T = decltype(threads)::value;
    constexpr bool F = decltype(filter)::value;
    const size_t lds = sizeof(int32_t) * (((size_t)(T / kWave + 1) << L.shift) + (F ? (size_t)d.N : 0));
    hipLaunchKernelGGL((token_bucket_kernel<T, F>), dim3(L.buckets), dim3(T), lds, s, of,
                       (int32_t)d.N, L.chunk, at(L.bstart), split, off, sorted, listed);
  };
  using std::bool_constant;
  using std::integral_constant;
  if (L.filtered) sort_buckets(integral_constant<int, 512>{}, bool_constant<true>{});
  else sort_buckets(integral_constant<int, 512>{}, bool_constant<false>{});
  if ((e = hipGetLastError()) != hipSuccess) return e;
  e = with_gradient_types(d, [&](auto wt, auto xt, auto ve, auto vz) {
    using WT = decltype(wt);
    using XT = decltype(xt);
    constexpr int VE = decltype(ve)::value, VZ = decltype(vz)::value;
    unsigned sum_blocks = 0;
    const Units u = make_units(L.chunks, (d.D + kWave * VE - 1) / (kWave * VE), &sum_blocks);
    const EmptySpans<WT, VZ> empty(gW, ldgw, d);
    hipLaunchKernelGGL((token_sum_kernel<WT, XT, VE, VZ>), dim3(sum_blocks + empty.blocks()),
                       dim3(256), 0, s, static_cast<const XT*>(g), ldg, off, sorted, (int32_t)d.V,
                       d.D, d.scale, static_cast<WT*>(gW), ldgw, runs, parts, L.part_ld, L.chunk,
                       u, sum_blocks, empty);
    return hipGetLastError();
  });
  if (e != hipSuccess || L.chunks < 2) return e;
  return with_type(d.wdtype, [&](auto wt) {
    using WT = decltype(wt);
    hipLaunchKernelGGL(token_join_kernel<WT>, dim3(kJoinBlocks), dim3(kJoinWaves * kWave), 0, s,
                       runs, d.D, d.scale, static_cast<WT*>(gW), ldgw, parts, L.part_ld);
    return hipGetLastError();
  });
}

}  // namespace tbe
