// Stable split of n keys into bins (at most 1024), the counting sort that
// orders assignments by expert and tokens by the upper part of their id.
//
// The keys are cut into at most 256 tiles of consecutive keys. split_count
// writes each tile's counts; in split_tile a 1024-thread workgroup per tile
// adds up the counts of all tiles itself (256 x bins values at most, read from
// L2 by many threads at once), which is cheaper than a launch for a scan.
// A tile is cut into 16 spans, one per wave; a wave ranks 64 keys at a time
// with one ballot per bit of the bin number, so equal keys keep their order.
// With one tile the counts come from its own histogram: one launch.
// A wave's keys of 8 rounds are loaded together and kept for the second pass:
// without that 262144 keys in 1001 bins took 14.5 us in place of 12.1. Bound by
// latency at the start and by the reading of all counts.
#pragma once

#include "lm.h"
#include "lm_device.h"

namespace tbe {

constexpr int kSplitThreads = 1024;
constexpr int kSplitWaves = kSplitThreads / kWave;

struct SplitLds {
  int32_t wave[kSplitWaves][kSplitBins];  // counts, then next place, per wave and bin
  int32_t total[kSplitBins];              // all tiles' counts of a bin
  int32_t before[kSplitBins];             // counts of the tiles before this one
  int32_t start[kSplitBins];              // first place of a bin
  int32_t sums[kSplitWaves];
};

// Exclusive scan over the 1024 threads of a workgroup (two barriers).
__device__ __forceinline__ int32_t block1024_exclusive(int32_t x, int32_t* sums) {
  const int lane = lane_id();
  const int wave = threadIdx.x / kWave;
  int32_t inc = x;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int32_t y = __shfl_up(inc, d);
    if (lane >= d) inc += y;
  }
  if (lane == kWave - 1) sums[wave] = inc;
  __syncthreads();
  int32_t base = 0;
#pragma unroll
  for (int w = 0; w < kSplitWaves; ++w) base += w < wave ? sums[w] : 0;
  __syncthreads();
  return base + inc - x;
}

// Lanes with the same `bin` as this lane, among the lanes with ok.
__device__ __forceinline__ uint64_t same_bin(uint32_t bin, bool ok, int bits) {
  uint64_t m = __ballot(ok);
  for (int b = 0; b < bits; ++b) {
    const bool bit = (bin >> b) & 1u;
    const uint64_t v = __ballot(bit);
    m &= bit ? v : ~v;
  }
  return m;
}

__device__ __forceinline__ uint64_t lanes_below() {
  return (uint64_t(1) << lane_id()) - 1;
}

constexpr int kSplitRounds = 8;  // rounds of 64 keys a wave has in registers

// A wave's keys of up to kSplitRounds rounds from j0 (key.load(j), or
// key.none() from `end` on): all loads are in flight together.
template <typename Key>
__device__ __forceinline__ void load_keys(const Key& key, int64_t j0, int64_t end, int step,
                                          typename Key::type (&k)[kSplitRounds]) {
#pragma unroll
  for (int q = 0; q < kSplitRounds; ++q) {
    const int64_t j = j0 + (int64_t)q * step + lane_id();
    k[q] = j < end ? key.load(j) : key.none();
  }
}

// counts[tile * stride + bin] of the tile this workgroup owns.
template <typename Key>
__device__ void split_count(int64_t n, SplitShape sh, int32_t bins, int32_t stride,
                            int32_t* __restrict__ counts, const Key& key) {
  __shared__ int32_t hist[kSplitBins];
  const int32_t tile = blockIdx.x;
  const int64_t a = (int64_t)tile * sh.len;
  const int64_t e = a + sh.len < n ? a + sh.len : n;
  for (int i = threadIdx.x; i < bins; i += kSplitThreads) hist[i] = 0;
  __syncthreads();
  for (int64_t j0 = a + wave_index() * kWave; j0 < e; j0 += kSplitRounds * kSplitThreads) {
    typename Key::type k[kSplitRounds];
    load_keys(key, j0, e, kSplitThreads, k);
#pragma unroll
    for (int q = 0; q < kSplitRounds; ++q)
      if (j0 + q * kSplitThreads + lane_id() < e)
        __hip_atomic_fetch_add(&hist[key.bin(k[q])], 1, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_WORKGROUP);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < stride; i += kSplitThreads)
    counts[(int64_t)tile * stride + i] = i < bins ? hist[i] : 0;
}

// Calls place(j, key, bin, p) for every key of this workgroup's tile: p is the
// place of key j in the stable order. Fills s.start (valid after the call in
// every thread).
template <typename Key, typename Place>
__device__ void split_tile(int64_t n, SplitShape sh, int32_t bins, int bits, int32_t stride,
                           const int32_t* __restrict__ counts, SplitLds& s, const Key& key,
                           Place place) {
  const int tid = threadIdx.x;
  const int wave = wave_index();
  const int lane = lane_id();
  const int32_t tile = blockIdx.x;
  // this tile's keys, a span of whole rounds of 64 per wave
  const int64_t a = (int64_t)tile * sh.len;
  const int64_t e = a + sh.len < n ? a + sh.len : n;
  const int32_t span = sh.len / kSplitWaves;
  const int64_t wa = a + (int64_t)wave * span;
  const int64_t we = wa + span < e ? wa + span : e;
  typename Key::type k[kSplitRounds];
  load_keys(key, wa, we, kWave, k);  // of a short span all, of a long one the first batch

  if (tid < bins) {
#pragma unroll
    for (int w = 0; w < kSplitWaves; ++w) s.wave[w][tid] = 0;
    s.total[tid] = s.before[tid] = 0;
  }
  __syncthreads();

  if (sh.tiles > 1) {
    // thread = (four bins, every groups-th tile): the loads of one thread do
    // not depend on each other
    const int cols = stride / 4;
    const int groups = kSplitThreads / cols;
    const int col = tid % cols, group = tid / cols;
    if (group < groups) {
      int4 tot = make_int4(0, 0, 0, 0), pre = make_int4(0, 0, 0, 0);
#pragma unroll 8
      for (int32_t t = group; t < sh.tiles; t += groups) {
        const int4 c = reinterpret_cast<const int4*>(counts + (int64_t)t * stride)[col];
        tot.x += c.x; tot.y += c.y; tot.z += c.z; tot.w += c.w;
        if (t < tile) { pre.x += c.x; pre.y += c.y; pre.z += c.z; pre.w += c.w; }
      }
      const int32_t tv[4] = {tot.x, tot.y, tot.z, tot.w};
      const int32_t pv[4] = {pre.x, pre.y, pre.z, pre.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (col * 4 + i >= bins) break;
        if (tv[i]) atomicAdd(&s.total[col * 4 + i], tv[i]);
        if (pv[i]) atomicAdd(&s.before[col * 4 + i], pv[i]);
      }
    }
  }

  for (int64_t j0 = wa; j0 < we; j0 += kSplitRounds * kWave) {
    if (j0 != wa) load_keys(key, j0, we, kWave, k);
#pragma unroll
    for (int q = 0; q < kSplitRounds; ++q)
      if (j0 + q * kWave + lane < we)
        __hip_atomic_fetch_add(&s.wave[wave][key.bin(k[q])], 1, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_WORKGROUP);
  }
  __syncthreads();

  int32_t tot = 0;
  if (tid < bins) {
    if (sh.tiles > 1) {
      tot = s.total[tid];
    } else {
#pragma unroll
      for (int w = 0; w < kSplitWaves; ++w) tot += s.wave[w][tid];
    }
  }
  const int32_t start = block1024_exclusive(tot, s.sums);
  if (tid < bins) {
    s.start[tid] = start;
    int32_t next = start + s.before[tid];
#pragma unroll
    for (int w = 0; w < kSplitWaves; ++w) {
      const int32_t c = s.wave[w][tid];
      s.wave[w][tid] = next;
      next += c;
    }
  }
  __syncthreads();

  const uint64_t below = lanes_below();
  for (int64_t j0 = wa; j0 < we; j0 += kSplitRounds * kWave) {
    if (span > kSplitRounds * kWave) load_keys(key, j0, we, kWave, k);
#pragma unroll
    for (int q = 0; q < kSplitRounds; ++q) {
      const int64_t j = j0 + q * kWave + lane;
      if (j - lane >= we) break;
      const bool ok = j < we;
      const int32_t bin = ok ? key.bin(k[q]) : 0;
      const uint64_t m = same_bin((uint32_t)bin, ok, bits);
      if (ok) {
        const int32_t p = s.wave[wave][bin] + __popcll(m & below);
        place(j, k[q], bin, p);
      }
      wave_lds_sync();  // every lane has read its bin's next place
      if (ok && (m & below) == 0) s.wave[wave][bin] += __popcll(m);
      wave_lds_sync();
    }
  }
}

}  // namespace tbe
