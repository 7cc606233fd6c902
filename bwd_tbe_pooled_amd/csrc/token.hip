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
  const void* ids;
  int32_t idx64, shift, buckets;
  int64_t V;
  __device__ __forceinline__ int32_t operator()(int64_t j) const {
    const int64_t v = load_id(ids, idx64, j);
    return v >= 0 && v < V ? (int32_t)(v >> shift) : buckets;  // padding: the last bin
  }
};

__global__ __launch_bounds__(kSplitThreads) void token_count_kernel(
    BucketOf of, int64_t N, SplitShape sh, int32_t stride, int32_t* __restrict__ counts) {
  split_count(N, sh, of.buckets + 1, stride, counts, of);
}

__global__ __launch_bounds__(kSplitThreads) void token_split_kernel(
    BucketOf of, int64_t N, SplitShape sh, int bits, int32_t stride,
    const int32_t* __restrict__ counts, int32_t* __restrict__ bstart, int32_t* __restrict__ lpos,
    int32_t* __restrict__ llow) {
  __shared__ SplitLds s;
  const int32_t low = (1 << of.shift) - 1;
  split_tile(N, sh, of.buckets + 1, bits, stride, counts, s, of,
             [&](int64_t j, int32_t bin, int32_t p) {
               if (bin == of.buckets) return;
               lpos[p] = (int32_t)j;
               llow[p] = (int32_t)load_id(of.ids, of.idx64, j) & low;
             });
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= of.buckets; i += kSplitThreads) bstart[i] = s.start[i];
}

constexpr int kBucketThreads = 512;
constexpr int kBucketWaves = kBucketThreads / kWave;
constexpr int kFilterTokens = 8192;      // tokens a workgroup filters by itself

// Sorts one bucket by the lower part of the id: sorted places pos/sid, and
// off[v] of the bucket's ids. FILTER: the bucket's tokens are picked out of
// all ids into LDS first.
template <bool FILTER>
__global__ __launch_bounds__(kBucketThreads) void token_bucket_kernel(
    BucketOf of, int32_t N, const int32_t* __restrict__ bstart, const int32_t* __restrict__ lpos,
    const int32_t* __restrict__ llow, int32_t* __restrict__ off, int32_t* __restrict__ pos,
    int32_t* __restrict__ sid) {
  extern __shared__ int32_t lds[];
  int32_t* const next = lds;  // [wave][low]: counts, then the next place
  int32_t* const list = lds + (kBucketWaves << of.shift);  // FILTER: pos | low << 13
  __shared__ int32_t sums[2 * kBucketWaves];
  const int tid = threadIdx.x;
  const int wave = wave_index();
  const int lane = lane_id();
  const int32_t b = blockIdx.x;
  const int shift = of.shift;
  const int32_t width = 1 << shift;
  const uint64_t below = lanes_below();
  int32_t base = 0, n = 0;

  if constexpr (FILTER) {
    // the wave's span of tokens: those of this bucket and of lower ones
    const int32_t span = ((N + kBucketThreads - 1) / kBucketThreads) * kWave;
    const int32_t wa = wave * span;
    const int32_t we = wa + span < N ? wa + span : N;
    int32_t mine = 0, lower = 0;
    for (int32_t j0 = wa; j0 < we; j0 += kWave) {
      const int32_t bin = j0 + lane < we ? of(j0 + lane) : of.buckets;
      mine += __popcll(__ballot(bin == b));
      lower += __popcll(__ballot(bin < b));
    }
    if (lane == 0) {
      sums[wave] = mine;
      sums[kBucketWaves + wave] = lower;
    }
    __syncthreads();
    int32_t at = 0;
#pragma unroll
    for (int w = 0; w < kBucketWaves; ++w) {
      at += w < wave ? sums[w] : 0;
      n += sums[w];
      base += sums[kBucketWaves + w];
    }
    for (int32_t j0 = wa; j0 < we; j0 += kWave) {
      const int32_t j = j0 + lane;
      const bool ok = j < we && of(j) == b;
      const uint64_t m = __ballot(ok);
      if (ok)
        list[at + __popcll(m & below)] =
            j | (((int32_t)load_id(of.ids, of.idx64, j) & (width - 1)) << 13);
      at += __popcll(m);
    }
  } else {
    base = bstart[b];
    n = bstart[b + 1] - base;
  }
  auto low_of = [&](int32_t i) { return FILTER ? list[i] >> 13 : llow[base + i]; };
  auto pos_of = [&](int32_t i) { return FILTER ? list[i] & (kFilterTokens - 1) : lpos[base + i]; };

  for (int i = tid; i < kBucketWaves * width; i += kBucketThreads) next[i] = 0;
  __syncthreads();
  const int32_t span = ((n + kBucketThreads - 1) / kBucketThreads) * kWave;
  const int32_t wa = wave * span;
  const int32_t we = wa + span < n ? wa + span : n;
  for (int32_t i = wa + lane; i < we; i += kWave)
    __hip_atomic_fetch_add(&next[(wave << shift) + low_of(i)], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  __syncthreads();

  // exclusive scan over the ids of the bucket; each thread has `per` of them
  const int32_t per = (width + kBucketThreads - 1) / kBucketThreads;
  int32_t mine = 0;
  for (int32_t q = 0; q < per; ++q) {
    const int32_t l = tid * per + q;
    if (l < width)
      for (int w = 0; w < kBucketWaves; ++w) mine += next[(w << shift) + l];
  }
  const int32_t inc = wave_inclusive_scan(mine);
  if (lane == kWave - 1) sums[wave] = inc;
  __syncthreads();
  int32_t run = base + inc - mine;
#pragma unroll
  for (int w = 0; w < kBucketWaves; ++w) run += w < wave ? sums[w] : 0;
  for (int32_t q = 0; q < per; ++q) {
    const int32_t l = tid * per + q;
    if (l >= width) break;
    const int64_t v = ((int64_t)b << shift) + l;
    if (v <= of.V) off[v] = run;
    for (int w = 0; w < kBucketWaves; ++w) {
      const int32_t c = next[(w << shift) + l];
      next[(w << shift) + l] = run;
      run += c;
    }
  }
  // the table's end, where it is the end of a bucket
  if (b == of.buckets - 1 && tid == 0 && ((int64_t)of.buckets << shift) == of.V) off[of.V] = base + n;
  __syncthreads();

  for (int32_t i0 = wa; i0 < we; i0 += kWave) {
    const int32_t i = i0 + lane;
    const bool ok = i < we;
    const int32_t low = ok ? low_of(i) : 0;
    const uint64_t m = same_bin((uint32_t)low, ok, shift);
    if (ok) {
      const int32_t p = next[(wave << shift) + low] + __popcll(m & below);
      pos[p] = pos_of(i);
      sid[p] = (b << shift) + low;
    }
    wave_lds_sync();
    if (ok && (m & below) == 0) next[(wave << shift) + low] += __popcll(m);
    wave_lds_sync();
  }
}

// --- sum -----------------------------------------------------------------------
constexpr int kZeroRows = 16;   // table rows a wave looks at for empty ones

// VE: columns per lane of the sums (16 bytes of g), VZ: of the zero rows.
template <typename WT, typename XT, int VE, int VZ>
__global__ __launch_bounds__(256) void token_sum_kernel(
    const XT* __restrict__ g, int64_t ldg, const int32_t* __restrict__ off,
    const int32_t* __restrict__ pos, const int32_t* __restrict__ sid, int32_t V, int32_t D,
    float scale, WT* __restrict__ gW, int64_t ldgw, float* __restrict__ parts, int64_t part_ld,
    int32_t chunk, Units units, uint32_t sum_blocks) {
  using RX = typename Pack<XT, VE>::raw;
  const int lane = lane_id();
  const int32_t nv = (D + VE - 1) / VE;

  if (blockIdx.x >= sum_blocks) {  // zero rows
    const int32_t v0 = ((int32_t)(blockIdx.x - sum_blocks) * 4 + wave_index()) * kZeroRows;
    const int32_t v = v0 + lane;
    const bool empty = lane < kZeroRows && v < V && off[v] == off[v + 1];
    uint64_t m = __ballot(empty);
    typename Pack<WT, VZ>::raw zero;
    zero_raw(zero);
    const int32_t nz = (D + VZ - 1) / VZ;
    while (m) {
      const int r = __builtin_ctzll(m);
      m &= m - 1;
      WT* row = gW + (int64_t)(v0 + r) * ldgw;
      for (int32_t i = lane; i < nz; i += kWave)
        store_pack_once<WT, VZ>(row + pack_column<VZ>(i, D), zero);
    }
    return;
  }

  const int32_t kept = off[V];
  for (UnitWalk u(units, blockIdx.x * 4 + wave_index()); u.valid(units); u.next(units)) {
    const int64_t b64 = u.row * chunk;
    if (b64 >= kept) continue;
    const int32_t b = (int32_t)b64;
    const int32_t e = kept - b > chunk ? b + chunk : kept;
    const int32_t i = u.seg * kWave + lane;
    const bool in = i < nv;
    const int32_t col = in ? pack_column<VE>(i, D) : 0;
    const XT* gc = g + col;
    float* part = parts + (u.row * 2) * part_ld + col;

    // leading places of a run that began before this chunk: its short rest
    // belongs to the wave of its start, a long run's piece to this one
    int32_t s0 = b;
    bool head = false;
    {
      const int32_t v = sid[b];
      const int32_t r0 = off[v], r1 = off[v + 1];
      if (r0 < b) {
        if (r1 - r0 > chunk) head = true;
        else s0 = r1;
      }
    }
    // the last run that starts here, if it crosses the border: whole if short
    int32_t s1 = e;
    bool tail = false;
    if (e < kept) {
      const int32_t v = sid[e - 1];
      const int32_t r0 = off[v], r1 = off[v + 1];
      if (r0 >= b && r1 > e) {
        if (r1 - r0 > chunk) tail = true;
        else s1 = r1;
      }
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
        if (k0 + q < s1 && in) r[q] = load_pack_once<XT, VE>(gc + (int64_t)pos[k0 + q] * ldg);
      }
#pragma unroll
      for (int q = 0; q < KU; ++q) {
        const int32_t k = k0 + q;
        if (k >= s1) break;
        float f[VE];
        widen<XT, VE>(r[q], f);
#pragma unroll
        for (int j = 0; j < VE; ++j) acc[j] += f[j];
        const int32_t v = sid[k];
        const bool last = k + 1 == s1;
        if (!last && sid[k + 1] == v) continue;
        // the run ends here: a whole one goes to the table, a piece of a
        // long one to this chunk's partial rows
        if (in) {
          if (head || (last && tail)) {
            store_pack<float, VE>(part + (head ? 0 : part_ld), narrow<float, VE>(acc));
          } else {
            float o[VE];
#pragma unroll
            for (int j = 0; j < VE; ++j) o[j] = acc[j] * scale;
            store_pack_once<WT, VE>(gW + (int64_t)v * ldgw + col, narrow<WT, VE>(o));
          }
        }
        head = false;
#pragma unroll
        for (int j = 0; j < VE; ++j) acc[j] = 0.f;
      }
    }
  }
}

// The run that starts in chunk c and has more than `chunk` tokens: its piece
// in c's second partial row and its pieces in the first rows of the chunks
// after it. 4 groups of 256 threads share the pieces, 4 columns per thread.
template <typename WT>
__global__ __launch_bounds__(1024) void token_join_kernel(
    const int32_t* __restrict__ off, const int32_t* __restrict__ sid, int32_t V, int32_t D,
    float scale, WT* __restrict__ gW, int64_t ldgw, const float* __restrict__ parts,
    int64_t part_ld, int32_t chunk, int64_t chunks) {
  __shared__ float4 red[3][256];
  const int32_t kept = off[V];
  const int group = threadIdx.x / 256;
  const int t = threadIdx.x % 256;
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int64_t e = (c + 1) * chunk;
    if (e >= kept) return;
    const int32_t v = sid[e - 1];
    const int32_t r0 = off[v], r1 = off[v + 1];
    if (r0 < c * chunk || r1 <= e || r1 - r0 <= chunk) continue;
    const int64_t pieces = (r1 - 1) / chunk - c;  // after the first one
    for (int32_t d0 = (blockIdx.y * 256 + t) * 4; d0 - t * 4 < D; d0 += gridDim.y * 1024) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      if (d0 < D) {
        // piece 0 is the run's first; rows are padded to whole float4s
#pragma unroll 8
        for (int64_t p = group; p <= pieces; p += 4) {
          const float4 f = *reinterpret_cast<const float4*>(
              parts + ((c + p) * 2 + (p == 0 ? 1 : 0)) * part_ld + d0);
          a.x += f.x; a.y += f.y; a.z += f.z; a.w += f.w;
        }
      }
      if (group) red[group - 1][t] = a;
      __syncthreads();
      if (group == 0 && d0 < D) {
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const float4 f = red[q][t];
          a.x += f.x; a.y += f.y; a.z += f.z; a.w += f.w;
        }
        const float o[4] = {a.x, a.y, a.z, a.w};
        WT* row = gW + (int64_t)v * ldgw;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (d0 + q < D) row[d0 + q] = round_to<WT>(o[q] * scale);
      }
      __syncthreads();
    }
  }
}

template <typename WT, typename XT, typename F>
hipError_t with_width(int32_t D, F f) {
  constexpr int VE = pack_elems<WT, XT>();
  if (D >= VE) return f(std::integral_constant<int, VE>{});
  return f(std::integral_constant<int, 1>{});
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
  // 64 sorted places a wave, fewer where that leaves the chip without waves
  const int32_t vec = d.xdtype == TBE_F32 ? 4 : 8;
  const int64_t segs = (d.D + 64 * vec - 1) / (64 * vec);
  L.chunk = d.N * segs >= 64 * 2048 ? 64 : 16;
  L.chunks = (d.N + L.chunk - 1) / L.chunk;
  L.part_ld = ((int64_t)d.D + 3) / 4 * 4;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += (bytes + 255) & ~size_t(255);
    return a;
  };
  const size_t n4 = sizeof(int32_t) * (size_t)d.N;
  L.off = take(sizeof(int32_t) * ((size_t)d.V + 1));
  L.pos = take(n4);
  L.sid = take(n4);
  if (!L.filtered) {
    L.lpos = take(n4);
    L.llow = take(n4);
    L.bstart = take(sizeof(int32_t) * ((size_t)L.buckets + 1));
    L.counts = take(sizeof(int32_t) * (size_t)split_shape(d.N).tiles * split_stride(L.buckets + 1));
  }
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
  int32_t *off = at(L.off), *pos = at(L.pos), *sid = at(L.sid);
  float* parts = reinterpret_cast<float*>(base + L.parts);
  const BucketOf of{ids, d.idx64, L.shift, L.buckets, d.V};
  const size_t lds = sizeof(int32_t) * ((size_t)kBucketWaves << L.shift);
  hipError_t e;
  if (L.filtered) {
    hipLaunchKernelGGL(token_bucket_kernel<true>, dim3(L.buckets), dim3(kBucketThreads),
                       lds + sizeof(int32_t) * (size_t)d.N, s, of, (int32_t)d.N, nullptr, nullptr, nullptr, off, pos, sid);
  } else {
    const SplitShape sh = split_shape(d.N);
    const int32_t stride = split_stride(L.buckets + 1);
    hipLaunchKernelGGL(token_count_kernel, dim3(sh.tiles), dim3(kSplitThreads), 0, s, of, d.N, sh,
                       stride, at(L.counts));
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(token_split_kernel, dim3(sh.tiles), dim3(kSplitThreads), 0, s, of, d.N, sh,
                       bits_for(L.buckets + 1), stride, at(L.counts), at(L.bstart), at(L.lpos),
                       at(L.llow));
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(token_bucket_kernel<false>, dim3(L.buckets), dim3(kBucketThreads), lds, s, of,
                       (int32_t)d.N, at(L.bstart), at(L.lpos), at(L.llow), off, pos, sid);
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  return with_type(d.wdtype, [&](auto wt) {
    using WT = decltype(wt);
    e = with_type(d.xdtype, [&](auto xt) {
      using XT = decltype(xt);
      auto go = [&](auto ve, auto vz) {
        constexpr int VE = decltype(ve)::value, VZ = decltype(vz)::value;
        unsigned sum_blocks = 0;
        const Units u = make_units(L.chunks, (d.D + kWave * VE - 1) / (kWave * VE), &sum_blocks);
        const unsigned zero_blocks = (unsigned)((d.V + 4 * kZeroRows - 1) / (4 * kZeroRows));
        hipLaunchKernelGGL((token_sum_kernel<WT, XT, VE, VZ>), dim3(sum_blocks + zero_blocks),
                           dim3(256), 0, s, static_cast<const XT*>(g), ldg, off, pos, sid,
                           (int32_t)d.V, d.D, d.scale, static_cast<WT*>(gW), ldgw, parts,
                           L.part_ld, L.chunk, u, sum_blocks);
        return hipGetLastError();
      };
      using std::integral_constant;
      if (d.D >= 8)
        return go(integral_constant<int, pack_elems<XT>()>{}, integral_constant<int, pack_elems<WT>()>{});
      return go(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    });
    if (e != hipSuccess || L.chunks < 2) return e;
    const unsigned panels = (unsigned)((d.D + 1023) / 1024);
    hipLaunchKernelGGL(token_join_kernel<WT>,
                       dim3((unsigned)(L.chunks < (1 << 16) ? L.chunks : (1 << 16)),
                            panels < 64 ? panels : 64),
                       dim3(1024), 0, s, off, sid, (int32_t)d.V, d.D, d.scale,
                       static_cast<WT*>(gW), ldgw, parts, L.part_ld, L.chunk, L.chunks);
    return hipGetLastError();
  });
}

}  // namespace tbe
