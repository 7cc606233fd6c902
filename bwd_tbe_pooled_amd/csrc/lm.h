// Host-side internals of the language-model operators: launchers and the
// layout of their workspaces.
#pragma once

#include <hip/hip_runtime.h>

#include "tbe_lm.h"

namespace tbe {

// Text behind tbe_last_error (api.cpp); returns TBE_ERR_HIP.
tbe_status hip_failure(hipError_t e, const char* what);

constexpr int kSplitBins = 1024;     // bins of one stable split, at most
// ids of one bucket of the token sort, at most, and the table rows this allows
constexpr int kBucketIds = 1024;
constexpr int64_t kTokenMaxRows = int64_t(kSplitBins - 1) * kBucketIds;

// Tiles of a stable split of n keys: tile length a multiple of 1024, at most
// 256 tiles.
struct SplitShape {
  int32_t tiles, len;
};
SplitShape split_shape(int64_t n, int32_t bins);

// Stable split of M assignments by expert (expert.hip's plan).
// counts: int32[tiles * stride(E + 1)], unused with one tile.
int32_t split_stride(int32_t bins);
hipError_t launch_expert_plan(const tbe_expert_desc& d, const void* ids, int32_t* offsets,
                              int32_t* order, int32_t* slots, int32_t* counts, hipStream_t s);
hipError_t launch_expert_dispatch(const tbe_expert_desc& d, const void* x, int64_t ldx,
                                  const int32_t* slots, void* xs, int64_t ldxs, hipStream_t s);
hipError_t launch_expert_combine(const tbe_expert_desc& d, const void* ys, int64_t ldys,
                                 const int32_t* slots, const float* w, void* out, int64_t ldo,
                                 hipStream_t s);
hipError_t launch_expert_combine_backward(const tbe_expert_desc& d, const void* dout, int64_t lddo,
                                          const void* ys, int64_t ldys, const int32_t* slots,
                                          const float* w, void* dys, int64_t lddys, float* dw,
                                          hipStream_t s);

// Token table's gradient: workspace regions, byte offsets.
struct TokenLayout {
  int32_t shift;      // ids of one bucket share id >> shift
  int32_t buckets;
  int32_t chunk;      // sorted places per wave of the sum
  int64_t chunks;
  int64_t part_ld;    // floats per partial row
  bool few;           // no sort, one launch (few tokens)
  bool filtered;      // one launch sorts
  size_t off;         // int32[V + 1]: first sorted place of each id
  size_t sorted;      // int2[N]: token and id (top bit: of a run longer than a chunk) at each sorted place
  size_t split;       // int2[N]: token and lower part of the id, before the sort inside buckets
  size_t bstart;      // int32[buckets + 1]
  size_t counts;      // split counts
  size_t listed;      // long runs: int32[4], of which 2 counts; int4[2][chunks]
  size_t parts;       // float[chunks][2][part_ld]
  size_t total;
};
TokenLayout token_layout(const tbe_token_desc& d);
hipError_t launch_token_forward(const tbe_token_desc& d, const void* W, int64_t ldw,
                                const void* ids, void* out, int64_t ldo, hipStream_t s);
hipError_t launch_token_backward(const tbe_token_desc& d, const TokenLayout& L, const void* g,
                                 int64_t ldg, const void* ids, void* gW, int64_t ldgw, void* ws,
                                 hipStream_t s);

// log2(e) / temperature: the kernels' powers are of 2.
inline float distill_factor(float temperature) {
  return (float)(1.4426950408889634 / (double)temperature);
}
hipError_t launch_distill_forward(const tbe_distill_desc& d, const void* x, int64_t ldx,
                                  const void* ids, const void* t, float* loss, float* stats,
                                  void* ws, hipStream_t s);
hipError_t launch_distill_backward(const tbe_distill_desc& d, const void* x, int64_t ldx,
                                   const void* ids, const void* t, const float* stats,
                                   const float* gl, void* gx, int64_t ldgx, hipStream_t s);
hipError_t launch_distill_step(const tbe_distill_desc& d, const void* x, int64_t ldx,
                               const void* ids, const void* t, const float* gl, float* loss,
                               void* gx, int64_t ldgx, void* ws, hipStream_t s);
size_t distill_workspace(const tbe_distill_desc& d);

// Layer norm. The backward's workgroups leave a partial row of dw and db each.
int32_t norm_partials(const tbe_norm_desc& d);
hipError_t launch_norm_forward(const tbe_norm_desc& d, const void* x, int64_t ldx, const void* w,
                               const void* b, void* y, int64_t ldy, float* stats, hipStream_t s);
hipError_t launch_norm_backward(const tbe_norm_desc& d, const void* dy, int64_t lddy, const void* x,
                                int64_t ldx, const void* w, const float* stats, void* dx,
                                int64_t lddx, void* dw, void* db, float* parts, hipStream_t s);

// Experts' products: workspace regions, byte offsets.
struct FfnLayout {
  int64_t ld;     // elements of a row of h; a row of the gradients of g and u has two of them
  size_t h;       // [M, ld]
  size_t dgu;     // [M, 2 ld], backward only
  size_t total;
};
FfnLayout ffn_layout(const tbe_ffn_desc& d);
struct FfnForward {
  const void* xs; int64_t ldxs;
  const int32_t* offsets;
  tbe_stack gate, up, down;
  void* pre; int64_t ldpre;
  void* ys; int64_t ldys;
  char* ws;
};
struct FfnBackward {
  const void* dys; int64_t lddys;
  const void* xs; int64_t ldxs;
  const int32_t* offsets;
  tbe_stack gate, up, down;
  const void* pre; int64_t ldpre;
  void* dxs; int64_t lddxs;
  tbe_stack dgate, dup, ddown;
  char* ws;
};
hipError_t launch_ffn_forward(const tbe_ffn_desc& d, const FfnForward& a, hipStream_t s);
hipError_t launch_ffn_backward(const tbe_ffn_desc& d, const FfnBackward& a, hipStream_t s);

constexpr int kAdamBlock = 256;   // elements that share a scale of an 8-bit moment
hipError_t launch_adamw(const tbe_adamw_desc& d, const tbe_adamw_tensor* tensors, int64_t count,
                        const int64_t* step, const float* lr, const float* scale, hipStream_t s);

}  // namespace tbe
