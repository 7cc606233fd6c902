// C ABI of the language-model operators: argument checks on the host before
// any launch, then the launchers on the caller's stream.
#include <algorithm>
#include <cmath>
#include <limits>
#include <new>

#include "lm.h"

using namespace tbe;

namespace {

constexpr int64_t kI32Lim = (int64_t(1) << 31) - 1;
constexpr int32_t kMaxD = 1 << 28;  // columns: offsets inside a row stay in 32 bits

#define TBE_TRY_HIP(expr)                                        \
  do {                                                           \
    (void)hipGetLastError(); /* an earlier runtime call's error */ \
    const hipError_t tbe_e_ = (expr);                            \
    if (tbe_e_ != hipSuccess) return hip_failure(tbe_e_, #expr); \
  } while (0)

bool type_ok(tbe_dtype t) { return t == TBE_F32 || t == TBE_F16 || t == TBE_BF16; }
bool idx_ok(int32_t i) { return i == 0 || i == 1; }
bool in_ld(int64_t ld) { return ld >= 0; }
bool out_ld(int64_t ld, int64_t width) { return ld >= width; }

tbe_status check(const tbe_token_desc* d) {
  if (!d || d->N < 0 || d->V < 1 || d->D < 1 || !idx_ok(d->idx64)) return TBE_ERR_ARG;
  if (!type_ok(d->wdtype) || !type_ok(d->xdtype)) return TBE_ERR_UNSUPPORTED;
  if (d->N >= (int64_t(1) << 30) || d->V > kTokenMaxRows || d->D > kMaxD) return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

tbe_status check(const tbe_expert_desc* d) {
  if (!d || d->N < 0 || d->K < 1 || d->E < 1 || d->D < 1 || !idx_ok(d->idx64)) return TBE_ERR_ARG;
  if (!type_ok(d->dtype)) return TBE_ERR_UNSUPPORTED;
  if (d->K > 64 || d->E > kSplitBins - 1 || d->D > kMaxD || d->N >= kI32Lim || d->N * d->K >= kI32Lim)
    return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

tbe_status check(const tbe_distill_desc* d) {
  if (!d || d->N < 0 || d->V < 1 || d->K < 1 || !idx_ok(d->idx64)) return TBE_ERR_ARG;
  if (!(d->temperature > 0.f) || !std::isfinite(d->temperature)) return TBE_ERR_ARG;
  if (!type_ok(d->dtype) || !type_ok(d->tdtype)) return TBE_ERR_UNSUPPORTED;
  // below 4.24e-39 (a subnormal number) the powers' factor is no float32
  if (!std::isfinite(distill_factor(d->temperature))) return TBE_ERR_UNSUPPORTED;
  if (d->N >= kI32Lim || d->V >= kI32Lim || d->K > 1024) return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

tbe_status check(const tbe_norm_desc* d) {
  if (!d || d->N < 0 || d->D < 1 || !(d->eps >= 0.f) || !std::isfinite(d->eps)) return TBE_ERR_ARG;
  if (!type_ok(d->dtype) || !type_ok(d->wdtype)) return TBE_ERR_UNSUPPORTED;
  if (d->N >= kI32Lim || d->D > kMaxD) return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}
size_t norm_bytes(const tbe_norm_desc& d) {
  return 256 + sizeof(float) * 2 * (size_t)norm_partials(d) * (size_t)d.D;
}

constexpr int64_t kFfnElems = int64_t(1) << 36;
// Rows: the kernels count a tile's rows, up to 256, from its first one in 32 bits.
constexpr int64_t kFfnRows = kI32Lim - 1024;
tbe_status check(const tbe_ffn_desc* d) {
  if (!d || d->M < 0 || d->E < 1 || d->D < 1 || d->F < 1) return TBE_ERR_ARG;
  if (d->act != TBE_ACT_SILU && d->act != TBE_ACT_GELU) return TBE_ERR_ARG;
  if (!type_ok(d->dtype)) return TBE_ERR_UNSUPPORTED;
  if (d->M > kFfnRows || d->E > 1023 || d->D > 65536 || d->F > 65536) return TBE_ERR_UNSUPPORTED;
  if (d->M * std::max(d->D, 2 * d->F) > kFfnElems) return TBE_ERR_UNSUPPORTED;
  return (int64_t)d->E * d->D * d->F > kFfnElems ? TBE_ERR_UNSUPPORTED : TBE_OK;
}
// E matrices of `rows` x `cols`.
bool in_stack(const tbe_stack* m) { return m && m->data && m->ld >= 0 && m->stride >= 0; }
bool out_stack(const tbe_stack* m, int32_t E, int64_t rows, int64_t cols) {
  if (!m || !m->data || m->ld < cols || m->stride < 0) return false;
  return E == 1 || m->stride / m->ld >= rows;
}

tbe_status check(const tbe_adamw_desc* d) {
  if (!d || (d->bits != 8 && d->bits != 32)) return TBE_ERR_ARG;
  if (!(d->beta1 >= 0 && d->beta1 < 1) || !(d->beta2 >= 0 && d->beta2 < 1)) return TBE_ERR_ARG;
  if (!(d->eps >= 0) || !std::isfinite((float)d->eps)) return TBE_ERR_ARG;
  if (!(d->weight_decay >= 0) || !std::isfinite((float)d->weight_decay)) return TBE_ERR_ARG;
  if (!type_ok(d->pdtype) || !type_ok(d->gdtype)) return TBE_ERR_UNSUPPORTED;
  // the kernel's reciprocal takes subnormal numbers for zeros, and 0 / eps would be NaN
  if (d->eps > 0 && (float)d->eps < std::numeric_limits<float>::min()) return TBE_ERR_UNSUPPORTED;
  if (d->cdtype != -1 && (d->pdtype != TBE_F32 || (d->cdtype != TBE_F16 && d->cdtype != TBE_BF16)))
    return TBE_ERR_UNSUPPORTED;
  return TBE_OK;
}

struct Range {
  uintptr_t a, z;
  bool operator<(const Range& o) const { return a < o.a; }
};
// Whether the tensors' parameters (or copies) overlap. Tensors in the order of
// their addresses, as in one buffer, are compared as they come; others are sorted.
tbe_status check_apart(const tbe_adamw_tensor* t, int64_t count, bool copies, size_t size) {
  auto range = [&](int64_t i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(copies ? t[i].c : t[i].p);
    return Range{a, a + (uintptr_t)t[i].n * size};
  };
  bool sorted = true;
  uintptr_t end = 0;
  for (int64_t i = 0; i < count && sorted; ++i) {
    if (t[i].n == 0) continue;
    const Range r = range(i);
    sorted = r.a >= end;
    end = r.z;
  }
  if (sorted) return TBE_OK;
  Range* r = new (std::nothrow) Range[(size_t)count];
  if (!r) return TBE_ERR_WORKSPACE;
  int64_t k = 0;
  for (int64_t i = 0; i < count; ++i)
    if (t[i].n > 0) r[k++] = range(i);
  std::sort(r, r + k);
  tbe_status status = TBE_OK;
  for (int64_t i = 1; i < k; ++i)
    if (r[i].a < r[i - 1].z) status = TBE_ERR_ARG;
  delete[] r;
  return status;
}

size_t type_size(tbe_dtype t) { return t == TBE_F32 ? 4 : 2; }

size_t expert_bytes(const tbe_expert_desc& d) {
  const SplitShape sh = split_shape(d.N * d.K, d.E + 1);
  const size_t counts = sh.tiles > 1 ? sizeof(int32_t) * (size_t)sh.tiles * split_stride(d.E + 1) : 0;
  return counts + 256;
}

tbe_status check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || have < need) return TBE_ERR_WORKSPACE;
  return reinterpret_cast<uintptr_t>(ws) % 256 == 0 ? TBE_OK : TBE_ERR_ARG;
}

#define TBE_CHECK(expr)                       \
  do {                                        \
    const tbe_status tbe_s_ = (expr);         \
    if (tbe_s_ != TBE_OK) return tbe_s_;      \
  } while (0)

}  // namespace

extern "C" {

tbe_status tbe_token_forward(const tbe_token_desc* d, const void* W, int64_t ldw, const void* ids,
                             void* out, int64_t ldo, void* stream) {
  TBE_CHECK(check(d));
  if (!W || !in_ld(ldw) || !out_ld(ldo, d->D)) return TBE_ERR_ARG;
  if (d->N == 0) return TBE_OK;
  if (!ids || !out) return TBE_ERR_ARG;
  TBE_TRY_HIP(launch_token_forward(*d, W, ldw, ids, out, ldo, (hipStream_t)stream));
  return TBE_OK;
}

size_t tbe_token_workspace_bytes(const tbe_token_desc* d) {
  return check(d) == TBE_OK ? token_layout(*d).total : 0;
}

tbe_status tbe_token_backward(const tbe_token_desc* d, const void* g, int64_t ldg, const void* ids,
                              void* gW, int64_t ldgw, void* ws, size_t ws_bytes, void* stream) {
  TBE_CHECK(check(d));
  if (!gW || !in_ld(ldg) || !out_ld(ldgw, d->D)) return TBE_ERR_ARG;
  if (d->N > 0 && (!g || !ids)) return TBE_ERR_ARG;
  const TokenLayout L = token_layout(*d);
  TBE_CHECK(check_ws(ws, ws_bytes, L.total));
  TBE_TRY_HIP(launch_token_backward(*d, L, g, ldg, ids, gW, ldgw, ws, (hipStream_t)stream));
  return TBE_OK;
}

size_t tbe_expert_workspace_bytes(const tbe_expert_desc* d) {
  return check(d) == TBE_OK ? expert_bytes(*d) : 0;
}

tbe_status tbe_expert_plan(const tbe_expert_desc* d, const void* ids, int32_t* offsets,
                           int32_t* order, int32_t* slots, void* ws, size_t ws_bytes,
                           void* stream) {
  TBE_CHECK(check(d));
  if (!offsets || (d->N > 0 && (!ids || !order || !slots))) return TBE_ERR_ARG;
  TBE_CHECK(check_ws(ws, ws_bytes, expert_bytes(*d)));
  TBE_TRY_HIP(launch_expert_plan(*d, ids, offsets, order, slots, static_cast<int32_t*>(ws),
                                 (hipStream_t)stream));
  return TBE_OK;
}

tbe_status tbe_expert_dispatch(const tbe_expert_desc* d, const void* x, int64_t ldx,
                               const int32_t* slots, void* xs, int64_t ldxs, void* stream) {
  TBE_CHECK(check(d));
  if (!in_ld(ldx) || !out_ld(ldxs, d->D)) return TBE_ERR_ARG;
  if (d->N == 0) return TBE_OK;
  if (!x || !slots || !xs) return TBE_ERR_ARG;
  TBE_TRY_HIP(launch_expert_dispatch(*d, x, ldx, slots, xs, ldxs, (hipStream_t)stream));
  return TBE_OK;
}

tbe_status tbe_expert_dispatch_backward(const tbe_expert_desc* d, const void* dxs, int64_t lddxs,
                                        const int32_t* slots, void* dx, int64_t lddx,
                                        void* stream) {
  TBE_CHECK(check(d));
  if (!in_ld(lddxs) || !out_ld(lddx, d->D)) return TBE_ERR_ARG;
  if (d->N == 0) return TBE_OK;
  if (!dxs || !slots || !dx) return TBE_ERR_ARG;
  TBE_TRY_HIP(launch_expert_combine(*d, dxs, lddxs, slots, nullptr, dx, lddx, (hipStream_t)stream));
  return TBE_OK;
}

tbe_status tbe_expert_combine(const tbe_expert_desc* d, const void* ys, int64_t ldys,
                              const int32_t* slots, const float* w, void* out, int64_t ldo,
                              void* stream) {
  TBE_CHECK(check(d));
  if (!in_ld(ldys) || !out_ld(ldo, d->D)) return TBE_ERR_ARG;
  if (d->N == 0) return TBE_OK;
  if (!ys || !slots || !w || !out) return TBE_ERR_ARG;
  TBE_TRY_HIP(launch_expert_combine(*d, ys, ldys, slots, w, out, ldo, (hipStream_t)stream));
  return TBE_OK;
}

tbe_status tbe_expert_combine_backward(const tbe_expert_desc* d, const void* dout, int64_t lddo,
                                       const void* ys, int64_t ldys, const int32_t* slots,
                                       const float* w, void* dys, int64_t lddys, float* dw,
                                       void* stream) {
  TBE_CHECK(check(d));
  if (!in_ld(lddo) || !in_ld(ldys) || !out_ld(lddys, d->D)) return TBE_ERR_ARG;
  if (d->N == 0) return TBE_OK;
  if (!dout || !ys || !slots || !w || !dys || !dw) return TBE_ERR_ARG;
  if (dys == ys && lddys != ldys) return TBE_ERR_ARG;
  TBE_TRY_HIP(launch_expert_combine_backward(*d, dout, lddo, ys, ldys, slots, w, dys, lddys, dw,
                                             (hipStream_t)stream));
  return TBE_OK;
}

size_t tbe_distill_workspace_bytes(const tbe_distill_desc* d) {
  return check(d) == TBE_OK ? distill_workspace(*d) : 0;
}

tbe_status tbe_distill_forward(const tbe_distill_desc* d, const void* x, int64_t ldx,
                               const void* ids, const void* t, float* loss, float* stats, void* ws,
                               size_t ws_bytes, void* stream) {
  TBE_CHECK(check(d));
  if (!in_ld(ldx)) return TBE_ERR_ARG;
  if (d->N > 0 && (!x || !ids || !t || !loss || !stats)) return TBE_ERR_ARG;
  TBE_CHECK(check_ws(ws, ws_bytes, distill_workspace(*d)));
  if (d->N == 0) return TBE_OK;
  TBE_TRY_HIP(launch_distill_forward(*d, x, ldx, ids, t, loss, stats, ws, (hipStream_t)stream));
  return TBE_OK;
}

tbe_status tbe_distill_backward(const tbe_distill_desc* d, const void* x, int64_t ldx,
                                const void* ids, const void* t, const float* stats,
                                const float* gl, void* gx, int64_t ldgx, void* stream) {
  TBE_CHECK(check(d));
  if (!in_ld(ldx) || !out_ld(ldgx, d->V)) return TBE_ERR_ARG;
  if (d->N == 0) return TBE_OK;
  if (!x || !ids || !t || !stats || !gl || !gx) return TBE_ERR_ARG;
  if (gx == x && ldgx != ldx) return TBE_ERR_ARG;
  TBE_TRY_HIP(launch_distill_backward(*d, x, ldx, ids, t, stats, gl, gx, ldgx,
                                      (hipStream_t)stream));
  return TBE_OK;
}

tbe_status tbe_distill_step(const tbe_distill_desc* d, const void* x, int64_t ldx, const void* ids,
                            const void* t, const float* gl, float* loss, void* gx, int64_t ldgx,
                            void* ws, size_t ws_bytes, void* stream) {
  TBE_CHECK(check(d));
  if (!in_ld(ldx) || !out_ld(ldgx, d->V)) return TBE_ERR_ARG;
  if (d->N > 0 && (!x || !ids || !t || !gl || !loss || !gx)) return TBE_ERR_ARG;
  if (d->N > 0 && gx == x && ldgx != ldx) return TBE_ERR_ARG;
  TBE_CHECK(check_ws(ws, ws_bytes, distill_workspace(*d)));
  if (d->N == 0) return TBE_OK;
  TBE_TRY_HIP(launch_distill_step(*d, x, ldx, ids, t, gl, loss, gx, ldgx, ws, (hipStream_t)stream));
  return TBE_OK;
}

tbe_status tbe_norm_forward(const tbe_norm_desc* d, const void* x, int64_t ldx, const void* w,
                            const void* b, void* y, int64_t ldy, float* stats, void* stream) {
  TBE_CHECK(check(d));
  if (!in_ld(ldx) || !out_ld(ldy, d->D)) return TBE_ERR_ARG;
  if (d->N == 0) return TBE_OK;
  if (!x || !y || !stats) return TBE_ERR_ARG;
  TBE_TRY_HIP(launch_norm_forward(*d, x, ldx, w, b, y, ldy, stats, (hipStream_t)stream));
  return TBE_OK;
}

size_t tbe_norm_workspace_bytes(const tbe_norm_desc* d) {
  return check(d) == TBE_OK ? norm_bytes(*d) : 0;
}

tbe_status tbe_norm_backward(const tbe_norm_desc* d, const void* dy, int64_t lddy, const void* x,
                             int64_t ldx, const void* w, const float* stats, void* dx,
                             int64_t lddx, void* dw, void* db, void* ws, size_t ws_bytes,
                             void* stream) {
  TBE_CHECK(check(d));
  if (!in_ld(lddy) || !in_ld(ldx) || !out_ld(lddx, d->D)) return TBE_ERR_ARG;
  if (d->N > 0 && (!dy || !x || !stats || !dx)) return TBE_ERR_ARG;
  TBE_CHECK(check_ws(ws, ws_bytes, norm_bytes(*d)));
  TBE_TRY_HIP(launch_norm_backward(*d, dy, lddy, x, ldx, w, stats, dx, lddx, dw, db,
                                   static_cast<float*>(ws), (hipStream_t)stream));
  return TBE_OK;
}

size_t tbe_ffn_workspace_bytes(const tbe_ffn_desc* d) {
  return check(d) == TBE_OK ? ffn_layout(*d).total : 0;
}

tbe_status tbe_ffn_forward(const tbe_ffn_desc* d, const void* xs, int64_t ldxs,
                           const int32_t* offsets, const tbe_stack* gate, const tbe_stack* up,
                           const tbe_stack* down, void* pre, int64_t ldpre, void* ys,
                           int64_t ldys, void* ws, size_t ws_bytes, void* stream) {
  TBE_CHECK(check(d));
  if (!in_stack(gate) || !in_stack(up) || !in_stack(down)) return TBE_ERR_ARG;
  if (!in_ld(ldxs) || !out_ld(ldys, d->D) || (pre && !out_ld(ldpre, 2 * (int64_t)d->F)))
    return TBE_ERR_ARG;
  if (!offsets || (d->M > 0 && (!xs || !ys))) return TBE_ERR_ARG;
  TBE_CHECK(check_ws(ws, ws_bytes, ffn_layout(*d).total));
  if (d->M == 0) return TBE_OK;
  TBE_TRY_HIP(launch_ffn_forward(*d, {xs, ldxs, offsets, *gate, *up, *down, pre, ldpre, ys, ldys,
                                      static_cast<char*>(ws)}, (hipStream_t)stream));
  return TBE_OK;
}

tbe_status tbe_ffn_backward(const tbe_ffn_desc* d, const void* dys, int64_t lddys, const void* xs,
                            int64_t ldxs, const int32_t* offsets, const tbe_stack* gate,
                            const tbe_stack* up, const tbe_stack* down, const void* pre,
                            int64_t ldpre, void* dxs, int64_t lddxs, const tbe_stack* dgate,
                            const tbe_stack* dup, const tbe_stack* ddown, void* ws,
                            size_t ws_bytes, void* stream) {
  TBE_CHECK(check(d));
  if (!in_stack(gate) || !in_stack(up) || !in_stack(down)) return TBE_ERR_ARG;
  if (!out_stack(dgate, d->E, d->F, d->D) || !out_stack(dup, d->E, d->F, d->D) ||
      !out_stack(ddown, d->E, d->D, d->F))
    return TBE_ERR_ARG;
  if (!in_ld(lddys) || !in_ld(ldxs) || !in_ld(ldpre) || !out_ld(lddxs, d->D)) return TBE_ERR_ARG;
  if (!offsets || (d->M > 0 && (!dys || !xs || !pre || !dxs))) return TBE_ERR_ARG;
  TBE_CHECK(check_ws(ws, ws_bytes, ffn_layout(*d).total));
  TBE_TRY_HIP(launch_ffn_backward(*d, {dys, lddys, xs, ldxs, offsets, *gate, *up, *down, pre, ldpre,
                                       dxs, lddxs, *dgate, *dup, *ddown, static_cast<char*>(ws)},
                                  (hipStream_t)stream));
  return TBE_OK;
}

tbe_status tbe_adamw_step(const tbe_adamw_desc* d, const tbe_adamw_tensor* t, int64_t count,
                          const int64_t* step, const float* lr, const float* scale, void* stream) {
  TBE_CHECK(check(d));
  if (count < 0 || (count > 0 && !t)) return TBE_ERR_ARG;
  if (count >= (int64_t(1) << 24)) return TBE_ERR_UNSUPPORTED;
  int64_t elements = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n < 0) return TBE_ERR_ARG;
    if (t[i].n >= (int64_t(1) << 40)) return TBE_ERR_UNSUPPORTED;
    if (t[i].n == 0) continue;
    elements += t[i].n;
    if (!t[i].p || !t[i].g || !t[i].m || !t[i].v || (d->cdtype >= 0 && !t[i].c)) return TBE_ERR_ARG;
    if (d->bits == 8 && (!t[i].mscale || !t[i].vscale ||
                         (reinterpret_cast<uintptr_t>(t[i].m) | reinterpret_cast<uintptr_t>(t[i].v)) % 8))
      return TBE_ERR_ARG;
  }
  if (!step || !lr) return TBE_ERR_ARG;
  TBE_CHECK(check_apart(t, count, false, type_size(d->pdtype)));
  if (d->cdtype >= 0) TBE_CHECK(check_apart(t, count, true, 2));
  if (elements == 0) return TBE_OK;
  TBE_TRY_HIP(launch_adamw(*d, t, count, step, lr, scale, (hipStream_t)stream));
  return TBE_OK;
}

}  // extern "C"
