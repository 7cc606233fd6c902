// C ABI of the language-model operators: argument checks on the host before
// any launch, then the launchers on the caller's stream.
#include <cmath>

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

}  // extern "C"
