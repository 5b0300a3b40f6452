// C ABI of the operators beside the routed-MoE call: the router, the MXFP4
// linear layer and the few-token MoE layer. Validation only; nothing here
// allocates device memory or synchronizes a stream.
#include <new>

#include "api_util.h"
#include "internal.h"
#include "ops.h"

using namespace qmoe;

namespace {

moe_status check_linear_shape(int64_t N, int64_t K) {
  if (N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (K % 32 != 0 || K > 65536 || N > ((int64_t)1 << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ router
moe_status moe_router_create(int64_t E, int64_t H, int x_type, const void* w, int w_type, int64_t max_M,
                             moe_router** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!w || !aligned16(w) || E <= 0 || H <= 0 || max_M < 0) return MOE_ERR_INVALID_ARG;
  if (!type16(x_type) || (w_type != MOE_BF16 && w_type != MOE_FP32)) return MOE_ERR_INVALID_ARG;
  if (E > kRouteMaxE || H % 8 != 0 || H > 65536 || max_M > kMaxRows) return MOE_ERR_UNSUPPORTED;
  int dev, cus;
  const void* ptrs[1] = {w};
  const moe_status st = device_of(ptrs, 1, &dev, &cus);
  if (st != MOE_OK) return st;
  moe_router* r = new (std::nothrow) moe_router;
  if (!r) return MOE_ERR_INVALID_ARG;
  *r = moe_router{E, H, max_M, x_type, w_type, dev, cus, w};
  *out = r;
  return MOE_OK;
}

void moe_router_destroy(moe_router* r) { delete r; }

const char* moe_router_kernel(const moe_router* r, int64_t M) {
  return r && M > 0 && M <= r->max_M ? router_kernel_name(M, r->E, r->num_cus) : nullptr;
}

moe_status moe_router_forward(const moe_router* r, int64_t M, const void* x, int64_t ldx, float* logits,
                              void* stream) {
  if (!r || M < 0 || M > r->max_M) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!x || !aligned16(x) || !logits || !aligned16(logits) || ldx < r->H || ldx % 8 != 0 || ldx > kMaxStride)
    return MOE_ERR_INVALID_ARG;
  if (ptr_device(x) != r->device || ptr_device(logits) != r->device) return MOE_ERR_DEVICE;
  const size_t out_bytes = 4 * (size_t)M * (size_t)r->E;
  if (overlaps(logits, out_bytes, x, span(M, ldx, r->H, 2)) ||
      overlaps(logits, out_bytes, r->w, (size_t)r->E * r->H * type_bytes(r->w_type)))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard guard(r->device);
  if (!guard.ok) return MOE_ERR_DEVICE;
  const RouterArgs a{M, r->E, r->H, ldx, x, r->w, logits, r->x_type, r->w_type};
  return launch_router(a, r->num_cus, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// ------------------------------------------------------------------ linear
moe_status moe_linear_pack_bytes(int64_t N, int64_t K, size_t* w_bytes, size_t* s_bytes) {
  const moe_status st = check_linear_shape(N, K);
  if (st != MOE_OK) return st;
  if (!w_bytes || !s_bytes) return MOE_ERR_INVALID_ARG;
  const size_t pieces = (size_t)((N + 15) / 16) * (size_t)((K + 127) / 128);
  *w_bytes = pieces * 1024;
  *s_bytes = pieces * 64;
  return MOE_OK;
}

moe_status moe_pack_linear(const void* w, const void* s, int64_t N, int64_t K, void* w_packed, void* s_packed,
                           void* stream) {
  size_t wb, sb;
  const moe_status st = moe_linear_pack_bytes(N, K, &wb, &sb);
  if (st != MOE_OK) return st;
  const void* ptrs[4] = {w, s, w_packed, s_packed};
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  const size_t wi = (size_t)N * (K / 2), si = (size_t)N * (K / 32);
  if (overlaps(w_packed, wb, w, wi) || overlaps(w_packed, wb, s, si) || overlaps(s_packed, sb, w, wi) ||
      overlaps(s_packed, sb, s, si) || overlaps(w_packed, wb, s_packed, sb))
    return MOE_ERR_INVALID_ARG;
  const int dev = ptr_device(w);
  if (dev < 0) return MOE_ERR_DEVICE;
  for (const void* q : ptrs)
    if (ptr_device(q) != dev) return MOE_ERR_DEVICE;
  DeviceGuard guard(dev);
  if (!guard.ok) return MOE_ERR_DEVICE;
  return launch_pack_linear(w, s, N, K, w_packed, s_packed, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_linear_create(int64_t N, int64_t K, int x_type, const void* w_packed, const void* s_packed,
                             const void* bias, int64_t max_M, moe_linear** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  moe_status st = check_linear_shape(N, K);
  if (st != MOE_OK) return st;
  if (!type16(x_type) || max_M < 0) return MOE_ERR_INVALID_ARG;
  if (max_M > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (!w_packed || !aligned16(w_packed) || !s_packed || !aligned16(s_packed) || !aligned16(bias))
    return MOE_ERR_INVALID_ARG;
  int dev, cus;
  const void* ptrs[3] = {w_packed, s_packed, bias};
  st = device_of(ptrs, 3, &dev, &cus);
  if (st != MOE_OK) return st;
  moe_linear* l = new (std::nothrow) moe_linear;
  if (!l) return MOE_ERR_INVALID_ARG;
  *l = moe_linear{N, K, max_M, x_type, dev, cus, (const uint8_t*)w_packed, (const uint8_t*)s_packed, bias};
  *out = l;
  return MOE_OK;
}

void moe_linear_destroy(moe_linear* l) { delete l; }

const char* moe_linear_kernel(const moe_linear* l, int64_t M) {
  return l && M > 0 && M <= l->max_M ? linear_kernel_name(M, l->N, l->K, l->x_type == MOE_FP16, l->num_cus) : nullptr;
}

moe_status moe_linear_forward(const moe_linear* l, int64_t M, const void* x, int64_t ldx, const void* residual,
                              int64_t ldr, void* y, int64_t ldy, int y_type, void* stream) {
  if (!l || M < 0 || M > l->max_M) return MOE_ERR_INVALID_ARG;
  if (y_type != l->x_type && y_type != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const size_t es = type_bytes(y_type);
  if (!x || !aligned16(x) || ldx < l->K || ldx % 8 != 0 || ldx > kMaxStride) return MOE_ERR_INVALID_ARG;
  if (!y || ((uintptr_t)y & (es - 1)) || ldy < l->N || ldy > kMaxStride) return MOE_ERR_INVALID_ARG;
  if (residual && (((uintptr_t)residual & (es - 1)) || ldr < l->N || ldr > kMaxStride))
    return MOE_ERR_INVALID_ARG;
  if (ptr_device(x) != l->device || ptr_device(y) != l->device || (residual && ptr_device(residual) != l->device))
    return MOE_ERR_DEVICE;
  size_t wb, sb;
  (void)moe_linear_pack_bytes(l->N, l->K, &wb, &sb);
  const size_t yb = span(M, ldy, l->N, es);
  if (overlaps(y, yb, x, span(M, ldx, l->K, 2)) || overlaps(y, yb, l->wp, wb) || overlaps(y, yb, l->sp, sb) ||
      (l->bias && overlaps(y, yb, l->bias, 2 * (size_t)l->N)))
    return MOE_ERR_INVALID_ARG;
  // in place (y is the residual itself) every element is read before it is written
  if (residual && !(residual == y && ldr == ldy) && overlaps(y, yb, residual, span(M, ldr, l->N, es)))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard guard(l->device);
  if (!guard.ok) return MOE_ERR_DEVICE;
  // columns that move together: groups of four, or pieces of 16 bytes
  auto fits = [&](int64_t n) {
    const uintptr_t bytes = (uintptr_t)n * es - 1;
    return l->N % n == 0 && ldy % n == 0 && ((uintptr_t)y & bytes) == 0 &&
           (!residual || (ldr % n == 0 && ((uintptr_t)residual & bytes) == 0));
  };
  const int vec = fits(16 / (int64_t)es) ? 2 : fits(4) ? 1 : 0;
  const LinearArgs a{M, l->N, l->K, ldx, ldr, ldy, x, l->wp, l->sp, l->bias, residual, y, l->x_type, y_type, vec};
  return launch_linear(a, l->num_cus, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// ------------------------------------------------------------------ layer
moe_status moe_layer_forward(moe_plan* plan, const moe_router* router, int64_t M, const void* x, const void* w13,
                             const void* s13, const void* w2, const void* s2, void* out, void* stream) {
  if (!plan || !router) return MOE_ERR_INVALID_ARG;
  if (M < 0 || M > plan->s.M) return MOE_ERR_INVALID_ARG;
  if (router->E != plan->s.E || router->H != plan->s.H || router->x_type != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (router->device != plan->device) return MOE_ERR_DEVICE;
  if (M > kSmallM || !layer_shape(plan->s)) return MOE_ERR_UNSUPPORTED;
  if (plan->shared_slot || plan->tpx.tp > 0 || plan->mid_fmt != MOE_MID_E4M3 ||
      plan->layout != MOE_LAYOUT_W13_PACKED)
    return MOE_ERR_UNSUPPORTED;
  if (!plan->ws) return MOE_ERR_WORKSPACE;
  if (M == 0) return MOE_OK;
  const void* ptrs[6] = {x, w13, s13, w2, s2, out};
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  for (const void* q : ptrs)
    if (ptr_device(q) != plan->device) return MOE_ERR_DEVICE;
  const size_t H = (size_t)plan->s.H, E = (size_t)plan->s.E, I = (size_t)plan->s.I, ob = (size_t)M * H * 2;
  if (overlaps(out, ob, x, ob) || overlaps(out, ob, plan->ws, plan->ws_bytes) ||
      overlaps(x, ob, plan->ws, plan->ws_bytes) ||
      overlaps(out, ob, router->w, E * H * type_bytes(router->w_type)) || overlaps(out, ob, w13, E * I * H) ||
      overlaps(out, ob, s13, E * I * H / 16) || overlaps(out, ob, w2, E * I * H / 2) ||
      overlaps(out, ob, s2, E * I * H / 32))
    return MOE_ERR_INVALID_ARG;
  DeviceGuard guard(plan->device);
  if (!guard.ok) return MOE_ERR_DEVICE;
  const LayerArgs a{M, x, w13, s13, w2, s2, out, (hipStream_t)stream};
  return launch_layer(plan, router, a) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
