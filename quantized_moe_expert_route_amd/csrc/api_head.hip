// C ABI of the operators on the output head's logits: scores of given tokens and
// distillation. Validation only; nothing here allocates device memory or
// synchronizes a stream.
#include <new>

#include "api_util.h"
#include "head.h"

using namespace qmoe;

namespace {

moe_status check_head(int64_t V, int64_t k, int64_t k_min, int type, int64_t max_M) {
  if (V <= 0 || k < k_min || max_M < 0 || (!type16(type) && type != MOE_FP32)) return MOE_ERR_INVALID_ARG;
  if (V > ((int64_t)1 << 24) || k > kMaxTop || max_M > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool rows_ok(const void* p, int64_t ld, int64_t V, size_t elem) {
  return p && ((uintptr_t)p & (elem - 1)) == 0 && ld >= V && ld <= kMaxStride;
}
bool dense_ok(const void* p) { return p && ((uintptr_t)p & 3) == 0; }

}  // namespace

extern "C" {

// ------------------------------------------------------------------ scores
moe_status moe_scores_create(int64_t V, int64_t top_k, int type, int64_t max_M, moe_scores** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  moe_status st = check_head(V, top_k, 0, type, max_M);
  if (st != MOE_OK) return st;
  if (top_k > V) return MOE_ERR_INVALID_ARG;
  int dev, cus;
  st = current_device(&dev, &cus);
  if (st != MOE_OK) return st;
  moe_scores* s = new (std::nothrow) moe_scores;
  if (!s) return MOE_ERR_INVALID_ARG;
  *s = moe_scores{V, top_k, max_M, type, dev, cus};
  *out = s;
  return MOE_OK;
}

void moe_scores_destroy(moe_scores* s) { delete s; }

const char* moe_scores_kernel(const moe_scores* s, int64_t M) {
  return s && M > 0 && M <= s->max_M ? scores_kernel_name(M, s->V, s->k, s->num_cus) : nullptr;
}

moe_status moe_scores_workspace_bytes(const moe_scores* s, int64_t M, size_t* bytes) {
  if (!s || !bytes || M < 0 || M > s->max_M) return MOE_ERR_INVALID_ARG;
  *bytes = scores_ws_bytes(M, s->V, s->k, s->num_cus);
  return MOE_OK;
}

moe_status moe_scores_forward(const moe_scores* s, int64_t M, const void* z, int64_t ldz, const int32_t* tokens,
                              float* logprobs, float* entropy, float* lse, float* top_logprobs, int32_t* top_ids,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!s || M < 0 || M > s->max_M) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const size_t es = type_bytes(s->type);
  if (!rows_ok(z, ldz, s->V, es)) return MOE_ERR_INVALID_ARG;
  if ((tokens != nullptr) != (logprobs != nullptr)) return MOE_ERR_INVALID_ARG;
  if (s->k > 0 ? !top_logprobs || !top_ids : top_logprobs || top_ids) return MOE_ERR_INVALID_ARG;
  const size_t need = scores_ws_bytes(M, s->V, s->k, s->num_cus);
  moe_status st = check_ws(workspace, workspace_bytes, need);
  if (st != MOE_OK) return st;
  const size_t col = 4 * (size_t)M, top = col * (size_t)s->k;
  const Buf b[] = {{logprobs, col, true}, {entropy, col, true}, {lse, col, true}, {top_logprobs, top, true},
                   {top_ids, top, true}, {workspace, need, true}, {tokens, col, false}, {z, span(M, ldz, s->V, es), false}};
  for (int i = 0; i < 7; ++i)
    if (b[i].p && ((uintptr_t)b[i].p & 3)) return MOE_ERR_INVALID_ARG;
  st = check_buffers(b, 8, s->device);
  if (st != MOE_OK) return st;
  DeviceGuard guard(s->device);
  if (!guard.ok) return MOE_ERR_DEVICE;
  const ScoresArgs a{M, s->V, ldz, z, tokens, logprobs, entropy, lse, top_logprobs, top_ids, (int)s->k, s->type, workspace};
  return launch_scores(a, s->num_cus, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// ------------------------------------------------------------------ distillation
moe_status moe_distill_create(int64_t V, int64_t k, int type, int grad_type, float temperature, int64_t max_M,
                              moe_distill** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  moe_status st = check_head(V, k, 1, type, max_M);
  if (st != MOE_OK) return st;
  if (grad_type != type && !type16(grad_type)) return MOE_ERR_INVALID_ARG;
  if (!(temperature >= 1e-6f && temperature <= 1e6f)) return MOE_ERR_INVALID_ARG;
  int dev, cus;
  st = current_device(&dev, &cus);
  if (st != MOE_OK) return st;
  moe_distill* d = new (std::nothrow) moe_distill;
  if (!d) return MOE_ERR_INVALID_ARG;
  *d = moe_distill{V, k, max_M, type, grad_type, temperature, dev, cus};
  *out = d;
  return MOE_OK;
}

void moe_distill_destroy(moe_distill* d) { delete d; }

const char* moe_distill_kernel(const moe_distill* d, int64_t M, int pass) {
  if (!d || M <= 0 || M > d->max_M || pass < kDistillForward || pass > kDistillBoth) return nullptr;
  return distill_kernel_name((DistillPass)pass, M, d->V, d->type, d->grad_type, d->num_cus);
}

moe_status moe_distill_workspace_bytes(const moe_distill* d, int64_t M, size_t* bytes) {
  if (!d || !bytes || M < 0 || M > d->max_M) return MOE_ERR_INVALID_ARG;
  *bytes = distill_ws_bytes(M, d->V, d->type, d->num_cus);
  return MOE_OK;
}

static moe_status distill(DistillPass pass, const moe_distill* d, int64_t M, const void* z, int64_t ldz,
                          const int32_t* ids, const float* t, const float* weight, float* loss, float* lse, void* dz,
                          int64_t lddz, void* workspace, size_t workspace_bytes, void* stream) {
  if (!d || M < 0 || M > d->max_M) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const size_t es = type_bytes(d->type), gs = type_bytes(d->grad_type);
  if (!rows_ok(z, ldz, d->V, es) || !dense_ok(ids) || !dense_ok(t) || ((uintptr_t)lse & 3)) return MOE_ERR_INVALID_ARG;
  if (pass != kDistillBackward && !dense_ok(loss)) return MOE_ERR_INVALID_ARG;
  if (pass == kDistillBackward && !lse) return MOE_ERR_INVALID_ARG;
  if (pass != kDistillForward && (!dense_ok(weight) || !rows_ok(dz, lddz, d->V, gs))) return MOE_ERR_INVALID_ARG;
  const size_t need = pass == kDistillBackward ? 0 : distill_ws_bytes(M, d->V, d->type, d->num_cus);
  moe_status st = check_ws(workspace, workspace_bytes, need);
  if (st != MOE_OK) return st;
  const size_t col = 4 * (size_t)M, top = col * (size_t)d->k;
  // in place (dz is z itself) every logit is read before its gradient is written
  const bool in_place = dz == z && lddz == ldz && d->grad_type == d->type;
  const Buf b[] = {{dz, span(M, lddz, d->V, gs), true},
                   {loss, col, true},
                   {lse, col, pass != kDistillBackward},
                   {workspace, need, true},
                   {z, in_place ? 0 : span(M, ldz, d->V, es), false},
                   {ids, top, false},
                   {t, top, false},
                   {weight, col, false}};
  st = check_buffers(b, 8, d->device);
  if (st != MOE_OK) return st;
  DeviceGuard guard(d->device);
  if (!guard.ok) return MOE_ERR_DEVICE;
  const DistillArgs a{M, d->V, ldz, lddz, z, ids, t, weight, loss, lse, dz, d->temperature, (int)d->k, d->type, d->grad_type, workspace};
  return launch_distill(pass, a, d->num_cus, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_distill_forward(const moe_distill* d, int64_t M, const void* z, int64_t ldz, const int32_t* ids,
                               const float* t, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                               void* stream) {
  return distill(kDistillForward, d, M, z, ldz, ids, t, nullptr, loss, lse, nullptr, 0, workspace, workspace_bytes, stream);
}

moe_status moe_distill_backward(const moe_distill* d, int64_t M, const void* z, int64_t ldz, const int32_t* ids,
                                const float* t, const float* lse, const float* weight, void* dz, int64_t lddz,
                                void* stream) {
  return distill(kDistillBackward, d, M, z, ldz, ids, t, weight, nullptr, const_cast<float*>(lse), dz, lddz, nullptr, 0, stream);
}

moe_status moe_distill_forward_backward(const moe_distill* d, int64_t M, const void* z, int64_t ldz,
                                        const int32_t* ids, const float* t, const float* weight, float* loss, void* dz,
                                        int64_t lddz, void* workspace, size_t workspace_bytes, void* stream) {
  return distill(kDistillBoth, d, M, z, ldz, ids, t, weight, loss, nullptr, dz, lddz, workspace, workspace_bytes, stream);
}

}  // extern "C"
