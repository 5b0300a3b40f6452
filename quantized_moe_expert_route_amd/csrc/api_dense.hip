// C ABI of the layers in 16 bits: the matrix product with its epilogue and the
// gated feed-forward block. Validation and the order of launches only; nothing
// here allocates device memory or synchronizes a stream.
#include <new>

#include "api_util.h"
#include "dense.h"

using namespace qmoe;

namespace {

// Largest row distance of an operand (N is dz's): the 256 rows of a tile lie within
// 2^31 bytes.
constexpr int64_t kMaxOperandLd = (int64_t)1 << 22;

// Sizes of w [N, K] that the products take.
moe_status check_sizes(int64_t N, int64_t K, int type, int64_t max_M) {
  if (N <= 0 || K <= 0 || max_M < 0 || !type16(type)) return MOE_ERR_INVALID_ARG;
  if (K % 8 != 0 || K > 65536 || N > kMaxOperandLd || max_M > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool operand_ok(const void* x, int64_t ldx, int64_t K) {
  return x && aligned16(x) && ldx >= K && ldx % 8 == 0 && ldx <= kMaxOperandLd;
}
bool matrix_ok(const void* p, int64_t ld, int64_t cols, size_t elem, int64_t max_ld = kMaxStride) {
  return p && ((uintptr_t)p & (elem - 1)) == 0 && ld >= cols && ld <= max_ld;
}

// Kernel of product 0 (forward, of this kind and N columns), 1 (dx) or 2 (dw [Nw, K]).
const char* kernel_of(GemmKind kind, int64_t M, int64_t N, int64_t Nw, int64_t K, int cus, int product) {
  switch (product) {
    case 0: return gemm_kernel_name(kind, M, N, K, cus);
    case 1: return gemm_kernel_name(kGemmInput, M, K, Nw, cus);
    case 2: return gemm_kernel_name(kGemmWeight, Nw, K, M, cus);
  }
  return nullptr;
}

int64_t up8(int64_t n) { return (n + 7) & ~(int64_t)7; }

// Workspace of a backward pass: dz, the partial sums of dbias, split sums.
struct Backward {
  size_t dz, part, split, bytes;
};
Backward backward_layout(int64_t M, int64_t N, int64_t K, bool dz, bool bias, int cus) {
  Backward l;
  size_t at = 0;
  l.dz = at;
  at += dz ? align256((size_t)M * up8(N) * 2) : 0;
  l.part = at;
  at += bias ? align256((size_t)dbias_parts(M) * N * 4) : 0;
  l.split = at;
  const size_t a = gemm_ws_bytes(kGemmInput, M, K, N, cus), b = gemm_ws_bytes(kGemmWeight, N, K, M, cus);
  l.bytes = at + (a > b ? a : b);
  return l;
}

// dx = dz w and dw = dz^T x of dz [M, N], w [N, K], x [M, K].
hipError_t products(int64_t M, int64_t N, int64_t K, int type, int cus, const void* dz, int64_t ldz, const void* w,
                    const void* x, int64_t ldx, void* dx, int64_t lddx, void* dw, uint8_t* ws, const Backward& l,
                    hipStream_t s) {
  hipError_t e = hipSuccess;
  GemmArgs g{};
  g.type = g.y_type = type;
  g.ws = ws ? ws + l.split : nullptr;
  if (dx && M > 0) {
    g.rows = M, g.cols = K, g.K = N;
    g.a = dz, g.lda = ldz, g.b = w, g.ldb = K;
    g.y = dx, g.ldy = lddx;
    e = launch_gemm(kGemmInput, g, cus, s);
  }
  if (dw && e == hipSuccess) {
    g.rows = N, g.cols = K, g.K = M;
    g.a = dz, g.lda = ldz, g.b = x, g.ldb = ldx;
    g.y = dw, g.ldy = K;
    e = launch_gemm(kGemmWeight, g, cus, s);
  }
  return e;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ dense
moe_status moe_dense_create(int64_t N, int64_t K, int type, const void* w, const void* bias, int activation,
                            int64_t max_M, moe_dense** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  moe_status st = check_sizes(N, K, type, max_M);
  if (st != MOE_OK) return st;
  if (!w || !aligned16(w) || ((uintptr_t)bias & 1) || activation < MOE_ACT_NONE || activation > MOE_ACT_GELU_TANH)
    return MOE_ERR_INVALID_ARG;
  int dev, cus;
  const void* ptrs[2] = {w, bias};
  st = device_of(ptrs, 2, &dev, &cus);
  if (st != MOE_OK) return st;
  moe_dense* d = new (std::nothrow) moe_dense;
  if (!d) return MOE_ERR_INVALID_ARG;
  *d = moe_dense{N, K, max_M, type, activation, dev, cus, w, bias};
  *out = d;
  return MOE_OK;
}

void moe_dense_destroy(moe_dense* d) { delete d; }

const char* moe_dense_kernel(const moe_dense* d, int64_t M, int product) {
  return d && M > 0 && M <= d->max_M ? kernel_of(kGemmForward, M, d->N, d->N, d->K, d->num_cus, product) : nullptr;
}

moe_status moe_dense_workspace_bytes(const moe_dense* d, int64_t M, int train, size_t* bytes) {
  if (!d || !bytes || M < 0 || M > d->max_M || train < 0 || train > 2) return MOE_ERR_INVALID_ARG;
  if (train == 2 && (d->act != MOE_ACT_NONE || d->N % 8 != 0)) train = 1;
  const size_t f = gemm_ws_bytes(kGemmForward, M, d->N, d->K, d->num_cus);
  const size_t b = train ? backward_layout(M, d->N, d->K, train == 1, train == 1, d->num_cus).bytes : 0;
  *bytes = f > b ? f : b;
  return MOE_OK;
}

moe_status moe_dense_forward(const moe_dense* d, int64_t M, const void* x, int64_t ldx, const void* residual,
                             int64_t ldr, void* y, int64_t ldy, int y_type, void* pre, int64_t ldp, int pre_type, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (!d || M < 0 || M > d->max_M) return MOE_ERR_INVALID_ARG;
  if (y_type != d->type && y_type != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (pre && pre_type != d->type && pre_type != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const size_t es = type_bytes(y_type);
  if (!operand_ok(x, ldx, d->K) || !matrix_ok(y, ldy, d->N, es)) return MOE_ERR_INVALID_ARG;
  if (residual && !matrix_ok(residual, ldr, d->N, es)) return MOE_ERR_INVALID_ARG;
  const size_t ps = type_bytes(pre_type);
  if (pre && !matrix_ok(pre, ldp, d->N, ps)) return MOE_ERR_INVALID_ARG;
  const size_t need = gemm_ws_bytes(kGemmForward, M, d->N, d->K, d->num_cus);
  moe_status st = check_ws(workspace, workspace_bytes, need);
  if (st != MOE_OK) return st;
  // in place (y is the residual itself) every element is read before it is written
  const bool in_place = residual == y && ldr == ldy;
  const Buf b[] = {{y, span(M, ldy, d->N, es), true},
                   {pre, span(M, ldp, d->N, ps), true},
                   {workspace, need, true},
                   {residual, in_place ? 0 : span(M, ldr, d->N, es), false},
                   {x, span(M, ldx, d->K, 2), false},
                   {d->w, 2 * (size_t)d->N * d->K, false},
                   {d->bias, 2 * (size_t)d->N, false}};
  st = check_buffers(b, 7, d->device);
  if (st != MOE_OK) return st;
  DeviceGuard guard(d->device);
  if (!guard.ok) return MOE_ERR_DEVICE;
  GemmArgs g{M, d->N, d->K, x, d->w, ldx, d->K, d->type, d->bias, residual, y, pre, ldr, ldy, ldp, d->act, y_type, pre_type, 0, 1,
             workspace};
  return launch_gemm(kGemmForward, g, d->num_cus, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_dense_backward(const moe_dense* d, int64_t M, const void* dy, int64_t lddy, const void* pre,
                              int64_t ldp, int pre_type, const void* x, int64_t ldx, void* dx, int64_t lddx, void* dw, void* dbias,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!d || M < 0 || M > d->max_M || (!dx && !dw && !dbias)) return MOE_ERR_INVALID_ARG;
  const int64_t N = d->N, K = d->K;
  if (d->act == MOE_ACT_NONE) pre = nullptr;
  if (pre && pre_type != d->type && pre_type != MOE_FP32) return MOE_ERR_INVALID_ARG;
  const size_t ps = type_bytes(pre_type);
  if (M > 0) {
    if (!matrix_ok(dy, lddy, N, 2) || (d->act != MOE_ACT_NONE && !matrix_ok(pre, ldp, N, ps))) return MOE_ERR_INVALID_ARG;
    if (dw && !operand_ok(x, ldx, K)) return MOE_ERR_INVALID_ARG;
    if (dx && !matrix_ok(dx, lddx, K, 2)) return MOE_ERR_INVALID_ARG;
  }
  if ((dw && !aligned16(dw)) || ((uintptr_t)dbias & 1)) return MOE_ERR_INVALID_ARG;
  // dy is dz itself where it needs no slope and its rows are an operand's
  const bool direct = d->act == MOE_ACT_NONE && N % 8 == 0 && (M == 0 || operand_ok(dy, lddy, N));
  const Backward l = backward_layout(M, N, K, !direct, !direct || dbias, d->num_cus);
  moe_status st = check_ws(workspace, workspace_bytes, l.bytes);
  if (st != MOE_OK) return st;
  const Buf b[] = {{dx, span(M, lddx, K, 2), true},
                   {dw, 2 * (size_t)N * K, true},
                   {dbias, 2 * (size_t)N, true},
                   {workspace, l.bytes, true},
                   {dy, span(M, lddy, N, 2), false},
                   {pre, span(M, ldp, N, ps), false},
                   {dw ? x : nullptr, span(M, ldx, K, 2), false},
                   {d->w, 2 * (size_t)N * K, false},
                   {d->bias, 2 * (size_t)N, false}};
  st = check_buffers(b, 9, d->device);
  if (st != MOE_OK) return st;
  DeviceGuard guard(d->device);
  if (!guard.ok) return MOE_ERR_DEVICE;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)workspace;
  const bool need_dz = !direct && (dx || dw);
  hipError_t e = hipSuccess;
  if (need_dz || dbias) {
    const SlopeArgs a{M, N, lddy, ldp, up8(N), dy, pre, need_dz ? ws + l.dz : nullptr, dbias, (float*)(ws + l.part), d->type, d->act, pre_type};
    e = launch_slope(a, s);
  }
  if (e == hipSuccess)
    e = products(M, N, K, d->type, d->num_cus, direct ? dy : ws + l.dz, direct ? lddy : up8(N), d->w, x, ldx, dx, lddx, dw, ws, l, s);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// ------------------------------------------------------------------ gated
moe_status moe_gated_create(int64_t I, int64_t H, int type, const void* w13, int activation, int64_t max_M,
                            moe_gated** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (I <= 0) return MOE_ERR_INVALID_ARG;
  if (I > kMaxOperandLd / 2) return MOE_ERR_UNSUPPORTED;
  moe_status st = check_sizes(2 * I, H, type, max_M);
  if (st != MOE_OK) return st;
  if (!w13 || !aligned16(w13) || activation <= MOE_ACT_NONE || activation > MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
  int dev, cus;
  const void* ptrs[1] = {w13};
  st = device_of(ptrs, 1, &dev, &cus);
  if (st != MOE_OK) return st;
  moe_gated* d = new (std::nothrow) moe_gated;
  if (!d) return MOE_ERR_INVALID_ARG;
  *d = moe_gated{I, H, max_M, type, activation, dev, cus, w13};
  *out = d;
  return MOE_OK;
}

void moe_gated_destroy(moe_gated* d) { delete d; }

const char* moe_gated_kernel(const moe_gated* d, int64_t M, int product) {
  return d && M > 0 && M <= d->max_M ? kernel_of(kGemmGated, M, d->I, 2 * d->I, d->H, d->num_cus, product) : nullptr;
}

moe_status moe_gated_workspace_bytes(const moe_gated* d, int64_t M, int train, size_t* bytes) {
  if (!d || !bytes || M < 0 || M > d->max_M || (train != 0 && train != 1)) return MOE_ERR_INVALID_ARG;
  const size_t f = gemm_ws_bytes(kGemmGated, M, d->I, d->H, d->num_cus);
  const size_t b = train ? backward_layout(M, 2 * d->I, d->H, true, false, d->num_cus).bytes : 0;
  *bytes = f > b ? f : b;
  return MOE_OK;
}

moe_status moe_gated_forward(const moe_gated* d, int64_t M, const void* x, int64_t ldx, void* h, int64_t ldh,
                             void* pre, int pre_type, void* workspace, size_t workspace_bytes, void* stream) {
  if (!d || M < 0 || M > d->max_M) return MOE_ERR_INVALID_ARG;
  if (pre && pre_type != d->type && pre_type != MOE_FP32) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const size_t ps = type_bytes(pre_type);
  if (!operand_ok(x, ldx, d->H) || !matrix_ok(h, ldh, d->I, 2) || ((uintptr_t)pre & (ps - 1))) return MOE_ERR_INVALID_ARG;
  const size_t need = gemm_ws_bytes(kGemmGated, M, d->I, d->H, d->num_cus);
  moe_status st = check_ws(workspace, workspace_bytes, need);
  if (st != MOE_OK) return st;
  const Buf b[] = {{h, span(M, ldh, d->I, 2), true},
                   {pre, span(M, 2 * d->I, 2 * d->I, ps), true},
                   {workspace, need, true},
                   {x, span(M, ldx, d->H, 2), false},
                   {d->w13, 4 * (size_t)d->I * d->H, false}};
  st = check_buffers(b, 5, d->device);
  if (st != MOE_OK) return st;
  DeviceGuard guard(d->device);
  if (!guard.ok) return MOE_ERR_DEVICE;
  GemmArgs g{M, d->I, d->H, x, d->w13, ldx, d->H, d->type, nullptr, nullptr, h, pre, 0, ldh, 2 * d->I, d->act, d->type, pre_type, 0, 1,
             workspace};
  return launch_gemm(kGemmGated, g, d->num_cus, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_gated_backward(const moe_gated* d, int64_t M, const void* dh, int64_t lddh, const void* pre,
                              int pre_type, const void* x, int64_t ldx, void* dx, int64_t lddx, void* dw13, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!d || M < 0 || M > d->max_M || (!dx && !dw13)) return MOE_ERR_INVALID_ARG;
  if (pre_type != d->type && pre_type != MOE_FP32) return MOE_ERR_INVALID_ARG;
  const size_t ps = type_bytes(pre_type);
  const int64_t N = 2 * d->I, H = d->H;
  if (M > 0) {
    if (!matrix_ok(dh, lddh, d->I, 2) || !pre || ((uintptr_t)pre & (ps - 1))) return MOE_ERR_INVALID_ARG;
    if (dw13 && !operand_ok(x, ldx, H)) return MOE_ERR_INVALID_ARG;
    if (dx && !matrix_ok(dx, lddx, H, 2)) return MOE_ERR_INVALID_ARG;
  }
  if (dw13 && !aligned16(dw13)) return MOE_ERR_INVALID_ARG;
  const Backward l = backward_layout(M, N, H, true, false, d->num_cus);
  moe_status st = check_ws(workspace, workspace_bytes, l.bytes);
  if (st != MOE_OK) return st;
  const Buf b[] = {{dx, span(M, lddx, H, 2), true},
                   {dw13, 2 * (size_t)N * H, true},
                   {workspace, l.bytes, true},
                   {dh, span(M, lddh, d->I, 2), false},
                   {pre, span(M, N, N, ps), false},
                   {dw13 ? x : nullptr, span(M, ldx, H, 2), false},
                   {d->w13, 2 * (size_t)N * H, false}};
  st = check_buffers(b, 7, d->device);
  if (st != MOE_OK) return st;
  DeviceGuard guard(d->device);
  if (!guard.ok) return MOE_ERR_DEVICE;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)workspace;
  const GatedSlopeArgs a{M, d->I, lddh, up8(N), dh, pre, ws + l.dz, d->type, d->act, pre_type};
  hipError_t e = launch_gated_slope(a, s);
  if (e == hipSuccess)
    e = products(M, N, H, d->type, d->num_cus, ws + l.dz, up8(N), d->w13, x, ldx, dx, lddx, dw13, ws, l, s);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
