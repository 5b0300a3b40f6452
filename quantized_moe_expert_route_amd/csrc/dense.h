// Handles and launch interface of the layers in 16 bits: the matrix product with
// its epilogue and the gated feed-forward block, forward and backward.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "qmoe.h"

struct moe_dense {
  int64_t N, K, max_M;
  int type, act;
  int device, num_cus;
  const void* w;
  const void* bias;
};

struct moe_gated {
  int64_t I, H, max_M;
  int type, act;
  int device, num_cus;
  const void* w13;
};

namespace qmoe {

// C [rows, cols] = A B^T over K elements, both operands of 16 bits. An operand's
// element (row, k) lies at row * ld + k, or for `by_k` at k * ld + row.
struct GemmArgs {
  int64_t rows, cols, K;
  const void* a;
  const void* b;
  int64_t lda, ldb;
  int type;
  // epilogue: y = act(C + bias) + residual, C itself to pre; gated: columns
  // [0, cols) gate and [cols, 2 cols) up of B's rows, y = act(gate) up, both to pre
  const void* bias;
  const void* residual;
  void* y;
  void* pre;
  int64_t ldr, ldy, ldp;
  int act, y_type, pre_type;
  int vec;  // set by launch_gemm: which of the matrices move in 16-byte pieces
  int splits;  // parts of K, set by launch_gemm
  void* ws;  // gemm_ws_bytes of the splits' sums
};

enum GemmKind {
  kGemmForward = 0,  // both operands along K: y = x w^T
  kGemmGated = 1,    // the same, two products
  kGemmInput = 2,    // b by_k: dx = dz w
  kGemmWeight = 3,   // both by_k: dw = dz^T x
};

hipError_t launch_gemm(GemmKind kind, const GemmArgs& a, int cus, hipStream_t stream);
// bytes of GemmArgs::ws that the launch wants for these sizes
size_t gemm_ws_bytes(GemmKind kind, int64_t rows, int64_t cols, int64_t K, int cus);

const char* gemm_kernel_name(GemmKind kind, int64_t rows, int64_t cols, int64_t K, int cus);  // rows, cols > 0

// dz [M, ldz] (ldz a multiple of 8 from N on, columns past N zero) = dy act'(pre),
// or dy itself without an activation; dbias [N] = its column sums before the rounding
// (NULL: none; dz NULL: only dbias). part: fp32 [dbias_parts(M), N].
struct SlopeArgs {
  int64_t M, N, lddy, ldp, ldz;
  const void* dy;
  const void* pre;
  void* dz;
  void* dbias;
  float* part;
  int type, act, pre_type;
};
constexpr int kBiasRows = 32;  // rows a partial sum of dbias takes (2^20 rows: 2^15 workgroups)
inline int64_t dbias_parts(int64_t M) { return (M + kBiasRows - 1) / kBiasRows; }
hipError_t launch_slope(const SlopeArgs& a, hipStream_t stream);

// dz [M, ldz] (from 2 I on zero) = [dh u act'(g), dh act(g)] of pre [M, 2 I] = [g u].
struct GatedSlopeArgs {
  int64_t M, I, lddh, ldz;
  const void* dh;
  const void* pre;
  void* dz;
  int type, act, pre_type;
};
hipError_t launch_gated_slope(const GatedSlopeArgs& a, hipStream_t stream);

}  // namespace qmoe
