// Handles and launch interface of the operators beside the routed-MoE call:
// the router, the MXFP4 linear layer, the few-token MoE layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "qmoe.h"

struct moe_router {
  int64_t E, H, max_M;
  int x_type, w_type;
  int device, num_cus;
  const void* w;
};

struct moe_linear {
  int64_t N, K, max_M;
  int x_type;
  int device, num_cus;
  const uint8_t* wp;
  const uint8_t* sp;
  const void* bias;
};

namespace qmoe {

struct RouterArgs {
  int64_t M, E, H, ldx;
  const void* x;
  const void* w;
  float* logits;
  int x_type, w_type;
};
hipError_t launch_router(const RouterArgs& a, int cus, hipStream_t stream, Ev ev = {});
const char* router_kernel_name(int64_t M, int64_t E, int cus);  // that it launches, M > 0

struct LinearArgs {
  int64_t M, N, K, ldx, ldr, ldy;
  const void* x;
  const uint8_t* wp;
  const uint8_t* sp;
  const void* bias;      // x's type, or NULL
  const void* residual;  // y's type, or NULL
  void* y;
  int x_type, y_type;
  int vec;  // N, the strides and the addresses allow four columns (1) or 16 bytes (2) in one access
};
hipError_t launch_pack_linear(const void* w, const void* s, int64_t N, int64_t K, void* wp, void* sp,
                              hipStream_t stream);
hipError_t launch_linear(const LinearArgs& a, int cus, hipStream_t stream);
const char* linear_kernel_name(int64_t M, int64_t N, int64_t K, bool f16, int cus);  // that it launches, M > 0

// Few-token MoE layer: most (token, slot) entries and the widest x a call takes
// (8 waves hold at most 8 K-steps of 128 each as register operands).
constexpr int kLayerMaxEntries = 256;
constexpr int kLayerMaxH = 8192;
constexpr int kLayerListBytes = 16 + (2 + 1 + 16) * kLayerMaxEntries;  // PickList of layer.hip

// Shapes of plans that moe_layer_forward may run on (others have no workspace for it).
inline bool layer_shape(const moe_shape& s) { return s.shared_I == 0 && s.H <= kLayerMaxH; }

struct LayerArgs {
  int64_t M;
  const void* x;
  const void* w13;
  const void* s13;
  const void* w2;
  const void* s2;
  void* out;
  hipStream_t stream;
};
// on the plan's workspace (topk_ids, topk_w and the regions of its own)
hipError_t launch_layer(const moe_plan* p, const moe_router* router, const LayerArgs& a);

}  // namespace qmoe
