// Handles and launch interface of the operators that read the output head's
// logits: the scores of given tokens, distillation from a teacher's top logits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "qmoe.h"

struct moe_scores {
  int64_t V, k, max_M;
  int type;
  int device, num_cus;
};

struct moe_distill {
  int64_t V, k, max_M;
  int type, grad_type;
  float temperature;
  int device, num_cus;
};

namespace qmoe {

constexpr int kMaxTop = 64;

struct ScoresArgs {
  int64_t M, V, ldz;
  const void* z;
  const int32_t* tokens;
  float* logprobs;
  float* entropy;
  float* lse;
  float* top_logprobs;
  int32_t* top_ids;
  int k, type;
  void* ws;
};
hipError_t launch_scores(const ScoresArgs& a, int cus, hipStream_t stream);
size_t scores_ws_bytes(int64_t M, int64_t V, int64_t k, int cus);
const char* scores_kernel_name(int64_t M, int64_t V, int64_t k, int cus);  // M > 0

struct DistillArgs {
  int64_t M, V, ldz, lddz;
  const void* z;
  const int32_t* ids;
  const float* t;
  const float* weight;
  float* loss;
  float* lse;  // written forward, read backward
  void* dz;
  float temperature;
  int k, type, grad_type;
  void* ws;
};
enum DistillPass { kDistillForward = 0, kDistillBackward = 1, kDistillBoth = 2 };
hipError_t launch_distill(DistillPass pass, const DistillArgs& a, int cus, hipStream_t stream);
size_t distill_ws_bytes(int64_t M, int64_t V, int type, int cus);
const char* distill_kernel_name(DistillPass pass, int64_t M, int64_t V, int type, int grad_type, int cus);  // M > 0

}  // namespace qmoe
