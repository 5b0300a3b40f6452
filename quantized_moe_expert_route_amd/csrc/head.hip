// What reads the output head's logits: scores of given tokens (log probability,
// entropy, largest alternatives) and distillation from a teacher's top logits.
#include <algorithm>

#include "head.h"
#include "mxfp4.h"

namespace qmoe {

__device__ __forceinline__ float load_logit(const void* p, int type, int64_t i) {
  if (type == MOE_FP32) return reinterpret_cast<const float*>(p)[i];
  const uint16_t b = reinterpret_cast<const uint16_t*>(p)[i];
  return type == MOE_FP16 ? fp16_value(b) : bf16_value(b);
}
__device__ __forceinline__ void store_grad(void* p, int type, int64_t i, float v) {
  if (type == MOE_FP32) reinterpret_cast<float*>(p)[i] = v;
  else reinterpret_cast<uint16_t*>(p)[i] = type == MOE_FP16 ? fp16_bits(v) : bf16_bits(v);
}
__device__ __forceinline__ const void* row_of(const void* z, int type, int64_t m, int64_t ld) {
  return reinterpret_cast<const uint8_t*>(z) + m * ld * (type == MOE_FP32 ? 4 : 2);
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

constexpr int kRowThreads = 256;

// Maximum (NaN if there is one) and the sums of e = exp(c z - max) and of e (c z -
// max) over a row, the same in all threads. An infinite maximum: sums NaN.
struct RowSums {
  float max;
  double sum, mean;
};
__device__ RowSums row_sums(const void* row, int type, int64_t V, float c) {
  constexpr int W = kRowThreads / 64;
  __shared__ float lm[W];
  __shared__ double ls[W], lt[W];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  float mx = -INFINITY;
  bool nan = false;
  for (int64_t v = threadIdx.x; v < V; v += kRowThreads) {
    const float z = load_logit(row, type, v) * c;
    nan |= z != z;
    mx = fmaxf(mx, z);
  }
  mx = wave_max(__ballot(nan) ? INFINITY : mx);
  const bool any = __ballot(nan) != 0;
  if (lane == 0) lm[wave] = any ? NAN : mx;
  __syncthreads();
  mx = lm[0];
  for (int w = 1; w < W; ++w) mx = mx != mx || lm[w] != lm[w] ? NAN : fmaxf(mx, lm[w]);
  double s = 0, t = 0;
  for (int64_t v = threadIdx.x; v < V; v += kRowThreads) {
    const float d = load_logit(row, type, v) * c - mx, e = expf(d);
    s += e;
    if (e != 0.f) t += (double)e * d;
  }
  s = wave_sum(s), t = wave_sum(t);
  if (lane == 0) ls[wave] = s, lt[wave] = t;
  __syncthreads();
  s = t = 0;
  for (int w = 0; w < W; ++w) s += ls[w], t += lt[w];
  return {mx, s, t};
}

__global__ __launch_bounds__(kRowThreads) void scores_kernel(const ScoresArgs a) {
  __shared__ uint64_t best[kRowThreads / 64];
  const int64_t m = blockIdx.x;
  const void* row = row_of(a.z, a.type, m, a.ldz);
  const RowSums r = row_sums(row, a.type, a.V, 1.f);
  const double logs = log(r.sum), lse = r.max + logs;
  if (threadIdx.x == 0) {
    if (a.tokens) {
      const int64_t t = a.tokens[m];
      a.logprobs[m] = t >= 0 && t < a.V ? (float)(load_logit(row, a.type, t) - lse) : NAN;
      if (!(fabsf(r.max) < INFINITY)) a.logprobs[m] = NAN;
    }
    if (a.entropy) a.entropy[m] = fabsf(r.max) < INFINITY ? (float)(logs - r.mean / r.sum) : NAN;
    if (a.lse) a.lse[m] = fabsf(r.max) < INFINITY ? (float)lse : r.max;
  }
  // one alternative after another: the largest key below the last one's
  uint64_t last = ~0ull;
  for (int j = 0; j < a.k; ++j) {
    uint64_t key = 0;
    for (int64_t v = threadIdx.x; v < a.V; v += kRowThreads) {
      const uint64_t q = ((uint64_t)order_key(load_logit(row, a.type, v)) << 32) | (uint32_t)~(uint32_t)v;
      if (q < last && q > key) key = q;
    }
    key = wave_max_u64(key);
    if ((threadIdx.x & 63) == 0) best[wave_id()] = key;
    __syncthreads();
    for (int w = 0; w < kRowThreads / 64; ++w) key = best[w] > key ? best[w] : key;
    __syncthreads();
    last = key;
    if (threadIdx.x == 0) {
      a.top_ids[m * a.k + j] = (int32_t)~(uint32_t)key;
      a.top_logprobs[m * a.k + j] = fabsf(r.max) < INFINITY ? (float)(key_to_float((uint32_t)(key >> 32)) - lse) : NAN;
    }
  }
}

size_t scores_ws_bytes(int64_t, int64_t, int64_t, int, int) { return 0; }

hipError_t launch_scores(const ScoresArgs& a, int, hipStream_t stream) {
  return launch_k(scores_kernel, dim3((unsigned)a.M), dim3(kRowThreads), 0, stream, Ev{}, a);
}

// ----------------------------------------------------------------- distillation
// The row's slots: token (-1 empty) and p, from the first wave.
__device__ bool teacher(const DistillArgs& a, int64_t m, int32_t* id, double* p, double* logp) {
  __shared__ int some;
  if (threadIdx.x < 64) {
    const int j = threadIdx.x;
    int32_t v = j < a.k ? a.ids[m * a.k + j] : -1;
    if (v < 0 || v >= a.V) v = -1;
    const float t = v >= 0 ? a.t[m * a.k + j] / a.temperature : -INFINITY;
    const float mx = wave_max(t);
    const double e = t > -INFINITY || t != t ? exp((double)t - mx) : 0.0;
    const double s = wave_sum(e);
    id[j] = v;
    p[j] = v >= 0 ? e / s : 0.0;
    logp[j] = (double)t - mx - log(s);
    const bool any = __ballot(v >= 0) != 0;
    if (j == 0) some = any;
  }
  __syncthreads();
  return some;
}

template <int PASS>
__global__ __launch_bounds__(kRowThreads) void distill_kernel(const DistillArgs a) {
  __shared__ int32_t id[64];
  __shared__ double p[64], logp[64];  // 64 bits: the loss of masked logits comes near binary32's largest number
  const int64_t m = blockIdx.x;
  const void* row = row_of(a.z, a.type, m, a.ldz);
  const float c = 1.f / a.temperature;
  const bool some = teacher(a, m, id, p, logp);
  double lse;
  if constexpr (PASS == kDistillBackward) {
    lse = a.lse[m];
  } else {
    const RowSums r = row_sums(row, a.type, a.V, c);
    const bool ok = fabsf(r.max) < INFINITY;
    lse = ok ? r.max + log(r.sum) : r.max;
    if (threadIdx.x < 64) {
      const int j = threadIdx.x;
      double l = 0;
      if (p[j] != 0) l = p[j] * (logp[j] - ((double)load_logit(row, a.type, id[j]) * c - lse));
      l = wave_sum(l);
      if (j == 0) a.loss[m] = !some ? 0.f : ok ? (float)l : NAN;
      if (j == 0 && a.lse) a.lse[m] = (float)lse;
    }
  }
  if constexpr (PASS == kDistillForward) return;
  if (!(fabs(lse) < INFINITY)) lse = NAN;
  uint8_t* out = reinterpret_cast<uint8_t*>(a.dz) + m * a.lddz * (a.grad_type == MOE_FP32 ? 4 : 2);
  const float f = some ? a.weight[m] * c : 0.f;
  // a slot's gradient, of its first slot: z is read before anything is written (dz may be z)
  float at = 0.f;
  bool mine = false;
  if (threadIdx.x < 64 && id[threadIdx.x] >= 0) {
    const int j = threadIdx.x;
    mine = true;
    double s = 0;
    for (int i = 0; i < a.k; ++i)
      if (id[i] == id[j]) {
        if (i < j) mine = false;
        s += p[i];
      }
    at = f * (float)(expf(load_logit(row, a.type, id[j]) * c - (float)lse) - s);
  }
  __syncthreads();
  for (int64_t v = threadIdx.x; v < a.V; v += kRowThreads)
    store_grad(out, a.grad_type, v, some ? f * expf(load_logit(row, a.type, v) * c - (float)lse) : 0.f);
  __syncthreads();
  if (mine) store_grad(out, a.grad_type, id[threadIdx.x], at);
}

size_t distill_ws_bytes(int64_t, int64_t, int, int) { return 0; }

hipError_t launch_distill(DistillPass pass, const DistillArgs& a, int, hipStream_t stream) {
  const dim3 grid((unsigned)a.M), block(kRowThreads);
  if (pass == kDistillForward) return launch_k(distill_kernel<kDistillForward>, grid, block, 0, stream, Ev{}, a);
  if (pass == kDistillBackward) return launch_k(distill_kernel<kDistillBackward>, grid, block, 0, stream, Ev{}, a);
  return launch_k(distill_kernel<kDistillBoth>, grid, block, 0, stream, Ev{}, a);
}

}  // namespace qmoe
