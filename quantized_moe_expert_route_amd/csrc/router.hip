// Router projection: logits[m][e] = sum_h x[m][h] w[e][h], one rounding to
// binary32. x bf16 or fp16, w bf16 or fp32.
//
// The sums are float64: the routing compares logits, and with sums exact to
// ~2^-50 two logits swap places only where their exact values round to the
// same binary32 number, whatever order or split a kernel adds in.
#include <algorithm>

#include "internal.h"
#include "mxfp4.h"
#include "ops.h"

namespace qmoe {

// 8 consecutive elements of a row as float.
template <int TYPE>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (TYPE == MOE_FP32) {
    const float4 a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    const float4 b = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 q = ld16(reinterpret_cast<const uint16_t*>(p) + i);
    const uint32_t d[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (TYPE == MOE_BF16) {
        v[2 * j] = __uint_as_float(d[j] << 16);
        v[2 * j + 1] = __uint_as_float(d[j] & 0xFFFF0000u);
      } else {
        v[2 * j] = fp16_value((uint16_t)(d[j] & 0xFFFFu));
        v[2 * j + 1] = fp16_value((uint16_t)(d[j] >> 16));
      }
    }
  }
}

__device__ __forceinline__ double shfl_xor_f64(double v, int o) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __shfl_xor((uint32_t)u, o, kWave), hi = __shfl_xor((uint32_t)(u >> 32), o, kWave);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// One expert and up to T tokens a workgroup: 256 threads over chunks of 8
// elements, one float64 sum per token and thread, added over lanes, then
// waves.
template <int XT, int WT, int T>
__global__ __launch_bounds__(256) void router_kernel(const RouterArgs a) {
  __shared__ double red[4][T];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t e = blockIdx.x, m0 = (int64_t)blockIdx.y * T;
  const int mt = (int)min((int64_t)T, a.M - m0);
  const int H = (int)a.H;
  double acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) acc[t] = 0.0;
  for (int c = threadIdx.x * 8; c < H; c += 256 * 8) {
    float w[8];
    load8<WT>(a.w, e * a.H + c, w);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      float x[8];
      load8<XT>(a.x, (m0 + min(t, mt - 1)) * a.ldx + c, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[t] = fma((double)x[i], (double)w[i], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) acc[t] += shfl_xor_f64(acc[t], o);
    if (lane == 0) red[wave][t] = acc[t];
  }
  __syncthreads();
  if ((int)threadIdx.x < mt) {
    const int t = threadIdx.x;
    a.logits[(m0 + t) * a.E + e] = (float)(red[0][t] + red[1][t] + red[2][t] + red[3][t]);
  }
}

template <int XT, int WT>
static hipError_t launch_types(const RouterArgs& a, hipStream_t stream) {
  if (a.M <= 1)
    return launch_k(router_kernel<XT, WT, 1>, dim3((unsigned)a.E, 1), dim3(256), 0, stream, Ev{}, a);
  if (a.M <= 4)
    return launch_k(router_kernel<XT, WT, 4>, dim3((unsigned)a.E, 1), dim3(256), 0, stream, Ev{}, a);
  return launch_k(router_kernel<XT, WT, 8>, dim3((unsigned)a.E, (unsigned)((a.M + 7) / 8)), dim3(256), 0, stream, Ev{},
                  a);
}

hipError_t launch_router(const RouterArgs& a, int cus, hipStream_t stream) {
  if (a.x_type == MOE_BF16)
    return a.w_type == MOE_BF16 ? launch_types<MOE_BF16, MOE_BF16>(a, stream)
                                : launch_types<MOE_BF16, MOE_FP32>(a, stream);
  return a.w_type == MOE_BF16 ? launch_types<MOE_FP16, MOE_BF16>(a, stream)
                              : launch_types<MOE_FP16, MOE_FP32>(a, stream);
}

}  // namespace qmoe
