// Matrix products of 16-bit operands with their epilogues, and the elementwise
// part of their backward passes.
//
// One product serves all: C [rows, cols] = A B^T, where forward both operands lie
// along K (y = x w^T), for the input's gradient B lies across it (dx = dz w), for the
// weight's both do (dw = dz^T x). Products of 16-bit values are exact in binary32
// and summed there by the MFMA, whose operand of a lane is 8 elements along K.
#include <algorithm>

#include "gemm_tile.h"

namespace qmoe {

// One element of C into y (and pre).
template <bool F16, GemmKind KIND>
__device__ __forceinline__ void store1(const GemmArgs& a, int64_t m, int64_t n, float c, float up) {
  uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + m * a.ldy + n;
  if constexpr (KIND == kGemmGated) {
    if (a.pre) {
      uint16_t* p = reinterpret_cast<uint16_t*>(a.pre) + m * a.ldp + n;
      p[0] = bits16<F16>(c);
      p[a.cols] = bits16<F16>(up);
    }
    *y = bits16<F16>(act_value(a.act, c) * up);
  } else if constexpr (KIND == kGemmForward) {
    if (a.bias) c += value16<F16>(reinterpret_cast<const uint16_t*>(a.bias)[n]);
    if (a.pre) reinterpret_cast<uint16_t*>(a.pre)[m * a.ldp + n] = bits16<F16>(c);
    c = act_value(a.act, c);
    if (a.y_type == MOE_FP32) {
      if (a.residual) c += reinterpret_cast<const float*>(a.residual)[m * a.ldr + n];
      reinterpret_cast<float*>(a.y)[m * a.ldy + n] = c;
    } else {
      if (a.residual) c += value16<F16>(reinterpret_cast<const uint16_t*>(a.residual)[m * a.ldr + n]);
      *y = bits16<F16>(c);
    }
  } else {
    *y = bits16<F16>(c);
  }
}

// 64 x 64 of C a workgroup, through LDS in K-steps of 32, every access checked.
template <bool F16, GemmKind KIND>
__global__ __launch_bounds__(256) void gemm_simple_kernel(const GemmArgs a, int tiles_m) {
  constexpr int B = KIND == kGemmGated ? 2 : 1;
  __shared__ uint16_t as[64][40], bs[B][64][40];  // rows of 32 K (and 8 of padding)
  const int wave = wave_id(), lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t m0 = (int64_t)(blockIdx.x % tiles_m) * 64, n0 = (int64_t)(blockIdx.x / tiles_m) * 64;
  auto stage = [&](uint16_t(&dst)[64][40], const void* p, int64_t ld, int64_t r0, int64_t rows, int64_t k0, bool by_k) {
    const uint16_t* src = reinterpret_cast<const uint16_t*>(p);
    for (int i = threadIdx.x; i < 64 * 32; i += 256) {
      const int row = by_k ? i & 63 : i >> 5, k = by_k ? i >> 6 : i & 31;
      const bool in = r0 + row < rows && k0 + k < a.K;
      dst[row][k] = in ? src[by_k ? (k0 + k) * ld + r0 + row : (r0 + row) * ld + k0 + k] : (uint16_t)0;
    }
  };
  v4f acc[B][4];
  for (int q = 0; q < B; ++q)
    for (int t = 0; t < 4; ++t) acc[q][t] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int64_t k0 = 0; k0 < a.K; k0 += 32) {
    stage(as, a.a, a.lda, m0, a.rows, k0, KIND == kGemmWeight);
    for (int q = 0; q < B; ++q)
      stage(bs[q], reinterpret_cast<const uint16_t*>(a.b) + q * a.cols * a.ldb, a.ldb, n0, a.cols, k0, KIND >= kGemmInput);
    __syncthreads();
    const uint4 x = ld16(&as[16 * wave + r][8 * g]);
    for (int q = 0; q < B; ++q)
      for (int t = 0; t < 4; ++t) acc[q][t] = mfma16<F16>(ld16(&bs[q][16 * t + r][8 * g]), x, acc[q][t]);
    __syncthreads();
  }
  const int64_t m = m0 + 16 * wave + r;
  if (m >= a.rows) return;
  for (int t = 0; t < 4; ++t)
    for (int i = 0; i < 4; ++i) {
      const int64_t n = n0 + 16 * t + 4 * g + i;
      if (n < a.cols) store1<F16, KIND>(a, m, n, acc[0][t][i], acc[B - 1][t][i]);
    }
}

template <bool F16, GemmKind KIND>
static hipError_t simple(const GemmArgs& a, hipStream_t stream) {
  const int64_t tm = (a.rows + 63) / 64, tn = (a.cols + 63) / 64;
  return launch_k(gemm_simple_kernel<F16, KIND>, dim3((unsigned)(tm * tn)), dim3(256), 0, stream, Ev{}, a, (int)tm);
}

size_t gemm_ws_bytes(GemmKind, int64_t, int64_t, int64_t, int, int) { return 0; }

template <bool F16, GemmKind KIND>
static hipError_t launch(const GemmArgs& a, hipStream_t stream) {
  if (a.rows <= 64) return simple<F16, KIND>(a, stream);
  return launch_tile<F16, KIND, 8, 4, 2, 4>(a, stream);
}

hipError_t launch_gemm(GemmKind kind, const GemmArgs& args, int, hipStream_t stream) {
  GemmArgs a = args;
  const int64_t es = a.y_type == MOE_FP32 ? 4 : 2;
  auto vec = [](const void* p, int64_t ld, int64_t elem) { return p && ((uintptr_t)p & 15) == 0 && ld * elem % 16 == 0; };
  a.vec = (vec(a.y, a.ldy, es) ? kVecY : 0) | (vec(a.residual, a.ldr, es) ? kVecResidual : 0) |
          (vec(a.pre, a.ldp, 2) && (kind != kGemmGated || a.cols % 8 == 0) ? kVecPre : 0) | (vec(a.bias, 0, 2) ? kVecBias : 0);
  const bool f16 = a.type == MOE_FP16;
  switch (kind) {
    case kGemmForward: return f16 ? launch<true, kGemmForward>(a, stream) : launch<false, kGemmForward>(a, stream);
    case kGemmGated: return f16 ? launch<true, kGemmGated>(a, stream) : launch<false, kGemmGated>(a, stream);
    case kGemmInput: return f16 ? launch<true, kGemmInput>(a, stream) : launch<false, kGemmInput>(a, stream);
    default: return f16 ? launch<true, kGemmWeight>(a, stream) : launch<false, kGemmWeight>(a, stream);
  }
}

// ----------------------------------------------------------------- backward, elementwise
// A thread takes one column of kBiasRows rows. dbias's partial sums are joined in
// the order of the rows by a second launch.
template <bool F16>
__global__ __launch_bounds__(256) void slope_kernel(const SlopeArgs a) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m0 = (int64_t)blockIdx.y * kBiasRows, m1 = min(m0 + kBiasRows, a.M);
  const int64_t cols = a.dz ? a.ldz : a.N;
  if (n >= cols) return;
  float sum = 0.f;
  for (int64_t m = m0; m < m1; ++m) {
    float v = 0.f;
    if (n < a.N) {
      v = value16<F16>(reinterpret_cast<const uint16_t*>(a.dy)[m * a.lddy + n]);
      float y;
      if (a.act) v *= act_slope(a.act, value16<F16>(reinterpret_cast<const uint16_t*>(a.pre)[m * a.ldp + n]), y);
    }
    if (a.dz) reinterpret_cast<uint16_t*>(a.dz)[m * a.ldz + n] = bits16<F16>(v);
    sum += v;
  }
  if (a.dbias && n < a.N) a.part[blockIdx.y * a.N + n] = sum;
}

template <bool F16>
__global__ __launch_bounds__(256) void dbias_kernel(const float* __restrict__ part, uint16_t* __restrict__ dbias, int64_t N,
                                                    int64_t parts) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float sum = 0.f;
  for (int64_t p = 0; p < parts; ++p) sum += part[p * N + n];
  dbias[n] = bits16<F16>(sum);
}

hipError_t launch_slope(const SlopeArgs& a, hipStream_t stream) {
  const bool f16 = a.type == MOE_FP16;
  const int64_t parts = dbias_parts(a.M);
  hipError_t e = hipSuccess;
  if (a.M > 0) {
    const dim3 grid((unsigned)(((a.dz ? a.ldz : a.N) + 255) / 256), (unsigned)parts);
    e = f16 ? launch_k(slope_kernel<true>, grid, dim3(256), 0, stream, Ev{}, a)
            : launch_k(slope_kernel<false>, grid, dim3(256), 0, stream, Ev{}, a);
  }
  if (e == hipSuccess && a.dbias) {
    const dim3 grid((unsigned)((a.N + 255) / 256));
    e = f16 ? launch_k(dbias_kernel<true>, grid, dim3(256), 0, stream, Ev{}, (const float*)a.part, (uint16_t*)a.dbias, a.N, parts)
            : launch_k(dbias_kernel<false>, grid, dim3(256), 0, stream, Ev{}, (const float*)a.part, (uint16_t*)a.dbias, a.N, parts);
  }
  return e;
}

template <bool F16>
__global__ __launch_bounds__(256) void gated_slope_kernel(const GatedSlopeArgs a) {
  const int64_t total = a.M * a.ldz;
  for (int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x; o < total; o += (int64_t)gridDim.x * 256) {
    const int64_t m = o / a.ldz, n = o - m * a.ldz;
    float v = 0.f;
    if (n < 2 * a.I) {
      const int64_t i = n < a.I ? n : n - a.I;
      const uint16_t* p = reinterpret_cast<const uint16_t*>(a.pre) + m * 2 * a.I + i;
      const float d = value16<F16>(reinterpret_cast<const uint16_t*>(a.dh)[m * a.lddh + i]);
      float value;
      const float slope = act_slope(a.act, value16<F16>(p[0]), value);
      v = n < a.I ? d * value16<F16>(p[a.I]) * slope : d * value;
    }
    reinterpret_cast<uint16_t*>(a.dz)[o] = bits16<F16>(v);
  }
}

hipError_t launch_gated_slope(const GatedSlopeArgs& a, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>((a.M * a.ldz + 255) / 256, 1 << 16));
  return a.type == MOE_FP16 ? launch_k(gated_slope_kernel<true>, grid, dim3(256), 0, stream, Ev{}, a)
                            : launch_k(gated_slope_kernel<false>, grid, dim3(256), 0, stream, Ev{}, a);
}

}  // namespace qmoe
