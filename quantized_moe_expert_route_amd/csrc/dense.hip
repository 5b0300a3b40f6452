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

namespace {

// The tiles a product may run on.
struct Tile {
  int rows, cols;  // of C (gated: of both products, half of them columns of y)
};
enum { k256x256, k256x192, k128x128, k64x64, kTiles };
constexpr Tile kTile[kTiles] = {{256, 256}, {256, 192}, {128, 128}, {64, 64}};

struct Choice {
  int tile, splits;
};

Choice choose(GemmKind kind, int64_t rows, int64_t cols, int64_t K, int cus) {
  // Rounds of workgroups over the CUs times a round's time per K-step
  constexpr int per[kTiles] = {100, 76, 36, 18};
  constexpr int wide[kTiles] = {1, 1, 2, 2};  // workgroups a CU
  const int64_t steps = std::max<int64_t>((K + 63) / 64, 1);
  Choice best{0, 1};
  int64_t least = INT64_MAX;
  for (int i = 0; i < kTiles; ++i) {
    const int64_t bn = kind == kGemmGated ? kTile[i].cols / 2 : kTile[i].cols;
    const int64_t tiles = ((rows + kTile[i].rows - 1) / kTile[i].rows) * ((cols + bn - 1) / bn);
    // splits of at least 8 steps each, while they fit the chip at once
    int64_t splits = std::min(std::max<int64_t>(cus * wide[i] / tiles, 1), std::max<int64_t>(steps / 8, 1));
    splits = std::min<int64_t>(splits, 32);
    const int64_t part = (steps + splits - 1) / splits;
    splits = (steps + part - 1) / part;  // none of them empty
    const int64_t rounds = (tiles * splits + cus * wide[i] - 1) / (cus * wide[i]);
    const int64_t cost = rounds * (part + 8) * per[i] * wide[i] + (splits > 1 ? 800 : 0);
    if (cost < least) least = cost, best = {i, (int)splits};
  }
  return best;
}

template <bool F16, GemmKind KIND>
hipError_t launch(GemmArgs a, const Choice& c, hipStream_t stream) {
  a.splits = c.splits;
  hipError_t e;
  switch (c.tile) {
    case k256x256: e = launch_tile<F16, KIND, 8, 4, 2, 4, 2>(a, stream); break;
    case k256x192: e = launch_tile<F16, KIND, 4, 6, 4, 2, 2>(a, stream); break;
    case k128x128: e = launch_tile<F16, KIND, 4, 4, 2, 2, 2>(a, stream); break;
    default: e = launch_tile<F16, KIND, 2, 2, 2, 2, 4>(a, stream); break;
  }
  if (e == hipSuccess && c.splits > 1) {
    const int64_t pieces = a.rows * ((a.cols + 7) / 8);
    e = launch_k(split_join_kernel<F16, KIND>, dim3((unsigned)std::min<int64_t>((pieces + 255) / 256, 4096)), dim3(256),
                 0, stream, Ev{}, a);
  }
  return e;
}

}  // namespace

size_t gemm_ws_bytes(GemmKind kind, int64_t rows, int64_t cols, int64_t K, int, int cus) {
  if (rows == 0 || cols == 0) return 0;
  const Choice c = choose(kind, rows, cols, K, cus);
  return c.splits > 1 ? (size_t)c.splits * rows * ((cols + 7) / 8 * 8) * (kind == kGemmGated ? 8 : 4) : 0;
}

hipError_t launch_gemm(GemmKind kind, const GemmArgs& args, int cus, hipStream_t stream) {
  GemmArgs a = args;
  const int64_t es = a.y_type == MOE_FP32 ? 4 : 2;
  auto vec = [](const void* p, int64_t ld, int64_t elem) { return p && ((uintptr_t)p & 15) == 0 && ld * elem % 16 == 0; };
  a.vec = (vec(a.y, a.ldy, es) ? kVecY : 0) | (vec(a.residual, a.ldr, es) ? kVecResidual : 0) |
          (vec(a.pre, a.ldp, 2) && (kind != kGemmGated || a.cols % 8 == 0) ? kVecPre : 0) | (vec(a.bias, 0, 2) ? kVecBias : 0);
  const bool f16 = a.type == MOE_FP16;
  const Choice c = choose(kind, a.rows, a.cols, a.K, cus);
  switch (kind) {
    case kGemmForward: return f16 ? launch<true, kGemmForward>(a, c, stream) : launch<false, kGemmForward>(a, c, stream);
    case kGemmGated: return f16 ? launch<true, kGemmGated>(a, c, stream) : launch<false, kGemmGated>(a, c, stream);
    case kGemmInput: return f16 ? launch<true, kGemmInput>(a, c, stream) : launch<false, kGemmInput>(a, c, stream);
    default: return f16 ? launch<true, kGemmWeight>(a, c, stream) : launch<false, kGemmWeight>(a, c, stream);
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
