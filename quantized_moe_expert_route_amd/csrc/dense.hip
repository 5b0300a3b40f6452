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
// A lane takes eight columns, a wave a row's 512 at a time; the four waves of a
// workgroup take kBiasRows rows in turn. dbias's sums of a workgroup are joined in the
// order of its waves, those of all workgroups in the order of the rows by a second
// launch. Bound by memory.
template <bool F16>
__global__ __launch_bounds__(256) void slope_kernel(const SlopeArgs a, int vec) {
  __shared__ float sums[4][512];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int64_t n = ((int64_t)blockIdx.x * 64 + lane) * 8;
  const int64_t m0 = (int64_t)blockIdx.y * kBiasRows, m1 = min(m0 + kBiasRows, a.M);
  const int left = (int)max((int64_t)0, min((int64_t)8, a.N - n));
  float sum[8] = {};
  if (left > 0) {
    with_act(a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll 4
      for (int64_t m = m0 + wave; m < m1; m += 4) {
        float v[8], p[8];
        read8<F16, false>(reinterpret_cast<const uint16_t*>(a.dy) + m * a.lddy + n, vec & 1, left, v);
        if constexpr (act != MOE_ACT_NONE) {
          read8<F16, false>(reinterpret_cast<const uint16_t*>(a.pre) + m * a.ldp + n, vec & 2, left, p);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float y;
            v[i] *= act_slope<act>(p[i], y);
          }
        }
        // (columns past N hold zeros)
        if (a.dz) write8<F16, false>(reinterpret_cast<uint16_t*>(a.dz) + m * a.ldz + n, true, 8, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += v[i];
      }
    });
  }
  if (!a.dbias) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[wave][i * 64 + lane] = sum[i];
  __syncthreads();
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int64_t c = (int64_t)blockIdx.x * 512 + (i & 63) * 8 + (i >> 6);
    if (c < a.N) a.part[blockIdx.y * a.N + c] = sums[0][i] + sums[1][i] + sums[2][i] + sums[3][i];
  }
}

// 64 columns a workgroup; its 16 waves take the partial sums in turn.
template <bool F16>
__global__ __launch_bounds__(1024) void dbias_kernel(const float* __restrict__ part, uint16_t* __restrict__ dbias, int64_t N,
                                                     int64_t parts) {
  __shared__ float sums[16][64];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int64_t n = (int64_t)blockIdx.x * 64 + lane;
  float sum = 0.f;
  if (n < N) {
#pragma unroll 8
    for (int64_t p = wave; p < parts; p += 16) sum += part[p * N + n];
  }
  sums[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && n < N) {
#pragma unroll
    for (int w = 1; w < 16; ++w) sum += sums[w][lane];
    dbias[n] = bits16<F16>(sum);
  }
}

static bool on16(const void* p, int64_t ld) { return ((uintptr_t)p & 15) == 0 && ld % 8 == 0; }

hipError_t launch_slope(const SlopeArgs& a, hipStream_t stream) {
  const bool f16 = a.type == MOE_FP16;
  const int64_t parts = dbias_parts(a.M);
  hipError_t e = hipSuccess;
  if (a.M > 0) {
    const int vec = (on16(a.dy, a.lddy) ? 1 : 0) | (a.pre && on16(a.pre, a.ldp) ? 2 : 0);
    const dim3 grid((unsigned)((a.N + 511) / 512), (unsigned)parts);
    e = f16 ? launch_k(slope_kernel<true>, grid, dim3(256), 0, stream, Ev{}, a, vec)
            : launch_k(slope_kernel<false>, grid, dim3(256), 0, stream, Ev{}, a, vec);
  }
  if (e == hipSuccess && a.dbias) {
    const dim3 grid((unsigned)((a.N + 63) / 64));
    e = f16 ? launch_k(dbias_kernel<true>, grid, dim3(1024), 0, stream, Ev{}, (const float*)a.part, (uint16_t*)a.dbias, a.N, parts)
            : launch_k(dbias_kernel<false>, grid, dim3(1024), 0, stream, Ev{}, (const float*)a.part, (uint16_t*)a.dbias, a.N, parts);
  }
  return e;
}

// Eight columns of I of a row a lane, both halves of dz. vec: 1 dh, 2 pre's and dz's
// rows and halves move in 16-byte pieces.
template <bool F16>
__global__ __launch_bounds__(256) void gated_slope_kernel(const GatedSlopeArgs a, int vec) {
  const int64_t pieces = (a.I + 7) / 8;
  with_act(a.act, [&](auto act) __attribute__((always_inline)) {
    if constexpr (act != MOE_ACT_NONE)
      for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = i * 8;
        if (i >= pieces) break;
        const int left = (int)min((int64_t)8, a.I - n);
        float d[8], g[8], u[8];
        const uint16_t* pre = reinterpret_cast<const uint16_t*>(a.pre) + m * 2 * a.I + n;
        uint16_t* dz = reinterpret_cast<uint16_t*>(a.dz) + m * a.ldz + n;
        read8<F16, false>(reinterpret_cast<const uint16_t*>(a.dh) + m * a.lddh + n, vec & 1, left, d);
        read8<F16, false>(pre, vec & 2, left, g);
        read8<F16, false>(pre + a.I, vec & 2, left, u);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float value;
          const float s = act_slope<act>(g[q], value);
          g[q] = d[q] * u[q] * s;
          u[q] = d[q] * value;
        }
        write8<F16, false>(dz, vec & 2, left, g);
        write8<F16, false>(dz + a.I, vec & 2, left, u);
        if (i == 0)  // what pads the row
          for (int64_t c = 2 * a.I; c < a.ldz; ++c) reinterpret_cast<uint16_t*>(a.dz)[m * a.ldz + c] = 0;
      }
  });
}

hipError_t launch_gated_slope(const GatedSlopeArgs& a, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  const int vec = (on16(a.dh, a.lddh) ? 1 : 0) | (on16(a.pre, a.I) ? 2 : 0);
  const dim3 grid((unsigned)((a.I + 2047) / 2048), (unsigned)std::min<int64_t>(a.M, 65535));
  return a.type == MOE_FP16 ? launch_k(gated_slope_kernel<true>, grid, dim3(256), 0, stream, Ev{}, a, vec)
                            : launch_k(gated_slope_kernel<false>, grid, dim3(256), 0, stream, Ev{}, a, vec);
}

}  // namespace qmoe
