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

// The kernels a product may run on: 16 TM rows by 16 TN columns a wave (gated: of both
// products, so half of them columns of y).
enum { k256x256, k256x192, k128x128, k64x64, k64x64Pair, kTiles, kWave16x16 = kTiles, kWave16x32, kWave32x16, kWave32x32, kChoices };
struct Choice {
  int kernel, splits;
};
struct Size {
  const char* name;
  int rows, cols;
};
constexpr Size kSize[kChoices] = {
    {"256 x 256 tile", 256, 256},
    {"256 x 192 tile", 256, 192},
    {"128 x 128 tile", 128, 128},
    {"64 x 64 tile", 64, 64},
    {"64 x 64 tile, two groups of waves", 64, 64},
    {"16 x 16, K split over the waves", 16, 16},
    {"16 x 32, K split over the waves", 16, 32},
    {"32 x 16, K split over the waves", 32, 16},
    {"32 x 32, K split over the waves", 32, 32},
};

Choice choose(GemmKind kind, int64_t rows, int64_t cols, int64_t K, int cus) {
  auto tiles_of = [&](int i) {
    const int64_t bn = kind == kGemmGated ? kSize[i].cols / 2 : kSize[i].cols;
    return ((rows + kSize[i].rows - 1) / kSize[i].rows) * ((cols + bn - 1) / bn);
  };
  auto rounds_of = [&](int i) { return (tiles_of(i) + cus - 1) / cus; };
  if (kind == kGemmForward || kind == kGemmGated) {
    // Few rows: no split sums to join by a second launch (weights from memory: 1 x 6144
    // x 2048 12.5 us by the 64 x 64 tiles, 9.1 by 16 x 32; 16 x 16384 x 6144 56.7 and 48.5; 4
    // x 512 x 8192 12.1, 10.9 and by 16 x 16 8.6; gated 4 x 2048 x 6144 19.3, 18.2 and 14.9).
    if (rows <= 16) return {rounds_of(kWave16x16) * 10 <= rounds_of(kWave16x32) * 18 ? kWave16x16 : kWave16x32, 1};
    // Tens of rows, while one round does (48 x 1536 x 1536: 9.5 us by 64 x 64, 7.4 by 32 x
    // 32, 5.9 by 32 x 16; 77 x 1543 x 1448 11.4, 9.3 and in two rounds 10.9; 64 x 6144 x 6144
    // 29.4, in two rounds 36.5), or weights are read once either way (24 x 16384 x 6144 55.3 and 51.4).
    if (rows <= 128) {
      if (rounds_of(kWave32x16) == 1) return {kWave32x16, 1};
      if (rounds_of(kWave32x32) == 1 || rows <= 32) return {kWave32x32, 1};
    }
  }
  // Tiles: rounds of workgroups over the CUs times a round's time, a K-step's per tile
  // and some steps' for its start and end, in units of 10 ns; split sums are written, read
  // and joined by a second launch besides. Fitted to 52 products of 8 .. 4096 rows, on which
  // the kernels chosen take 0.8 % longer than the best tile and split on average, 10 % at
  // most (512 x 1024 x 1024: 64 x 64 whole 9.0 us, in 2 splits 10.8; 512 x 6144 x 6144: 256 x
  // 192 in 4 splits 51, 128 x 128 in 2 58; 1024 x 6144 x 2048 39 by 128 x 128, 42 by 256 x 192;
  // 4096 x 6144 x 2048 89, by 256 x 256 114; with two groups of waves 64 x 64 tiles that are
  // alone on their CUs take 12.5 us for 14.0, 333 x 2320 x 2056, and 16.4 for 18.8, 704 x 1000 x 3000).
  constexpr int per[kTiles] = {160, 143, 59, 25, 63};
  constexpr int start[kTiles] = {18, 18, 18, 18, 11};
  constexpr int wide[kTiles] = {1, 1, 2, 2, 1};    // workgroups a CU
  constexpr int groups[kTiles] = {1, 1, 1, 1, 2};  // of waves, which share the steps
  const int64_t steps = std::max<int64_t>((K + 63) / 64, 1);
  Choice best{0, 1};
  int64_t least = INT64_MAX;
  for (int i = 0; i < kTiles; ++i) {
    const int64_t tiles = tiles_of(i), room = cus * wide[i];
    if (i == k64x64Pair && tiles > cus) continue;
    // splits of at least 8 steps each, while they fit the chip at once
    const int64_t most = std::min<int64_t>({std::max<int64_t>(room / tiles, 1), std::max<int64_t>(steps / 8, 1), 16});
    for (int64_t want : {(int64_t)1, most / 2, most}) {
      const int64_t part = (steps + std::max<int64_t>(want, 1) - 1) / std::max<int64_t>(want, 1);
      const int64_t splits = (steps + part - 1) / part;  // none of them empty
      int64_t cost = (tiles * splits + room - 1) / room * ((part + groups[i] - 1) / groups[i] + start[i]) * per[i] * wide[i];
      if (splits > 1) cost += 960 + splits * rows * cols * (kind == kGemmGated ? 2 : 1) / 30000;
      if (cost < least) least = cost, best = {i, (int)splits};
    }
  }
  return best;
}

template <bool F16, GemmKind KIND>
hipError_t launch(GemmArgs a, const Choice& c, int cus, hipStream_t stream) {
  a.splits = c.splits;
  if constexpr (KIND == kGemmForward || KIND == kGemmGated) {
    switch (c.kernel) {
      case kWave16x16: return launch_wave<F16, KIND, 1, 1, 4>(a, cus, stream);
      case kWave16x32: return launch_wave<F16, KIND, 1, 2, 3>(a, cus, stream);
      case kWave32x16: return launch_wave<F16, KIND, 2, 1, 2>(a, cus, stream);
      case kWave32x32: return launch_wave<F16, KIND, 2, 2, 2>(a, cus, stream);
    }
  }
  hipError_t e;
  switch (c.kernel) {
    case k256x256: e = launch_tile<F16, KIND, 8, 4, 2, 4, 2>(a, stream); break;
    case k256x192: e = launch_tile<F16, KIND, 4, 6, 4, 2, 2>(a, stream); break;
    case k128x128: e = launch_tile<F16, KIND, 4, 4, 2, 2, 2>(a, stream); break;
    case k64x64Pair: e = launch_tile<F16, KIND, 2, 2, 2, 2, 4, 2>(a, stream); break;
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

size_t gemm_ws_bytes(GemmKind kind, int64_t rows, int64_t cols, int64_t K, int cus) {
  if (rows == 0 || cols == 0) return 0;
  const Choice c = choose(kind, rows, cols, K, cus);
  return c.splits > 1 ? (size_t)c.splits * rows * ((cols + 7) / 8 * 8) * (kind == kGemmGated ? 8 : 4) : 0;
}

const char* gemm_kernel_name(GemmKind kind, int64_t rows, int64_t cols, int64_t K, int cus) {
  return kSize[choose(kind, rows, cols, K, cus).kernel].name;
}

hipError_t launch_gemm(GemmKind kind, const GemmArgs& args, int cus, hipStream_t stream) {
  GemmArgs a = args;
  const int64_t es = a.y_type == MOE_FP32 ? 4 : 2, ps = a.pre_type == MOE_FP32 ? 4 : 2;
  auto vec = [](const void* p, int64_t ld, int64_t elem) { return p && ((uintptr_t)p & 15) == 0 && ld * elem % 16 == 0; };
  a.vec = (vec(a.y, a.ldy, es) ? kVecY : 0) | (vec(a.residual, a.ldr, es) ? kVecResidual : 0) |
          (vec(a.pre, a.ldp, ps) && (kind != kGemmGated || a.cols * ps % 16 == 0) ? kVecPre : 0) | (vec(a.bias, 0, 2) ? kVecBias : 0);
  const bool f16 = a.type == MOE_FP16;
  const Choice c = choose(kind, a.rows, a.cols, a.K, cus);
  switch (kind) {
    case kGemmForward: return f16 ? launch<true, kGemmForward>(a, c, cus, stream) : launch<false, kGemmForward>(a, c, cus, stream);
    case kGemmGated: return f16 ? launch<true, kGemmGated>(a, c, cus, stream) : launch<false, kGemmGated>(a, c, cus, stream);
    case kGemmInput: return f16 ? launch<true, kGemmInput>(a, c, cus, stream) : launch<false, kGemmInput>(a, c, cus, stream);
    default: return f16 ? launch<true, kGemmWeight>(a, c, cus, stream) : launch<false, kGemmWeight>(a, c, cus, stream);
  }
}

// ----------------------------------------------------------------- backward, elementwise
// Up to 8 values of pre.
template <bool F16>
__device__ __forceinline__ void read_pre(const void* pre, int type, int64_t at, bool vec, int n, float (&v)[8]) {
  if (type == MOE_FP32) read8<F16, true>(reinterpret_cast<const float*>(pre) + at, vec, n, v);
  else read8<F16, false>(reinterpret_cast<const uint16_t*>(pre) + at, vec, n, v);
}

// Eight columns a lane; a wave takes RL rows of 512 / RL columns at a time, the W waves
// of a workgroup `rows` rows together. dbias's sums of a workgroup are joined in a fixed
// order, those of several workgroups by a second launch. Bound by memory: 4096 x 6144 33 us
// (4.6 TB/s: dy and pre read, dz written), dbias's second launch 5 us.
template <bool F16, int RL, int W>
__global__ __launch_bounds__(64 * W) void slope_kernel(const SlopeArgs a, int vec, int rows) {
  constexpr int L = 64 / RL, C = 8 * L;  // lanes of a row, columns
  __shared__ float sums[W][C];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int64_t n = (int64_t)blockIdx.x * C + (lane % L) * 8;
  const int64_t m0 = (int64_t)blockIdx.y * rows, m1 = min(m0 + rows, a.M);
  const int left = (int)max((int64_t)0, min((int64_t)8, a.N - n));
  float sum[8] = {};
  if (left > 0) {
    with_act(a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll 4
      for (int64_t m = m0 + RL * wave + lane / L; m < m1; m += RL * W) {
        float v[8], p[8];
        read8<F16, false>(reinterpret_cast<const uint16_t*>(a.dy) + m * a.lddy + n, vec & 1, left, v);
        if constexpr (act != MOE_ACT_NONE) {
          read_pre<F16>(a.pre, a.pre_type, m * a.ldp + n, vec & 2, left, p);
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
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = L; o < 64; o *= 2) sum[i] += __shfl_xor(sum[i], o, kWave);
    if (lane < L) sums[wave][i * L + lane] = sum[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < C; i += 64 * W) {
    const int64_t c = (int64_t)blockIdx.x * C + (i % L) * 8 + i / L;
    if (c >= a.N) continue;
    float v = sums[0][i];
#pragma unroll
    for (int w = 1; w < W; ++w) v += sums[w][i];
    if (gridDim.y == 1) reinterpret_cast<uint16_t*>(a.dbias)[c] = bits16<F16>(v);
    else a.part[blockIdx.y * a.N + c] = v;
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

static bool on16(const void* p, int64_t ld, int64_t elem) { return ((uintptr_t)p & 15) == 0 && ld * elem % 16 == 0; }

hipError_t launch_slope(const SlopeArgs& a, hipStream_t stream) {
  const bool f16 = a.type == MOE_FP16;
  const int vec = (on16(a.dy, a.lddy, 2) ? 1 : 0) | (a.pre && on16(a.pre, a.ldp, a.pre_type == MOE_FP32 ? 4 : 2) ? 2 : 0);
  // Up to 128 rows a workgroup takes all of 64 columns, and dbias needs no second launch (77 x
  // 1543: 6 us, 9.4 + 3.4 by two); above, whole lines of a row a wave (4096 x 6144 33 us, by 64
  // columns 40 to 59). No rows: dbias is zero.
  const bool few = a.M <= 128;
  const int64_t parts = few ? 1 : dbias_parts(a.M);
  const dim3 grid((unsigned)(few ? (a.N + 63) / 64 : (a.N + 511) / 512), (unsigned)parts);
  hipError_t e = few ? f16 ? launch_k(slope_kernel<true, 8, 16>, grid, dim3(1024), 0, stream, Ev{}, a, vec, 128)
                           : launch_k(slope_kernel<false, 8, 16>, grid, dim3(1024), 0, stream, Ev{}, a, vec, 128)
                     : f16 ? launch_k(slope_kernel<true, 1, 4>, grid, dim3(256), 0, stream, Ev{}, a, vec, kBiasRows)
                           : launch_k(slope_kernel<false, 1, 4>, grid, dim3(256), 0, stream, Ev{}, a, vec, kBiasRows);
  if (e == hipSuccess && a.dbias && parts > 1) {
    const dim3 cols((unsigned)((a.N + 63) / 64));
    e = f16 ? launch_k(dbias_kernel<true>, cols, dim3(1024), 0, stream, Ev{}, (const float*)a.part, (uint16_t*)a.dbias, a.N, parts)
            : launch_k(dbias_kernel<false>, cols, dim3(1024), 0, stream, Ev{}, (const float*)a.part, (uint16_t*)a.dbias, a.N, parts);
  }
  return e;
}

// Eight columns of I of a row a lane, both halves of dz. Bound by memory: 4096 x 2 2048 23
// us (3.6 TB/s; pre in 32 bits 25, 4.7 TB/s). vec: the rows and halves of dh
// (1), pre (2) and dz (4) move in 16-byte pieces.
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
        uint16_t* dz = reinterpret_cast<uint16_t*>(a.dz) + m * a.ldz + n;
        read8<F16, false>(reinterpret_cast<const uint16_t*>(a.dh) + m * a.lddh + n, vec & 1, left, d);
        read_pre<F16>(a.pre, a.pre_type, m * 2 * a.I + n, vec & 2, left, g);
        read_pre<F16>(a.pre, a.pre_type, m * 2 * a.I + a.I + n, vec & 2, left, u);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float value;
          const float s = act_slope<act>(g[q], value);
          // (an infinite u beside a gate that passes nothing: 0, as h has it)
          g[q] = s == 0.f && fabsf(u[q]) == INFINITY ? d[q] * s : d[q] * u[q] * s;
          u[q] = d[q] * value;
        }
        write8<F16, false>(dz, vec & 4, left, g);
        write8<F16, false>(dz + a.I, vec & 4, left, u);
        if (i == 0)  // what pads the row
          for (int64_t c = 2 * a.I; c < a.ldz; ++c) reinterpret_cast<uint16_t*>(a.dz)[m * a.ldz + c] = 0;
      }
  });
}

hipError_t launch_gated_slope(const GatedSlopeArgs& a, hipStream_t stream) {
  if (a.M == 0) return hipSuccess;
  const int vec = (on16(a.dh, a.lddh, 2) ? 1 : 0) | (on16(a.pre, a.I, a.pre_type == MOE_FP32 ? 4 : 2) ? 2 : 0) | (a.I % 8 == 0 ? 4 : 0);
  const dim3 grid((unsigned)((a.I + 2047) / 2048), (unsigned)std::min<int64_t>(a.M, 65535));
  return a.type == MOE_FP16 ? launch_k(gated_slope_kernel<true>, grid, dim3(256), 0, stream, Ev{}, a, vec)
                            : launch_k(gated_slope_kernel<false>, grid, dim3(256), 0, stream, Ev{}, a, vec);
}

}  // namespace qmoe
