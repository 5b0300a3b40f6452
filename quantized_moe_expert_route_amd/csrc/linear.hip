// Linear layer on MXFP4 weights with 16-bit activations:
//   y[m][n] = sum_k x[m][k] E2M1(w[n][k]) 2^(s[n][k/32] - 127) (+ bias[n]) (+ residual[m][n])
// products exact, sums in binary32, one rounding to y's type.
//
// Weights are packed once (moe_pack_linear): a K-step of 128 of a block of 16
// rows is 1 KB contiguous, lane 16 g + r holding row r, dword j the 8 codes
// of K 32 j + 8 g .. + 7, so that one MFMA (K = 32) covers exactly the MX
// block j of every row and the activations' operand of a lane is 16
// contiguous bytes, 64 over the four lane groups:
//   wp [ceil(N/16)][ceil(K/128)][4 g][16 r][4 j] dwords, codes past N or K zero
//   sp [ceil(N/16)][ceil(K/128)][16 r][4 j] bytes, past N or K 127 (2^0)
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "mxfp4.h"
#include "ops.h"

namespace qmoe {

// ----------------------------------------------------------------- packing
__global__ __launch_bounds__(256) void pack_linear_kernel(const uint8_t* __restrict__ w, uint32_t* __restrict__ wp,
                                                          int64_t dwords, int nks, int64_t N, int64_t K) {
  for (int64_t o = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; o < dwords; o += (int64_t)gridDim.x * blockDim.x) {
    const int j = (int)(o & 3), r = (int)((o >> 2) & 15), g = (int)((o >> 6) & 3);
    const int64_t rest = o >> 8;
    const int64_t n = rest / nks * 16 + r, k = rest % nks * 128 + 32 * j + 8 * g;
    wp[o] = n < N && k < K ? *reinterpret_cast<const uint32_t*>(w + n * (K / 2) + k / 2) : 0u;
  }
}

__global__ __launch_bounds__(256) void pack_linear_scale_kernel(const uint8_t* __restrict__ s,
                                                                uint8_t* __restrict__ sp, int64_t bytes, int nks,
                                                                int64_t N, int64_t K) {
  for (int64_t o = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; o < bytes; o += (int64_t)gridDim.x * blockDim.x) {
    const int j = (int)(o & 3), r = (int)((o >> 2) & 15);
    const int64_t rest = o >> 6;
    const int64_t n = rest / nks * 16 + r, b = rest % nks * 4 + j;
    sp[o] = n < N && b < K / 32 ? s[n * (K / 32) + b] : (uint8_t)127;
  }
}

hipError_t launch_pack_linear(const void* w, const void* s, int64_t N, int64_t K, void* wp, void* sp,
                              hipStream_t stream) {
  const int64_t nrb = (N + 15) / 16, nks = (K + 127) / 128;
  const int64_t dwords = nrb * nks * 256, bytes = nrb * nks * 64;
  hipError_t e = launch_k(pack_linear_kernel, dim3((unsigned)std::min<int64_t>((dwords + 255) / 256, 1 << 16)),
                          dim3(256), 0, stream, Ev{}, (const uint8_t*)w, (uint32_t*)wp, dwords, (int)nks, N, K);
  if (e == hipSuccess)
    e = launch_k(pack_linear_scale_kernel, dim3((unsigned)std::min<int64_t>((bytes + 255) / 256, 1 << 16)), dim3(256),
                 0, stream, Ev{}, (const uint8_t*)s, (uint8_t*)sp, bytes, (int)nks, N, K);
  return e;
}

// ----------------------------------------------------------------- epilogue
// Four consecutive columns n .. n + 3 of row m (n a multiple of 4). `a.vec`: all
// of a row's groups of four lie inside N and are aligned (uniform over the
// call), so that they move as one piece.
__device__ __forceinline__ void store4(const LinearArgs& a, int64_t m, int64_t n, v4f v) {
  const bool f16 = a.x_type == MOE_FP16;
  if (n >= a.N) return;
  const int left = (int)min((int64_t)4, a.N - n);
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) {
        const uint16_t b = reinterpret_cast<const uint16_t*>(a.bias)[n + i];
        v[i] += f16 ? fp16_value(b) : bf16_value(b);
      }
  }
  if (a.y_type == MOE_FP32) {
    float* y = reinterpret_cast<float*>(a.y) + m * a.ldy + n;
    const float* res = reinterpret_cast<const float*>(a.residual) + m * a.ldr + n;
    if (a.vec) {
      if (a.residual) v += *reinterpret_cast<const v4f*>(res);
      *reinterpret_cast<v4f*>(y) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) y[i] = v[i] + (a.residual ? res[i] : 0.f);
    }
    return;
  }
  uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + m * a.ldy + n;
  const uint16_t* res = reinterpret_cast<const uint16_t*>(a.residual) + m * a.ldr + n;
  if (a.vec) {
    if (a.residual) {
      const uint2 p = *reinterpret_cast<const uint2*>(res);
      const uint16_t b[4] = {(uint16_t)p.x, (uint16_t)(p.x >> 16), (uint16_t)p.y, (uint16_t)(p.y >> 16)};
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += f16 ? fp16_value(b[i]) : bf16_value(b[i]);
    }
    uint16_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f16 ? fp16_bits(v[i]) : bf16_bits(v[i]);
    *reinterpret_cast<uint2*>(y) = make_uint2((uint32_t)o[0] | ((uint32_t)o[1] << 16), (uint32_t)o[2] | ((uint32_t)o[3] << 16));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) {
        if (a.residual) v[i] += f16 ? fp16_value(res[i]) : bf16_value(res[i]);
        y[i] = f16 ? fp16_bits(v[i]) : bf16_bits(v[i]);
      }
  }
}

// scale_operand of a byte number known after unrolling
__device__ __forceinline__ float scale_of(uint32_t d, int j) {
  return j == 0 ? scale_operand<0>(d) : j == 1 ? scale_operand<1>(d) : j == 2 ? scale_operand<2>(d) : scale_operand<3>(d);
}

// ----------------------------------------------------------------- few rows
// A workgroup of W waves computes 16 columns of y at a time for up to 16 rows
// of x; the waves split K. Wave w owns K-steps w S .. w S + S - 1 of 128 and
// keeps its fragments of x as MFMA operands in registers over all the tiles
// of the workgroup. Its weights stream through a ring of D tiles' registers:
// the piece of a tile D ahead is requested as soon as a slot's products are
// issued, so a wave has about S D KB under way at any time. The W partial
// sums of a tile are added in wave order through LDS.
template <bool F16>
struct WeightStep {  // one K-step of 16 weight rows: a lane's codes and scales
  uint4 q;
  uint4 sc;  // bf16: .x is the lane's row's four scales; fp16: rows 4 g .. 4 g + 3
  __device__ __forceinline__ void load(const LinearArgs& a, size_t piece, int lane) {
    q = ld16(a.wp + piece * 1024 + 16 * lane);
    if constexpr (F16) sc = ld16(a.sp + piece * 64 + 16 * (lane >> 4));
    else sc.x = ld4(a.sp + piece * 64 + 4 * (lane & 15));
  }
  __device__ __forceinline__ void clear() { q = make_uint4(0, 0, 0, 0); }
  // against CT column tiles of x: acc[u] += w x[u]
  template <int CT>
  __device__ __forceinline__ void mul_columns(const uint4 (&x)[CT][4], v4f (&acc)[CT]) const {
    const uint32_t d[4] = {q.x, q.y, q.z, q.w}, rs[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (F16) {
        const v8h wf = fp4x8_f16(d[j]);
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = e8m0_value((rs[i] >> (8 * j)) & 255u);
#pragma unroll
        for (int u = 0; u < CT; ++u) {
          const v4f p = mfma_f16(wf, __builtin_bit_cast(v8h, x[u][j]), v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[u][i] += p[i] * f[i];
        }
      } else {
        const v8s wf = fp4x8_bf16(d[j], scale_of(sc.x, j));
#pragma unroll
        for (int u = 0; u < CT; ++u) acc[u] = mfma_bf16(wf, __builtin_bit_cast(v8s, x[u][j]), acc[u]);
      }
    }
  }
};

template <bool F16, int W, int S, int D>
__global__ __launch_bounds__(64 * W) void linear_rows_kernel(const LinearArgs a) {
  __shared__ v4f red[2][W][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int K = (int)a.K, nks = (K + 127) / 128;
  const bool row = r < a.M;
  const int ntiles = (int)((a.N + 15) / 16), step = gridDim.x;
  const int own = (ntiles - (int)blockIdx.x + step - 1) / step;  // this workgroup's tiles (grid <= ntiles)

  WeightStep<F16> ring[D][S];
  auto load = [&](int d, int s, int i) {
    // past the last step of K or the last tile: that one again, not used
    const int tile = blockIdx.x + min(i, own - 1) * step;
    ring[d][s].load(a, (size_t)tile * nks + min(wave * S + s, nks - 1), lane);
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
#pragma unroll
    for (int s = 0; s < S; ++s) load(d, s, d);
  uint4 xf[S][1][4];
  const uint16_t* xr = reinterpret_cast<const uint16_t*>(a.x) + (row ? r : 0) * a.ldx;
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = 128 * (wave * S + s) + 32 * j + 8 * g;
      xf[s][0][j] = row && k < K ? ld16(xr + k) : make_uint4(0, 0, 0, 0);
    }

  auto tile_done = [&](int i, const v4f& acc) {
    const int buf = i & 1;
    red[buf][wave][lane] = acc;
    barrier_lds();
    // lane holds rows 4 g .. 4 g + 3 (columns of y) of column r (row of x)
    if (wave == i % W && row) {
      v4f v = red[buf][0][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) v += red[buf][w][lane];
      store4(a, r, (int64_t)(blockIdx.x + i * step) * 16 + 4 * g, v);
    }
  };
  auto compute = [&](int d, int i, auto reload) {
    v4f acc[1] = {{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      // a step past the last takes no part (its codes could meet a scale that
      // overflows, and zero times that is not zero)
      if (wave * S + s >= nks) ring[d][s].clear();
      ring[d][s].template mul_columns<1>(xf[s], acc);
      if constexpr (reload) load(d, s, i + D);
    }
    tile_done(i, acc[0]);
  };
  int i = 0;
  for (; i + D < own; i += D)
#pragma unroll
    for (int d = 0; d < D; ++d) compute(d, i + d, std::true_type{});
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (i + d < own) compute(d, i + d, std::false_type{});
}

// K beyond the W S steps that the waves hold: segment after segment, x loaded
// again for each (from the cache), the next segment's weights under way.
template <bool F16, int W, int S>
__global__ __launch_bounds__(64 * W) void linear_rows_long_kernel(const LinearArgs a) {
  __shared__ v4f red[2][W][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int K = (int)a.K, nks = (K + 127) / 128, nseg = (nks + W * S - 1) / (W * S);
  const bool row = r < a.M;
  const uint16_t* xr = reinterpret_cast<const uint16_t*>(a.x) + (row ? r : 0) * a.ldx;
  const int ntiles = (int)((a.N + 15) / 16);
  uint4 xf[S][1][4];
  WeightStep<F16> cur[S], next[S];
  auto load_w = [&](int tile, int seg) {
#pragma unroll
    for (int s = 0; s < S; ++s)
      next[s].load(a, (size_t)tile * nks + min((seg * W + wave) * S + s, nks - 1), lane);
  };
  int buf = 0;
  load_w(blockIdx.x, 0);
  for (int tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
    v4f acc[1] = {{0.f, 0.f, 0.f, 0.f}};
    for (int seg = 0; seg < nseg; ++seg) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = 128 * ((seg * W + wave) * S + s) + 32 * j + 8 * g;
          xf[s][0][j] = row && k < K ? ld16(xr + k) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
      for (int s = 0; s < S; ++s) cur[s] = next[s];
      if (seg + 1 < nseg) load_w(tile, seg + 1);
      else load_w(min(tile + (int)gridDim.x, ntiles - 1), 0);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if ((seg * W + wave) * S + s >= nks) cur[s].clear();
        cur[s].template mul_columns<1>(xf[s], acc);
      }
    }
    red[buf][wave][lane] = acc[0];
    barrier_lds();
    if (wave == buf && row) {
      v4f v = red[buf][0][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) v += red[buf][w][lane];
      store4(a, r, (int64_t)tile * 16 + 4 * g, v);
    }
    buf ^= 1;
  }
}

// OCC workgroups fit a CU's registers: one a tile while they all fit at once,
// else OCC a CU, each over several tiles.
template <bool F16, int W, int S, int OCC>
static hipError_t launch_rows(const LinearArgs& a, int cus, hipStream_t stream) {
  const int64_t tiles = (a.N + 15) / 16;
  if (tiles <= OCC * cus)
    return launch_k(linear_rows_kernel<F16, W, S, 1>, dim3((unsigned)tiles), dim3(64 * W), 0, stream, Ev{}, a);
  return launch_k(linear_rows_kernel<F16, W, S, S == 1 ? 4 : 2>, dim3((unsigned)(OCC * cus)), dim3(64 * W), 0, stream,
                  Ev{}, a);
}

// ----------------------------------------------------------------- tens of rows
// 16 R columns of y for 16 CT rows of x a workgroup. The 8 waves take K-steps
// in turn, weights and x both straight from memory to registers, one K-step
// ahead: no operand is shared between waves, so the loop has no barrier. The
// partial sums are joined through LDS at the end, R sub-tiles' columns at a
// time. x is read once per 16 R columns (from the L2): R = 2 where there are
// tiles enough.
template <bool F16, int CT, int R>
__global__ __launch_bounds__(512) void linear_mid_kernel(const LinearArgs a, int tiles_n) {
  constexpr int W = 8;
  __shared__ v4f red[W][CT][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int K = (int)a.K, nks = (K + 127) / 128;
  const int tile = (int)(blockIdx.x % tiles_n) * R;
  const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * (16 * CT);
  const int last = (int)((a.N + 15) / 16) - 1;
  const uint16_t* xr[CT];
#pragma unroll
  for (int u = 0; u < CT; ++u)
    xr[u] = reinterpret_cast<const uint16_t*>(a.x) + min(m0 + 16 * u + r, a.M - 1) * a.ldx + 8 * g;
  WeightStep<F16> w[R], nw[R];
  uint4 x[CT][4], nx[CT][4];
  auto load = [&](int ks) {
    const int kc = min(ks, nks - 1);
#pragma unroll
    for (int t = 0; t < R; ++t) nw[t].load(a, (size_t)min(tile + t, last) * nks + kc, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = 128 * kc + 32 * j;
      const bool in = k < K;  // K is a multiple of 32: whole operands
#pragma unroll
      for (int u = 0; u < CT; ++u) nx[u][j] = in ? ld16(xr[u] + k) : make_uint4(0, 0, 0, 0);
    }
  };
  v4f acc[R][CT];
#pragma unroll
  for (int t = 0; t < R; ++t)
#pragma unroll
    for (int u = 0; u < CT; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
  load(wave);
  for (int ks = wave; ks < nks; ks += W) {
#pragma unroll
    for (int t = 0; t < R; ++t) w[t] = nw[t];
#pragma unroll
    for (int u = 0; u < CT; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[u][j] = nx[u][j];
    load(ks + W);
#pragma unroll
    for (int t = 0; t < R; ++t) w[t].template mul_columns<CT>(x, acc[t]);
  }
#pragma unroll
  for (int t = 0; t < R; ++t) {
    if (t) __syncthreads();
#pragma unroll
    for (int u = 0; u < CT; ++u) red[wave][u][lane] = acc[t][u];
    __syncthreads();
    if (wave < CT) {
      v4f v = red[0][wave][lane];
#pragma unroll
      for (int q = 1; q < W; ++q) v += red[q][wave][lane];
      const int64_t m = m0 + 16 * wave + r;
      if (m < a.M && tile + t <= last) store4(a, m, (int64_t)(tile + t) * 16 + 4 * g, v);
    }
  }
}

// ----------------------------------------------------------------- many rows
// Where x's 16-byte chunk c (of a row's 16 in a K-step) of row m of a 16-row
// block lies in LDS, in chunks: operand j = c / 4 of the block is 64
// consecutive chunks, lane 16 g + r reading row r, g = c % 4. The rows of a
// group are exchanged by r ^ c, so that the 16 lanes that write a row's
// chunks, like the 16 that read a group, meet all banks.
__device__ __forceinline__ int x_slot(int block, int c, int m) {
  return (block * 4 + (c >> 2)) * 64 + 16 * (c & 3) + (m ^ c);
}

// A workgroup of WN x WM waves computes BN = 16 TN WN columns of y for BM =
// 16 TM WM rows of x; a wave 16 TN x 16 TM of it. x goes through LDS (two
// buffers of one K-step of 128; whole 256-byte row pieces are read, and kept
// in registers for two steps until their buffer is free); weights go straight
// from their packed form to registers, PW steps ahead, and are widened there:
// a wave's rows are read by WM waves only. With one step ahead a step took
// 2.2 us, the weights' latency, where its products take 0.85.
template <bool F16, int TN, int TM, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM) void linear_tile_kernel(const LinearArgs a, int tiles_m, int tiles_n) {
  constexpr int W = WN * WM, BM = 16 * TM * WM, BN = 16 * TN * WN;
  constexpr int NX = BM / 4 / W;  // pieces of 4 rows x 128 K staged by a wave
  constexpr int PW = 4;           // weight steps in registers
  static_assert(BM % (4 * W) == 0, "whole pieces");
  __shared__ uint4 xs[2][BM * 16];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int wn = wave % WN, wm = wave / WN;
  const int K = (int)a.K, nks = (K + 127) / 128;

  // Workgroups go to the eight XCDs in turn: XCD x takes a contiguous eighth
  // of the tiles, walked in groups of 8 row blocks, so that the tiles it runs
  // at a time share their x rows and weight rows in its L2.
  const int total = tiles_m * tiles_n;
  int id;
  {
    const int xcd = blockIdx.x & 7, at = blockIdx.x >> 3;
    const int per = total >> 3, rest = total & 7;
    id = xcd * per + min(xcd, rest) + at;
  }
  constexpr int GM = 8;
  const int group = id / (GM * tiles_n), first = group * GM, rows = min(GM, tiles_m - first);
  const int in = id - group * GM * tiles_n;
  const int64_t m0 = (int64_t)(first + in % rows) * BM;
  const int64_t n0 = (int64_t)(in / rows) * BN;

  const uint16_t* xr[NX];
#pragma unroll
  for (int i = 0; i < NX; ++i)
    xr[i] = reinterpret_cast<const uint16_t*>(a.x) + min(m0 + 4 * (wave * NX + i) + g, a.M - 1) * a.ldx;
  uint4 xv[2][NX];
  auto load_x = [&](uint4(&v)[NX], int ks) {
    const int k = 128 * min(ks, nks - 1);
    // K's last step may end inside a row piece: zero there (as the codes are)
    const bool in_k = k + 8 * r < K;
    const int at = in_k ? k + 8 * r : 0;
#pragma unroll
    for (int i = 0; i < NX; ++i) v[i] = ld16(xr[i] + at);
    if (k + 128 > K) {
#pragma unroll
      for (int i = 0; i < NX; ++i) v[i] = in_k ? v[i] : make_uint4(0, 0, 0, 0);
    }
  };
  auto put_x = [&](const uint4(&v)[NX], int buf) {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int piece = wave * NX + i;
      xs[buf][x_slot(piece >> 2, r, 4 * (piece & 3) + g)] = v[i];
    }
  };
  // row blocks past N: the last one again (not stored)
  size_t rb[TN];
#pragma unroll
  for (int t = 0; t < TN; ++t)
    rb[t] = (size_t)min(n0 / 16 + wn * TN + t, (a.N + 15) / 16 - 1) * nks;
  uint4 q[PW][TN];
  uint32_t sc[PW][TN];
  auto load_w = [&](int p, int ks) {
    const int kc = min(ks, nks - 1);
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      q[p][t] = ld16(a.wp + (rb[t] + kc) * 1024 + 16 * lane);
      sc[p][t] = ld4(a.sp + (rb[t] + kc) * 64 + 4 * r);
    }
  };

  v4f acc[TN][TM];
#pragma unroll
  for (int t = 0; t < TN; ++t)
#pragma unroll
    for (int u = 0; u < TM; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
  load_x(xv[0], 0);
  load_x(xv[1], 1);
#pragma unroll
  for (int p = 0; p < PW; ++p) load_w(p, p);
  put_x(xv[0], 0);
  load_x(xv[0], 2);
  barrier_lds();
  for (int k0 = 0; k0 < nks; k0 += PW) {
#pragma unroll
    for (int p = 0; p < PW; ++p) {
      const int ks = k0 + p;
      if (ks >= nks) break;
      // step ks + 1's x into the buffer that step ks - 1 was read from
      put_x(xv[(p + 1) & 1], (p + 1) & 1);
      load_x(xv[(p + 1) & 1], ks + 3);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v8s wf[TN];
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          const uint32_t d = j == 0 ? q[p][t].x : j == 1 ? q[p][t].y : j == 2 ? q[p][t].z : q[p][t].w;
          wf[t] = fp4x8_bf16(d, scale_of(sc[p][t], j));
        }
#pragma unroll
        for (int u = 0; u < TM; ++u) {
          const uint4 f = xs[p & 1][x_slot(wm * TM + u, 4 * j + g, r)];
          if constexpr (F16) {
            v8s hi, lo;
            fp16x8_planes(f, hi, lo);
#pragma unroll
            for (int t = 0; t < TN; ++t) acc[t][u] = mfma_bf16(wf[t], lo, mfma_bf16(wf[t], hi, acc[t][u]));
          } else {
#pragma unroll
            for (int t = 0; t < TN; ++t) acc[t][u] = mfma_bf16(wf[t], __builtin_bit_cast(v8s, f), acc[t][u]);
          }
        }
      }
      load_w(p, ks + PW);
      barrier_lds();
    }
  }
#pragma unroll
  for (int u = 0; u < TM; ++u) {
    const int64_t m = m0 + 16 * (wm * TM + u) + r;
    if (m >= a.M) continue;
#pragma unroll
    for (int t = 0; t < TN; ++t) store4(a, m, n0 + 16 * (wn * TN + t) + 4 * g, acc[t][u]);
  }
}

template <bool F16, int TN, int TM, int WN, int WM>
static hipError_t launch_tile(const LinearArgs& a, hipStream_t stream) {
  const int64_t tm = (a.M + 16 * TM * WM - 1) / (16 * TM * WM), tn = (a.N + 16 * TN * WN - 1) / (16 * TN * WN);
  return launch_k(linear_tile_kernel<F16, TN, TM, WN, WM>, dim3((unsigned)(tm * tn)), dim3(64 * WN * WM), 0, stream,
                  Ev{}, a, (int)tm, (int)tn);
}

template <bool F16>
static hipError_t launch_16_rows(const LinearArgs& a, int cus, hipStream_t stream) {
  const int64_t nks = (a.K + 127) / 128;
  if (nks <= 8) return launch_rows<F16, 8, 1, 3>(a, cus, stream);
  if (nks <= 16) return launch_rows<F16, 8, 2, 2>(a, cus, stream);
  if (nks <= 24) return launch_rows<F16, 8, 3, 1>(a, cus, stream);
  if (nks <= 32) return launch_rows<F16, 8, 4, 1>(a, cus, stream);
  // (fp16 carries four scale dwords a step: 6 steps do not fit the registers)
  if constexpr (!F16)
    if (nks <= 48) return launch_rows<F16, 8, 6, 1>(a, cus, stream);
  const dim3 grid((unsigned)std::min<int64_t>((a.N + 15) / 16, cus));
  return launch_k(linear_rows_long_kernel<F16, 8, 4>, grid, dim3(512), 0, stream, Ev{}, a);
}

template <bool F16, int CT>
static hipError_t launch_mid(const LinearArgs& a, int cus, hipStream_t stream) {
  const int64_t tiles = (a.N + 15) / 16, rows = (a.M + 16 * CT - 1) / (16 * CT);
  if (tiles * rows <= cus)
    return launch_k(linear_mid_kernel<F16, CT, 1>, dim3((unsigned)(tiles * rows)), dim3(512), 0, stream, Ev{}, a,
                    (int)tiles);
  const int64_t pairs = (tiles + 1) / 2;
  return launch_k(linear_mid_kernel<F16, CT, 2>, dim3((unsigned)(pairs * rows)), dim3(512), 0, stream, Ev{}, a,
                  (int)pairs);
}

template <bool F16>
static hipError_t launch_type(const LinearArgs& a, int cus, hipStream_t stream) {
  if (a.M <= 16) return launch_16_rows<F16>(a, cus, stream);
  if (a.M <= 32) return launch_mid<F16, 2>(a, cus, stream);
  if (a.M <= 64 || getenv("LMID")) return launch_mid<F16, 4>(a, cus, stream);
  if (getenv("LT2")) return launch_tile<F16, 2, 4, 4, 2>(a, stream);
  return launch_tile<F16, 4, 4, 4, 2>(a, stream);
}

hipError_t launch_linear(const LinearArgs& a, int cus, hipStream_t stream) {
  return a.x_type == MOE_FP16 ? launch_type<true>(a, cus, stream) : launch_type<false>(a, cus, stream);
}

}  // namespace qmoe
