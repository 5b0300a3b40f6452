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
    // 253 and 254 become 255, NaN: 4 x 2^126 and 2 x 2^127 are above bf16's
    // largest number, so the kernels that fold the scale into the weight would
    // not agree with those that scale the sums
    const uint8_t v = n < N && b < K / 32 ? s[n * (K / 32) + b] : (uint8_t)127;
    sp[o] = v < 253 ? v : (uint8_t)255;
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
// call), so that they move as one piece; 2: so are pieces of 16 bytes.
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

// 16 bytes of row m from column n on, from their sums.
__device__ __forceinline__ void store_piece(const LinearArgs& a, int64_t m, int64_t n, const float* sums) {
  const bool f16 = a.x_type == MOE_FP16;
  float v[8];
  const int cols = a.y_type == MOE_FP32 ? 4 : 8;
  *reinterpret_cast<v4f*>(v) = *reinterpret_cast<const v4f*>(sums);
  if (cols == 8) *reinterpret_cast<v4f*>(v + 4) = *reinterpret_cast<const v4f*>(sums + 4);
  auto add16 = [&](const uint16_t* b, int i) { v[i] += f16 ? fp16_value(b[i]) : bf16_value(b[i]); };
  if (a.bias) {
    const uint16_t* b = reinterpret_cast<const uint16_t*>(a.bias) + n;
    union {
      uint2 q[2];
      uint16_t b[8];
    } w;
    w.q[0] = *reinterpret_cast<const uint2*>(b);
    if (cols == 8) w.q[1] = *reinterpret_cast<const uint2*>(b + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) add16(w.b, i);
    if (cols == 8) {
#pragma unroll
      for (int i = 4; i < 8; ++i) add16(w.b, i);
    }
  }
  if (cols == 4) {
    v4f t = *reinterpret_cast<v4f*>(v);
    if (a.residual) t += *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(a.residual) + m * a.ldr + n);
    *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.y) + m * a.ldy + n) = t;
    return;
  }
  union {
    uint4 q;
    uint16_t b[8];
  } w;
  if (a.residual) {
    w.q = ld16(reinterpret_cast<const uint16_t*>(a.residual) + m * a.ldr + n);
#pragma unroll
    for (int i = 0; i < 8; ++i) add16(w.b, i);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) w.b[i] = f16 ? fp16_bits(v[i]) : bf16_bits(v[i]);
  *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.y) + m * a.ldy + n) = w.q;
}

// scale_operand of a byte number known after unrolling
__device__ __forceinline__ float scale_of(uint32_t d, int j) {
  return j == 0 ? scale_operand<0>(d) : j == 1 ? scale_operand<1>(d) : j == 2 ? scale_operand<2>(d) : scale_operand<3>(d);
}

__device__ __forceinline__ float scale_value(uint32_t d, int j) {
  return j == 0 ? e8m0_value<0>(d) : j == 1 ? e8m0_value<1>(d) : j == 2 ? e8m0_value<2>(d) : e8m0_value<3>(d);
}

// Where x's 16-byte chunk c (of a row's 16 in a K-step) of row m of a 16-row
// block lies in LDS, in chunks: operand j = c / 4 of the block is 64
// consecutive chunks, lane 16 g + r reading row r, g = c % 4. The rows of a
// group are exchanged by r ^ c, so that the 16 lanes that write a row's
// chunks, like the 16 that read a group, meet all banks.
__device__ __forceinline__ int x_slot(int block, int c, int m) {
  return (block * 4 + (c >> 2)) * 64 + 16 * (c & 3) + (m ^ c);
}

// ----------------------------------------------------------------- few rows
// A workgroup of W waves computes 16 columns of y at a time for up to 16 rows
// of x; the waves split K. Wave w owns K-steps w S .. w S + S - 1 of 128 and
// keeps its fragments of x as MFMA operands in registers over all the tiles
// of the workgroup. Its weights stream through a ring of D tiles' registers:
// the piece of a tile D ahead is requested as soon as a slot's products are
// issued, so a wave has about S D KB under way at any time. The W partial
// sums of a tile are added in wave order through LDS. Bound by the weights'
// bytes once there are many (4 x 131072 x 6144: 73 us, 5.9 TB/s), by the start
// and x's way to every CU below (16 x 8192 x 6144: 8.7 us, 3.1 TB/s; 1 x 6144 x
// 2048: 4.5 us).
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
  // MFMA j (K 32 j .. + 31) against CT column tiles: acc[u] += w x[u]
  template <int CT>
  __device__ __forceinline__ void mul(int j, const uint4 (&x)[CT], v4f (&acc)[CT]) const {
    const uint32_t d = j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w;
    if constexpr (F16) {
      const uint32_t rs[4] = {sc.x, sc.y, sc.z, sc.w};
      const v8h wf = fp4x8_f16(d);
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = scale_value(rs[i], j);
#pragma unroll
      for (int u = 0; u < CT; ++u) {
        const v4f p = mfma_f16(wf, __builtin_bit_cast(v8h, x[u]), v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[u][i] += p[i] * f[i];
      }
    } else {
      const v8s wf = fp4x8_bf16(d, scale_of(sc.x, j));
#pragma unroll
      for (int u = 0; u < CT; ++u) acc[u] = mfma_bf16(wf, __builtin_bit_cast(v8s, x[u]), acc[u]);
    }
  }
};

template <bool F16, int W, int S, int D>
__global__ __launch_bounds__(64 * W) void linear_rows_kernel(const LinearArgs a) {
  __shared__ v4f red[2][W][64];
  __shared__ uint4 xs[W][256];
  const int wave = wave_id(), lane = threadIdx.x & 63;
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
  // x: whole 256-byte row pieces, four rows a load, turned into operands
  // through 4 KB of LDS of the wave's own as the first tile's steps come to
  // them. (Every CU reads all of x: 16 x 6144 is 50 MB from the L2s, 2.6 us of
  // their bandwidth, so the first products do not wait for all of it.)
  uint4 xf[S][4][1], xv[S][4];
  const uint16_t* xp = reinterpret_cast<const uint16_t*>(a.x);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    load(0, s, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // rows past M and pieces past K: others again (no branch: the compiler
      // counts the loads under way). Rows past M are not stored, pieces past K
      // become zero on their way to LDS.
      const int k = 128 * (wave * S + s) + 8 * r, m = min(4 * i + g, (int)a.M - 1);
      xv[s][i] = ld16(xp + m * a.ldx + (k < K ? k : 0));
    }
  }
#pragma unroll
  for (int d = 1; d < D; ++d)
#pragma unroll
    for (int s = 0; s < S; ++s) load(d, s, d);
  auto operands = [&](int s) {
    uint4* mine = &xs[wave][0];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (128 * (wave * S + s) + 128 > K && 128 * (wave * S + s) + 8 * r >= K) xv[s][i] = make_uint4(0, 0, 0, 0);
      mine[x_slot(0, r, 4 * i + g)] = xv[s][i];
    }
    wave_lds_order();
#pragma unroll
    for (int j = 0; j < 4; ++j) xf[s][j][0] = mine[x_slot(0, 4 * j + g, r)];
    wave_lds_order();
  };

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
  auto compute = [&](int d, int i, auto reload, auto first) __attribute__((always_inline)) {
    v4f acc[1] = {{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if constexpr (first) operands(s);
      // a step past the last takes no part (its codes could meet a scale that
      // overflows, and zero times that is not zero)
      if (wave * S + s >= nks) ring[d][s].clear();
#pragma unroll
      for (int j = 0; j < 4; ++j) ring[d][s].template mul<1>(j, xf[s][j], acc);
      if constexpr (reload) load(d, s, i + D);
    }
    tile_done(i, acc[0]);
  };
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  if constexpr (D == 1) {  // one tile
    compute(0, 0, no, yes);
  } else {
    compute(0, 0, yes, yes);
#pragma unroll
    for (int d = 1; d < D; ++d)
      if (d < own) compute(d, d, yes, no);
    int i = D;
    for (; i + D < own; i += D)
#pragma unroll
      for (int d = 0; d < D; ++d) compute(d, i + d, yes, no);
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (i + d < own) compute(d, i + d, no, no);
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
// in turn and share no operand, so the loop has no barrier: weights go from
// memory to registers, x through a piece of LDS of the wave's own (whole
// 256-byte row pieces are read: operand-shaped loads, 64 bytes of 16 rows
// each, took three times as long), both P of the wave's steps ahead. The
// partial sums are joined through LDS at the end. x is read once per 16 R
// columns (from the L2): R = 2 where there are tiles enough. Bound by the L2
// reads and the loads' latency: 32 x 6144 x 6144 9.7 us, 64 rows 16.9 us (192 MB
// from the L2s, 11 TB/s). 16 rows of a K that the kernel above does not take: 16 x
// 8192 x 7168 10.9 us, x 8192 11.2, x 16384 18.4; 4 x 131072 x 8192 143 us (4.0 TB/s
// of weights; the kernel above at K 6144 5.9).
template <bool F16, int CT, int R>
__global__ __launch_bounds__(512) void linear_mid_kernel(const LinearArgs a, int tiles_n) {
  constexpr int W = 8, P = CT == 1 ? 4 : 2;
  __shared__ uint4 xs[W][CT * 256];  // and the partial sums [W][CT][64]
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int K = (int)a.K, nks = (K + 127) / 128;
  const int tile = (int)(blockIdx.x % tiles_n) * R;
  const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * (16 * CT);
  const int last = (int)((a.N + 15) / 16) - 1;
  const uint16_t* xr[CT * 4];
#pragma unroll
  for (int i = 0; i < CT * 4; ++i)
    xr[i] = reinterpret_cast<const uint16_t*>(a.x) + min(m0 + 4 * i + g, a.M - 1) * a.ldx;
  WeightStep<F16> w[P][R];
  uint4 xv[P][CT * 4];
  auto load_w = [&](int p, int ks) {
#pragma unroll
    for (int t = 0; t < R; ++t)
      w[p][t].load(a, (size_t)min(tile + t, last) * nks + min(ks, nks - 1), ks < nks ? lane : 0);
  };
  auto load_x = [&](int p, int ks) {
    const int k = 128 * min(ks, nks - 1);
    const int at = k + 8 * r < K ? k + 8 * r : 0;
    // past the last step: one address for all lanes, hardly any traffic
#pragma unroll
    for (int i = 0; i < CT * 4; ++i) xv[p][i] = ld16(ks < nks ? xr[i] + at : reinterpret_cast<const uint16_t*>(a.x));
  };
  v4f acc[R][CT];
#pragma unroll
  for (int t = 0; t < R; ++t)
#pragma unroll
    for (int u = 0; u < CT; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int p = 0; p < P; ++p) load_w(p, wave + p * W);
#pragma unroll
  for (int p = 0; p < P; ++p) load_x(p, wave + p * W);
  auto step = [&](int p, int ks) __attribute__((always_inline)) {
    if (128 * ks + 128 > K && 128 * ks + 8 * r >= K) {  // past K: zero (as the codes are)
#pragma unroll
      for (int i = 0; i < CT * 4; ++i) xv[p][i] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < CT * 4; ++i) xs[wave][x_slot(i >> 2, r, 4 * (i & 3) + g)] = xv[p][i];
    wave_lds_order();
    load_x(p, ks + P * W);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 x[CT];
#pragma unroll
      for (int u = 0; u < CT; ++u) x[u] = xs[wave][x_slot(u, 4 * j + g, r)];
#pragma unroll
      for (int t = 0; t < R; ++t) w[p][t].template mul<CT>(j, x, acc[t]);
    }
    wave_lds_order();
    load_w(p, ks + P * W);
  };
  // out of the loop itself, not round its end: paths that met there would make
  // the next round wait for all loads
  for (int k0 = wave;; k0 += P * W) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (k0 + p * W >= nks) goto done;
      step(p, k0 + p * W);
    }
  }
done:
  v4f(*const red)[CT][64] = reinterpret_cast<v4f(*)[CT][64]>(&xs[0][0]);
#pragma unroll
  for (int t = 0; t < R; ++t) {
    __syncthreads();
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
// A workgroup of WN x WM waves computes BN = 16 TN WN columns of y for BM =
// 16 TM WM rows of x; a wave 16 TN x 16 TM of it. x goes through LDS (two
// buffers of one K-step of 128; whole 256-byte row pieces are read, and kept
// in registers for two steps until their buffer is free); weights go straight
// from their packed form to registers, PW steps ahead, and are widened there:
// a wave's rows are read by WM waves only. x's operands are read from LDS RD - 1
// ahead of their MFMAs, in a fixed order: read where they are needed, two waves
// a SIMD did not hide the LDS (with the rows of a tile in one wave 241 -> 235
// us at 4096 x 6144 x 6144, fp16 464 -> 447). fp16 x is split into two bf16 on its
// way into LDS (exact; the same products, twice the MFMAs). With one step of
// weights ahead a K-step took 2.2 us, their latency, where its products take
// 0.85. 4096 x 6144 x 6144: 235 us, 1310 TFLOP/s (fp16: 447 us), bound by MFMAs
// and the widening between them (with the residual, 253 us: MFMAs busy 49 % of the
// SIMDs' time, vector ALUs 28 %, and the two overlap by a quarter only; fp16 54 and
// 54 %); 256 rows 31 us, 192 workgroups for 256 CUs, MFMAs busy 25 %.
template <bool F16, int TN, int TM, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM) void linear_tile_kernel(const LinearArgs a, int tiles_m, int tiles_n) {
  constexpr int W = WN * WM, BM = 16 * TM * WM, BN = 16 * TN * WN;
  constexpr int NX = BM / 4 / W;  // pieces of 4 rows x 128 K staged by a wave
  constexpr int PW = 4;           // weight steps in registers
  constexpr int RD = 4;           // operands of x in registers
  static_assert(BM % (4 * W) == 0, "whole pieces");
  constexpr int P = F16 ? 2 : 1;  // bf16 planes of x
  __shared__ uint4 xs[2][P][BM * 16];
  const int wave = wave_id(), lane = threadIdx.x & 63;
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
    const int at = k + 8 * r < K ? k + 8 * r : 0;
    // past the last step: one address for all lanes, hardly any traffic
#pragma unroll
    for (int i = 0; i < NX; ++i) v[i] = ld16(ks < nks ? xr[i] + at : reinterpret_cast<const uint16_t*>(a.x));
  };
  auto put_x = [&](uint4(&v)[NX], int buf, int ks) {
    // K's last step may end inside a row piece: zero there (as the codes are;
    // not at the load, which would be waited for)
    if (128 * ks + 128 > K && 128 * ks + 8 * r >= K) {
#pragma unroll
      for (int i = 0; i < NX; ++i) v[i] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int piece = wave * NX + i;
      const int at = x_slot(piece >> 2, r, 4 * (piece & 3) + g);
      if constexpr (F16) {
        v8s hi, lo;
        fp16x8_planes(v[i], hi, lo);
        xs[buf][0][at] = __builtin_bit_cast(uint4, hi);
        xs[buf][P - 1][at] = __builtin_bit_cast(uint4, lo);
      } else {
        xs[buf][0][at] = v[i];
      }
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
    const int kc = min(ks, nks - 1), used = ks < nks ? ~0 : 0;
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      q[p][t] = ld16(a.wp + (rb[t] + kc) * 1024 + 16 * (lane & used));
      sc[p][t] = ld4(a.sp + (rb[t] + kc) * 64 + 4 * (r & used));
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
  put_x(xv[0], 0, 0);
  load_x(xv[0], 2);
  barrier_lds();
  auto step = [&](int p, int ks) __attribute__((always_inline)) {
    constexpr int NF = 4 * TM * P;
    v8s f[RD], wf[TN];
    // operand i: MFMA j's of row tile u, the lower plane first
    auto operand = [&](int i) __attribute__((always_inline)) {
      const int j = i / (TM * P), u = i / P % TM, pl = P - 1 - i % P;
      f[i % RD] = __builtin_bit_cast(v8s, xs[p & 1][pl][x_slot(wm * TM + u, 4 * j + g, r)]);
    };
#pragma unroll
    for (int i = 0; i < RD - 1; ++i) operand(i);
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const int j = i / (TM * P), u = i / P % TM;
      if (i + RD - 1 < NF) operand(i + RD - 1);
      if (i % (TM * P) == 0) {
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          const uint32_t d = j == 0 ? q[p][t].x : j == 1 ? q[p][t].y : j == 2 ? q[p][t].z : q[p][t].w;
          wf[t] = fp4x8_bf16(d, scale_of(sc[p][t], j));
        }
      }
#pragma unroll
      for (int t = 0; t < TN; ++t) acc[t][u] = mfma_bf16(wf[t], f[i % RD], acc[t][u]);
      __builtin_amdgcn_sched_barrier(0x16);  // ALU work and memory loads may move across, LDS and MFMAs not
      if (i == TM * P - 1) {
        // step ks + 1's x into the buffer that step ks - 1 was read from
        put_x(xv[(p + 1) & 1], (p + 1) & 1, ks + 1);
        load_x(xv[(p + 1) & 1], ks + 3);
      }
    }
    load_w(p, ks + PW);
    barrier_lds();
  };
  // out of the loop itself, not round its end: paths that met there would make
  // the next round wait for all loads
  for (int k0 = 0;; k0 += PW) {
#pragma unroll
    for (int p = 0; p < PW; ++p) {
      if (k0 + p >= nks) goto done;
      step(p, k0 + p);
    }
  }
done:
  if (a.vec == 2) {
    // 16 rows of y at a time through LDS of the wave's own (the last step's
    // barrier freed it), so that residual and y move in 16-byte pieces along a
    // row: 4096 x 6144 x 6144 with residual 259 us, 266 where each lane moved
    // the 8-byte pieces its sums lie in
    constexpr int C = 16 * TN, S = C + 4;  // (+ 4: 16 rows of a column on all banks)
    static_assert(sizeof(xs) >= 4 * W * 16 * S, "the sums fit x's buffers");
    float* mine = reinterpret_cast<float*>(xs) + wave * 16 * S;
    const int es = a.y_type == MOE_FP32 ? 4 : 2, e = 16 / es;  // bytes, elements a piece
    const int per_row = C / e;
#pragma unroll
    for (int u = 0; u < TM; ++u) {
#pragma unroll
      for (int t = 0; t < TN; ++t) *reinterpret_cast<v4f*>(&mine[r * S + 16 * t + 4 * g]) = acc[t][u];
      wave_lds_order();
      for (int i = lane; i < 16 * per_row; i += 64) {
        const int row = i / per_row, c = i % per_row * e;
        const int64_t m = m0 + 16 * (wm * TM + u) + row, n = n0 + C * wn + c;
        if (m < a.M && n < a.N) store_piece(a, m, n, &mine[row * S + c]);
      }
      wave_lds_order();
    }
    return;
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

template <bool F16, int CT, int R>
static hipError_t launch_mid(const LinearArgs& a, hipStream_t stream) {
  const int64_t tiles = (a.N + 16 * R - 1) / (16 * R), rows = (a.M + 16 * CT - 1) / (16 * CT);
  return launch_k(linear_mid_kernel<F16, CT, R>, dim3((unsigned)(tiles * rows)), dim3(512), 0, stream, Ev{}, a,
                  (int)tiles);
}

// The kernels a call may run, by the rules of `choose`: name, and per type of x
// the launch (NULL: not for that type).
namespace {

typedef hipError_t (*Launch)(const LinearArgs& a, int cus, hipStream_t stream);
struct Choice {
  const char* name;
  Launch launch[2];  // bf16, fp16 x
};

// up to 16 rows: K-steps a wave, workgroups a CU
template <bool F16, int S, int OCC>
hipError_t rows(const LinearArgs& a, int cus, hipStream_t stream) {
  return launch_rows<F16, 8, S, OCC>(a, cus, stream);
}
template <bool F16, int CT, int R>
hipError_t mid(const LinearArgs& a, int, hipStream_t stream) {
  return launch_mid<F16, CT, R>(a, stream);
}
template <bool F16, int TN, int TM, int WN, int WM>
hipError_t tile(const LinearArgs& a, int, hipStream_t stream) {
  return launch_tile<F16, TN, TM, WN, WM>(a, stream);
}

enum { kMid1 = 6, kMidRows = 8, kChoices = 13 };
constexpr Choice kChoice[kChoices] = {
    {"rows, 1 K-step a wave", {rows<false, 1, 3>, rows<true, 1, 3>}},
    {"rows, 2 K-steps a wave", {rows<false, 2, 2>, rows<true, 2, 2>}},
    {"rows, 3 K-steps a wave", {rows<false, 3, 1>, rows<true, 3, 1>}},
    // more K-steps a wave (fp16 4, bf16 7 and 8) fit the registers as well, are not
    // there, and go to the ones below
    {"rows, 4 K-steps a wave", {rows<false, 4, 1>, nullptr}},
    {"rows, 5 K-steps a wave", {rows<false, 5, 1>, nullptr}},
    {"rows, 6 K-steps a wave", {rows<false, 6, 1>, nullptr}},
    {"16 x 16, K split over the waves", {mid<false, 1, 1>, mid<true, 1, 1>}},
    {"16 x 32, K split over the waves", {mid<false, 1, 2>, mid<true, 1, 2>}},
    {"32 x 16, K split over the waves", {mid<false, 2, 1>, mid<true, 2, 1>}},
    {"32 x 32, K split over the waves", {mid<false, 2, 2>, mid<true, 2, 2>}},
    // all rows of a tile by every wave (weights widened once a workgroup, not
    // twice) where that measured faster: bf16 M 256 by the first 30.9 against
    // 32.5 us, M 4096 by the third 235 against 246; by the second 310 against 304
    {"64 x 128 tile", {tile<false, 1, 4, 8, 1>, tile<true, 1, 4, 8, 1>}},
    {"128 x 128 tile", {tile<false, 2, 4, 4, 2>, tile<true, 2, 4, 4, 2>}},
    {"128 x 256 tile", {tile<false, 2, 8, 8, 1>, tile<true, 4, 4, 4, 2>}},
};

int choose(int64_t M, int64_t N, int64_t K, bool f16, int cus) {
  const int64_t tiles = (N + 15) / 16;
  if (M <= 16) {
    const int64_t S = ((K + 127) / 128 + 7) / 8;
    if (S <= (f16 ? 3 : 6)) return (int)S - 1;
    // a longer K: x from the L2 for every 16 or 32 columns
    return tiles <= cus ? kMid1 : kMid1 + 1;
  }
  // Rounds of workgroups over the CUs times a round's time per K-step, in
  // units of 10 ns (N and K 6144, bf16 x; M 32: 14.4 us by the first against 9.6
  // by the second; M 64: 20.8, 16.9 and 30.7 by the first three; M 128: 26 and 31
  // by the second and third, M 256: 46.6, 31.4 and 49 by the second to fourth;
  // M 1024: 83, 98 and 71, M 4096: 312, 304 and 235 by the last three. fp16 x: M
  // 64 25, 21 and 59 by the first three, M 256 61, 59 and 97 by the second to
  // fourth, M 4096 604, 593 and 452 by the last three).
  auto cost = [&](int64_t bm, int64_t bn, int per) {
    const int64_t groups = ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
    return ((groups + cus - 1) / cus) * per;
  };
  const int64_t c[5] = {cost(32, 16, f16 ? 16 : 14), cost(32, 32, f16 ? 22 : 16), cost(64, 128, f16 ? 105 : 60),
                        cost(128, 128, f16 ? 195 : 97), cost(128, 256, f16 ? 280 : 150)};
  return kMidRows + (int)(std::min_element(c, c + 5) - c);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, int cus, hipStream_t stream) {
  const bool f16 = a.x_type == MOE_FP16;
  return kChoice[choose(a.M, a.N, a.K, f16, cus)].launch[f16](a, cus, stream);
}

const char* linear_kernel_name(int64_t M, int64_t N, int64_t K, bool f16, int cus) {
  return kChoice[choose(M, N, K, f16, cus)].name;
}

}  // namespace qmoe
