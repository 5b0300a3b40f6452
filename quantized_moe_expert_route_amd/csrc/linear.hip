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
// A workgroup of W waves computes 16 columns of y for up to 16 rows of x at a
// time. The waves split K: wave w owns S K-steps of 128 in every segment of
// W S steps, and keeps its fragments of x in registers over all the tiles of
// the workgroup while one segment covers K. The W partial sums are added in
// wave order through LDS.
template <bool F16, int W, int S>
__global__ __launch_bounds__(64 * W) void linear_rows_kernel(const LinearArgs a) {
  __shared__ v4f red[2][W][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int K = (int)a.K, nks = (K + 127) / 128, nseg = (nks + W * S - 1) / (W * S);
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  const bool row = m0 + r < a.M;
  const uint16_t* xr = reinterpret_cast<const uint16_t*>(a.x) + (row ? m0 + r : 0) * a.ldx;
  const int ntiles = (int)((a.N + 15) / 16);

  uint4 xf[S][4], q[S], nq[S];
  uint4 sc[S], nsc[S];  // bf16: .x is the row's four scales; fp16: rows 4g..4g+3
  auto load_x = [&](int seg) {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = 128 * ((seg * W + wave) * S + s) + 32 * j + 8 * g;
        xf[s][j] = row && k < K ? ld16(xr + k) : make_uint4(0, 0, 0, 0);
      }
  };
  auto load_w = [&](int tile, int seg, uint4(&qq)[S], uint4(&ss)[S]) {
    const size_t base = (size_t)tile * nks;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      // past the last step: that step again, with x zero
      const size_t p = base + min((seg * W + wave) * S + s, nks - 1);
      qq[s] = ld16(a.wp + p * 1024 + 16 * lane);
      if (F16) ss[s] = ld16(a.sp + p * 64 + 16 * g);
      else ss[s].x = ld4(a.sp + p * 64 + 4 * r);
    }
  };

  int tile = blockIdx.x, seg = 0, buf = 0;
  if (tile >= ntiles) return;
  load_w(tile, 0, nq, nsc);
  load_x(0);
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  while (tile < ntiles) {
#pragma unroll
    for (int s = 0; s < S; ++s) { q[s] = nq[s]; sc[s] = nsc[s]; }
    int ntile = tile, nsg = seg + 1;
    if (nsg == nseg) { nsg = 0; ntile += gridDim.x; }
    if (ntile < ntiles) load_w(ntile, nsg, nq, nsc);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      // a step past the last one takes no part (its codes could meet a scale
      // that overflows, and zero times that is not zero)
      const bool in = (seg * W + wave) * S + s < nks;
      const uint32_t d[4] = {in ? q[s].x : 0u, in ? q[s].y : 0u, in ? q[s].z : 0u, in ? q[s].w : 0u};
      const uint32_t rs[4] = {sc[s].x, sc[s].y, sc[s].z, sc[s].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (F16) {
          const v4f z = {0.f, 0.f, 0.f, 0.f};
          const v4f p = mfma_f16(fp4x8_f16(d[j]), __builtin_bit_cast(v8h, xf[s][j]), z);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] += p[i] * e8m0_value((rs[i] >> (8 * j)) & 255u);
        } else {
          acc = mfma_bf16(fp4x8_bf16(d[j], scale_of(sc[s].x, j)), __builtin_bit_cast(v8s, xf[s][j]), acc);
        }
      }
    }
    if (nsg == 0) {
      red[buf][wave][lane] = acc;
      acc = v4f{0.f, 0.f, 0.f, 0.f};
      barrier_lds();
      // lane holds rows 4 g .. 4 g + 3 (columns of y) of column r (row of x)
      if (wave == buf && row) {
        v4f v = red[buf][0][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) v += red[buf][w][lane];
        store4(a, m0 + r, (int64_t)tile * 16 + 4 * g, v);
      }
      buf ^= 1;
    }
    if (nseg > 1 && ntile < ntiles) load_x(nsg);
    tile = ntile;
    seg = nsg;
  }
}

template <bool F16, int S>
static hipError_t launch_rows(const LinearArgs& a, int cus, hipStream_t stream) {
  const int64_t tiles = (a.N + 15) / 16;
  const dim3 grid((unsigned)std::min<int64_t>(tiles, 2 * cus), (unsigned)((a.M + 15) / 16));
  return launch_k(linear_rows_kernel<F16, 8, S>, grid, dim3(512), 0, stream, Ev{}, a);
}

// ----------------------------------------------------------------- many rows
// A workgroup of WN x WM waves computes BN = 16 TN WN columns of y for BM =
// 16 TM WM rows of x; a wave 16 TN x 16 TM of it. x goes through LDS in the
// MFMA's operand order (a fragment of 16 rows x 32 K is 1 KB contiguous, read
// back in lane order), two buffers of one K-step of 128, the next step's x in
// registers meanwhile; weights go straight from their packed form to
// registers, one K-step ahead, and are widened there: a wave's rows are read
// by WM waves only.
template <bool F16, int TN, int TM, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM) void linear_tile_kernel(const LinearArgs a, int tiles_m, int tiles_n) {
  constexpr int W = WN * WM, BM = 16 * TM * WM, BN = 16 * TN * WN;
  constexpr int NF = BM / 16 * 4;        // fragments of a K-step
  constexpr int NX = (NF + W - 1) / W;   // of them staged by a wave
  __shared__ uint4 xs[2][NF][64];
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

  const uint16_t* xp = reinterpret_cast<const uint16_t*>(a.x);
  const uint16_t* xr[NX];
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    const int f = min(wave + i * W, NF - 1);
    xr[i] = xp + min(m0 + 16 * (f >> 2) + r, a.M - 1) * a.ldx + 32 * (f & 3) + 8 * g;
  }
  uint4 xv[NX];
  auto load_x = [&](int ks) {
    if (128 * ks + 128 <= K) {
#pragma unroll
      for (int i = 0; i < NX; ++i) xv[i] = ld16(xr[i] + 128 * ks);
    } else {
#pragma unroll
      for (int i = 0; i < NX; ++i) {
        const int k = 128 * ks + 32 * (min(wave + i * W, NF - 1) & 3) + 8 * g;
        xv[i] = k < K ? ld16(xr[i] + 128 * ks) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  auto put_x = [&](int buf) {
#pragma unroll
    for (int i = 0; i < NX; ++i)
      if (NF % W == 0 || wave + i * W < NF) xs[buf][wave + i * W][lane] = xv[i];
  };
  // row blocks past N: the last one again (not stored)
  size_t rb[TN];
#pragma unroll
  for (int t = 0; t < TN; ++t)
    rb[t] = (size_t)min(n0 / 16 + wn * TN + t, (a.N + 15) / 16 - 1) * nks;
  uint4 q[TN], nq[TN];
  uint32_t sc[TN], nsc[TN];
  auto load_w = [&](int ks) {
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      nq[t] = ld16(a.wp + (rb[t] + ks) * 1024 + 16 * lane);
      nsc[t] = ld4(a.sp + (rb[t] + ks) * 64 + 4 * r);
    }
  };

  v4f acc[TN][TM];
#pragma unroll
  for (int t = 0; t < TN; ++t)
#pragma unroll
    for (int u = 0; u < TM; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
  load_x(0);
  load_w(0);
  put_x(0);
  barrier_lds();
  for (int ks = 0; ks < nks; ++ks) {
#pragma unroll
    for (int t = 0; t < TN; ++t) { q[t] = nq[t]; sc[t] = nsc[t]; }
    if (ks + 1 < nks) {
      load_x(ks + 1);
      load_w(ks + 1);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v8s wf[TN];
#pragma unroll
      for (int t = 0; t < TN; ++t) {
        const uint32_t d = j == 0 ? q[t].x : j == 1 ? q[t].y : j == 2 ? q[t].z : q[t].w;
        wf[t] = fp4x8_bf16(d, scale_of(sc[t], j));
      }
#pragma unroll
      for (int u = 0; u < TM; ++u) {
        const uint4 f = xs[ks & 1][(wm * TM + u) * 4 + j][lane];
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
    if (ks + 1 < nks) {
      put_x((ks + 1) & 1);  // the buffer of step ks - 1: read by nobody since the last barrier
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

hipError_t launch_linear(const LinearArgs& a, int cus, hipStream_t stream) {
  const int64_t nks = (a.K + 127) / 128;
  const bool f16 = a.x_type == MOE_FP16;
  if (a.M > 64) return f16 ? launch_tile<true, 4, 4, 4, 2>(a, stream) : launch_tile<false, 4, 4, 4, 2>(a, stream);
  if (nks <= 8) return f16 ? launch_rows<true, 1>(a, cus, stream) : launch_rows<false, 1>(a, cus, stream);
  if (nks <= 16) return f16 ? launch_rows<true, 2>(a, cus, stream) : launch_rows<false, 2>(a, cus, stream);
  if (nks <= 32) return f16 ? launch_rows<true, 4>(a, cus, stream) : launch_rows<false, 4>(a, cus, stream);
  return f16 ? launch_rows<true, 6>(a, cus, stream) : launch_rows<false, 6>(a, cus, stream);
}

}  // namespace qmoe
