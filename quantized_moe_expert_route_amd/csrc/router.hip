// Router projection: logits[m][e] = sum_h x[m][h] w[e][h], one rounding to
// binary32. x bf16 or fp16, w bf16 or fp32.
//
// Up to 16 tokens the sums are float64: the routing compares logits, and with
// sums exact to ~2^-50 two logits swap places only where their exact values
// round to the same binary32 number. Above, they are binary32 sums of exact
// products, off by at most (48 + H / 32) 2^-23 of the products' magnitudes, so
// that of two experts whose logits lie that near the other may be picked.
#include <algorithm>

#include "internal.h"
#include "mxfp4.h"
#include "ops.h"

namespace qmoe {

// 8 consecutive elements of a row, as loaded and as float.
template <int TYPE>
struct Raw8 {
  uint4 v[TYPE == MOE_FP32 ? 2 : 1];
};
template <int TYPE>
__device__ __forceinline__ void raw8(const void* p, int64_t i, Raw8<TYPE>& q) {
  if constexpr (TYPE == MOE_FP32) {
    q.v[0] = ld16(reinterpret_cast<const float*>(p) + i);
    q.v[1] = ld16(reinterpret_cast<const float*>(p) + i + 4);
  } else {
    q.v[0] = ld16(reinterpret_cast<const uint16_t*>(p) + i);
  }
}
template <int TYPE>
__device__ __forceinline__ void values8(const Raw8<TYPE>& q, float (&v)[8]) {
  const uint32_t d[4] = {q.v[0].x, q.v[0].y, q.v[0].z, q.v[0].w};
  if constexpr (TYPE == MOE_FP32) {
    const uint32_t u[4] = {q.v[1].x, q.v[1].y, q.v[1].z, q.v[1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(d[i]);
      v[4 + i] = __uint_as_float(u[i]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = TYPE == MOE_BF16 ? __uint_as_float(d[j] << 16) : fp16_value((uint16_t)(d[j] & 0xFFFFu));
      v[2 * j + 1] = TYPE == MOE_BF16 ? __uint_as_float(d[j] & 0xFFFF0000u) : fp16_value((uint16_t)(d[j] >> 16));
    }
  }
}

__device__ __forceinline__ double shfl_xor_f64(double v, int o) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __shfl_xor((uint32_t)u, o, kWave), hi = __shfl_xor((uint32_t)(u >> 32), o, kWave);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

constexpr int kRouterWaves = 12;  // 3 a SIMD: 168 registers a lane

// Up to 16 tokens: one expert and T tokens a workgroup. A wave takes 512
// elements of H at a time, 8 a lane, all T tokens' pieces under way at once;
// the lanes' float64 sums are added by exchanging halves (T values shrink to
// one a lane), then the waves'. Every workgroup reads all of x: 16 x 6144 is
// 50 MB from the L2s, 2.6 us, about the time of the float64 products. H 6144, 256
// experts: 3.3 us at 1 token, 4.2 at 4 (fp32 weights), 7.6 at 16.
template <int XT, int WT, int T>
__global__ __launch_bounds__(64 * kRouterWaves) void router_kernel(const RouterArgs a) {
  __shared__ double red[kRouterWaves][T];
  const int wave = wave_id(), lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int64_t e = blockIdx.x;
  const int mt = (int)a.M, H = (int)a.H;
  double acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) acc[t] = 0.0;
#pragma unroll 1
  for (int c = (wave * 64 + lane) * 8; c < H; c += waves * 512) {
    Raw8<WT> wr;
    Raw8<XT> xr[T];
    raw8<WT>(a.w, e * a.H + c, wr);
#pragma unroll
    for (int t = 0; t < T; ++t) raw8<XT>(a.x, min(t, mt - 1) * a.ldx + c, xr[t]);
    double w[8];
    float f[8];
    values8<WT>(wr, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (double)f[i];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      values8<XT>(xr[t], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[t] = fma((double)f[i], w[i], acc[t]);
    }
  }
  int bit = 32;
#pragma unroll
  for (int n = T / 2; n >= 1; n >>= 1, bit >>= 1) {
    const bool up = lane & bit;  // keeps the upper half of the tokens
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const double give = up ? acc[i] : acc[i + n];
      acc[i] = (up ? acc[i + n] : acc[i]) + shfl_xor_f64(give, bit);
    }
  }
  for (; bit >= 1; bit >>= 1) acc[0] += shfl_xor_f64(acc[0], bit);
  constexpr int kLanes = 64 / T;
  if (lane % kLanes == 0) red[wave][lane / kLanes] = acc[0];
  __syncthreads();
  if ((int)threadIdx.x < mt) {
    double v = 0.0;
    for (int w = 0; w < waves; ++w) v += red[w][threadIdx.x];
    a.logits[threadIdx.x * a.E + e] = (float)v;
  }
}

// 8 elements as P planes of bf16 whose sum they are: bf16 is one, fp16 two,
// fp32 three (each plane keeps the upper 8 significant bits of what is left:
// 24 = 3 x 8, exact down to bf16's smallest number). A value that is not
// finite is so in the first, the others zero: sums with it come out as an
// infinity or a NaN, if not always the right one of the two (infinity times
// another's zero plane), and are formed anew by redo_odd.
template <int TYPE>
constexpr int kPlanes = TYPE == MOE_BF16 ? 1 : TYPE == MOE_FP16 ? 2 : 3;

template <int TYPE>
__device__ __forceinline__ void planes8(const Raw8<TYPE>& q, v8s (&out)[kPlanes<TYPE>]) {
  if constexpr (TYPE == MOE_BF16) {
    out[0] = __builtin_bit_cast(v8s, q.v[0]);
  } else if constexpr (TYPE == MOE_FP16) {
    fp16x8_planes(q.v[0], out[0], out[1]);
  } else {
    const uint32_t d[8] = {q.v[0].x, q.v[0].y, q.v[0].z, q.v[0].w, q.v[1].x, q.v[1].y, q.v[1].z, q.v[1].w};
    uint32_t h[4], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t hi = d[i] & 0xFFFF0000u;
      const bool fine = (d[i] & 0x7F800000u) != 0x7F800000u;
      const float r1 = fine ? __uint_as_float(d[i]) - __uint_as_float(hi) : 0.f;
      const uint32_t mi = __float_as_uint(r1) & 0xFFFF0000u;
      const uint32_t lo = __float_as_uint(r1 - __uint_as_float(mi));
      if (i & 1) {
        h[i >> 1] |= hi;
        m[i >> 1] |= mi;
        l[i >> 1] |= lo & 0xFFFF0000u;
      } else {
        h[i >> 1] = hi >> 16;
        m[i >> 1] = mi >> 16;
        l[i >> 1] = lo >> 16;
      }
    }
    out[0] = as_v8s(h[0], h[1], h[2], h[3]);
    out[1] = as_v8s(m[0], m[1], m[2], m[3]);
    out[2] = as_v8s(l[0], l[1], l[2], l[3]);
  }
}

__device__ __forceinline__ bool odd(float v) { return !(fabsf(v) < INFINITY); }

// Logits e .. e + 3 of token m as the few-token kernel forms them, where what
// this thread stored is not finite: planes of infinities, or a partial sum
// above binary32's range. One logit a lane at a time: a call with an infinite
// token takes some ms (4096 tokens, 256 experts, H 6144: 2.7, an infinity in
// every token 6.3), with NaN, which end their sum, 10 to 20 us more.
template <int XT, int WT>
__device__ __forceinline__ void redo_odd(const RouterArgs& a, int64_t m, int e) {
#pragma unroll 1
  for (int i = e; i < min(e + 4, (int)a.E); ++i) {
    float* const at = a.logits + m * a.E + i;
    if (!odd(*at)) continue;
    double sum = 0.0;
#pragma unroll 1
    for (int64_t c = 0; c < a.H && sum == sum; c += 8) {  // (a NaN stays one)
      Raw8<WT> wr;
      Raw8<XT> xr;
      raw8<WT>(a.w, i * a.H + c, wr);
      raw8<XT>(a.x, m * a.ldx + c, xr);
      float w[8], x[8];
      values8<WT>(wr, w);
      values8<XT>(xr, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) sum = fma((double)x[q], (double)w[q], sum);
    }
    *at = (float)sum;
  }
}

// Up to some hundred tokens: tiles of 16 TN experts x 16 TM tokens on the bf16 MFMA
// (binary32 sums of exact products, planes as above). The W waves of a
// workgroup split K in pieces of 64, so that no operand is shared between
// them: each goes from memory to the wave's registers, without LDS or
// barriers in the loop. The W partial tiles are added in wave order. 77 tokens,
// 161 experts, H 2056 5.3 us (fp16 x); 256 tokens, 256 experts, H 6144 13 us, 1024
// tokens 25: no rate is near its limit (107 and 245 MB from the L2s, MFMAs busy 2
// and 5 % of the time); what is left are the latency of loads of 64 bytes from each
// of 16 rows and the start.
template <int XT, int WT, int TN, int TM, int W>
__global__ __launch_bounds__(64 * W) void router_tile_kernel(const RouterArgs a, int tiles_e) {
  __shared__ v4f red[W][TN * TM > 4 ? 4 : TN * TM][64];
  constexpr int C = TN * TM > 4 ? 4 : TN * TM;  // sub-tiles joined at a time
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int e0 = (int)(blockIdx.x % tiles_e) * 16 * TN;
  const int64_t m0 = (int64_t)(blockIdx.x / tiles_e) * 16 * TM;
  const int H = (int)a.H;
  int64_t wo[TN], xo[TM];
#pragma unroll
  for (int t = 0; t < TN; ++t) wo[t] = (int64_t)min(e0 + 16 * t + r, (int)a.E - 1) * H;
#pragma unroll
  for (int u = 0; u < TM; ++u) xo[u] = min(m0 + 16 * u + r, a.M - 1) * a.ldx;
  v4f acc[TN][TM];
#pragma unroll
  for (int t = 0; t < TN; ++t)
#pragma unroll
    for (int u = 0; u < TM; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
  // piece c: K 64 c .. + 63, lane group g its elements 16 g .. + 15 as two
  // operands; past H they are taken as zero (H is a multiple of 8)
  Raw8<WT> wr[2][TN];
  Raw8<XT> xr[2][TM];
  auto load = [&](int c) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = 64 * c + 16 * g + 8 * j;
      const int kc = min(k, H - 8);
#pragma unroll
      for (int t = 0; t < TN; ++t) raw8<WT>(a.w, wo[t] + kc, wr[j][t]);
#pragma unroll
      for (int u = 0; u < TM; ++u) raw8<XT>(a.x, xo[u] + kc, xr[j][u]);
    }
    if (64 * c + 64 > H) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (64 * c + 16 * g + 8 * j >= H) {
#pragma unroll
          for (int t = 0; t < TN; ++t)
            for (auto& v : wr[j][t].v) v = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int u = 0; u < TM; ++u)
            for (auto& v : xr[j][u].v) v = make_uint4(0, 0, 0, 0);
        }
    }
  };
  const int pieces = (H + 63) / 64;
  for (int c = wave; c < pieces; c += W) {
    load(c);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      v8s wf[TN][kPlanes<WT>];
#pragma unroll
      for (int t = 0; t < TN; ++t) planes8<WT>(wr[j][t], wf[t]);
#pragma unroll
      for (int u = 0; u < TM; ++u) {
        v8s xf[kPlanes<XT>];
        planes8<XT>(xr[j][u], xf);
#pragma unroll
        for (int t = 0; t < TN; ++t)
#pragma unroll
          for (int p = kPlanes<WT> - 1; p >= 0; --p)
#pragma unroll
            for (int q = kPlanes<XT> - 1; q >= 0; --q) acc[t][u] = mfma_bf16(wf[t][p], xf[q], acc[t][u]);
      }
    }
  }
  // lane (g, r): experts 4 g .. + 3 of token r of a sub-tile
#pragma unroll
  for (int s0 = 0; s0 < TN * TM; s0 += C) {
    if (s0) __syncthreads();
#pragma unroll
    for (int s = 0; s < C; ++s) red[wave][s][lane] = acc[(s0 + s) / TM][(s0 + s) % TM];
    __syncthreads();
    for (int i = threadIdx.x; i < C * 64; i += 64 * W) {
      const int s = i >> 6, l = i & 63;
      v4f v = red[0][s][l];
#pragma unroll
      for (int w = 1; w < W; ++w) v += red[w][s][l];
      const int64_t m = m0 + 16 * ((s0 + s) % TM) + (l & 15);
      const int e = e0 + 16 * ((s0 + s) / TM) + 4 * (l >> 4);
      if (m < a.M) {
        float odds = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (e + q < a.E) a.logits[m * a.E + e + q] = v[q];
          odds = fmaf(v[q], 0.f, odds);
        }
        if (odds != 0.f) redo_odd<XT, WT>(a, m, e);
      }
    }
  }
}

// Many tokens: 64 experts x 64 tokens a workgroup. x and the weights go through
// LDS as they are (whole 256- or 512-byte row pieces are read, two K-steps of
// 128 ahead in registers, two LDS buffers), each operand where lane 16 g + r
// reads it, rows exchanged against bank conflicts as in the linear layer. Wave
// w multiplies K's quarter w % 4 of every step for half of the tokens, so that
// an operand read from LDS serves two or four MFMAs; planes are formed there.
// 4096 tokens, 256 experts, H 6144, bf16: 31 us for 411 MB from the L2s (x once per
// 64 experts, the weights once per 64 tokens, 201 MB each) through 256 workgroups,
// one a CU; MFMAs busy 15 % of the time. fp32 weights: 92 us, three MFMAs a product
// and the planes' vector work.
// (With every wave loading its own operands, 64 bytes of 16 rows each, 4096
// tokens of H 6144 to 256 experts took 49 us: the memory pipeline's time.)
template <int XT, int WT>
__global__ __launch_bounds__(512) void router_wide_kernel(const RouterArgs a, int tiles_e) {
  constexpr int NW = WT == MOE_FP32 ? 4 : 2;  // 16-byte pieces of a step's weights a thread
  __shared__ uint4 sx[2][4 * 256], sw[2][NW * 512];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int wk = wave & 3, wm = wave >> 2;
  const int H = (int)a.H, nks = (H + 127) / 128;
  // XCD x (workgroups go to the eight in turn) takes a contiguous eighth of the
  // tiles, the experts of the same tokens side by side
  const int total = gridDim.x, per = total >> 3, rest = total & 7, xcd = blockIdx.x & 7;
  const int id = xcd * per + min(xcd, rest) + (blockIdx.x >> 3);
  const int e0 = id % tiles_e * 64;
  const int64_t m0 = (int64_t)(id / tiles_e) * 64;

  // piece i of this thread: row (thread + 512 i) / pieces of a row
  const uint16_t* xr[2];
  int64_t wr[NW];
  constexpr int kWP = WT == MOE_FP32 ? 32 : 16;
  const int xc = threadIdx.x & 15, wc = threadIdx.x & (kWP - 1);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    xr[i] = reinterpret_cast<const uint16_t*>(a.x) + min(m0 + (threadIdx.x >> 4) + 32 * i, a.M - 1) * a.ldx;
#pragma unroll
  for (int i = 0; i < NW; ++i)
    wr[i] = (int64_t)min(e0 + (int)(threadIdx.x / kWP) + 512 / kWP * i, (int)a.E - 1) * H;
  const int xe = 8 * xc, we = (kWP == 32 ? 4 : 8) * wc;  // first element of the piece
  uint4 xv[2][2], wv[2][NW];
  auto load = [&](int p, int ks) __attribute__((always_inline)) {
    const int k = 128 * min(ks, nks - 1);  // pieces past H: the row's first (zero below)
#pragma unroll
    for (int i = 0; i < 2; ++i) xv[p][i] = ld16(xr[i] + (k + xe < H ? k + xe : 0));
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int64_t at = wr[i] + (k + we < H ? k + we : 0);
      if constexpr (WT == MOE_FP32) wv[p][i] = ld16(reinterpret_cast<const float*>(a.w) + at);
      else wv[p][i] = ld16(reinterpret_cast<const uint16_t*>(a.w) + at);
    }
  };
  // chunk c of row m of a 16-row block
  auto slot = [](int block, int c, int m) { return (block * 4 + (c >> 2)) * 64 + 16 * (c & 3) + (m ^ c); };
  auto put = [&](int p, int buf, int ks) __attribute__((always_inline)) {
    const bool xin = 128 * ks + xe < H, win = 128 * ks + we < H;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = (threadIdx.x >> 4) + 32 * i;
      sx[buf][slot(row >> 4, xc, row & 15)] = xin ? xv[p][i] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int row = threadIdx.x / kWP + 512 / kWP * i;
      // fp32: an operand's 8 elements are two pieces, kept 1024 apart
      const int at = kWP == 32 ? (wc & 1) * 1024 + slot(row >> 4, wc >> 1, row & 15) : slot(row >> 4, wc, row & 15);
      sw[buf][at] = win ? wv[p][i] : make_uint4(0, 0, 0, 0);
    }
  };
  v4f acc[4][2];
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
  load(0, 0);
  load(1, 1);
  put(0, 0, 0);
  load(0, 2);
  barrier_lds();
  auto step = [&](int p, int ks) __attribute__((always_inline)) {
    put(p ^ 1, p ^ 1, ks + 1);  // into the buffer that step ks - 1 was read from
    load(p ^ 1, ks + 3);
    v8s xf[2][kPlanes<XT>];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Raw8<XT> q;
      q.v[0] = sx[p][slot(2 * wm + u, 4 * wk + g, r)];
      planes8<XT>(q, xf[u]);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      Raw8<WT> q;
      q.v[0] = sw[p][slot(t, 4 * wk + g, r)];
      if constexpr (WT == MOE_FP32) q.v[1] = sw[p][1024 + slot(t, 4 * wk + g, r)];
      v8s wf[kPlanes<WT>];
      planes8<WT>(q, wf);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = kPlanes<WT> - 1; i >= 0; --i)
#pragma unroll
          for (int j = kPlanes<XT> - 1; j >= 0; --j) acc[t][u] = mfma_bf16(wf[i], xf[u][j], acc[t][u]);
    }
    barrier_lds();
  };
  for (int k0 = 0;; k0 += 2) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (k0 + p >= nks) goto done;
      step(p, k0 + p);
    }
  }
done:
  // the four quarters' sums in order, through LDS; lane (g, r): experts 4 g ..
  // + 3 of token r
  v4f(*const red)[8][64] = reinterpret_cast<v4f(*)[8][64]>(&sx[0][0]);  // [3][8][64]: 24 of sx's 32 KB
  float odds = 0.f;  // NaN once a sum is not finite (columns past E repeat the last expert's)
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    __syncthreads();
    if (wm == half && wk > 0) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) red[wk - 1][2 * t + u][lane] = acc[t][u];
    }
    __syncthreads();
    if (wm == half && wk == 0) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          v4f v = acc[t][u];
#pragma unroll
          for (int i = 0; i < 3; ++i) v += red[i][2 * t + u][lane];
#pragma unroll
          for (int q = 0; q < 4; ++q) odds = fmaf(v[q], 0.f, odds);
          const int64_t m = m0 + 16 * (2 * wm + u) + r;
          const int e = e0 + 16 * t + 4 * g;
          if (m < a.M) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (e + q < a.E) a.logits[m * a.E + e + q] = v[q];
          }
        }
    }
  }
  if (odds != 0.f) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      const int64_t m = m0 + 16 * (2 * wm + (i & 1)) + r;
      if (m < a.M) redo_odd<XT, WT>(a, m, e0 + 16 * (i >> 1) + 4 * g);
    }
  }
}

template <int XT, int WT, int TN, int TM, int W>
static hipError_t launch_tiles(const RouterArgs& a, hipStream_t stream, Ev ev) {
  const int64_t te = (a.E + 16 * TN - 1) / (16 * TN), tm = (a.M + 16 * TM - 1) / (16 * TM);
  return launch_k(router_tile_kernel<XT, WT, TN, TM, W>, dim3((unsigned)(te * tm)), dim3(64 * W), 0, stream, ev, a,
                  (int)te);
}

// Up to 16 tokens by 1, 4, 8 or 16 of them a workgroup. Above, 64 x 64 tiles where
// they occupy half of the CUs, else the larger of two that still give every CU a
// workgroup (H 6144, 256 experts, bf16: 2048 tokens 31 us by the first, 49 by the
// second; 1024 tokens 30 and 25; 256 tokens 28 us by the first and 13 by the third)
enum { kTokens1, kTokens4, kTokens8, kTokens16, kWide, kTiles2, kTiles1 };
static const char* const kNames[] = {"1 token", "4 tokens", "8 tokens", "16 tokens",
                                     "64 x 64 tile", "32 x 32, K split over the waves",
                                     "16 x 16, K split over the waves"};
static int64_t tiles_of(int64_t M, int64_t E, int t) { return ((E + t - 1) / t) * ((M + t - 1) / t); }
static int choose(int64_t M, int64_t E, int cus) {
  if (M <= 16) return M <= 1 ? kTokens1 : M <= 4 ? kTokens4 : M <= 8 ? kTokens8 : kTokens16;
  return tiles_of(M, E, 64) >= cus / 2 ? kWide : tiles_of(M, E, 32) >= cus ? kTiles2 : kTiles1;
}

template <int XT, int WT>
static hipError_t launch_types(const RouterArgs& a, int cus, hipStream_t stream, Ev ev) {
  const dim3 grid((unsigned)a.E), block(64 * (unsigned)std::min<int64_t>(kRouterWaves, (a.H + 511) / 512));
  switch (choose(a.M, a.E, cus)) {
    case kTokens1: return launch_k(router_kernel<XT, WT, 1>, grid, block, 0, stream, ev, a);
    case kTokens4: return launch_k(router_kernel<XT, WT, 4>, grid, block, 0, stream, ev, a);
    case kTokens8: return launch_k(router_kernel<XT, WT, 8>, grid, block, 0, stream, ev, a);
    case kTokens16: return launch_k(router_kernel<XT, WT, 16>, grid, block, 0, stream, ev, a);
    case kWide:
      return launch_k(router_wide_kernel<XT, WT>, dim3((unsigned)tiles_of(a.M, a.E, 64)), dim3(512), 0, stream, ev, a,
                      (int)((a.E + 63) / 64));
    case kTiles2: return launch_tiles<XT, WT, 2, 2, 8>(a, stream, ev);
    default: return launch_tiles<XT, WT, 1, 1, 16>(a, stream, ev);
  }
}

const char* router_kernel_name(int64_t M, int64_t E, int cus) { return kNames[choose(M, E, cus)]; }

hipError_t launch_router(const RouterArgs& a, int cus, hipStream_t stream, Ev ev) {
  if (a.x_type == MOE_BF16)
    return a.w_type == MOE_BF16 ? launch_types<MOE_BF16, MOE_BF16>(a, cus, stream, ev)
                                : launch_types<MOE_BF16, MOE_FP32>(a, cus, stream, ev);
  return a.w_type == MOE_BF16 ? launch_types<MOE_FP16, MOE_BF16>(a, cus, stream, ev)
                              : launch_types<MOE_FP16, MOE_FP32>(a, cus, stream, ev);
}

}  // namespace qmoe
