// The whole MoE layer of up to 16 tokens from their hidden states, activations
// kept in 16 bits:
//   logits = x router^T (router.hip); top-k, weights as in route_common.h;
//   h = SiLU(x Wg^T) (x Wu^T) per (token, slot), binary32;
//   out[t] = sum_j w[t][j] h[t][j] W2[e_j]^T, one rounding to bf16.
// h enters the down product scaled by its routing weight and split into two
// bf16 (the value and the remainder, 16 significant bits: its rounding error
// of 2^-17 stays far below the output's 2^-9).
//
// With at most 16 tokens the MFMA's 16 columns hold the whole batch, so
// nothing is sorted or gathered: an active expert's gate/up rows meet all
// tokens' x, and the columns of tokens that did not pick it are dropped; the
// down product of 16 output columns runs over every active expert, a token's
// column being zero where it did not pick the expert, which also combines.
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "mxfp4.h"
#include "ops.h"
#include "route_common.h"

namespace qmoe {

constexpr int kLayerWaves = 8;

// Which experts the batch picked, and which slot of a token an expert is.
struct ActiveList {
  int n;
  uint16_t expert[kLayerMaxEntries];       // active experts, ascending
  uint8_t slot[kLayerMaxEntries][kSmallM]; // [active][token]: the token's slot, 255: none
};

// From ids[t * k + j] in LDS (every thread of a 512-thread workgroup).
__device__ __forceinline__ void build_active(const uint16_t* ids, int M, int k, int E, uint16_t* index,
                                             ActiveList& list) {
  const int n = M * k;
  for (int e = threadIdx.x; e < E; e += blockDim.x) index[e] = 0;
  for (int i = threadIdx.x; i < kLayerMaxEntries * kSmallM / 4; i += blockDim.x)
    reinterpret_cast<uint32_t*>(list.slot)[i] = 0xFFFFFFFFu;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) index[ids[i]] = 1;
  __syncthreads();
  if (threadIdx.x < 64) {
    int base = 0;
    for (int c = 0; c < E; c += 64) {
      const int e = c + (int)threadIdx.x;
      const bool on = e < E && index[e] != 0;
      const unsigned long long hits = __ballot(on);
      if (on) {
        const int at = base + __popcll(hits & ((1ull << threadIdx.x) - 1));
        list.expert[at] = (uint16_t)e;
        index[e] = (uint16_t)at;
      }
      base += __popcll(hits);
    }
    if (threadIdx.x == 0) list.n = base;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) list.slot[index[ids[i]]][i / k] = (uint8_t)(i % k);
  __syncthreads();
}

// Chunk c (8 elements of a K-step of 128) of token m's x in a wave's LDS: the
// packed gate/up weights give lane group g K elements 32 g + 8 j .. of MFMA j,
// so chunk c = 4 g + j is operand j's; rows exchanged by c against bank
// conflicts (writes: one row's 16 chunks; reads: one group's 16 rows).
__device__ __forceinline__ int x13_slot(int c, int m) { return (c & 3) * 64 + 16 * (c >> 2) + (m ^ c); }

// Gate/up of every active expert. Work item: 8 columns of I of one active
// expert: one MFMA row tile of its 8 gate rows and its 8 up rows (half of a
// packed 16-row block each, in 128-byte runs). Wave w holds K-steps w S ..
// w S + S - 1 of x as MFMA operands in registers over all items of the
// workgroup; the items' weights stream through a ring of two items' registers
// (one where x takes more), each slot requested again as soon as its products
// are issued.
template <int S, int EC>
__global__ __launch_bounds__(64 * kLayerWaves) void layer_gate_up_kernel(
    const uint16_t* __restrict__ x, const float* __restrict__ logits, const uint8_t* __restrict__ w13p,
    const uint8_t* __restrict__ s13p, int* __restrict__ topk_ids, float* __restrict__ topk_w,
    uint16_t* __restrict__ gp, int M, int H, int E, int I, int k, float scaling) {
  __shared__ ActiveList list;
  __shared__ uint16_t index[kRouteMaxE];
  __shared__ uint16_t ids[kLayerMaxEntries];
  __shared__ float sel[kLayerMaxEntries], wts[kLayerMaxEntries];
  __shared__ float red[2][kLayerWaves][4 * 80];
  __shared__ uint4 xs[kLayerWaves][256];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int nks = H / 128, nkq = H / 512, nit = I / 8;

  uint4 xv[S][4];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ks = wave * S + s, m = 4 * i + g;
      xv[s][i] = m < M && ks < nks ? ld16(x + (size_t)m * H + 128 * ks + 8 * r) : make_uint4(0, 0, 0, 0);
    }

  for (int t = wave; t < M; t += kLayerWaves) {
    uint32_t key[EC], sel_e = 0;
    float sel_l = 0.f;
    load_keys<EC>(logits + (size_t)t * E, E, lane, key);
    topk_wave<EC>(key, k, lane, sel_e, sel_l);
    if (lane < k) {
      ids[t * k + lane] = (uint16_t)sel_e;
      sel[t * k + lane] = sel_l;
      if (blockIdx.x == 0) topk_ids[t * k + lane] = (int)sel_e;
    }
  }
  __syncthreads();
  build_active(ids, M, k, E, index, list);

  const int items = list.n * nit, step = gridDim.x;
  const int own = ((int)blockIdx.x < items) ? (items - (int)blockIdx.x + step - 1) / step : 0;
  // lane r < 8: gate row r of the item, else up row r - 8
  constexpr int D = S > 6 ? 1 : 2;
  uint4 q[D][S];
  uint32_t sc[D][S];
  auto load = [&](int d, int s, int i) {
    const int it = blockIdx.x + min(i, own - 1) * step, a = it / nit, c = it - a * nit;
    const uint32_t rb = (uint32_t)list.expert[a] * (I / 8) + (c >> 1) + (r >= 8 ? I / 16 : 0);
    const uint32_t row = 8 * (c & 1) + (r & 7);
    const int ks = min(wave * S + s, nks - 1);
    q[d][s] = ld16(w13p + ((size_t)rb * nks + ks) * 1024 + 256 * g + 16 * row);
    sc[d][s] = ld4(s13p + ((size_t)rb * nkq + (ks >> 2)) * 256 + 64 * g + 4 * row);
  };
  if (own > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int s = 0; s < S; ++s) load(d, s, d);
  }
  // the routing weights, while the first weights are on their way: sigmoid
  // scores (float64, one rounding), renormalized over the token's slots
  if ((int)threadIdx.x < M * k) wts[threadIdx.x] = (float)(1.0 / (1.0 + exp(-(double)sel[threadIdx.x])));
  barrier_lds();
  float weight = 0.f;
  if ((int)threadIdx.x < M * k) {
    const int t0 = threadIdx.x / k * k;
    float sum = 0.f;
    for (int j = 0; j < k; ++j) sum += wts[t0 + j];
    weight = __fdiv_rn(wts[threadIdx.x], sum + 1e-20f) * scaling;
  }
  barrier_lds();
  if ((int)threadIdx.x < M * k) {
    wts[threadIdx.x] = weight;
    if (blockIdx.x == 0) topk_w[threadIdx.x] = weight;
  }

  uint4 xf[S][4];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    uint4* mine = &xs[wave][0];
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[x13_slot(r, 4 * i + g)] = xv[s][i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // LDS keeps a wave's order
#pragma unroll
    for (int j = 0; j < 4; ++j) xf[s][j] = mine[x13_slot(4 * g + j, r)];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  barrier_lds();

  auto compute = [&](int d, int i, auto reload) {
    v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int ks = wave * S + s;
      const float f = scale_operand<0>(sc[d][s] >> (8 * (ks & 3)));
      const bool in = ks < nks;  // x is zero past the last step; so are the codes, whatever their scale
      const uint32_t c[4] = {in ? q[d][s].x : 0u, in ? q[d][s].y : 0u, in ? q[d][s].z : 0u, in ? q[d][s].w : 0u};
#pragma unroll
      for (int j = 0; j < 4; ++j) acc = mfma_bf16(fp4x8_bf16(c[j], f), __builtin_bit_cast(v8s, xf[s][j]), acc);
      if constexpr (reload) load(d, s, i + D);
    }
    // lane (g, r): rows 4 g .. 4 g + 3 of token r (rows 0-7 gate, 8-15 up); 80
    // floats a group keep the transposed reads below off each other's banks
    const int buf = i & 1;
    *reinterpret_cast<v4f*>(&red[buf][wave][80 * g + 4 * r]) = acc;
    barrier_lds();
    const int th = (int)threadIdx.x - 128 * (i & 3);  // two waves in turn
    if (th >= 0 && th < 128) {
      const int it = blockIdx.x + i * step, a = it / nit, c = it - a * nit;
      const int t = th >> 3, n = th & 7;
      const int slot = list.slot[a][t];
      if (slot != 255) {
        const int at = 80 * (n >> 2) + 4 * t + (n & 3);
        float G = 0.f, U = 0.f;
#pragma unroll
        for (int w = 0; w < kLayerWaves; ++w) {
          G += red[buf][w][at];
          U += red[buf][w][at + 160];
        }
        const int entry = t * k + slot;
        const float v = G / (1.0f + expf(-G)) * U * wts[entry];
        const uint16_t hi = bf16_bits(v);
        const float rest = v - bf16_value(hi);
        const size_t o = (size_t)entry * I + 8 * c + n;
        gp[o] = hi;
        gp[(size_t)M * k * I + o] = fabsf(rest) < INFINITY ? bf16_bits(rest) : (uint16_t)0;
      }
    }
  };
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  int i = 0;
  for (; i + D < own; i += D)
#pragma unroll
    for (int d = 0; d < D; ++d) compute(d, i + d, yes);
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (i + d < own) compute(d, i + d, no);
}

// Down and combine: cw (a multiple of 8, at most 16 R) columns of out a
// workgroup, every active expert. Wave w takes experts w, w + 8, ..., a
// K-step of 128 at a time: R row tiles' weights PW steps ahead, and the
// tokens' weighted h (two bf16 a value; loaded only by the lanes of tokens
// that picked the expert) two steps ahead.
template <int NB, int R>
__global__ __launch_bounds__(64 * kLayerWaves) void layer_down_kernel(
    const uint16_t* __restrict__ gp, const int* __restrict__ topk_ids, const uint8_t* __restrict__ w2,
    const uint8_t* __restrict__ s2, uint16_t* __restrict__ out, int M, int H, int E, int k, int cw) {
  __shared__ ActiveList list;
  __shared__ uint16_t index[kRouteMaxE];
  __shared__ uint16_t ids[kLayerMaxEntries];
  __shared__ v4f red[kLayerWaves][R][64];
  constexpr int I = 128 * NB;
  constexpr int PW = NB == 3 ? 6 : 8, PG = 2;
  static_assert(PW % NB == 0 && PW % PG == 0, "whole experts a round");
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  for (int i = threadIdx.x; i < M * k; i += blockDim.x) ids[i] = (uint16_t)topk_ids[i];
  __syncthreads();
  build_active(ids, M, k, E, index, list);
  const size_t plane = (size_t)M * k * I;
  const int c0 = blockIdx.x * cw, cols = min(cw, H - c0);
  const int experts = (list.n - wave + kLayerWaves - 1) / kLayerWaves;  // of this wave
  const int units = experts > 0 ? experts * NB : 0;                     // K-steps of all of them

  uint4 q[PW][R];
  uint32_t sc[PW][R];
  uint4 hi[PG][4], lo[PG][4];
  int row[R];  // rows past the workgroup's columns: the last one again (not stored)
#pragma unroll
  for (int t = 0; t < R; ++t) row[t] = c0 + min(16 * t + r, cols - 1);
  auto load_w = [&](int p, int u, int b) {
    const int a = wave + kLayerWaves * min(u / NB, experts - 1);
    const size_t base = (size_t)list.expert[a] * H;
#pragma unroll
    for (int t = 0; t < R; ++t) {
      q[p][t] = ld16(w2 + (base + row[t]) * (I / 2) + 64 * b + 16 * g);
      sc[p][t] = ld4(s2 + (base + row[t]) * (I / 32) + 4 * b);
    }
  };
  auto slot_of = [&](int u) -> int {
    const int a = wave + kLayerWaves * min(u / NB, experts - 1);
    return r < M ? list.slot[a][r] : 255;
  };
  auto load_g = [&](int p, int u, int b) {
    const int slot = slot_of(u);
    const uint16_t* h = gp + (size_t)(r * k + slot) * I + 128 * b + 32 * g;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[p][j] = make_uint4(0, 0, 0, 0);
      lo[p][j] = make_uint4(0, 0, 0, 0);
    }
    if (slot != 255) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        hi[p][j] = ld16(h + 8 * j);
        lo[p][j] = ld16(h + plane + 8 * j);
      }
    }
  };
  v4f acc[R], d[R];
#pragma unroll
  for (int t = 0; t < R; ++t) acc[t] = d[t] = v4f{0.f, 0.f, 0.f, 0.f};
  if (units > 0) {
#pragma unroll
    for (int p = 0; p < PW; ++p) load_w(p, p, p % NB);
#pragma unroll
    for (int p = 0; p < PG; ++p) load_g(p, p, p % NB);
  }
  for (int u0 = 0; u0 < units; u0 += PW) {
#pragma unroll
    for (int p = 0; p < PW; ++p) {
      const int u = u0 + p;
      if (u >= units) break;
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const float f = scale_operand<0>(sc[p][t] >> (8 * g));
        const uint32_t w[4] = {q[p][t].x, q[p][t].y, q[p][t].z, q[p][t].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const v8s wf = fp4x8_bf16(w[j], f);
          d[t] = mfma_bf16(wf, __builtin_bit_cast(v8s, lo[p % PG][j]), d[t]);
          d[t] = mfma_bf16(wf, __builtin_bit_cast(v8s, hi[p % PG][j]), d[t]);
        }
      }
      load_w(p, u + PW, p % NB);
      if (p % NB == NB - 1) {
        // a token that did not pick the expert takes nothing from it, also
        // where its weights are not finite
        const bool mine = slot_of(u) != 255;
#pragma unroll
        for (int t = 0; t < R; ++t) {
          if (mine) acc[t] += d[t];
          d[t] = v4f{0.f, 0.f, 0.f, 0.f};
        }
      }
      load_g(p % PG, u + PG, (p + PG) % NB);
    }
  }
#pragma unroll
  for (int t = 0; t < R; ++t) red[wave][t][lane] = acc[t];
  __syncthreads();
  if (wave < R && r < M) {
    const int n = 16 * wave + 4 * g;
    v4f v = red[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kLayerWaves; ++w) v += red[w][wave][lane];
    if (n < cols) {
      uint2 o;
      o.x = (uint32_t)bf16_bits(v[0]) | ((uint32_t)bf16_bits(v[1]) << 16);
      o.y = (uint32_t)bf16_bits(v[2]) | ((uint32_t)bf16_bits(v[3]) << 16);
      *reinterpret_cast<uint2*>(out + (size_t)r * H + c0 + n) = o;
    }
  }
}

template <int S>
static hipError_t launch_gate_up_s(const moe_plan* p, const LayerArgs& a, const float* logits, uint16_t* gp) {
  const int E = (int)p->s.E, I = (int)p->s.I, k = (int)p->s.top_k;
  const int64_t items = std::min<int64_t>(E, a.M * k) * (I / 8);
  const dim3 grid((unsigned)std::min<int64_t>(items, p->num_cus));
  auto go = [&](auto kern) {
    return launch_k(kern, grid, dim3(64 * kLayerWaves), 0, a.stream, Ev{}, (const uint16_t*)a.x, logits,
                    (const uint8_t*)a.w13, (const uint8_t*)a.s13, wsp<int>(p, p->L.topk_ids),
                    wsp<float>(p, p->L.topk_w), gp, (int)a.M, (int)p->s.H, E, I, k, p->s.routed_scaling);
  };
  return E <= 256 ? go(layer_gate_up_kernel<S, 4>) : go(layer_gate_up_kernel<S, 16>);
}

hipError_t launch_layer(const moe_plan* p, const moe_router* router, const LayerArgs& a) {
  float* logits = wsp<float>(p, p->X.layer_logits);
  uint16_t* gp = wsp<uint16_t>(p, p->X.layer_g);
  const RouterArgs ra{a.M, p->s.E, p->s.H, p->s.H, a.x, router->w, logits, router->x_type, router->w_type};
  hipError_t e = launch_router(ra, p->num_cus, a.stream);
  if (e != hipSuccess) return e;
  const int H = (int)p->s.H, nks = H / 128;
  e = nks <= 8    ? launch_gate_up_s<1>(p, a, logits, gp)
      : nks <= 16 ? launch_gate_up_s<2>(p, a, logits, gp)
      : nks <= 32 ? launch_gate_up_s<4>(p, a, logits, gp)
      : nks <= 48 ? launch_gate_up_s<6>(p, a, logits, gp)
                  : launch_gate_up_s<8>(p, a, logits, gp);
  if (e != hipSuccess) return e;
  // one workgroup a CU, each the same number of columns: a multiple of 8
  // (H 6144 on 256 CUs: 24), in one or two 16-row tiles
  const int cw = std::min(32, (H / 8 + p->num_cus - 1) / p->num_cus * 8);
  const dim3 grid((unsigned)((H + cw - 1) / cw));
  auto go = [&](auto kern) {
    return launch_k(kern, grid, dim3(64 * kLayerWaves), 0, a.stream, Ev{}, (const uint16_t*)gp,
                    wsp<int>(p, p->L.topk_ids), (const uint8_t*)a.w2, (const uint8_t*)a.s2, (uint16_t*)a.out, (int)a.M,
                    H, (int)p->s.E, (int)p->s.top_k, cw);
  };
  switch (2 * (p->s.I / 128) + (cw > 16 ? 1 : 0)) {
    case 2: return go(layer_down_kernel<1, 1>);
    case 3: return go(layer_down_kernel<1, 2>);
    case 4: return go(layer_down_kernel<2, 1>);
    case 5: return go(layer_down_kernel<2, 2>);
    case 6: return go(layer_down_kernel<3, 1>);
    case 7: return go(layer_down_kernel<3, 2>);
    case 8: return go(layer_down_kernel<4, 1>);
    default: return go(layer_down_kernel<4, 2>);
  }
}

}  // namespace qmoe
