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

// Gate/up of every active expert. Work item: 16 columns of I of one active
// expert, its gate rows and its up rows. Wave w holds K-steps w S .. w S + S-1
// of x as MFMA operands in registers over all items of the workgroup.
template <int S, int EC>
__global__ __launch_bounds__(64 * kLayerWaves) void layer_gate_up_kernel(
    const uint16_t* __restrict__ x, const float* __restrict__ logits, const uint8_t* __restrict__ w13p,
    const uint8_t* __restrict__ s13p, int* __restrict__ topk_ids, float* __restrict__ topk_w,
    uint16_t* __restrict__ gp, int M, int H, int E, int I, int k, float scaling) {
  __shared__ ActiveList list;
  __shared__ uint16_t index[kRouteMaxE];
  __shared__ uint16_t ids[kLayerMaxEntries];
  __shared__ float wts[kLayerMaxEntries];
  __shared__ float red[2][2][kLayerWaves][4 * 80];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int nks = H / 128, nkq = H / 512, nit = I / 16;

  uint4 xf[S][4];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int ks = wave * S + s;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      xf[s][j] = r < M && ks < nks ? ld16(x + (size_t)r * H + 128 * ks + 32 * g + 8 * j) : make_uint4(0, 0, 0, 0);
  }

  for (int t = wave; t < M; t += kLayerWaves) {
    uint32_t sel_e = 0;
    float w = 0.f;
    route_token<EC>(logits + (size_t)t * E, E, k, scaling, 0, lane, sel_e, w);
    if (lane < k) {
      ids[t * k + lane] = (uint16_t)sel_e;
      wts[t * k + lane] = w;
      if (blockIdx.x == 0) {
        topk_ids[t * k + lane] = (int)sel_e;
        topk_w[t * k + lane] = w;
      }
    }
  }
  __syncthreads();
  build_active(ids, M, k, E, index, list);

  const int items = list.n * nit;
  int buf = 0;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int a = it / nit, c = it % nit;
    const size_t rbg = (size_t)list.expert[a] * (2 * nit) + c, rbu = rbg + nit;
    uint4 qg[S], qu[S];
    uint32_t sg[S], su[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int ks = min(wave * S + s, nks - 1);
      qg[s] = ld16(w13p + (rbg * nks + ks) * 1024 + 16 * lane);
      qu[s] = ld16(w13p + (rbu * nks + ks) * 1024 + 16 * lane);
      sg[s] = ld4(s13p + (rbg * nkq + (ks >> 2)) * 256 + 4 * lane);
      su[s] = ld4(s13p + (rbu * nkq + (ks >> 2)) * 256 + 4 * lane);
    }
    v4f ag = {0.f, 0.f, 0.f, 0.f}, au = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int ks = wave * S + s;
      if (ks >= nks) break;
      const float fg = scale_operand<0>(sg[s] >> (8 * (ks & 3))), fu = scale_operand<0>(su[s] >> (8 * (ks & 3)));
      const uint32_t dg[4] = {qg[s].x, qg[s].y, qg[s].z, qg[s].w}, du[4] = {qu[s].x, qu[s].y, qu[s].z, qu[s].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v8s xb = __builtin_bit_cast(v8s, xf[s][j]);
        ag = mfma_bf16(fp4x8_bf16(dg[j], fg), xb, ag);
        au = mfma_bf16(fp4x8_bf16(du[j], fu), xb, au);
      }
    }
    // lane (g, r): rows (columns of I) 4 g .. 4 g + 3 of token r; 80 floats a
    // group keep the transposed reads below off each other's banks
    *reinterpret_cast<v4f*>(&red[buf][0][wave][80 * g + 4 * r]) = ag;
    *reinterpret_cast<v4f*>(&red[buf][1][wave][80 * g + 4 * r]) = au;
    barrier_lds();
    if (threadIdx.x < 256) {
      const int t = threadIdx.x >> 4, n = threadIdx.x & 15;
      const int slot = list.slot[a][t];
      if (slot != 255) {
        const int at = 80 * (n >> 2) + 4 * t + (n & 3);
        float G = 0.f, U = 0.f;
#pragma unroll
        for (int w = 0; w < kLayerWaves; ++w) {
          G += red[buf][0][w][at];
          U += red[buf][1][w][at];
        }
        const int entry = t * k + slot;
        const float v = G / (1.0f + expf(-G)) * U * wts[entry];
        const uint16_t hi = bf16_bits(v);
        const float rest = v - bf16_value(hi);
        const size_t o = (size_t)entry * I + 16 * c + n;
        gp[o] = hi;
        gp[(size_t)M * k * I + o] = fabsf(rest) < INFINITY ? bf16_bits(rest) : (uint16_t)0;
      }
    }
    buf ^= 1;
  }
}

// Down and combine: 16 columns of out, every active expert; the waves take
// the experts in turn.
template <int NB>
__global__ __launch_bounds__(64 * kLayerWaves) void layer_down_kernel(
    const uint16_t* __restrict__ gp, const int* __restrict__ topk_ids, const uint8_t* __restrict__ w2,
    const uint8_t* __restrict__ s2, uint16_t* __restrict__ out, int M, int H, int E, int k) {
  __shared__ ActiveList list;
  __shared__ uint16_t index[kRouteMaxE];
  __shared__ uint16_t ids[kLayerMaxEntries];
  __shared__ v4f red[2][kLayerWaves][64];
  constexpr int I = 128 * NB;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  for (int i = threadIdx.x; i < M * k; i += blockDim.x) ids[i] = (uint16_t)topk_ids[i];
  __syncthreads();
  build_active(ids, M, k, E, index, list);
  const size_t plane = (size_t)M * k * I;
  int buf = 0;
  for (int tile = blockIdx.x; tile < H / 16; tile += gridDim.x) {
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    for (int a = wave; a < list.n; a += kLayerWaves) {
      const size_t row = (size_t)list.expert[a] * H + 16 * tile + r;
      const int slot = r < M ? list.slot[a][r] : 255;
      uint4 q[NB];
      uint32_t sc[NB];
      uint4 hi[NB][4], lo[NB][4];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        q[b] = ld16(w2 + row * (I / 2) + 64 * b + 16 * g);
        sc[b] = ld4(s2 + row * (I / 32) + 4 * b);
      }
      const uint16_t* p = gp + (size_t)(r * k + (slot == 255 ? 0 : slot)) * I + 32 * g;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          hi[b][j] = slot != 255 ? ld16(p + 128 * b + 8 * j) : make_uint4(0, 0, 0, 0);
          lo[b][j] = slot != 255 ? ld16(p + plane + 128 * b + 8 * j) : make_uint4(0, 0, 0, 0);
        }
      v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float f = scale_operand<0>(sc[b] >> (8 * g));
        const uint32_t w[4] = {q[b].x, q[b].y, q[b].z, q[b].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const v8s wf = fp4x8_bf16(w[j], f);
          d = mfma_bf16(wf, __builtin_bit_cast(v8s, lo[b][j]), d);
          d = mfma_bf16(wf, __builtin_bit_cast(v8s, hi[b][j]), d);
        }
      }
      // a token that did not pick the expert takes nothing from it, also
      // where its weights are not finite
      if (slot != 255) acc += d;
    }
    red[buf][wave][lane] = acc;
    barrier_lds();
    if (wave == buf && r < M) {
      v4f v = red[buf][0][lane];
#pragma unroll
      for (int w = 1; w < kLayerWaves; ++w) v += red[buf][w][lane];
      uint2 o;
      o.x = (uint32_t)bf16_bits(v[0]) | ((uint32_t)bf16_bits(v[1]) << 16);
      o.y = (uint32_t)bf16_bits(v[2]) | ((uint32_t)bf16_bits(v[3]) << 16);
      *reinterpret_cast<uint2*>(out + (size_t)r * H + 16 * tile + 4 * g) = o;
    }
    buf ^= 1;
  }
}

template <int S>
static hipError_t launch_gate_up_s(const moe_plan* p, const LayerArgs& a, const float* logits, uint16_t* gp) {
  const int E = (int)p->s.E, I = (int)p->s.I, k = (int)p->s.top_k;
  const int64_t items = std::min<int64_t>(E, a.M * k) * (I / 16);
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
  const dim3 grid((unsigned)std::min(H / 16, 2 * p->num_cus));
  auto go = [&](auto kern) {
    return launch_k(kern, grid, dim3(64 * kLayerWaves), 0, a.stream, Ev{}, (const uint16_t*)gp,
                    wsp<int>(p, p->L.topk_ids), (const uint8_t*)a.w2, (const uint8_t*)a.s2, (uint16_t*)a.out, (int)a.M,
                    H, (int)p->s.E, (int)p->s.top_k);
  };
  switch (p->s.I / 128) {
    case 1: return go(layer_down_kernel<1>);
    case 2: return go(layer_down_kernel<2>);
    case 3: return go(layer_down_kernel<3>);
    default: return go(layer_down_kernel<4>);
  }
}

}  // namespace qmoe
