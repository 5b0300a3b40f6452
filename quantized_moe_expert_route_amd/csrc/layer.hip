// The whole MoE layer of up to 16 tokens from their hidden states, activations
// unquantized:
//   logits = x router^T (router.hip); top-k, weights as in route_common.h;
//   h = SiLU(x Wg^T) (x Wu^T) per (token, slot), binary32;
//   out[t] = sum_j w[t][j] h[t][j] W2[e_j]^T, one rounding to bf16.
// h enters the down product scaled by its routing weight, in binary32, as the
// three bf16 whose sum it is (8 significant bits each).
//
// With at most 16 tokens the MFMA's 16 columns hold the whole batch, so
// nothing is sorted or gathered: an active expert's gate/up rows meet all
// tokens' x, and the columns of tokens that did not pick it are dropped; the
// down product of some output columns runs over every active expert with the
// tokens that picked it, which also combines.
#include <stddef.h>

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
  int pad[3];
  uint16_t expert[kLayerMaxEntries];        // active experts, ascending
  uint8_t slot[kLayerMaxEntries][kSmallM];  // [active][token]: the token's slot, 255: none
};

// The same for the down launch: which tokens picked an expert.
struct PickList {
  int n;
  int pad[3];
  uint16_t expert[kLayerMaxEntries];
  uint8_t count[kLayerMaxEntries];          // tokens that picked it
  uint8_t pick[kLayerMaxEntries][kSmallM];  // they, ascending: 16 token + slot
};
static_assert(sizeof(PickList) == kLayerListBytes && sizeof(PickList) % 16 == 0, "copied in 16-byte pieces");
static_assert(offsetof(ActiveList, slot) == offsetof(PickList, count), "the same head");

// Top-k of T tokens' keys by one wave (of two the second may be all zero:
// unused), their rounds side by side so that one's lane exchanges hide the
// other's. A lane first sorts its own keys (EC <= 4; above, it looks for its
// largest every round); a round takes the largest of the lanes' first keys and
// drops it; of equal ones the lowest expert id 64 c + lane. Lane j < k gets
// slot j's expert and logit. (Looking through all keys every round took 2.6
// us for 8 of 256.)
template <int EC, int T>
__device__ __forceinline__ void topk_tokens(uint32_t (&key)[T][EC], bool second, int k, int lane,
                                            uint32_t (&sel_e)[T], float (&sel_l)[T]) {
  constexpr bool kSorted = EC <= 4;
  uint32_t id[T][EC];
#pragma unroll
  for (int t = 0; t < T; ++t) {
#pragma unroll
    for (int c = 0; c < EC; ++c) id[t][c] = 64 * c + lane;
    if constexpr (kSorted) {  // stable: equal keys keep the lower id first
#pragma unroll
      for (int pass = 0; pass < EC - 1; ++pass)
#pragma unroll
        for (int c = 0; c + 1 < EC - pass; ++c) {
          const bool swap = key[t][c + 1] > key[t][c];
          const uint32_t k0 = key[t][c], k1 = key[t][c + 1], i0 = id[t][c], i1 = id[t][c + 1];
          key[t][c] = swap ? k1 : k0;
          key[t][c + 1] = swap ? k0 : k1;
          id[t][c] = swap ? i1 : i0;
          id[t][c + 1] = swap ? i0 : i1;
        }
    }
  }
  for (int j = 0; j < k; ++j) {
    uint32_t top[T], first[T], win[T];
    unsigned long long hits[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      uint32_t m = key[t][0];
      first[t] = id[t][0];
      if constexpr (!kSorted) {
#pragma unroll
        for (int c = 1; c < EC; ++c) {
          first[t] = key[t][c] > m ? id[t][c] : first[t];
          m = max(m, key[t][c]);
        }
      }
      top[t] = wave_max_u32(m);
      hits[t] = __ballot(m == top[t]);
      win[t] = __builtin_amdgcn_readlane(first[t], __builtin_ctzll(hits[t]));
    }
    bool equal = hits[0] & (hits[0] - 1);
    if constexpr (T == 2) equal = equal || (second && (hits[1] & (hits[1] - 1)));
    if (equal) {
#pragma unroll
      for (int t = 0; t < T; ++t) win[t] = wave_min_u32((hits[t] >> lane) & 1 ? first[t] : 0xFFFFFFFFu);
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if constexpr (kSorted) {
        const bool mine = first[t] == win[t];
#pragma unroll
        for (int c = 0; c < EC; ++c) {
          key[t][c] = mine ? (c + 1 < EC ? key[t][c + 1 < EC ? c + 1 : c] : 0u) : key[t][c];
          if (c + 1 < EC) id[t][c] = mine ? id[t][c + 1] : id[t][c];
        }
      } else {
#pragma unroll
        for (int c = 0; c < EC; ++c) key[t][c] = win[t] == id[t][c] ? 0u : key[t][c];
      }
      if (lane == j) {
        sel_e[t] = win[t];
        sel_l[t] = key_to_float(top[t]);
      }
    }
  }
}

// Chunk c (8 elements of a K-step of 128) of token m's x in a wave's LDS: the
// packed gate/up weights give lane group g K elements 32 g + 8 j .. of MFMA j,
// so chunk c = 4 g + j is operand j's; rows exchanged by c against bank
// conflicts (writes: one row's 16 chunks; reads: one group's 16 rows).
__device__ __forceinline__ int x13_slot(int c, int m) { return (c & 3) * 64 + 16 * (c >> 2) + (m ^ c); }

// Weighted h of the batch, as the down launch's lanes read it: per entry
// t * k + j and K-step of 128, operand j (K 32 g + 8 j .. + 7 of lane group g)
// is 192 bytes: the four groups' first bf16, then their second and third.
constexpr int kHParts = 3;
constexpr int kHStep = 128 * kHParts;
__device__ __forceinline__ size_t h_at(int entry, int nb, int col, int part) {
  const int e = col & 127;
  return ((size_t)entry * nb + (col >> 7)) * kHStep + (((e >> 3) & 3) * (4 * kHParts) + part * 4 + (e >> 5)) * 8 + (e & 7);
}

constexpr int kHoldItems = 16;  // finished items a gate/up workgroup holds before it stores them

// Gate/up of every active expert. Work item: 8 columns of I of one active
// expert: one MFMA row tile of its 8 gate rows and its 8 up rows (half of a
// packed 16-row block each, in 128-byte runs; the other half goes to a
// workgroup of the same XCD). Wave w holds K-steps w S .. w S + S - 1 of x as
// MFMA operands in registers over all items of the workgroup; the items'
// weights stream through a ring of two items' registers (one where x takes
// more), each slot requested again as soon as its products are issued.
// Results wait in LDS and are stored 16 items at a time: the compiler drains
// all loads before it lets a store's counter mix with them. H 6144, I 256, 8 of
// 256 experts: 4 tokens 16 us, of which 4.6 pass before weights move (logits,
// top-k, list), 16 tokens 31 us (6.7); then 4.4 TB/s of them (51 and 108 MB), a
// third of the time with the vector ALUs at work and a twelfth with the MFMAs.
//
// T tokens a wave are routed, x comes operand-shaped up to 4 tokens (few
// lines a load), else in whole row pieces turned round in LDS.
template <int S, int EC, int T>
__global__ __launch_bounds__(64 * kLayerWaves) void layer_gate_up_kernel(
    const uint16_t* __restrict__ x, const float* __restrict__ logits, const uint8_t* __restrict__ w13p,
    const uint8_t* __restrict__ s13p, int* __restrict__ topk_ids, float* __restrict__ topk_w,
    uint16_t* __restrict__ gp, PickList* __restrict__ batch, int M, int H, int E, int I, int k, float scaling) {
  __shared__ __align__(16) ActiveList list;
  __shared__ __align__(16) uint32_t mask[kRouteMaxE / 32];  // picked experts
  __shared__ uint16_t ids[kLayerMaxEntries];
  __shared__ float wts[kLayerMaxEntries];
  __shared__ float red[2][kLayerWaves][4 * 80];
  __shared__ uint4 xs[kLayerWaves][256];
  __shared__ float hold[kHoldItems * 128];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int nks = H / 128, nkq = H / 512, nit = I / 8;

  // the wave's tokens' logits first (loads return in order), then x
  static_assert(kSmallM == 2 * kLayerWaves, "at most two tokens a wave");
  uint32_t key[T][EC];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int token = wave + kLayerWaves * t;
    load_keys<EC>(logits + (size_t)min(token, M - 1) * E, E, lane, key[t]);
    if (token >= M) {
#pragma unroll
      for (int c = 0; c < EC; ++c) key[t][c] = 0;
    }
  }
  const bool few = M <= 4;
  uint4 xv[S][4];
  int now = 1;
  asm volatile("" : "+s"(now));  // (a branch the compiler must keep, or it asks for x only where it is used)
  if (now) {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // rows past M and steps past the last: the last ones again (no branch:
        // the compiler counts the loads under way). Columns of tokens past M
        // are dropped, steps past the last become zero below.
        const int ks = min(wave * S + s, nks - 1), m = min(few ? r : 4 * i + g, M - 1), c = few ? 4 * g + i : r;
        xv[s][i] = ld16(x + (size_t)m * H + 128 * ks + 8 * c);
      }
  } else {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[s][i] = make_uint4(0, 0, 0, 0);
  }
  if (threadIdx.x < kRouteMaxE / 32) mask[threadIdx.x] = 0;
  for (int i = threadIdx.x; i < kLayerMaxEntries; i += 64 * kLayerWaves)
    reinterpret_cast<uint4*>(list.slot)[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
  barrier_lds();
  uint32_t sel_e[T];
  float sel_l[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    sel_e[t] = 0;
    sel_l[t] = 0.f;
  }
  if (wave < M) {
    topk_tokens<EC, T>(key, wave + kLayerWaves < M, k, lane, sel_e, sel_l);
#pragma unroll
    for (int t = 0; t < T; ++t)
      if (lane < k && wave + kLayerWaves * t < M) {
        ids[(wave + kLayerWaves * t) * k + lane] = (uint16_t)sel_e[t];
        atomicOr(&mask[sel_e[t] >> 5], 1u << (sel_e[t] & 31));
      }
  }
  barrier_lds();
  // an expert's place in the list: the picked ones below it
  auto place_in = [](const uint32_t(&words)[2 * EC], int e) {
    int at = 0;
#pragma unroll
    for (int w = 0; w < 2 * EC; ++w) {
      const uint32_t below = w < (e >> 5) ? ~0u : w == (e >> 5) ? (1u << (e & 31)) - 1 : 0u;
      at += __popc(words[w] & below);
    }
    return at;
  };
  {
    uint32_t words[2 * EC];
#pragma unroll
    for (int w = 0; w < 2 * EC; ++w) words[w] = mask[w];
    auto place = [&](int e) { return place_in(words, e); };
    for (int e = threadIdx.x; e < E; e += 64 * kLayerWaves)
      if ((mask[e >> 5] >> (e & 31)) & 1) list.expert[place(e)] = (uint16_t)e;
    if ((int)threadIdx.x < M * k) list.slot[place(ids[threadIdx.x])][threadIdx.x / k] = (uint8_t)(threadIdx.x % k);
    if (threadIdx.x == 64 * kLayerWaves - 1) {
      int all = 0;
#pragma unroll
      for (int w = 0; w < 2 * EC; ++w) all += __popc(words[w]);
      list.n = all;
    }
  }
  barrier_lds();

  // workgroups 16 v + x and 16 v + x + 8 (one XCD) take the halves 2 p, 2 p + 1
  const int items = list.n * nit, step = gridDim.x, id = blockIdx.x;
  const int first = step % 16 == 0 ? (id & ~15) + 2 * (id & 7) + ((id >> 3) & 1) : id;
  const int own = first < items ? (items - first + step - 1) / step : 0;
  // lane r < 8: gate row r of the item, else up row r - 8
  constexpr int D = S > 6 ? 1 : 2;
  uint4 q[D][S];
  uint32_t sc[D][S];
  auto item_row = [&](int i) -> uint32_t {  // the item's (gate or up) row of this lane, in 16-row blocks' order
    const int it = own > 0 ? first + min(i, own - 1) * step : 0, a = it / nit, c = it - a * nit;
    return (uint32_t)list.expert[a] * (2 * I) + 8 * c + (r >= 8 ? I : 0) + (r & 7);
  };
  auto load = [&](int d, int s, uint32_t row) {
    const size_t rb = row >> 4;
    // a step past the last: one address a block, hardly any traffic
    const int ks = min(wave * S + s, nks - 1), used = wave * S + s < nks ? ~0 : 0;
    q[d][s] = ld16(w13p + (rb * nks + ks) * 1024 + ((256 * g + 16 * (row & 15)) & used));
    sc[d][s] = ld4(s13p + (rb * nkq + (ks >> 2)) * 256 + ((64 * g + 4 * (row & 15)) & used));
  };
  // (a workgroup without an item asks for the first one's: no branch, so that x
  // is not waited for together with these)
#pragma unroll
  for (int d = 0; d < D; ++d) {
    const uint32_t row = item_row(d);
#pragma unroll
    for (int s = 0; s < S; ++s) load(d, s, row);
  }
  // The routing weights, while the first weights are on their way: sigmoid
  // scores (float64, one rounding), renormalized over the token's slots in
  // slot order. They are first read behind the first item's barrier.
  if (wave < M) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const float w = route_weight(sel_l[t], k, lane, scaling);
      if (lane < k && wave + kLayerWaves * t < M) wts[(wave + kLayerWaves * t) * k + lane] = w;
    }
  }

  uint4 xf[S][4];
  if (few) {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) xf[s][j] = xv[s][j];
  } else {
    uint4* mine = &xs[wave][0];
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) mine[x13_slot(r, 4 * i + g)] = xv[s][i];
      wave_lds_order();
#pragma unroll
      for (int j = 0; j < 4; ++j) xf[s][j] = mine[x13_slot(4 * g + j, r)];
      wave_lds_order();
    }
  }
  // x is waited for here, once: left to its first use, inside the loop, the
  // wait would be for all loads, every round
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (wave * S + s >= nks) xf[s][j] = make_uint4(0, 0, 0, 0);
      asm volatile("" : "+v"(xf[s][j].x), "+v"(xf[s][j].y), "+v"(xf[s][j].z), "+v"(xf[s][j].w));
    }

  auto flush = [&](int i0, int i1) {  // store items i0 .. i1 - 1
    for (int v = threadIdx.x; v < (i1 - i0) * 128; v += 64 * kLayerWaves) {
      const int it = first + (i0 + (v >> 7)) * step, a = it / nit, c = it - a * nit;
      const int t = (v & 127) >> 3, n = v & 7, slot = list.slot[a][t];
      if (slot == 255) continue;
      // the upper 8 significant bits of what is left, three times: exact (down
      // to bf16's smallest number); an infinity or NaN stays in the first
      float rest = hold[v];
#pragma unroll
      for (int p = 0; p < kHParts; ++p) {
        const uint32_t u = __float_as_uint(rest) & 0xFFFF0000u;
        gp[h_at(t * k + slot, I / 128, 8 * c + n, p)] = (uint16_t)(u >> 16);
        rest = (u & 0x7F800000u) == 0x7F800000u ? 0.f : rest - __uint_as_float(u);
      }
    }
  };
  auto compute = [&](int d, int i, auto reload) __attribute__((always_inline)) {
    const uint32_t next = reload ? item_row(i + D) : 0;
    v4f acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int ks = wave * S + s;
      const float f = scale_operand<0>(sc[d][s] >> (8 * (ks & 3)));
      const bool in = ks < nks;  // x is zero past the last step; so are the codes, whatever their scale
      const uint32_t c[4] = {in ? q[d][s].x : 0u, in ? q[d][s].y : 0u, in ? q[d][s].z : 0u, in ? q[d][s].w : 0u};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[j & 1] = mfma_bf16(fp4x8_bf16(c[j], f), __builtin_bit_cast(v8s, xf[s][j]), acc[j & 1]);
      if constexpr (reload) load(d, s, next);
    }
    // lane (g, r): rows 4 g .. 4 g + 3 of token r (rows 0-7 gate, 8-15 up); 80
    // floats a group keep the transposed reads below off each other's banks
    const int buf = i & 1;
    *reinterpret_cast<v4f*>(&red[buf][wave][80 * g + 4 * r]) = acc[0] + acc[1];
    barrier_lds();
    const int th = (int)threadIdx.x - 128 * (i & 3);  // two waves in turn
    if (th >= 0 && th < 128) {
      const int it = first + i * step, a = it / nit;
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
        hold[(i % kHoldItems) * 128 + th] = G / (1.0f + expf(-G)) * U * wts[t * k + slot];
      }
    }
    if ((i + 1) % kHoldItems == 0) {
      barrier_lds();
      flush(i + 1 - kHoldItems, i + 1);
      barrier_lds();
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
  barrier_lds();
  flush(own / kHoldItems * kHoldItems, own);
  if (blockIdx.x == 0) {  // for the down launch and the caller
    if ((int)threadIdx.x < M * k) {
      topk_ids[threadIdx.x] = ids[threadIdx.x];
      topk_w[threadIdx.x] = wts[threadIdx.x];
      // this token's rank among those that picked the expert
      uint32_t words[2 * EC];
#pragma unroll
      for (int w = 0; w < 2 * EC; ++w) words[w] = mask[w];
      const int at = place_in(words, ids[threadIdx.x]), t = threadIdx.x / k;
      uint32_t tokens = 0;
#pragma unroll
      for (int m = 0; m < kSmallM; ++m) tokens |= (uint32_t)(list.slot[at][m] != 255) << m;
      const int rank = __popc(tokens & ((1u << t) - 1));
      batch->pick[at][rank] = (uint8_t)(16 * t + list.slot[at][t]);
      if ((tokens >> t) == 1) batch->count[at] = (uint8_t)(rank + 1);
    }
    for (int i = threadIdx.x; i < (int)offsetof(PickList, count) / 16; i += 64 * kLayerWaves)
      reinterpret_cast<uint4*>(batch)[i] = reinterpret_cast<const uint4*>(&list)[i];
  }
}

// Down and combine: 8 C8 columns of out a workgroup, over every active expert.
// Wave w takes experts w, w + 8, ...: an expert's rows of these columns are one
// run of 512 C8 NB bytes, read PE experts ahead in whole lines and turned
// into MFMA operands through LDS of the wave's own (operand-shaped loads, 64
// bytes of 16 rows, cost the memory pipeline four times as much). The tokens'
// weighted h is loaded UH K-steps ahead by the lanes of tokens that picked the
// expert: loads return in order, so h asked for when it is needed would wait
// for all weights under way (and copied to LDS beforehand, it cost 3 to 6 us
// with nothing else moving).
// An expert is picked by few of the tokens, so the 16 MFMA columns hold all three
// parts of h at once: column c < 15 is part c / 5 of the (c % 5)th token that
// picked the expert; more than five take further passes over the same weights.
// Which tokens a column holds changes from expert to expert, so the sums stay in
// LDS of the wave's own, per part and token, and the parts are added at the end.
// Bound by loads' latency, not by a rate: few experts a wave, and the waves' ends
// spread (their experts are fixed, so that the sums' order is). H 6144, I 256, 8
// of 256 experts: 4 tokens 11.2 us (26 MB of weights, 2.3 TB/s; with h 41 MB from
// the L2s), 16 tokens 20.3 (54 MB, 2.6 TB/s; 108 MB); where h was cut to two bf16
// and the sums stayed in registers 10.6 and 18.5.
template <int NB>
struct DownRows {  // a row's 4 NB chunks of 16 bytes in LDS, exchanged against bank conflicts
  static constexpr int kStride = NB == 3 ? 16 : 4 * NB;
  __device__ static __forceinline__ int at(int row, int chunk) {
    const int x = NB == 1 ? (row >> 2) & 3 : NB == 2 ? (row >> 1) & 7 : row & 15;
    return row * kStride + (chunk ^ x);
  }
};

template <int NB, int C8>
__global__ __launch_bounds__(64 * kLayerWaves) void layer_down_kernel(
    const uint16_t* __restrict__ gp, const PickList* __restrict__ batch, const uint8_t* __restrict__ w2,
    const uint8_t* __restrict__ s2, uint16_t* __restrict__ out, int M, int H, int k) {
  typedef DownRows<NB> Rows;
  constexpr int I = 128 * NB, R = (C8 + 1) / 2;      // R MFMA row tiles
  constexpr int kRows = 8 * C8 * Rows::kStride;      // chunks of a wave's rows in LDS
  constexpr int NL = (8 * C8 * 4 * NB + 63) / 64;    // loads of an expert's rows
  // (H 4096, I 256, 16 tokens: 21.1 us with 4 experts ahead, 22.0 with 6, no registers for 8)
  constexpr int PE = NL >= 5 ? 2 : NL >= 3 || NB == 4 || NL * NB == 4 ? 4 : 8;
  constexpr int UH = NB == 3 ? 3 : 4;
  static_assert(PE * NB % UH == 0, "whole rounds of h");
  __shared__ __align__(16) PickList list;
  __shared__ uint4 area[kLayerWaves * kRows];
  // [.][.][token][4 t + g]: columns 16 t + 4 g .. + 3 (one more, or all tokens met the same banks)
  __shared__ v4f sums[kLayerWaves][kHParts][kSmallM][4 * R + 1];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  for (int i = threadIdx.x; i < (int)sizeof(PickList) / 16; i += 64 * kLayerWaves)
    reinterpret_cast<uint4*>(&list)[i] = reinterpret_cast<const uint4*>(batch)[i];
  __syncthreads();
  const int c0 = blockIdx.x * 8 * C8, cols = min(8 * C8, H - c0);
  const int experts = (list.n - wave + kLayerWaves - 1) / kLayerWaves;  // of this wave
  uint4* mine = area + wave * kRows;
  // The wave's expert i. Past its last, that one again (with none, the list's
  // first), by one address for all lanes: asked for without a branch, but
  // hardly any traffic.
  auto at = [&](int i) __attribute__((always_inline)) {
    return experts > 0 ? wave + kLayerWaves * min(i, experts - 1) : 0;
  };

  typedef uint32_t scales __attribute__((ext_vector_type(NB == 1 ? 2 : NB), aligned(4)));
  uint4 q[PE][NL];
  uint32_t sc[PE][R][NB];
  auto load = [&](int p, int i) __attribute__((always_inline)) {
    const size_t row0 = (size_t)list.expert[at(i)] * H + c0;
    const int used = i < experts ? ~0 : 0;
#pragma unroll
    for (int l = 0; l < NL; ++l)  // columns past H: the last chunk again
      q[p][l] = ld16(w2 + row0 * (I / 2) + 16 * (min(64 * l + lane, cols * 4 * NB - 1) & used));
#pragma unroll
    for (int t = 0; t < R; ++t) {
      const uint8_t* src = s2 + (row0 + (min(16 * t + r, cols - 1) & used)) * (I / 32);
      if constexpr (NB == 1) {
        sc[p][t][0] = ld4(src);
      } else {
        const scales v = *reinterpret_cast<const scales*>(src);
#pragma unroll
        for (int b = 0; b < NB; ++b) sc[p][t][b] = v[b];
      }
    }
  };
  // Token and slot (16 token + slot) of this lane's column in a pass over the
  // wave's expert i, -1: none; n: the tokens that picked it, none past the last
  // expert. Both bytes are read whatever comes of them: a branch would wait for
  // the one and then for the other. (Column 15 is nobody's and reads what column
  // 10 does.)
  const int c5 = r % 5, part = min(r / 5, kHParts - 1);
  auto column = [&](int i, int pass, int& n) __attribute__((always_inline)) -> int {
    const int q = 5 * pass + c5, who = list.pick[at(i)][min(q, kSmallM - 1)];
    n = list.count[at(i)] & (i < experts ? 255 : 0);
    return who | (q < n ? 0 : -1);
  };
  auto load_h = [&](uint4(&hv)[4], int who, int b) __attribute__((always_inline)) {
    // (no branch round the loads: the compiler counts those under way. Without a
    // token the first entry's, for a column that is not used)
    const int w = max(who, 0), entry = (w >> 4) * k + (w & 15);
    const uint16_t* src = gp + (size_t)(entry * NB + b) * kHStep + (part * 4 + g) * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) hv[j] = ld16(src + 32 * kHParts * j);
  };
  int n_ahead;
  uint4 hv[UH][4];
  load(0, 0);
#pragma unroll
  for (int u = 0; u < UH; ++u) load_h(hv[u], column(u / NB, 0, n_ahead), u % NB);
#pragma unroll
  for (int p = 1; p < PE; ++p) load(p, p);
  for (int i = lane; i < kHParts * kSmallM * (4 * R + 1); i += 64) (&sums[wave][0][0][0])[i] = v4f{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](int p, int b, const uint4(&x)[4], v4f(&d)[R]) __attribute__((always_inline)) {
    uint4 w[R];
#pragma unroll
    for (int t = 0; t < R; ++t) w[t] = mine[Rows::at(min(16 * t + r, 8 * C8 - 1), 4 * b + g)];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const uint32_t c = j == 0 ? w[t].x : j == 1 ? w[t].y : j == 2 ? w[t].z : w[t].w;
        d[t] = mfma_bf16(fp4x8_bf16(c, scale_operand<0>(sc[p][t][b] >> (8 * g))), __builtin_bit_cast(v8s, x[j]), d[t]);
      }
  };
  auto expert = [&](int p, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      const int n = min(64 * l + lane, cols * 4 * NB - 1);
      mine[Rows::at(n / (4 * NB), n % (4 * NB))] = q[p][l];
    }
    wave_lds_order();
    v4f d[R];
    // a token that did not pick the expert takes nothing from it, also where
    // its weights are not finite
    auto begin = [&](int who) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < R; ++t) d[t] = sums[wave][part][max(who, 0) >> 4][4 * t + g];
    };
    auto end = [&](int who) __attribute__((always_inline)) {
      if (who >= 0 && r < 5 * kHParts) {
#pragma unroll
        for (int t = 0; t < R; ++t) sums[wave][part][who >> 4][4 * t + g] = d[t];
      }
    };
    int n, n_same;
    const int who = column(i, 0, n);
    begin(who);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int u = p * NB + b;
      multiply(p, b, hv[u % UH], d);
      load_h(hv[u % UH], column(i + (b + UH) / NB, 0, n_ahead), (b + UH) % NB);
      if constexpr (NB * R > 4 || C8 == 2) __builtin_amdgcn_sched_barrier(0);  // one K-step's operands at a time in registers
    }
    end(who);
    // (further passes ask for h when they need it, and so wait for the weights
    // under way too: 16 tokens seldom pick one of many experts more than five times)
    const int tokens = __builtin_amdgcn_readfirstlane(n);
    for (int pass = 1; 5 * pass < tokens; ++pass) {
      wave_lds_order();  // other lanes' sums than before
      const int more = column(i, pass, n_same);
      begin(more);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint4 x[4];
        load_h(x, more, b);
        multiply(p, b, x, d);
      }
      end(more);
    }
    wave_lds_order();
    load(p, i + PE);
  };
  // out of the loop itself, not round its end: paths that met there would make
  // the next round wait for all loads
  for (int i0 = 0;; i0 += PE) {
#pragma unroll
    for (int p = 0; p < PE; ++p) {
      if (i0 + p >= experts) goto done;
      expert(p, i0 + p);
    }
  }
done:
  wave_lds_order();
  // a token's three parts, the smallest first, then the waves in order
#pragma unroll
  for (int t = 0; t < R; ++t)
    sums[wave][0][r][4 * t + g] += sums[wave][1][r][4 * t + g] + sums[wave][2][r][4 * t + g];
  __syncthreads();
  if (wave < R && r < M) {
    const int n = 16 * wave + 4 * g;
    v4f v = sums[0][0][r][4 * wave + g];
#pragma unroll
    for (int w = 1; w < kLayerWaves; ++w) v += sums[w][0][r][4 * wave + g];
    if (n < cols) {
      uint2 o;
      o.x = (uint32_t)bf16_bits(v[0]) | ((uint32_t)bf16_bits(v[1]) << 16);
      o.y = (uint32_t)bf16_bits(v[2]) | ((uint32_t)bf16_bits(v[3]) << 16);
      *reinterpret_cast<uint2*>(out + (size_t)r * H + c0 + n) = o;
    }
  }
}

template <int S>
static hipError_t launch_gate_up_s(const moe_plan* p, const LayerArgs& a, const float* logits, uint16_t* gp, Ev ev) {
  const int E = (int)p->s.E, I = (int)p->s.I, k = (int)p->s.top_k;
  const int64_t items = std::min<int64_t>(E, a.M * k) * (I / 8);
  const dim3 grid((unsigned)std::min<int64_t>(items, p->num_cus));
  auto go = [&](auto kern) {
    return launch_k(kern, grid, dim3(64 * kLayerWaves), 0, a.stream, ev, (const uint16_t*)a.x, logits,
                    (const uint8_t*)a.w13, (const uint8_t*)a.s13, wsp<int>(p, p->L.topk_ids),
                    wsp<float>(p, p->L.topk_w), gp, wsp<PickList>(p, p->X.layer_list), (int)a.M, (int)p->s.H, E, I, k, p->s.routed_scaling);
  };
  if (E <= 256) return a.M <= kLayerWaves ? go(layer_gate_up_kernel<S, 4, 1>) : go(layer_gate_up_kernel<S, 4, 2>);
  return a.M <= kLayerWaves ? go(layer_gate_up_kernel<S, 16, 1>) : go(layer_gate_up_kernel<S, 16, 2>);
}

template <int NB, int C8>
static hipError_t launch_down_c8(const moe_plan* p, const LayerArgs& a, const uint16_t* gp, Ev ev) {
  const int H = (int)p->s.H;
  const dim3 grid((unsigned)((H + 8 * C8 - 1) / (8 * C8)));
  return launch_k(layer_down_kernel<NB, C8>, grid, dim3(64 * kLayerWaves), 0, a.stream, ev, gp,
                  wsp<PickList>(p, p->X.layer_list), (const uint8_t*)a.w2, (const uint8_t*)a.s2, (uint16_t*)a.out,
                  (int)a.M, H, (int)p->s.top_k);
}

template <int NB>
static hipError_t launch_down_nb(const moe_plan* p, const LayerArgs& a, int c8, const uint16_t* gp, Ev ev) {
  switch (c8) {
    case 1: return launch_down_c8<NB, 1>(p, a, gp, ev);
    case 2: return launch_down_c8<NB, 2>(p, a, gp, ev);
    case 3: return launch_down_c8<NB, 3>(p, a, gp, ev);
    default: return launch_down_c8<NB, 4>(p, a, gp, ev);
  }
}

hipError_t launch_layer(const moe_plan* p, const moe_router* router, const LayerArgs& a) {
  float* logits = wsp<float>(p, p->X.layer_logits);
  uint16_t* gp = wsp<uint16_t>(p, p->X.layer_g);
  const RouterArgs ra{a.M, p->s.E, p->s.H, p->s.H, a.x, router->w, logits, router->x_type, router->w_type};
  // stages: route (the router), gate_up (with the top-k), down (with the
  // combine); the others record empty intervals
  Ev ev[kStages];
  if (p->n_events)
    for (int i = 0; i < kStages; ++i) ev[i] = Ev{p->events[2 * i], p->events[2 * i + 1]};
  if (p->call_start) {
    ev[0].start = p->call_start;
    ev[5].stop = p->call_stop;
  }
  hipError_t e = launch_router(ra, p->num_cus, a.stream, ev[0]);
  if (e == hipSuccess) e = record_empty(p, ev[1], a.stream);
  if (e != hipSuccess) return e;
  const int H = (int)p->s.H, nks = H / 128;
  switch ((nks + kLayerWaves - 1) / kLayerWaves) {  // K-steps a wave
    case 1: e = launch_gate_up_s<1>(p, a, logits, gp, ev[2]); break;
    case 2: e = launch_gate_up_s<2>(p, a, logits, gp, ev[2]); break;
    case 3: e = launch_gate_up_s<3>(p, a, logits, gp, ev[2]); break;
    case 4: e = launch_gate_up_s<4>(p, a, logits, gp, ev[2]); break;
    case 5: e = launch_gate_up_s<5>(p, a, logits, gp, ev[2]); break;
    case 6: e = launch_gate_up_s<6>(p, a, logits, gp, ev[2]); break;
    case 7: e = launch_gate_up_s<7>(p, a, logits, gp, ev[2]); break;
    default: e = launch_gate_up_s<8>(p, a, logits, gp, ev[2]); break;
  }
  for (int i = 3; i <= 4 && e == hipSuccess; ++i) e = record_empty(p, ev[i], a.stream);
  if (e != hipSuccess) return e;
  // one workgroup a CU, each the same number of columns: a multiple of 8
  // (H 6144 on 256 CUs: 24)
  const int c8 = std::min(4, (H / 8 + p->num_cus - 1) / p->num_cus);
  switch (p->s.I / 128) {
    case 1: e = launch_down_nb<1>(p, a, c8, gp, ev[5]); break;
    case 2: e = launch_down_nb<2>(p, a, c8, gp, ev[5]); break;
    case 3: e = launch_down_nb<3>(p, a, c8, gp, ev[5]); break;
    default: e = launch_down_nb<4>(p, a, c8, gp, ev[5]); break;
  }
  return e == hipSuccess ? record_empty(p, ev[6], a.stream) : e;
}

}  // namespace qmoe
