// Tiles of C [rows, cols] = A B^T of 16-bit operands: staging, fragments, the main
// loop and the epilogue, for operands that lie along K or across it.
//
// A workgroup of WM x WN waves computes BM = 16 TM WM rows by BN = 16 TN WN columns,
// a wave 16 TM x 16 TN of them, in K-steps of 64 from S buffers of LDS. Memory goes
// straight to LDS (16 bytes a lane, 1 KB an instruction, in LDS in lane order), so
// the tile's way through LDS needs no registers and what lies past a matrix's edge
// comes as zeros from the buffer's bound.
//
// LDS of an operand of R rows (or columns) and 64 k:
//  along K:  [R][64], 128-byte rows of eight 16-byte chunks; chunk c of row r lies at
//            c ^ (r >> 1 & 7): the 16 lanes that read a chunk column meet all banks.
//            A lane's MFMA operand, 8 k of its row, is one 16-byte read.
//  across K: [64][R]; the lane's 8 k come by two transposing reads, of which 16 lanes
//            take 4 k by 16 rows (32 bytes a k). The 32-byte blocks of k are exchanged
//            by the bits of k that tell apart the 8 k a half wave reads at a time.
#pragma once

#include <algorithm>
#include <type_traits>

#include "act.h"
#include "dense.h"
#include "mxfp4.h"

namespace qmoe {

template <bool F16>
__device__ __forceinline__ v4f mfma16(uint4 a, uint4 b, v4f c) {
  if constexpr (F16) return mfma_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c);
  else return mfma_bf16(__builtin_bit_cast(v8s, a), __builtin_bit_cast(v8s, b), c);
}
template <bool F16>
__device__ __forceinline__ float value16(uint16_t b) { return F16 ? fp16_value(b) : bf16_value(b); }
template <bool F16>
__device__ __forceinline__ uint16_t bits16(float v) { return F16 ? fp16_bits(v) : bf16_bits(v); }

// ----------------------------------------------------------------- memory to LDS
constexpr uint32_t kOutside = 0x80000000u;  // an offset past every buffer's bound

// Buffer descriptor of 2^31 bytes from p on (raw, 32-bit elements).
__device__ __forceinline__ v4i buffer_at(const void* p) {
  const uint64_t u = (uint64_t)p;
  return v4i{(int)__builtin_amdgcn_readfirstlane((uint32_t)u),
             (int)(__builtin_amdgcn_readfirstlane((uint32_t)(u >> 32)) & 0xFFFF), (int)kOutside, 0x00020000};
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// 16 bytes a lane from `offset` to LDS at `lds` + 16 lane; zeros where the offset is
// kOutside. In assembly, so that the compiler does not wait for it before every
// read of LDS: wait_and_barrier does that. No register is written but M0, which the
// compiler sets anew where it needs it (it warns that it does not keep M0's value over
// the block: it need not).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(v4i buffer, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(offset), "s"(buffer)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// All but the N newest of the wave's loads to LDS have arrived, its reads of LDS too; then the
// workgroup's barrier.
template <int N>
__device__ __forceinline__ void wait_and_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// ----------------------------------------------------------------- an operand's tile
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

template <bool BY_K, int R, int W>
struct Operand {
  static constexpr int kBytes = R * 128;
  static constexpr int kLoads = R / 8 / W;  // load instructions a wave
  static_assert(R % (8 * W) == 0, "whole loads");
  static_assert(!BY_K || R % 64 == 0, "whole groups of blocks");
  uint32_t off[kLoads];
  int left[kLoads];  // K from this lane's piece on, at the start

  // across K: how the 32-byte blocks of row k are exchanged
  static __device__ __forceinline__ int swap(int k) {
    if constexpr (R % 128 == 0) return (k & 3) | ((k >> 3 & 1) << 2);
    else return (k >> 1 & 1) | ((k >> 3 & 1) << 1);  // rows of an odd multiple of 128 bytes: k & 1 is another half of the banks
  }

  // rows: how many of the tile's rows the matrix has
  __device__ __forceinline__ void init(int wave, int lane, int64_t ld, int64_t rows) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int piece = (i * W + wave) * 64 + lane;
      if constexpr (BY_K) {
        const int k = piece / (R / 8), at = piece % (R / 8);
        const int col = (((at >> 1) ^ swap(k)) << 1 | (at & 1)) * 8;
        off[i] = col < rows ? (uint32_t)(k * ld * 2 + col * 2) : kOutside;
        left[i] = -k;
      } else {
        const int row = piece >> 3, chunk = (piece & 7) ^ (row >> 1 & 7);
        off[i] = row < rows ? (uint32_t)(row * ld * 2 + chunk * 16) : kOutside;
        left[i] = -8 * chunk;
      }
    }
  }
  // the tile's last step, with `k` of K left: what is past them comes as zeros
  __device__ __forceinline__ void last(int k) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (left[i] + k <= 0) off[i] = kOutside;
  }
  // offset i with k of K left
  __device__ __forceinline__ uint32_t offset(int i, int k) const { return left[i] + k > 0 ? off[i] : kOutside; }
  // load i of the wave's. second: buffer of the rows from R / 2 on (gated: the other half of B's rows)
  __device__ __forceinline__ void load(int i, v4i buffer, v4i second, uint32_t lds, int wave) const {
    load_lds16(!BY_K && i * W + wave >= R / 16 ? second : buffer, off[i], lds + (uint32_t)(i * W + wave) * 1024);
  }

  // MFMA operand of K 32 j .. + 31 of the tile's row block b (16 rows)
  static __device__ __forceinline__ uint4 fragment(const uint8_t* lds, int b, int j, int r, int g) {
    if constexpr (BY_K) {
      const int k = 32 * j + 8 * g + (r >> 2);
      const uint8_t* p = lds + k * (2 * R) + ((b ^ swap(8 * g + (r >> 2))) * 32) + (r & 3) * 8;
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p);
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * 2 * R));
      const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
      return make_uint4(l.x, l.y, h.x, h.y);
    } else {
      return ld16(lds + (16 * b + r) * 128 + (((4 * j + g) ^ (r >> 1)) * 16));
    }
  }
};

// ----------------------------------------------------------------- epilogue
// What of a call's matrices moves in 16-byte pieces along a row.
enum { kVecY = 1, kVecResidual = 2, kVecPre = 4, kVecBias = 8 };

// Up to 8 values at p, of 16 bits (WIDE: of 32).
template <bool F16, bool WIDE>
__device__ __forceinline__ void read8(const void* p, bool vec, int n, float (&v)[8]) {
  if constexpr (WIDE) {
    const float* f = reinterpret_cast<const float*>(p);
    if (vec && n == 8) {
      *reinterpret_cast<v4f*>(v) = *reinterpret_cast<const v4f*>(f);
      *reinterpret_cast<v4f*>(v + 4) = *reinterpret_cast<const v4f*>(f + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? f[i] : 0.f;
    }
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    union {
      uint4 q;
      uint16_t b[8];
    } w;
    if (vec && n == 8) {
      w.q = ld16(h);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w.b[i] = i < n ? h[i] : (uint16_t)0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = value16<F16>(w.b[i]);
  }
}
template <bool F16, bool WIDE>
__device__ __forceinline__ void write8(void* p, bool vec, int n, const float (&v)[8]) {
  if constexpr (WIDE) {
    float* f = reinterpret_cast<float*>(p);
    if (vec && n == 8) {
      *reinterpret_cast<v4f*>(f) = *reinterpret_cast<const v4f*>(v);
      *reinterpret_cast<v4f*>(f + 4) = *reinterpret_cast<const v4f*>(v + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) f[i] = v[i];
    }
  } else {
    uint16_t* h = reinterpret_cast<uint16_t*>(p);
    union {
      uint4 q;
      uint16_t b[8];
    } w;
#pragma unroll
    for (int i = 0; i < 8; ++i) w.b[i] = bits16<F16>(v[i]);
    if (vec && n == 8) {
      *reinterpret_cast<uint4*>(h) = w.q;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) h[i] = w.b[i];
    }
  }
}

template <bool F16>
__device__ __forceinline__ void write_pre(const GemmArgs& a, int64_t at, int n, const float (&v)[8]) {
  if (a.pre_type == MOE_FP32) write8<F16, true>(reinterpret_cast<float*>(a.pre) + at, a.vec & kVecPre, n, v);
  else write8<F16, false>(reinterpret_cast<uint16_t*>(a.pre) + at, a.vec & kVecPre, n, v);
}

// Eight columns n .. n + 7 of row m from their sums (n < cols); gated: `up` the
// second product's.
template <bool F16, GemmKind KIND>
__device__ __forceinline__ void store8(const GemmArgs& a, int64_t m, int64_t n, float (&c)[8], const float (&up)[8]) {
  const int left = (int)min((int64_t)8, a.cols - n);
  const bool vy = a.vec & kVecY;
  uint16_t* y16 = reinterpret_cast<uint16_t*>(a.y) + m * a.ldy + n;
  if constexpr (KIND == kGemmGated) {
    if (a.pre) {
      write_pre<F16>(a, m * a.ldp + n, left, c);
      write_pre<F16>(a, m * a.ldp + a.cols + n, left, up);
    }
    with_act(a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = act_value<act>(c[i]) * up[i];
    });
    write8<F16, false>(y16, vy, left, c);
  } else if constexpr (KIND == kGemmForward) {
    float t[8];
    if (a.bias) {
      read8<F16, false>(reinterpret_cast<const uint16_t*>(a.bias) + n, a.vec & kVecBias, left, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] += t[i];
    }
    if (a.pre) write_pre<F16>(a, m * a.ldp + n, left, c);
    with_act(a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = act_value<act>(c[i]);
    });
    if (a.y_type == MOE_FP32) {
      if (a.residual) {
        read8<F16, true>(reinterpret_cast<const float*>(a.residual) + m * a.ldr + n, a.vec & kVecResidual, left, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] += t[i];
      }
      write8<F16, true>(reinterpret_cast<float*>(a.y) + m * a.ldy + n, vy, left, c);
    } else {
      if (a.residual) {
        read8<F16, false>(reinterpret_cast<const uint16_t*>(a.residual) + m * a.ldr + n, a.vec & kVecResidual, left, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] += t[i];
      }
      write8<F16, false>(y16, vy, left, c);
    }
  } else {
    write8<F16, false>(y16, vy, left, c);
  }
}

// Tile of workgroup `block`. Workgroups go to the eight XCDs in turn: XCD x takes a
// contiguous eighth of the tiles, walked in groups of GM row blocks, so that the tiles
// it runs at a time share operands in its L2.
__device__ __forceinline__ void tile_of(int block, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int GM = 8;
  const int total = tiles_m * tiles_n;
  const int xcd = block & 7, at = block >> 3, per = total >> 3, rest = total & 7;
  const int id = xcd * per + min(xcd, rest) + at;
  const int group = id / (GM * tiles_n), first = group * GM, rows = min(GM, tiles_m - first);
  const int in = id - group * GM * tiles_n;
  tm = first + in % rows;
  tn = in / rows;
}

// A split's sums (a.splits > 1: workgroups take parts of K, joined by split_join_kernel):
// fp32 [split][rows][columns of B's rows, padded to 8].
__device__ __forceinline__ float* split_sums(const GemmArgs& a, int split, int64_t m, bool gated) {
  const int64_t ld = (a.cols + 7) / 8 * 8 * (gated ? 2 : 1);
  return reinterpret_cast<float*>(a.ws) + (split * a.rows + m) * ld;
}

// Large products are bound by the MFMAs and the power they may draw: 4096 x 6144 x 6144 291
// us forward, 264 and 261 for the gradients (1062 to 1185 TFLOP/s; a library's products of
// the size 281 to 341). There 32 x 32 MFMAs, other orders of the MFMAs and of the tiles
// and waves' priorities gave the same times at another clock, and a step without its
// barrier 2 %. Eight waves, so that a wave's sums and both halves' operands fit its
// registers: four waves of 128 x 128 moved sums between the two register files.
// KG groups of WM x WN waves take the K-steps in turn, each through buffers of its own, and
// join their sums at the end: small tiles leave most of a SIMD's time to the LDS's latency.
template <bool F16, GemmKind KIND, int TM, int TN, int WM, int WN, int S, int KG>
__global__ __launch_bounds__(64 * WM * WN * KG) void gemm_tile_kernel(const GemmArgs a, int tiles_m, int tiles_n) {
  constexpr int W = WM * WN, BM = 16 * TM * WM, BN = 16 * TN * WN;
  constexpr bool gated = KIND == kGemmGated;
  constexpr int cols = gated ? BN / 2 : BN;  // columns of y a tile
  typedef Operand<KIND == kGemmWeight, BM, W> OpA;
  typedef Operand<KIND == kGemmInput || KIND == kGemmWeight, BN, W> OpB;
  constexpr int kStage = OpA::kBytes + OpB::kBytes, kLoads = OpA::kLoads + OpB::kLoads;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[KG * S * kStage];
  const int group = KG > 1 ? wave_id() / W : 0, wave = wave_id() - group * W;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wm = wave / WN, wn = wave % WN;
  const int tiles = tiles_m * tiles_n, split = blockIdx.x / tiles;
  int tm, tn;
  tile_of(blockIdx.x - split * tiles, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * cols;

  OpA la;
  OpB lb;
  la.init(wave, lane, a.lda, a.rows - m0);
  if constexpr (gated) {
    // rows [0, BN / 2) of B's tile: gate; from BN / 2 on: up, the same columns
    lb.init(wave, lane, a.ldb, BN);
#pragma unroll
    for (int i = 0; i < OpB::kLoads; ++i) {
      const int piece = (i * W + wave) * 64 + lane, row = (piece >> 3) % (BN / 2), chunk = (piece & 7) ^ (piece >> 4 & 7);
      lb.off[i] = n0 + row < a.cols ? (uint32_t)(row * a.ldb * 2 + chunk * 16) : kOutside;
    }
  } else {
    lb.init(wave, lane, a.ldb, a.cols - n0);
  }
  // this split's part of K
  const int64_t part = ((a.K + 63) / 64 + a.splits - 1) / a.splits * 64, k0 = split * part;
  const int64_t K = min(part, a.K - k0);
  const int steps = (int)((K + 64 * KG - 1) / (64 * KG));  // of a group
  const int64_t step_a = KIND == kGemmWeight ? 64 * a.lda : 64, step_b = KIND >= kGemmInput ? 64 * a.ldb : 64;
  const uint16_t* pa = reinterpret_cast<const uint16_t*>(a.a) + (KIND == kGemmWeight ? m0 : m0 * a.lda) + k0 / 64 * step_a;
  const uint16_t* pb = reinterpret_cast<const uint16_t*>(a.b) + (KIND >= kGemmInput ? n0 : n0 * a.ldb) + k0 / 64 * step_b;
  uint8_t* const own = lds + group * (S * kStage);
  const uint32_t base = __builtin_amdgcn_readfirstlane(lds_address(own));

  // Loads of the group's step t to buffer t % S, one at a time.
  v4i ba, bb, bc;
  uint32_t at;
  auto begin_loads = [&](int t, int buffer) __attribute__((always_inline)) {
    const int64_t kt = (int64_t)t * KG + group;
    if (t + 1 >= steps) {  // (past the last step: zeros, not used)
      la.last((int)(K - kt * 64));
      lb.last((int)(K - kt * 64));
    }
    at = base + (uint32_t)buffer * kStage;
    ba = buffer_at(pa + kt * step_a), bb = buffer_at(pb + kt * step_b);
    bc = gated ? buffer_at(pb + a.cols * a.ldb + kt * step_b) : bb;
  };
  auto load = [&](int n) __attribute__((always_inline)) {
    if (n < OpA::kLoads) la.load(n, ba, ba, at, wave);
    else lb.load(n - OpA::kLoads, bb, bc, at + OpA::kBytes, wave);
  };

  v4f acc[TN][TM];
#pragma unroll
  for (int t = 0; t < TN; ++t)
#pragma unroll
    for (int u = 0; u < TM; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
  // column block t of the wave in B's tile
  auto block_n = [&](int t) { return gated ? (t < TN / 2 ? wn * (TN / 2) + t : BN / 32 + wn * (TN / 2) + t - TN / 2) : wn * TN + t; };
  // A step is two halves of 32 k. While the MFMAs of one half run, the operands of the
  // next are read from LDS, so that they are there when the step's one barrier ends.
  uint4 fa[2][TM], fb[2][TN];
  auto read = [&](int i, int j, int buffer) __attribute__((always_inline)) {  // operand i of half j of a step
    const uint8_t* sa = own + buffer * kStage;
    if (i < TN) fb[j][i] = OpB::fragment(sa + OpA::kBytes, block_n(i), j, r, g);
    else fa[j][i - TN] = OpA::fragment(sa, wm * TM + i - TN, j, r, g);
  };
  // The reads go among the first three quarters of the MFMAs; so do, over all of the
  // second half's, the loads: issued in a row after the barrier they held up all waves
  // at once (4096 x 4096 x 6144 190 -> 172 us).
  auto half = [&](int j, int next) __attribute__((always_inline)) {
    constexpr int all = TM * TN, reads = TM + TN;
    constexpr int gap = all * 3 / 4 / reads > 0 ? all * 3 / 4 / reads : 1, every = all / kLoads > 0 ? all / kLoads : 1;
    static_assert(all >= reads && all >= kLoads, "one read and one load an MFMA at most");
#pragma unroll
    for (int i = 0; i < all; ++i) {
      const int u = i / TN, t = i % TN;
      if (i % gap == 0 && i / gap < reads) read(i / gap, j ^ 1, next);
      acc[t][u] = mfma16<F16>(fb[j][t], fa[j][u], acc[t][u]);
      if (j == 1 && i % every == every - 1 && i / every < kLoads) load(i / every);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int t = 0; t < S; ++t) {
    begin_loads(t, t);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) load(n);
  }
  wait_and_barrier<(S - 1) * kLoads>();
#pragma unroll
  for (int i = 0; i < TM + TN; ++i) read(i, 0, 0);
  int buffer = 0;
  for (int t = 0; t < steps; ++t) {
    const int next = buffer + 1 == S ? 0 : buffer + 1;
    half(0, buffer);
    // step t has been read by all waves, step t + 1 has arrived
    wait_and_barrier<(S - 2) * kLoads>();
    begin_loads(t + S, buffer);
    half(1, next);
    buffer = next;
  }
  // 16 rows of sums at a time through LDS of the wave's own, so that all that moves
  // in the epilogue moves in 16-byte pieces along a row
  wait_and_barrier<0>();
  constexpr int C = 16 * TN, P = C + 4;
  constexpr int pieces = (gated ? C / 2 : C) / 8;
  constexpr int rows = KG > 1 ? TM : 1;  // blocks of 16 rows at a time
  float* mine = reinterpret_cast<float*>(lds) + wave * 16 * P * rows;
  constexpr int other = W * 16 * P * rows;  // from a group's sums to the next one's
  static_assert(S * kStage >= W * 16 * P * rows * 4, "the sums fit the operands' buffers");
#pragma unroll
  for (int u0 = 0; u0 < TM; u0 += rows) {
#pragma unroll
    for (int u = 0; u < rows; ++u)
#pragma unroll
      for (int t = 0; t < TN; ++t) *reinterpret_cast<v4f*>(&mine[group * other + (16 * u + r) * P + 16 * t + 4 * g]) = acc[t][u0 + u];
    if constexpr (KG > 1) barrier_lds();
    else wave_lds_order();
#pragma unroll
    for (int i = lane + 64 * group; i < 16 * rows * pieces; i += 64 * KG) {
      const int row = i / pieces, c = i % pieces * 8;
      const int64_t m = m0 + 16 * (wm * TM + u0) + row, n = n0 + (gated ? C / 2 : C) * wn + c;
      float v[8], up[8];
#pragma unroll
      for (int q = 0; q < 8; q += 4) {
        auto sum = [&](int at) __attribute__((always_inline)) {
          v4f s = *reinterpret_cast<const v4f*>(&mine[at]);
#pragma unroll
          for (int k = 1; k < KG; ++k) s += *reinterpret_cast<const v4f*>(&mine[k * other + at]);
          return s;
        };
        *reinterpret_cast<v4f*>(v + q) = sum(row * P + c + q);
        if constexpr (gated) *reinterpret_cast<v4f*>(up + q) = sum(row * P + C / 2 + c + q);
      }
      if (m < a.rows && n < a.cols) {
        if (a.splits > 1) {
          float* p = split_sums(a, split, m, gated) + n;
          write8<F16, true>(p, true, 8, v);
          if constexpr (gated) write8<F16, true>(p + (a.cols + 7) / 8 * 8, true, 8, up);
        } else {
          store8<F16, KIND>(a, m, n, v, up);
        }
      }
    }
    if constexpr (KG == 1) wave_lds_order();
  }
}

// The splits' sums, added in their order, and the epilogue: a launch of its own, 4 us, so
// that no workgroup waits for another (atomics would add in any order).
template <bool F16, GemmKind KIND>
__global__ __launch_bounds__(256) void split_join_kernel(const GemmArgs a) {
  constexpr bool gated = KIND == kGemmGated;
  const int64_t pieces = (a.cols + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.rows * pieces; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / pieces, n = (i - m * pieces) * 8;
    float v[8] = {}, up[8] = {};
    for (int s = 0; s < a.splits; ++s) {
      float t[8];
      const float* p = split_sums(a, s, m, gated) + n;
      read8<F16, true>(p, true, 8, t);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] += t[q];
      if constexpr (gated) {
        read8<F16, true>(p + pieces * 8, true, 8, t);
#pragma unroll
        for (int q = 0; q < 8; ++q) up[q] += t[q];
      }
    }
    store8<F16, KIND>(a, m, n, v, up);
  }
}

// ----------------------------------------------------------------- few rows
// 16 TM rows by 16 TN columns (gated: 8 TN of both products) a workgroup at a time. Its
// eight waves share no operand: they take the K-steps of 64 in turn, each through S
// buffers of its own, without a barrier, and join their sums through LDS at the end of a
// tile. A workgroup takes tiles one after another; the loads run on over their ends.
// Bound by the weights' way from memory: 16 x 16384 x 6144 39 us (5.1 TB/s) over copies of the
// weights in turn, 49 where each call's are cold in every cache.
template <bool F16, GemmKind KIND, int TM, int TN, int S>
__global__ __launch_bounds__(512) void gemm_wave_kernel(const GemmArgs a, int tiles_m, int tiles_n) {
  constexpr int W = 8, BM = 16 * TM, BN = 16 * TN;
  constexpr bool gated = KIND == kGemmGated;
  constexpr int cols = gated ? BN / 2 : BN;
  static_assert(KIND == kGemmForward || gated, "operands along K");
  typedef Operand<false, BM, 1> OpA;
  typedef Operand<false, BN, 1> OpB;
  constexpr int kStage = OpA::kBytes + OpB::kBytes, kLoads = OpA::kLoads + OpB::kLoads;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[W * S * kStage];
  __shared__ float sums[W][BM][BN];
  const int wave = wave_id(), lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int tiles = tiles_m * tiles_n, step = gridDim.x;
  const int steps = (int)((a.K + 63) / 64), per = (steps + W - 1) / W;  // K-steps, of a wave (some of them past K)
  const uint32_t base = __builtin_amdgcn_readfirstlane(lds_address(lds)) + wave * (S * kStage);
  const uint8_t* mine = lds + wave * (S * kStage);

  // Loads run S steps ahead: those of step `at` of tile `tile`.
  OpA la;
  OpB lb;
  const uint16_t *pa, *pb;
  int tile = blockIdx.x, at = 0, buffer = 0;
  auto begin_tile = [&]() __attribute__((always_inline)) {
    if (tile >= tiles) return;
    const int64_t m0 = (int64_t)(tile / tiles_n) * BM, n0 = (int64_t)(tile % tiles_n) * cols;
    la.init(0, lane, a.lda, a.rows - m0);
    if constexpr (gated) {
      lb.init(0, lane, a.ldb, BN);
#pragma unroll
      for (int i = 0; i < OpB::kLoads; ++i) {
        const int piece = i * 64 + lane, row = (piece >> 3) % (BN / 2), chunk = (piece & 7) ^ (piece >> 4 & 7);
        lb.off[i] = n0 + row < a.cols ? (uint32_t)(row * a.ldb * 2 + chunk * 16) : kOutside;
      }
    } else {
      lb.init(0, lane, a.ldb, a.cols - n0);
    }
    pa = reinterpret_cast<const uint16_t*>(a.a) + m0 * a.lda;
    pb = reinterpret_cast<const uint16_t*>(a.b) + n0 * a.ldb;
  };
  auto load = [&]() __attribute__((always_inline)) {
    const int t = at * W + wave, left = tile < tiles ? (int)min(a.K - (int64_t)t * 64, (int64_t)64) : 0;
    const int64_t k = left > 0 ? (int64_t)t * 64 : 0;
    const v4i ba = buffer_at(pa + k), bb = buffer_at(pb + k);
    const v4i bc = gated ? buffer_at(pb + a.cols * a.ldb + k) : bb;
    const uint32_t to = base + (uint32_t)buffer * kStage;
#pragma unroll
    for (int i = 0; i < OpA::kLoads; ++i) load_lds16(ba, la.offset(i, left), to + i * 1024);
#pragma unroll
    for (int i = 0; i < OpB::kLoads; ++i)
      load_lds16(gated && i >= OpB::kLoads / 2 ? bc : bb, lb.offset(i, left), to + OpA::kBytes + i * 1024);
    buffer = buffer + 1 == S ? 0 : buffer + 1;
    if (++at == per) {
      at = 0;
      tile += step;
      begin_tile();
    }
  };
  begin_tile();
#pragma unroll
  for (int i = 0; i < S; ++i) load();
  int from = 0;
  for (int now = blockIdx.x; now < tiles; now += step) {
    v4f acc[TN][TM];
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int u = 0; u < TM; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < per; ++i) {
      asm volatile("s_waitcnt vmcnt(%0)" : : "n"((S - 1) * kLoads) : "memory");
      const uint8_t* sa = mine + from * kStage;
      const uint8_t* sb = sa + OpA::kBytes;
      uint4 fa[2][TM], fb[2][TN];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int t = 0; t < TN; ++t) fb[j][t] = OpB::fragment(sb, t, j, r, g);
#pragma unroll
        for (int u = 0; u < TM; ++u) fa[j][u] = OpA::fragment(sa, u, j, r, g);
      }
      from = from + 1 == S ? 0 : from + 1;
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");  // read before it is loaded anew
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int t = 0; t < TN; ++t)
#pragma unroll
          for (int u = 0; u < TM; ++u) acc[t][u] = mfma16<F16>(fb[j][t], fa[j][u], acc[t][u]);
      load();
    }
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int u = 0; u < TM; ++u) *reinterpret_cast<v4f*>(&sums[wave][16 * u + r][16 * t + 4 * g]) = acc[t][u];
    barrier_lds();
    const int64_t m0 = (int64_t)(now / tiles_n) * BM, n0 = (int64_t)(now % tiles_n) * cols;
    constexpr int pieces = cols / 8;
    for (int i = threadIdx.x; i < BM * pieces; i += 64 * W) {
      const int row = i / pieces, c = i % pieces * 8;
      float v[8] = {}, up[8] = {};
#pragma unroll
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[q] += sums[w][row][c + q];
          if constexpr (gated) up[q] += sums[w][row][cols + c + q];
        }
      if (m0 + row < a.rows && n0 + c < a.cols) store8<F16, KIND>(a, m0 + row, n0 + c, v, up);
    }
    barrier_lds();
  }
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");  // no load to LDS outlives the workgroup
}

template <bool F16, GemmKind KIND, int TM, int TN, int S>
hipError_t launch_wave(const GemmArgs& a, int cus, hipStream_t stream) {
  constexpr int cols = 16 * TN / (KIND == kGemmGated ? 2 : 1);
  const int64_t tm = (a.rows + 16 * TM - 1) / (16 * TM), tn = (a.cols + cols - 1) / cols;
  return launch_k(gemm_wave_kernel<F16, KIND, TM, TN, S>, dim3((unsigned)std::min<int64_t>(tm * tn, cus)), dim3(512), 0,
                  stream, Ev{}, a, (int)tm, (int)tn);
}

template <bool F16, GemmKind KIND, int TM, int TN, int WM, int WN, int S, int KG = 1>
hipError_t launch_tile(const GemmArgs& a, hipStream_t stream) {
  constexpr int BM = 16 * TM * WM, cols = 16 * TN * WN / (KIND == kGemmGated ? 2 : 1);
  const int64_t tm = (a.rows + BM - 1) / BM, tn = (a.cols + cols - 1) / cols;
  return launch_k(gemm_tile_kernel<F16, KIND, TM, TN, WM, WN, S, KG>, dim3((unsigned)(tm * tn * a.splits)),
                  dim3(64 * WM * WN * KG), 0, stream, Ev{}, a, (int)tm, (int)tn);
}

}  // namespace qmoe
