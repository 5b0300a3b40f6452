// What reads the output head's logits: scores of given tokens (log probability,
// entropy, largest alternatives) and distillation from a teacher's top logits.
//
// One pass over a row forms, a thread over its elements and the threads at the end,
//   m near max z, s = sum exp(c (z - m)), t = sum exp(c (z - m)) c (z - m)
// (c = 1 / temperature), the sums moved on by exp(c (m_old - m)) whenever m grows, so
//   lse = c m + log s,  entropy = log s - t / s.
// m starts at the type's lowest number, not at -inf: a row (or thread) of nothing but
// -inf has s = 0 and no NaN. A NaN or +inf makes s NaN. Sums of a thread are binary32,
// those over threads and what follows binary64.
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "head.h"
#include "mxfp4.h"

namespace qmoe {

constexpr float kLog2e = 1.4426950408889634f;

// ----------------------------------------------------------------- elements
template <int TYPE>
struct Logit {
  static constexpr int kBytes = TYPE == MOE_FP32 ? 4 : 2, kPiece = 16 / kBytes;  // elements of 16 bytes
  // 16 bytes of -inf: what lies outside a row
  static __device__ __forceinline__ uint4 none() {
    const uint32_t w = TYPE == MOE_FP32 ? 0xFF800000u : TYPE == MOE_FP16 ? 0xFC00FC00u : 0xFF80FF80u;
    return make_uint4(w, w, w, w);
  }
  static __device__ __forceinline__ float load(const void* row, int64_t i) {
    if constexpr (TYPE == MOE_FP32) return reinterpret_cast<const float*>(row)[i];
    else if constexpr (TYPE == MOE_FP16) return fp16_value(reinterpret_cast<const uint16_t*>(row)[i]);
    else return bf16_value(reinterpret_cast<const uint16_t*>(row)[i]);
  }
  static __device__ __forceinline__ void store(void* row, int64_t i, float v) {
    if constexpr (TYPE == MOE_FP32) reinterpret_cast<float*>(row)[i] = v;
    else if constexpr (TYPE == MOE_FP16) reinterpret_cast<uint16_t*>(row)[i] = fp16_bits(v);
    else reinterpret_cast<uint16_t*>(row)[i] = bf16_bits(v);
  }
  static __device__ __forceinline__ float value(uint4 q, int i) {
    const uint32_t d = TYPE == MOE_FP32 ? (i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w)
                                        : (i / 2 == 0 ? q.x : i / 2 == 1 ? q.y : i / 2 == 2 ? q.z : q.w);
    if constexpr (TYPE == MOE_FP32) return __uint_as_float(d);
    else if constexpr (TYPE == MOE_FP16) return (float)__builtin_bit_cast(f16x2, d)[i & 1];
    else return __uint_as_float(i & 1 ? d & 0xFFFF0000u : d << 16);
  }
};

// A row as 16-byte pieces on 16-byte boundaries: `head` elements before them, `tail`
// elements behind. Elements have any alignment of their own size.
template <int TYPE>
struct Row {
  const uint8_t* p;
  int64_t V, pieces;
  int head, tail;
  __device__ __forceinline__ Row(const void* z, int64_t m, int64_t ld, int64_t n) {
    constexpr int b = Logit<TYPE>::kBytes, e = Logit<TYPE>::kPiece;
    p = reinterpret_cast<const uint8_t*>(z) + m * ld * b;
    V = n;
    head = (int)min((int64_t)(((16 - ((uintptr_t)p & 15)) & 15) / b), n);
    pieces = (n - head) / e;
    tail = (int)(n - head - pieces * e);
  }
  __device__ __forceinline__ uint4 piece_once(int64_t i) const {
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const v4i*>(p + head * Logit<TYPE>::kBytes + i * 16)));
  }
  __device__ __forceinline__ uint4 piece(int64_t i) const { return ld16(p + head * Logit<TYPE>::kBytes + i * 16); }
  __device__ __forceinline__ int64_t first(int64_t i) const { return head + i * Logit<TYPE>::kPiece; }  // its first element
  __device__ __forceinline__ int edges() const { return head + tail; }  // elements outside the pieces,
  __device__ __forceinline__ int64_t edge(int i) const { return i < head ? i : V - edges() + i; }  // the i-th of them
};

// The wave's sum, uniform: within rows of 16 lanes by DPP, the four rows' as scalars
// (by six exchanges through LDS it took 0.25 us, and a row's way through a workgroup
// has several).
template <int CTRL>
__device__ __forceinline__ double dpp_other(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_other<0xB1>(v);   // lane ^ 1
  v += dpp_other<0x4E>(v);   // lane ^ 2
  v += dpp_other<0x141>(v);  // half row mirrored
  v += dpp_other<0x140>(v);  // row mirrored
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
// The wave's largest number, NaN only if all are.
template <int CTRL>
__device__ __forceinline__ float dpp_other(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp_other<0xB1>(v));
  v = fmaxf(v, dpp_other<0x4E>(v));
  v = fmaxf(v, dpp_other<0x141>(v));
  v = fmaxf(v, dpp_other<0x140>(v));
  auto at = [&](int lane) { return __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(v), lane)); };
  return fmaxf(fmaxf(at(0), at(16)), fmaxf(at(32), at(48)));
}

// ----------------------------------------------------------------- sums of a row
// A thread's sums, N elements at a time: each N by themselves, then added to the rest, with
// more than kChain of them (LONG) with the rounding errors carried along: a chain of plain additions of like
// terms rounds them all the same way (it lost 3e-4 of a sum of 2^15). Carrying them costs 1 %
// of 2048 x 131072. m stays while the elements pass it by no more than a factor 2^kOver of
// the sums: of a row that rises slowly every N elements would scale the sums, by a
// rounded factor each time. (SHORT: of some hundred elements at most, m is their largest.)
constexpr float kOver = 6.f;
constexpr int kChain = 32;
template <bool MEAN, bool SHORT = false>
struct Sums {
  float m = -FLT_MAX, s = 0.f, t = 0.f;
  float s_over = 0.f, t_over = 0.f;  // what the sums hold too much
  static __device__ __forceinline__ void carry(float& sum, float& over, float v) {
    const float y = v - over, n = sum + y;
    over = (n - sum) - y;
    sum = n;
  }
  // N elements, in units of 1 / cl (cl = c log2 e: t is in log2 units); returns the largest
  template <bool LONG = false, int N>
  __device__ __forceinline__ float add(const float (&v)[N], float cl) {
    const float bound = SHORT ? m : m + kOver / cl;
    float top = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, v[i]);
    // (a factor is 0 long before -1e4; no infinity, which zero sums would turn into NaN)
    const float mn = SHORT ? fmaxf(m, top) : top > bound ? top : m;
    const float back = fmaxf((m - mn) * cl, -1e4f), f = __builtin_amdgcn_exp2f(back);
    if constexpr (MEAN) t = (t + s * back) * f;
    s *= f;
    if constexpr (LONG) {
      if constexpr (MEAN) t_over = (t_over + s_over * back) * f;
      s_over *= f;
    }
    m = mn;
    float ps = 0.f, pt = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = (v[i] - m) * cl, e = __builtin_amdgcn_exp2f(d);
      ps += e;
      if constexpr (MEAN) pt += e * fmaxf(d, -1e4f);
    }
    if constexpr (LONG) {
      carry(s, s_over, ps);
      if constexpr (MEAN) carry(t, t_over, pt);
    } else {
      s += ps;
      if constexpr (MEAN) t += pt;
    }
    return top;
  }
};

struct Total {
  float m;
  double s, t;  // t in natural units
};
// Over the workgroup's threads (THREADS of them), the same in all.
template <int THREADS, bool MEAN>
__device__ __forceinline__ Total join(const Sums<MEAN>& a, float cl) {
  constexpr int W = THREADS / 64;
  __shared__ float lm[W];
  __shared__ double ls[W], lt[W];
  const int wave = wave_id(), lane = threadIdx.x & 63;
  float m = row_max(a.m);
  if (lane == 0) lm[wave] = m;
  __syncthreads();
  m = row_max(lm[lane % W]);
  const float back = fmaxf((a.m - m) * cl, -1e4f);
  const double f = __builtin_amdgcn_exp2f(back);
  const double mine = (double)a.s - a.s_over;
  const double s = wave_sum(mine * f);
  if (lane == 0) ls[wave] = s;
  if constexpr (MEAN) {
    const double t = wave_sum(((double)a.t - a.t_over + mine * back) * f);
    if (lane == 0) lt[wave] = t;
  }
  __syncthreads();
  Total r{m, wave_sum(lane < W ? ls[lane] : 0.0), 0};
  if constexpr (MEAN) r.t = wave_sum(lane < W ? lt[lane] : 0.0) * 0.69314718055994531;
  return r;
}

// ----------------------------------------------------------------- the k largest
// Keys order elements by value, then by falling id. Candidates are collected in LDS
// while they reach a threshold below which no element can be among the k largest.
__device__ __forceinline__ uint64_t key_of(float v, int64_t id) {
  return ((uint64_t)order_key(v) << 32) | (uint32_t)~(uint32_t)id;
}

template <int THREADS, int STRETCHES = 1>
struct Candidates {
  static constexpr int kStretches = STRETCHES;  // of a thread's pieces
  static constexpr int kKeys = THREADS == 128 ? 512 : 2048;  // candidates held
  uint64_t key[kKeys];
  uint64_t top[kMaxTop];  // the k largest, in order
  uint64_t at_least;      // the threshold
  int n;                  // candidates met; those past kKeys are not held
  int reached[2][THREADS / 64];  // by a wave's threshold: how many of the threads' best do
  int stretches;  // of threads, whose best element reaches the threshold: thread + THREADS
  uint16_t stretch[kStretches * THREADS];  // stretch, in no order
  uint16_t high[kStretches * THREADS];     // of the stretches' best elements the upper 16 bits
  uint32_t best[THREADS];    // the threads' best elements (order_key)
};

// The candidates held, largest first, c.n of them at most k; the threshold is the k-th.
template <int THREADS, int S>
__device__ void sort_candidates(Candidates<THREADS, S>& c, int k) {
  __syncthreads();
  const int n = min(c.n, c.kKeys);
  int size = 2;
  while (size < n) size *= 2;
#pragma unroll 1
  for (int i = n + threadIdx.x; i < size; i += THREADS) c.key[i] = 0;
  __syncthreads();
#pragma unroll 1
  for (int run = 2; run <= size; run *= 2)
#pragma unroll 1
    for (int step = run / 2; step > 0; step /= 2) {
#pragma unroll 1
      for (int i = threadIdx.x; i < size / 2; i += THREADS) {
        const int lo = (i & ~(step - 1)) * 2 | (i & (step - 1)), hi = lo + step;
        const uint64_t a = c.key[lo], b = c.key[hi];
        if ((a < b) == ((lo & run) == 0)) c.key[lo] = b, c.key[hi] = a;
      }
      __syncthreads();
    }
  if (threadIdx.x == 0) {
    c.n = min(n, k);
    if (n >= k) c.at_least = c.key[k - 1];
  }
  __syncthreads();
}

// c.top: the k largest of the candidates (zeros behind fewer). A few hundred are
// ranked by counting the larger ones, more are sorted.
template <int THREADS, int S>
__device__ void rank_candidates(Candidates<THREADS, S>& c, int k) {
  __syncthreads();
  const int n = c.n;
  if (n > THREADS) {
    sort_candidates(c, k);
    for (int j = threadIdx.x; j < k; j += THREADS) c.top[j] = j < c.n ? c.key[j] : 0;
  } else {
    for (int j = n + threadIdx.x; j < k; j += THREADS) c.top[j] = 0;
    if ((int)threadIdx.x < n) {
      const uint64_t key = c.key[threadIdx.x];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) rank += c.key[j] > key;
      if (rank < k) c.top[rank] = key;
    }
  }
  __syncthreads();
}

// A thread's N elements v with ids first .. as candidates; those of `left` that found
// no room stay in it.
template <int THREADS, int S, int N>
__device__ __forceinline__ void offer(Candidates<THREADS, S>& c, const float (&v)[N], int64_t first, uint32_t& left) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!(left >> i & 1)) continue;
    const uint64_t key = key_of(v[i], first + i);
    if (key >= c.at_least) {
      if (c.n > c.kKeys) continue;
      const int at = atomicAdd(&c.n, 1);
      if (at >= c.kKeys) continue;
      c.key[at] = key;
    }
    left &= ~(1u << i);
  }
}

// The k largest of a segment again, of which more candidates reach the threshold than
// fit (or fewer than k: `from` is 0 then): whenever they are full, they are sorted, all
// but k dropped and the threshold raised.
template <int TYPE, int THREADS, int S>
__device__ __forceinline__ void reselect(Candidates<THREADS, S>& c, const Row<TYPE>& row, int64_t p0, int64_t p1, bool edges, uint64_t from, int k) {
  if (threadIdx.x == 0) c.n = 0, c.at_least = from;
  __syncthreads();
  const int64_t inner = (p1 - p0) * Logit<TYPE>::kPiece, all = inner + (edges ? row.edges() : 0);
#pragma unroll 1
  for (int64_t base = 0; base < all; base += THREADS) {
    const int64_t i = base + threadIdx.x;
    uint32_t left = i < all;
    const int64_t first = !left ? 0 : i < inner ? row.first(p0) + i : row.edge((int)(i - inner));
    const float v[1] = {left ? Logit<TYPE>::load(row.p, first) : 0.f};
#pragma unroll 1
    for (;;) {
      offer(c, v, first, left);
      __syncthreads();
      const bool full = c.n >= c.kKeys;
      __syncthreads();
      if (!full) break;
      sort_candidates(c, k);
    }
  }
}

// The k largest of a segment whose threads hold their own elements' maxima: at least k
// elements reach the k-th largest of these, and hardly more do (131072 elements of 512
// threads, k 32: 33 where nothing ties), all of them elements of threads whose maximum
// reaches it, in stretches of `span` of a thread's pieces whose maximum (c.high) does.
// Those are read again (whole threads: 1.4 times the memory's traffic, a 16-byte piece
// costs a line). The threshold is taken from the maxima's upper 16 bits.
template <int TYPE, int THREADS, int S>
__device__ void select(Candidates<THREADS, S>& c, const Row<TYPE>& row, int64_t p0, int64_t p1, int span, bool edges, float edge, float best,
                       int k) {
  constexpr int E = Logit<TYPE>::kPiece, W = THREADS / 64;
  const uint32_t mine = order_key(best);
  c.best[threadIdx.x] = mine;
  if (threadIdx.x == 0) c.n = 0, c.stretches = 0;
  __syncthreads();
  // The largest 16-bit threshold that k maxima reach. The waves try a digit's values, one
  // each (two waves: a bit at a time by the first).
  uint32_t b[W], at = 0;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int w = 0; w < W; ++w) b[w] = c.best[64 * w + lane] >> 16;
  auto reached = [&](uint32_t from) __attribute__((always_inline)) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) n += __popcll(__ballot(b[w] >= from));
    return n;
  };
  if constexpr (W >= 8) {
    constexpr int B = W == 16 ? 4 : 3;
    const int wave = wave_id();
    int round = 0;
#pragma unroll 1
    for (int shift = 16; shift > 0; round ^= 1) {
      shift = shift > B ? shift - B : 0;
      const int n = reached(at | (uint32_t)wave << shift);
      if (lane == 0) c.reached[round][wave] = n;
      __syncthreads();
      // the largest value that suffices (in a shorter last digit, a value that sets bits
      // already decided changes nothing or does not suffice)
      const uint64_t enough = __ballot(lane < W && c.reached[round][lane % W] >= k);
      at |= (uint32_t)(63 - __clzll(enough)) << shift;
    }
    if (threadIdx.x == 0) c.at_least = (uint64_t)at << 48;
  } else if (threadIdx.x < 64) {
#pragma unroll 1
    for (uint32_t bit = 1u << 15; bit > 0; bit >>= 1)
      if (reached(at | bit) >= k) at |= bit;
    if (threadIdx.x == 0) c.at_least = (uint64_t)at << 48;
  }
  __syncthreads();
  const uint64_t at_least = c.at_least;
  if (mine >= (uint32_t)(at_least >> 32)) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int at = i * THREADS + threadIdx.x;
      if (S == 1 || c.high[at] >= (uint32_t)(at_least >> 48)) c.stretch[atomicAdd(&c.stretches, 1)] = (uint16_t)at;
    }
  }
  if (edges && (int)threadIdx.x < row.edges()) {
    float v[1] = {edge};
    uint32_t left = 1;
    offer(c, v, row.edge(threadIdx.x), left);
  }
  __syncthreads();
  const int n = c.stretches;
#pragma unroll 1
  for (int i = threadIdx.x; i < span * n; i += THREADS) {
    const int r = i / n, at = c.stretch[i - r * n];
    const int64_t p = p0 + ((int64_t)(at / THREADS) * span + r) * THREADS + at % THREADS;
    if (p >= p1) continue;
    const uint4 q = row.piece(p);
    float v[E], top;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      v[e] = Logit<TYPE>::value(q, e);
      top = e ? fmaxf(top, v[e]) : v[e];
    }
    if (order_key(top) < (uint32_t)(at_least >> 32)) continue;
    uint32_t left = (1u << E) - 1;
    offer(c, v, row.first(p), left);
  }
  __syncthreads();
  // too few where elements are NaN or -inf (the maxima start above -inf), too many of
  // equal ones
  const int met = c.n;
  __syncthreads();
  if (met < k || met > c.kKeys) reselect<TYPE>(c, row, p0, p1, edges, met < k ? 0 : at_least, k);
  rank_candidates(c, k);
}

// ----------------------------------------------------------------- scores
// A segment of a row a workgroup. Few rows are split over `parts` workgroups, whose
// sums and k keys go to the workspace and are joined by scores_join_kernel.
struct ScoresPart {
  float m;
  float pad;
  double s, t;
};

// (Log probabilities from the distance to m: lse has lost log s where all logits are the
// type's lowest number.)
__device__ void write_scores(const ScoresArgs& a, int64_t m, const Total& r, float given, const uint64_t* top) {
  const bool ok = r.m < INFINITY && r.s > 0;  // not NaN either
  const double logs = log(r.s), lse = r.m + logs;
  if (threadIdx.x == 0) {
    if (a.tokens) {
      const int64_t t = a.tokens[m];
      a.logprobs[m] = ok && t >= 0 && t < a.V ? (float)(((double)given - r.m) - logs) : NAN;
    }
    if (a.entropy) a.entropy[m] = ok ? (float)(logs - r.t / r.s) : NAN;
    if (a.lse) a.lse[m] = ok ? (float)lse : r.m == INFINITY ? INFINITY : r.s == 0 ? -INFINITY : NAN;
  }
  for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
    const uint64_t key = top[j];
    a.top_ids[m * a.k + j] = (int32_t)~(uint32_t)key;
    a.top_logprobs[m * a.k + j] = ok ? (float)(((double)key_to_float((uint32_t)(key >> 32)) - r.m) - logs) : NAN;
  }
}

template <int TYPE>
__device__ __forceinline__ float given_logit(const ScoresArgs& a, const Row<TYPE>& row, int64_t m) {
  const int64_t t = a.tokens ? a.tokens[m] : -1;
  return t >= 0 && t < a.V ? Logit<TYPE>::load(row.p, t) : 0.f;
}

// (at most 64 registers for 512 threads: four workgroups a CU). N elements a thread and
// tile, the next tile's under way meanwhile. Bound by memory: 2048 x 131072 bf16 94 us (5.7
// TB/s) without alternatives, whose logits are read past the caches; 114 with 32 of them: the
// search for the threshold and the second reading of some 33 threads' pieces, S stretches a
// thread, are a workgroup's own latency, and the logits pass through the caches for it.
template <int TYPE, int THREADS, int N, bool TOP, int S, bool LONG = false>
__global__ __launch_bounds__(THREADS, THREADS == 512 ? 8 : 4) void scores_kernel(const ScoresArgs a, int parts) {
  constexpr int E = Logit<TYPE>::kPiece, NP = N / E;  // pieces
  __shared__ std::conditional_t<TOP, Candidates<THREADS, S>, int> c;
  const uint64_t* top = nullptr;
  const int64_t m = blockIdx.x / parts;
  const int part = blockIdx.x % parts;
  const Row<TYPE> row(a.z, m, a.ldz, a.V);
  const int64_t per = (row.pieces + parts - 1) / parts;
  const int64_t p0 = min(per * part, row.pieces), p1 = min(p0 + per, row.pieces);
  const bool edges = part == 0;
  Sums<true> sums;

  uint4 q[NP];
  auto load = [&](int64_t base) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int64_t p = base + u * THREADS + threadIdx.x;
      if constexpr (!TOP && THREADS == 512) q[u] = p < p1 ? row.piece_once(p) : Logit<TYPE>::none();
      else q[u] = p < p1 ? row.piece(p) : Logit<TYPE>::none();
    }
  };
  load(p0);
  float edge[1] = {edges && (int)threadIdx.x < row.edges() ? Logit<TYPE>::load(row.p, row.edge(threadIdx.x)) : -INFINITY};
  const float given = parts == 1 ? given_logit<TYPE>(a, row, m) : 0.f;  // (two loads one behind the other, beside the tile's)
  float best = fmaxf(sums.add(edge, kLog2e), -FLT_MAX);
  const int tiles = (int)((p1 - p0 + NP * THREADS - 1) / (NP * THREADS)), span = (tiles + S - 1) / S;  // a stretch's tiles
  int64_t base = p0;
  auto sum_tile = [&]() __attribute__((always_inline)) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = Logit<TYPE>::value(q[i / E], i % E);
    load(base += NP * THREADS);
    return sums.template add<LONG>(v, kLog2e);
  };
  if constexpr (S == 1) {
    for (int t = 0; t < tiles; ++t) best = fmaxf(best, sum_tile());
  } else {
    int t = 0;
#pragma unroll 1
    for (int stretch = 0; stretch < S; ++stretch) {
      float high = -INFINITY;
      for (int end = min(t + span, tiles); t < end; ++t) high = fmaxf(high, sum_tile());
      best = fmaxf(best, high);
      c.high[stretch * THREADS + threadIdx.x] = (uint16_t)(order_key(high) >> 16);
    }
  }
  const Total r = join<THREADS>(sums, kLog2e);
  if constexpr (TOP) {
    select<TYPE>(c, row, p0, p1, span * NP, edges, edge[0], best, a.k);
    top = c.top;
  }
  if (parts == 1) {
    write_scores(a, m, r, given, top);
    return;
  }
  if (threadIdx.x == 0) reinterpret_cast<ScoresPart*>(a.ws)[blockIdx.x] = {r.m, 0.f, r.s, r.t};
  uint64_t* keys = reinterpret_cast<uint64_t*>(reinterpret_cast<ScoresPart*>(a.ws) + a.M * parts) + (int64_t)blockIdx.x * a.k;
  for (int j = threadIdx.x; j < a.k; j += THREADS) keys[j] = top[j];
}

constexpr int kMaxParts = 32;
static_assert(kMaxParts * kMaxTop <= Candidates<256>::kKeys, "the parts' keys are sorted at once");

template <int TYPE>
__global__ __launch_bounds__(256) void scores_join_kernel(const ScoresArgs a, int parts) {
  __shared__ Candidates<256> c;
  const int64_t m = blockIdx.x;
  const Row<TYPE> row(a.z, m, a.ldz, a.V);
  const float given = given_logit<TYPE>(a, row, m);
  const ScoresPart* p = reinterpret_cast<const ScoresPart*>(a.ws) + m * parts;
  const uint64_t* keys = reinterpret_cast<const uint64_t*>(reinterpret_cast<const ScoresPart*>(a.ws) + a.M * parts) + m * parts * a.k;
  if (threadIdx.x == 0) c.n = 0;
  __syncthreads();
  if (a.k) {
    // at least k of the keys reach the least of the parts' q-th, and the largest of their k-th
    const int i = threadIdx.x & 63, q = (a.k + parts - 1) / parts;
    const uint64_t least = ~wave_max_u64(i < parts ? ~keys[(int64_t)i * a.k + q - 1] : 0);
    const uint64_t last = wave_max_u64(i < parts ? keys[(int64_t)i * a.k + a.k - 1] : 0);
    const uint64_t at_least = least > last ? least : last;
    for (int j = threadIdx.x; j < parts * a.k; j += 256) {
      const uint64_t key = keys[j];
      if (key >= at_least && key) c.key[atomicAdd(&c.n, 1)] = key;
    }
  }
  Total r{-FLT_MAX, 0, 0};
  {  // every wave the same
    const int i = threadIdx.x & 63;
    const ScoresPart mine = i < parts ? p[i] : ScoresPart{-FLT_MAX, 0.f, 0, 0};
    r.m = row_max(mine.m);
    const double back = fmax((double)mine.m - r.m, -1e4), f = exp(back);
    r.s = wave_sum(mine.s * f);
    r.t = wave_sum((mine.t + mine.s * back) * f);
  }
  if (a.k) rank_candidates(c, a.k);
  write_scores(a, m, r, given, c.top);
}

namespace {

// Workgroups a row of the sums: their join is a launch of its own, so a row is split only
// where one workgroup takes longer. (A CU forms the sums of 131072 elements in 9 us: 16 x
// 131072 fp32, 20.2 us by a workgroup a row, 14.0 by 16 and a join.)
int parts_of(int64_t M, int64_t V, int cus) {
  if (V <= 65536) return 1;
  const int64_t room = 4 * (int64_t)cus / std::max<int64_t>(M, 1);
  return (int)std::max<int64_t>(1, std::min<int64_t>({room, V / 16384, (int64_t)kMaxParts}));
}
// Up to a row a CU, a workgroup has 1024 threads and twice the loads under way.
bool few_rows(int64_t M, int parts, int cus) { return M <= cus && parts == 1; }

// Threads of a workgroup, and how it goes through its row or part of one.
enum Threads { kRow128, kRow1024, kRowLong, kRowStretches, kRow512 };
constexpr const char* kRowName[] = {"128 threads", "1024 threads", "512 threads, long sums", "512 threads, in stretches", "512 threads"};
constexpr const char* kPartName = "parts of a row, 512 threads";
// (Stretches pay where lines read twice do, many long rows: 2048 x 131072 bf16 125.5 us
// without, 111 with them, fp32 1024 x 131072 119 and 102; 4096 x 8000 49 and 54, 16 x 131072
// 13.2 and 14.7. Threads: 4096 x 1000 17 us by 128, 50 by 512; 77 x 30011 11.5 by 1024, 10.5 by
// 512, 200 x 65000 15.5 and 16.1. Both sums in one kernel: fp32's would not fit 64 registers.)
Threads row_of(int64_t M, int64_t V, int64_t k, int parts, int cus) {
  if (V <= 4096) return kRow128;
  if (few_rows(M, parts, cus)) return kRow1024;
  if (V / parts > kChain * 512 * 16) return kRowLong;
  return k > 0 && M > cus && V > 32768 ? kRowStretches : kRow512;
}

template <int TYPE, bool TOP>
hipError_t scores(const ScoresArgs& a, int cus, hipStream_t stream) {
  const int parts = parts_of(a.M, a.V, cus);
  constexpr int S = TOP ? 4 : 1;
  const dim3 grid((unsigned)(a.M * parts));
  hipError_t e;
  switch (row_of(a.M, a.V, a.k, parts, cus)) {
    case kRow128: e = launch_k(scores_kernel<TYPE, 128, 16, TOP, 1>, grid, dim3(128), 0, stream, Ev{}, a, parts); break;
    case kRow1024: e = launch_k(scores_kernel<TYPE, 1024, 32, TOP, 1>, grid, dim3(1024), 0, stream, Ev{}, a, parts); break;
    case kRowLong: e = launch_k(scores_kernel<TYPE, 512, 16, TOP, S, true>, grid, dim3(512), 0, stream, Ev{}, a, parts); break;
    case kRowStretches: e = launch_k(scores_kernel<TYPE, 512, 16, TOP, S>, grid, dim3(512), 0, stream, Ev{}, a, parts); break;
    default: e = launch_k(scores_kernel<TYPE, 512, 16, TOP, 1>, grid, dim3(512), 0, stream, Ev{}, a, parts); break;
  }
  if (e == hipSuccess && parts > 1)
    e = launch_k(scores_join_kernel<TYPE>, dim3((unsigned)a.M), dim3(256), 0, stream, Ev{}, a, parts);
  return e;
}
template <int TYPE>
hipError_t scores(const ScoresArgs& a, int cus, hipStream_t stream) {
  return a.k ? scores<TYPE, true>(a, cus, stream) : scores<TYPE, false>(a, cus, stream);
}

}  // namespace

size_t scores_ws_bytes(int64_t M, int64_t V, int64_t k, int cus) {
  const int parts = parts_of(M, V, cus);
  return parts > 1 ? (size_t)M * parts * (sizeof(ScoresPart) + 8 * (size_t)k) : 0;
}

const char* scores_kernel_name(int64_t M, int64_t V, int64_t k, int cus) {
  const int parts = parts_of(M, V, cus);
  return parts > 1 ? kPartName : kRowName[row_of(M, V, k, parts, cus)];
}

hipError_t launch_scores(const ScoresArgs& a, int cus, hipStream_t stream) {
  return a.type == MOE_FP32   ? scores<MOE_FP32>(a, cus, stream)
         : a.type == MOE_FP16 ? scores<MOE_FP16>(a, cus, stream)
                              : scores<MOE_BF16>(a, cus, stream);
}

// ----------------------------------------------------------------- distillation
// The row's slots in LDS, from the first wave: token (-1 empty, as is one of t = -inf) and p, log p in 64
// bits (the loss of masked logits comes near binary32's largest number).
struct Teacher {
  int32_t id[64];
  double p[64], logp[64];
  int some;  // a slot is filled
};
__device__ void read_teacher(const DistillArgs& a, int64_t m, Teacher& w) {
  if (threadIdx.x < 64) {
    const int j = threadIdx.x;
    int32_t v = j < a.k ? a.ids[m * a.k + j] : -1;
    if (v < 0 || v >= a.V) v = -1;
    const float t = v >= 0 ? a.t[m * a.k + j] : -INFINITY;
    if (t == -INFINITY) v = -1;
    const double d = ((double)t - row_max(t)) / a.temperature;
    const double e = v >= 0 ? exp(d) : 0.0;
    const double s = wave_sum(e);
    w.id[j] = v;
    w.p[j] = v >= 0 ? e / s : 0.0;
    w.logp[j] = d - log(s);
    const bool any = __ballot(v >= 0) != 0;
    if (j == 0) w.some = any;
  }
  __syncthreads();
}

// The loss, and lse where asked for, of a row with these sums; z the logit at the
// thread's slot (first wave).
__device__ __forceinline__ void write_loss(const DistillArgs& a, int64_t m, const Teacher& w, const Total& r, float z) {
  if (threadIdx.x >= 64) return;
  const int j = threadIdx.x;
  const double c = 1.f / a.temperature;
  const bool ok = r.m < INFINITY && r.s > 0;
  const double logs = log(r.s), lse = r.m * c + logs;
  double l = 0;
  if (w.p[j] != 0) l = w.p[j] * (w.logp[j] - (((double)z - r.m) * c - logs));
  l = wave_sum(l);
  if (j == 0) {
    a.loss[m] = !w.some ? 0.f : ok ? (float)l : NAN;
    if (a.lse) a.lse[m] = ok ? (float)lse : r.m == INFINITY ? INFINITY : r.s == 0 ? -INFINITY : NAN;
  }
}
template <int TYPE>
__device__ __forceinline__ float slot_logit(const Row<TYPE>& row, const Teacher& w) {
  return threadIdx.x < 64 && w.id[threadIdx.x] >= 0 ? Logit<TYPE>::load(row.p, w.id[threadIdx.x]) : 0.f;
}

// A row's gradient f exp2((z - shift) cl), zero for a row without a slot (some = 0).
struct Slope {
  float shift, f, cl;
  int some;
  __device__ __forceinline__ float at(float z) const { return some ? f * __builtin_amdgcn_exp2f((z - shift) * cl) : 0.f; }
};

// The gradient at the thread's slot's token, where the logit is z; `mine`: this is the
// first of the token's slots.
__device__ __forceinline__ float slot_grad(const DistillArgs& a, int64_t m, const Teacher& w, const Slope& g, float z, bool& mine) {
  const int j = threadIdx.x;
  double q = 0;
  mine = true;
#pragma unroll 4
  for (int i = 0; i < a.k; ++i)
    if (w.id[i] == w.id[j]) {
      if (i < j) mine = false;
      q += w.p[i];
    }
  return (float)(g.at(z) - a.weight[m] / a.temperature * q);
}

template <bool ONCE>
__device__ __forceinline__ void store16(uint8_t* p, uint4 v) {
  if constexpr (ONCE) __builtin_nontemporal_store(__builtin_bit_cast(v4i, v), reinterpret_cast<v4i*>(p));
  else *reinterpret_cast<uint4*>(p) = v;
}

// A piece's gradients to elements o .. of a row of dz; `vec`: on 16 bytes for whole
// pieces of dz's type. ONCE: past the caches.
template <int GRAD, bool ONCE, int E>
__device__ __forceinline__ void store_grads(uint8_t* out, uint32_t o, bool vec, const float (&g)[E]) {
  if constexpr (GRAD == MOE_FP32) {
    if (vec) store16<ONCE>(out + o * 4, __builtin_bit_cast(uint4, make_float4(g[0], g[1], g[2], g[3])));
    else {
#pragma unroll
      for (int i = 0; i < E; ++i) Logit<GRAD>::store(out, o + i, g[i]);
    }
  } else {
    union {
      uint16_t b[E];
      uint4 q4;
      uint2 q2;
    } s;
#pragma unroll
    for (int i = 0; i < E; ++i) s.b[i] = GRAD == MOE_FP16 ? fp16_bits(g[i]) : bf16_bits(g[i]);
    if (E == 8 && vec) store16<ONCE>(out + o * 2, s.q4);
    else if (E == 4 && ((uintptr_t)(out + o * 2) & 7) == 0) *reinterpret_cast<uint2*>(out + o * 2) = s.q2;
    else {
#pragma unroll
      for (int i = 0; i < E; ++i) reinterpret_cast<uint16_t*>(out)[o + i] = s.b[i];
    }
  }
}
template <int GRAD>
__device__ __forceinline__ uint8_t* grad_row(const DistillArgs& a, int64_t m) {
  return reinterpret_cast<uint8_t*>(a.dz) + m * a.lddz * Logit<GRAD>::kBytes;
}

// Gradients of more bytes are written past the caches, which would not hold them for
// their reader, and the logits' second reading finds more of them there.
constexpr int64_t kOnce = (int64_t)128 << 20;

// The gradient of pieces [p0, p1) of a row (and of the elements outside the pieces).
template <int TYPE, int GRAD, int THREADS>
__device__ void write_grad(const DistillArgs& a, int64_t m, const Row<TYPE>& row, int64_t p0, int64_t p1, bool edges,
                           const Teacher& w, const Slope& g) {
  constexpr int E = Logit<TYPE>::kPiece, NP = 2;
  uint8_t* out = grad_row<GRAD>(a, m);
  // every logit is read before its gradient is written (dz may be z); other workgroups
  // write the slots of other pieces
  float slot = 0.f;
  bool mine = false;
  if (threadIdx.x < 64 && w.id[threadIdx.x] >= 0) {
    const int64_t v = w.id[threadIdx.x], p = (v - row.head) / E;
    if (v < row.head || v >= row.V - row.tail ? edges : p >= p0 && p < p1)
      slot = slot_grad(a, m, w, g, Logit<TYPE>::load(row.p, v), mine);
  }
  const bool at_edge = edges && (int)threadIdx.x < row.edges();
  const float edge = at_edge ? Logit<TYPE>::load(row.p, row.edge(threadIdx.x)) : 0.f;
  __syncthreads();
  if (at_edge) Logit<GRAD>::store(out, row.edge(threadIdx.x), g.at(edge));
  const bool vec = ((uintptr_t)(out + (int64_t)row.head * Logit<GRAD>::kBytes) & 15) == 0;  // dz's pieces lie as z's
  auto pieces = [&](auto once) __attribute__((always_inline)) {
    for (int64_t base = p0; base < p1; base += NP * THREADS) {
      uint4 q[NP];
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        const int64_t p = base + u * THREADS + threadIdx.x;
        if (p < p1) q[u] = row.piece(p);
      }
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        const int64_t p = base + u * THREADS + threadIdx.x;
        if (p >= p1) continue;
        float v[E];
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = g.at(Logit<TYPE>::value(q[u], i));
        store_grads<GRAD, decltype(once)::value>(out, (uint32_t)row.first(p), vec, v);
      }
    }
  };
  if (a.M * a.lddz * Logit<GRAD>::kBytes > kOnce) pieces(std::true_type{});
  else pieces(std::false_type{});
  __syncthreads();
  if (mine) Logit<GRAD>::store(out, w.id[threadIdx.x], slot);
}

template <int TYPE, int THREADS, int N>
__device__ Sums<false> sum_pieces(const Row<TYPE>& row, int64_t p0, int64_t p1, bool edges, float cl) {
  constexpr int E = Logit<TYPE>::kPiece, NP = N / E;
  Sums<false> sums;
  uint4 q[NP];
  auto load = [&](int64_t base) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int64_t p = base + u * THREADS + threadIdx.x;
      q[u] = p < p1 ? row.piece(p) : Logit<TYPE>::none();
    }
  };
  load(p0);
  float edge[1] = {edges && (int)threadIdx.x < row.edges() ? Logit<TYPE>::load(row.p, row.edge(threadIdx.x)) : -INFINITY};
  sums.add(edge, cl);
  auto sum_tiles = [&](auto chain) __attribute__((always_inline)) {
    for (int64_t base = p0; base < p1; base += NP * THREADS) {
      float v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = Logit<TYPE>::value(q[i / E], i % E);
      load(base + NP * THREADS);
      sums.template add<decltype(chain)::value>(v, cl);
    }
  };
  if (THREADS == 128 || p1 - p0 <= kChain * NP * THREADS) sum_tiles(std::false_type{});
  else sum_tiles(std::true_type{});
  return sums;
}

// Forward: a row's sums by `parts` workgroups; with one of them the loss too.
template <int TYPE, int THREADS, int N>
__global__ __launch_bounds__(THREADS) void distill_sums_kernel(const DistillArgs a, int parts) {
  __shared__ Teacher w;
  const int64_t m = blockIdx.x / parts;
  const int part = blockIdx.x % parts;
  const float cl = 1.f / a.temperature * kLog2e;
  const Row<TYPE> row(a.z, m, a.ldz, a.V);
  const int64_t per = (row.pieces + parts - 1) / parts;
  const int64_t p0 = min(per * part, row.pieces), p1 = min(p0 + per, row.pieces);
  const Total r = join<THREADS>(sum_pieces<TYPE, THREADS, N>(row, p0, p1, part == 0, cl), cl);
  if (parts == 1) {
    read_teacher(a, m, w);
    write_loss(a, m, w, r, slot_logit(row, w));
  } else if (threadIdx.x == 0) {
    reinterpret_cast<ScoresPart*>(a.ws)[blockIdx.x] = {r.m, 0.f, r.s, 0};
  }
}

__device__ Total joined(const DistillArgs& a, int64_t row, int parts) {
  const ScoresPart* p = reinterpret_cast<const ScoresPart*>(a.ws) + row * parts;
  const double c = 1.f / a.temperature;
  const int i = threadIdx.x & 63;  // every wave the same
  const float m = i < parts ? p[i].m : -FLT_MAX;
  const float top = row_max(m);
  return {top, wave_sum(i < parts ? p[i].s * exp(((double)m - top) * c) : 0.0), 0};
}

// Forward, the parts' sums joined: the loss.
template <int TYPE>
__global__ __launch_bounds__(64) void distill_loss_kernel(const DistillArgs a, int parts) {
  __shared__ Teacher w;
  const int64_t m = blockIdx.x;
  read_teacher(a, m, w);
  write_loss(a, m, w, joined(a, m, parts), slot_logit(Row<TYPE>(a.z, m, a.ldz, a.V), w));
}

// Largest magnitude of an lse that the gradient is taken from: rounded to 32 bits it is off by
// 2^-18 there, and so is the gradient. Rows past it (small temperatures; rows of nothing
// but the type's lowest number) are summed again, by each of their workgroups.
constexpr float kNearLse = 128.f;

// The gradient from lse (backward), or from the parts' sums.
template <int TYPE, int GRAD, int THREADS, bool SUMS>
__global__ __launch_bounds__(THREADS) void distill_grad_kernel(const DistillArgs a, int parts) {
  __shared__ Teacher w;
  const int64_t m = blockIdx.x / parts;
  const int part = blockIdx.x % parts;
  const float c = 1.f / a.temperature;
  const Row<TYPE> row(a.z, m, a.ldz, a.V);
  const int64_t per = (row.pieces + parts - 1) / parts;
  const int64_t p0 = min(per * part, row.pieces), p1 = min(p0 + per, row.pieces);
  read_teacher(a, m, w);
  const float lse = SUMS ? 0.f : a.lse[m];
  float shift, f = a.weight[m] * c;
  if (!SUMS && fabsf(lse) <= kNearLse) {
    // exp(c z - lse) = exp(c (z - shift)) r with shift = lse T rounded
    shift = lse * a.temperature;
    f *= expf(__builtin_fmaf(shift, c, -lse));
  } else {
    Total r{};
    if constexpr (SUMS) r = joined(a, m, parts);
    else if (w.some) r = join<THREADS>(sum_pieces<TYPE, THREADS, 16>(row, 0, row.pieces, true, c * kLog2e), c * kLog2e);
    shift = r.m;
    f = r.m < INFINITY && r.s > 0 ? (float)(f / r.s) : NAN;
  }
  write_grad<TYPE, GRAD, THREADS>(a, m, row, p0, p1, part == 0, w, Slope{shift, f, c * kLog2e, w.some});
}

// Forward and backward: a row a workgroup.
template <int TYPE, int GRAD, int THREADS>
__global__ __launch_bounds__(THREADS) void distill_both_kernel(const DistillArgs a) {
  __shared__ Teacher w;
  const int64_t m = blockIdx.x;
  const float c = 1.f / a.temperature, cl = c * kLog2e;
  const Row<TYPE> row(a.z, m, a.ldz, a.V);
  const Total r = join<THREADS>(sum_pieces<TYPE, THREADS, 16>(row, 0, row.pieces, true, cl), cl);
  read_teacher(a, m, w);
  write_loss(a, m, w, r, slot_logit(row, w));
  const float f = r.m < INFINITY && r.s > 0 ? (float)(a.weight[m] * c / r.s) : NAN;
  write_grad<TYPE, GRAD, THREADS>(a, m, row, 0, row.pieces, true, w, Slope{r.m, f, cl, w.some});
}

// The same for rows of at most 1024 H pieces, which the threads hold between the sums
// and the gradient: every logit is read once. A workgroup takes rows one after another
// and loads a piece of the next as soon as that piece's gradient is on its way, and sums
// it `lag` pieces later, so that memory is not left idle for a row's sums. Bound by memory:
// 2048 x 131072 bf16 228 us, 2048 x 32000 fp32 107 with its second launch (4.7 and 4.9
// TB/s; with accesses through the caches 251 and 118). dz's elements have z's size and
// its rows z's alignment. The rows' sums and their logits at the slots go to the
// workspace for distill_finish_kernel, which writes the loss and the gradient at the
// slots: 64-bit functions here left no registers for the pieces.
__device__ __forceinline__ float* slot_logits(const DistillArgs& a, int64_t m) {
  return reinterpret_cast<float*>(reinterpret_cast<ScoresPart*>(a.ws) + a.M) + m * kMaxTop;
}

template <int TYPE, int GRAD, int H>
__global__ __launch_bounds__(1024, H <= 8 ? 8 : 4) void distill_held_kernel(const DistillArgs a) {
  constexpr int E = Logit<TYPE>::kPiece, G = 16 / E, W = 16;  // pieces summed at a time, waves
  static_assert(H % G == 0, "whole groups");
  __shared__ float lm[W];
  __shared__ double ls[W];
  __shared__ int some;
  const float c = 1.f / a.temperature, cl = c * kLog2e;
  const int wave = wave_id(), lane = threadIdx.x & 63;
  uint4 q[H];
  uint32_t tid = threadIdx.x;
  // Offsets are formed anew for every row, and the pieces' values for the sums and
  // again for the gradient: kept over either they would not fit the registers.
  auto fresh = [](uint4& p) __attribute__((always_inline)) { asm volatile("" : "+v"(p.x), "+v"(p.y), "+v"(p.z), "+v"(p.w)); };
  auto load = [&](const Row<TYPE>& row, int h) __attribute__((always_inline)) {
    const uint32_t p = h * 1024 + tid;
    const v4i* from = reinterpret_cast<const v4i*>(row.p + row.head * Logit<TYPE>::kBytes + p * 16u);
    q[h] = p < (uint32_t)row.pieces ? __builtin_bit_cast(uint4, __builtin_nontemporal_load(from)) : Logit<TYPE>::none();
  };
  Sums<false, true> sums;
  float edge;
  auto begin = [&](const Row<TYPE>& row) __attribute__((always_inline)) {
    asm volatile("" : "+v"(tid));
    edge = (int)tid < row.edges() ? Logit<TYPE>::load(row.p, row.edge(tid)) : -INFINITY;
    sums = Sums<false, true>{};
  };
  auto add = [&](const Row<TYPE>& row, int h) __attribute__((always_inline)) {  // pieces h .. h + G - 1
    if (row.pieces <= h * 1024) return;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      // (after the last group's sums: else all groups' values come first)
      asm volatile("" : "+v"(q[h + i].x), "+v"(q[h + i].y), "+v"(q[h + i].z), "+v"(q[h + i].w), "+v"(sums.s), "+v"(sums.m));
    }
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = Logit<TYPE>::value(q[h + i / E], i % E);
    sums.add(v, cl);
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int lag = 4;
  static_assert(lag % G == 0, "whole groups");
  {
    const Row<TYPE> row(a.z, blockIdx.x, a.ldz, a.V);
#pragma unroll
    for (int h = 0; h < H; ++h) load(row, h);
    begin(row);
#pragma unroll
    for (int h = 0; h < H - lag; h += G) add(row, h);
  }
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const Row<TYPE> row(a.z, m, a.ldz, a.V);
    if (threadIdx.x < 64) {
      int32_t id = -1;
      if (lane < a.k) {
        const int64_t at = m * a.k + lane;
        if (a.t[at] != -INFINITY) id = a.ids[at];
      }
      const bool in = id >= 0 && id < a.V;
      if (in) slot_logits(a, m)[lane] = Logit<TYPE>::load(row.p, id);
      const bool any = __ballot(in) != 0;
      if (lane == 0) some = any;
    }
#pragma unroll
    for (int h = H - lag; h < H; h += G) add(row, h);
    const float last[1] = {edge};
    sums.add(last, cl);
    // the sums of the threads, in 64 bits
    float top = row_max(sums.m);
    if (lane == 0) lm[wave] = top;
    __syncthreads();
    top = row_max(lm[lane % W]);
    const float part = sums.s * __builtin_amdgcn_exp2f(fmaxf((sums.m - top) * cl, -1e4f));
    const double ws = wave_sum((double)part);
    if (lane == 0) ls[wave] = ws;
    __syncthreads();
    const double s = wave_sum(lane < W ? ls[lane] : 0.0);
    if (threadIdx.x == 0) reinterpret_cast<ScoresPart*>(a.ws)[m] = {top, 0.f, s, 0};
    const Slope g{top, top < INFINITY && s > 0 ? (float)(a.weight[m] * c / s) : NAN, cl, some};
    uint8_t* out = grad_row<GRAD>(a, m);
    asm volatile("" : "+v"(tid));
    if ((int)tid < row.edges()) Logit<GRAD>::store(out, row.edge(tid), g.at(edge));
    const int64_t mn = m + gridDim.x;
    const Row<TYPE> next(a.z, mn < a.M ? mn : m, a.ldz, mn < a.M ? a.V : 0);
    begin(next);
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const uint32_t p = h * 1024 + tid;
      fresh(q[h]);
      if (p < (uint32_t)row.pieces) {
        float v[E];
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = g.at(Logit<TYPE>::value(q[h], i));
        store_grads<GRAD, true>(out + row.head * Logit<GRAD>::kBytes, p * (uint32_t)E, true, v);
      }
      load(next, h);
      __builtin_amdgcn_sched_barrier(0);
      if (h >= lag && (h + 1) % G == 0) add(next, h + 1 - G - lag);
    }
    __syncthreads();  // (all have read `some`)
  }
}

// A row a wave: the loss, and the gradient at the slots over what stands there.
template <int TYPE, int GRAD>
__global__ __launch_bounds__(64) void distill_finish_kernel(const DistillArgs a) {
  __shared__ Teacher w;
  const int64_t m = blockIdx.x;
  const int j = threadIdx.x;
  const ScoresPart r = reinterpret_cast<const ScoresPart*>(a.ws)[m];
  const float c = 1.f / a.temperature;
  read_teacher(a, m, w);
  const float z = w.id[j] >= 0 ? slot_logits(a, m)[j] : 0.f;
  write_loss(a, m, w, Total{r.m, r.s, 0}, z);
  if (w.id[j] < 0) return;
  const Slope g{r.m, r.m < INFINITY && r.s > 0 ? (float)(a.weight[m] * c / r.s) : NAN, c * kLog2e, w.some};
  bool mine;
  const float v = slot_grad(a, m, w, g, z, mine);
  if (mine) Logit<GRAD>::store(grad_row<GRAD>(a, m), w.id[j], v);
}

namespace {

// Workgroups a row of the gradient, which needs no join: while the chip has room for
// them (four of 512 threads a CU), a tile's elements each at least.
int grad_parts(int64_t M, int64_t V, int cus) {
  const int64_t room = 4 * (int64_t)cus / std::max<int64_t>(M, 1);
  return (int)std::max<int64_t>(1, std::min<int64_t>({room, V / 8192, (int64_t)kMaxParts}));
}

// How forward and backward at once go: kAlone, a row a workgroup, which reads it twice
// (the second time from the L2 or the memory-side cache); kHeld, the row held between; kSplit, as the two calls
// but with the sums in full. (bf16: 16 x 131072 14.2 us split, 24.3 alone, 100 rows 26.0 and 28.6;
// 2048 x 131072 231 held, 264 alone; 2048 x 32768 67.7 and 68.1, 4096 x 18000 95 and 77; 300 x
// 131072, which is two rounds, 61 and 46.)
enum Both { kAlone, kHeld, kSplit };
Both choose_both(int64_t M, int64_t V, int type, bool alike, int cus) {
  const int64_t bytes = V * (type == MOE_FP32 ? 4 : 2), kb = 1024;
  if (2 * M <= cus && V > 65536) return kSplit;
  // held: rounds of rows over the workgroups that are at most an eighth empty
  const int64_t room = bytes <= 128 * kb ? 2 * cus : cus, rounds = (M + room - 1) / room;
  return alike && bytes > 64 * kb && bytes <= 256 * kb && rounds * room * 7 <= M * 8 ? kHeld : kAlone;
}

template <int TYPE, int GRAD>
hipError_t distill(DistillPass pass, const DistillArgs& a, int cus, hipStream_t stream) {
  const bool small = a.V <= 4096;
  // (over z itself no workgroup may read what another one writes: rows are not split)
  const int gparts = pass == kDistillBackward && a.dz == a.z ? 1 : grad_parts(a.M, a.V, cus);
  const dim3 rows((unsigned)a.M), grads((unsigned)(a.M * gparts));
  if (pass == kDistillBackward)
    return small ? launch_k(distill_grad_kernel<TYPE, GRAD, 128, false>, grads, dim3(128), 0, stream, Ev{}, a, gparts)
                 : launch_k(distill_grad_kernel<TYPE, GRAD, 512, false>, grads, dim3(512), 0, stream, Ev{}, a, gparts);
  int parts = parts_of(a.M, a.V, cus);
  const bool few = few_rows(a.M, parts, cus);
  if (pass == kDistillBoth) {
    constexpr bool same = Logit<TYPE>::kBytes == Logit<GRAD>::kBytes;
    const bool alike = same && (((uintptr_t)a.z - (uintptr_t)a.dz) & 15) == 0 &&
                       (a.ldz - a.lddz) * Logit<TYPE>::kBytes % 16 == 0;
    const Both how = choose_both(a.M, a.V, a.type, alike, cus);
    if constexpr (same) {
      if (how == kHeld) {
        const bool half = a.V * Logit<TYPE>::kBytes <= 128 * 1024;
        // (as many workgroups as fit at once)
        const dim3 grid((unsigned)std::min<int64_t>(a.M, half ? 2 * cus : cus));
        const hipError_t e = half ? launch_k(distill_held_kernel<TYPE, GRAD, 8>, grid, dim3(1024), 0, stream, Ev{}, a)
                                  : launch_k(distill_held_kernel<TYPE, GRAD, 16>, grid, dim3(1024), 0, stream, Ev{}, a);
        return e != hipSuccess ? e : launch_k(distill_finish_kernel<TYPE, GRAD>, rows, dim3(64), 0, stream, Ev{}, a);
      }
    }
    if (how == kAlone)
      return small ? launch_k(distill_both_kernel<TYPE, GRAD, 128>, rows, dim3(128), 0, stream, Ev{}, a)
             : few || a.V > 32768 ? launch_k(distill_both_kernel<TYPE, GRAD, 1024>, rows, dim3(1024), 0, stream, Ev{}, a)
                 : launch_k(distill_both_kernel<TYPE, GRAD, 512>, rows, dim3(512), 0, stream, Ev{}, a);
    parts = std::max(gparts, 2);  // (more than 65536 elements, eight rooms a row: gparts is 8 at least)
  }
  const dim3 grid((unsigned)(a.M * parts));
  hipError_t e = small ? launch_k(distill_sums_kernel<TYPE, 128, 16>, grid, dim3(128), 0, stream, Ev{}, a, parts)
                 : few && pass == kDistillForward
                     ? launch_k(distill_sums_kernel<TYPE, 1024, 32>, grid, dim3(1024), 0, stream, Ev{}, a, parts)
                     : launch_k(distill_sums_kernel<TYPE, 512, 16>, grid, dim3(512), 0, stream, Ev{}, a, parts);
  if (e == hipSuccess && parts > 1) e = launch_k(distill_loss_kernel<TYPE>, rows, dim3(64), 0, stream, Ev{}, a, parts);
  if (e == hipSuccess && pass == kDistillBoth)
    e = launch_k(distill_grad_kernel<TYPE, GRAD, 512, true>, grid, dim3(512), 0, stream, Ev{}, a, parts);
  return e;
}

}  // namespace

size_t distill_ws_bytes(int64_t M, int64_t V, int type, int cus) {
  if (M == 0) return 0;
  size_t n = 0;  // bytes a row
  auto need = [&](size_t bytes) { n = std::max(n, bytes); };
  const int parts = parts_of(M, V, cus);
  if (parts > 1) need(parts * sizeof(ScoresPart));
  const Both how = choose_both(M, V, type, true, cus);
  if (how == kSplit) need(std::max(grad_parts(M, V, cus), 2) * sizeof(ScoresPart));
  if (how == kHeld) need(sizeof(ScoresPart) + kMaxTop * sizeof(float));
  return (size_t)M * n;
}

const char* distill_kernel_name(DistillPass pass, int64_t M, int64_t V, int type, int grad_type, int cus) {
  const int parts = pass == kDistillBackward ? grad_parts(M, V, cus) : parts_of(M, V, cus);
  const bool few = few_rows(M, parts, cus);
  if (pass == kDistillBoth) {
    const bool same = (type == MOE_FP32) == (grad_type == MOE_FP32);
    const Both how = choose_both(M, V, type, same, cus);
    if (how == kHeld) return "rows held in registers";
    if (how == kSplit) return kPartName;
    return kRowName[V <= 4096 ? kRow128 : few || V > 32768 ? kRow1024 : kRow512];
  }
  if (parts > 1) return kPartName;
  return kRowName[V <= 4096 ? kRow128 : few && pass == kDistillForward ? kRow1024 : kRow512];
}

hipError_t launch_distill(DistillPass pass, const DistillArgs& a, int cus, hipStream_t stream) {
  switch (a.type) {
    case MOE_FP32:
      return a.grad_type == MOE_FP32   ? distill<MOE_FP32, MOE_FP32>(pass, a, cus, stream)
             : a.grad_type == MOE_FP16 ? distill<MOE_FP32, MOE_FP16>(pass, a, cus, stream)
                                       : distill<MOE_FP32, MOE_BF16>(pass, a, cus, stream);
    case MOE_FP16:
      return a.grad_type == MOE_FP16 ? distill<MOE_FP16, MOE_FP16>(pass, a, cus, stream)
                                     : distill<MOE_FP16, MOE_BF16>(pass, a, cus, stream);
    default:
      return a.grad_type == MOE_FP16 ? distill<MOE_BF16, MOE_FP16>(pass, a, cus, stream)
                                     : distill<MOE_BF16, MOE_BF16>(pass, a, cus, stream);
  }
}

}  // namespace qmoe
