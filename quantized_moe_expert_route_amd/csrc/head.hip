// What reads the output head's logits: scores of given tokens (log probability,
// entropy, largest alternatives) and distillation from a teacher's top logits.
//
// One pass over a row forms, a thread over its elements and the threads at the end,
//   m = max z, s = sum exp(c (z - m)), t = sum exp(c (z - m)) c (z - m)
// (c = 1 / temperature), the sums moved on by exp(c (m_old - m)) whenever m grows, so
//   lse = c m + log s,  entropy = log s - t / s.
// m starts at the type's lowest number, not at -inf: a row (or thread) of nothing but
// -inf has s = 0 and no NaN. A NaN or +inf makes s NaN. Sums of a thread are binary32,
// those over threads and what follows binary64.
#include <float.h>

#include <algorithm>

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
  __device__ __forceinline__ uint4 piece(int64_t i) const { return ld16(p + head * Logit<TYPE>::kBytes + i * 16); }
  __device__ __forceinline__ int64_t first(int64_t i) const { return head + i * Logit<TYPE>::kPiece; }  // its first element
  __device__ __forceinline__ int edges() const { return head + tail; }  // elements outside the pieces,
  __device__ __forceinline__ int64_t edge(int i) const { return i < head ? i : V - edges() + i; }  // the i-th of them
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// ----------------------------------------------------------------- sums of a row
template <bool MEAN>
struct Sums {
  float m = -FLT_MAX, s = 0.f, t = 0.f;
  // N elements, in units of 1 / cl (cl = c log2 e: t is in log2 units)
  template <int N>
  __device__ __forceinline__ float add(const float (&v)[N], float cl) {
    float top = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, v[i]);
    // (a factor is 0 long before -1e4; no infinity, which zero sums would turn into NaN)
    const float mn = fmaxf(m, top), back = fmaxf((m - mn) * cl, -1e4f), f = __builtin_amdgcn_exp2f(back);
    if constexpr (MEAN) t = (t + s * back) * f;
    s *= f;
    m = mn;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = (v[i] - m) * cl, e = __builtin_amdgcn_exp2f(d);
      s += e;
      if constexpr (MEAN) t += e * fmaxf(d, -1e4f);
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
  float m = wave_max(a.m);
  if (lane == 0) lm[wave] = m;
  __syncthreads();
  m = lm[0];
#pragma unroll
  for (int w = 1; w < W; ++w) m = fmaxf(m, lm[w]);
  const float back = fmaxf((a.m - m) * cl, -1e4f);
  const double f = __builtin_amdgcn_exp2f(back);
  double s = a.s * f, t = 0;
  if constexpr (MEAN) t = ((double)a.t + (double)a.s * back) * f;
  s = wave_sum(s);
  if constexpr (MEAN) t = wave_sum(t);
  if (lane == 0) ls[wave] = s, lt[wave] = t;
  __syncthreads();
  s = t = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) s += ls[w], t += lt[w];
  return {m, s, t * 0.69314718055994531};
}

// ----------------------------------------------------------------- the k largest
// Keys order elements by value, then by falling id. Candidates are collected in LDS
// while they reach a threshold below which no element can be among the k largest.
__device__ __forceinline__ uint64_t key_of(float v, int64_t id) {
  return ((uint64_t)order_key(v) << 32) | (uint32_t)~(uint32_t)id;
}

constexpr int kKeys = 2048;  // candidates held
struct Candidates {
  uint64_t key[kKeys];
  uint64_t at_least;  // the threshold
  uint64_t wave[16];
  int n;              // candidates met; those past kKeys are not held
};

// The threshold that a tile's best elements give, `best` a thread's: every wave has q
// threads at or above its q-th best, all waves together at least k above the least of
// these.
template <int THREADS>
__device__ __forceinline__ void raise_threshold(Candidates& c, uint64_t best, int k) {
  constexpr int W = THREADS / 64;
  const int q = (k + W - 1) / W;
  uint64_t at = 0;
  for (int i = 0; i < q; ++i) {
    at = wave_max_u64(best);
    if (best == at) best = 0;  // keys differ, but for 0
  }
  if ((threadIdx.x & 63) == 0) c.wave[wave_id()] = at;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < W; ++w) at = c.wave[w] < at ? c.wave[w] : at;
    if (at > c.at_least) c.at_least = at;
  }
  __syncthreads();
}

// The candidates held, largest first, c.n of them at most k; the threshold is the k-th.
template <int THREADS>
__device__ void sort_candidates(Candidates& c, int k) {
  __syncthreads();
  const int n = min(c.n, kKeys);
  int size = 2;
  while (size < n) size *= 2;
  for (int i = n + threadIdx.x; i < size; i += THREADS) c.key[i] = 0;
  __syncthreads();
  for (int run = 2; run <= size; run *= 2)
    for (int step = run / 2; step > 0; step /= 2) {
      for (int i = threadIdx.x; i < size / 2; i += THREADS) {
        const int lo = (i / step) * 2 * step + i % step, hi = lo + step;
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

// A thread's N elements v with ids first .. as candidates; those of `left` that found
// no room stay in it.
template <int N>
__device__ __forceinline__ void offer(Candidates& c, const float (&v)[N], int64_t first, uint32_t& left) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!(left >> i & 1)) continue;
    const uint64_t key = key_of(v[i], first + i);
    if (key >= c.at_least) {
      if (c.n > kKeys) continue;
      const int at = atomicAdd(&c.n, 1);
      if (at >= kKeys) continue;
      c.key[at] = key;
    }
    left &= ~(1u << i);
  }
}

// The k largest of a segment again, for rows whose candidates were more than fit: the
// threshold is raised by every tile, and whenever the candidates are full they are
// sorted and all but k dropped.
template <int TYPE, int THREADS>
__device__ void reselect(Candidates& c, const Row<TYPE>& row, int64_t p0, int64_t p1, bool edges, int k) {
  constexpr int E = Logit<TYPE>::kPiece;
  __syncthreads();
  if (threadIdx.x == 0) c.n = 0, c.at_least = 0;
  __syncthreads();
  for (int64_t base = edges ? p0 - THREADS : p0; base < p1; base += THREADS) {
    float v[E];
    uint32_t left = 0;
    int64_t first = 0;
    if (base < p0) {  // the elements outside the pieces
      const bool in = (int)threadIdx.x < row.edges();
      first = row.edge(in ? threadIdx.x : 0);
      v[0] = in ? Logit<TYPE>::load(row.p, first) : 0.f;
#pragma unroll
      for (int i = 1; i < E; ++i) v[i] = 0.f;
      left = in;
    } else {
      const int64_t p = base + threadIdx.x;
      const uint4 q = row.piece(p < p1 ? p : p0);
      first = row.first(p);
      left = p < p1 ? (1u << E) - 1 : 0;
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = Logit<TYPE>::value(q, i);
    }
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (left >> i & 1) {
        const uint64_t key = key_of(v[i], first + i);
        best = key > best ? key : best;
      }
    raise_threshold<THREADS>(c, best, k);
    for (;;) {
      offer(c, v, first, left);
      __syncthreads();
      const bool full = c.n >= kKeys;
      __syncthreads();
      if (!full) break;
      sort_candidates<THREADS>(c, k);
    }
  }
}

// ----------------------------------------------------------------- scores
// A segment of a row a workgroup. Few rows are split over `parts` workgroups, whose
// sums and k keys go to the workspace and are joined by scores_join_kernel.
struct ScoresPart {
  float m;
  float pad;
  double s, t;
};

__device__ void write_scores(const ScoresArgs& a, int64_t m, const Total& r, float given, const Candidates& c) {
  const bool ok = r.m < INFINITY && r.s > 0;  // not NaN either
  const double logs = log(r.s), lse = r.m + logs;
  if (threadIdx.x == 0) {
    if (a.tokens) {
      const int64_t t = a.tokens[m];
      a.logprobs[m] = ok && t >= 0 && t < a.V ? (float)(given - lse) : NAN;
    }
    if (a.entropy) a.entropy[m] = ok ? (float)(logs - r.t / r.s) : NAN;
    if (a.lse) a.lse[m] = ok ? (float)lse : r.m == INFINITY ? INFINITY : r.s == 0 ? -INFINITY : NAN;
  }
  for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
    const uint64_t key = c.key[j];
    a.top_ids[m * a.k + j] = (int32_t)~(uint32_t)key;
    a.top_logprobs[m * a.k + j] = ok ? (float)(key_to_float((uint32_t)(key >> 32)) - lse) : NAN;
  }
}

template <int TYPE>
__device__ __forceinline__ float given_logit(const ScoresArgs& a, const Row<TYPE>& row, int64_t m) {
  const int64_t t = a.tokens ? a.tokens[m] : -1;
  return t >= 0 && t < a.V ? Logit<TYPE>::load(row.p, t) : 0.f;
}

template <int TYPE, int THREADS, bool TOP>
__global__ __launch_bounds__(THREADS) void scores_kernel(const ScoresArgs a, int parts) {
  constexpr int E = Logit<TYPE>::kPiece, NP = 16 / E, N = NP * E;  // pieces, elements a thread and tile
  __shared__ Candidates c;
  const int64_t m = blockIdx.x / parts;
  const int part = blockIdx.x % parts;
  const Row<TYPE> row(a.z, m, a.ldz, a.V);
  const int64_t per = (row.pieces + parts - 1) / parts;
  const int64_t p0 = min(per * part, row.pieces), p1 = min(p0 + per, row.pieces);
  const bool edges = part == 0;
  const float given = parts == 1 ? given_logit<TYPE>(a, row, m) : 0.f;
  if (TOP && threadIdx.x == 0) c.n = 0, c.at_least = 0;
  Sums<true> sums;

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
  sums.add(edge, kLog2e);
  for (int64_t base = p0; base < p1 || base == p0; base += NP * THREADS) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = Logit<TYPE>::value(q[i / E], i % E);
    load(base + NP * THREADS);
    const float top = sums.add(v, kLog2e);
    if constexpr (TOP) {
      if (base == p0) {
        uint64_t best = edges && (int)threadIdx.x < row.edges() ? key_of(edge[0], row.edge(threadIdx.x)) : 0;
#pragma unroll
        for (int u = 0; u < NP; ++u) {
          const int64_t p = base + u * THREADS + threadIdx.x;
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const uint64_t key = p < p1 ? key_of(v[u * E + i], row.first(p) + i) : 0;
            best = key > best ? key : best;
          }
        }
        raise_threshold<THREADS>(c, best, a.k);
        uint32_t left = edges && (int)threadIdx.x < row.edges();
        offer(c, edge, row.edge(threadIdx.x), left);
      }
      // (the first tile's NaN raise the threshold, but not `top`; a NaN threshold lets all pass)
      if (base == p0 || !(top < key_to_float((uint32_t)(c.at_least >> 32)))) {
#pragma unroll
        for (int u = 0; u < NP; ++u) {
          const int64_t p = base + u * THREADS + threadIdx.x;
          float w[E];
#pragma unroll
          for (int i = 0; i < E; ++i) w[i] = v[u * E + i];
          uint32_t left = p < p1 ? (1u << E) - 1 : 0;
          offer(c, w, row.first(p), left);
        }
      }
    }
  }
  const Total r = join<THREADS>(sums, kLog2e);  // (its barriers: all candidates are in)
  if constexpr (TOP) {
    if (c.n > kKeys) reselect<TYPE, THREADS>(c, row, p0, p1, edges, a.k);
    sort_candidates<THREADS>(c, a.k);
  }
  if (parts == 1) {
    write_scores(a, m, r, given, c);
    return;
  }
  if (threadIdx.x == 0) reinterpret_cast<ScoresPart*>(a.ws)[blockIdx.x] = {r.m, 0.f, r.s, r.t};
  uint64_t* keys = reinterpret_cast<uint64_t*>(reinterpret_cast<ScoresPart*>(a.ws) + a.M * parts) + (int64_t)blockIdx.x * a.k;
  for (int j = threadIdx.x; j < a.k; j += THREADS) keys[j] = j < c.n ? c.key[j] : 0;
}

constexpr int kMaxParts = 32;
static_assert(kMaxParts * kMaxTop <= kKeys, "the parts' keys are sorted at once");

template <int TYPE>
__global__ __launch_bounds__(256) void scores_join_kernel(const ScoresArgs a, int parts) {
  __shared__ Candidates c;
  const int64_t m = blockIdx.x;
  const Row<TYPE> row(a.z, m, a.ldz, a.V);
  const float given = given_logit<TYPE>(a, row, m);
  const ScoresPart* p = reinterpret_cast<const ScoresPart*>(a.ws) + m * parts;
  const uint64_t* keys = reinterpret_cast<const uint64_t*>(reinterpret_cast<const ScoresPart*>(a.ws) + a.M * parts) + m * parts * a.k;
  for (int j = threadIdx.x; j < parts * a.k; j += 256) c.key[j] = keys[j];
  if (threadIdx.x == 0) c.n = parts * a.k, c.at_least = 0;
  Total r{-FLT_MAX, 0, 0};
  for (int i = 0; i < parts; ++i) r.m = fmaxf(r.m, p[i].m);
  for (int i = 0; i < parts; ++i) {
    const double back = fmax((double)p[i].m - r.m, -1e4), f = exp(back);
    r.s += p[i].s * f;
    r.t += (p[i].t + p[i].s * back) * f;
  }
  if (a.k) sort_candidates<256>(c, a.k);
  write_scores(a, m, r, given, c);
}

namespace {

// Workgroups a row: the chip has room for four of 512 threads a CU; a part has at least
// a tile's elements.
int parts_of(int64_t M, int64_t V, int cus) {
  const int64_t room = 4 * (int64_t)cus / std::max<int64_t>(M, 1), tiles = V / 8192;
  return (int)std::max<int64_t>(1, std::min<int64_t>({room, tiles, (int64_t)kMaxParts}));
}

template <int TYPE>
hipError_t scores(const ScoresArgs& a, int cus, hipStream_t stream) {
  const int parts = parts_of(a.M, a.V, cus);
  const dim3 grid((unsigned)(a.M * parts));
  hipError_t e;
  if (a.V <= 4096)
    e = a.k ? launch_k(scores_kernel<TYPE, 128, true>, grid, dim3(128), 0, stream, Ev{}, a, parts)
            : launch_k(scores_kernel<TYPE, 128, false>, grid, dim3(128), 0, stream, Ev{}, a, parts);
  else
    e = a.k ? launch_k(scores_kernel<TYPE, 512, true>, grid, dim3(512), 0, stream, Ev{}, a, parts)
            : launch_k(scores_kernel<TYPE, 512, false>, grid, dim3(512), 0, stream, Ev{}, a, parts);
  if (e == hipSuccess && parts > 1)
    e = launch_k(scores_join_kernel<TYPE>, dim3((unsigned)a.M), dim3(256), 0, stream, Ev{}, a, parts);
  return e;
}

}  // namespace

size_t scores_ws_bytes(int64_t M, int64_t V, int64_t k, int, int cus) {
  const int parts = parts_of(M, V, cus);
  return parts > 1 ? (size_t)M * parts * (sizeof(ScoresPart) + 8 * (size_t)k) : 0;
}

hipError_t launch_scores(const ScoresArgs& a, int cus, hipStream_t stream) {
  return a.type == MOE_FP32   ? scores<MOE_FP32>(a, cus, stream)
         : a.type == MOE_FP16 ? scores<MOE_FP16>(a, cus, stream)
                              : scores<MOE_BF16>(a, cus, stream);
}

// ----------------------------------------------------------------- distillation
// The row's slots in LDS, from the first wave: token (-1 empty) and p, log p in 64
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
    const float t = v >= 0 ? a.t[m * a.k + j] / a.temperature : -INFINITY;
    const float mx = wave_max(t);
    const double e = t > -INFINITY || t != t ? exp((double)t - mx) : 0.0;
    const double s = wave_sum(e);
    w.id[j] = v;
    w.p[j] = v >= 0 ? e / s : 0.0;
    w.logp[j] = (double)t - mx - log(s);
    const bool any = __ballot(v >= 0) != 0;
    if (j == 0) w.some = any;
  }
  __syncthreads();
}

// The loss, and lse where asked for, of a row with these sums (first wave).
template <int TYPE>
__device__ void write_loss(const DistillArgs& a, int64_t m, const Row<TYPE>& row, const Teacher& w, const Total& r) {
  if (threadIdx.x >= 64) return;
  const int j = threadIdx.x;
  const double c = 1.f / a.temperature;
  const bool ok = r.m < INFINITY && r.s > 0;
  const double lse = r.m * c + log(r.s);
  double l = 0;
  if (w.p[j] != 0) l = w.p[j] * (w.logp[j] - (Logit<TYPE>::load(row.p, w.id[j]) * c - lse));
  l = wave_sum(l);
  if (j == 0) {
    a.loss[m] = !w.some ? 0.f : ok ? (float)l : NAN;
    if (a.lse) a.lse[m] = ok ? (float)lse : r.m == INFINITY ? INFINITY : r.s == 0 ? -INFINITY : NAN;
  }
}

// Gradient of pieces [p0, p1) of a row (and of the elements outside the pieces):
// f exp2(z cl - at), the teacher's tokens by themselves. Every logit is read before its
// gradient is written (dz may be z).
template <int TYPE, int GRAD, int THREADS>
__device__ void write_grad(const DistillArgs& a, int64_t m, const Row<TYPE>& row, int64_t p0, int64_t p1, bool edges,
                           const Teacher& w, float shift, float f, float cl) {
  constexpr int E = Logit<TYPE>::kPiece;
  uint8_t* out = reinterpret_cast<uint8_t*>(a.dz) + m * a.lddz * Logit<GRAD>::kBytes;
  auto grad = [&](float z) __attribute__((always_inline)) { return f * __builtin_amdgcn_exp2f((z - shift) * cl); };
  // the gradient at a slot's token, by the first of its slots
  float at = 0.f;
  bool mine = false;
  if (threadIdx.x < 64 && w.id[threadIdx.x] >= 0) {
    const int j = threadIdx.x;
    const int64_t v = w.id[j], p = v - row.head;
    mine = v < row.head || v >= row.V - row.tail ? edges : p / E >= p0 && p / E < p1;
    double s = 0;
    for (int i = 0; i < a.k; ++i)
      if (w.id[i] == w.id[j]) {
        if (i < j) mine = false;
        s += w.p[i];
      }
    if (mine) at = (float)(grad(Logit<TYPE>::load(row.p, v)) - a.weight[m] / a.temperature * s);
  }
  const float edge = edges && (int)threadIdx.x < row.edges() ? Logit<TYPE>::load(row.p, row.edge(threadIdx.x)) : 0.f;
  __syncthreads();
  if (edges && (int)threadIdx.x < row.edges()) Logit<GRAD>::store(out, row.edge(threadIdx.x), w.some ? grad(edge) : 0.f);
  const int64_t o0 = row.head;
  const bool vec = ((uintptr_t)(out + o0 * Logit<GRAD>::kBytes) & 15) == 0;  // dz's pieces lie as z's
  constexpr int NP = 2;
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
      float g[E];
#pragma unroll
      for (int i = 0; i < E; ++i) g[i] = w.some ? grad(Logit<TYPE>::value(q[u], i)) : 0.f;
      const int64_t o = row.first(p);
      if constexpr (GRAD == MOE_FP32) {
        if (vec) *reinterpret_cast<float4*>(out + o * 4) = make_float4(g[0], g[1], g[2], g[3]);
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
        if (E == 8 && vec) *reinterpret_cast<uint4*>(out + o * 2) = s.q4;
        else if (E == 4 && ((uintptr_t)(out + o * 2) & 7) == 0) *reinterpret_cast<uint2*>(out + o * 2) = s.q2;
        else {
#pragma unroll
          for (int i = 0; i < E; ++i) reinterpret_cast<uint16_t*>(out)[o + i] = s.b[i];
        }
      }
    }
  }
  __syncthreads();
  if (mine) Logit<GRAD>::store(out, w.id[threadIdx.x], at);
}

template <int TYPE, int THREADS>
__device__ Sums<false> sum_pieces(const Row<TYPE>& row, int64_t p0, int64_t p1, bool edges, float cl) {
  constexpr int E = Logit<TYPE>::kPiece, NP = 16 / E, N = NP * E;
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
  for (int64_t base = p0; base < p1; base += NP * THREADS) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = Logit<TYPE>::value(q[i / E], i % E);
    load(base + NP * THREADS);
    sums.add(v, cl);
  }
  return sums;
}

// Forward: a row's sums by `parts` workgroups; with one of them the loss too.
template <int TYPE, int THREADS>
__global__ __launch_bounds__(THREADS) void distill_sums_kernel(const DistillArgs a, int parts) {
  __shared__ Teacher w;
  const int64_t m = blockIdx.x / parts;
  const int part = blockIdx.x % parts;
  const float cl = 1.f / a.temperature * kLog2e;
  const Row<TYPE> row(a.z, m, a.ldz, a.V);
  const int64_t per = (row.pieces + parts - 1) / parts;
  const int64_t p0 = min(per * part, row.pieces), p1 = min(p0 + per, row.pieces);
  const Total r = join<THREADS>(sum_pieces<TYPE, THREADS>(row, p0, p1, part == 0, cl), cl);
  if (parts == 1) {
    read_teacher(a, m, w);
    write_loss<TYPE>(a, m, row, w, r);
  } else if (threadIdx.x == 0) {
    reinterpret_cast<ScoresPart*>(a.ws)[blockIdx.x] = {r.m, 0.f, r.s, 0};
  }
}

__device__ Total joined(const DistillArgs& a, int64_t m, int parts) {
  const ScoresPart* p = reinterpret_cast<const ScoresPart*>(a.ws) + m * parts;
  Total r{-FLT_MAX, 0, 0};
  const double c = 1.f / a.temperature;
  for (int i = 0; i < parts; ++i) r.m = fmaxf(r.m, p[i].m);
  for (int i = 0; i < parts; ++i) r.s += p[i].s * exp(((double)p[i].m - r.m) * c);
  return r;
}

// Forward, the parts' sums joined: the loss. (PARTS workgroups with the gradient.)
template <int TYPE>
__global__ __launch_bounds__(64) void distill_loss_kernel(const DistillArgs a, int parts) {
  __shared__ Teacher w;
  const int64_t m = blockIdx.x;
  read_teacher(a, m, w);
  write_loss<TYPE>(a, m, Row<TYPE>(a.z, m, a.ldz, a.V), w, joined(a, m, parts));
}

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
  float shift, f = a.weight[m] * c;
  if constexpr (SUMS) {
    const Total r = joined(a, m, parts);
    shift = r.m;
    f = r.m < INFINITY && r.s > 0 ? (float)(f / r.s) : NAN;
  } else {
    // exp(c z - lse) = exp(c (z - shift)) r with shift = lse T rounded
    const float lse = a.lse[m];
    shift = lse * a.temperature;
    f = fabsf(lse) < INFINITY ? f * expf(__builtin_fmaf(shift, c, -lse)) : NAN;
  }
  write_grad<TYPE, GRAD, THREADS>(a, m, row, p0, p1, part == 0, w, shift, f, c * kLog2e);
}

// Forward and backward: a row a workgroup.
template <int TYPE, int GRAD, int THREADS>
__global__ __launch_bounds__(THREADS) void distill_both_kernel(const DistillArgs a) {
  __shared__ Teacher w;
  const int64_t m = blockIdx.x;
  const float c = 1.f / a.temperature, cl = c * kLog2e;
  const Row<TYPE> row(a.z, m, a.ldz, a.V);
  const Total r = join<THREADS>(sum_pieces<TYPE, THREADS>(row, 0, row.pieces, true, cl), cl);
  read_teacher(a, m, w);
  write_loss<TYPE>(a, m, row, w, r);
  const float f = r.m < INFINITY && r.s > 0 ? (float)(a.weight[m] * c / r.s) : NAN;
  write_grad<TYPE, GRAD, THREADS>(a, m, row, 0, row.pieces, true, w, r.m, f, cl);
}

size_t distill_ws_bytes(int64_t M, int64_t V, int, int cus) {
  const int parts = parts_of(M, V, cus);
  return parts > 1 ? (size_t)M * parts * sizeof(ScoresPart) : 0;
}

namespace {

template <int TYPE, int GRAD>
hipError_t distill(DistillPass pass, const DistillArgs& a, int cus, hipStream_t stream) {
  const int parts = parts_of(a.M, a.V, cus);
  const dim3 grid((unsigned)(a.M * parts));
  const bool small = a.V <= 4096;
  const dim3 block(small ? 128 : 512);
  if (pass == kDistillBackward)
    return small ? launch_k(distill_grad_kernel<TYPE, GRAD, 128, false>, grid, block, 0, stream, Ev{}, a, parts)
                 : launch_k(distill_grad_kernel<TYPE, GRAD, 512, false>, grid, block, 0, stream, Ev{}, a, parts);
  if (pass == kDistillBoth && parts == 1)
    return small ? launch_k(distill_both_kernel<TYPE, GRAD, 128>, grid, block, 0, stream, Ev{}, a)
                 : launch_k(distill_both_kernel<TYPE, GRAD, 512>, grid, block, 0, stream, Ev{}, a);
  hipError_t e = small ? launch_k(distill_sums_kernel<TYPE, 128>, grid, block, 0, stream, Ev{}, a, parts)
                       : launch_k(distill_sums_kernel<TYPE, 512>, grid, block, 0, stream, Ev{}, a, parts);
  if (e == hipSuccess && parts > 1)
    e = launch_k(distill_loss_kernel<TYPE>, dim3((unsigned)a.M), dim3(64), 0, stream, Ev{}, a, parts);
  if (e == hipSuccess && pass == kDistillBoth)
    e = launch_k(distill_grad_kernel<TYPE, GRAD, 512, true>, grid, block, 0, stream, Ev{}, a, parts);
  return e;
}

}  // namespace

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
