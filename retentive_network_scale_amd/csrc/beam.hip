// A step of a beam search: the selection of the K best continuations of every request, and the
// reordering of the beams' states (language.h).
//
// Selection takes two launches.  The first reads the logits once: a workgroup keeps a slice of one
// beam's row in registers, leaves the slice's maximum and the sum of the exponentials beside it, and its K best
// logits in order.  To find those, each wave takes the K-th best of its lanes' best values, found bit by
// bit, and the workgroup the largest of these as a bound: at least K elements reach it and few others.
// Those are gathered and ranked by counting, ordered by value and index as one whole number, so that none
// are equal.  Where more reach it than there is room for (rows of equal values), the bound is found again
// from the lanes' best as such whole numbers, which at most K lanes reach.
// The second launch, a workgroup a request, joins the slices' sums to the beams' log-sums and does the
// same with the lists' heads and the lists.
// 64 requests, 8 beams, 32000 bf16 logits (33 MB): 14 us, 2.3 TB/s, and 8 for the second launch, a chain of four
// dependent loads and barriers.  The first is bound by the chain of a slice: load, bound, gather, rank, each waiting
// for the one before; ranking all 256 lanes' best by counting took 29 us.
// A request of few slices takes one launch, whose waves keep a slice each and whose workgroup joins them.
#include <math.h>

#include <algorithm>

#include "language.hpp"

using namespace ret;

namespace {

constexpr int NT = 256;
constexpr int MAXK = LANGUAGE_MAX_BEAMS;
typedef unsigned long long u64;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

struct Cand {
  float value;
  int index;  // in the row; -1: none
};

// A slice's part of its row's log-sum: the maximum m and the sum of exp(x - m) over all other elements.  In a confident
// row these are far below 1 and would be lost beside it.
struct Sum {
  float m, rest;
};

struct SelectArgs {
  const void *logits;
  const float *scores;
  const uint8_t *ended;
  int *tokens, *parents;
  float *out_scores;
  Sum *sums;    // [B W][slices]
  Cand *cands;   // [B W][slices][K], best first
  long long ld;
  int B, W, V, K, eos, slices;
};

// Whole numbers in the order of the values (NaN of either sign at the ends).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ u64 ordered(double v) {
  const u64 b = (u64)__double_as_longlong(v);
  return b ^ ((u64)((long long)b >> 63) | 0x8000000000000000ull);
}
// -0 is 0: the two compare equal, and the index has to decide.
__device__ __forceinline__ u64 key_of(float v, int index) { return (u64)ordered(v + 0.0f) << 32 | (uint32_t)~index; }

// The K-th largest of the lanes' values (K <= 64) as a whole number in their order.
__device__ __forceinline__ uint32_t kth_of_wave(uint32_t mine, int K) {
  uint32_t t = 0;
#pragma unroll
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t c = t | 1u << bit;
    if (__popcll(__ballot(mine >= c)) >= K) t = c;
  }
  return t;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xffffffffu));
}

// Each chunk's maximum in a lane, and the lane's; they pass over NaN, which spoils the sum.
template <int C>
__device__ __forceinline__ float tops_of(const float (&x)[C][8], float (&tops)[C]) {
  float top = -INFINITY;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    tops[c] = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) tops[c] = fmaxf(tops[c], x[c][i]);
    top = fmaxf(top, tops[c]);
  }
  return top;
}
// The wave's part of a slice's sum for the slice's maximum m, less the `same` elements that are m; where m is -inf nothing
// but a NaN shows.  Only a chunk that holds m somewhere in the wave looks for it: 1024 requests, 4 beams, V 32000 take
// 77 us, with a choice for every element and sums in fp64 87.
template <int C>
__device__ __forceinline__ float rest_of_wave(const float (&x)[C][8], const float (&tops)[C], float m, int &same) {
  float s = 0.0f;
  same = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = __builtin_amdgcn_exp2f((x[c][i] - m) * kLog2e);
    if (__any(tops[c] == m))
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool top = x[c][i] == m;
        e[i] = top ? 0.0f : e[i];
        same += __popcll(__ballot(top));
      }
    s += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
  }
  return wave_sum(s);
}
// m and what stands beside it, of all parts: rest, and how many elements are m.
__device__ __forceinline__ Sum sum_of(float m, float rest, int same) {
  return {m, m == -INFINITY ? rest : rest + (float)(same - 1)};
}

// E elements of a row a thread, in E / 8 chunks.
template <typename T, int E>
__global__ __launch_bounds__(NT) void slice_kernel(SelectArgs a) {
  constexpr int CAP = MAXK * E;  // elements that can reach an exact bound: of K - 1 threads with a better one, and one more
  __shared__ u64 list[CAP];
  __shared__ u64 best[NT];
  __shared__ float red[NT / 64];
  __shared__ float rests[NT / 64];
  __shared__ int sames[NT / 64];
  __shared__ uint32_t kth[NT / 64];
  __shared__ u64 bound;
  __shared__ int count;
  const int tid = threadIdx.x, slice = blockIdx.x;
  const long long row = blockIdx.y + (long long)blockIdx.z * 65535;
  if (row >= (long long)a.B * a.W) return;
  // an ended beam and one without a score offer nothing of their logits
  if ((a.ended && a.ended[row]) || !isfinite(a.scores[row])) return;
  const int first = slice * (NT * E);
  const T *src = (const T *)a.logits + row * a.ld;
  float x[E / 8][8];  // -inf behind the row's end
  if (first + NT * E <= a.V) {
#pragma unroll
    for (int c = 0; c < E / 8; ++c) load8(src + first + (c * NT + tid) * 8, x[c]);
  } else {
#pragma unroll
    for (int c = 0; c < E / 8; ++c) {
      const int left = a.V - first - (c * NT + tid) * 8;
      load8(src + first + (c * NT + tid) * 8, left, x[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[c][i] = i < left ? x[c][i] : -INFINITY;
    }
  }
  float tops[E / 8];
  const float top = tops_of(x, tops);
  const uint32_t t = kth_of_wave(ordered(top + 0.0f), a.K);
  float m = top;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if ((tid & 63) == 0) red[tid >> 6] = m, kth[tid >> 6] = t;
  if (tid == 0) bound = 0, count = 0;
  __syncthreads();
  m = red[0];
  uint32_t most = kth[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) m = fmaxf(m, red[w]), most = max(most, kth[w]);
  const float least = value_of(most);
  // gather what reaches the bound
  auto put = [&](u64 k) {
    const int to = atomicAdd(&count, 1);
    if (to < CAP) list[to] = k;
  };
  if (top >= least)
#pragma unroll
    for (int c = 0; c < E / 8; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = first + (c * NT + tid) * 8 + i;
        if (x[c][i] >= least && at < a.V) put(key_of(x[c][i], at));
      }
  int same;
  const float rest = rest_of_wave(x, tops, m, same);
  if ((tid & 63) == 0) rests[tid >> 6] = rest, sames[tid >> 6] = same;
  __syncthreads();  // the list is written too
  int n = count;
  if (n > CAP) {  // the same for all threads
    u64 mine = 0;
#pragma unroll
    for (int c = 0; c < E / 8; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = first + (c * NT + tid) * 8 + i;
        const u64 k = at < a.V ? key_of(x[c][i], at) : 0;
        mine = k > mine ? k : mine;
      }
    best[tid] = mine;
    __syncthreads();
    if (tid == 0) count = 0;
    int rank = 0;
    for (int j = 0; j < NT; ++j) rank += best[j] > mine;
    if (mine && rank == a.K - 1) bound = mine;
    __syncthreads();
    const u64 b = bound;
#pragma unroll
    for (int c = 0; c < E / 8; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = first + (c * NT + tid) * 8 + i;
        if (at < a.V && key_of(x[c][i], at) >= b) put(key_of(x[c][i], at));
      }
    __syncthreads();
    n = count;
  }
  Cand *out = a.cands + (row * a.slices + slice) * a.K;
  for (int e = tid; e < n; e += NT) {
    const u64 k = list[e];
    int r = 0;
    for (int j = 0; j < n; ++j) r += list[j] > k;
    if (r < a.K) out[r] = {value_of((uint32_t)(k >> 32)), (int)~(uint32_t)k};
  }
  for (int e = n + tid; e < a.K; e += NT) out[e] = {0.0f, -1};
  if (tid == 0) {
    float s = 0.0f;
    int every = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) s += rests[w], every += sames[w];
    a.sums[row * a.slices + slice] = sum_of(m, s, every);
  }
}

// A candidate of a request: its score, and what decides between equal ones, the lower beam, then the larger logit, then
// the lower token.  Far from zero many logits have one score (all of a beam's at the type's lowest value), so the
// logit has to be compared itself: a slice's list is in this order only then.
struct Key {
  u64 score, tie;
  static constexpr uint32_t LAST = LANGUAGE_MAX_VOCAB - 1;
  static __device__ __forceinline__ u64 tie_of(int w, float value, int v) {
    return (u64)(MAXK - 1 - w) << 56 | (u64)ordered(value) << 24 | (LAST - v);
  }
  __device__ __forceinline__ int beam() const { return MAXK - 1 - (int)(tie >> 56); }
  __device__ __forceinline__ int token() const { return (int)(LAST - ((uint32_t)tie & LAST)); }
  __device__ __forceinline__ bool above(const Key &o) const {
    return score > o.score || (score == o.score && tie > o.tie);
  }
};
static_assert((Key::LAST & LANGUAGE_MAX_VOCAB) == 0 && LANGUAGE_MAX_VOCAB == 1 << 24, "a token in 24 bits");

// What a workgroup of NTH threads needs to choose a request's K (KM at most) of its lists' candidates.
template <int NTH, int LISTS, int KM>
struct Join {
  double lse[MAXK];
  int kind[MAXK];  // 0: an ordinary beam, 1: ended, 2: nothing to offer
  Key head[LISTS];
  Key list[KM * KM];
  Key bound;
  int count;
};

// Request b, from its lists' sums ([lists]) and candidates ([lists][K]), in memory or in LDS.
template <int NTH, int LISTS, int KM>
__device__ __forceinline__ void join(const SelectArgs &a, long long b, const Sum *sums, const Cand *cands,
                                     Join<NTH, LISTS, KM> &lds) {
  constexpr int CAP2 = KM * KM;
  const int tid = threadIdx.x, lists = a.W * a.slices;
  if (tid == 0) lds.bound = {0, 0}, lds.count = 0;
  // few candidates are all on their way from the start
  constexpr int EACH = 4;
  const bool ahead = lists * a.K <= EACH * NTH;
  Cand own[EACH];
  if (ahead)
#pragma unroll
    for (int u = 0; u < EACH; ++u)
      if (u * NTH + tid < lists * a.K) own[u] = cands[u * NTH + tid];
  // a beam's log-sum by a wave, its slices by the lanes
  for (int w = tid >> 6; w < a.W; w += NTH / 64) {
    const long long row = b * a.W + w;
    const float own = a.scores[row];
    const bool end = a.ended && a.ended[row];
    float m = -INFINITY;
    double s = 0.0;
    int tops = 0;
    if (!end && isfinite(own)) {
      for (int i = tid & 63; i < a.slices; i += 64) m = fmaxf(m, sums[w * a.slices + i].m);
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
      for (int i = tid & 63; i < a.slices; i += 64) {
        const Sum v = sums[w * a.slices + i];
        tops += v.m == m;
        // a slice of nothing but -inf adds its sum, 0 or NaN
        s += v.m == m || v.m == -INFINITY ? (double)v.rest : (1.0 + (double)v.rest) * exp((double)v.m - (double)m);
      }
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, 64), tops += __shfl_xor(tops, off, 64);
    }
    if ((tid & 63) == 0) {
      const double l = (double)m + log1p(s + (tops - 1));
      lds.lse[w] = l;
      lds.kind[w] = !isfinite(own) ? 2 : end ? 1 : isfinite(l) ? 0 : 2;
    }
  }
  __syncthreads();
  // Candidate j of a list as a key; {0, 0}: none
  auto key_of_cand = [&](int list, int j, const Cand &c) -> Key {
    const int w = list / a.slices, slice = list - w * a.slices;
    const long long row = b * a.W + w;
    int v;
    float value = 0.0f;
    double score;
    if (lds.kind[w] == 0) {
      if (c.index < 0) return {0, 0};
      v = c.index;
      value = c.value;
      score = (double)a.scores[row] + ((double)c.value - lds.lse[w]);
    } else {
      // the tokens in their order, after the end token where the beam has ended: in the first list
      if (slice) return {0, 0};
      const bool end = lds.kind[w] == 1 && a.eos >= 0 && a.eos < a.V;
      v = !end ? j : j == 0 ? a.eos : j - 1 < a.eos ? j - 1 : j;
      if (v >= a.V) return {0, 0};
      score = end && j == 0 ? (double)a.scores[row] : -INFINITY;
    }
    return {ordered(score + 0.0), Key::tie_of(w, value, v)};
  };
  auto key_at = [&](int list, int j) { return key_of_cand(list, j, cands[list * a.K + j]); };
  Key mine[EACH];
  if (ahead) {
#pragma unroll
    for (int u = 0; u < EACH; ++u) {
      const int e = u * NTH + tid, l = e / a.K, j = e - l * a.K;
      mine[u] = {0, 0};
      if (e < lists * a.K) {
        mine[u] = key_of_cand(l, j, own[u]);
        if (j == 0) lds.head[l] = mine[u];
      }
    }
  } else {
    for (int l = tid; l < lists; l += NTH) lds.head[l] = key_at(l, 0);
  }
  __syncthreads();
  for (int l = tid; l < lists; l += NTH) {
    const Key k = lds.head[l];
    if (!k.score) continue;
    int r = 0;
    for (int j = 0; j < lists; ++j) r += lds.head[j].above(k);
    if (r == a.K - 1) lds.bound = k;
  }
  __syncthreads();
  // what reaches the bound: prefixes of at most K lists
  auto put = [&](const Key &k) {
    const int to = atomicAdd(&lds.count, 1);
    if (to < CAP2) lds.list[to] = k;
  };
  if (ahead) {
#pragma unroll
    for (int u = 0; u < EACH; ++u)
      if (mine[u].score && !lds.bound.above(mine[u])) put(mine[u]);
  } else {
    for (int l = tid; l < lists; l += NTH)
      for (int j = 0; j < a.K; ++j) {
        const Key k = key_at(l, j);
        if (!k.score || lds.bound.above(k)) break;
        put(k);
      }
  }
  __syncthreads();
  const int n = min(lds.count, CAP2);
  for (int e = tid; e < n; e += NTH) {
    const Key k = lds.list[e];
    int r = 0;
    for (int j = 0; j < n; ++j) r += lds.list[j].above(k);
    if (r < a.K) {
      const u64 o = k.score;
      a.tokens[b * a.K + r] = k.token();
      a.parents[b * a.K + r] = k.beam();
      a.out_scores[b * a.K + r] =
          (float)__longlong_as_double((long long)(o ^ (o >> 63 ? 0x8000000000000000ull : ~0ull)));
    }
  }
}

template <int LISTS, int KM>
__global__ __launch_bounds__(NT) void join_kernel(SelectArgs a) {
  __shared__ Join<NT, LISTS, KM> lds;
  const long long b = blockIdx.x, lists = (long long)a.W * a.slices;
  join(a, b, a.sums + b * lists, a.cands + b * lists * a.K, lds);
}

// Both steps in one launch, for requests of few slices and candidates: a wave takes a slice of 2048 elements of a
// beam at a time, the workgroup's NTH / 64 waves take turns.  One beam of 32000 fp32 logits: 10.5 us, and 5.3 + 4.8
// in two launches, which cost a call 5 us more (15.7 against 10.9).
constexpr int SLICE = 2048, FEW_LISTS = 32, JOIN_LISTS = 512, FEW_K = 32;
template <typename T, int NTH>
__global__ __launch_bounds__(NTH) void request_kernel(SelectArgs a) {
  constexpr int CAP = 64;  // elements gathered by a wave
  __shared__ Join<NTH, FEW_LISTS, FEW_K> lds;
  __shared__ Sum sums[FEW_LISTS];
  __shared__ Cand cands[FEW_LISTS * FEW_K];
  __shared__ u64 list[NTH / 64][CAP];
  __shared__ int counts[NTH / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lists = a.W * a.slices;
  const long long b = blockIdx.x;
  for (int l = wave; l < lists; l += NTH / 64) {
    const int w = l / a.slices, first = (l - w * a.slices) * SLICE;
    const long long row = b * a.W + w;
    if ((a.ended && a.ended[row]) || !isfinite(a.scores[row])) continue;
    const T *src = (const T *)a.logits + row * a.ld;
    float x[4][8], tops[4];  // -inf behind the row's end
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int at = first + (c * 64 + lane) * 8, left = a.V - at;
      load8(src + at, left, x[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[c][i] = i < left ? x[c][i] : -INFINITY;
    }
    const float top = tops_of(x, tops);
    const float least = value_of(kth_of_wave(ordered(top + 0.0f), a.K));
    float m = top;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    if (lane == 0) counts[wave] = 0;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = first + (c * 64 + lane) * 8 + i;
        if (x[c][i] >= least && at < a.V) {
          const int to = atomicAdd(&counts[wave], 1);
          if (to < CAP) list[wave][to] = key_of(x[c][i], at);
        }
      }
    int same;
    const float rest = rest_of_wave(x, tops, m, same);
    if (lane == 0) sums[l] = sum_of(m, rest, same);
    __builtin_amdgcn_wave_barrier();
    const int n = *(volatile int *)&counts[wave];
    Cand *out = cands + l * a.K;
    if (n <= CAP) {
      if (lane < n) {
        const u64 k = list[wave][lane];
        int r = 0;
        for (int j = 0; j < n; ++j) r += list[wave][j] > k;
        if (r < a.K) out[r] = {value_of((uint32_t)(k >> 32)), (int)~(uint32_t)k};
      }
      for (int e = n + lane; e < a.K; e += 64) out[e] = {0.0f, -1};
    } else {  // rows of equal values: one after the other
      u64 last = ~0ull;
      for (int r = 0; r < a.K; ++r) {
        u64 best = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int at = first + (c * 64 + lane) * 8 + i;
            const u64 k = at < a.V ? key_of(x[c][i], at) : 0;
            best = k < last && k > best ? k : best;
          }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
          const u64 other = __shfl_xor(best, off, 64);
          best = other > best ? other : best;
        }
        if (lane == 0) out[r] = best ? Cand{value_of((uint32_t)(best >> 32)), (int)~(uint32_t)best} : Cand{0.0f, -1};
        last = best;
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  join(a, b, sums, cands, lds);
}

// ----------------------------------------------------------------------------- reorder
// MT tensors at most: of few all arguments are read at once, in one trip to the memory they lie in (two tensors
// of 131 KB a beam: 8.8 us with arguments for 64, read one after the other).
template <int MT>
struct ReorderArgs {
  void *states[MT];
  long long bytes[MT];
  unsigned first[MT + 1];  // workgroups of a request in front of tensor i; behind the last their number, then ~0
  const int *parents;
  int W;
};

// A thread holds the same few bytes of every beam of a request: it reads the parents' before it
// writes, so the exchange needs no second buffer.  WM beams at most, T at a time.
template <typename T, int WM>
__device__ __forceinline__ void reorder_at(char *base, long long bytes, long long off, const int (&parent)[WM]) {
  T v[WM] = {};
#pragma unroll
  for (int w = 0; w < WM; ++w)
    if (parent[w] != w) v[w] = *(const T *)(base + parent[w] * bytes + off);
#pragma unroll
  for (int w = 0; w < WM; ++w)
    if (parent[w] != w) *(T *)(base + w * bytes + off) = v[w];
}

template <int WM, int MT>
__global__ __launch_bounds__(NT) void reorder_kernel(ReorderArgs<MT> a) {
  using Wide = std::conditional_t<(WM <= 16), u32x4, std::conditional_t<(WM <= 32), u32x2, uint32_t>>;
  const long long b = blockIdx.y;
  long long bytes = a.bytes[0];
  char *tensor = (char *)a.states[0];
  unsigned from = 0, to = a.first[1];
  if constexpr (MT <= 4) {
#pragma unroll
    for (int i = 1; i < MT; ++i)
      if (blockIdx.x >= a.first[i])
        bytes = a.bytes[i], tensor = (char *)a.states[i], from = a.first[i], to = a.first[i + 1];
  } else {
    // indexed where they lie: the argument itself would be copied to be indexed
    const auto *lie = (const __attribute__((address_space(4))) ReorderArgs<MT> *)__builtin_amdgcn_kernarg_segment_ptr();
    int i = 0;
#pragma unroll
    for (int j = 1; j < MT; ++j) i += blockIdx.x >= a.first[j];
    bytes = lie->bytes[i], tensor = (char *)lie->states[i], from = lie->first[i], to = lie->first[i + 1];
  }
  char *base = tensor + b * a.W * bytes;
  int parent[WM];
#pragma unroll
  for (int w = 0; w < WM; ++w) {
    const int p = a.parents[b * a.W + min(w, a.W - 1)];  // all read at once
    parent[w] = w < a.W && (unsigned)p < (unsigned)a.W ? p : w;
  }
  const long long at = (long long)(blockIdx.x - from) * NT + threadIdx.x, step = (long long)(to - from) * NT;
  const unsigned low = (unsigned)(uintptr_t)tensor | (unsigned)bytes;
  if (low % sizeof(Wide) == 0)
    for (long long e = at * sizeof(Wide); e < bytes; e += step * sizeof(Wide))
      reorder_at<Wide, WM>(base, bytes, e, parent);
  else if (low % 4 == 0)
    for (long long e = at * 4; e < bytes; e += step * 4) reorder_at<uint32_t, WM>(base, bytes, e, parent);
  else
    for (long long e = at; e < bytes; e += step) reorder_at<uint8_t, WM>(base, bytes, e, parent);
}

template <int MT>
hipError_t launch_reorder(const ReorderArgs<MT> &a, dim3 grid, hipStream_t st) {
  if (a.W <= 4)
    hipLaunchKernelGGL((reorder_kernel<4, MT>), grid, dim3(NT), 0, st, a);
  else if (a.W <= 8)
    hipLaunchKernelGGL((reorder_kernel<8, MT>), grid, dim3(NT), 0, st, a);
  else if (a.W <= 16)
    hipLaunchKernelGGL((reorder_kernel<16, MT>), grid, dim3(NT), 0, st, a);
  else if (a.W <= 32)
    hipLaunchKernelGGL((reorder_kernel<32, MT>), grid, dim3(NT), 0, st, a);
  else
    hipLaunchKernelGGL((reorder_kernel<64, MT>), grid, dim3(NT), 0, st, a);
  return hipGetLastError();
}

// Elements of a row a thread keeps: 32 where that gives enough workgroups, else 8.
int per_thread(long long rows, int V) { return rows * rec_cdiv(V, NT * 32) >= 256 ? 32 : 8; }

// Whether one launch does: few slices and candidates a request.
bool one_launch(long long W, int V, int K) { return W * rec_cdiv(V, SLICE) <= FEW_LISTS && K <= FEW_K; }

struct SelectWs {
  int slices;
  size_t cands, bytes;
};
SelectWs select_ws(long long B, int W, int V, int K) {
  SelectWs w = {};
  if (one_launch(W, V, K)) return w;
  const long long rows = B * W;
  w.slices = (int)rec_cdiv(V, NT * per_thread(rows, V));
  w.cands = rec_align((size_t)rows * w.slices * sizeof(Sum));
  w.bytes = w.cands + rec_align((size_t)rows * w.slices * K * sizeof(Cand));
  return w;
}

ret_status_t check_sizes(int B, int W, int V, int K) {
  if (B < 0 || W <= 0 || V <= 0 || K <= 0) return rec_fail(RET_ERR_INVALID_ARG, "sizes must be positive");
  if ((long long)W * V < K) return rec_fail(RET_ERR_INVALID_ARG, "K above W V");
  if (W > LANGUAGE_MAX_BEAMS || K > LANGUAGE_MAX_BEAMS || V > LANGUAGE_MAX_VOCAB || (long long)B * W > LANGUAGE_MAX_BEAM_ROWS ||
      W * rec_cdiv(V, NT * 8) > LANGUAGE_MAX_BEAM_LISTS)
    return rec_fail(RET_ERR_UNSUPPORTED, "B, W, V or K too large");
  return RET_OK;
}

}  // namespace

extern "C" size_t beam_select_workspace_bytes(int B, int W, int V, int K) {
  if (check_sizes(B, W, V, K) != RET_OK || B == 0) return 0;
  return select_ws(B, W, V, K).bytes;
}

extern "C" ret_status_t beam_select(const void *logits, const float *scores, const unsigned char *ended, int *tokens,
                                    int *parents, float *out_scores, int B, int W, int V, int K, long long logits_ld,
                                    int eos, ret_dtype_t dtype, void *workspace, size_t workspace_bytes,
                                    void *hip_stream) {
  ret_status_t s = check_sizes(B, W, V, K);
  if (s != RET_OK) return s;
  if (!rec_dtype_ok(dtype)) return rec_fail(RET_ERR_INVALID_ARG, "unknown dtype");
  if (logits_ld < V) return rec_fail(RET_ERR_INVALID_ARG, "a row stride is shorter than its row");
  if (ended && (eos < 0 || eos >= V)) return rec_fail(RET_ERR_INVALID_ARG, "eos outside 0..V-1");
  if (logits_ld > (1LL << 31)) return rec_fail(RET_ERR_UNSUPPORTED, "logits_ld too large");
  if (B == 0) return rec_status(hipSuccess);
  if (!logits || !scores || !tokens || !parents || !out_scores)
    return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  const long long rows = (long long)B * W;
  const size_t e = rec_esize(dtype), picked = (size_t)B * K * 4;
  if (!rec_aligned(logits, e) || !rec_aligned(scores, 4) || !rec_aligned(tokens, 4) || !rec_aligned(parents, 4) ||
      !rec_aligned(out_scores, 4))
    return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const SelectWs w = select_ws(B, W, V, K);
  if (w.bytes && (!workspace || workspace_bytes < w.bytes))
    return rec_fail(RET_ERR_WORKSPACE, "workspace of %zu bytes needed", w.bytes);
  const RecSpan ins[] = {rec_rows("logits", logits, rows, logits_ld, V, e), {"scores", scores, (size_t)rows * 4},
                         {"ended", ended, (size_t)rows}};
  const RecSpan outs[] = {{"tokens", tokens, picked}, {"parents", parents, picked}, {"out_scores", out_scores, picked},
                          {"workspace", workspace, w.bytes}};
  if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
  if (w.bytes && !rec_aligned(workspace, 16))
    return rec_fail(RET_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  SelectArgs a = {};
  a.logits = logits, a.scores = scores, a.ended = ended, a.tokens = tokens, a.parents = parents;
  a.out_scores = out_scores, a.ld = logits_ld;
  a.B = B, a.W = W, a.V = V, a.K = K, a.eos = eos, a.slices = w.slices;
  hipStream_t st = (hipStream_t)hip_stream;
  if (one_launch(W, V, K)) {
    a.slices = (int)rec_cdiv(V, SLICE);
    // four waves also where 16 would not fit a grid
    const bool small = W * a.slices <= 4 || !rec_grid_ok((double)B, 1024);
    if (dtype == RET_BF16) {
      if (small)
        hipLaunchKernelGGL((request_kernel<uint16_t, 256>), dim3((unsigned)B), dim3(256), 0, st, a);
      else
        hipLaunchKernelGGL((request_kernel<uint16_t, 1024>), dim3((unsigned)B), dim3(1024), 0, st, a);
    } else {
      if (small)
        hipLaunchKernelGGL((request_kernel<float, 256>), dim3((unsigned)B), dim3(256), 0, st, a);
      else
        hipLaunchKernelGGL((request_kernel<float, 1024>), dim3((unsigned)B), dim3(1024), 0, st, a);
    }
    return rec_status(hipGetLastError());
  }
  a.sums = (Sum *)workspace;
  a.cands = (Cand *)((char *)workspace + w.cands);
  const dim3 grid((unsigned)w.slices, (unsigned)std::min<long long>(rows, 65535), (unsigned)rec_cdiv(rows, 65535));
  const bool many = per_thread(rows, V) == 32;
  if (dtype == RET_BF16) {
    if (many)
      hipLaunchKernelGGL((slice_kernel<uint16_t, 32>), grid, dim3(NT), 0, st, a);
    else
      hipLaunchKernelGGL((slice_kernel<uint16_t, 8>), grid, dim3(NT), 0, st, a);
  } else {
    if (many)
      hipLaunchKernelGGL((slice_kernel<float, 32>), grid, dim3(NT), 0, st, a);
    else
      hipLaunchKernelGGL((slice_kernel<float, 8>), grid, dim3(NT), 0, st, a);
  }
  // LDS for the lists and K that there are: 25 KB or 98
  if (W * w.slices <= JOIN_LISTS && K <= FEW_K)
    hipLaunchKernelGGL((join_kernel<JOIN_LISTS, FEW_K>), dim3((unsigned)B), dim3(NT), 0, st, a);
  else
    hipLaunchKernelGGL((join_kernel<LANGUAGE_MAX_BEAM_LISTS, MAXK>), dim3((unsigned)B), dim3(NT), 0, st, a);
  return rec_status(hipGetLastError());
}

extern "C" ret_status_t beam_reorder(void *const *states, const long long *bytes, int count, const int *parents, int B,
                                     int W, void *hip_stream) {
  if (count < 0 || B < 0 || W <= 0) return rec_fail(RET_ERR_INVALID_ARG, "sizes must be positive");
  if (count > LANGUAGE_MAX_REORDERED || W > LANGUAGE_MAX_BEAMS || B > LANGUAGE_MAX_REORDER_BATCH)
    return rec_fail(RET_ERR_UNSUPPORTED, "too many tensors, requests or beams");
  if (count == 0 || B == 0) return rec_status(hipSuccess);
  if (!states || !bytes || !parents) return rec_fail(RET_ERR_INVALID_ARG, "NULL pointer");
  if (!rec_aligned(parents, 4)) return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  ReorderArgs<LANGUAGE_MAX_REORDERED> a = {};
  a.parents = parents, a.W = W;
  int n = 0;  // tensors that hold anything
  const RecSpan par = {"parents", parents, (size_t)B * W * 4};
  RecSpan all[LANGUAGE_MAX_REORDERED];
  unsigned blocks = 0;
  for (int i = 0; i < count; ++i) {
    if (bytes[i] < 0) return rec_fail(RET_ERR_INVALID_ARG, "sizes must be positive");
    if (bytes[i] > (1LL << 40) || (double)bytes[i] * B * W > (double)(1LL << 44))
      return rec_fail(RET_ERR_UNSUPPORTED, "a tensor is too large");
    if (bytes[i] == 0) continue;
    if (!states[i]) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
    all[n] = {"a tensor", states[i], (size_t)bytes[i] * B * W};
    if (rec_overlap(all[n], par)) return rec_fail(RET_ERR_INVALID_ARG, "a tensor overlaps parents");
    for (int j = 0; j < n; ++j)
      if (rec_overlap(all[n], all[j])) return rec_fail(RET_ERR_INVALID_ARG, "two tensors overlap");
    a.states[n] = states[i];
    a.bytes[n] = bytes[i];
    a.first[n] = blocks;
    blocks += (unsigned)std::min<long long>(4096, rec_cdiv(bytes[i], NT * 16));
    a.first[++n] = blocks;
  }
  if (n == 0) return rec_status(hipSuccess);
  for (int i = n + 1; i <= LANGUAGE_MAX_REORDERED; ++i) a.first[i] = ~0u;
  if (!rec_grid_ok((double)blocks * B, NT)) return rec_fail(RET_ERR_UNSUPPORTED, "too many workgroups for one launch");
  const dim3 grid(blocks, (unsigned)B);
  hipStream_t st = (hipStream_t)hip_stream;
  if (n > 4) return rec_status(launch_reorder(a, grid, st));
  ReorderArgs<4> few = {};
  for (int i = 0; i < 4; ++i) few.states[i] = a.states[i], few.bytes[i] = a.bytes[i], few.first[i + 1] = a.first[i + 1];
  few.parents = parents, few.W = W;
  return rec_status(launch_reorder(few, grid, st));
}
