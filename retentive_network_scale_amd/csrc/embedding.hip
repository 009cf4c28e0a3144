// Scaled embedding and its gradient by sorted tokens (language.h).
//
// The lookup streams: eight elements a thread, each moved once.  Bound by bytes written: 16384 tokens of 2048
// bf16 channels (67 MB, from 5000 distinct rows) take 24 us, 64 tokens 2.6.
//
// The gradient of a row is a sum over the tokens that name it, in their order.  Three launches:
//   1. Sort.  The tokens are ordered by (id modulo the number of workgroups, id, token).  Each workgroup
//      owns the ids of one remainder, so that the frequent ones, which come first in a vocabulary, are spread, and
//      reads all tokens twice: once to count, once to place.  What has a smaller remainder tells
//      where its part of the order begins, so the workgroups need nothing from each other.
//   2. Long runs.  Tokens come with the frequencies of words, so one id can have a tenth of them.  The
//      order is cut into pieces of `piece` tokens, and runs longer than one are summed piece by piece.
//   3. Rows.  Every row of the table's gradient is written once: the sum of a short run's tokens or of
//      a long run's pieces, or zero.
// 16384 tokens of 2048 bf16 channels, V 32000: 14, 10.5 and 46 us.  The last writes 131 MB and reads 67 and is bound by
// bytes (4.3 TB/s with the pieces'); the first by its chain: ids, counts, their running sum, ids again.
#include <algorithm>
#include <type_traits>

#include "language.hpp"

using namespace ret;

namespace {

constexpr int NT = 256;

// ------------------------------------------------------------------------------ lookup
// Threads of a row: tpr (a power of two up to NT); a workgroup takes NT / tpr rows at a time.
template <typename TI, typename TO>
__global__ __launch_bounds__(NT) void lookup_kernel(const int *ids, const TI *table, TO *out, long long n, int V, int D,
                                                    int tpr, float scale) {
  const int col = threadIdx.x & (tpr - 1), rows = NT / tpr;
  const long long t = (long long)blockIdx.x * rows + threadIdx.x / tpr;
  if (t >= n) return;
  const int id = ids[t];
  const bool in = (unsigned)id < (unsigned)V;
  const TI *src = table + (long long)(in ? id : 0) * D;
  TO *dst = out + t * D;
  for (int c = col * 8; c < D; c += tpr * 8) {
    float r[8];
    load8(src + c, in ? D - c : 0, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = in ? r[i] * scale : 0.0f;
    store8(dst + c, D - c, r);
  }
}

// -------------------------------------------------------------------------------- sort
constexpr int SORT_NT = 1024, SORT_WAVES = SORT_NT / 64;
constexpr int MAX_RANGE = 512;  // ids of a workgroup: 32 KB of counters
constexpr int CHUNK = 512;      // tokens that a wave looks through before it places what it found

// Workgroup b of 2^shift owns the ids b, b + 2^shift, ..: `range` of them at most, `bits` the width of their
// number.  order[j]: the token at place j; runs[v]: the places of v's tokens, from .x up to .y; *total:
// the number of tokens with an id in the table.  Wave w of a workgroup reads the w-th part of the tokens.
__global__ __launch_bounds__(SORT_NT) void sort_kernel(const int *ids, int *order, int2 *runs, int *total, int n, int V,
                                                       int shift, int bits) {
  __shared__ int at[SORT_WAVES][MAX_RANGE];  // tokens of a wave for an id, then where its next one goes
  __shared__ int2 found[SORT_WAVES][CHUNK];
  __shared__ int red[SORT_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int own = blockIdx.x, groups = 1 << shift, mine = own < V ? (V - 1 - own) / groups + 1 : 0;
  const int part = ((n + SORT_WAVES * 64 - 1) / (SORT_WAVES * 64)) * 64;
  const long long lo = (long long)wave * part, hi = lo + part < n ? lo + part : n;
  for (int i = lane; i < mine; i += 64) at[wave][i] = 0;
  __syncthreads();
  int below = 0;
#pragma unroll 8
  for (long long t = lo + lane; t < hi; t += 64) {
    const int id = ids[t];
    if ((unsigned)id < (unsigned)V) {
      const int rem = id & (groups - 1);
      below += rem < own;
      if (rem == own) atomicAdd(&at[wave][id >> shift], 1);
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) below += __shfl_xor(below, off, 64);
  if (lane == 0) red[wave] = below;
  __syncthreads();
  // wave 0: the counts' running sum over (id, wave), from the tokens of smaller remainders on
  if (wave == 0) {
    int base = 0;
#pragma unroll
    for (int w = 0; w < SORT_WAVES; ++w) base += red[w];
    for (int i0 = 0; i0 < mine; i0 += 64) {
      const int i = i0 + lane;
      int c[SORT_WAVES], sum = 0;
#pragma unroll
      for (int w = 0; w < SORT_WAVES; ++w) c[w] = i < mine ? at[w][i] : 0;
#pragma unroll
      for (int w = 0; w < SORT_WAVES; ++w) sum += c[w];
      int incl = sum;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int up = __shfl_up(incl, off, 64);
        if (lane >= off) incl += up;
      }
      int p = base + incl - sum;
      if (i < mine) {
        runs[own + (i << shift)] = make_int2(p, p + sum);
#pragma unroll
        for (int w = 0; w < SORT_WAVES; ++w) {
          at[w][i] = p;
          p += c[w];
        }
      }
      base += __shfl(incl, 63, 64);
    }
    if (own == groups - 1 && lane == 0) *total = base;
  }
  __syncthreads();
  for (long long t0 = lo; t0 < hi; t0 += CHUNK) {
    // the tokens of the workgroup's ids, in order (a wave's LDS operations keep theirs)
    int many = 0;
#pragma unroll
    for (int u = 0; u < CHUNK / 64; ++u) {
      const long long t = t0 + u * 64 + lane;
      const int id = t < hi ? ids[t] : -1;
      const bool in = (unsigned)id < (unsigned)V && (id & (groups - 1)) == own;
      const unsigned long long some = __ballot(in);
      if (in) found[wave][many + __popcll(some & ((1ull << lane) - 1))] = make_int2(id >> shift, (int)t);
      many += __popcll(some);
    }
    __builtin_amdgcn_wave_barrier();
    for (int j0 = 0; j0 < many; j0 += 64) {
      const bool in = j0 + lane < many;
      const int2 f = in ? found[wave][j0 + lane] : make_int2(0, 0);
      unsigned long long same = __ballot(in);  // the lanes of the same id, from one comparison a bit
      for (int bit = 0; bit < bits; ++bit) {
        const bool one = f.x >> bit & 1;
        const unsigned long long set = __ballot(one);
        same &= one ? set : ~set;
      }
      // the first lane of an id takes the places of all of them
      const int leader = __ffsll((long long)same) - 1;
      int to = 0;
      if (in && lane == leader) to = atomicAdd(&at[wave][f.x], __popcll(same));
      to = __shfl(to, leader, 64);
      if (in) order[to + __popcll(same & ((1ull << lane) - 1))] = f.y;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// -------------------------------------------------------------------------------- sums
// Adds tokens to CH chunks of eight columns, the first at c, chunk k `step` further on; AHEAD tokens' loads are
// under way at a time.  token(j): the j-th of `many`.
template <typename TI, int CH, int AHEAD, typename F>
__device__ __forceinline__ void add_tokens(const TI *d_o, F token, int many, long long ld, int c, int step, int D,
                                           float (&sum)[CH][8]) {
  for (int j = 0; j < many; j += AHEAD) {
    Raw8<TI> r[AHEAD][CH];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const bool in = j + u < many;
      const TI *src = d_o + token(in ? j + u : j) * ld + c;
#pragma unroll
      for (int k = 0; k < CH; ++k) r[u][k].load(src + k * step, in ? D - c - k * step : 0);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float v[8];
        r[u][k].get(v);
        if (j + u < many)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[k][i] += v[i];
      }
  }
}

constexpr int MAX_PIECE = 4096;

// Piece blockIdx.x of the order: the part of the run that its first place belongs to, and of the run
// that its last place belongs to where that is another, each only if the run is longer than a piece.
template <typename TI>
__global__ __launch_bounds__(NT) void piece_kernel(const int *ids, const TI *d_o, const int *order, const int2 *runs,
                                                   const int *total, float *part, int D, long long ld, int piece) {
  __shared__ int tokens[MAX_PIECE];
  const int j0 = blockIdx.x * piece, c = (blockIdx.y * NT + threadIdx.x) * 8;
  const int j1 = min(j0 + piece, *total);
  for (int j = j0 + threadIdx.x; j < j1; j += NT) tokens[j - j0] = order[j];
  __syncthreads();
  if (j0 >= j1) return;
  const int a = ids[tokens[0]], z = ids[tokens[j1 - j0 - 1]];
  const int2 run[2] = {runs[a], runs[z]};
#pragma unroll
  for (int slot = 0; slot < 2; ++slot) {
    const int s = run[slot].x, e = run[slot].y;
    if ((slot == 1 && z == a) || e - s <= piece || c >= D) continue;
    const int from = max(s, j0), many = min(e, j1) - from;
    float sum[1][8] = {};
    add_tokens<TI, 1, 16>(d_o, [&](int j) { return tokens[from - j0 + j]; }, many, ld, c, 0, D, sum);
    store8(part + (2LL * blockIdx.x + slot) * D + c, D - c, sum[0]);
  }
}

// Eight columns from c of the sum over a long run's pieces, places s .. e of the order.
__device__ __forceinline__ void add_pieces(const float *part, int s, int e, int piece, int c, int D, float (&sum)[8]) {
  constexpr int AHEAD = 8;
  const int p0 = s / piece, p1 = (e - 1) / piece;
  for (int p = p0; p <= p1; p += AHEAD) {
    Raw8<float> r[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)  // a run that begins inside its first piece is that piece's second slot
      r[u].load(part + (2LL * min(p + u, p1) + (p + u == p0 && s % piece != 0)) * D + c, p + u <= p1 ? D - c : 0);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      float v[8];
      r[u].get(v);
      if (p + u <= p1)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += v[i];
    }
  }
}

// A row of the gradient by tpr lanes (a power of two up to a wave), CH chunks of eight columns each at a
// time: a wave a row rather than a workgroup, since a row's time is that of its run, the run's tokens
// and their rows, one after the other.  A long run's pieces in rows of a wave (CH > 1) are added by the whole
// workgroup, a chunk a thread, more of them at a time: one id with 1600 of 16384 tokens took its wave 90 us.
template <typename TI, typename TO, int CH>
__global__ __launch_bounds__(NT) void rows_kernel(const TI *d_o, const int *order, const int2 *runs, const float *part,
                                                  TO *dtable, int V, int D, long long ld, int piece, int tpr,
                                                  float scale) {
  const int col = threadIdx.x & (tpr - 1), rows = NT / tpr, step = tpr * 8;
  const int v0 = blockIdx.x * rows, v = v0 + threadIdx.x / tpr;
  const int2 run = runs && v < V ? runs[v] : make_int2(0, 0);
  const int s = run.x, e = run.y;
  if (v < V && (CH == 1 || e - s <= piece)) {
    for (int c = col * 8; c < D + col * 8; c += CH * step) {  // all of a row's lanes stay together
      float sum[CH][8] = {};
      if (e - s <= piece) {
        for (int j = s; j < e; j += tpr) {
          const int mine = order[min(j + col, e - 1)];
          const int first = (threadIdx.x & 63) - col;
          add_tokens<TI, CH, 4>(d_o, [&](int i) { return __shfl(mine, first + i, 64); }, min(tpr, e - j), ld, c, step, D,
                                sum);
        }
      } else {
        add_pieces(part, s, e, piece, c, D, sum[0]);
      }
#pragma unroll
      for (int k = 0; k < CH; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[k][i] *= scale;
        store8(dtable + (long long)v * D + c + k * step, D - c - k * step, sum[k]);
      }
    }
  }
  if constexpr (CH > 1) {
    if (!runs) return;
    for (int i = 0; i < rows && v0 + i < V; ++i) {
      const int2 other = runs[v0 + i];
      if (other.y - other.x <= piece) continue;
      for (int c = threadIdx.x * 8; c < D; c += NT * 8) {
        float sum[8] = {};
        add_pieces(part, other.x, other.y, piece, c, D, sum);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] *= scale;
        store8(dtable + (long long)(v0 + i) * D + c, D - c, sum);
      }
    }
  }
}

int threads_per_row(int D, int most) {
  int t = 1;
  while (t < most && t * 8 < D) t *= 2;
  return t;
}

// Tokens of a piece: about a quarter of the square root of their number, 4096 at most (of 2^28), so that neither a
// piece nor the list of pieces of one id is long.
int piece_of(long long n) {
  int p = 32;
  while (16LL * p * p < n) p *= 2;
  return p;
}

struct EmbedWs {
  size_t order, runs, total, part, bytes;
};
EmbedWs embed_ws(long long n, int V, int D) {
  EmbedWs w;
  w.order = 0;
  w.runs = rec_align((size_t)n * 4);
  w.total = w.runs + rec_align((size_t)V * 8);
  w.part = w.total + 256;
  w.bytes = w.part + rec_align((size_t)rec_cdiv(n, piece_of(n)) * 2 * D * 4);
  return w;
}

ret_status_t check_sizes(long long n, int V, int D, ret_dtype_t in, ret_dtype_t out) {
  if (n < 0 || V <= 0 || D <= 0) return rec_fail(RET_ERR_INVALID_ARG, "sizes must be positive");
  if (!rec_dtype_ok(in) || !rec_dtype_ok(out)) return rec_fail(RET_ERR_INVALID_ARG, "unknown dtype");
  if (n > LANGUAGE_MAX_TOKENS || V > LANGUAGE_MAX_VOCAB || D > LANGUAGE_MAX_CHANNELS ||
      n * D > LANGUAGE_MAX_ELEMENTS || (long long)V * D > LANGUAGE_MAX_ELEMENTS)
    return rec_fail(RET_ERR_UNSUPPORTED, "n, V or D too large");
  if (!rec_grid_ok((double)rec_cdiv(n, NT / threads_per_row(D, NT)), NT) ||
      !rec_grid_ok((double)rec_cdiv(V, NT / threads_per_row(D, 64)), NT))
    return rec_fail(RET_ERR_UNSUPPORTED, "too many rows for one launch");
  return RET_OK;
}

}  // namespace

extern "C" ret_status_t embedding(const int *ids, const void *table, void *out, long long n, int V, int D, float scale,
                                  ret_dtype_t in_dtype, ret_dtype_t out_dtype, void *hip_stream) {
  ret_status_t s = check_sizes(n, V, D, in_dtype, out_dtype);
  if (s != RET_OK) return s;
  if (n == 0) return rec_status(hipSuccess);
  if (!ids || !table || !out) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  const size_t ie = rec_esize(in_dtype), oe = rec_esize(out_dtype);
  if (!rec_aligned(ids, 4) || !rec_aligned(table, ie) || !rec_aligned(out, oe))
    return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const RecSpan ins[] = {{"ids", ids, (size_t)n * 4}, {"table", table, (size_t)V * D * ie}};
  const RecSpan outs[] = {{"out", out, (size_t)n * D * oe}};
  if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
  const int tpr = threads_per_row(D, NT);
  const unsigned grid = (unsigned)rec_cdiv(n, NT / tpr);
  return rec_status(with_types(in_dtype, out_dtype, [&](auto ti, auto to) {
    hipLaunchKernelGGL((lookup_kernel<std::remove_pointer_t<decltype(ti)>, std::remove_pointer_t<decltype(to)>>),
                       dim3(grid), dim3(NT), 0, (hipStream_t)hip_stream, ids, (decltype(ti))table, (decltype(to))out, n,
                       V, D, tpr, scale);
    return hipGetLastError();
  }));
}

extern "C" size_t embedding_bwd_workspace_bytes(long long n, int V, int D) {
  if (check_sizes(n, V, D, RET_F32, RET_F32) != RET_OK || n == 0) return 0;
  return embed_ws(n, V, D).bytes;
}

extern "C" ret_status_t embedding_bwd(const int *ids, const void *d_o, void *dtable, long long n, int V, int D,
                                      long long o_ld, float scale, ret_dtype_t in_dtype, ret_dtype_t out_dtype,
                                      void *workspace, size_t workspace_bytes, void *hip_stream) {
  ret_status_t s = check_sizes(n, V, D, in_dtype, out_dtype);
  if (s != RET_OK) return s;
  if (o_ld < D) return rec_fail(RET_ERR_INVALID_ARG, "a row stride is shorter than its row");
  if (o_ld > (1LL << 31)) return rec_fail(RET_ERR_UNSUPPORTED, "o_ld too large");
  if (!dtable || (n > 0 && (!ids || !d_o))) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  const size_t ie = rec_esize(in_dtype), oe = rec_esize(out_dtype);
  if (!rec_aligned(ids, 4) || !rec_aligned(d_o, ie) || !rec_aligned(dtable, oe))
    return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const EmbedWs w = embed_ws(n, V, D);
  if (n > 0) {
    if (!workspace || workspace_bytes < w.bytes)
      return rec_fail(RET_ERR_WORKSPACE, "workspace of %zu bytes needed", w.bytes);
    const RecSpan ins[] = {{"ids", ids, (size_t)n * 4}, rec_rows("d_o", d_o, n, o_ld, D, ie)};
    const RecSpan outs[] = {{"dtable", dtable, (size_t)V * D * oe}, {"workspace", workspace, w.bytes}};
    if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
    if (!rec_aligned(workspace, 16)) return rec_fail(RET_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  }
  hipStream_t st = (hipStream_t)hip_stream;
  char *ws = (char *)workspace;
  int *order = n ? (int *)(ws + w.order) : nullptr, *total = n ? (int *)(ws + w.total) : nullptr;
  int2 *runs = n ? (int2 *)(ws + w.runs) : nullptr;
  float *part = n ? (float *)(ws + w.part) : nullptr;
  const int piece = piece_of(n), tpr = threads_per_row(D, 64);
  if (n > 0) {
    int shift = 8, bits = 0;  // 256 workgroups, or more where they would own more ids than they can count
    while (V > MAX_RANGE << shift) ++shift;
    while (1LL << (shift + bits) < V) ++bits;
    hipLaunchKernelGGL(sort_kernel, dim3(1u << shift), dim3(SORT_NT), 0, st, ids, order, runs, total, (int)n, V, shift,
                       bits);
  }
  return rec_status(with_types(in_dtype, out_dtype, [&](auto ti, auto to) {
    using TI = std::remove_pointer_t<decltype(ti)>;
    using TO = std::remove_pointer_t<decltype(to)>;
    if (n > piece)
      hipLaunchKernelGGL((piece_kernel<TI>), dim3((unsigned)rec_cdiv(n, piece), (unsigned)rec_cdiv(D, NT * 8)), dim3(NT),
                         0, st, ids, (const TI *)d_o, order, runs, total, part, D, o_ld, piece);
    auto rows = [&](auto chunks) {
      hipLaunchKernelGGL((rows_kernel<TI, TO, decltype(chunks)::value>), dim3((unsigned)rec_cdiv(V, NT / tpr)), dim3(NT), 0,
                         st, (const TI *)d_o, order, runs, part, (TO *)dtable, V, D, o_ld, piece, tpr, scale);
    };
    if (D <= 512)
      rows(std::integral_constant<int, 1>{});
    else if (D <= 1024)
      rows(std::integral_constant<int, 2>{});
    else
      rows(std::integral_constant<int, 4>{});
    return hipGetLastError();
  }));
}
