// Products with bias, activation and residual, and their gradients (language.h): the entry points, the
// product for few tokens, and the elementwise part of the gradients.  linear_mm.hpp has the tiled
// product.
#include "linear.hpp"

using namespace ret;

namespace {

// --------------------------------------------------------------------------- few tokens
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;

// Adds the lanes' N values over lanes: each step halves the number of values a lane holds, as long as
// there is more than one.
template <int N, int OFF, int C>
__device__ __forceinline__ void fold(float (&v)[C], int lane) {
  if constexpr (OFF > 0) {
    if constexpr (N > 1) {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float mine = lane & OFF ? v[i + N / 2] : v[i], other = lane & OFF ? v[i] : v[i + N / 2];
        v[i] = mine + __shfl_xor(other, OFF, 64);
      }
      fold<N / 2, OFF / 2>(v, lane);
    } else {
      v[0] += __shfl_xor(v[0], OFF, 64);
      fold<1, OFF / 2>(v, lane);
    }
  }
}

// A workgroup takes RW rows of w, its four waves take turns along k, 512 at a time, a lane 8 of them; M tokens at
// most.  w is read once at full width, x comes from the caches.  Each wave's RW M sums end in as many lanes,
// and the waves' are added in LDS.  Bound by the launch and the way from memory for one token (N 4096, K 2048,
// 16.8 MB: 3.4 us) and by the caches' way for x with more of them.
template <int M, int RW>
__global__ __launch_bounds__(256) void rows_kernel(const uint16_t *x, const uint16_t *w, int tokens, int N, int K,
                                                   long long x_ld, Finish f) {
  constexpr int C = M * RW;
  static_assert(C <= 64 && (C & (C - 1)) == 0, "sums of a wave");
  __shared__ float red[4][C];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n0 = blockIdx.x * RW;
  float acc[C] = {};  // [RW][M]
  auto add = [&](const Raw8<uint16_t> (&wv)[RW], const Raw8<uint16_t> &xv, int m) {
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[r * M + m] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, wv[r].w[0].w[i]),
                                                         __builtin_bit_cast(bf16x2, xv.w[0].w[i]), acc[r * M + m], false);
  };
  const int whole = K / 512 * 512;
  for (int k = wave * 512 + lane * 8; k < whole; k += 2048) {
    Raw8<uint16_t> wv[RW], xv;
#pragma unroll
    for (int r = 0; r < RW; ++r) wv[r].load(w + (long long)min(n0 + r, N - 1) * K + k, 8);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      xv.load(x + min(m, tokens - 1) * x_ld + k, 8);
      add(wv, xv, m);
    }
  }
  if (whole < K && wave == (whole / 512 & 3)) {
    const int k = whole + lane * 8;
    Raw8<uint16_t> wv[RW], xv;
#pragma unroll
    for (int r = 0; r < RW; ++r) wv[r].load(w + (long long)min(n0 + r, N - 1) * K + k, K - k);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      xv.load(x + min(m, tokens - 1) * x_ld + k, K - k);
      add(wv, xv, m);
    }
  }
  fold<C, 32>(acc, lane);
  if (lane % (64 / C) == 0) red[wave][lane / (64 / C)] = acc[0];
  __syncthreads();
  const int value = threadIdx.x, m = value % M, col = n0 + value / M;
  if (value < C && m < tokens && col < N) {
    float v = red[0][value] + red[1][value] + red[2][value] + red[3][value];
    const long long at = (long long)m * N + col;
    if (f.bias) v += bf2f(f.bias[col]);
    if (f.pre) f.pre[at] = f2bf(v);
    v = act_value(v, f.act, f.out_bf16);
    if (f.residual) v += load_elem(f.residual, at, f.res_bf16);
    store_elem(f.out, at, v, f.out_bf16);
  }
}

// ------------------------------------------------------------------- a batch of single tokens
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;

// A workgroup takes 16 rows of w and all tokens, 16 FM at most; its eight waves take turns along k, 64 at a time,
// and their sums meet in LDS: one launch, where tiles need parts of k and a second one.  Operands go straight from
// memory to the matrix cores' registers, four steps ahead.  Bound by the rate at which a CU takes 16 rows' lines in
// a load, 0.88 us for 16 rows of 1000 k (36 GB/s a CU); 32 tokens, N 4096, K 2048: 8.1 us.
template <int FM>
__global__ __launch_bounds__(512) void batch_kernel(const uint16_t *x, const uint16_t *w, int tokens, int N, int K,
                                                    long long x_ld, Finish f) {
  constexpr int WAVES = 8, AHEAD = 4, PITCH = 16 + 4, THREADS = 16 * FM * 2;  // of eight sums each
  __shared__ __attribute__((aligned(16))) float red[WAVES][16 * FM][PITCH];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const uint16_t *rows[FM + 1];  // rows behind the last are the last once more
#pragma unroll
  for (int i = 0; i < FM; ++i) rows[i] = x + min(i * 16 + l16, tokens - 1) * x_ld + g * 8;
  rows[FM] = w + (long long)min(n0 + l16, N - 1) * K + g * 8;
  f32x4 acc[FM] = {};
  struct Chunk {
    Words4 r[FM + 1][2];
  };
  auto load = [&](Chunk &c, int k) {
#pragma unroll
    for (int i = 0; i < FM + 1; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) c.r[i][h] = *(const Words4 *)(rows[i] + k + h * 32);
  };
  auto multiply = [&](const Chunk &c) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < FM; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, c.r[FM][h]),
                                                         __builtin_bit_cast(bf16x8, c.r[i][h]), acc[i], 0, 0, 0);
  };
  // what the sums need at the end, on its way early
  const int t = threadIdx.x, m = t / 2, col = t % 2 * 8, left = t < THREADS && m < tokens ? N - n0 - col : 0;
  const long long at = (long long)m * N + n0 + col;
  float bias[8] = {};
  if (f.bias) load8(f.bias + n0 + col, left, bias);
  Residual8 res;
  res.load(f, at, left);

  const int whole = K / 64, mine = whole > wave ? (whole - wave + WAVES - 1) / WAVES : 0;
  const int groups = mine / AHEAD, rest = mine % AHEAD;
  auto k_of = [&](int c) { return (wave + c * WAVES) * 64; };
  if (groups > 0) {
    Chunk now[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) load(now[u], k_of(u));
    for (int i = 1; i < groups; ++i) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        multiply(now[u]);
        load(now[u], k_of(i * AHEAD + u));
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) multiply(now[u]);
  }
  if (rest > 0) {
    Chunk now[AHEAD - 1];
#pragma unroll
    for (int u = 0; u < AHEAD - 1; ++u)
      if (u < rest) load(now[u], k_of(groups * AHEAD + u));
#pragma unroll
    for (int u = 0; u < AHEAD - 1; ++u)
      if (u < rest) multiply(now[u]);
  }
  if (whole * 64 < K && wave == whole % WAVES) {
    Chunk end;
#pragma unroll
    for (int i = 0; i < FM + 1; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Raw8<uint16_t> r;
        r.load(rows[i] + whole * 64 + h * 32, K - whole * 64 - g * 8 - h * 32);
        end.r[i][h] = r.w[0];
      }
    multiply(end);
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) *(f32x4 *)&red[wave][i * 16 + l16][4 * g] = acc[i];
  __syncthreads();
  if (left <= 0) return;
  float z[8] = {};
#pragma unroll
  for (int v = 0; v < WAVES; ++v) {
    const f32x4 lo = *(const f32x4 *)&red[v][m][col], hi = *(const f32x4 *)&red[v][m][col + 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] += lo[i], z[i + 4] += hi[i];
  }
  finish8(f, at, left, bias, res, z);
}

// ----------------------------------------------------------------- dz and the bias's gradient
// Columns blockIdx.y * 512 + 8 lane .., rows blockIdx.x * 4 + wave, then parts * 4 further on.
// dz [M][ldz] (columns behind N zero) and one partial row of sums a workgroup; either may be NULL.
// dz is rounded to bf16, as an operand of two products on the bf16 matrix cores: the gradients are off by 2.35e-3
// (relative, of normal values) where those of an unrounded dz, rounded at the end, are by 1.66e-3; two bf16 terms
// would keep it at twice the products' work.  The bias's sums take it unrounded.
// Bound by bytes: 403 MB in 75 us (M 16384, N 4096), the copy rate.
__global__ __launch_bounds__(256) void dz_kernel(const uint16_t *d_o, const uint16_t *pre, uint16_t *dz, float *part,
                                                 long long M, int N, int ldz, int parts, int act) {
  __shared__ float red[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.y * 512 + lane * 8, n = N - c;
  float sum[8] = {};
  if (n > 0) {
    for (long long m = (long long)blockIdx.x * 4 + wave; m < M; m += (long long)parts * 4) {
      float d[8], z[8];
      load8(d_o + m * N + c, n, d);
      if (act) {
        load8(pre + m * N + c, n, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= act_slope(z[i], act);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += d[i];
      if (dz) {
        if (n < 8)
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = i < n ? d[i] : 0.0f;
        store8(dz + m * ldz + c, d);
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[wave][lane * 8 + i] = sum[i];
  __syncthreads();
  for (int e = threadIdx.x; e < 512; e += 256) {
    const int col = blockIdx.y * 512 + e;
    if (col < N) part[(long long)blockIdx.x * N + col] = red[0][e] + red[1][e] + red[2][e] + red[3][e];
  }
}

__global__ __launch_bounds__(1024) void bias_join_kernel(const float *part, int parts, int N, float *dbias) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (n < N)
#pragma unroll 8
    for (int p = wave; p < parts; p += 16) s += part[(long long)p * N + n];
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && n < N) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += red[w][lane];
    dbias[n] = s;
  }
}

// ------------------------------------------------------------------------------- host
// Whether rows_kernel serves a call.  It and the tiles take, in us, for 8 tokens 5.8 and 8.8 (N 4096, K 2048); it and
// batch_kernel for 16 tokens 7.5 and 9.8 (2048, 4096), where that has half the CUs, but 8.9 and 6.3 (4096, 2048) and 6.5
// and 4.1 (1000, 1000).  Rows of odd length, of which a lane's 16 bytes begin at any two, cost it three times as much:
// 16 tokens 28 us, the tiles 12 (2048, 4095).
bool few(long long M, long long N, long long K) {
  return M <= 8 || (M <= 16 && K >= 2 * N && N * K <= 1 << 23 && K % 2 == 0);
}

template <int M, int RW>
hipError_t launch_rows(const void *x, const void *w, int tokens, int N, int K, long long x_ld, const Finish &f,
                       hipStream_t st) {
  hipLaunchKernelGGL((rows_kernel<M, RW>), dim3((unsigned)rec_cdiv(N, RW)), dim3(256), 0, st, (const uint16_t *)x,
                     (const uint16_t *)w, tokens, N, K, x_ld, f);
  return hipGetLastError();
}

// Whether batch_kernel does, among the others: its time as measured (in us, without the launch) against the tiles'
// estimate.  For 32 tokens it and the tiles take 8.1 and 10.6 (N 4096, K 2048), 4.6 and 7.1 (1000, 1000), 13.2 and 9.6
// (2048, 4096), 48 and 22 (32000, 2048).  With rows of odd length it takes three times as much and the tiles 1.5 times:
// for 16 tokens 8.8 and 16.6 (4096, 1401) but 16.6 and 11.4 (4096, 2047), for 33 10.6 and 12.1 (1000, 999), for 64 14.1
// and 12.4 (1000, 999) and 36 and 20 (4096, 2047); there rows that are the last once more cost little.
bool batch(long long M, long long N, long long K) {
  if (M > 64) return false;
  const double each = 0.88e-3 * K * rec_cdiv(rec_cdiv(N, 16), 256);
  if (K % 2) return each * (M / 16.0 + 1) < 2.75;
  return each * ((M <= 16 ? 1 : M <= 32 ? 2 : 4) + 1) < mm_plan(M, N, K).us;
}

template <int FM>
hipError_t launch_batch(const void *x, const void *w, int tokens, int N, int K, long long x_ld, const Finish &f,
                        hipStream_t st) {
  hipLaunchKernelGGL(batch_kernel<FM>, dim3((unsigned)rec_cdiv(N, 16)), dim3(512), 0, st, (const uint16_t *)x,
                     (const uint16_t *)w, tokens, N, K, x_ld, f);
  return hipGetLastError();
}

ret_status_t check_sizes(long long M, int N, int K) {
  if (M < 0 || N <= 0 || K <= 0) return rec_fail(RET_ERR_INVALID_ARG, "sizes must be positive");
  if (M > LANGUAGE_MAX_TOKENS || N > LANGUAGE_MAX_FEATURES || K > LANGUAGE_MAX_FEATURES ||
      (double)M * N > (double)LANGUAGE_MAX_ELEMENTS || (double)M * K > (double)LANGUAGE_MAX_ELEMENTS ||
      (double)N * K > (double)LANGUAGE_MAX_ELEMENTS)
    return rec_fail(RET_ERR_UNSUPPORTED, "M, N or K too large");
  return RET_OK;
}

bool act_ok(int act) { return act == LINEAR_ACT_NONE || act == LINEAR_ACT_GELU || act == LINEAR_ACT_SILU; }

struct BwdWs {
  int ldz, parts;  // of dz; rows of partial sums of the bias
  size_t dz, bias, product, bytes;
};
BwdWs bwd_ws(long long M, int N, int K) {
  BwdWs w;
  w.ldz = (N + 7) / 8 * 8;
  const long long cols = rec_cdiv(N, 512);
  w.parts = (int)std::max<long long>(1, std::min<long long>(rec_cdiv(M, 4), std::max<long long>(1, 2048 / cols)));
  w.dz = 0;
  w.bias = rec_align((size_t)M * w.ldz * 2);
  w.product = w.bias + rec_align((size_t)w.parts * N * 4);
  w.bytes = w.product + std::max(mm_plan(M, K, N).bytes, mm_plan(N, K, M).bytes);
  return w;
}

}  // namespace

extern "C" size_t linear_workspace_bytes(long long M, int N, int K) {
  if (check_sizes(M, N, K) != RET_OK || few(M, N, K) || batch(M, N, K)) return 0;
  return mm_plan(M, N, K).bytes;
}

extern "C" ret_status_t linear(const void *x, const void *w, const void *bias, const void *residual, void *out,
                               void *pre, long long M, int N, int K, long long x_ld, int act,
                               ret_dtype_t residual_dtype, ret_dtype_t out_dtype, void *workspace,
                               size_t workspace_bytes, void *hip_stream) {
  ret_status_t s = check_sizes(M, N, K);
  if (s != RET_OK) return s;
  if (!rec_dtype_ok(out_dtype) || !rec_dtype_ok(residual_dtype))
    return rec_fail(RET_ERR_INVALID_ARG, "unknown dtype");
  if (!act_ok(act)) return rec_fail(RET_ERR_INVALID_ARG, "unknown activation");
  if (x_ld < K) return rec_fail(RET_ERR_INVALID_ARG, "a row stride is shorter than its row");
  if (x_ld > (1LL << 31)) return rec_fail(RET_ERR_UNSUPPORTED, "x_ld too large");
  if (M == 0) return rec_status(hipSuccess);
  if (!x || !w || !out) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  const size_t oe = rec_esize(out_dtype), re = rec_esize(residual_dtype), mn = (size_t)M * N;
  if (!rec_aligned(x, 2) || !rec_aligned(w, 2) || !rec_aligned(bias, 2) || !rec_aligned(residual, re) ||
      !rec_aligned(out, oe) || !rec_aligned(pre, 2))
    return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const size_t need = linear_workspace_bytes(M, N, K);
  if (need && (!workspace || workspace_bytes < need))
    return rec_fail(RET_ERR_WORKSPACE, "workspace of %zu bytes needed", need);
  const bool in_place = residual == out && residual_dtype == out_dtype;
  const RecSpan ins[] = {rec_rows("x", x, M, x_ld, K, 2), {"w", w, (size_t)N * K * 2}, {"bias", bias, (size_t)N * 2},
                         {"residual", in_place ? nullptr : residual, mn * re}};
  const RecSpan outs[] = {{"out", out, mn * oe}, {"pre", pre, mn * 2}, {"workspace", workspace, need}};
  if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
  if (need && !rec_aligned(workspace, 16)) return rec_fail(RET_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  Finish f = {};
  f.bias = (const uint16_t *)bias, f.residual = residual, f.out = out, f.pre = (uint16_t *)pre;
  f.act = act, f.res_bf16 = residual_dtype == RET_BF16, f.out_bf16 = out_dtype == RET_BF16;
  hipStream_t st = (hipStream_t)hip_stream;
  if (few(M, N, K)) {
    const int m = (int)M;
    return rec_status(m == 1   ? launch_rows<1, 4>(x, w, m, N, K, x_ld, f, st)
                      : m == 2 ? launch_rows<2, 4>(x, w, m, N, K, x_ld, f, st)
                      : m <= 4 ? launch_rows<4, 4>(x, w, m, N, K, x_ld, f, st)
                      : m <= 8 ? launch_rows<8, 4>(x, w, m, N, K, x_ld, f, st)
                               : launch_rows<16, 4>(x, w, m, N, K, x_ld, f, st));
  }
  if (batch(M, N, K)) {
    const int m = (int)M;
    return rec_status(m <= 16   ? launch_batch<1>(x, w, m, N, K, x_ld, f, st)
                      : m <= 32 ? launch_batch<2>(x, w, m, N, K, x_ld, f, st)
                                : launch_batch<4>(x, w, m, N, K, x_ld, f, st));
  }
  MmArgs a = {};
  a.p = (const uint16_t *)x, a.q = (const uint16_t *)w, a.ldp = x_ld, a.ldq = K;
  a.M = M, a.N = N, a.K = K, a.f = f;
  return rec_status(mm_forward(a, workspace, st));
}

extern "C" size_t linear_bwd_workspace_bytes(long long M, int N, int K) {
  if (check_sizes(M, N, K) != RET_OK || M == 0) return 0;
  return bwd_ws(M, N, K).bytes;
}

extern "C" ret_status_t linear_bwd(const void *x, const void *w, const void *d_o, const void *pre, void *dx, void *dw,
                                   float *dbias, long long M, int N, int K, long long x_ld, int act,
                                   ret_dtype_t out_dtype, void *workspace, size_t workspace_bytes, void *hip_stream) {
  ret_status_t s = check_sizes(M, N, K);
  if (s != RET_OK) return s;
  if (!rec_dtype_ok(out_dtype)) return rec_fail(RET_ERR_INVALID_ARG, "unknown dtype");
  if (!act_ok(act)) return rec_fail(RET_ERR_INVALID_ARG, "unknown activation");
  if (x_ld < K) return rec_fail(RET_ERR_INVALID_ARG, "a row stride is shorter than its row");
  if (x_ld > (1LL << 31)) return rec_fail(RET_ERR_UNSUPPORTED, "x_ld too large");
  if (M > 0 && (!d_o || (act && !pre) || (dx && !w) || (dw && !x)))
    return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  const size_t oe = rec_esize(out_dtype);
  if (!rec_aligned(x, 2) || !rec_aligned(w, 2) || !rec_aligned(d_o, 2) || !rec_aligned(pre, 2) ||
      !rec_aligned(dx, oe) || !rec_aligned(dw, oe) || !rec_aligned(dbias, 4))
    return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const BwdWs v = bwd_ws(M, N, K);
  const size_t need = M > 0 ? v.bytes : 0, mn = (size_t)M * N * 2;
  if (need && (!workspace || workspace_bytes < need))
    return rec_fail(RET_ERR_WORKSPACE, "workspace of %zu bytes needed", need);
  const RecSpan ins[] = {rec_rows("x", dw ? x : nullptr, M, x_ld, K, 2), {"w", dx ? w : nullptr, (size_t)N * K * 2},
                         {"d_o", d_o, mn}, {"pre", act ? pre : nullptr, mn}};
  const RecSpan outs[] = {{"dx", dx, (size_t)M * K * oe}, {"dw", dw, (size_t)N * K * oe}, {"dbias", dbias, (size_t)N * 4},
                          {"workspace", workspace, need}};
  if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
  if (need && !rec_aligned(workspace, 16)) return rec_fail(RET_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  hipStream_t st = (hipStream_t)hip_stream;
  char *ws = (char *)workspace;
  const uint16_t *dz = (const uint16_t *)d_o;
  long long ldz = N;
  const bool make_dz = act && (dx || dw) && M > 0;
  if (make_dz) dz = (const uint16_t *)(ws + v.dz), ldz = v.ldz;
  float *part = (float *)(ws + v.bias);
  if (M > 0 && (make_dz || dbias))
    hipLaunchKernelGGL(dz_kernel, dim3((unsigned)v.parts, (unsigned)rec_cdiv(N, 512)), dim3(256), 0, st,
                       (const uint16_t *)d_o, (const uint16_t *)pre, make_dz ? (uint16_t *)dz : nullptr,
                       dbias ? part : nullptr, M, N, v.ldz, v.parts, act);
  if (dbias)
    hipLaunchKernelGGL(bias_join_kernel, dim3((unsigned)rec_cdiv(N, 64)), dim3(1024), 0, st, part, M > 0 ? v.parts : 0,
                       N, dbias);
  hipError_t e = hipGetLastError();
  Finish f = {};
  f.out_bf16 = out_dtype == RET_BF16;
  MmArgs a = {};
  a.p = dz, a.ldp = ldz;
  if (e == hipSuccess && dx && M > 0) {
    f.out = dx;
    a.q = (const uint16_t *)w, a.ldq = K, a.M = M, a.N = K, a.K = N, a.f = f;
    e = mm_dx(a, ws + v.product, st);
  }
  if (e == hipSuccess && dw) {
    f.out = dw;
    a.q = (const uint16_t *)x, a.ldq = x_ld, a.M = N, a.N = K, a.K = M, a.f = f;
    e = mm_dw(a, ws + v.product, st);
  }
  return rec_status(e);
}
