// Products with bias, activation and residual, and their gradients (language.h): the entry points, the
// product for few tokens, and the elementwise part of the gradients.  linear_mm.hpp has the tiled
// product.
#include "linear.hpp"

using namespace ret;

namespace {

// --------------------------------------------------------------------------- few tokens
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;

// Eight bf16 elements as they are, the first n of them (any alignment).
__device__ __forceinline__ Words4 raw8(const uint16_t *p, int n) {
  Words4 v = {{0u, 0u, 0u, 0u}};
  if (n >= 8) return *(const Words4 *)p;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) v.w[i / 2] |= (uint32_t)p[i] << (i % 2 * 16);
  return v;
}

// A wave takes RW rows of w, which it reads at full width, a lane 8 k of each 512; M tokens at most.  The
// lanes' RW M sums are added so that each step halves their number: value i ends in lane i 64 / (RW M).
// Bound by the launch and the way from memory: one token, N 4096, K 2048 (16.8 MB).
template <int M, int RW>
__global__ __launch_bounds__(256) void rows_kernel(const uint16_t *x, const uint16_t *w, int tokens, int N, int K,
                                                   long long x_ld, Finish f) {
  constexpr int C = M * RW, UNROLL = M <= 2 ? 4 : M <= 8 ? 2 : 1;
  static_assert(C <= 64 && (C & (C - 1)) == 0, "sums of a wave");
  const int lane = threadIdx.x & 63;
  const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * RW;
  if (n0 >= N) return;
  float acc[C] = {};  // [RW][M]
  auto add = [&](const Words4 (&wv)[RW], const Words4 &xv, int m) {
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[r * M + m] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, wv[r].w[i]),
                                                         __builtin_bit_cast(bf16x2, xv.w[i]), acc[r * M + m], false);
  };
  const int whole = K / 512 * 512;
#pragma unroll UNROLL
  for (int k = lane * 8; k < whole; k += 512) {
    Words4 wv[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) wv[r] = *(const Words4 *)(w + (long long)min(n0 + r, N - 1) * K + k);
#pragma unroll
    for (int m = 0; m < M; ++m) add(wv, *(const Words4 *)(x + min(m, tokens - 1) * x_ld + k), m);
  }
  if (whole < K) {
    const int k = whole + lane * 8;
    Words4 wv[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) wv[r] = raw8(w + (long long)min(n0 + r, N - 1) * K + k, K - k);
#pragma unroll
    for (int m = 0; m < M; ++m) add(wv, raw8(x + min(m, tokens - 1) * x_ld + k, K - k), m);
  }
  int n = C;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    if (n > 1) {
      n /= 2;
#pragma unroll
      for (int i = 0; i < C / 2; ++i)
        if (i < n) {
          const bool up = lane & off;
          const float mine = up ? acc[i + n] : acc[i], other = up ? acc[i] : acc[i + n];
          acc[i] = mine + __shfl_xor(other, off, 64);
        }
    } else {
      acc[0] += __shfl_xor(acc[0], off, 64);
    }
  }
  const int value = lane / (64 / C), m = value % M, col = n0 + value / M;
  if (lane % (64 / C) == 0 && m < tokens && col < N) {
    float v = acc[0];
    const long long at = (long long)m * N + col;
    if (f.bias) v += bf2f(f.bias[col]);
    if (f.pre) f.pre[at] = f2bf(v);
    v = act_value(v, f.act);
    if (f.residual) v += load_elem(f.residual, at, f.res_bf16);
    store_elem(f.out, at, v, f.out_bf16);
  }
}

// ----------------------------------------------------------------- dz and the bias's gradient
// Columns blockIdx.y * 512 + 8 lane .., rows blockIdx.x * 4 + wave, then parts * 4 further on.
// dz [M][ldz] (columns behind N zero) and one partial row of sums a workgroup; either may be NULL.
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
constexpr long long FEW = 16;  // tokens that rows_kernel serves

template <int M, int RW>
hipError_t launch_rows(const void *x, const void *w, int tokens, int N, int K, long long x_ld, const Finish &f,
                       hipStream_t st) {
  hipLaunchKernelGGL((rows_kernel<M, RW>), dim3((unsigned)rec_cdiv(N, 4 * RW)), dim3(256), 0, st, (const uint16_t *)x,
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
  if (check_sizes(M, N, K) != RET_OK || M <= FEW) return 0;
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
  if (M <= FEW) {
    const int m = (int)M;
    return rec_status(m == 1   ? launch_rows<1, 2>(x, w, m, N, K, x_ld, f, st)
                      : m == 2 ? launch_rows<2, 2>(x, w, m, N, K, x_ld, f, st)
                      : m <= 4 ? launch_rows<4, 2>(x, w, m, N, K, x_ld, f, st)
                      : m <= 8 ? launch_rows<8, 2>(x, w, m, N, K, x_ld, f, st)
                               : launch_rows<16, 4>(x, w, m, N, K, x_ld, f, st));
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
