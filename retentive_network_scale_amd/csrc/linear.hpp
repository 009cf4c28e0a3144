// What the products of language.h share: activations, the way from a sum to the output, and the plan of a
// product (linear_mm.hpp has its kernel).
#pragma once

#include <algorithm>
#include <type_traits>

#include "language.hpp"

namespace ret {

constexpr int BK = 64;  // k of a tile

// ------------------------------------------------------------------------ activations
// gelu(z) = z Phi(z) = max(z, 0) - |z| Phi(-|z|), so that small results keep their relative accuracy, in two forms.
//
// For results that leave in bf16: Phi(-a), a >= 0, as 2^p(a), p a polynomial fitted to log2 Phi(-a) on 0..6 (a minimax
// fit of degree 7 made for this file; 5.7e-6 of the value at most, evaluated in fp32).  Behind 6 it falls faster
// than Phi does, to zero at 14: good to 4e-4 of the value at 7, 6e-3 at 8, where that is 6e-16.
__device__ __forceinline__ float normal_tail(float a) {
  float p = -1.834846444e-06f;
  p = fmaf(p, a, 6.159897748e-05f);
  p = fmaf(p, a, -9.305300191e-04f);
  p = fmaf(p, a, 8.507910185e-03f);
  p = fmaf(p, a, -5.396010354e-02f);
  p = fmaf(p, a, -4.584643543e-01f);
  p = fmaf(p, a, -1.151251078e+00f);
  p = fmaf(p, a, -9.999952912e-01f);
  return __builtin_amdgcn_exp2f(p);
}
__device__ __forceinline__ float gelu_bf16(float z) {
  const float a = fminf(fabsf(z), 14.0f);
  return fmaf(0.5f, fabsf(z), 0.5f * z) - a * normal_tail(a);
}
// For results that leave in fp32: Phi(-a) = e^(-a a / 2) m(a), m a polynomial in 1 / (1 + 0.35 a) (of degree 7, fitted
// here for the relative error on 0..14, 5.2 half steps of fp32).  (10 + 2 a a) half steps of the value in all, most of
// them the exponential's argument's, until it leaves fp32's range behind 13.  23 issue slots against 17.
__device__ __forceinline__ float gelu_f32(float z) {
  const float a = fminf(fabsf(z), 14.0f), t = __builtin_amdgcn_rcpf(fmaf(0.35f, a, 1.0f));
  float m = 4.8942431807518005e-02f;
  m = fmaf(m, t, -2.0211923122406006e-01f);
  m = fmaf(m, t, 2.4064074456691742e-01f);
  m = fmaf(m, t, -1.7023373395204544e-02f);
  m = fmaf(m, t, 1.5596145391464233e-01f);
  m = fmaf(m, t, 1.3335511088371277e-01f);
  m = fmaf(m, t, 1.4027033746242523e-01f);
  m = fmaf(m, t, -2.7315489205648191e-05f);
  return fmaf(0.5f, fabsf(z), 0.5f * z) - a * (__builtin_amdgcn_exp2f(a * (-0.5f * kLog2e) * a) * m);
}
// Phi(z) + z phi(z), for the gradients, whose sums (dbias) stay in fp32: p is of degree 10 here, fitted on 0..6 for
// the absolute error, 3.2e-8 at most; behind 6 it falls as the other does.
__device__ __forceinline__ float gelu_slope(float z) {
  const float a = fminf(fabsf(z), 14.0f);
  float p = -2.643092323e-08f;
  p = fmaf(p, a, 8.022586258e-07f);
  p = fmaf(p, a, -1.040739517e-05f);
  p = fmaf(p, a, 7.340624143e-05f);
  p = fmaf(p, a, -2.696193114e-04f);
  p = fmaf(p, a, -2.047829366e-05f);
  p = fmaf(p, a, 6.972098723e-03f);
  p = fmaf(p, a, -5.245869979e-02f);
  p = fmaf(p, a, -4.592149258e-01f);
  p = fmaf(p, a, -1.151104927e+00f);
  p = fmaf(p, a, -1.000000000e+00f);
  const float t = __builtin_amdgcn_exp2f(p);
  const float phi = 0.3989422804f * __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2e));
  return fmaf(z, phi, z >= 0.0f ? 1.0f - t : t);
}
__device__ __forceinline__ float act_value(float z, int act, bool out_bf16) {
  if (act == LINEAR_ACT_GELU) return out_bf16 ? gelu_bf16(z) : gelu_f32(z);
  return act == LINEAR_ACT_SILU ? z * sigmoid(z) : z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == LINEAR_ACT_GELU) return gelu_slope(z);
  const float s = sigmoid(z);
  return act == LINEAR_ACT_SILU ? s * (1.0f + z * (1.0f - s)) : 1.0f;
}

// --------------------------------------------------------------------------- epilogue
struct Finish {
  const uint16_t *bias;
  const void *residual;
  void *out;
  uint16_t *pre;
  int act, res_bf16, out_bf16;
  __host__ __device__ bool fine() const { return act == LINEAR_ACT_GELU && !out_bf16; }
};

// Eight elements of the residual on their way, of either type.
struct Residual8 {
  Raw8<uint16_t> h;
  Raw8<float> s;
  __device__ __forceinline__ void load(const Finish &f, long long at, int left) {
    if (!f.residual) return;
    if (f.res_bf16)
      h.load((const uint16_t *)f.residual + at, left);
    else
      s.load((const float *)f.residual + at, left);
  }
  __device__ __forceinline__ void add(const Finish &f, float (&z)[8]) const {
    if (!f.residual) return;
    float r[8];
    if (f.res_bf16)
      h.get(r);
    else
      s.get(r);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += r[i];
  }
};

// Eight of z's elements, `left` of which exist, at `at` of [M][N]: bias (zero where there is none), activation,
// residual.  FINE: the activation is gelu for fp32.
template <bool FINE>
__device__ __forceinline__ void finish8(const Finish &f, long long at, int left, const float (&bias)[8],
                                        const Residual8 &res, float (&z)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] += bias[i];
  if (f.pre) store8(f.pre + at, left, z);
  if constexpr (FINE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = gelu_f32(z[i]);
  } else if (f.act == LINEAR_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = gelu_bf16(z[i]);
  } else if (f.act == LINEAR_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= sigmoid(z[i]);
  }
  res.add(f, z);
  if (!FINE && f.out_bf16)
    store8((uint16_t *)f.out + at, left, z);
  else
    store8((float *)f.out + at, left, z);
}
__device__ __forceinline__ void finish8(const Finish &f, long long at, int left, const float (&bias)[8],
                                        const Residual8 &res, float (&z)[8]) {
  if (f.fine())
    finish8<true>(f, at, left, bias, res, z);
  else
    finish8<false>(f, at, left, bias, res, z);
}

struct MmArgs {
  const uint16_t *p, *q;
  long long ldp, ldq;
  long long M;  // P's rows
  int N;        // Q's rows
  long long K;
  long long kpart;  // k of a part, a multiple of BK
  float *part;      // [parts][M][N], or NULL: finish
  Finish f;
};

struct MmPlan {
  int rows, cols;  // of a tile: 64 x 64, 64 x 128, 128 x 128 or 256 x 256
  int parts;
  long long kpart;
  size_t bytes;  // of the parts' sums
  double us;     // the estimate
};

// Tile and parts of k by an estimate of the time, in us.  A step (64 k) of a tile takes `alone` where a CU has
// one workgroup and `each` for every workgroup of the fullest CU (measured with 16 tokens, and with
// 1024 tiles, K 2048: a 128 x 128 tile fetches twice the bytes of a 256 x 256 one for its work, and a 64 x 64
// one four times); `end` is its way from sums to output.  Parts of k cost their sums' way to memory and back
// and a launch, 5 us.  At M 16384, N 4096, K 2048 tiles of 256 x 256 take 215 us and of 128 x 128 248; at M 1024 64 x 64,
// 128 x 128 and 256 x 256 31, 25 and 47, at M 200 12, 21 and 45; M 777, N 2304, K 1000 with 64 x 128 12.1, with
// the better of its neighbours 13.3; four parts for M 16, N 2048, K 4096: 18.8 -> 10.7 us.
inline MmPlan mm_plan(long long M, long long N, long long K) {
  struct {
    int rows, cols;
    double alone, each, end;
  } const kinds[] = {{64, 64, 0.27, 0.23, 0.7}, {64, 128, 0.38, 0.35, 1.0}, {128, 128, 0.50, 0.53, 1.5}, {256, 256, 1.25, 1.70, 3.0}};
  const long long steps = std::max<long long>(1, rec_cdiv(K, BK));
  MmPlan best = {};
  double least = 1e300;
  for (const auto &k : kinds) {
    const long long tiles = std::max<long long>(1, rec_cdiv(M, k.rows) * rec_cdiv(N, k.cols));
    for (long long parts = 1; parts <= 32 && (parts == 1 || 2 * parts <= steps); parts *= 2) {
      const long long each = rec_cdiv(steps, parts), real = rec_cdiv(steps, each);
      if (real != parts || !rec_grid_ok((double)tiles, 512)) continue;
      const double fullest = (double)rec_cdiv(tiles * parts, 256);
      double t = each * std::max(k.alone, fullest * k.each) + k.end;
      if (parts > 1) t += 5.0 + (double)M * N * (8 * parts + 2) / 4.5e6;
      if (t < least) {
        least = t;
        best.rows = k.rows;
        best.cols = k.cols;
        best.parts = (int)parts;
        best.kpart = each * BK;
      }
    }
  }
  best.us = least;
  best.bytes = best.parts > 1 ? rec_align((size_t)best.parts * M * N * 4) : 0;
  return best;
}

// The products on `ws`, mm_plan's bytes: forward (both operands with k along their rows), dx (P with k
// along, Q across) and dw (both across).
hipError_t mm_forward(MmArgs a, void *ws, hipStream_t st);
hipError_t mm_forward_fine(MmArgs a, void *ws, hipStream_t st);  // gelu for fp32
hipError_t mm_dx(MmArgs a, void *ws, hipStream_t st);
hipError_t mm_dw(MmArgs a, void *ws, hipStream_t st);

}  // namespace ret
