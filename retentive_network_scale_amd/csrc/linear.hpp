// What the products of language.h share: activations, the way from a sum to the output, and the plan of a
// product (linear_mm.hpp has its kernel).
#pragma once

#include <algorithm>
#include <type_traits>

#include "language.hpp"

namespace ret {


constexpr int BK = 64;  // k of a tile

// ------------------------------------------------------------------------ activations
// Phi(-a) for a >= 0 as 2^p(a), p a polynomial fitted to log2 Phi(-a) on 0..6 (a minimax fit of degree 7
// made for this file; 5.7e-6 of the value at most, evaluated in fp32); behind 6 it stays at 1e-9.
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
// z Phi(z) = max(z, 0) - |z| Phi(-|z|), so that small results keep their relative accuracy.
__device__ __forceinline__ float gelu(float z) {
  const float a = fminf(fabsf(z), 6.0f);
  return fmaf(0.5f, fabsf(z), 0.5f * z) - a * normal_tail(a);
}
// Phi(z) + z phi(z), for the gradients, whose sums (dbias) stay in fp32: p is of degree 10 here, fitted for
// the absolute error, 3.2e-8 at most.
__device__ __forceinline__ float gelu_slope(float z) {
  const float a = fminf(fabsf(z), 6.0f);
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
__device__ __forceinline__ float act_value(float z, int act) {
  return act == LINEAR_ACT_GELU ? gelu(z) : act == LINEAR_ACT_SILU ? z * sigmoid(z) : z;
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
};

struct __attribute__((packed, aligned(2))) Words2 {
  uint32_t w[2];
};
// Four consecutive elements, whatever their alignment.
__device__ __forceinline__ void load4(const void *p, long long off, bool bf16, float (&r)[4]) {
  if (bf16) {
    const Words2 v = *(const Words2 *)((const uint16_t *)p + off);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r[2 * i] = __uint_as_float(v.w[i] << 16);
      r[2 * i + 1] = __uint_as_float(v.w[i] & 0xffff0000u);
    }
  } else {
    const Words4 v = *(const Words4 *)((const float *)p + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __uint_as_float(v.w[i]);
  }
}
__device__ __forceinline__ void put4(void *p, long long off, bool bf16, const float (&r)[4]) {
  if (bf16) {
    *(Words2 *)((uint16_t *)p + off) = {{pack_bf2(r[0], r[1]), pack_bf2(r[2], r[3])}};
  } else {
    Words4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.w[i] = __float_as_uint(r[i]);
    *(Words4 *)((float *)p + off) = v;
  }
}

// z's elements n..n+3 of row m (of N a row), as far as there are any: bias, activation, residual.
__device__ __forceinline__ void finish4(const Finish &f, long long m, int n, int N, float (&z)[4]) {
  const long long at = m * N + n;
  if (n + 4 <= N) {
    float r[4];
    if (f.bias) {
      load4(f.bias, n, true, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] += r[i];
    }
    if (f.pre) put4(f.pre, at, true, z);
    if (f.act)
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = act_value(z[i], f.act);
    if (f.residual) {
      load4(f.residual, at, f.res_bf16, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] += r[i];
    }
    put4(f.out, at, f.out_bf16, z);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) {
        float v = z[i];
        if (f.bias) v += bf2f(f.bias[n + i]);
        if (f.pre) f.pre[at + i] = f2bf(v);
        v = act_value(v, f.act);
        if (f.residual) v += load_elem(f.residual, at + i, f.res_bf16);
        store_elem(f.out, at + i, v, f.out_bf16);
      }
  }
}

struct MmArgs {
  const uint16_t *p, *q;
  long long ldp, ldq;
  long long M;  // P's rows
  int N;        // Q's rows
  long long K;
  long long kpart;  // k of a part, a multiple of BK
  float *part;      // [parts][M][N rounded up to 4], or NULL: finish
  Finish f;
};

struct MmPlan {
  int tile;  // rows and columns of a tile: 64, 128 or 256
  int parts;
  long long kpart;
  size_t bytes;  // of the parts' sums
};

// The largest tile that still gives every CU a workgroup, and else parts of k until there are about
// two a CU, none shorter than four tiles of k.
inline MmPlan mm_plan(long long M, long long N, long long K) {
  MmPlan p;
  auto tiles = [&](int t) { return rec_cdiv(M, t) * rec_cdiv(N, t); };
  p.tile = tiles(256) >= 256 ? 256 : tiles(128) >= 256 ? 128 : 64;
  const long long steps = std::max<long long>(1, rec_cdiv(K, BK)), n = std::max<long long>(1, tiles(p.tile));
  long long parts = n >= 256 ? 1 : std::min<long long>(rec_cdiv(512, n), steps / 4);
  parts = std::max<long long>(1, std::min<long long>(parts, 64));
  p.kpart = rec_cdiv(steps, parts) * BK;
  p.parts = (int)std::max<long long>(1, rec_cdiv(K, p.kpart));
  p.bytes = p.parts > 1 ? rec_align((size_t)p.parts * M * ((N + 3) / 4 * 4) * 4) : 0;
  return p;
}

// The products on `ws`, mm_plan's bytes: forward (both operands with k along their rows), dx (P with k
// along, Q across) and dw (both across).
hipError_t mm_forward(MmArgs a, void *ws, hipStream_t st);
hipError_t mm_dx(MmArgs a, void *ws, hipStream_t st);
hipError_t mm_dw(MmArgs a, void *ws, hipStream_t st);

}  // namespace ret
