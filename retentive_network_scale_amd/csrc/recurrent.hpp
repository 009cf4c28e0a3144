// Host and device helpers shared by the recurrent-layer operators (recurrent.h).
#pragma once

#include <stdarg.h>
#include <stdio.h>

#include "common.hpp"
#include "recurrent.h"

// Defined in abi.hip: records the message returned by retention_last_error().
ret_status_t retention_fail_(ret_status_t s, const char *msg);

namespace ret {

// ------------------------------------------------------------------ host side
inline ret_status_t rec_fail(ret_status_t s, const char *fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return retention_fail_(s, msg);
}

inline ret_status_t rec_status(hipError_t e) {
  return e == hipSuccess ? retention_fail_(RET_OK, "") : rec_fail(RET_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
}

inline size_t rec_esize(ret_dtype_t t) { return t == RET_BF16 ? 2 : 4; }
inline bool rec_dtype_ok(ret_dtype_t t) { return t == RET_F32 || t == RET_BF16; }
inline size_t rec_align(size_t x) { return (x + 255) & ~(size_t)255; }
inline long long rec_cdiv(long long a, long long b) { return (a + b - 1) / b; }

// A tensor of a call: its bytes from p on (rows * ld less the gap behind the last row).
struct RecSpan {
  const char *name;
  const void *p;
  size_t n;
};
inline RecSpan rec_rows(const char *name, const void *p, long long rows, long long ld, long long width, size_t e) {
  return {name, p, p && rows > 0 ? (size_t)((rows - 1) * ld + width) * e : 0};
}
inline bool rec_overlap(const RecSpan &a, const RecSpan &b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + b.n && b0 < a0 + a.n;
}
// The first output that meets an input or another output, as an error; RET_OK if none.
template <int NI, int NO>
inline ret_status_t rec_check_overlap(const RecSpan (&ins)[NI], const RecSpan (&outs)[NO]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (rec_overlap(outs[o], ins[i]))
        return rec_fail(RET_ERR_INVALID_ARG, "%s overlaps %s", outs[o].name, ins[i].name);
    for (int i = 0; i < o; ++i)
      if (rec_overlap(outs[o], outs[i]))
        return rec_fail(RET_ERR_INVALID_ARG, "%s overlaps %s", outs[o].name, outs[i].name);
  }
  return RET_OK;
}
// Whether a launch's threads can be counted in 32 bits, as HIP requires.
inline bool rec_grid_ok(double blocks, int threads) { return blocks * threads < 4294967296.0; }
inline bool rec_aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// ------------------------------------------------------------------ device side
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kLog2eLow = (float)(1.4426950408889634 - (double)1.4426950408889634f);

// Four consecutive elements to base + off: the first n of them, or all, aligned (VEC).
template <bool VEC>
__device__ __forceinline__ void store4(void *base, long long off, int n, const float (&r)[4], bool bf16) {
  if constexpr (VEC) {
    if (bf16)
      *(uint2 *)((uint16_t *)base + off) = make_uint2(pack_bf2(r[0], r[1]), pack_bf2(r[2], r[3]));
    else
      *(float4 *)((float *)base + off) = make_float4(r[0], r[1], r[2], r[3]);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < n) store_elem(base, off + c, r[c], bf16);
  }
}

// log(1 + e^x) = max(x, 0) + log1p(e), e = e^-|x|.  The exponential's argument is taken to
// base 2 in two parts, so that far negative x keep their relative accuracy; 1 + e rounds,
// and what it lost is added to the logarithm (over s = 1 + e, which matters only where s
// is near 1).  The hardware's exp2 and log2 are good to 2 half steps, near 1 too: 3 half
// steps in all, measured over e^-18 .. 20.  Below -150 e is 0 in fp32 anyway: x of -inf or
// the type's lowest value (a token that does nothing) gives 0; NaN stays NaN.
__device__ __forceinline__ float softplus(float x) {
  const float a = -fabsf(x), m = a < -150.0f ? -150.0f : a;
  const float hi = m * kLog2e, lo = fmaf(m, kLog2eLow, fmaf(m, kLog2e, -hi));
  float e = __builtin_amdgcn_exp2f(hi);
  e = fmaf(e, lo * kLn2, e);
  const float s = 1.0f + e, lost = e - (s - 1.0f);
  return (x > 0.0f ? x : 0.0f) + fmaf(__builtin_amdgcn_logf(s), kLn2, lost);
}

// x / (1 + e^-x) to within two roundings: the exponential's argument to base 2 in two parts
// around its nearest whole number, the quotient with one correction.  The convolution uses
// it, since its result may be rounded to bf16 and then drive a state in fp32: a few units
// of 2^-24 more turn more of the values next to a rounding border into the other neighbour.
__device__ __forceinline__ float silu(float x) {
  const float t = __builtin_amdgcn_fmed3f(-x, -150.0f, 150.0f);
  float hi = t * kLog2e;
  asm("" : "+v"(hi));  // the product as rounded, also where it is subtracted from
  const float lo = fmaf(t, kLog2eLow, fmaf(t, kLog2e, -hi)), n = rintf(hi);
  const float d = 1.0f + ldexpf(__builtin_amdgcn_exp2f((hi - n) + lo), (int)n), r = __builtin_amdgcn_rcpf(d);
  const float q = x * r;
  return __builtin_amdgcn_div_fixupf(fmaf(fmaf(-q, d, x), r, q), d, x);
}

// The same within a few roundings, where the result is not rounded on the way.
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

}  // namespace ret
