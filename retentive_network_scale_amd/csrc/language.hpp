// Device helpers shared by the operators of language.h (host helpers: recurrent.hpp).
#pragma once

#include "language.h"
#include "recurrent.hpp"

namespace ret {

// Eight consecutive elements in one access (two for fp32), whatever their alignment: the
// global memory path takes any address, and a row of odd length costs a few lines more.
struct __attribute__((packed, aligned(2))) Words4 {
  uint32_t w[4];
};
// Eight elements as they come from memory, for loads that are to be under way while others are used.
template <typename T>
struct Raw8 {
  Words4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T *p, int n) {
    if (n >= 8) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = ((const Words4 *)p)[i];
    } else {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = {{0u, 0u, 0u, 0u}};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) {
          if constexpr (sizeof(T) == 2)
            w[0].w[i / 2] |= (uint32_t)p[i] << (i % 2 * 16);
          else
            w[i / 4].w[i % 4] = __float_as_uint(p[i]);
        }
    }
  }
  __device__ __forceinline__ void get(float (&r)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 2)
        r[i] = __uint_as_float(i % 2 ? w[0].w[i / 2] & 0xffff0000u : w[0].w[i / 2] << 16);
      else
        r[i] = __uint_as_float(w[i / 4].w[i % 4]);
    }
  }
};

// Eight elements, the first n of them (n <= 0: none; the others are zero).
template <typename T>
__device__ __forceinline__ void load8(const T *p, int n, float (&r)[8]) {
  Raw8<T> v;
  v.load(p, n);
  v.get(r);
}
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&r)[8]) {
  load8(p, 8, r);
}
__device__ __forceinline__ void store8(uint16_t *p, const float (&r)[8]) {
  Words4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.w[i] = pack_bf2(r[2 * i], r[2 * i + 1]);
  *(Words4 *)p = v;
}
__device__ __forceinline__ void store8(float *p, const float (&r)[8]) {
  Words4 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a.w[i] = __float_as_uint(r[i]);
    b.w[i] = __float_as_uint(r[4 + i]);
  }
  *(Words4 *)p = a;
  *(Words4 *)(p + 4) = b;
}

template <typename T>
__device__ __forceinline__ void store8(T *p, int n, const float (&r)[8]) {
  if (n >= 8) {
    store8(p, r);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) store_elem(p, i, r[i], sizeof(T) == 2);
  }
}

// Calls f with a null pointer of the element type that each dtype stands for.
template <typename F>
inline auto with_types(ret_dtype_t in, ret_dtype_t out, F f) {
  if (in == RET_BF16) return out == RET_BF16 ? f((uint16_t *)0, (uint16_t *)0) : f((uint16_t *)0, (float *)0);
  return out == RET_BF16 ? f((float *)0, (uint16_t *)0) : f((float *)0, (float *)0);
}

}  // namespace ret
