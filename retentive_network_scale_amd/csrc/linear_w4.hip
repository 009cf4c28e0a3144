// Products with 4-bit weights for few tokens (recurrent.h): out = x W^T with
// W[n, k] = (q[n, k] - zero[n, g]) scale[n, g], g = k / group.
//
// The weights go to the matrix cores as whole numbers.  A nibble q placed in the top
// four mantissa bits of a bf16 with exponent 4 is exactly 16 + q, two of them per
// shift-and-mask of the packed word; a second product with the constant -(16 + zero)
// on the same accumulator takes the offset out again.  A group's sum is thus one of
// exact bf16 products in fp32, and its scale is applied in fp32.
//
// A workgroup covers 16 rows of W and up to 64 tokens; its waves share out the blocks
// of K (128 of them for groups of 128, 64 and 32 below) and meet in LDS.  Inside a
// block, lane (n = lane & 15, kq = lane >> 4) reads WORDS consecutive words of its row,
// eight weights each; a product step takes one word of every lane, so that the four kq
// cover WORDS * 8 apart ranges of K.  x is read by the same map.  Which k sits in which
// slot of a step does not matter, as long as both operands agree: the packed order
// (0 4 1 5 2 6 3 7) of a word's nibbles is matched by permuting x.
#include <algorithm>

#include "launch.hpp"
#include "recurrent.hpp"

using namespace ret;

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

struct W4Args {
  const uint16_t *x, *scale;
  const uint32_t *q;
  const uint8_t *zero;
  void *out;
  long long x_ld;
  int M, N, K, group, out_bf16;
};

// Eight elements of x, as loaded and in the order 0 4 1 5 2 6 3 7.
template <bool VEC>
__device__ __forceinline__ u32x4 load_x(const uint16_t *p) {
  if constexpr (VEC) return *(const u32x4 *)p;
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (uint32_t)p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
  return v;
}
__device__ __forceinline__ bf16x8 permuted(u32x4 v) {
  u32x4 r;
  r[0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100);
  r[1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302);
  r[2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100);
  r[3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302);
  return __builtin_bit_cast(bf16x8, r);
}

// Eight weights of a word as 16 + q, same order.
__device__ __forceinline__ bf16x8 unpack(uint32_t w) {
  u32x4 r;
  r[0] = (w << 3 & 0x00780078u) | 0x41804180u;
  r[1] = (w >> 1 & 0x00780078u) | 0x41804180u;
  r[2] = (w >> 5 & 0x00780078u) | 0x41804180u;
  r[3] = (w >> 9 & 0x00780078u) | 0x41804180u;
  return __builtin_bit_cast(bf16x8, r);
}

// MT tiles of 16 tokens; WORDS words of a row per lane and block; WAVES waves.
template <int MT, int WORDS, int WAVES, bool VEC>
__global__ __launch_bounds__(WAVES * 64) void w4_kernel(W4Args a) {
  __shared__ f32x4 red[WAVES][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, kq = lane >> 4;
  const int n = blockIdx.x * 16 + col, nr = min(n, a.N - 1), m0 = blockIdx.y * MT * 16;
  constexpr int KB = WORDS * 32;  // k per block
  constexpr int U = 16 / (WORDS * MT) < 1 ? 1 : 16 / (WORDS * MT) > 4 ? 4 : 16 / (WORDS * MT);
  const int groups = a.K / a.group;
  const uint32_t *q = a.q + (long long)nr * (a.K / 8) + kq * WORDS;
  const uint16_t *scale = a.scale + (long long)nr * groups;
  const uint8_t *zero = a.zero ? a.zero + (long long)nr * groups : nullptr;
  const uint16_t *x[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) x[m] = a.x + (long long)min(m0 + m * 16 + col, a.M - 1) * a.x_ld + kq * WORDS * 8;
  f32x4 tot[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) tot[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int blocks = a.K / KB;
  for (int kb0 = wave; kb0 < blocks; kb0 += WAVES * U) {
    // everything that U blocks need is requested before the first is used: a wave has few
    // blocks, and their latency is most of its time.  Blocks behind the end: the last one
    // again, with scale 0.
    uint32_t w[U][WORDS], z[U];
    u32x4 xv[U][MT][WORDS];
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(kb0 + u * WAVES, blocks - 1), g = (int)((long long)kb * KB / a.group);
      if constexpr (WORDS == 4) {
        const u32x4 v = *(const u32x4 *)(q + (long long)kb * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[u][i] = v[i];
      } else if constexpr (WORDS == 2) {
        const uint2 v = *(const uint2 *)(q + (long long)kb * 8);
        w[u][0] = v.x;
        w[u][1] = v.y;
      } else {
        w[u][0] = q[(long long)kb * 4];
      }
      z[u] = zero ? zero[g] & 15u : 8u;
      s[u] = kb0 + u * WAVES < blocks ? bf2f(scale[g]) : 0.0f;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < WORDS; ++i) xv[u][m][i] = load_x<VEC>(x[m] + (long long)kb * KB + i * 8);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t off = (0xC180u | z[u] << 3) * 0x10001u;
      const bf16x8 minus = __builtin_bit_cast(bf16x8, u32x4{off, off, off, off});
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
          const bf16x8 xp = permuted(xv[u][m][i]);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xp, unpack(w[u][i]), acc, 0, 0, 0);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xp, minus, acc, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[m][i] += s[u] * acc[i];
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) red[wave][m][lane] = tot[m];
  __syncthreads();
  // lane (n = lane & 15, rows (lane >> 4) * 4 ..) of tile m
  for (int m = wave; m < MT; m += WAVES) {
    f32x4 y = red[0][m][lane];
#pragma unroll
    for (int k = 1; k < WAVES; ++k) y += red[k][m][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = m0 + m * 16 + kq * 4 + i;
      if (row < a.M && n < a.N) store_elem(a.out, (long long)row * a.N + n, y[i], a.out_bf16);
    }
  }
}

template <int MT, int WORDS, int WAVES>
hipError_t launch_w(const W4Args &a, bool vec, hipStream_t st) {
  const dim3 grid((unsigned)rec_cdiv(a.N, 16), (unsigned)rec_cdiv(a.M, MT * 16));
  if (vec)
    hipLaunchKernelGGL((w4_kernel<MT, WORDS, WAVES, true>), grid, dim3(WAVES * 64), 0, st, a);
  else
    hipLaunchKernelGGL((w4_kernel<MT, WORDS, WAVES, false>), grid, dim3(WAVES * 64), 0, st, a);
  return hipGetLastError();
}
// Sixteen waves a workgroup where the grid alone does not give every CU eight.
template <int MT>
hipError_t launch_mt(const W4Args &a, bool vec, hipStream_t st) {
  const bool few = rec_cdiv(a.N, 16) * rec_cdiv(a.M, MT * 16) <= 256;
  if (a.group % 128 == 0) return few ? launch_w<MT, 4, 16>(a, vec, st) : launch_w<MT, 4, 8>(a, vec, st);
  if (a.group == 64) return few ? launch_w<MT, 2, 16>(a, vec, st) : launch_w<MT, 2, 8>(a, vec, st);
  return few ? launch_w<MT, 1, 16>(a, vec, st) : launch_w<MT, 1, 8>(a, vec, st);
}

}  // namespace

namespace ret {

// The checks of linear_w4's arguments, as a message or nullptr.
const char *w4_refusal(const void *q, const void *scale, int N, int K, int group, bool *unsupported) {
  *unsupported = false;
  if (!q || !scale) return "NULL tensor pointer";
  if (N <= 0 || K <= 0 || group <= 0) return "sizes must be positive";
  if (!rec_aligned(q, 16)) return "q must be 16-byte aligned";
  if (!rec_aligned(scale, 2)) return "a pointer is not aligned to its elements";
  *unsupported = true;
  if (group != 32 && group != 64 && group % 128) return "group must be 32, 64 or a multiple of 128";
  if (K % group) return "K must be a multiple of group";
  return nullptr;
}

hipError_t launch_w4(const void *x, const void *q, const void *scale, const void *zero, void *out, int M, int N, int K,
                     int group, long long x_ld, bool out_bf16, hipStream_t st) {
  W4Args a;
  a.x = (const uint16_t *)x;
  a.q = (const uint32_t *)q;
  a.scale = (const uint16_t *)scale;
  a.zero = (const uint8_t *)zero;
  a.out = out;
  a.x_ld = x_ld;
  a.M = M;
  a.N = N;
  a.K = K;
  a.group = group;
  a.out_bf16 = out_bf16;
  const bool vec = x_ld % 8 == 0 && rec_aligned(x, 16);
  // Tokens per workgroup: 64 read a weight once; where that leaves CUs idle, fewer tokens
  // and more workgroups, whose weights then come from L2 (N / 16 workgroups apart, a
  // multiple of the eight dies in the usual case).
  const long long rows = rec_cdiv(N, 16);
  if (M > 32 && rows * rec_cdiv(M, 64) >= 512) return launch_mt<4>(a, vec, st);
  if (M > 16 && rows * rec_cdiv(M, 32) >= 512) return launch_mt<2>(a, vec, st);
  return launch_mt<1>(a, vec, st);
}

}  // namespace ret

extern "C" ret_status_t linear_w4(const void *x, const void *q, const void *scale, const void *zero, void *out, int M,
                                  int N, int K, int group, long long x_ld, ret_dtype_t out_dtype, void *hip_stream) {
  if (M < 0) return rec_fail(RET_ERR_INVALID_ARG, "sizes must be positive");
  if (!rec_dtype_ok(out_dtype)) return rec_fail(RET_ERR_INVALID_ARG, "unknown dtype");
  bool unsupported;
  if (const char *msg = w4_refusal(q, scale, N, K, group, &unsupported))
    return rec_fail(unsupported ? RET_ERR_UNSUPPORTED : RET_ERR_INVALID_ARG, "%s", msg);
  if (x_ld < K) return rec_fail(RET_ERR_INVALID_ARG, "a row stride is shorter than its row");
  if (M > W4_MAX_ROWS || x_ld > (1LL << 31)) return rec_fail(RET_ERR_UNSUPPORTED, "M or x_ld too large");
  if (M == 0) return rec_status(hipSuccess);
  if (!x || !out) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  const size_t oe = rec_esize(out_dtype);
  if (!rec_aligned(x, 2) || !rec_aligned(out, oe))
    return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const size_t ng = (size_t)N * (K / group);
  const RecSpan ins[] = {rec_rows("x", x, M, x_ld, K, 2), {"q", q, (size_t)N * (K / 2)}, {"scale", scale, ng * 2},
                         {"zero", zero, ng}};
  const RecSpan outs[] = {{"out", out, (size_t)M * N * oe}};
  const ret_status_t s = rec_check_overlap(ins, outs);
  if (s != RET_OK) return s;
  return rec_status(launch_w4(x, q, scale, zero, out, M, N, K, group, x_ld, out_dtype == RET_BF16,
                              (hipStream_t)hip_stream));
}
