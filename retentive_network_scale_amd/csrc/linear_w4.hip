// Products with 4-bit weights for few tokens (recurrent.h): out = x W^T with
// W[n, k] = (q[n, k] - zero[n, g]) scale[n, g], g = k / group.
//
// The weights go to the matrix cores as whole numbers.  A nibble q placed in the top
// four mantissa bits of a bf16 with exponent 4 is exactly 16 + q, two of them per
// shift-and-mask of the packed word; a second product with the constant -(16 + zero)
// on the same accumulator takes the offset out again.  A group's sum is thus one of
// exact bf16 products in fp32, and its scale is applied in fp32.
//
// A workgroup covers NN tiles of 16 rows of W and MT of 16 tokens, its waves share out K
// and meet in LDS.  Both operands go through LDS, a chunk of K at a time, requested while the
// chunk before is worked on and read from memory along the rows: lanes that fetched their
// matrix operands themselves, from 16 rows each, took 64 address cycles a load and met in
// few L2 channels (rows lie a power of two apart): 20 us for 64 tokens, N = 2048, K = 4096.
//
// Which k sits in which slot of a matrix step does not matter, as long as both operands
// agree: lane (n = lane & 15, kq = lane >> 4) takes WORDS consecutive words of its row,
// eight weights each, and a step takes one word of every lane.
#include <algorithm>

#include "launch.hpp"
#include "recurrent.hpp"

using namespace ret;

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

constexpr int KS = 8;  // waves of a workgroup

struct W4Args {
  const void *x;  // bf16, or fp32 where the kernel reads it in two parts
  const uint16_t *scale;
  const uint32_t *q;
  const uint8_t *zero;
  void *out;
  long long x_ld;
  int M, N, K, group, out_bf16;
  int *pos;  // a decode step's positions, advanced beside the products, or NULL
};

// Eight elements of x, and in the order 0 4 1 5 2 6 3 7, that of a word's nibbles below.
template <bool VEC>
__device__ __forceinline__ u32x4 load_x(const uint16_t *p) {
  if constexpr (VEC) return *(const u32x4 *)p;
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (uint32_t)p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
  return v;
}
__device__ __forceinline__ u32x4 permuted(u32x4 v) {
  u32x4 r;
  r[0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100);
  r[1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302);
  r[2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100);
  r[3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302);
  return r;
}

// Eight fp32 elements of x as two bf16 parts in that order, hi + lo, lo the remainder's: 2^-16 of
// the value at most is lost.
__device__ __forceinline__ void split_x(u32x4 a, u32x4 b, u32x4 &hi, u32x4 &lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float u = __uint_as_float(a[i]), v = __uint_as_float(b[i]);
    hi[i] = pack_bf2(u, v);
    lo[i] = pack_bf2(u - __uint_as_float(hi[i] << 16), v - __uint_as_float(hi[i] & 0xffff0000u));
  }
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

// NN tiles of 16 rows of W, MT tiles of 16 tokens; the KS waves share out the blocks of
// WORDS * 32 elements of K, which come KC elements a chunk.  XR: rows of x kept, 16 MT, or 4
// for at most four tokens, which leaves room for chunks twice as long (K = 2048 is one: 7.8 ->
// 5.4 us for one token, N 12288).  Bound by the latency of the launch and one dependent chain
// (load, LDS, matrix steps, the join), until N K is some 2^27 (M 16, N 8192, K 8192: 14 us for
// 35 MB; M 64, N 16384, K 8192: 58 us for 67 MB and 34 GFLOP with both steps).  The tile of 64 rows
// and 32 tokens is bound by no unit (matrix cores busy 21 %, vector unit 35 %, LDS 18 %): its 104 KB of
// LDS leave a CU one workgroup, whose loads and matrix steps take turns around a chunk's barriers.
// SPLIT: x is fp32 (16-byte aligned, VEC) and multiplied in its two parts, whose rows of LDS and
// matrix steps are twice as many: 9.2 us instead of 6.4 (M 16, N 2048, K 4096), 13.8 instead of 9.6
// (M 64).  An accumulator for each part, or shorter chunks, were no faster.
template <int NN, int MT, int XR, int KC, int WORDS, bool VEC, bool SPLIT>
__global__ __launch_bounds__(KS * 64, NN * MT > 2 || SPLIT || (KC > 1024 && XR > 4) ? 2 : 4) void w4_kernel(W4Args a) {
  constexpr int PARTS = SPLIT ? 2 : 1;
  constexpr int NTH = KS * 64;
  constexpr int KB = WORDS * 32, NB = KC / KB, U = NB / KS;         // per block; blocks of a chunk, of a wave
  constexpr int XROW = KC + 8, QROW = KC / 8 + 4;  // 16 bytes more: a quarter wave's rows start in different banks
  constexpr int XQ = XR * (KC / 8) / NTH, QQ = (16 * NN * (KC / 32) + NTH - 1) / NTH;  // a thread's 16 bytes of x and q
  constexpr int NR = 16 * NN, SQ = (NB * NR + NTH - 1) / NTH;  // rows of W; a thread's scales
  __shared__ union {
    struct {
      uint16_t x[PARTS][XR][XROW];
      uint32_t q[NR][QROW];
      float scale[NB][NR];
      uint32_t minus[NB][NR];  // -(16 + zero), twice
    } c;
    f32x4 red[KS][NN * MT][64];
  } lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, kq = lane >> 4;
  const int n0 = blockIdx.x * NR, m0 = blockIdx.y * MT * 16;
  const int rows = min(a.M - m0, MT * 16), groups = a.K / a.group, blocks = a.K / KB;
  const unsigned per = a.group / KB;  // blocks per group; 1 for the groups of 32 and 64
  // the thread's share of a chunk: q and x by 16 bytes along their rows, blocks' scales and zero points
  u32x4 qv[QQ], xv[XQ][PARTS];
  uint16_t sv[SQ];
  uint8_t zv[SQ];
#pragma unroll
  for (int i = 0; i < QQ; ++i) qv[i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < XQ; ++i)
#pragma unroll
    for (int k = 0; k < PARTS; ++k) xv[i][k] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < SQ; ++i) sv[i] = 0, zv[i] = 8;
  const int sr = min(n0 + tid % NR, a.N - 1);
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < QQ; ++i) {
      const int e = i * NTH + tid, r = e / (KC / 32), c = e % (KC / 32) * 32;
      if (r < NR && k0 + c < a.K)
        qv[i] = *(const u32x4 *)(a.q + (long long)min(n0 + r, a.N - 1) * (a.K / 8) + (k0 + c) / 8);
    }
#pragma unroll
    for (int i = 0; i < SQ; ++i) {
      const unsigned sb = (i * NTH + tid) / NR, kb = k0 / KB + sb, g = WORDS < 4 || per == 1 ? kb : kb / per;
      if (sb < NB && (int)kb < blocks) {
        sv[i] = a.scale[(long long)sr * groups + g];
        if (a.zero) zv[i] = a.zero[(long long)sr * groups + g];
      }
    }
#pragma unroll
    for (int i = 0; i < XQ; ++i) {
      const int e = i * NTH + tid, r = e / (KC / 8), c = e % (KC / 8) * 8;
      if (r < rows && k0 + c < a.K) {
        const long long at = (long long)(m0 + r) * a.x_ld + k0 + c;
        if constexpr (SPLIT)
#pragma unroll
          for (int k = 0; k < PARTS; ++k) xv[i][k] = ((const u32x4 *)((const float *)a.x + at))[k];
        else
          xv[i][0] = load_x<VEC>((const uint16_t *)a.x + at);
      }
    }
  };
  f32x4 tot[NN][MT];
#pragma unroll
  for (int t = 0; t < NN; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) tot[t][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  fetch(0);
  for (int k0 = 0; k0 < a.K; k0 += KC) {
    if (k0) __syncthreads();  // the chunk before has been read
#pragma unroll
    for (int i = 0; i < QQ; ++i) {
      const int e = i * NTH + tid, r = e / (KC / 32);
      if (r < NR) *(u32x4 *)&lds.c.q[r][e % (KC / 32) * 4] = qv[i];
    }
#pragma unroll
    for (int i = 0; i < SQ; ++i) {
      const int sb = (i * NTH + tid) / NR;
      if (sb < NB) {
        lds.c.scale[sb][tid % NR] = bf2f(sv[i]);
        lds.c.minus[sb][tid % NR] = (0xC180u | (zv[i] & 15u) << 3) * 0x10001u;
      }
    }
#pragma unroll
    for (int i = 0; i < XQ; ++i) {
      const int e = i * NTH + tid, r = e / (KC / 8);
      if (r < rows) {
        u32x4 part[PARTS];
        if constexpr (SPLIT)
          split_x(xv[i][0], xv[i][1], part[0], part[1]);
        else
          part[0] = permuted(xv[i][0]);
#pragma unroll
        for (int k = 0; k < PARTS; ++k) *(u32x4 *)&lds.c.x[k][r][e % (KC / 8) * 8] = part[k];
      }
    }
    __syncthreads();
    if (k0 + KC < a.K) fetch(k0 + KC);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = wave * U + u;
      if (k0 / KB + kb >= blocks) break;
      bf16x8 minus[NN];
      float sc[NN];
      uint32_t wq[NN][WORDS];
#pragma unroll
      for (int t = 0; t < NN; ++t) {
        const uint32_t off = lds.c.minus[kb][t * 16 + col];
        minus[t] = __builtin_bit_cast(bf16x8, u32x4{off, off, off, off});
        sc[t] = lds.c.scale[kb][t * 16 + col];
        const uint32_t *w = &lds.c.q[t * 16 + col][kb * (KB / 8) + kq * WORDS];
        if constexpr (WORDS == 4)
          *(u32x4 *)wq[t] = *(const u32x4 *)w;
        else if constexpr (WORDS == 2)
          *(uint2 *)wq[t] = *(const uint2 *)w;
        else
          wq[t][0] = w[0];
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        // rows without a token hold anything (or another's): they reach only their own rows of the result
        f32x4 acc[NN] = {};
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
#pragma unroll
          for (int k = 0; k < PARTS; ++k) {
            const bf16x8 xf = *(const bf16x8 *)&lds.c.x[k][(m * 16 + col) % XR][kb * KB + kq * WORDS * 8 + i * 8];
#pragma unroll
            for (int t = 0; t < NN; ++t) {
              acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, unpack(wq[t][i]), acc[t], 0, 0, 0);
              acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, minus[t], acc[t], 0, 0, 0);
            }
          }
#pragma unroll
        for (int t = 0; t < NN; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) tot[t][m][i] += sc[t] * acc[t][i];
      }
    }
  }
  if (a.pos && blockIdx.x == 0 && wave == 0)
    for (int b = m0 + lane; b < m0 + rows; b += 64) a.pos[b] += 1;
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NN; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) lds.red[wave][t * MT + m][lane] = tot[t][m];
  __syncthreads();
  // lane (n = lane & 15, rows (lane >> 4) * 4 ..) of a tile
  for (int e = wave; e < NN * MT; e += KS) {
    f32x4 y = lds.red[0][e][lane];
#pragma unroll
    for (int k = 1; k < KS; ++k) y += lds.red[k][e][lane];
    const int n = n0 + e / MT * 16 + col;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = m0 + e % MT * 16 + kq * 4 + i;
      if (row < a.M && n < a.N) store_elem(a.out, (long long)row * a.N + n, y[i], a.out_bf16);
    }
  }
}

enum XKind { BF16_ROWS, BF16_WIDE, F32_PARTS };  // x by elements or by 16 bytes, or fp32 in two parts

template <int NN, int MT, int XR, int KC, int WORDS>
hipError_t launch_w(const W4Args &a, XKind x, hipStream_t st) {
  const dim3 grid((unsigned)rec_cdiv(a.N, 16 * NN), (unsigned)rec_cdiv(a.M, MT * 16));
  if (x == F32_PARTS) {
    if constexpr (NN * MT <= 2)
      hipLaunchKernelGGL((w4_kernel<NN, MT, XR, KC, WORDS, true, true>), grid, dim3(KS * 64), 0, st, a);
    else
      return hipErrorInvalidValue;  // both parts of the larger tile do not fit LDS
  } else if (x == BF16_WIDE) {
    hipLaunchKernelGGL((w4_kernel<NN, MT, XR, KC, WORDS, true, false>), grid, dim3(KS * 64), 0, st, a);
  } else {
    hipLaunchKernelGGL((w4_kernel<NN, MT, XR, KC, WORDS, false, false>), grid, dim3(KS * 64), 0, st, a);
  }
  return hipGetLastError();
}
template <int NN, int MT, int KC, int XR = 16 * MT>
hipError_t launch_mt(const W4Args &a, XKind x, hipStream_t st) {
  if (a.group % 128 == 0) return launch_w<NN, MT, XR, KC, 4>(a, x, st);
  return a.group == 64 ? launch_w<NN, MT, XR, KC, 2>(a, x, st) : launch_w<NN, MT, XR, KC, 1>(a, x, st);
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
  if (N > 1 << 26 || K > 1 << 26) return "N or K above 2^26";
  return nullptr;
}

hipError_t launch_w4(const void *x, const void *q, const void *scale, const void *zero, void *out, int M, int N, int K,
                     int group, long long x_ld, bool out_bf16, hipStream_t st, int *pos, bool x_f32) {
  W4Args a;
  a.pos = pos;
  a.x = x;
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
  const XKind kind = x_f32 ? F32_PARTS : x_ld % 8 == 0 && rec_aligned(x, 16) ? BF16_WIDE : BF16_ROWS;
  // A larger tile reads x and W fewer times from L2, a smaller one gives more workgroups.
  // Measured, us, for tiles of 16 x 16, 32 x 16, 64 x 32 (rows of W x tokens): M 16, N 2048,
  // K 4096: 6.9, 7.9, 14.6; M 64, N 2048, K 4096: 10.2, 8.2, 14.7; M 16, N 12288, K 2048: 9.4,
  // 7.3, 8.5; M 32: 15.5, 10.9, 9.3; M 64, N 16384, K 8192: 126, 75, 58.  So the larger one
  // as soon as it still gives about a workgroup per CU.
  if (M <= 4) return launch_mt<1, 1, 2048, 4>(a, kind, st);
  if (!x_f32 && M > 16 && rec_cdiv(N, 64) * rec_cdiv(M, 32) >= 192) return launch_mt<4, 2, 1024>(a, kind, st);
  if (rec_cdiv(N, 32) * rec_cdiv(M, 16) >= 192) return launch_mt<2, 1, 1024>(a, kind, st);
  // Chunks twice as long, whose LDS leaves a CU one workgroup, where there are no more than that:
  // M 16, N 2048, K 4096, groups of 64: 7.3 -> 6.4 us, K 2048: 4.8 -> 4.3 us.  For 32 rows of W they
  // took longer from K 4096 on (M 64, N 2048: 8.3 -> 8.9 us).
  if (rec_cdiv(N, 16) * rec_cdiv(M, 16) <= 256 && K > 1024) return launch_mt<1, 1, 2048>(a, kind, st);
  return launch_mt<1, 1, 1024>(a, kind, st);
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
