// The tiled product of language.h's linear and its gradients, on the matrix cores.
//
// One kernel serves the three products of a layer.  It sums out[m][n] = sum_k P(m, k) Q(n, k):
//   forward  P = x,  Q = w         both with k along their rows
//   dx       P = dz, Q = w         w's rows run along n: its tiles are read transposed from LDS
//   dw       P = dz, Q = x         both with k across their rows
// Tiles of 64 k reach LDS by DMA, two buffers in turn, so that one is filled while the other is
// multiplied; the 16-byte chunks of a row are permuted, so that the operand reads meet no bank twice.
// Operands whose rows are not 16-byte aligned take the same way through registers.
// Where there are too few tiles for the chip, k is cut, the parts' sums go to the workspace in
// fp32, and a second launch joins them in order and finishes.
#pragma once

#include "linear.hpp"

namespace ret {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((address_space(3))) void lds_void;

// A tile of R rows and BK k of an operand in LDS.
//   KROWS: [R][BK], chunk c (16 bytes) of row r at c ^ (r & 7): the eight rows that a read
//     takes together then lie in different banks
//   else: [BK][R], chunk c of row k at c ^ 2 (k & 3), for reads that transpose
template <int R, bool KROWS, int NT, bool DMA>
struct Operand {
  static constexpr int BYTES = R * BK * 2, NJ = BYTES / 1024 / (NT / 64);
  static_assert(NJ >= 1 && BYTES % (1024 * (NT / 64)) == 0, "whole wave loads");
  const uint16_t *base;  // of the tile's rows (KROWS) or columns
  long long ld, K;
  int width;  // rows of the operand from the tile on, R at most
  u32x4 reg[DMA ? 1 : NJ];

  __device__ __forceinline__ void start(const uint16_t *p, long long ld_, long long rows, long long r0, long long K_) {
    base = KROWS ? p + r0 * ld_ : p + r0;
    ld = ld_;
    K = K_;
    width = rows - r0 < R ? (int)(rows - r0) : R;
  }
  // Place of chunk j of this thread: row of the LDS tile and (unpermuted) chunk in it.
  static __device__ __forceinline__ void place(int j, int &row, int &c) {
    const int off = ((threadIdx.x >> 6) * NJ + j) * 1024 + (threadIdx.x & 63) * 16;
    constexpr int RB = KROWS ? BK * 2 : R * 2;
    row = off / RB;
    c = (off % RB) / 16 ^ (KROWS ? row & 7 : 2 * (row & 3));
  }
  // The tile at k0 on its way to `lds` (DMA) or to registers; k from `kend` on is zero.
  __device__ __forceinline__ void fetch(uint16_t *lds, long long k0, long long kend) {
    if constexpr (DMA) {
      // rows are whole 16-byte chunks; what lies behind the range reads as zero
      const int left = kend - k0 < BK ? (int)(kend - k0) : BK;
      const uint16_t *b = KROWS ? base + k0 : base + k0 * ld;
      const long long last = KROWS ? (long long)(width - 1) * ld + left : (long long)(left - 1) * ld + width;
      const __amdgpu_buffer_rsrc_t rs =
          __builtin_amdgcn_make_buffer_rsrc((void *)b, (short)0, (int)(last * 2), 0x00020000);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        int row, c;
        place(j, row, c);
        int off = row * (int)ld * 2 + c * 16;
        if (KROWS && c * 8 >= left) off = (int)0x80000000u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(lds + ((threadIdx.x >> 6) * NJ + j) * 512), 16, off, 0,
                                                 0, 0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        int row, c;
        place(j, row, c);
        const long long k = k0 + (KROWS ? c * 8 : row);
        const int r = KROWS ? row : c * 8;
        const uint16_t *src = KROWS ? base + r * ld + k : base + k * ld + r;
        int n = 0;  // elements of the chunk that exist
        if (KROWS ? r < width : k < kend) n = (int)(KROWS ? (kend - k < 8 ? kend - k : 8) : (width - r < 8 ? width - r : 8));
        u32x4 v = {0u, 0u, 0u, 0u};
        if (n >= 8) {
          const Words4 w = *(const Words4 *)src;
          v = u32x4{w.w[0], w.w[1], w.w[2], w.w[3]};
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < n) v[i / 2] |= (uint32_t)src[i] << (i % 2 * 16);
        }
        reg[j] = v;
      }
    }
  }
  __device__ __forceinline__ void commit(uint16_t *lds) {
    if constexpr (!DMA)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        *(u32x4 *)(lds + ((threadIdx.x >> 6) * NJ + j) * 512 + (threadIdx.x & 63) * 8) = reg[j];
  }
  // Matrix operand: lane (l16, g) holds k = 32 ks + 8 g .. + 7 of row r0 + l16.
  static __device__ __forceinline__ bf16x8 read(const uint16_t *lds, int r0, int ks, int l16, int g) {
    if constexpr (KROWS) {
      return *(const bf16x8 *)(lds + (r0 + l16) * BK + ((ks * 4 + g) ^ (l16 & 7)) * 8);
    } else {
      // within 16 lanes, lane r receives element r % 4 of the pieces that lanes 4 j + r / 4 address
      const int row = ks * 32 + 8 * g + (l16 >> 2), c = (r0 >> 3) + ((l16 & 3) >> 1);
      const uint16_t *p = lds + row * R + ((c ^ 2 * (row & 3)) << 3) + 4 * (l16 & 1);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p + 4 * R));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// BM x BN of out by WM x WN waves.
template <int BM, int BN, int WM, int WN, bool PK, bool QK, bool DMA>
__global__ __launch_bounds__(WM *WN * 64, 2) void mm_kernel(MmArgs a) {
  constexpr int NT = WM * WN * 64, FM = BM / WM / 16, FN = BN / WN / 16;
  __shared__ __attribute__((aligned(1024))) uint16_t lds[2][(BM + BN) * BK];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
  const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
  // Workgroups go round the eight XCDs, each with an L2 of its own: an XCD takes neighbouring tiles,
  // in groups of rows of tiles that share their columns of Q.
  const unsigned tn = (a.N + BN - 1) / BN, tm = (unsigned)((a.M + BM - 1) / BM), tiles = tm * tn;
  unsigned t = blockIdx.x;
  {
    const unsigned per = tiles / 8, rest = tiles % 8, x = t % 8;
    t = t / 8 + x * per + min(x, rest);
  }
  constexpr unsigned GM = 8;
  const unsigned gr = t / (GM * tn), in = t - gr * GM * tn, gm = min(GM, tm - gr * GM);
  const long long m0 = (long long)(gr * GM + in % gm) * BM;
  const int n0 = (int)(in / gm) * BN;
  const long long kb = (long long)blockIdx.y * a.kpart, ke = kb + a.kpart < a.K ? kb + a.kpart : a.K;

  Operand<BM, PK, NT, DMA> P;
  Operand<BN, QK, NT, DMA> Q;
  P.start(a.p, a.ldp, a.M, m0, a.K);
  Q.start(a.q, a.ldq, a.N, n0, a.K);
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int buf = 0;
  if (kb < ke) {
    P.fetch(lds[0], kb, ke);
    Q.fetch(lds[0] + BM * BK, kb, ke);
  }
  for (long long k0 = kb; k0 < ke; k0 += BK) {
    uint16_t *cur = lds[buf], *next = lds[buf ^ 1];
    P.commit(cur);
    Q.commit(cur + BM * BK);
    __syncthreads();  // this tile is there, and all have left the other buffer
    if (k0 + BK < ke) {
      P.fetch(next, k0 + BK, ke);
      Q.fetch(next + BM * BK, k0 + BK, ke);
    }
#pragma unroll
    for (int ks = 0; ks < BK / 32; ++ks) {
      bf16x8 fp[FM], fq[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) fq[j] = Q.read(cur + BM * BK, wn + j * 16, ks, l16, g);
#pragma unroll
      for (int i = 0; i < FM; ++i) fp[i] = P.read(cur, wm + i * 16, ks, l16, g);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[j], fp[i], acc[i][j], 0, 0, 0);
    }
    buf ^= 1;
  }
  // lane (l16, g): row l16 of P's, rows 4 g .. + 3 of Q's
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const long long m = m0 + wm + i * 16 + l16;
    if (m >= a.M) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int n = n0 + wn + j * 16 + 4 * g;
      if (n >= a.N) continue;
      float z[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      if (a.part) {
        const long long nr = (a.N + 3) / 4 * 4;
        *(f32x4 *)(a.part + ((long long)blockIdx.y * a.M + m) * nr + n) = acc[i][j];
      } else {
        finish4(a.f, m, n, a.N, z);
      }
    }
  }
}

// The parts' sums, in order.
__global__ __launch_bounds__(256) void mm_join_kernel(const float *part, int parts, long long M, int N, Finish f) {
  const unsigned nq = (N + 3) / 4;
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  if (e >= M * nq) return;
  const long long m = e / nq;
  const int n = (int)(e - m * nq) * 4;
  float z[4] = {};
  for (int p = 0; p < parts; ++p) {
    const f32x4 v = *(const f32x4 *)(part + (p * M + m) * nq * 4 + n);
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] += v[i];
  }
  finish4(f, m, n, N, z);
}

template <int T, int WM, int WN, bool PK, bool QK>
hipError_t launch_tile(const MmArgs &a, int parts, bool dma, hipStream_t st) {
  const dim3 grid((unsigned)(rec_cdiv(a.M, T) * rec_cdiv(a.N, T)), (unsigned)parts);
  if (dma)
    hipLaunchKernelGGL((mm_kernel<T, T, WM, WN, PK, QK, true>), grid, dim3(WM * WN * 64), 0, st, a);
  else
    hipLaunchKernelGGL((mm_kernel<T, T, WM, WN, PK, QK, false>), grid, dim3(WM * WN * 64), 0, st, a);
  return hipGetLastError();
}

// Rows of `width` elements whose 16-byte chunks are whole and aligned, within a buffer's reach.
bool chunked(const void *p, long long ld, long long width) {
  return rec_aligned(p, 16) && ld % 8 == 0 && width % 8 == 0 && ld <= (1 << 21);
}

template <bool PK, bool QK>
hipError_t product(MmArgs a, void *ws, hipStream_t st) {
  const MmPlan p = mm_plan(a.M, a.N, a.K);
  a.kpart = p.kpart;
  a.part = p.parts > 1 ? (float *)ws : nullptr;
  const bool dma = chunked(a.p, a.ldp, PK ? a.K : a.M) && chunked(a.q, a.ldq, QK ? a.K : a.N);
  hipError_t e = p.tile == 256   ? launch_tile<256, 2, 4, PK, QK>(a, p.parts, dma, st)
                 : p.tile == 128 ? launch_tile<128, 2, 2, PK, QK>(a, p.parts, dma, st)
                                 : launch_tile<64, 2, 2, PK, QK>(a, p.parts, dma, st);
  if (e != hipSuccess || p.parts == 1) return e;
  const long long quads = a.M * ((a.N + 3) / 4);
  hipLaunchKernelGGL(mm_join_kernel, dim3((unsigned)rec_cdiv(quads, 256)), dim3(256), 0, st, a.part, p.parts, a.M, a.N,
                     a.f);
  return hipGetLastError();
}

}  // namespace
}  // namespace ret
