// The tiled product of language.h's linear and its gradients, on the matrix cores.
//
// One kernel serves the three products of a layer.  It sums out[m][n] = sum_k P(m, k) Q(n, k):
//   forward  P = x,  Q = w         both with k along their rows
//   dx       P = dz, Q = w         w's rows run along n: its tiles are read transposed from LDS
//   dw       P = dz, Q = x         both with k across their rows
// Tiles of 64 k reach LDS by DMA, two to four in turn, so that one is filled while another is multiplied, and the
// operands of the next matrix step are read from LDS while the present one's are multiplied.
// Operands whose rows are not 16-byte aligned take the same way through registers (M 64, N 4096, K 2048 11.7 us,
// K 2047 20.0; M 300, N 1001, K 999 12.7 against 7.9 for 1000 and 1000).
// Where there are too few tiles for the chip, k is cut, the parts' sums go to the workspace in
// fp32, and a second launch joins them in order and finishes.
//
// M 16384, features 2048 -> 4096 (275 GFLOP): 215 us without and 237 us with gelu, whose 18 operations an
// element follow the last matrix step with nothing to hide behind; dx 211 us, dw 260 us and 17 us to join two
// parts.  The largest library product reaches 1385 TFLOP/s here, so 199 us would be the floor.  What is left is the
// wait at a tile's middle: with one workgroup a CU, whose 128 KB of LDS hold two tiles, all waves stand there.
#pragma once

#include "linear.hpp"

namespace ret {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((address_space(3))) void lds_void;

// A tile of R rows and 64 k of an operand in LDS, in two halves of 32 k, one matrix step each.
//   KROWS (k along the rows in memory): groups of 8 rows, of each 8 rows of 32 k and then 8 rows of
//     the next 32: a wave load takes 8 whole lines of 128 bytes (tiles of 32 k fetched every line
//     twice and were bound by it: 128 x 128 tiles took 0.29 us a step of 32 k).  Chunk c (16 bytes) of
//     a half's row r is at c ^ (r / 2 & 3): the 8 rows that a read takes together meet no bank twice.
//   else: [64][R], chunk c of row k at c ^ turn(k), for reads that transpose.  In rows of 256 columns the
//     rows k + 8 .. are turned further than k ..: 32 lanes take them together (dx 234 -> 215 us; 128 columns
//     were slower with it, 296 -> 321 us, and 64 have no chunks for it).
//
// DMA: 16-byte chunks straight to LDS.  WIDE: the same chunks at any address through registers, DEPTH tiles under
// way (M 300, N 1001, K 999 with a branch around each row's end and one tile: 21.8 us, without and with four: 12.7).
// SINGLE: element by element, for rows of fewer than 8.
enum Way { DMA, WIDE, SINGLE };
template <int R, bool KROWS, int NT, Way WAY, int DEPTH>
struct Operand {
  static constexpr int SIZE = R * BK, NJ = SIZE * 2 / 1024 / (NT / 64);  // elements; wave loads of a wave
  static_assert(NJ >= 1 && SIZE * 2 % (1024 * (NT / 64)) == 0, "whole wave loads");
  const uint16_t *base;  // of the tile's rows (KROWS) or columns
  long long ld;
  int width;  // rows of the operand from the tile on, R at most
  u32x4 reg[DEPTH][NJ];

  __device__ __forceinline__ void start(const uint16_t *p, long long ld_, long long rows, long long r0) {
    base = KROWS ? p + r0 * ld_ : p + r0;
    ld = ld_;
    width = rows - r0 < R ? (int)(rows - r0) : R;
  }
  // The wave, as a scalar.
  static __device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
  static __device__ __forceinline__ int turn(int k) { return 2 * (R >= 256 ? (k & 3) | (k >> 1 & 4) : k & 3); }
  // What chunk j of this thread holds: a row and one of its 16-byte chunks (KROWS: of k, else of columns).
  static __device__ __forceinline__ void place(int j, int &row, int &c) {
    const int piece = wave() * NJ + j, lane = threadIdx.x & 63;
    if constexpr (KROWS) {
      const int r = lane >> 2 & 7;
      row = piece * 8 + r;
      c = (lane >> 5) * 4 + ((lane & 3) ^ (r >> 1));
    } else {
      const int off = piece * 1024 + lane * 16;
      row = off / (R * 2);
      c = off % (R * 2) / 16 ^ turn(row);
    }
  }
  // The tile at k0 on its way to `lds` (DMA) or to reg[d]; k from `kend` on is zero.
  __device__ __forceinline__ void fetch(uint16_t *lds, int d, long long k0, long long kend) {
    const int left = kend - k0 < BK ? (int)(kend - k0) : BK;
    if constexpr (WAY == DMA) {
      // rows are whole 16-byte chunks; what lies behind the range reads as zero
      const uint16_t *b = KROWS ? base + k0 : base + k0 * ld;
      const long long last = left <= 0 ? 0 : KROWS ? (long long)(width - 1) * ld + left : (long long)(left - 1) * ld + width;
      const __amdgpu_buffer_rsrc_t rs =
          __builtin_amdgcn_make_buffer_rsrc((void *)b, (short)0, (int)(last * 2), 0x00020000);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        int row, c;
        place(j, row, c);
        int off = row * (int)ld * 2 + c * 16;
        if (KROWS && c * 8 >= left) off = (int)0x80000000u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(lds + (wave() * NJ + j) * 512), 16, off, 0, 0, 0);
      }
    } else if constexpr (WAY == WIDE) {
      // Every lane loads, with no branch, which would hold up the loads under way: rows behind the last are the
      // last once more, and a row's last chunk ends with the row.
      const char *b = (const char *)(KROWS ? base + k0 - 8 : base + k0 * ld - 8);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        int row, c;
        place(j, row, c);
        row = min(row, (KROWS ? width : left) - 1);
        // a row's offset in 64 bits: rows are up to 2^31 elements apart
        const uint64_t off = (uint64_t)(uint32_t)row * (uint32_t)ld + (uint32_t)(min(c * 8, (KROWS ? left : width) - 8) + 8);
        const Words4 w = *(const Words4 *)(b + off * 2);
        reg[d][j] = u32x4{w.w[0], w.w[1], w.w[2], w.w[3]};
      }
    } else {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        int row, c;
        place(j, row, c);
        const uint16_t *src = KROWS ? base + row * ld + k0 + c * 8 : base + (k0 + row) * ld + c * 8;
        const int n = row < (KROWS ? width : left) ? (KROWS ? left : width) - c * 8 : 0;
        reg[d][j] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < n) reg[d][j][i / 2] |= (uint32_t)src[i] << (i % 2 * 16);
      }
    }
  }
  // The tile of `left` k in reg[d] to LDS.
  __device__ __forceinline__ void commit(uint16_t *lds, int d, int left) {
    if constexpr (WAY != DMA) {
      const bool cut = WAY == WIDE && (left < BK || (!KROWS && width < R));
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        u32x4 v = reg[d][j];
        if (cut) {
          int row, c;
          place(j, row, c);
          const int s = 16 * (c * 8 - min(c * 8, (KROWS ? left : width) - 8));  // bits that the chunk was read early
          uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
          lo = s == 0 ? lo : s < 64 ? lo >> s | hi << (64 - s) : s < 128 ? hi >> (s - 64) : 0;
          hi = s < 64 ? hi >> s : 0;
          if (!KROWS && row >= left) lo = hi = 0;
          v = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
        }
        *(u32x4 *)(lds + (wave() * NJ + j) * 512 + (threadIdx.x & 63) * 8) = v;
      }
    }
  }
  // Matrix operand of half h: lane (l16, g) holds k = 32 h + 8 g .. + 7 of row r0 + l16.
  static __device__ __forceinline__ bf16x8 read(const uint16_t *lds, int r0, int h, int l16, int g) {
    if constexpr (KROWS) {
      return *(const bf16x8 *)(lds + (r0 / 8 + (l16 >> 3)) * 512 + h * 256 + (l16 & 7) * 32 + (g ^ (l16 >> 1 & 3)) * 8);
    } else {
      // within 16 lanes, lane r receives element r % 4 of the pieces that lanes 4 j + r / 4 address
      const int row = h * 32 + 8 * g + (l16 >> 2), c = (r0 >> 3) + ((l16 & 3) >> 1);
      const uint16_t *p = lds + row * R + ((c ^ turn(row)) << 3) + 4 * (l16 & 1);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p + 4 * R));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// Waits until at most N of this wave's loads are under way, and for its LDS operations.
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0070);
}
// A barrier that waits for nothing by itself; memory operations stay on their side of it.
__device__ __forceinline__ void meet() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// BM x BN of out by WM x WN waves, with a ring of NB tiles in LDS.  A wave multiplies the operands of a half
// tile while it reads those of the next half.  The barrier in the middle of a tile tells that all
// have read it, so that tile i + NB takes its place, and that tile i + 1 has come.
// FINE: finish8's.  A kernel of its own: with both kinds of gelu in one, the large product without any took 241 us
// instead of 226, going round their code.
template <int BM, int BN, int WM, int WN, int NB, bool PK, bool QK, Way WAY, bool FINE>
__global__ __launch_bounds__(WM *WN * 64, 2) void mm_kernel(MmArgs a) {
  constexpr int NT = WM * WN * 64, FM = BM / WM / 16, FN = BN / WN / 16;
  // WIDE's tiles under way: as many as there are registers for beside the sums
  constexpr int DEPTH = WAY != WIDE ? 1 : BM * BN <= 4096 ? 4 : BM * BN <= 16384 ? 2 : 1;
  using OpP = Operand<BM, PK, NT, WAY, DEPTH>;
  using OpQ = Operand<BN, QK, NT, WAY, DEPTH>;
  constexpr int SIZE = OpP::SIZE + OpQ::SIZE, LOADS = OpP::NJ + OpQ::NJ;
  __shared__ __attribute__((aligned(1024))) uint16_t lds[NB * SIZE];
  const int lane = threadIdx.x & 63, wave = OpP::wave(), l16 = lane & 15, g = lane >> 4;
  const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
  // Workgroups go round the eight XCDs, each with an L2 of its own: an XCD takes neighbouring tiles,
  // in groups of rows of tiles that share their columns of Q.
  const unsigned tn = (a.N + BN - 1) / BN, tm = (unsigned)((a.M + BM - 1) / BM), tiles = tm * tn;
  unsigned t = blockIdx.x;
  {
    const unsigned per = tiles / 8, rest = tiles % 8, x = t % 8;
    t = t / 8 + x * per + min(x, rest);
  }
  constexpr unsigned GM = 4;
  const unsigned gr = t / (GM * tn), in = t - gr * GM * tn, gm = min(GM, tm - gr * GM);
  const long long m0 = (long long)(gr * GM + in % gm) * BM;
  const int n0 = (int)(in / gm) * BN;
  const long long kb = (long long)blockIdx.y * a.kpart, ke = kb + a.kpart < a.K ? kb + a.kpart : a.K;
  const int tiles_k = (int)((ke - kb + BK - 1) / BK);

  OpP P;
  OpQ Q;
  P.start(a.p, a.ldp, a.M, m0);
  Q.start(a.q, a.ldq, a.N, n0);
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  bf16x8 fp[2][FM], fq[2][FN];
  auto fetch = [&](int i, int slot) {  // a place in LDS, or in registers
    P.fetch(lds + slot * SIZE, slot, kb + (long long)i * BK, ke);
    Q.fetch(lds + slot * SIZE + OpP::SIZE, slot, kb + (long long)i * BK, ke);
  };
  auto read = [&](int slot, int h) {
#pragma unroll
    for (int j = 0; j < FN; ++j) fq[h][j] = OpQ::read(lds + slot * SIZE + OpP::SIZE, wn + j * 16, h, l16, g);
#pragma unroll
    for (int i = 0; i < FM; ++i) fp[h][i] = OpP::read(lds + slot * SIZE, wm + i * 16, h, l16, g);
  };
  auto multiply = [&](int h) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[h][j], fp[h][i], acc[i][j], 0, 0, 0);
  };
  // the reads, and then the loads, go out between the matrix instructions: loads issued in a row keep a wave from
  // its matrix instructions (fwd 221 -> 215 us)
  auto interleave = [](auto loads) {
    constexpr int READS = (PK ? FM : 2 * FM) + (QK ? FN : 2 * FN), REST = FM * FN - READS;
#pragma unroll
    for (int r = 0; r < READS; ++r) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // an LDS read
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // and a matrix instruction
    }
    if constexpr (decltype(loads)::value)
#pragma unroll
      for (int r = 0; r < LOADS; ++r) {
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // a load from memory
        __builtin_amdgcn_sched_group_barrier(0x008, REST / LOADS > 1 ? REST / LOADS : 1, 0);
      }
  };
  if constexpr (WAY == DMA) {
    // tiles behind the last are fetched as zeros, so that all steps are alike
#pragma unroll
    for (int i = 0; i < NB; ++i) fetch(i, i);
    wait_loads<(NB - 1) * LOADS>();
    meet();
    read(0, 0);
    int slot = 0;  // of tile i
    for (int i = 0; i < tiles_k; ++i) {
      read(slot, 1);
      multiply(0);
      interleave(std::false_type{});
      wait_loads<(NB - 2) * LOADS>();
      meet();
      const int free = slot;
      slot = slot + 1 == NB ? 0 : slot + 1;
      read(slot, 0);
      fetch(i + NB, free);
      multiply(1);
      interleave(std::true_type{});
    }
  } else if (tiles_k > 0) {
    // steps behind the last tile have it once more, as zeros: all are alike, with no branch around a load
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) fetch(min(d, tiles_k - 1), d);
    for (int i0 = 0; i0 < tiles_k; i0 += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        const int i = i0 + d, slot = DEPTH > 1 ? d & 1 : i & 1;
        const long long rest = ke - kb - (long long)i * BK;
        const int left = rest < BK ? (rest > 0 ? (int)rest : 0) : BK;
        P.commit(lds + slot * SIZE, d, left);
        Q.commit(lds + slot * SIZE + OpP::SIZE, d, left);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // for LDS only: the next tiles stay under way
        meet();                              // this tile is there, and all have left the other place
        fetch(min(i + DEPTH, tiles_k - 1), d);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          read(slot, h);
          multiply(h);
        }
      }
    }
  }
  // Lane (l16, g) holds row l16 of P's and rows 4 g .. + 3 of Q's of each 16 x 16; through LDS, 16 rows of P's
  // at a time, they become runs of eight neighbours, which are finished and stored together.
  wait_loads<0>();
  meet();
  // The bias is read once and the residual 16 rows ahead.
  constexpr int TN = BN / WN, PITCH = TN + 4, ROWS = 512 / TN, PASSES = 16 / ROWS;  // ROWS rows in a pass of 64 lanes
  static_assert(NT / 64 * 16 * PITCH * 4 <= (int)sizeof(lds) && ROWS <= 16, "the waves' patches");
  float *patch = (float *)lds + wave * 16 * PITCH;
  const int c = lane % (TN / 8) * 8, r0 = lane / (TN / 8), n = n0 + wn + c;
  float bias[8] = {};
  if (a.f.bias && !a.part) load8(a.f.bias + n, a.N - n, bias);
  Residual8 res[2][PASSES];
  auto row = [&](int i, int q) { return m0 + wm + i * 16 + q * ROWS + r0; };
  auto ahead = [&](int i) {
#pragma unroll
    for (int q = 0; q < PASSES; ++q)
      if (!a.part) res[i & 1][q].load(a.f, row(i, q) * a.N + n, row(i, q) < a.M ? a.N - n : 0);
  };
  ahead(0);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (i + 1 < FM) ahead(i + 1);
#pragma unroll
    for (int j = 0; j < FN; ++j) *(f32x4 *)(patch + l16 * PITCH + j * 16 + 4 * g) = acc[i][j];
#pragma unroll
    for (int q = 0; q < PASSES; ++q) {
      const int r = q * ROWS + r0;
      const f32x4 lo = *(const f32x4 *)(patch + r * PITCH + c), hi = *(const f32x4 *)(patch + r * PITCH + c + 4);
      float z[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      const long long m = row(i, q);
      if (m < a.M && n < a.N) {
        if (a.part)
          store8(a.part + ((long long)blockIdx.y * a.M + m) * a.N + n, a.N - n, z);
        else
          finish8<FINE>(a.f, m * a.N + n, a.N - n, bias, res[i & 1][q], z);
      }
    }
  }
}

// The parts' sums, in order.
__global__ __launch_bounds__(256) void mm_join_kernel(const float *part, int parts, long long M, int N, Finish f) {
  const unsigned runs = (N + 7) / 8;
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  if (e >= M * runs) return;
  const long long m = e / runs;
  const int n = (int)(e - m * runs) * 8;
  Residual8 res;
  res.load(f, m * N + n, N - n);
  float z[8] = {};
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    float v[8];
    load8(part + (p * M + m) * N + n, N - n, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += v[i];
  }
  float bias[8] = {};
  if (f.bias) load8(f.bias + n, N - n, bias);
  finish8(f, m * N + n, N - n, bias, res, z);
}

template <int BM, int BN, int WM, int WN, int NB, bool PK, bool QK, Way WAY, bool FINE>
hipError_t launch_tile(const MmArgs &a, int parts, hipStream_t st) {
  const dim3 grid((unsigned)(rec_cdiv(a.M, BM) * rec_cdiv(a.N, BN)), (unsigned)parts);
  hipLaunchKernelGGL((mm_kernel<BM, BN, WM, WN, NB, PK, QK, WAY, FINE>), grid, dim3(WM * WN * 64), 0, st, a);
  return hipGetLastError();
}

template <bool PK, bool QK, Way WAY, bool FINE>
hipError_t launch(const MmArgs &a, const MmPlan &p, hipStream_t st) {
  // Tiles in LDS.  The smallest tiles are for calls of one workgroup a CU, whose w comes from memory: four of them
  // (M 32, N 8192, K 2048: 18.2 -> 11.8 us).  128 x 128 with four: 27.4 -> 26.6 us (M 777, N 4096) but 33 -> 50 (N 8192).
  constexpr int NB = WAY == DMA ? 3 : 2, NB64 = WAY == DMA ? 4 : 2;
  if (p.rows == 256) return launch_tile<256, 256, 2, 4, 2, PK, QK, WAY, FINE>(a, p.parts, st);
  if (p.rows == 128) return launch_tile<128, 128, 2, 2, 2, PK, QK, WAY, FINE>(a, p.parts, st);
  if (p.cols == 128) return launch_tile<64, 128, 2, 2, NB, PK, QK, WAY, FINE>(a, p.parts, st);
  return launch_tile<64, 64, 2, 2, NB64, PK, QK, WAY, FINE>(a, p.parts, st);
}

// Rows of `width` elements whose 16-byte chunks are whole and aligned, within a buffer's reach.
bool chunked(const void *p, long long ld, long long width) {
  return rec_aligned(p, 16) && ld % 8 == 0 && width % 8 == 0 && ld <= (1 << 21);
}

template <bool PK, bool QK, bool FINE = false>
hipError_t product(MmArgs a, void *ws, hipStream_t st) {
  const MmPlan p = mm_plan(a.M, a.N, a.K);
  a.kpart = p.kpart;
  a.part = p.parts > 1 ? (float *)ws : nullptr;
  const long long wp = PK ? a.K : a.M, wq = QK ? a.K : a.N;
  const Way way = chunked(a.p, a.ldp, wp) && chunked(a.q, a.ldq, wq) ? DMA : wp >= 8 && wq >= 8 ? WIDE : SINGLE;
  // SINGLE in one size: 128 x 128 of the largest output still are a grid
  const hipError_t e = way == DMA    ? launch<PK, QK, DMA, FINE>(a, p, st)
                       : way == WIDE ? launch<PK, QK, WIDE, FINE>(a, p, st)
                                     : launch_tile<128, 128, 2, 2, 2, PK, QK, SINGLE, FINE>(a, p.parts, st);
  if (e != hipSuccess || p.parts == 1) return e;
  const long long runs = a.M * ((a.N + 7) / 8);
  hipLaunchKernelGGL(mm_join_kernel, dim3((unsigned)rec_cdiv(runs, 256)), dim3(256), 0, st, a.part, p.parts, a.M, a.N,
                     a.f);
  return hipGetLastError();
}

}  // namespace
}  // namespace ret
