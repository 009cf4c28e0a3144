// Selective state space scan (recurrent.h): h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t,
// y_t = C_t . h_t + D u_t, gated by silu(z_t); its gradients; its single-token form.
//
// Layout of the passes: a wave works alone on CW = 16 CJ neighbouring channels of one
// group (of B and C) of one sequence.  A lane holds CJ channels, those of lane & 15, and
// NS states, those of its row of 16 lanes (lane >> 4), N <= 4 NS: the recurrence never
// leaves a lane, a sum over a channel's states is NS terms and two steps across the rows.
// Tokens come in tiles of 16: a lane reads four channels of CJ tokens, computes the time
// step, dt u and the gated gradient once, in fp32, and leaves them in the wave's part of
// LDS, from where all four rows read them back.  The loads of the next tile are in flight
// meanwhile.
//
// What bounds it: the vector unit.  Per token, channel and state the exponential (two issue
// slots by the counters), its argument, the decay and the product with C, 5 slots; N = 16
// of them and some 30 to 50 slots of softplus, gate and conversions stand against 8 bytes
// of a bf16 token and channel, and the chip has 39e12 lanes' slots a second against 5e12
// bytes.  So dt u B is left to the matrix cores (quad_outer).
//
// Long sequences are cut into segments, so that few channels still fill the chip: the
// decay of a state over a segment is exp(A sum dt), so the states entering the
// segments follow from each segment's own final state and its sum of time steps
// (states pass, combination), and the output pass runs all segments at once.
#include <algorithm>

#include "recurrent.hpp"

using namespace ret;

namespace {

constexpr int TT = 16;  // tokens per staged tile
constexpr int NT = 256;

struct ScanArgs {
  const void *u, *delta, *Bm, *Cm, *z, *d_o;
  const float *A, *Dskip, *bias, *h0, *dhT;
  const int *lengths;
  void *out;
  float *hT;
  long long u_ld, delta_ld, z_ld, b_ld, c_ld;
  int waves;                     // of a pass
  int B, L, D, N, G, Dg, tiles;  // Dg = D / G channels per group, tiles of them per workgroup
  int seg_len, nseg, softplus, out_bf16;
  int span, nspan, span_len;  // spans: segments that a workgroup of the backward's main pass walks; their tokens
  int vec;  // everything may be accessed by fours: channels, states, B and C
  // workspace: segment states [B * nseg][D][N], sums of dt [B * nseg][D]
  float *seg, *sdt;
  // backward
  void *du, *ddelta, *dz;
  float *gseg;        // gradients entering the segments from behind, [B * nseg][D][N]
  float *ck, *ckdt;   // per sub-tile: state relative to the segment, sum of dt before it
  float *bcpart;      // [tiles][B * L][G][2][N]
  float *dApart, *dDpart, *dbpart;  // [B * nspan][D][N], [B * nspan][D]
  float *dh0;
  int subs;           // sub-tiles per segment
};

// Channels per lane of a pass where there are channels enough: up to 16 elements per lane
// share what a token costs beside them (scan_plan says where).  Four channels instead of two were no faster for
// outputs and slower for checkpoints (223 against 179 us at B 2, L 4096, D 4096, N 16), where
// they leave two waves per SIMD.
constexpr int wide_cj(int NS) { return NS <= 8 ? 2 : 1; }

// Channels per lane and tokens per sub-tile of the backward's main pass: a sub-tile's
// states, SUB CJ NS fp32, stay in 64 registers.
constexpr int bwd_cj(int NS) { return NS >= 8 ? 1 : 2; }
constexpr int bwd_sub(int NS) { return std::min(TT, 64 / (NS * bwd_cj(NS))); }
constexpr int BWD_WAVES = 4, PASS_WAVES = 4;
constexpr int SIMDS = 1024;  // of the chip

// What a workgroup works on: a segment, or a span of them.
struct Where {
  int b, s, g, tile, len, t_lo, t_hi;
};
template <bool SPANS>
__device__ __forceinline__ Where where(const ScanArgs &a, int id) {
  Where w;
  w.tile = id % a.tiles;
  id /= a.tiles;
  w.g = id % a.G;
  id /= a.G;
  const int parts = SPANS ? a.nspan : a.nseg;
  w.s = id % parts;
  w.b = id / parts;
  w.len = a.lengths ? min(max(a.lengths[w.b], 0), a.L) : a.L;
  const int p = SPANS ? w.s : w.s / a.span;  // segments end with their span
  const long long end = (long long)(p + 1) * a.span_len, lo = (long long)p * a.span_len + (SPANS ? 0 : w.s % a.span * a.seg_len);
  w.t_lo = (int)min(min(lo, end), (long long)w.len);
  w.t_hi = (int)min(SPANS ? end : min(lo + a.seg_len, end), (long long)w.len);
  return w;
}

// Between a wave's own writes to its LDS and its reads of other lanes' values (and the
// other way round): the hardware keeps a wave's LDS operations in order, this keeps the
// compiler's.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The sum over the four rows of a wave, for four tokens at once: lane row r gets token r.
// The swaps exchange the halves (rows) of two registers, so that each addition sums both.
__device__ __forceinline__ float swap_add32(float x, float y) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap_add16(float x, float y) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float row_sums(const float (&y)[4]) {
  return swap_add16(swap_add32(y[0], y[2]), swap_add32(y[1], y[3]));
}

// Sum over the 16 lanes of a row, in all of them (row rotations by 8, 4, 2, 1).
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row16_sum(float x) {
  x += dpp<0x128>(x);
  x += dpp<0x124>(x);
  x += dpp<0x122>(x);
  x += dpp<0x121>(x);
  return x;
}

// c[i] += x_{n0 + i} y for the lane's four states, where the lanes of a quad hold x_{n0} ..
// x_{n0 + 3} of their row and y is the lane's own (its channel's): an outer product per
// quad, one step of the matrix cores (16 blocks of 4 x 4, in fp32) for four multiplications
// of the vector unit, which is what bounds these kernels.
typedef __attribute__((ext_vector_type(4))) float f32x4;
__device__ __forceinline__ f32x4 quad_outer(float x, float y, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_4x4x1f32(x, y, c, 0, 0, 0);
}

// h <- e h + dtu B for one channel's NS states: Bq are the quad's values of B, Bv the lane's.
template <int NS>
__device__ __forceinline__ void advance(float (&h)[NS], const float (&e)[NS], float dtu, const float (&Bq)[(NS + 3) / 4],
                                        const float (&Bv)[NS]) {
  if constexpr (NS % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
      const f32x4 r = quad_outer(Bq[i / 4], dtu, f32x4{e[i] * h[i], e[i + 1] * h[i + 1], e[i + 2] * h[i + 2], e[i + 3] * h[i + 3]});
#pragma unroll
      for (int k = 0; k < 4; ++k) h[i + k] = r[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) h[i] = e[i] * h[i] + dtu * Bv[i];
  }
}

// A to base 2, kept finite: a rate of the lowest value or -inf still decays at once, and a
// time step of 0 (a masked token, one behind the end) still leaves the state as it is.
__device__ __forceinline__ float rate2(float A) {
  const float r = A * kLog2e;
  return r < -3e38f ? -3e38f : r;
}

// NS states of a lane from n0 on.  VEC: N and n0 are multiples of four, p is aligned.
template <int NS, bool VEC>
__device__ __forceinline__ void load_state(const float *p, int N, int n0, bool ok, float (&h)[NS]) {
  if constexpr (VEC && NS % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (ok && n0 + i < N) v = *(const float4 *)(p + n0 + i);
      h[i] = v.x;
      h[i + 1] = v.y;
      h[i + 2] = v.z;
      h[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) h[i] = ok && n0 + i < N ? p[n0 + i] : 0.0f;
  }
}
template <int NS, bool VEC>
__device__ __forceinline__ void store_state(float *p, int N, int n0, bool ok, const float (&h)[NS]) {
  if constexpr (VEC && NS % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NS; i += 4)
      if (ok && n0 + i < N) *(float4 *)(p + n0 + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (ok && n0 + i < N) p[n0 + i] = h[i];
  }
}

// Four neighbouring elements as they come from memory.  VEC: all four are there, p is
// aligned to them; otherwise n of them are, and the others read as 0.
template <typename T, bool VEC>
struct Quad;
template <bool VEC>
struct Quad<uint16_t, VEC> {
  uint2 v;
  __device__ __forceinline__ void load(const uint16_t *p, int n) {
    if constexpr (VEC) {
      v = *(const uint2 *)p;
    } else {
      v = make_uint2(0u, 0u);
      if (n > 0) v.x = p[0];
      if (n > 1) v.x |= (uint32_t)p[1] << 16;
      if (n > 2) v.y = p[2];
      if (n > 3) v.y |= (uint32_t)p[3] << 16;
    }
  }
  __device__ __forceinline__ void get(float (&r)[4]) const {
    r[0] = __uint_as_float(v.x << 16);
    r[1] = __uint_as_float(v.x & 0xffff0000u);
    r[2] = __uint_as_float(v.y << 16);
    r[3] = __uint_as_float(v.y & 0xffff0000u);
  }
};
template <bool VEC>
struct Quad<float, VEC> {
  float4 v;
  __device__ __forceinline__ void load(const float *p, int n) {
    if constexpr (VEC) {
      v = *(const float4 *)p;
    } else {
      v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (n > 0) v.x = p[0];
      if (n > 1) v.y = p[1];
      if (n > 2) v.z = p[2];
      if (n > 3) v.w = p[3];
    }
  }
  __device__ __forceinline__ void get(float (&r)[4]) const {
    r[0] = v.x;
    r[1] = v.y;
    r[2] = v.z;
    r[3] = v.w;
  }
};

// The CJ neighbouring values of a lane in a row of LDS (four where it staged them, one or two channels in a pass).
template <int CJ>
__device__ __forceinline__ void get_lane(const float *p, float (&r)[CJ]) {
  if constexpr (CJ == 4) {
    const float4 v = *(const float4 *)p;
    r[0] = v.x;
    r[1] = v.y;
    r[2] = v.z;
    r[3] = v.w;
  } else if constexpr (CJ == 2) {
    const float2 v = *(const float2 *)p;
    r[0] = v.x;
    r[1] = v.y;
  } else {
    r[0] = p[0];
  }
}
template <int CJ>
__device__ __forceinline__ void put_lane(float *p, const float (&r)[CJ]) {
  if constexpr (CJ == 2)
    *(float2 *)p = make_float2(r[0], r[1]);
  else
    p[0] = r[0];
}
template <int NS>
__device__ __forceinline__ void get_states(const float *p, float (&r)[NS]) {
  if constexpr (NS % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
      const float4 v = *(const float4 *)(p + i);
      r[i] = v.x;
      r[i + 1] = v.y;
      r[i + 2] = v.z;
      r[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) r[i] = p[i];
  }
}

// The quad's values of a row of states: the lane's is the one of its place in the quad.
template <int NS>
__device__ __forceinline__ void get_quad(const float *p, int lane, float (&r)[(NS + 3) / 4]) {
  if constexpr (NS % 4 == 0)
#pragma unroll
    for (int i = 0; i < NS; i += 4) r[i / 4] = p[i + (lane & 3)];
}

// A lane's share of a tile of B or C: quads of states, NS of them per token.  Wide loads
// are not predicated: tokens and states outside read the nearest ones inside, and put()
// zeroes them.
template <typename T, int NS, bool VEC>
struct StatesIn {
  static constexpr int NQ = (TT * NS + 63) / 64;
  Quad<T, VEC> q[NQ];
  __device__ __forceinline__ void load(const void *src, long long ld, const ScanArgs &a, const Where &w, int t0, int lane) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int id = i * 64 + lane, t = t0 + id / NS, n = id % NS * 4;
      const T *p = (const T *)src + (long long)w.b * a.L * ld + (long long)w.g * a.N;
      if constexpr (VEC)
        q[i].load(p + (long long)min(max(t, w.t_lo), w.t_hi - 1) * ld + min(n, a.N - 4), 4);
      else
        q[i].load(p + (long long)t * ld + n, id < TT * NS && t >= w.t_lo && t < w.t_hi ? a.N - n : 0);
    }
  }
  __device__ __forceinline__ void put(float *dst, const ScanArgs &a, const Where &w, int t0, int lane) const {  // [TT][4 NS]
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int id = i * 64 + lane;
      const bool there = t0 + id / NS < w.t_hi && id % NS * 4 < a.N;
      float r[4];
      q[i].get(r);
      if (TT * NS % 64 == 0 || id < TT * NS)
        *(float4 *)(dst + id * 4) = make_float4(there ? r[0] : 0.0f, there ? r[1] : 0.0f, there ? r[2] : 0.0f,
                                                there ? r[3] : 0.0f);
    }
  }
};

// A lane's share of a tile of channels: CJ quads, of tokens TT / CJ apart and channels
// d .. d + 3 (of which nc are the lane's own: none, if the group ends before them; the wide
// load then reads the group's last four).  Its users zero what is outside.
template <typename T, int CJ, bool VEC>
struct ChannelsIn {
  Quad<T, VEC> q[CJ];
  __device__ __forceinline__ void load(const void *src, long long ld, const ScanArgs &a, const Where &w, int t0, int tt,
                                       long long d, int nc) {
    const T *p = (const T *)src + (long long)w.b * a.L * ld + d;
#pragma unroll
    for (int i = 0; i < CJ; ++i) {
      const int t = t0 + i * (TT / CJ) + tt;
      if constexpr (VEC)
        q[i].load(p + (long long)min(max(t, w.t_lo), w.t_hi - 1) * ld, 4);
      else
        q[i].load(p + (long long)t * ld, t >= w.t_lo && t < w.t_hi ? nc : 0);
    }
  }
};

// The n values that a lane's four channels have, the others 0 (or anything, where n is 0).
template <bool VEC>
__device__ __forceinline__ void load_channels(const float *p, int n, float (&r)[4]) {
  if constexpr (VEC) {
    const float4 v = *(const float4 *)p;
    r[0] = v.x;
    r[1] = v.y;
    r[2] = v.z;
    r[3] = v.w;
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) r[c] = c < n ? p[c] : 0.0f;
  }
}

enum { OUTPUT, STATES, CHECKPOINTS };

// A wave's part of LDS in a pass.
template <int NS, int CJ, int MODE>
struct PassLds {
  float dt[TT][16 * CJ], du[TT][16 * CJ];  // dt, dt u; OUTPUT: y replaces dt u
  float dy[MODE == CHECKPOINTS ? TT : 1][16 * CJ];
  float B[TT][4 * NS], C[MODE == STATES ? 1 : TT][4 * NS];
};

// One pass over a segment.  Bound by the vector unit: at B 1, L 32768, D 2048, N 16, bf16
// OUTPUT takes 286 us (537 MB; busy 93 %), STATES 218 us (88 %), and CHECKPOINTS 173 us (87 %)
// at B 2, L 4096, D 4096.
//   OUTPUT: from the state entering the segment, the gated outputs; the last segment
//     writes the final state.
//   STATES: from zero, the segment's own final state and its sum of dt.
//   CHECKPOINTS (backward): as STATES, also the state and the sum of dt before every
//     sub-tile, and the gradient that the segment's own outputs send to the state in
//     front of it, sum_t exp(A sum dt) C_t dy_t.
template <typename T, int NS, int CJ, int MODE, bool VEC>
__global__ __launch_bounds__(64 * PASS_WAVES, MODE == CHECKPOINTS && NS * CJ >= 16 ? 2 : 3) void scan_pass_kernel(ScanArgs a) {
  constexpr int NP = 4 * NS, CW = 16 * CJ, SUB = bwd_sub(NS);
  extern __shared__ __align__(16) char shared[];
  PassLds<NS, CJ, MODE> *lds = (PassLds<NS, CJ, MODE> *)shared;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), id = blockIdx.x * (blockDim.x >> 6) + wave;
  if (id >= a.waves) return;
  float(*const dts)[CW] = lds[wave].dt, (*const dus)[CW] = lds[wave].du, (*const dys)[CW] = lds[wave].dy;
  float(*const Bs)[NP] = lds[wave].B, (*const Cs)[NP] = lds[wave].C;
  const Where w = where<false>(a, id);
  const bool last = w.s == a.nseg - 1;
  const int lane = threadIdx.x & 63, row = lane >> 4, c0 = (lane & 15) * CJ, n0 = row * NS;
  const int rel = w.tile * CW + c0;
  const long long d = (long long)w.g * a.Dg + rel;
  const long long sd = ((long long)w.b * a.nseg + w.s) * a.D + d;
  // the lane's part of the staging
  const int tt = lane / (4 * CJ), cq = lane % (4 * CJ) * 4, relq = w.tile * CW + cq;
  const int nc = min(max(a.Dg - relq, 0), 4);
  const long long dq = (long long)w.g * a.Dg + (VEC ? min(relq, a.Dg - 4) : relq);
  ChannelsIn<T, CJ, VEC> un, xn, zn, gn;
  StatesIn<T, NS, VEC> bn, cn;
  auto fetch = [&](int t0) {
    un.load(a.u, a.u_ld, a, w, t0, tt, dq, nc);
    xn.load(a.delta, a.delta_ld, a, w, t0, tt, dq, nc);
    bn.load(a.Bm, a.b_ld, a, w, t0, lane);
    if constexpr (MODE != STATES) {
      if (a.z) zn.load(a.z, a.z_ld, a, w, t0, tt, dq, nc);
      cn.load(a.Cm, a.c_ld, a, w, t0, lane);
    }
    if constexpr (MODE == CHECKPOINTS) gn.load(a.d_o, a.D, a, w, t0, tt, dq, nc);
  };
  if (w.t_lo < w.t_hi) fetch(w.t_lo);
  float A2[CJ][NS], h[CJ][NS], gs[CJ][NS], pr[CJ][NS], sum[CJ];
#pragma unroll
  for (int j = 0; j < CJ; ++j) {
    load_state<NS, VEC>(a.A + (d + j) * a.N, a.N, n0, rel + j < a.Dg, A2[j]);
    sum[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      A2[j][i] = rate2(A2[j][i]);
      h[j][i] = 0.0f;
      gs[j][i] = 0.0f;
      pr[j][i] = 1.0f;
    }
    if constexpr (MODE == OUTPUT) {
      if (a.nseg > 1)
        load_state<NS, VEC>(a.seg + (sd + j) * a.N, a.N, n0, rel + j < a.Dg, h[j]);
      else if (a.h0)
        load_state<NS, VEC>(a.h0 + (sd + j) * a.N, a.N, n0, rel + j < a.Dg, h[j]);
    }
  }
  float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f}, Dsk[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (a.bias) load_channels<VEC>(a.bias + dq, nc, bias);
  if (MODE == OUTPUT && a.Dskip) load_channels<VEC>(a.Dskip + dq, nc, Dsk);
  for (int t0 = w.t_lo; t0 < w.t_hi; t0 += TT) {
    ChannelsIn<T, CJ, VEC> uc, zc;
#pragma unroll
    for (int i = 0; i < CJ; ++i) {
      const int k = i * (TT / CJ) + tt;
      const bool live = t0 + k < w.t_hi && nc > 0;
      float u[4], x[4], z[4], g[4], dt[4], dtu[4];
      un.q[i].get(u);
      xn.q[i].get(x);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float v = x[c] + bias[c];
        const bool there = VEC ? live : live && c < nc;
        dt[c] = there ? a.softplus ? softplus(v) : v : 0.0f;
        dtu[c] = there ? dt[c] * u[c] : 0.0f;
      }
      *(float4 *)&dts[k][cq] = make_float4(dt[0], dt[1], dt[2], dt[3]);
      *(float4 *)&dus[k][cq] = make_float4(dtu[0], dtu[1], dtu[2], dtu[3]);
      if constexpr (MODE == CHECKPOINTS) {
        gn.q[i].get(g);
        if (a.z) {
          zn.q[i].get(z);
#pragma unroll
          for (int c = 0; c < 4; ++c) g[c] *= z[c] * sigmoid(z[c]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) g[c] = (VEC ? live : live && c < nc) ? g[c] : 0.0f;
        *(float4 *)&dys[k][cq] = make_float4(g[0], g[1], g[2], g[3]);
      }
      uc.q[i] = un.q[i];
      if (MODE == OUTPUT && a.z) zc.q[i] = zn.q[i];
    }
    bn.put(&Bs[0][0], a, w, t0, lane);
    if constexpr (MODE != STATES) cn.put(&Cs[0][0], a, w, t0, lane);
    fetch(t0 + TT);
    wave_sync();
    // Unrolled over all of the tile (tokens behind the end have no time step and leave the state),
    // so that the reads of later tokens go ahead of the chain: uncut, 1024 waves, N 16, 4096
    // tokens: 518 -> 443 us.  Not with two states a lane (575 -> 623 us) and for
    // checkpoints, which would spill.
    constexpr int AHEAD = MODE == CHECKPOINTS || NS == 2 ? 1 : 4;
    const int nt = AHEAD == 4 ? TT : min(TT, w.t_hi - t0);
#pragma unroll AHEAD
    for (int t4 = 0; t4 < nt; t4 += 4) {
      if constexpr (MODE == CHECKPOINTS) {
        if (t4 % SUB == 0) {
          const long long k = ((long long)w.b * a.nseg + w.s) * a.subs + (t0 - w.t_lo + t4) / SUB;
#pragma unroll
          for (int j = 0; j < CJ; ++j) {
            store_state<NS, VEC>(a.ck + (k * a.D + d + j) * a.N, a.N, n0, rel + j < a.Dg, h[j]);
            if (rel + j < a.Dg && row == 0) a.ckdt[k * a.D + d + j] = sum[j];
          }
        }
      }
      float y[CJ][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float dt[CJ], dtu[CJ], dy[CJ], Bv[NS], Cv[NS], Bq[(NS + 3) / 4];
        get_lane(&dts[t4 + k][c0], dt);
        get_lane(&dus[t4 + k][c0], dtu);
        get_quad<NS>(&Bs[t4 + k][n0], lane, Bq);
        if constexpr (NS % 4) get_states(&Bs[t4 + k][n0], Bv);
        if constexpr (MODE != STATES) get_states(&Cs[t4 + k][n0], Cv);
        if constexpr (MODE == CHECKPOINTS) get_lane(&dys[t4 + k][c0], dy);
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
          float acc = 0.0f;
          if constexpr (MODE != OUTPUT) sum[j] += dt[j];
          float e[NS];
#pragma unroll
          for (int i = 0; i < NS; ++i) e[i] = __builtin_amdgcn_exp2f(dt[j] * A2[j][i]);
          advance(h[j], e, dtu[j], Bq, Bv);
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            if constexpr (MODE == OUTPUT) acc += h[j][i] * Cv[i];
            if constexpr (MODE == CHECKPOINTS) {
              pr[j][i] *= e[i];
              gs[j][i] += pr[j][i] * (dy[j] * Cv[i]);
            }
          }
          y[j][k] = acc;
        }
      }
      if constexpr (MODE == OUTPUT) {
        float v[CJ];
#pragma unroll
        for (int j = 0; j < CJ; ++j) v[j] = row_sums(y[j]);
        put_lane(&dus[t4 + row][c0], v);  // the wave is past these tokens' dt u
      }
    }
    wave_sync();
    if constexpr (MODE == OUTPUT) {
#pragma unroll
      for (int i = 0; i < CJ; ++i) {
        const int k = i * (TT / CJ) + tt;
        float u[4], z[4], o[4];
        const float4 y = *(const float4 *)&dus[k][cq];
        uc.q[i].get(u);
        o[0] = y.x + Dsk[0] * u[0];
        o[1] = y.y + Dsk[1] * u[1];
        o[2] = y.z + Dsk[2] * u[2];
        o[3] = y.w + Dsk[3] * u[3];
        if (a.z) {
          zc.q[i].get(z);
#pragma unroll
          for (int c = 0; c < 4; ++c) o[c] *= z[c] * sigmoid(z[c]);
        }
        if (t0 + k < w.t_hi && nc > 0)
          store4<VEC>(a.out, ((long long)w.b * a.L + t0 + k) * a.D + dq, nc, o, a.out_bf16);
      }
      wave_sync();
    }
  }
#pragma unroll
  for (int j = 0; j < CJ; ++j) {
    const bool ok = rel + j < a.Dg;
    if constexpr (MODE == OUTPUT) {
      if (last && a.hT) store_state<NS, VEC>(a.hT + ((long long)w.b * a.D + d + j) * a.N, a.N, n0, ok, h[j]);
    } else {
      store_state<NS, VEC>(a.seg + (sd + j) * a.N, a.N, n0, ok, h[j]);
      if (ok && row == 0) a.sdt[sd + j] = sum[j];
      if constexpr (MODE == CHECKPOINTS) store_state<NS, VEC>(a.gseg + (sd + j) * a.N, a.N, n0, ok, gs[j]);
    }
  }
}

// Segment states -> states entering the segments, in place (blockIdx.y 0), and gradients of
// the segments -> gradients entering them from behind (1).  One thread per (sequence,
// channel, state); the chain over segments is short next to its loads, which go ahead by 32.
// Bound by their latency: 4 to 16 us (128 segments of 32768 states).
__global__ __launch_bounds__(NT) void scan_combine_kernel(ScanArgs a) {
  const long long DN = (long long)a.D * a.N, id = (long long)blockIdx.x * NT + threadIdx.x;
  if (id >= a.B * DN) return;
  constexpr int U = 32;
  const long long b = id / DN, e = id % DN, d = e / a.N;
  const bool back = blockIdx.y != 0;
  const float A2 = rate2(a.A[e]);
  // from the first segment on, or from the last back
  const long long first = b * a.nseg + (back ? a.nseg - 1 : 0), way = back ? -1 : 1;
  const float *sdt = a.sdt + first * a.D + d;
  float *S = (back ? a.gseg : a.seg) + first * DN + e;
  const float *h = back ? a.dhT : a.h0;
  float own[U], dt[U], carry = h ? h[id] : 0.0f;
  for (int s0 = 0; s0 < a.nseg; s0 += U) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const long long s = way * min(s0 + k, a.nseg - 1);
      own[k] = S[s * DN];
      dt[k] = sdt[s * a.D];
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (s0 + k < a.nseg) {
        S[way * (s0 + k) * DN] = carry;
        carry = __builtin_amdgcn_exp2f(A2 * dt[k]) * carry + own[k];
      }
  }
}

// The backward's sums over a wave's channels, for one token: the products of a lane, NS of
// dB and NS of dC, are summed over the row's 16 lanes.  Four states of both together: the
// first two steps halve the number of registers as well, since the bank mask of a row
// operation lets two sums share one (lanes 0-7 keep the first, 8-15 the second; then banks
// of four): 16 additions for eight sums instead of 32.  out: [2][4 NS] of the token.
template <int NS>
__device__ __forceinline__ void channel_sums(const float (&pB)[NS], const float (&pC)[NS], int lane, float *out) {
  const int row = lane >> 4;
  if constexpr (NS % 4 == 0) {
    const int bank = (lane >> 2) & 3, state = (bank & 1) * 2 + (bank >> 1);
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
      float b, c, t0, t1, t2, t3;
      // two instructions, or that many idle slots, between a register's write and its use by a row operation
      asm("s_nop 1\n"
          "v_add_f32_dpp %2, %6, %6 row_ror:8 row_mask:0xf bank_mask:0x3\n"
          "v_add_f32_dpp %2, %7, %7 row_ror:8 row_mask:0xf bank_mask:0xc\n"
          "v_add_f32_dpp %3, %8, %8 row_ror:8 row_mask:0xf bank_mask:0x3\n"
          "v_add_f32_dpp %3, %9, %9 row_ror:8 row_mask:0xf bank_mask:0xc\n"
          "v_add_f32_dpp %4, %10, %10 row_ror:8 row_mask:0xf bank_mask:0x3\n"
          "v_add_f32_dpp %4, %11, %11 row_ror:8 row_mask:0xf bank_mask:0xc\n"
          "v_add_f32_dpp %5, %12, %12 row_ror:8 row_mask:0xf bank_mask:0x3\n"
          "v_add_f32_dpp %5, %13, %13 row_ror:8 row_mask:0xf bank_mask:0xc\n"
          "v_add_f32_dpp %0, %2, %2 row_half_mirror row_mask:0xf bank_mask:0x5\n"
          "v_add_f32_dpp %0, %3, %3 row_half_mirror row_mask:0xf bank_mask:0xa\n"
          "v_add_f32_dpp %1, %4, %4 row_half_mirror row_mask:0xf bank_mask:0x5\n"
          "v_add_f32_dpp %1, %5, %5 row_half_mirror row_mask:0xf bank_mask:0xa\n"
          "v_add_f32_dpp %0, %0, %0 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n"
          "s_nop 0\n"
          "v_add_f32_dpp %1, %1, %1 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n"
          "v_add_f32_dpp %0, %0, %0 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n"
          "s_nop 0\n"
          "v_add_f32_dpp %1, %1, %1 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n"
          : "=&v"(b), "=&v"(c), "=&v"(t0), "=&v"(t1), "=&v"(t2), "=&v"(t3)
          : "v"(pB[i]), "v"(pB[i + 1]), "v"(pB[i + 2]), "v"(pB[i + 3]), "v"(pC[i]), "v"(pC[i + 1]), "v"(pC[i + 2]),
            "v"(pC[i + 3]));
      out[(lane & 1) * 4 * NS + row * NS + i + state] = lane & 1 ? c : b;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const float b = row16_sum(pB[i]), c = row16_sum(pC[i]);
      out[(lane & 1) * 4 * NS + row * NS + i] = lane & 1 ? c : b;
    }
  }
}

// The backward's main pass over a span of segments, tiles and sub-tiles from the last to
// the first: each sub-tile's states are computed again from its checkpoint and kept in
// registers; then the gradient of the state runs against time, computing the decays once
// more (keeping them too took the registers that hold the next checkpoint's loads).  The
// waves of a workgroup work on neighbouring channels and meet once per tile, to add up
// their sums for dB and dC.  Bound by the vector unit (busy 82 %): 460 us at B 2, L 4096,
// D 4096, N 16, bf16; with the decays kept in registers 580 became 760 us.
template <typename T, int NS, bool VEC>
__global__ __launch_bounds__(64 * BWD_WAVES, NS >= 16 ? 1 : 2) void scan_bwd_kernel(ScanArgs a) {
  constexpr int NP = 4 * NS, CJ = bwd_cj(NS), CW = 16 * CJ, SUB = bwd_sub(NS);
  struct WaveLds {
    float dt[TT][CW];
    float du[TT][CW];  // dt u, then sum_n g B
    float dy[TT][CW];  // dy, then sum_n A w
    float y[TT][CW];   // C . h
    float B[TT][NP], C[TT][NP];
  };
  __shared__ __align__(16) WaveLds lds[BWD_WAVES];
  __shared__ float part[2][BWD_WAVES][TT][2][NP];  // each wave's sums over its channels
  const Where w = where<true>(a, blockIdx.x);
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int row = lane >> 4, c0 = (lane & 15) * CJ, n0 = row * NS;
  const int base = (w.tile * waves + wave) * CW, rel = base + c0;
  const long long d = (long long)w.g * a.Dg + rel;
  const long long bs = (long long)w.b * a.nspan + w.s;
  WaveLds &s = lds[wave];
  const int tt = lane / (4 * CJ), cq = lane % (4 * CJ) * 4, relq = base + cq;
  const int nc = min(max(a.Dg - relq, 0), 4);
  const long long dq = (long long)w.g * a.Dg + (VEC ? min(relq, a.Dg - 4) : relq);
  ChannelsIn<T, CJ, VEC> un, xn, zn, gn;
  StatesIn<T, NS, VEC> bn, cn;
  auto fetch = [&](int t0) {
    un.load(a.u, a.u_ld, a, w, t0, tt, dq, nc);
    xn.load(a.delta, a.delta_ld, a, w, t0, tt, dq, nc);
    if (a.z) zn.load(a.z, a.z_ld, a, w, t0, tt, dq, nc);
    gn.load(a.d_o, a.D, a, w, t0, tt, dq, nc);
    bn.load(a.Bm, a.b_ld, a, w, t0, lane);
    cn.load(a.Cm, a.c_ld, a, w, t0, lane);
  };
  const int ntile = (w.t_hi - w.t_lo + TT - 1) / TT;
  if (ntile > 0) fetch(w.t_lo + (ntile - 1) * TT);
  float A2[CJ][NS], carry[CJ][NS], dA[CJ][NS];
#pragma unroll
  for (int j = 0; j < CJ; ++j) {
    const bool ok = rel + j < a.Dg;
    load_state<NS, VEC>(a.A + (d + j) * a.N, a.N, n0, ok, A2[j]);
    const int end = min((w.s + 1) * a.span, a.nseg) - 1;  // the span's last segment
    load_state<NS, VEC>(a.gseg + (((long long)w.b * a.nseg + end) * a.D + d + j) * a.N, a.N, n0, ok, carry[j]);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      A2[j][i] = rate2(A2[j][i]);
      dA[j][i] = 0.0f;
    }
  }
  float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f}, Dsk[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  float sD[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sb[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (a.bias) load_channels<VEC>(a.bias + dq, nc, bias);
  if (a.Dskip) load_channels<VEC>(a.Dskip + dq, nc, Dsk);
  // the state in front of a sub-tile: its checkpoint, and what the segment's entering
  // state has become; loaded one sub-tile ahead
  float hck[CJ][NS], hin[CJ][NS], before[CJ];
  const int last = w.t_hi - w.t_lo - 1;  // of the span's tokens
  int ck_seg = max(last, 0) / a.seg_len, ck_sub = max(last, 0) % a.seg_len / SUB;
  auto checkpoint = [&]() {  // the next one towards the span's start, and then the one before it
    const long long seg = (long long)w.b * a.nseg + w.s * a.span + ck_seg, k = seg * a.subs + ck_sub;
#pragma unroll
    for (int j = 0; j < CJ; ++j) {
      const bool ok = rel + j < a.Dg && ck_seg >= 0;
      load_state<NS, VEC>(a.ck + (k * a.D + d + j) * a.N, a.N, n0, ok, hck[j]);
      load_state<NS, VEC>(a.seg + (seg * a.D + d + j) * a.N, a.N, n0, ok, hin[j]);
      before[j] = ok ? a.ckdt[k * a.D + d + j] : 0.0f;
    }
    if (--ck_sub < 0) {
      --ck_seg;
      ck_sub = a.subs - 1;
    }
  };
  if (ntile > 0) checkpoint();
  for (int tile = ntile - 1; tile >= 0; --tile) {
    const int t0 = w.t_lo + tile * TT;
#pragma unroll
    for (int i = 0; i < CJ; ++i) {
      const int k = i * (TT / CJ) + tt;
      const bool live = t0 + k < w.t_hi && nc > 0;
      float u[4], x[4], z[4], g[4], dt[4], dtu[4];
      un.q[i].get(u);
      xn.q[i].get(x);
      gn.q[i].get(g);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float v = x[c] + bias[c];
        const bool there = VEC ? live : live && c < nc;
        dt[c] = there ? a.softplus ? softplus(v) : v : 0.0f;
        dtu[c] = there ? dt[c] * u[c] : 0.0f;
      }
      if (a.z) {
        zn.q[i].get(z);
#pragma unroll
        for (int c = 0; c < 4; ++c) g[c] *= z[c] * sigmoid(z[c]);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) g[c] = (VEC ? live : live && c < nc) ? g[c] : 0.0f;
      *(float4 *)&s.dt[k][cq] = make_float4(dt[0], dt[1], dt[2], dt[3]);
      *(float4 *)&s.du[k][cq] = make_float4(dtu[0], dtu[1], dtu[2], dtu[3]);
      *(float4 *)&s.dy[k][cq] = make_float4(g[0], g[1], g[2], g[3]);
    }
    bn.put(&s.B[0][0], a, w, t0, lane);
    cn.put(&s.C[0][0], a, w, t0, lane);
    wave_sync();
    const int nt = min(TT, w.t_hi - t0);
    float(*ps)[2][NP] = part[tile & 1][wave];
    for (int t1 = (nt - 1) / SUB * SUB; t1 >= 0; t1 -= SUB) {
      float h[CJ][NS], hstart[CJ][NS], hh[SUB][CJ][NS], y[CJ][4];
#pragma unroll
      for (int j = 0; j < CJ; ++j)
#pragma unroll
        for (int i = 0; i < NS; ++i)
          h[j][i] = hstart[j][i] = hck[j][i] + __builtin_amdgcn_exp2f(A2[j][i] * before[j]) * hin[j][i];
      checkpoint();
#pragma unroll
      for (int t = 0; t < SUB; ++t) {
        float dt[CJ], dtu[CJ], Bv[NS], Cv[NS], Bq[(NS + 3) / 4];
        get_lane(&s.dt[t1 + t][c0], dt);
        get_lane(&s.du[t1 + t][c0], dtu);
        get_quad<NS>(&s.B[t1 + t][n0], lane, Bq);
        if constexpr (NS % 4) get_states(&s.B[t1 + t][n0], Bv);
        get_states(&s.C[t1 + t][n0], Cv);
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
          float acc = 0.0f, e[NS];
#pragma unroll
          for (int i = 0; i < NS; ++i) e[i] = __builtin_amdgcn_exp2f(dt[j] * A2[j][i]);
          advance(h[j], e, dtu[j], Bq, Bv);
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            hh[t][j][i] = h[j][i];
            acc += h[j][i] * Cv[i];
          }
          y[j][t & 3] = acc;
        }
        if ((t & 3) == 3) {
          float v[CJ];
#pragma unroll
          for (int j = 0; j < CJ; ++j) v[j] = row_sums(y[j]);
          put_lane(&s.y[t1 + (t & ~3) + row][c0], v);
        }
      }
#pragma unroll
      for (int t4 = SUB - 4; t4 >= 0; t4 -= 4) {
        float gB[CJ][4], sA[CJ][4];
#pragma unroll
        for (int q = 3; q >= 0; --q) {
          const int t = t4 + q;
          float dt[CJ], dtu[CJ], dy[CJ], Bv[NS], Cv[NS], Cq[(NS + 3) / 4], pB[NS], pC[NS];
          get_lane(&s.dt[t1 + t][c0], dt);
          get_lane(&s.du[t1 + t][c0], dtu);
          get_lane(&s.dy[t1 + t][c0], dy);
          get_states(&s.B[t1 + t][n0], Bv);
          get_quad<NS>(&s.C[t1 + t][n0], lane, Cq);
          if constexpr (NS % 4) get_states(&s.C[t1 + t][n0], Cv);
#pragma unroll
          for (int j = 0; j < CJ; ++j) {
            gB[j][q] = sA[j][q] = 0.0f;
            float gt[NS];
            if constexpr (NS % 4 == 0) {
#pragma unroll
              for (int i = 0; i < NS; i += 4) {
                const f32x4 r = quad_outer(Cq[i / 4], dy[j], f32x4{carry[j][i], carry[j][i + 1], carry[j][i + 2], carry[j][i + 3]});
#pragma unroll
                for (int k = 0; k < 4; ++k) gt[i + k] = r[k];
              }
            } else {
#pragma unroll
              for (int i = 0; i < NS; ++i) gt[i] = Cv[i] * dy[j] + carry[j][i];
            }
#pragma unroll
            for (int i = 0; i < NS; ++i) {
              const float g = gt[i];
              carry[j][i] = __builtin_amdgcn_exp2f(dt[j] * A2[j][i]) * g;
              const float wv = carry[j][i] * (t > 0 ? hh[t > 0 ? t - 1 : 0][j][i] : hstart[j][i]);
              sA[j][q] += A2[j][i] * wv;  // times log2 e; taken out below
              dA[j][i] += dt[j] * wv;
              gB[j][q] += g * Bv[i];
              pB[i] = j ? pB[i] + g * dtu[j] : g * dtu[j];
              pC[i] = j ? pC[i] + dy[j] * hh[t][j][i] : dy[j] * hh[t][j][i];
            }
          }
          channel_sums(pB, pC, lane, &ps[t1 + t][0][0]);
        }
        float vB[CJ], vA[CJ];
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
          vB[j] = row_sums(gB[j]);
          vA[j] = kLn2 * row_sums(sA[j]);
        }
        // the wave is past these tokens
        put_lane(&s.du[t1 + t4 + row][c0], vB);
        put_lane(&s.dy[t1 + t4 + row][c0], vA);
      }
    }
    wave_sync();
    // the inputs stayed in registers; the next tile's take their place as they are used
    const ChannelsIn<T, CJ, VEC> uc = un, xc = xn, zc = zn, gc = gn;
    fetch(t0 - TT);
#pragma unroll
    for (int i = 0; i < CJ; ++i) {
      const int k = i * (TT / CJ) + tt;
      float u[4], x[4], z[4], g[4], dt[4], gB[4], sA[4], y[4], du[4], dd[4], dz[4];
      uc.q[i].get(u);
      xc.q[i].get(x);
      gc.q[i].get(g);
      get_lane(&s.dt[k][cq], dt);
      get_lane(&s.du[k][cq], gB);
      get_lane(&s.dy[k][cq], sA);
      get_lane(&s.y[k][cq], y);
      if (a.z) zc.q[i].get(z);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float dy = g[c];
        if (a.z) {
          const float sg = sigmoid(z[c]), gate = z[c] * sg;
          dy *= gate;
          dz[c] = g[c] * (y[c] + Dsk[c] * u[c]) * (sg + gate * (1.0f - sg));
        }
        du[c] = gB[c] * dt[c] + dy * Dsk[c];
        dd[c] = sA[c] + gB[c] * u[c];
        if (a.softplus) {  // no slope (a masked token): 0, also where a rate of the lowest value made the sum overflow
          const float slope = sigmoid(x[c] + bias[c]);
          dd[c] = slope == 0.0f ? 0.0f : dd[c] * slope;
        }
        const bool live = t0 + k < w.t_hi && c < nc;
        sD[c] += live ? dy * u[c] : 0.0f;
        sb[c] += live ? dd[c] : 0.0f;
      }
      if (t0 + k < w.t_hi && nc > 0) {
        const long long o = ((long long)w.b * a.L + t0 + k) * a.D + dq;
        store4<VEC>(a.du, o, nc, du, a.out_bf16);
        store4<VEC>(a.ddelta, o, nc, dd, a.out_bf16);
        if (a.z) store4<VEC>(a.dz, o, nc, dz, a.out_bf16);
      }
    }
    __syncthreads();
    // the other half of part is written before the next barrier, this one behind it
    for (int e = threadIdx.x; e < nt * 2 * NP; e += blockDim.x) {
      const int t = e / (2 * NP), k = e / NP % 2, n = e % NP;
      if (n >= a.N) continue;
      float x = part[tile & 1][0][t][k][n];
      for (int v = 1; v < waves; ++v) x += part[tile & 1][v][t][k][n];
      a.bcpart[((((long long)w.tile * a.B + w.b) * a.L + t0 + t) * a.G + w.g) * 2 * a.N + k * a.N + n] = x;
    }
  }
#pragma unroll
  for (int j = 0; j < CJ; ++j) {
    const bool ok = rel + j < a.Dg;
    store_state<NS, VEC>(a.dApart + (bs * a.D + d + j) * a.N, a.N, n0, ok, dA[j]);
    if (w.s == 0 && a.dh0) store_state<NS, VEC>(a.dh0 + ((long long)w.b * a.D + d + j) * a.N, a.N, n0, ok, carry[j]);
  }
  // dD and the bias's gradient: the lanes that staged a channel's tokens
  wave_sync();
  *(float4 *)&s.dt[tt][cq] = make_float4(sD[0], sD[1], sD[2], sD[3]);
  *(float4 *)&s.du[tt][cq] = make_float4(sb[0], sb[1], sb[2], sb[3]);
  wave_sync();
  if (lane < CW && base + lane < a.Dg) {
    float x = 0.0f, y = 0.0f;
#pragma unroll
    for (int k = 0; k < TT / CJ; ++k) {
      x += s.dt[k][lane];
      y += s.du[k][lane];
    }
    const long long e = bs * a.D + (long long)w.g * a.Dg + base + lane;
    a.dDpart[e] = x;
    a.dbpart[e] = y;
  }
}

// Rows behind the sequences' ends: zero gradients of u, delta and z.
__global__ __launch_bounds__(NT) void scan_bwd_tail_kernel(ScanArgs a) {
  for (long long r = blockIdx.x; r < (long long)a.B * a.L; r += gridDim.x) {
    if (r % a.L < min(max(a.lengths[r / a.L], 0), a.L)) continue;
    for (int d = threadIdx.x; d < a.D; d += NT) {
      store_elem(a.du, r * a.D + d, 0.0f, a.out_bf16);
      store_elem(a.ddelta, r * a.D + d, 0.0f, a.out_bf16);
      if (a.dz) store_elem(a.dz, r * a.D + d, 0.0f, a.out_bf16);
    }
  }
}

// The backward's last sums, over the workgroups of the main pass, in their order: dB and dC
// over a group's channel tiles (the first bc_blocks workgroups, a thread a value), and dA,
// dD and the bias's gradient over sequences and spans (COLS values a workgroup, ROWS threads
// each, in double: thousands of partial sums may come together).
constexpr int COLS = 32, ROWS = 16;
__global__ __launch_bounds__(COLS * ROWS) void scan_reduce_kernel(ScanArgs a, void *dB, void *dC, float *dA, float *dD,
                                                                  float *dbias, long long bc_blocks) {
  constexpr int U = 8;
  if (blockIdx.x < bc_blocks) {
    const long long total = (long long)a.B * a.L * a.G * 2 * a.N, step = bc_blocks * (COLS * ROWS);
    for (long long id = (long long)blockIdx.x * (COLS * ROWS) + threadIdx.x; id < total; id += step) {
      const long long rg = id / (2 * a.N), r = rg / a.G;
      const int k = (int)(id - rg * 2 * a.N);
      float x = 0.0f;
      if (!a.lengths || r % a.L < a.lengths[r / a.L])
        for (int t = 0; t < a.tiles; t += U) {
          float v[U];
#pragma unroll
          for (int i = 0; i < U; ++i) v[i] = t + i < a.tiles ? a.bcpart[(t + i) * total + id] : 0.0f;
#pragma unroll
          for (int i = 0; i < U; ++i) x += v[i];
        }
      store_elem(k < a.N ? dB : dC, rg * a.N + (k < a.N ? k : k - a.N), x, a.out_bf16);
    }
    return;
  }
  __shared__ double red[ROWS][COLS];
  const int c = threadIdx.x % COLS, r0 = threadIdx.x / COLS, rows = a.B * a.nspan;
  long long col = (blockIdx.x - bc_blocks) * COLS + c, cols = (long long)a.D * a.N;
  const float *part = a.dApart;
  float *out = dA;
  if (col >= cols) {
    col -= cols;
    cols = a.D;
    part = a.dDpart;
    out = dD;
    if (col >= cols) {
      col -= cols;
      part = a.dbpart;
      out = dbias;
    }
  }
  const bool there = col < cols && out;
  double x = 0.0;
  if (there)
    for (int r = r0; r < rows; r += U * ROWS) {
      float v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) v[k] = r + k * ROWS < rows ? part[(r + k * ROWS) * cols + col] : 0.0f;
#pragma unroll
      for (int k = 0; k < U; ++k) x += v[k];
    }
  red[r0][c] = x;
  __syncthreads();
  if (r0 != 0 || !there) return;
#pragma unroll
  for (int k = 1; k < ROWS; ++k) x += red[k][c];
  out[col] = (float)x;
}

__global__ __launch_bounds__(NT) void state_copy_kernel(float *dst, const float *src, long long n) {
  for (long long i = (long long)blockIdx.x * NT + threadIdx.x; i < n; i += (long long)gridDim.x * NT)
    dst[i] = src ? src[i] : 0.0f;
}
hipError_t state_copy(float *dst, const float *src, long long n, hipStream_t st) {
  if (!dst || dst == src || n == 0) return hipSuccess;
  hipLaunchKernelGGL(state_copy_kernel, dim3((unsigned)std::min<long long>(rec_cdiv(n, NT), 4096)), dim3(NT), 0, st,
                     dst, src, n);
  return hipGetLastError();
}

constexpr int STEP_CH = 64;  // channels of a workgroup's four waves

// One token: a wave's lanes as in the passes above with one channel each; bound by reading
// and writing the states once: 15.5 us for B 128, D 4096, N 16, 75 MB, 4.9 TB/s.
// SQ sequences share their channels' A and have their loads in flight together.
template <typename T, int NS, int SQ, bool VEC>
__global__ __launch_bounds__(NT) void scan_step_kernel(ScanArgs a) {
  const int tid = threadIdx.x, lane = tid & 63, row = lane >> 4, ch = (tid >> 6) * 16 + (lane & 15);
  int id = blockIdx.x;
  const int tile = id % a.tiles;
  id /= a.tiles;
  const int g = id % a.G;
  const int b0 = id / a.G * SQ;
  const int rel = tile * STEP_CH + ch, n0 = row * NS;
  const bool ok = rel < a.Dg;
  const long long d = (long long)g * a.Dg + rel;
  constexpr int bf = sizeof(T) == 2;
  float A[NS], h[SQ][NS], u[SQ], x[SQ], z[SQ], y[SQ];
  constexpr bool VQ = VEC && NS % 4 == 0;  // a lane's states come in whole quads
  Quad<T, VQ> Bq[SQ][(NS + 3) / 4], Cq[SQ][(NS + 3) / 4];
#pragma unroll
  for (int q = 0; q < SQ; ++q) {
    const long long b = min(b0 + q, a.B - 1);
    load_state<NS, VEC>(a.hT + (b * a.D + d) * a.N, a.N, n0, ok, h[q]);
    u[q] = ok ? load_elem(a.u, b * a.u_ld + d, bf) : 0.0f;
    x[q] = ok ? load_elem(a.delta, b * a.delta_ld + d, bf) : 0.0f;
    z[q] = ok && a.z ? load_elem(a.z, b * a.z_ld + d, bf) : 0.0f;
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
      // states behind N (their A, and so their state, is 0 and stays unwritten): any quad inside
      const int at = VQ ? min(n0 + i, a.N - 4) : n0 + i, n = min(a.N - n0 - i, NS - i);
      Bq[q][i / 4].load((const T *)a.Bm + b * a.b_ld + (long long)g * a.N + at, n);
      Cq[q][i / 4].load((const T *)a.Cm + b * a.c_ld + (long long)g * a.N + at, n);
    }
  }
  load_state<NS, VEC>(a.A + d * a.N, a.N, n0, ok, A);
  const float bias = ok && a.bias ? a.bias[d] : 0.0f, skip = ok && a.Dskip ? a.Dskip[d] : 0.0f;
#pragma unroll
  for (int i = 0; i < NS; ++i) A[i] = rate2(A[i]);
#pragma unroll
  for (int q = 0; q < SQ; ++q) {
    const float dt = a.softplus ? softplus(x[q] + bias) : x[q] + bias, dtu = dt * u[q];
    y[q] = 0.0f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      float Bv[4], Cv[4];
      Bq[q][i / 4].get(Bv);
      Cq[q][i / 4].get(Cv);
      h[q][i] = __builtin_amdgcn_exp2f(dt * A[i]) * h[q][i] + dtu * Bv[i % 4];
      y[q] += !VQ || n0 + i < a.N ? h[q][i] * Cv[i % 4] : 0.0f;
    }
    if (b0 + q < a.B) store_state<NS, VEC>(a.hT + ((long long)(b0 + q) * a.D + d) * a.N, a.N, n0, ok, h[q]);
  }
#pragma unroll
  for (int q = 0; q < SQ; ++q) {
    y[q] += __shfl_xor(y[q], 16, 64);
    y[q] += __shfl_xor(y[q], 32, 64);
    y[q] += skip * u[q];
    if (a.z) y[q] *= z[q] * sigmoid(z[q]);
    if (ok && row == q % 4 && b0 + q < a.B) store_elem(a.out, (long long)(b0 + q) * a.D + d, y[q], a.out_bf16);
  }
}

// ------------------------------------------------------------------ host side
int state_regs(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

struct ScanPlan {
  int cj, seg_len, nseg, subs, span, nspan, span_len;
  int bwd_waves, bwd_tiles;
  size_t seg, sdt, gseg, ck, ckdt, bcpart, dApart, dDpart, dbpart, total;
};

// The parts of a workspace for nseg segments of in all subs sub-tiles per sequence, in nspan spans.
void scan_layout(ScanPlan &p, int B, int L, int D, int N, int G, bool bwd, size_t nseg, size_t subs, size_t nspan) {
  size_t off = 0;
  auto take = [&off](size_t floats) {
    const size_t at = off;
    off += rec_align(floats * 4);
    return at;
  };
  const size_t DN = (size_t)D * N;
  p.seg = p.sdt = p.gseg = p.ck = p.ckdt = p.bcpart = p.dApart = p.dDpart = p.dbpart = 0;
  if (bwd || nseg > 1) {
    p.seg = take(B * nseg * DN);
    p.sdt = take(B * nseg * D);
  }
  if (bwd) {
    p.gseg = take(B * nseg * DN);
    p.ck = take(B * subs * DN);
    p.ckdt = take(B * subs * D);
    p.bcpart = take((size_t)p.bwd_tiles * B * L * G * 2 * N);
    p.dApart = take(B * nspan * DN);
    p.dDpart = take(B * nspan * D);
    p.dbpart = take(B * nspan * D);
  }
  p.total = off;
}

// How a call is cut.  Waves of 16 wide_cj channels share a token's LDS reads and sums
// among up to 16 elements per lane; waves of 16 channels are more.  The wide ones are taken
// where they still give three waves per SIMD: 24 sequences of 2048 tokens, D 2048, N 16
// (1536 wide waves) 581 us with them and 459 without, 32 of them 575 and 564, 48 801 and 813; in
// segments, one sequence of 1500 tokens 52 and 43.  A sequence is
// cut into segments only where its channels give less than a wave per SIMD (1024), since
// that computes every exponential twice, and from 257 tokens on, since it takes three
// launches.  Uncut and cut, us: 512 waves, N 16: L 100 22 and 29, L 333 50 and 52, L 777 107
// and 81, L 4096 527 and 256; 256 waves: L 100 24 and 30, L 333 48 and 34.
ScanPlan scan_plan(int B, int L, int D, int N, int G, bool bwd) {
  ScanPlan p;
  const int NS = state_regs(N), SUB = bwd_sub(NS), Dg = D / G;
  const int wide = wide_cj(NS);
  const long long groups = (long long)B * G, ww = groups * rec_cdiv(Dg, 16 * wide), w16 = groups * rec_cdiv(Dg, 16);
  // Segments of at least four tiles; of two, where many states make a tile long and there would be
  // less than two waves per SIMD (1000 tokens, D 512, N 64: 46 -> 35 us; N 16: 27 either way).
  const long long most = rec_cdiv(L, (NS >= 8 && w16 * rec_cdiv(L, 4 * TT) < 2 * SIMDS ? 2 : 4) * TT);
  if (bwd) {
    // The main pass, at two waves per SIMD, takes few long spans: each starts with loads that
    // nothing hides.  The checkpoints' pass, at four, cuts them further.
    const int cw = 16 * bwd_cj(NS);
    p.bwd_waves = (int)std::min<long long>(BWD_WAVES, rec_cdiv(Dg, cw));
    p.bwd_tiles = (int)rec_cdiv(Dg, (long long)cw * p.bwd_waves);
    const long long spans = std::min(rec_cdiv(2048, groups * p.bwd_tiles * p.bwd_waves), rec_cdiv(L, 2 * TT));
    p.span_len = (int)(rec_cdiv(rec_cdiv(L, spans), TT) * TT);
    p.nspan = (int)rec_cdiv(L, p.span_len);
    p.cj = ww * rec_cdiv(L, 2 * TT) >= 3 * SIMDS ? wide : 1;
    const long long cut = std::min<long long>(std::max<long long>(4096 / ((p.cj == 1 ? w16 : ww) * p.nspan), 1),
                                              rec_cdiv(p.span_len, 2 * TT));
    p.seg_len = (int)(rec_cdiv(rec_cdiv(p.span_len, cut), TT) * TT);
    p.span = (int)rec_cdiv(p.span_len, p.seg_len);
    p.nseg = p.nspan * p.span;
  } else {
    p.bwd_waves = p.bwd_tiles = 0;
    p.cj = ww >= 3 * SIMDS ? wide : 1;
    long long nseg = 1;
    if (w16 < SIMDS && L > 256) {
      p.cj = ww * most >= 3 * SIMDS ? wide : 1;
      nseg = std::min(most, rec_cdiv(8192, p.cj == 1 ? w16 : ww));
    }
    p.seg_len = p.span_len = (int)(rec_cdiv(rec_cdiv(L, nseg), TT) * TT);
    p.nseg = p.nspan = (int)rec_cdiv(L, p.seg_len);
    p.span = 1;
  }
  p.subs = p.seg_len / SUB;
  scan_layout(p, B, L, D, N, G, bwd, p.nseg, (size_t)p.nseg * p.subs, p.nspan);
  return p;
}

// Bytes that serve every call of at most L tokens: the plan's counts of segments and spans rise
// and fall with L, so each is replaced by a bound that only rises.
size_t scan_bytes(int B, int L, int D, int N, int G, bool bwd) {
  ScanPlan p;
  const int NS = state_regs(N), Dg = D / G, wide = wide_cj(NS);
  const long long groups = (long long)B * G, ww = groups * rec_cdiv(Dg, 16 * wide), w16 = groups * rec_cdiv(Dg, 16);
  if (!bwd) {
    if (w16 >= SIMDS || L <= 256) return 0;
    // the most segments by their length, of four tiles or (up to `fine` tokens) two; more of them
    // never turn wide waves narrow again
    const long long fine = NS >= 8 ? 4 * TT * ((2 * SIMDS - 1) / w16) : 0;
    const long long most = std::max(rec_cdiv(L, 4 * TT), rec_cdiv(std::min<long long>(L, fine), 2 * TT));
    scan_layout(p, B, L, D, N, G, false, std::min(most, rec_cdiv(8192, ww * most >= 3 * SIMDS ? ww : w16)), 0, 0);
    return p.total;
  }
  const int cw = 16 * bwd_cj(NS);
  p.bwd_waves = (int)std::min<long long>(BWD_WAVES, rec_cdiv(Dg, cw));
  p.bwd_tiles = (int)rec_cdiv(Dg, (long long)cw * p.bwd_waves);
  // In tiles.  s spans of n = ceil(tiles / s) cover at most tiles + min(n, s) - 1.  A span in c
  // segments adds at most min(ceil(n / c), c) - 1: over all spans no more than there are segments
  // (at most `cut`), and where c > 1 no more than half of what they cover.
  const long long tiles = rec_cdiv(L, TT), cap = rec_cdiv(2048, groups * p.bwd_tiles * p.bwd_waves);
  const long long spans = std::min(cap, rec_cdiv(tiles, 2));
  const long long cover = tiles + (rec_cdiv(tiles, 2) <= cap ? 1 : std::min(rec_cdiv(tiles, cap), cap));
  const long long cut = 4096 / (ww * rec_cdiv(L, 2 * TT) >= 3 * SIMDS ? ww : w16);
  const long long all = cover + std::min(cut, cover / 2);
  scan_layout(p, B, L, D, N, G, true, std::min(std::max(cut, spans), std::max(all / 2, 1LL)),
              (size_t)all * (TT / bwd_sub(NS)), spans);
  return p.total;
}

// Sizes a call takes, the header's limits.  They keep every grid below 2^32 threads: 64
// times the waves, 256 times the workgroups of a single token, a thread a state.
bool plan_ok(int B, int L, int D, int N, int G) {
  return B > 0 && L > 0 && D > 0 && N > 0 && G > 0 && D % G == 0 && N <= RECURRENT_MAX_STATE &&
         D <= RECURRENT_MAX_CHANNELS && (long long)B * L <= RECURRENT_MAX_TOKENS &&
         (double)B * L * D <= RECURRENT_MAX_ELEMENTS && (double)B * L * G * N <= RECURRENT_MAX_ELEMENTS &&
         (double)B * D * N <= RECURRENT_MAX_STATES && (double)B * G * rec_cdiv(D / G, 16) < 1 << 24;
}

ret_status_t check_sizes(int B, int L, int D, int N, int G, ret_dtype_t in_dtype, ret_dtype_t out_dtype) {
  if (B <= 0 || L < 0 || D <= 0 || N <= 0 || G <= 0)
    return rec_fail(RET_ERR_INVALID_ARG, "sizes must be positive (B=%d L=%d D=%d N=%d G=%d)", B, L, D, N, G);
  if (D % G) return rec_fail(RET_ERR_INVALID_ARG, "D=%d is not a multiple of G=%d", D, G);
  if (!rec_dtype_ok(in_dtype) || !rec_dtype_ok(out_dtype)) return rec_fail(RET_ERR_INVALID_ARG, "unknown dtype");
  if (N > RECURRENT_MAX_STATE) return rec_fail(RET_ERR_UNSUPPORTED, "N=%d above %d", N, RECURRENT_MAX_STATE);
  if (!plan_ok(B, std::max(L, 1), D, N, G))
    return rec_fail(RET_ERR_UNSUPPORTED, "too many tokens (B=%d L=%d D=%d)", B, L, D);
  return RET_OK;
}

// Rows of four channels that may be read at once: every row of p starts at a multiple
// of four elements, aligned to them.
bool wide(const void *p, long long ld, size_t e) { return !p || (ld % 4 == 0 && rec_aligned(p, 4 * e)); }

template <typename K>
hipError_t launch(K kernel, long long blocks, int threads, hipStream_t st, const ScanArgs &a, size_t lds = 0) {
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), lds, st, a);
  return hipGetLastError();
}

// Where rows or states cannot be accessed by fours, one kernel per type and NS will do:
// the narrow one.
template <typename T, int NS, int CJ, int MODE, bool VEC>
hipError_t launch_pass_kernel(ScanArgs a, hipStream_t st) {
  a.tiles = (int)rec_cdiv(a.Dg, 16 * CJ);
  // the waves do not meet: workgroups of four spread them evenly over the SIMDs, of one over the
  // CUs (each with the LDS of its waves: with that of four, three fitted a CU at N 64, and
  // 1024 waves took two turns, 2885 us instead of 1080 for 4096 tokens)
  const long long waves = (long long)a.B * a.nseg * a.G * a.tiles;
  a.waves = (int)waves;
  const int per = waves > SIMDS ? PASS_WAVES : 1;
  return launch(scan_pass_kernel<T, NS, CJ, MODE, VEC>, rec_cdiv(waves, per), 64 * per, st, a,
                per * sizeof(PassLds<NS, CJ, MODE>));
}
template <typename T, int NS, int MODE>
hipError_t launch_pass(const ScanArgs &a, int cj, hipStream_t st) {
  if (!a.vec) return launch_pass_kernel<T, NS, 1, MODE, false>(a, st);
  return cj == 1 ? launch_pass_kernel<T, NS, 1, MODE, true>(a, st)
                 : launch_pass_kernel<T, NS, wide_cj(NS), MODE, true>(a, st);
}
template <typename T, int MODE>
hipError_t launch_pass(const ScanArgs &a, int cj, hipStream_t st) {
  switch (state_regs(a.N)) {
    case 1: return launch_pass<T, 1, MODE>(a, cj, st);
    case 2: return launch_pass<T, 2, MODE>(a, cj, st);
    case 4: return launch_pass<T, 4, MODE>(a, cj, st);
    case 8: return launch_pass<T, 8, MODE>(a, cj, st);
    default: return launch_pass<T, 16, MODE>(a, cj, st);
  }
}
template <int MODE>
hipError_t launch_pass(const ScanArgs &a, bool bf, int cj, hipStream_t st) {
  return bf ? launch_pass<uint16_t, MODE>(a, cj, st) : launch_pass<float, MODE>(a, cj, st);
}

template <typename T, bool VEC>
hipError_t launch_bwd(ScanArgs a, const ScanPlan &p, hipStream_t st) {
  a.tiles = p.bwd_tiles;
  const long long blocks = (long long)a.B * a.nspan * a.G * a.tiles;
  const int threads = 64 * p.bwd_waves;
  switch (state_regs(a.N)) {
    case 1: return launch(scan_bwd_kernel<T, 1, VEC>, blocks, threads, st, a);
    case 2: return launch(scan_bwd_kernel<T, 2, VEC>, blocks, threads, st, a);
    case 4: return launch(scan_bwd_kernel<T, 4, VEC>, blocks, threads, st, a);
    case 8: return launch(scan_bwd_kernel<T, 8, VEC>, blocks, threads, st, a);
    default: return launch(scan_bwd_kernel<T, 16, VEC>, blocks, threads, st, a);
  }
}
template <typename T>
hipError_t launch_bwd(const ScanArgs &a, const ScanPlan &p, hipStream_t st) {
  return a.vec ? launch_bwd<T, true>(a, p, st) : launch_bwd<T, false>(a, p, st);
}

template <typename T, int SQ, bool VEC>
hipError_t launch_step(ScanArgs a, hipStream_t st) {
  a.tiles = (int)rec_cdiv(a.Dg, STEP_CH);
  const long long blocks = rec_cdiv(a.B, SQ) * a.G * a.tiles;
  switch (state_regs(a.N)) {
    case 1: return launch(scan_step_kernel<T, 1, SQ, VEC>, blocks, NT, st, a);
    case 2: return launch(scan_step_kernel<T, 2, SQ, VEC>, blocks, NT, st, a);
    case 4: return launch(scan_step_kernel<T, 4, SQ, VEC>, blocks, NT, st, a);
    case 8: return launch(scan_step_kernel<T, 8, SQ, VEC>, blocks, NT, st, a);
    default: return launch(scan_step_kernel<T, 16, SQ, VEC>, blocks, NT, st, a);
  }
}
// Four sequences a workgroup where that still leaves four workgroups a CU.
template <typename T>
hipError_t launch_step(const ScanArgs &a, hipStream_t st) {
  const bool many = (long long)a.B * a.G * rec_cdiv(a.Dg, STEP_CH) >= 4096;
  if (!a.vec) return launch_step<T, 1, false>(a, st);
  return many ? launch_step<T, 4, true>(a, st) : launch_step<T, 1, true>(a, st);
}

hipError_t launch_combine(const ScanArgs &a, hipStream_t st) {
  const dim3 grid((unsigned)rec_cdiv((long long)a.B * a.D * a.N, NT), a.gseg ? 2 : 1);
  hipLaunchKernelGGL(scan_combine_kernel, grid, dim3(NT), 0, st, a);
  return hipGetLastError();
}

ScanArgs scan_args(const void *u, const void *delta, const float *A, const void *Bm, const void *Cm,
                   const float *D_skip, const void *z, const float *bias, const int *lengths, int B, int L, int D,
                   int N, int G, long long u_ld, long long delta_ld, long long z_ld, long long b_ld, long long c_ld,
                   int softplus, ret_dtype_t in_dtype, ret_dtype_t out_dtype) {
  ScanArgs a = {};
  a.u = u;
  a.delta = delta;
  a.A = A;
  a.Bm = Bm;
  a.Cm = Cm;
  a.Dskip = D_skip;
  a.z = z;
  a.bias = bias;
  a.lengths = lengths;
  a.u_ld = u_ld;
  a.delta_ld = delta_ld;
  a.z_ld = z_ld;
  a.b_ld = b_ld;
  a.c_ld = c_ld;
  a.B = B;
  a.L = L;
  a.D = D;
  a.N = N;
  a.G = G;
  a.Dg = D / G;
  a.softplus = softplus != 0;
  a.out_bf16 = out_dtype == RET_BF16;
  const size_t e = rec_esize(in_dtype);
  a.vec = a.Dg % 4 == 0 && N % 4 == 0 && wide(u, u_ld, e) && wide(delta, delta_ld, e) && wide(z, z_ld, e) &&
          wide(Bm, b_ld, e) && wide(Cm, c_ld, e) && wide(D_skip, 0, 4) && wide(bias, 0, 4);
  return a;
}

// Whether states are aligned for access by fours: the caller's, A, and the workspace's.
bool wide_states(const ScanArgs &a) {
  const void *ps[] = {a.A, a.h0, a.hT, a.dhT, a.dh0, a.seg};
  for (const void *p : ps)
    if (!rec_aligned(p, 16)) return false;
  return true;
}

// Pointers, strides and alignment of the inputs that all three calls share.
ret_status_t check_inputs(const ScanArgs &a, size_t e) {
  if (!a.u || !a.delta || !a.A || !a.Bm || !a.Cm) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  const long long bc = (long long)a.G * a.N;
  if (a.u_ld < a.D || a.delta_ld < a.D || (a.z && a.z_ld < a.D) || a.b_ld < bc || a.c_ld < bc)
    return rec_fail(RET_ERR_INVALID_ARG, "a row stride is shorter than its row");
  const long long most = 1LL << 31;
  if (a.u_ld > most || a.delta_ld > most || (a.z && a.z_ld > most) || a.b_ld > most || a.c_ld > most)
    return rec_fail(RET_ERR_UNSUPPORTED, "a row stride above 2^31");
  const void *es[] = {a.u, a.delta, a.Bm, a.Cm, a.z, a.d_o};
  for (const void *p : es)
    if (!rec_aligned(p, e)) return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const void *fs[] = {a.A, a.Dskip, a.bias, a.h0, a.dhT, a.hT, a.dh0, a.lengths};
  for (const void *p : fs)
    if (!rec_aligned(p, 4)) return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  return RET_OK;
}

}  // namespace

extern "C" {

size_t selective_scan_workspace_bytes(int B, int L, int D, int N, int G) {
  return plan_ok(B, L, D, N, G) ? scan_bytes(B, L, D, N, G, false) : 0;
}

size_t selective_scan_bwd_workspace_bytes(int B, int L, int D, int N, int G) {
  return plan_ok(B, L, D, N, G) ? scan_bytes(B, L, D, N, G, true) : 0;
}

ret_status_t selective_scan(const void *u, const void *delta, const float *A, const void *Bm, const void *Cm,
                            const float *D_skip, const void *z, const float *delta_bias, void *out,
                            const int *lengths, const float *state_in, float *state_out, int B, int L, int D, int N,
                            int G, long long u_ld, long long delta_ld, long long z_ld, long long b_ld, long long c_ld,
                            int delta_softplus, ret_dtype_t in_dtype, ret_dtype_t out_dtype, void *workspace,
                            size_t workspace_bytes, void *hip_stream) {
  ret_status_t s = check_sizes(B, L, D, N, G, in_dtype, out_dtype);
  if (s != RET_OK) return s;
  const size_t e = rec_esize(in_dtype), oe = rec_esize(out_dtype), ns = (size_t)B * D * N * 4;
  const long long rows = (long long)B * L;
  ScanArgs a = scan_args(u, delta, A, Bm, Cm, D_skip, z, delta_bias, lengths, B, L, D, N, G, u_ld, delta_ld, z_ld, b_ld,
                         c_ld, delta_softplus, in_dtype, out_dtype);
  a.h0 = state_in;
  a.hT = state_out;
  a.out = out;
  hipStream_t st = (hipStream_t)hip_stream;
  const RecSpan hi = {"state_in", state_in, state_in ? ns : 0}, ho = {"state_out", state_out, state_out ? ns : 0};
  if (state_in != state_out && rec_overlap(hi, ho))
    return rec_fail(RET_ERR_INVALID_ARG, "state_out partially overlaps state_in");
  if (L == 0) {
    if (!rec_aligned(state_in, 4) || !rec_aligned(state_out, 4))
      return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
    return rec_status(state_copy(state_out, state_in, (long long)B * D * N, st));
  }
  if ((s = check_inputs(a, e)) != RET_OK) return s;
  if (!out) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!rec_aligned(out, oe)) return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const ScanPlan p = scan_plan(B, L, D, N, G, false);
  if (p.total && (!workspace || workspace_bytes < p.total))
    return rec_fail(RET_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", p.total, workspace_bytes);
  if (!rec_aligned(workspace, 16)) return rec_fail(RET_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  const RecSpan ins[] = {rec_rows("u", u, rows, u_ld, D, e), rec_rows("delta", delta, rows, delta_ld, D, e),
                         rec_rows("z", z, rows, z_ld, D, e), rec_rows("Bm", Bm, rows, b_ld, (long long)G * N, e),
                         rec_rows("Cm", Cm, rows, c_ld, (long long)G * N, e), {"A", A, (size_t)D * N * 4},
                         {"D_skip", D_skip, (size_t)D * 4}, {"delta_bias", delta_bias, (size_t)D * 4},
                         {"lengths", lengths, (size_t)B * 4}};
  const RecSpan outs[] = {{"out", out, (size_t)rows * D * oe}, ho, {"the workspace", workspace, p.total}};
  if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
  const RecSpan hin[] = {hi}, others[] = {outs[0], outs[2]};
  if ((s = rec_check_overlap(hin, others)) != RET_OK) return s;
  a.seg_len = a.span_len = p.seg_len;
  a.nseg = p.nseg;
  a.span = 1;
  a.seg = (float *)((char *)workspace + p.seg);
  a.sdt = (float *)((char *)workspace + p.sdt);
  const bool bf = in_dtype == RET_BF16;
  a.vec = a.vec && wide(out, D, oe) && wide_states(a);
  hipError_t err = hipSuccess;
  if (p.nseg > 1) {
    if ((err = launch_pass<STATES>(a, bf, p.cj, st)) != hipSuccess || (err = launch_combine(a, st)) != hipSuccess)
      return rec_status(err);
  }
  return rec_status(launch_pass<OUTPUT>(a, bf, p.cj, st));
}

ret_status_t selective_scan_bwd(const void *u, const void *delta, const float *A, const void *Bm, const void *Cm,
                                const float *D_skip, const void *z, const float *delta_bias, const void *d_o,
                                const int *lengths, const float *state_in, const float *d_state_out, void *du,
                                void *ddelta, float *dA, void *dB, void *dC, float *dD, void *dz, float *ddelta_bias,
                                float *d_state_in, int B, int L, int D, int N, int G, long long u_ld,
                                long long delta_ld, long long z_ld, long long b_ld, long long c_ld,
                                int delta_softplus, ret_dtype_t in_dtype, ret_dtype_t out_dtype, void *workspace,
                                size_t workspace_bytes, void *hip_stream) {
  ret_status_t s = check_sizes(B, L, D, N, G, in_dtype, out_dtype);
  if (s != RET_OK) return s;
  const size_t e = rec_esize(in_dtype), oe = rec_esize(out_dtype), ns = (size_t)B * D * N * 4;
  const long long rows = (long long)B * L, bc = (long long)G * N;
  hipStream_t st = (hipStream_t)hip_stream;
  ScanArgs a = scan_args(u, delta, A, Bm, Cm, D_skip, z, delta_bias, lengths, B, L, D, N, G, u_ld, delta_ld, z_ld, b_ld,
                         c_ld, delta_softplus, in_dtype, out_dtype);
  a.h0 = state_in;
  a.dhT = d_state_out;
  a.d_o = d_o;
  a.du = du;
  a.ddelta = ddelta;
  a.dz = dz;
  a.dh0 = d_state_in;
  if (!dA) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  const void *fs[] = {dA, dD, ddelta_bias, d_state_in, d_state_out};
  for (const void *q : fs)
    if (!rec_aligned(q, 4)) return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  ScanPlan p = {};
  if (L > 0) p = scan_plan(B, L, D, N, G, true);
  const RecSpan dho = {"d_state_out", d_state_out, d_state_out ? ns : 0};
  const RecSpan outs[] = {{"du", du, (size_t)rows * D * oe}, {"ddelta", ddelta, (size_t)rows * D * oe},
                          {"dA", dA, (size_t)D * N * 4}, {"dB", dB, (size_t)rows * bc * oe},
                          {"dC", dC, (size_t)rows * bc * oe}, {"dD", dD, (size_t)D * 4},
                          {"dz", dz, (size_t)rows * D * oe}, {"ddelta_bias", ddelta_bias, (size_t)D * 4},
                          {"d_state_in", d_state_in, d_state_in ? ns : 0},
                          {"the workspace", workspace, p.total}};
  const RecSpan ins[] = {rec_rows("u", u, rows, u_ld, D, e), rec_rows("delta", delta, rows, delta_ld, D, e),
                         rec_rows("z", z, rows, z_ld, D, e), rec_rows("Bm", Bm, rows, b_ld, bc, e),
                         rec_rows("Cm", Cm, rows, c_ld, bc, e), {"A", A, (size_t)D * N * 4},
                         {"D_skip", D_skip, (size_t)D * 4}, {"delta_bias", delta_bias, (size_t)D * 4},
                         {"d_o", d_o, (size_t)rows * D * e}, {"state_in", state_in, ns}, dho,
                         {"lengths", lengths, (size_t)B * 4}};
  if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
  if (L == 0) {  // the state passes through; sums over no tokens
    hipError_t err;
    if ((err = state_copy(dA, nullptr, (long long)D * N, st)) != hipSuccess ||
        (err = state_copy(dD, nullptr, D, st)) != hipSuccess ||
        (err = state_copy(ddelta_bias, nullptr, D, st)) != hipSuccess)
      return rec_status(err);
    return rec_status(state_copy(d_state_in, d_state_out, (long long)B * D * N, st));
  }
  if ((s = check_inputs(a, e)) != RET_OK) return s;
  if (!d_o || !du || !ddelta || !dB || !dC) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!dz != !z) return rec_fail(RET_ERR_INVALID_ARG, "dz and z come together");
  const void *os[] = {du, ddelta, dB, dC, dz};
  for (const void *q : os)
    if (!rec_aligned(q, oe)) return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  if (!workspace || workspace_bytes < p.total)
    return rec_fail(RET_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", p.total, workspace_bytes);
  if (!rec_aligned(workspace, 16)) return rec_fail(RET_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  char *ws = (char *)workspace;
  a.seg_len = p.seg_len;
  a.nseg = p.nseg;
  a.subs = p.subs;
  a.span = p.span;
  a.nspan = p.nspan;
  a.span_len = p.span_len;
  a.seg = (float *)(ws + p.seg);
  a.sdt = (float *)(ws + p.sdt);
  a.gseg = (float *)(ws + p.gseg);
  a.ck = (float *)(ws + p.ck);
  a.ckdt = (float *)(ws + p.ckdt);
  a.bcpart = (float *)(ws + p.bcpart);
  a.dApart = (float *)(ws + p.dApart);
  a.dDpart = (float *)(ws + p.dDpart);
  a.dbpart = (float *)(ws + p.dbpart);
  const bool bf = in_dtype == RET_BF16;
  a.vec = a.vec && wide(d_o, D, e) && wide(du, D, oe) && wide(ddelta, D, oe) && wide(dz, D, oe) && wide_states(a);
  hipError_t err;
  if ((err = launch_pass<CHECKPOINTS>(a, bf, p.cj, st)) != hipSuccess || (err = launch_combine(a, st)) != hipSuccess ||
      (err = bf ? launch_bwd<uint16_t>(a, p, st) : launch_bwd<float>(a, p, st)) != hipSuccess)
    return rec_status(err);
  // grids of at most 2^20 workgroups, which walk what is more
  if (lengths && (err = launch(scan_bwd_tail_kernel, std::min(rows, 1LL << 20), NT, st, a)) != hipSuccess)
    return rec_status(err);
  a.tiles = p.bwd_tiles;
  const long long bc_blocks = std::min(rec_cdiv(rows * 2 * bc, COLS * ROWS), 1LL << 20);
  const long long cols = (long long)D * (N + 2);
  hipLaunchKernelGGL(scan_reduce_kernel, dim3((unsigned)(bc_blocks + rec_cdiv(cols, COLS))), dim3(COLS * ROWS), 0, st, a,
                     dB, dC, dA, dD, ddelta_bias, bc_blocks);
  if ((err = hipGetLastError()) != hipSuccess) return rec_status(err);
  return rec_status(hipSuccess);
}

ret_status_t selective_scan_step(const void *u, const void *delta, const float *A, const void *Bm, const void *Cm,
                                 const float *D_skip, const void *z, const float *delta_bias, void *out, float *state,
                                 int B, int D, int N, int G, long long u_ld, long long delta_ld, long long z_ld,
                                 long long b_ld, long long c_ld, int delta_softplus, ret_dtype_t in_dtype,
                                 ret_dtype_t out_dtype, void *hip_stream) {
  ret_status_t s = check_sizes(B, 1, D, N, G, in_dtype, out_dtype);
  if (s != RET_OK) return s;
  const size_t e = rec_esize(in_dtype), oe = rec_esize(out_dtype);
  ScanArgs a = scan_args(u, delta, A, Bm, Cm, D_skip, z, delta_bias, nullptr, B, 1, D, N, G, u_ld, delta_ld, z_ld, b_ld,
                         c_ld, delta_softplus, in_dtype, out_dtype);
  a.out = out;
  a.hT = state;
  if ((s = check_inputs(a, e)) != RET_OK) return s;
  if (!out || !state) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!rec_aligned(out, oe)) return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const long long bc = (long long)G * N;
  const RecSpan ins[] = {rec_rows("u", u, B, u_ld, D, e), rec_rows("delta", delta, B, delta_ld, D, e),
                         rec_rows("z", z, B, z_ld, D, e), rec_rows("Bm", Bm, B, b_ld, bc, e),
                         rec_rows("Cm", Cm, B, c_ld, bc, e), {"A", A, (size_t)D * N * 4},
                         {"D_skip", D_skip, (size_t)D * 4}, {"delta_bias", delta_bias, (size_t)D * 4}};
  const RecSpan outs[] = {{"out", out, (size_t)B * D * oe}, {"state", state, (size_t)B * D * N * 4}};
  if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
  a.vec = a.vec && wide_states(a);
  hipStream_t st = (hipStream_t)hip_stream;
  return rec_status(in_dtype == RET_BF16 ? launch_step<uint16_t>(a, st) : launch_step<float>(a, st));
}

}  // extern "C"
