// Selective state space scan (recurrent.h): h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t,
// y_t = C_t . h_t + D u_t, gated by silu(z_t); its gradients; its single-token form.
//
// Layout of every kernel here: a workgroup of four waves covers 64 channels of one
// group (of B and C) of one sequence; a wave covers 16 channels, lane & 15, and its four
// rows of 16 lanes (lane >> 4) hold NS of the states each, N <= 4 NS.  Sums over a
// channel's states are NS terms in registers and two steps across the rows; the
// recurrence itself never leaves a lane.  Tokens are staged in tiles of 16: thread
// (token, four channels) computes the time step, u dt and the gated gradient once, in
// fp32, into LDS, from where all four rows read them.
//
// Long sequences are cut into segments, so that few channels still fill the chip: the
// decay of a state over a segment is exp(A sum dt), so the states entering the
// segments follow from each segment's own final state and its sum of time steps
// (states pass, combination), and the output pass runs all segments at once.
#include <algorithm>

#include "recurrent.hpp"

using namespace ret;

namespace {

constexpr int CH = 64;  // channels per workgroup
constexpr int TT = 16;  // tokens per staged tile
constexpr int NT = 256;

struct ScanArgs {
  const void *u, *delta, *Bm, *Cm, *z, *d_o;
  const float *A, *Dskip, *bias, *h0, *dhT;
  const int *lengths;
  void *out;
  float *hT;
  long long u_ld, delta_ld, z_ld, b_ld, c_ld;
  int B, L, D, N, G, Dg, tiles;  // Dg = D / G channels per group, tiles of 64 of them
  int seg_len, nseg, softplus, out_bf16;
  // workspace: segment states [B * nseg][D][N], sums of dt [B * nseg][D]
  float *seg, *sdt;
  // backward
  void *du, *ddelta, *dz;
  float *gseg;        // gradients entering the segments from behind, [B * nseg][D][N]
  float *ck, *ckdt;   // per sub-tile: state relative to the segment, sum of dt before it
  float *bcpart;      // [tiles][B * L][G][2][N]
  float *dApart, *dDpart, *dbpart;  // [B * nseg][D][N], [B * nseg][D]
  float *dh0;
  int subs;           // sub-tiles per segment
};

// What a block works on.
struct Where {
  int b, s, g, tile, len, t_lo, t_hi;
};
__device__ __forceinline__ Where where(const ScanArgs &a) {
  Where w;
  int id = blockIdx.x;
  w.tile = id % a.tiles;
  id /= a.tiles;
  w.g = id % a.G;
  id /= a.G;
  w.s = id % a.nseg;
  w.b = id / a.nseg;
  w.len = a.lengths ? min(max(a.lengths[w.b], 0), a.L) : a.L;
  w.t_lo = min(w.s * a.seg_len, w.len);
  w.t_hi = min(w.t_lo + a.seg_len, w.len);
  return w;
}

// The sum over the four rows of a wave, for four tokens at once: lane row r gets token r.
__device__ __forceinline__ float row_sums(const float (&y)[4], int row) {
  float s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    s[j] = y[j] + __shfl_xor(y[j], 16, 64);
    s[j] += __shfl_xor(s[j], 32, 64);
  }
  return row == 0 ? s[0] : row == 1 ? s[1] : row == 2 ? s[2] : s[3];
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

template <int NS>
__device__ __forceinline__ void load_state(const float *p, int N, int n0, bool ok, float (&h)[NS]) {
#pragma unroll
  for (int i = 0; i < NS; ++i) h[i] = ok && n0 + i < N ? p[n0 + i] : 0.0f;
}
template <int NS>
__device__ __forceinline__ void store_state(float *p, int N, int n0, bool ok, const float (&h)[NS]) {
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (ok && n0 + i < N) p[n0 + i] = h[i];
}

// B or C of the tile's tokens t0.. into dst[16][4 NS], zero behind N and behind t_hi.
template <typename T, int NS>
__device__ __forceinline__ void stage_bc(const void *src, long long ld, const ScanArgs &a, const Where &w, int t0,
                                         float (*dst)[4 * NS]) {
  for (int e = threadIdx.x; e < TT * 4 * NS; e += NT) {
    const int tt = e / (4 * NS), n = e % (4 * NS);
    float x = 0.0f;
    if (n < a.N && t0 + tt < w.t_hi)
      x = load_elem(src, ((long long)w.b * a.L + t0 + tt) * ld + (long long)w.g * a.N + n, sizeof(T) == 2);
    dst[tt][n] = x;
  }
}

enum { OUTPUT, STATES, CHECKPOINTS };

// One pass over a segment.
//   OUTPUT: from the state entering the segment, the gated outputs; the last segment
//     writes the final state.
//   STATES: from zero, the segment's own final state and its sum of dt.
//   CHECKPOINTS (backward): as STATES, also the state and the sum of dt before every
//     SUB tokens, and the gradient that the segment's own outputs send to the state in
//     front of it, sum_t exp(A sum dt) C_t dy_t.
template <typename T, int NS, bool VEC, int MODE>
__global__ __launch_bounds__(NT) void scan_pass_kernel(ScanArgs a) {
  constexpr int NP = 4 * NS, SUB = NS <= 4 ? 16 : 64 / NS;
  __shared__ float2 dtx[TT][CH];  // (dt, dt u)
  __shared__ float Bs[TT][NP];
  __shared__ float Cs[MODE == STATES ? 1 : TT][NP];
  __shared__ float ys[MODE == STATES ? 1 : TT][CH];  // OUTPUT: y; CHECKPOINTS: dy
  const Where w = where(a);
  const bool last = w.s == a.nseg - 1;
  const int tid = threadIdx.x, lane = tid & 63, row = lane >> 4, ch = (tid >> 6) * 16 + (lane & 15);
  const int rel = w.tile * CH + ch, n0 = row * NS;
  const bool ok = rel < a.Dg;
  const long long d = (long long)w.g * a.Dg + rel;
  const long long sd = ((long long)w.b * a.nseg + w.s) * a.D + d;
  float A2[NS], h[NS], gs[NS], pr[NS], sum = 0.0f;
  load_state(a.A + d * a.N, a.N, n0, ok, A2);
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    A2[i] *= kLog2e;
    h[i] = 0.0f;
    gs[i] = 0.0f;
    pr[i] = 1.0f;
  }
  if constexpr (MODE == OUTPUT) {
    if (a.nseg > 1)
      load_state(a.seg + sd * a.N, a.N, n0, ok, h);
    else if (a.h0)
      load_state(a.h0 + sd * a.N, a.N, n0, ok, h);
  }
  // the thread's part of the staging: one token, four channels
  const int tt = tid >> 4, cq = (tid & 15) * 4, relq = w.tile * CH + cq;
  const int nc = min(max(a.Dg - relq, 0), 4);
  const long long dq = (long long)w.g * a.Dg + relq;
  float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f}, Dsk[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (c < nc) {
      if (a.bias) bias[c] = a.bias[dq + c];
      if (a.Dskip) Dsk[c] = a.Dskip[dq + c];
    }
  for (int t0 = w.t_lo; t0 < w.t_hi; t0 += TT) {
    const long long r = (long long)w.b * a.L + t0 + tt;
    const bool live = t0 + tt < w.t_hi && nc > 0;
    float u[4] = {0.0f, 0.0f, 0.0f, 0.0f}, z[4] = {0.0f, 0.0f, 0.0f, 0.0f}, x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (live) {
      load4<T, VEC>((const T *)a.u + r * a.u_ld + dq, nc, u);
      load4<T, VEC>((const T *)a.delta + r * a.delta_ld + dq, nc, x);
      if (MODE != STATES && a.z) load4<T, VEC>((const T *)a.z + r * a.z_ld + dq, nc, z);
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float v = x[c] + bias[c], dt = !live || c >= nc ? 0.0f : a.softplus ? softplus(v) : v;
      dtx[tt][cq + c] = make_float2(dt, live && c < nc ? dt * u[c] : 0.0f);
    }
    stage_bc<T, NS>(a.Bm, a.b_ld, a, w, t0, Bs);
    if constexpr (MODE != STATES) stage_bc<T, NS>(a.Cm, a.c_ld, a, w, t0, Cs);
    if constexpr (MODE == CHECKPOINTS) {
      float g[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (live) load4<T, VEC>((const T *)a.d_o + r * a.D + dq, nc, g);
#pragma unroll
      for (int c = 0; c < 4; ++c) ys[tt][cq + c] = a.z ? g[c] * z[c] * sigmoid(z[c]) : g[c];
    }
    __syncthreads();
    const int nt = min(TT, w.t_hi - t0);
    for (int t4 = 0; t4 < nt; t4 += 4) {
      if constexpr (MODE == CHECKPOINTS) {
        if (t4 % SUB == 0) {
          const long long k = ((long long)w.b * a.nseg + w.s) * a.subs + (t0 - w.t_lo + t4) / SUB;
          store_state(a.ck + (k * a.D + d) * a.N, a.N, n0, ok, h);
          if (ok && row == 0) a.ckdt[k * a.D + d] = sum;
        }
      }
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = dtx[t4 + j][ch];
        float acc = 0.0f;
        const float dy = MODE == CHECKPOINTS ? ys[t4 + j][ch] : 0.0f;
        if constexpr (MODE != OUTPUT) sum += v.x;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const float e = __builtin_amdgcn_exp2f(v.x * A2[i]);
          h[i] = e * h[i] + v.y * Bs[t4 + j][n0 + i];
          if constexpr (MODE == OUTPUT) acc += h[i] * Cs[t4 + j][n0 + i];
          if constexpr (MODE == CHECKPOINTS) {
            pr[i] *= e;
            gs[i] += pr[i] * (dy * Cs[t4 + j][n0 + i]);
          }
        }
        y[j] = acc;
      }
      if constexpr (MODE == OUTPUT) {
        const float v = row_sums(y, row);
        ys[t4 + row][ch] = v;
      }
    }
    if constexpr (MODE == OUTPUT) {
      __syncthreads();
      if (live) {
        float o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          o[c] = ys[tt][cq + c] + Dsk[c] * u[c];
          if (a.z) o[c] *= z[c] * sigmoid(z[c]);
        }
        store4<VEC>(a.out, r * a.D + dq, nc, o, a.out_bf16);
      }
    }
  }
  if constexpr (MODE == OUTPUT) {
    if (last && a.hT) store_state(a.hT + ((long long)w.b * a.D + d) * a.N, a.N, n0, ok, h);
  } else {
    store_state(a.seg + sd * a.N, a.N, n0, ok, h);
    if (ok && row == 0) a.sdt[sd] = sum;
    if constexpr (MODE == CHECKPOINTS) store_state(a.gseg + sd * a.N, a.N, n0, ok, gs);
  }
}

// Segment states -> states entering the segments, in place; with gseg also the
// gradients entering them from behind.  One thread per (sequence, channel, state).
__global__ __launch_bounds__(NT) void scan_combine_kernel(ScanArgs a) {
  const long long DN = (long long)a.D * a.N, id = (long long)blockIdx.x * NT + threadIdx.x;
  if (id >= a.B * DN) return;
  const long long b = id / DN, e = id % DN, d = e / a.N;
  const float A2 = a.A[e] * kLog2e;
  float carry = a.h0 ? a.h0[id] : 0.0f;
  float *S = a.seg + b * a.nseg * DN + e;
  const float *sdt = a.sdt + b * a.nseg * a.D + d;
  for (int s = 0; s < a.nseg; ++s) {
    const float own = S[s * DN];
    S[s * DN] = carry;
    carry = __builtin_amdgcn_exp2f(A2 * sdt[(long long)s * a.D]) * carry + own;
  }
  if (!a.gseg) return;
  float *Gs = a.gseg + b * a.nseg * DN + e;
  carry = a.dhT ? a.dhT[id] : 0.0f;
  for (int s = a.nseg - 1; s >= 0; --s) {
    const float own = Gs[s * DN];
    Gs[s * DN] = carry;
    carry = __builtin_amdgcn_exp2f(A2 * sdt[(long long)s * a.D]) * carry + own;
  }
}

// The backward's main pass over a segment, tiles and sub-tiles from the last to the
// first: each sub-tile's states are computed again from its checkpoint and kept in
// registers with their decays; then the gradient of the state runs against time.
template <typename T, int NS, bool VEC>
__global__ __launch_bounds__(NT) void scan_bwd_kernel(ScanArgs a) {
  constexpr int NP = 4 * NS, SUB = NS <= 4 ? 16 : 64 / NS;
  __shared__ float2 dtx[TT][CH];       // (dt, dt u), then (sum g B, sum A w)
  __shared__ float dys[TT][CH];        // dy, then C . h
  __shared__ float Bs[TT][NP], Cs[TT][NP];
  __shared__ float part[4][TT][2][NP];  // each wave's sums over its channels
  const Where w = where(a);
  const int tid = threadIdx.x, lane = tid & 63, row = lane >> 4, wave = tid >> 6, ch = wave * 16 + (lane & 15);
  const int rel = w.tile * CH + ch, n0 = row * NS;
  const bool ok = rel < a.Dg;
  const long long d = (long long)w.g * a.Dg + rel;
  const long long bs = (long long)w.b * a.nseg + w.s, sd = bs * a.D + d;
  float A1[NS], hin[NS], carry[NS], dA[NS];
  load_state(a.A + d * a.N, a.N, n0, ok, A1);
  load_state(a.seg + sd * a.N, a.N, n0, ok, hin);
  load_state(a.gseg + sd * a.N, a.N, n0, ok, carry);
#pragma unroll
  for (int i = 0; i < NS; ++i) dA[i] = 0.0f;
  const int tt = tid >> 4, cq = (tid & 15) * 4, relq = w.tile * CH + cq;
  const int nc = min(max(a.Dg - relq, 0), 4);
  const long long dq = (long long)w.g * a.Dg + relq;
  float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f}, Dsk[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  float sD[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sb[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (c < nc) {
      if (a.bias) bias[c] = a.bias[dq + c];
      if (a.Dskip) Dsk[c] = a.Dskip[dq + c];
    }
  const int ntile = (w.t_hi - w.t_lo + TT - 1) / TT;
  for (int tile = ntile - 1; tile >= 0; --tile) {
    const int t0 = w.t_lo + tile * TT;
    const long long r = (long long)w.b * a.L + t0 + tt;
    const bool live = t0 + tt < w.t_hi && nc > 0;
    float u[4] = {0.0f, 0.0f, 0.0f, 0.0f}, z[4] = {0.0f, 0.0f, 0.0f, 0.0f}, x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float go[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dt[4], dy[4];
    if (live) {
      load4<T, VEC>((const T *)a.u + r * a.u_ld + dq, nc, u);
      load4<T, VEC>((const T *)a.delta + r * a.delta_ld + dq, nc, x);
      load4<T, VEC>((const T *)a.d_o + r * a.D + dq, nc, go);
      if (a.z) load4<T, VEC>((const T *)a.z + r * a.z_ld + dq, nc, z);
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[c] += bias[c];
      dt[c] = !live || c >= nc ? 0.0f : a.softplus ? softplus(x[c]) : x[c];
      dy[c] = a.z ? go[c] * z[c] * sigmoid(z[c]) : go[c];
      dtx[tt][cq + c] = make_float2(dt[c], live && c < nc ? dt[c] * u[c] : 0.0f);
      dys[tt][cq + c] = dy[c];
    }
    stage_bc<T, NS>(a.Bm, a.b_ld, a, w, t0, Bs);
    stage_bc<T, NS>(a.Cm, a.c_ld, a, w, t0, Cs);
    __syncthreads();
    const int nt = min(TT, w.t_hi - t0);
    for (int t1 = (nt - 1) / SUB * SUB; t1 >= 0; t1 -= SUB) {
      float h[NS], hh[SUB][NS], aa[SUB][NS], y[4];
      const long long k = bs * a.subs + (tile * TT + t1) / SUB;
      load_state(a.ck + (k * a.D + d) * a.N, a.N, n0, ok, h);
      const float before = ok ? a.ckdt[k * a.D + d] : 0.0f;
      float hstart[NS];
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        h[i] += __builtin_amdgcn_exp2f(A1[i] * kLog2e * before) * hin[i];
        hstart[i] = h[i];
      }
      float ysum[SUB / 4];
#pragma unroll
      for (int t = 0; t < SUB; ++t) {
        const float2 v = dtx[t1 + t][ch];
        float acc = 0.0f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          aa[t][i] = __builtin_amdgcn_exp2f(v.x * (A1[i] * kLog2e));
          h[i] = aa[t][i] * h[i] + v.y * Bs[t1 + t][n0 + i];
          hh[t][i] = h[i];
          acc += h[i] * Cs[t1 + t][n0 + i];
        }
        y[t & 3] = acc;
        if ((t & 3) == 3) ysum[t >> 2] = row_sums(y, row);
      }
#pragma unroll
      for (int t4 = SUB - 4; t4 >= 0; t4 -= 4) {
        float gB[4], sA[4];
#pragma unroll
        for (int j = 3; j >= 0; --j) {
          const int t = t4 + j;
          const float2 v = dtx[t1 + t][ch];
          const float dyv = dys[t1 + t][ch];
          gB[j] = sA[j] = 0.0f;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const float Bv = Bs[t1 + t][n0 + i], Cv = Cs[t1 + t][n0 + i];
            const float g = Cv * dyv + carry[i];
            carry[i] = aa[t][i] * g;
            const float wv = carry[i] * (t > 0 ? hh[t - 1][i] : hstart[i]);
            sA[j] += A1[i] * wv;
            dA[i] += v.x * wv;
            gB[j] += g * Bv;
            const float pB = row16_sum(g * v.y), pC = row16_sum(dyv * hh[t][i]);
            if ((lane & 15) == 0) {
              part[wave][t1 + t][0][n0 + i] = pB;
              part[wave][t1 + t][1][n0 + i] = pC;
            }
          }
        }
        const float vB = row_sums(gB, row), vA = row_sums(sA, row);
        // only this wave reads these channels' entries, and it is past these tokens
        dtx[t1 + t4 + row][ch] = make_float2(vB, vA);
        dys[t1 + t4 + row][ch] = ysum[t4 >> 2];
      }
    }
    __syncthreads();
    if (live) {
      float gu[4], gd[4], gz[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 v = dtx[tt][cq + c];
        gu[c] = v.x * dt[c] + dy[c] * Dsk[c];
        gd[c] = v.y + v.x * u[c];
        if (a.softplus) gd[c] *= sigmoid(x[c]);
        const float y = dys[tt][cq + c] + Dsk[c] * u[c], sg = sigmoid(z[c]);
        gz[c] = go[c] * y * sg * (1.0f + z[c] * (1.0f - sg));
        sD[c] += dy[c] * u[c];
        sb[c] += gd[c];
      }
      store4<VEC>(a.du, r * a.D + dq, nc, gu, a.out_bf16);
      store4<VEC>(a.ddelta, r * a.D + dq, nc, gd, a.out_bf16);
      if (a.z) store4<VEC>(a.dz, r * a.D + dq, nc, gz, a.out_bf16);
    }
    for (int e = tid; e < nt * 2 * a.N; e += NT) {
      const int t = e / (2 * a.N), k = e / a.N % 2, n = e % a.N;
      a.bcpart[((((long long)w.tile * a.B + w.b) * a.L + t0 + t) * a.G + w.g) * 2 * a.N + k * a.N + n] =
          part[0][t][k][n] + part[1][t][k][n] + part[2][t][k][n] + part[3][t][k][n];
    }
  }
  store_state(a.dApart + sd * a.N, a.N, n0, ok, dA);
  if (w.s == 0 && a.dh0) store_state(a.dh0 + ((long long)w.b * a.D + d) * a.N, a.N, n0, ok, carry);
  // dD and the bias's gradient: the 16 token threads of each channel
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 4; ++c) dtx[tt][cq + c] = make_float2(sD[c], sb[c]);
  __syncthreads();
  if (tid < CH && w.tile * CH + tid < a.Dg) {
    float2 t = make_float2(0.0f, 0.0f);
    for (int k = 0; k < TT; ++k) {
      t.x += dtx[k][tid].x;
      t.y += dtx[k][tid].y;
    }
    const long long e = bs * a.D + (long long)w.g * a.Dg + w.tile * CH + tid;
    a.dDpart[e] = t.x;
    a.dbpart[e] = t.y;
  }
}

// Rows behind the sequences' ends: zero gradients of u, delta and z.
__global__ __launch_bounds__(NT) void scan_bwd_tail_kernel(ScanArgs a) {
  const long long r = blockIdx.x, b = r / a.L;
  if (r % a.L < min(max(a.lengths[b], 0), a.L)) return;
  for (int d = threadIdx.x; d < a.D; d += NT) {
    store_elem(a.du, r * a.D + d, 0.0f, a.out_bf16);
    store_elem(a.ddelta, r * a.D + d, 0.0f, a.out_bf16);
    if (a.dz) store_elem(a.dz, r * a.D + d, 0.0f, a.out_bf16);
  }
}

// dB and dC: the sum over the group's channel tiles, in their order.
__global__ __launch_bounds__(NT) void scan_reduce_bc_kernel(ScanArgs a, void *dB, void *dC) {
  const long long total = (long long)a.B * a.L * a.G * 2 * a.N, id = (long long)blockIdx.x * NT + threadIdx.x;
  if (id >= total) return;
  const int n = id % a.N, k = id / a.N % 2;
  const long long rg = id / (2 * a.N), r = rg / a.G;
  float x = 0.0f;
  if (!a.lengths || r % a.L < a.lengths[r / a.L])
    for (int t = 0; t < a.tiles; ++t) x += a.bcpart[t * total + id];
  store_elem(k ? dC : dB, rg * a.N + n, x, a.out_bf16);
}

// Column sums of part[rows][cols]; double, as thousands of rows may come together.
__global__ __launch_bounds__(NT) void column_sum_kernel(const float *part, float *out, int rows, long long cols) {
  __shared__ double red[4][64];
  const long long col = (long long)blockIdx.x * 64 + (threadIdx.x & 63);
  const int w = threadIdx.x >> 6;
  double x = 0.0;
  if (col < cols)
    for (int r = w; r < rows; r += 4) x += part[r * cols + col];
  red[w][threadIdx.x & 63] = x;
  __syncthreads();
  if (w == 0 && col < cols)
    out[col] = (float)(red[0][threadIdx.x] + red[1][threadIdx.x] + red[2][threadIdx.x] + red[3][threadIdx.x]);
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

// One token: a wave's lanes as in the passes above, the state read and written once.
template <typename T, int NS>
__global__ __launch_bounds__(NT) void scan_step_kernel(ScanArgs a) {
  const int tid = threadIdx.x, lane = tid & 63, row = lane >> 4, ch = (tid >> 6) * 16 + (lane & 15);
  int id = blockIdx.x;
  const int tile = id % a.tiles;
  id /= a.tiles;
  const int g = id % a.G;
  const long long b = id / a.G;
  const int rel = tile * CH + ch, n0 = row * NS;
  const bool ok = rel < a.Dg;
  const long long d = (long long)g * a.Dg + rel;
  float A[NS], h[NS];
  float *S = a.hT + (b * a.D + d) * a.N;
  load_state(a.A + d * a.N, a.N, n0, ok, A);
  load_state(S, a.N, n0, ok, h);
  constexpr int bf = sizeof(T) == 2;
  float u = 0.0f, dt = 0.0f;
  if (ok) {
    u = load_elem(a.u, b * a.u_ld + d, bf);
    dt = load_elem(a.delta, b * a.delta_ld + d, bf) + (a.bias ? a.bias[d] : 0.0f);
    if (a.softplus) dt = softplus(dt);
  }
  float y = 0.0f;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = n0 + i;
    const float Bv = n < a.N ? load_elem(a.Bm, b * a.b_ld + (long long)g * a.N + n, bf) : 0.0f;
    const float Cv = n < a.N ? load_elem(a.Cm, b * a.c_ld + (long long)g * a.N + n, bf) : 0.0f;
    h[i] = __builtin_amdgcn_exp2f(dt * (A[i] * kLog2e)) * h[i] + dt * u * Bv;
    y += h[i] * Cv;
  }
  store_state(S, a.N, n0, ok, h);
  y += __shfl_xor(y, 16, 64);
  y += __shfl_xor(y, 32, 64);
  if (ok && row == 0) {
    if (a.Dskip) y += a.Dskip[d] * u;
    if (a.z) {
      const float z = load_elem(a.z, b * a.z_ld + d, bf);
      y *= z * sigmoid(z);
    }
    store_elem(a.out, b * a.D + d, y, a.out_bf16);
  }
}

// ------------------------------------------------------------------ host side
int state_regs(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

struct ScanPlan {
  int tiles, seg_len, nseg, subs;
  size_t seg, sdt, gseg, ck, ckdt, bcpart, dApart, dDpart, dbpart, total;
};

// Segments: about `want` workgroups in all, of at least a tile each.
ScanPlan scan_plan(int B, int L, int D, int N, int G, bool bwd) {
  ScanPlan p;
  p.tiles = (int)rec_cdiv(D / G, CH);
  const long long blocks = (long long)B * G * p.tiles, want = 1024;
  long long nseg = std::min<long long>(rec_cdiv(want, blocks), rec_cdiv(L, 4 * TT));
  if (!bwd && 2 * blocks >= want) nseg = 1;
  p.seg_len = (int)(rec_cdiv(rec_cdiv(L, std::max<long long>(nseg, 1)), TT) * TT);
  p.nseg = (int)rec_cdiv(L, p.seg_len);
  const int NS = state_regs(N), SUB = NS <= 4 ? 16 : 64 / NS;
  p.subs = p.seg_len / SUB;
  size_t off = 0;
  auto take = [&off](size_t floats) {
    const size_t at = off;
    off += rec_align(floats * 4);
    return at;
  };
  const size_t bs = (size_t)B * p.nseg, DN = (size_t)D * N;
  p.seg = p.sdt = p.gseg = p.ck = p.ckdt = p.bcpart = p.dApart = p.dDpart = p.dbpart = 0;
  if (bwd || p.nseg > 1) {
    p.seg = take(bs * DN);
    p.sdt = take(bs * D);
  }
  if (bwd) {
    p.gseg = take(bs * DN);
    p.ck = take(bs * p.subs * DN);
    p.ckdt = take(bs * p.subs * D);
    p.bcpart = take((size_t)p.tiles * B * L * G * 2 * N);
    p.dApart = take(bs * DN);
    p.dDpart = take(bs * D);
    p.dbpart = take(bs * D);
  }
  p.total = off;
  return p;
}

// Sizes a call takes: within the header's limits, and a workgroup grid that can be launched.
bool plan_ok(int B, int L, int D, int N, int G) {
  return B > 0 && L > 0 && D > 0 && N > 0 && G > 0 && D % G == 0 && N <= RECURRENT_MAX_STATE &&
         (long long)B * L <= RECURRENT_MAX_TOKENS && (double)B * L * D <= RECURRENT_MAX_ELEMENTS &&
         (double)B * D * N <= RECURRENT_MAX_ELEMENTS && (double)B * G * rec_cdiv(D / G, CH) < 2e9 &&
         (double)B * L * G * N <= RECURRENT_MAX_ELEMENTS;
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
hipError_t launch(K kernel, long long blocks, hipStream_t st, const ScanArgs &a) {
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(NT), 0, st, a);
  return hipGetLastError();
}

template <typename T, bool VEC, int MODE>
hipError_t launch_pass(const ScanArgs &a, hipStream_t st) {
  const long long blocks = (long long)a.B * a.nseg * a.G * a.tiles;
  switch (state_regs(a.N)) {
    case 1: return launch(scan_pass_kernel<T, 1, VEC, MODE>, blocks, st, a);
    case 2: return launch(scan_pass_kernel<T, 2, VEC, MODE>, blocks, st, a);
    case 4: return launch(scan_pass_kernel<T, 4, VEC, MODE>, blocks, st, a);
    case 8: return launch(scan_pass_kernel<T, 8, VEC, MODE>, blocks, st, a);
    default: return launch(scan_pass_kernel<T, 16, VEC, MODE>, blocks, st, a);
  }
}
template <int MODE>
hipError_t launch_pass(const ScanArgs &a, bool bf, bool vec, hipStream_t st) {
  if (bf) return vec ? launch_pass<uint16_t, true, MODE>(a, st) : launch_pass<uint16_t, false, MODE>(a, st);
  return vec ? launch_pass<float, true, MODE>(a, st) : launch_pass<float, false, MODE>(a, st);
}

template <typename T, bool VEC>
hipError_t launch_bwd(const ScanArgs &a, hipStream_t st) {
  const long long blocks = (long long)a.B * a.nseg * a.G * a.tiles;
  switch (state_regs(a.N)) {
    case 1: return launch(scan_bwd_kernel<T, 1, VEC>, blocks, st, a);
    case 2: return launch(scan_bwd_kernel<T, 2, VEC>, blocks, st, a);
    case 4: return launch(scan_bwd_kernel<T, 4, VEC>, blocks, st, a);
    case 8: return launch(scan_bwd_kernel<T, 8, VEC>, blocks, st, a);
    default: return launch(scan_bwd_kernel<T, 16, VEC>, blocks, st, a);
  }
}
hipError_t launch_bwd(const ScanArgs &a, bool bf, bool vec, hipStream_t st) {
  if (bf) return vec ? launch_bwd<uint16_t, true>(a, st) : launch_bwd<uint16_t, false>(a, st);
  return vec ? launch_bwd<float, true>(a, st) : launch_bwd<float, false>(a, st);
}

template <typename T>
hipError_t launch_step(const ScanArgs &a, hipStream_t st) {
  const long long blocks = (long long)a.B * a.G * a.tiles;
  switch (state_regs(a.N)) {
    case 1: return launch(scan_step_kernel<T, 1>, blocks, st, a);
    case 2: return launch(scan_step_kernel<T, 2>, blocks, st, a);
    case 4: return launch(scan_step_kernel<T, 4>, blocks, st, a);
    case 8: return launch(scan_step_kernel<T, 8>, blocks, st, a);
    default: return launch(scan_step_kernel<T, 16>, blocks, st, a);
  }
}

hipError_t launch_combine(const ScanArgs &a, hipStream_t st) {
  return launch(scan_combine_kernel, rec_cdiv((long long)a.B * a.D * a.N, NT), st, a);
}

hipError_t column_sum(const float *part, float *out, int rows, long long cols, hipStream_t st) {
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)rec_cdiv(cols, 64)), dim3(NT), 0, st, part, out, rows, cols);
  return hipGetLastError();
}

ScanArgs scan_args(const void *u, const void *delta, const float *A, const void *Bm, const void *Cm,
                   const float *D_skip, const void *z, const float *bias, const int *lengths, int B, int L, int D,
                   int N, int G, long long u_ld, long long delta_ld, long long z_ld, long long b_ld, long long c_ld,
                   int softplus, ret_dtype_t out_dtype) {
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
  a.tiles = (int)rec_cdiv(a.Dg, CH);
  a.softplus = softplus != 0;
  a.out_bf16 = out_dtype == RET_BF16;
  return a;
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
  return plan_ok(B, L, D, N, G) ? scan_plan(B, L, D, N, G, false).total : 0;
}

size_t selective_scan_bwd_workspace_bytes(int B, int L, int D, int N, int G) {
  return plan_ok(B, L, D, N, G) ? scan_plan(B, L, D, N, G, true).total : 0;
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
                         c_ld, delta_softplus, out_dtype);
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
  a.seg_len = p.seg_len;
  a.nseg = p.nseg;
  a.seg = (float *)((char *)workspace + p.seg);
  a.sdt = (float *)((char *)workspace + p.sdt);
  const bool bf = in_dtype == RET_BF16;
  const bool vec = a.Dg % 4 == 0 && wide(u, u_ld, e) && wide(delta, delta_ld, e) && wide(z, z_ld, e) &&
                   wide(out, D, oe);
  hipError_t err = hipSuccess;
  if (p.nseg > 1) {
    if ((err = launch_pass<STATES>(a, bf, vec, st)) != hipSuccess || (err = launch_combine(a, st)) != hipSuccess)
      return rec_status(err);
  }
  return rec_status(launch_pass<OUTPUT>(a, bf, vec, st));
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
                         c_ld, delta_softplus, out_dtype);
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
  const RecSpan dho = {"d_state_out", d_state_out, d_state_out ? ns : 0};
  const RecSpan outs[] = {{"du", du, (size_t)rows * D * oe}, {"ddelta", ddelta, (size_t)rows * D * oe},
                          {"dA", dA, (size_t)D * N * 4}, {"dB", dB, (size_t)rows * bc * oe},
                          {"dC", dC, (size_t)rows * bc * oe}, {"dD", dD, (size_t)D * 4},
                          {"dz", dz, (size_t)rows * D * oe}, {"ddelta_bias", ddelta_bias, (size_t)D * 4},
                          {"d_state_in", d_state_in, d_state_in ? ns : 0},
                          {"the workspace", L ? workspace : nullptr, workspace_bytes}};
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
  const ScanPlan p = scan_plan(B, L, D, N, G, true);
  if (!workspace || workspace_bytes < p.total)
    return rec_fail(RET_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", p.total, workspace_bytes);
  if (!rec_aligned(workspace, 16)) return rec_fail(RET_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  char *ws = (char *)workspace;
  a.seg_len = p.seg_len;
  a.nseg = p.nseg;
  a.subs = p.subs;
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
  const bool vec = a.Dg % 4 == 0 && wide(u, u_ld, e) && wide(delta, delta_ld, e) && wide(z, z_ld, e) &&
                   wide(d_o, D, e) && wide(du, D, oe) && wide(ddelta, D, oe) && wide(dz, D, oe);
  hipError_t err;
  if ((err = launch_pass<CHECKPOINTS>(a, bf, vec, st)) != hipSuccess || (err = launch_combine(a, st)) != hipSuccess ||
      (err = launch_bwd(a, bf, vec, st)) != hipSuccess)
    return rec_status(err);
  if (lengths && (err = launch(scan_bwd_tail_kernel, rows, st, a)) != hipSuccess) return rec_status(err);
  hipLaunchKernelGGL(scan_reduce_bc_kernel, dim3((unsigned)rec_cdiv(rows * 2 * bc, NT)), dim3(NT), 0, st, a, dB, dC);
  if ((err = hipGetLastError()) != hipSuccess) return rec_status(err);
  const int parts = B * p.nseg;
  if ((err = column_sum(a.dApart, dA, parts, (long long)D * N, st)) != hipSuccess) return rec_status(err);
  if (dD && (err = column_sum(a.dDpart, dD, parts, D, st)) != hipSuccess) return rec_status(err);
  if (ddelta_bias && (err = column_sum(a.dbpart, ddelta_bias, parts, D, st)) != hipSuccess) return rec_status(err);
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
                         c_ld, delta_softplus, out_dtype);
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
  hipStream_t st = (hipStream_t)hip_stream;
  return rec_status(in_dtype == RET_BF16 ? launch_step<uint16_t>(a, st) : launch_step<float>(a, st));
}

}  // extern "C"
