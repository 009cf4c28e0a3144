// Short causal depthwise convolution (recurrent.h): c_t = act(bias + sum_j w_j x_{t-K+1+j}),
// its gradients and its single-token form.
//
// Every kernel streams: a thread keeps VC neighbouring channels (four, where rows are
// aligned to them), their taps and a window of the last K inputs in registers and walks
// a run of tokens, so each input is read once but for the K - 1 in front of a run.  The
// loads of a step's tokens go out together.  Bound by the bytes, each moved once: the forward
// takes 63 us for 268 MB (4.2 TB/s) at B 4, L 4096, D 4096, bf16 (the vector unit is busy 81 %); runs of 128 tokens and
// steps of four were no faster.
#include <algorithm>
#include <type_traits>

#include "recurrent.hpp"

using namespace ret;

namespace {

constexpr int NT = 256;
constexpr int STEP = 8;    // tokens whose loads the forward issues together
constexpr int WAVES = NT / 64;

struct ConvArgs {
  const void *x, *w, *bias, *h0, *d_o, *dhT;
  const int *lengths;
  void *out, *hT, *dx, *dh0;
  float *part;  // [B * runs / WAVES][D][K + 1]: dw, dbias
  long long x_ld;
  int B, L, D, K, run, runs, silu;
  long long main_threads, state_at;  // runs' threads; the first of the state's, a workgroup's start behind them
};

// VC neighbouring channels as they come from memory.
template <typename T, int VC>
struct Raw {
  using V = std::conditional_t<VC == 1, T, std::conditional_t<sizeof(T) == 2, uint2, float4>>;
  V v;
  __device__ __forceinline__ void load(const T *p) { v = *(const V *)p; }
  __device__ __forceinline__ void get(float (&r)[VC]) const {
    if constexpr (VC == 4 && sizeof(T) == 2) {
      r[0] = __uint_as_float(v.x << 16);
      r[1] = __uint_as_float(v.x & 0xffff0000u);
      r[2] = __uint_as_float(v.y << 16);
      r[3] = __uint_as_float(v.y & 0xffff0000u);
    } else if constexpr (VC == 4) {
      r[0] = v.x;
      r[1] = v.y;
      r[2] = v.z;
      r[3] = v.w;
    } else if constexpr (sizeof(T) == 2) {
      r[0] = bf2f(v);
    } else {
      r[0] = v;
    }
  }
};
template <typename T, int VC>
__device__ __forceinline__ void loadc(const T *p, float (&r)[VC]) {
  Raw<T, VC> v;
  v.load(p);
  v.get(r);
}

template <typename T, int VC>
__device__ __forceinline__ void storec(T *p, const float (&r)[VC]) {
  if constexpr (VC == 4)
    store4<true>(p, 0, 4, r, sizeof(T) == 2);
  else
    store_elem(p, 0, r[0], sizeof(T) == 2);
}

// Input t of sequence b (t < 0: from the state in front), VC channels from d; t >= -(K - 1).
template <typename T, int K, int VC>
__device__ __forceinline__ void input_at(const ConvArgs &a, long long b, int t, int d, float (&r)[VC]) {
  if (t >= 0) {
    loadc<T, VC>((const T *)a.x + (b * a.L + t) * a.x_ld + d, r);
  } else if (a.h0) {
    loadc<T, VC>((const T *)a.h0 + (b * (K - 1) + t + K - 1) * a.D + d, r);
  } else {
#pragma unroll
    for (int c = 0; c < VC; ++c) r[c] = 0.0f;
  }
}

template <typename T, int K, int VC>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int d, float (&w)[K][VC], float (&bias)[VC]) {
#pragma unroll
  for (int c = 0; c < VC; ++c) {
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][c] = load_elem(a.w, (long long)(d + c) * K + j, sizeof(T) == 2);
    bias[c] = a.bias ? load_elem(a.bias, d + c, sizeof(T) == 2) : 0.0f;
  }
}

// bias + sum_j w_j x_{i+j}, the products added in their order and each fused with its sum: written
// out, so that a token has the same bits in a prompt and as a step (left to the compiler, two taps
// were fused the one way here and the other way there).
template <int K, int VC, int W>
__device__ __forceinline__ float taps_at(const float (&w)[K][VC], const float (&x)[W][VC], float bias, int i, int c) {
  float s = w[0][c] * x[i][c];
#pragma unroll
  for (int j = 1; j < K; ++j) s = fmaf(w[j][c], x[i + j][c], s);
  return s + bias;
}

__device__ __forceinline__ int length_of(const ConvArgs &a, long long b) {
  return a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;
}

// Threads below main_threads: (sequence, run, channels).  From state_at on: the final
// state, (sequence, tap, channels).
template <typename T, int K, int VC>
__global__ __launch_bounds__(NT) void conv_fwd_kernel(ConvArgs a) {
  const int dv = a.D / VC;
  long long id = (long long)blockIdx.x * NT + threadIdx.x;
  if (id >= a.main_threads) {
    id -= a.state_at;
    if (id < 0 || !a.hT || id >= (long long)a.B * (K - 1) * dv) return;
    const int d = (int)(id % dv) * VC, j = (int)(id / dv % (K - 1));
    const long long b = id / dv / (K - 1);
    float r[VC];
    input_at<T, K, VC>(a, b, length_of(a, b) - (K - 1) + j, d, r);
    storec<T, VC>((T *)a.hT + (b * (K - 1) + j) * a.D + d, r);
    return;
  }
  const int d = (int)(id % dv) * VC;
  const long long b = id / dv / a.runs;
  const int t0 = (int)(id / dv % a.runs) * a.run, t1 = min(t0 + a.run, length_of(a, b));
  if (t0 >= t1) return;
  float w[K][VC], bias[VC], win[K - 1 + STEP][VC];
  load_taps<T, K, VC>(a, d, w, bias);
  Raw<T, VC> next[STEP];
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < STEP; ++i) next[i].load((const T *)a.x + (b * a.L + min(t + i, t1 - 1)) * a.x_ld + d);
  };
  fetch(t0);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) input_at<T, K, VC>(a, b, t0 - (K - 1) + j, d, win[j]);
  for (int t = t0; t < t1; t += STEP) {
#pragma unroll
    for (int i = 0; i < STEP; ++i) next[i].get(win[K - 1 + i]);
    fetch(t + STEP);
#pragma unroll
    for (int i = 0; i < STEP; ++i) {
      float y[VC];
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        const float s = taps_at(w, win, bias[c], i, c);
        y[c] = a.silu ? silu(s) : s;
      }
      if (t + i < t1) storec<T, VC>((T *)a.out + (b * a.L + t + i) * a.D + d, y);
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int c = 0; c < VC; ++c) win[j][c] = win[STEP + j][c];
  }
}

// Gradients.  With g_t = d_o_t act'(pre_t): dx_s = sum_j w_j g_{s+K-1-j}, dw_j = sum_t g_t
// x_{t-K+1+j}, dbias = sum_t g_t.  A thread walks its run's tokens and K - 1 more, whose
// g the last inputs of the run need; the first run also covers the K - 1 inputs of the
// state in front.  The workgroup's waves take neighbouring runs of the same channels and
// add up their dw and dbias.  Bound by its three streams of memory; four waves per SIMD
// (128 registers, where the taps allow it) instead of three took it from 111 to 92 us at best at B 4, L 4096, D 4096,
// bf16 (96 on average: 403 MB, 4.2 TB/s).
template <typename T, int K, int VC>
__global__ __launch_bounds__(NT, K <= 3 || (K == 4 && sizeof(T) == 2) ? 4 : 2) void conv_bwd_kernel(ConvArgs a) {
  constexpr int S = 4;
  __shared__ float red[WAVES][VC * (K + 1)][64];
  const int dv = a.D / VC, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int chunks = (dv + 63) / 64, groups = (a.runs + WAVES - 1) / WAVES;
  const int chunk = (int)(blockIdx.x % chunks) * 64 + lane, rg = (int)(blockIdx.x / chunks % groups);
  const long long b = blockIdx.x / chunks / groups;
  const int k = rg * WAVES + wave, d = min(chunk, dv - 1) * VC;
  const int len = length_of(a, b), t0 = k * a.run, t1 = min(t0 + a.run, len);
  float dw[K][VC], db[VC];
#pragma unroll
  for (int c = 0; c < VC; ++c) {
    db[c] = 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][c] = 0.0f;
  }
  if (chunk < dv && k < a.runs) {
    if (t0 < t1 || k == 0) {
      float w[K][VC], bias[VC], x[K - 1 + S][VC], g[K - 1 + S][VC];
      load_taps<T, K, VC>(a, d, w, bias);
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        input_at<T, K, VC>(a, b, t0 - (K - 1) + j, d, x[j]);
#pragma unroll
        for (int c = 0; c < VC; ++c) g[j][c] = 0.0f;
      }
      // token t closes input s = t - (K - 1); the first run starts with s = -(K - 1)
      const int end = max(t1, t0) + K - 1;
      Raw<T, VC> xr[S] = {}, gr[S] = {};  // the next step's
      auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < S; ++i) {  // tokens behind the end: any inside, and no g
          const int r = min(t + i, len - 1);
          xr[i].load((const T *)a.x + (b * a.L + r) * a.x_ld + d);
          gr[i].load((const T *)a.d_o + (b * a.L + r) * a.D + d);
        }
      };
      if (len > 0) fetch(t0);
      for (int t = t0; t < end; t += S) {
        float go[S][VC];
#pragma unroll
        for (int i = 0; i < S; ++i) {
          xr[i].get(x[K - 1 + i]);
          gr[i].get(go[i]);
        }
        if (len > 0) fetch(t + S);
#pragma unroll
        for (int i = 0; i < S; ++i) {
#pragma unroll
          for (int c = 0; c < VC; ++c) {
            float s = bias[c];
#pragma unroll
            for (int j = 0; j < K; ++j) s += w[j][c] * x[i + j][c];
            const float sg = sigmoid(s), v = a.silu ? go[i][c] * sg * (1.0f + s * (1.0f - sg)) : go[i][c];
            g[K - 1 + i][c] = t + i < len ? v : 0.0f;
            if (t + i < t1) {
              db[c] += g[K - 1 + i][c];
#pragma unroll
              for (int j = 0; j < K; ++j) dw[j][c] += g[K - 1 + i][c] * x[i + j][c];
            }
          }
        }
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const int s = t + i - (K - 1);
          if (t + i >= end || (s < t0 && k > 0)) continue;  // the run in front closes the latter
          float dx[VC];
          const int q = s - (len - (K - 1));  // its place in the final state
          if (a.dhT && q >= 0 && q < K - 1) {
            loadc<T, VC>((const T *)a.dhT + (b * (K - 1) + q) * a.D + d, dx);
          } else {
#pragma unroll
            for (int c = 0; c < VC; ++c) dx[c] = 0.0f;
          }
#pragma unroll
          for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int j = 0; j < K; ++j) dx[c] += w[j][c] * g[K - 1 + i - j][c];
          if (s >= 0)
            storec<T, VC>((T *)a.dx + (b * a.L + s) * a.D + d, dx);
          else if (a.dh0)
            storec<T, VC>((T *)a.dh0 + (b * (K - 1) + s + K - 1) * a.D + d, dx);
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
#pragma unroll
          for (int c = 0; c < VC; ++c) {
            x[j][c] = x[S + j][c];
            g[j][c] = g[S + j][c];
          }
      }
    }
    // rows behind the end
    for (int t = max(t0, len); t < min(t0 + a.run, a.L); ++t) {
      float zero[VC];
#pragma unroll
      for (int c = 0; c < VC; ++c) zero[c] = 0.0f;
      storec<T, VC>((T *)a.dx + (b * a.L + t) * a.D + d, zero);
    }
  }
#pragma unroll
  for (int c = 0; c < VC; ++c) {
#pragma unroll
    for (int j = 0; j < K; ++j) red[wave][c * (K + 1) + j][lane] = dw[j][c];
    red[wave][c * (K + 1) + K][lane] = db[c];
  }
  __syncthreads();
  float *p = a.part + (b * groups + rg) * a.D * (K + 1) + (long long)(blockIdx.x % chunks) * 64 * VC * (K + 1);
  const int have = min(dv - (int)(blockIdx.x % chunks) * 64, 64) * VC * (K + 1);
  for (int e = threadIdx.x; e < have; e += NT) {
    const int l = e / (VC * (K + 1)), i = e % (VC * (K + 1));
    float s = red[0][i][l];
#pragma unroll
    for (int v = 1; v < WAVES; ++v) s += red[v][i][l];
    p[e] = s;
  }
}

// dw and dbias: the sums over the workgroups along the tokens, in a fixed order and in double.
// A workgroup takes COLS columns of part, its threads' rows run ROWS apart, eight loads ahead.
constexpr int COLS = 32, ROWS = 16;
__global__ __launch_bounds__(COLS * ROWS) void conv_sum_kernel(const float *part, float *dw, float *dbias,
                                                               long long rows, int D, int K) {
  __shared__ double red[ROWS][COLS];
  const int c = threadIdx.x % COLS, r0 = threadIdx.x / COLS;
  const long long col = (long long)blockIdx.x * COLS + c, cols = (long long)D * (K + 1);
  constexpr int U = 8;
  double x = 0.0;
  if (col < cols)
    for (long long r = r0; r < rows; r += U * ROWS) {
      float v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) v[k] = r + k * ROWS < rows ? part[(r + k * ROWS) * cols + col] : 0.0f;
#pragma unroll
      for (int k = 0; k < U; ++k) x += v[k];
    }
  red[r0][c] = x;
  __syncthreads();
  if (r0 != 0 || col >= cols) return;
#pragma unroll
  for (int k = 1; k < ROWS; ++k) x += red[k][c];
  const long long d = col / (K + 1);
  const int j = (int)(col % (K + 1));
  if (j < K)
    dw[d * K + j] = (float)x;
  else if (dbias)
    dbias[d] = (float)x;
}
hipError_t conv_sum(const float *part, float *dw, float *dbias, long long rows, int D, int K, hipStream_t st) {
  hipLaunchKernelGGL(conv_sum_kernel, dim3((unsigned)rec_cdiv((long long)D * (K + 1), COLS)), dim3(COLS * ROWS), 0, st,
                     part, dw, dbias, rows, D, K);
  return hipGetLastError();
}

// One token, bound by its launch (2.5 to 4 us).
template <typename T, int K, int VC>
__global__ __launch_bounds__(NT) void conv_step_kernel(ConvArgs a) {
  const int dv = a.D / VC;
  const long long id = (long long)blockIdx.x * NT + threadIdx.x;
  if (id >= (long long)a.B * dv) return;
  const int d = (int)(id % dv) * VC;
  const long long b = id / dv;
  float w[K][VC], bias[VC], x[K][VC], y[VC];
  load_taps<T, K, VC>(a, d, w, bias);
  T *S = (T *)a.hT + b * (K - 1) * a.D + d;
#pragma unroll
  for (int j = 0; j < K - 1; ++j) loadc<T, VC>(S + (long long)j * a.D, x[j]);
  loadc<T, VC>((const T *)a.x + b * a.x_ld + d, x[K - 1]);
#pragma unroll
  for (int c = 0; c < VC; ++c) {
    const float s = taps_at(w, x, bias[c], 0, c);
    y[c] = a.silu ? silu(s) : s;
  }
  storec<T, VC>((T *)a.out + b * a.D + d, y);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) storec<T, VC>(S + (long long)j * a.D, x[j + 1]);
}

// ------------------------------------------------------------------ host side
enum { FWD, BWD, ONE };

template <int WHAT, typename T, int K, int VC>
hipError_t launch_k(const ConvArgs &a, long long threads, hipStream_t st) {
  dim3 grid((unsigned)rec_cdiv(threads, NT));
  if (WHAT == BWD) grid.x = (unsigned)(rec_cdiv(a.D / VC, 64) * rec_cdiv(a.runs, WAVES) * a.B);
  if constexpr (WHAT == FWD)
    hipLaunchKernelGGL((conv_fwd_kernel<T, K, VC>), grid, dim3(NT), 0, st, a);
  else if constexpr (WHAT == BWD)
    hipLaunchKernelGGL((conv_bwd_kernel<T, K, VC>), grid, dim3(NT), 0, st, a);
  else
    hipLaunchKernelGGL((conv_step_kernel<T, K, VC>), grid, dim3(NT), 0, st, a);
  return hipGetLastError();
}
template <int WHAT, typename T, int VC>
hipError_t launch_vc(const ConvArgs &a, long long threads, hipStream_t st) {
  switch (a.K) {
    case 2: return launch_k<WHAT, T, 2, VC>(a, threads, st);
    case 3: return launch_k<WHAT, T, 3, VC>(a, threads, st);
    case 4: return launch_k<WHAT, T, 4, VC>(a, threads, st);
    case 5: return launch_k<WHAT, T, 5, VC>(a, threads, st);
    case 6: return launch_k<WHAT, T, 6, VC>(a, threads, st);
    case 7: return launch_k<WHAT, T, 7, VC>(a, threads, st);
    default: return launch_k<WHAT, T, 8, VC>(a, threads, st);
  }
}
template <int WHAT>
hipError_t launch(const ConvArgs &a, bool bf, int vc, long long threads, hipStream_t st) {
  if (bf) return vc > 1 ? launch_vc<WHAT, uint16_t, 4>(a, threads, st) : launch_vc<WHAT, uint16_t, 1>(a, threads, st);
  return vc > 1 ? launch_vc<WHAT, float, 4>(a, threads, st) : launch_vc<WHAT, float, 1>(a, threads, st);
}

ret_status_t check_sizes(int B, int L, int D, int K, long long x_ld, ret_dtype_t dtype) {
  if (B <= 0 || L < 0 || D <= 0 || K <= 0)
    return rec_fail(RET_ERR_INVALID_ARG, "sizes must be positive (B=%d L=%d D=%d K=%d)", B, L, D, K);
  if (!rec_dtype_ok(dtype)) return rec_fail(RET_ERR_INVALID_ARG, "unknown dtype");
  if (K < 2 || K > RECURRENT_MAX_TAPS)
    return rec_fail(RET_ERR_UNSUPPORTED, "K=%d outside 2..%d", K, RECURRENT_MAX_TAPS);
  if (x_ld < D) return rec_fail(RET_ERR_INVALID_ARG, "a row stride is shorter than its row");
  if (x_ld > (1LL << 31)) return rec_fail(RET_ERR_UNSUPPORTED, "a row stride above 2^31");
  if (D > RECURRENT_MAX_CHANNELS || (long long)B * std::max(L, 1) > RECURRENT_MAX_TOKENS ||
      (double)B * L * D > RECURRENT_MAX_ELEMENTS || (double)B * K * D > RECURRENT_MAX_STATES)
    return rec_fail(RET_ERR_UNSUPPORTED, "too many tokens (B=%d L=%d D=%d)", B, L, D);
  return RET_OK;
}

// Channels a thread takes: four where every tensor of the call allows it.
int channels(const void *const *ps, int n, int D, long long x_ld, size_t e) {
  if (D % 4 || x_ld % 4) return 1;
  for (int i = 0; i < n; ++i)
    if (!rec_aligned(ps[i], 4 * e)) return 1;
  return 4;
}

// Tokens a thread walks: long runs reread fewer of the K - 1 tokens in front, short
// ones give more threads; about four workgroups a CU are wanted.
void set_runs(ConvArgs &a, int vc, int most) {
  const long long per = (long long)a.B * (a.D / vc);
  int run = most;
  while (run > STEP && per * rec_cdiv(a.L, run) < 1024LL * NT) run /= 2;
  a.run = run;
  a.runs = (int)rec_cdiv(a.L, run);
  a.main_threads = per * a.runs;
}
constexpr int FWD_RUN = 64, BWD_RUN = 64;

// Partial sums of the backward for at most L tokens: workgroups along the tokens, of the kernel that
// has the most.  Runs are halved where 64-token ones give less than 1024 NT threads, so that fewer
// tokens can have more runs: at most the twice as many that were too few before the last halving.
long long bwd_parts(int B, int L, int D) {
  long long most = 0;
  for (int vc : {1, 4})
    if (D % vc == 0) {
      const long long enough = (1024LL * NT - 1) / ((long long)B * (D / vc));
      const long long runs = std::max(rec_cdiv(L, BWD_RUN), std::min(rec_cdiv(L, STEP), 2 * enough));
      most = std::max(most, B * rec_cdiv(runs, WAVES));
    }
  return most;
}

}  // namespace

extern "C" {

ret_status_t causal_conv1d(const void *x, const void *w, const void *bias, void *out, const int *lengths,
                           const void *state_in, void *state_out, int B, int L, int D, int K, long long x_ld, int silu,
                           ret_dtype_t dtype, void *hip_stream) {
  ret_status_t s = check_sizes(B, L, D, K, x_ld, dtype);
  if (s != RET_OK) return s;
  if (!w || (L > 0 && (!x || !out))) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  const size_t e = rec_esize(dtype), ns = (size_t)B * (K - 1) * D * e;
  const void *ps[] = {x, out, state_in, state_out, w, bias};
  for (const void *p : ps)
    if (!rec_aligned(p, e)) return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  if (!rec_aligned(lengths, 4)) return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const long long rows = (long long)B * L;
  const RecSpan ins[] = {rec_rows("x", x, rows, x_ld, D, e), {"w", w, (size_t)D * K * e}, {"bias", bias, (size_t)D * e},
                         {"state_in", state_in, ns}, {"lengths", lengths, (size_t)B * 4}};
  const RecSpan outs[] = {{"out", out, (size_t)rows * D * e}, {"state_out", state_out, ns}};
  if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
  ConvArgs a = {};
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.out = out;
  a.lengths = lengths;
  a.h0 = state_in;
  a.hT = state_out;
  a.B = B;
  a.L = L;
  a.D = D;
  a.K = K;
  a.x_ld = x_ld;
  a.silu = silu != 0;
  const int vc = channels(ps, 4, D, x_ld, e);
  if (L > 0) {
    set_runs(a, vc, FWD_RUN);
    a.state_at = rec_cdiv(a.main_threads, NT) * NT;
  }
  const long long threads = a.state_at + (state_out ? (long long)B * (K - 1) * (D / vc) : 0);
  if (threads == 0) return rec_status(hipSuccess);
  if (!rec_grid_ok((double)rec_cdiv(threads, NT), NT))
    return rec_fail(RET_ERR_UNSUPPORTED, "too many tokens (B=%d L=%d D=%d)", B, L, D);
  return rec_status(launch<FWD>(a, dtype == RET_BF16, vc, threads, (hipStream_t)hip_stream));
}

size_t causal_conv1d_bwd_workspace_bytes(int B, int L, int D, int K) {
  if (B <= 0 || L <= 0 || D <= 0 || K < 2 || K > RECURRENT_MAX_TAPS) return 0;
  if (D > RECURRENT_MAX_CHANNELS || (long long)B * L > RECURRENT_MAX_TOKENS ||
      (double)B * L * D > RECURRENT_MAX_ELEMENTS)
    return 0;
  return rec_align((size_t)bwd_parts(B, L, D) * D * (K + 1) * 4);
}

ret_status_t causal_conv1d_bwd(const void *x, const void *w, const void *bias, const void *d_o, const int *lengths,
                               const void *state_in, const void *d_state_out, void *dx, float *dw, float *dbias,
                               void *d_state_in, int B, int L, int D, int K, long long x_ld, int silu,
                               ret_dtype_t dtype, void *workspace, size_t workspace_bytes, void *hip_stream) {
  ret_status_t s = check_sizes(B, L, D, K, x_ld, dtype);
  if (s != RET_OK) return s;
  if (!w || !dw || (L > 0 && (!x || !d_o || !dx))) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  const size_t e = rec_esize(dtype), ns = (size_t)B * (K - 1) * D * e;
  const void *ps[] = {x, d_o, dx, state_in, d_state_out, d_state_in, w, bias};
  for (const void *p : ps)
    if (!rec_aligned(p, e)) return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const void *fs[] = {lengths, dw, dbias};
  for (const void *p : fs)
    if (!rec_aligned(p, 4)) return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const long long rows = (long long)B * L;
  const int vc = channels(ps, 6, D, x_ld, e);
  ConvArgs a = {};
  a.B = B;
  a.L = L;
  a.D = D;
  if (L > 0) set_runs(a, vc, BWD_RUN);
  const long long parts = L > 0 ? B * rec_cdiv(a.runs, WAVES) : 0;
  const size_t need = rec_align((size_t)parts * D * (K + 1) * 4);
  const RecSpan ins[] = {rec_rows("x", x, rows, x_ld, D, e), {"w", w, (size_t)D * K * e}, {"bias", bias, (size_t)D * e},
                         {"d_o", d_o, (size_t)rows * D * e}, {"state_in", state_in, ns},
                         {"d_state_out", d_state_out, ns}, {"lengths", lengths, (size_t)B * 4}};
  const RecSpan outs[] = {{"dx", dx, (size_t)rows * D * e}, {"dw", dw, (size_t)D * K * 4},
                          {"dbias", dbias, (size_t)D * 4}, {"d_state_in", d_state_in, ns},
                          {"the workspace", L ? workspace : nullptr, need}};
  if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
  if (L > 0 && (!workspace || workspace_bytes < need))
    return rec_fail(RET_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  if (!rec_aligned(workspace, 16)) return rec_fail(RET_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.d_o = d_o;
  a.lengths = lengths;
  a.h0 = state_in;
  a.dhT = d_state_out;
  a.dx = dx;
  a.dh0 = d_state_in;
  a.part = (float *)workspace;
  a.K = K;
  a.x_ld = x_ld;
  a.silu = silu != 0;
  hipStream_t st = (hipStream_t)hip_stream;
  const bool bf = dtype == RET_BF16;
  if (L == 0) {  // the state passes through, the sums are empty: the step's work without tokens
    hipError_t err = hipSuccess;
    if (d_state_in) {
      ConvArgs c = {};
      c.B = B;
      c.D = D;
      c.K = K;
      c.h0 = d_state_out;
      c.hT = d_state_in;
      const void *qs[] = {d_state_out, d_state_in};
      const int sv = channels(qs, 2, D, 0, e);
      err = launch<FWD>(c, bf, sv, (long long)B * (K - 1) * (D / sv), st);
    }
    if (err == hipSuccess) err = conv_sum(nullptr, dw, dbias, 0, D, K, st);
    return rec_status(err);
  }
  if (!rec_grid_ok((double)rec_cdiv(D / vc, 64) * rec_cdiv(a.runs, WAVES) * B, NT))
    return rec_fail(RET_ERR_UNSUPPORTED, "too many tokens (B=%d L=%d D=%d)", B, L, D);
  hipError_t err = launch<BWD>(a, bf, vc, a.main_threads, st);
  if (err != hipSuccess) return rec_status(err);
  return rec_status(conv_sum(a.part, dw, dbias, parts, D, K, st));
}

ret_status_t causal_conv1d_step(const void *x, const void *w, const void *bias, void *out, void *state, int B, int D,
                                int K, long long x_ld, int silu, ret_dtype_t dtype, void *hip_stream) {
  ret_status_t s = check_sizes(B, 1, D, K, x_ld, dtype);
  if (s != RET_OK) return s;
  if (!x || !w || !out || !state) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  const size_t e = rec_esize(dtype);
  const void *ps[] = {x, out, state, w, bias};
  for (const void *p : ps)
    if (!rec_aligned(p, e)) return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const RecSpan ins[] = {rec_rows("x", x, B, x_ld, D, e), {"w", w, (size_t)D * K * e}, {"bias", bias, (size_t)D * e}};
  const RecSpan outs[] = {{"out", out, (size_t)B * D * e}, {"state", state, (size_t)B * (K - 1) * D * e}};
  if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
  ConvArgs a = {};
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.out = out;
  a.hT = state;
  a.B = B;
  a.D = D;
  a.K = K;
  a.x_ld = x_ld;
  a.silu = silu != 0;
  const int vc = channels(ps, 3, D, x_ld, e);
  return rec_status(launch<ONE>(a, dtype == RET_BF16, vc, (long long)B * (D / vc), (hipStream_t)hip_stream));
}

}  // extern "C"
