// GroupNorm of every token and head with a gate, and its gradients (language.h).
//
// A group of TPR lanes holds a row of W channels in registers, eight neighbouring ones in each of C
// chunks, so a row is read once: the mean first, then the squared differences from it.
// The gradients need the same statistics and three more sums over the row; a workgroup stays with one
// head and walks its tokens, so that the sums over tokens (dweight, dbias) stay in registers until
// its end, are joined in LDS, and leave one partial row a workgroup for a second launch.
// Bound by bytes: B 4, H 8, L 4096, W 512, bf16 with weight and bias, 403 MB forward in 91 us (4.4 TB/s) and 671 MB
// in 160 for the gradients (4.2 TB/s; 5 us for the second launch), beside a vector unit busy 78 and 90 %.  With ragged
// lengths, half of the tokens on average, 130 us for both launches of the gradients.
#include <algorithm>
#include <type_traits>

#include "language.hpp"

using namespace ret;

namespace {

constexpr int NT = 256;      // forward
constexpr int BWD_NT = 512;  // gradients

struct NormArgs {
  const void *x, *gate, *d_o;
  const float *weight, *bias;
  void *out, *dx, *dgate;
  float *part;  // [parts][2][H W]: dweight, dbias
  const int *lengths;
  long long x_sb, x_sh, x_sl, gate_ld;
  int B, H, L, W, silu, parts;
  float eps;
};

template <int TPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = TPR / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// The activation of a gate and its derivative.
__device__ __forceinline__ float act_of(float g, int silu) { return silu ? g * sigmoid(g) : g; }
__device__ __forceinline__ void act_both(float g, int silu, float &act, float &slope) {
  act = g;
  slope = 1.0f;
  if (silu) {
    const float s = sigmoid(g);
    act = g * s;
    slope = fmaf(act, 1.0f - s, s);
  }
}

// Row statistics: x becomes x - mean (zero behind W), the result is 1 / sqrt(var + eps).
template <int TPR, int C>
__device__ __forceinline__ float normalise(float (&x)[C][8], int col, int W, float eps) {
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < C; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[k][i];
  const float mean = row_sum<TPR>(s) / (float)W;
  float q = 0.0f;
#pragma unroll
  for (int k = 0; k < C; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[k][i] = (k * TPR + col) * 8 + i < W ? x[k][i] - mean : 0.0f;
      q += x[k][i] * x[k][i];
    }
  return 1.0f / sqrtf(row_sum<TPR>(q) / (float)W + eps);
}

// The forward kernel, for the head blockIdx.y: tokens blockIdx.x * RB + row, then parts * RB further on, whose
// loads are under way while one is computed.
template <typename TI, typename TO, int TPR, int C>
__global__ __launch_bounds__(NT) void norm_fwd_kernel(NormArgs a) {
  constexpr int RB = NT / TPR;
  const int col = threadIdx.x & (TPR - 1), h = blockIdx.y;
  float w[C][8], bias[C][8];
#pragma unroll
  for (int k = 0; k < C; ++k) {
    const int c = (k * TPR + col) * 8;
    if (a.weight) load8(a.weight + (long long)h * a.W + c, a.W - c, w[k]);
    if (a.bias) load8(a.bias + (long long)h * a.W + c, a.W - c, bias[k]);
  }
  const unsigned tokens = (unsigned)a.B * a.L, step = a.parts * RB;
  Raw8<TI> xr[C], gr[C];
  bool live = false;
  auto fetch = [&](unsigned tok) {
    const unsigned b = tok / (unsigned)a.L, t = tok - b * a.L;
    live = tok < tokens && (!a.lengths || (int)t < a.lengths[b]);
    const TI *xp = (const TI *)a.x + (long long)b * a.x_sb + h * a.x_sh + t * a.x_sl;
    const TI *gp = (const TI *)a.gate + tok * a.gate_ld + (long long)h * a.W;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int c = (k * TPR + col) * 8, n = live ? a.W - c : 0;
      xr[k].load(xp + c, n);
      if (a.gate) gr[k].load(gp + c, n);
    }
  };
  unsigned tok = blockIdx.x * RB + threadIdx.x / TPR;
  fetch(tok);
  for (; tok < tokens; tok += step) {
    const bool now = live;
    float x[C][8], g[C][8];
#pragma unroll
    for (int k = 0; k < C; ++k) {
      xr[k].get(x[k]);
      if (a.gate) gr[k].get(g[k]);
    }
    fetch(tok + step);
    if (!now) continue;
    const float r = normalise<TPR, C>(x, col, a.W, a.eps);
    TO *out = (TO *)a.out + (long long)tok * a.H * a.W + (long long)h * a.W;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int c = (k * TPR + col) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float n = x[k][i] * r;
        if (a.weight) n *= w[k][i];
        if (a.bias) n += bias[k][i];
        x[k][i] = a.gate ? n * act_of(g[k][i], a.silu) : act_of(n, a.silu);
      }
      store8(out + c, a.W - c, x[k]);
    }
  }
}

// blockIdx.y: the head; blockIdx.x of a.parts: tokens blockIdx.x * RB + row, then parts * RB further on, whose
// loads are under way while one is computed.
template <typename TI, typename TO, int TPR, int C, bool SUMS>
__global__ __launch_bounds__(BWD_NT) void norm_bwd_kernel(NormArgs a) {
  constexpr int RB = BWD_NT / TPR;
  const int col = threadIdx.x & (TPR - 1), h = blockIdx.y;
  float dw[SUMS ? C : 1][8] = {}, db[SUMS ? C : 1][8] = {};
  float w[C][8], bias[C][8];
#pragma unroll
  for (int k = 0; k < C; ++k) {
    const int c = (k * TPR + col) * 8;
    if (a.weight) load8(a.weight + (long long)h * a.W + c, a.W - c, w[k]);
    if (a.bias) load8(a.bias + (long long)h * a.W + c, a.W - c, bias[k]);
  }
  const unsigned tokens = (unsigned)a.B * a.L, step = a.parts * RB;
  Raw8<TI> xr[C], gr[C], dr[C];
  bool live = false;
  auto fetch = [&](unsigned tok) {
    const unsigned b = tok / (unsigned)a.L, t = tok - b * a.L;
    live = tok < tokens && (!a.lengths || (int)t < a.lengths[b]);
    const TI *xp = (const TI *)a.x + (long long)b * a.x_sb + h * a.x_sh + t * a.x_sl;
    const TI *gp = (const TI *)a.gate + tok * a.gate_ld + (long long)h * a.W;
    const TI *dp = (const TI *)a.d_o + (long long)tok * a.H * a.W + (long long)h * a.W;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int c = (k * TPR + col) * 8, n = live ? a.W - c : 0;
      xr[k].load(xp + c, n);
      dr[k].load(dp + c, n);
      if (a.gate) gr[k].load(gp + c, n);
    }
  };
  unsigned tok = blockIdx.x * RB + threadIdx.x / TPR;
  fetch(tok);
  for (; tok < tokens; tok += step) {
    const unsigned b = tok / (unsigned)a.L, t = tok - b * a.L;
    const bool now = live;
    float x[C][8], g[C][8], d[C][8];
#pragma unroll
    for (int k = 0; k < C; ++k) {
      xr[k].get(x[k]);
      dr[k].get(d[k]);
      if (a.gate) gr[k].get(g[k]);
    }
    fetch(tok + step);
    TO *dgate = (TO *)a.dgate + (long long)tok * a.H * a.W + (long long)h * a.W;
    TO *dx = (TO *)a.dx + (((long long)b * a.H + h) * a.L + t) * a.W;
    if (!now) {  // zero whatever weight and bias are
      const float zero[8] = {};
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int c = (k * TPR + col) * 8;
        if (a.gate) store8(dgate + c, a.W - c, zero);
        store8(dx + c, a.W - c, zero);
      }
      continue;
    }
    const float r = normalise<TPR, C>(x, col, a.W, a.eps);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int c = (k * TPR + col) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = x[k][i] * r;
        float n = xh, dn;
        if (a.weight) n *= w[k][i];
        if (a.bias) n += bias[k][i];
        if (a.gate) {
          float act, slope;
          act_both(g[k][i], a.silu, act, slope);
          dn = d[k][i] * act;
          g[k][i] = d[k][i] * n * slope;
        } else {
          float act, slope;
          act_both(n, a.silu, act, slope);
          dn = d[k][i] * slope;
        }
        if constexpr (SUMS) {
          dw[k][i] += dn * xh;
          db[k][i] += dn;
        }
        if (a.weight) dn *= w[k][i];
        x[k][i] = xh;
        d[k][i] = dn;
        s1 += dn;
        s2 += dn * xh;
      }
      if (a.gate) store8(dgate + c, a.W - c, g[k]);
    }
    s1 = row_sum<TPR>(s1) / (float)a.W;
    s2 = row_sum<TPR>(s2) / (float)a.W;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int c = (k * TPR + col) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) d[k][i] = r * (d[k][i] - s1 - x[k][i] * s2);
      store8(dx + c, a.W - c, d[k]);
    }
  }
  if constexpr (SUMS) {
    // the workgroup's RB rows, one after the other
    __shared__ float red[BWD_NT / 64][2][64 * 8];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < C; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // rows within the wave first
#pragma unroll
        for (int off = TPR; off < 64; off <<= 1) {
          dw[k][i] += __shfl_xor(dw[k][i], off, 64);
          db[k][i] += __shfl_xor(db[k][i], off, 64);
        }
      }
      __syncthreads();
      if (lane < TPR)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          red[wave][0][lane * 8 + i] = dw[k][i];
          red[wave][1][lane * 8 + i] = db[k][i];
        }
      __syncthreads();
      for (int e = threadIdx.x; e < 2 * TPR * 8; e += BWD_NT) {
        const int which = e / (TPR * 8), c = e % (TPR * 8), ch = k * TPR * 8 + c;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < BWD_NT / 64; ++w) s += red[w][which][c];
        if (ch < a.W) a.part[((long long)blockIdx.x * 2 + which) * a.H * a.W + (long long)h * a.W + ch] = s;
      }
    }
  }
}

// dweight and dbias: 64 channels a workgroup, its waves share out the parts.
__global__ __launch_bounds__(1024) void norm_join_kernel(const float *part, int parts, long long width, float *dweight,
                                                         float *dbias) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, which = blockIdx.y;
  const long long ch = (long long)blockIdx.x * 64 + lane;
  float *out = which ? dbias : dweight;
  if (!out) return;
  float s = 0.0f;
  if (ch < width)
#pragma unroll 8
    for (int p = wave; p < parts; p += 16) s += part[((long long)p * 2 + which) * width + ch];
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && ch < width) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += red[w][lane];
    out[ch] = s;
  }
}

// Workgroups of a head: 4096 threads for each of the 256 CUs together, and no more than there are tokens for.
int parts_of(long long tokens, int H, int tpr, int threads) {
  const long long most = rec_cdiv(tokens, threads / tpr), want = std::max<long long>(1, 2048 * BWD_NT / threads / H);
  return (int)std::max<long long>(1, std::min(most, want));
}

int tpr_of(int W) { return W <= 64 ? 8 : W <= 128 ? 16 : W <= 256 ? 32 : 64; }

// Calls f with the row's lanes and chunks as constants.
template <typename F>
hipError_t with_width(int W, F f) {
#define NORM_AT(T, C) return f(std::integral_constant<int, T>{}, std::integral_constant<int, C>{})
  if (W <= 64) NORM_AT(8, 1);
  if (W <= 128) NORM_AT(16, 1);
  if (W <= 256) NORM_AT(32, 1);
  if (W <= 512) NORM_AT(64, 1);
  NORM_AT(64, 2);
#undef NORM_AT
}

ret_status_t check_sizes(int B, int H, int L, int W) {
  if (B <= 0 || H <= 0 || L < 0 || W <= 0) return rec_fail(RET_ERR_INVALID_ARG, "sizes must be positive");
  const long long tokens = (long long)B * L, width = (long long)H * W;
  if (W > LANGUAGE_MAX_NORM_WIDTH || width > LANGUAGE_MAX_CHANNELS || H > 65535 || tokens > LANGUAGE_MAX_TOKENS ||
      (double)tokens * width > (double)LANGUAGE_MAX_ELEMENTS)
    return rec_fail(RET_ERR_UNSUPPORTED, "B, H, L or W too large");
  return RET_OK;
}

// The last element of x that a call reads, counted from its first, + 1.
size_t x_extent(int B, int H, int L, int W, long long sb, long long sh, long long sl) {
  return (size_t)((B - 1) * sb + (H - 1) * sh + (L - 1) * sl + W);
}

ret_status_t check_common(const NormArgs &a, ret_dtype_t in, ret_dtype_t out) {
  const ret_status_t s = check_sizes(a.B, a.H, a.L, a.W);
  if (s != RET_OK) return s;
  if (!rec_dtype_ok(in) || !rec_dtype_ok(out)) return rec_fail(RET_ERR_INVALID_ARG, "unknown dtype");
  if (!(a.eps > 0.0f) || a.eps > 3.4e38f) return rec_fail(RET_ERR_INVALID_ARG, "eps must be finite and above 0");
  if (a.L == 0) return RET_OK;  // strides of nothing
  if ((a.B > 1 && a.x_sb < a.W) || (a.H > 1 && a.x_sh < a.W) || (a.L > 1 && a.x_sl < a.W) || a.x_sb < 0 || a.x_sh < 0 ||
      a.x_sl < 0 || (a.gate && a.gate_ld < (long long)a.H * a.W))
    return rec_fail(RET_ERR_INVALID_ARG, "a stride is shorter than its row");
  if (a.x_sb > LANGUAGE_MAX_ELEMENTS || a.x_sh > LANGUAGE_MAX_ELEMENTS || a.x_sl > (1LL << 31) ||
      a.gate_ld > (1LL << 31) || (double)a.B * (double)a.x_sb > 4.0 * LANGUAGE_MAX_ELEMENTS)
    return rec_fail(RET_ERR_UNSUPPORTED, "a stride is too large");
  return RET_OK;
}

}  // namespace

extern "C" ret_status_t group_norm_gate(const void *x, const void *gate, const float *weight, const float *bias,
                                        void *out, const int *lengths, int B, int H, int L, int W, long long x_sb,
                                        long long x_sh, long long x_sl, long long gate_ld, int silu, float eps,
                                        ret_dtype_t in_dtype, ret_dtype_t out_dtype, void *hip_stream) {
  NormArgs a = {};
  a.x = x, a.gate = gate, a.weight = weight, a.bias = bias, a.out = out, a.lengths = lengths;
  a.x_sb = x_sb, a.x_sh = x_sh, a.x_sl = x_sl, a.gate_ld = gate_ld;
  a.B = B, a.H = H, a.L = L, a.W = W, a.silu = silu, a.eps = eps;
  ret_status_t s = check_common(a, in_dtype, out_dtype);
  if (s != RET_OK) return s;
  if (L == 0) return rec_status(hipSuccess);
  if (!x || !out) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  const size_t ie = rec_esize(in_dtype), oe = rec_esize(out_dtype), width = (size_t)H * W;
  const long long tokens = (long long)B * L;
  if (!rec_aligned(x, ie) || !rec_aligned(gate, ie) || !rec_aligned(weight, 4) || !rec_aligned(bias, 4) ||
      !rec_aligned(out, oe) || !rec_aligned(lengths, 4))
    return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  const RecSpan ins[] = {{"x", x, x_extent(B, H, L, W, x_sb, x_sh, x_sl) * ie},
                         rec_rows("gate", gate, tokens, gate_ld, (long long)width, ie),
                         {"weight", weight, width * 4},
                         {"bias", bias, width * 4},
                         {"lengths", lengths, (size_t)B * 4}};
  const RecSpan outs[] = {{"out", out, (size_t)tokens * width * oe}};
  if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
  a.parts = parts_of(tokens, H, tpr_of(W), NT);
  return rec_status(with_types(in_dtype, out_dtype, [&](auto ti, auto to) {
    return with_width(W, [&](auto tpr, auto chunks) {
      hipLaunchKernelGGL((norm_fwd_kernel<std::remove_pointer_t<decltype(ti)>, std::remove_pointer_t<decltype(to)>,
                                          decltype(tpr)::value, decltype(chunks)::value>),
                         dim3((unsigned)a.parts, (unsigned)H), dim3(NT), 0, (hipStream_t)hip_stream, a);
      return hipGetLastError();
    });
  }));
}

extern "C" size_t group_norm_gate_bwd_workspace_bytes(int B, int H, int L, int W) {
  if (check_sizes(B, H, L, W) != RET_OK || L == 0) return 0;
  return rec_align((size_t)parts_of((long long)B * L, H, tpr_of(W), BWD_NT) * 2 * H * W * 4);
}

extern "C" ret_status_t group_norm_gate_bwd(const void *x, const void *gate, const float *weight, const float *bias,
                                            const void *d_o, const int *lengths, void *dx, void *dgate, float *dweight,
                                            float *dbias, int B, int H, int L, int W, long long x_sb, long long x_sh,
                                            long long x_sl, long long gate_ld, int silu, float eps,
                                            ret_dtype_t in_dtype, ret_dtype_t out_dtype, void *workspace,
                                            size_t workspace_bytes, void *hip_stream) {
  NormArgs a = {};
  a.x = x, a.gate = gate, a.weight = weight, a.bias = bias, a.d_o = d_o, a.lengths = lengths;
  a.dx = dx, a.dgate = dgate, a.part = (float *)workspace;
  a.x_sb = x_sb, a.x_sh = x_sh, a.x_sl = x_sl, a.gate_ld = gate_ld;
  a.B = B, a.H = H, a.L = L, a.W = W, a.silu = silu, a.eps = eps;
  ret_status_t s = check_common(a, in_dtype, out_dtype);
  if (s != RET_OK) return s;
  const size_t ie = rec_esize(in_dtype), oe = rec_esize(out_dtype), width = (size_t)H * W;
  const long long tokens = (long long)B * L;
  const bool sums = dweight || dbias;
  if (L > 0 && (!x || !d_o || !dx || !dgate != !gate)) return rec_fail(RET_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!rec_aligned(x, ie) || !rec_aligned(gate, ie) || !rec_aligned(d_o, ie) || !rec_aligned(weight, 4) ||
      !rec_aligned(bias, 4) || !rec_aligned(dx, oe) || !rec_aligned(dgate, oe) || !rec_aligned(dweight, 4) ||
      !rec_aligned(dbias, 4) || !rec_aligned(lengths, 4))
    return rec_fail(RET_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  a.parts = parts_of(tokens, H, tpr_of(W), BWD_NT);
  const size_t need = sums && L > 0 ? (size_t)a.parts * 2 * width * 4 : 0;
  if (need && (!workspace || workspace_bytes < need))
    return rec_fail(RET_ERR_WORKSPACE, "workspace of %zu bytes needed", need);
  const RecSpan ins[] = {{"x", x, L ? x_extent(B, H, L, W, x_sb, x_sh, x_sl) * ie : 0},
                         rec_rows("gate", gate, tokens, gate_ld, (long long)width, ie),
                         {"weight", weight, width * 4},
                         {"bias", bias, width * 4},
                         {"d_o", d_o, (size_t)tokens * width * ie},
                         {"lengths", lengths, (size_t)B * 4}};
  const RecSpan outs[] = {{"dx", dx, (size_t)tokens * width * oe},
                          {"dgate", dgate, (size_t)tokens * width * oe},
                          {"dweight", dweight, width * 4},
                          {"dbias", dbias, width * 4},
                          {"workspace", workspace, need}};
  if ((s = rec_check_overlap(ins, outs)) != RET_OK) return s;
  if (need && !rec_aligned(workspace, 16)) return rec_fail(RET_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  hipStream_t st = (hipStream_t)hip_stream;
  if (L == 0) a.parts = 0;  // sums of nothing
  return rec_status(with_types(in_dtype, out_dtype, [&](auto ti, auto to) {
    return with_width(W, [&](auto tpr, auto chunks) {
      using TI = std::remove_pointer_t<decltype(ti)>;
      using TO = std::remove_pointer_t<decltype(to)>;
      constexpr int T = decltype(tpr)::value, C = decltype(chunks)::value;
      const dim3 grid((unsigned)a.parts, (unsigned)H);
      if (L > 0) {
        if (sums)
          hipLaunchKernelGGL((norm_bwd_kernel<TI, TO, T, C, true>), grid, dim3(BWD_NT), 0, st, a);
        else
          hipLaunchKernelGGL((norm_bwd_kernel<TI, TO, T, C, false>), grid, dim3(BWD_NT), 0, st, a);
      }
      if (sums)
        hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)rec_cdiv((long long)width, 64), 2), dim3(1024), 0, st,
                           a.part, a.parts, (long long)width, dweight, dbias);
      return hipGetLastError();
    });
  }));
}
