// Sums of partial results over the workgroups that made them (recurrent.hpp).
#include "recurrent.hpp"

namespace ret {

// A workgroup takes COLS columns, its threads' rows run ROWS apart, eight loads ahead.
constexpr int COLS = 32, ROWS = 16;

__global__ __launch_bounds__(COLS * ROWS) void column_sum_kernel(const float *part, float *out, float *last,
                                                                 long long rows, long long cols, int group) {
  __shared__ double red[ROWS][COLS];
  const int c = threadIdx.x % COLS, r0 = threadIdx.x / COLS;
  const long long col = (long long)blockIdx.x * COLS + c;
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
  if (group == 0)
    out[col] = (float)x;
  else if (col % group < group - 1)
    out[col / group * (group - 1) + col % group] = (float)x;
  else if (last)
    last[col / group] = (float)x;
}

hipError_t column_sum(const float *part, float *out, float *last, long long rows, long long cols, int group,
                      hipStream_t st) {
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)rec_cdiv(cols, COLS)), dim3(COLS * ROWS), 0, st, part, out, last,
                     rows, cols, group);
  return hipGetLastError();
}

}  // namespace ret
