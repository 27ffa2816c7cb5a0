// Internal launch interface of the block norms between their C ABI
// (blocknorm_api.cu) and the kernels (blocknorm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace blocknorm {

constexpr int kMaxD = 8192;
constexpr int kParts = 152 * 4;  // partial rows of the sums over rows: four blocks an SM

struct Args {
  const void *a, *b;     // add: x, residual; gated: o, z
  const float *w, *scale;
  const void *dout, *dh;  // gradients of the output (type of a) and of h (type of b)
  void *out, *h;
  float* rstd;
  void *da, *db;
  float *dw, *dscale, *part;
  long long rows, a_t, b_t;  // rows in all (tokens * H); elements from token to token
  int H, D;
  float eps;
};
// The partial rows a backward writes (its blocks).
int part_rows(long long rows, int D);
cudaError_t launch_add(const Args& p, bool a_bf16, bool b_bf16, bool backward, cudaStream_t s);
cudaError_t launch_gated(const Args& p, bool bf16, bool backward, cudaStream_t s);

}  // namespace blocknorm
