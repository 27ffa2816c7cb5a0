// Internal launch interface of the norms of queries and keys with the position
// rotation between their C ABI (qkrope_api.cu) and the kernels (qkrope.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qkrope {

constexpr int kMaxD = 256;
constexpr int kSms = 152;        // of the GPU that plans go by
constexpr int kParts = kSms * 2;  // partial rows of the weights' gradients: two blocks an SM

struct Args {
  const void *q, *k;
  const float *wq, *wk;
  const double* freq;
  const int* positions;
  const void *dqo, *dko;
  void *qo, *ko;      // the outputs, or q's and k's gradients
  float *dwq, *dwk, *part;
  long long q_t, k_t, rows, T;  // elements from token to token; tokens * (Hq + Hk)
  int Hq, Hk, D, half, interleaved;
  float eps;
};
// The partial rows a backward writes (its blocks).
int part_rows(long long rows);
cudaError_t launch(const Args& p, bool bf16, bool backward, cudaStream_t s);

}  // namespace qkrope
