// The tensor maps and the states' images that linattn_api.cu places for the bfloat16 kernels.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <stddef.h>
#include <stdint.h>

namespace linattn {

// q, k, v and do as (size, head, token, batch row); a box is 64 columns of 128 tokens of a head. Columns past
// the size and tokens past T arrive as zeros.
struct Maps {
  CUtensorMap q, k, v, d;
};

// A state as the gradients' products read it: [part][64 keys][64 values], tiles of 64 rows (values).
constexpr uint32_t kImagePiece = 64 * 128;
#ifdef __CUDACC__
__host__ __device__
#endif
constexpr size_t image_bytes(int K, int V) {
  return (size_t)3 * ((K + 63) / 64) * ((V + 63) / 64) * kImagePiece;
}

}  // namespace linattn
