// Internal interface of the products of 8-bit floating-point codes (fp8.cu: entries; fp8_tc.cu:
// the kernel).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "qlinear.h"

namespace qfp8 {

// D[row][m] = sum_b sx[m][b] sw[..] sum_{i in block b} W . q[m][i] over the rows m of every expert:
//   forward   rows n, sum over k;   backward   rows k, sum over n
// of W [E][N][K], sw [E][N / 128][K / 128].
struct Product {
  bool bf16, backward;
  const uint8_t* q;        // [M][K] (backward [M][N])
  const float* sx;         // [M][blocks]
  const int* offsets;      // [E + 1] on the device, or null: one expert, all rows
  const uint8_t* w;
  const float* sw;
  void* y;                 // [M][N] (backward [M][K])
  int M, E, N, K;
  uint32_t* err;           // sticky flags
  uint32_t* counters;      // arrivals, zero between calls
  float* partials;
  size_t partial_bytes;
  cudaStream_t stream;
};

constexpr int kMaxExperts = 1024;

ql_status launch_product(const Product& p);
size_t product_partial_bytes(int M, int E);  // bound over every call with at most M rows

}  // namespace qfp8
