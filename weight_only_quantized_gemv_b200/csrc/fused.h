// Internal interfaces of the fused linear layers (fused.cu: entries, gradient kernel;
// fused_tc.cu: tensor-core products; qlinear.cu: GEMV with an epilogue).
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "qlinear.h"

namespace qfused {

// What happens to an output element z (fp32) of the forward products, bias added first:
//   linear: y = act(z) + residual, z kept if zsave
//   gated : the packed columns alternate 16 gate / 16 up; h = act(g) u, (g, u) kept if zsave
// The backward products store dx = the sum, times the row's power of two if dz was scaled
// (unscale[m]: the exponent field of that fp32 power; readable up to a multiple of 8 rows).
struct Epilogue {
  const __half* bias;      // linear [N]; gated [2][F]; or null
  const __half* residual;  // [M][N] or null (linear)
  __half* y;               // [M][N], gated [M][F], backward [M][K]
  __half* zsave;           // [M][N], gated [M][2][F], or null
  const uint8_t* unscale;  // backward: [M], or null
  int act;
  int gated;
};

// y[m][n] = sum_k x[m][k] W[n][k] (forward), or y[m][k] = sum_n x[m][n] W[n][k] (backward: x
// holds dz, its columns in packed order), then the epilogue.
struct Product {
  int fmt;
  bool backward;
  const __half* x;
  const void* packed;
  const void* p0;
  const void* p1;
  Epilogue epi;
  int M, N, K;
  uint32_t* err;        // sticky wait flags
  uint32_t* counters;   // arrivals, zero between calls
  float* partials;
  size_t partial_bytes;  // room at partials (QL_ERR_WORKSPACE if it is too little)
  cudaStream_t stream;
};

// Workspace: one layout for every entry and shape, so that calls of different layers may share
// one (the counters of any call sit where every other call's counters sit, never under its
// partial sums).
constexpr size_t kErrBytes = 256;
constexpr size_t kTcCounterBytes = 16384 - kErrBytes;     // tensor-core products
constexpr size_t kVecCounterOffset = 16384;               // GEMV, column sums
constexpr size_t kVecCounterBytes = 65536;                // grown for N > 524288
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline size_t vec_counter_bytes(int N) {
  const size_t need = ((size_t)N + 127) / 128 * 16;
  return need > kVecCounterBytes ? align_up(need, 256) : kVecCounterBytes;
}
inline size_t partial_offset(int N) { return kVecCounterOffset + vec_counter_bytes(N); }

// tensor-core products (fused_tc.cu)
ql_status launch_tc(const Product& p);
size_t tc_partial_bytes(int M);  // bound over every call with at most M rows

// Limit of a barrier wait of the tensor-core products and the delays of qlinear_debug_wait_test:
// worker 0's copies of the activations (low half) and its first MMA (high half).
struct WaitTest {
  uint32_t limit_us, delays;
};
WaitTest wait_test();

// GEMV with an epilogue (qlinear.cu), M <= 16.  QL_ERR_SHAPE and 0 bytes: it has no plan for the
// shape (its unit arithmetic is 32-bit), which then is the tensor-core product's.
ql_status launch_gemv(const Product& p);
ql_status gemv_partial_bytes(int fmt, int M, int N, int K, bool gated, size_t* bytes);

}  // namespace qfused
