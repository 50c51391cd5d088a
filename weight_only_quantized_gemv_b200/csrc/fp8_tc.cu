// Products of e4m3 codes with a scale per 128 (fp8.h): one thread per output, tiles of 32 x 32 in
// shared memory.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8.cuh"
#include "fp8.h"
#include "fused.h"

using namespace qfp8;

namespace {

struct Params {
  const uint8_t *q, *w;
  const float *sx, *sw;
  const int* offsets;
  void* y;
  uint32_t* err;
  int M, N, K, bf16, mtiles;
};

__device__ __forceinline__ float decode(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

constexpr int kTile = 32;

template <bool BWD>
__global__ void __launch_bounds__(kTile* kTile) product_kernel(const Params P) {
  __shared__ float qs[kTile][kTile + 1], ws[kTile][kTile + 1];
  const int C = BWD ? P.N : P.K, R = BWD ? P.K : P.N;
  const int tx = threadIdx.x % kTile, ty = threadIdx.x / kTile;
  const int e = blockIdx.z, r0 = blockIdx.x * kTile;
  // the expert's rows: what comes before the largest offset so far belongs to others
  int lo = 0, hi = P.M;
  if (P.offsets) {
    for (int i = 0; i <= e; ++i) lo = max(lo, min(P.offsets[i], P.M));
    hi = max(lo, min(P.offsets[e + 1], P.M));
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0 &&
        (lo != P.offsets[e] || hi != P.offsets[e + 1]))
      atomicOr(P.err, 4u);
  }
  const int m0 = lo + blockIdx.y * kTile;
  if (m0 >= hi) return;
  const uint8_t* w = P.w + (size_t)e * P.N * P.K;
  const float* sw = P.sw + (size_t)e * blocks_of(P.N) * blocks_of(P.K);
  const int m = m0 + ty, r = r0 + tx;
  float sum = 0.f;
  for (int b = 0; b < blocks_of(C); ++b) {
    float part = 0.f;
    for (int c0 = b * kBlock; c0 < min(C, (b + 1) * kBlock); c0 += kTile) {
      __syncthreads();
      qs[ty][tx] = m < hi && c0 + tx < C ? decode(P.q[(size_t)m * C + c0 + tx]) : 0.f;
      if (BWD)  // ws[c][r]
        ws[ty][tx] = c0 + ty < C && r < R ? decode(w[(size_t)(c0 + ty) * P.K + r]) : 0.f;
      else
        ws[tx][ty] = c0 + tx < C && r0 + ty < R ? decode(w[(size_t)(r0 + ty) * P.K + c0 + tx]) : 0.f;
      __syncthreads();
      for (int i = 0; i < kTile; ++i) part = fmaf(qs[ty][i], ws[i][tx], part);
    }
    if (m < hi && r < R) {
      const int nb = BWD ? b : r / kBlock, kb = BWD ? r / kBlock : b;
      sum = fmaf(part, P.sx[(size_t)m * blocks_of(C) + b] * sw[(size_t)nb * blocks_of(P.K) + kb],
                 sum);
    }
  }
  if (m < hi && r < R) {
    const size_t o = (size_t)m * R + r;
    if (P.bf16)
      static_cast<__nv_bfloat16*>(P.y)[o] = __float2bfloat16_rn(sum);
    else
      static_cast<__half*>(P.y)[o] = __float2half_rn(sum);
  }
}

}  // namespace

namespace qfp8 {

size_t product_partial_bytes(int, int) { return 256; }

ql_status launch_product(const Product& p) {
  Params P{p.q, p.w, p.sx, p.sw, p.offsets, p.y, p.err, p.M, p.N, p.K, p.bf16, 0};
  const int R = p.backward ? p.K : p.N;
  const dim3 grid((R + kTile - 1) / kTile, (p.M + kTile - 1) / kTile, p.E);
  if (grid.y > 65535) return QL_ERR_SHAPE;
  if (p.backward)
    product_kernel<true><<<grid, kTile * kTile, 0, p.stream>>>(P);
  else
    product_kernel<false><<<grid, kTile * kTile, 0, p.stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? QL_OK : QL_ERR_CUDA;
}

}  // namespace qfp8
