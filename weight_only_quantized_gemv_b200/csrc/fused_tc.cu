// Products of the fused linear layers with the epilogue (fused.h), for every format, direction
// and size.  A block computes 32 tokens x one 128-column block of the weights (forward) or one
// 128-k group (backward), decoding one 128 x 128 unit of weights at a time into shared memory;
// sums in fp32.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "act.cuh"
#include "dequant_frag.cuh"
#include "fused.h"
#include "kernels.cuh"
#include "layout.h"

using namespace qlayout;

namespace {

constexpr int kTok = 32;

struct PlainParams {
  const __half* x;
  const uint8_t* qw;
  const void* p0;
  const void* p1;
  qfused::Epilogue epi;
  int M, N, K, G, ntiles;
  bool backward;
};

// row r (packed column), k granule of the unit (b, g): eight fp16 weights
template <int FMT>
__device__ void decode_unit(const PlainParams& P, int b, int g, int warp, int lane,
                            const float* lut, __half (*w)[kGroup + 8]) {
  const int gi = lane >> 2, t = lane & 3;
  constexpr int KW = qlk::Fmt<FMT>::kWords;
  const bool in = warp < tiles_in_block(b, P.ntiles);
  uint32_t words[KW];
  __half2 zb[2][2], s2 = __float2half2_rn(0.f);
  float4 am = make_float4(0.f, 0.f, 0.f, 0.f);
  if (in) {
    const long long ch = chunk_index(b, g, warp, P.G, P.ntiles);
    const uint32_t* src = reinterpret_cast<const uint32_t*>(P.qw + ch * chunk_bytes(FMT));
#pragma unroll
    for (int i = 0; i < KW; ++i) words[i] = src[word_index(i, lane)];
    if constexpr (FMT == kLUT4) {
      am = *reinterpret_cast<const float4*>(static_cast<const float*>(P.p1) + ch * 32 + gi * 4);
    } else {
      s2 = *reinterpret_cast<const __half2*>(static_cast<const __half*>(P.p0) + ch * 16 + gi * 2);
      const __half2 z2 =
          *reinterpret_cast<const __half2*>(static_cast<const __half*>(P.p1) + ch * 16 + gi * 2);
      qdq::zero_bias<FMT>(__low2float(z2), __high2float(z2), zb);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (in) {
        if constexpr (FMT == kLUT4)
          v = qdq::lut_pair8(words, 2 * i, h, lut,
                             i >= 2 ? (h ? am.w : am.z) : (h ? am.y : am.x));
        else
          v = qdq::uniform_pair8<FMT>(words, 2 * i, h, zb, h ? __high2half2(s2) : __low2half2(s2));
      }
      *reinterpret_cast<uint4*>(&w[16 * warp + gi + 8 * h][32 * i + 8 * t]) = v;
    }
}

template <int FMT>
__global__ void __launch_bounds__(256) plain_kernel(const PlainParams P) {
  __shared__ __align__(16) __half w[128][kGroup + 8];
  __shared__ __half xs[kTok][kGroup];
  __shared__ float lut[16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (FMT == kLUT4 && tid < 16) lut[tid] = __half2float(static_cast<const __half*>(P.p0)[tid]);
  __syncthreads();
  const int out = blockIdx.x;                 // block (forward) or group (backward)
  const int m0 = blockIdx.y * kTok;
  const int nblocks = (P.ntiles + kBlockTiles - 1) / kBlockTiles;
  const int steps = P.backward ? nblocks : P.G;
  const int width = P.backward ? P.N : P.K;   // columns of x
  // thread: outputs r = 32 j + lane (j < 4), tokens warp + 8 i (i < 4)
  float acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  for (int st = 0; st < steps; ++st) {
    const int b = P.backward ? st : out, g = P.backward ? out : st;
    decode_unit<FMT>(P, b, g, warp, lane, lut, w);
    for (int e = tid; e < kTok * kGroup; e += 256) {
      const int m = m0 + e / kGroup, c = st * kGroup + e % kGroup;
      xs[e / kGroup][e % kGroup] =
          (m < P.M && c < width) ? P.x[(size_t)m * width + c] : __float2half(0.f);
    }
    __syncthreads();
    for (int c = 0; c < kGroup; ++c) {
      float wv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        wv[j] = __half2float(P.backward ? w[c][32 * j + lane] : w[32 * j + lane][c]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float xv = __half2float(xs[warp + 8 * i][c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xv, wv[j], acc[i][j]);
      }
    }
    __syncthreads();
  }
  const qfused::Epilogue& E = P.epi;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + warp + 8 * i;
    if (m >= P.M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = out * 128 + 32 * j + lane;
      float z = acc[i][j];
      if (P.backward) {
        E.y[(size_t)m * P.K + r] = __float2half_rn(z);
      } else if (E.gated) {
        // packed column r: tile r / 16, even = gate; the partner sits 16 lanes away
        const int F = P.N / 2, f = (r >> 5) * 16 + (r & 15), up = (r >> 4) & 1;
        const bool ok = r < P.N;
        if (ok && E.bias) z += __half2float(E.bias[up * F + f]);
        const float other = __shfl_xor_sync(0xffffffffu, z, 16);
        if (ok && E.zsave) E.zsave[((size_t)m * 2 + up) * F + f] = __float2half_rn(z);
        if (ok && !up) E.y[(size_t)m * F + f] = __float2half_rn(qact::act_forward(E.act, z) * other);
      } else if (r < P.N) {
        if (E.bias) z += __half2float(E.bias[r]);
        const size_t o = (size_t)m * P.N + r;
        if (E.zsave) E.zsave[o] = __float2half_rn(z);
        float y = qact::act_forward(E.act, z);
        if (E.residual) y += __half2float(E.residual[o]);
        E.y[o] = __float2half_rn(y);
      }
    }
  }
}

}  // namespace

namespace qfused {

size_t tc_partial_bytes(int) { return 256; }

ql_status launch_tc(const Product& p) {
  PlainParams P{p.x, static_cast<const uint8_t*>(p.packed), p.p0, p.p1, p.epi, p.M, p.N, p.K,
                p.K / kGroup, p.N / kTileN, p.backward};
  const dim3 grid((unsigned)(p.backward ? P.G : (P.ntiles + 7) / 8),
                  (unsigned)((p.M + kTok - 1) / kTok));
  switch (p.fmt) {
    case kW2: plain_kernel<kW2><<<grid, 256, 0, p.stream>>>(P); break;
    case kW4: plain_kernel<kW4><<<grid, 256, 0, p.stream>>>(P); break;
    case kW8: plain_kernel<kW8><<<grid, 256, 0, p.stream>>>(P); break;
    default: plain_kernel<kLUT4><<<grid, 256, 0, p.stream>>>(P); break;
  }
  return cudaGetLastError() == cudaSuccess ? QL_OK : QL_ERR_CUDA;
}

}  // namespace qfused
