// Entries of the fused linear layers (include/qlinear.h) and the gradient kernel of their
// backward passes.
//
// Forward: one launch, the GEMV kernel with an epilogue or the tensor-core product with one.
// Backward: dz = dy act'(z) (or the gated pair) and the column sums in one pass over the
// activations, then dx = dz W^T on the tensor cores.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "act.cuh"
#include "fused.h"
#include "kernels.cuh"
#include "layout.h"

using namespace qlayout;

namespace {

constexpr int kMaxRows = 1 << 24, kMaxColumns = 1 << 30;
constexpr int kGemvRows = 16;  // the GEMV up to here, the tensor-core product above

bool fmt_ok(int fmt) { return fmt == kW2 || fmt == kW4 || fmt == kW8 || fmt == kLUT4; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool shape_ok(int M, int N, int K) {
  // (the kernels count rows, columns and units in 32 bits)
  return M >= 1 && M <= kMaxRows && N >= kTileN && N <= kMaxColumns && N % kTileN == 0 &&
         K >= kGroup && K <= kMaxColumns && K % kGroup == 0 &&
         (long long)((N + 127) / 128) * (K / kGroup) < (1LL << 31);
}

// ---------------------------------------------------------------------------
// dz and its column sums.
//
// One pass over dy and z (dh, g, u): bound by memory (6 bytes an element, gated 10, read and
// written once).  A thread takes eight consecutive columns as 16-byte vectors, a warp 256
// columns, the eight warps of a block every eighth row of the block's strip; the fp32 sums of
// a column over the strip meet in shared memory, and with more than one strip in the
// workspace, where the last block of a column range to arrive adds the strips in their order.
constexpr int kGradCols = 256, kGradWarps = 8;

struct GradParams {
  const __half* dy;   // [M][W]
  const __half* z;    // linear [M][W] or null (act none); gated [M][2][W]
  __half* dz;         // [M][W]; gated [M][2W] in packed column order; null: not written
  float* dbias;       // [W]; gated [2][W]; or null
  float* partials;    // [strips][W] ([strips][2][W])
  uint32_t* counters; // one per column range
  int M, W, act, rows;  // rows per strip
};

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// From L2: this grid may start before the one that writes the data has ended, and the
// read-only path asks for data that nobody writes during the grid's whole life.
__device__ __forceinline__ uint4 load8(const __half* p) {
  return __ldcg(reinterpret_cast<const uint4*>(p));
}

// d *= act'(z); the activation's branch outside the loop
template <int ACT>
__device__ __forceinline__ void times_gradient_of(float (&d)[8], const float (&z)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float f, df;
    qact::act_both(ACT, z[e], f, df);
    d[e] *= df;
  }
}
__device__ __forceinline__ void times_gradient(int act, float (&d)[8], const float (&z)[8]) {
  switch (act) {
    case QL_ACT_RELU: return times_gradient_of<QL_ACT_RELU>(d, z);
    case QL_ACT_GELU: return times_gradient_of<QL_ACT_GELU>(d, z);
    case QL_ACT_GELU_TANH: return times_gradient_of<QL_ACT_GELU_TANH>(d, z);
    case QL_ACT_SILU: return times_gradient_of<QL_ACT_SILU>(d, z);
    default: return;
  }
}
// dg = dh u act'(g), dh becomes du = dh act(g)
template <int ACT>
__device__ __forceinline__ void gated_gradients_of(float (&dh)[8], const float (&g)[8],
                                                   const float (&u)[8], float (&dg)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float f, df;
    qact::act_both(ACT, g[e], f, df);
    dg[e] = dh[e] * u[e] * df;
    dh[e] *= f;
  }
}
__device__ __forceinline__ void gated_gradients(int act, float (&dh)[8], const float (&g)[8],
                                                const float (&u)[8], float (&dg)[8]) {
  switch (act) {
    case QL_ACT_RELU: return gated_gradients_of<QL_ACT_RELU>(dh, g, u, dg);
    case QL_ACT_GELU: return gated_gradients_of<QL_ACT_GELU>(dh, g, u, dg);
    case QL_ACT_GELU_TANH: return gated_gradients_of<QL_ACT_GELU_TANH>(dh, g, u, dg);
    case QL_ACT_SILU: return gated_gradients_of<QL_ACT_SILU>(dh, g, u, dg);
    default: return gated_gradients_of<QL_ACT_NONE>(dh, g, u, dg);
  }
}

template <bool GATED>
__global__ void __launch_bounds__(32 * kGradWarps, GATED ? 3 : 4) grad_kernel(const GradParams P) {
  constexpr int NB = GATED ? 2 : 1;
  __shared__ float red[NB][kGradWarps][kGradCols];
  __shared__ uint32_t last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.x * kGradCols, c = c0 + 8 * lane;
  const int m0 = blockIdx.y * P.rows;
  const int m1 = m0 + P.rows < P.M ? m0 + P.rows : P.M;
  const bool in = c < P.W;  // W is a multiple of 8: a thread's columns are all in or all out
  float sum[NB][8];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[b][e] = 0.f;
  qlk::grid_dependents_launch();
  qlk::grid_dependency_wait();
  if (in) {
    // kRows rows at a time: their loads are in flight together
    constexpr int kRows = GATED ? 2 : 4;
    for (int mm = m0 + warp; mm < m1; mm += kRows * kGradWarps) {
      uint4 vd[kRows], va[kRows], vb[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int m = mm + i * kGradWarps;
        if (m >= m1) continue;
        const size_t row = (size_t)m * P.W;
        vd[i] = load8(P.dy + row + c);
        if constexpr (GATED) {
          va[i] = load8(P.z + 2 * row + c);
          vb[i] = load8(P.z + 2 * row + P.W + c);
        } else if (P.z) {
          va[i] = load8(P.z + row + c);
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int m = mm + i * kGradWarps;
        if (m >= m1) continue;
        const size_t row = (size_t)m * P.W;
        float d[8], a[8];
        unpack8(vd[i], d);
        if constexpr (GATED) {
          float u[8], dg[8];
          unpack8(va[i], a);
          unpack8(vb[i], u);
          gated_gradients(P.act, d, a, u, dg);  // d becomes du
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            sum[0][e] += dg[e];
            sum[1][e] += d[e];
          }
          // packed order: gate column f at 32 (f / 16) + f % 16, its up column 16 further
          __half* o = P.dz + 2 * row + 32 * (c >> 4) + (c & 15);
          *reinterpret_cast<uint4*>(o) = pack8(dg);
          *reinterpret_cast<uint4*>(o + 16) = pack8(d);
        } else {
          if (P.z) {
            unpack8(va[i], a);
            times_gradient(P.act, d, a);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[0][e] += d[e];
          if (P.dz) *reinterpret_cast<uint4*>(P.dz + row + c) = pack8(d);
        }
      }
    }
  }
  if (!P.dbias) return;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 8; ++e) red[b][warp][8 * lane + e] = sum[b][e];
  __syncthreads();
  const int cc = c0 + threadIdx.x;
  float s[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    s[b] = 0.f;
#pragma unroll
    for (int w = 0; w < kGradWarps; ++w) s[b] += red[b][w][threadIdx.x];
  }
  if (gridDim.y == 1) {
    if (cc < P.W)
#pragma unroll
      for (int b = 0; b < NB; ++b) P.dbias[(size_t)b * P.W + cc] = s[b];
    return;
  }
  if (cc < P.W)
#pragma unroll
    for (int b = 0; b < NB; ++b) P.partials[((size_t)blockIdx.y * NB + b) * P.W + cc] = s[b];
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = qlk::arrive_acq_rel(P.counters + blockIdx.x) + 1 == gridDim.y;
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (cc < P.W)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float t = 0.f;
#pragma unroll 8
      for (unsigned y = 0; y < gridDim.y; ++y)
        t += __ldcg(P.partials + ((size_t)y * NB + b) * P.W + cc);
      P.dbias[(size_t)b * P.W + cc] = t;
    }
  if (threadIdx.x == 0) P.counters[blockIdx.x] = 0u;  // ready for the next call
}

// Rows per strip: 64 (eight a warp), or fewer, down to one a warp, while the blocks do not fill
// the SMs twice; at most kMaxStrips strips are joined.
constexpr int kMaxStrips = 64;
int grad_rows(int M, int W, int sms) {
  const long long cols = (W + kGradCols - 1) / kGradCols;
  const int least = ((M + kMaxStrips - 1) / kMaxStrips + kGradWarps - 1) / kGradWarps * kGradWarps;
  int rows = 64;
  while (rows > kGradWarps && cols * ((M + rows - 1) / rows) < 2LL * sms) rows /= 2;
  return rows > least ? rows : least;
}
int grad_strips(int M, int W, int sms) {
  const int rows = grad_rows(M, W, sms);
  return (M + rows - 1) / rows;
}

// ---------------------------------------------------------------------------
// argument checks

struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.p && b.p && x < y + b.bytes && y < x + a.bytes;
}
// no output overlaps an input or another output
bool disjoint(const Span* outs, int nout, const Span* ins, int nin) {
  for (int i = 0; i < nout; ++i) {
    for (int j = i + 1; j < nout; ++j)
      if (overlap(outs[i], outs[j])) return false;
    for (int j = 0; j < nin; ++j)
      if (overlap(outs[i], ins[j])) return false;
  }
  return true;
}

ql_status check_weights(int fmt, const void* packed, const void* p0, const void* p1) {
  if (!packed || !p0 || !p1) return QL_ERR_NULL;
  if (!aligned(packed, 32) || !aligned(p1, 16) || !aligned(p0, fmt == kLUT4 ? 2 : 16))
    return QL_ERR_ALIGN;
  return QL_OK;
}
size_t packed_size(int fmt, int N, int K) { return qlinear_packed_bytes(fmt, N, K); }
size_t p0_size(int fmt, int N, int K) {
  return fmt == kLUT4 ? 32 : qlinear_params_bytes(fmt, N, K);
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}

// dz follows the partial sums
size_t grad_partial_bytes(int M, int N) {  // bound over every M up to this one
  return (size_t)(M < 64 * kGradWarps ? (M + kGradWarps - 1) / kGradWarps : kMaxStrips) * N *
         sizeof(float);
}
size_t backward_partial_bytes(int M, int N) {
  const size_t a = qfused::tc_partial_bytes(M), b = grad_partial_bytes(M, N);
  return qfused::align_up(a > b ? a : b, 256);
}

// Runs a forward product: the GEMV up to 16 rows, the tensor-core product above.
ql_status forward(qfused::Product& p, void* workspace, size_t workspace_bytes) {
  const size_t off = qfused::partial_offset(p.N);
  if (!workspace || workspace_bytes < off) return QL_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return QL_ERR_ALIGN;
  p.partial_bytes = workspace_bytes - off;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.err = static_cast<uint32_t*>(workspace);
  p.counters = reinterpret_cast<uint32_t*>(
      ws + (p.M <= kGemvRows ? qfused::kVecCounterOffset : qfused::kErrBytes));
  p.partials = reinterpret_cast<float*>(ws + off);
  return p.M <= kGemvRows ? qfused::launch_gemv(p) : qfused::launch_tc(p);
}

template <bool GATED>
ql_status launch_grad(const GradParams& g, int strips, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((g.W + kGradCols - 1) / kGradCols), (unsigned)strips);
  cfg.blockDim = dim3(32 * kGradWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, grad_kernel<GATED>, g) != cudaSuccess) return QL_ERR_CUDA;
  return QL_OK;
}

// dz (unless dy serves as it is) and dbias, then dx = dz W^T.  W: columns of dy.
ql_status backward(qfused::Product& p, const __half* dy, const __half* z, int W, float* dbias,
                   void* workspace, size_t workspace_bytes) {
  const bool gated = p.epi.gated, dz_is_dy = !gated && p.epi.act == QL_ACT_NONE;
  const int sms = sm_count();
  if (sms <= 0) return QL_ERR_CUDA;
  const size_t off = qfused::partial_offset(p.N);
  const size_t part = backward_partial_bytes(p.M, p.N);
  const size_t dz_bytes = dz_is_dy ? 0 : (size_t)p.M * p.N * sizeof(__half);
  if (!workspace || workspace_bytes < off + part + dz_bytes) return QL_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return QL_ERR_ALIGN;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  __half* dz = reinterpret_cast<__half*>(ws + off + part);
  p.err = static_cast<uint32_t*>(workspace);
  p.counters = reinterpret_cast<uint32_t*>(ws + qfused::kErrBytes);
  p.partials = reinterpret_cast<float*>(ws + off);
  p.partial_bytes = part;
  p.x = dz_is_dy ? dy : dz;
  if (!dz_is_dy || dbias) {
    GradParams g;
    g.dy = dy;
    g.z = dz_is_dy ? nullptr : z;
    g.dz = dz_is_dy ? nullptr : dz;
    g.dbias = dbias;
    g.partials = p.partials;
    g.counters = reinterpret_cast<uint32_t*>(ws + qfused::kVecCounterOffset);
    g.M = p.M;
    g.W = W;
    g.act = p.epi.act;
    g.rows = grad_rows(p.M, W, sms);
    const int strips = grad_strips(p.M, W, sms);
    const ql_status s = gated ? launch_grad<true>(g, strips, p.stream)
                              : launch_grad<false>(g, strips, p.stream);
    if (s != QL_OK) return s;
  }
  p.epi.act = QL_ACT_NONE;
  p.epi.gated = 0;
  return qfused::launch_tc(p);
}

}  // namespace

// ---------------------------------------------------------------------------
// exported entry points

extern "C" size_t qlinear_fused_workspace_bytes(int fmt, int M, int N, int K, int backward) {
  if (!fmt_ok(fmt) || !shape_ok(M, N, K)) return 0;
  size_t part = 0;
  for (int m = 1; m <= M && m <= kGemvRows; ++m)
    for (int gated = 0; gated < (N % (2 * kTileN) ? 1 : 2); ++gated) {
      const size_t b = qfused::gemv_partial_bytes(fmt, m, N, K, gated != 0);
      if (!b) return 0;
      if (b > part) part = b;
    }
  if (qfused::tc_partial_bytes(M) > part) part = qfused::tc_partial_bytes(M);
  if (backward) {
    const size_t b = backward_partial_bytes(M, N) + (size_t)M * N * sizeof(__half);
    if (b > part) part = b;
  }
  return qfused::partial_offset(N) + qfused::align_up(part, 256);
}

extern "C" ql_status qlinear_linear(int fmt, const uint16_t* x, const void* packed,
                                    const void* p0, const void* p1, const uint16_t* bias,
                                    const uint16_t* residual, int act, uint16_t* y, uint16_t* z,
                                    int M, int N, int K, void* workspace, size_t workspace_bytes,
                                    ql_stream_t stream) {
  if (!fmt_ok(fmt) || !qact::act_ok(act)) return QL_ERR_UNSUPPORTED;
  if (!x || !y) return QL_ERR_NULL;
  if (!shape_ok(M, N, K)) return QL_ERR_SHAPE;
  if (const ql_status s = check_weights(fmt, packed, p0, p1)) return s;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(z, 16) || !aligned(bias, 16) ||
      !aligned(residual, 16))
    return QL_ERR_ALIGN;
  const size_t mn = (size_t)M * N * 2;
  const Span outs[3] = {{y, mn}, {z, mn}, {workspace, workspace_bytes}};
  const Span ins[6] = {{x, (size_t)M * K * 2}, {bias, (size_t)N * 2},
                       {residual == y ? nullptr : residual, mn},
                       {packed, packed_size(fmt, N, K)}, {p0, p0_size(fmt, N, K)},
                       {p1, qlinear_params_bytes(fmt, N, K)}};
  if (!disjoint(outs, 3, ins, 6)) return QL_ERR_ALIAS;
  qfused::Product p{};
  p.fmt = fmt;
  p.x = reinterpret_cast<const __half*>(x);
  p.packed = packed;
  p.p0 = p0;
  p.p1 = p1;
  p.epi = qfused::Epilogue{reinterpret_cast<const __half*>(bias),
                           reinterpret_cast<const __half*>(residual),
                           reinterpret_cast<__half*>(y), reinterpret_cast<__half*>(z), act, 0};
  p.M = M;
  p.N = N;
  p.K = K;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  return forward(p, workspace, workspace_bytes);
}

extern "C" ql_status qlinear_gated(int fmt, const uint16_t* x, const void* packed, const void* p0,
                                   const void* p1, const uint16_t* bias, int act, uint16_t* h,
                                   uint16_t* gu, int M, int F, int K, void* workspace,
                                   size_t workspace_bytes, ql_stream_t stream) {
  if (!fmt_ok(fmt) || !qact::act_ok(act)) return QL_ERR_UNSUPPORTED;
  if (!x || !h) return QL_ERR_NULL;
  if (F < kTileN || F % kTileN || F > kMaxColumns / 2 || !shape_ok(M, 2 * F, K)) return QL_ERR_SHAPE;
  if (const ql_status s = check_weights(fmt, packed, p0, p1)) return s;
  if (!aligned(x, 16) || !aligned(h, 16) || !aligned(gu, 16) || !aligned(bias, 16))
    return QL_ERR_ALIGN;
  const int N = 2 * F;
  const size_t mf = (size_t)M * F * 2;
  const Span outs[3] = {{h, mf}, {gu, 2 * mf}, {workspace, workspace_bytes}};
  const Span ins[5] = {{x, (size_t)M * K * 2}, {bias, (size_t)N * 2},
                       {packed, packed_size(fmt, N, K)}, {p0, p0_size(fmt, N, K)},
                       {p1, qlinear_params_bytes(fmt, N, K)}};
  if (!disjoint(outs, 3, ins, 5)) return QL_ERR_ALIAS;
  qfused::Product p{};
  p.fmt = fmt;
  p.x = reinterpret_cast<const __half*>(x);
  p.packed = packed;
  p.p0 = p0;
  p.p1 = p1;
  p.epi = qfused::Epilogue{reinterpret_cast<const __half*>(bias), nullptr,
                           reinterpret_cast<__half*>(h), reinterpret_cast<__half*>(gu), act, 1};
  p.M = M;
  p.N = N;
  p.K = K;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  return forward(p, workspace, workspace_bytes);
}

extern "C" ql_status qlinear_linear_backward(int fmt, const uint16_t* dy, const uint16_t* z,
                                             const void* packed, const void* p0, const void* p1,
                                             int act, uint16_t* dx, float* dbias, int M, int N,
                                             int K, void* workspace, size_t workspace_bytes,
                                             ql_stream_t stream) {
  if (!fmt_ok(fmt) || !qact::act_ok(act)) return QL_ERR_UNSUPPORTED;
  if (!dy || !dx || (!z && act != QL_ACT_NONE)) return QL_ERR_NULL;
  if (!shape_ok(M, N, K)) return QL_ERR_SHAPE;
  if (const ql_status s = check_weights(fmt, packed, p0, p1)) return s;
  if (!aligned(dy, 16) || !aligned(z, 16) || !aligned(dx, 16) || !aligned(dbias, 16))
    return QL_ERR_ALIGN;
  const size_t mn = (size_t)M * N * 2;
  const Span outs[3] = {{dx, (size_t)M * K * 2}, {dbias, (size_t)N * 4},
                        {workspace, workspace_bytes}};
  const Span ins[5] = {{dy, mn}, {z, mn}, {packed, packed_size(fmt, N, K)},
                       {p0, p0_size(fmt, N, K)}, {p1, qlinear_params_bytes(fmt, N, K)}};
  if (!disjoint(outs, 3, ins, 5)) return QL_ERR_ALIAS;
  qfused::Product p{};
  p.fmt = fmt;
  p.backward = true;
  p.packed = packed;
  p.p0 = p0;
  p.p1 = p1;
  p.epi = qfused::Epilogue{nullptr, nullptr, reinterpret_cast<__half*>(dx), nullptr, act, 0};
  p.M = M;
  p.N = N;
  p.K = K;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  return backward(p, reinterpret_cast<const __half*>(dy), reinterpret_cast<const __half*>(z), N,
                  dbias, workspace, workspace_bytes);
}

extern "C" ql_status qlinear_gated_backward(int fmt, const uint16_t* dh, const uint16_t* gu,
                                            const void* packed, const void* p0, const void* p1,
                                            int act, uint16_t* dx, float* dbias, int M, int F,
                                            int K, void* workspace, size_t workspace_bytes,
                                            ql_stream_t stream) {
  if (!fmt_ok(fmt) || !qact::act_ok(act)) return QL_ERR_UNSUPPORTED;
  if (!dh || !gu || !dx) return QL_ERR_NULL;
  if (F < kTileN || F % kTileN || F > kMaxColumns / 2 || !shape_ok(M, 2 * F, K)) return QL_ERR_SHAPE;
  if (const ql_status s = check_weights(fmt, packed, p0, p1)) return s;
  if (!aligned(dh, 16) || !aligned(gu, 16) || !aligned(dx, 16) || !aligned(dbias, 16))
    return QL_ERR_ALIGN;
  const int N = 2 * F;
  const size_t mf = (size_t)M * F * 2;
  const Span outs[3] = {{dx, (size_t)M * K * 2}, {dbias, (size_t)N * 4},
                        {workspace, workspace_bytes}};
  const Span ins[5] = {{dh, mf}, {gu, 2 * mf}, {packed, packed_size(fmt, N, K)},
                       {p0, p0_size(fmt, N, K)}, {p1, qlinear_params_bytes(fmt, N, K)}};
  if (!disjoint(outs, 3, ins, 5)) return QL_ERR_ALIAS;
  qfused::Product p{};
  p.fmt = fmt;
  p.backward = true;
  p.packed = packed;
  p.p0 = p0;
  p.p1 = p1;
  p.epi = qfused::Epilogue{nullptr, nullptr, reinterpret_cast<__half*>(dx), nullptr, act, 1};
  p.M = M;
  p.N = N;
  p.K = K;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  return backward(p, reinterpret_cast<const __half*>(dh), reinterpret_cast<const __half*>(gu), F,
                  dbias, workspace, workspace_bytes);
}
