// Entries of the fused linear layers (include/qlinear.h) and the gradient kernels of their
// backward passes.
//
// Forward: one launch, the GEMV kernel with an epilogue or the tensor-core product with one.
// Backward: dz = dy act'(z) (or the gated pair), with its column sums where they are asked for,
// then dx = dz W^T on the tensor cores.
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
// dz for the product, and its column sums.
//
// The tensor cores take fp16, whose range gradients leave: dh u act'(g) passes 65504 for ordinary
// values, and unscaled gradients fall below 6e-8.  So a row of dz is multiplied by a power of two,
// and the product's epilogue divides its fp32 sums by it, both without rounding.  It is the one
// that brings the row's largest |dy| (gated: |dh u|, |dh g|) into [2^14, 2^15): |act'| <= 1.13 and
// |act(g)| <= |g|, so nothing overflows, and every element down to 2^-28 of that keeps 11 bits.
// (Rows, because a row of dx contracts one row of dz: nothing of one row shows in another.)
//
// Without column sums one kernel does both, a block to a row.  With them the same kernel only finds
// the factors (kFactor), and a second one with blocks of its own shape, whose columns' sums it
// keeps, writes dz.  Measured, cold: both at once, gated SiLU, 1024 x 14336 33 us for 147 MB
// (4.5 TB/s; blocks of 384 threads that keep three vectors 35); factors of 2048 x 28672 20 us for
// 117 MB (5.8 TB/s), then dz and sums with GELU 111 us for 352 MB, bound by the issue of its
// expf, polynomial and division (94 us with the epilogue's fast forms, which the fp32 sums do not
// get; four blocks an SM and two rows at a time 111, three and four 117); with ReLU, 777 x 12288,
// 7 and 15 us.
constexpr int kDzThreads = 512;
constexpr float kLargest = 3.402823466e38f;
enum { kFactor, kStore };

struct DzParams {
  const __half* dy;  // [M][W]
  const __half* z;   // [M][W]; gated [M][2][W]
  __half* dz;        // [M][W]; gated [M][2W] in packed column order
  uint8_t* unscale;  // [M]: the fp32 exponent field of the factor that undoes a row's scaling
  int W, act;
};

// A thread takes eight consecutive columns as 16-byte vectors, a warp 256 columns, the eight warps
// of a block every eighth row of the block's strip; the fp32 sums of a column over the strip meet
// in shared memory, and with more than one strip in the workspace, where the last block of a
// column range to arrive adds the strips in their order.
constexpr int kGradCols = 256, kGradWarps = 8;

struct GradParams {
  DzParams d;         // z: null without an activation, dz: then null (dy serves as it is)
  float* dbias;       // [W]; gated [2][W]
  float* partials;    // [strips][W] ([strips][2][W])
  uint32_t* counters; // one per column range
  int M, rows;        // rows per strip
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
template <int ACT, bool FAST>
__device__ __forceinline__ void times_gradient_of(float (&d)[8], const float (&z)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float f, df;
    qact::act_both<FAST>(ACT, z[e], f, df);
    d[e] *= df;
  }
}
template <bool FAST>
__device__ __forceinline__ void times_gradient(int act, float (&d)[8], const float (&z)[8]) {
  switch (act) {
    case QL_ACT_RELU: return times_gradient_of<QL_ACT_RELU, FAST>(d, z);
    case QL_ACT_GELU: return times_gradient_of<QL_ACT_GELU, FAST>(d, z);
    case QL_ACT_GELU_TANH: return times_gradient_of<QL_ACT_GELU_TANH, FAST>(d, z);
    case QL_ACT_SILU: return times_gradient_of<QL_ACT_SILU, FAST>(d, z);
    default: return;
  }
}
// dg = dh u act'(g), dh becomes du = dh act(g)
template <int ACT, bool FAST>
__device__ __forceinline__ void gated_gradients_of(float (&dh)[8], const float (&g)[8],
                                                   const float (&u)[8], float (&dg)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float f, df;
    qact::act_both<FAST>(ACT, g[e], f, df);
    dg[e] = dh[e] * u[e] * df;
    dh[e] *= f;
  }
}
template <bool FAST>
__device__ __forceinline__ void gated_gradients(int act, float (&dh)[8], const float (&g)[8],
                                                const float (&u)[8], float (&dg)[8]) {
  switch (act) {
    case QL_ACT_RELU: return gated_gradients_of<QL_ACT_RELU, FAST>(dh, g, u, dg);
    case QL_ACT_GELU: return gated_gradients_of<QL_ACT_GELU, FAST>(dh, g, u, dg);
    case QL_ACT_GELU_TANH: return gated_gradients_of<QL_ACT_GELU_TANH, FAST>(dh, g, u, dg);
    case QL_ACT_SILU: return gated_gradients_of<QL_ACT_SILU, FAST>(dh, g, u, dg);
    default: return gated_gradients_of<QL_ACT_NONE, FAST>(dh, g, u, dg);
  }
}

// Eight columns of a row: dz, or (gated) dg in d[0] and du in d[1].
template <bool GATED>
struct Inputs8 {
  uint4 dy, a, b;  // z; or g, u
};
template <bool GATED>
__device__ __forceinline__ void load_inputs(const __half* dy, const __half* z, size_t row, int W,
                                            int c, Inputs8<GATED>& in) {
  in.dy = load8(dy + row + c);
  if constexpr (GATED) {
    in.a = load8(z + 2 * row + c);
    in.b = load8(z + 2 * row + W + c);
  } else if (z) {
    in.a = load8(z + row + c);
  }
}
template <bool GATED, bool FAST>
__device__ __forceinline__ void gradients8(int act, bool has_z, const Inputs8<GATED>& in,
                                           float (&d)[GATED ? 2 : 1][8]) {
  float a[8];
  if constexpr (GATED) {
    float u[8];
    unpack8(in.dy, d[1]);
    unpack8(in.a, a);
    unpack8(in.b, u);
    gated_gradients<FAST>(act, d[1], a, u, d[0]);  // d[1] becomes du
  } else {
    unpack8(in.dy, d[0]);
    if (has_z) {
      unpack8(in.a, a);
      times_gradient<FAST>(act, d[0], a);
    }
  }
}

// The size that a row's factor goes by, over eight columns: |dy|, or (gated) |dh| max(|g|, |u|).
// Without NaN (fmaxf drops it) and infinities: most make the row's dx not finite, but ReLU has no
// gradient at g = -infinity, and the rest of the row keeps its factor.
template <bool GATED>
__device__ __forceinline__ float size8(const Inputs8<GATED>& in) {
  float d[8], top = 0.f;
  unpack8(in.dy, d);
  if constexpr (GATED) {
    float g[8], u[8];
    unpack8(in.a, g);
    unpack8(in.b, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] *= fmaxf(fabsf(g[e]), fabsf(u[e]));
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(d[e]));
  if (top > kLargest) {
    top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fabsf(d[e]) <= kLargest ? fmaxf(top, fabsf(d[e])) : top;
  }
  return top;
}

// dz of eight columns, each element times `scale`.
template <bool GATED>
__device__ __forceinline__ void store_dz(__half* dz, size_t row, int c, float scale,
                                         const float (&d)[GATED ? 2 : 1][8]) {
  float v[8];
#pragma unroll
  for (int b = 0; b < (GATED ? 2 : 1); ++b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = d[b][e] * scale;
    // packed order: gate column f at 32 (f / 16) + f % 16, its up column 16 further
    __half* o = GATED ? dz + 2 * row + 32 * (size_t)(c >> 4) + (c & 15) + 16 * b : dz + row + c;
    *reinterpret_cast<uint4*>(o) = pack8(v);
  }
}

// A block takes a row.  A thread's first V vectors stay in its registers between the search for
// the row's factor and the stores; what a wide row has beyond them is read again (from L2).
template <bool GATED, int WHAT>
__global__ void __launch_bounds__(kDzThreads, 2) dz_kernel(const DzParams P) {
  constexpr int NB = GATED ? 2 : 1, V = GATED ? 2 : 3;
  __shared__ float red[kDzThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t row = (size_t)blockIdx.x * P.W;
  const int step = 8 * (int)blockDim.x, c0 = 8 * (int)threadIdx.x;  // W is a multiple of 8
  const __half* z = GATED || WHAT == kStore ? P.z : nullptr;  // (a linear factor needs dy alone)
  qlk::grid_dependents_launch();
  qlk::grid_dependency_wait();
  Inputs8<GATED> in[V];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c0 + i * step < P.W) load_inputs<GATED>(P.dy, z, row, P.W, c0 + i * step, in[i]);
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c0 + i * step < P.W) top = fmaxf(top, size8<GATED>(in[i]));
#pragma unroll 4
  for (int c = c0 + V * step; c < P.W; c += step) {
    Inputs8<GATED> more;
    load_inputs<GATED>(P.dy, GATED ? z : nullptr, row, P.W, c, more);
    top = fmaxf(top, size8<GATED>(more));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) red[warp] = top;
  __syncthreads();
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) top = fmaxf(top, red[w]);
  // 2^k (-18 <= k <= 62: sizes are products of at most two fp16); a row of zeros stays as it is
  const int k = top > 0.f ? 14 - ((int)(__float_as_uint(top) >> 23) - 127) : 0;
  if (threadIdx.x == 0) P.unscale[blockIdx.x] = (uint8_t)(127 - k);
  if constexpr (WHAT == kStore) {
    const float scale = __uint_as_float((uint32_t)(127 + k) << 23);
    float d[NB][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c0 + i * step < P.W) {
        gradients8<GATED, true>(P.act, true, in[i], d);
        store_dz<GATED>(P.dz, row, c0 + i * step, scale, d);
      }
#pragma unroll 2
    for (int c = c0 + V * step; c < P.W; c += step) {
      Inputs8<GATED> more;
      load_inputs<GATED>(P.dy, z, row, P.W, c, more);
      gradients8<GATED, true>(P.act, true, more, d);
      store_dz<GATED>(P.dz, row, c, scale, d);
    }
  }
}

template <bool GATED>
__global__ void __launch_bounds__(32 * kGradWarps, GATED ? 3 : 4) grad_kernel(const GradParams P) {
  constexpr int NB = GATED ? 2 : 1;
  __shared__ float red[NB][kGradWarps][kGradCols];
  __shared__ uint32_t last;
  const DzParams& D = P.d;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.x * kGradCols, c = c0 + 8 * lane;
  const int m0 = blockIdx.y * P.rows;
  const int m1 = m0 + P.rows < P.M ? m0 + P.rows : P.M;
  const bool in = c < D.W;  // W is a multiple of 8: a thread's columns are all in or all out
  float sum[NB][8];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[b][e] = 0.f;
  qlk::grid_dependents_launch();
  qlk::grid_dependency_wait();
  if (in) {
    // kRows rows at a time: their loads are in flight together
    constexpr int kRows = 2;
    for (int mm = m0 + warp; mm < m1; mm += kRows * kGradWarps) {
      Inputs8<GATED> in8[kRows];
      uint32_t unscale[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int m = mm + i * kGradWarps;
        if (m >= m1) continue;
        load_inputs<GATED>(D.dy, D.z, (size_t)m * D.W, D.W, c, in8[i]);
        if (D.dz) unscale[i] = __ldcg(D.unscale + m);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int m = mm + i * kGradWarps;
        if (m >= m1) continue;
        float d[NB][8];
        gradients8<GATED, false>(D.act, D.z != nullptr, in8[i], d);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[b][e] += d[b][e];
        if (D.dz)
          store_dz<GATED>(D.dz, (size_t)m * D.W, c, __uint_as_float((254u - unscale[i]) << 23), d);
      }
    }
  }
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
    if (cc < D.W)
#pragma unroll
      for (int b = 0; b < NB; ++b) P.dbias[(size_t)b * D.W + cc] = s[b];
    return;
  }
  if (cc < D.W)
#pragma unroll
    for (int b = 0; b < NB; ++b) P.partials[((size_t)blockIdx.y * NB + b) * D.W + cc] = s[b];
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = qlk::arrive_acq_rel(P.counters + blockIdx.x) + 1 == gridDim.y;
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (cc < D.W)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float t = 0.f;
#pragma unroll 8
      for (unsigned y = 0; y < gridDim.y; ++y)
        t += __ldcg(P.partials + ((size_t)y * NB + b) * D.W + cc);
      P.dbias[(size_t)b * D.W + cc] = t;
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

// A dz block's threads: a vector of eight columns each, up to kDzThreads.
int dz_threads(int W) {
  const int t = (W / 8 + 31) / 32 * 32;
  return t < kDzThreads ? t : kDzThreads;
}

// the rows' exponents and dz follow the partial sums
size_t dz_bytes(int M, int N) {
  return qfused::align_up(M, 256) + (size_t)M * N * sizeof(__half);
}
size_t grad_partial_bytes(int M, int N) {  // bound over every M up to this one
  return (size_t)(M < 64 * kGradWarps ? (M + kGradWarps - 1) / kGradWarps : kMaxStrips) * N *
         sizeof(float);
}
size_t backward_partial_bytes(int M, int N) {
  const size_t a = qfused::tc_partial_bytes(M), b = grad_partial_bytes(M, N);
  return qfused::align_up(a > b ? a : b, 256);
}

// Runs a forward product: the GEMV up to 16 rows if it has a plan, else the tensor-core product.
ql_status forward(qfused::Product& p, void* workspace, size_t workspace_bytes) {
  const size_t off = qfused::partial_offset(p.N);
  if (!workspace || workspace_bytes < off) return QL_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return QL_ERR_ALIGN;
  p.partial_bytes = workspace_bytes - off;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.err = static_cast<uint32_t*>(workspace);
  p.partials = reinterpret_cast<float*>(ws + off);
  if (p.M <= kGemvRows) {
    p.counters = reinterpret_cast<uint32_t*>(ws + qfused::kVecCounterOffset);
    const ql_status s = qfused::launch_gemv(p);
    if (s != QL_ERR_SHAPE) return s;
  }
  p.counters = reinterpret_cast<uint32_t*>(ws + qfused::kErrBytes);
  return qfused::launch_tc(p);
}

template <class Params>
ql_status launch_early(void (*kernel)(Params), dim3 grid, int threads, const Params& p,
                       cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? QL_OK : QL_ERR_CUDA;
}

// dz (unless dy serves as it is) and its column sums (if asked for), then dx = dz W^T.  W: columns
// of dy.
template <bool GATED>
ql_status gradients(const GradParams& g, int sms, cudaStream_t st) {
  const DzParams& d = g.d;
  const int threads = dz_threads(d.W);
  if (!g.dbias) return launch_early(dz_kernel<GATED, kStore>, dim3(g.M), threads, d, st);
  if (d.dz)
    if (const ql_status s =
            launch_early(dz_kernel<GATED, kFactor>, dim3(g.M), threads, d, st))
      return s;
  const dim3 grid((unsigned)((d.W + kGradCols - 1) / kGradCols),
                  (unsigned)grad_strips(g.M, d.W, sms));
  return launch_early(grad_kernel<GATED>, grid, 32 * kGradWarps, g, st);
}

ql_status backward(qfused::Product& p, const __half* dy, const __half* z, int W, float* dbias,
                   void* workspace, size_t workspace_bytes) {
  const bool gated = p.epi.gated, dz_is_dy = !gated && p.epi.act == QL_ACT_NONE;
  const int sms = sm_count();
  if (sms <= 0) return QL_ERR_CUDA;
  const size_t off = qfused::partial_offset(p.N);
  const size_t part = backward_partial_bytes(p.M, p.N);
  if (!workspace || workspace_bytes < off + part + (dz_is_dy ? 0 : dz_bytes(p.M, p.N)))
    return QL_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return QL_ERR_ALIGN;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* unscale = ws + off + part;
  __half* dz = reinterpret_cast<__half*>(unscale + qfused::align_up(p.M, 256));
  p.err = static_cast<uint32_t*>(workspace);
  p.counters = reinterpret_cast<uint32_t*>(ws + qfused::kErrBytes);
  p.partials = reinterpret_cast<float*>(ws + off);
  p.partial_bytes = part;
  p.x = dz_is_dy ? dy : dz;
  p.epi.unscale = dz_is_dy ? nullptr : unscale;
  if (!dz_is_dy || dbias) {
    GradParams g;
    g.d = DzParams{dy, dz_is_dy ? nullptr : z, dz_is_dy ? nullptr : dz, unscale, W, p.epi.act};
    g.dbias = dbias;
    g.partials = p.partials;
    g.counters = reinterpret_cast<uint32_t*>(ws + qfused::kVecCounterOffset);
    g.M = p.M;
    g.rows = grad_rows(p.M, W, sms);
    const ql_status s = gated ? gradients<true>(g, sms, p.stream)
                              : gradients<false>(g, sms, p.stream);
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
      size_t b;
      if (qfused::gemv_partial_bytes(fmt, m, N, K, gated != 0, &b) != QL_OK) return 0;
      if (b > part) part = b;
    }
  if (qfused::tc_partial_bytes(M) > part) part = qfused::tc_partial_bytes(M);
  if (backward) {
    const size_t b = backward_partial_bytes(M, N) + dz_bytes(M, N);
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
                           reinterpret_cast<__half*>(y), reinterpret_cast<__half*>(z),
                           nullptr, act, 0};
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
                           reinterpret_cast<__half*>(h), reinterpret_cast<__half*>(gu),
                           nullptr, act, 1};
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
  p.epi = qfused::Epilogue{nullptr, nullptr, reinterpret_cast<__half*>(dx), nullptr, nullptr,
                           act, 0};
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
  p.epi = qfused::Epilogue{nullptr, nullptr, reinterpret_cast<__half*>(dx), nullptr, nullptr,
                           act, 1};
  p.M = M;
  p.N = N;
  p.K = K;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  return backward(p, reinterpret_cast<const __half*>(dh), reinterpret_cast<const __half*>(gu), F,
                  dbias, workspace, workspace_bytes);
}
