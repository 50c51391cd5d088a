// Entries of the 8-bit floating-point path (include/qlinear.h) and its kernels over rows: RMS norm,
// gated activation and plain quantization with e4m3 output, and their backward passes.  The
// products are in fp8_tc.cu.
//
// All of them are bound by memory: they read and write each element once, as 16-byte vectors of
// eight columns (8 bytes of codes), and a block's scale is a maximum over sixteen lanes.
#include <cuda_runtime.h>
#include <stdint.h>

#include "act.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "fused.h"
#include "kernels.cuh"

using namespace qfp8;

namespace {

constexpr int kMaxRows = 1 << 24, kMaxColumns = 1 << 30;
constexpr int kMaxNorm = 32768;  // columns of a norm: 1024 threads of four vectors

// From L2: a grid may start before the one that writes its input has ended, and the read-only
// path asks for data that nobody writes during the grid's whole life.
__device__ __forceinline__ uint4 load16(const void* p) {
  return __ldcg(reinterpret_cast<const uint4*>(p));
}

// 16 bytes into shared memory, past L1.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The sum over a group of whole warps, in every one of its threads; `red` has a word per warp and
// two of them are used in turn, `barrier` is the group's own (0: the block is the group).
__device__ __forceinline__ float group_sum(float v, float (&red)[32], int tid, int threads,
                                           int barrier) {
  const int lane = tid & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) red[tid >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(threads) : "memory");
  v = lane < threads >> 5 ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------------------
// RMS norm

struct NormParams {
  const uint16_t* x;         // rows ldx apart
  const uint16_t* residual;  // [M][K] or null
  const uint16_t* weight;    // [K]
  uint16_t* total;           // [M][K] or null
  uint16_t* y;               // [M][K] or null
  uint8_t* q;                // [M][K] or null
  float* scales;             // [M][blocks]
  float* rstd;               // [M] or null
  long long ldx;
  float eps;
  int M, K;
};

// A block takes a row; a thread keeps its V vectors in registers between the sum of squares and the
// output, so that the row is read once.  Measured, cold, bf16, with residual, total, y and codes:
// 4096 x 8192 47.4 us for 302 MB (6.4 TB/s, 97 % of a copy's rate); with V = 4, where 48 bytes
// spill, 4096 x 12288 74.3 us, 16384 93.2 us and 32768 200 us (6.1, 6.5 and 6.1 TB/s).
template <bool BF16, int V>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams P) {
  __shared__ float red[32];
  const int row = blockIdx.x, step = 8 * (int)blockDim.x, c0 = 8 * (int)threadIdx.x;
  const size_t base = (size_t)row * P.K;
  qlk::grid_dependents_launch();
  qlk::grid_dependency_wait();
  // (the weight too: it is trained, by work that may be the stream's last before this)
  uint4 a[V], r[V], w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = c0 + i * step;
    if (c >= P.K) continue;
    a[i] = load16(P.x + (size_t)row * P.ldx + c);
    if (P.residual) r[i] = load16(P.residual + base + c);
    w[i] = load16(P.weight + c);
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = c0 + i * step;
    if (c >= P.K) continue;
    float t[8];
    unpack8<BF16>(a[i], t);
    if (P.residual) {
      float u[8];
      unpack8<BF16>(r[i], u);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] += u[e];
      a[i] = pack8<BF16>(t);  // the stream as it is stored: what follows goes by it
      unpack8<BF16>(a[i], t);
    }
    if (P.total) *reinterpret_cast<uint4*>(P.total + base + c) = a[i];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(t[e], t[e], sum);
  }
  const float rstd = rsqrtf(group_sum(sum, red, threadIdx.x, blockDim.x, 0) / (float)P.K + P.eps);
  if (P.rstd && threadIdx.x == 0) P.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = c0 + i * step;
    float t[8] = {};
    if (c < P.K) {
      float g[8];
      unpack8<BF16>(a[i], t);
      unpack8<BF16>(w[i], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = t[e] * rstd * g[e];
      if (P.y) *reinterpret_cast<uint4*>(P.y + base + c) = pack8<BF16>(t);
    }
    if (P.q) {
      const float scale = scale_of(top_of_block(top8(t)));
      if (c < P.K) {
        *reinterpret_cast<uint2*>(P.q + base + c) = encode8(t, scale);
        if ((threadIdx.x & 15) == 0) P.scales[(size_t)row * blocks_of(P.K) + c / kBlock] = scale;
      }
    }
  }
}

struct NormGradParams {
  const uint16_t* dy;      // [M][K]
  const uint16_t* total;   // [M][K]
  const float* rstd;       // [M]
  const uint16_t* weight;  // [K]
  const uint16_t* dtotal;  // [M][K] or null
  const int* offsets;      // PART, [E + 1]: rows outside of offsets[0] .. offsets[E] have no dy
  uint16_t* dx;            // [M][K]
  float* partials;         // [blocks][K] or null: sums of dy t rstd over a block's rows
  int M, E, K, threads;    // threads of a group
};

// A block is up to eight groups of P.threads threads.  A group takes a row at a time and keeps the
// sums of the columns in registers; the groups' meet at the end, so that a block leaves one set of
// sums.  A thread copies its own vectors of the S - 1 rows ahead into shared memory (no other
// thread reads them), since the wait for a row's sum leaves no other way to keep enough loads under
// way.  Measured, cold, bf16, with dtotal and dweight: 4096 x 8192 54.7 us (4.9 TB/s), 2047 x 8192
// 32.6 us (4.1), 700 x 14336 25.7 us (3.1), the join among them: the passes between a row's
// arrival and its barrier, which issue in 60 % of the slots.  (Addresses in 64 bits took 57.6 us,
// 34.2 and 28.8.)  V = 4 spills 104 to 120 bytes: 1024 x 20480 66.2 us, 1024 x 32768 86.5 us.
//
// PART: rows may be without a dy (of no expert: nobody wrote it).  Such a row adds to no sum, and
// its dx is dtotal, or 0.  (An instance of its own: the tests of rows cost the others 1 to 2 %.)
template <bool BF16, bool PART, int V, int S>
__global__ void __launch_bounds__(1024) norm_grad_kernel(const NormGradParams P) {
  extern __shared__ __align__(16) uint4 stages[];  // [group][S][array][V][thread]; then the sums
  __shared__ float red[8][2][32];
  const int threads = P.threads, groups = (int)blockDim.x / threads;
  const int group = (int)threadIdx.x / threads, tid = (int)threadIdx.x - group * threads;
  const int step = 8 * threads, c0 = 8 * tid;
  const int arrays = P.dtotal ? 3 : 2;
  const int hop = V * threads, stage = arrays * hop;  // vectors
  const uint32_t mine = qlk::smem_addr(stages + group * S * stage + tid);
  uint4 w[V];
  float dw[V][8] = {};
  qlk::grid_dependents_launch();
  qlk::grid_dependency_wait();
  int lo = 0, hi = P.M;
  if constexpr (PART) {
    lo = max(__ldcg(P.offsets), 0);
    hi = min(__ldcg(P.offsets + P.E), P.M);
  }
  auto has_dy = [&](int row) { return !PART || (row >= lo && row < hi); };
  auto copy = [&](int row, int s) {
    if (row < P.M) {
      const bool own = has_dy(row);
      const size_t at = (size_t)row * P.K + c0;
      const uint32_t o = mine + 16 * s * stage;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c0 + i * step < P.K) {
          if (own) {
            copy16(o + 16 * i * threads, P.total + at + i * step);
            copy16(o + 16 * (i * threads + hop), P.dy + at + i * step);
          }
          if (P.dtotal) copy16(o + 16 * (i * threads + 2 * hop), P.dtotal + at + i * step);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int rows = (int)gridDim.x * groups;
  int row = (int)blockIdx.x * groups + group;
#pragma unroll
  for (int s = 0; s < S - 1; ++s) copy(row + s * rows, s);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    w[i] = make_uint4(0, 0, 0, 0);
    if (c0 + i * step < P.K) w[i] = load16(P.weight + c0 + i * step);
  }
  for (int s = 0, half = 0; row < P.M; row += rows, half ^= 1) {
    copy(row + (S - 1) * rows, s + S - 1 < S ? s + S - 1 : s - 1);
    const float rstd = __ldcg(P.rstd + row);
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    const uint32_t x = mine + 16 * s * stage;
    if (!has_dy(row)) {  // for the whole group, which uses neither its barrier nor this half
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c0 + i * step < P.K) {
          uint4 t = make_uint4(0, 0, 0, 0);
          if (P.dtotal) t = qlk::lds128(x + 16 * (i * threads + 2 * hop));
          *reinterpret_cast<uint4*>(P.dx + (size_t)row * P.K + c0 + i * step) = t;
        }
      s = s + 1 < S ? s + 1 : 0;
      half ^= 1;
      continue;
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (c0 + i * step >= P.K) continue;
      float t[8], g[8], v[8];
      unpack8<BF16>(qlk::lds128(x + 16 * i * threads), t);
      unpack8<BF16>(qlk::lds128(x + 16 * (i * threads + hop)), g);
      unpack8<BF16>(w[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = t[e] * rstd;
        sum = fmaf(g[e] * v[e], n, sum);
        dw[i][e] = fmaf(g[e], n, dw[i][e]);
      }
    }
    const float mean = group_sum(sum, red[group][half], tid, threads, 1 + group) / (float)P.K;
    const float back = -rstd * mean;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = c0 + i * step;
      if (c >= P.K) continue;
      float t[8], g[8], v[8];
      unpack8<BF16>(qlk::lds128(x + 16 * i * threads), t);
      unpack8<BF16>(qlk::lds128(x + 16 * (i * threads + hop)), g);
      unpack8<BF16>(w[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = rstd * fmaf(g[e], v[e], back * t[e]);
      if (P.dtotal) {
        unpack8<BF16>(qlk::lds128(x + 16 * (i * threads + 2 * hop)), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] += g[e];
      }
      *reinterpret_cast<uint4*>(P.dx + (size_t)row * P.K + c) = pack8<BF16>(t);
    }
    s = s + 1 < S ? s + 1 : 0;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (!P.partials) return;
  // the groups' sums, added in their order: [group - 1][V][2][thread]
  float4* const sums = reinterpret_cast<float4*>(stages) + tid;
  if (groups > 1) {
    __syncthreads();
    if (group > 0)
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) {
        const float* d = &dw[i >> 1][4 * (i & 1)];
        sums[(group - 1) * 2 * hop + i * threads] = make_float4(d[0], d[1], d[2], d[3]);
      }
    __syncthreads();
    if (group > 0) return;
  }
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) {
    const float* d = &dw[i >> 1][4 * (i & 1)];
    float4 t = make_float4(d[0], d[1], d[2], d[3]);
    for (int g = 1; g < groups; ++g) {
      const float4 o = sums[(g - 1) * 2 * hop + i * threads];
      t.x += o.x;
      t.y += o.y;
      t.z += o.z;
      t.w += o.w;
    }
    const int c = c0 + (i >> 1) * step + 4 * (i & 1);
    if (c < P.K) *reinterpret_cast<float4*>(P.partials + (size_t)blockIdx.x * P.K + c) = t;
  }
}

// dweight[c] = the blocks' sums, added in a fixed order: warp w of a block takes every W-th, its
// lanes the columns, and they meet in shared memory.  W is 32 while the blocks are one wave of two
// to an SM, above that 16.  Measured, with the gradients before it, us of 32 and of 16: 2047 x 8192
// 32.6 and 33.3, 700 x 14336 27.0 and 25.7; without the weight's sums 28.3 and 20.2.
template <int W>
__global__ void __launch_bounds__(32 * W) norm_join_kernel(const float* partials, float* dweight,
                                                           int blocks, int K) {
  __shared__ float red[W][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = 32 * blockIdx.x + lane;
  qlk::grid_dependents_launch();
  qlk::grid_dependency_wait();
  float s = 0.f;
  if (c < K)
#pragma unroll 5
    for (int b = warp; b < blocks; b += W) s += __ldcg(partials + (size_t)b * K + c);
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < K) {
#pragma unroll
    for (int w = 1; w < W; ++w) s += red[w][lane];
    dweight[c] = s;
  }
}

// ---------------------------------------------------------------------------
// quantization of rows: of x, of act(g) u, or of the gated pair's gradients.
//
// The gradients of a pair have their codes F columns apart.  Where F is a multiple of 128 both lie
// at the same place of their blocks and a thread makes both (kPair); where it is not, a thread
// makes one and the inputs are read twice (kGatedGrad).

enum { kPlain, kGated, kGatedGrad, kPair };

struct CodeParams {
  const uint16_t* x;   // kPlain: rows ldx apart; else gu [M][2 F]
  const uint16_t* dh;  // gradients: [M][F]
  uint8_t* q;          // [M][C]
  float* scales;       // [M][blocks of C]
  long long ldx;
  int M, C, F, act;    // C columns of output: K, F, 2 F
  int slots;           // vectors of eight columns in a row, whole blocks of sixteen (kPair: of F)
  float inv_slots;     // 1 / slots
};

constexpr int kCodeThreads = 256;

template <int WHAT>
struct Inputs {
  uint4 a, b, c;  // x; or g, u; and dh
};
template <int WHAT>
__device__ __forceinline__ void load_inputs(const CodeParams& P, int row, int c,
                                            Inputs<WHAT>& in) {
  if constexpr (WHAT == kPlain) {
    in.a = load16(P.x + (size_t)row * P.ldx + c);
  } else {
    const int f = WHAT == kGatedGrad && c >= P.F ? c - P.F : c;
    const uint16_t* gu = P.x + (size_t)row * 2 * P.F + f;
    in.a = load16(gu);
    in.b = load16(gu + P.F);
    if constexpr (WHAT != kGated) in.c = load16(P.dh + (size_t)row * P.F + f);
  }
}
// The activation, and with it the derivative, from the sigmoid with the short exponential and
// reciprocal: the values are coded in 8 bits.  (Where e^-x leaves the normal numbers the sigmoid is
// 0 or 1; x times what is lost is below 2^-119.)
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == QL_ACT_SILU) {
    return z * rcp_fast(1.f + exp2_fast(z * -1.44269504f));
  } else {
    return qact::act_forward(ACT, z);
  }
}
template <int ACT>
__device__ __forceinline__ void act_pair(float z, float& f, float& df) {
  if constexpr (ACT == QL_ACT_SILU) {
    const float e = exp2_fast(fabsf(z) * -1.44269504f), r = rcp_fast(1.f + e), er = e * r;
    const float s = z < 0.f ? er : r, c = z < 0.f ? r : er;  // sigma(z), 1 - sigma(z)
    f = z * s;
    df = fmaf(f, c, s);
  } else {
    qact::act_both<true>(ACT, z, f, df);
  }
}

// v: the values to code (kPair: dg, and du in w)
template <int WHAT, bool BF16, int ACT>
__device__ __forceinline__ void code_values(const Inputs<WHAT>& in, bool second, float (&v)[8],
                                            float (&w)[8]) {
  unpack8<BF16>(in.a, v);
  if constexpr (WHAT == kPlain) return;
  float u[8];
  unpack8<BF16>(in.b, u);
  if constexpr (WHAT == kGated) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = act_value<ACT>(v[e]) * u[e];
  } else {
    float d[8];
    unpack8<BF16>(in.c, d);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float y, dy;
      act_pair<ACT>(v[e], y, dy);
      const float dg = d[e] * u[e] * dy, du = d[e] * y;
      v[e] = WHAT == kGatedGrad && second ? du : dg;
      w[e] = du;
    }
  }
}
// The whole warp: sixteen lanes to a block, `in`: the lane's vector lies within its row.
__device__ __forceinline__ void store_codes(const CodeParams& P, bool in, int row, int c,
                                            const float (&v)[8], uint32_t top) {
  const float scale = scale_of(top_of_block(top));
  if (in) {
    *reinterpret_cast<uint2*>(P.q + (size_t)row * P.C + c) = encode8(v, scale);
    if ((threadIdx.x & 15) == 0) P.scales[(size_t)row * blocks_of(P.C) + c / kBlock] = scale;
  }
}

// U vectors to a thread: all of their loads are under way before the first is used.  Measured,
// cold, bf16, 1024 x 14336: plain 10.1 us for 44 MB (4.3 TB/s), gated SiLU 14.6 us for 73 MB (5.0),
// its gradients 24.9 us for 117 MB (4.7): bound by issue (80 % of the slots), GELU more so (22.9
// and 30.8 us).  A thread to one gradient took 38 us, a 64-bit division for a vector's row 5 us
// more.
template <int WHAT, bool BF16, int ACT, int U>
__global__ void __launch_bounds__(kCodeThreads) code_kernel(const CodeParams P) {
  qlk::grid_dependents_launch();
  qlk::grid_dependency_wait();
  constexpr int kStep = kCodeThreads * U;
  const long long n = (long long)P.M * P.slots;
  for (long long base = (long long)blockIdx.x * kStep; base < n;
       base += (long long)gridDim.x * kStep) {
    // (a 64-bit division costs as much as coding a vector)
    const int row0 = n >> 32 ? (int)(base / P.slots) : (int)((unsigned)base / (unsigned)P.slots);
    const int at0 = (int)(base - (long long)row0 * P.slots) + (int)threadIdx.x;
    int row[U], c[U];
    bool in[U];
    Inputs<WHAT> x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      // the quotient by the reciprocal is at most one off (at < 2 slots + 512)
      const int at = at0 + i * kCodeThreads;
      int r = __float2int_rz(__int2float_rn(at) * P.inv_slots), rest = at - r * P.slots;
      if (rest < 0) {
        --r;
        rest += P.slots;
      } else if (rest >= P.slots) {
        ++r;
        rest -= P.slots;
      }
      row[i] = row0 + r;
      c[i] = 8 * rest;
      in[i] = row[i] < P.M && c[i] < P.C;
      x[i].a = x[i].b = x[i].c = make_uint4(0, 0, 0, 0);
      if (in[i]) load_inputs<WHAT>(P, row[i], c[i], x[i]);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float v[8], w[8];
      code_values<WHAT, BF16, ACT>(x[i], c[i] >= P.F, v, w);
      store_codes(P, in[i], row[i], c[i], v,
                  WHAT == kPlain ? top_of_words<BF16>(x[i].a) : top8(v));
      if constexpr (WHAT == kPair) store_codes(P, in[i], row[i], P.F + c[i], w, top8(w));
    }
  }
}

// ---------------------------------------------------------------------------
// weights: a block of threads to a 128 x 128 block.  Measured, cold, bf16: 28672 x 8192 118 us (6.0
// TB/s), 4096 x 4096 15.3 us (3.3).

struct WeightParams {
  const uint16_t* w;  // [E][N][K]
  uint8_t* q;
  float* scales;      // [E][N / 128][K / 128]
  int N, K;
};

template <bool BF16>
__global__ void __launch_bounds__(256) weight_kernel(const WeightParams P) {
  __shared__ uint32_t red[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nb = blocks_of(P.N), kb = blocks_of(P.K);
  const long long b = blockIdx.x;
  const int k = (int)(b % kb) * kBlock + 8 * (threadIdx.x & 15);
  const long long rest = b / kb;
  const int n0 = (int)(rest % nb) * kBlock + (int)(threadIdx.x >> 4);
  const size_t base = (size_t)(rest / nb) * P.N * P.K + k;
  uint4 v[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    if (k < P.K && n0 + 16 * i < P.N) v[i] = load16(P.w + base + (size_t)(n0 + 16 * i) * P.K);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack8<BF16>(v[i], f);
    top = max(top, top8(f));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) red[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, red[i]);
  const float scale = scale_of(top);
  if (threadIdx.x == 0) P.scales[b] = scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (k >= P.K || n0 + 16 * i >= P.N) continue;
    float f[8];
    unpack8<BF16>(v[i], f);
    *reinterpret_cast<uint2*>(P.q + base + (size_t)(n0 + 16 * i) * P.K) = encode8(f, scale);
  }
}

// ---------------------------------------------------------------------------
// argument checks and launches

bool type_ok(int type) { return type == QL_TYPE_F16 || type == QL_TYPE_BF16; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool cols_ok(int c) { return c >= 16 && c <= kMaxColumns && c % 16 == 0; }

struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
// no output overlaps an input or another output
template <int NO, int NI>
bool disjoint(const Span (&outs)[NO], const Span (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return false;
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i], ins[j])) return false;
  }
  return true;
}
size_t strided(int M, long long ld, int K) { return ((size_t)(M - 1) * ld + K) * 2; }
size_t scale_bytes(int M, int C) { return (size_t)M * blocks_of(C) * 4; }

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}

// The kernel may start while the one before it ends (it waits for that one's results itself).
template <class... Params, class... Args>
ql_status launch_early_smem(void (*kernel)(Params...), unsigned grid, int threads, size_t smem,
                            ql_stream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? QL_OK : QL_ERR_CUDA;
}
template <class... Params, class... Args>
ql_status launch_early(void (*kernel)(Params...), unsigned grid, int threads, ql_stream_t stream,
                       const Args&... args) {
  return launch_early_smem(kernel, grid, threads, 0, stream, args...);
}

// Threads of a norm's block, for V vectors each.
int norm_threads(int K, int V) { return (K / 8 + 32 * V - 1) / (32 * V) * 32; }
int norm_vectors(int K) { return K <= 2048 ? 1 : K <= 8192 ? 2 : 4; }

template <bool BF16>
ql_status launch_norm(const NormParams& P, ql_stream_t st) {
  const int V = norm_vectors(P.K), t = norm_threads(P.K, V);
  if (V == 1) return launch_early(norm_kernel<BF16, 1>, P.M, t, st, P);
  if (V == 2) return launch_early(norm_kernel<BF16, 2>, P.M, t, st, P);
  return launch_early(norm_kernel<BF16, 4>, P.M, t, st, P);
}

// The norm's gradient: one block per SM, its groups filling it.
constexpr int kGradSmem = 200 * 1024;
int norm_grad_vectors(int K) { return K <= 2048 ? 1 : K <= 16384 ? 2 : 4; }
int norm_grad_blocks(int M, int sms) { return M < sms ? M : sms; }
template <bool BF16, bool PART, int V, int S>
ql_status launch_norm_grad_as(const NormGradParams& P, int blocks, int groups, size_t bytes,
                              ql_stream_t st) {
  auto kernel = norm_grad_kernel<BF16, PART, V, S>;
  // (set with each launch: it is the current device's)
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGradSmem) !=
      cudaSuccess)
    return QL_ERR_CUDA;
  // (the groups' sums, two thirds of a stage's two arrays and more, use the same memory)
  return launch_early_smem(kernel, blocks, groups * P.threads, groups * S * bytes, st, P);
}
template <bool BF16, bool PART, int V>
ql_status launch_norm_grad_v(NormGradParams P, int blocks, ql_stream_t st) {
  P.threads = norm_threads(P.K, V);
  const size_t bytes = (size_t)(P.dtotal ? 3 : 2) * V * P.threads * 16;  // of a row
  int groups = P.M < 2 * blocks ? 1 : 1024 / P.threads < 8 ? 1024 / P.threads : 8;
  // the next row, at least, is on its way
  while (groups > 1 && 2 * bytes * groups > kGradSmem) --groups;
  // as many stages as there is room for: four with one vector to a thread (192 KB at most), four or
  // two with two, two or one with four
  constexpr int kMost = V == 4 ? 2 : 4, kLeast = V == 1 ? 4 : kMost / 2;
  if (groups * kMost * bytes <= kGradSmem)
    return launch_norm_grad_as<BF16, PART, V, kMost>(P, blocks, groups, bytes, st);
  return launch_norm_grad_as<BF16, PART, V, kLeast>(P, blocks, groups, bytes, st);
}
template <bool BF16, bool PART>
ql_status launch_norm_grad_rows(const NormGradParams& P, int blocks, ql_stream_t st) {
  const int V = norm_grad_vectors(P.K);
  if (V == 1) return launch_norm_grad_v<BF16, PART, 1>(P, blocks, st);
  if (V == 2) return launch_norm_grad_v<BF16, PART, 2>(P, blocks, st);
  return launch_norm_grad_v<BF16, PART, 4>(P, blocks, st);
}
template <bool BF16>
ql_status launch_norm_grad(const NormGradParams& P, int blocks, ql_stream_t st) {
  return P.offsets ? launch_norm_grad_rows<BF16, true>(P, blocks, st)
                   : launch_norm_grad_rows<BF16, false>(P, blocks, st);
}

template <int WHAT, bool BF16, int ACT>
ql_status launch_codes_as(CodeParams P, ql_stream_t st) {
  P.slots = blocks_of(WHAT == kPair ? P.F : P.C) * 16;
  P.inv_slots = 1.f / (float)P.slots;
  const long long n = (long long)P.M * P.slots, most = 1 << 20;
  // two vectors to a thread once there are enough threads with one for every SM of a B200 (148)
  const int U = n >= 2048LL * 148 ? 2 : 1;
  const long long blocks = (n + kCodeThreads * U - 1) / (kCodeThreads * U);
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  return U == 2 ? launch_early(code_kernel<WHAT, BF16, ACT, 2>, grid, kCodeThreads, st, P)
                : launch_early(code_kernel<WHAT, BF16, ACT, 1>, grid, kCodeThreads, st, P);
}
template <int WHAT, bool BF16>
ql_status launch_codes(const CodeParams& P, ql_stream_t st) {
  if constexpr (WHAT == kPlain) {
    return launch_codes_as<WHAT, BF16, QL_ACT_NONE>(P, st);
  } else {
    switch (P.act) {
      case QL_ACT_RELU: return launch_codes_as<WHAT, BF16, QL_ACT_RELU>(P, st);
      case QL_ACT_GELU: return launch_codes_as<WHAT, BF16, QL_ACT_GELU>(P, st);
      case QL_ACT_GELU_TANH: return launch_codes_as<WHAT, BF16, QL_ACT_GELU_TANH>(P, st);
      case QL_ACT_SILU: return launch_codes_as<WHAT, BF16, QL_ACT_SILU>(P, st);
      default: return launch_codes_as<WHAT, BF16, QL_ACT_NONE>(P, st);
    }
  }
}
template <int WHAT>
ql_status codes(int type, const CodeParams& P, ql_stream_t st) {
  return type == QL_TYPE_BF16 ? launch_codes<WHAT, true>(P, st) : launch_codes<WHAT, false>(P, st);
}

// Sums of a call's parts lie where those of the other fused layers do, behind their counters, so
// that one workspace serves all of them (fused.h).
constexpr size_t kPartials = qfused::kVecCounterOffset + qfused::kVecCounterBytes;

// The checks and the launch of a product; C columns of q, R of the output.
ql_status product(int type, const uint8_t* q, const float* scales, const int* offsets,
                  const uint8_t* w, const float* wscales, void* y, int M, int E, int N, int K,
                  bool backward, bool grouped, void* workspace, size_t workspace_bytes,
                  ql_stream_t stream) {
  if (!type_ok(type)) return QL_ERR_UNSUPPORTED;
  if (!q || !scales || !w || !wscales || !y || (grouped && !offsets)) return QL_ERR_NULL;
  if (M < 1 || M > kMaxRows || !cols_ok(N) || !cols_ok(K) || E < 1 || E > kMaxExperts)
    return QL_ERR_SHAPE;
  const int C = backward ? N : K, R = backward ? K : N;
  // a tensor map's strides, an expert's codes among them, are below 2^40 bytes
  if ((long long)N * K >= (1LL << 40)) return QL_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(scales, 4) || !aligned(w, 16) || !aligned(wscales, 4) ||
      !aligned(y, 16) || !aligned(offsets, 4))
    return QL_ERR_ALIGN;
  if (!workspace || workspace_bytes < kPartials) return QL_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return QL_ERR_ALIGN;
  const Span outs[2] = {{y, (size_t)M * R * 2}, {workspace, workspace_bytes}};
  const Span ins[5] = {{q, (size_t)M * C}, {scales, scale_bytes(M, C)},
                       {offsets, (size_t)(E + 1) * 4}, {w, (size_t)E * N * K},
                       {wscales, (size_t)E * blocks_of(N) * blocks_of(K) * 4}};
  if (!disjoint(outs, ins)) return QL_ERR_ALIAS;
  Product p{};
  p.bf16 = type == QL_TYPE_BF16;
  p.backward = backward;
  p.q = q;
  p.sx = scales;
  p.offsets = offsets;
  p.w = w;
  p.sw = wscales;
  p.y = y;
  p.M = M;
  p.E = E;
  p.N = N;
  p.K = K;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.err = reinterpret_cast<uint32_t*>(ws);
  p.counters = reinterpret_cast<uint32_t*>(ws + qfused::kErrBytes);
  p.partials = reinterpret_cast<float*>(ws + kPartials);
  p.partial_bytes = workspace_bytes - kPartials;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  return launch_product(p);
}

// The checks and the launches of the norm's backward pass; offsets: null, or [E + 1].
ql_status norm_backward(int type, const void* dy, const void* total, const float* rstd,
                        const void* weight, const void* dtotal, const int* offsets, void* dx,
                        float* dweight, int M, int E, int K, void* workspace,
                        size_t workspace_bytes, ql_stream_t stream) {
  if (!type_ok(type)) return QL_ERR_UNSUPPORTED;
  if (!dy || !total || !rstd || !weight || !dx) return QL_ERR_NULL;
  if (M < 1 || M > kMaxRows || !cols_ok(K) || K > kMaxNorm) return QL_ERR_SHAPE;
  if (!aligned(dy, 16) || !aligned(total, 16) || !aligned(rstd, 4) || !aligned(weight, 16) ||
      !aligned(dtotal, 16) || !aligned(offsets, 4) || !aligned(dx, 16) || !aligned(dweight, 4))
    return QL_ERR_ALIGN;
  const int sms = sm_count();
  if (sms <= 0) return QL_ERR_CUDA;
  const int blocks = norm_grad_blocks(M, sms);
  if (dweight) {
    if (!workspace || workspace_bytes < kPartials + (size_t)blocks * K * 4)
      return QL_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return QL_ERR_ALIGN;
  }
  const size_t mk = (size_t)M * K * 2;
  const Span outs[3] = {{dx, mk}, {dweight, (size_t)K * 4},
                        {dweight ? workspace : nullptr, workspace_bytes}};
  const Span ins[6] = {{dy, mk}, {total, mk}, {rstd, (size_t)M * 4}, {weight, (size_t)K * 2},
                       {dtotal == dx ? nullptr : dtotal, mk}, {offsets, (size_t)(E + 1) * 4}};
  if (!disjoint(outs, ins)) return QL_ERR_ALIAS;
  NormGradParams P{};
  P.dy = static_cast<const uint16_t*>(dy);
  P.total = static_cast<const uint16_t*>(total);
  P.rstd = rstd;
  P.weight = static_cast<const uint16_t*>(weight);
  P.dtotal = static_cast<const uint16_t*>(dtotal);
  P.offsets = offsets;
  P.dx = static_cast<uint16_t*>(dx);
  P.partials = dweight ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kPartials)
                       : nullptr;
  P.M = M;
  P.E = E;
  P.K = K;
  const ql_status s = type == QL_TYPE_BF16 ? launch_norm_grad<true>(P, blocks, stream)
                                           : launch_norm_grad<false>(P, blocks, stream);
  if (s != QL_OK || !dweight) return s;
  const unsigned joins = (unsigned)((K + 31) / 32);
  const float* sums = P.partials;
  return joins <= 2u * (unsigned)sms
             ? launch_early(norm_join_kernel<32>, joins, 32 * 32, stream, sums, dweight, blocks, K)
             : launch_early(norm_join_kernel<16>, joins, 32 * 16, stream, sums, dweight, blocks, K);
}

}  // namespace

// ---------------------------------------------------------------------------
// exported entry points

extern "C" ql_status qlinear_fp8_quantize(int type, const void* x, long long ldx, uint8_t* q,
                                          float* scales, int M, int K, ql_stream_t stream) {
  if (!type_ok(type)) return QL_ERR_UNSUPPORTED;
  if (!x || !q || !scales) return QL_ERR_NULL;
  if (M < 1 || M > kMaxRows || !cols_ok(K) || ldx < K || ldx > (1LL << 40)) return QL_ERR_SHAPE;
  if (!aligned(x, 16) || ldx % 8 || !aligned(q, 16) || !aligned(scales, 4)) return QL_ERR_ALIGN;
  const Span outs[2] = {{q, (size_t)M * K}, {scales, scale_bytes(M, K)}};
  const Span ins[1] = {{x, strided(M, ldx, K)}};
  if (!disjoint(outs, ins)) return QL_ERR_ALIAS;
  CodeParams P{};
  P.x = static_cast<const uint16_t*>(x);
  P.q = q;
  P.scales = scales;
  P.ldx = ldx;
  P.M = M;
  P.C = K;
  return codes<kPlain>(type, P, stream);
}

extern "C" ql_status qlinear_fp8_gated(int type, int act, const void* gu, uint8_t* q,
                                       float* scales, int M, int F, ql_stream_t stream) {
  if (!type_ok(type) || !qact::act_ok(act)) return QL_ERR_UNSUPPORTED;
  if (!gu || !q || !scales) return QL_ERR_NULL;
  if (M < 1 || M > kMaxRows || !cols_ok(F) || F > kMaxColumns / 2) return QL_ERR_SHAPE;
  if (!aligned(gu, 16) || !aligned(q, 16) || !aligned(scales, 4)) return QL_ERR_ALIGN;
  const Span outs[2] = {{q, (size_t)M * F}, {scales, scale_bytes(M, F)}};
  const Span ins[1] = {{gu, (size_t)M * F * 4}};
  if (!disjoint(outs, ins)) return QL_ERR_ALIAS;
  CodeParams P{};
  P.x = static_cast<const uint16_t*>(gu);
  P.q = q;
  P.scales = scales;
  P.M = M;
  P.C = P.F = F;
  P.act = act;
  return codes<kGated>(type, P, stream);
}

extern "C" ql_status qlinear_fp8_gated_backward(int type, int act, const void* dh, const void* gu,
                                                uint8_t* q, float* scales, int M, int F,
                                                ql_stream_t stream) {
  if (!type_ok(type) || !qact::act_ok(act)) return QL_ERR_UNSUPPORTED;
  if (!dh || !gu || !q || !scales) return QL_ERR_NULL;
  if (M < 1 || M > kMaxRows || !cols_ok(F) || F > kMaxColumns / 2) return QL_ERR_SHAPE;
  if (!aligned(dh, 16) || !aligned(gu, 16) || !aligned(q, 16) || !aligned(scales, 4))
    return QL_ERR_ALIGN;
  const Span outs[2] = {{q, (size_t)M * F * 2}, {scales, scale_bytes(M, 2 * F)}};
  const Span ins[2] = {{dh, (size_t)M * F * 2}, {gu, (size_t)M * F * 4}};
  if (!disjoint(outs, ins)) return QL_ERR_ALIAS;
  CodeParams P{};
  P.x = static_cast<const uint16_t*>(gu);
  P.dh = static_cast<const uint16_t*>(dh);
  P.q = q;
  P.scales = scales;
  P.M = M;
  P.C = 2 * F;
  P.F = F;
  P.act = act;
  return F % kBlock == 0 ? codes<kPair>(type, P, stream) : codes<kGatedGrad>(type, P, stream);
}

extern "C" ql_status qlinear_fp8_quantize_weights(int type, const void* w, uint8_t* q,
                                                  float* scales, int E, int N, int K,
                                                  ql_stream_t stream) {
  if (!type_ok(type)) return QL_ERR_UNSUPPORTED;
  if (!w || !q || !scales) return QL_ERR_NULL;
  if (E < 1 || E > kMaxExperts || !cols_ok(N) || !cols_ok(K)) return QL_ERR_SHAPE;
  const long long blocks = (long long)E * blocks_of(N) * blocks_of(K);
  if (blocks >= (1LL << 31)) return QL_ERR_SHAPE;
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(scales, 4)) return QL_ERR_ALIGN;
  const size_t count = (size_t)E * N * K;
  const Span outs[2] = {{q, count}, {scales, (size_t)blocks * 4}};
  const Span ins[1] = {{w, count * 2}};
  if (!disjoint(outs, ins)) return QL_ERR_ALIAS;
  const WeightParams P{static_cast<const uint16_t*>(w), q, scales, N, K};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (type == QL_TYPE_BF16)
    weight_kernel<true><<<(unsigned)blocks, 256, 0, st>>>(P);
  else
    weight_kernel<false><<<(unsigned)blocks, 256, 0, st>>>(P);
  return cudaGetLastError() == cudaSuccess ? QL_OK : QL_ERR_CUDA;
}

extern "C" ql_status qlinear_rmsnorm(int type, const void* x, long long ldx, const void* residual,
                                     const void* weight, float eps, void* total, void* y,
                                     uint8_t* q, float* scales, float* rstd, int M, int K,
                                     ql_stream_t stream) {
  if (!type_ok(type)) return QL_ERR_UNSUPPORTED;
  if (!x || !weight || (!q && !y) || (!q != !scales)) return QL_ERR_NULL;
  if (M < 1 || M > kMaxRows || !cols_ok(K) || K > kMaxNorm || ldx < K || ldx > (1LL << 40) ||
      !(eps >= 0.f))
    return QL_ERR_SHAPE;
  if (!aligned(x, 16) || ldx % 8 || !aligned(residual, 16) || !aligned(weight, 16) ||
      !aligned(total, 16) || !aligned(y, 16) || !aligned(q, 16) || !aligned(scales, 4) ||
      !aligned(rstd, 4))
    return QL_ERR_ALIGN;
  const size_t mk = (size_t)M * K * 2;
  // the stream may be updated in place: each thread reads an element before it writes it
  const bool in_x = total == x && ldx == K, in_r = total == residual;
  const Span outs[5] = {{total, mk}, {y, mk}, {q, mk / 2}, {scales, scale_bytes(M, K)},
                        {rstd, (size_t)M * 4}};
  const Span ins[3] = {{in_x ? nullptr : x, strided(M, ldx, K)},
                       {in_r ? nullptr : residual, mk}, {weight, (size_t)K * 2}};
  const Span others[4] = {outs[1], outs[2], outs[3], outs[4]};
  const Span whole[2] = {{x, strided(M, ldx, K)}, {residual, mk}};
  if (!disjoint(outs, ins) || !disjoint(others, whole)) return QL_ERR_ALIAS;
  NormParams P{};
  P.x = static_cast<const uint16_t*>(x);
  P.residual = static_cast<const uint16_t*>(residual);
  P.weight = static_cast<const uint16_t*>(weight);
  P.total = static_cast<uint16_t*>(total);
  P.y = static_cast<uint16_t*>(y);
  P.q = q;
  P.scales = scales;
  P.rstd = rstd;
  P.ldx = ldx;
  P.eps = eps;
  P.M = M;
  P.K = K;
  return type == QL_TYPE_BF16 ? launch_norm<true>(P, stream) : launch_norm<false>(P, stream);
}

extern "C" size_t qlinear_rmsnorm_workspace_bytes(int M, int K) {
  if (M < 1 || M > kMaxRows || !cols_ok(K) || K > kMaxNorm) return 0;
  const int sms = sm_count();
  return sms > 0 ? kPartials + qfused::align_up((size_t)norm_grad_blocks(M, sms) * K * 4, 256)
                 : 0;
}

extern "C" ql_status qlinear_rmsnorm_backward(int type, const void* dy, const void* total,
                                              const float* rstd, const void* weight,
                                              const void* dtotal, void* dx, float* dweight, int M,
                                              int K, void* workspace, size_t workspace_bytes,
                                              ql_stream_t stream) {
  return norm_backward(type, dy, total, rstd, weight, dtotal, nullptr, dx, dweight, M, 0, K,
                       workspace, workspace_bytes, stream);
}
extern "C" ql_status qlinear_rmsnorm_backward_grouped(
    int type, const void* dy, const void* total, const float* rstd, const void* weight,
    const void* dtotal, const int* offsets, void* dx, float* dweight, int M, int E, int K,
    void* workspace, size_t workspace_bytes, ql_stream_t stream) {
  if (!type_ok(type)) return QL_ERR_UNSUPPORTED;
  if (!offsets) return QL_ERR_NULL;
  if (E < 1 || E > kMaxExperts) return QL_ERR_SHAPE;
  return norm_backward(type, dy, total, rstd, weight, dtotal, offsets, dx, dweight, M, E, K,
                       workspace, workspace_bytes, stream);
}

extern "C" size_t qlinear_fp8_workspace_bytes(int M, int E, int N, int K) {
  if (M < 1 || M > kMaxRows || !cols_ok(N) || !cols_ok(K) || E < 1 || E > kMaxExperts) return 0;
  const size_t part = product_partial_bytes(M, E);
  return part ? kPartials + qfused::align_up(part, 256) : 0;
}

extern "C" ql_status qlinear_fp8_linear(int type, const uint8_t* q, const float* scales,
                                        const uint8_t* w, const float* wscales, void* y, int M,
                                        int N, int K, void* workspace, size_t workspace_bytes,
                                        ql_stream_t stream) {
  return product(type, q, scales, nullptr, w, wscales, y, M, 1, N, K, false, false, workspace,
                 workspace_bytes, stream);
}
extern "C" ql_status qlinear_fp8_linear_backward(int type, const uint8_t* q, const float* scales,
                                                 const uint8_t* w, const float* wscales, void* dx,
                                                 int M, int N, int K, void* workspace,
                                                 size_t workspace_bytes, ql_stream_t stream) {
  return product(type, q, scales, nullptr, w, wscales, dx, M, 1, N, K, true, false, workspace,
                 workspace_bytes, stream);
}
extern "C" ql_status qlinear_fp8_grouped(int type, const uint8_t* q, const float* scales,
                                         const int* offsets, const uint8_t* w,
                                         const float* wscales, void* y, int M, int E, int N, int K,
                                         void* workspace, size_t workspace_bytes,
                                         ql_stream_t stream) {
  return product(type, q, scales, offsets, w, wscales, y, M, E, N, K, false, true, workspace,
                 workspace_bytes, stream);
}
extern "C" ql_status qlinear_fp8_grouped_backward(int type, const uint8_t* q, const float* scales,
                                                  const int* offsets, const uint8_t* w,
                                                  const float* wscales, void* dx, int M, int E,
                                                  int N, int K, void* workspace,
                                                  size_t workspace_bytes, ql_stream_t stream) {
  return product(type, q, scales, offsets, w, wscales, dx, M, E, N, K, true, true, workspace,
                 workspace_bytes, stream);
}
