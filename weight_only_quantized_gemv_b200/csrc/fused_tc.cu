// Products of the fused linear layers on the fifth-generation tensor cores (tcgen05), with
// the dequantization inside and bias, activation, residual or the gated product in the
// epilogue (fused.h):
//
//   forward   D[n][m] = sum_k W[n][k] x[m][k]        rows n: output columns
//   backward  D[k][m] = sum_n W[n][k] dz[m][n]       rows k: input columns
//
// The weights are the MMA's A operand (128 rows per CTA), the activations its B operand.
// One pipeline stage is one unit of the packed layout, the 128 x 128 weights of a
// (128-column block, 128-k group), in both directions:
//  * eight warps decode a unit, one 16-column tile each, into two 128-row x 64-k panels of
//    fp16 with the 128-byte swizzle (row n, 16-byte granule c at granule c ^ (n mod 8)).
//    Read as K-major rows that is W[n][k], contracted over k; read as MN-major that is
//    W^T, contracted over n.  Only the descriptors and the order of the units differ.
//  * the unit's codes and parameters are one contiguous run of the packed arrays: plain bulk
//    copies into a ring of their own, filled ahead by a producer warp.
//  * x (dz) arrives by tensor copies, two 64-column boxes per stage.
//
// Roles of the 24 warps: 0 copies of x, 1 MMA issue and tensor memory, 2 copies of codes,
// 4..7 epilogue, 8..23 two teams of eight decoding warps that take the stages in turn, so that
// the latency of one unit's decoding (wait, shared loads, stores, proxy fence, arrival) is
// hidden behind the other's.
//
// PAIR: a cluster of two CTAs on two SMs computes 256 rows with tcgen05 cta_group::2; each CTA
// decodes its own 128 rows and copies half of the tokens, which halves what the tokens cost
// in shared memory and L2.
//
// Work: tiles of 128 (PAIR 256) rows x bn tokens.  Whole waves of tiles go round the
// workers; the remaining tiles, at least one wave where there is one, are cut into equal
// runs of stages (stream-K), whose partial sums meet in the workspace: the last contributor
// to arrive adds them in worker order, nobody waits.
//
// Every barrier wait is bounded in time (100 ms against microseconds); one that runs out sets
// a flag in the workspace's error word, all roles leave their loops, and the CTA waits for its
// own copies and MMAs, frees its tensor memory and exits.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "act.cuh"
#include "dequant_frag.cuh"
#include "fused.h"
#include "kernels.cuh"
#include "layout.h"
#include "tc.cuh"

using namespace qlayout;
using namespace qtc;

namespace {

constexpr uint32_t kErrStage = 1u, kErrAcc = 2u;
constexpr int kTeams = 2, kTeamWarps = 8;

template <int BNX_, int FMT_, bool PAIR_>
struct TcCfg {
  static constexpr int BNX = BNX_, FMT = FMT_;     // most tokens per tile, format
  static constexpr bool PAIR = PAIR_;
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int kBRows = BNX / kCtas;       // most tokens one CTA copies
  static constexpr int kHalfA = 128 * 128;         // bytes of a 128-row x 64-column panel
  static constexpr int kHalfB = kBRows * 128;
  static constexpr int kABytes = 2 * kHalfA;
  static constexpr int kStageBytes = kABytes + 2 * kHalfB;
  // codes of 8 chunks, then their scales and zeros (LUT4: absmax)
  static constexpr int kChunk = FMT == kW2 ? 512 : FMT == kW8 ? 2048 : 1024;
  static constexpr int kCodeBytes = kBlockTiles * kChunk;
  static constexpr int kParChunk = FMT == kLUT4 ? 128 : 32;  // per tile and array
  static constexpr int kSlot = kCodeBytes + (FMT == kLUT4 ? 1 : 2) * kBlockTiles * kParChunk;
  static constexpr int S = 3;
  static constexpr int kBudget = 232448 - 1024 - 512;        // alignment, barriers
  static constexpr int SC0 = (kBudget - S * kStageBytes) / kSlot;
  static constexpr int SC = SC0 < 12 ? SC0 : 12;
  static_assert(SC >= 2, "code ring");
  static constexpr int kRingC = S * kStageBytes;
  static constexpr int kBarOff = kRingC + SC * kSlot;
  // full[S] empty[S] accf[2] acce[2] fin cfull[SC] cempty[SC], tensor memory base, abort, lut
  static constexpr int kMiscOff = kBarOff + 8 * (2 * S + 5 + 2 * SC);
  static constexpr int kLutOff = kMiscOff + 16;
  static constexpr int kSmem = kLutOff + 64 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
  static constexpr int kEpiWarp0 = 4, kDqWarp0 = 8;
  static constexpr int kWarps = kDqWarp0 + kTeams * kTeamWarps;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr uint32_t kTmemCols = 2 * BNX;
  static constexpr uint32_t kFullCount = 1 + kCtas * kTeamWarps;
  static constexpr uint32_t kAccEmptyCount = kCtas * 4;
};

struct TcParams {
  const uint8_t* qw;
  const void* p0;
  const void* p1;
  qfused::Epilogue epi;
  float* partials;
  uint32_t* counters;
  uint32_t* err;
  int M, N, K, G, ntiles, nblocks;
  int ld;        // row stride of the output: N forward, K backward (gated: F)
  int rows;      // valid rows of D: N or K
  int rblocks;   // 128-row blocks
  int steps;     // units per tile: groups (forward) or blocks (backward)
  int bn, mtiles, tiles, whole;  // tokens per tile; tiles [0, whole) are not split
};

// The work of a worker (CTA or pair): whole tiles w, w + W, ..., then its run of the stages of
// tiles [whole, tiles), cut at tile boundaries.
struct Segments {
  long long u, u1;
  int t, w, W;
  bool first;  // no stage of the run has been handed out yet
  __device__ __forceinline__ void init(const TcParams& P, int w_, int W_) {
    w = w_;
    W = W_;
    t = w_;
    const long long U = (long long)(P.tiles - P.whole) * P.steps;
    u = w * U / W;
    u1 = (w + 1) * U / W;
    first = true;
  }
  // tile, stages [k0, k1); slot: workspace slot of a partial sum (0: the run's first segment)
  __device__ __forceinline__ bool next(const TcParams& P, int& tile, int& k0, int& k1, int& slot) {
    slot = 0;
    if (t < P.whole) {
      tile = t;
      t += W;
      k0 = 0;
      k1 = P.steps;
      return true;
    }
    if (u >= u1) return false;
    const int tt = (int)(u / P.steps);
    tile = P.whole + tt;
    k0 = (int)(u - (long long)tt * P.steps);
    k1 = (u1 - u < (long long)(P.steps - k0)) ? k0 + (int)(u1 - u) : P.steps;
    u += k1 - k0;
    slot = first ? 0 : 1;
    first = false;
    return true;
  }
};

__device__ __forceinline__ long long run_begin(int w, long long U, int W) { return w * U / W; }
__device__ __forceinline__ int worker_of(long long u, long long U, int W) {
  return (int)(((u + 1) * W - 1) / U);
}

// ---------------------------------------------------------------------------
// bounded waits

struct WaitCtx {
  volatile uint32_t* abort;  // shared memory
  uint32_t* err;             // global memory
};
constexpr uint64_t kWaitNs = 100ull * 1000 * 1000;

__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, WaitCtx w, uint32_t bit,
                                       bool cluster, bool patient, bool honor_abort) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    if (patient && it >= 64) {  // long waits: suspend up to 500 ns at a time
      uint32_t done;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(done)
          : "r"(bar), "r"(parity), "r"(500u)
          : "memory");
      if (done) return true;
    }
    if (mbar_ready(bar, parity, cluster)) return true;
    if (it >= 256) __nanosleep(32);
    if ((it & 63u) == 63u) {
      if (honor_abort && *w.abort) break;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0)
        t0 = now;
      else if (now - t0 > kWaitNs)
        break;
    }
  }
  atomicOr(w.err, bit);
  *w.abort = 1u;
  return false;
}

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const WaitCtx& w, uint32_t bit,
                                     bool cluster = false, bool patient = false,
                                     bool honor_abort = true) {
  if (mbar_ready(bar, parity, cluster)) return true;
  return wait_slow(bar, parity, w, bit, cluster, patient, honor_abort);
}

// A whole warp: every lane sees the phase complete (the usual case), or one lane waits.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtx& w,
                                          uint32_t bit, int lane, bool patient = false) {
  if (__all_sync(0xffffffffu, mbar_ready(bar, parity, false))) return true;
  bool ok = true;
  if (lane == 0) ok = wait_slow(bar, parity, w, bit, false, patient, true);
  return __shfl_sync(0xffffffffu, ok, 0);
}

// ---------------------------------------------------------------------------
// decoding: one warp, one 16-column tile of a unit, into rows 16 tile .. 16 tile + 15 of the
// two A panels.  Lane (gi, t) holds, per pair of steps i, the eight k 32 i + 8 t .. + 7 of
// rows gi and gi + 8: granule 4 (i mod 2) + t of panel i / 2.  Lanes with odd gi take the
// pairs in the order 1, 0, 3, 2: the eight lanes of a store phase (two rows, four t) then
// write eight distinct granules, without bank conflicts.

template <int FMT>
__device__ __forceinline__ uint32_t a_address(uint32_t a, int row, int i, int t) {
  return a + (i >> 1) * (128 * 128) + row * 128 + (((4 * (i & 1) + t) ^ (row & 7)) << 4);
}

template <class C>
__device__ __forceinline__ void decode_tile(uint32_t slot, uint32_t a, int tile, int lane,
                                            const float* lut) {
  constexpr int FMT = C::FMT;
  constexpr int KW = qlk::Fmt<FMT>::kWords, KP = KW / 4;  // words per lane, per step pair
  const int gi = lane >> 2, t = lane & 3;
  const int swap = gi & 1;
  uint32_t w[KW];
  const uint32_t cs = slot + tile * C::kChunk + lane * 16;
  if constexpr (FMT == kW8) {  // a quad is a pair: the swap is in the address
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = qlk::lds128(cs + (i ^ swap) * 512);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  } else {
    uint32_t r[KW];
#pragma unroll
    for (int q = 0; q < KW / 4; ++q) {
      const uint4 v = qlk::lds128(cs + q * 512);
      r[4 * q] = v.x;
      r[4 * q + 1] = v.y;
      r[4 * q + 2] = v.z;
      r[4 * q + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < KP; ++k) w[KP * i + k] = swap ? r[KP * (i ^ 1) + k] : r[KP * i + k];
  }
  const uint32_t pa = slot + C::kCodeBytes + tile * C::kParChunk;
  if constexpr (FMT == kLUT4) {
    const uint4 am = qlk::lds128(pa + gi * 16);  // [64-block][row half]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float m = __uint_as_float(i >= 2 ? (h ? am.w : am.z) : (h ? am.y : am.x));
        const uint4 v = qdq::lut_pair8(w + KP * i, 0, h, lut, m);
        sts128(a_address<FMT>(a, 16 * tile + gi + 8 * h, i ^ swap, t), v);
      }
  } else {
    const __half2 s2 = qdq::u32_as_h2(qlk::lds32(pa + gi * 4));
    const __half2 z2 = qdq::u32_as_h2(qlk::lds32(pa + kBlockTiles * C::kParChunk + gi * 4));
    __half2 zb[2][2];
    qdq::zero_bias<FMT>(__low2float(z2), __high2float(z2), zb);
    const __half2 sl = __low2half2(s2), sh = __high2half2(s2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 v = qdq::uniform_pair8<FMT>(w + KP * i, 0, h, zb, h ? sh : sl);
        sts128(a_address<FMT>(a, 16 * tile + gi + 8 * h, i ^ swap, t), v);
      }
  }
}

// Rows of a tile past the last column, contracted in the backward product: zeros.
template <int FMT>
__device__ __forceinline__ void zero_tile(uint32_t a, int tile, int lane) {
  const int gi = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      sts128(a_address<FMT>(a, 16 * tile + gi + 8 * h, i ^ (gi & 1), t), make_uint4(0, 0, 0, 0));
}

// ---------------------------------------------------------------------------
// epilogue: 16 tokens (m0 .. m0 + count - 1 of them real) of one row per lane

__device__ __forceinline__ void finish16(const TcParams& P, const float (&v)[16], int m0, int count,
                                         int row) {
  const qfused::Epilogue& E = P.epi;
  const bool in = row < P.rows;
  if (E.gated) {
    // rows alternate 16 gate / 16 up; the lanes exchange, per pair of tokens, so that the gate
    // lanes finish the even token and the up lanes the odd one
    const int F = P.ld, f = (row >> 5) * 16 + (row & 15), up = (row >> 4) & 1;
    const float bias = in && E.bias ? __half2float(E.bias[(size_t)up * F + f]) : 0.f;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float z0 = v[e] + bias, z1 = v[e + 1] + bias;
      if (E.zsave && in) {
        __half* o = E.zsave + ((size_t)(m0 + e) * 2 + up) * F + f;
        if (e < count) o[0] = __float2half_rn(z0);
        if (e + 1 < count) o[(size_t)2 * F] = __float2half_rn(z1);
      }
      const float other = __shfl_xor_sync(0xffffffffu, up ? z0 : z1, 16);
      const float g = up ? other : z0, u = up ? z1 : other;
      if (in && e + up < count)
        E.y[(size_t)(m0 + e + up) * F + f] = __float2half_rn(qact::act_forward(E.act, g) * u);
    }
    return;
  }
  if (!in) return;
  const float bias = E.bias ? __half2float(E.bias[row]) : 0.f;
  const size_t o = (size_t)m0 * P.ld + row;
  float r[16];
#pragma unroll
  for (int e = 0; e < 16; ++e)
    r[e] = E.residual && e < count ? __half2float(E.residual[o + (size_t)e * P.ld]) : 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    if (e >= count) break;
    const float z = v[e] + bias;
    if (E.zsave) E.zsave[o + (size_t)e * P.ld] = __float2half_rn(z);
    E.y[o + (size_t)e * P.ld] = __float2half_rn(qact::act_forward(E.act, z) + r[e]);
  }
}

// A-operand descriptor of the backward product: MN-major, 128-byte swizzle, 64-wide MN panels
// 16384 bytes apart (leading offset), 8-row groups of the contraction 1024 bytes apart
// (stride).  Forward: K-major (desc_sw128).
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(128 * 128 / 16) << 16) | (64ull << 32) |
         (1ull << 46) | (2ull << 61);
}
constexpr uint32_t kTransposeA = 1u << 15;  // instruction descriptor: A is MN-major

template <int BNX, int FMT, bool PAIR, bool BWD>
__global__ void __launch_bounds__(TcCfg<BNX, FMT, PAIR>::kThreads, 1)
    fused_tc_kernel(const TcParams P, const __grid_constant__ CUtensorMap xmap) {
  using C = TcCfg<BNX, FMT, PAIR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = qlk::smem_addr(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (ring - raw);
  const uint32_t bars = ring + C::kBarOff;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (C::S + s); };
  auto accf = [&](int a) { return bars + 8 * (2 * C::S + a); };
  auto acce = [&](int a) { return bars + 8 * (2 * C::S + 2 + a); };
  const uint32_t fin = bars + 8 * (2 * C::S + 4);
  auto cfull = [&](int c) { return bars + 8 * (2 * C::S + 5 + c); };
  auto cempty = [&](int c) { return bars + 8 * (2 * C::S + 5 + C::SC + c); };
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::kMiscOff);
  float* lut = reinterpret_cast<float*>(smem + C::kLutOff);
  const WaitCtx W{misc + 1, P.err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const bool leader = rank == 0;
  const int wk = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int nwk = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  auto lead = [&](uint32_t b) { return (PAIR && !leader) ? cluster_addr(b, 0) : b; };
  auto arrive_lead = [&](uint32_t b) {
    if (PAIR && !leader)
      mbar_arrive_remote(cluster_addr(b, 0));
    else
      qlk::mbar_arrive(b);
  };
  auto commit_both = [&](uint32_t b) {
    tc_commit<PAIR>(b);
    if constexpr (PAIR) tc_commit<PAIR>(cluster_addr(b, 1));
  };

  if (FMT == kLUT4 && threadIdx.x < 16)
    lut[threadIdx.x] = __half2float(static_cast<const __half*>(P.p0)[threadIdx.x]);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) {
      qlk::mbar_init(full(s), C::kFullCount);
      qlk::mbar_init(empty(s), 1);
    }
    for (int c = 0; c < C::SC; ++c) {
      qlk::mbar_init(cfull(c), 1);
      qlk::mbar_init(cempty(c), kTeamWarps);
    }
    for (int a = 0; a < 2; ++a) {
      qlk::mbar_init(accf(a), 1);
      qlk::mbar_init(acce(a), C::kAccEmptyCount);
    }
    qlk::mbar_init(fin, 1);
    misc[1] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<PAIR>(ring + C::kMiscOff, C::kTmemCols);
  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  qlk::grid_dependents_launch();

  Segments sg;
  sg.init(P, wk, nwk);
  int tile, k0, k1, slot;

  if (warp == 0) {
    // ---- copies of x (dz)
    if (lane == 0) {
      qlk::grid_dependency_wait();
      int s = 0, ph = 1, n = 0;
      bool ok = true;
      const uint32_t bytes = (uint32_t)P.bn * 256u;  // both CTAs, both boxes
      while (ok && sg.next(P, tile, k0, k1, slot)) {
        const int m = (tile % P.mtiles) * P.bn + (int)rank * (P.bn / C::kCtas);
        for (int k = k0; k < k1; ++k) {
          if (n >= C::S && !(ok = wait(empty(s), ph, W, kErrStage))) break;
          const uint32_t b = ring + s * C::kStageBytes + C::kABytes;
          if (leader) qlk::mbar_arrive_expect_tx(full(s), bytes);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (PAIR)
              tma_2d_pair(b + h * C::kHalfB, &xmap, k * 128 + h * 64, m, lead(full(s)));
            else
              tma_2d(b + h * C::kHalfB, &xmap, k * 128 + h * 64, m, full(s));
          }
          ++n;
          if (++s == C::S) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // no copy is in flight when the CTA exits (the leader's barriers count both CTAs')
      if (leader)
        for (int i = n > C::S ? n - C::S : 0; i < n; ++i)
          wait(full(i % C::S), (i / C::S) & 1, W, kErrStage, PAIR, false, false);
    }
  } else if (warp == 2) {
    // ---- copies of the units' codes and parameters
    if (lane == 0) {
      int c = 0, ph = 1, n = 0;
      bool ok = true;
      const uint64_t pol = qlk::evict_first_policy();
      while (ok && sg.next(P, tile, k0, k1, slot)) {
        const int rb = (tile / P.mtiles) * C::kCtas + (int)rank;
        for (int k = k0; k < k1; ++k) {
          if (n >= C::SC) {
            if (n == C::SC) qlk::grid_dependency_wait();
            if (!(ok = wait(cempty(c), ph, W, kErrStage))) break;
          }
          const int b = BWD ? k : rb, g = BWD ? rb : k;
          const uint32_t dst = ring + C::kRingC + c * C::kSlot;
          if (rb < P.rblocks) {
            const int tb = tiles_in_block(b, P.ntiles);
            const long long ch = chunk_index(b, g, 0, P.G, P.ntiles);
            const uint32_t cb = tb * C::kChunk, pb = tb * C::kParChunk;
            qlk::mbar_arrive_expect_tx(cfull(c), cb + (FMT == kLUT4 ? 1 : 2) * pb);
            if (P.mtiles == 1)  // read once
              qlk::bulk_g2s(dst, P.qw + ch * C::kChunk, cb, cfull(c), pol);
            else
              qlk::bulk_g2s(dst, P.qw + ch * C::kChunk, cb, cfull(c));
            const uint32_t pd = dst + C::kCodeBytes;
            if constexpr (FMT == kLUT4) {
              qlk::bulk_g2s(pd, static_cast<const float*>(P.p1) + ch * 32, pb, cfull(c));
            } else {
              qlk::bulk_g2s(pd, static_cast<const __half*>(P.p0) + ch * 16, pb, cfull(c));
              qlk::bulk_g2s(pd + kBlockTiles * C::kParChunk,
                            static_cast<const __half*>(P.p1) + ch * 16, pb, cfull(c));
            }
          } else {  // no rows for this CTA of the pair
            qlk::mbar_arrive(cfull(c));
          }
          ++n;
          if (++c == C::SC) {
            c = 0;
            ph ^= 1;
          }
        }
      }
      for (int i = n > C::SC ? n - C::SC : 0; i < n; ++i)
        wait(cfull(i % C::SC), (i / C::SC) & 1, W, kErrStage, false, false, false);
    }
  } else if (warp == 1) {
    // ---- MMA issue (the leader of a pair)
    if (lane == 0 && leader) {
      qlk::grid_dependency_wait();
      const uint32_t idesc = idesc_f16(128 * C::kCtas, P.bn) | (BWD ? kTransposeA : 0u);
      int s = 0, ph = 0, j = 0;
      bool ok = true;
      for (; ok && sg.next(P, tile, k0, k1, slot); ++j) {
        const int a = j & 1;
        if (j >= 2 && !(ok = wait(acce(a), ((j >> 1) - 1) & 1, W, kErrAcc, PAIR))) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(a * BNX);
        for (int k = k0; k < k1; ++k) {
          if (!(ok = wait(full(s), ph, W, kErrStage, PAIR))) break;
          tc_fence_after();
          const uint32_t pa = ring + s * C::kStageBytes, pb = pa + C::kABytes;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t ad = BWD ? desc_mn(pa + 2048 * kk)
                                    : desc_sw128(pa + (kk >> 2) * C::kHalfA + 32 * (kk & 3));
            const uint64_t bd = desc_sw128(pb + (kk >> 2) * C::kHalfB + 32 * (kk & 3));
            tc_mma<PAIR>(d, ad, bd, idesc, (k != k0) || (kk != 0));
          }
          commit_both(empty(s));
          if (++s == C::S) {
            s = 0;
            ph ^= 1;
          }
        }
        if (ok) commit_both(accf(a));
      }
      tc_commit<PAIR>(fin);
      wait(fin, 0, W, kErrAcc, false, false, false);
    }
  } else if (warp >= C::kDqWarp0) {
    // ---- decoding teams
    const int team = (warp - C::kDqWarp0) / kTeamWarps, dt = (warp - C::kDqWarp0) % kTeamWarps;
    int n = 0, s = 0, sph = 1, c = 0, cph = 0;
    bool ok = true;
    while (ok && sg.next(P, tile, k0, k1, slot)) {
      const int rb = (tile / P.mtiles) * C::kCtas + (int)rank;
      for (int k = k0; k < k1; ++k, ++n) {
        if ((n & 1) == team) {
          const int tb = rb < P.rblocks ? tiles_in_block(BWD ? k : rb, P.ntiles) : 0;
          if (n >= C::S) {
            if (n <= C::S + 1) qlk::grid_dependency_wait();
            if (!(ok = warp_wait(empty(s), sph, W, kErrStage, lane))) break;
          }
          if (!(ok = warp_wait(cfull(c), cph, W, kErrStage, lane))) break;
          const uint32_t a = ring + s * C::kStageBytes;
          if (dt < tb)
            decode_tile<C>(ring + C::kRingC + c * C::kSlot, a, dt, lane, lut);
          else if (BWD)
            zero_tile<FMT>(a, dt, lane);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // visible to the MMAs
          __syncwarp();
          if (lane == 0) {
            qlk::mbar_arrive(cempty(c));
            arrive_lead(full(s));
          }
        }
        if (++s == C::S) {
          s = 0;
          sph ^= 1;
        }
        if (++c == C::SC) {
          c = 0;
          cph ^= 1;
        }
      }
    }
  } else if (warp >= C::kEpiWarp0) {
    // ---- epilogue: accumulator lanes 32 q .. 32 q + 31
    qlk::grid_dependency_wait();
    const int q = warp & 3;
    const long long U = (long long)(P.tiles - P.whole) * P.steps;
    for (int j = 0; sg.next(P, tile, k0, k1, slot); ++j) {
      const int a = j & 1;
      if (!warp_wait(accf(a), (j >> 1) & 1, W, kErrAcc, lane, true)) break;
      tc_fence_after();
      const int lrow = 32 * q + lane;
      const int row = ((tile / P.mtiles) * C::kCtas + (int)rank) * 128 + lrow;
      const int m0 = (tile % P.mtiles) * P.bn;
      const int cols = P.M - m0 < P.bn ? P.M - m0 : P.bn;
      const uint32_t tb = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(a * BNX);
      if (k0 == 0 && k1 == P.steps) {
        for (int c0 = 0; c0 < cols; c0 += 16) {
          uint32_t r[16];
          tmem_ld16(tb + (uint32_t)c0, r);
          tc_wait_ld();
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(r[e]);
          finish16(P, v, m0 + c0, cols - c0, row);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_lead(acce(a));
        continue;
      }
      // part of a tile: [token][row] partial sums, one row of 128 per token
      float* mine = P.partials + (size_t)(2 * blockIdx.x + slot) * 128 * P.bn + lrow;
      for (int c0 = 0; c0 < cols; c0 += 16) {
        uint32_t r[16];
        tmem_ld16(tb + (uint32_t)c0, r);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (c0 + e < cols) __stcg(mine + (size_t)(c0 + e) * 128, __uint_as_float(r[e]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_lead(acce(a));
      const long long ub = (long long)(tile - P.whole) * P.steps;
      const int wf = worker_of(ub, U, nwk), wl = worker_of(ub + P.steps - 1, U, nwk);
      uint32_t* counter = P.counters + ((size_t)(tile - P.whole) * C::kCtas + rank) * 4 + q;
      uint32_t prev = 0;
      if (lane == 0) prev = qlk::arrive_acq_rel(counter);
      prev = __shfl_sync(0xffffffffu, prev, 0);
      if (prev + 1 != (uint32_t)(wl - wf + 1)) continue;
      __syncwarp();
      for (int c0 = 0; c0 < cols; c0 += 16) {
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
        for (int w = wf; w <= wl; ++w) {
          const int cta = w * C::kCtas + (int)rank;
          const int sl = run_begin(w, U, nwk) >= ub ? 0 : 1;
          const float* src = P.partials + (size_t)(2 * cta + sl) * 128 * P.bn + lrow;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (c0 + e < cols) v[e] += __ldcg(src + (size_t)(c0 + e) * 128);
        }
        finish16(P, v, m0 + c0, cols - c0, row);
      }
      if (lane == 0) *counter = 0u;  // ready for the next call
    }
  }

  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<PAIR>(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// host side

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                       &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  fn.store(f, std::memory_order_release);
  return f;
}

// fp16 [rows][cols], box 64 columns x box_rows rows, 128-byte swizzle; outside: zeros
bool encode_rows(CUtensorMap* map, const void* base, int rows, int cols, int box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

// attr: two entries, the cluster first (the occupancy query takes that one alone)
template <int BNX, int FMT, bool PAIR>
void launch_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, unsigned ctas,
                   cudaStream_t st) {
  using C = TcCfg<BNX, FMT, PAIR>;
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3(ctas);
  cfg->blockDim = dim3(C::kThreads);
  cfg->dynamicSmemBytes = C::kSmem;
  cfg->stream = st;
  int n = 0;
  if constexpr (PAIR) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = n + 1;
}

// Workers resident at once, once per instance and device.
template <int BNX, int FMT, bool PAIR, bool BWD>
int resident_workers(int dev, int sms) {
  using C = TcCfg<BNX, FMT, PAIR>;
  static std::atomic<int> known[kMaxDevices];
  if (dev < 0 || dev >= kMaxDevices) return 0;
  int n = known[dev].load(std::memory_order_acquire);
  if (n > 0) return n;
  auto fn = fused_tc_kernel<BNX, FMT, PAIR, BWD>;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
    return 0;
  if constexpr (PAIR) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    launch_config<BNX, FMT, PAIR>(&cfg, attr, 2 * (sms / 2), nullptr);
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) n = 0;
  } else {
    int occ = 0;
    n = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, C::kThreads, C::kSmem) ==
                    cudaSuccess && occ >= 1
            ? sms
            : 0;
  }
  if (n > 0) known[dev].store(n, std::memory_order_release);
  return n;
}

// Tokens per tile and the tile form: one CTA for up to 64 tokens (in steps of 16), else a pair
// with up to 256 (in steps of 32); more tokens in equal tiles.
struct Tokens {
  bool pair;
  int bn, mtiles;
};
Tokens token_tiles(int M) {
  if (M <= 64) return Tokens{false, (M + 15) / 16 * 16, 1};
  const int mt = (M + 255) / 256;
  const int bn = ((M + mt - 1) / mt + 31) / 32 * 32;
  return Tokens{true, bn, (M + bn - 1) / bn};
}

template <int BNX, int FMT, bool PAIR, bool BWD>
ql_status launch_as(const qfused::Product& p, const Tokens& tk) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return QL_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return QL_ERR_CUDA;
  const int maxw = resident_workers<BNX, FMT, PAIR, BWD>(dev, sms);
  if (maxw <= 0) return QL_ERR_CUDA;
  constexpr int ctas = PAIR ? 2 : 1;
  TcParams P;
  P.qw = static_cast<const uint8_t*>(p.packed);
  P.p0 = p.p0;
  P.p1 = p.p1;
  P.epi = p.epi;
  P.partials = p.partials;
  P.counters = p.counters;
  P.err = p.err;
  P.M = p.M;
  P.N = p.N;
  P.K = p.K;
  P.G = p.K / kGroup;
  P.ntiles = p.N / kTileN;
  P.nblocks = (P.ntiles + kBlockTiles - 1) / kBlockTiles;
  P.rows = BWD ? p.K : p.N;
  P.ld = BWD ? p.K : p.epi.gated ? p.N / 2 : p.N;
  P.rblocks = BWD ? P.G : P.nblocks;
  P.steps = BWD ? P.nblocks : P.G;
  P.bn = tk.bn;
  P.mtiles = tk.mtiles;
  const long long tiles = (long long)((P.rblocks + ctas - 1) / ctas) * tk.mtiles;
  if (tiles >= (1LL << 31)) return QL_ERR_SHAPE;
  P.tiles = (int)tiles;
  // whole waves of tiles, then the rest shared out by stage: the remainder together with one
  // whole wave, so that a tile is cut in a few long runs
  const int rem = P.tiles % maxw;
  P.whole = rem == 0 ? P.tiles : P.tiles < maxw ? 0 : P.tiles - rem - maxw;
  const long long units = (long long)(P.tiles - P.whole) * P.steps;
  const int workers = P.whole > 0 || units >= maxw ? maxw : (int)units;
  CUtensorMap xmap;
  if (!encode_rows(&xmap, p.x, p.M, BWD ? p.N : p.K, tk.bn / ctas)) return QL_ERR_CUDA;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  launch_config<BNX, FMT, PAIR>(&cfg, attr, (unsigned)(workers * ctas), p.stream);
  if (cudaLaunchKernelEx(&cfg, fused_tc_kernel<BNX, FMT, PAIR, BWD>, P, xmap) != cudaSuccess)
    return QL_ERR_CUDA;
  return QL_OK;
}

template <int FMT, bool BWD>
ql_status launch_fmt(const qfused::Product& p) {
  const Tokens tk = token_tiles(p.M);
  if (!tk.pair) return launch_as<64, FMT, false, BWD>(p, tk);
  return tk.bn <= 128 ? launch_as<128, FMT, true, BWD>(p, tk)
                      : launch_as<256, FMT, true, BWD>(p, tk);
}

}  // namespace

namespace qfused {

// Two fp32 partial tiles of 128 rows per CTA; the tokens of a tile with at most M rows.
size_t tc_partial_bytes(int M) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  const int bn = M >= 256 ? 256 : (M + 31) / 32 * 32;
  return (size_t)2 * sms * 128 * bn * sizeof(float);
}

ql_status launch_tc(const Product& p) {
  switch (p.fmt) {
    case kW2: return p.backward ? launch_fmt<kW2, true>(p) : launch_fmt<kW2, false>(p);
    case kW4: return p.backward ? launch_fmt<kW4, true>(p) : launch_fmt<kW4, false>(p);
    case kW8: return p.backward ? launch_fmt<kW8, true>(p) : launch_fmt<kW8, false>(p);
    default: return p.backward ? launch_fmt<kLUT4, true>(p) : launch_fmt<kLUT4, false>(p);
  }
}

}  // namespace qfused
