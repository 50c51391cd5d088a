// Products of e4m3 codes with a scale per 128 on the fifth-generation tensor cores (tcgen05):
//
//   forward   D[n][m] = sum_b sx[m][b] sw[n / 128][b] sum_{k in block b} W[n][k] q[m][k]
//   backward  D[k][m] = sum_b sd[m][b] sw[b][k / 128] sum_{n in block b} W[n][k] q[m][n]
//
// for one matrix or for one per expert, whose rows of q follow one another.
//
// A pipeline step is one block of the summed index: 128 bytes of every row, the width of the
// 128-byte swizzle.  Both operands come by tensor copies.  The backward product reads the same
// 128 x 128 block of the weights MN-major (its rows are then the summed index), so that only the
// copies' coordinates and the descriptors differ.
//
// The scales differ from block to block, so the tensor cores' sum covers one block: a step's four
// MMAs write a fresh accumulator in tensor memory, and the epilogue warps add it, times sx sw, to
// fp32 sums in registers.  A warp makes the products of scales, steps ahead, in shared memory.
//
// Two kernels, by the rows of q that an average expert has (of all E: the host does not read the
// offsets, so rows on few experts get narrow tiles, each of which reads the weights again.  64
// experts of 2048 x 4096, 1024 rows: on all of them 113 us, on 8 or fewer 66; by one matrix 29):
//   up to 64     fp8_tc_kernel: the weights are the MMA's A operand (128 rows), q's rows its B
//                operand, any multiple of 16 of them.  Bound by reading the weights.
//   above        fp8_wide_kernel: q's rows are the A operand, 256 of D's rows the B operand.
//
// Work: whole waves of tiles go round the workers; the rest are cut by steps (schedule), and the
// parts' sums meet in the workspace: the last contributor to arrive adds them in worker order,
// nobody waits.  For experts all of this is computed on the device, from the offsets.
//
// Every barrier wait is bounded in time as in the fused products (fused_tc.cu).
//
// Measured, us (in brackets the bytes' or the operations' time at the card's rates: a copy's 6.55
// TB/s, twice cuBLAS' bf16 1.63 PFLOP/s): 1 x 28672 x 8192 39.8 (35.9), 33 rows 44.8 (36.2), 128 x
// 8192 x 28672 56 (36), 777 x 4096 x 12304 backward 64 (24; weights in L2: 53), 2048 x 8192 x 4096
// 73 (42), 4096 x 28672 x 8192 871 to 896 (589; call after call at the power limit of 1000 W, 1.5
// GHz, 985 to 1030).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "fp8.cuh"
#include "fp8.h"
#include "fused.h"
#include "kernels.cuh"
#include "tc.cuh"
#define QTC_WAIT_SLOW __forceinline__
#include "tc_pipe.cuh"

using namespace qtc;
using namespace qfp8;

namespace {

constexpr uint32_t kErrStage = 1u, kErrAcc = 2u, kErrOffsets = 4u;
constexpr int kTokStride = 80;  // bytes of a staged row of q's outputs: 32 of them and 16 more

// Few rows of q.  A thread of the epilogue holds two neighbouring columns (rows of q) of each eight
// (tcgen05.ld 16x256b), so a step's scales are one 8-byte shared load per four of its packed
// multiply-adds.  Warps: 0 copies, 1 MMA issue and tensor memory, 2 scales, 4 .. 7 epilogue.
template <int BNX_>
struct Cfg {
  static constexpr int BNX = BNX_;                 // most rows of q per tile
  static constexpr int kCtas = 1, kBlocks = 1;
  static constexpr int kGran = 16;                 // a tile's rows of q: a multiple
  static constexpr int kBRows = BNX;
  static constexpr int kABytes = 128 * 128;
  static constexpr int kBBytes = BNX * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kEpiWarps = 4, kEpiWarp0 = 4;
  static constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
  static constexpr int kAcc = 4;                   // accumulators
  static constexpr uint32_t kTmemCols = kAcc * BNX;
  // A call is bound by reading the weights: two CTAs on an SM keep more of them on their way, and
  // where one is enough the next call's first weights come while this one ends.
  static constexpr int kPerSm = 2;
  static constexpr size_t kTileBytes = 128 * BNX * 4;  // of a CTA's sums
  static constexpr int S = 104 * 1024 / kStageBytes;
  static constexpr int kStagingOff = S * kStageBytes;
  static constexpr int kStaging = 16 * kTokStride;           // per epilogue warp
  static constexpr int kScaleOff = kStagingOff + kEpiWarps * kStaging;
  static constexpr int kBarOff = kScaleOff + kAcc * BNX * 4;
  // full[S] empty[S] accf[kAcc] acce[kAcc] sempty[kAcc] fin
  static constexpr int kBars = 2 * S + 3 * kAcc + 1;
  static constexpr int kMiscOff = kBarOff + 8 * kBars;       // tensor memory's base, abort flag
  static constexpr int kTableOff = kMiscOff + 16;            // start[E + 1], tiles before [E + 1]
  static constexpr int smem(int E) { return kTableOff + 8 * (E + 1); }
  static constexpr int kMaxSmem = kTableOff + 8 * (kMaxExperts + 1);
  static_assert(kPerSm * (kTableOff + 8 * 256 + 1024) <= 233472, "shared memory");
};

struct Params {
  const float* sx;
  const float* sw;
  const int* offsets;
  void* y;
  float* partials;
  uint32_t* counters;
  uint32_t* err;
  int M, E, R;        // rows of q, experts, rows of D
  int steps;          // blocks of the summed index
  int nb, kb;         // blocks of the weights' N and K
  int rtiles;         // tiles of D's rows
  int bf16;
  int vec;            // scales of a row that one load may take
  uint32_t wait_us, test_us;
};

struct Tile {
  int e, rt, m0, rows, bn;  // expert, tile of D's rows, first row of q, how many, padded
};

// The call's tiles: those of expert e are pre[e] .. pre[e + 1] - 1, rows of q varying fastest, so
// that the workers that are at the same weights read them from L2.
struct Plan {
  const int* start;  // shared memory
  const int* pre;
  int tiles, whole, runners;
};

// The experts' first rows and tiles of BN rows of q, by one warp.
template <int BN>
__device__ __forceinline__ void make_table(const Params& P, int* start, int* pre, int lane) {
  if (P.offsets) qlk::grid_dependency_wait();
  int top = 0, before = 0;
  bool bad = false;
  for (int b = 0; b <= P.E; b += 32) {
    const int j = b + lane;
    const int raw = j > P.E ? 0 : P.offsets ? __ldcg(P.offsets + j) : j ? P.M : 0;
    int v = min(max(raw, 0), P.M);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, u);
    }
    v = max(v, top);
    top = __shfl_sync(0xffffffffu, v, 31);
    if (j <= P.E) {
      start[j] = v;
      bad |= v != raw;
    }
  }
  __syncwarp();
  if (lane == 0) pre[0] = 0;
  for (int b = 0; b < P.E; b += 32) {
    const int j = b + lane;
    int v = j < P.E ? (start[j + 1] - start[j] + BN - 1) / BN * P.rtiles : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    v += before;
    before = __shfl_sync(0xffffffffu, v, 31);
    if (j < P.E) pre[j + 1] = v;
  }
  if (blockIdx.x == 0 && __any_sync(0xffffffffu, bad) && lane == 0) atomicOr(P.err, kErrOffsets);
}

// The last expert with pre[e] <= t (one with tiles).
__device__ __forceinline__ int expert_of(const Params& P, const Plan& plan, int t) {
  int e = 0, hi = P.E;
  while (hi - e > 1) {
    const int mid = (e + hi) >> 1;
    if (plan.pre[mid] <= t)
      e = mid;
    else
      hi = mid;
  }
  return e;
}

// Tiles of equal width, a multiple of the granularity; or (wide_tile_of) of BNX rows of q.
template <class C>
__device__ __forceinline__ Tile tile_of(const Params& P, const Plan& plan, int t) {
  const int e = expert_of(P, plan, t);
  Tile r;
  r.e = e;
  const int lo = plan.start[e], cnt = plan.start[e + 1] - lo;
  const int mt = (cnt + C::BNX - 1) / C::BNX, l = t - plan.pre[e];
  r.rt = l / mt;
  r.bn = ((cnt + mt - 1) / mt + C::kGran - 1) / C::kGran * C::kGran;
  const int m = (l - r.rt * mt) * r.bn;
  r.m0 = lo + m;
  r.rows = min(r.bn, cnt - m);
  return r;
}
template <class C>
__device__ __forceinline__ Tile wide_tile_of(const Params& P, const Plan& plan, int t) {
  const int e = expert_of(P, plan, t);
  const int lo = plan.start[e], cnt = plan.start[e + 1] - lo;
  const int mt = (cnt + C::BNX - 1) / C::BNX, l = t - plan.pre[e], rt = l / mt;
  const int m = C::BNX * (l - rt * mt);
  return Tile{e, rt, lo + m, min(C::BNX, cnt - m), C::BNX};
}

// The work of a worker (CTA or pair): whole tiles w, w + W, ..., then its run of the steps of
// tiles [whole, tiles), cut at tile boundaries.
struct Segments {
  int t, W, rt, rk, left;
  bool first;
  __device__ __forceinline__ void init(const Plan& p, int steps, int w, int W_) {
    W = W_;
    t = w;
    const long long U = (long long)(p.tiles - p.whole) * steps;
    const long long u = w < p.runners ? run_begin(w, U, p.runners) : 0;
    left = w < p.runners ? (int)(run_begin(w + 1, U, p.runners) - u) : 0;
    rt = p.whole + (int)(u / steps);
    rk = (int)(u % steps);
    first = true;
  }
  __device__ __forceinline__ bool next(const Plan& p, int steps, int& tile, int& k0, int& k1,
                                       int& slot) {
    if (t < p.whole) {
      tile = t;
      t += W;
      k0 = 0;
      k1 = steps;
      return true;
    }
    if (left <= 0) return false;
    tile = rt++;
    k0 = rk;
    k1 = left < steps - rk ? rk + left : steps;
    left -= k1 - k0;
    rk = 0;
    slot = first ? 0 : 1;
    first = false;
    return true;
  }
};

// The R tiles behind the whole waves, over `runners` workers: each in f equal parts (f workers to a
// tile), or (RUNS) where that would leave many workers idle in W equal runs.  A call that is bound
// by reading the weights has no use for runs: fewer workers read as fast, and sums of parts cost.
constexpr int kMaxParts = 8;
template <bool RUNS>
__device__ __forceinline__ void schedule(Plan& p, int steps, int W) {
  const int R = p.tiles % W;
  p.whole = p.tiles - R;
  p.runners = 0;
  if (R == 0) return;
  const int f = min(min(W / R, steps), kMaxParts);
  const bool runs = RUNS && f < kMaxParts && (long long)R * steps >= W && 100 * R * f < 60 * W;
  p.runners = runs ? W : R * f;
}

// ---------------------------------------------------------------------------
// instructions

// Operand descriptors in two words, as in fused_tc.cu: 8-row groups 1024 bytes apart, 128-byte
// swizzle.  Instruction descriptor: A, B MN-major.
constexpr uint32_t kDescHi = 64u | (1u << 14) | (2u << 29);
constexpr uint32_t kDescLo = 1u << 16;
constexpr uint32_t kTransposeA = 1u << 15, kTransposeB = 1u << 16;

// e4m3 operands, fp32 accumulator
template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc,
                                    uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(kDescHi), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(kDescHi), "r"(accumulate)
        : "memory");
}

// Arrive on the barrier `bar` of this CTA (PAIR: of both, at the same offset) once the MMAs issued
// so far have completed.
template <bool PAIR>
__device__ __forceinline__ void commit_both(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], m;\n\t}" ::"r"(bar)
        : "memory");
  else
    tc_commit<false>(bar);
}

template <bool PAIR>
__device__ __forceinline__ void copy_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                        int c2, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// 16 lanes of tensor memory x 16 columns: register 4 i + 2 h + c holds row lane / 4 + 8 h of column
// 8 i + 2 (lane mod 4) + c.
__device__ __forceinline__ void tmem_ld_16x16(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// The loads above have arrived.  (Their registers go through it, so that no use moves ahead of it.)
__device__ __forceinline__ void wait_loads(uint32_t (&a)[8], uint32_t (&b)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]),
                 "+r"(a[6]), "+r"(a[7]), "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]),
                 "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7])
               :
               : "memory");
}

// Lane 0 arrives on two barriers, without a branch: a shared::cluster address, one of this CTA's.
__device__ __forceinline__ void arrive_both(uint32_t cluster_bar, uint32_t bar, int lane) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %2, 0;\n\t"
      "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%1];\n\t}" ::"r"(cluster_bar),
      "r"(bar), "r"(lane)
      : "memory");
}

using pair_t = unsigned long long;  // two fp32
__device__ __forceinline__ pair_t lds_pair(uint32_t a) {
  pair_t v;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void add_scaled(pair_t& acc, uint32_t lo, uint32_t hi, pair_t s) {
  asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(lo), "r"(hi), "l"(s));
}
__device__ __forceinline__ float2 halves(pair_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ pair_t add_pairs(pair_t a, pair_t b) {
  pair_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 32 lanes of tensor memory x 32 columns: register i holds column i of the lane's row.
__device__ __forceinline__ void tmem_ld_32x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, "
      "%24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void wait_loads(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Four 8 x 8 matrices of 16-bit values, transposed: lane 8 j + i gives the address of row i of
// matrix j.
__device__ __forceinline__ void store_transposed(uint32_t a, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

// ---------------------------------------------------------------------------

// Tensor maps: the weights [E][N][K], boxes of 128 x 128; q, boxes of 128 columns x 128, 64, 32 and
// 16 rows.
struct Maps {
  CUtensorMap w, q[4];
};

template <int BNX, bool BWD>
__global__ void __launch_bounds__(Cfg<BNX>::kThreads, Cfg<BNX>::kPerSm)
    fp8_tc_kernel(const Params P, const __grid_constant__ Maps maps) {
  using C = Cfg<BNX>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t ring = qlk::smem_addr(smem);  // 1024-byte aligned, as the swizzle wants
  const uint32_t bars = ring + C::kBarOff;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (C::S + s); };
  auto accf = [&](int a) { return bars + 8 * (2 * C::S + a); };
  auto acce = [&](int a) { return bars + 8 * (2 * C::S + C::kAcc + a); };
  auto sempty = [&](int a) { return bars + 8 * (2 * C::S + 2 * C::kAcc + a); };
  const uint32_t fin = bars + 8 * (2 * C::S + 3 * C::kAcc);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::kMiscOff);
  int* const start = reinterpret_cast<int*>(smem + C::kTableOff);
  int* const pre = start + P.E + 1;
  const WaitCtx W{ring + C::kMiscOff + 4, P.err, P.wait_us};
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  const int wk = (int)blockIdx.x, nwk = (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) {
      qlk::mbar_init(full(s), 1);
      qlk::mbar_init(empty(s), 1);
    }
    for (int a = 0; a < C::kAcc; ++a) {
      qlk::mbar_init(accf(a), 2);  // the MMAs, the scales
      qlk::mbar_init(acce(a), C::kEpiWarps);
      qlk::mbar_init(sempty(a), C::kEpiWarps);
    }
    qlk::mbar_init(fin, 1);
    misc[1] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) make_table<BNX>(P, start, pre, lane);
  sync_all<false>();
  if (warp == 1) tmem_alloc<false>(ring + C::kMiscOff, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  qlk::grid_dependents_launch();  // (behind the allocation: the next grid's must not come first)

  Plan plan{start, pre, pre[P.E], 0, 0};
  schedule<false>(plan, P.steps, nwk);
  Segments sg;
  sg.init(plan, P.steps, wk, nwk);
  int t, k0, k1, slot = 0;

  if (warp < C::kEpiWarp0) {
    if (warp == 0) {
      // ---- copies
      if (lane == 0) {
        int s = 0, ph = 1, n = 0;
        bool ok = true;
        if (P.offsets == nullptr && (P.test_us & 0xFFFFu) == 0) {
          // the weights of the first stages, while the kernels before this one end
          Segments ahead = sg;
          while (n < C::S && ahead.next(plan, P.steps, t, k0, k1, slot)) {
            const Tile T = tile_of<C>(P, plan, t);
            const int row = T.rt * 128;
            for (int k = k0; k < k1 && n < C::S; ++k, ++n) {
              qlk::mbar_arrive_expect_tx(full(n), C::kABytes + T.bn * 128);
              copy_3d<false>(ring + n * C::kStageBytes, &maps.w, BWD ? row : k * 128,
                             BWD ? k * 128 : row, T.e, full(n));
            }
          }
        }
        const int early = n;
        n = 0;
        qlk::grid_dependency_wait();
        if ((P.test_us & 0xFFFFu) && wk == 0) qlk::test_delay(P.test_us & 0xFFFFu);
        while (ok && sg.next(plan, P.steps, t, k0, k1, slot)) {
          const Tile T = tile_of<C>(P, plan, t);
          const int row = T.rt * 128;
#pragma unroll 1
          for (int k = k0; k < k1; ++k) {
            if (n >= C::S && !(ok = wait<64>(empty(s), ph, W, kErrStage))) break;
            const uint32_t a = ring + s * C::kStageBytes, b = a + C::kABytes;
            if (n >= early) {
              qlk::mbar_arrive_expect_tx(full(s), C::kABytes + T.bn * 128);
              copy_3d<false>(a, &maps.w, BWD ? row : k * 128, BWD ? k * 128 : row, T.e, full(s));
            }
            int at = 0;
#pragma unroll
            for (int i = 0; i < 3; ++i) {  // 64, 32 and 16 rows
              const int rows = 64 >> i;
              if (rows > BNX || !(T.bn & rows)) continue;
              tma_2d(b + at * 128, &maps.q[i + 1], k * 128, T.m0 + at, full(s));
              at += rows;
            }
            ++n;
            if (++s == C::S) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        // no copy is in flight at the end.  (Of a stage whose weights came early and whose rows of
        // q do not any more, since a wait ran out, the bytes on their way have long arrived.)
        for (int i = n > C::S ? n - C::S : 0; i < n; ++i)
          wait<0>(full(i % C::S), (i / C::S) & 1, W, kErrStage, false);
        if (!ok || n < early) qlk::test_delay(kSettleUs);
      }
    } else if (warp == 1) {
      // ---- MMA issue
      qlk::grid_dependency_wait();
      if ((P.test_us >> 16) && wk == 0) qlk::test_delay(P.test_us >> 16);
      int s = 0, ph = 0, a = 0, aph = 1, n = 0;
      bool ok = true;
      while (ok && sg.next(plan, P.steps, t, k0, k1, slot)) {
        const Tile T = tile_of<C>(P, plan, t);
        // (the type fields of e4m3 are zeros, as those of fp16 in kind::f16)
        const uint32_t idesc = idesc_f16(128, T.bn) | (BWD ? kTransposeA : 0u);
#pragma unroll 1
        for (int k = k0; k < k1; ++k, ++n) {
          if (n >= C::kAcc && !(ok = warp_wait<64>(acce(a), aph, W, kErrAcc, lane))) break;
          if (!(ok = warp_wait<64>(full(s), ph, W, kErrStage, lane))) break;
          tc_fence_after();
          const uint32_t pa = ((ring + s * C::kStageBytes) >> 4) | kDescLo;
          const uint32_t pb = pa + (C::kABytes >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma<false>(tmem + a * BNX, pa + (BWD ? 256 : 2) * kk, pb + 2 * kk, idesc, kk != 0);
            tc_commit<false>(empty(s));
            tc_commit<false>(accf(a));
          }
          __syncwarp();
          if (++s == C::S) {
            s = 0;
            ph ^= 1;
          }
          if (++a == C::kAcc) {
            a = 0;
            aph ^= 1;
          }
        }
      }
      if (n > 0) {
        if (elect_one()) tc_commit<false>(fin);
        __syncwarp();
        warp_wait<0>(fin, 0, W, kErrAcc, lane, false);
      }
    } else if (warp == 2) {
      // ---- products of scales: columns lane + 32 i of the tile, four steps in registers while the
      // four before them are handed out
      constexpr int kPer = (BNX + 31) / 32, kAhead = 4;
      qlk::grid_dependency_wait();
      int a = 0, aph = 1, n = 0;
      bool ok = true;
      while (ok && sg.next(plan, P.steps, t, k0, k1, slot)) {
        const Tile T = tile_of<C>(P, plan, t);
        const float* sw =
            P.sw + (size_t)T.e * P.nb * P.kb + (size_t)T.rt * (BWD ? 1 : P.kb);
        const int hop = BWD ? P.kb : 1;
        const float* sx = P.sx + (size_t)(T.m0 + lane) * P.steps;
        const size_t skip = (size_t)32 * P.steps;
        float v[kPer][kAhead], w[kAhead];
        auto load = [&](int k) {
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            const bool in = k + j < k1;
            w[j] = in ? __ldg(sw + (size_t)(k + j) * hop) : 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
              v[i][j] = in && lane + 32 * i < T.rows ? __ldcg(sx + i * skip + k + j) : 0.f;
          }
        };
        load(k0);
#pragma unroll 1
        for (int k = k0; ok && k < k1; k += kAhead) {
          float s[kPer][kAhead];
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int i = 0; i < kPer; ++i) s[i][j] = v[i][j] * w[j];
          load(k + kAhead);
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            if (k + j >= k1) break;
            if (n >= C::kAcc && !(ok = warp_wait<64>(sempty(a), aph, W, kErrAcc, lane))) break;
            float* o = reinterpret_cast<float*>(smem + C::kScaleOff) + a * BNX + lane;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
              if (lane + 32 * i < BNX) o[32 * i] = s[i][j];
            __syncwarp();
            if (lane == 0) qlk::mbar_arrive(accf(a));
            ++n;
            if (++a == C::kAcc) {
              a = 0;
              aph ^= 1;
            }
          }
        }
      }
    }
  } else {
    // ---- epilogue: accumulator lanes 32 q .. 32 q + 31
    qlk::grid_dependency_wait();
    constexpr int kChunks = BNX / 16;
    const int q = warp & 3;
    const long long U = (long long)(plan.tiles - plan.whole) * P.steps;
    const uint32_t staging = ring + C::kStagingOff + q * C::kStaging;
    int a = 0, aph = 0;
    bool ok = true;
    while (ok && sg.next(plan, P.steps, t, k0, k1, slot)) {
      const Tile T = tile_of<C>(P, plan, t);
      const int chunks = T.bn / 16;
      pair_t acc[kChunks][2][2][2];                 // [chunk][16 lanes][8 columns][8 lanes]
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[c][i >> 2][(i >> 1) & 1][i & 1] = 0ull;
#pragma unroll 1
      for (int k = k0; k < k1; ++k) {
        if (!(ok = warp_wait<256>(accf(a), aph, W, kErrAcc, lane))) break;
        tc_fence_after();
        const uint32_t ta = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(a * BNX);
        const uint32_t sa = ring + C::kScaleOff + 4 * (a * BNX + 2 * (lane & 3));
        uint32_t r[2][2][8];
        tmem_ld_16x16(ta, r[0][0]);
        tmem_ld_16x16(ta + (16u << 16), r[0][1]);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c < chunks) {
            const pair_t s0 = lds_pair(sa + 64 * c), s1 = lds_pair(sa + 64 * c + 32);
            wait_loads(r[c & 1][0], r[c & 1][1]);
            if (c + 1 < kChunks && c + 1 < chunks) {
              tmem_ld_16x16(ta + 16 * (c + 1), r[(c + 1) & 1][0]);
              tmem_ld_16x16(ta + 16 * (c + 1) + (16u << 16), r[(c + 1) & 1][1]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  add_scaled(acc[c][h][i][e], r[c & 1][h][4 * i + 2 * e],
                             r[c & 1][h][4 * i + 2 * e + 1], i ? s1 : s0);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          qlk::mbar_arrive(acce(a));
          qlk::mbar_arrive(sempty(a));
        }
        if (++a == C::kAcc) {
          a = 0;
          aph ^= 1;
        }
      }
      if (!ok) break;
      if (k0 != 0 || k1 != P.steps) {
        // part of a tile: the last contributor goes on, with the sums of all
        constexpr size_t kWarpBytes = (size_t)32 * BNX * 4;
        uint8_t* base = reinterpret_cast<uint8_t*>(P.partials) + q * kWarpBytes + 16 * lane;
        constexpr size_t kSlot = C::kEpiWarps * kWarpBytes;
        uint8_t* mine = base + (size_t)(2 * blockIdx.x + slot) * kSlot;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (c < chunks)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                __stcg(reinterpret_cast<ulonglong2*>(mine + (size_t)(4 * c + 2 * h + i) * 512),
                       make_ulonglong2(acc[c][h][i][0], acc[c][h][i][1]));
        __syncwarp();
        const long long ub = (long long)(t - plan.whole) * P.steps;
        const int wf = worker_of(ub, U, plan.runners);
        const int wl = worker_of(ub + P.steps - 1, U, plan.runners);
        uint32_t* counter = P.counters + (size_t)(t - plan.whole) * C::kEpiWarps + q;
        uint32_t prev = 0;
        if (lane == 0) prev = arrive_weight(counter, 1u);
        prev = __shfl_sync(0xffffffffu, prev, 0);
        if (prev != (uint32_t)(wl - wf)) continue;
        __syncwarp();
        // slot 0 of every contributor (their runs start in this tile), but slot 1 of one whose run
        // started in an earlier tile
        const int first = run_begin(wf, U, plan.runners) >= ub ? 0 : 1;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (c < chunks)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[c][i >> 2][(i >> 1) & 1][i & 1] = 0ull;
#pragma unroll 1
        for (int w = wf; w <= wl; ++w) {
          const uint8_t* src = base + (size_t)(2 * w + (w == wf ? first : 0)) * kSlot;
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < chunks)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const ulonglong2 v = __ldcg(
                      reinterpret_cast<const ulonglong2*>(src + (size_t)(4 * c + 2 * h + i) * 512));
                  acc[c][h][i][0] = add_pairs(acc[c][h][i][0], v.x);
                  acc[c][h][i][1] = add_pairs(acc[c][h][i][1], v.y);
                }
        }
        if (lane == 0) *counter = 0u;  // ready for the next call
      }
      // 16 rows of q at a time through shared memory: 64 contiguous bytes of a row of y per warp
      const int n = T.rt * 128 + 32 * q + 8 * (lane & 3);
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        if (c < chunks) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 v = halves(acc[c][j >> 1][i][j & 1]);
              p[j] = P.bf16 ? pack2<true>(v.x, v.y) : pack2<false>(v.x, v.y);
            }
            store_transposed(staging + (8 * i + (lane & 7)) * kTokStride + (lane >> 3) * 16, p);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int row = 16 * c + 8 * i + (lane >> 2);
            const uint4 v =
                qlk::lds128(staging + (8 * i + (lane >> 2)) * kTokStride + (lane & 3) * 16);
            if (row < T.rows && n < P.R)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.y) + (size_t)(T.m0 + row) * P.R +
                                        n) = v;
          }
        }
    }
  }

  tc_fence_before();
  sync_all<false>();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<false>(tmem, C::kTmemCols);
  }
}

// --------------------------------------------------------------------------- Many rows of q: they
// are the MMA's A operand, 128 per CTA, and 256 of D's rows its B operand.  A thread of the
// epilogue holds a row of q and 128 of D's rows, one block of the weights: a step has one product
// of scales per thread.  (The other way round a step's scales are as many shared loads as a quarter
// of its multiply-adds: 585 against 346 cycles.)
//
// PAIR: a cluster of two CTAs on two SMs computes a tile of 256 rows of q with tcgen05
// cta_group::2; each copies its 128 rows and one of the two blocks of weights, 64 KB a step for
// both, which the L2 gives in about 0.40 us.  Single CTAs copy both blocks, 48 KB: weights come at
// twice the rate, rows of q in tiles of 128.  They take calls of up to 128 rows, which the weights
// bound (128 x 8192 x 28672 56 against 68 us; 200 x 8192 x 8192 31.6 against 28.9), and of up to
// 288 per expert, whose last tiles are half as empty.  (Random splits: 64 experts of 2048 x 4096,
// 256 rows each 221 against 230 us, 312 rows 252 against 249, backward 272 against 266, 512 rows
// 378 against 371; 8 of 14336 x 4096, backward, 256 rows 194 against 202, 312 rows 222 against
// 233, 437 rows 280 against 270.  Where the two are equal goes by how the tiles fill the last wave:
// between 300 and 400 rows here.)
//
// A step of a pair takes 0.54 us and more: 512 cycles of MMAs, the copies' 0.40 us, and in the
// epilogue 128 multiply-adds of two warps to a scheduler, 346 cycles, which overlap but for what
// the way of an accumulator from the MMAs to the epilogue and back costs, with two of them in
// tensor memory. Without the multiply-adds 4096 x 28672 x 8192 takes 737 us, without the MMAs 692,
// with the copies alone 624.  Measured and left: packed multiply-adds (988 us: the pairs' registers
// spill), two accumulators of 128 columns a step (909), sixteen epilogue warps (887), polls instead
// of suspended waits (892), one warp to issue the MMAs (885).  Two warps issue them, a step each in
// turn.
//
// Warps: 0 copies, 1 and 3 MMA issue (1 the tensor memory), 2 scales, 4 .. 11 epilogue.
template <bool PAIR_>
struct Wide {
  static constexpr bool PAIR = PAIR_;
  static constexpr int kCtas = PAIR ? 2 : 1, kBlocks = 2, kBRows = 128, kPerSm = 1;
  static constexpr int BNX = 128 * kCtas;          // rows of q per tile
  static constexpr int kBytes = 128 * 128;         // of 128 rows of an operand, per step
  static constexpr int kOwn = 2 / kCtas;           // of the tile's two blocks of weights, a CTA's
  static constexpr int kStageBytes = (1 + kOwn) * kBytes, S = 200 * 1024 / kStageBytes;
  static_assert(S % 2 == 0, "a stage's barrier is always the same MMA warp's (a parity wait)");
  static constexpr int kEpiWarps = 8, kEpiWarp0 = 4;
  static constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
  static constexpr int kAcc = 2;
  static constexpr size_t kTileBytes = 128 * 256 * 4;  // of a CTA's sums
  static constexpr int kStagingOff = S * kStageBytes;
  static constexpr int kStaging = 32 * kTokStride; // per epilogue warp: 32 rows of 32 columns
  static constexpr int kScaleWarps = 1;
  // products of scales [kAcc][2 blocks][128 rows]
  static constexpr int kScaleOff = kStagingOff + kEpiWarps * kStaging;
  static constexpr int kBarOff = kScaleOff + kAcc * 256 * 4;
  // full[S] empty[S] accf[2] acce[2] sempty[2] fin[2]
  static constexpr int kBars = 2 * S + 4 * kAcc;
  static constexpr int kMiscOff = kBarOff + 8 * kBars;
  static constexpr int kTableOff = kMiscOff + 16;
  static constexpr int smem(int E) { return kTableOff + 8 * (E + 1); }
  static constexpr int kMaxSmem = kTableOff + 8 * (kMaxExperts + 1);
  static_assert(kMaxSmem <= 232448, "shared memory");
  // setmaxnreg: the epilogue's threads hold 128 sums each
  static constexpr int kRegsEpi = 216, kRegsOther = 72;
  static_assert(kThreads == 384 && 2 * kRegsEpi + kRegsOther <= 3 * 168, "registers");
};

template <bool PAIR, bool BWD>
__global__ void __launch_bounds__(Wide<PAIR>::kThreads, 1)
    fp8_wide_kernel(const Params P, const __grid_constant__ Maps maps) {
  using C = Wide<PAIR>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t ring = qlk::smem_addr(smem);
  const uint32_t bars = ring + C::kBarOff;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (C::S + s); };
  auto accf = [&](int a) { return bars + 8 * (2 * C::S + a); };
  auto acce = [&](int a) { return bars + 8 * (2 * C::S + C::kAcc + a); };
  auto sempty = [&](int a) { return bars + 8 * (2 * C::S + 2 * C::kAcc + a); };
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::kMiscOff);
  int* const start = reinterpret_cast<int*>(smem + C::kTableOff);
  int* const pre = start + P.E + 1;
  const WaitCtx W{ring + C::kMiscOff + 4, P.err, P.wait_us};
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? blockIdx.x & 1u : 0u;  // of the cluster (2, 1, 1)
  const bool leader = rank == 0;
  const int wk = (int)blockIdx.x / C::kCtas, nwk = (int)gridDim.x / C::kCtas;
  auto lead = [&](uint32_t b) { return PAIR && !leader ? cluster_addr(b, 0) : b; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) {
      qlk::mbar_init(full(s), 1);
      qlk::mbar_init(empty(s), 1);
    }
    for (int a = 0; a < C::kAcc; ++a) {
      qlk::mbar_init(accf(a), 1 + C::kScaleWarps);
      qlk::mbar_init(acce(a), C::kCtas * C::kEpiWarps);
      qlk::mbar_init(sempty(a), C::kEpiWarps);
      qlk::mbar_init(bars + 8 * (2 * C::S + 3 * C::kAcc + a), 1);  // fin
    }
    misc[1] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) make_table<C::BNX>(P, start, pre, lane);
  sync_all<PAIR>();
  if (warp == 1) tmem_alloc<PAIR>(ring + C::kMiscOff, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  qlk::grid_dependents_launch();  // (behind the allocation: the next grid's must not come first)

  Plan plan{start, pre, pre[P.E], 0, 0};
  schedule<PAIR>(plan, P.steps, nwk);
  Segments sg;
  sg.init(plan, P.steps, wk, nwk);
  int t, k0, k1, slot = 0;

  if (warp < C::kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == 0) {
      // ---- copies
      if (lane == 0) {
        int s = 0, ph = 1, n = 0;
        bool ok = true;
        qlk::grid_dependency_wait();
        if ((P.test_us & 0xFFFFu) && wk == 0) qlk::test_delay(P.test_us & 0xFFFFu);
        while (ok && sg.next(plan, P.steps, t, k0, k1, slot)) {
          const Tile T = wide_tile_of<C>(P, plan, t);
          const int row = (T.rt * 2 + (int)rank * C::kOwn) * 128;  // of D
          // rows of q that the CTAs copy, in units of 32 (the others' products are not stored)
          const int need = (T.rows + 31) & ~31, mine = min(max(need - (int)rank * 128, 0), 128);
          const uint32_t bytes = 2 * C::kBytes + need * 128;  // of both CTAs of a pair
#pragma unroll 1
          for (int k = k0; k < k1; ++k) {
            if (n >= C::S && !(ok = wait<64>(empty(s), ph, W, kErrStage))) break;
            const uint32_t a = ring + s * C::kStageBytes;
            if (leader) qlk::mbar_arrive_expect_tx(full(s), bytes);
            int at = 0;
#pragma unroll
            for (int i = 0; i < 3; ++i) {  // 128, 64 and 32 rows
              if (!(mine & (128 >> i))) continue;
              const int m = T.m0 + (int)rank * 128 + at;
              if constexpr (PAIR)
                tma_2d_pair(a + at * 128, &maps.q[i], k * 128, m, lead(full(s)));
              else
                tma_2d(a + at * 128, &maps.q[i], k * 128, m, full(s));
              at += 128 >> i;
            }
#pragma unroll
            for (int b = 0; b < C::kOwn; ++b) {
              const int r = row + b * 128;
              copy_3d<PAIR>(a + (1 + b) * C::kBytes, &maps.w, BWD ? r : k * 128,
                            BWD ? k * 128 : r, T.e, lead(full(s)));
            }
            ++n;
            if (++s == C::S) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        // (as in fp8_tc_kernel)
        for (int i = n > C::S ? n - C::S : 0; ok && i < n; ++i)
          ok = wait<0>(empty(i % C::S), (i / C::S) & 1, W, kErrStage);
        if (leader)
          for (int i = n > C::S ? n - C::S : 0; i < n; ++i)
            wait<0>(full(i % C::S), (i / C::S) & 1, W, kErrStage, false);
        if (PAIR && !ok) qlk::test_delay(kSettleUs);
      }
    } else if (warp & 1) {
      // ---- MMA issue by the leader: warp 1 the even steps, warp 3 the odd ones, an accumulator
      // each. What a warp takes to see its barriers complete and to issue is then hidden behind the
      // other step's MMAs.
      if (leader) {
        qlk::grid_dependency_wait();
        if ((P.test_us >> 16) && wk == 0) qlk::test_delay(P.test_us >> 16);
        constexpr uint32_t idesc = idesc_f16(128 * C::kCtas, 256) | (BWD ? kTransposeB : 0u);
        // (read MN-major a single CTA's two blocks of the weights are panels 16384 bytes apart)
        constexpr uint32_t kDescLoB = BWD ? (uint32_t)(C::kBytes / 16) << 16 : kDescLo;
        const int a = warp >> 1;
        const uint32_t fin = bars + 8 * (2 * C::S + 3 * C::kAcc + a);
        int s = a, ph = 0, aph = 1, n = 0;
        bool ok = true, mine = a == 0;
        while (ok && sg.next(plan, P.steps, t, k0, k1, slot)) {
#pragma unroll 1
          for (int k = k0; k < k1; ++k, mine = !mine) {
            if (!mine) continue;
            if (!(ok = warp_wait<0>(full(s), ph, W, kErrStage, lane))) break;
            if (n > 0 && !(ok = warp_wait<0>(acce(a), aph, W, kErrAcc, lane))) break;
            tc_fence_after();
            const uint32_t st = (ring + s * C::kStageBytes) >> 4;
            const uint32_t pa = st | kDescLo, pb = (st + (C::kBytes >> 4)) | kDescLoB;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma<PAIR>(tmem + a * 256, pa + 2 * kk, pb + (BWD ? 256 : 2) * kk, idesc, kk != 0);
              commit_both<PAIR>(accf(a));
              commit_both<PAIR>(empty(s));
            }
            __syncwarp();
            ++n;
            aph ^= 1;
            if ((s += 2) >= C::S) {
              s -= C::S;
              ph ^= 1;
            }
          }
        }
        if (n > 0) {
          if (elect_one()) tc_commit<PAIR>(fin);
          __syncwarp();
          warp_wait<0>(fin, 0, W, kErrAcc, lane, false);
        }
        if (PAIR && (!ok || misc[1])) qlk::test_delay(kSettleUs);
      }
    } else {
      // ---- products of scales: rows 32 i + lane of this CTA's, by both blocks of the weights.
      // Two steps at a time, the next two on their way while they are handed out.
      qlk::grid_dependency_wait();
      int a = 0, aph = 1, n = 0;
      bool ok = true;
      while (ok && sg.next(plan, P.steps, t, k0, k1, slot)) {
        const Tile T = wide_tile_of<C>(P, plan, t);
        const int last = T.rows - 1 - (int)rank * 128, least = -(int)rank * 128;
        const float* sx = P.sx + (size_t)(T.m0 - least) * P.steps;
        int row[4];  // of the tile's rows, in scales
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = max(min(lane + 32 * i, last), least) * P.steps;
        // the blocks of the weights (the second may lie behind the last: any scale does)
        const float* sw =
            P.sw + (size_t)T.e * P.nb * P.kb + (size_t)(2 * T.rt) * (BWD ? 1 : P.kb);
        const int other = 2 * T.rt + 1 < (BWD ? P.kb : P.nb) ? (BWD ? 1 : P.kb) : 0;
        const int hop = BWD ? P.kb : 1;
        float v[4][2], w[2][2];
        auto load = [&](int k) {  // steps k, k + 1, k even
          if (k >= k1) return;
          const int k2 = min(k + 1, P.steps - 1);
          w[0][0] = __ldg(sw + (size_t)k * hop);
          w[0][1] = __ldg(sw + (size_t)k2 * hop);
          w[1][0] = __ldg(sw + other + (size_t)k * hop);
          w[1][1] = __ldg(sw + other + (size_t)k2 * hop);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (P.vec == 2) {
              const float2 x = __ldcg(reinterpret_cast<const float2*>(sx + row[i] + k));
              v[i][0] = x.x;
              v[i][1] = x.y;
            } else {
              v[i][0] = __ldcg(sx + row[i] + k);
              v[i][1] = __ldcg(sx + row[i] + k2);
            }
          }
        };
        load(k0 & ~1);
#pragma unroll 1
        for (int k = k0 & ~1; ok && k < k1; k += 2) {
          float f[2][8];  // [step][block of the weights, row]
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) f[j][i] = v[i & 3][j] * w[i >> 2][j];
          load(k + 2);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (k + j < k0 || k + j >= k1) continue;
            if (n >= C::kAcc && !(ok = warp_wait<0>(sempty(a), aph, W, kErrAcc, lane))) break;
            float* o = reinterpret_cast<float*>(smem + C::kScaleOff) + a * 256 + lane;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[32 * i] = f[j][i];
            __syncwarp();
            if (lane == 0) qlk::mbar_arrive(accf(a));
            ++n;
            if (++a == C::kAcc) {
              a = 0;
              aph ^= 1;
            }
          }
        }
      }
    }
  } else {
    // ---- epilogue: rows 32 q + lane of this CTA's rows of q, columns of group g
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsEpi));
    qlk::grid_dependency_wait();
    const int ew = warp - C::kEpiWarp0, q = warp & 3, g = ew >> 2;
    const long long U = (long long)(plan.tiles - plan.whole) * P.steps;
    const uint32_t staging = ring + C::kStagingOff + ew * C::kStaging;
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(g * 128);
    const uint32_t sq = ring + C::kScaleOff + 4 * (128 * g + 32 * q + lane);
    const uint32_t free = lead(acce(0));  // the leader's
    int a = 0, aph = 0;
    bool ok = true;
    while (ok && sg.next(plan, P.steps, t, k0, k1, slot)) {
      const Tile T = wide_tile_of<C>(P, plan, t);
      float acc[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) acc[c] = 0.f;
#pragma unroll 1
      for (int k = k0; k < k1; ++k) {
        if (!(ok = warp_wait<0>(accf(a), aph, W, kErrAcc, lane))) break;
        tc_fence_after();
        const uint32_t ta = tq + (uint32_t)(a * 256);
        uint32_t r[2][32];
        tmem_ld_32x32(ta, r[0]);
        const float f = __uint_as_float(qlk::lds32(sq + a * 1024));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          wait_loads(r[c & 1]);
          if (c < 3) {
            tmem_ld_32x32(ta + 32 * (c + 1), r[(c + 1) & 1]);
          } else {  // the accumulator is free
            tc_fence_before();
            __syncwarp();
            // (the loads have completed, nothing in memory is to be ordered: the other CTA's arrival
            // says only when, and the default scope is enough, see arrive_stage in fused_tc.cu)
            arrive_both(free + 8 * a, sempty(0) + 8 * a, lane);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i)
            acc[32 * c + i] = fmaf(__uint_as_float(r[c & 1][i]), f, acc[32 * c + i]);
        }
        if (++a == C::kAcc) {
          a = 0;
          aph ^= 1;
        }
      }
      if (!ok) break;
      if (k0 != 0 || k1 != P.steps) {
        // part of a tile (as in fp8_tc_kernel)
        constexpr size_t kWarpBytes = 32 * 128 * 4, kSlot = C::kEpiWarps * kWarpBytes;
        uint8_t* base = reinterpret_cast<uint8_t*>(P.partials) + ew * kWarpBytes + 16 * lane;
        uint8_t* mine = base + (size_t)(2 * blockIdx.x + slot) * kSlot;
#pragma unroll
        for (int c = 0; c < 32; ++c)
          __stcg(reinterpret_cast<float4*>(mine + c * 512),
                 make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]));
        __syncwarp();
        const long long ub = (long long)(t - plan.whole) * P.steps;
        const int wf = worker_of(ub, U, plan.runners);
        const int wl = worker_of(ub + P.steps - 1, U, plan.runners);
        uint32_t* counter =
            P.counters + ((size_t)(t - plan.whole) * C::kCtas + rank) * C::kEpiWarps + ew;
        uint32_t prev = 0;
        if (lane == 0) prev = arrive_weight(counter, 1u);
        prev = __shfl_sync(0xffffffffu, prev, 0);
        if (prev != (uint32_t)(wl - wf)) continue;
        __syncwarp();
        const int first = run_begin(wf, U, plan.runners) >= ub ? 0 : 1;
#pragma unroll
        for (int c = 0; c < 128; ++c) acc[c] = 0.f;
#pragma unroll 1
        for (int w2 = wf; w2 <= wl; ++w2) {
          const uint8_t* src =
              base + (size_t)(2 * (w2 * C::kCtas + (int)rank) + (w2 == wf ? first : 0)) * kSlot;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(src + c * 512));
            acc[4 * c] += x.x;
            acc[4 * c + 1] += x.y;
            acc[4 * c + 2] += x.z;
            acc[4 * c + 3] += x.w;
          }
        }
        if (lane == 0) *counter = 0u;  // ready for the next call
      }
      // 32 columns at a time through shared memory: 64 contiguous bytes of a row of y per warp
      const int m = T.m0 + (int)rank * 128 + 32 * q + (lane >> 2);
      const int n = (T.rt * 2 + g) * 128 + 8 * (lane & 3);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x0 = acc[32 * c + 8 * i + 2 * j], x1 = acc[32 * c + 8 * i + 2 * j + 1];
            p[j] = P.bf16 ? pack2<true>(x0, x1) : pack2<false>(x0, x1);
          }
          sts128(staging + lane * kTokStride + 16 * i, make_uint4(p[0], p[1], p[2], p[3]));
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x =
              qlk::lds128(staging + (8 * i + (lane >> 2)) * kTokStride + 16 * (lane & 3));
          if (m + 8 * i < T.m0 + T.rows && n + 32 * c < P.R)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.y) + (size_t)(m + 8 * i) * P.R + n +
                                      32 * c) = x;
        }
      }
    }
  }

  tc_fence_before();
  sync_all<PAIR>();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<PAIR>(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// host side

constexpr int kMaxDevices = 64;

bool encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, int box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return false;
  const cuuint64_t strides[2] = {dims[0], dims[0] * dims[1]};
  const cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// attr: two entries, the cluster first (the occupancy query takes that one alone)
template <class C>
void launch_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, unsigned ctas, int E,
                   cudaStream_t st) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3(ctas);
  cfg->blockDim = dim3(C::kThreads);
  cfg->dynamicSmemBytes = C::smem(E);
  cfg->stream = st;
  int n = 0;
  if constexpr (C::kCtas == 2) {
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

using Kernel = void (*)(const Params, const Maps);
constexpr int kLongRun = 8;

// Workers resident at once, once per kernel and device.
template <class C, Kernel kernel>
int resident_workers(int dev, int sms) {
  static std::atomic<int> known[kMaxDevices];
  if (dev < 0 || dev >= kMaxDevices) return 0;
  int n = known[dev].load(std::memory_order_acquire);
  if (n > 0) return n;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kMaxSmem) !=
      cudaSuccess)
    return 0;
  if constexpr (C::kCtas == 2) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    launch_config<C>(&cfg, attr, 2 * (sms / 2), kMaxExperts, nullptr);
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
  } else {
    // (the query answers 1 for every kernel that allocates tensor memory; two do run at once, as
    // timestamps show, and nothing rests on it)
    int occ = 0;
    n = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, C::kThreads, C::kMaxSmem) ==
                    cudaSuccess && occ >= 1
            ? sms
            : 0;
  }
  if (n > 0) known[dev].store(n, std::memory_order_release);
  return n;
}

// C: rows of q (BNX) and blocks of 128 rows of D (kBlocks) per tile.
template <class C, Kernel kernel, bool BWD>
ql_status launch_as(const Product& p) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return QL_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return QL_ERR_CUDA;
  const int maxw = resident_workers<C, kernel>(dev, sms);
  if (maxw <= 0) return QL_ERR_CUDA;
  Params P;
  P.sx = p.sx;
  P.sw = p.sw;
  P.offsets = p.offsets;
  P.y = p.y;
  P.partials = p.partials;
  P.counters = p.counters;
  P.err = p.err;
  P.M = p.M;
  P.E = p.E;
  P.R = BWD ? p.K : p.N;
  P.nb = blocks_of(p.N);
  P.kb = blocks_of(p.K);
  P.steps = BWD ? P.nb : P.kb;
  P.rtiles = (blocks_of(P.R) + C::kBlocks - 1) / C::kBlocks;
  P.bf16 = p.bf16;
  P.vec = P.steps % 2 == 0 && (uintptr_t)p.sx % 8 == 0 ? 2 : 1;
  // no more tiles than these, whatever the offsets
  const long long tiles = (long long)P.rtiles * (p.offsets ? p.M / C::BNX + (p.E < p.M ? p.E : p.M)
                                                           : (p.M + C::BNX - 1) / C::BNX);
  // (a worker's tile number passes the last one by less than the workers)
  if (tiles >= (1LL << 31) - (1 << 16)) return QL_ERR_SHAPE;
  // (fewer tiles than workers are split)
  if ((size_t)C::kPerSm * maxw * C::kCtas * C::kEpiWarps * sizeof(uint32_t) >
      qfused::kTcCounterBytes)
    return QL_ERR_UNSUPPORTED;
  if (p.partial_bytes < (size_t)2 * C::kPerSm * sms * C::kTileBytes) return QL_ERR_WORKSPACE;
  const qfused::WaitTest wt = qfused::wait_test();
  P.wait_us = (wt.limit_us < 1000000000u ? wt.limit_us : 1000000000u) + 4u * (uint32_t)P.steps;
  P.test_us = wt.delays;
  Maps maps;
  const cuuint64_t wdims[3] = {(cuuint64_t)p.K, (cuuint64_t)p.N, (cuuint64_t)p.E};
  const cuuint64_t qdims[2] = {(cuuint64_t)(BWD ? p.N : p.K), (cuuint64_t)p.M};
  if (!encode(&maps.w, p.w, 3, wdims, 128)) return QL_ERR_CUDA;
  for (int i = 0; i < 4; ++i)  // (narrow tiles: 64, 32 and 16 rows; wide ones: 128, 64 and 32)
    if ((128 >> i) <= C::kBRows && (i < 3 || C::kBRows < 128) &&
        !encode(&maps.q[i], p.q, 2, qdims, 128 >> i))
      return QL_ERR_CUDA;
  // every worker that can run: how many have work is known on the device.  A second CTA on each SM
  // where both have kLongRun steps and more
  const long long units = tiles * P.steps;
  const int most = units >= (long long)2 * maxw * kLongRun && p.E < 256 ? C::kPerSm * maxw : maxw;
  const int workers = units < most ? (int)units : most;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  launch_config<C>(&cfg, attr, (unsigned)(workers * C::kCtas), p.E, p.stream);
  return cudaLaunchKernelEx(&cfg, kernel, P, maps) == cudaSuccess ? QL_OK : QL_ERR_CUDA;
}

template <int BNX, bool BWD>
ql_status launch_narrow(const Product& p) {
  return launch_as<Cfg<BNX>, fp8_tc_kernel<BNX, BWD>, BWD>(p);
}

template <bool BWD>
ql_status launch(const Product& p) {
  const int rows = (p.M + p.E - 1) / p.E;  // of an average expert
  if (rows <= 16) return launch_narrow<16, BWD>(p);
  if (rows <= 32) return launch_narrow<32, BWD>(p);
  if (rows <= 64) return launch_narrow<64, BWD>(p);
  if (rows <= (p.offsets ? 288 : 128))
    return launch_as<Wide<false>, fp8_wide_kernel<false, BWD>, BWD>(p);
  return launch_as<Wide<true>, fp8_wide_kernel<true, BWD>, BWD>(p);
}

}  // namespace

namespace qfp8 {

// Two fp32 partial tiles of 128 rows per CTA (two CTAs to an SM up to 64 rows), of the widest tile
// that a call with at most M rows has.
size_t product_partial_bytes(int M, int E) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  const int rows = (M + E - 1) / E;
  int bn = 16;
  while (bn < 256 && bn < rows) bn *= 2;
  return (size_t)2 * sms * 128 * (bn <= 64 ? 2 * bn : 256) * sizeof(float);
}

ql_status launch_product(const Product& p) {
  return p.backward ? launch<true>(p) : launch<false>(p);
}

}  // namespace qfp8
