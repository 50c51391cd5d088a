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
// Roles of the 24 or 28 warps: 0 copies of x, 1 MMA issue and tensor memory, 2 copies of codes,
// then four or eight epilogue warps, and two teams of eight decoding warps that take the stages
// in turn, so that the latency of one unit's decoding (wait, shared loads, stores, proxy fence,
// arrival) is hidden behind the other's.
//
// PAIR: a cluster of two CTAs on two SMs computes 256 rows with tcgen05 cta_group::2; each CTA
// decodes its own 128 rows and copies half of the tokens, which halves what the tokens cost
// in shared memory and L2.
//
// Work: tiles of 128 (PAIR 256) rows x bn tokens.  Whole waves of tiles go round the
// workers; the remaining tiles are cut into equal parts, or with one whole wave into equal
// runs of stages (schedule), whose partial sums meet in the workspace: the last contributor
// to arrive adds them in worker order, nobody waits.
//
// Measured, W4: 8192 x 8192 with 512 tokens 55 us (1.25 PFLOP/s; the tensor pipe is busy for 76 %
// of the cycles in which an SM has work), 8192 x 18944 with 32 tokens 37 us against 13 us for its
// bytes (decoding: 57 % of the issue slots, the tensor pipe 35 %), 8192 x 28672 with 2048 tokens
// 662 us (1.45 PFLOP/s) in a run of 20 calls; with GELU, bias, residual and the pre-activation kept
// 762 us in such a run, 876 us (1.10 PFLOP/s) call after call for seconds, at the power limit.
//
// The weights and, backward, dz (its rows scaled, fused.cu) are rounded to fp16 once: the operand
// type of kind::f16.  That adds about one rounding each to the output's own (2.1e-4 in the relative
// L2 norm becomes 2.8e-4, with two of them 3.3e-4 to 4.2e-4); keeping dz in two halves would double
// the MMAs.
//
// Every barrier wait is bounded in time (100 ms against microseconds, and 4 us more for each stage
// of a tile, several times what one takes, since the epilogue waits for a whole tile;
// qlinear_debug_wait_test sets another limit); one that runs out sets a flag in the workspace's
// error word, all roles leave their loops, and the CTA waits for its own copies and MMAs, frees its
// tensor memory and exits.
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

// EP: epilogue warps per quadrant of the accumulators.  Two where one would finish a tile later
// than the MMAs the next (launch_fmt), one elsewhere, which leaves the decoding more registers
// (32 x 18944 x 8192: 35.5 against 38.0 us).
template <int BNX_, int FMT_, bool PAIR_, int EP>
struct TcCfg {
  static constexpr int kEpiPer = EP;
  static constexpr int kMembers = kEpiPer + kTeams * kTeamWarps / 4;  // ... with the decoding warps
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
  // A team of decoding warps must follow every phase of a barrier that it waits for (a parity
  // says "this phase or the one before the last"), and the teams take the stages in turn.  So
  // the barriers that tell them of codes in the SC slots and of the S stages handed back are
  // kTeams times as many, each of which then belongs to one team.
  static constexpr int SE = kTeams * S;
  static constexpr int kBudget = 232448 - 768;               // barriers
  static constexpr int SC0 = (kBudget - S * kStageBytes) / kSlot;
  static constexpr int SC = SC0 < 12 ? SC0 : 12;
  static constexpr int SF = kTeams * SC;
  static_assert(SC >= 2, "code ring");
  static constexpr int kRingC = S * kStageBytes;
  static constexpr int kLutOff = kRingC + SC * kSlot;        // LUT4: the table, 64 bytes
  static_assert(FMT != kLUT4 || kLutOff % 256 == 0, "table address");
  static constexpr int kBarOff = kLutOff + (FMT == kLUT4 ? 64 : 0);
  // full[S] empty[SE] accf[2] acce[2] fin cfull[SF] cempty[SC] tail[4][2] last; then the tensor
  // memory's base, the abort flag, arrivals before the last segment's per quadrant
  static constexpr int kTailBar = S + SE + 5 + SF + SC;
  static constexpr int kLastBar = kTailBar + 8;
  static constexpr int kMiscOff = kBarOff + 8 * (kLastBar + 1);
  static constexpr int kSpareOff = kMiscOff + 24;  // a word per decoding warp
  static constexpr int kSmem = kSpareOff + 4 * kTeams * kTeamWarps;
  static_assert(kSmem <= 232448, "shared memory");
  static constexpr int kSpin = BNX == 256 ? 64 : 0;          // polls before a suspended wait
  static constexpr int kEpiWarp0 = 4, kDqWarp0 = kEpiWarp0 + 4 * kEpiPer;
  static constexpr int kWarps = kDqWarp0 + kTeams * kTeamWarps;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr uint32_t kTmemCols = 2 * BNX;
  static constexpr uint32_t kFullCount = 1 + kCtas * kTeamWarps;
  static constexpr uint32_t kAccEmptyCount = kCtas * 4 * kEpiPer;
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
  int runners;                   // workers that share the stages of tiles [whole, tiles)
  uint32_t wait_us;              // limit of a wait (the longest, for a tile, included)
  uint32_t test_us;              // tests of the waits: delays (qfused::WaitTest)
};

__device__ __forceinline__ long long run_begin(int w, long long U, int W) { return w * U / W; }
__device__ __forceinline__ int worker_of(long long u, long long U, int W) {
  return (int)(((u + 1) * W - 1) / U);
}

// The work of a worker (CTA or pair): whole tiles w, w + W, ..., then its run of the stages of
// tiles [whole, tiles), cut at tile boundaries.
struct Segments {
  int t, W;         // next whole tile of this worker, workers
  int rt, rk, left; // the run: next tile and stage, stages left
  bool first;       // no stage of the run has been handed out yet
  __device__ __forceinline__ void init(const TcParams& P, int w, int W_) {
    W = W_;
    t = w;
    const long long U = (long long)(P.tiles - P.whole) * P.steps;
    const long long u = w < P.runners ? run_begin(w, U, P.runners) : 0;  // (no runners: 0 tiles)
    left = w < P.runners ? (int)(run_begin(w + 1, U, P.runners) - u) : 0;
    rt = P.whole + (int)(u / P.steps);
    rk = (int)(u % P.steps);
    first = true;
  }
  // tile, stages [k0, k1); slot: workspace slot of a partial sum (0: the run's first segment)
  __device__ __forceinline__ bool next(const TcParams& P, int& tile, int& k0, int& k1, int& slot) {
    if (t < P.whole) {
      tile = t;
      t += W;
      k0 = 0;
      k1 = P.steps;
      return true;
    }
    if (left <= 0) return false;
    tile = rt++;
    k0 = rk;
    k1 = left < P.steps - rk ? rk + left : P.steps;
    left -= k1 - k0;
    rk = 0;
    slot = first ? 0 : 1;
    first = false;
    return true;
  }
  __device__ __forceinline__ bool done(const TcParams& P) const {  // no segment is left
    return t >= P.whole && left <= 0;
  }
};

// ---------------------------------------------------------------------------
// bounded waits

struct WaitCtx {
  uint32_t abort;  // shared-memory address of the CTA's abort flag
  uint32_t* err;   // global memory
  uint32_t limit_us;
};

// Suspends the thread until the phase completes, or for up to kSuspendNs; whether it completed.
// (Polling instead took as many issue slots as the decoding.)
constexpr uint32_t kSuspendNs = 20000;
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity, bool cluster) {
  uint32_t done;
  if (cluster)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kSuspendNs)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kSuspendNs)
        : "memory");
  return done != 0;
}

// The phase has not completed within one suspension: keep waiting up to the limit, or until
// another role has given up; then set the flag.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint32_t abort, uint32_t* err,
                                       uint32_t limit_us, uint32_t bit, bool honor_abort,
                                       bool cluster) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (try_wait(bar, parity, cluster)) return true;
    if (honor_abort) {
      uint32_t a;
      asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(a) : "r"(abort) : "memory");
      if (a) break;
    }
    if (globaltimer_ns() - t0 > 1000ull * limit_us) break;
  }
  atomicOr(err, bit);
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(1u) : "memory");
  return false;
}

// Waking up from a suspended wait takes hundreds of cycles; polling takes issue slots.  So the
// waits between the pipeline's roles (SPIN > 0) poll SPIN times first where the MMAs set the pace
// (256-token tiles: 190 against 290 us on 1024 x 4096 x 28672 backward) and suspend at once where
// the decoding does (32 rows, 8192 x 18944: 35.1 against 37.6 us).
// CLUSTER: some of the arrivals come from the pair's other CTA (acquire at cluster scope).

// One thread.
template <int SPIN>
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const WaitCtx& w, uint32_t bit,
                                     bool honor_abort = true) {
#pragma unroll 1
  for (int i = 0; i < SPIN; ++i)
    if (mbar_ready(bar, parity, false)) return true;
  return try_wait(bar, parity, false) ||
         wait_slow(bar, parity, w.abort, w.err, w.limit_us, bit, honor_abort, false);
}

// A whole warp: every lane sees the phase complete (the usual case), or one lane waits on.
template <int SPIN, bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtx& w,
                                          uint32_t bit, int lane, bool honor_abort = true) {
#pragma unroll 1
  for (int i = 0; i < SPIN; ++i)
    if (__all_sync(0xffffffffu, mbar_ready(bar, parity, CLUSTER))) return true;
  if (__all_sync(0xffffffffu, try_wait(bar, parity, CLUSTER))) return true;
  bool ok = true;
  if (lane == 0)
    ok = wait_slow(bar, parity, w.abort, w.err, w.limit_us, bit, honor_abort, CLUSTER);
  return __shfl_sync(0xffffffffu, ok, 0);
}

// A role that gave up: what it has sent to the pair's other CTA, or has that CTA's barriers count,
// arrives long before this ends (nothing is left to wait on).
constexpr uint32_t kSettleUs = 20000;

// ---------------------------------------------------------------------------
// decoding: one warp, one 16-column tile of a unit, into rows 16 tile .. 16 tile + 15 of the
// two A panels.  Lane (gi, t) holds, per pair of steps i, the eight k 32 i + 8 t .. + 7 of
// rows gi and gi + 8: granule 4 (i mod 2) + t of panel i / 2.  Lanes with odd gi take the
// pairs in the order 1, 0, 3, 2: the eight lanes of a store phase (two rows, four t) then
// write eight distinct granules, without bank conflicts.

struct Decoded {
  uint4 v[4][2];  // [pair of steps, in the lane's order][row gi, gi + 8]
};

// Eight weights fp16(s (q - z)) of a pair of steps for row half h (see uniform_pair8), with the
// field and the exponent of 2^(10 - shift) put together by one logic operation.
template <int FMT>
__device__ __forceinline__ uint4 uniform8(const uint32_t* w, int h, const __half2 (&zb)[2][2],
                                          __half2 scale) {
  uint32_t o[4];
#pragma unroll
  for (int ss = 0; ss < 2; ++ss)
#pragma unroll
    for (int dkp = 0; dkp < 2; ++dkp) {
      const uint32_t word = FMT == kW8 ? w[2 * ss + h] : FMT == kW2 ? w[0] : w[ss];
      const uint32_t v = dkp ? word >> 8 : word;
      const uint32_t mask = FMT == kW8   ? 0x00FF00FFu
                            : FMT == kW4 ? (h ? 0x00F000F0u : 0x000F000Fu)
                                         : 0x00030003u << (4 * ss + 2 * h);
      const uint32_t magic = qdq::magic_half(qdq::field_shift<FMT>(ss, h)) * 0x10001u;
      uint32_t f;
      asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(f) : "r"(v), "r"(mask), "r"(magic));
      o[2 * ss + dkp] = qdq::h2_as_u32(__hmul2(__hsub2(qdq::u32_as_h2(f), zb[ss][h]), scale));
    }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// LUT4: eight weights fp16(fp32(lut[q]) * absmax) of a pair of steps for row half h (see
// lut_pair8).  `table`: shared-memory address of the 16 entries in fp32, a multiple of 256, so
// that a byte permute of the codes (times 4, by two shifts a word) makes the address of an entry.
// Entries lie in different banks.  (Looked up by byte permutes in registers instead, with no
// shared loads, it took 107 against 88 us: 64 x 28672 x 8192.)
__device__ __forceinline__ uint4 lut8(uint32_t table, const uint32_t* w, int h, float a) {
  uint32_t o[4];
#pragma unroll
  for (int ss = 0; ss < 2; ++ss) {
    const uint32_t even = (w[ss] << 2) & 0x3C3C3C3Cu, odd = (w[ss] >> 2) & 0x3C3C3C3Cu;
#pragma unroll
    for (int dkp = 0; dkp < 2; ++dkp) {
      const uint32_t byte = 0x7650u + h + 2 * dkp;
      const float lo = __uint_as_float(qlk::lds32(__byte_perm(even, table, byte)));
      const float hi = __uint_as_float(qlk::lds32(__byte_perm(odd, table, byte)));
      o[2 * ss + dkp] = qdq::h2_as_u32(__floats2half2_rn(__fmul_rn(lo, a), __fmul_rn(hi, a)));
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The code slot is handed back (`release`, `spare`: a shared word of the warp) as soon as every
// lane holds its words.  The barrier arrival does not wait for shared loads in flight; the
// store of a value made from all of them does, and the arrival comes after it.
template <class C>
__device__ __forceinline__ void decode_tile(uint32_t slot, int tile, int lane, uint32_t table,
                                            uint32_t release, uint32_t spare, Decoded& d) {
  constexpr int FMT = C::FMT;
  constexpr int KW = qlk::Fmt<FMT>::kWords, KP = KW / 4;  // words per lane, per step pair
  const int gi = lane >> 2;
  const int swap = gi & 1;
  uint32_t w[KW];
  const uint32_t cs = slot + tile * C::kChunk + lane * 16;
  if constexpr (FMT == kW8) {  // a quad is a pair: the order is in the address
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
  uint4 am = make_uint4(0, 0, 0, 0);  // LUT4 [64-block][row half]; else scales, zeros
  if constexpr (FMT == kLUT4) {
    am = qlk::lds128(pa + gi * 16);
  } else {
    am.x = qlk::lds32(pa + gi * 4);
    am.y = qlk::lds32(pa + kBlockTiles * C::kParChunk + gi * 4);
  }
  uint32_t all = am.x ^ am.y ^ am.z ^ am.w;
#pragma unroll
  for (int k = 0; k < KW; ++k) all ^= w[k];
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(spare), "r"(all) : "memory");
  __syncwarp();
  if (lane == 0) qlk::mbar_arrive(release);
  if constexpr (FMT == kLUT4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        d.v[i][h] = lut8(table, w + KP * i, h,
                         __uint_as_float(i >= 2 ? (h ? am.w : am.z) : (h ? am.y : am.x)));
  } else {
    const __half2 s2 = qdq::u32_as_h2(am.x), z2 = qdq::u32_as_h2(am.y);
    // z + 2^(10 - shift): exact in fp16 for integer zeros up to 1024
    __half2 zb[2][2];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        zb[p][h] = __hadd2(h ? __high2half2(z2) : __low2half2(z2),
                           qdq::u32_as_h2(qdq::magic_half(qdq::field_shift<FMT>(p, h)) * 0x10001u));
    const __half2 sl = __low2half2(s2), sh = __high2half2(s2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        d.v[i][h] = uniform8<FMT>(w + KP * i, h, zb, h ? sh : sl);
  }
}

__device__ __forceinline__ void store_tile(uint32_t a, int tile, int lane, const Decoded& d) {
  const int gi = lane >> 2, t = lane & 3;
  const uint32_t row = a + (16 * tile + gi) * 128;
  // granule 4 (pair mod 2) + t of a row, at granule ^ (row mod 8) = ^ gi
  const uint32_t g0 = ((uint32_t)((4 * (gi & 1) + t) ^ gi)) << 4, g1 = g0 ^ 64u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      sts128(row + (i >> 1) * (128 * 128) + h * 8 * 128 + ((i & 1) ? g1 : g0), d.v[i][h]);
}

// ---------------------------------------------------------------------------
// epilogue: kTok tokens m0 .. (the first `count` of them real) of one row per lane

constexpr int kTok = 8;

// Between "one row, two tokens" and "two rows, one token" (packed fp16): lanes l and l ^ 1 hold
// neighbouring rows; the even one ends up with the first token of both, the odd one with the
// second.  The same exchange goes back.
__device__ __forceinline__ uint32_t exchange_rows(uint32_t v, int lane) {
  const uint32_t o = __shfl_xor_sync(0xffffffffu, v, 1);
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(o), "r"((lane & 1) ? 0x3276u : 0x5410u));
  return r;
}

// The warp's values of N tokens, the first `count` of them real, `stride` elements apart; `o`
// points at token 0 of the lane's row, `in`: the row exists.  Two rows in one 4-byte store.
template <int N>
__device__ __forceinline__ void store_tokens(__half* o, size_t stride, const float (&v)[N],
                                             int count, int lane, bool in) {
  const int odd = lane & 1;
  __half* p = o + odd * stride - odd;
#pragma unroll
  for (int e = 0; e < N; e += 2, p += 2 * stride) {
    const __half2 h = __floats2half2_rn(v[e], v[e + 1]);
    const uint32_t w = exchange_rows(qdq::h2_as_u32(h), lane);
    if (in && e + odd < count) *reinterpret_cast<uint32_t*>(p) = w;
  }
}

template <int ACT, int N>
__device__ __forceinline__ void act_each(float (&v)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = qact::act_forward(ACT, v[e]);
}
template <int N>
__device__ __forceinline__ void act_all(int act, float (&v)[N]) {  // one branch for all values
  switch (act) {
    case QL_ACT_RELU: return act_each<QL_ACT_RELU>(v);
    case QL_ACT_GELU: return act_each<QL_ACT_GELU>(v);
    case QL_ACT_GELU_TANH: return act_each<QL_ACT_GELU_TANH>(v);
    case QL_ACT_SILU: return act_each<QL_ACT_SILU>(v);
    default: return;
  }
}

// rows alternate 16 gate / 16 up: the lanes exchange, per pair of tokens, so that the gate
// lanes finish the even token and the up lanes the odd one
__device__ __forceinline__ void finish_gated(const TcParams& P, float (&v)[kTok], int m0, int count,
                                             int row, float bias, int lane) {
  const qfused::Epilogue& E = P.epi;
  const bool in = row < P.rows;
  const int F = P.ld, f = (row >> 5) * 16 + (row & 15), up = (row >> 4) & 1;
#pragma unroll
  for (int e = 0; e < kTok; ++e) v[e] += bias;
  if (E.zsave)
    store_tokens(E.zsave + ((size_t)m0 * 2 + up) * F + f, (size_t)2 * F, v, count, lane, in);
  float g[kTok / 2], u[kTok / 2];
#pragma unroll
  for (int e = 0; e < kTok / 2; ++e) {
    const float other = __shfl_xor_sync(0xffffffffu, up ? v[2 * e] : v[2 * e + 1], 16);
    g[e] = up ? other : v[2 * e];
    u[e] = up ? v[2 * e + 1] : other;
  }
  act_all(E.act, g);
#pragma unroll
  for (int e = 0; e < kTok / 2; ++e) g[e] *= u[e];
  // this lane's tokens: up, up + 2, ..
  store_tokens(E.y + (size_t)(m0 + up) * F + f, (size_t)2 * F, g, (count - up + 1) / 2, lane, in);
}

// Backward: the sums of kTok tokens back from their rows' scaling (fused.cu), exactly.
__device__ __forceinline__ uint2 load_unscale(const TcParams& P, int m) {
  return __ldcg(reinterpret_cast<const uint2*>(P.epi.unscale + m));
}
__device__ __forceinline__ void unscale_tokens(float (&v)[kTok], uint2 x) {
#pragma unroll
  for (int e = 0; e < kTok; ++e) {
    const uint32_t w = e < 4 ? x.x : x.y;
    const int up = 23 - 8 * (e & 3);  // the byte's way to the exponent field
    v[e] *= __uint_as_float((up >= 0 ? w << up : w >> -up) & 0x7F800000u);
  }
}

// The warp's residual of kTok tokens, two rows in one 4-byte load each (exchanged when used).
__device__ __forceinline__ void load_residual(const TcParams& P, uint32_t (&r)[kTok / 2], int m0,
                                              int count, int row, int lane) {
  if (!P.epi.residual) return;
  const int odd = lane & 1;
  const __half* p = P.epi.residual + (size_t)(m0 + odd) * P.ld + row - odd;
#pragma unroll
  for (int e = 0; e < kTok; e += 2, p += 2 * (size_t)P.ld)
    if (row < P.rows && e + odd < count) r[e / 2] = *reinterpret_cast<const uint32_t*>(p);
}

__device__ __forceinline__ void finish(const TcParams& P, float (&v)[kTok], int m0, int count,
                                       int row, float bias, const uint32_t (&residual)[kTok / 2],
                                       int lane) {
  const qfused::Epilogue& E = P.epi;
  const bool in = row < P.rows;
  const size_t o = (size_t)m0 * P.ld + row;
#pragma unroll
  for (int e = 0; e < kTok; ++e) v[e] += bias;
  if (E.zsave) store_tokens(E.zsave + o, P.ld, v, count, lane, in);
  act_all(E.act, v);
  if (E.residual) {
#pragma unroll
    for (int e = 0; e < kTok; e += 2) {
      const float2 r = __half22float2(qdq::u32_as_h2(exchange_rows(residual[e / 2], lane)));
      v[e] += r.x;
      v[e + 1] += r.y;
    }
  }
  store_tokens(E.y + o, P.ld, v, count, lane, in);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

// Operand descriptors, in two words: the low one holds the address (16-byte units) and the
// leading offset, the high one is the same for all (stride 1024 bytes between 8-row groups,
// 128-byte swizzle).  K-major rows of 128 bytes; the backward product reads A MN-major: its
// 64-wide MN panels are 16384 bytes apart (leading offset).
constexpr uint32_t kDescHi = 64u | (1u << 14) | (2u << 29);
constexpr uint32_t kDescLoK = 1u << 16, kDescLoMn = (128u * 128u / 16u) << 16;
constexpr uint32_t kTransposeA = 1u << 15;  // instruction descriptor: A is MN-major

// Split-sum arrival with a weight; the count before it.
__device__ __forceinline__ uint32_t arrive_weight(uint32_t* counter, uint32_t weight) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
               : "=r"(old)
               : "l"(counter), "r"(weight)
               : "memory");
  return old;
}

// A stage of the pair's other CTA is complete: arrive on the leader's barrier.  The default scope
// (the CTA) orders nothing between the two CTAs in the memory model, so this is what it rests on:
// no thread of the leader reads what the arrival stands for.  A pair's MMA takes each half of
// its operands from the shared memory of the SM that holds it, which has no copy elsewhere: the
// decoding warps' stores are there, and visible to that SM's tensor core, once their proxy fence
// has completed, and the arrival, a release for the CTA, is issued after it.  It only says when.
// (Copied tokens complete on the leader's barrier themselves.)
// A release at cluster scope takes longer than the ring of three stages hides, even when a warp of
// its own passes a stage on for all eight: 512 x 8192 x 8192 78 against 60 us (at the default scope
// that way 61), 2048 x 28672 x 8192 1010 against 750, timed in turn.
__device__ __forceinline__ void arrive_stage(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Every thread of the CTA (PAIR: of both CTAs).  The roles leave their warps divergent, so the
// lanes meet first, and the cluster barrier is the form that does not ask for it.
template <bool PAIR>
__device__ __forceinline__ void sync_all() {
  __syncwarp();
  if constexpr (PAIR)
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  else
    __syncthreads();
  __syncwarp();
}

// One lane of the warp, the same every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc,
                                    uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(kDescHi), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(kDescHi), "r"(accumulate)
        : "memory");
}

template <int BNX, int FMT, bool PAIR, bool BWD, int EP>
__global__ void __launch_bounds__(TcCfg<BNX, FMT, PAIR, EP>::kThreads, 1)
    fused_tc_kernel(const TcParams P, const __grid_constant__ CUtensorMap xmap) {
  using C = TcCfg<BNX, FMT, PAIR, EP>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t ring = qlk::smem_addr(smem_raw);  // 1024-byte aligned, as the swizzle wants
  uint8_t* smem = smem_raw;
  const uint32_t bars = ring + C::kBarOff;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int e) { return bars + 8 * (C::S + e); };
  auto accf = [&](int a) { return bars + 8 * (C::S + C::SE + a); };
  auto acce = [&](int a) { return bars + 8 * (C::S + C::SE + 2 + a); };
  const uint32_t fin = bars + 8 * (C::S + C::SE + 4);
  auto cfull = [&](int f) { return bars + 8 * (C::S + C::SE + 5 + f); };
  auto cempty = [&](int c) { return bars + 8 * (C::S + C::SE + 5 + C::SF + c); };
  const uint32_t lastf = bars + 8 * C::kLastBar;  // the worker's last accumulator is complete
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::kMiscOff);
  const WaitCtx W{ring + C::kMiscOff + 4, P.err, P.wait_us};
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? blockIdx.x & 1u : 0u;  // of the cluster (2, 1, 1)
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
    reinterpret_cast<float*>(smem + C::kLutOff)[threadIdx.x] =
        __half2float(static_cast<const __half*>(P.p0)[threadIdx.x]);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) qlk::mbar_init(full(s), C::kFullCount);
    for (int e = 0; e < C::SE; ++e) qlk::mbar_init(empty(e), 1);
    for (int f = 0; f < C::SF; ++f) qlk::mbar_init(cfull(f), 1);
    for (int c = 0; c < C::SC; ++c) qlk::mbar_init(cempty(c), kTeamWarps);
    for (int a = 0; a < 2; ++a) {
      qlk::mbar_init(accf(a), 1);
      qlk::mbar_init(acce(a), C::kAccEmptyCount);
    }
    qlk::mbar_init(fin, 1);
    qlk::mbar_init(lastf, 1);
    for (int i = 0; i < 4; ++i) {
      qlk::mbar_init(bars + 8 * C::kTailBar + 16 * i, C::kMembers);
      qlk::mbar_init(bars + 8 * C::kTailBar + 16 * i + 8, 1);
    }
    misc[1] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  sync_all<PAIR>();  // barriers are set up (a pair's allocation also wants both CTAs running)
  if (warp == 1) tmem_alloc<PAIR>(ring + C::kMiscOff, C::kTmemCols);
  tc_fence_before();
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
      int s = 0, n = 0, e = 0, eph = 0;  // e: the barrier of stage n - S
      bool ok = true;
      const uint32_t bytes = (uint32_t)P.bn * 256u;  // both CTAs, both boxes
      if ((P.test_us & 0xFFFFu) && wk == 0) qlk::test_delay(P.test_us & 0xFFFFu);
      while (ok && sg.next(P, tile, k0, k1, slot)) {
        const int m = (tile % P.mtiles) * P.bn + (int)rank * (P.bn / C::kCtas);
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {
          if (n >= C::S) {
            if (!(ok = wait<C::kSpin>(empty(e), eph, W, kErrStage))) break;
            if (++e == C::SE) {
              e = 0;
              eph ^= 1;
            }
          }
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
          if (++s == C::S) s = 0;
        }
      }
      // all stages are handed back (a pair's other CTA gets these arrivals from the leader: none
      // may be on its way when it exits), and no copy is in flight (the leader's barriers count
      // both CTAs')
      for (int i = n > C::S ? n - C::S : 0; ok && i < n; ++i) {
        ok = wait<0>(empty(e), eph, W, kErrStage);
        if (++e == C::SE) {
          e = 0;
          eph ^= 1;
        }
      }
      if (leader)
        for (int i = n > C::S ? n - C::S : 0; i < n; ++i)
          wait<0>(full(i % C::S), (i / C::S) & 1, W, kErrStage, false);
      if (PAIR && !ok) qlk::test_delay(kSettleUs);
    }
  } else if (warp == 2) {
    // ---- copies of the units' codes and parameters: lanes 0, 1, 2 each issue one of a unit's
    // copies (LUT4: two) with one instruction
    {
      int c = 0, ph = 1, n = 0, f = 0;
      bool ok = true;
      const uint8_t* base = P.qw;      // this lane's array, bytes per chunk of it
      uint32_t per = C::kChunk, off = 0;
      if (lane >= 1) {
        base = static_cast<const uint8_t*>(FMT == kLUT4 || lane >= 2 ? P.p1 : P.p0);
        per = C::kParChunk;
        off = C::kCodeBytes + (lane >= 2 ? kBlockTiles * C::kParChunk : 0);
      }
      constexpr int kCopies = FMT == kLUT4 ? 2 : 3;
      while (ok && sg.next(P, tile, k0, k1, slot)) {
        const int rb = (tile / P.mtiles) * C::kCtas + (int)rank;
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {
          if (n >= C::SC) {
            if (n == C::SC) qlk::grid_dependency_wait();
            if (!(ok = warp_wait<C::kSpin>(cempty(c), ph, W, kErrStage, lane))) break;
          }
          const int b = BWD ? k : rb, g = BWD ? rb : k;
          if (rb < P.rblocks) {
            const int tb = tiles_in_block(b, P.ntiles);
            const long long ch = chunk_index(b, g, 0, P.G, P.ntiles);
            if (lane == 0)
              qlk::mbar_arrive_expect_tx(cfull(f), tb * (C::kChunk + (kCopies - 1) * C::kParChunk));
            __syncwarp();
            if (lane < kCopies)
              qlk::bulk_g2s(ring + C::kRingC + c * C::kSlot + off, base + ch * per, tb * per,
                            cfull(f));
          } else if (lane == 0) {  // no rows for this CTA of the pair
            qlk::mbar_arrive(cfull(f));
          }
          ++n;
          f = f + 1 == C::SF ? 0 : f + 1;
          if (++c == C::SC) {
            c = 0;
            ph ^= 1;
          }
        }
      }
      for (int i = n > C::SC ? n - C::SC : 0; i < n; ++i)  // none in flight at the end
        warp_wait<0>(cfull(i % C::SF), (i / C::SF) & 1, W, kErrStage, lane, false);
    }
  } else if (warp == 1) {
    // ---- MMA issue (the leader of a pair).  The whole warp runs the loop, so that the
    // descriptors stay in uniform registers; one elected lane issues.
    if (leader) {
      qlk::grid_dependency_wait();
      const uint32_t idesc = idesc_f16(128 * C::kCtas, P.bn) | (BWD ? kTransposeA : 0u);
      if ((P.test_us >> 16) && wk == 0) qlk::test_delay(P.test_us >> 16);
      int s = 0, ph = 0, e = 0, j = 0;
      bool ok = true, ready = false;
      for (; ok && sg.next(P, tile, k0, k1, slot); ++j) {
        const int a = j & 1;
        if (j >= 2 && !(ok = warp_wait<0, PAIR>(acce(a), ((j >> 1) - 1) & 1, W, kErrAcc, lane)))
          break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(a * BNX);
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {
          if (!ready && !(ok = warp_wait<C::kSpin, PAIR>(full(s), ph, W, kErrStage, lane))) break;
          tc_fence_after();
          const uint32_t st = (ring + s * C::kStageBytes) >> 4;
          const uint32_t pa = st | (BWD ? kDescLoMn : kDescLoK);
          const uint32_t pb = (st + (C::kABytes >> 4)) | kDescLoK;
          const int s1 = s + 1 == C::S ? 0 : s + 1, ph1 = s + 1 == C::S ? ph ^ 1 : ph;
          // the next stage's barrier is looked at while this stage's MMAs are issued
          const bool next_ready = mbar_ready(full(s1), ph1, PAIR);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma<PAIR>(d, pa + (BWD ? 128 * kk : (kk >> 2) * (C::kHalfA >> 4) + 2 * (kk & 3)),
                        pb + (kk >> 2) * (C::kHalfB >> 4) + 2 * (kk & 3), idesc,
                        kk == 0 ? (uint32_t)(k != k0) : 1u);
            commit_both(empty(e));
          }
          e = e + 1 == C::SE ? 0 : e + 1;
          ready = __all_sync(0xffffffffu, next_ready);
          s = s1;
          ph = ph1;
        }
        if (ok && elect_one()) commit_both(sg.done(P) ? lastf : accf(a));
        __syncwarp();
      }
      if (elect_one()) tc_commit<PAIR>(fin);
      __syncwarp();
      warp_wait<0>(fin, 0, W, kErrAcc, lane, false);
      if (PAIR && (!ok || misc[1])) qlk::test_delay(kSettleUs);
    }
  } else if (warp >= C::kEpiWarp0) {
    const bool decoder = warp >= C::kDqWarp0;
    int j = 0;  // segment
    bool ok = true;
    if (decoder) {
      // ---- decoding teams
      const int team = (warp - C::kDqWarp0) / kTeamWarps;
      const int dt = (warp - C::kDqWarp0) % kTeamWarps;
      // the team's stages n = team, team + 2, ...: slots n mod S and n mod SC, the barriers of
      // codes n mod SF and of stage n - S
      int s = team, c = team, f = team, fph = 0, e = (C::S ^ team) & 1, eph = 0;
      int n0 = 0;  // stages before the segment
      for (; ok && sg.next(P, tile, k0, k1, slot); ++j) {
        const int rb = (tile / P.mtiles) * C::kCtas + (int)rank;
        const int ftb = rb < P.rblocks ? (BWD ? kBlockTiles : tiles_in_block(rb, P.ntiles)) : 0;
#pragma unroll 1
        for (int k = k0 + ((n0 ^ team) & 1); k < k1; k += kTeams) {
          const int n = n0 + k - k0;
          // Codes beyond the first SC units, and stages handed back, come once the kernels before
          // this one have ended: no limited wait for them may start earlier.
          constexpr int kFree = C::SC < C::S ? C::SC : C::S;
          if (n >= kFree && n < kFree + kTeams) qlk::grid_dependency_wait();
          // decode into registers while the MMAs may still read the stage
          if (!(ok = warp_wait<C::kSpin>(cfull(f), fph, W, kErrStage, lane))) break;
          const bool have = dt < (BWD && k == P.steps - 1 ? min(ftb, tiles_in_block(k, P.ntiles)) : ftb);
          Decoded d;
          if (have) {
            decode_tile<C>(ring + C::kRingC + c * C::kSlot, dt, lane, ring + C::kLutOff, cempty(c),
                           ring + C::kSpareOff + 4 * (warp - C::kDqWarp0), d);
          } else {
            if (lane == 0) qlk::mbar_arrive(cempty(c));
            if (BWD) {  // rows past the last column are contracted: zeros
#pragma unroll
              for (int i = 0; i < 8; ++i) d.v[i >> 1][i & 1] = make_uint4(0, 0, 0, 0);
            }
          }
          if (n >= C::S) {
            if (!(ok = warp_wait<C::kSpin>(empty(e), eph, W, kErrStage, lane))) break;
            if ((e += kTeams) >= C::SE) {
              e -= C::SE;
              eph ^= 1;
            }
          }
          if (BWD || have) store_tile(ring + s * C::kStageBytes, dt, lane, d);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // visible to the MMAs
          __syncwarp();
          if (lane == 0) {
            if (PAIR && !leader)
              arrive_stage(lead(full(s)));
            else
              qlk::mbar_arrive(full(s));
          }
          if ((s += kTeams) >= C::S) s -= C::S;
          if ((c += kTeams) >= C::SC) c -= C::SC;
          if ((f += kTeams) >= C::SF) {
            f -= C::SF;
            fph ^= 1;
          }
        }
        n0 += k1 - k0;
      }
      --j;
    }
    // ---- epilogue: accumulator lanes 32 q .. 32 q + 31, the tokens in chunks of kTok.  The
    // epilogue warps take every segment but the worker's last, while the next one is
    // multiplied; nothing follows the last, so the decoding warps share its chunks.
    qlk::grid_dependency_wait();
    const int q = warp & 3;
    const int member =  // of the quadrant's
        decoder ? C::kEpiPer + (warp - C::kDqWarp0) / 4 : (warp - C::kEpiWarp0) / 4;
    const uint32_t tail = bars + 8 * C::kTailBar + 16 * q;          // two barriers
    const long long U = (long long)(P.tiles - P.whole) * P.steps;
    const qfused::Epilogue& E = P.epi;
    for (; ok; ++j) {
      if (!decoder && !sg.next(P, tile, k0, k1, slot)) break;
      const bool last = decoder || sg.done(P);
      const int a = j & 1;
      // the last accumulator has a barrier of its own, which completes once: the decoding warps
      // have not followed the phases of the others (all see it complete, or all time out)
      if (!(last ? warp_wait<0>(lastf, 0, W, kErrAcc, lane, false)
                 : warp_wait<0>(accf(a), (j >> 1) & 1, W, kErrAcc, lane)))
        break;
      tc_fence_after();
      const int lrow = 32 * q + lane;
      const int row = ((tile / P.mtiles) * C::kCtas + (int)rank) * 128 + lrow;
      const int m0 = (tile % P.mtiles) * P.bn;
      const int cols = P.M - m0 < P.bn ? P.M - m0 : P.bn;
      const uint32_t tb = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(a * BNX);
      int step = (last ? C::kMembers : C::kEpiPer) * kTok, c_first = member * kTok;
      float bias = 0.f;
      if (E.bias && row < P.rows)
        bias = __half2float(E.bias[E.gated ? (size_t)((row >> 4) & 1) * P.ld + (row >> 5) * 16 +
                                                 (row & 15)
                                           : (size_t)row]);
      const bool whole = k0 == 0 && k1 == P.steps;
      int wf = 0, wl = 0, first_slot = 0;
      uint32_t* counter = nullptr;
      if (!whole) {
        // part of a tile: partial sums [token / 4][row][token mod 4]; the last contributor of
        // the tile goes on, with the sums in place of the accumulator
        float* mine = P.partials + (size_t)(2 * blockIdx.x + slot) * 128 * P.bn + 4 * lrow;
#pragma unroll 1
        for (int c0 = c_first; c0 < cols; c0 += step) {
          uint32_t r[8];
          __syncwarp();
          tmem_ld8(tb + (uint32_t)c0, r);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < kTok; e += 4)
            __stcg(reinterpret_cast<uint4*>(mine + (size_t)(c0 + e) * 128),
                   make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]));
        }
        tc_fence_before();
        __syncwarp();
        const long long ub = (long long)(tile - P.whole) * P.steps;
        wf = worker_of(ub, U, P.runners);
        first_slot = run_begin(wf, U, P.runners) >= ub ? 0 : 1;
        wl = worker_of(ub + P.steps - 1, U, P.runners);
        counter = P.counters + ((size_t)(tile - P.whole) * C::kCtas + rank) * 4 + q;
        uint32_t prev = 0;
        if (!last) {
          if (lane == 0) {
            arrive_lead(acce(a));
            prev = arrive_weight(counter, 1u);
          }
          prev = __shfl_sync(0xffffffffu, prev, 0) + 1u;
          c_first = 0;  // the last of a tile's warps joins all of its tokens
          step = kTok;
        } else {
          // the members' sums are written, then one arrival for all of them
          if (lane == 0) qlk::mbar_arrive(tail);
          if (member == 0) {
            if (!warp_wait<0>(tail, 0, W, kErrAcc, lane, false)) break;
            if (lane == 0) {
              misc[2 + q] = arrive_weight(counter, C::kEpiPer);
              qlk::mbar_arrive(tail + 8);
            }
          }
          if (!warp_wait<0>(tail + 8, 0, W, kErrAcc, lane, false)) break;
          prev = misc[2 + q] + C::kEpiPer;
        }
        // (every contributor counts kEpiPer: its warps one each, or all in one arrival)
        if (prev != (uint32_t)(C::kEpiPer * (wl - wf + 1))) {
          if (last) break;
          continue;
        }
        __syncwarp();
      }
      uint32_t res[kTok / 2] = {};
      load_residual(P, res, m0 + c_first, cols - c_first, row, lane);
      uint2 back = {};
      if (BWD && E.unscale && c_first < cols) back = load_unscale(P, m0 + c_first);
#pragma unroll 1
      for (int c0 = c_first; c0 < cols; c0 += step) {
        uint32_t res_next[kTok / 2] = {};
        if (c0 + step < cols)
          load_residual(P, res_next, m0 + c0 + step, cols - c0 - step, row, lane);
        uint2 back_next = {};
        if (BWD && E.unscale && c0 + step < cols) back_next = load_unscale(P, m0 + c0 + step);
        float v[kTok];
        if (whole) {
          uint32_t r[8];
          __syncwarp();
          tmem_ld8(tb + (uint32_t)c0, r);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < kTok; ++e) v[e] = __uint_as_float(r[e]);
        } else {
#pragma unroll
          for (int e = 0; e < kTok; ++e) v[e] = 0.f;
          // slot 0 of every contributor (their runs start in this tile), but slot 1 of one
          // whose run started in an earlier tile
          const float* src = P.partials + (size_t)(2 * (wf * C::kCtas + (int)rank) + first_slot) *
                                              128 * P.bn + (size_t)c0 * 128 + 4 * lrow;
          size_t hop = (size_t)(2 * C::kCtas - first_slot) * 128 * P.bn;
#pragma unroll 4
          for (int w = wf; w <= wl; ++w) {
#pragma unroll
            for (int e = 0; e < kTok; e += 4) {
              const float4 f = __ldcg(reinterpret_cast<const float4*>(src + (size_t)e * 128));
              v[e] += f.x;
              v[e + 1] += f.y;
              v[e + 2] += f.z;
              v[e + 3] += f.w;
            }
            src += hop;
            hop = (size_t)(2 * C::kCtas) * 128 * P.bn;
          }
        }
        if (BWD && E.unscale) unscale_tokens(v, back);
        back = back_next;
        if (E.gated)
          finish_gated(P, v, m0 + c0, cols - c0, row, bias, lane);
        else
          finish(P, v, m0 + c0, cols - c0, row, bias, res, lane);
#pragma unroll
        for (int e = 0; e < kTok / 2; ++e) res[e] = res_next[e];
      }
      if (!whole && lane == 0 && (!last || member == 0)) *counter = 0u;  // ready for the next call
      if (last) break;
      if (whole) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_lead(acce(a));
      }
    }
  }

  tc_fence_before();
  sync_all<PAIR>();
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
template <int BNX, int FMT, bool PAIR, int EP>
void launch_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, unsigned ctas,
                   cudaStream_t st) {
  using C = TcCfg<BNX, FMT, PAIR, EP>;
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
template <int BNX, int FMT, bool PAIR, bool BWD, int EP>
int resident_workers(int dev, int sms) {
  using C = TcCfg<BNX, FMT, PAIR, EP>;
  static std::atomic<int> known[kMaxDevices];
  if (dev < 0 || dev >= kMaxDevices) return 0;
  int n = known[dev].load(std::memory_order_acquire);
  if (n > 0) return n;
  auto fn = fused_tc_kernel<BNX, FMT, PAIR, BWD, EP>;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
    return 0;
  if constexpr (PAIR) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    launch_config<BNX, FMT, PAIR, EP>(&cfg, attr, 2 * (sms / 2), nullptr);
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

// Whole waves of tiles, then the remaining R tiles over `runners` workers by stage, in one of
// two ways:
//  * parts: each of the R tiles in f equal parts, f <= W / R.  The workers stay in step and
//    read the same tokens at the same time; the parts of a tile are joined by 20 or 24 warps.
//  * runs (stream-K): R tiles and one whole wave in W equal runs.  No worker idles, but each is
//    at a depth of its own, and most sums are joined by four warps beside the next tile.
// In us: a stage takes about max(0.45, bn / 465), joining one more part bn / 160 + 0.3, and runs
// cost more than their stages: bn / 14 + 1, and bn / 6.5 + 2 where there is no whole wave, since
// the joins then all fall at the end.  Measured, tokens x columns x k, runs against parts:
// 64 x 28672 x 8192 56 / 66, 96 x 28672 x 8192 62 / 71, 256 x 28672 x 8192 103 / 102,
// 513 x 28672 x 4096 127 / 118, 64 x 12288 x 4096 27 / 20, 200 x 12288 x 4096 53 / 28.
struct Schedule {
  int whole, runners;
};
Schedule schedule(int tiles, int steps, int W, int bn) {
  const int R = tiles % W;
  if (R == 0) return Schedule{tiles, 0};
  const float stage = bn > 209 ? bn / 465.f : 0.45f, join = bn / 160.f + 0.3f;
  int f = 1;
  float parts = steps * stage;
  for (int g = 2; g <= W / R && g <= steps; ++g) {
    const float t = (steps + g - 1) / g * stage + g * join;
    if (t < parts) {
      parts = t;
      f = g;
    }
  }
  const float runs =
      steps * stage * R / W + (tiles < W ? bn / 6.5f + 2.f : bn / 14.f + 1.f);
  if (runs < parts) {
    const int t = tiles < W ? tiles : R + W;  // shared out
    const long long units = (long long)t * steps;
    return Schedule{tiles - t, units < W ? (int)units : W};
  }
  return Schedule{tiles - R, R * f};
}

template <int BNX, int FMT, bool PAIR, bool BWD, int EP = 1>
ql_status launch_as(const qfused::Product& p, const Tokens& tk) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return QL_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return QL_ERR_CUDA;
  const int maxw = resident_workers<BNX, FMT, PAIR, BWD, EP>(dev, sms);
  if (maxw <= 0) return QL_ERR_CUDA;
  if (p.partial_bytes < (size_t)2 * sms * 128 * tk.bn * sizeof(float)) return QL_ERR_WORKSPACE;
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
  const Schedule sc = schedule(P.tiles, P.steps, maxw, tk.bn);
  P.whole = sc.whole;
  P.runners = sc.runners;
  const qfused::WaitTest wt = qfused::wait_test();
  P.wait_us = (wt.limit_us < 1000000000u ? wt.limit_us : 1000000000u) + 4u * (uint32_t)P.steps;
  P.test_us = wt.delays;
  if ((size_t)(P.tiles - P.whole) * ctas * 4 * sizeof(uint32_t) > qfused::kTcCounterBytes)
    return QL_ERR_UNSUPPORTED;  // more than five hundred SMs
  const int workers = P.whole > 0 ? maxw : P.runners;
  CUtensorMap xmap;
  if (!encode_rows(&xmap, p.x, p.M, BWD ? p.N : p.K, tk.bn / ctas)) return QL_ERR_CUDA;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  launch_config<BNX, FMT, PAIR, EP>(&cfg, attr, (unsigned)(workers * ctas), p.stream);
  if (cudaLaunchKernelEx(&cfg, fused_tc_kernel<BNX, FMT, PAIR, BWD, EP>, P, xmap) != cudaSuccess)
    return QL_ERR_CUDA;
  return QL_OK;
}

template <int FMT, bool BWD>
ql_status launch_fmt(const qfused::Product& p) {
  const Tokens tk = token_tiles(p.M);
  if (!tk.pair)
    return tk.bn <= 32 ? launch_as<32, FMT, false, BWD>(p, tk)
                       : launch_as<64, FMT, false, BWD>(p, tk);
  if (tk.bn <= 128) return launch_as<128, FMT, true, BWD>(p, tk);
  if constexpr (!BWD) {
    // Per 256 tokens a stage takes about 1100 cycles, the epilogue of one warp per quadrant
    // 48000, and 32000 more for each array beside the output: with two warps 2048 x 28672 x 8192
    // with GELU and the pre-activation kept takes 785 against 952 us, without it 824 against 787
    // (30 calls each in turn); gated 513 x 28672 x 4096 with both kept 172 against 191.
    const int arrays = (p.epi.zsave != nullptr) + (p.epi.residual != nullptr);
    if (p.K / kGroup < 44 + 30 * arrays) return launch_as<256, FMT, true, BWD, 2>(p, tk);
  }
  return launch_as<256, FMT, true, BWD>(p, tk);
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
