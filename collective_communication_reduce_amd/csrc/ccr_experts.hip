// Device kernels of the experts' matrix products, written for gfx950 (CDNA4:
// wave64, 256 CUs in 8 XCDs, MFMA matrix cores, 160 KB LDS per CU).
//
// Every expert e owns a run of rows x (its tokens) and a weight W_e [F x H]:
//
//   product   out[i, f]  = sum_h x[i, h] W_e[f, h]
//   dgrad     dx[i, h]   = sum_f dout[i, f] W_e[f, h]
//   wgrad     dW_e[f, h] = sum_i dout[i, f] x[i, h]
//
// One launch covers all experts (up to kExpertGroups of them): the host lists
// the experts with work and the first tile of each, so the grid holds exactly
// the tiles there are, however ragged the rows.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "ccr_device.h"
#include "ccr_experts.h"
#include "ccr_internal.h"

namespace ccr {
namespace {

// Source of the lanes that lie past the end of the contraction.
__device__ const u32x4 zero_vector = {0, 0, 0, 0};

// D (rows: a's, columns: b's) += a b^T over half a K-step.
template <int ES>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 d) {
  if constexpr (ES == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), d, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      d = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, (uint32_t)a[i]),
                                               __builtin_bit_cast(float, (uint32_t)b[i]), d, 0, 0, 0);
    return d;
  }
}

// ------------------------------------------------------- small and mid tiles
// OP as in the table above.  Tile BM x BN of the output; WK groups of WM x WN
// waves, each of which takes every WK-th K-step over the whole tile; a ring of
// NBUF rounds of WK K-steps in LDS.  Per round one barrier: behind it the
// round's vectors are in LDS and the round before is read by every wave, so its
// buffer takes the loads of the round NBUF - 1 ahead.  What bounds it: few rows,
// HBM (the weights of 64 experts, 2048 x 1024 bf16, for 288 rows: 57.5 us, 4.7
// TB/s) or, with few tiles, a tile's latency; tile 64, reads from L2 (21 TB/s
// over the chip); fp32, the matrix units (8192 rows, 4096 x 4096: 1.94 ms, 142
// TFLOP/s).
template <ExpertOp OP, int ES, int OS, int BM, int BN, int WM, int WN, int WK, int NBUF>
__global__ __launch_bounds__(WM * WN * WK * 64) void experts_ring_kernel(const ExpertTable tab,
                                                                         const ExpertShape sh) {
  constexpr bool kACol = OP == ExpertOp::kWgrad;       // a: x, dout, dout
  constexpr bool kBCol = OP != ExpertOp::kProduct;     // b: W, W, x
  constexpr int NT = WM * WN * 64;                     // threads of a group
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 blocks per wave
  constexpr int kABytes = BM * KB, kStepBytes = (BM + BN) * KB, kBuf = WK * kStepBytes;
  using LoadA = Loader<ES, BM, kACol, false, NT>;
  using LoadB = Loader<ES, BN, kBCol, false, NT>;
  constexpr int kLoads = LoadA::kLoads + LoadB::kLoads;
  static_assert(LoadA::kLoads * NT == BM * 8 && LoadB::kLoads * NT == BN * 8, "whole loads");
  static_assert((NBUF - 2) * kLoads <= 63, "the wait count has 6 bits");
  static_assert(WK == 1 || WK * BM * BN * 4 <= NBUF * kBuf, "the groups' sums fit the ring");
  __shared__ __align__(1024) char lds[NBUF * kBuf];
  const int t = kACol ? xcd_turns(blockIdx.x, gridDim.x) : xcd_tile(blockIdx.x, gridDim.x);
  const Where at = place_of<OP, BM, BN>(tab, sh, t);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = w / (WM * WN), wg = w % (WM * WN);
  const int wm = (wg / WN) * (BM / WM), wn = (wg % WN) * (BN / WN);
  LoadA la;
  LoadB lb;
  la.init(at.a, (OP == ExpertOp::kProduct ? sh.H : sh.F) * ES, at.m0, at.M, threadIdx.x % NT);
  lb.init(at.b, sh.H * ES, at.n0, at.N, threadIdx.x % NT);
  constexpr int kStep = LoadA::kStep;
  // Step 0 holds the contraction's odd end (`rest` values, then zeros; no value
  // for a weight gradient without rows), so that every later step is whole.
  // Past the last step the loads bring the last whole step again (or, where
  // there is none, each operand's first vector): the count of loads on their
  // way stays the same.
  const int whole = (int)((at.C - 1) / kStep), nk = whole + 1;
  const int rest = (int)(at.C - (int64_t)whole * kStep);
  const int64_t da = la.stride(), db = lb.stride();
  const uint32_t lds0 = (uint32_t)(uintptr_t)(CCR_LDS char*)lds + wk * kStepBytes + wg * 1024;
  const char *pa, *pb;  // step j, or the last whole one before it
  int j = 0;
  auto go_to = [&](int step) {
    j = step < whole ? step : whole;
    pa = la.base + (kACol ? rest * la.ld : rest * ES) + (j - 1) * da;
    pb = lb.base + (kBCol ? rest * lb.ld : rest * ES) + (j - 1) * db;
  };
  auto issue = [&](uint32_t to) {
#pragma unroll
    for (int i = 0; i < LoadA::kLoads; i++) load_lds(to + i * NT * 16, (uint32_t)la.off[i], pa);
#pragma unroll
    for (int i = 0; i < LoadB::kLoads; i++)
      load_lds(to + kABytes + i * NT * 16, (uint32_t)lb.off[i], pb);
    const int next = j + WK < whole ? j + WK : whole;
    pa += (next - j) * da;
    pb += (next - j) * db;
    j = next;
  };
  if (wk == 0 || wk >= nk) {  // the partial step, or zeros for a group without a step
    const int until = wk == 0 ? rest : 0;
    const char* zero = reinterpret_cast<const char*>(&zero_vector);
#pragma unroll
    for (int i = 0; i < LoadA::kLoads; i++)
      load_lds(lds0 + i * NT * 16, la.k[i] < until ? la.base + la.off[i] : zero);
#pragma unroll
    for (int i = 0; i < LoadB::kLoads; i++)
      load_lds(lds0 + kABytes + i * NT * 16, lb.k[i] < until ? lb.base + lb.off[i] : zero);
    go_to(wk + WK);
  } else {
    go_to(wk);
    issue(lds0);
  }
  if (whole == 0) {
    pa = rest ? la.base : reinterpret_cast<const char*>(&zero_vector);
    pb = rest ? lb.base : reinterpret_cast<const char*>(&zero_vector);
#pragma unroll
    for (int i = 0; i < LoadA::kLoads; i++) la.off[i] = 0;
#pragma unroll
    for (int i = 0; i < LoadB::kLoads; i++) lb.off[i] = 0;
  }
#pragma unroll
  for (int i = 1; i < NBUF - 1; i++) issue(lds0 + i * kBuf);
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; i++)
#pragma unroll
    for (int n = 0; n < TN; n++) acc[i][n] = f32x4{0, 0, 0, 0};
  // fp32 results are summed in chains of 64 matrix instructions (256 values of
  // fp32, 2048 of bf16), and the chains' sums apart: the error grows with the
  // length of a chain of additions.  Over 4096 fp32 values it is 3e-7 of the
  // result, 1e-6 in one chain; the cost is 2%.
  constexpr int kChain = ES == 4 ? 8 : 32;  // K-steps
  f32x4 sum[OS == 4 ? TM : 1][OS == 4 ? TN : 1] = {};
  auto collect = [&]() {
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
      for (int n = 0; n < TN; n++) {
        sum[i][n] += acc[i][n];
        acc[i][n] = f32x4{0, 0, 0, 0};
      }
  };
  int cur = 0, free = (NBUF - 1) * kBuf;  // byte offsets of this round's buffer and of the one read before
  const int rounds = (nk + WK - 1) / WK;
  for (int r = 0; r < rounds;) {
    const int until = OS == 4 && r + kChain < rounds ? r + kChain : rounds;
#pragma unroll 1
    for (; r < until; r++) {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NBUF - 2) * kLoads) : "memory");
      const char* from = lds + cur + wk * kStepBytes;
      u32x4 a[2][TM], b[2][TN];
#pragma unroll
      for (int h = 0; h < 2; h++) {
#pragma unroll
        for (int i = 0; i < TM; i++) a[h][i] = fragment<ES, BM, kACol, false>(from, wm, i, h);
#pragma unroll
        for (int n = 0; n < TN; n++) b[h][n] = fragment<ES, BN, kBCol, false>(from + kABytes, wn, n, h);
      }
      issue(lds0 + free);
      free = cur;
      cur = cur + kBuf == NBUF * kBuf ? 0 : cur + kBuf;
      if (WK > 1 && r * WK + wk >= nk) continue;  // this group has no step in the last round
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int i = 0; i < TM; i++)
#pragma unroll
          for (int n = 0; n < TN; n++) acc[i][n] = mma<ES>(b[h][n], a[h][i], acc[i][n]);
    }
    if constexpr (OS == 4) collect();
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  // D holds b's rows (the output's columns) down its registers: lane l has
  // output row l % 16 and columns 4 (l / 16) + (0..3) of each 16 x 16 block.
  const int l = threadIdx.x & 63;
  if constexpr (WK == 1) {
#pragma unroll
    for (int i = 0; i < TM; i++) {
      const int64_t m = at.m0 + wm + i * 16 + (l & 15);
      if (m >= at.M) continue;
#pragma unroll
      for (int n = 0; n < TN; n++) {
        const int64_t c = at.n0 + wn + n * 16 + (l >> 4) * 4;
        if (c < at.N) store4<OS>(at.c + (m * at.N + c) * OS, OS == 4 ? sum[i][n] : acc[i][n], sh.add);
      }
    }
  } else {
    // the groups' sums, added in the groups' order
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    f32x4* part = reinterpret_cast<f32x4*>(lds);  // [WK][BM][BN / 4]
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
      for (int n = 0; n < TN; n++)
        part[(wk * BM + wm + i * 16 + (l & 15)) * (BN / 4) + (wn + n * 16) / 4 + (l >> 4)] =
            OS == 4 ? sum[i][n] : acc[i][n];
    __syncthreads();
    for (int q = threadIdx.x; q < BM * BN / 4; q += NT * WK) {
      const int64_t m = at.m0 + q / (BN / 4), c = at.n0 + q % (BN / 4) * 4;
      f32x4 v = part[q];
#pragma unroll
      for (int k = 1; k < WK; k++) v += part[k * BM * BN / 4 + q];
      if (m < at.M && c < at.N) store4<OS>(at.c + (m * at.N + c) * OS, v, sh.add);
    }
  }
}

// ------------------------------------------------------------- large tiles
// bf16 products of 256 x 256 tiles: four waves, one to a SIMD, each with a
// 128 x 128 part of the tile in its accumulators.  Per K-step of 64 a wave
// reads 32 KiB from LDS for 128 MFMAs.
//
// All of the CU's LDS is a ring of five 32 KiB slots, each one operand's part
// of one K-step (whole 128-byte lines of memory).  A step runs in two phases
// of 32 k: in the first, the fragments of its second half are read; then a
// barrier, after which its slots are free and the next step's are full; in the
// second, the fragments of the next step's first half are read.  The loads of
// the slots set free go out in the second phase and the beginning of the next
// step's first: b of step s + 2, needed one step later, then a of step s + 3,
// needed two steps later.
//
// With one wave to a SIMD nothing hides an instruction that stalls, so reads
// and loads are placed one by one between the products.  Measured at 8192^3
// against reads and loads in groups of three before every eight products:
// 1283 -> 1433 TFLOP/s (dgrad).  A training layer's product (196,608 rows of 64
// experts, 2048 x 1024) takes 705 to 728 us, 1.13 to 1.17 PFLOP/s, and is bound by
// power: the matrix units are 64% busy at 1.65 GHz, and where gaps are filled the
// clock falls.  The gradients of 49,152 rows of 16 experts (2048 x 1408: 271 and
// 275 us, 1.04 and 1.03 PFLOP/s) run at 2.06 GHz with the matrix units 50% busy:
// the start and the stores of a tile, the last round's empty units and, in the input
// gradient, LDS conflicts (33% of the LDS cycles) count there.

// A fragment as fragment() gives it, read in parts.
template <bool COL, bool PAIRED>
struct Frag {
  static constexpr int kReads = COL ? 2 : 1;
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  u32x4 whole;
  u32x2 half[2];

  template <int X>
  __device__ __forceinline__ void read(const char* lds, int x0, int i, int h, int part) {
    if constexpr (!COL) whole = fragment<2, X, false, PAIRED>(lds, x0, i, h);
    else half[part] = __builtin_bit_cast(u32x2, fragment_half<X, PAIRED>(lds, x0, i, h, part));
  }
  __device__ __forceinline__ u32x4 v() const {
    if constexpr (COL) return __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3);
    else return whole;
  }
};

// D += a b^T with D held in accumulation registers.  Written in assembly
// because all 256 of them are accumulators here, which the compiler's own
// allocation mixes with the fragments and moves about in the loop.  No two
// products in a row touch the same D, so no wait states are due between them;
// drain() provides those before D is read.  The compiler does not know of them:
// were it to copy an accumulator inside the loop, the copy would miss the last
// sums.  It has no cause to while every D is read in place after drain(); the
// build reads the assembly of these kernels and refuses one that does.
__device__ __forceinline__ void mma_acc(u32x4 a, u32x4 b, f32x4& d) {
  asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(d) : "v"(a), "v"(b));
}
__device__ __forceinline__ void drain(f32x4* d) {
  asm volatile("s_nop 15\n\ts_nop 15"
               : "+a"(d[0]), "+a"(d[1]), "+a"(d[2]), "+a"(d[3]), "+a"(d[4]), "+a"(d[5]), "+a"(d[6]),
                 "+a"(d[7]));
}

// Eight neighbouring bf16 values of an output row.
__device__ __forceinline__ void store8(char* p, f32x4 lo, f32x4 hi) {
  const bf16x4 a = __builtin_convertvector(lo, bf16x4), b = __builtin_convertvector(hi, bf16x4);
  *reinterpret_cast<bf16x8*>(p) = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// One workgroup to a compute unit, each taking every gridDim.x-th tile.  The
// first loads of its next tile go out before this tile's results are written,
// so that neither their latency nor the launch of a workgroup lies between two
// tiles.
//
// fp32 results are summed in chains of up to kChainSteps K-steps (8192 rows), so
// that their error does not grow with an expert's rows.  All accumulation
// registers hold one chain, and the chains are joined in the tile's results: each
// one after the first goes through the loop as a tile of its own that adds to what
// the one before stored.  RMS error of 262,144 rows of normal values 5.9e-7 of the
// results, 3.3e-6 in one chain; the joining costs 4% at 20,512 rows and 10% at
// 65,536 (4096 x 4096: 1.54 -> 1.69 ms).  Chains of 4096 rows: 4.2e-7, but 18%
// and 21%, and a fifth more for experts of 4096 to 8192 rows too.
constexpr int kChainSteps = 128;
template <ExpertOp OP, int OS>
__global__ __launch_bounds__(256, 1) void experts_big_kernel(const ExpertTable tab, const ExpertShape sh,
                                                             int tiles) {
  constexpr int ES = 2, BM = 256, BN = 256, NT = 256, T = 8;
  constexpr bool kACol = OP == ExpertOp::kWgrad;
  constexpr bool kBCol = OP != ExpertOp::kProduct;
  constexpr int kSlot = BM * KB, kSlots = 5;
  static_assert(BM == BN, "both operands fill a slot");
  using LoadA = Loader<ES, BM, kACol, false, NT>;
  // Paired fragments of b give 16-byte stores of bf16 (dgrad of 8 x 4096 rows,
  // 2048 x 1024: 122 us, unpaired 130), though in a column image their reads meet
  // on half of the banks.  fp32 results are stored by 16 bytes either way.
  constexpr bool kPaired = OS == 2;
  using LoadB = Loader<ES, BN, kBCol, kPaired, NT>;
  constexpr int kStep = LoadA::kStep;
  constexpr int kLoads = LoadA::kLoads;  // of one slot
  static_assert(kLoads == 8 && LoadB::kLoads == 8, "the wait counts below");
  constexpr bool kChains = OP == ExpertOp::kWgrad && OS == 4;
  constexpr int64_t kChain = (int64_t)kChainSteps * kStep;  // values
  constexpr int kEarlyA = 5;  // loads of a that go out in a step's second phase
  __shared__ __align__(1024) char lds[kSlots * kSlot];
  const int l = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (w >> 1) * 128, wn = (w & 1) * 128;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(CCR_LDS char*)lds + w * 1024;

  LoadA la;
  LoadB lb;
  const char *pa, *pb;  // the step whose loads are next, of a and of b
  int64_t da, db;
  int ja, jb, whole;
  // A slot's loads, one at a time: load i of the slot at `to`.
  auto load_at = [&](int i, uint32_t to, const int* off, const char* p) {
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3"
                 ::"s"(to), "n"(i * NT * 16), "v"(off[i]), "s"(p) : "memory", "scc");
  };
  auto load_a = [&](int i, uint32_t to) { load_at(i, to, la.off, pa); };
  auto load_b = [&](int i, uint32_t to) { load_at(i, to, lb.off, pb); };
  // Past the last step the loads bring the last whole step again (or, where
  // there is none, each operand's first vector) into slots that are not read
  // any more: the loop keeps no branch, and the count of loads on their way
  // stays the same.
  auto next_a = [&]() {
    pa += ja < whole ? da : 0;
    ja++;
  };
  auto next_b = [&]() {
    pb += jb < whole ? db : 0;
    jb++;
  };
  auto load_whole = [&](auto& load, uint32_t to, int n) {
#pragma unroll
    for (int i = 0; i < n; i++) load(i, to);
  };
  // A tile's first loads: step 0, which holds the contraction's odd end (`rest`
  // values, then zeros; no value for a weight gradient without rows), so that
  // every later step is whole; step 1; the first of a's step 2.
  auto begin = [&](const Where& at) {
    la.init(at.a, (OP == ExpertOp::kProduct ? sh.H : sh.F) * ES, at.m0, at.M, threadIdx.x);
    lb.init(at.b, sh.H * ES, at.n0, at.N, threadIdx.x);
    whole = (int)((at.C - 1) / kStep);
    const int rest = (int)(at.C - (int64_t)whole * kStep);
    const char* zero = reinterpret_cast<const char*>(&zero_vector);
#pragma unroll
    for (int i = 0; i < kLoads; i++)
      load_lds(lds0 + i * NT * 16, la.k[i] < rest ? la.base + la.off[i] : zero);
#pragma unroll
    for (int i = 0; i < kLoads; i++)
      load_lds(lds0 + kSlot + i * NT * 16, lb.k[i] < rest ? lb.base + lb.off[i] : zero);
    pa = la.base + (kACol ? rest * la.ld : rest * ES);
    pb = lb.base + (kBCol ? rest * lb.ld : rest * ES);
    da = la.stride();
    db = lb.stride();
    ja = jb = 1;
    if (whole == 0) {
      pa = rest ? la.base : zero;
      pb = rest ? lb.base : zero;
#pragma unroll
      for (int i = 0; i < kLoads; i++) la.off[i] = lb.off[i] = 0;
    }
    load_whole(load_a, lds0 + 2 * kSlot, kLoads);
    next_a();
    load_whole(load_b, lds0 + 3 * kSlot, kLoads);
    next_b();
    load_whole(load_a, lds0 + 4 * kSlot, kEarlyA);
  };

  // Fragments are read in units: one LDS read each, two to a fragment from a
  // column image.
  using FragA = Frag<kACol, false>;
  using FragB = Frag<kBCol, kPaired>;
  constexpr int kUnitsB = T * FragB::kReads, kUnits = kUnitsB + T * FragA::kReads;
  FragA a[2][T];
  FragB b[2][T];
  auto read = [&](int u, int h, const char* at_a, const char* at_b) {  // b's first, then a's
    if (u < kUnitsB) {
      constexpr int n = FragB::kReads;
      b[h][u / n].template read<BN>(at_b, wn, u / n, h, u % n);
    } else {
      constexpr int n = FragA::kReads;
      a[h][(u - kUnitsB) / n].template read<BM>(at_a, wm, (u - kUnitsB) / n, h, (u - kUnitsB) % n);
    }
  };

  // tile t: the first of its chains, which takes what the others leave over
  auto place = [&](int t) {
    Where x = place_of<OP, BM, BN>(tab, sh, t);
    x.add = sh.add;
    if (kChains && x.C > kChain) {
      x.left = (x.C - 1) / kChain * kChain;
      x.C -= x.left;
    }
    return x;
  };
  auto rest_of = [&](Where x) {  // its next chain
    x.a += x.C * sh.F * ES;
    x.b += x.C * sh.H * ES;
    x.C = kChain;
    x.left -= kChain;
    x.add = true;
    return x;
  };

  int r = 0;
  Where at = place(tile_of<kACol>(blockIdx.x, 0, tiles));
  begin(at);
  // all but step 1 and part of a's step 2
  asm volatile("s_waitcnt vmcnt(21)\n\ts_barrier" ::: "memory");
  static_assert(2 * kLoads + kEarlyA == 21, "as waited for");
#pragma unroll 1
  for (;;) {
    const int nk = whole + 1;
    Where next;
    bool again = true;
    if (kChains && at.left > 0) {
      next = rest_of(at);
    } else {
      r++;
      const int t = tile_of<kACol>(blockIdx.x, r, tiles);
      again = t >= 0;
      next = place(again ? t : 0);
    }
#pragma unroll
    for (int u = 0; u < kUnits; u++) read(u, 0, lds, lds + kSlot);
    f32x4 acc[T][T];
#pragma unroll
    for (int i = 0; i < T; i++)
#pragma unroll
      for (int j = 0; j < T; j++) {
        acc[i][j] = f32x4{0, 0, 0, 0};
        asm volatile("" : "+a"(acc[i][j]));
      }
    int s = 0, slot = 0;  // the step that runs, and the slot of its a
    auto ahead = [&](int n) {  // the slot n places on
      const int x = slot + n;
      return x < kSlots ? x : x - kSlots;
    };
    // A phase's reads are done after kReadSlots of its 64 products; a load goes
    // out every kLoadEvery products.  (Between 32 and 56, and at 4, the rate
    // stays within 1%.)
    constexpr int kReadSlots = 48, kLoadEvery = 5;
#pragma unroll 1
    do {
      {
        const char* at_a = lds + slot * kSlot;
        const char* at_b = lds + ahead(1) * kSlot;
        const uint32_t to = lds0 + ahead(4) * kSlot;
#pragma unroll
        for (int n = 0; n < T * T; n++) {
          mma_acc(b[0][n % T].v(), a[0][n / T].v(), acc[n / T][n % T]);
          if (n < kReadSlots) {
#pragma unroll
            for (int u = n * kUnits / kReadSlots; u < (n + 1) * kUnits / kReadSlots; u++)
              read(u, 1, at_a, at_b);
          }
          if (n % kLoadEvery == 2 && n / kLoadEvery < kLoads - kEarlyA)
            load_a(kEarlyA + n / kLoadEvery, to);  // the rest of a's step s + 2
          __builtin_amdgcn_sched_barrier(0);
        }
        next_a();
      }
      // step s is read by every wave; step s + 1 is in LDS, a's step s + 2 may be
      // on its way
      asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      {
        const char* at_a = lds + ahead(2) * kSlot;
        const char* at_b = lds + ahead(3) * kSlot;
        const uint32_t to_b = lds0 + slot * kSlot, to_a = lds0 + ahead(1) * kSlot;
#pragma unroll
        for (int n = 0; n < T * T; n++) {
          mma_acc(b[1][n % T].v(), a[1][n / T].v(), acc[n / T][n % T]);
          // (after the last step this reads what the slots held; unused)
          if (n < kReadSlots) {
#pragma unroll
            for (int u = n * kUnits / kReadSlots; u < (n + 1) * kUnits / kReadSlots; u++)
              read(u, 0, at_a, at_b);
          }
          const int i = n / kLoadEvery;
          if (n % kLoadEvery == 2 && i < kLoads) load_b(i, to_b);
          else if (n % kLoadEvery == 2 && i < kLoads + kEarlyA) load_a(i - kLoads, to_a);
          __builtin_amdgcn_sched_barrier(0);
        }
        static_assert((kLoads + kEarlyA - 1) * kLoadEvery + 2 < T * T, "a phase holds its loads");
        next_b();
      }
      slot = ahead(2);
    } while (++s < nk);
    drain(acc[T - 1]);
    // The last loads of this tile are done, and every wave has read what it
    // needs of the slots (at the last step's barrier): the next tile's go out.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    if (again) begin(next);

    // D holds b's rows (the output's columns) down its registers: lane l has
    // output row l % 16 of each block and columns 4 (l / 16) + (0..3) of it, or of
    // a pair of blocks columns 8 (l / 16) + (0..7).
    const bool inside = at.m0 + BM <= at.M && at.n0 + BN <= at.N, full = inside && !at.add;
    const int64_t n = at.n0 + wn + (l >> 4) * (kPaired ? 8 : 4);
    char* out = at.c + ((at.m0 + wm + (l & 15)) * at.N + n) * OS;
    const int64_t down = 16 * at.N * OS;
    auto column = [](int j) { return kPaired ? (j >> 1) * 32 + (j & 1) * 4 : j * 16; };
    if (full) {
#pragma unroll
      for (int i = 0; i < T; i++) {
#pragma unroll
        for (int j = 0; j < T; j += 2) {
          asm volatile("" : "+a"(acc[i][j]), "+a"(acc[i][j + 1]));  // read out row by row
          if constexpr (kPaired) {
            store8(out + column(j) * OS, acc[i][j], acc[i][j + 1]);
          } else {
            store4<OS>(out + column(j) * OS, acc[i][j], false);
            store4<OS>(out + column(j + 1) * OS, acc[i][j + 1], false);
          }
        }
        out += down;
        __builtin_amdgcn_sched_barrier(0);
      }
    } else if (kChains && inside) {  // a row of blocks at a time, its old values read together
#pragma unroll
      for (int i = 0; i < T; i++) {
        f32x4 old[T];
#pragma unroll
        for (int j = 0; j < T; j++) old[j] = *reinterpret_cast<const f32x4*>(out + column(j) * OS);
#pragma unroll
        for (int j = 0; j < T; j++) {
          asm volatile("" : "+a"(acc[i][j]));
          store4<OS>(out + column(j) * OS, acc[i][j] + old[j], false);
        }
        out += down;
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < T; i++) {
        const bool in = at.m0 + wm + i * 16 + (l & 15) < at.M;
#pragma unroll
        for (int j = 0; j < T; j++) {
          asm volatile("" : "+a"(acc[i][j]));
          if (in && n + column(j) < at.N) store4<OS>(out + column(j) * OS, acc[i][j], at.add);
        }
        out += down;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (!again) return;
    at = next;
    // the next tile's step 0; its step 1 and part of a's step 2, and in a full
    // tile the results' stores, may be on their way here.  (What place() loads of
    // the table at the loop's start is waited for behind all of them.)
    constexpr int kStores = kPaired ? T * T / 2 : T * T;
    if (full) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(21 + kStores < 63 ? 21 + kStores : 63) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    asm volatile("s_barrier" ::: "memory");
  }
}

template <ExpertOp OP, int ES, int OS>
hipError_t launch_as(const ExpertTable& tab, const ExpertShape& sh, ExpertTile tile, int tiles,
                     hipStream_t stream) {
  switch (tile) {
    case ExpertTile::k16:  // 64 KiB of LDS: two workgroups to a compute unit
      experts_ring_kernel<OP, ES, OS, 16, 16, 1, 1, 4, 4><<<(unsigned)tiles, 256, 0, stream>>>(tab, sh);
      break;
    case ExpertTile::k32:  // 32 KiB: five
      experts_ring_kernel<OP, ES, OS, 32, 32, 2, 2, 1, 4><<<(unsigned)tiles, 256, 0, stream>>>(tab, sh);
      break;
    case ExpertTile::k64:  // 48 KiB: three
      experts_ring_kernel<OP, ES, OS, 64, 64, 2, 2, 1, 3><<<(unsigned)tiles, 256, 0, stream>>>(tab, sh);
      break;
    case ExpertTile::k128:  // 128 KiB: one
      experts_ring_kernel<OP, ES, OS, 128, 128, 2, 4, 1, 4><<<(unsigned)tiles, 512, 0, stream>>>(tab, sh);
      break;
    case ExpertTile::k256:
      if constexpr (ES == 2)
        experts_big_kernel<OP, OS><<<(unsigned)(tiles < kCus ? tiles : kCus), 256, 0, stream>>>(tab, sh,
                                                                                              tiles);
      else
        return hipErrorInvalidValue;
      break;
  }
  return hipGetLastError();
}

}  // namespace

ExpertTileSize expert_tile_size(ExpertTile tile) {
  switch (tile) {
    case ExpertTile::k16: return {16, 16};
    case ExpertTile::k32: return {32, 32};
    case ExpertTile::k64: return {64, 64};
    case ExpertTile::k128: return {128, 128};
    default: return {256, 256};
  }
}

// The variant with the shortest estimated time.  A tile of s K-steps is taken
// to cost c0 + c1 s + its output at an even share of 4.9 TB/s, and tiles to
// run in rounds of one to a compute unit (of the smaller tiles, of which a unit
// holds several, in fractions of a round).  A tile with a unit to itself takes
// alone s instead of c1 s: in few tiles the groups of k16 share a long
// contraction, in many its short rows cost it twice the loads of k32 (and more
// where they are rows of 16 columns: input and weight gradients).  Rows
// that are not whole lines of 128 bytes cost the tiles up to 64, whose reads
// from L2 bound them, a third more, as each read touches two lines (4 x 3000
// rows, 1000 x 1000 against 1024 x 1024: tile 64 57 and 42 us, tile 256 31.9 and
// 30.0).  The constants in us were fitted to all three products of 38 shapes from 1 to
// 16000 rows; where the choice matters:
//   us at tile                        16     32     64    128    256
//   1 row, 2048 x 1024               3.8    6.2    9.3   14.6   36.7
//   1 row, 8192 x 1024               6.7   17.4
//   5 x 1 row, 2048 x 1024           5.1    6.3   10.1   14.7   37.1
//   2 x 100 rows, 2856 x 120         4.4    7.8
//   8 x 16 rows, 512 x 512           3.3    3.5    4.4    6.0   13.9
//   6 x 120 rows, 512 x 512          8.2    4.2
//   64 x 4 rows, 2048 x 1024        48.7   39.5
//   4 x 500 rows, 1024 x 1024              13.2    9.1   11.4   26.7
//   8 x 200 rows, 2048 x 2048              41.3   30.5   21.7   44.2
//   8 x 2000 rows, 1024 x 1024             95.3   59.4   50.6   35.7
//   4 x 1500 rows, 2048 x 2048              131   77.7   62.4   50.4
// (products in bf16).  fp32 products of 8 x 16 rows, 512 x 512: 3.9, 6.0, 11.2,
// 32.3; of 1 row, 8192 x 1024: 17.8, 55.1; weight gradients (fp32 out) of 64 x 4
// rows, 2048 x 1024, from tile 32 on: 268, 161, 181, 109.  Large fp32 products
// run at the rate of the matrix units from tile 64 on.  8-bit rows have constants
// of their own, fitted to the products of 22 shapes from 1 to 90,000 rows (their
// rows are whole lines); where the choice matters, us of the whole call, of which
// the host's part hides all below 8.5:
//   us at tile                        16     32     64    128    256
//   1 row, 8192 x 1024              10.7   13.3   18.4   34.4   73.3
//   64 x 5 rows, 2048 x 1024        36.5   23.4   25.4   27.4   31.3
//   8 x 16 rows, 4096 x 4096        27.4   22.3   21.8   23.5   43.5
//   64 x 100 rows, 2048 x 1024       208   63.4   36.2   33.4   34.5
//   8 x 200 rows, 2048 x 2048        103   30.9   22.5   16.2   26.6
//   4 x 500 rows, 1024 x 1024       47.6   12.2    8.5    9.9   16.9
//   8 x 500 rows, 7168 x 2048        480    183    107   73.8   77.6
//   16 x 700 rows, 2048 x 1024       327   82.0   50.2   40.9   31.5
ExpertTile expert_tile(ExpertOp op, int es, int os, const ExpertShape& sh, const int64_t* rows, int n) {
  struct Cost {
    ExpertTile tile;
    double c0, c1, alone;
  };
  const bool f32 = es == 4;
  const Cost of_rows8[] = {{ExpertTile::k16, 1.2, 0.06, 0.05},
                           {ExpertTile::k32, 0.22, 0.096, 0.12},
                           {ExpertTile::k64, 0.6, 0.22, 0.2},
                           {ExpertTile::k128, 2.6, 0.58, 0.45},
                           {ExpertTile::k256, 5.0, 1.3, 1.1}};
  const Cost of_values[] = {{ExpertTile::k16, 0.3, op == ExpertOp::kProduct ? 0.07 : 0.09, f32 ? 0.058 : 0.03},
                            {ExpertTile::k32, 0.25, f32 ? 0.15 : 0.09, f32 ? 0.2 : 0.11},
                            {ExpertTile::k64, 0.4, f32 ? 0.52 : 0.2, f32 ? 0.52 : 0.2},
                            {ExpertTile::k128, 2.0, f32 ? 2.0 : 0.5, f32 ? 2.0 : 0.44},
                            {ExpertTile::k256, 1.0, 1.42, 1.1}};
  const bool odd_lines = es > 1 && (sh.H * es % 128 || (op != ExpertOp::kProduct && sh.F * es % 128));
  ExpertTile best = ExpertTile::k16;
  double least = 0;
  for (const Cost& c : es == 1 ? of_rows8 : of_values) {
    if (c.tile == ExpertTile::k256 && es == 4) continue;
    const ExpertTileSize x = expert_tile_size(c.tile);
    const int step = KB / es;
    const double fixed = c.c0 + (double)x.rows * x.cols * os / 19000.0;
    const double c1 = c.c1 * (odd_lines && x.rows <= 64 ? 1.35 : 1.0);
    const int64_t across = ((op == ExpertOp::kProduct ? sh.F : sh.H) + x.cols - 1) / x.cols;
    double tiles = 0, work = 0, most = 0, longest = 0;
    for (int i = 0; i < n; i++) {
      const int64_t down = ((op == ExpertOp::kWgrad ? sh.F : rows[i]) + x.rows - 1) / x.rows;
      const int64_t k = op == ExpertOp::kProduct ? sh.H : op == ExpertOp::kDgrad ? sh.F : rows[i];
      const double steps = (double)((k + step - 1) / step);
      const double t = fixed + c1 * steps, alone = fixed + c.alone * steps;
      tiles += (double)(down * across);
      work += t * (double)(down * across);
      most = t > most ? t : most;
      longest = alone > longest ? alone : longest;
    }
    double est = work / kCus;
    if (x.rows >= 128 && op != ExpertOp::kWgrad) est = most * ceil(tiles / kCus);
    else if (x.rows >= 128 && est > most) est += most / 4;  // the last round's unevenness
    if (est < longest) est = longest;
    if (least == 0 || est < least) {
      least = est;
      best = c.tile;
    }
  }
  return best;
}

hipError_t launch_experts(ExpertOp op, int es, int os, const ExpertTable& tab, const ExpertShape& sh,
                          ExpertTile tile, int tiles, hipStream_t stream) {
  if (tiles <= 0) return hipSuccess;
  switch (op) {
    case ExpertOp::kProduct:
      return es == 4 ? launch_as<ExpertOp::kProduct, 4, 4>(tab, sh, tile, tiles, stream)
                     : launch_as<ExpertOp::kProduct, 2, 2>(tab, sh, tile, tiles, stream);
    case ExpertOp::kDgrad:
      return es == 4 ? launch_as<ExpertOp::kDgrad, 4, 4>(tab, sh, tile, tiles, stream)
                     : launch_as<ExpertOp::kDgrad, 2, 2>(tab, sh, tile, tiles, stream);
    default:
      if (es == 4) return launch_as<ExpertOp::kWgrad, 4, 4>(tab, sh, tile, tiles, stream);
      return os == 4 ? launch_as<ExpertOp::kWgrad, 2, 4>(tab, sh, tile, tiles, stream)
                     : launch_as<ExpertOp::kWgrad, 2, 2>(tab, sh, tile, tiles, stream);
  }
}

}  // namespace ccr
