// Device kernels of the experts' product on 8-bit rows (ccr_rows.h states their
// format), written for gfx950 (CDNA4: wave64, 256 CUs in 8 XCDs, matrix
// instructions with block scales, 160 KB LDS per CU):
//
//   out[i, f] = sum_h x[i, h] W_e[f, h],  x and W_e in e4m3 with a power of two
//               for every 32 values of h
//
// The matrix instruction multiplies 16 x 128 by 128 x 16 values and takes the
// scales of both sides, so a K-step is one 128-byte line of each row and four of
// its scale bytes, and nothing is rounded but the result.  (Within the
// instruction, the products of 16 neighbouring values are aligned to the largest
// of them and keep 13 bits below it; the sums are fp32.  On rows of normal values
// that is an error of 1.5e-5 of the results, 1% of what rounding them to bf16
// makes.)

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccr_device.h"
#include "ccr_experts.h"
#include "ccr_internal.h"

namespace ccr {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// As load_lds(), 4 bytes per lane.
__device__ __forceinline__ void load_lds4(uint32_t lds, const char* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory");
}

// A 16-row fragment (the i-th from row x0 on) of a K-step: lane l holds row
// l % 16 and, with g = l / 16, the vectors g and 4 + g of its line: k = 16 g +
// (0..15) and 64 + 16 g + (0..15), as the matrix instruction takes them.
template <int X>
__device__ __forceinline__ i32x8 fragment8(const char* lds, int x0, int i) {
  const u32x4 v[2] = {fragment<1, X, false, false>(lds, x0, i, 0), fragment<1, X, false, false>(lds, x0, i, 1)};
  return __builtin_bit_cast(i32x8, v);
}

// The scale that lane l gives for a fragment: of row l % 16, of values 32 g +
// (0..31) of the step.  scales: four bytes per row.
__device__ __forceinline__ int fragment_scale(const char* scales, int x0, int i) {
  const int l = threadIdx.x & 63;
  return (uint8_t)scales[(x0 + i * 16 + (l & 15)) * 4 + (l >> 4)];
}

// D (rows: a's, columns: b's) += a b^T over a K-step.
__device__ __forceinline__ f32x4 mma8(i32x8 a, i32x8 b, f32x4 d, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, d, 0, 0, 0, sa, 0, sb);
}

// Tile BM x BN of the output; WK groups of WM x WN waves, each of which takes
// every WK-th K-step over the whole tile; a ring of NBUF rounds of WK K-steps in
// LDS, a step being the tile's lines of a, of b, and their scales.  Per round one
// barrier: behind it the round's vectors are in LDS and the round before is read
// by every wave, so its buffer takes the loads of the round NBUF - 1 ahead.
template <int BM, int BN, int WM, int WN, int WK, int NBUF>
__global__ __launch_bounds__(WM * WN * WK * 64) void experts8_ring_kernel(const ExpertTable tab,
                                                                          const ExpertShape sh, int64_t row_bytes) {
  constexpr int NT = WM * WN * 64;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
  constexpr int kABytes = BM * KB, kTile = (BM + BN) * KB;
  using LoadA = Loader<1, BM, false, false, NT>;
  using LoadB = Loader<1, BN, false, false, NT>;
  constexpr int kScaleLoads = (BM + BN + NT - 1) / NT;  // of one dword per lane
  constexpr int kStepBytes = kTile + kScaleLoads * NT * 4, kBuf = WK * kStepBytes;
  constexpr int kLoads = LoadA::kLoads + LoadB::kLoads + kScaleLoads;
  static_assert(LoadA::kLoads * NT == BM * 8 && LoadB::kLoads * NT == BN * 8, "whole loads");
  static_assert((NBUF - 2) * kLoads <= 63, "the wait count has 6 bits");
  static_assert(WK == 1 || WK * BM * BN * 4 <= NBUF * kBuf, "the groups' sums fit the ring");
  __shared__ __align__(1024) char lds[NBUF * kBuf];
  const Where at = place_of<ExpertOp::kProduct, BM, BN>(tab, sh, xcd_tile(blockIdx.x, gridDim.x));
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = w / (WM * WN), wg = w % (WM * WN);
  const int wm = (wg / WN) * (BM / WM), wn = (wg % WN) * (BN / WN);
  const int thread = threadIdx.x % NT;
  LoadA la;
  LoadB lb;
  la.init(at.a, row_bytes, at.m0, at.M, thread);
  lb.init(at.b, row_bytes, at.n0, at.N, thread);
  const int nk = (int)((sh.H + KB - 1) / KB);
  // this lane's rows of scales: those of a, then of b; past them the first ones again
  const char* scale[kScaleLoads];
#pragma unroll
  for (int i = 0; i < kScaleLoads; i++) {
    const int q = (i * NT + thread) % (BM + BN);
    const int64_t r = q < BM ? q : q - BM, left = q < BM ? at.M - at.m0 : at.N - at.n0;
    scale[i] = (q < BM ? la.base : lb.base) + (r < left ? r : left - 1) * row_bytes + (int64_t)nk * KB;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(CCR_LDS char*)lds + wk * kStepBytes;
  int j = wk < nk ? wk : nk - 1;  // the step that is loaded next; past the last one, that one again
  auto issue = [&](uint32_t to) {
    const char *pa = la.base + (int64_t)j * KB, *pb = lb.base + (int64_t)j * KB;
#pragma unroll
    for (int i = 0; i < LoadA::kLoads; i++) load_lds(to + wg * 1024 + i * NT * 16, (uint32_t)la.off[i], pa);
#pragma unroll
    for (int i = 0; i < LoadB::kLoads; i++)
      load_lds(to + kABytes + wg * 1024 + i * NT * 16, (uint32_t)lb.off[i], pb);
#pragma unroll
    for (int i = 0; i < kScaleLoads; i++) load_lds4(to + kTile + wg * 256 + i * NT * 4, scale[i] + j * 4);
    j = j + WK < nk ? j + WK : nk - 1;
  };
#pragma unroll
  for (int i = 0; i < NBUF - 1; i++) issue(lds0 + i * kBuf);
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; i++)
#pragma unroll
    for (int n = 0; n < TN; n++) acc[i][n] = f32x4{0, 0, 0, 0};
  int cur = 0, free = (NBUF - 1) * kBuf;  // byte offsets of this round's buffer and of the one read before
  const int rounds = (nk + WK - 1) / WK;
#pragma unroll 1
  for (int r = 0; r < rounds; r++) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NBUF - 2) * kLoads) : "memory");
    const char* from = lds + cur + wk * kStepBytes;
    i32x8 a[TM], b[TN];
    int sa[TM], sb[TN];
#pragma unroll
    for (int i = 0; i < TM; i++) {
      a[i] = fragment8<BM>(from, wm, i);
      sa[i] = fragment_scale(from + kTile, wm, i);
    }
#pragma unroll
    for (int n = 0; n < TN; n++) {
      b[n] = fragment8<BN>(from + kABytes, wn, n);
      sb[n] = fragment_scale(from + kTile, BM + wn, n);
    }
    issue(lds0 + free);
    free = cur;
    cur = cur + kBuf == NBUF * kBuf ? 0 : cur + kBuf;
    if (WK > 1 && r * WK + wk >= nk) continue;  // this group has no step in the last round
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
      for (int n = 0; n < TN; n++) acc[i][n] = mma8(b[n], a[i], acc[i][n], sb[n], sa[i]);
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
        if (c < at.N) store4<2>(at.c + (m * at.N + c) * 2, acc[i][n], false);
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
        part[(wk * BM + wm + i * 16 + (l & 15)) * (BN / 4) + (wn + n * 16) / 4 + (l >> 4)] = acc[i][n];
    __syncthreads();
    for (int q = threadIdx.x; q < BM * BN / 4; q += NT * WK) {
      const int64_t m = at.m0 + q / (BN / 4), c = at.n0 + q % (BN / 4) * 4;
      f32x4 v = part[q];
#pragma unroll
      for (int k = 1; k < WK; k++) v += part[k * BM * BN / 4 + q];
      if (m < at.M && c < at.N) store4<2>(at.c + (m * at.N + c) * 2, v, false);
    }
  }
}

}  // namespace

hipError_t launch_experts8(const ExpertTable& tab, const ExpertShape& sh, ExpertTile tile, int tiles,
                           hipStream_t stream) {
  if (tiles <= 0) return hipSuccess;
  const int64_t row = q8_row_bytes(sh.H);
  switch (tile) {
    case ExpertTile::k16:
      experts8_ring_kernel<16, 16, 1, 1, 4, 4><<<(unsigned)tiles, 256, 0, stream>>>(tab, sh, row);
      break;
    case ExpertTile::k32:
      experts8_ring_kernel<32, 32, 2, 2, 1, 4><<<(unsigned)tiles, 256, 0, stream>>>(tab, sh, row);
      break;
    case ExpertTile::k64:
      experts8_ring_kernel<64, 64, 2, 2, 1, 3><<<(unsigned)tiles, 256, 0, stream>>>(tab, sh, row);
      break;
    default:
      experts8_ring_kernel<128, 128, 2, 4, 1, 4><<<(unsigned)tiles, 512, 0, stream>>>(tab, sh, row);
      break;
  }
  return hipGetLastError();
}

}  // namespace ccr
