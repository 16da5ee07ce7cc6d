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

#include <type_traits>

#include "ccr_device.h"
#include "ccr_internal.h"

namespace ccr {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
using dev::f32x4;
using dev::u32x4;

#define CCR_LDS __attribute__((address_space(3)))
#define CCR_GLOBAL __attribute__((address_space(1)))

// Source of the lanes that lie past the end of the contraction.
__device__ const u32x4 zero_vector = {0, 0, 0, 0};

// What one K-step of a tile holds of one operand, 128 bytes of K per row:
// 64 bf16 or 32 fp32.
template <int ES>
constexpr int kStep = 128 / ES;

// LDS image of an operand tile of X rows (the tile's m or n) by one K-step,
// in 16-byte vectors.  Loads go straight from memory to LDS, which fixes each
// lane's LDS place (its wave's base + 16 x lane), so the bank swizzle is
// applied to the address a lane reads from.
//
// Row image (K contiguous in memory): X rows of 8 vectors; vector c of row r
// sits at c ^ ((r >> 1) & 7), so 16 lanes that read the same vector of 16
// consecutive rows touch all 64 banks once.
// Column image (the tile's X contiguous): kStep rows of X / (16 / ES)
// vectors; vector c of row k sits at c ^ swz(k), which spreads the rows that
// one transposing read touches over the banks.
template <int ES, int X>
__device__ __forceinline__ int col_swz(int k) {
  constexpr int kPerRow = X * ES / 16;
  if constexpr (ES == 2) return ((((k & 3) | ((k >> 1) & 4)) << 1)) & (kPerRow - 1);
  else return (((k >> 2) & 3) << 2) & (kPerRow - 1);
}

// One operand's loads of a K-step: NT threads bring X x 128 bytes.  Lanes
// past the tile's last row (or column) read a row inside it: their products
// are not stored.  Lanes past the contraction's end read zeros.
template <int ES, int X, bool COL, int NT>
struct Loader {
  static constexpr int kLoads = X * 8 / NT;
  static constexpr int kPerRow = X * ES / 16;  // vectors per row of a column image
  const char* base;  // the tile's first row (row image) or column (column image)
  int64_t ld;        // bytes from one memory row to the next
  int off[kLoads];   // byte offset of this lane's vector from base, K-step 0
  int k[kLoads];     // first k of the vector

  // p: the operand's first byte; x0: the tile's first row or column; extent:
  // how many there are
  __device__ __forceinline__ void init(const char* p, int64_t ld_bytes, int64_t x0, int64_t extent) {
    ld = ld_bytes;
    const int left = (int)(extent - x0 < X ? extent - x0 : X);
    base = COL ? p + x0 * ES : p + x0 * ld;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int q = i * NT + threadIdx.x;
      if constexpr (COL) {
        const int kr = q / kPerRow;
        const int c = (q % kPerRow) ^ col_swz<ES, X>(kr);
        off[i] = (int)(kr * ld) + (c * (16 / ES) < left ? c * 16 : 0);
        k[i] = kr;
      } else {
        const int r = q >> 3;
        const int c = (q & 7) ^ ((r >> 1) & 7);
        off[i] = (int)((r < left ? r : left - 1) * ld) + c * 16;
        k[i] = c * (16 / ES);
      }
    }
  }

  // K-step s of nk; `rest` = k values the last step holds.
  __device__ __forceinline__ void issue(char* lds, int64_t s, int rest, bool last) const {
    const char* from = base + (COL ? s * kStep<ES> * ld : s * 128);
    char* const to = lds + (threadIdx.x & ~63) * 16;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const char* g = from + off[i];
      if (last && k[i] >= rest) g = reinterpret_cast<const char*>(&zero_vector);
      __builtin_amdgcn_global_load_lds((const CCR_GLOBAL unsigned*)g,
                                       (CCR_LDS unsigned*)(to + i * NT * 16), 16, 0, 0);
    }
  }
};

// A 16-row fragment of half a K-step: 4 registers per lane.  Lane l holds row
// l % 16 and, with g = l / 16, k = 32 h + 8 g + (0..7) in bf16 or
// k = 16 h + 4 g + (0..3) in fp32.  Both operands use the same k for the same
// lane and register, which is all a product needs.
template <int ES, int X, bool COL>
__device__ __forceinline__ u32x4 fragment(const char* lds, int x0, int h) {
  const int l = threadIdx.x & 63, j = l & 15, g = l >> 4;
  if constexpr (!COL) {
    const int r = x0 + j;
    return *reinterpret_cast<const u32x4*>(lds + r * 128 + (((h * 4 + g) ^ ((r >> 1) & 7)) << 4));
  } else if constexpr (ES == 2) {
    // two transposing reads of 4 k x 16 columns per 16 lanes: lane j gives the
    // address of 4 columns of row j / 4 and receives column j of the 4 rows
    s16x4 v[2];
#pragma unroll
    for (int u = 0; u < 2; u++) {
      const int k = h * 32 + g * 8 + u * 4 + (j >> 2);
      const int c = (x0 >> 3) + ((j & 3) >> 1);
      v[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (CCR_LDS s16x4*)(lds + k * (X * 2) + ((c ^ col_swz<ES, X>(k)) << 4) + (j & 1) * 8));
    }
    u32x4 r;
    __builtin_memcpy(&r, v, 16);
    return r;
  } else {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int k = h * 16 + g * 4 + i;
      const int c = (x0 + j) >> 2;
      r[i] = *reinterpret_cast<const uint32_t*>(lds + k * (X * 4) + ((c ^ col_swz<ES, X>(k)) << 4) +
                                                (j & 3) * 4);
    }
    return r;
  }
}

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

// Four consecutive values of an output row, rounded once to the output type;
// adding to what is there first when `add`.
template <int OS>
__device__ __forceinline__ void store4(char* p, f32x4 v, bool add) {
  if constexpr (OS == 4) {
    f32x4* q = reinterpret_cast<f32x4*>(p);
    if (add) v += *q;
    *q = v;
  } else {
    bf16x4* q = reinterpret_cast<bf16x4*>(p);
    if (add) v += __builtin_convertvector(*q, f32x4);
    *q = __builtin_convertvector(v, bf16x4);
  }
}

// Which tile of the launch this workgroup takes.  Workgroups go to the XCDs
// round robin; each XCD takes a contiguous run of tiles, so the tiles that
// share an expert's weights meet in one L2.
__device__ __forceinline__ int xcd_tile(int b, int n) {
  const int per = n >> 3, rem = n & 7, x = b & 7;
  return x * per + (x < rem ? x : rem) + (b >> 3);
}

// The group of tile t: the last one whose first tile is at or before it.
__device__ __forceinline__ int group_of(const ExpertTable& tab, int t) {
  const int lane = threadIdx.x & 63;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kExpertGroups; i += 64)
    n += __popcll(__ballot(i + lane < tab.n && tab.tile0[i + lane] <= t));
  return n - 1;
}

// OP as in the table above.  Tile BM x BN of the output, WM x WN waves.
template <ExpertOp OP, int ES, int OS, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void experts_kernel(const ExpertTable tab,
                                                               const ExpertShape sh) {
  constexpr bool kACol = OP == ExpertOp::kWgrad;       // a: x, dout, dout
  constexpr bool kBCol = OP != ExpertOp::kProduct;     // b: W, W, x
  constexpr int NT = WM * WN * 64;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 blocks per wave
  constexpr int kABytes = BM * 128, kBuf = (BM + BN) * 128;
  __shared__ __align__(1024) char lds[2 * kBuf];
  const int t = xcd_tile(blockIdx.x, gridDim.x);
  const int gi = __builtin_amdgcn_readfirstlane(group_of(tab, t));
  const ExpertGroup g = tab.g[gi];
  const int64_t M = OP == ExpertOp::kWgrad ? sh.F : g.rows;
  const int64_t N = OP == ExpertOp::kProduct ? sh.F : sh.H;
  const int64_t C = OP == ExpertOp::kProduct ? sh.H : OP == ExpertOp::kDgrad ? sh.F : g.rows;
  const int mt = (int)((M + BM - 1) / BM);
  const int in = t - tab.tile0[gi];
  const int64_t m0 = (int64_t)(in % mt) * BM, n0 = (int64_t)(in / mt) * BN;
  const int64_t lda = (OP == ExpertOp::kProduct ? sh.H : sh.F) * ES;
  const int64_t ldb = sh.H * ES;
  Loader<ES, BM, kACol, NT> la;
  Loader<ES, BN, kBCol, NT> lb;
  la.init(g.a, lda, m0, M);
  lb.init(g.b, ldb, n0, N);
  const int64_t nk = (C + kStep<ES> - 1) / kStep<ES>;
  const int rest = (int)(C - (nk - 1) * kStep<ES>);
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; i++)
#pragma unroll
    for (int j = 0; j < TN; j++) acc[i][j] = f32x4{0, 0, 0, 0};
  const int w = threadIdx.x >> 6;
  const int wm = (w / WN) * (BM / WM), wn = (w % WN) * (BN / WN);

  if (nk > 0) {
    la.issue(lds, 0, rest, nk == 1);
    lb.issue(lds + kABytes, 0, rest, nk == 1);
  }
  for (int64_t s = 0; s < nk; s++) {
    // this step's vectors are in LDS for every wave, and every wave has read
    // the step before
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const char* cur = lds + (s & 1) * kBuf;
    u32x4 a[2][TM], b[2][TN];
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int i = 0; i < TM; i++) a[h][i] = fragment<ES, BM, kACol>(cur, wm + i * 16, h);
#pragma unroll
      for (int j = 0; j < TN; j++) b[h][j] = fragment<ES, BN, kBCol>(cur + kABytes, wn + j * 16, h);
    }
    if (s + 1 < nk) {
      char* next = lds + ((s + 1) & 1) * kBuf;
      la.issue(next, s + 1, rest, s + 2 == nk);
      lb.issue(next + kABytes, s + 1, rest, s + 2 == nk);
    }
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) acc[i][j] = mma<ES>(b[h][j], a[h][i], acc[i][j]);
  }

  // D holds b's rows (the output's columns) down its registers: lane l has
  // output row l % 16 and columns 4 (l / 16) + (0..3) of each 16 x 16 block.
  const int l = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < TM; i++) {
    const int64_t m = m0 + wm + i * 16 + (l & 15);
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < TN; j++) {
      const int64_t n = n0 + wn + j * 16 + (l >> 4) * 4;
      if (n < N) store4<OS>(g.c + (m * N + n) * OS, acc[i][j], sh.add);
    }
  }
}

// ------------------------------------------------------------- large tiles
// bf16 products of 256 x 256 tiles: four waves, one to a SIMD, each with a
// 128 x 128 part of the tile in its accumulators.  Per K-step of 64 a wave
// reads 32 KiB from LDS for 128 MFMAs.
//
// Two LDS buffers of one K-step each, two register sets of half a step each:
// while a half's products run, the other half's fragments are read, and while
// the second half's run, the loads of the step after the next go out into the
// buffer just read empty.  So loads have a whole K-step to arrive, and there
// is one barrier per K-step, in its middle.
//
// The loads are written in assembly (they have no result register, only LDS)
// because the compiler would otherwise wait for all of them before any later
// LDS read.
__device__ __forceinline__ void load_lds(uint32_t lds, uint32_t off, const char* base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               ::"s"(lds), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void load_lds(uint32_t lds, const char* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               ::"s"(lds), "v"(p) : "memory");
}

// D += a b^T with D held in accumulation registers.  Written in assembly
// because all 256 of them are accumulators here, which the compiler's own
// allocation mixes with the fragments and moves about in the loop.  No two
// products in a row touch the same D, so no wait states are due between them;
// drain() provides those before D is read.
__device__ __forceinline__ void mma_acc(u32x4 a, u32x4 b, f32x4& d) {
  asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(d) : "v"(a), "v"(b));
}
__device__ __forceinline__ void drain(f32x4* d) {
  asm volatile("s_nop 15\n\ts_nop 15"
               : "+a"(d[0]), "+a"(d[1]), "+a"(d[2]), "+a"(d[3]), "+a"(d[4]), "+a"(d[5]), "+a"(d[6]),
                 "+a"(d[7]));
}

template <ExpertOp OP, int OS>
__global__ __launch_bounds__(256, 1) void experts_big_kernel(const ExpertTable tab, const ExpertShape sh) {
  constexpr int ES = 2, BM = 256, BN = 256, NT = 256, T = 8;
  constexpr bool kACol = OP == ExpertOp::kWgrad;
  constexpr bool kBCol = OP != ExpertOp::kProduct;
  constexpr int kABytes = BM * 128, kBuf = (BM + BN) * 128;
  using LoadA = Loader<ES, BM, kACol, NT>;
  using LoadB = Loader<ES, BN, kBCol, NT>;
  __shared__ __align__(1024) char lds[2 * kBuf];
  const int t = xcd_tile(blockIdx.x, gridDim.x);
  const int gi = __builtin_amdgcn_readfirstlane(group_of(tab, t));
  const ExpertGroup g = tab.g[gi];
  const int64_t M = OP == ExpertOp::kWgrad ? sh.F : g.rows;
  const int64_t N = OP == ExpertOp::kProduct ? sh.F : sh.H;
  const int64_t C = OP == ExpertOp::kProduct ? sh.H : OP == ExpertOp::kDgrad ? sh.F : g.rows;
  const int mt = (int)((M + BM - 1) / BM);
  const int in = t - tab.tile0[gi];
  const int64_t m0 = (int64_t)(in % mt) * BM, n0 = (int64_t)(in / mt) * BN;
  const int64_t lda = (OP == ExpertOp::kProduct ? sh.H : sh.F) * ES;
  const int64_t ldb = sh.H * ES;
  const int l = threadIdx.x & 63;
  if (OP == ExpertOp::kWgrad && C == 0) {  // an expert without a row
    for (int i = threadIdx.x; i < BM * (BN / 4); i += NT) {
      const int64_t m = m0 + i / (BN / 4), n = n0 + i % (BN / 4) * 4;
      if (m < M && n < N) store4<OS>(g.c + (m * N + n) * OS, f32x4{0, 0, 0, 0}, sh.add);
    }
    return;
  }
  LoadA la;
  LoadB lb;
  la.init(g.a, lda, m0, M);
  lb.init(g.b, ldb, n0, N);
  const int nk = (int)((C + kStep<ES> - 1) / kStep<ES>);
  const int rest = (int)(C - (int64_t)(nk - 1) * kStep<ES>);
  f32x4 acc[T][T];
#pragma unroll
  for (int i = 0; i < T; i++)
#pragma unroll
    for (int j = 0; j < T; j++) acc[i][j] = f32x4{0, 0, 0, 0};
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (w >> 1) * 128, wn = (w & 1) * 128;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(CCR_LDS char*)lds + w * 1024;

  // K-step 0 is the partial one (rest values, then zeros), so that every later
  // step is whole: step s > 0 starts at k = rest + 64 (s - 1).
  const char* pa = la.base + (kACol ? rest * la.ld : rest * ES);
  const char* pb = lb.base + (kBCol ? rest * lb.ld : rest * ES);
  const int64_t da = kACol ? kStep<ES> * la.ld : 128, db = kBCol ? kStep<ES> * lb.ld : 128;
  constexpr int kLoads = LoadA::kLoads + LoadB::kLoads;
  auto load_first = [&]() {
    const char* zero = reinterpret_cast<const char*>(&zero_vector);
#pragma unroll
    for (int i = 0; i < LoadA::kLoads; i++)
      load_lds(lds0 + i * NT * 16, la.k[i] < rest ? la.base + la.off[i] : zero);
#pragma unroll
    for (int i = 0; i < LoadB::kLoads; i++)
      load_lds(lds0 + kABytes + i * NT * 16, lb.k[i] < rest ? lb.base + lb.off[i] : zero);
  };
  // load i (a's, then b's) of the step at pa, pb
  auto load = [&](int i, uint32_t to) {
    if (i < LoadA::kLoads) load_lds(to + i * NT * 16, (uint32_t)la.off[i], pa);
    else load_lds(to + kABytes + (i - LoadA::kLoads) * NT * 16, (uint32_t)lb.off[i - LoadA::kLoads], pb);
  };

  u32x4 a[2][T], b[2][T];
  // fragment i of half h from the buffer at cur: b's, then a's
  auto read = [&](int i, int h, const char* cur) {
    if (i < T) b[h][i] = fragment<ES, BN, kBCol>(cur + kABytes, wn + i * 16, h);
    else a[h][i - T] = fragment<ES, BM, kACol>(cur, wm + (i - T) * 16, h);
  };

  {
    load_first();
    if (nk > 1) {
#pragma unroll
      for (int i = 0; i < kLoads; i++) load(i, lds0 + kBuf);
      pa += da;
      pb += db;
      asm volatile("s_waitcnt vmcnt(16)" ::: "memory");
      static_assert(kLoads == 16, "the second step's loads may be in flight");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    asm volatile("s_barrier" ::: "memory");
#pragma unroll
    for (int i = 0; i < 2 * T; i++) read(i, 0, lds);
    int cur = 0;  // byte offset of step s's buffer
    int s = 0;
#pragma unroll 1
    do {
#pragma unroll
      for (int i = 0; i < T; i++) {
        if (i < 6) {
#pragma unroll
          for (int x = 0; x < 3; x++)
            if (i * 3 + x < 2 * T) read(i * 3 + x, 1, lds + cur);
        }
#pragma unroll
        for (int j = 0; j < T; j++) mma_acc(b[0][j], a[0][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
      // step s is read by every wave; step s + 1 is in LDS
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      const uint32_t to = lds0 + cur;
      cur ^= kBuf;
      const bool more = s + 2 < nk;
#pragma unroll
      for (int i = 0; i < T; i++) {
        // after the last step this reads what the buffer held before; unused
        if (i < 6) {
#pragma unroll
          for (int x = 0; x < 3; x++)
            if (i * 3 + x < 2 * T) read(i * 3 + x, 0, lds + cur);
        }
        if (more) {
#pragma unroll
          for (int x = 0; x < kLoads / T; x++) load(i * (kLoads / T) + x, to);
        }
#pragma unroll
        for (int j = 0; j < T; j++) mma_acc(b[1][j], a[1][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
      pa += da;
      pb += db;
    } while (++s < nk);
    drain(acc[T - 1]);
  }

#pragma unroll
  for (int i = 0; i < T; i++) {
    const int64_t m = m0 + wm + i * 16 + (l & 15);
#pragma unroll
    for (int j = 0; j < T; j++) {
      asm volatile("" : "+a"(acc[i][j]));  // read out row by row, not all at once
      const int64_t n = n0 + wn + j * 16 + (l >> 4) * 4;
      if (m < M && n < N) store4<OS>(g.c + (m * N + n) * OS, acc[i][j], sh.add);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <ExpertOp OP, int ES, int OS>
hipError_t launch_as(const ExpertTable& tab, const ExpertShape& sh, ExpertTile tile, int tiles,
                     hipStream_t stream) {
  if constexpr (ES == 2)
    if (tile.m == 256) {
      experts_big_kernel<OP, OS><<<(unsigned)tiles, 256, 0, stream>>>(tab, sh);
      return hipGetLastError();
    }
  experts_kernel<OP, ES, OS, 128, 128, 2, 2><<<(unsigned)tiles, 256, 0, stream>>>(tab, sh);
  return hipGetLastError();
}

}  // namespace

ExpertTile expert_tile(ExpertOp op, int es, const ExpertShape& sh, int64_t max_rows, int64_t rows) {
  if (es == 2 && rows >= 4096) return ExpertTile{256, 256};
  return ExpertTile{128, 128};
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
