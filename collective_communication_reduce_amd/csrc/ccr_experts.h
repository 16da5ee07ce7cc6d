// What the kernels of the experts' matrix products share: the LDS image of an
// operand's tile and the loads that fill it, the tiles of a launch and who takes
// them.  Included by the .hip sources of the products only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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

// LDS image of an operand tile of X rows (the tile's m or n) by one K-step of
// KB = 128 bytes per row (64 bf16 or 32 fp32), in 16-byte vectors.  Loads go
// straight from memory to LDS, which fixes each lane's LDS place (its wave's
// base + 16 x lane), so the bank swizzle is applied to the address a lane reads
// from.
//
// Row image (K contiguous in memory): X rows of 8 vectors; vector c of
// row r sits at c ^ row_swz(r).  A 16-byte read serves 16 lanes at a time, of
// two 16-lane groups (0-3, 12-15 of the one, 4-11 of the other): the swizzle
// puts the 16 vectors they ask for, of 16 rows, on all 64 banks once.
// Column image (the tile's X contiguous): KB / ES rows of X / (16 / ES)
// vectors; vector c of row k sits at c ^ col_swz(k), which spreads the rows
// that one transposing read touches over the banks.
//
// PAIRED: how a fragment's 16 rows (or columns) lie in the tile.  Plain, they
// are 16 neighbours.  Paired, fragments 2 i and 2 i + 1 share 32 neighbours, in
// turns of four: row q of fragment 2 i + u is 8 (q / 4) + 4 u + q % 4 of them,
// so that the four results a lane holds of each are eight neighbours.
template <bool PAIRED>
__device__ __forceinline__ int row_swz(int r) {
  return PAIRED ? ((r >> 1) & 1) | ((r >> 2) & 6) : (r >> 1) & 7;
}
template <int ES, int X, bool PAIRED>
__device__ __forceinline__ int col_swz(int k) {
  constexpr int kPerRow = X * ES / 16;
  if constexpr (ES == 4) return (((k >> 2) & 3) << 2) & (kPerRow - 1);
  else if constexpr (PAIRED) return ((k & 3) << 2) & (kPerRow - 1);
  else return ((((k & 3) | ((k >> 1) & 4)) << 1)) & (kPerRow - 1);
}

// One operand's loads of a K-step: NT threads bring X x KB bytes.  Lanes past
// the tile's last row (or column) read a row inside it: their products are
// not stored.  Lanes past the contraction's end read zeros.
constexpr int KB = 128;

template <int ES, int X, bool COL, bool PAIRED, int NT>
struct Loader {
  static constexpr int kLoads = X * (KB / 16) / NT;
  static constexpr int kStep = KB / ES;        // k values per step
  static constexpr int kPerRow = X * ES / 16;  // vectors per row of a column image
  const char* base;  // the tile's first row (row image) or column (column image)
  int64_t ld;        // bytes from one memory row to the next
  int off[kLoads];   // byte offset of this lane's vector from base, K-step 0
  int k[kLoads];     // first k of the vector

  // p: the operand's first byte; x0: the tile's first row or column; extent:
  // how many there are; thread: this thread's number among the NT
  __device__ __forceinline__ void init(const char* p, int64_t ld_bytes, int64_t x0, int64_t extent,
                                       int thread) {
    ld = ld_bytes;
    const int left = (int)(extent - x0 < X ? extent - x0 : X);
    base = COL ? p + x0 * ES : p + x0 * ld;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int q = i * NT + thread;
      if constexpr (COL) {
        const int kr = q / kPerRow;
        const int c = (q % kPerRow) ^ col_swz<ES, X, PAIRED>(kr);
        off[i] = (int)(kr * ld) + (c * (16 / ES) < left ? c * 16 : 0);
        k[i] = kr;
      } else {
        const int r = q / (KB / 16);
        const int c = (q % (KB / 16)) ^ row_swz<PAIRED>(r);
        off[i] = (int)((r < left ? r : left - 1) * ld) + c * 16;
        k[i] = c * (16 / ES);
      }
    }
  }

  // bytes from one K-step to the next
  __device__ __forceinline__ int64_t stride() const { return COL ? kStep * ld : KB; }
};

// Half of a bf16 fragment from a column image: a transposing read of 4 k x 16
// columns per 16 lanes.  Lane j gives the address of 4 columns of row j / 4 and
// receives column j of the 4 rows.  The fragment is the i-th from column x0 on.
template <int X, bool PAIRED>
__device__ __forceinline__ s16x4 fragment_half(const char* lds, int x0, int i, int h, int u) {
  const int l = threadIdx.x & 63, j = l & 15, g = l >> 4;
  const int k = h * 32 + g * 8 + u * 4 + (j >> 2);
  const int x = PAIRED ? x0 + (i >> 1) * 32 + (j & 3) * 8 + (i & 1) * 4 : x0 + i * 16 + (j & 3) * 4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (CCR_LDS s16x4*)(lds + k * (X * 2) + (((x >> 3) ^ col_swz<2, X, PAIRED>(k)) << 4) + (x & 4) * 2));
}

// A 16-row fragment (the i-th from row x0 on) of 64 bytes of K (part h of the
// step): 4 registers per lane.  Lane l holds row l % 16 and, with g = l / 16,
// k = 32 h + 8 g + (0..7) in bf16 or k = 16 h + 4 g + (0..3) in fp32.  Both
// operands use the same k for the same lane and register, which is all a
// product needs.
template <int ES, int X, bool COL, bool PAIRED>
__device__ __forceinline__ u32x4 fragment(const char* lds, int x0, int i, int h) {
  static_assert(ES != 4 || !PAIRED, "fp32 results are 16 bytes by fours");
  const int l = threadIdx.x & 63, j = l & 15, g = l >> 4;
  if constexpr (!COL) {
    const int r = PAIRED ? x0 + (i >> 1) * 32 + (j >> 2) * 8 + (i & 1) * 4 + (j & 3) : x0 + i * 16 + j;
    return *reinterpret_cast<const u32x4*>(lds + r * KB + (((h * 4 + g) ^ row_swz<PAIRED>(r)) << 4));
  } else if constexpr (ES == 2) {
    const s16x4 v[2] = {fragment_half<X, PAIRED>(lds, x0, i, h, 0),
                        fragment_half<X, PAIRED>(lds, x0, i, h, 1)};
    u32x4 r;
    __builtin_memcpy(&r, v, 16);
    return r;
  } else {
    u32x4 r;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const int k = h * 16 + g * 4 + e;
      const int c = (x0 + i * 16 + j) >> 2;
      r[e] = *reinterpret_cast<const uint32_t*>(
          lds + k * (X * 4) + ((c ^ col_swz<4, X, false>(k)) << 4) + (j & 3) * 4);
    }
    return r;
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

// The same for tiles that do not take equally long (weight gradients, listed
// from the longest on): the XCDs take turns at runs of kRun tiles, short enough
// to share the long ones out, long enough to meet in an L2.  Tiles of 64,
// weights 3016 x 336 of 8 experts of 40 to 17625 rows: 1024 us in contiguous
// runs, 203 us so; with runs of 8 tiles equal experts lose a fifth (8 x 2000
// rows: 43 -> 53 us).
__device__ __forceinline__ int xcd_turns(int b, int n) {
  constexpr int kRun = 16;
  const int i = b >> 3, t = ((i / kRun) * 8 + (b & 7)) * kRun + i % kRun;
  return b < n / (8 * kRun) * (8 * kRun) ? t : b;
}

// The tile that workgroup b of kCus takes in its round r, -1 for none.
// Products and input gradients, whose tiles take equally long: xcd_tile's
// contiguous runs.  Weight gradients, whose tiles take as long as their expert has rows and are listed
// from the longest on: each round's tiles are dealt out in one piece, the later
// rounds in reverse, so that who had a long tile gets a short one (a training
// layer of 16 experts of 518 to 5999 rows: 323 us with contiguous runs, 274 us so).
constexpr int kCus = 256;
template <bool UNEQUAL>
__device__ __forceinline__ int tile_of(int b, int r, int n) {
  if (!UNEQUAL || n <= kCus) return b + r * kCus < n ? xcd_tile(b + r * kCus, n) : -1;
  const int place = (b & 7) * (kCus / 8) + (b >> 3);
  const int t = r == 0 ? place : r * kCus + kCus - 1 - place;
  return t < n ? t : -1;
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

// Tile `in` of a group of mt x nt tiles: strips of 8 tiles in m, column after
// column, so the 32 tiles that an XCD's compute units hold at a time are about
// 8 x 4 and share their operands in its L2.
__device__ __forceinline__ void tile_at(int in, int mt, int nt, int* m, int* n) {
  constexpr int kStrip = 8;
  const int strip = in / (kStrip * nt), r = in - strip * kStrip * nt;
  const int left = mt - strip * kStrip, h = left < kStrip ? left : kStrip;
  *n = r / h;
  *m = strip * kStrip + (r - *n * h);
}

// What a workgroup computes: its expert's operands and sizes (output M x N,
// contraction C) and its tile's corner.  left: values of the contraction that
// follow these C, to be added to the tile afterwards; add: these C are such ones.
struct Where {
  const char *a, *b;
  char* c;
  int64_t M, N, C, m0, n0;
  int64_t left = 0;
  bool add = false;
};
template <ExpertOp OP, int BM, int BN>
__device__ __forceinline__ Where place_of(const ExpertTable& tab, const ExpertShape& sh, int t) {
  const int gi = __builtin_amdgcn_readfirstlane(group_of(tab, t));
  const ExpertGroup& g = tab.g[gi];
  Where at;
  at.a = g.a;
  at.b = g.b;
  at.c = g.c;
  at.M = g.m;
  at.N = OP == ExpertOp::kProduct ? sh.F : sh.H;
  at.C = OP == ExpertOp::kProduct ? sh.H : OP == ExpertOp::kDgrad ? sh.F : g.rows;
  int tm, tn;
  tile_at(t - tab.tile0[gi], (int)((at.M + BM - 1) / BM), (int)((at.N + BN - 1) / BN), &tm, &tn);
  at.m0 = (int64_t)tm * BM;
  at.n0 = (int64_t)tn * BN;
  return at;
}

// The loads are written in assembly (they have no result register, only LDS)
// because the compiler would otherwise wait for all of them before any later
// LDS read.  m0 holds the LDS place; a load must not follow its write directly,
// which is why write, wait state and load are one block that nothing can be
// moved into or out of.  (m0 is reserved and cannot be named as clobbered; the
// compiler has no use of its own for it in these kernels.)
__device__ __forceinline__ void load_lds(uint32_t lds, uint32_t off, const char* base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               ::"s"(lds), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void load_lds(uint32_t lds, const char* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               ::"s"(lds), "v"(p) : "memory");
}

}  // namespace
}  // namespace ccr
