// Device kernels of the global gradient norm and of clipping, written for
// gfx950 (CDNA4: wave64, 256 CUs in 8 XCDs, HBM3E).
//
//   norm = sqrt(sum over every tensor, over every element, of g^2)
//   out  = g * min(1, max_norm / (norm + 1e-6))
//
// Both are streaming passes bound by HBM.  The tensors of a call are cut into
// tiles and the tiles dealt round robin to at most kGradSlots workgroups, so a
// call over hundreds of small tensors takes a launch per 200 of them (133 where
// results go elsewhere): 500 tensors of 2700 values, norm 17.4 us with launches
// of 112, 11.4 so, clipping 32.9 and 20.0.  Each workgroup leaves one fp64 partial in its own slot of the caller's
// work array; the slots are added in a fixed order, so the norm has the same
// bits on every run.  Squares are taken and added in
// fp64: the square of any fp32 value is exact in it and neither overflows nor
// underflows, and at HBM rate its cost does not show.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccr_device.h"
#include "ccr_internal.h"

namespace ccr {
namespace {

using dev::u32x4;

// 16-byte vectors per thread and tile.  Clipping 200 Mi values of both types:
// 8: 432 us, 4: 335, 2: 348, 1: 411.
constexpr int kVecs = 4;
constexpr int64_t kTileVecs = kBlock * kVecs;  // 16 KiB

// A tensor as the kernels walk it: `head` elements up to the first 16-byte
// boundary, then whole vectors, then a tail shorter than one.
struct Span {
  const char* src;
  char* dst;
  int64_t count, nvec;
  int head, tail;
};

template <int ES>
__device__ __forceinline__ Span span_of(const GradTensor& t) {
  Span s;
  s.src = t.src;
  s.dst = t.dst;
  s.count = t.count;
  const int64_t to_edge = ((16 - (int)(reinterpret_cast<uintptr_t>(t.src) & 15)) & 15) / ES;
  s.head = (int)(to_edge < t.count ? to_edge : t.count);
  s.nvec = (t.count - s.head) * ES >> 4;
  s.tail = (int)(t.count - s.head - s.nvec * (16 / ES));
  return s;
}

template <int ES>
__device__ __forceinline__ float element(const char* p, int64_t i) {
  if constexpr (ES == 4) return reinterpret_cast<const float*>(p)[i];
  else return dev::bf16_lo(reinterpret_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ double square(float x) { return (double)x * (double)x; }

template <int ES>
__device__ __forceinline__ double squares(u32x4 v, double acc) {
#pragma unroll
  for (int j = 0; j < 4; j++) {
    if constexpr (ES == 4) {
      acc += square(__builtin_bit_cast(float, (uint32_t)v[j]));
    } else {
      acc += square(dev::bf16_lo(v[j]));
      acc += square(dev::bf16_hi(v[j]));
    }
  }
  return acc;
}

// A tile's vectors: thread's of the kBlock threads that share it; past the
// tensor's end zeros if FILL, else anything.
template <int ES, bool NT, bool FILL>
__device__ __forceinline__ void tile_load(const Span& s, int64_t tile, int thread, u32x4* x) {
  const u32x4* v = reinterpret_cast<const u32x4*>(s.src + (int64_t)s.head * ES);
  const int64_t first = tile * kTileVecs + thread;
#pragma unroll
  for (int u = 0; u < kVecs; u++) {
    const int64_t i = first + u * kBlock;
    if constexpr (FILL) x[u] = i < s.nvec ? dev::load16<NT>(v + i) : u32x4{0, 0, 0, 0};
    else if (i < s.nvec) x[u] = dev::load16<NT>(v + i);
  }
}

template <int ES>
__device__ __forceinline__ double tile_sum(const Span& s, int64_t tile, int thread, const u32x4* x,
                                           double acc) {
#pragma unroll
  for (int u = 0; u < kVecs; u++) acc = squares<ES>(x[u], acc);
  if (tile == 0 && thread < s.head) acc += square(element<ES>(s.src, thread));
  if (tile == 0 && thread < s.tail) acc += square(element<ES>(s.src, s.count - s.tail + thread));
  return acc;
}

template <int ES, bool NT>
__device__ __forceinline__ double tile_squares(const GradTensor& t, int64_t tile, double acc) {
  const Span s = span_of<ES>(t);
  u32x4 x[kVecs];
  tile_load<ES, NT, true>(s, tile, threadIdx.x, x);
  return tile_sum<ES>(s, tile, threadIdx.x, x, acc);
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off);
  return x;
}

// The sum over the workgroup, in every thread; `part` holds a double per wave.
template <int WAVES = kBlock / 64>
__device__ __forceinline__ double block_sum(double x, double* part) {
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0;
#pragma unroll
  for (int w = 0; w < WAVES; w++) s += part[w];
  return s;
}

// The tensor that holds tile `tile` (the last whose first tile is at or before
// it) and the tile's number in it.  Every lane looks at a few first tiles.
struct Place {
  GradTensor t;
  int64_t tile;
};
__device__ __forceinline__ Place place_of(const GradTable& tab, int64_t tile) {
  const int lane = threadIdx.x & 63;
  constexpr int kLooks = (kGradTensors + 63) / 64;
  int first[kLooks];
#pragma unroll
  for (int i = 0; i < kLooks; i++) {  // all on their way before the first is used
    const int j = i * 64 + lane;
    first[i] = tab.tile0[j < tab.n ? j : 0];
  }
  int n = 0;
#pragma unroll
  for (int i = 0; i < kLooks; i++)
    n += __popcll(__ballot((i * 64 + lane < tab.n) & (first[i] <= (int)tile)));
  n = __builtin_amdgcn_readfirstlane(n - 1);
  const uint64_t* w = tab.word + n * tab.words;
  Place p;
  // as global memory, or the accesses would be flat ones
  typedef __attribute__((address_space(1))) char* Global;
  p.t.src = (const char*)reinterpret_cast<Global>(w[0]);
  p.t.dst = (char*)reinterpret_cast<Global>(w[tab.words == 3 ? 2 : 0]);
  p.t.count = (int64_t)(w[1] >> 1);
  p.t.es = w[1] & 1 ? 2 : 4;
  p.tile = tile - tab.tile0[n];
  return p;
}

// One partial per workgroup: work[b] = (add ? work[b] : 0) + its tiles' sum.
// Tiles below `stream` are loaded non-temporally.
__global__ __launch_bounds__(kBlock) void grad_squares_kernel(const GradTable tab, int64_t stream,
                                                              double* work, int add) {
  __shared__ double part[kBlock / 64];
  double acc = 0;
  for (int64_t tile = blockIdx.x; tile < tab.ntiles; tile += gridDim.x) {
    const Place p = place_of(tab, tile);
    if (tile < stream)
      acc = p.t.es == 4 ? tile_squares<4, true>(p.t, p.tile, acc) : tile_squares<2, true>(p.t, p.tile, acc);
    else
      acc = p.t.es == 4 ? tile_squares<4, false>(p.t, p.tile, acc) : tile_squares<2, false>(p.t, p.tile, acc);
  }
  const double s = block_sum(acc, part);
  if (threadIdx.x == 0) work[blockIdx.x] = add ? work[blockIdx.x] + s : s;
}

// The sum of the slots, the same additions in the same order in every
// workgroup that makes it.
__device__ __forceinline__ double total_of(const double* work, int slots, double* part) {
  double acc = 0;
  for (int i = threadIdx.x; i < slots; i += kBlock) acc += work[i];
  return block_sum(acc, part);
}

__global__ __launch_bounds__(kBlock) void grad_norm_kernel(const double* work, int slots, float* norm) {
  __shared__ double part[kBlock / 64];
  const double s = total_of(work, slots, part);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

// Each result is rounded once more than the fp32 product: to its own type.
template <int ES>
__device__ __forceinline__ u32x4 scaled(u32x4 v, float c) {
  u32x4 r;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    if constexpr (ES == 4) {
      r[j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, (uint32_t)v[j]) * c);
    } else {
      dev::f32x2 f = {dev::bf16_lo(v[j]) * c, dev::bf16_hi(v[j]) * c};
      r[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, dev::bf16x2));
    }
  }
  return r;
}

template <int ES>
__device__ __forceinline__ void scale_element(const Span& s, int64_t i, float c) {
  const float r = element<ES>(s.src, i) * c;
  if constexpr (ES == 4) reinterpret_cast<float*>(s.dst)[i] = r;
  else reinterpret_cast<__bf16*>(s.dst)[i] = static_cast<__bf16>(r);
}

template <int ES, bool NT>
__device__ __forceinline__ void tile_store(const Span& s, int64_t tile, int thread, const u32x4* x,
                                           float c) {
  char* const out = s.dst + (int64_t)s.head * ES;
  const int64_t first = tile * kTileVecs + thread;
  if ((reinterpret_cast<uintptr_t>(out) & 15) == 0) {
#pragma unroll
    for (int u = 0; u < kVecs; u++) {
      const int64_t i = first + u * kBlock;
      if (i < s.nvec) dev::store16<NT>(reinterpret_cast<u32x4*>(out) + i, scaled<ES>(x[u], c));
    }
  } else {  // the result's buffer starts at another offset within 16 bytes
#pragma unroll
    for (int u = 0; u < kVecs; u++) {
      const int64_t i = first + u * kBlock;
      if (i >= s.nvec) continue;
      const u32x4 r = scaled<ES>(x[u], c);
      if constexpr (ES == 4) {
#pragma unroll
        for (int j = 0; j < 4; j++) reinterpret_cast<uint32_t*>(out)[4 * i + j] = r[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
          reinterpret_cast<uint16_t*>(out)[8 * i + j] = (uint16_t)(r[j >> 1] >> (16 * (j & 1)));
      }
    }
  }
  if (tile == 0 && thread < s.head) scale_element<ES>(s, thread, c);
  if (tile == 0 && thread < s.tail) scale_element<ES>(s, s.count - s.tail + thread, c);
}

template <int ES, bool NT>
__device__ __forceinline__ void tile_scale(const GradTensor& t, int64_t tile, float c) {
  const Span s = span_of<ES>(t);
  u32x4 x[kVecs];
  tile_load<ES, NT, false>(s, tile, threadIdx.x, x);
  tile_store<ES, NT>(s, tile, threadIdx.x, x, c);
}

// min(1, max_norm / (norm + 1e-6)).  A NaN stays; an infinite max_norm only
// measures, whatever the norm.
__device__ __forceinline__ float factor_of(float norm, float max_norm) {
  const float q = max_norm / (norm + 1e-6f);
  return q > 1.0f || max_norm == __builtin_inff() ? 1.0f : q;
}

// out = g * factor over the tiles, the last tile
// first: the pass before left the end of the gradients in the last-level
// cache.  Every workgroup adds the slots itself (16 KiB from L2), which saves
// a launch between the two passes.  In place, a factor of 1 writes nothing.
// NT: loads and stores are non-temporal.  The launch bound keeps all
// kGradSlots workgroups resident, eight to a compute unit: with two registers
// more, and so seven, 200 Mi values of both types take 361 us, not 331.
template <bool NT>
__global__ __launch_bounds__(kBlock, 8) void grad_clip_kernel(const GradTable tab, const double* work,
                                                           int slots, float max_norm, float* norm) {
  __shared__ double part[kBlock / 64];
  const float nv = (float)sqrt(total_of(work, slots, part));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = nv;
  const float c = factor_of(nv, max_norm);
  for (int64_t tile = tab.ntiles - 1 - blockIdx.x; tile >= 0; tile -= gridDim.x) {
    const Place p = place_of(tab, tile);
    if (c == 1.0f && p.t.src == p.t.dst) continue;
    if (p.t.es == 4) tile_scale<4, NT>(p.t, p.tile, c);
    else tile_scale<2, NT>(p.t, p.tile, c);
  }
}

// A call of up to grad_small_tiles tiles: one workgroup of kGroups times kBlock
// threads, each kBlock of them with up to kMine tiles in registers, makes the
// norm and the clipping in one launch and one pass over the gradients.  It is
// bound by latency: the launch, the loads, the stores.  The norm alone saves a
// launch, clipping a read of cold gradients too, so it pays up to more tiles.  us
// in one launch / in two, replayed from a graph, of whole tiles of fp32:
//   tiles              1         4         6         8        10        11        12
//   norm, warm     2.2/3.7   2.8/4.1   3.2/4.2   3.8/4.2   4.2/4.2   4.4/4.2   4.8/4.2
//   norm, cold     2.9/4.2   3.4/4.5   4.0/4.6   5.7/4.6   6.6/4.6   6.9/4.6   7.5/4.6
//   clip, warm     2.9/5.4   3.9/6.1   4.5/6.2   5.6/6.3   6.1/6.3   6.3/6.4   7.1/6.4
//   clip, cold     3.6/6.6   5.3/8.8   6.5/9.3   7.5/9.5   8.3/9.5   8.8/9.5   9.6/9.5
constexpr int kGroups = 4;
template <bool CLIP>
constexpr int kMine = (grad_small_tiles(CLIP) + kGroups - 1) / kGroups;
template <bool CLIP>
__global__ __launch_bounds__(kBlock * kGroups) void grad_small_kernel(const GradTable tab, float max_norm,
                                                                      float* norm) {
  __shared__ double part[kGroups * kBlock / 64];
  const int thread = threadIdx.x % kBlock;
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / kBlock);
  u32x4 x[kMine<CLIP>][kVecs];
  Place p[kMine<CLIP>];
#pragma unroll
  for (int m = 0; m < kMine<CLIP>; m++) {
    const int tile = m * kGroups + group;
    if (tile >= tab.ntiles) continue;
    p[m] = place_of(tab, tile);
    if (p[m].t.es == 4) tile_load<4, false, true>(span_of<4>(p[m].t), p[m].tile, thread, x[m]);
    else tile_load<2, false, true>(span_of<2>(p[m].t), p[m].tile, thread, x[m]);
  }
  double acc = 0;
#pragma unroll
  for (int m = 0; m < kMine<CLIP>; m++) {
    if (m * kGroups + group >= tab.ntiles) continue;
    acc = p[m].t.es == 4 ? tile_sum<4>(span_of<4>(p[m].t), p[m].tile, thread, x[m], acc)
                         : tile_sum<2>(span_of<2>(p[m].t), p[m].tile, thread, x[m], acc);
  }
  const float nv = (float)sqrt(block_sum<kGroups * kBlock / 64>(acc, part));
  if (threadIdx.x == 0) *norm = nv;
  if constexpr (CLIP) {
    const float c = factor_of(nv, max_norm);
#pragma unroll
    for (int m = 0; m < kMine<CLIP>; m++) {
      if (m * kGroups + group >= tab.ntiles || (c == 1.0f && p[m].t.src == p[m].t.dst)) continue;
      if (p[m].t.es == 4) tile_store<4, false>(span_of<4>(p[m].t), p[m].tile, thread, x[m], c);
      else tile_store<2, false>(span_of<2>(p[m].t), p[m].tile, thread, x[m], c);
    }
  }
}

}  // namespace

int64_t grad_tile_bytes() { return kTileVecs * 16; }

int64_t grad_tiles(const void* p, int64_t count, int es) {
  const int64_t to_edge = ((16 - (int)(reinterpret_cast<uintptr_t>(p) & 15)) & 15) / es;
  const int64_t nvec = count > to_edge ? (count - to_edge) * es >> 4 : 0;
  const int64_t t = (nvec + kTileVecs - 1) / kTileVecs;
  return t > 0 ? t : 1;
}

hipError_t launch_grad_squares(const GradTable& tab, int grid, int64_t stream_tiles, double* work,
                               bool add, hipStream_t stream) {
  grad_squares_kernel<<<(unsigned)grid, kBlock, 0, stream>>>(tab, stream_tiles, work, add ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_grad_small(const GradTable& tab, bool clip, float max_norm, float* norm,
                             hipStream_t stream) {
  if (clip) grad_small_kernel<true><<<1, kBlock * kGroups, 0, stream>>>(tab, max_norm, norm);
  else grad_small_kernel<false><<<1, kBlock * kGroups, 0, stream>>>(tab, max_norm, norm);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const double* work, int slots, float* norm, hipStream_t stream) {
  grad_norm_kernel<<<1, kBlock, 0, stream>>>(work, slots, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradTable& tab, int grid, bool nontemporal, const double* work,
                            int slots, float max_norm, float* norm, hipStream_t stream) {
  if (nontemporal)
    grad_clip_kernel<true><<<(unsigned)grid, kBlock, 0, stream>>>(tab, work, slots, max_norm, norm);
  else
    grad_clip_kernel<false><<<(unsigned)grid, kBlock, 0, stream>>>(tab, work, slots, max_norm, norm);
  return hipGetLastError();
}

}  // namespace ccr
