// Rows of values on the device, shared by the kernels that stream them (the
// gated sum's neighbours: norms, 8-bit rows): 16-byte vectors to and from fp32,
// sums over a wave, and the 8-bit row format.  gfx950 only.
//
// An 8-bit row of H values: q8_values(H) bytes of e4m3 (H rounded up to whole
// groups of 128, zeros behind the H), then a scale byte for each 32 of them, then
// zeros up to a whole number of 128-byte lines.  Scale byte b stands for 2^(b -
// 127), the form the matrix instructions take; it is the smallest one whose
// block's largest magnitude is at most 448 times it (448 is e4m3's largest value,
// so nothing saturates), 0 for a block of zeros, 255 (NaN) for a block that holds
// an infinity or a NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccr_device.h"
#include "ccr_internal.h"

namespace ccr {
namespace dev {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int ES>
constexpr int kPer = 16 / ES;  // values per 16-byte vector

template <int ES>
__device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
  for (int j = 0; j < 4; j++) {
    if constexpr (ES == 4) {
      f[j] = __builtin_bit_cast(float, (uint32_t)v[j]);
    } else {
      f[2 * j] = bf16_lo(v[j]);
      f[2 * j + 1] = bf16_hi(v[j]);
    }
  }
}

template <int ES>
__device__ __forceinline__ u32x4 pack(const float* f) {
  u32x4 v;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    if constexpr (ES == 4) {
      v[j] = __builtin_bit_cast(uint32_t, f[j]);
    } else {
      f32x2 p = {f[2 * j], f[2 * j + 1]};
      v[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
    }
  }
  return v;
}

// The sum over each N neighbouring lanes, in all of them.
template <int N, typename T>
__device__ __forceinline__ T lanes_sum(T x) {
#pragma unroll
  for (int off = N / 2; off >= 1; off >>= 1) x += __shfl_xor(x, off);
  return x;
}

// The sum over the workgroup's kBlock threads, in every thread, added in the
// same order whatever the timing; `part` holds a T per wave and is free again
// after the next barrier.
template <typename T>
__device__ __forceinline__ T block_sum(T x, T* part) {
  x = lanes_sum<64>(x);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  T s = 0;
#pragma unroll
  for (int w = 0; w < kBlock / 64; w++) s += part[w];
  return s;
}

// The scale byte of a block from the bits of its largest magnitude (as unsigned
// numbers they order magnitudes, infinity and NaN above all others).
__device__ __forceinline__ int q8_scale(uint32_t top) {
  const int b = (int)(top >> 23) + ((top & 0x7fffff) > 0x600000) - 8;  // 448 = 1.75 * 2^8
  return top >= 0x7f800000 ? 255 : b > 0 ? b : 0;
}

// One lane's P values of a block of 32 that P-th parts of lanes (neighbours, the
// first a multiple of 32 / P) hold together: its bytes, and the block's scale.
template <int P>
__device__ __forceinline__ void q8_pack(const float* f, uint32_t* bytes, int* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < P; j++) {
    const uint32_t m = __builtin_bit_cast(uint32_t, f[j]) & 0x7fffffff;
    top = top > m ? top : m;
  }
  // over the block's neighbouring lanes: pairs, quads, halves of a row mirrored
  static_assert(P >= 4 && P <= 16, "two to eight lanes");
  auto merge = [&](int o) { top = top > (uint32_t)o ? top : (uint32_t)o; };
  merge(__builtin_amdgcn_mov_dpp((int)top, 0xb1, 0xf, 0xf, true));
  if constexpr (P < 16) merge(__builtin_amdgcn_mov_dpp((int)top, 0x4e, 0xf, 0xf, true));
  if constexpr (P < 8) merge(__builtin_amdgcn_mov_dpp((int)top, 0x141, 0xf, 0xf, true));
  const int b = q8_scale(top);
  *scale = b;
  const float inv = __builtin_bit_cast(float, (uint32_t)(b < 255 ? 254 - b : 0) << 23);  // 2^(127 - b)
#pragma unroll
  for (int j = 0; j < P / 4; j++) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j] * inv, f[4 * j + 1] * inv, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j + 2] * inv, f[4 * j + 3] * inv, w, true);
    bytes[j] = b < 255 ? (uint32_t)w : 0x7f7f7f7fu;
  }
}

// What scale byte b stands for.
__device__ __forceinline__ float q8_factor(int b) {
  const uint32_t bits = b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : (uint32_t)b << 23;
  return __builtin_bit_cast(float, bits);
}

}  // namespace dev
}  // namespace ccr
