// Device kernels of the root-mean-square norm with the residual's addition, its
// gradients, and 8-bit rows, written for gfx950 (CDNA4: wave64, 256 CUs in 8 XCDs,
// HBM3E).
//
//   h = round(x + residual)             (x itself without a residual)
//   r = 1 / sqrt(mean(h^2) + eps)
//   y = h r w                           rounded once, to the rows' type or 8 bits
//
//   g = w dy,  hh = h r
//   dx = r (g - hh mean(g hh)) + dh     rounded once
//   dw = sum over rows of dy hh         fp32
//
// Every value is read once and written once: bound by HBM.  Squares are taken
// and added in fp64 (no finite row overflows), everything else in fp32.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccr_device.h"
#include "ccr_internal.h"
#include "ccr_rows.h"

namespace ccr {
namespace {

using namespace dev;

// The P weights of vector i.
template <int P, int WES>
__device__ __forceinline__ void load_weight(const char* w, int64_t i, float* f) {
  if constexpr (P * WES == 16) {
    unpack<WES>(reinterpret_cast<const u32x4*>(w)[i], f);
  } else if constexpr (P * WES == 32) {  // bf16 rows, fp32 weights
    unpack<4>(reinterpret_cast<const u32x4*>(w)[2 * i], f);
    unpack<4>(reinterpret_cast<const u32x4*>(w)[2 * i + 1], f + 4);
  } else {  // fp32 rows, bf16 weights
    const u32x2 v = reinterpret_cast<const u32x2*>(w)[i];
    f[0] = bf16_lo(v[0]);
    f[1] = bf16_hi(v[0]);
    f[2] = bf16_lo(v[1]);
    f[3] = bf16_hi(v[1]);
  }
}

// One lane's part of an 8-bit row: the P values of vector i (all lanes of a
// block take part, those past the row's end with zeros).
template <int P>
__device__ __forceinline__ void store_q8(char* q, int64_t i, int64_t values, const float* f) {
  uint32_t bytes[P / 4];
  int scale;
  q8_pack<P>(f, bytes, &scale);
  if (i * P >= values) return;
  if constexpr (P == 8) *reinterpret_cast<u32x2*>(q + i * 8) = u32x2{bytes[0], bytes[1]};
  else *reinterpret_cast<uint32_t*>(q + i * 4) = bytes[0];
  if (i % (32 / P) == 0) q[values + i / (32 / P)] = (char)scale;
}

// The zeros behind an 8-bit row's scales.
template <int TPR>
__device__ __forceinline__ void pad_q8(char* q, int64_t values, int64_t row_bytes, int thread) {
  const int64_t from = values + values / 32;
  for (int64_t i = from + thread * 4; i < row_bytes; i += TPR * 4) *reinterpret_cast<uint32_t*>(q + i) = 0;
}

// A row per TPR threads (a part of a wave, a wave, or the workgroup), NV vectors of
// it in each thread's registers; NV = 0: a row of any length, read twice.  8 x 4096
// rows of 2048 bf16 with residual: 92 us, 5.8 TB/s; to 8 bits 88.
template <int ES, int WES, int TPR, int NV, bool ADD>
__global__ __launch_bounds__(kBlock) void norm_kernel(const NormArgs a, int64_t T, int64_t vpr, int64_t values,
                                                      int64_t q_bytes, double inv_H, float eps,
                                                      int64_t blocks_per_rank) {
  constexpr int P = kPer<ES>, kRows = kBlock / TPR;
  __shared__ double part[kBlock / 64];
  const int rank = (int)(blockIdx.x / blocks_per_rank);
  const int tid = TPR == kBlock ? threadIdx.x : threadIdx.x % TPR;
  const int64_t t = (blockIdx.x % blocks_per_rank) * kRows + (TPR == kBlock ? 0 : threadIdx.x / TPR);
  if (t >= T) return;  // uniform over the threads of a row
  const u32x4* x = reinterpret_cast<const u32x4*>(a.x[rank]) + t * vpr;
  const u32x4* res = ADD ? reinterpret_cast<const u32x4*>(a.res[rank]) + t * vpr : nullptr;
  u32x4* h = ADD ? reinterpret_cast<u32x4*>(a.h[rank]) + t * vpr : nullptr;
  u32x4* y = a.y[rank] ? reinterpret_cast<u32x4*>(a.y[rank]) + t * vpr : nullptr;
  char* q = a.q[rank] ? a.q[rank] + t * q_bytes : nullptr;
  const char* w = a.w[rank];
  double sum = 0;
  auto joined = [&](int64_t i) {  // vector i of h
    u32x4 v = x[i];
    if constexpr (ADD) {
      if constexpr (ES == 4) v = add_f32x4(v, res[i]);
      else v = add_bf16x8(v, res[i]);
    }
    return v;
  };
  auto squares = [&](u32x4 v) {
    float f[P];
    unpack<ES>(v, f);
#pragma unroll
    for (int j = 0; j < P; j++) sum = __builtin_fma((double)f[j], (double)f[j], sum);
  };
  auto finish = [&]() {
    if constexpr (TPR == kBlock) sum = block_sum(sum, part);
    else sum = lanes_sum<TPR>(sum);
    // In fp64, where the mean of any finite values has a root: the instruction's 2^-23
    // and a Newton step, which 0 and infinity do without (a division, a root and
    // another division were most of a short row's instructions).
    const double m = __builtin_fma(sum, inv_H, (double)eps), y = __builtin_amdgcn_rsq(m);
    const double half = 0.5 * m * y, better = __builtin_fma(y, __builtin_fma(-half, y, 0.5), y);
    return m > 0.0 && m < __builtin_inf() ? better : y;
  };
  // Where the root is beyond fp32 or among its subnormal numbers (rows below 2^-128,
  // above 2^126) values and root are multiplied at other scales, which changes
  // neither's digits: `up` on the one side, its inverse on the other.
  float r, up = 1.0f;
  auto emit = [&](int64_t i, u32x4 v) {  // of every vector up to the 8-bit row's end
    float f[P], g[P];
    if (i < vpr) {
      unpack<ES>(v, f);
      load_weight<P, WES>(w, i, g);
    }
    if (__builtin_expect(up != 1.0f, 0)) {
#pragma unroll
      for (int j = 0; j < P; j++) f[j] *= up;
    }
#pragma unroll
    for (int j = 0; j < P; j++) f[j] = i < vpr ? f[j] * r * g[j] : 0.0f;
    if (y && i < vpr) y[i] = pack<ES>(f);
    if (q) store_q8<P>(q, i, values, f);
  };
  auto root = [&]() {
    const double d = finish();
    r = (float)d;
    if (a.rstd[rank] && tid == 0) a.rstd[rank][t] = r;
    if (!(r >= 0x1p-126f && r < __builtin_inff())) {
      up = r < 1.0f ? 0x1p-64f : 0x1p64f;
      r = (float)(d * (r < 1.0f ? 0x1p64 : 0x1p-64));
    }
  };
  const int64_t end = q ? values / P : vpr;
  if constexpr (NV > 0) {
    u32x4 v[NV];
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const int64_t i = tid + n * TPR;
      v[n] = i < vpr ? joined(i) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const int64_t i = tid + n * TPR;
      if (ADD && i < vpr) h[i] = v[n];
      squares(v[n]);
    }
    root();
#pragma unroll
    for (int n = 0; n < NV; n++)
      if (n * TPR < end) emit(tid + n * TPR, v[n]);
  } else {
    for (int64_t i = tid; i < vpr; i += TPR) {
      const u32x4 v = joined(i);
      if (ADD) h[i] = v;
      squares(v);
    }
    root();
    const u32x4* from = ADD ? h : x;
    for (int64_t n = 0; n < end; n += TPR) {
      const int64_t i = n + tid;
      emit(i, i < vpr ? from[i] : u32x4{0, 0, 0, 0});
    }
  }
  if (q) pad_q8<TPR>(q, values, q_bytes, tid);
}

// ---------------------------------------------------------------- backward
// Every workgroup takes every slots-th row (or, of short rows, as many as it
// holds at a time) of its rank, so that it can add up dw in its registers; after
// every kPiece of its rows, and at the end, what it has goes to its slot of the work
// array, and norm_dw_kernel adds the slots (8 x 4096 rows of 2048 bf16 with dh: 115
// and 5 us, 4.7 TB/s).  So no sum of dw is a chain of more than kPiece rows, however
// many there are (of R T < 2^24 rows a slot has up to 136 pieces): chains of 4096
// were off by 980 units of 2^-24.
constexpr int kPiece = 128;
template <int ES, int WES, int TPR, int NV, bool ADD>
__global__ __launch_bounds__(kBlock) void norm_bwd_kernel(const NormBwdArgs a, int64_t T, int64_t vpr, float H,
                                                          int slots, float* work) {
  constexpr int P = kPer<ES>, kRows = kBlock / TPR;
  __shared__ float part[2][kBlock / 64];
  __shared__ float wave_dw[TPR == kBlock ? 1 : kRows][TPR == kBlock ? 1 : TPR * NV * P];
  const int rank = blockIdx.x / slots, slot = blockIdx.x % slots;
  const int tid = TPR == kBlock ? threadIdx.x : threadIdx.x % TPR;
  const int sub = TPR == kBlock ? 0 : threadIdx.x / TPR;
  const u32x4* dy = reinterpret_cast<const u32x4*>(a.dy[rank]);
  const u32x4* h = reinterpret_cast<const u32x4*>(a.h[rank]);
  const u32x4* dh = reinterpret_cast<const u32x4*>(a.dh[rank]);
  u32x4* dx = reinterpret_cast<u32x4*>(a.dx[rank]);
  const float* rstd = a.rstd[rank];
  float w[NV][P], dw[NV][P];
#pragma unroll
  for (int n = 0; n < NV; n++) {
    const int64_t i = tid + n * TPR;
#pragma unroll
    for (int j = 0; j < P; j++) w[n][j] = dw[n][j] = 0.0f;
    if (i < vpr) load_weight<P, WES>(a.w[rank], i, w[n]);
  }
  // A row is loaded while the one before is summed, where a lane has one vector of
  // it; with more it has loads enough on their way.
  constexpr bool kAhead = NV == 1;
  struct Row {
    u32x4 d[NV], h[NV], e[NV];
    float r;
  };
  auto load = [&](int64_t t, Row& x) {
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const int64_t i = tid + n * TPR;
      x.d[n] = x.h[n] = x.e[n] = u32x4{0, 0, 0, 0};
      if (t < T && i < vpr) {
        x.d[n] = dy[t * vpr + i];
        x.h[n] = h[t * vpr + i];
        if (ADD) x.e[n] = dh[t * vpr + i];
      }
    }
    x.r = t < T ? rstd[t] : 0.0f;
  };
  int turn = 0;
  const int64_t step = (int64_t)slots * kRows;
  const int64_t first = (int64_t)slot * kRows;
  int64_t t = first + sub;
  float* out = work + (int64_t)blockIdx.x * vpr * P;
  Row x, next;
  if (kAhead) load(t, next);
  for (int64_t from = first; from < T; from += kPiece * step) {  // uniform over the workgroup
    const int64_t to = T < from + kPiece * step ? T : from + kPiece * step;
    for (; t < to; t += step) {
      if (kAhead) {
        x = next;
        load(t + step, next);
      } else {
        load(t, x);
      }
      const float r = x.r;
      float s = 0;
#pragma unroll
      for (int n = 0; n < NV; n++) {
        float d[P], f[P];
        unpack<ES>(x.d[n], d);
        unpack<ES>(x.h[n], f);
#pragma unroll
        for (int j = 0; j < P; j++) {
          const float hh = f[j] * r;
          s = __builtin_fmaf(w[n][j] * d[j], hh, s);
          dw[n][j] = __builtin_fmaf(d[j], hh, dw[n][j]);
        }
      }
      // two arrays in turn: a wave may be a row ahead of one that still reads
      if constexpr (TPR == kBlock) s = block_sum(s, part[turn]);
      else s = lanes_sum<TPR>(s);
      turn ^= 1;
      s /= H;
#pragma unroll
      for (int n = 0; n < NV; n++) {
        const int64_t i = tid + n * TPR;
        float d[P], f[P], e[P], o[P];
        unpack<ES>(x.d[n], d);
        unpack<ES>(x.h[n], f);
        if (ADD) unpack<ES>(x.e[n], e);
#pragma unroll
        for (int j = 0; j < P; j++) {
          o[j] = r * (w[n][j] * d[j] - f[j] * r * s);
          if (ADD) o[j] += e[j];
        }
        if (i < vpr) dx[t * vpr + i] = pack<ES>(o);
      }
    }
    if constexpr (TPR == kBlock) {
#pragma unroll
      for (int n = 0; n < NV; n++) {
        const int64_t i = tid + n * TPR;
        if (i >= vpr) continue;
#pragma unroll
        for (int j = 0; j < P; j += 4) {
          f32x4* o = reinterpret_cast<f32x4*>(out + i * P + j);
          const f32x4 v = {dw[n][j], dw[n][j + 1], dw[n][j + 2], dw[n][j + 3]};
          *o = from == first ? v : *o + v;
        }
      }
    } else {
      if (from != first) __syncthreads();  // the piece before is read
#pragma unroll
      for (int n = 0; n < NV; n++)
#pragma unroll
        for (int j = 0; j < P; j++) wave_dw[sub][(tid + n * TPR) * P + j] = dw[n][j];
      __syncthreads();
      for (int64_t c = threadIdx.x; c < vpr * P; c += kBlock) {
        float v = 0;
#pragma unroll
        for (int k = 0; k < kRows; k++) v += wave_dw[k][c];
        out[c] = from == first ? v : out[c] + v;
      }
    }
#pragma unroll
    for (int n = 0; n < NV; n++)
#pragma unroll
      for (int j = 0; j < P; j++) dw[n][j] = 0.0f;
  }
}

// Rows of any length: dx in two passes over a row, a workgroup to each.
template <int ES, int WES, bool ADD>
__global__ __launch_bounds__(kBlock) void norm_bwd_long_kernel(const NormBwdArgs a, int64_t T, int64_t vpr,
                                                               float H) {
  constexpr int P = kPer<ES>;
  __shared__ float part[kBlock / 64];
  const int rank = (int)(blockIdx.x / T);
  const int64_t t = blockIdx.x % T;
  const u32x4* dy = reinterpret_cast<const u32x4*>(a.dy[rank]) + t * vpr;
  const u32x4* h = reinterpret_cast<const u32x4*>(a.h[rank]) + t * vpr;
  const u32x4* dh = ADD ? reinterpret_cast<const u32x4*>(a.dh[rank]) + t * vpr : nullptr;
  u32x4* dx = reinterpret_cast<u32x4*>(a.dx[rank]) + t * vpr;
  const float r = a.rstd[rank][t];
  float s = 0;
  for (int64_t i = threadIdx.x; i < vpr; i += kBlock) {
    float d[P], f[P], w[P];
    unpack<ES>(dy[i], d);
    unpack<ES>(h[i], f);
    load_weight<P, WES>(a.w[rank], i, w);
#pragma unroll
    for (int j = 0; j < P; j++) s = __builtin_fmaf(w[j] * d[j], f[j] * r, s);
  }
  s = block_sum(s, part) / H;
  for (int64_t i = threadIdx.x; i < vpr; i += kBlock) {
    float d[P], f[P], w[P], e[P];
    unpack<ES>(dy[i], d);
    unpack<ES>(h[i], f);
    load_weight<P, WES>(a.w[rank], i, w);
    if (ADD) unpack<ES>(dh[i], e);
    float o[P];
#pragma unroll
    for (int j = 0; j < P; j++) {
      o[j] = r * (w[j] * d[j] - f[j] * r * s);
      if (ADD) o[j] += e[j];
    }
    dx[i] = pack<ES>(o);
  }
}

// ... and their dw: a workgroup takes kBlock vectors of every slots-th row.
template <int ES>
__global__ __launch_bounds__(kBlock) void norm_dw_long_kernel(const NormBwdArgs a, int64_t T, int64_t vpr,
                                                              int slots, float* work) {
  constexpr int P = kPer<ES>;
  const int rank = blockIdx.x / slots, slot = blockIdx.x % slots;
  const int64_t i = (int64_t)blockIdx.y * kBlock + threadIdx.x;
  if (i >= vpr) return;
  const u32x4* dy = reinterpret_cast<const u32x4*>(a.dy[rank]);
  const u32x4* h = reinterpret_cast<const u32x4*>(a.h[rank]);
  float sum[P] = {};
  for (int64_t from = slot; from < T; from += (int64_t)kPiece * slots) {  // in pieces, as above
    float dw[P] = {};
    for (int64_t k = 0, t = from; k < kPiece && t < T; k++, t += slots) {
      const float r = a.rstd[rank][t];
      float d[P], f[P];
      unpack<ES>(dy[t * vpr + i], d);
      unpack<ES>(h[t * vpr + i], f);
#pragma unroll
      for (int j = 0; j < P; j++) dw[j] = __builtin_fmaf(d[j], f[j] * r, dw[j]);
    }
#pragma unroll
    for (int j = 0; j < P; j++) sum[j] += dw[j];
  }
  float* out = work + ((int64_t)blockIdx.x * vpr + i) * P;
#pragma unroll
  for (int j = 0; j < P; j++) out[j] = sum[j];
}

// dw (+)= the slots' sums, in a fixed order: a workgroup takes 64 columns, 16
// threads (four columns each) to a slot.
constexpr int kDwBlock = 1024;
__global__ __launch_bounds__(kDwBlock) void norm_dw_kernel(const NormBwdArgs a, const float* work, int slots,
                                                           int64_t H, bool add) {
  constexpr int kWaves = kDwBlock / 64;
  __shared__ f32x4 part[kWaves][16];
  const int rank = blockIdx.y, col = threadIdx.x & 15, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + col * 4;
  const float* from = work + (int64_t)rank * slots * H + c;
  f32x4 s = {0, 0, 0, 0};
  if (c < H)
#pragma unroll 4
    for (int k = threadIdx.x >> 4; k < slots; k += kDwBlock / 16) s += *reinterpret_cast<const f32x4*>(from + k * H);
#pragma unroll
  for (int off = 16; off <= 32; off <<= 1)
#pragma unroll
    for (int j = 0; j < 4; j++) s[j] += __shfl_xor(s[j], off);
  if ((threadIdx.x & 63) < 16) part[wave][col] = s;
  __syncthreads();
  if (threadIdx.x < 16 && c < H) {
    s = part[0][col];
#pragma unroll
    for (int k = 1; k < kWaves; k++) s += part[k][col];
    float* dw = a.dw[rank] + c;  // of a float's alignment
#pragma unroll
    for (int j = 0; j < 4; j++) dw[j] = add ? dw[j] + s[j] : s[j];
  }
}

// -------------------------------------------------------------- 8-bit rows
// To 8 bits or back: a wave takes U times 64 vectors of a row's values, 4 where
// they are there for it, so that it has 4 loads on their way (2 x 11,264 rows of
// 2048 bf16: 39 us with one and its place in 64-bit divisions by lanes, 29 so); or
// ROWS whole rows of up to 64 / ROWS vectors (1,048,576 rows of 64 bf16: 237 us with
// one row to a wave, 117 so).  Back, a lane reads as many bytes as make a vector (16
// bytes and four stores of 64 bytes' distance to fp32 rows of 2048: 103 us for 2^26
// values, 60 so).
template <int ES, int U, int ROWS, bool BACK>
__global__ __launch_bounds__(kBlock) void q8_kernel(const Q8Args a, int R, int64_t vpr, int64_t values,
                                                    int64_t q_bytes, int64_t chunks) {
  constexpr int P = kPer<ES>, kLanes = 64 / ROWS;
  const int lane = threadIdx.x & (kLanes - 1), row = (threadIdx.x & 63) / kLanes;
  const int64_t unit = (int64_t)blockIdx.x * (kBlock / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int rank = 0;
  int64_t t, c = 0;
  if constexpr (ROWS == 1) {
    while (rank < R && unit >= a.first[rank + 1] * chunks) rank++;
    if (rank == R) return;
    const int64_t k = unit - a.first[rank] * chunks;
    t = k / chunks;
    c = k - t * chunks;
  } else {
    t = unit * ROWS + row;  // of all ranks' rows
    while (rank < R && t >= a.first[rank + 1]) rank++;
    if (rank == R) return;  // whole rows' lanes
    t -= a.first[rank];
  }
  const int64_t i0 = c * (64 * U) + lane;
  u32x4* x = reinterpret_cast<u32x4*>(const_cast<char*>(a.rows[rank])) + t * vpr;
  char* q = a.q[rank] + t * q_bytes;
  if constexpr (!BACK) {
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; u++) v[u] = i0 + u * 64 < vpr ? x[i0 + u * 64] : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < U; u++) {
      float f[P];
      unpack<ES>(v[u], f);
      store_q8<P>(q, i0 + u * 64, values, f);
    }
    if (c == chunks - 1) pad_q8<kLanes>(q, values, q_bytes, lane);
  } else {
    uint32_t bytes[U][P / 4];
    uint8_t scale[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t i = i0 + u * 64 < vpr ? i0 + u * 64 : 0;
      __builtin_memcpy(bytes[u], __builtin_assume_aligned(q + i * P, P), P);
      scale[u] = (uint8_t)q[values + i / (32 / P)];
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const float s = q8_factor(scale[u]);
      float f[P];
#pragma unroll
      for (int j = 0; j < P / 4; j++) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)bytes[u][j], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)bytes[u][j], true);
        f[4 * j] = lo[0] * s;
        f[4 * j + 1] = lo[1] * s;
        f[4 * j + 2] = hi[0] * s;
        f[4 * j + 3] = hi[1] * s;
      }
      if (i0 + u * 64 < vpr) x[i0 + u * 64] = pack<ES>(f);
    }
  }
}

template <int ES, bool BACK>
hipError_t launch_q8_as(const Q8Args& a, int R, int64_t H, hipStream_t stream) {
  const int64_t grid64 = q8_grid(ES, a.first[R], H);
  if (grid64 == 0) return hipSuccess;
  if (grid64 > kMaxGridWorkgroups) return hipErrorInvalidValue;
  const unsigned grid = (unsigned)grid64;
  const int64_t vpr = H * ES >> 4, values = q8_values(H), row = q8_row_bytes(H), chunks = q8_chunks(ES, H);
  if constexpr (ES == 2) {
    if (q8_rows(ES, H) == 4) {
      q8_kernel<ES, 1, 4, BACK><<<grid, kBlock, 0, stream>>>(a, R, vpr, values, row, chunks);
      return hipGetLastError();
    }
  }
  if (q8_rows(ES, H) == 2) q8_kernel<ES, 1, 2, BACK><<<grid, kBlock, 0, stream>>>(a, R, vpr, values, row, chunks);
  else if (q8_unroll(ES, H) == 4) q8_kernel<ES, 4, 1, BACK><<<grid, kBlock, 0, stream>>>(a, R, vpr, values, row, chunks);
  else q8_kernel<ES, 1, 1, BACK><<<grid, kBlock, 0, stream>>>(a, R, vpr, values, row, chunks);
  return hipGetLastError();
}

template <int ES, int WES, bool ADD, int TPR, int NV>
hipError_t launch_norm_as(const NormArgs& a, const NormShape& n, hipStream_t stream) {
  constexpr int kRows = kBlock / TPR;
  const int64_t vpr = n.H * ES >> 4, per_rank = (n.T + kRows - 1) / kRows;
  if (per_rank * n.R > kMaxGridWorkgroups) return hipErrorInvalidValue;
  const unsigned grid = (unsigned)(per_rank * n.R);
  norm_kernel<ES, WES, TPR, NV, ADD><<<grid, kBlock, 0, stream>>>(a, n.T, vpr, q8_values(n.H), q8_row_bytes(n.H),
                                                                  1.0 / (double)n.H, n.eps, per_rank);
  return hipGetLastError();
}

// v: vectors that a row's registers have to hold, up to the end of the 8-bit row
// where there is one.  Short rows share a wave, long ones leave the registers; a
// lane has one vector on its way where the residual makes that two loads and two
// stores, else four.  us for 2^26 bf16 values, with residual / to 8 bits without:
//   rows of            64        256       512       1024      2048      8192     16384
//   8 lanes         97
//   16 lanes       147/122     97/40    105/40
//   a wave         441         136       92/55     96/38    101/39
//   the workgroup  1183        325      177       106        90/54    102/40   108
//   read twice     1265        335      186       119       106       114      120
// The gradients':
//   16 lanes        89          83       79
//   32 lanes                    81        83        80        81
//   a wave         266          91       81        84        81
//   the workgroup  1022        283      161        96        80        86      110
//   read twice     1325        359      206       145       138       157      168
template <int ES, int WES, bool ADD>
hipError_t launch_norm_w(const NormArgs& a, const NormShape& n, hipStream_t stream) {
  const int64_t v = (a.q[0] ? q8_values(n.H) : n.H) * ES >> 4;
  if (v <= 8) return launch_norm_as<ES, WES, ADD, 8, 1>(a, n, stream);
  if (v <= 16) return launch_norm_as<ES, WES, ADD, 16, 1>(a, n, stream);
  if (v <= 32) return launch_norm_as<ES, WES, ADD, 16, 2>(a, n, stream);
  if (v <= 64) return launch_norm_as<ES, WES, ADD, ADD ? 64 : 16, ADD ? 1 : 4>(a, n, stream);
  if (v <= 128) return launch_norm_as<ES, WES, ADD, 64, 2>(a, n, stream);
  if (v <= kBlock) return launch_norm_as<ES, WES, ADD, ADD ? kBlock : 64, ADD ? 1 : 4>(a, n, stream);
  if (v <= 2 * kBlock) return launch_norm_as<ES, WES, ADD, kBlock, 2>(a, n, stream);
  if (v <= 4 * kBlock) return launch_norm_as<ES, WES, ADD, kBlock, 4>(a, n, stream);
  if (v <= 8 * kBlock) return launch_norm_as<ES, WES, ADD, kBlock, 8>(a, n, stream);
  return launch_norm_as<ES, WES, ADD, kBlock, 0>(a, n, stream);
}
template <int ES, int WES>
hipError_t launch_norm_of(const NormArgs& a, const NormShape& n, hipStream_t stream) {
  return n.add ? launch_norm_w<ES, WES, true>(a, n, stream) : launch_norm_w<ES, WES, false>(a, n, stream);
}

template <int ES, int WES, int TPR, int NV>
hipError_t launch_norm_bwd_as(const NormBwdArgs& a, const NormShape& n, float* work, hipStream_t stream) {
  const int64_t vpr = n.H * ES >> 4;
  constexpr int kRows = NV > 0 ? kBlock / TPR : 1;
  const int64_t most = norm_slots(n.R, n.T), of = (n.T + kRows - 1) / kRows;  // none without a row
  const int slots = (int)(of < most ? of : most);
  const unsigned grid = (unsigned)(slots * n.R);
  if constexpr (NV > 0) {
    if (n.add)
      norm_bwd_kernel<ES, WES, TPR, NV, true><<<grid, kBlock, 0, stream>>>(a, n.T, vpr, (float)n.H, slots, work);
    else
      norm_bwd_kernel<ES, WES, TPR, NV, false><<<grid, kBlock, 0, stream>>>(a, n.T, vpr, (float)n.H, slots, work);
  } else {
    if (n.T * n.R > kMaxGridWorkgroups) return hipErrorInvalidValue;
    if (n.add)
      norm_bwd_long_kernel<ES, WES, true><<<(unsigned)(n.T * n.R), kBlock, 0, stream>>>(a, n.T, vpr, (float)n.H);
    else
      norm_bwd_long_kernel<ES, WES, false><<<(unsigned)(n.T * n.R), kBlock, 0, stream>>>(a, n.T, vpr, (float)n.H);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    norm_dw_long_kernel<ES><<<dim3(grid, (unsigned)((vpr + kBlock - 1) / kBlock)), kBlock, 0, stream>>>(
        a, n.T, vpr, slots, work);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  norm_dw_kernel<<<dim3((unsigned)((n.H + 63) / 64), n.R), kDwBlock, 0, stream>>>(a, work, slots, n.H, n.accumulate);
  return hipGetLastError();
}

template <int ES, int WES>
hipError_t launch_norm_bwd_w(const NormBwdArgs& a, const NormShape& n, float* work, hipStream_t stream) {
  const int64_t v = n.H * ES >> 4;
  if (v <= 16) return launch_norm_bwd_as<ES, WES, 16, 1>(a, n, work, stream);
  if (v <= 32) return launch_norm_bwd_as<ES, WES, 32, 1>(a, n, work, stream);
  if (v <= 64) return launch_norm_bwd_as<ES, WES, 64, 1>(a, n, work, stream);
  if (v <= 128) return launch_norm_bwd_as<ES, WES, 32, 4>(a, n, work, stream);
  if (v <= kBlock) return launch_norm_bwd_as<ES, WES, kBlock, 1>(a, n, work, stream);
  if (v <= 2 * kBlock) return launch_norm_bwd_as<ES, WES, kBlock, 2>(a, n, work, stream);
  if (v <= 4 * kBlock) return launch_norm_bwd_as<ES, WES, kBlock, 4>(a, n, work, stream);
  if (v <= 8 * kBlock) return launch_norm_bwd_as<ES, WES, kBlock, 8>(a, n, work, stream);
  return launch_norm_bwd_as<ES, WES, kBlock, 0>(a, n, work, stream);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, const NormShape& n, hipStream_t stream) {
  if (n.es == 4) return n.wes == 4 ? launch_norm_of<4, 4>(a, n, stream) : launch_norm_of<4, 2>(a, n, stream);
  return n.wes == 4 ? launch_norm_of<2, 4>(a, n, stream) : launch_norm_of<2, 2>(a, n, stream);
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, const NormShape& n, float* work, hipStream_t stream) {
  if (n.T == 0) {  // no slot: dw is 0
    norm_dw_kernel<<<dim3((unsigned)((n.H + 63) / 64), n.R), kDwBlock, 0, stream>>>(a, work, 0, n.H, n.accumulate);
    return hipGetLastError();
  }
  if (n.es == 4)
    return n.wes == 4 ? launch_norm_bwd_w<4, 4>(a, n, work, stream) : launch_norm_bwd_w<4, 2>(a, n, work, stream);
  return n.wes == 4 ? launch_norm_bwd_w<2, 4>(a, n, work, stream) : launch_norm_bwd_w<2, 2>(a, n, work, stream);
}

hipError_t launch_q8(bool to_q8, int es, const Q8Args& a, int R, int64_t H, hipStream_t stream) {
  if (to_q8) return es == 4 ? launch_q8_as<4, false>(a, R, H, stream) : launch_q8_as<2, false>(a, R, H, stream);
  return es == 4 ? launch_q8_as<4, true>(a, R, H, stream) : launch_q8_as<2, true>(a, R, H, stream);
}

}  // namespace ccr
