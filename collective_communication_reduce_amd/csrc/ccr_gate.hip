// Device kernels of the gated sum that ends an expert-parallel layer, and of
// its gradients, written for gfx950 (CDNA4: wave64, 256 CUs in 8 XCDs, HBM3E).
//
// Per token, with S the set the softmax runs over (the K choices, or all E
// experts) and e_k the expert of choice k:
//
//   w_k       = exp(l[e_k] - m) / sum_{S} exp(l - m),  m = max_{S} l
//   y         = sum_k w_k row_k
//   drow_k    = w_k dy
//   g_k       = <dy, row_k>,  s = sum_k w_k g_k
//   dl[e_k]  += w_k (g_k - s)         (S = the choices)
//   dl[e]     = sum_{k: e_k = e} w_k g_k - p_e s   (S = all experts)
//
// An absent choice (its expert id outside [0, E), or its logit -inf) has
// weight 0 and its row is not read.  Everything is one pass over the rows,
// bound by HBM: 16-byte loads, all K rows of a column in flight together,
// fp32 sums, one rounding to the row type.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccr_device.h"
#include "ccr_internal.h"

namespace ccr {
namespace {

using dev::u32x4;

template <int ES>
constexpr int kPer = 16 / ES;  // values per 16-byte vector

template <int ES>
__device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
  for (int j = 0; j < 4; j++) {
    if constexpr (ES == 4) {
      f[j] = __builtin_bit_cast(float, (uint32_t)v[j]);
    } else {
      f[2 * j] = dev::bf16_lo(v[j]);
      f[2 * j + 1] = dev::bf16_hi(v[j]);
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
      dev::f32x2 p = {f[2 * j], f[2 * j + 1]};
      v[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, dev::bf16x2));
    }
  }
  return v;
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x = fmaxf(x, __shfl_xor(x, off));
  return x;
}
__device__ __forceinline__ float wave_add(float x) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off);
  return x;
}

constexpr float kNegInf = -__builtin_inff();

// exp(l - m), 0 for l = -inf also where every l is
__device__ __forceinline__ float term(float l, float m) { return l == kNegInf ? 0.0f : expf(l - m); }

// A token's softmax, computed by each wave for itself.  Lane k < K holds
// choice k: its expert (-1: absent) and its weight.
struct Choice {
  int e;
  float w;
  float m, s;  // maximum and sum of the softmax, in every lane
};

template <bool ALL>
__device__ __forceinline__ Choice choices(const float* logits, const int32_t* topk, int E, int K) {
  const int lane = threadIdx.x & 63;
  Choice c;
  c.e = lane < K ? topk[lane] : -1;
  if (c.e >= E) c.e = -1;
  const float l = c.e >= 0 ? logits[c.e] : kNegInf;
  if (l == kNegInf) c.e = -1;
  float sum = 0;
  if constexpr (ALL) {
    float m = kNegInf;
    for (int e = lane; e < E; e += 64) m = fmaxf(m, logits[e]);
    c.m = wave_max(m);
    for (int e = lane; e < E; e += 64) sum += term(logits[e], c.m);
    c.s = wave_add(sum);
  } else {
    c.m = wave_max(l);
    c.s = wave_add(term(l, c.m));
  }
  // c.s is 0 only where no logit is above -inf; a NaN in the set reaches
  // every weight through the sum
  c.w = c.e >= 0 ? term(l, c.m) / c.s : 0.0f;
  return c;
}

// One token per TPT threads (a wave, or the whole workgroup); KM >= K rows
// are held at once.  NTL, NTS: the rows are loaded, the results stored
// non-temporally.
template <int ES, int TPT, int KM, bool ALL, bool NTL, bool NTS>
__global__ __launch_bounds__(kBlock) void gate_sum_kernel(const GateArgs a, int64_t T, int E, int K,
                                                          int64_t vpr, int64_t blocks_per_rank) {
  constexpr int kTok = kBlock / TPT;
  constexpr int P = kPer<ES>;
  const int r = (int)(blockIdx.x / blocks_per_rank);
  const int64_t t = (blockIdx.x % blocks_per_rank) * kTok + (TPT == kBlock ? 0 : threadIdx.x / TPT);
  if (t >= T) return;
  const Choice c = choices<ALL>(a.logits[r] + t * E, a.topk[r] + t * K, E, K);
  const u32x4* rows = reinterpret_cast<const u32x4*>(a.rows[r]) + t * K * vpr;
  u32x4* y = reinterpret_cast<u32x4*>(a.y[r]) + t * vpr;
  float w[KM];
  bool have[KM];
#pragma unroll
  for (int k = 0; k < KM; k++) {
    w[k] = __shfl(c.w, k);
    have[k] = __builtin_amdgcn_readfirstlane(__shfl(c.e, k)) >= 0;  // uniform per wave
  }
  for (int64_t i = threadIdx.x % TPT; i < vpr; i += TPT) {
    u32x4 v[KM];
#pragma unroll
    for (int k = 0; k < KM; k++)
      if (have[k]) v[k] = dev::load16<NTL>(rows + k * vpr + i);
    float acc[P] = {};
#pragma unroll
    for (int k = 0; k < KM; k++)
      if (have[k]) {
        float f[P];
        unpack<ES>(v[k], f);
#pragma unroll
        for (int j = 0; j < P; j++) acc[j] = __builtin_fmaf(w[k], f[j], acc[j]);
      }
    dev::store16<NTS>(y + i, pack<ES>(acc));
  }
}

template <int ES, int TPT, int KM, bool ALL, bool NTS>
__global__ __launch_bounds__(kBlock) void gate_sum_bwd_kernel(const GateArgs a, int64_t T, int E,
                                                              int K, int64_t vpr,
                                                              int64_t blocks_per_rank) {
  constexpr int kTok = kBlock / TPT;
  constexpr int P = kPer<ES>;
  __shared__ float part[kBlock / 64][KM];
  const int lane = threadIdx.x & 63;
  const int r = (int)(blockIdx.x / blocks_per_rank);
  const int64_t t = (blockIdx.x % blocks_per_rank) * kTok + (TPT == kBlock ? 0 : threadIdx.x / TPT);
  if (t >= T) return;  // uniform over the threads of a token
  const float* logits = a.logits[r] + t * E;
  const Choice c = choices<ALL>(logits, a.topk[r] + t * K, E, K);
  const u32x4* rows = reinterpret_cast<const u32x4*>(a.rows[r]) + t * K * vpr;
  const u32x4* dy = reinterpret_cast<const u32x4*>(a.dy[r]) + t * vpr;
  u32x4* drows = reinterpret_cast<u32x4*>(a.drows[r]) + t * K * vpr;
  float w[KM], g[KM];
  int ex[KM];
#pragma unroll
  for (int k = 0; k < KM; k++) {
    w[k] = __shfl(c.w, k);
    ex[k] = __builtin_amdgcn_readfirstlane(__shfl(c.e, k));
    g[k] = 0.0f;
  }
  for (int64_t i = threadIdx.x % TPT; i < vpr; i += TPT) {
    const u32x4 dv = dy[i];
    u32x4 v[KM];
#pragma unroll
    for (int k = 0; k < KM; k++)
      if (ex[k] >= 0) v[k] = rows[k * vpr + i];
    float d[P];
    unpack<ES>(dv, d);
#pragma unroll
    for (int k = 0; k < KM; k++) {
      float o[P] = {};
      if (ex[k] >= 0) {
        float f[P];
        unpack<ES>(v[k], f);
#pragma unroll
        for (int j = 0; j < P; j++) {
          g[k] = __builtin_fmaf(d[j], f[j], g[k]);
          o[j] = w[k] * d[j];
        }
      }
      if (k < K) dev::store16<NTS>(drows + k * vpr + i, pack<ES>(o));
    }
  }
#pragma unroll
  for (int k = 0; k < KM; k++) g[k] = wave_add(g[k]);
  if constexpr (TPT == kBlock) {
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < KM; k++) part[threadIdx.x >> 6][k] = g[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KM; k++) {
      g[k] = 0.0f;
      for (int x = 0; x < kBlock / 64; x++) g[k] += part[x][k];
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < KM; k++)
    if (ex[k] >= 0) s = __builtin_fmaf(w[k], g[k], s);
  float* dl = a.dlogits[r] + t * E;
  for (int e = threadIdx.x % TPT; e < E; e += TPT) {
    float d = 0.0f;
#pragma unroll
    for (int k = 0; k < KM; k++)
      if (ex[k] == e) d += ALL ? w[k] * g[k] : w[k] * (g[k] - s);
    if constexpr (ALL) {
      const float l = logits[e];
      if (c.s != 0.0f && l != kNegInf) d -= term(l, c.m) / c.s * s;
    }
    dl[e] = d;
  }
}

// How a call's rows and results pass the caches.  Results that an L2 holds
// (2 MiB) are stored as usual: one token's sum takes 4.0 us so, 5.0 us with
// non-temporal stores.  Larger ones are stored non-temporally, which also
// speeds up a call with its reader behind it: the backward of 8192 tokens x 2
// rows of 512 alone 9.5 -> 7.6 us, with a norm over its result 18.7 -> 16.8 us;
// of 2 x 4096 tokens x 6 rows of 2048 82 -> 66 us.  The forward loads its rows
// non-temporally when rows and results exceed the last-level cache (8 x 4096
// tokens x 6 rows of 2048: 167 -> 155 us, 6.1 TB/s); within it that is slower
// (8192 x 2 x 512: 5.3 -> 6.7 us), and so it is for the backward at any size
// (66 -> 69 us).
struct Caching {
  bool nt_load, nt_store;
};

template <int ES, int TPT, int KM, bool ALL>
hipError_t launch_gate_as(bool bwd, const GateArgs& a, int R, int64_t T, int E, int K, int64_t vpr,
                          Caching c, hipStream_t stream) {
  constexpr int kTok = kBlock / TPT;
  const int64_t per_rank = (T + kTok - 1) / kTok;
  if (per_rank * R > kMaxGridWorkgroups) return hipErrorInvalidValue;
  const unsigned grid = (unsigned)(per_rank * R);
  if (bwd && c.nt_store)
    gate_sum_bwd_kernel<ES, TPT, KM, ALL, true><<<grid, kBlock, 0, stream>>>(a, T, E, K, vpr, per_rank);
  else if (bwd)
    gate_sum_bwd_kernel<ES, TPT, KM, ALL, false><<<grid, kBlock, 0, stream>>>(a, T, E, K, vpr, per_rank);
  else if (c.nt_load)
    gate_sum_kernel<ES, TPT, KM, ALL, true, true><<<grid, kBlock, 0, stream>>>(a, T, E, K, vpr, per_rank);
  else if (c.nt_store)
    gate_sum_kernel<ES, TPT, KM, ALL, false, true><<<grid, kBlock, 0, stream>>>(a, T, E, K, vpr, per_rank);
  else
    gate_sum_kernel<ES, TPT, KM, ALL, false, false><<<grid, kBlock, 0, stream>>>(a, T, E, K, vpr, per_rank);
  return hipGetLastError();
}

template <int ES, int TPT, bool ALL>
hipError_t launch_gate_k(bool bwd, const GateArgs& a, int R, int64_t T, int E, int K, int64_t vpr,
                         Caching c, hipStream_t stream) {
  if (K <= 2) return launch_gate_as<ES, TPT, 2, ALL>(bwd, a, R, T, E, K, vpr, c, stream);
  if (K <= 4) return launch_gate_as<ES, TPT, 4, ALL>(bwd, a, R, T, E, K, vpr, c, stream);
  if (K <= 8) return launch_gate_as<ES, TPT, 8, ALL>(bwd, a, R, T, E, K, vpr, c, stream);
  return launch_gate_as<ES, TPT, 16, ALL>(bwd, a, R, T, E, K, vpr, c, stream);
}

// A row of up to 64 vectors takes one wave, a longer one the workgroup.
template <int ES, bool ALL>
hipError_t launch_gate_t(bool bwd, const GateArgs& a, int R, int64_t T, int E, int K, int64_t vpr,
                         Caching c, hipStream_t stream) {
  return vpr <= 64 ? launch_gate_k<ES, 64, ALL>(bwd, a, R, T, E, K, vpr, c, stream)
                   : launch_gate_k<ES, kBlock, ALL>(bwd, a, R, T, E, K, vpr, c, stream);
}

}  // namespace

hipError_t launch_gate_sum(bool bwd, bool over_all, int es, const GateArgs& a, int R, int64_t T,
                           int E, int K, int64_t row_bytes, bool large, hipStream_t stream) {
  if (R <= 0 || T <= 0) return hipSuccess;
  const int64_t vpr = row_bytes >> 4, result = R * T * row_bytes * (bwd ? K : 1);
  const bool nt_store = large || result > (int64_t(2) << 20);
  const Caching c{large && !bwd, nt_store};
  if (es == 4)
    return over_all ? launch_gate_t<4, true>(bwd, a, R, T, E, K, vpr, c, stream)
                    : launch_gate_t<4, false>(bwd, a, R, T, E, K, vpr, c, stream);
  return over_all ? launch_gate_t<2, true>(bwd, a, R, T, E, K, vpr, c, stream)
                  : launch_gate_t<2, false>(bwd, a, R, T, E, K, vpr, c, stream);
}

}  // namespace ccr
