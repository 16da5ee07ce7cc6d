// Device kernels of the router in front of an expert-parallel exchange, and of
// its gradient, written for gfx950 (CDNA4: wave64, 256 CUs in 8 XCDs).
//
// Per token, over its E logits l:
//
//   s      = softmax(l), or 1 / (1 + exp(-l)) each
//   key    = s + bias (no bias: the logits order the experts, s grows with l)
//   groups of E / G experts: their value is the sum of their one or two largest
//            keys; the experts of the best groups stay
//   topk   = the K largest keys, equal ones by expert
//   w_k    = s_k, over the sum of the chosen ones if renormalised, times a scale
//
// Choices are those of 64-bit arithmetic, so that they do not hang on a
// rounding: keys are computed in fp32, and where two that decide lie nearer to
// each other than their error bound, the wave's tokens are chosen again in fp64
// (one token in some hundred).  Keys are compared as unsigned numbers in the
// order of the values, NaN above all (it reaches the weights), 0 for an expert
// that cannot be chosen.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccr_device.h"
#include "ccr_internal.h"

namespace ccr {
namespace {

constexpr float kNegInf = -__builtin_inff();

// Over the LPT neighbouring lanes that share a token (16: a row of the wave's
// lanes, by its own exchanges; 64: the wave).
template <int LPT, typename T, typename F>
__device__ __forceinline__ T reduce(T x, F&& f) {
#pragma unroll
  for (int off = 1; off < LPT; off <<= 1) x = f(x, __shfl_xor(x, off));
  return x;
}
template <int LPT, typename T>
__device__ __forceinline__ T sum_of(T x) {
  return reduce<LPT>(x, [](T a, T b) { return a + b; });
}
template <int LPT, typename T>
__device__ __forceinline__ T max_of(T x) {
  return reduce<LPT>(x, [](T a, T b) { return a > b ? a : b; });
}

// Keys in the order of their values: larger numbers for larger values, NaN
// largest; never 0.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);  // -0 is 0
  return x != x ? 0xffffffffu : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x + 0.0);
  return x != x ? ~0ull : b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// 1 / (1 + exp(-l)) without overflow, and its complement.
template <typename T>
struct Sigmoid {
  T s, rest;
};
__device__ __forceinline__ Sigmoid<float> sigmoid(float l) {
  const float t = expf(-fabsf(l)), q = 1.0f / (1.0f + t);
  return l >= 0 ? Sigmoid<float>{q, t * q} : Sigmoid<float>{t * q, q};
}
__device__ __forceinline__ Sigmoid<double> sigmoid(double l) {
  const double t = exp(-fabs(l)), q = 1.0 / (1.0 + t);
  return l >= 0 ? Sigmoid<double>{q, t * q} : Sigmoid<double>{t * q, q};
}
__device__ __forceinline__ float exponential(float x) { return expf(x); }
__device__ __forceinline__ double exponential(double x) { return exp(x); }

// The scores of a lane's J experts; l: the logits, -inf where there is none.
template <int LPT, int J, typename T>
__device__ __forceinline__ void scores(const float* l, bool sig, T* s) {
  if (sig) {
#pragma unroll
    for (int j = 0; j < J; j++) s[j] = sigmoid((T)l[j]).s;
    return;
  }
  float m = kNegInf;
#pragma unroll
  for (int j = 0; j < J; j++) m = fmaxf(m, l[j]);
  m = max_of<LPT>(m);
  T sum = 0;
#pragma unroll
  for (int j = 0; j < J; j++) {
    s[j] = l[j] == kNegInf ? T(0) : exponential((T)l[j] - (T)m);
    sum += s[j];
  }
  sum = sum_of<LPT>(sum);
  const T inv = sum == T(0) ? T(0) : T(1) / sum;
#pragma unroll
  for (int j = 0; j < J; j++) s[j] *= inv;
}

// What the wave's lanes wrote to LDS before is there for all of them after.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Where a wave's tokens keep keys and group values while groups are chosen.
template <int LPT, int J>
struct GroupRoom {
  static constexpr int kTok = 64 / LPT;
  double key[kTok][LPT * J];
  double value[kTok][kRouteGroups];
  uint8_t keep[kTok][kRouteGroups];
};

struct Chosen {
  int32_t id;
  float s;
};

// One round of choosing for the wave's tokens; T: the arithmetic of the keys.
// Lane k of a token ends with its k-th choice (id -1: none left).  Returns
// whether any decision of the lane's token was nearer than `tol` (T = float).
template <int LPT, int J, bool GROUPS, typename T>
__device__ __forceinline__ bool choose(const float* l, const float* s32, const float* bias, bool with_bias,
                                       const RouteShape& n, GroupRoom<LPT, J>* room, Chosen (*out)[16],
                                       bool* taken) {
  using U = decltype(ordered(T(0)));
  constexpr bool kExact = sizeof(T) == 8;
  const int sub = threadIdx.x % LPT, tok = (threadIdx.x & 63) / LPT;
  const uint64_t mine = (LPT == 64 ? ~0ull : ((1ull << (LPT & 63)) - 1)) << (tok * LPT);
  T s[J];
  const bool need = with_bias || (GROUPS && n.group_top == 2);
  if constexpr (kExact) {
    if (need) scores<LPT, J, T>(l, n.sigmoid, s);
  } else {
#pragma unroll
    for (int j = 0; j < J; j++) s[j] = s32[j];
  }
  T v[J];
#pragma unroll
  for (int j = 0; j < J; j++) v[j] = with_bias ? s[j] + (T)bias[j] : (T)l[j];
  // fp32 scores are off by up to 2^-21 (sigmoid) or 2^-20 (softmax) of the
  // largest one, the sum with the bias by 2^-24 of itself
  float top = 1.0f;
  if (!kExact && !n.sigmoid) {
    top = 0;
#pragma unroll
    for (int j = 0; j < J; j++) top = fmaxf(top, s32[j]);
    top = max_of<LPT>(top);
  }
  const float err = n.sigmoid ? 0x1p-21f : 0x1p-20f * top;
  bool near = false;
  U key[J];
#pragma unroll
  for (int j = 0; j < J; j++) key[j] = l[j] == kNegInf ? U(0) : ordered(v[j]);
  if constexpr (GROUPS) {
    // a group's value: of one key that key, of two their sum (of scores, where
    // the keys are logits); a group's masked experts add nothing
    const bool real = n.group_top == 2 && !with_bias;
#pragma unroll
    for (int j = 0; j < J; j++) {
      const int e = sub * J + j;
      if (e < n.E) room->key[tok][e] = l[j] == kNegInf ? (double)kNegInf : (double)(real ? s[j] : v[j]);
    }
    wave_sync();
    const int eg = n.E / n.groups;
    for (int g = sub; g < n.groups; g += LPT) {
      double a = kNegInf, b = kNegInf;
      bool nan = false;
      for (int i = 0; i < eg; i++) {
        const double x = room->key[tok][g * eg + i];
        nan |= x != x;
        if (x > a) {
          b = a;
          a = x;
        } else if (x > b) {
          b = x;
        }
      }
      double y = a;
      if (n.group_top == 2 && b != (double)kNegInf) y = kExact ? a + b : (double)((float)a + (float)b);
      room->value[tok][g] = nan ? __builtin_nan("") : y;
    }
    wave_sync();
    double low = __builtin_inf(), high = kNegInf;  // the worst kept value, the best other one
    for (int g = sub; g < n.groups; g += LPT) {
      const double y = room->value[tok][g];
      const uint64_t o = ordered(y);
      int rank = 0;
      for (int i = 0; i < n.groups; i++) {
        const uint64_t p = ordered(room->value[tok][i]);
        rank += p > o || (p == o && i < g);
      }
      const bool keep = rank < n.kept;
      room->keep[tok][g] = keep;
      if (keep && y < low) low = y;
      if (!keep && y > high) high = y;
    }
    wave_sync();
    if (!kExact && need && n.kept < n.groups) {
      low = reduce<LPT>(low, [](double a, double b) { return a < b ? a : b; });
      high = max_of<LPT>(high);
      near |= !(low - high > 4 * (double)err + 0x1p-21 * (fabs(low) + fabs(high)));
    }
#pragma unroll
    for (int j = 0; j < J; j++) {
      const int e = sub * J + j;
      if (e < n.E && !room->keep[tok][e / eg]) key[j] = 0;
    }
  }
#pragma unroll
  for (int j = 0; j < J; j++) taken[j] = false;
  U before = 0;
  const bool check = !kExact && with_bias;
  const int rounds = n.K + (check ? 1 : 0);  // one more for the key that just missed
  for (int k = 0; k < rounds; k++) {
    U m = 0;
#pragma unroll
    for (int j = 0; j < J; j++) m = key[j] > m ? key[j] : m;
    const U best = max_of<LPT>(m);
    if (check && k > 0 && best != 0) {
      const float a = value_of((uint32_t)before), b = value_of((uint32_t)best);
      near |= !(a - b > 2 * err + 0x1p-23f * (fabsf(a) + fabsf(b)));
    }
    before = best;
    if (k == n.K) break;
    const uint64_t who = __ballot(m == best && best != 0) & mine;
    if (who == 0) {
      if (sub == 0) out[tok][k] = Chosen{-1, 0.0f};
    } else if (__ffsll((unsigned long long)who) - 1 == (int)(threadIdx.x & 63)) {
      bool open = true;
#pragma unroll
      for (int j = 0; j < J; j++)
        if (open && key[j] == best) {
          open = false;
          key[j] = 0;
          taken[j] = true;
          out[tok][k] = Chosen{sub * J + j, s32[j]};
        }
    }
  }
  wave_sync();
  return near;
}

// A token per LPT lanes, J neighbouring experts to a lane; a workgroup takes
// every slots-th step of its rank's tokens.  STATS: it counts its tokens'
// choices and sums their scores, in its slot of the work array or, alone, in
// the results.
template <int LPT, int J, bool GROUPS, bool STATS>
__global__ __launch_bounds__(kBlock) void route_kernel(const RouteArgs a, const RouteShape n, int slots,
                                                       float* work) {
  constexpr int kTok = 64 / LPT, kWaves = kBlock / 64;
  __shared__ Chosen chosen[kWaves][kTok][16];
  __shared__ GroupRoom<GROUPS ? LPT : 64, GROUPS ? J : 1> rooms[GROUPS ? kWaves : 1];
  __shared__ float sum_part[STATS ? kWaves * kTok : 1][STATS ? LPT * J : 1];
  __shared__ int count_part[STATS ? kWaves * kTok : 1][STATS ? LPT * J : 1];
  const int rank = blockIdx.x / slots, slot = blockIdx.x % slots;
  const int wave = threadIdx.x >> 6, sub = threadIdx.x % LPT, tok = (threadIdx.x & 63) / LPT;
  const float* logits = a.logits[rank];
  const bool with_bias = a.bias[rank] != nullptr;
  float bias[J], sums[J];
  int counts[J];
#pragma unroll
  for (int j = 0; j < J; j++) {
    const int e = sub * J + j;
    bias[j] = with_bias && e < n.E ? a.bias[rank][e] : 0.0f;
    sums[j] = 0;
    counts[j] = 0;
  }
  for (int64_t t0 = ((int64_t)slot * kWaves + wave) * kTok; t0 < n.T; t0 += (int64_t)slots * kWaves * kTok) {
    const int64_t t = t0 + tok;
    const bool live = t < n.T;
    float l[J], s[J];
#pragma unroll
    for (int j = 0; j < J; j++) {
      const int e = sub * J + j;
      l[j] = live && e < n.E ? logits[t * n.E + e] : kNegInf;
    }
    scores<LPT, J, float>(l, n.sigmoid, s);
    bool taken[J];
    auto* room = reinterpret_cast<GroupRoom<LPT, J>*>(&rooms[GROUPS ? wave : 0]);
    const bool near = choose<LPT, J, GROUPS, float>(l, s, bias, with_bias, n, room, chosen[wave], taken);
    if (__ballot(near && live))
      choose<LPT, J, GROUPS, double>(l, s, bias, with_bias, n, room, chosen[wave], taken);
    Chosen c = sub < n.K ? chosen[wave][tok][sub & 15] : Chosen{-1, 0.0f};
    const float total = sum_of<LPT>(c.s);
    float w = c.s;
    if (n.renorm) w = total == 0.0f ? 0.0f : w / total;
    if (live && sub < n.K) {
      a.topk[rank][t * n.K + sub] = c.id;
      a.weights[rank][t * n.K + sub] = w * n.scale;
    }
    wave_sync();
    if constexpr (STATS) {
#pragma unroll
      for (int j = 0; j < J; j++)
        if (live && sub * J + j < n.E) {
          sums[j] += l[j] == kNegInf ? 0.0f : s[j];
          counts[j] += taken[j];
        }
    }
  }
  if constexpr (STATS) {
#pragma unroll
    for (int j = 0; j < J; j++) {
      sum_part[wave * kTok + tok][sub * J + j] = sums[j];
      count_part[wave * kTok + tok][sub * J + j] = counts[j];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n.E; e += kBlock) {
      float s = 0;
      int c = 0;
#pragma unroll
      for (int k = 0; k < kWaves * kTok; k++) {
        s += sum_part[k][e];
        c += count_part[k][e];
      }
      if (slots == 1) {
        if (a.sums[rank]) a.sums[rank][e] = s;
        if (a.counts[rank]) a.counts[rank][e] = c;
      } else {
        float* out = work + (int64_t)blockIdx.x * 2 * n.E;
        out[e] = s;
        reinterpret_cast<int*>(out)[n.E + e] = c;
      }
    }
  }
}

// The slots' counts and sums, in the slots' order: a workgroup takes 64 experts,
// a wave of it every fourth slot.
__global__ __launch_bounds__(kBlock) void route_stats_kernel(const RouteArgs a, const float* work, int slots, int E) {
  __shared__ double sum_part[kBlock / 64][64];
  __shared__ int64_t count_part[kBlock / 64][64];
  const int rank = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  const float* from = work + (int64_t)rank * slots * 2 * E;
  double s = 0;
  int64_t c = 0;
  if (e < E)
    for (int k = wave; k < slots; k += kBlock / 64) {
      s += (double)from[(int64_t)k * 2 * E + e];
      c += reinterpret_cast<const int*>(from)[((int64_t)k * 2 + 1) * E + e];
    }
  sum_part[wave][lane] = s;
  count_part[wave][lane] = c;
  __syncthreads();
  if (wave == 0 && e < E) {
#pragma unroll
    for (int k = 1; k < kBlock / 64; k++) {
      s += sum_part[k][lane];
      c += count_part[k][lane];
    }
    if (a.sums[rank]) a.sums[rank][e] = (float)s;
    if (a.counts[rank]) a.counts[rank][e] = c;
  }
}

// ---------------------------------------------------------------- backward
// With c_k the chosen scores and u_k = scale dw_k, the gradient of the scores
// is, at the k-th choice, u_k, or renormalised (u_k - sum u c / C) / C with
// C = sum c; at every expert, that of the sums of scores; and that of the logits
// s (ds - sum s ds) for a softmax, s (1 - s) ds for sigmoids.
template <int LPT, int J>
__global__ __launch_bounds__(kBlock) void route_bwd_kernel(const RouteBwdArgs a, const RouteShape n,
                                                           int64_t blocks_per_rank) {
  constexpr int kTok = 64 / LPT, kWaves = kBlock / 64;
  __shared__ Chosen back[kWaves][kTok][16];
  const int rank = (int)(blockIdx.x / blocks_per_rank);
  const int wave = threadIdx.x >> 6, sub = threadIdx.x % LPT, tok = (threadIdx.x & 63) / LPT;
  const int64_t t = ((int64_t)(blockIdx.x % blocks_per_rank) * kWaves + wave) * kTok + tok;
  const bool live = t < n.T;
  const float* logits = a.logits[rank] + (live ? t : 0) * n.E;
  float l[J], s[J], ds[J];
#pragma unroll
  for (int j = 0; j < J; j++) {
    const int e = sub * J + j;
    l[j] = live && e < n.E ? logits[e] : kNegInf;
  }
  float m = 0, inv = 0;
  if (!n.sigmoid) {
    m = kNegInf;
#pragma unroll
    for (int j = 0; j < J; j++) m = fmaxf(m, l[j]);
    m = max_of<LPT>(m);
    float sum = 0;
#pragma unroll
    for (int j = 0; j < J; j++) {
      s[j] = l[j] == kNegInf ? 0.0f : expf(l[j] - m);
      sum += s[j];
    }
    sum = sum_of<LPT>(sum);
    inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int j = 0; j < J; j++) s[j] *= inv;
  }
  // lane k < K: the k-th choice and its score
  int id = -1;
  float c = 0, u = 0;
  if (live && sub < n.K) {
    id = a.topk[rank][t * n.K + sub];
    if (id < 0 || id >= n.E) id = -1;
    const float lk = id >= 0 ? logits[id] : kNegInf;
    if (lk == kNegInf) id = -1;
    if (id >= 0) {
      c = n.sigmoid ? sigmoid(lk).s : expf(lk - m) * inv;
      u = a.dweights[rank][t * n.K + sub] * n.scale;
    }
  }
  if (n.renorm) {
    const float total = sum_of<LPT>(c), dot = sum_of<LPT>(u * c);
    u = id < 0 || total == 0.0f ? 0.0f : (u - dot / total) / total;
  }
  if (sub < 16) back[wave][tok][sub] = Chosen{id, u};
  wave_sync();
  const float* dsums = a.dsums[rank];
#pragma unroll
  for (int j = 0; j < J; j++) {
    const int e = sub * J + j;
    ds[j] = dsums && e < n.E ? dsums[e] : 0.0f;
  }
  for (int k = 0; k < n.K; k++) {
    const Chosen b = back[wave][tok][k];
#pragma unroll
    for (int j = 0; j < J; j++) ds[j] += b.id == sub * J + j ? b.s : 0.0f;
  }
  float dot = 0;
  if (!n.sigmoid) {
#pragma unroll
    for (int j = 0; j < J; j++) dot = __builtin_fmaf(s[j], ds[j], dot);
    dot = sum_of<LPT>(dot);
  }
#pragma unroll
  for (int j = 0; j < J; j++) {
    const int e = sub * J + j;
    float d;
    if (n.sigmoid) {
      const Sigmoid<float> x = sigmoid(l[j]);
      d = x.s * x.rest * ds[j];
    } else {
      d = s[j] * (ds[j] - dot);
    }
    if (live && e < n.E) a.dlogits[rank][t * n.E + e] = l[j] == kNegInf ? 0.0f : d;
  }
}

hipError_t launch_stats(const RouteArgs& a, const RouteShape& n, const float* work, int slots, hipStream_t stream) {
  route_stats_kernel<<<dim3((unsigned)((n.E + 63) / 64), (unsigned)n.R), kBlock, 0, stream>>>(a, work, slots, n.E);
  return hipGetLastError();
}

template <int LPT, int J>
hipError_t launch_route_as(const RouteArgs& a, const RouteShape& n, bool stats, float* work, hipStream_t stream) {
  const int slots = route_slots(n.R, n.T);
  const unsigned grid = (unsigned)(slots * n.R);
  const bool groups = n.kept < n.groups;
  if (groups && stats) route_kernel<LPT, J, true, true><<<grid, kBlock, 0, stream>>>(a, n, slots, work);
  else if (groups) route_kernel<LPT, J, true, false><<<grid, kBlock, 0, stream>>>(a, n, slots, work);
  else if (stats) route_kernel<LPT, J, false, true><<<grid, kBlock, 0, stream>>>(a, n, slots, work);
  else route_kernel<LPT, J, false, false><<<grid, kBlock, 0, stream>>>(a, n, slots, work);
  hipError_t e = hipGetLastError();
  return e != hipSuccess || !stats || slots == 1 ? e : launch_stats(a, n, work, slots, stream);
}

template <int LPT, int J>
hipError_t launch_route_bwd_as(const RouteBwdArgs& a, const RouteShape& n, hipStream_t stream) {
  constexpr int kTokens = kBlock / LPT;
  const int64_t per_rank = (n.T + kTokens - 1) / kTokens;
  if (per_rank * n.R > kMaxGridWorkgroups) return hipErrorInvalidValue;
  route_bwd_kernel<LPT, J><<<(unsigned)(per_rank * n.R), kBlock, 0, stream>>>(a, n, per_rank);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, const RouteShape& n, float* work, hipStream_t stream) {
  bool stats = false;
  for (int r = 0; r < n.R; r++) stats |= a.counts[r] || a.sums[r];
  if (n.T <= 0) return stats ? launch_stats(a, n, work, 0, stream) : hipSuccess;  // no slot: zeros
  if (n.E <= 64) return launch_route_as<16, 4>(a, n, stats, work, stream);
  if (n.E <= 256) return launch_route_as<16, 16>(a, n, stats, work, stream);
  return launch_route_as<64, 16>(a, n, stats, work, stream);
}

hipError_t launch_route_bwd(const RouteBwdArgs& a, const RouteShape& n, hipStream_t stream) {
  if (n.T <= 0) return hipSuccess;
  if (n.E <= 64) return launch_route_bwd_as<16, 4>(a, n, stream);
  if (n.E <= 256) return launch_route_bwd_as<16, 16>(a, n, stream);
  return launch_route_bwd_as<64, 16>(a, n, stream);
}

}  // namespace ccr
