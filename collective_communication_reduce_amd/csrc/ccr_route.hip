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

// Over the LPT neighbouring lanes that share a token, every lane's own result.
// Within a row of 16 lanes the exchanges are operands of the operation (quads,
// then halves and the row mirrored: after each step the lanes below it agree, so
// a mirror image is as good as any other lane of the other half).  As LDS
// permutes the router of 256 experts took twice as long.
template <int CTRL, typename T>
__device__ __forceinline__ T across(T x) {
  return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
template <int N, typename T, typename F>
__device__ __forceinline__ T reduce(T x, F&& f) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (N > 1) x = f(x, across<0xb1>(x));
    if constexpr (N > 2) x = f(x, across<0x4e>(x));
    if constexpr (N > 4) x = f(x, across<0x141>(x));
    if constexpr (N > 8) x = f(x, across<0x140>(x));
    if constexpr (N > 16) x = f(x, __shfl_xor(x, 16));
    if constexpr (N > 32) x = f(x, __shfl_xor(x, 32));
  } else {
#pragma unroll
    for (int off = 1; off < N; off <<= 1) x = f(x, __shfl_xor(x, off));
  }
  return x;
}
template <int N, typename T>
__device__ __forceinline__ T sum_of(T x) {
  return reduce<N>(x, [](T a, T b) { return a + b; });
}
template <int N, typename T>
__device__ __forceinline__ T max_of(T x) {
  return reduce<N>(x, [](T a, T b) { return a > b ? a : b; });
}
template <int N, typename T>
__device__ __forceinline__ T min_of(T x) {
  return reduce<N>(x, [](T a, T b) { return a < b ? a : b; });
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

constexpr uint32_t kNone = 0xffffffffu;  // no choice

// Where the experts of a token lie: group g's on the lanes g q .. g q + q - 1, J
// neighbours to a lane (without groups, one group on all lanes).  A lane's place
// is where it would be if every lane held J.
struct Layout {
  int eg, q;  // experts of a group, lanes of a group (a power of two)
};

// J values from p, the first n of them (the others: none).  Rows of logits need
// not be aligned to more than a value.
template <int J>
__device__ __forceinline__ void load_some(const float* p, int n, float none, float* v) {
  struct Four {
    float f[4];
  };
  if (n >= J) {
#pragma unroll
    for (int j = 0; j < J; j += 4) {
      Four x;
      __builtin_memcpy(&x, p + j, 16);
#pragma unroll
      for (int i = 0; i < 4; i++) v[j + i] = x.f[i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < J; j++) v[j] = j < n ? p[j] : none;
  }
}

// ------------------------------------------------------------ 64 bits, exactly
// One token's choice by a whole wave, keys in fp64.
template <int E>
struct ExactRoom {
  double key[E];
  double value[kRouteGroups];
  uint8_t keep[kRouteGroups];
};

template <int J, bool GROUPS>
__device__ __forceinline__ void choose_exactly(const float* logits, const float* bias, const RouteShape& n,
                                            ExactRoom<GROUPS ? 64 * J : 1>* room, const Layout at, int J32,
                                            uint32_t* out) {
  const int lane = threadIdx.x & 63;
  const bool real = GROUPS && n.group_top == 2;  // values, not only their order, count
  float l[J];
  double s[J], v[J];
#pragma unroll
  for (int j = 0; j < J; j++) l[j] = lane * J + j < n.E ? logits[lane * J + j] : kNegInf;
  if (bias || real) scores<64, J, double>(l, n.sigmoid, s);
  uint64_t key[J];
#pragma unroll
  for (int j = 0; j < J; j++) {
    v[j] = bias && lane * J + j < n.E ? s[j] + (double)bias[lane * J + j] : (double)l[j];
    key[j] = l[j] == kNegInf ? 0 : ordered(v[j]);
  }
  if constexpr (GROUPS) {
    // a group's value: of one key that key, of two their sum (of scores, where
    // the keys are logits); a group's masked experts add nothing
#pragma unroll
    for (int j = 0; j < J; j++)
      if (lane * J + j < n.E)
        room->key[lane * J + j] = l[j] == kNegInf ? (double)kNegInf : real && !bias ? s[j] : v[j];
    wave_sync();
    if (lane < n.groups) {
      const int eg = n.E / n.groups;
      double a = kNegInf, b = kNegInf;
      bool nan = false;
      for (int i = 0; i < eg; i++) {
        const double x = room->key[lane * eg + i];
        nan |= x != x;
        if (x > a) {
          b = a;
          a = x;
        } else if (x > b) {
          b = x;
        }
      }
      room->value[lane] = nan ? __builtin_nan("") : n.group_top == 2 && b != (double)kNegInf ? a + b : a;
    }
    wave_sync();
    if (lane < n.groups) {
      const uint64_t o = ordered(room->value[lane]);
      int rank = 0;
      for (int i = 0; i < n.groups; i++) {
        const uint64_t p = ordered(room->value[i]);
        rank += p > o || (p == o && i < lane);
      }
      room->keep[lane] = rank < n.kept;
    }
    wave_sync();
#pragma unroll
    for (int j = 0; j < J; j++)
      if (lane * J + j < n.E && !room->keep[(lane * J + j) / (n.E / n.groups)]) key[j] = 0;
  }
  for (int k = 0; k < n.K; k++) {
    uint64_t m = 0;
#pragma unroll
    for (int j = 0; j < J; j++) m = key[j] > m ? key[j] : m;
    const uint64_t best = max_of<64>(m);
    const uint64_t who = __ballot(m == best);
    if (best == 0) {
      if (lane == 0) out[k] = kNone;
    } else if (__ffsll((unsigned long long)who) - 1 == lane) {
      bool open = true;
#pragma unroll
      for (int j = 0; j < J; j++)
        if (open && key[j] == best) {
          open = false;
          key[j] = 0;
          const int e = lane * J + j, g = e / at.eg, i = e - g * at.eg;
          out[k] = (uint32_t)((g * at.q + i / J32) * J32 + i % J32) << 16 | (uint32_t)e;
        }
    }
  }
  wave_sync();
}

// ------------------------------------------------------------------ 32 bits
// The wave's tokens' choices; l, s, bias: those of this lane's J experts, of
// which e0 is the first.  Choice k of a token goes to out[tok][k], place and
// expert.  Returns whether a decision of this lane's token was too near to make.
template <int LPT, int J, bool GROUPS>
__device__ __forceinline__ bool choose(const float* l, const float* s, const float* bias, bool with_bias, int e0,
                                       const RouteShape& n, int q, uint32_t (*out)[16]) {
  const int sub = threadIdx.x % LPT, tok = (threadIdx.x & 63) / LPT;
  uint32_t key[J];
#pragma unroll
  for (int j = 0; j < J; j++) key[j] = l[j] == kNegInf ? 0 : ordered(with_bias ? s[j] + bias[j] : l[j]);
  // fp32 scores are off by up to 2^-21 (sigmoid) or 2^-20 (softmax) of the
  // largest one, the sum with the bias by 2^-24 of itself
  float err = 0x1p-21f;
  if (!n.sigmoid && (with_bias || (GROUPS && n.group_top == 2))) {
    float top = 0;
#pragma unroll
    for (int j = 0; j < J; j++) top = fmaxf(top, s[j]);
    err = 0x1p-20f * max_of<LPT>(top);
  }
  bool near = false;
  if constexpr (GROUPS) {
    // the two largest keys (scores, where the keys are logits) of the group
    const bool of_scores = n.group_top == 2 && !with_bias;
    uint32_t a = 0, b = 0;
    auto merge = [&](uint32_t c, uint32_t d) {  // c >= d
      b = max(min(a, c), max(b, d));
      a = max(a, c);
    };
#pragma unroll
    for (int j = 0; j < J; j++) merge(of_scores && key[j] ? ordered(s[j]) : key[j], 0);
    if (q > 1) merge(across<0xb1>(a), across<0xb1>(b));
    if (q > 2) merge(across<0x4e>(a), across<0x4e>(b));
    if (q > 4) merge(across<0x141>(a), across<0x141>(b));
    if (q > 8) merge(across<0x140>(a), across<0x140>(b));
    if constexpr (LPT == 64) {
      if (q > 16) merge(__shfl_xor(a, 16), __shfl_xor(b, 16));
    }
    if (n.group_top == 2 && b != 0) a = ordered(value_of(a) + value_of(b));
    const int g = sub / q;
    if (g >= n.groups) a = 0;
    int rank = 0;
    const int first = threadIdx.x & 63 & ~(LPT - 1);
    for (int i = 0; i < n.groups; i++) {
      const uint32_t o = __shfl(a, first + i * q);
      rank += o > a || (o == a && i < g);
    }
    const bool keep = rank < n.kept && g < n.groups;
    if (with_bias || n.group_top == 2) {
      const uint32_t low = min_of<LPT>(keep ? a : ~0u), high = max_of<LPT>(keep ? 0u : a);
      const float x = value_of(low), y = value_of(high);
      near |= high != 0 && !(x - y > 4 * err + 0x1p-21f * (fabsf(x) + fabsf(y)));
    }
    if (!keep) {
#pragma unroll
      for (int j = 0; j < J; j++) key[j] = 0;
    }
  }
  uint32_t before = 0;
  const int rounds = n.K + (with_bias ? 1 : 0);  // one more for the key that just missed
  for (int k = 0; k < rounds; k++) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < J; j++) m = max(m, key[j]);
    const uint32_t best = max_of<LPT>(m);
    if (with_bias && k > 0 && best != 0) {
      const float x = value_of(before), y = value_of(best);
      near |= !(x - y > 2 * err + 0x1p-23f * (fabsf(x) + fabsf(y)));
    }
    before = best;
    if (k == n.K) break;
    const int winner = min_of<LPT>(m == best ? sub : LPT);  // the lowest lane that has it
    bool open = winner == sub && best != 0;
    int at = 0;
#pragma unroll
    for (int j = 0; j < J; j++) {
      const bool hit = open && key[j] == best;
      key[j] = hit ? 0 : key[j];
      at = hit ? j : at;
      open = open && !hit;
    }
    if (winner == sub) out[tok][k] = best == 0 ? kNone : (uint32_t)(sub * J + at) << 16 | (uint32_t)(e0 + at);
  }
  wave_sync();
  return near;
}

// A token per LPT lanes, J experts to a lane; a workgroup takes every slots-th
// step of its rank's tokens.  STATS: it counts its tokens' choices and sums their
// scores, in its slot of the work array or, alone, in the results.
template <int LPT, int J, bool GROUPS, bool STATS>
__global__ __launch_bounds__(kBlock) void route_kernel(const RouteArgs a, const RouteShape n, const Layout at,
                                                       bool exact, int slots, float* work) {
  constexpr int kTok = 64 / LPT, kWaves = kBlock / 64, kPlaces = LPT * J;
  constexpr int kExactJ = (kPlaces + 63) / 64;
  __shared__ uint32_t chosen[kWaves][kTok][16];
  __shared__ __align__(16) float score[kWaves][kTok][kPlaces];
  __shared__ ExactRoom<GROUPS ? 64 * kExactJ : 1> rooms[GROUPS ? kWaves : 1];
  __shared__ int count[STATS ? kPlaces : 1];
  const int rank = blockIdx.x / slots, slot = blockIdx.x % slots;
  const int wave = threadIdx.x >> 6, sub = threadIdx.x % LPT, tok = (threadIdx.x & 63) / LPT;
  const float* logits = a.logits[rank];
  const bool with_bias = a.bias[rank] != nullptr;
  const int g = sub / at.q, i0 = sub % at.q * J, e0 = g * at.eg + i0;
  const int mine = g * at.eg < n.E ? max(0, min(J, at.eg - i0)) : 0;
  float bias[J], sums[J];
  if (with_bias) load_some<J>(a.bias[rank] + (mine > 0 ? e0 : 0), mine, 0.0f, bias);
  if constexpr (STATS) {
#pragma unroll
    for (int j = 0; j < J; j++) sums[j] = 0;
    for (int e = threadIdx.x; e < kPlaces; e += kBlock) count[e] = 0;
    __syncthreads();
  }
  for (int64_t t0 = ((int64_t)slot * kWaves + wave) * kTok; t0 < n.T; t0 += (int64_t)slots * kWaves * kTok) {
    const int64_t t = t0 + tok;
    const bool live = t < n.T;
    float l[J], s[J];
    load_some<J>(logits + (live && mine > 0 ? t * n.E + e0 : 0), live ? mine : 0, kNegInf, l);
    scores<LPT, J, float>(l, n.sigmoid, s);
#pragma unroll
    for (int j = 0; j < J; j += 4)
      *reinterpret_cast<dev::f32x4*>(&score[wave][tok][sub * J + j]) = dev::f32x4{s[j], s[j + 1], s[j + 2], s[j + 3]};
    if constexpr (STATS) {
#pragma unroll
      for (int j = 0; j < J; j++) sums[j] += l[j] == kNegInf ? 0.0f : s[j];
    }
    bool near = exact;
    if (!exact) near = choose<LPT, J, GROUPS>(l, s, bias, with_bias, e0, n, at.q, chosen[wave]);
    for (uint64_t todo = __ballot(near && live && sub == 0); todo; todo &= todo - 1) {
      const int k = (__ffsll((unsigned long long)todo) - 1) / LPT;
      choose_exactly<kExactJ, GROUPS>(logits + (t0 + k) * n.E, a.bias[rank], n, &rooms[GROUPS ? wave : 0], at, J,
                                      chosen[wave][k]);
    }
    wave_sync();
    const uint32_t c = live && sub < n.K ? chosen[wave][tok][sub & 15] : kNone;
    float w = c != kNone ? score[wave][tok][c >> 16] : 0.0f;
    if (n.renorm) {
      const float total = sum_of<LPT>(w);
      w = total == 0.0f ? 0.0f : w / total;
    }
    if (live && sub < n.K) {
      a.topk[rank][t * n.K + sub] = c != kNone ? (int)(c & 0xffff) : -1;
      a.weights[rank][t * n.K + sub] = w * n.scale;
    }
    if constexpr (STATS) {
      if (c != kNone) atomicAdd(&count[c >> 16], 1);  // whole numbers: the order does not show
    }
    wave_sync();
  }
  if constexpr (STATS) {
#pragma unroll
    for (int j = 0; j < J; j++) score[wave][tok][sub * J + j] = sums[j];
    __syncthreads();
    for (int e = threadIdx.x; e < n.E; e += kBlock) {
      const int eg = e / at.eg, i = e - eg * at.eg, p = (eg * at.q + i / J) * J + i % J;
      float s = 0;
#pragma unroll
      for (int k = 0; k < kWaves * kTok; k++) s += score[k / kTok][k % kTok][p];
      if (slots == 1) {
        if (a.sums[rank]) a.sums[rank][e] = s;
        if (a.counts[rank]) a.counts[rank][e] = count[p];
      } else {
        float* out = work + (int64_t)blockIdx.x * 2 * n.E;
        out[e] = s;
        reinterpret_cast<int*>(out)[n.E + e] = count[p];
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
  struct Part {
    int id;
    float u;
  };
  __shared__ Part back[kWaves][kTok][16];
  const int rank = (int)(blockIdx.x / blocks_per_rank);
  const int wave = threadIdx.x >> 6, sub = threadIdx.x % LPT, tok = (threadIdx.x & 63) / LPT;
  const int64_t t = ((int64_t)(blockIdx.x % blocks_per_rank) * kWaves + wave) * kTok + tok;
  const bool live = t < n.T;
  const float* logits = a.logits[rank] + (live ? t : 0) * n.E;
  const int e0 = sub * J, mine = max(0, min(J, n.E - e0));
  float l[J], s[J], ds[J];
  load_some<J>(logits + (mine > 0 ? e0 : 0), live ? mine : 0, kNegInf, l);
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
  if (sub < 16) back[wave][tok][sub] = Part{id, u};
  wave_sync();
  const float* dsums = a.dsums[rank];
  load_some<J>(dsums ? dsums + (mine > 0 ? e0 : 0) : nullptr, dsums ? mine : 0, 0.0f, ds);
  for (int k = 0; k < n.K; k++) {
    const Part b = back[wave][tok][k];
#pragma unroll
    for (int j = 0; j < J; j++) ds[j] += b.id == e0 + j ? b.u : 0.0f;
  }
  float dot = 0;
  if (!n.sigmoid) {
#pragma unroll
    for (int j = 0; j < J; j++) dot = __builtin_fmaf(s[j], ds[j], dot);
    dot = sum_of<LPT>(dot);
  }
  float d[J];
#pragma unroll
  for (int j = 0; j < J; j++) {
    if (n.sigmoid) {
      const Sigmoid<float> x = sigmoid(l[j]);
      d[j] = x.s * x.rest * ds[j];
    } else {
      d[j] = s[j] * (ds[j] - dot);
    }
    if (l[j] == kNegInf) d[j] = 0.0f;
  }
  float* out = a.dlogits[rank] + t * n.E + e0;
  if (live && mine == J) {
#pragma unroll
    for (int j = 0; j < J; j += 4) __builtin_memcpy(out + j, d + j, 16);
  } else if (live) {
#pragma unroll
    for (int j = 0; j < J; j++)
      if (j < mine) out[j] = d[j];
  }
}

hipError_t launch_stats(const RouteArgs& a, const RouteShape& n, const float* work, int slots, hipStream_t stream) {
  route_stats_kernel<<<dim3((unsigned)((n.E + 63) / 64), (unsigned)n.R), kBlock, 0, stream>>>(a, work, slots, n.E);
  return hipGetLastError();
}

template <int LPT, int J>
hipError_t launch_route_as(const RouteArgs& a, const RouteShape& n, const Layout& at, bool exact, bool stats,
                           float* work, hipStream_t stream) {
  const int slots = route_slots(n.R, n.T);
  const unsigned grid = (unsigned)(slots * n.R);
  const bool groups = n.kept < n.groups;
  if (groups && stats) route_kernel<LPT, J, true, true><<<grid, kBlock, 0, stream>>>(a, n, at, exact, slots, work);
  else if (groups) route_kernel<LPT, J, true, false><<<grid, kBlock, 0, stream>>>(a, n, at, exact, slots, work);
  else if (stats) route_kernel<LPT, J, false, true><<<grid, kBlock, 0, stream>>>(a, n, at, exact, slots, work);
  else route_kernel<LPT, J, false, false><<<grid, kBlock, 0, stream>>>(a, n, at, exact, slots, work);
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

// Lanes of a group where `lanes` share a token and hold J experts each; 0 where
// the groups do not fit.
int lanes_of(int lanes, int J, int groups, int eg) {
  int q = 1;
  while (2 * q * groups <= lanes) q *= 2;
  return groups <= lanes && q * J >= eg ? q : 0;
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, const RouteShape& n, float* work, hipStream_t stream) {
  bool stats = false;
  for (int r = 0; r < n.R; r++) stats |= a.counts[r] || a.sums[r];
  if (n.T <= 0) return stats ? launch_stats(a, n, work, 0, stream) : hipSuccess;  // no slot: zeros
  const int groups = n.kept < n.groups ? n.groups : 1, eg = n.E / groups;
  if (const int q = lanes_of(16, 4, groups, eg)) return launch_route_as<16, 4>(a, n, Layout{eg, q}, false, stats, work, stream);
  if (const int q = lanes_of(16, 16, groups, eg)) return launch_route_as<16, 16>(a, n, Layout{eg, q}, false, stats, work, stream);
  if (const int q = lanes_of(64, 4, groups, eg)) return launch_route_as<64, 4>(a, n, Layout{eg, q}, false, stats, work, stream);
  if (const int q = lanes_of(64, 16, groups, eg)) return launch_route_as<64, 16>(a, n, Layout{eg, q}, false, stats, work, stream);
  // groups that do not fit the lanes: every token by the whole wave, in 64 bits
  return launch_route_as<64, 16>(a, n, Layout{n.E, 64}, true, stats, work, stream);
}

hipError_t launch_route_bwd(const RouteBwdArgs& a, const RouteShape& n, hipStream_t stream) {
  if (n.T <= 0) return hipSuccess;
  if (n.E <= 64) return launch_route_bwd_as<16, 4>(a, n, stream);
  if (n.E <= 256) return launch_route_bwd_as<16, 16>(a, n, stream);
  return launch_route_bwd_as<64, 16>(a, n, stream);
}

}  // namespace ccr
