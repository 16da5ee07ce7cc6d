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
//            (in fp64 where a chosen s_k is below fp32's normal numbers)
//
// Choices are those of 64-bit arithmetic, so that they do not hang on a
// rounding: keys are computed in fp32, and where two that decide lie nearer to
// each other than their error bound, the token is chosen again in fp64 by its whole
// wave (one in some hundred of random logits; every token whose deciding keys are
// equal where there is a bias: 8 x 4096 tokens of 256 zeros with a bias of zeros 85
// us, random ones 27, in 8 groups 117 and 36).  Keys are compared as unsigned numbers in the
// order of the values, NaN above all (it reaches the weights), 0 for an expert
// that cannot be chosen.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ccr_device.h"
#include "ccr_internal.h"

namespace ccr {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

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
// The same for 64 bits, and the rows of 16 and halves of 32 lanes against each other.
template <int CTRL, typename T>
__device__ __forceinline__ T other(T x) {
  if constexpr (sizeof(T) == 4) {
    return across<CTRL>(x);
  } else {
    const u32x2 v = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(T, u32x2{across<CTRL>(v[0]), across<CTRL>(v[1])});
  }
}
template <typename T, typename F, typename S>
__device__ __forceinline__ T swapped(T x, F&& f, S&& swap) {
  if constexpr (sizeof(T) == 4) {
    const auto r = swap(__builtin_bit_cast(uint32_t, x));
    return f(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1]));
  } else {
    const u32x2 v = __builtin_bit_cast(u32x2, x);
    const auto lo = swap(v[0]), hi = swap(v[1]);
    return f(__builtin_bit_cast(T, u32x2{(uint32_t)lo[0], (uint32_t)hi[0]}),
             __builtin_bit_cast(T, u32x2{(uint32_t)lo[1], (uint32_t)hi[1]}));
  }
}
template <int N, typename T, typename F>
__device__ __forceinline__ T reduce(T x, F&& f) {
  if constexpr (N > 1) x = f(x, other<0xb1>(x));
  if constexpr (N > 2) x = f(x, other<0x4e>(x));
  if constexpr (N > 4) x = f(x, other<0x141>(x));
  if constexpr (N > 8) x = f(x, other<0x140>(x));
  if constexpr (N > 16)
    x = swapped(x, f, [](uint32_t v) { return __builtin_amdgcn_permlane16_swap(v, v, false, false); });
  if constexpr (N > 32)
    x = swapped(x, f, [](uint32_t v) { return __builtin_amdgcn_permlane32_swap(v, v, false, false); });
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
// largest; never 0 (nor, of 32 bits, the largest number).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);  // -0 is 0
  return x != x ? 0xfffffffeu : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x + 0.0);
  return x != x ? ~0ull : b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ double value_of(uint64_t k) {
  return __builtin_bit_cast(double, k >> 63 ? k & ~(1ull << 63) : ~k);
}

// exp(x), x <= 0: 2^n 2^f with n + f = x log2(e), whose last bits the second
// product adds; off by two units of its 24 bits at most.
__device__ __forceinline__ float exponential(float x) {
  constexpr double kLog2e = 1.4426950408889634;
  constexpr float kHigh = (float)kLog2e, kLow = (float)(kLog2e - (double)kHigh);
  const float y = x < -200.0f ? -200.0f : x;  // 0 from -104 on; NaN stays
  const float n = __builtin_rintf(y * kHigh);
  const float f = __builtin_fmaf(y, kLow, __builtin_fmaf(y, kHigh, -n));
  return ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}
__device__ __forceinline__ double exponential(double x) { return exp(x); }

// 1 / (1 + exp(-l)) without overflow, and its complement.
template <typename T>
struct Sigmoid {
  T s, rest;
};
__device__ __forceinline__ Sigmoid<float> sigmoid(float l) {
  const float t = exponential(-fabsf(l)), d = 1.0f + t, r = __builtin_amdgcn_rcpf(d);
  const float q = __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.0f), r);  // 1 / d
  return l >= 0 ? Sigmoid<float>{q, t * q} : Sigmoid<float>{t * q, q};
}
__device__ __forceinline__ Sigmoid<double> sigmoid(double l) {
  const double t = exp(-fabs(l)), q = 1.0 / (1.0 + t);
  return l >= 0 ? Sigmoid<double>{q, t * q} : Sigmoid<double>{t * q, q};
}

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
  int eg, log_q;  // experts of a group, log2 of its lanes
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
  uint64_t key[E];
  uint64_t value[kRouteGroups];
  uint8_t keep[kRouteGroups];
};

template <int J, bool GROUPS>
__device__ __forceinline__ void choose_exactly(const float* logits, const float* bias, const RouteShape& n,
                                            ExactRoom<GROUPS ? 64 * J : 1>* room, const Layout at, int J32,
                                            uint32_t* out) {
  int lane = threadIdx.x & 63;
  int eg = at.eg, size = n.groups;
  // seldom used: nothing of this is worth a register of the caller's loop
  asm volatile("" : "+v"(lane), "+s"(eg), "+s"(size));
  size = n.E / size;
  const bool real = GROUPS && n.group_top == 2;  // values, not only their order, count
  float l[J], with[J];
  double s[J], v[J];
#pragma unroll
  for (int j = 0; j < J; j++) {
    l[j] = lane * J + j < n.E ? logits[lane * J + j] : kNegInf;
    with[j] = bias && lane * J + j < n.E ? bias[lane * J + j] : 0.0f;
  }
  if (bias || real) scores<64, J, double>(l, n.sigmoid, s);
  uint64_t key[J];
#pragma unroll
  for (int j = 0; j < J; j++) {
    v[j] = bias ? s[j] + (double)with[j] : (double)l[j];
    key[j] = l[j] == kNegInf ? 0 : ordered(v[j]);
  }
  if constexpr (GROUPS) {
    // a group's value: of one key that key, of two their sum (of scores, where
    // the keys are logits); an expert that cannot be chosen is none of the two
#pragma unroll
    for (int j = 0; j < J; j++)
      if (lane * J + j < n.E) room->key[lane * J + j] = key[j] != 0 && real && !bias ? ordered(s[j]) : key[j];
    wave_sync();
    if (lane < n.groups) {
      uint64_t a = 0, b = 0;
#pragma unroll 8
      for (int i = 0; i < size; i++) {
        const uint64_t x = room->key[lane * size + i], low = a < x ? a : x;
        b = b > low ? b : low;
        a = a > x ? a : x;
      }
      room->value[lane] = n.group_top == 2 && b != 0 ? ordered(value_of(a) + value_of(b)) : a;
    }
    wave_sync();
    if (lane < n.groups) {
      const uint64_t o = room->value[lane];
      int rank = 0;
#pragma unroll 4
      for (int i = 0; i < n.groups; i++) {
        const uint64_t p = room->value[i];
        rank += p > o || (p == o && i < lane);
      }
      room->keep[lane] = rank < n.kept;
    }
    wave_sync();
#pragma unroll
    for (int j = 0; j < J; j++)
      if (lane * J + j < n.E && !room->keep[(lane * J + j) / size]) key[j] = 0;
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
          const int e = lane * J + j, g = e / eg, i = e - g * eg;
          out[k] = (uint32_t)(((g << at.log_q) + i / J32) * J32 + i % J32) << 16 | (uint32_t)e;
        }
    }
  }
  wave_sync();
}

// ------------------------------------------------------------------ 32 bits
// A network that sorts N numbers, N a power of two: sorts halves and merges them,
// the merge splitting even and odd places (Batcher).
template <int N>
struct Network {
  int n = 0, a[64] = {}, b[64] = {};
  constexpr Network() {
    for (int p = 1; p < N; p *= 2)
      for (int k = p; k >= 1; k /= 2)
        for (int j = k % p; j + k < N; j += 2 * k)
          for (int i = 0; i < k && i + j + k < N; i++)
            if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
              a[n] = i + j;
              b[n] = i + j + k;
              n++;
            }
  }
};

// What a wave's lanes tell each other of their tokens.
template <int LPT, int J>
struct Room {
  static constexpr int kTok = 64 / LPT;
  uint32_t chosen[kTok][16];                       // choice k: its place and expert
  u32x2 pick[kTok][16];                       // choice k: its lane and how often the lane had its key before; its key
  __align__(16) uint32_t group[kTok][LPT];         // groups' values
  __align__(16) uint32_t of_place[kTok][LPT * J];  // keys, then scores
  // The word of a place: a lane's vectors in another order from lane to lane, or
  // those of every fourth lane would lie in the same banks.
  static __device__ __forceinline__ int at(int lane, int j) {
    return J < 16 ? lane * J + j : lane * J + (((j >> 2) ^ (lane >> 2 & 3)) << 2 | (j & 3));
  }
  template <typename T>
  __device__ __forceinline__ void put(int tok, int lane, const T* v) {
#pragma unroll
    for (int j = 0; j < J; j += 4) {
      const T four[4] = {v[j], v[j + 1], v[j + 2], v[j + 3]};
      *reinterpret_cast<dev::u32x4*>(&of_place[tok][at(lane, j)]) = __builtin_bit_cast(dev::u32x4, four);
    }
  }
};

// The wave's tokens' choices; l, s, bias: those of this lane's J experts.  Returns
// whether a decision of this lane's token was too near to make.
//
// Each lane sorts its keys (they alone: 2 instructions to a comparison), and a
// round takes the largest of the lanes' first ones.  Which expert a choice is, the
// K lanes of the choices find at the end, all at once, among the winners' keys.
// (Searching and striking out in every round took twice the instructions.)
template <int LPT, int J, bool GROUPS>
__device__ __forceinline__ bool choose(const float* l, const float* s, const float* bias, bool with_bias,
                                       const RouteShape& n, const Layout at, int lane, Room<LPT, J>* room) {
  const int sub = lane % LPT, tok = lane / LPT;
  const bool of_scores = GROUPS && n.group_top == 2 && !with_bias;  // groups' values
  uint32_t key[J];
#pragma unroll
  for (int j = 0; j < J; j++) key[j] = l[j] == kNegInf ? 0 : ordered(with_bias ? s[j] + bias[j] : l[j]);
  room->put(tok, sub, key);
  // fp32 scores are off by up to 2^-22 (sigmoid: the exponential's two units at a
  // quarter, one each of the sum, the reciprocal and the product) or 2^-20 of the
  // largest one (softmax), the sum with the bias by 2^-24 of itself
  float err = 0x1p-22f;
  if (!n.sigmoid && (with_bias || of_scores)) {
    float top = 0;
#pragma unroll
    for (int j = 0; j < J; j++) top = fmaxf(top, s[j]);
    err = 0x1p-20f * max_of<LPT>(top);
  }
  bool near = false, keep = true;
  uint32_t a = 0, b = 0;
  auto merge = [&](uint32_t c, uint32_t d) {  // c >= d
    b = max(min(a, c), max(b, d));
    a = max(a, c);
  };
  if (of_scores) {
#pragma unroll
    for (int j = 0; j < J; j++) merge(key[j] ? ordered(s[j]) : 0, 0);
  }
  constexpr Network<J> net;
#pragma unroll
  for (int c = 0; c < net.n; c++) {
    const uint32_t x = key[net.a[c]], y = key[net.b[c]];
    key[net.a[c]] = max(x, y);
    key[net.b[c]] = min(x, y);
  }
  if constexpr (GROUPS) {
    // the two largest keys (scores, where the keys are logits) of the group
    if (!of_scores) {
      a = key[0];
      b = key[1];
    }
    const int q = 1 << at.log_q, g = sub >> at.log_q;
    if (q > 1) merge(across<0xb1>(a), across<0xb1>(b));
    if (q > 2) merge(across<0x4e>(a), across<0x4e>(b));
    if (q > 4) merge(across<0x141>(a), across<0x141>(b));
    if (q > 8) merge(across<0x140>(a), across<0x140>(b));
    if constexpr (LPT == 64) {
      if (q > 16) merge(__shfl_xor(a, 16), __shfl_xor(b, 16));
    }
    // The group's value, of one key or two, and what it may be off by: its keys'
    // scores, and the roundings of the keys and of their sum, which are shares of the
    // keys themselves: they may cancel.  Infinite keys are exact.
    const bool two = n.group_top == 2 && b != 0;
    const float first = value_of(a), second = two ? value_of(b) : 0.0f, parts = fabsf(first) + fabsf(second);
    float off = fmaxf(fabsf(first), fabsf(second)) == -kNegInf ? 0.0f : 2 * err + 0x1p-21f * parts;
    asm volatile("" : "+v"(off));  // one register over the loop below, not its parts
    if (two) a = ordered(first + second);
    if ((sub & (q - 1)) == 0) room->group[tok][g] = g < n.groups ? a : 0;
    wave_sync();
    // how many groups are before this one: a larger value, or as large and left
    int rank = 0;
    for (int i = 0; i < n.groups; i += 4) {
      const dev::u32x4 o = *reinterpret_cast<const dev::u32x4*>(&room->group[tok][i]);
#pragma unroll
      for (int k = 0; k < 4; k++) rank += i + k < n.groups && o[k] >= a + (i + k < g ? 0 : 1);
    }
    keep = rank < n.kept && g < n.groups;
    if (with_bias || n.group_top == 2) {
      // Every kept group's least value against the others' largest; a sum beyond fp32
      // and NaN are undecided.  A group of no expert that can be chosen (0) is kept
      // only if all others are such groups.
      const float least = value_of(a) - off, most = value_of(a) + off;
      const float low = min_of<LPT>(!keep || a == 0 ? -kNegInf : least == least ? least : kNegInf);
      const float high = max_of<LPT>(keep || a == 0 || g >= n.groups ? kNegInf : most == most ? most : -kNegInf);
      near |= high != kNegInf && !(low > high);  // -infinity: no group is left out that could stay
    }
  }
  const uint64_t left = ((1ull << sub) - 1) << tok * LPT;  // the token's lanes before this one
  uint32_t before = 0, mine = ~0u;
  int again = 0;
  const int rounds = n.K + (with_bias ? 1 : 0);  // one more for the key that just missed
  for (int k = 0; k < rounds; k++) {
    const uint32_t m = keep ? key[0] : 0, best = max_of<LPT>(m);
    if (with_bias && k > 0 && best != 0) {
      const float x = value_of(before), y = value_of(best);
      near |= !(x - y > 2 * err + 0x1p-23f * (fabsf(x) + fabsf(y)));
    }
    before = best;
    if (k == n.K) break;
    const bool won = m == best && (__ballot(m == best) & left) == 0;  // the lowest lane that has it
    if (won) {
      again = best == mine ? again + 1 : 0;
      mine = best;
      room->pick[tok][k] = u32x2{(uint32_t)sub << 8 | (uint32_t)again, best};
    }
#pragma unroll
    for (int j = 0; j < J; j++) {
      uint32_t here = key[j], next = j + 1 < J ? key[j + 1] : 0;
      asm("" : "+v"(here), "+v"(next));  // two numbers: as two places to load from they made the array an indexed one
      key[j] = won ? next : here;
    }
  }
  wave_sync();
  if (sub < n.K) {
    const u32x2 p = room->pick[tok][sub];
    const int from = (int)(p[0] >> 8);
    int skip = (int)(p[0] & 255), j = -1;
#pragma unroll
    for (int v = 0; v < J; v += 4) {
      const dev::u32x4 x = *reinterpret_cast<const dev::u32x4*>(&room->of_place[tok][Room<LPT, J>::at(from, v)]);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const bool same = x[i] == p[1];
        j = same && skip == 0 ? v + i : j;
        skip -= same;
      }
    }
    room->chosen[tok][sub] = p[1] == 0 ? kNone : (uint32_t)(from * J + j) << 16 |
                                                     (uint32_t)((from >> at.log_q) * at.eg + (from & ((1 << at.log_q) - 1)) * J + j);
  }
  return near;
}

// The renormalised weights of a wave's tokens from t0 on in 64 bits, where a chosen
// score, or a softmax's exponential before its division by at most 1024, is below
// 2^-116: scores in fp32 lose their digits from 2^-126 on.  (Behind the tokens' loop,
// by the lanes that wrote topk; within it, it cost registers.)
template <int LPT>
__device__ __forceinline__ void precise_weights(const float* logits, const RouteShape& n, int64_t t0,
                                                const int32_t* topk, float* weights) {
  const int lane = threadIdx.x & 63, sub = lane % LPT;
  const int64_t t = t0 + lane / LPT;
  const bool here = t < n.T && sub < n.K;
  const int e = here ? topk[t * n.K + sub] : -1;
  double x = 0;
  if (e >= 0) {
    const float* row = logits + t * n.E;
    float m = kNegInf;  // the row's largest, NaN with one
    if (!n.sigmoid)
      for (int i = 0; i < n.E; i++) m = row[i] > m || row[i] != row[i] ? row[i] : m;
    const double l = (double)row[e];
    x = n.sigmoid ? sigmoid(l).s : m < -kNegInf ? exp(l - (double)m) : __builtin_nan("");
  }
  const bool tiny = max_of<LPT>(e >= 0 && x < 0x1p-116 ? 1 : 0) != 0;
  const double sum = sum_of<LPT>(x);
  if (here && tiny) weights[t * n.K + sub] = (sum == 0.0 ? 0.0f : (float)(x / sum)) * n.scale;
}

// A token per LPT lanes, J experts to a lane; a workgroup takes every slots-th
// step of its rank's tokens.  STATS: it counts its tokens' choices and sums their
// scores, in its slot of the work array or, alone, in the results.
template <int LPT, int J, bool GROUPS, bool STATS>
__global__ __launch_bounds__(kBlock, LPT == 16 ? 4 : LPT == 32 ? 3 : 2) void route_kernel(const RouteArgs a, const RouteShape n, const Layout at,
                                                       bool exact, int slots, float* work) {
  constexpr int kTok = 64 / LPT, kWaves = kBlock / 64, kPlaces = LPT * J;
  constexpr int kExactJ = (kPlaces + 63) / 64;
  __shared__ Room<LPT, J> all_rooms[kWaves];
  __shared__ ExactRoom<GROUPS ? 64 * kExactJ : 1> rooms[GROUPS ? kWaves : 1];
  __shared__ int count[STATS ? kPlaces : 1];
  const int rank = blockIdx.x / slots, slot = blockIdx.x % slots;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Room<LPT, J>& room = all_rooms[wave];
  const float* logits = a.logits[rank];
  const bool with_bias = a.bias[rank] != nullptr;
  float sums[J];
  if constexpr (STATS) {
#pragma unroll
    for (int j = 0; j < J; j++) sums[j] = 0;
    for (int e = threadIdx.x; e < kPlaces; e += kBlock) count[e] = 0;
    __syncthreads();
  }
  uint64_t tiny = 0;
  for (int64_t t0 = ((int64_t)slot * kWaves + wave) * kTok; t0 < n.T; t0 += (int64_t)slots * kWaves * kTok) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // what follows from it costs less anew than registers between the steps
    const int sub = lane % LPT, tok = lane / LPT;
    const int g = sub >> at.log_q, i0 = (sub & ((1 << at.log_q) - 1)) * J, e0 = g * at.eg + i0;
    const int mine = g * at.eg < n.E ? max(0, min(J, at.eg - i0)) : 0;
    const int64_t t = t0 + tok;
    const bool live = t < n.T;
    float l[J], s[J], bias[J];
    load_some<J>(logits + (live && mine > 0 ? t * n.E + e0 : 0), live ? mine : 0, kNegInf, l);
    if (with_bias) load_some<J>(a.bias[rank] + (mine > 0 ? e0 : 0), mine, 0.0f, bias);
    scores<LPT, J, float>(l, n.sigmoid, s);
    if constexpr (STATS) {
#pragma unroll
      for (int j = 0; j < J; j++) sums[j] += s[j];
    }
    bool near = exact;
    if (!exact) near = choose<LPT, J, GROUPS>(l, s, bias, with_bias, n, at, lane, &room);
    for (uint64_t todo = __ballot(near && live && sub == 0); todo; todo &= todo - 1) {
      const int k = (__ffsll((unsigned long long)todo) - 1) / LPT;
      choose_exactly<kExactJ, GROUPS>(logits + (t0 + k) * n.E, a.bias[rank], n, &rooms[GROUPS ? wave : 0], at, J,
                                      room.chosen[k]);
    }
    wave_sync();
    room.put(tok, sub, s);
    wave_sync();
    const uint32_t c = live && sub < n.K ? room.chosen[tok][sub & 15] : kNone;
    float w = c != kNone ? __builtin_bit_cast(float, room.of_place[tok][room.at((int)(c >> 16) / J, (int)(c >> 16) % J)]) : 0.0f;
    if (n.renorm) {
      const float total = sum_of<LPT>(w);
      tiny |= __ballot(c != kNone && w < 0x1p-115f);
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
  if (tiny)
    for (int64_t t0 = ((int64_t)slot * kWaves + wave) * kTok; t0 < n.T; t0 += (int64_t)slots * kWaves * kTok)
      precise_weights<LPT>(logits, n, t0, a.topk[rank], a.weights[rank]);
  if constexpr (STATS) {
    const int lane = threadIdx.x & 63;
    room.put(lane / LPT, lane % LPT, sums);
    __syncthreads();
    for (int e = threadIdx.x; e < n.E; e += kBlock) {
      const int eg = e / at.eg, i = e - eg * at.eg, of = (eg << at.log_q) + i / J, p = of * J + i % J;
      float s = 0;
#pragma unroll
      for (int k = 0; k < kWaves * kTok; k++)
        s += __builtin_bit_cast(float, all_rooms[k / kTok].of_place[k % kTok][room.at(of, i % J)]);
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

// The slots' counts and sums, in an order of their own: a workgroup takes 64
// experts, a wave of it every 16th slot (with 4 waves the reads of the slots were
// most of the kernel: 9.8 us at 8 ranks of 128 slots and 256 experts).
constexpr int kStatsBlock = 1024;
__global__ __launch_bounds__(kStatsBlock) void route_stats_kernel(const RouteArgs a, const float* work, int slots, int E) {
  constexpr int kWaves = kStatsBlock / 64;
  __shared__ double sum_part[kWaves][64];
  __shared__ int64_t count_part[kWaves][64];
  const int rank = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  const float* from = work + (int64_t)rank * slots * 2 * E;
  double s = 0;
  int64_t c = 0;
  if (e < E) {
#pragma unroll 4
    for (int k = wave; k < slots; k += kWaves) {
      s += (double)from[(int64_t)k * 2 * E + e];
      c += reinterpret_cast<const int*>(from)[((int64_t)k * 2 + 1) * E + e];
    }
  }
  sum_part[wave][lane] = s;
  count_part[wave][lane] = c;
  __syncthreads();
  if (wave == 0 && e < E) {
#pragma unroll
    for (int k = 1; k < kWaves; k++) {
      s += sum_part[k][lane];
      c += count_part[k][lane];
    }
    if (a.sums[rank]) a.sums[rank][e] = (float)s;
    if (a.counts[rank]) a.counts[rank][e] = c;
  }
}

// A choice's share of the sum of its token's chosen scores, 0 without one (have):
// c / sum c, or where a chosen score is below fp32's normal numbers from its logit
// lk (m: the row's largest) in 64 bits.
template <int LPT>
__device__ __forceinline__ float share(float c, float lk, float m, bool have, bool sig) {
  const float total = sum_of<LPT>(c);
  float w = total == 0.0f ? 0.0f : c / total;
  const uint64_t tiny = __ballot(have && c < 0x1p-126f);
  if (tiny) {
    const double x = !have ? 0.0 : sig ? sigmoid((double)lk).s : exp((double)lk - (double)m);
    const double sum = sum_of<LPT>(x);
    const int first = (threadIdx.x & 63) / LPT * LPT;  // the token's lanes
    if (tiny << (64 - LPT - first) >> (64 - LPT)) w = sum == 0.0 ? 0.0f : (float)(x / sum);
  }
  return w;
}

// ---------------------------------------------------------------- backward
// With c_k the chosen scores and u_k = scale dw_k, the gradient of the scores
// is u_k at the k-th choice and, at every expert, that of the sums of scores; that
// of the logits is s (ds - sum s ds) for a softmax, s (1 - s) ds for sigmoids.
//
// Renormalised, the choices' part is (u_k - sum w u) / C with C = sum c and w = c /
// C, and adds to the logits' gradient w_k (u_k - sum w u), for sigmoids times 1 - c_k
// (a softmax's own sum over it is 0).  So no score divides another's: 1 / C may be
// beyond fp32.  Of choices with scores below its normal numbers w is that of 64 bits.
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
  float c = 0, u = 0, lk = kNegInf;
  if (live && sub < n.K) {
    id = a.topk[rank][t * n.K + sub];
    if (id < 0 || id >= n.E) id = -1;
    if (id >= 0) lk = logits[id];
    if (lk == kNegInf) id = -1;
    if (id >= 0) {
      c = n.sigmoid ? sigmoid(lk).s : expf(lk - m) * inv;
      u = a.dweights[rank][t * n.K + sub] * n.scale;
    }
  }
  if (n.renorm) {
    float w = share<LPT>(c, lk, m, id >= 0, n.sigmoid);
    w *= u - sum_of<LPT>(w * u);
    u = n.sigmoid ? w * sigmoid(lk).rest : w;
  }
  if (sub < 16) back[wave][tok][sub] = Part{id, u};
  wave_sync();
  const float* dsums = a.dsums[rank];
  load_some<J>(dsums ? dsums + (mine > 0 ? e0 : 0) : nullptr, dsums ? mine : 0, 0.0f, ds);
  float chosen[J];
#pragma unroll
  for (int j = 0; j < J; j++) chosen[j] = 0.0f;
  for (int k = 0; k < n.K; k++) {
    const Part b = back[wave][tok][k];
#pragma unroll
    for (int j = 0; j < J; j++) chosen[j] += b.id == e0 + j ? b.u : 0.0f;
  }
  if (!n.renorm) {
#pragma unroll
    for (int j = 0; j < J; j++) ds[j] += chosen[j];
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
    if (n.renorm) d[j] += chosen[j];
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
  route_stats_kernel<<<dim3((unsigned)((n.E + 63) / 64), (unsigned)n.R), kStatsBlock, 0, stream>>>(a, work, slots, n.E);
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
  // As few lanes to a token as hold its experts: what all lanes do for a choice is
  // shared by more tokens (65,536 tokens, us; 16 lanes with 4 and 16 experts each, 32
  // and 64 with 16; E = 64: 18, 41; 256: 45, 89, 228; 512: 83, 234; 256 in 32
  // groups, which 32 lanes hold: 105, 281).
  const int groups = n.kept < n.groups ? n.groups : 1, eg = n.E / groups;
  if (const int q = lanes_of(16, 4, groups, eg)) return launch_route_as<16, 4>(a, n, Layout{eg, __builtin_ctz((unsigned)q)}, false, stats, work, stream);
  if (const int q = lanes_of(16, 16, groups, eg)) return launch_route_as<16, 16>(a, n, Layout{eg, __builtin_ctz((unsigned)q)}, false, stats, work, stream);
  if (const int q = lanes_of(32, 16, groups, eg)) return launch_route_as<32, 16>(a, n, Layout{eg, __builtin_ctz((unsigned)q)}, false, stats, work, stream);
  if (const int q = lanes_of(64, 16, groups, eg)) return launch_route_as<64, 16>(a, n, Layout{eg, __builtin_ctz((unsigned)q)}, false, stats, work, stream);
  // groups that do not fit the lanes: every token by the whole wave, in 64 bits (32,768
  // tokens of 48 groups of 21 experts: 410 us; of 64 groups of 16, which fit: 176)
  return launch_route_as<64, 16>(a, n, Layout{n.E, 6}, true, stats, work, stream);
}

hipError_t launch_route_bwd(const RouteBwdArgs& a, const RouteShape& n, hipStream_t stream) {
  if (n.T <= 0) return hipSuccess;
  // likewise (on one more step of lanes or experts each: E = 64: 12 us, 25; 256: 48, 53;
  // 512: 87, 104)
  if (n.E <= 64) return launch_route_bwd_as<16, 4>(a, n, stream);
  if (n.E <= 256) return launch_route_bwd_as<16, 16>(a, n, stream);
  if (n.E <= 512) return launch_route_bwd_as<32, 16>(a, n, stream);
  return launch_route_bwd_as<64, 16>(a, n, stream);
}

}  // namespace ccr
