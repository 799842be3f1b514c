// route.cu -- tokens to experts: scores, the choice of k of them, their weights, and
// the order that sorts the chosen (token, expert) pairs by expert.
//
// A warp takes a token, lane l its experts l, l + 32, ....  The choice compares
// score + bias, numbers that may be closer than FP32 tells apart, so it is made in
// FP32 first, with a bound on the error of each difference; where one of the
// comparisons that decide the outcome falls below it, the token is chosen again in
// 64 bits (about one token in a thousand).  Without a bias the scores are in the
// order of the logits, which need no rounding.  Ties go to the lowest index.
//
// Sorting: a block takes 128 tokens and holds a bit for each (expert, token), so
// that a pair's place among its expert's is a count of bits: no atomics on places,
// and tokens stay in order.  With more than one block the counts go through memory
// and a second kernel adds up those of the blocks before.
//
// The instructions of the choice bound it, about 1500 a token of 256 experts at 2.9 a
// clock, on 128 of 152 SMs (a block for each 128 tokens), and then the block with the
// most tokens that need 64 bits: 16384 x 256, sigmoid, bias, 4 of 8 groups, 8 chosen, 54
// to 60 us a call by the inputs (the logits are 17 MB, 2.5 us), 68000 clocks of an
// average block and 99000 of the busiest.  128 x 256 is one block and takes 32 us.  Loops
// that are not written out matter: a choice's code written out does not stay in the
// instruction cache (74 against 58 us under the profiler).  So do the tokens that need 64
// bits: chosen by a warp alone, with the other warps waiting, 70 us with an L2 flush, by
// all warps together 62.
#include <cfloat>

#include "experts.h"
#include "kernels.h"

namespace g07 {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr float kUnit = 1.2e-7f;  // a unit in the last place of FP32, relative: 2^-23
constexpr int kChunk = kRouteChunk;
constexpr int kWords = kChunk / 32;
// A token's choice is a chain of reductions: up to 256 experts, whose keys leave room
// for it, 32 warps of an SM hide one another's.
template <int V>
constexpr int kThreads = V <= 8 ? 1024 : 512;

// FP32 and 64-bit values as unsigned numbers in the same order; 0 is below all of
// them and stands for "not to be chosen": NaN and -infinity.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v);
  return v > -INFINITY ? b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u)
                       : 0u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ unsigned long long key_of(double v) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(v));
  return v > -INFINITY
             ? b ^ (static_cast<unsigned long long>(static_cast<long long>(b) >> 63) | (1ull << 63))
             : 0ull;
}
__device__ __forceinline__ double value_of(unsigned long long key) {
  return __longlong_as_double(
      static_cast<long long>(key >> 63 ? key ^ (1ull << 63) : ~key));
}
// -0 and +0 are equal numbers; keys have to be too.
template <typename V>
__device__ __forceinline__ V plain_zero(V v) {
  return v + V(0);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
  const uint32_t hi = static_cast<uint32_t>(v >> 32), top = __reduce_max_sync(kAll, hi);
  const uint32_t lo = __reduce_max_sync(kAll, hi == top ? static_cast<uint32_t>(v) : 0u);
  return static_cast<unsigned long long>(top) << 32 | lo;
}

template <typename Key>
struct Choice {
  int index;  // lane j < k: the j-th expert or -1
  Key key;    // of it; 0: none
  Key rest;   // the largest of this lane's that are not chosen
};

// The k largest keys, lowest index first among equals.  key[i] belongs to expert
// i * 32 + lane; those that are not chosen are left.
template <int V, typename Key>
__device__ __forceinline__ Choice<Key> pick(Key (&key)[V], int k) {
  const int lane = threadIdx.x & 31;
  Choice<Key> c{-1, 0, 0};
  Key mine = 0;
  auto largest = [&]() {
    mine = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) mine = key[i] > mine ? key[i] : mine;
  };
  largest();
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    const Key top = warp_max(mine);
    if (top == 0) break;
    unsigned at = 0x7FFFFFFFu;
    if (mine == top) {
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (key[i] == top) at = static_cast<unsigned>(i * 32 + lane);
    }
    at = __reduce_min_sync(kAll, at);
    if (lane == j) {
      c.index = static_cast<int>(at);
      c.key = top;
    }
    if (static_cast<int>(at & 31u) == lane) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == static_cast<int>(at >> 5)) key[i] = 0;
      largest();
    }
  }
  c.rest = mine;
  return c;
}

// Leaves only the keys of the `kept` groups with the largest sums of their
// group_top (1 or 2) largest values; a group without a key that can be chosen is
// last.  slack: how far the scores in such a sum, together, may be off; negative: the
// values are exact.  FP32 keys that are not: true where another choice of groups is
// within reach.
template <int V, typename Key>
__device__ __forceinline__ bool keep_groups(Key (&key)[V], int groups, int size, int kept,
                                            int group_top, float slack) {
  const int lane = threadIdx.x & 31;
  Key sum = 0;            // lane g: group g
  float rounding = 0.0f;  // of the sum
  auto put = [&](int g, Key first, Key second) {
    const bool two = group_top != 1 && second != 0;
    if (lane != g) return;
    sum = first;
    if constexpr (sizeof(Key) == 4) rounding = 2.0f * kUnit * fabsf(value_of(first));
    if (!two) return;
    auto v = value_of(first) + value_of(second);
    if constexpr (sizeof(Key) == 4) {
      rounding += 2.0f * kUnit * fabsf(value_of(second));
      // (masks of the type's lowest value add up to less than FP32 holds: held at its
      // lowest, within the bound of which 64 bits decide)
      v = fmaxf(v, -FLT_MAX);
    }
    sum = key_of(plain_zero(v));
  };
  if (size == 32) {  // a group is one key of each lane
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const Key first = warp_max(key[i]);
      const int holder = __ffs(__ballot_sync(kAll, key[i] == first)) - 1;
      put(i, first, warp_max(lane == holder ? Key(0) : key[i]));
    }
  } else {
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
      const int lo = g * size, hi = lo + size;
      Key mine = 0, next = 0;  // this lane's two largest
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        if (e >= lo && e < hi) {
          if (key[i] > mine) {
            next = mine;
            mine = key[i];
          } else if (key[i] > next) {
            next = key[i];
          }
        }
      }
      const Key first = warp_max(mine);
      const int holder = __ffs(__ballot_sync(kAll, mine == first)) - 1;
      put(g, first, warp_max(lane == holder ? next : mine));
    }
  }
  unsigned keep = 0;
  Key left = sum;
#pragma unroll 1
  for (int j = 0; j < kept; ++j) {
    const Key top = warp_max(left);
    if (top == 0) break;  // the others have nothing to choose
    const int at = __ffs(__ballot_sync(kAll, left == top)) - 1;
    keep |= 1u << at;
    if (lane == at) left = 0;
  }
  bool close = false;
  if constexpr (sizeof(Key) == 4) {
    if (slack >= 0.0f) {
      // Each value was rounded at its own size, half a unit of it, and so was their sum:
      // where they cancel, the sum's size says nothing of its error.  (A bound that is
      // infinite, or no number, leaves it open.)
      const float v = value_of(sum), off = slack + rounding;
      const bool in = keep >> lane & 1u;
      const Key least = __reduce_min_sync(kAll, in ? key_of(v - off) : kAll);
      const Key most = warp_max(in || sum == 0 ? 0u : key_of(v + off));
      close = most != 0 && most >= least;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int g = size == 32 ? i : (i * 32 + lane) / size;
    if (g >= groups || !(keep >> g & 1u)) key[i] = 0;
  }
  return close;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// The sigmoid times e^-shift, shift <= 0 the largest of several logits (0 if that is
// positive), for quotients of sigmoids: by itself it leaves FP32 below a logit of -88,
// where the quotients are ordinary numbers.  0 where 64 bits have no sigmoid either.
__device__ __forceinline__ float sigmoid_over(float l, float shift) {
  const float e = expf(-fabsf(l));
  const float top = l >= 0.0f ? 1.0f : l < -709.7f ? 0.0f : expf(l - shift);
  return top / (1.0f + e);
}

// The logit of this lane's expert e (0 for -1), from the token's.
template <int V>
__device__ __forceinline__ float logit_of(const float (&l)[V], int e) {
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float x = __shfl_sync(kAll, l[i], e & 31);
    if (i == e >> 5) v = x;
  }
  return v;
}

// The choice in 64 bits, from the definition: the token's logits, and in `score` the
// sigmoid of each, or its exponential for softmax.
template <int V>
__device__ __forceinline__ int choose_64(const RouteArgs& a, const float (&l)[V],
                                         const double* score, float* weight) {
  const int lane = threadIdx.x & 31;
  double total = 0.0;
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) total += i * 32 + lane < a.E ? score[i * 32 + lane] : 0.0;
    total = warp_sum(total);
  }
  unsigned long long key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    key[i] = 0ull;
    if (e < a.E && l[i] > -INFINITY) {
      double v = a.sigmoid ? score[e] : score[e] / total;
      if (a.bias) v += static_cast<double>(__ldg(a.bias + e));
      key[i] = key_of(plain_zero(v));
    }
  }
  if (a.kept < a.groups) keep_groups<V>(key, a.groups, a.E / a.groups, a.kept, a.group_top, -1.0f);
  if (!a.bias) {  // in the order of the logits
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] != 0) key[i] = key_of(plain_zero(static_cast<double>(l[i])));
  }
  const int first = pick<V>(key, a.k).index;
  const int at = lane < a.k ? first : -1;
  double w = at < 0 ? 0.0 : a.sigmoid ? score[at] : score[at] / total;
  if (a.renorm && !a.sigmoid) {  // over the chosen alone, as FP32 does: theirs may all be 0
    const float chosen = logit_of<V>(l, first);
    const float most = value_of(warp_max(at >= 0 ? key_of(plain_zero(chosen)) : 0u));
    if (at >= 0) w = exp(static_cast<double>(chosen) - static_cast<double>(most));
  }
  if (a.renorm) {
    const double sum = warp_sum(w);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  *weight = static_cast<float>(w) * a.scale;
  return at;
}

// Experts (lane j: the j-th or -1) and weights of a token from its logits
// (-infinity past the last expert); *unsure: a comparison was too close to tell.
template <int V>
__device__ __forceinline__ int route_token(const RouteArgs& a, const float (&l)[V], float* weight,
                                           bool* unsure) {
  const int lane = threadIdx.x & 31;
  *unsure = false;
  bool nan = false;
  float mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    nan |= l[i] != l[i];
    mine = fmaxf(mine, l[i]);
  }
  const float top = value_of(warp_max(key_of(plain_zero(mine))));  // (NaN: no key)
  const bool any = __any_sync(kAll, mine > -INFINITY);
  nan = __any_sync(kAll, nan);
  // Scores that are not numbers choose nothing, and show in the weights.
  if (nan || (!a.sigmoid && any && top == INFINITY)) {
    *weight = __int_as_float(0x7FC00000);
    return -1;
  }
  if (!any) {
    *weight = 0.0f;
    return -1;
  }

  // Softmax's sum over all: for the weights themselves unless they are
  // renormalised, else for the choice alone.
  const bool scores = a.bias || (a.kept < a.groups && a.group_top > 1);
  float total = 1.0f;
  float s[V];
  if (a.sigmoid) {
    if (scores) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = __fdividef(1.0f, 1.0f + __expf(-l[i]));
    }
  } else if (scores || !a.renorm) {
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = expf(l[i] - top);
      total += s[i];
    }
    total = warp_sum(total);
    const float inverse = __fdividef(1.0f, total);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] *= inverse;
  }

  // How far a difference of two scores in FP32 may be off.  Sigmoid: the
  // exponential's 2 + 1.2 |l| units in the last place weigh s (1 - s), at most 1/4
  // and with |l| 0.23, the quotient adds 2 units; softmax: 2 units each for
  // exponential, sum (of up to 1024 numbers, 32 a lane and 5 steps: 40) and
  // quotient, of at most the largest score.  Two scores (of two experts, or the two
  // in a group's sum), and half a unit of each sum with the bias.
  const float slack = a.sigmoid ? 8.0f * kUnit : 96.0f * kUnit * __fdividef(1.0f, total);
  auto told = [&](float hi, float lo) {
    return hi - lo > slack + 2.0f * kUnit * fmaxf(fabsf(hi), fabsf(lo));
  };

  uint32_t key[V];
  bool close = false;
  if (a.kept < a.groups) {
    if (scores) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        const float v = s[i] + (a.bias && e < a.E ? __ldg(a.bias + e) : 0.0f);
        key[i] = l[i] > -INFINITY ? key_of(plain_zero(v)) : 0u;
      }
      close = keep_groups<V>(key, a.groups, a.E / a.groups, a.kept, a.group_top, slack);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = key_of(plain_zero(l[i]));
      keep_groups<V>(key, a.groups, a.E / a.groups, a.kept, a.group_top, -1.0f);
    }
    if (!a.bias) {  // within the groups by the logits
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] != 0) key[i] = key_of(plain_zero(l[i]));
    }
  } else if (a.bias) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      key[i] = l[i] > -INFINITY && e < a.E ? key_of(plain_zero(s[i] + __ldg(a.bias + e))) : 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = key_of(plain_zero(l[i]));
  }

  const Choice<uint32_t> c = pick<V>(key, a.k);
  const float chosen = logit_of<V>(l, c.index);
  const int at = lane < a.k ? c.index : -1;
  if (a.bias) {
    // every two that follow each other have to be told apart, or equal in everything
    const uint32_t before = __shfl_up_sync(kAll, c.key, 1);
    const int other = __shfl_up_sync(kAll, c.index, 1);
    const float its = __shfl_up_sync(kAll, chosen, 1);
    bool near = lane > 0 && c.key != 0 && !told(value_of(before), value_of(c.key));
    if (near && its == chosen) near = __ldg(a.bias + other) != __ldg(a.bias + c.index);
    // and so has everything that is left from the last: behind one that is its equal
    // there may be another that is not
    const uint32_t last = __shfl_sync(kAll, c.key, a.k - 1);
    const bool behind = last != 0 && c.rest != 0 && !told(value_of(last), value_of(c.rest));
    if (__any_sync(kAll, behind)) {
      const float last_logit = __shfl_sync(kAll, chosen, a.k - 1);
      const float last_bias = __ldg(a.bias + __shfl_sync(kAll, c.index, a.k - 1));
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] != 0 && !told(value_of(last), value_of(key[i])))
          near |= l[i] != last_logit || __ldg(a.bias + i * 32 + lane) != last_bias;
    }
    close |= __any_sync(kAll, near);
  }
  *unsure = close;

  // Weights, from the scores without the bias: FP32 as the outputs are, which leaves 6e-8
  // of them against 64 bits (16384 x 256), where scores in 64 bits would leave half of that
  // for 64-bit exponentials of every token.
  float w = 0.0f;
  if (!a.renorm) {
    if (at >= 0) w = a.sigmoid ? 1.0f / (1.0f + expf(-chosen)) : expf(chosen - top) / total;
  } else {
    const float most = value_of(warp_max(at >= 0 ? key_of(plain_zero(chosen)) : 0u));
    if (at >= 0) w = a.sigmoid ? sigmoid_over(chosen, fminf(most, 0.0f)) : expf(chosen - most);
    const float sum = warp_sum(w);
    w = sum > 0.0f ? w / sum : 0.0f;
  }
  *weight = w * a.scale;
  return at;
}

// A block of 128 tokens: choices, weights and, for a single block, the sorted order;
// else the number of its tokens for each expert.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads<V>) route_kernel(RouteArgs a) {
  constexpr int kWarps = kThreads<V> / 32;
  extern __shared__ double score[];  // [E], of a token that needs 64 bits
  uint32_t* bits = reinterpret_cast<uint32_t*>(score + a.E);  // [E][kWords]: tokens of each expert
  __shared__ int warp_total[kWarps], unsure[kChunk], unsure_count;
  grid_dependency_wait();
  grid_dependents_go();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) unsure_count = 0;
  const int t0 = static_cast<int>(blockIdx.x) * kChunk;
  const int tokens = a.T - t0 < kChunk ? a.T - t0 : kChunk;
  for (int i = threadIdx.x; i < a.E * kWords; i += kThreads<V>) bits[i] = 0;
  __syncthreads();
  auto load = [&](int t, float (&l)[V]) {
    const T* row = static_cast<const T*>(a.logits) + (t0 + t) * a.ld;
#pragma unroll
    for (int i = 0; i < V; ++i)
      l[i] = i * 32 + lane < a.E ? to_f32(row[i * 32 + lane]) : -INFINITY;
  };
  auto put = [&](int t, int at, float w) {
    if (lane < a.k) {
      const int64_t o = static_cast<int64_t>(t0 + t) * a.k + lane;
      a.index[o] = at;
      a.weight[o] = w;
      if (at >= 0) atomicOr(&bits[at * kWords + (t >> 5)], 1u << (t & 31));
    }
  };
#pragma unroll 1
  for (int t = warp; t < tokens; t += kWarps) {
    float l[V];
    load(t, l);
    float w;
    bool close;
    const int at = route_token<V>(a, l, &w, &close);
    if (close) {
      if (lane == 0) unsure[atomicAdd(&unsure_count, 1)] = t;
    } else {
      put(t, at, w);
    }
  }
  __syncthreads();
  // What FP32 could not tell, token by token: every thread an expert's score (a warp by
  // itself would keep its block, and the kernel, waiting for its 64-bit exponentials),
  // then a warp the choice.
  const int again = unsure_count;
#pragma unroll 1
  for (int u = 0; u < again; ++u) {
    const int t = unsure[u];
    float l[V];
    load(t, l);
    float top = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
    const T* row = static_cast<const T*>(a.logits) + (t0 + t) * a.ld;
    for (int e = threadIdx.x; e < a.E; e += kThreads<V>) {
      const double x = static_cast<double>(to_f32(row[e]));
      score[e] = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - static_cast<double>(top));
    }
    __syncthreads();
    if (warp == 0) {
      float w;
      const int at = choose_64<V>(a, l, score, &w);
      put(t, at, w);
    }
    __syncthreads();
  }
  __syncthreads();
  auto count = [&](int e) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) n += __popc(bits[e * kWords + i]);
    return n;
  };
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < a.E; e += kThreads<V>)
      a.counts[static_cast<int64_t>(blockIdx.x) * route_count_stride(a.E) + e] =
          static_cast<uint8_t>(count(e));
    return;
  }
  // The only block: each thread holds the experts 2 i and 2 i + 1.
  int* start = reinterpret_cast<int*>(bits + a.E * kWords);
  const int e0 = 2 * static_cast<int>(threadIdx.x);
  const int n0 = e0 < a.E ? count(e0) : 0, n1 = e0 + 1 < a.E ? count(e0 + 1) : 0;
  int upto = n0 + n1;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int v = __shfl_up_sync(kAll, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) warp_total[warp] = upto;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < kWarps; ++i) {
    before += i < warp ? warp_total[i] : 0;
    all += warp_total[i];
  }
  const int at0 = before + upto - n0 - n1;
  if (e0 < a.E) {
    start[e0] = at0;
    a.offsets[e0] = at0;
  }
  if (e0 + 1 < a.E) {
    start[e0 + 1] = at0 + n0;
    a.offsets[e0 + 1] = at0 + n0;
  }
  if (threadIdx.x == 0) a.offsets[a.E] = all;
  __syncthreads();
  const int pairs = tokens * a.k;
  for (int i = threadIdx.x; i < pairs; i += kThreads<V>) {
    const int t = i / a.k, e = a.index[i];
    int place = -1;
    if (e >= 0) {
      place = start[e];
      for (int w = 0; w < t >> 5; ++w) place += __popc(bits[e * kWords + w]);
      place += __popc(bits[e * kWords + (t >> 5)] & ((1u << (t & 31)) - 1u));
      a.source[place] = t;
    }
    a.slot[i] = place;
    if (i >= all) a.source[i] = -1;
  }
}

// The sorted order, a block for each 128 tokens, from the counts of all blocks.
__global__ void __launch_bounds__(1024) route_sort_kernel(RouteArgs a) {
  extern __shared__ uint32_t bits[];  // [E][kWords], then [E] starts
  __shared__ int warp_total[32];
  grid_dependency_wait();
  grid_dependents_go();
  int* start = reinterpret_cast<int*>(bits + a.E * kWords);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = static_cast<int>(gridDim.x), chunk = static_cast<int>(blockIdx.x);
  const int t0 = chunk * kChunk;
  const int tokens = a.T - t0 < kChunk ? a.T - t0 : kChunk;
  for (int i = threadIdx.x; i < a.E * (kWords + 1); i += 1024) bits[i] = 0;
  __syncthreads();
  // the experts' counts, four to a word: all of them, and those before this block.  The
  // blocks are shared among as many threads as there are.
  const int words = route_count_stride(a.E) / 4, parts = 1024 / words;
  const int e4 = static_cast<int>(threadIdx.x) % words, part = static_cast<int>(threadIdx.x) / words;
  if (part < parts) {
    const uint32_t* counts = reinterpret_cast<const uint32_t*>(a.counts) + e4;
    int total[4] = {0, 0, 0, 0}, earlier[4] = {0, 0, 0, 0};
#pragma unroll 8
    for (int c = part; c < chunks; c += parts) {
      const uint32_t n = __ldg(counts + static_cast<int64_t>(c) * words);
      const uint32_t m = c < chunk ? n : 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        total[i] += static_cast<int>(n >> (8 * i) & 255u);
        earlier[i] += static_cast<int>(m >> (8 * i) & 255u);
      }
    }
    // (sums of whole numbers: the order of the atomics does not matter)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e4 * 4 + i;
      if (e < a.E) {
        atomicAdd(&start[e], total[i]);
        atomicAdd(reinterpret_cast<int*>(&bits[e * kWords]), earlier[i]);
      }
    }
  }
  __syncthreads();
  const bool mine = static_cast<int>(threadIdx.x) < a.E;
  const int n = mine ? start[threadIdx.x] : 0;
  const int earlier = mine ? static_cast<int>(bits[threadIdx.x * kWords]) : 0;
  int upto = n;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int v = __shfl_up_sync(kAll, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) warp_total[warp] = upto;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < 32; ++i) {
    before += i < warp ? warp_total[i] : 0;
    all += warp_total[i];
  }
  if (mine) {
    start[threadIdx.x] = before + upto - n + earlier;
    bits[threadIdx.x * kWords] = 0;
    if (chunk == 0) a.offsets[threadIdx.x] = before + upto - n;
  }
  if (chunk == 0 && threadIdx.x == 0) a.offsets[a.E] = all;
  __syncthreads();
  const int pairs = tokens * a.k;
  const int64_t first = static_cast<int64_t>(t0) * a.k;
  for (int i = threadIdx.x; i < pairs; i += 1024) {
    const int x = a.index[first + i], t = i / a.k;
    if (x >= 0) atomicOr(&bits[x * kWords + (t >> 5)], 1u << (t & 31));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += 1024) {
    const int t = i / a.k, x = a.index[first + i];
    int place = -1;
    if (x >= 0) {
      place = start[x];
      for (int w = 0; w < t >> 5; ++w) place += __popc(bits[x * kWords + w]);
      place += __popc(bits[x * kWords + (t >> 5)] & ((1u << (t & 31)) - 1u));
      a.source[place] = t0 + t;
    }
    a.slot[first + i] = place;
    if (first + i >= all) a.source[first + i] = -1;
  }
}

// The gradient of the weights with respect to a token's logits: with w_j = scale *
// s_j (/ S, S = sum of the chosen s when renormalised), d the gradient of w,
//   ds_j = scale * (d_j - sum_i d_i s_i / S) / S   (scale * d_j),
// then sigmoid: ds s (1 - s); softmax: s (ds - sum ds s), which for renormalised
// weights is a softmax over the chosen experts alone, and 0 for all others.
template <typename T, int V>
__global__ void __launch_bounds__(256) route_bwd_kernel(RouteArgs a) {
  grid_dependency_wait();
  grid_dependents_go();
  const int lane = threadIdx.x & 31;
  const int t = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  int at = -1;
  float d = 0.0f, l = 0.0f;
  if (lane < a.k) {
    const int64_t o = static_cast<int64_t>(t) * a.k + lane;
    at = __ldg(a.chosen + o);
    if (at < 0 || at >= a.E) at = -1;
    if (at >= 0) {
      d = a.scale * __ldg(a.d_weight + o);
      l = to_f32(row[at]);
    }
  }
  float g = 0.0f;       // of the chosen logit
  float rest = 0.0f;    // softmax over all: every expert's share of it
  float top = 0.0f;
  const bool over_all = !a.sigmoid && !a.renorm;
  float all[V];
  if (a.renorm) {
    float most = at >= 0 ? l : -INFINITY;
#pragma unroll
    for (int i = 16; i; i >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, i));
    if (most == -INFINITY) most = 0.0f;  // closed experts: scores of 0
    float s = 0.0f;
    if (at >= 0) s = a.sigmoid ? sigmoid_over(l, fminf(most, 0.0f)) : expf(l - most);
    const float sum = warp_sum(s);
    s = sum > 0.0f ? s / sum : s;
    const float dot = warp_sum(d * s);
    g = s * (d - dot);
    if (a.sigmoid && at >= 0) g /= 1.0f + expf(l);
  } else if (a.sigmoid) {
    const float s = at >= 0 ? 1.0f / (1.0f + expf(-l)) : 0.0f;
    g = at >= 0 ? d * s / (1.0f + expf(l)) : 0.0f;
  } else {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      all[i] = i * 32 + lane < a.E ? to_f32(row[i * 32 + lane]) : -INFINITY;
      top = fmaxf(top, all[i]);
    }
#pragma unroll
    for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, i));
    if (top == -INFINITY) top = 0.0f;  // a token of padding: scores of 0
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      all[i] = expf(all[i] - top);
      sum += all[i];
    }
    sum = warp_sum(sum);
    const float inverse = sum == 0.0f ? 0.0f : 1.0f / sum;
    g = at >= 0 ? expf(l - top) * inverse * d : 0.0f;
    rest = -warp_sum(g) * inverse;
  }
  T* out = static_cast<T*>(a.d_logits) + t * a.ld_d;
  float o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = over_all ? all[i] * rest : 0.0f;
  for (int j = 0; j < a.k; ++j) {  // in the order of the choice: the same expert twice adds up
    const int e = __shfl_sync(kAll, at, j);
    const float v = __shfl_sync(kAll, g, j);
    if (e >= 0 && (e & 31) == lane) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == e >> 5) o[i] += v;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i * 32 + lane < a.E) out[i * 32 + lane] = from_f32<T>(o[i]);
}

template <int V>
cudaError_t route_of(const RouteArgs& a, bool gradient, cudaStream_t stream) {
  if (gradient) {
    const dim3 grid((a.T + 7) / 8);
    const cudaError_t e =
        a.bf16 ? launch_pdl(route_bwd_kernel<__nv_bfloat16, V>, grid, dim3(256), 0, stream, a)
               : launch_pdl(route_bwd_kernel<float, V>, grid, dim3(256), 0, stream, a);
    if (e == cudaSuccess) note_launches(1);
    return e;
  }
  const int chunks = a.T > kChunk ? (a.T + kChunk - 1) / kChunk : 1;  // (no token: offsets of 0)
  const size_t sort = static_cast<size_t>(a.E) * (kWords + 1) * 4;
  const size_t smem = static_cast<size_t>(a.E) * sizeof(double) + sort;  // at most 28 KB
  cudaError_t e = a.bf16 ? launch_pdl(route_kernel<__nv_bfloat16, V>, dim3(chunks), dim3(kThreads<V>),
                                      smem, stream, a)
                         : launch_pdl(route_kernel<float, V>, dim3(chunks), dim3(kThreads<V>), smem,
                                      stream, a);
  if (e == cudaSuccess && chunks > 1)
    e = launch_pdl(route_sort_kernel, dim3(chunks), dim3(1024), sort, stream, a);
  if (e == cudaSuccess) note_launches(chunks > 1 ? 2 : 1);
  return e;
}

cudaError_t by_experts(const RouteArgs& a, bool gradient, cudaStream_t stream) {
  if (a.E <= 32) return route_of<1>(a, gradient, stream);
  if (a.E <= 64) return route_of<2>(a, gradient, stream);
  if (a.E <= 128) return route_of<4>(a, gradient, stream);
  if (a.E <= 256) return route_of<8>(a, gradient, stream);
  if (a.E <= 512) return route_of<16>(a, gradient, stream);
  return route_of<32>(a, gradient, stream);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  return by_experts(a, false, stream);
}
cudaError_t launch_route_bwd(const RouteArgs& a, cudaStream_t stream) {
  return by_experts(a, true, stream);
}

}  // namespace g07
