// Routing to experts by scores.
//
// Per token: scores s = softmax(l) or sigmoid(l) of the router's logits; choice
// c = s + b with a balancing bias b (without one the order of c is that of l, so
// the logits themselves are compared); with groups, only the experts of the
// top_groups best groups stay (a group's mark is its largest choice, or the sum
// of its two largest); the top K of what stays, larger choice first, ties to the
// lower index; weights are the chosen scores, optionally over their sum, times a
// factor.
//
// The order of two close choices decides whole numbers, so c and the marks are
// formed in 64 bits whenever they are more than a logit.
//
// Layout: 16 lanes per token, lane i holds experts i*V .. i*V+V-1 (V = E/16
// rounded up to a power of two), so a token's logits are read as one contiguous
// run and lower lanes hold lower indices.  Values become unsigned keys of the
// same order, with 0 for an expert that is taken, masked or beyond E; every
// round takes the largest key (four lane exchanges), the lowest lane holding it
// and that lane's lowest place.  Keys of real experts are never 0, so the ids of
// a token are distinct and in range even for logits that are not finite.
#include "kernels.h"

namespace clha {

constexpr int kRL = 16;              // lanes per token (>= kMaxTopK)
constexpr int kRTokens = 256 / kRL;  // tokens per workgroup

template <typename T>
__device__ __forceinline__ T lane_max(T v) {
#pragma unroll
  for (int o = 1; o < kRL; o <<= 1) {
    const T w = __shfl_xor(v, o, kRL);
    v = w > v ? w : v;
  }
  return v;
}
__device__ __forceinline__ double lane_sum(double v) {
#pragma unroll
  for (int o = 1; o < kRL; o <<= 1) v += __shfl_xor(v, o, kRL);
  return v;
}

// Order-preserving unsigned keys (x + 0 makes the two zeros equal); never 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t k = u >> 31 ? ~u : u | 0x80000000u;
  return k ? k : 1u;
}
__device__ __forceinline__ unsigned long long order_key(double x) {
  const unsigned long long u = __double_as_longlong(x + 0.0);
  const unsigned long long k = u >> 63 ? ~u : u | (1ull << 63);
  return k ? k : 1ull;
}

template <bool WIDE>
struct KeyOf {
  typedef uint32_t type;
};
template <>
struct KeyOf<true> {
  typedef unsigned long long type;
};

// WIDE: the choice is s + b in 64 bits (a bias is given); otherwise the logit.
// GROUPS: more than one group.
template <int V, bool WIDE, bool GROUPS>
__global__ __launch_bounds__(256) void score_route_kernel(const float* __restrict__ logits,
                                                          const float* __restrict__ bias, int64_t n, int E, int K,
                                                          RouteArgs a, int32_t* __restrict__ topk,
                                                          float* __restrict__ weights, int32_t* __restrict__ iota,
                                                          int* __restrict__ status, int layer, int has_layer) {
  typedef typename KeyOf<WIDE>::type Key;
  __shared__ double member[GROUPS ? kRTokens * kMaxExperts : 1];
  __shared__ double mark[GROUPS ? kRTokens * kMaxExperts : 1];
  __shared__ uint32_t keep[GROUPS ? kRTokens * (kMaxExperts / 32) : 1];
  const int lane = threadIdx.x % kRL, slot = threadIdx.x / kRL;
  const int64_t t = (int64_t)blockIdx.x * kRTokens + slot;
  const float* row = logits + (t < n ? t : n - 1) * E;   // tokens past the end repeat the last one
  float l[V];
  bool bad = false;
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane * V + j;
    l[j] = e < E ? row[e] : 0.0f;
    if (e < E) {
      bad |= !isfinite(l[j]);
      top = fmaxf(top, l[j]);
    }
  }
  top = lane_max(top);
  const bool soft = a.score == kScoreSoftmax;
  double s[V];          // scores in 64 bits, where the choice or the marks need them
  double den = 1.0;     // sum of exp(l - top)
  const bool marks_by_score = GROUPS && a.group_score == kGroupTop2;
  if (WIDE || marks_by_score) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = lane * V + j;
      s[j] = soft ? exp((double)l[j] - (double)top) : 1.0 / (1.0 + exp(-(double)l[j]));
      if (e < E) sum += s[j];
    }
    if (soft) {
      den = lane_sum(sum);
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] /= den;
    }
  } else if (soft && !a.renormalize) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane * V + j < E) sum += (double)expf(l[j] - top);
    den = lane_sum(sum);
  }
  Key key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane * V + j;
    if constexpr (WIDE) {
      const float b = e < E ? bias[e] : 0.0f;
      bad |= !isfinite(b);
      s[j] += (double)b;
      key[j] = e < E ? order_key(s[j]) : 0;
    } else {
      key[j] = e < E ? order_key(l[j]) : 0;
    }
  }
  if constexpr (GROUPS) {
    const int per = E / a.n_groups;
    double* mem = member + slot * kMaxExperts;
    double* mk = mark + slot * kMaxExperts;
    uint32_t* kp = keep + slot * (kMaxExperts / 32);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane * V + j < E) mem[lane * V + j] = WIDE || marks_by_score ? s[j] : (double)l[j];
    if (lane < kMaxExperts / 32) kp[lane] = 0;
    __syncthreads();
    for (int g = lane; g < a.n_groups; g += kRL) {
      double m1 = -INFINITY, m2 = -INFINITY;
      for (int i = 0; i < per; ++i) {
        const double v = mem[g * per + i];
        m2 = fmax(m2, fmin(m1, v));
        m1 = fmax(m1, v);
      }
      mk[g] = a.group_score == kGroupTop2 && per > 1 ? m1 + m2 : m1;
    }
    __syncthreads();
    for (int g = lane; g < a.n_groups; g += kRL) {
      const unsigned long long mine = order_key(mk[g]);
      int better = 0;
      for (int o = 0; o < a.n_groups; ++o) {
        const unsigned long long other = order_key(mk[o]);
        better += other > mine || (other == mine && o < g);
      }
      if (better < a.top_groups) atomicOr(&kp[g >> 5], 1u << (g & 31));
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = (lane * V + j) / per;
      if (lane * V + j < E && !((kp[g >> 5] >> (g & 31)) & 1u)) key[j] = 0;
    }
  }
  int chosen = 0;   // of round `lane`
  for (int k = 0; k < K; ++k) {
    Key best = 0;
    int at = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    }
    const Key m = lane_max(best);
    const unsigned long long vote = __ballot(best == m);
    const int first = __ffs((unsigned)(vote >> ((threadIdx.x & 63) / kRL * kRL)) & 0xffffu) - 1;
    const int e = __shfl(lane * V + at, first, kRL);
    if (lane == k) chosen = e;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane == first && j == at) key[j] = 0;
  }
  // weights, in 64 bits: one chosen expert per lane
  const bool mine = lane < K;
  const float lc = row[mine ? chosen : 0];
  double w = 0.0;
  if (soft && a.renormalize) {
    // the softmax's own sum cancels; relative to the largest chosen logit nothing underflows to 0/0
    const float lm = lane_max(mine ? lc : -INFINITY);
    w = mine ? exp((double)lc - (double)lm) : 0.0;
  } else if (mine) {
    w = soft ? exp((double)lc - (double)top) / den : 1.0 / (1.0 + exp(-(double)lc));
  }
  if (a.renormalize) {
    const double sum = lane_sum(w);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (t < n) {
    if (mine) {
      topk[t * K + lane] = chosen;
      if (weights) weights[t * K + lane] = (float)(w * (double)a.scale);
    }
    if (iota && lane == 0) iota[t] = (int32_t)t;
    if (bad) {
      atomicOr(status, kStatusNonfinite);
      if (has_layer)
        atomicCAS(reinterpret_cast<unsigned long long*>(status + kStatusLayer), 0ull,
                  (1ull << 32) | (unsigned long long)(uint32_t)layer);
      else
        atomicOr(status + kStatusRoute, 1);
    }
  }
}

namespace {
struct RouteCall {
  const float *logits, *bias;
  int64_t n;
  int E, K;
  RouteArgs a;
  int32_t* topk;
  float* weights;
  int32_t* iota;
  int* status;
  int layer, has_layer;
};

template <int V, bool WIDE, bool GROUPS>
void run_route(const RouteCall& c, hipStream_t s) {
  hipLaunchKernelGGL((score_route_kernel<V, WIDE, GROUPS>), dim3((unsigned)((c.n + kRTokens - 1) / kRTokens)),
                     dim3(256), 0, s, c.logits, c.bias, c.n, c.E, c.K, c.a, c.topk, c.weights, c.iota, c.status,
                     c.layer, c.has_layer);
}
template <int V>
void run_route_v(const RouteCall& c, hipStream_t s) {
  const bool groups = c.a.n_groups > 1;
  if (c.bias) {
    if (groups) run_route<V, true, true>(c, s);
    else run_route<V, true, false>(c, s);
  } else {
    if (groups) run_route<V, false, true>(c, s);
    else run_route<V, false, false>(c, s);
  }
}
}  // namespace

void launch_score_route(const float* logits, const float* bias, int64_t n, int E, int K, const RouteArgs& a,
                        int32_t* topk, float* weights, int32_t* iota, int* status, int layer, bool has_layer,
                        hipStream_t s) {
  const RouteCall c{logits, bias, n, E, K, a, topk, weights, iota, status, layer, has_layer ? 1 : 0};
  if (E <= 16) run_route_v<1>(c, s);
  else if (E <= 32) run_route_v<2>(c, s);
  else if (E <= 64) run_route_v<4>(c, s);
  else if (E <= 128) run_route_v<8>(c, s);
  else run_route_v<16>(c, s);
}

}  // namespace clha
