// The router on sm_103a: logits -> scores -> groups -> the best experts and
// their weights; and its gradient.
//
// A warp takes a token, a lane every 32nd expert. Experts are taken one by one:
// the warp's largest key by one reduction, its lowest index by another, both of
// the integer unit (a float's bits, turned so that they order as integers).
//
// A choice hangs on the last bit, and fp32 scores carry errors of a few. So
// without a bias experts are compared by their logits, which order as the scores
// do and are exact; and where a choice by scores (a bias, a sum over a group) is
// closer than the errors that they can have, the token is done again in 64 bits.
// The bound of a score's error: an exponential of 2 ulp, a division, a sum over
// up to 32 values a lane and 5 steps across lanes, an argument rounded once;
// under 4 ulp of 1 for a sigmoid, under 47 * 2^-24 of the largest score for a
// softmax. kSigmoidNear and kSoftmaxNear are twice that, and kSumNear what the
// rounded sums of two such values add, relative to the largest.
//
// What bounds it: a call of few tokens its launch; with many, the reductions'
// latency (about 60 cycles an expert taken), of which each SM has up to 64 warps'
// in flight. The bytes (1 KB of logits a token) take a tenth of the time.
#include <math.h>

#include "common.cuh"
#include "kernels.cuh"

namespace ep {

namespace {

constexpr int kWarps = 4;  // tokens of a block
constexpr unsigned kAll = 0xffffffffu;
constexpr float kSigmoidNear = 0x1p-20f, kSoftmaxNear = 0x1p-17f, kSumNear = 0x1p-21f;
constexpr float kTiny = 1e-20f;  // added to the sum that weights are divided by

__device__ __forceinline__ float inf() { return __int_as_float(0x7F800000); }

__device__ __forceinline__ float logit(const RouteParams& p, int64_t at) {
  return p.bf16 ? bf16_lo(__ldg(static_cast<const uint16_t*>(p.logits) + at))
                : __ldg(static_cast<const float*>(p.logits) + at);
}

// An order-preserving integer of a float that is no NaN, above 0 unless it is -inf.
__device__ __forceinline__ unsigned key_of(float v) {
  if (v == -inf()) return 0u;
  const unsigned u = __float_as_uint(v + 0.0f);  // -0 and 0 are the same
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(unsigned k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The scores of a token: exp(z - top) / sum, or 1 / (1 + exp(-z)). A NaN scores 0.
struct Scorer {
  bool sigmoid;
  float top, sum;
  __device__ __forceinline__ float term(float z) const {
    return z != z ? 0.0f : z == top ? 1.0f : expf(z - top);  // (several infinities share the sum)
  }
  __device__ __forceinline__ float operator()(float z) const {
    if (sigmoid) return z != z ? 0.0f : 1.0f / (1.0f + expf(-z));
    return top == -inf() ? 0.0f : term(z) / sum;
  }
};

template <int V>
__device__ __forceinline__ Scorer scorer(const RouteParams& p, const float (&z)[V]) {
  Scorer s{p.sigmoid != 0, 0.0f, 0.0f};
  if (s.sigmoid) return s;
  float top = -inf();
#pragma unroll
  for (int j = 0; j < V; ++j) top = fmaxf(top, z[j]);  // a NaN is left out
  s.top = warp_max(top);
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) sum += s.term(z[j]);
  s.sum = warp_sum(sum);
  return s;
}

// Group g's place of an expert in shared memory: a word more after each 32, so
// that lanes that walk through groups of 32 meet different banks.
__device__ __forceinline__ int place(int e) { return e + (e >> 5); }

// The groups that are kept, as bits; T is float or double, `values` the warp's
// choice values (-inf: cannot be chosen). near < 0: exact. Otherwise `close` is
// set where the last kept and the first left out are closer than that.
template <typename T>
__device__ unsigned keep_groups(const RouteParams& p, const T* values, T near, bool& close) {
  const int lane = threadIdx.x & 31, size = p.E / p.groups;
  const T none = -static_cast<T>(inf());
  T best = none, second = none, largest = 0;
  if (lane < p.groups) {
    for (int i = 0; i < size; ++i) {
      const T v = values[place(lane * size + i)];
      if (v > best) {
        second = best;
        best = v;
      } else if (v > second) {
        second = v;
      }
    }
    if (p.group_best == 2 && second > none) {
      largest = fabs(best) > fabs(second) ? fabs(best) : fabs(second);
      best += second;
    }
  }
  int ahead = 0;
  for (int h = 0; h < p.groups; ++h) {
    const T other = __shfl_sync(kAll, best, h);
    ahead += other > best || (other == best && h < lane);
  }
  const bool kept = best > none && ahead < p.topk_groups;
  if (near >= 0) {
    T least = kept ? best : -none, most = kept ? none : best;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const T a = __shfl_xor_sync(kAll, least, o), b = __shfl_xor_sync(kAll, most, o), c = __shfl_xor_sync(kAll, largest, o);
      least = a < least ? a : least;
      most = b > most ? b : most;
      largest = c > largest ? c : largest;
    }
    // (Where a group has one expert, its value counts once; `near` is for two.)
    const T m = fabs(most) > largest ? fabs(most) : largest;
    close = most > none && least - most <= near + static_cast<T>(kSumNear) * m;
  }
  return __ballot_sync(kAll, kept);
}

__device__ __forceinline__ bool can_choose(float z, float b) { return z > -inf() && b > -inf(); }  // no NaN either

// A token's choice in 64 bits: lane k returns the k-th expert, or -1.
template <int V>
__device__ __noinline__ int choose_exactly(const RouteParams& p, int64_t token, double* values) {
  const int lane = threadIdx.x & 31;
  const double none = -static_cast<double>(inf());
  double c[V];
  float top = -inf();
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * 32 + lane;
    const float z = e < p.E ? logit(p, token * p.stride + e) : -inf();
    top = fmaxf(top, z);
    c[j] = z;
  }
  top = warp_max(top);
  double sum = 0.0;
  if (!p.sigmoid) {
#pragma unroll
    for (int j = 0; j < V; ++j) sum += c[j] != c[j] ? 0.0 : c[j] == top ? 1.0 : exp(c[j] - top);
    sum = warp_sum(sum);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * 32 + lane;
    const float b = e < p.E && p.bias ? __ldg(p.bias + e) : 0.0f;
    const double z = c[j];
    c[j] = none;
    if (e < p.E && can_choose(static_cast<float>(z), b))
      c[j] = (p.sigmoid ? 1.0 / (1.0 + exp(-z)) : (z == top ? 1.0 : exp(z - top)) / sum) + b;
  }
  if (p.groups > 1) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane < p.E) values[place(j * 32 + lane)] = c[j];
    __syncwarp();
    bool close = false;
    const unsigned kept = keep_groups<double>(p, values, -1.0, close);
    const int size = p.E / p.groups;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane >= p.E || !(kept >> ((j * 32 + lane) / size) & 1)) c[j] = none;
  }
  if (!p.bias) {  // within the groups the logits say it, however close the scores
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (c[j] > none) c[j] = logit(p, token * p.stride + j * 32 + lane);
  }
  int mine = -1;
  for (int k = 0; k < p.K; ++k) {
    double best = none;
    int at = INT32_MAX;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (c[j] > best) {
        best = c[j];
        at = j * 32 + lane;
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double other = __shfl_xor_sync(kAll, best, o);
      const int other_at = __shfl_xor_sync(kAll, at, o);
      if (other > best || (other == best && other_at < at)) {
        best = other;
        at = other_at;
      }
    }
    if (at == INT32_MAX) break;
    if (lane == k) mine = at;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane == at) c[j] = none;
  }
  return mine;
}

size_t values_bytes(const RouteParams& p) {
  return p.groups > 1 ? sizeof(double) * kWarps * (p.E + p.E / 32 + 1) : 0;
}

// V: experts a lane.
template <int V>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteParams p) {
  extern __shared__ double shared_values[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  double* values = shared_values + w * (p.E + p.E / 32 + 1);
  grid_dependency_wait();
  launch_dependents();
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kWarps + w;
  if (token >= p.N) return;
  const int64_t row = token * p.stride;
  float z[V];
#pragma unroll
  for (int j = 0; j < V; ++j) z[j] = j * 32 + lane < p.E ? logit(p, row + j * 32 + lane) : -inf();
  const Scorer score = scorer(p, z);
  // By what experts are chosen: the logits, or the biased scores.
  const bool by_score = p.bias || (p.groups > 1 && p.group_best == 2);
  const float near = p.sigmoid ? kSigmoidNear : kSoftmaxNear / score.sum;  // (the largest score is 1 / sum)
  unsigned key[V];
  float c[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * 32 + lane;
    const float b = p.bias && e < p.E ? __ldg(p.bias + e) : 0.0f;
    const bool can = can_choose(z[j], b);
    const float s = by_score || p.scores ? score(z[j]) : 0.0f;
    if (p.scores && e < p.E) p.scores[token * p.E + e] = s;
    c[j] = !can ? -inf() : by_score ? s + b : z[j];
    key[j] = !can ? 0u : key_of(p.bias ? c[j] : z[j]);
  }
  bool close = false;
  if (p.groups > 1) {
    float* group_values = reinterpret_cast<float*>(values);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane < p.E) group_values[place(j * 32 + lane)] = c[j];
    __syncwarp();
    const unsigned kept = keep_groups<float>(p, group_values, by_score ? 2.0f * near : -1.0f, close);
    const unsigned size = p.E / p.groups, inverse = size > 1 ? 0xFFFFFFFFu / size + 1 : 0;  // e / size for e < 1024
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const unsigned e = j * 32 + lane, g = size > 1 ? __umulhi(e, inverse) : e;
      if (!(kept >> (g & 31) & 1)) key[j] = 0u;
    }
  }
  int mine = -1;
  float before = 0.0f;
  // With a bias one more is taken, to see how far it is behind.
  const int takes = p.K + (p.bias ? 1 : 0);
  for (int k = 0; k < takes && !close; ++k) {
    unsigned best = 0;
    int at = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    const unsigned most = __reduce_max_sync(kAll, best);
    if (most == 0u) break;
    if (p.bias) {
      const float v = of_key(most);
      close = k > 0 && before - v <= near + kSumNear * fmaxf(fabsf(before), fabsf(v));
      before = v;
    }
    const int e = static_cast<int>(__reduce_min_sync(kAll, best == most ? static_cast<unsigned>(at * 32 + lane) : ~0u));
    if (lane == k && k < p.K) mine = e;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane == e) key[j] = 0u;
  }
  if (close) mine = choose_exactly<V>(p, token, values);
  float s = mine >= 0 ? score(logit(p, row + mine)) : 0.0f;
  if (p.renormalize) s = s / (warp_sum(s) + kTiny);
  if (lane < p.K) {
    p.idx[token * p.K + lane] = mine;
    p.weights[token * p.K + lane] = s * p.scale;
  }
}

template <int V>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(const RouteParams p) {
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  launch_dependents();
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (token >= p.N) return;
  const int64_t row = token * p.stride;
  float s[V], d[V];
#pragma unroll
  for (int j = 0; j < V; ++j) s[j] = j * 32 + lane < p.E ? logit(p, row + j * 32 + lane) : -inf();
  // Lane k has the k-th chosen expert.
  int e = -1;
  float dw = 0.0f;
  if (lane < p.K) {
    e = __ldg(p.chosen + token * p.K + lane);
    if (e < -1 || e >= p.E) {
      flag(p.status, EP_ST_BAD_INDEX);
      e = -1;
    }
    if (e >= 0) dw = __ldg(p.grad_weights + token * p.K + lane) * p.scale;
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    d[j] = p.grad_scores && j * 32 + lane < p.E ? __ldg(p.grad_scores + token * p.E + j * 32 + lane) : 0.0f;
  const Scorer score = scorer(p, s);
  if (p.renormalize) {
    const float w = e >= 0 ? score(logit(p, row + e)) : 0.0f;
    const float sum = warp_sum(w) + kTiny;
    dw = (dw - warp_sum(dw * (w / sum))) / sum;
  }
  for (int k = 0; k < p.K; ++k) {
    const int at = __shfl_sync(kAll, e, k);
    const float add = __shfl_sync(kAll, dw, k);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane == at) d[j] += add;
  }
  float dot = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    s[j] = score(s[j]);
    if (s[j] != 0.0f) dot += s[j] * d[j];
  }
  if (!p.sigmoid) dot = warp_sum(dot);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = j * 32 + lane;
    if (i >= p.E) continue;
    // (An expert that scores 0 moves nothing, whatever its gradient.)
    const float dz = s[j] == 0.0f ? 0.0f : p.sigmoid ? s[j] * (1.0f - s[j]) * d[j] : s[j] * (d[j] - dot);
    if (p.bf16)
      static_cast<__nv_bfloat16*>(p.grad_logits)[token * p.E + i] = __float2bfloat16(dz);
    else
      static_cast<float*>(p.grad_logits)[token * p.E + i] = dz;
  }
}

template <int V>
cudaError_t launch(const RouteParams& p, bool backward, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.N) + kWarps - 1) / kWarps)), block(kWarps * 32);
  return backward ? launch_kernel(route_backward_kernel<V>, grid, block, 0, s, /*dependent=*/true, p)
                  : launch_kernel(route_kernel<V>, grid, block, values_bytes(p), s, /*dependent=*/true, p);
}

cudaError_t launch_any(const RouteParams& p, bool backward, cudaStream_t s) {
  if (p.N <= 0) return cudaSuccess;
  const int per = (p.E + 31) / 32;
  if (per <= 1) return launch<1>(p, backward, s);
  if (per <= 2) return launch<2>(p, backward, s);
  if (per <= 4) return launch<4>(p, backward, s);
  if (per <= 8) return launch<8>(p, backward, s);
  if (per <= 16) return launch<16>(p, backward, s);
  return launch<32>(p, backward, s);
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, cudaStream_t s) { return launch_any(p, false, s); }
cudaError_t launch_route_backward(const RouteParams& p, cudaStream_t s) { return launch_any(p, true, s); }

}  // namespace ep
