// The router on sm_103a: logits -> scores -> groups -> the best experts and
// their weights; and its gradient.
//
// A warp takes a token, a lane neighbouring experts (up to 32), which it sorts. Experts
// are then taken one by one: the warp's largest key by a reduction of the integer
// unit (a float's bits, turned so that they order as integers), and of the lanes
// that show it the first.
//
// A choice hangs on the last bit, and fp32 scores carry errors of a few. So
// without a bias experts are compared by their logits, which order as the scores
// do and are exact; and where a choice by scores (a bias, a sum over a group) is
// closer than the errors that they can have, the experts that it is between are
// compared in 64 bits (some of 10,000 tokens; done for all of a token's experts
// it made 16384 tokens take 36 us instead of 25, since an SM has two units of
// 64-bit arithmetic and the token is waited for at the end).
// The bound of a score's error: an exponential of 2 ulp, a reciprocal of 1, a
// product, a sum over up to 32 values a lane and 5 steps across lanes, an argument
// rounded once; under 4 ulp of 1 for a sigmoid, under 48 * 2^-24 of the largest for a
// softmax. kSigmoidNear and kSoftmaxNear are twice that, and kSumNear what the
// rounded sums of two such values add, relative to the largest.
//
// What bounds it: a call of few tokens its launch (4 us on the device, 12 from
// Python); with many, its instructions (about 1200 a token of 256 experts in 8
// groups, 4 issued in 5 cycles). The bytes (1 KB of logits a token) take a tenth of
// the time. Measured: 16384 tokens x 256 experts, 8 of 4 of 8 groups with a bias 22 us;
// softmax alone 16 us; 131072 tokens 150 and 116 us. The gradient of 16384 x 256: sigmoid
// 9.9 us, 3.5 TB/s, softmax 14.9 us; 131072 tokens 70 us.
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

// An order-preserving integer of a float that is no NaN; kNone of -inf.
constexpr unsigned kNone = 0x007FFFFFu;
__device__ __forceinline__ unsigned key_of(float v) {
  const unsigned u = __float_as_uint(v + 0.0f);  // -0 and 0 are the same
  return u ^ (static_cast<unsigned>(static_cast<int>(u) >> 31) | 0x80000000u);
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
  float top, sum, inverse;
  __device__ __forceinline__ float term(float z) const {
    return z != z ? 0.0f : z == top ? 1.0f : expf(z - top);  // (several infinities share the sum)
  }
  __device__ __forceinline__ float operator()(float z) const {
    if (sigmoid) {
      float r;  // (within an ulp)
      asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + expf(-z)));
      return z != z ? 0.0f : r;
    }
    return top == -inf() ? 0.0f : term(z) * inverse;
  }
};

// The sigmoid's derivative s (1 - s) as e / (1 + e)^2 with e = exp(-|z|): 1 - s would
// keep two bits of an expert whose logit is 15, and none from 18 on. A NaN has none.
__device__ __forceinline__ float sigmoid_slope(float z) {
  const float e = expf(-fabsf(z));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));  // (of a number from 1 to 2)
  return z != z ? 0.0f : e * r * r;
}

template <int V>
__device__ __forceinline__ Scorer scorer(const RouteParams& p, const float (&z)[V]) {
  Scorer s{p.sigmoid != 0, 0.0f, 0.0f, 0.0f};
  if (s.sigmoid) return s;
  float top = -inf();
#pragma unroll
  for (int j = 0; j < V; ++j) top = fmaxf(top, z[j]);  // a NaN is left out
  s.top = warp_max(top);
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) sum += s.term(z[j]);
  s.sum = warp_sum(sum);
  s.inverse = 1.0f / s.sum;
  return s;
}

// Group g's place of an expert in shared memory: a word more after each 32, so
// that lanes that walk through groups of 32 meet different banks.
__device__ __forceinline__ int place(int e) { return e + (e >> 5); }

// Whether this lane's group g is kept; every lane knows its group's best two
// values (-inf: none), and lanes g * lanes on are group g's. near < 0: the values
// are exact. Otherwise `close` is set where the last group kept and the first left
// out are closer than that. (Of two values half the sum is compared: the sum of two of
// the type's lowest would be -inf, a group of which no expert is left. What is lost of
// numbers below 2^-125 is below any `near`.)
__device__ __forceinline__ bool keeps_group(const RouteParams& p, float best, float second, int g, int lanes, float near,
                                            bool& close) {
  const float none = -inf();
  float largest = 0.0f;
  if (p.group_best == 2) {
    near *= 0.5f;
    best *= 0.5f;
    if (second > none) {
      largest = fmaxf(fabsf(best), 0.5f * fabsf(second));
      best = fmaf(0.5f, second, best);
    }
  }
  const bool real = g < p.groups;
  int ahead = 0;
  for (int h = 0; h < p.groups; ++h) {
    const float other = __shfl_sync(kAll, best, h * lanes);
    ahead += other > best || (other == best && h < g);
  }
  const bool kept = real && best > none && ahead < p.topk_groups;
  if (near >= 0.0f) {
    const float least = of_key(__reduce_min_sync(kAll, kept ? key_of(best) : ~0u));
    const unsigned out = __reduce_max_sync(kAll, real && !kept ? key_of(best) : kNone);
    const float most = of_key(out), m = fmaxf(fabsf(most), __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(largest))));
    close = out != kNone && least - most <= near + kSumNear * m;
  }
  return kept;
}

// The groups that are kept, as bits; `values` are the warp's choice values.
__device__ unsigned keep_groups(const RouteParams& p, const float* values, float near, bool& close) {
  const int lane = threadIdx.x & 31, size = p.E / p.groups;
  float best = -inf(), second = -inf();
  if (lane < p.groups) {
    for (int i = 0; i < size; ++i) {
      const float v = values[place(lane * size + i)];
      second = fmaxf(second, fminf(best, v));
      best = fmaxf(best, v);
    }
  }
  return __ballot_sync(kAll, keeps_group(p, best, second, lane, 1, near, close));
}


__device__ __forceinline__ bool can_choose(float z, float b) { return z > -inf() && b > -inf(); }  // no NaN either

// An order-preserving integer of a double that is no NaN, above 0 unless it is -inf.
__device__ __forceinline__ unsigned long long key_of(double v) {
  if (v == -static_cast<double>(inf())) return 0ull;
  const unsigned long long u = __double_as_longlong(v + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}

// The groups that are kept, as bits; lane g has group g's best two keys (0: none).
__device__ __forceinline__ unsigned kept_by_key(const RouteParams& p, unsigned long long best, unsigned long long second) {
  const int lane = threadIdx.x & 31;
  const auto value = [](unsigned long long k) { return __longlong_as_double(k >> 63 ? k & ~(1ull << 63) : ~k); };
  if (p.group_best == 2 && second) best = key_of(value(best) + value(second));
  int ahead = 0;
  for (int h = 0; h < p.groups; ++h) {
    const unsigned long long other = __shfl_sync(kAll, best, h);
    ahead += other > best || (other == best && h < lane);
  }
  return __ballot_sync(kAll, lane < p.groups && best && ahead < p.topk_groups);
}

// A token's choice in 64 bits: lane k returns the k-th expert, or -1. (The SM has
// two units of 64-bit arithmetic: all but the scores and the groups' sums is done
// in integers.)
template <int V>
__device__ __noinline__ int choose_exactly(const RouteParams& p, int64_t token, unsigned long long* values) {
  const int lane = threadIdx.x & 31;
  float z[V];
  float top = -inf();
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * 32 + lane;
    z[j] = e < p.E ? logit(p, token * p.stride + e) : -inf();
    top = fmaxf(top, z[j]);
  }
  top = warp_max(top);
  double c[V], sum = 0.0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    c[j] = z[j] == top && !p.sigmoid ? 1.0 : exp(p.sigmoid ? -static_cast<double>(z[j]) : static_cast<double>(z[j]) - top);
    if (z[j] != z[j]) c[j] = 0.0;
    sum += c[j];
  }
  if (!p.sigmoid) sum = warp_sum(sum);
  unsigned long long key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * 32 + lane;
    const float b = e < p.E && p.bias ? __ldg(p.bias + e) : 0.0f;
    key[j] = 0ull;
    if (e < p.E && can_choose(z[j], b)) key[j] = key_of((p.sigmoid ? 1.0 / (1.0 + c[j]) : c[j] / sum) + b);
  }
  if (p.groups > 1) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane < p.E) values[place(j * 32 + lane)] = key[j];
    __syncwarp();
    const int size = p.E / p.groups;
    unsigned long long best = 0ull, second = 0ull;
    if (lane < p.groups) {
      for (int i = 0; i < size; ++i) {
        const unsigned long long v = values[place(lane * size + i)], low = min(v, best);
        best = max(v, best);
        second = max(second, low);
      }
    }
    const unsigned kept = kept_by_key(p, best, second);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * 32 + lane;
      if (e >= p.E || !(kept >> (e / size) & 1)) key[j] = 0ull;
      // Within the groups, without a bias, the logits say it, however close the scores.
      if (!p.bias && key[j]) key[j] = key_of(static_cast<double>(z[j]));
    }
  }
  int mine = -1;
  for (int k = 0; k < p.K; ++k) {
    unsigned long long best = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) best = max(best, key[j]);
    const unsigned high = __reduce_max_sync(kAll, static_cast<unsigned>(best >> 32));
    const unsigned low = __reduce_max_sync(kAll, best >> 32 == high ? static_cast<unsigned>(best) : 0u);
    const unsigned long long most = static_cast<unsigned long long>(high) << 32 | low;
    if (!most) break;
    unsigned at = ~0u;
#pragma unroll
    for (int j = V - 1; j >= 0; --j)
      if (key[j] == most) at = j * 32 + lane;
    at = __reduce_min_sync(kAll, at);
    if (lane == k) mine = at;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * 32 + lane == at) key[j] = 0ull;
  }
  return mine;
}

// What a token's softmax in 64 bits is divided by, and its largest logit.
template <int V>
__device__ __forceinline__ double exact_sum(const RouteParams& p, int64_t row, float& top) {
  const int lane = threadIdx.x & 31;
  top = 0.0f;
  if (p.sigmoid) return 1.0;
  float z[V];
  top = -inf();
#pragma unroll
  for (int j = 0; j < V; ++j) {
    z[j] = j * 32 + lane < p.E ? logit(p, row + j * 32 + lane) : -inf();
    top = fmaxf(top, z[j]);
  }
  top = warp_max(top);
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < V; ++j) sum += z[j] == top ? 1.0 : z[j] != z[j] ? 0.0 : exp(static_cast<double>(z[j]) - top);
  return warp_sum(sum);
}

// The key in 64 bits of expert e, which can be chosen.
__device__ __forceinline__ unsigned long long exact_key(const RouteParams& p, int64_t row, int e, float top, double sum) {
  const float z = logit(p, row + e);
  const double c = p.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(z)))
                             : (z == top ? 1.0 : exp(static_cast<double>(z) - top)) / sum;
  return key_of(c + (p.bias ? __ldg(p.bias + e) : 0.0f));
}

// The groups that are kept, as bits, by sums in 64 bits of the experts that can be
// among their groups' best; 0 if these are more than 32.
template <int V>
__device__ __noinline__ unsigned keep_groups_exactly(const RouteParams& p, int64_t token, Scorer score, float near,
                                                     unsigned long long* shared) {
  const int lane = threadIdx.x & 31, size = p.E / p.groups;
  const int64_t row = token * p.stride;
  float* values = reinterpret_cast<float*>(shared);
  int* list = reinterpret_cast<int*>(values + p.E + p.E / 32 + 1);
  float c[V];
  __syncwarp();
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * 32 + lane;
    c[j] = -inf();
    if (e < p.E) {
      const float z = logit(p, row + e), b = p.bias ? __ldg(p.bias + e) : 0.0f;
      if (can_choose(z, b)) c[j] = score(z) + b;
      values[place(e)] = c[j];
    }
  }
  __syncwarp();
  float best = -inf(), second = -inf();
  if (lane < p.groups) {
    for (int i = 0; i < size; ++i) {
      const float v = values[place(lane * size + i)];
      second = fmaxf(second, fminf(best, v));
      best = fmaxf(best, v);
    }
  }
  const float last = p.group_best == 2 && second > -inf() ? second : best;
  const float least = last == inf() ? last : last - (near + kSumNear * fabsf(last));
  int count = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * 32 + lane;
    const float of_group = __shfl_sync(kAll, least, min(e, p.E - 1) / size);
    const unsigned some = __ballot_sync(kAll, c[j] > -inf() && c[j] >= of_group);
    const int at = count + __popc(some & lanemask_lt());
    if ((some >> lane & 1) && at < 32) list[at] = e;
    count += __popc(some);
  }
  __syncwarp();
  if (count > 32) return 0u;
  float top;
  const double sum = exact_sum<V>(p, row, top);
  const int e = lane < count ? list[lane] : -1, group = lane < count ? e / size : -1;
  const unsigned long long key = lane < count ? exact_key(p, row, e, top, sum) : 0ull;
  unsigned long long first = 0ull, next = 0ull;
  for (int h = 0; h < count; ++h) {
    const unsigned long long other = __shfl_sync(kAll, key, h);
    if (__shfl_sync(kAll, group, h) == lane) {
      next = max(next, min(first, other));
      first = max(first, other);
    }
  }
  return kept_by_key(p, first, next);
}

// The first `count` lanes' experts in the order of their values in 64 bits: lane k
// returns the k-th, or -1.
template <int V>
__device__ __noinline__ int order_exactly(const RouteParams& p, int64_t token, int mine, int count) {
  const int lane = threadIdx.x & 31;
  const int64_t row = token * p.stride;
  float top;
  const double sum = exact_sum<V>(p, row, top);
  const unsigned long long key = lane < count ? exact_key(p, row, mine, top, sum) : 0ull;
  int ahead = 0;
  for (int h = 0; h < count; ++h) {
    const unsigned long long other = __shfl_sync(kAll, key, h);
    const int e = __shfl_sync(kAll, mine, h);
    ahead += other > key || (other == key && e < mine);
  }
  int result = -1;
  for (int k = 0; k < min(p.K, count); ++k) {
    const int from = __ffs(__ballot_sync(kAll, lane < count && ahead == k)) - 1;
    const int e = __shfl_sync(kAll, mine, from);
    if (lane == k) result = e;
  }
  return result;
}

size_t values_bytes(const RouteParams& p) {
  return p.groups > 1 ? sizeof(unsigned long long) * kWarps * (p.E + p.E / 32 + 1) : 0;
}

// A lane's V experts, lane * V and on, of one row: 16 bytes at a time where the
// row allows it (`vec`). Places behind the last expert hold `none`.
template <int V>
__device__ __forceinline__ void load_row(const RouteParams& p, const void* from, int64_t row, bool bf16, bool vec,
                                         float none, float (&z)[V]) {
  const int e0 = (threadIdx.x & 31) * V;
  if (V >= 4 && vec) {
    if (e0 >= p.E) {
#pragma unroll
      for (int j = 0; j < V; ++j) z[j] = none;
    } else if (bf16) {
      const uint2* at = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(from) + row + e0);
#pragma unroll
      for (int j = 0; j + 3 < V; j += 4) {
        const uint2 v = __ldg(at + j / 4);
        z[j] = bf16_lo(v.x), z[j + 1] = bf16_hi(v.x), z[j + 2] = bf16_lo(v.y), z[j + 3] = bf16_hi(v.y);
      }
    } else {
      const float4* at = reinterpret_cast<const float4*>(static_cast<const float*>(from) + row + e0);
#pragma unroll
      for (int j = 0; j + 3 < V; j += 4) {
        const float4 v = __ldg(at + j / 4);
        z[j] = v.x, z[j + 1] = v.y, z[j + 2] = v.z, z[j + 3] = v.w;
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = e0 + j;
    z[j] = e >= p.E ? none
           : bf16   ? bf16_lo(__ldg(static_cast<const uint16_t*>(from) + row + e))
                    : __ldg(static_cast<const float*>(from) + row + e);
  }
}

template <int V>
__device__ __forceinline__ void store_row(const RouteParams& p, void* to, int64_t row, bool bf16, bool vec,
                                          const float (&v)[V]) {
  const int e0 = (threadIdx.x & 31) * V;
  if (V >= 4 && vec) {
    if (e0 >= p.E) return;
#pragma unroll
    for (int j = 0; j + 3 < V; j += 4) {
      if (bf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(to) + row + e0 + j) =
            make_uint2(pack_bf16x2(v[j], v[j + 1]), pack_bf16x2(v[j + 2], v[j + 3]));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(to) + row + e0 + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (e0 + j >= p.E) break;
    if (bf16)
      static_cast<__nv_bfloat16*>(to)[row + e0 + j] = __float2bfloat16(v[j]);
    else
      static_cast<float*>(to)[row + e0 + j] = v[j];
  }
}

// Keys down, the lower place first where two are equal, and their places with them.
template <int V>
__device__ __forceinline__ void sort_down(unsigned (&key)[V], unsigned& order) {
  unsigned at[V];
#pragma unroll
  for (int j = 0; j < V; ++j) at[j] = j;
  // Odd-even merge sort's exchanges; equal keys keep their order by comparing places too.
  const auto exchange = [&](int i, int j) {
    const bool swap = key[j] > key[i] || (key[j] == key[i] && at[j] < at[i]);
    const unsigned k = key[i], a = at[i];
    key[i] = swap ? key[j] : k;
    at[i] = swap ? at[j] : a;
    key[j] = swap ? k : key[j];
    at[j] = swap ? a : at[j];
  };
  if (V == 2) exchange(0, 1);
  if (V == 4 || V == 8) {
#pragma unroll
    for (int o = 0; o < V; o += 4) {
      exchange(o, o + 1);
      exchange(o + 2, o + 3);
      exchange(o, o + 2);
      exchange(o + 1, o + 3);
      exchange(o + 1, o + 2);
    }
  }
  if (V == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) exchange(i, i + 4);
    exchange(2, 4);
    exchange(3, 5);
    exchange(1, 2);
    exchange(3, 4);
    exchange(5, 6);
  }
  order = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) order |= at[j] << (4 * (j & 7));
}

// V: experts a lane. (Ten blocks an SM for up to 256 experts, in 48 registers, of which
// V = 8 spills 144 bytes and V = 4 68. With seven blocks and 72 registers, without
// spills to speak of, softmax alone took 17.4 us instead of 16.4 for 16384 tokens and 128
// instead of 116 for 131072; with groups and a bias 156 instead of 149 to 154.)
template <int V>
__global__ void __launch_bounds__(kWarps * 32, V <= 8 ? 10 : V == 16 ? 4 : 3) route_kernel(const RouteParams p) {
  extern __shared__ unsigned long long shared_values[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, e0 = lane * V;
  unsigned long long* values = shared_values + w * (p.E + p.E / 32 + 1);
  grid_dependency_wait();
  launch_dependents();
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kWarps + w;
  if (token >= p.N) return;
  const int64_t row = token * p.stride;
  float z[V], b[V];
  load_row(p, p.logits, row, p.bf16, p.vec_logits, -inf(), z);
  if (p.bias)
    load_row(p, p.bias, 0, false, p.vec_bias, 0.0f, b);
  else
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = 0.0f;
  const Scorer score = scorer(p, z);
  // By what experts are chosen: the logits, or the biased scores.
  const bool by_score = p.bias || (p.groups > 1 && p.group_best == 2);
  const float near = p.sigmoid ? kSigmoidNear : kSoftmaxNear * score.inverse;  // (the largest score is 1 / sum)
  float c[V];
#pragma unroll
  for (int j = 0; j < V; ++j) c[j] = by_score || p.scores ? score(z[j]) : 0.0f;
  if (p.scores) store_row(p, p.scores, token * p.E, false, p.vec_scores, c);
  unsigned key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float v = by_score ? c[j] + b[j] : z[j];
    c[j] = can_choose(z[j], b[j]) ? v : -inf();
    key[j] = key_of(p.bias ? c[j] : c[j] > -inf() ? z[j] : -inf());
  }
  bool all = false;  // the whole token is to be done again
  if (p.groups > 1) {
    const unsigned size = p.E / p.groups, lanes = size / V;
    const float group_near = by_score ? 2.0f * near : -1.0f;
    bool close = false;
    const auto exactly = [&]() {
      const unsigned kept = keep_groups_exactly<V>(p, token, score, near, values);
      all = kept == 0u;
      return kept;
    };
    if (lanes * V == size && (lanes & (lanes - 1)) == 0) {
      // A group is a power of two of lanes: its best two by exchanges among them.
      float best = -inf(), second = -inf();
#pragma unroll
      for (int j = 0; j < V; ++j) {
        second = fmaxf(second, fminf(best, c[j]));
        best = fmaxf(best, c[j]);
      }
      for (unsigned o = 1; o < lanes; o <<= 1) {
        const float other = __shfl_xor_sync(kAll, best, o), other_second = __shfl_xor_sync(kAll, second, o);
        second = fmaxf(fminf(best, other), fmaxf(second, other_second));
        best = fmaxf(best, other);
      }
      const int group = e0 < p.E ? e0 / size : p.groups;
      bool kept = keeps_group(p, best, second, group, lanes, group_near, close);
      if (close) kept = exactly() >> (group & 31) & 1;
      if (!kept) {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = kNone;
      }
    } else {
      float* group_values = reinterpret_cast<float*>(values);
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (e0 + j < p.E) group_values[place(e0 + j)] = c[j];
      __syncwarp();
      unsigned kept = keep_groups(p, group_values, group_near, close);
      if (close) kept = exactly();
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (e0 + j >= p.E || !(kept >> ((e0 + j) / size) & 1)) key[j] = kNone;
    }
  }
  // Each lane's experts best first, `order` their places, four bits each: from
  // there on a lane shows its first alone, and the one that is taken is dropped.
  unsigned order = 0x76543210u;
  if (V <= 8) sort_down(key, order);
  int mine = -1, taken = 0;
  unsigned value = kNone;  // the key of the k-th taken, in lane k
  const auto largest = [&]() {
    unsigned best = key[0];
    if (V > 8) {
#pragma unroll
      for (int j = 1; j < V; ++j) best = max(best, key[j]);
    }
    return best;
  };
  const auto take = [&](unsigned best, unsigned most) {
    // Lower lanes hold lower indices.
    const int owner = __ffs(__ballot_sync(kAll, best == most)) - 1;
    int at = order & 15;
    if (V > 8) {
#pragma unroll
      for (int j = V - 1; j >= 0; --j)
        if (key[j] == most) at = j;
    }
    const int e = owner * V + __shfl_sync(kAll, at, owner);
    if (lane == taken) {
      mine = e;
      value = most;
    }
    if (V > 8) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (e0 + j == e) key[j] = kNone;
    } else if (lane == owner) {
#pragma unroll
      for (int j = 0; j + 1 < V; ++j) key[j] = key[j + 1];
      key[V - 1] = kNone;
      order >>= 4;
    }
    ++taken;
  };
  if (!all) {
    unsigned most = kNone;
    while (taken < p.K) {
      const unsigned best = largest();
      const unsigned next = __reduce_max_sync(kAll, best);
      if (next == kNone) break;
      most = next;
      take(best, most);
    }
    // What is as near to the last one as two scores' errors is taken too.
    while (p.bias) {
      const unsigned best = largest();
      const unsigned next = __reduce_max_sync(kAll, best);
      const float kth = of_key(most), v = of_key(next);
      if (next == kNone || !(kth - v <= near + kSumNear * fmaxf(fabsf(kth), fabsf(v)))) break;
      all = taken == 32;
      if (all) break;
      take(best, next);
    }
  }
  if (all) {
    mine = choose_exactly<V>(p, token, values);
  } else if (p.bias) {
    const float v = of_key(value), n = of_key(__shfl_down_sync(kAll, value, 1));
    const bool near_next = lane + 1 < taken && v - n <= near + kSumNear * fmaxf(fabsf(v), fabsf(n));
    if (__any_sync(kAll, near_next)) mine = order_exactly<V>(p, token, mine, taken);
  }
  float s = mine >= 0 ? score(logit(p, row + mine)) : 0.0f;
  if (p.renormalize) s = s / (warp_sum(s) + kTiny);
  if (lane < p.K) {
    p.idx[token * p.K + lane] = mine;
    p.weights[token * p.K + lane] = s * p.scale;
  }
}

template <int V>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(const RouteParams p) {
  const int lane = threadIdx.x & 31, e0 = lane * V;
  grid_dependency_wait();
  launch_dependents();
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (token >= p.N) return;
  const int64_t row = token * p.stride;
  float s[V], d[V];
  load_row(p, p.logits, row, p.bf16, p.vec_logits, -inf(), s);
  // Lane k has the k-th chosen expert.
  int e = -1;
  float dw = 0.0f, z = 0.0f;
  if (lane < p.K) {
    e = __ldg(p.chosen + token * p.K + lane);
    dw = __ldg(p.grad_weights + token * p.K + lane);
    if (e < -1 || e >= p.E) {
      flag(p.status, EP_ST_BAD_INDEX);
      e = -1;
    }
  }
  if (p.grad_scores) {
    load_row(p, p.grad_scores, token * p.E, false, p.vec_scores, 0.0f, d);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = 0.0f;
  }
  if (e >= 0) z = logit(p, row + e);
  dw = e >= 0 ? dw * p.scale : 0.0f;
  const Scorer score = scorer(p, s);
  if (p.renormalize) {
    // Where one score has most of the sum, gradients relative to its own: its own less the
    // mean would be a difference of nearly equal numbers. (Where none has, the mean is no
    // one's, and a difference from some large gradient would cost the small ones their bits.)
    const float w = e >= 0 ? score(z) : 0.0f;
    const float sum = warp_sum(w) + kTiny;
    const unsigned bits = __float_as_uint(w), most = __reduce_max_sync(kAll, bits);
    float base = __shfl_sync(kAll, dw, __ffs(__ballot_sync(kAll, bits == most)) - 1);
    if (__uint_as_float(most) <= 0.5f * sum) base = 0.0f;
    dw = e >= 0 ? dw - base : 0.0f;
    dw = (dw - warp_sum(dw * (w / sum)) + base * (kTiny / sum)) / sum;  // (the quotients add up to 1 - kTiny / sum)
  }
  for (int k = 0; k < p.K; ++k) {
    const int at = __shfl_sync(kAll, e, k) - e0;
    const float add = __shfl_sync(kAll, dw, k);
    if (at >= 0 && at < V) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j == at) d[j] += add;
    }
  }
  // (An expert that scores 0, or whose score does not move, moves nothing, whatever its gradient.)
  if (p.sigmoid) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float slope = sigmoid_slope(s[j]);
      d[j] = slope == 0.0f ? 0.0f : slope * d[j];
    }
  } else {
    float base = 0.0f, dot = 0.0f;
    if (score.inverse > 0.5f) {  // the largest score is most of their sum, 1: as above
      bool largest = false;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (s[j] == score.top) {
          base = d[j];
          largest = true;
        }
      }
      base = __shfl_sync(kAll, base, __ffs(__ballot_sync(kAll, largest)) - 1);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s[j] = score(s[j]);
      d[j] -= base;
      if (s[j] != 0.0f) dot += s[j] * d[j];
    }
    dot = warp_sum(dot);
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = s[j] == 0.0f ? 0.0f : s[j] * (d[j] - dot);
  }
  store_row(p, p.grad_logits, token * p.E, p.bf16, p.vec_grad, d);
}

template <int V>
cudaError_t launch(const RouteParams& p, bool backward, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.N) + kWarps - 1) / kWarps)), block(kWarps * 32);
  return backward ? launch_kernel(route_backward_kernel<V>, grid, block, 0, s, /*dependent=*/true, p)
                  : launch_kernel(route_kernel<V>, grid, block, values_bytes(p), s, /*dependent=*/true, p);
}

cudaError_t launch_any(RouteParams p, bool backward, cudaStream_t s) {
  if (p.N <= 0) return cudaSuccess;
  const int per = (p.E + 31) / 32;
  // Rows of whole sixteen bytes (of eight in BF16), and a lane's experts all there or none.
  const int unit = per <= 4 ? 4 : per <= 8 ? 8 : per <= 16 ? 16 : 32;
  const bool whole = p.E % unit == 0;
  const auto vec = [&](const void* at, int64_t stride, bool bf16) {
    return whole && stride % 4 == 0 && reinterpret_cast<uintptr_t>(at) % (bf16 ? 8 : 16) == 0;
  };
  p.vec_logits = vec(p.logits, p.N > 1 ? p.stride : 0, p.bf16);
  p.vec_bias = vec(p.bias, 0, false);
  p.vec_scores = vec(backward ? static_cast<const void*>(p.grad_scores) : p.scores, p.E, false);
  p.vec_grad = vec(p.grad_logits, p.E, p.bf16);
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
