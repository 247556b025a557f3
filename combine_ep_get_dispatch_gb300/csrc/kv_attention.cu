// Attention of a call's new tokens over the paged E4M3 cache on sm_103a.
//
// Mathematics: for a query row, running maximum m and sum l over the keys seen
// so far, s_j = scale <q, k_j>: each key rescales what was summed by
// exp(m - m') and adds exp(s_j - m') (and that times v_j); out = o / l and
// lse = m + log(l). Key and value blocks enter as code * scale.
//
// This form: a warp for each (token, query head), a lane D / 32 channels.
#include "common.cuh"
#include "kernels.cuh"

namespace ep {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float decode1(uint8_t c) {
  uint32_t f2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f2) : "h"(static_cast<uint16_t>(c)));
  return __low2float(*reinterpret_cast<const __half2*>(&f2));
}

template <int kD>
__global__ void __launch_bounds__(kThreads) kv_attention_kernel(const KVAttentionParams p) {
  constexpr int kC = kD / 32;
  const KVParams& c = p.c;
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  if (c.cu && blockIdx.x == 0)
    for (int b = threadIdx.x; b < c.B; b += kThreads)
      if (c.cu[b] < 0 || c.cu[b + 1] < c.cu[b] || c.cu[b + 1] > c.N) flag(c.status, EP_ST_BAD_INDEX);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = i / p.QH;
  const int h = static_cast<int>(i % p.QH);
  if (t >= c.N) return;
  int b = static_cast<int>(t), t0 = b, n = 1;
  if (c.cu) {
    int lo = 0, hi = c.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (__ldg(c.cu + mid) <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    t0 = __ldg(c.cu + b);
    n = __ldg(c.cu + b + 1) - t0;
    if (t0 < 0 || n < 0 || t0 + static_cast<int64_t>(n) > c.N) {
      flag(c.status, EP_ST_BAD_INDEX);
      n = 0;
    }
  }
  int len = __ldg(c.lens + b);
  int64_t last = static_cast<int64_t>(len) - n + (t - t0);  // the token's position
  if (t >= t0 + static_cast<int64_t>(n) || t < t0) last = -1;
  const int64_t cap = static_cast<int64_t>(c.MP) * c.P;
  if (len > cap) flag(c.status, EP_ST_CAPACITY);
  const int64_t stop = last + 1 < cap ? last + 1 : cap;
  int64_t j = p.window > 0 && last - p.window + 1 > 0 ? last - p.window + 1 : 0;
  const int kvh = h / p.G;
  float q[kC], o[kC], m = -INFINITY, l = 0.0f;
  const __nv_bfloat16* qp = reinterpret_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride + h * kD + lane * kC;
#pragma unroll
  for (int x = 0; x < kC; ++x) {
    q[x] = __bfloat162float(qp[x]) * p.scale_log2;
    o[x] = 0.0f;
  }
  while (j < stop) {
    const int64_t end = min(stop, ((j >> c.log2P) + 1) << c.log2P);
    const int page = __ldg(c.table + static_cast<int64_t>(b) * c.MP + (j >> c.log2P));
    if (page < 0 || page >= c.pages) {
      flag(c.status, EP_ST_BAD_INDEX);
      j = end;
      continue;
    }
    const int64_t block = static_cast<int64_t>(page) * c.KH + kvh;
    const float ks = c.k_scale[block], vs = c.v_scale[block];
    for (; j < end; ++j) {
      const int64_t at = (block * c.P + (j & (c.P - 1))) * kD + lane * kC;
      float s = 0.0f;
#pragma unroll
      for (int x = 0; x < kC; ++x) s = fmaf(q[x], decode1(c.k[at + x]), s);
#pragma unroll
      for (int w = 16; w >= 1; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      s *= ks;
      const float m2 = fmaxf(m, s);
      const float alpha = m2 == -INFINITY ? 1.0f : exp2f(m - m2), e = m2 == -INFINITY ? 0.0f : exp2f(s - m2);
      l = l * alpha + e;
#pragma unroll
      for (int x = 0; x < kC; ++x) o[x] = fmaf(e, decode1(c.v[at + x]) * vs, o[x] * alpha);
      m = m2;
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  __nv_bfloat16* op = reinterpret_cast<__nv_bfloat16*>(p.out) + (t * p.QH + h) * kD + lane * kC;
#pragma unroll
  for (int x = 0; x < kC; ++x) op[x] = __float2bfloat16(o[x] * inv);
  if (p.lse && lane == 0) p.lse[t * p.QH + h] = (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

size_t kv_attention_ws_bytes(int, int, int, int) { return 256; }

cudaError_t launch_kv_attention(const KVAttentionParams& p, cudaStream_t s) {
  if (p.c.N <= 0) return cudaSuccess;
  const int64_t grid = (static_cast<int64_t>(p.c.N) * p.QH + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_kernel(p.c.D == 64 ? kv_attention_kernel<64> : kv_attention_kernel<128>,
                       dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, /*dependent=*/true, p);
}

}  // namespace ep
