// The experts' products with 4-bit weights on sm_103a: y_row = x_row W_e^T.
//
// This form: a block for 4 outputs of an expert, a warp each (with GLU, a
// gate and its up); every row in turn, fp32 fused multiply-adds.
#include "common.cuh"
#include "kernels.cuh"

namespace ep {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float e2m1(unsigned c) {
  const unsigned m = c & 7u;
  const float v = m < 2u ? 0.5f * m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
  return c & 8u ? -v : v;
}

__device__ __forceinline__ float ue8m0(unsigned b) {
  if (b == 255u) return __uint_as_float(0x7FC00000u);
  return b ? __uint_as_float(b << 23) : __uint_as_float(0x00400000u);
}

__device__ __forceinline__ float x_value(const ExpertLinearParams& p, int64_t row, int k) {
  if (!p.x_scale) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p.x)[row * p.K + k]) << 16);
  uint32_t f2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f2) : "h"(static_cast<uint16_t>(static_cast<const uint8_t*>(p.x)[row * p.K + k])));
  return __low2float(*reinterpret_cast<const __half2*>(&f2)) * ue8m0(p.x_scale[row * (p.K / 128) + k / 128]);
}

__device__ float dot(const ExpertLinearParams& p, int e, int m, int64_t row, int lane) {
  const uint8_t* w = p.w + (static_cast<int64_t>(e) * p.M + m) * (p.K / 2);
  const uint8_t* ws = p.w_scale + (static_cast<int64_t>(e) * p.M + m) * (p.K / 32);
  float acc = 0.0f;
  for (int k = 2 * lane; k < p.K; k += 64) {
    const unsigned c = w[k / 2];
    const float s = ue8m0(ws[k / 32]);
    acc = fmaf(x_value(p, row, k), e2m1(c & 15u) * s, acc);
    acc = fmaf(x_value(p, row, k + 1), e2m1(c >> 4) * s, acc);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  return acc;
}

__global__ void __launch_bounds__(kThreads) expert_linear_kernel(const ExpertLinearParams p) {
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  const int outs = p.glu ? p.M / 2 : p.M;
  const int m = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), e = blockIdx.y;
  if (m >= outs) return;
  const int n = p.count[e];
  const int64_t first = p.offset ? p.offset[e] : e * p.region;
  int64_t before = 0;  // rows of the experts before this one
  for (int i = 0; i < e; ++i) before += p.offset ? max(0, p.count[i]) : min(p.region, static_cast<int64_t>(max(0, p.count[i])));
  for (int j = 0; j < n; ++j) {
    const int64_t row = first + j;
    if (row < 0 || row >= p.x_rows || (!p.offset && j >= p.region) || before + j >= p.max_rows) {
      flag(p.status, EP_ST_CAPACITY);
      break;
    }
    float v = dot(p, e, m, row, lane);
    if (p.glu) {
      const float u = dot(p, e, m + outs, row, lane);
      v = v / (1.0f + expf(-v)) * u;
    }
    if (lane == 0) reinterpret_cast<__nv_bfloat16*>(p.y)[row * outs + m] = __float2bfloat16(v);
  }
}

}  // namespace

size_t expert_linear_ws_bytes(int, int64_t, int, bool) { return 256; }

cudaError_t launch_expert_linear(const ExpertLinearParams& p, cudaStream_t s) {
  if (p.max_rows <= 0 || p.x_rows <= 0) return cudaSuccess;
  const int outs = p.glu ? p.M / 2 : p.M;
  return launch_kernel(expert_linear_kernel, dim3((outs + 3) / 4, p.E), dim3(kThreads), 0, s, /*dependent=*/true, p);
}

}  // namespace ep
