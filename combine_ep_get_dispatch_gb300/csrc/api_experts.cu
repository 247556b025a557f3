// The C ABI of the router and of the experts' products with 8-bit weights
// (include/ep.h): argument checks and kernel launches. No entry point
// allocates, frees or synchronises.
#include <math.h>
#include <stdint.h>

#include "ep.h"
#include "kernels.cuh"

namespace {

using namespace ep;

inline bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) == 0; }
int cuda_rc(cudaError_t e) { return e == cudaSuccess ? EP_OK : EP_ERR_CUDA; }

// Sizes that ep_route and ep_route_backward share; fills p.
int route_setup(const void* logits, int flags, int64_t stride, int N, int E, int K, float scale, RouteParams& p) {
  if (flags & ~(EP_ROUTE_BF16 | EP_ROUTE_SIGMOID | EP_ROUTE_RENORMALIZE)) return EP_ERR_INVALID_ARG;
  if (N < 0 || E < 1 || E > EP_MAX_EXPERTS || K < 1 || K > EP_MAX_TOPK || K > E || !isfinite(scale))
    return EP_ERR_INVALID_ARG;
  if (N > 0 && (!logits || (N > 1 && stride < E))) return EP_ERR_INVALID_ARG;
  if (!aligned(logits, flags & EP_ROUTE_BF16 ? 2 : 4)) return EP_ERR_ALIGNMENT;
  p = RouteParams{};
  p.logits = logits;
  p.stride = stride;
  p.N = N;
  p.E = E;
  p.K = K;
  p.bf16 = (flags & EP_ROUTE_BF16) != 0;
  p.sigmoid = (flags & EP_ROUTE_SIGMOID) != 0;
  p.renormalize = (flags & EP_ROUTE_RENORMALIZE) != 0;
  p.scale = scale;
  return EP_OK;
}

bool linear_fp8_sizes_ok(int E, int64_t max_rows) {
  return E >= 1 && E <= EP_MAX_EXPERTS && max_rows >= 0 && max_rows <= (INT32_MAX >> 4);
}

}  // namespace

extern "C" {

int ep_route(const void* logits, int64_t logits_stride, int num_tokens, int num_experts, int num_topk, const float* bias,
             int num_groups, int topk_groups, int group_best, int flags, float scale, int32_t* topk_idx,
             float* topk_weights, float* scores, void* stream) {
  RouteParams p{};
  const int rc = route_setup(logits, flags, logits_stride, num_tokens, num_experts, num_topk, scale, p);
  if (rc != EP_OK) return rc;
  if (num_groups < 1 || num_groups > EP_MAX_ROUTE_GROUPS || num_experts % num_groups != 0) return EP_ERR_INVALID_ARG;
  if (topk_groups < 1 || topk_groups > num_groups || group_best < 1 || group_best > 2) return EP_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!topk_idx || !topk_weights)) return EP_ERR_INVALID_ARG;
  if (!aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_weights, 4) || !aligned(scores, 4))
    return EP_ERR_ALIGNMENT;
  p.bias = bias;
  p.groups = topk_groups < num_groups ? num_groups : 1;  // with every group kept there is nothing to choose
  p.topk_groups = topk_groups;
  p.group_best = group_best;
  p.idx = topk_idx;
  p.weights = topk_weights;
  p.scores = scores;
  return cuda_rc(launch_route(p, static_cast<cudaStream_t>(stream)));
}

int ep_route_backward(const float* grad_weights, const float* grad_scores, const void* logits, int64_t logits_stride,
                      const int32_t* topk_idx, int num_tokens, int num_experts, int num_topk, int flags, float scale,
                      void* grad_logits, int32_t* status, void* stream) {
  RouteParams p{};
  const int rc = route_setup(logits, flags, logits_stride, num_tokens, num_experts, num_topk, scale, p);
  if (rc != EP_OK) return rc;
  if (num_tokens > 0 && (!grad_weights || !topk_idx || !grad_logits)) return EP_ERR_INVALID_ARG;
  if (!aligned(grad_weights, 4) || !aligned(grad_scores, 4) || !aligned(topk_idx, 4) || !aligned(grad_logits, p.bf16 ? 2 : 4))
    return EP_ERR_ALIGNMENT;
  p.grad_weights = grad_weights;
  p.grad_scores = grad_scores;
  p.chosen = topk_idx;
  p.grad_logits = grad_logits;
  p.status = status;
  return cuda_rc(launch_route_backward(p, static_cast<cudaStream_t>(stream)));
}

size_t ep_expert_linear_fp8_workspace_bytes(int num_experts, int64_t max_rows) {
  if (!linear_fp8_sizes_ok(num_experts, max_rows)) return 0;
  return expert_linear_fp8_ws_bytes(num_experts, max_rows);
}

int ep_expert_linear_fp8(const uint8_t* x, const void* x_scale, int64_t x_rows, int in_features,
                         const int32_t* row_count, const int32_t* row_offset, int64_t rows_per_expert, int num_experts,
                         int64_t max_rows, const uint8_t* w, const float* w_scale, int out_features, int flags, void* y,
                         void* y_scale, void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  constexpr int kKnown = EP_LINEAR_GLU | EP_LINEAR_TRANSPOSED | EP_LINEAR_X_UE8M0 | EP_LINEAR_OUT_FP8 |
                         EP_LINEAR_OUT_ROUND_SCALE | EP_LINEAR_OUT_UE8M0;
  if (!linear_fp8_sizes_ok(num_experts, max_rows) || x_rows < 0 || x_rows > INT32_MAX) return EP_ERR_INVALID_ARG;
  if (flags & ~kKnown) return EP_ERR_INVALID_ARG;
  const bool glu = flags & EP_LINEAR_GLU, transposed = flags & EP_LINEAR_TRANSPOSED, fp8 = flags & EP_LINEAR_OUT_FP8;
  if ((glu && transposed) || (!fp8 && (flags & (EP_LINEAR_OUT_ROUND_SCALE | EP_LINEAR_OUT_UE8M0))))
    return EP_ERR_INVALID_ARG;
  if (in_features < 128 || in_features > EP_MAX_HIDDEN || in_features % 128 != 0) return EP_ERR_INVALID_ARG;
  const int unit = (fp8 || transposed ? 128 : 8) * (glu ? 2 : 1);
  if (out_features < unit || out_features > (1 << 20) || out_features % unit != 0) return EP_ERR_INVALID_ARG;
  if (!expert_linear_fp8_units_ok(num_experts, max_rows, out_features, glu)) return EP_ERR_INVALID_ARG;
  if (!row_offset && (rows_per_expert < 0 || rows_per_expert > INT32_MAX)) return EP_ERR_INVALID_ARG;
  if (!row_count || !w || !w_scale) return EP_ERR_INVALID_ARG;
  if (x_rows > 0 && max_rows > 0 && (!x || !x_scale || !y || (fp8 && !y_scale))) return EP_ERR_INVALID_ARG;
  const bool x_ue8m0 = flags & EP_LINEAR_X_UE8M0, out_ue8m0 = flags & EP_LINEAR_OUT_UE8M0;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(w_scale, 4) ||
      !aligned(x_scale, x_ue8m0 ? 1 : 4) || !aligned(y_scale, out_ue8m0 ? 1 : 4))
    return EP_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < expert_linear_fp8_ws_bytes(num_experts, max_rows)) return EP_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return EP_ERR_ALIGNMENT;
  ExpertLinearFp8Params p{};
  p.x = x;
  p.x_scale = x_scale;
  p.x_rows = x_rows;
  p.count = row_count;
  p.offset = row_offset;
  p.region = rows_per_expert;
  p.E = num_experts;
  p.K = in_features;
  p.M = out_features;
  p.glu = glu;
  p.transposed = transposed;
  p.x_ue8m0 = x_ue8m0;
  p.out_fp8 = fp8;
  p.out_pow2 = (flags & (EP_LINEAR_OUT_ROUND_SCALE | EP_LINEAR_OUT_UE8M0)) != 0;
  p.out_ue8m0 = out_ue8m0;
  p.max_rows = max_rows;
  p.w = w;
  p.w_scale = w_scale;
  p.y = y;
  p.y_scale = y_scale;
  p.ws = static_cast<uint8_t*>(workspace);
  p.status = status;
  return cuda_rc(launch_expert_linear_fp8(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
