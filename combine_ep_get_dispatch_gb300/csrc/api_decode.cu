// The C ABI of the decode step's operators (include/ep.h): argument checks
// and kernel launches. No entry point allocates, frees or synchronises.
#include <math.h>
#include <stdint.h>

#include "ep.h"
#include "kernels.cuh"

namespace {

using namespace ep;

inline bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) == 0; }
int cuda_rc(cudaError_t e) { return e == cudaSuccess ? EP_OK : EP_ERR_CUDA; }

// Checks of the cache and the call's tokens; fills p.
int cache_setup(const ep_kv_cache_t* C, const int32_t* seq_lens, const int32_t* cu_tokens, int N, int32_t* status,
                KVParams& p) {
  if (!C || N < 0) return EP_ERR_INVALID_ARG;
  const int P = C->page_size, D = C->head_dim;
  if (P != 16 && P != 32 && P != 64 && P != 128) return EP_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return EP_ERR_INVALID_ARG;
  if (C->num_pages < 0 || C->num_heads < 1 || C->num_heads > 1024 || C->num_seqs < 0 || C->max_pages < 0)
    return EP_ERR_INVALID_ARG;
  if (static_cast<int64_t>(C->max_pages) * P > INT32_MAX || C->num_seqs > (1 << 28)) return EP_ERR_INVALID_ARG;
  if (!cu_tokens && N != C->num_seqs) return EP_ERR_INVALID_ARG;
  if (N > 0) {
    if (!seq_lens || C->num_seqs < 1 || C->num_pages < 1) return EP_ERR_INVALID_ARG;
    if (static_cast<int64_t>(C->num_pages) * C->num_heads > INT32_MAX) return EP_ERR_INVALID_ARG;
    if (C->max_pages > 0 && !C->page_table) return EP_ERR_INVALID_ARG;
    if (!C->k || !C->v || !C->k_scale || !C->v_scale) return EP_ERR_INVALID_ARG;
  }
  if (!aligned(C->k, 16) || !aligned(C->v, 16)) return EP_ERR_ALIGNMENT;
  p = KVParams{};
  p.k = C->k;
  p.v = C->v;
  p.k_scale = C->k_scale;
  p.v_scale = C->v_scale;
  p.table = C->page_table;
  p.lens = seq_lens;
  p.cu = cu_tokens;
  p.pages = C->num_pages;
  p.KH = C->num_heads;
  p.P = P;
  p.D = D;
  p.B = C->num_seqs;
  p.MP = C->max_pages;
  p.log2P = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
  p.N = N;
  p.status = status;
  return EP_OK;
}

// Token rows of `heads` heads: the stride leaves room for them and keeps
// 16-byte vectors aligned.
bool stride_ok(int64_t stride, int64_t heads, int D) { return stride >= heads * D && stride % 8 == 0; }

bool linear_sizes_ok(int E, int64_t max_rows, int K) {
  return E >= 1 && E <= EP_MAX_EXPERTS && max_rows >= 0 && max_rows <= (INT32_MAX >> 4) && K >= 128 &&
         K <= EP_MAX_HIDDEN && K % 128 == 0;
}

}  // namespace

extern "C" {

int ep_kv_append(const ep_kv_cache_t* C, const int32_t* seq_lens, const int32_t* cu_tokens, int num_tokens,
                 const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q, int64_t q_stride,
                 void* q_out, int64_t q_out_stride, int num_q_heads, const float* rope, int rope_rows, int rope_dim,
                 int interleaved, int32_t* status, void* stream) {
  KVAppendParams p{};
  const int rc = cache_setup(C, seq_lens, cu_tokens, num_tokens, status, p.c);
  if (rc != EP_OK) return rc;
  const int D = C->head_dim;
  if (rope_dim < 0 || rope_dim > D || rope_dim % 16 != 0 || rope_rows < 0) return EP_ERR_INVALID_ARG;
  if ((rope_dim > 0) != (rope != nullptr)) return EP_ERR_INVALID_ARG;
  if ((q != nullptr) != (q_out != nullptr)) return EP_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!k || !v)) return EP_ERR_INVALID_ARG;
  if (!stride_ok(k_stride, C->num_heads, D) || !stride_ok(v_stride, C->num_heads, D)) return EP_ERR_INVALID_ARG;
  if (q) {
    if (num_q_heads < 1 || num_q_heads > 4096) return EP_ERR_INVALID_ARG;
    if (!stride_ok(q_stride, num_q_heads, D) || !stride_ok(q_out_stride, num_q_heads, D)) return EP_ERR_INVALID_ARG;
  }
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(rope, 16))
    return EP_ERR_ALIGNMENT;
  p.k_new = static_cast<const uint16_t*>(k);
  p.v_new = static_cast<const uint16_t*>(v);
  p.q = static_cast<const uint16_t*>(q);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_stride = q_stride;
  p.q_out_stride = q_out_stride;
  p.QH = q ? num_q_heads : 0;
  p.rope = rope;
  p.rope_rows = rope_rows;
  p.rot = rope_dim;
  p.interleaved = interleaved != 0;
  return cuda_rc(launch_kv_append(p, static_cast<cudaStream_t>(stream)));
}

size_t ep_kv_attention_workspace_bytes(int num_tokens, int num_q_heads, int num_heads, int head_dim) {
  if (num_tokens < 0 || num_heads < 1 || num_heads > 1024 || num_q_heads < 1 || num_q_heads > 4096 ||
      num_q_heads % num_heads != 0 || (head_dim != 64 && head_dim != 128))
    return 0;
  return kv_attention_ws_bytes(num_tokens, num_q_heads, num_heads, head_dim);
}

int ep_kv_attention(const ep_kv_cache_t* C, const int32_t* seq_lens, const int32_t* cu_tokens, int num_tokens,
                    const void* q, int64_t q_stride, int num_q_heads, float scale, int window, void* out, float* lse,
                    void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  KVAttentionParams p{};
  const int rc = cache_setup(C, seq_lens, cu_tokens, num_tokens, status, p.c);
  if (rc != EP_OK) return rc;
  const int D = C->head_dim;
  if (num_q_heads < 1 || num_q_heads > 4096 || num_q_heads % C->num_heads != 0 || window < 0)
    return EP_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, num_q_heads, D) || !isfinite(scale)) return EP_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!q || !out)) return EP_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16)) return EP_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kv_attention_ws_bytes(num_tokens, num_q_heads, C->num_heads, D))
    return EP_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return EP_ERR_ALIGNMENT;
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_stride;
  p.QH = num_q_heads;
  p.G = num_q_heads / C->num_heads;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.window = window;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.ws = static_cast<uint8_t*>(workspace);
  return cuda_rc(launch_kv_attention(p, static_cast<cudaStream_t>(stream)));
}

size_t ep_expert_linear_workspace_bytes(int num_experts, int64_t max_rows, int in_features, int x_is_fp8) {
  if (!linear_sizes_ok(num_experts, max_rows, in_features)) return 0;
  return expert_linear_ws_bytes(num_experts, max_rows, in_features, x_is_fp8 != 0);
}

int ep_expert_linear(const void* x, const uint8_t* x_scale, int64_t x_rows, int in_features,
                     const int32_t* row_count, const int32_t* row_offset, int64_t rows_per_expert, int num_experts,
                     int64_t max_rows, const uint8_t* w, const uint8_t* w_scale, int out_features, int flags, void* y,
                     void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  if (!linear_sizes_ok(num_experts, max_rows, in_features) || x_rows < 0) return EP_ERR_INVALID_ARG;
  if (flags & ~EP_LINEAR_GLU) return EP_ERR_INVALID_ARG;
  if (x_scale && x_rows > INT32_MAX) return EP_ERR_INVALID_ARG;
  const int glu = flags & EP_LINEAR_GLU;
  if (out_features < 8 || out_features > (1 << 20) || out_features % (glu ? 16 : 8) != 0) return EP_ERR_INVALID_ARG;
  if (!row_offset && (rows_per_expert < 0 || rows_per_expert > INT32_MAX)) return EP_ERR_INVALID_ARG;
  if (!row_count || !w || !w_scale) return EP_ERR_INVALID_ARG;
  if (x_rows > 0 && max_rows > 0 && (!x || !y)) return EP_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(w, 32) || !aligned(w_scale, 16)) return EP_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < expert_linear_ws_bytes(num_experts, max_rows, in_features, x_scale != nullptr))
    return EP_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return EP_ERR_ALIGNMENT;
  ExpertLinearParams p{};
  p.x = x;
  p.x_scale = x_scale;
  p.x_rows = x_rows;
  p.count = row_count;
  p.offset = row_offset;
  p.region = rows_per_expert;
  p.E = num_experts;
  p.K = in_features;
  p.M = out_features;
  p.glu = glu ? 1 : 0;
  p.max_rows = max_rows;
  p.w = w;
  p.w_scale = w_scale;
  p.y = static_cast<uint16_t*>(y);
  p.ws = static_cast<uint8_t*>(workspace);
  p.status = status;
  return cuda_rc(launch_expert_linear(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
