// Logits of the sparse-attention indexer over a paged key cache:
//   logits[r, t] = s_t * sum_h w[r, h] * max(0, q[r, h, :] . k[t, :]).
// One thread a (row, token): plain fp32.
#include <cuda_fp8.h>

#include "paged.cuh"

namespace ltk {
namespace paged {
namespace {

constexpr int kThreads = 128;

struct LogitsParams {
  topk_index_logits_args a;
  Rows R;
};

template <typename T>
__device__ __forceinline__ float as_float(T x) { return static_cast<float>(x); }

template <typename T>
__global__ void __launch_bounds__(kThreads) index_logits_kernel(const LogitsParams p) {
  __shared__ float q[128 * 128];
  dependent_wait();
  dependent_launch();
  const topk_index_logits_args& a = p.a;
  for (int64_t row = blockIdx.x; row < p.R.num_rows; row += gridDim.x) {
    const int len = row_length(p.R, row, threadIdx.x == 0);
    const T* qr = static_cast<const T*>(a.q) + row * a.q_row_stride;
    __syncthreads();
    for (int i = threadIdx.x; i < a.heads * a.dim; i += kThreads) q[i] = as_float(qr[(i / a.dim) * a.q_head_stride + i % a.dim]);
    __syncthreads();
    for (int t = threadIdx.x; t < len; t += kThreads) {
      int64_t block;
      int place;
      float sum = -INFINITY;
      if (locate(p.R, row_request(p.R, row), t, &block, &place)) {
        const T* k = static_cast<const T*>(a.keys) + block * a.key_block_stride + place * a.key_token_stride;
        sum = 0;
        for (int h = 0; h < a.heads; ++h) {
          float dot = 0;
          for (int d = 0; d < a.dim; ++d) dot += q[h * a.dim + d] * as_float(k[d]);
          sum += a.weights[row * a.weight_row_stride + h] * (dot < 0 ? 0 : dot);
        }
        if (a.key_scales) sum *= a.key_scales[block * a.scale_block_stride + place * a.scale_token_stride];
      }
      a.logits[row * a.logits_row_stride + t] = sum;
    }
  }
}

}  // namespace
}  // namespace paged
}  // namespace ltk

extern "C" int topk_index_logits(const topk_index_logits_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_index_logits_args& a = *args;
  int rc = check_rows(a.rows);
  if (rc != TOPK_OK) return rc;
  if (a.max_len < 1 || a.max_len > INT32_MAX || a.logits_row_stride < 0) return TOPK_ERR_INVALID_ARG;
  const int size = a.dtype == TOPK_DTYPE_F8E4M3 ? 1 : 2, piece = 16 / size;
  if (a.dtype != TOPK_DTYPE_F16 && a.dtype != TOPK_DTYPE_BF16 && a.dtype != TOPK_DTYPE_F8E4M3) return TOPK_ERR_UNSUPPORTED;
  if (a.heads < 1 || a.heads > 128 || a.dim < piece || a.dim > 128 || a.dim % piece != 0) return TOPK_ERR_UNSUPPORTED;
  if (a.rows.num_rows == 0) return TOPK_OK;
  rc = check_row_pointers(a.rows);
  if (rc != TOPK_OK) return rc;
  if (a.q == nullptr || a.weights == nullptr || a.keys == nullptr || a.logits == nullptr || a.workspace == nullptr)
    return TOPK_ERR_INVALID_ARG;
  if (misaligned(a.q, 16) || a.q_row_stride % piece || a.q_head_stride % piece || misaligned(a.keys, 16) ||
      a.key_block_stride % piece || a.key_token_stride % piece || misaligned(a.weights, 4) ||
      misaligned(a.key_scales, 4) || misaligned(a.logits, 4) || misaligned(a.workspace, 16))
    return TOPK_ERR_MISALIGNED;
  const int sms = num_sms();
  if (sms < 1) return TOPK_ERR_CUDA;
  LogitsParams p{};
  p.a = a;
  p.R = make_rows(a.rows, a.max_len, a.workspace);
  const int64_t grid = a.rows.num_rows < sms * 2 ? a.rows.num_rows : sms * 2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (size == 1) return launch(index_logits_kernel<__nv_fp8_e4m3>, p, grid, kThreads, 0, s);
  if (a.dtype == TOPK_DTYPE_F16) return launch(index_logits_kernel<__half>, p, grid, kThreads, 0, s);
  return launch(index_logits_kernel<__nv_bfloat16>, p, grid, kThreads, 0, s);
}
