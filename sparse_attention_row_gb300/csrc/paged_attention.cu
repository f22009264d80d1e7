// Attention of each row's heads over a paged cache. One CTA a (row, head):
// every warp takes every fourth token with an online softmax in fp32; the
// warps' sums are joined at the end.
#include "paged.cuh"

namespace ltk {
namespace paged {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxQk = 576, kMaxV = 512;

struct AttentionParams {
  topk_attention_args a;
  Rows R;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) paged_attention_kernel(const AttentionParams p) {
  __shared__ float sum_l[4], sum_m[4];
  __shared__ float acc[4][kMaxV];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  dependent_wait();
  dependent_launch();
  const topk_attention_args& a = p.a;
  for (int64_t u = blockIdx.x; u < p.R.num_rows * a.heads; u += gridDim.x) {
    const int64_t row = u / a.heads;
    const int head = static_cast<int>(u % a.heads), kvh = head / (a.heads / a.kv_heads);
    const int len = row_length(p.R, row, threadIdx.x == 0);
    const T* q = static_cast<const T*>(a.q) + row * a.q_row_stride + head * a.q_head_stride;
    float o[kMaxV / 32] = {}, m = -INFINITY, l = 0;
    const int n = len == 0 ? 0 : (a.indices ? a.num_indices : len);
    for (int i = warp; i < n; i += 4) {
      const int t = a.indices ? a.indices[row * a.index_row_stride + i] : i;
      if (t < 0 || t >= len) continue;
      int64_t block;
      int place;
      if (!locate(p.R, row_request(p.R, row), t, &block, &place)) continue;
      const T* k = static_cast<const T*>(a.k) + block * a.k_block_stride + place * a.k_token_stride + kvh * a.k_head_stride;
      const T* v = a.v ? static_cast<const T*>(a.v) + block * a.v_block_stride + place * a.v_token_stride + kvh * a.v_head_stride : k;
      float s = 0;
      for (int d = lane; d < a.dk; d += 32) s += static_cast<float>(q[d]) * static_cast<float>(k[d]);
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
      s *= a.scale;
      const float m2 = s > m ? s : m, base = m2 == -INFINITY ? 0.f : m2;
      const float w = expf(m - base), e = expf(s - base);
      l = l * w + e;
      for (int j = 0; j < kMaxV / 32; ++j)
        if (j * 32 + lane < a.dv) o[j] = o[j] * w + e * static_cast<float>(v[j * 32 + lane]);
      m = m2;
    }
    for (int j = 0; j < kMaxV / 32; ++j) acc[warp][j * 32 + lane] = o[j];
    sum_m[warp] = m;
    sum_l[warp] = l;
    __syncthreads();
    float mm = -INFINITY, ll = 0;
    for (int w = 0; w < 4; ++w) mm = fmaxf(mm, sum_m[w]);
    const float base = mm == -INFINITY ? 0.f : mm;
    for (int w = 0; w < 4; ++w) ll += sum_l[w] * expf(sum_m[w] - base);
    T* out = static_cast<T*>(a.out) + row * a.out_row_stride + head * a.out_head_stride;
    for (int d = threadIdx.x; d < a.dv; d += kThreads) {
      float x = 0;
      for (int w = 0; w < 4; ++w) x += acc[w][d] * expf(sum_m[w] - base);
      out[d] = static_cast<T>(ll == 0.f ? 0.f : x / ll);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row * a.heads + head] = ll == 0.f ? -INFINITY : base + logf(ll);
    __syncthreads();
  }
}

}  // namespace
}  // namespace paged
}  // namespace ltk

extern "C" size_t topk_attention_workspace_size(int device) {
  topk_device_props p{};
  if (topk_query_device(device, &p) != TOPK_OK) return 0;
  return TOPK_PAGED_WORKSPACE_BYTES;
}

extern "C" int topk_paged_attention(const topk_attention_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_attention_args& a = *args;
  int rc = check_rows(a.rows);
  if (rc != TOPK_OK) return rc;
  if (!(a.scale > 0.f) || a.scale > 3.4e38f || a.heads < 1 || a.kv_heads < 1 || a.heads % a.kv_heads != 0) return TOPK_ERR_INVALID_ARG;
  if (a.indices != nullptr && (a.num_indices < 1 || a.num_indices > (1 << 20) || a.index_row_stride < 0)) return TOPK_ERR_INVALID_ARG;
  if ((a.dtype != TOPK_DTYPE_F16 && a.dtype != TOPK_DTYPE_BF16) || a.heads > 1024 || a.dk < 8 || a.dk > kMaxQk || a.dk % 8 ||
      a.dv < 8 || a.dv > kMaxV || a.dv % 8 || (a.v == nullptr && a.dv > a.dk))
    return TOPK_ERR_UNSUPPORTED;
  if (a.rows.num_rows == 0) return TOPK_OK;
  rc = check_row_pointers(a.rows);
  if (rc != TOPK_OK) return rc;
  if (a.q == nullptr || a.k == nullptr || a.out == nullptr || a.workspace == nullptr) return TOPK_ERR_INVALID_ARG;
  if (misaligned(a.q, 16) || a.q_row_stride % 8 || a.q_head_stride % 8 || misaligned(a.k, 16) || a.k_block_stride % 8 ||
      a.k_token_stride % 8 || a.k_head_stride % 8 || misaligned(a.out, 16) || a.out_row_stride % 8 || a.out_head_stride % 8 ||
      misaligned(a.indices, 4) || misaligned(a.lse, 4) || misaligned(a.workspace, 16) ||
      (a.v && (misaligned(a.v, 16) || a.v_block_stride % 8 || a.v_token_stride % 8 || a.v_head_stride % 8)))
    return TOPK_ERR_MISALIGNED;
  const int sms = num_sms();
  if (sms < 1) return TOPK_ERR_CUDA;
  if (a.workspace_bytes < TOPK_PAGED_WORKSPACE_BYTES) return TOPK_ERR_WORKSPACE_TOO_SMALL;
  AttentionParams p{};
  p.a = a;
  p.R = make_rows(a.rows, INT32_MAX, a.workspace);
  const int64_t units = a.rows.num_rows * a.heads, grid = units < sms * 8 ? units : sms * 8;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.dtype == TOPK_DTYPE_F16) return launch(paged_attention_kernel<__half>, p, grid, kThreads, 0, s);
  return launch(paged_attention_kernel<__nv_bfloat16>, p, grid, kThreads, 0, s);
}
