// Host side of cache_map.cuh: tensor maps of a paged cache.
#include "cache_map.cuh"

#include <numeric>

namespace ltk {
namespace paged {
namespace {

using Encode = decltype(&cuTensorMapEncodeTiled);

Encode encoder() {
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<Encode>(f);
  }();
  return fn;
}

bool encode(CUtensorMap* map, const void* base, CUtensorMapDataType type, int size, int dim, int64_t rows, int64_t step, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(step) * size};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / size), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t each[2] = {1, 1};
  return encoder()(map, type, 2, const_cast<void*>(base), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int make_cache_map(CacheMap* m, const void* base, int size, int dtype, int64_t num_blocks, int block_size, int dim,
                   int64_t block_stride, int64_t token_stride, int most_rows) {
  if (encoder() == nullptr) return TOPK_ERR_CUDA;
  const CUtensorMapDataType type = dtype == TOPK_DTYPE_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : dtype == TOPK_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  m->elements = 128 / size;
  // a stride that is never taken does not count
  if (num_blocks < 2) block_stride = 0;
  if (block_size < 2) token_stride = 0;
  if (block_stride < 0 || token_stride < 0) return TOPK_ERR_UNSUPPORTED;
  int64_t step = std::gcd(block_stride, token_stride);
  if (step == 0) step = (dim + 15) / 16 * 16;  // one token in all (or all the same)
  const int64_t last = num_blocks > 0 ? (num_blocks - 1) * block_stride + (block_size - 1) * token_stride : 0;
  if (last / step >= INT32_MAX - 1 || step * size >= (int64_t{1} << 40)) return TOPK_ERR_UNSUPPORTED;
  m->rows = static_cast<int32_t>(last / step + 1);
  m->block_step = block_stride / step;
  m->token_step = token_stride / step;
  if (!encode(&m->gather, base, type, size, dim, m->rows, step, 1)) return TOPK_ERR_UNSUPPORTED;
  m->run_rows = 0;
  int run = 1;
  while (run < most_rows && block_size % (run * 2) == 0) run *= 2;
  if (run >= 8 && token_stride > 0 && block_stride % token_stride == 0) {
    m->run_total = static_cast<int32_t>(last / token_stride + 1);
    m->run_block_step = block_stride / token_stride;
    if (encode(&m->run, base, type, size, dim, m->run_total, token_stride, run)) m->run_rows = run;
  }
  return TOPK_OK;
}

}  // namespace paged
}  // namespace ltk
