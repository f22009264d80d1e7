// What the paged calls (topk_kv_map, topk_index_logits, topk_paged_attention)
// share: the rows of a call as their kernels see them, argument checks, the
// launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <climits>

#include "libtopk.h"
#include "topk_internal.h"

namespace ltk {
namespace paged {

// topk_paged_rows for a kernel. Lengths are clamped into [0, max_len].
struct Rows {
  int64_t num_rows;
  int64_t num_requests;
  int64_t num_blocks;
  int64_t table_stride;
  const int32_t* lengths;
  const int32_t* row_request;
  const int32_t* block_table;
  int32_t next_n;
  int32_t block_size;
  uint32_t block_mul, block_shift;  // x / block_size = (high word of x * block_mul + x) >> block_shift, 0 <= x < 2^31
  int32_t max_len;
  uint32_t* status;
};

__device__ __forceinline__ int64_t row_request(const Rows& R, int64_t row) {
  return R.row_request ? static_cast<int64_t>(R.row_request[row]) : static_cast<uint32_t>(row) / static_cast<uint32_t>(R.next_n);  // rows are below 2^31
}

// The table's column of a token (division by an invariant, Granlund and Montgomery 1994).
__device__ __forceinline__ int block_column(const Rows& R, int x) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(x), R.block_mul) + static_cast<uint32_t>(x)) >> R.block_shift);
}

// Tokens that a row sees, from its entry in `lengths` and its request; 0 for a padding row (negative request).
__device__ __forceinline__ int seen_tokens(const Rows& R, int32_t n, int64_t request) {
  if (request < 0 || request >= R.num_requests) return 0;
  return n < 0 ? 0 : (n > R.max_len ? R.max_len : n);
}

__device__ __forceinline__ int row_length(const Rows& R, int64_t row) {
  const int32_t n = R.lengths[row];
  return seen_tokens(R, n, row_request(R, row));
}

// Reports what was wrong with the rows: one CTA does it, when its work is done.
__device__ __forceinline__ void report_rows(const Rows& R, int tid, int threads) {
  uint32_t bits = 0;
  for (int64_t row = tid; row < R.num_rows; row += threads) {
    const int32_t n = R.lengths[row];
    const int64_t b = row_request(R, row);
    if (b >= R.num_requests) bits |= TOPK_DEV_BAD_BLOCK;
    if (b >= 0 && b < R.num_requests && (n < 0 || n > R.max_len)) bits |= TOPK_DEV_LENGTH_CLAMPED;
  }
  if (bits) atomicOr(R.status, bits);
}

// Programmatic dependent launch: wait for the kernel before this one on the stream, before the first
// access to global memory; and let the next one start early in the same way. A kernel that has begun before the
// last one has ended may not use loads of data that nothing writes while it runs (__ldg): what they read is what it waits for.
__device__ __forceinline__ void dependent_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependent_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Checks what can be checked of the rows before the pointers are looked at.
inline int check_rows(const topk_paged_rows& r) {
  if (r.num_rows < 0 || r.num_rows > INT32_MAX || r.next_n < 1 || r.block_size < 1 || r.num_requests < 0 ||
      r.num_requests > INT32_MAX || r.num_blocks < 0 || r.num_blocks > INT32_MAX || r.max_blocks < 1 ||
      r.table_stride < r.max_blocks)
    return TOPK_ERR_INVALID_ARG;
  if (r.row_request == nullptr && (r.num_rows % r.next_n != 0 || r.num_rows / r.next_n > r.num_requests))
    return TOPK_ERR_INVALID_ARG;
  return TOPK_OK;
}

inline int check_row_pointers(const topk_paged_rows& r) {
  if (r.lengths == nullptr || r.block_table == nullptr) return TOPK_ERR_INVALID_ARG;
  if (misaligned(r.lengths, 4) || misaligned(r.row_request, 4) || misaligned(r.block_table, 4))
    return TOPK_ERR_MISALIGNED;
  return TOPK_OK;
}

inline Rows make_rows(const topk_paged_rows& r, int64_t columns, void* workspace) {
  Rows R{};
  R.num_rows = r.num_rows;
  R.num_requests = r.num_requests;
  R.num_blocks = r.num_blocks;
  R.table_stride = r.table_stride;
  R.lengths = r.lengths;
  R.row_request = r.row_request;
  R.block_table = r.block_table;
  R.next_n = r.next_n;
  R.block_size = r.block_size;
  while ((1ull << R.block_shift) < static_cast<uint64_t>(r.block_size)) ++R.block_shift;
  R.block_mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << R.block_shift) - r.block_size)) / r.block_size + 1);
  const int64_t held = r.max_blocks > INT32_MAX / r.block_size ? INT32_MAX : r.max_blocks * r.block_size;
  R.max_len = static_cast<int32_t>(held < columns ? held : columns);
  R.status = static_cast<uint32_t*>(workspace);
  return R;
}

template <typename Args>
inline int launch(void (*kernel)(Args), const Args& args, int64_t grid, int threads, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent_launch_default() ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, args) != cudaSuccess) {
    cudaGetLastError();
    return TOPK_ERR_CUDA;
  }
  return TOPK_OK;
}

// Lets a kernel use `smem` bytes of shared memory. Asked of the runtime once for each kernel and device: `granted` (one
// for each kernel, its own static array) holds what was granted.
constexpr int kMaxDevices = 64;
template <typename Kernel>
inline int allow_smem(Kernel* kernel, size_t smem, int device, int* granted) {
  if (device >= 0 && device < kMaxDevices && __atomic_load_n(&granted[device], __ATOMIC_ACQUIRE) >= static_cast<int>(smem)) return TOPK_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess) {
    cudaGetLastError();
    return TOPK_ERR_CUDA;
  }
  if (device >= 0 && device < kMaxDevices) __atomic_store_n(&granted[device], static_cast<int>(smem), __ATOMIC_RELEASE);
  return TOPK_OK;
}

// SMs of the current device (cached); 0 if it cannot be queried.
int num_sms();

}  // namespace paged
}  // namespace ltk
