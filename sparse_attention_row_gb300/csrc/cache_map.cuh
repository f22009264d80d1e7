// Tensor maps of a paged cache, and copies of its tokens through them by TMA.
//
// The cache is a list of rows, one token each, whose addresses are base + row * step;
// `step` is the largest one that the strides of blocks and tokens are multiples of, so
// that any of them fits. Where a block's tokens come in runs of 8 to 64 (its size is a
// multiple of that, and its stride one of the tokens'), a run is fetched at once;
// elsewhere four rows by their numbers (tile::gather4). What is masked has a row number
// past the last, which reads as zeros; of a run that begins in the cache the tokens past
// the length are fetched with it. Either way 128 bytes of each token at a time, swizzled.
//
// This is for streams of whole pages. An instruction takes its warp 70 cycles for 512
// bytes and 180 for 8 KB, so scattered tokens are better copied by cp.async
// (token_copies.cuh); but those wait for a place among an SM's outstanding reads, of which
// a stream from HBM in pieces of 128 bytes a token takes all: 14 to 25 bytes a cycle.
#pragma once

#include <cuda.h>

#include "paged.cuh"

namespace ltk {
namespace paged {

struct CacheMap {
  CUtensorMap gather;  // rows by number, box 1 x 128 bytes
  CUtensorMap run;     // run_rows consecutive tokens of a block, box run_rows x 128 bytes
  int64_t block_step, token_step;  // of row numbers, in `gather`
  int64_t run_block_step;          // in `run`, whose tokens are one row apart
  int32_t rows, run_total;         // of both: what is past them reads as zeros
  int32_t run_rows;                // 0: no runs
  int32_t elements;                // of 128 bytes
};

// Row number of a token; past the end where it is masked.
__device__ __forceinline__ int gather_row(const CacheMap& m, bool on, int64_t block, int place) {
  return on ? static_cast<int>(block * m.block_step + place * m.token_step) : m.rows;
}
__device__ __forceinline__ int run_row(const CacheMap& m, bool on, int64_t block, int place) {
  return on ? static_cast<int>(block * m.run_block_step + place) : m.run_total;
}

// An arrival on `bar` that also makes its phase wait for `bytes` of copies.
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void fetch_run(const CacheMap& m, uint32_t dst, int column, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(&m.run), "r"(column * m.elements), "r"(row), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void fetch_four(const CacheMap& m, uint32_t dst, int column, const int (&row)[4], uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(dst),
      "l"(&m.gather), "r"(column * m.elements), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(bar)
      : "memory");
}

// Builds the maps of a cache [num_blocks, block_size, dim] with these strides in elements of `size` bytes (multiples of
// 16 bytes, as is `base`); runs of at most `most_rows` tokens, a power of two up to 64. TOPK_ERR_UNSUPPORTED where a row
// number would not fit 31 bits.
int make_cache_map(CacheMap* m, const void* base, int size, int dtype, int64_t num_blocks, int block_size, int dim,
                   int64_t block_stride, int64_t token_stride, int most_rows);

}  // namespace paged
}  // namespace ltk
