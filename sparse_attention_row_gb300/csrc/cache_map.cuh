// Tensor maps of a paged cache, and the copies of a tile's tokens through them.
//
// The cache is a list of rows, one token (of one head) each, whose addresses are
// base + row * step; `step` is the largest one that the strides of blocks, tokens and
// heads are multiples of, so that any of them fits. A tile's tokens are fetched
// four rows at a time by their row numbers (tile::gather4), in columns of 128 bytes,
// swizzled; a masked token's row number is one past the last, which reads as zeros.
// Where a tile holds nothing but consecutive tokens of whole runs of a block (a dense
// cache, not a row's last tile), up to 32 rows are fetched at once.
// Copies by 16-byte cp.async with an arrival for each thread, which this replaces, bring
// an SM 36 bytes a cycle whatever else runs (32 KB in 900 cycles, measured); a latent
// tile (147 KB) then takes longer to arrive than to be multiplied.
#pragma once

#include <cuda.h>

#include "paged.cuh"
#include "umma.cuh"

namespace ltk {
namespace paged {

struct CacheMap {
  CUtensorMap gather;  // rows by number, box 1 x 128 bytes
  CUtensorMap run;     // run_rows consecutive tokens, box run_rows x 128 bytes
  int64_t block_step, token_step, head_step;              // of row numbers, in `gather`
  int64_t run_block_step, run_head_step;                  // in `run`, whose tokens are one row apart
  int32_t rows, run_total;                                // of both: what is past them reads as zeros
  int32_t run_rows;                                       // 0: no runs
  int32_t elements;                                       // of 128 bytes
};

// Row numbers of this thread's token; past the end where it is masked.
__device__ __forceinline__ int gather_row(const CacheMap& m, bool on, int64_t block, int place, int head) {
  return on ? static_cast<int>(block * m.block_step + place * m.token_step + head * m.head_step) : m.rows;
}
__device__ __forceinline__ int run_row(const CacheMap& m, bool on, int64_t block, int place, int head) {
  return on ? static_cast<int>(block * m.run_block_step + place + head * m.run_head_step) : m.run_total;
}

__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// A copying warp's 32 tokens of a tile.
struct TokenRows {
  int row[4];   // gather: the four rows of this lane's group (lane % 8); runs: row[0], the first of this lane's run
  int run;      // rows of a run, 0: gather
  // `mine`: the row number of this lane's token.
  __device__ __forceinline__ void set(int mine, int run_rows, int lane) {
    run = run_rows;
    if (run) {
      row[0] = __shfl_sync(~0u, mine, (lane * run) & 31);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) row[i] = __shfl_sync(~0u, mine, (lane & 7) * 4 + i);
    }
  }
  // Columns [chunk, chunk + chunks) (at most two) of the warp's tokens to `dst` + 16 KB a column; `dst` is the place of the
  // warp's first token. One lane per copy.
  __device__ __forceinline__ void fetch(const CacheMap& m, uint32_t dst, int chunk, int chunks, uint32_t bar, int lane) const {
    if (lane == 0) expect_bytes(bar, chunks * 32 * 128);
    __syncwarp();
    if (run) {
      const int copies = 32 / run, i = lane & (copies - 1), c = lane / copies;
      if (c < chunks)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                dst + c * (128 * 128) + i * run * 128),
            "l"(&m.run), "r"((chunk + c) * m.elements), "r"(row[0]), "r"(bar)
            : "memory");
    } else if (lane < chunks * 8) {
      const int c = lane >> 3;
      asm volatile(
          "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
          "%5, %6}], [%7];" ::"r"(dst + c * (128 * 128) + (lane & 7) * 512),
          "l"(&m.gather), "r"((chunk + c) * m.elements), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(bar)
          : "memory");
    }
  }
};

// Builds the maps of a cache [num_blocks, block_size, heads, dim] with these strides in elements of `size` bytes (multiples
// of 16 bytes, as is `base`). TOPK_ERR_UNSUPPORTED where a row number would not fit 31 bits.
int make_cache_map(CacheMap* m, const void* base, int size, int bf16_or_f16_or_8bit, int64_t num_blocks, int block_size, int heads,
                   int dim, int64_t block_stride, int64_t token_stride, int64_t head_stride);

}  // namespace paged
}  // namespace ltk
