// The forms of the attention kernel (paged_attention.cu), and what each of them is given beside the call's arguments.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "libtopk.h"
#include "paged.cuh"

namespace ltk {
namespace paged {

enum class Form {
  kPlain,   // topk_paged_attention
  kBlocks,  // topk_block_attention: index lists name blocks, one list for each row and key-value head
  kTail,    // topk_shared_attention, the tokens behind the prefixes: rows begin at a page of their own
  kShared,  // topk_shared_attention, the prefixes: units are runs of rows that share one
  kWhole,   // topk_shared_attention, each row by itself: the prefix's pages are found in its row of their table
};

// Neighbouring rows that share a prefix.
struct SharedRun {
  int32_t row0, rows;
  int32_t prefix;  // row of the prefixes' table
  int32_t length;  // tokens shared: whole pages
};

// What requests begin with.
struct Prefixes {
  const int32_t* of;  // [requests]
  const int32_t* lens;
  const int32_t* table;
  int64_t count, stride;
  int64_t most;  // tokens of a row of the table
};

// Tokens of a request's prefix, whole pages; 0: nothing shared. `prefix`: which one.
__device__ __forceinline__ int prefix_tokens(const Prefixes& p, const Rows& R, int64_t request, int32_t* prefix) {
  if (request < 0 || request >= R.num_requests) return 0;
  *prefix = p.of[request];
  if (*prefix < 0 || *prefix >= p.count) return 0;
  const int64_t n = p.lens[*prefix];
  if (n <= 0) return 0;
  return block_column(R, static_cast<int>(n < p.most ? n : p.most)) * R.block_size;
}

// The same for a row: 0 also where one of its request's rows, which read what follows together, sees less. Rows that bring
// their requests read by themselves, and each decides for itself. By a whole warp, each lane with a row of its own (or past the last one): requests of many rows are looked through by all lanes.
__device__ __forceinline__ int row_prefix_tokens(const Prefixes& p, const Rows& R, int64_t row, int32_t* prefix) {
  const bool real = row >= 0 && row < R.num_rows;
  const int64_t request = real ? row_request(R, row) : -1;
  int n = prefix_tokens(p, R, request, prefix);
  if (R.row_request) return n > 0 && seen_tokens(R, R.lengths[row], request) >= n ? n : 0;
  constexpr int kFew = 4;
  if (R.next_n <= kFew) {
    for (int j = 0; j < R.next_n; ++j)
      if (n > 0 && seen_tokens(R, R.lengths[request * R.next_n + j], request) < n) n = 0;
    return n;
  }
  const int lane = threadIdx.x & 31;
  __syncwarp();
  for (unsigned todo = __ballot_sync(~0u, n > 0); todo;) {
    const int first = __ffs(todo) - 1;
    const int64_t which = __shfl_sync(~0u, request, first);
    const int need = __shfl_sync(~0u, n, first);
    bool less = false;
    for (int j = lane; j < R.next_n; j += 32) less |= seen_tokens(R, R.lengths[which * R.next_n + j], which) < need;
    less = __any_sync(~0u, less);
    const bool mine = request == which;
    if (mine && less) n = 0;
    todo &= ~__ballot_sync(~0u, mine);
  }
  return n;
}

struct FormArgs {
  // kBlocks
  const int32_t* blocks;
  int64_t block_row_stride, block_head_stride;
  int64_t num_chosen;
  // kTail
  const int32_t* skip;  // [rows] columns of the request's table before the row's first token
  // kShared
  const SharedRun* runs;
  const int32_t* run_count;
  Prefixes prefixes;  // and kWhole
  float* tail_lse;    // [slices][2][column blocks][columns]: of what is behind the prefix, for the join
};

int attend_plain(const topk_attention_args& a, const FormArgs& f, void* stream);
int attend_blocks(const topk_attention_args& a, const FormArgs& f, void* stream);
int attend_tail(const topk_attention_args& a, const FormArgs& f, void* stream);
int attend_shared(const topk_attention_args& a, const FormArgs& f, void* stream);
int attend_whole(const topk_attention_args& a, const FormArgs& f, void* stream);

constexpr int kMaxQk = 576, kMaxV = 512;

// What all forms refuse; of pointers only where there are rows.
inline int check_attention(const topk_attention_args& a) {
  int rc = check_rows(a.rows);
  if (rc != TOPK_OK) return rc;
  if (!(a.scale > 0.f) || a.scale > 3.4e38f || a.heads < 1 || a.kv_heads < 1 || a.heads % a.kv_heads != 0)
    return TOPK_ERR_INVALID_ARG;
  if (a.indices != nullptr && (a.num_indices < 1 || a.num_indices > (1 << 20) || a.index_row_stride < 0))
    return TOPK_ERR_INVALID_ARG;
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
  return TOPK_OK;
}

// Columns (rows and heads) of a unit at most, where rows share a prefix: kWideCols in wide_prefix.cu, which takes keys and values
// of up to 128 dims that are not one, kSharedCols in the kernel of all forms. Past kSharedCols that one reads a prefix more than once,
// and the wide one is the faster: 32 heads over 8, a prefix of 16 K tokens, in us wide against narrow: 72 columns 43, 50; 256 58, 78;
// 512 85, 112; of 64 dims 96 columns 41, 51. Few units bring them closer: 16 heads over 2, 32 K tokens: 80 columns 41, 42; 256 47, 47;
// 512 52, 63; over one 256 47, 42. All of one prefix: of several, runs have fewer columns than rows times heads say, and the wide kernel's
// units are then in part empty (32 rows of 32 heads over 8, 16 K tokens: one prefix 47, eight of 4 rows each 138).
constexpr int kSharedCols = 64, kWideCols = 256;

int attend_wide(const topk_attention_args& a, const FormArgs& f, void* scratch, void* stream);
size_t wide_scratch(int sms);

inline bool takes_wide(const topk_attention_args& a) {
  const int group = a.heads / a.kv_heads;
  return a.v != nullptr && a.dk <= 128 && a.dv <= 128 && group <= kWideCols && a.rows.num_rows * group > kSharedCols;
}

// Rows of a run: what fills a unit's columns.
inline int rows_of_run(const topk_attention_args& a) {
  const int group = a.heads / a.kv_heads, cols = takes_wide(a) ? kWideCols : kSharedCols, rows = group >= cols ? 1 : cols / group;
  return rows < a.rows.num_rows ? rows : static_cast<int>(a.rows.num_rows);
}

}  // namespace paged
}  // namespace ltk
