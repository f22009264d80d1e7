// topk_block_attention: the attention kernel whose index lists name blocks (paged_attention.cu), one list for each row and
// key-value head. A list's entry stands for block_size tokens; tiles of 128 of them are found in two steps as ever, the
// position now from the list's entry and the place in the block.
#define LTK_ATTENTION_FORM kBlocks
#define LTK_ATTENTION_CALL attend_blocks
#include "paged_attention.cu"

extern "C" int topk_block_attention(const topk_block_attention_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_block_attention_args& b = *args;
  if (b.attention.indices != nullptr || b.num_chosen < 1 || b.block_row_stride < 0 || b.block_head_stride < 0) return TOPK_ERR_INVALID_ARG;
  if (b.attention.rows.block_size < 1 || b.num_chosen >= (int64_t{1} << 30) / b.attention.rows.block_size) return TOPK_ERR_INVALID_ARG;
  if (b.attention.rows.num_rows > 0) {
    if (b.blocks == nullptr) return TOPK_ERR_INVALID_ARG;
    if (misaligned(b.blocks, 4)) return TOPK_ERR_MISALIGNED;
  }
  FormArgs f{};
  f.blocks = b.blocks;
  f.block_row_stride = b.block_row_stride;
  f.block_head_stride = b.block_head_stride;
  f.num_chosen = b.num_chosen;
  return attend_blocks(b.attention, f, stream);
}
