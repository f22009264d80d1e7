// Block tables and slot maps of one step, from the requests' lengths: which
// blocks each request takes from the free list, and for every new token its
// slot, the length that it sees and its request.
//
// Two exclusive sums over the requests (new tokens; blocks taken) place
// everything. They are short (a few thousand requests at most), so every CTA
// computes both from the start of the lists, a segment of requests at a time
// in shared memory, and then writes its own slice of the token lists: one
// launch, nothing exchanged between CTAs but a ticket. A token finds its
// request by a binary search in the segment's starts. A block taken in this
// call always holds a new token at its first place, so the thread that lists
// that token also enters the block in the table.
//
// `taken` may be updated in place: a CTA draws a ticket after its last read of
// it, and the one that draws the last ticket writes taken_out (and sets the
// ticket back to zero).
//
// Bound by latency: 16 bytes are written a token.
#include "paged.cuh"

namespace ltk {
namespace paged {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 4;                    // requests a thread scans
constexpr int kSegment = kThreads * kPer;  // requests of one segment
constexpr int kSlice = 2048;               // tokens that make a CTA worth its scan
constexpr int kTicketWord = 8;             // of the workspace

struct MapParams {
  topk_kv_map_args a;
  int block_shift;
};

__device__ __forceinline__ int64_t blocks_for(const MapParams& p, int64_t tokens) {
  const int64_t up = tokens + p.a.block_size - 1;
  const int64_t n = p.block_shift >= 0 ? up >> p.block_shift : up / p.a.block_size;
  return n < p.a.max_blocks ? n : p.a.max_blocks;
}

__device__ __forceinline__ int64_t context(const MapParams& p, int64_t r) {
  return p.a.context_lens[r] < 0 ? 0 : p.a.context_lens[r];
}

__global__ void __launch_bounds__(kThreads) kv_map_kernel(const MapParams p) {
  __shared__ int64_t start[kSegment];      // first new token of each request of the segment
  __shared__ int64_t first[kSegment];      // blocks taken before each
  __shared__ int64_t warp_tokens[kWarps], warp_blocks[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const topk_kv_map_args& a = p.a;
  uint32_t* status = static_cast<uint32_t*>(a.workspace);
  dependent_wait();
  dependent_launch();
  const int64_t taken = *a.taken;
  const int64_t slice = (a.max_tokens + gridDim.x - 1) / gridDim.x;  // tokens of this CTA: [t0, t1)
  const int64_t t0 = slice * blockIdx.x;
  const int64_t t1 = t0 + slice < a.max_tokens ? t0 + slice : a.max_tokens;
  int64_t tokens = 0, blocks = 0;  // before the segment
  uint32_t flags = 0;
  for (int64_t r0 = 0; r0 < a.num_requests; r0 += kSegment) {
    const int n = static_cast<int>(a.num_requests - r0 < kSegment ? a.num_requests - r0 : kSegment);
    int64_t my_new[kPer], my_take[kPer], sum_new, sum_take, seg_tokens, seg_blocks, at, took;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = tid * kPer + i;
      my_new[i] = j < n && a.new_lens[r0 + j] > 0 ? a.new_lens[r0 + j] : 0;
    }
    for (bool cut = false;;) {
      sum_new = sum_take = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int j = tid * kPer + i;
        const int64_t c = j < n ? context(p, r0 + j) : 0;
        my_take[i] = blocks_for(p, c + my_new[i]) - blocks_for(p, c);
        sum_new += my_new[i];
        sum_take += my_take[i];
      }
      int64_t pre_new = sum_new, pre_take = sum_take;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(~0u, pre_new, d), y = __shfl_up_sync(~0u, pre_take, d);
        if (lane >= d) {
          pre_new += x;
          pre_take += y;
        }
      }
      if (lane == 31) {
        warp_tokens[warp] = pre_new;
        warp_blocks[warp] = pre_take;
      }
      __syncthreads();
      seg_tokens = seg_blocks = 0;
      at = tokens + pre_new - sum_new;
      took = blocks + pre_take - sum_take;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
          at += warp_tokens[w];
          took += warp_blocks[w];
        }
        seg_tokens += warp_tokens[w];
        seg_blocks += warp_blocks[w];
      }
      if (cut || tokens + seg_tokens <= a.max_tokens) break;
      // more tokens than the lists hold: what is past their end gets no blocks either
      cut = true;
      flags |= TOPK_DEV_TOKENS_DROPPED;
      int64_t s = at;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int64_t room = a.max_tokens > s ? a.max_tokens - s : 0;
        s += my_new[i];
        my_new[i] = my_new[i] < room ? my_new[i] : room;
      }
      __syncthreads();  // the sums are written again
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = tid * kPer + i;
      start[j] = at;
      first[j] = took;
      if (j < n && (r0 / kSegment) % gridDim.x == blockIdx.x) a.token_start[r0 + j] = static_cast<int32_t>(at);
      at += my_new[i];
      took += my_take[i];
    }
    __syncthreads();
    const int64_t lo = t0 > tokens ? t0 : tokens, end = tokens + seg_tokens, hi = t1 < end ? t1 : end;
    for (int64_t t = lo + tid; t < hi; t += kThreads) {
      int j = 0;  // the last request whose start is at or before t: it holds t, since later ones start after it
#pragma unroll
      for (int step = kSegment / 2; step > 0; step >>= 1)
        if (start[j + step] <= t) j += step;
      const int64_t r = r0 + j;
      const int64_t c = context(p, r);
      const int64_t pos = c + (t - start[j]);
      const int64_t col = p.block_shift >= 0 ? pos >> p.block_shift : pos / a.block_size;
      const int64_t place = pos - col * a.block_size;
      const int64_t have = blocks_for(p, c);
      int64_t block = -1;
      if (col >= a.max_blocks) {
        flags |= TOPK_DEV_TABLE_FULL;
      } else if (col < have) {
        block = a.block_table[r * a.table_stride + col];
      } else {
        const int64_t i = taken + first[j] + (col - have);
        if (i >= 0 && i < a.num_free)
          block = a.free_blocks[i];
        else
          flags |= TOPK_DEV_BLOCKS_EXHAUSTED;
        if (place == 0) a.block_table[r * a.table_stride + col] = static_cast<int32_t>(block);
      }
      a.slots[t] = block < 0 ? -1 : block * a.block_size + place;
      a.row_lens[t] = static_cast<int32_t>(pos + 1 < INT32_MAX ? pos + 1 : INT32_MAX);
      a.row_request[t] = static_cast<int32_t>(r);
    }
    tokens += seg_tokens;
    blocks += seg_blocks;
    __syncthreads();  // the next segment writes the starts again
  }
  for (int64_t t = (t0 > tokens ? t0 : tokens) + tid; t < t1; t += kThreads) {
    a.slots[t] = -1;
    a.row_lens[t] = 0;
    a.row_request[t] = -1;
  }
  if (flags) atomicOr(status, flags);
  if (tid == 0) {
    if (blockIdx.x == 0) a.token_start[a.num_requests] = static_cast<int32_t>(tokens);
    bool last = true;
    if (gridDim.x > 1) {
      __threadfence();
      last = atomicAdd(status + kTicketWord, 1u) + 1 == gridDim.x;
      if (last) status[kTicketWord] = 0;
    }
    const int64_t after = taken + blocks;
    if (last) *a.taken_out = static_cast<int32_t>(after < a.num_free ? after : (taken > a.num_free ? taken : a.num_free));
  }
}

}  // namespace

int num_sms() {
  static int cached[64];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  sms = __atomic_load_n(&cached[dev], __ATOMIC_RELAXED);
  if (sms > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  __atomic_store_n(&cached[dev], sms, __ATOMIC_RELAXED);
  return sms;
}

}  // namespace paged
}  // namespace ltk

extern "C" int topk_kv_map(const topk_kv_map_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_kv_map_args& a = *args;
  if (a.num_requests < 0 || a.num_requests > INT32_MAX || a.block_size < 1 || a.max_blocks < 1 ||
      a.max_blocks > INT32_MAX || a.table_stride < a.max_blocks || a.num_free < 0 || a.num_free > INT32_MAX ||
      a.max_tokens < 0 || a.max_tokens > INT32_MAX)
    return TOPK_ERR_INVALID_ARG;
  if (a.token_start == nullptr || a.taken == nullptr || a.taken_out == nullptr || a.workspace == nullptr ||
      (a.num_requests > 0 && (a.context_lens == nullptr || a.new_lens == nullptr || a.block_table == nullptr)) ||
      (a.num_free > 0 && a.free_blocks == nullptr) ||
      (a.max_tokens > 0 && (a.slots == nullptr || a.row_lens == nullptr || a.row_request == nullptr)))
    return TOPK_ERR_INVALID_ARG;
  if (misaligned(a.context_lens, 4) || misaligned(a.new_lens, 4) || misaligned(a.block_table, 4) ||
      misaligned(a.free_blocks, 4) || misaligned(a.taken, 4) || misaligned(a.taken_out, 4) || misaligned(a.slots, 8) ||
      misaligned(a.row_lens, 4) || misaligned(a.row_request, 4) || misaligned(a.token_start, 4) ||
      misaligned(a.workspace, 16))
    return TOPK_ERR_MISALIGNED;
  const int sms = num_sms();
  if (sms < 1) return TOPK_ERR_CUDA;
  MapParams p{};
  p.a = a;
  p.block_shift = -1;
  for (int s = 0; s < 31; ++s)
    if ((1ll << s) == a.block_size) p.block_shift = s;
  int64_t grid = (a.max_tokens + kSlice - 1) / kSlice;
  grid = grid < 1 ? 1 : (grid > 2ll * sms ? 2ll * sms : grid);
  return launch(kv_map_kernel, p, grid, kThreads, 0, static_cast<cudaStream_t>(stream));
}
