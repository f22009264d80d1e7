// Block tables and slot maps of one step, from the requests' lengths: which
// blocks each request takes from the free list, and for every new token its
// slot, the length that it sees and its request.
//
// Two exclusive sums over the requests (new tokens; blocks taken) place
// everything. They are short (a few thousand requests at most), so every CTA
// computes both from the start of the lists, a segment of requests at a time
// in shared memory, and then writes its own chunks of the token lists: one
// launch, nothing exchanged between CTAs but a ticket. A token finds its
// request by a binary search in the segment's starts. A block taken in this
// call always holds a new token at its first place, so the thread that lists
// that token also enters the block in the table.
//
// `taken` may be updated in place: a CTA draws a ticket after its last read of
// it, and the one that draws the last ticket writes taken_out (and sets the
// ticket back to zero).
//
// Bound by latency (4.8 us for 64 requests with a token each), and by the 16 bytes that
// are written a token: lists for two million tokens, half of them new ones of 512 requests,
// take 16 us (2 TB/s).
#include "paged.cuh"

namespace ltk {
namespace paged {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 4;                    // requests a thread scans
constexpr int kSegment = kThreads * kPer;  // requests of one segment
constexpr int kChunk = 2048;               // consecutive tokens of a CTA; chunks are dealt to the CTAs in turn
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

__global__ void __launch_bounds__(kThreads, 3) kv_map_kernel(const MapParams p) {
  __shared__ uint32_t start[kSegment];  // first new token of each request of the segment, from the segment's first
  __shared__ uint32_t first[kSegment];  // blocks taken before each, likewise
  __shared__ int64_t warp_tokens[kWarps], warp_blocks[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const topk_kv_map_args& a = p.a;
  uint32_t* status = static_cast<uint32_t*>(a.workspace);
  dependent_wait();
  dependent_launch();
  const int64_t taken = *a.taken;
  // this CTA's first chunk that ends after token x
  const auto first_chunk = [&](int64_t x) {
    const int64_t chunk = x / kChunk;
    return (chunk + gridDim.x - 1 - blockIdx.x) / gridDim.x * gridDim.x + blockIdx.x;
  };
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
      start[j] = static_cast<uint32_t>(at - tokens);
      first[j] = static_cast<uint32_t>(took - blocks);
      if (j < n && (r0 / kSegment) % gridDim.x == blockIdx.x) a.token_start[r0 + j] = static_cast<int32_t>(at);
      at += my_new[i];
      took += my_take[i];
    }
    __syncthreads();
    const int64_t end = tokens + seg_tokens;
    // Token numbers are below 2^31 and positions below 2^32, so 32 bits do from here on.
    const uint32_t n_tokens = static_cast<uint32_t>(seg_tokens);
    const int64_t taken_here = taken + blocks;
    for (int64_t chunk = first_chunk(tokens); chunk * kChunk < end; chunk += gridDim.x) {
      const int64_t chunk0 = chunk * kChunk - tokens;  // from the segment's first token
#pragma unroll 2
      for (int i = 0; i < kChunk; i += kThreads) {
        const int64_t t64 = chunk0 + i + tid;
        if (t64 < 0 || t64 >= n_tokens) continue;
        const uint32_t t = static_cast<uint32_t>(t64);
        uint32_t j = 0;  // the last request whose start is at or before t: it holds t, since later ones start after it
#pragma unroll
        for (uint32_t step = kSegment / 2; step > 0; step >>= 1)
          if (start[j + step] <= t) j += step;
        const int32_t r = static_cast<int32_t>(r0) + static_cast<int32_t>(j);
        const int32_t c = max(a.context_lens[r], 0);
        const uint32_t pos = static_cast<uint32_t>(c) + (t - start[j]);
        const uint32_t size = a.block_size, columns = static_cast<uint32_t>(a.max_blocks);
        const uint32_t col = p.block_shift >= 0 ? pos >> p.block_shift : pos / size;
        const uint32_t place = pos - col * size;
        const uint32_t have = min(p.block_shift >= 0 ? (c + (size - 1)) >> p.block_shift : (c + (size - 1)) / size, columns);
        int32_t* entry = a.block_table + r * a.table_stride + col;
        int32_t block = -1;
        bool had = false;  // whether the table or the free list names a block
        if (col >= columns) {
          flags |= TOPK_DEV_TABLE_FULL;
        } else if (col < have) {
          block = *entry;
          had = true;
        } else {
          const int64_t n = taken_here + first[j] + (col - have);
          had = n >= 0 && n < a.num_free;
          if (had)
            block = a.free_blocks[n];
          else
            flags |= TOPK_DEV_BLOCKS_EXHAUSTED;
          if (place == 0) *entry = block;
        }
        if (had && block < 0) flags |= TOPK_DEV_BAD_BLOCK;  // where an earlier step ran out of blocks, for one
        const int64_t at = tokens + t;
        a.slots[at] = block < 0 ? -1 : static_cast<int64_t>(block) * size + place;
        a.row_lens[at] = static_cast<int32_t>(min(pos, 0x7FFFFFFEu) + 1);
        a.row_request[at] = r;
      }
    }
    tokens += seg_tokens;
    blocks += seg_blocks;
    __syncthreads();  // the next segment writes the starts again
  }
  for (int64_t chunk = first_chunk(tokens); chunk * kChunk < a.max_tokens; chunk += gridDim.x) {
#pragma unroll
    for (int i = 0; i < kChunk; i += kThreads) {
      const int64_t t = chunk * kChunk + i + tid;
      if (t < tokens || t >= a.max_tokens) continue;
      a.slots[t] = -1;
      a.row_lens[t] = 0;
      a.row_request[t] = -1;
    }
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
  int64_t grid = (a.max_tokens + kChunk - 1) / kChunk;
  grid = grid < 1 ? 1 : (grid > 3ll * sms ? 3ll * sms : grid);
  return launch(kv_map_kernel, p, grid, kThreads, 0, static_cast<cudaStream_t>(stream));
}
