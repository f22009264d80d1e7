// Mean keys of pages (topk_block_means) and the scores that rows give blocks by them (topk_block_scores).
//
//   means[b, g, :] = 1/n sum_t k[b, t, g, :]           scores[r, g, j] = (sum_h q[r, h, :]) . means[page of j, g, :]
//
// Means. The keys of a page are a matrix, tokens by (head, dim), and a unit is 512 bytes of its width; a thread sums 16 bytes of
// a token's row over every fourth token, 16 loads at a time, and the threads of one column meet in shared memory, in
// a fixed order. Units are found as the map finds its tokens: every CTA sums the requests' pages up. Bound by HBM for
// prompts (64 K tokens of 2 KB: 26 us, 5.2 TB/s; 16 loads at a time and no 64-bit divisions against 8 and some: 33 us), by latency
// for the page or so that a decode step touches of each request (5 us).
//
// Scores. All rows' blocks are dealt to the CTAs in equal shares, in order, after every CTA has summed them up.
//
//   few rows (one of a request, or up to four of large groups): the sum over a group's heads comes first, in shared memory; a warp has 32 blocks of one
//   head, and eight lanes read a mean, 128 bytes at a time, and multiply it with the rows' queries. Bound by the means' way from
//   HBM: 64 rows of 64 heads over 32 K to 131 K tokens in blocks of 64 take 33 us, 5.2 TB/s. (A thread to each mean reads the same
//   bytes, but 16 of every line at a time: 50 us.)
//
//   many rows: tensor cores, which take the heads one by one, since a sum of them would not fit the input type: S [128 blocks x 128
//   columns] = means . Q^T, a thread a block, which sums a row's heads up as it reads them from tensor memory. Bound by the chain of
//   a tile's copy, product and sums, which the CTAs on an SM overlap (three with one place for the means and 128 dims: 1024 rows
//   of one request, 32 heads over 4, 32 K tokens take 15.5 us, 4096 rows 42; fused multiply-adds 34 and 120; two CTAs with two places
//   were 15% slower than three). At the start all CTAs' queries and means come at once: 36 bytes a cycle and SM. The sums are trees over 64 columns at a
//   time, with the rows' tests behind them (32 and one after the other, a branch for each row: 18 and 49 us).
#include "attention_parts.cuh"
#include "paged.cuh"
#include "token_copies.cuh"
#include "umma.cuh"

namespace ltk {
namespace paged {
namespace {

constexpr int kMaxDk = 576;

template <bool kBf16>
__device__ __forceinline__ float2 widen2(uint32_t x) {
  if constexpr (kBf16)
    return __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(x));
  else
    return __half22float2(reinterpret_cast<const __half2&>(x));
}

// A load that stays where it is written, among others that are under way at the same time.
__device__ __forceinline__ uint4 fetch(const uint16_t* at) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at) : "memory");
  return v;
}

template <bool kBf16>
__device__ __forceinline__ void widen(const uint4& x, float (&v)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = widen2<kBf16>(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

template <bool kBf16>
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
  if constexpr (kBf16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return reinterpret_cast<const uint32_t&>(x);
  } else {
    const __half2 x = __floats2half2_rn(lo, hi);
    return reinterpret_cast<const uint32_t&>(x);
  }
}

// ---- means ------------------------------------------------------------------

constexpr int kMeanThreads = 128;
constexpr int kMeanColumns = 32;  // of 16 bytes: a unit is so much of a page's width
constexpr int kTeams = kMeanThreads / kMeanColumns;  // which take its tokens in turn
constexpr int kSegment = 1024;  // requests whose pages are summed up at a time

struct MeanParams {
  topk_block_means_args a;
  Rows R;           // for the division by block_size
  int32_t columns;  // of 16 bytes in a token's row of keys
  uint32_t widths;  // units of a page
};

// New pages of a request: the first one's column, and how many.
__device__ __forceinline__ int touched(const MeanParams& p, int64_t r, int32_t* first, int64_t* total) {
  const int64_t had = p.a.context_lens[r] > 0 ? p.a.context_lens[r] : 0, more = p.a.new_lens[r] > 0 ? p.a.new_lens[r] : 0;
  *total = had + more < INT32_MAX ? had + more : INT32_MAX;  // positions stay below 2^31
  *first = block_column(p.R, static_cast<int>(had));
  return more == 0 || *total <= had ? 0 : block_column(p.R, static_cast<int>(*total - 1)) - *first + 1;
}

template <bool kBf16>
__global__ void __launch_bounds__(kMeanThreads, 5) means_kernel(const __grid_constant__ MeanParams p) {
  __shared__ uint32_t start[kSegment + 1];
  __shared__ uint32_t warp_sum[kMeanThreads / 32];
  __shared__ float4 part[kMeanThreads][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const topk_block_means_args& a = p.a;
  constexpr int kPer = kSegment / kMeanThreads;
  dependent_wait();
  dependent_launch();
  uint32_t flags = 0;
  for (int64_t r0 = 0; r0 < a.num_requests; r0 += kSegment) {
    // the segment's new pages, and each request's first among them
    uint32_t mine[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t r = r0 + tid * kPer + i;
      int32_t first;
      int64_t total;
      mine[i] = r < a.num_requests ? touched(p, r, &first, &total) : 0;
      if (mine[i] > 0 && first + static_cast<int64_t>(mine[i]) > a.max_blocks) {
        flags |= TOPK_DEV_TABLE_FULL;
        mine[i] = first < a.max_blocks ? static_cast<uint32_t>(a.max_blocks - first) : 0;
      }
      sum += mine[i];
    }
    uint32_t pre = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(~0u, pre, d);
      if (lane >= d) pre += x;
    }
    if (lane == 31) warp_sum[warp] = pre;
    __syncthreads();
    uint32_t at = pre - sum, all = 0;
    for (int w = 0; w < kMeanThreads / 32; ++w) {
      if (w < warp) at += warp_sum[w];
      all += warp_sum[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      start[tid * kPer + i] = at;
      at += mine[i];
    }
    __syncthreads();
    for (uint32_t v = blockIdx.x; v < all * p.widths; v += gridDim.x) {
      const uint32_t u = v / p.widths;
      const int c = static_cast<int>(v - u * p.widths) * kMeanColumns + lane;
      uint32_t j = 0;  // the last request whose start is at or before u
#pragma unroll
      for (uint32_t step = kSegment / 2; step > 0; step >>= 1)
        if (start[j + step] <= u) j += step;
      int32_t first;
      int64_t total;
      touched(p, r0 + j, &first, &total);
      const int32_t column = first + static_cast<int32_t>(u - start[j]);
      const int64_t page = a.block_table[(r0 + j) * a.table_stride + column];
      if (page < 0 || page >= a.num_blocks) {
        flags |= TOPK_DEV_BAD_BLOCK;
        continue;
      }
      const int64_t left = total - static_cast<int64_t>(column) * a.block_size;
      const int held = static_cast<int>(left < a.block_size ? left : a.block_size);
      const int per_head = a.dk / 8, head = c / per_head, d = (c - head * per_head) * 8;
      float s[8] = {};
      if (c < p.columns) {
        const uint16_t* k = static_cast<const uint16_t*>(a.k) + page * a.k_block_stride + head * a.k_head_stride + d;
        constexpr int kAtOnce = 16;
        const int64_t step = kTeams * a.k_token_stride;
        k += warp * a.k_token_stride;
        for (int t = warp; t < held; t += kAtOnce * kTeams, k += kAtOnce * step) {
          uint4 x[kAtOnce];
          const int here = (held - t + kTeams - 1) / kTeams;  // tokens left of this team's
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) x[i] = fetch(i < here ? k + i * step : k);
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            float v8[8];
            widen<kBf16>(x[i], v8);
            if (i < here) {
#pragma unroll
              for (int e = 0; e < 8; ++e) s[e] += v8[e];
            }
          }
        }
      }
      part[tid][0] = make_float4(s[0], s[1], s[2], s[3]);
      part[tid][1] = make_float4(s[4], s[5], s[6], s[7]);
      __syncthreads();
      if (warp == 0 && c < p.columns) {
#pragma unroll
        for (int i = 1; i < kTeams; ++i) {
          const float4 x = part[tid + i * kMeanColumns][0], y = part[tid + i * kMeanColumns][1];
          s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w;
          s[4] += y.x, s[5] += y.y, s[6] += y.z, s[7] += y.w;
        }
        const float n = static_cast<float>(held);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.means) + page * a.mean_block_stride + head * a.mean_head_stride + d) =
            make_uint4(narrow<kBf16>(s[0] / n, s[1] / n), narrow<kBf16>(s[2] / n, s[3] / n), narrow<kBf16>(s[4] / n, s[5] / n),
                       narrow<kBf16>(s[6] / n, s[7] / n));
      }
      __syncthreads();  // the next unit writes the parts again
    }
    __syncthreads();  // the next segment writes the starts again
  }
  if (flags) atomicOr(p.R.status, flags);
}

// ---- scores -----------------------------------------------------------------

struct ScoreParams {
  topk_block_scores_args a;
  Rows R;
  int32_t group;
  int32_t tile_rows;      // rows of a tile: of one request where next_n says whose they are, else neighbours
  int32_t request_tiles;  // tiles of a request, 0: of all rows
  int64_t tiles;
  int32_t heads;    // of a window: those whose queries are held at a time
  int32_t windows;  // of the heads
  int32_t slices;
};

__device__ __forceinline__ int seen_blocks(const ScoreParams& p, int tokens) {
  return tokens == 0 ? 0 : static_cast<int>(min(static_cast<int64_t>(block_column(p.R, tokens - 1)) + 1, p.a.max_columns));
}

__device__ __forceinline__ int steps_of(int blocks, int size) { return static_cast<int>((blocks + (size - 1u)) / size); }  // without a sum past 2^31

// The rows [row0, end) of a tile, and within them runs of rows of the same request: those from row0 on.
struct TileRows {
  int64_t row0, end;
  __device__ __forceinline__ TileRows(const ScoreParams& p, int64_t tile) {
    if (p.request_tiles > 0) {
      const int64_t request = p.request_tiles == 1 ? tile : static_cast<uint32_t>(tile) / static_cast<uint32_t>(p.request_tiles);  // there are no more tiles than rows
      row0 = request * p.R.next_n + (tile - request * p.request_tiles) * p.tile_rows;
      end = min(row0 + p.tile_rows, (request + 1) * p.R.next_n);
    } else {
      row0 = tile * p.tile_rows;
      end = min(row0 + p.tile_rows, p.R.num_rows);
    }
  }
  // Length of the run at row0, its request, and the blocks that its rows see at most.
  __device__ __forceinline__ int run(const ScoreParams& p, int64_t* request, int* most) const {
    *request = row_request(p.R, row0);
    *most = 0;
    if (p.request_tiles > 0) {  // all rows of the tile; loads that do not wait for one another
      const int n = static_cast<int>(end - row0);
      int32_t longest = 0;
#pragma unroll 16
      for (int i = 0; i < n; ++i) longest = max(longest, p.R.lengths[row0 + i]);
      *most = seen_blocks(p, seen_tokens(p.R, longest, *request));
      return n;
    }
    int n = 0;
    for (; row0 + n < end; ++n) {
      if (n > 0 && row_request(p.R, row0 + n) != *request) break;
      *most = max(*most, seen_blocks(p, seen_tokens(p.R, p.R.lengths[row0 + n], *request)));
    }
    return n;
  }
  // Steps of `size` blocks for all runs.
  __device__ __forceinline__ int64_t steps(const ScoreParams& p, int size) const {
    TileRows t = *this;
    int64_t sum = 0, request;
    int most;
    while (t.row0 < t.end) {
      t.row0 += t.run(p, &request, &most);
      sum += steps_of(most, size);
    }
    return sum;
  }
};

// A CTA's share of all tiles' steps, which are dealt to the slices in equal numbers, in order.
struct Share {
  int64_t tile, skip, left;  // the first step: so many steps into that tile; and how many there are
};

template <int kThreads>
__device__ __forceinline__ Share find_share(const ScoreParams& p, int slice, int size, int times) {
  __shared__ int64_t sums[kThreads / 32];
  __shared__ Share share;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t per = (p.tiles + kThreads - 1) / kThreads, t0 = min(per * tid, p.tiles), t1 = min(t0 + per, p.tiles);
  int64_t mine = 0;
  for (int64_t t = t0; t < t1; ++t) mine += TileRows(p, t).steps(p, size) * times;
  int64_t pre = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, pre, d);
    if (lane >= d) pre += x;
  }
  if (lane == 31) sums[warp] = pre;
  if (tid == 0) share = Share{0, 0, 0};
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) pre += sums[w];
    total += sums[w];
  }
  const int64_t begin = slice_begin(total, p.slices, slice);
  int64_t at = pre - mine;
  if (begin >= at && begin < pre) {
    for (int64_t t = t0; t < t1; ++t) {
      const int64_t n = t + 1 < t1 ? TileRows(p, t).steps(p, size) * times : pre - at;  // of the last one what is left
      if (begin < at + n) {
        share = Share{t, begin - at, slice_begin(total, p.slices, slice + 1) - begin};
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  return share;
}

// Every row's number of blocks, and what was wrong with the rows.
__device__ __forceinline__ void write_lens(const ScoreParams& p) {
  uint32_t bits = 0;
  const int64_t all = p.R.num_rows * p.a.kv_heads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < all; i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i / p.a.kv_heads, request = row_request(p.R, row);
    const int32_t given = p.R.lengths[row], n = seen_tokens(p.R, given, request);
    if (request >= p.R.num_requests) bits |= TOPK_DEV_BAD_BLOCK;
    if (request >= 0 && request < p.R.num_requests && (given < 0 || given > p.R.max_len)) bits |= TOPK_DEV_LENGTH_CLAMPED;
    if (n > 0 && block_column(p.R, n - 1) >= p.a.max_columns) bits |= TOPK_DEV_LENGTH_CLAMPED;
    p.a.score_lens[i] = seen_blocks(p, n);
  }
  if (bits) atomicOr(p.R.status, bits);
}

// What stands for a block's score: those that are always selected, and those that cannot be.
__device__ __forceinline__ float final_score(const ScoreParams& p, float score, bool read, int block, int blocks) {
  return !read ? -INFINITY : block < p.a.sink_blocks || block >= blocks - p.a.recent_blocks ? INFINITY : score;
}

// -- few rows

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewRows = 4;
// Queries of a tile's rows and some of its heads. Of the 48 KB that a launch may have without asking for more, the kernel's own arrays and
// what the system keeps of each CTA's take 1 KB (432 dims of seven heads and four rows, 48 384 bytes, are refused at the launch).
constexpr int kQueryBytes = 46 * 1024;
constexpr int kTurnBlocks = 32;

template <int kRows, bool kBf16>
__global__ void __launch_bounds__(kFewThreads, 2) few_kernel(const __grid_constant__ ScoreParams p) {
  constexpr int kAtOnce = kRows > 2 ? 1 : 2;  // pieces of each mean
  constexpr int kMeans = kRows > 2 ? 4 : 8;
  extern __shared__ __align__(16) float q_sum[];  // [kRows][heads of the window][dk]
  __shared__ int32_t seen[kRows];
  const topk_block_scores_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane & 7, four = lane >> 3;
  const int window = blockIdx.x % p.windows, slice = blockIdx.x / p.windows;
  const int head0 = window * p.heads, heads = min(p.heads, a.kv_heads - head0), pieces = a.dk / 8;
  dependent_wait();
  dependent_launch();
  write_lens(p);
  const Share share = find_share<kFewThreads>(p, slice, kTurnBlocks, 1);
  uint32_t flags = 0;
  int64_t tile = share.tile, skip = share.skip, left = share.left;
  for (; left > 0; ++tile) {
    TileRows t(p, tile);
    while (left > 0 && t.row0 < t.end) {
      int64_t request;
      int most;
      const int64_t row0 = t.row0;
      const int rows = t.run(p, &request, &most), groups = steps_of(most, kTurnBlocks);
      t.row0 += rows;
      if (skip >= groups) {
        skip -= groups;
        continue;
      }
      const int first = static_cast<int>(skip), count = static_cast<int>(min(static_cast<int64_t>(groups - first), left));
      skip = 0;
      left -= count;
      __syncthreads();  // the last rows' queries have been read
      if (tid < kRows) seen[tid] = tid < rows ? seen_blocks(p, seen_tokens(p.R, p.R.lengths[row0 + tid], request)) : 0;
      for (int i = tid; i < kRows * heads * pieces; i += kFewThreads) {
        const int at = i / pieces, d = (i - at * pieces) * 8, r = at / heads, head = head0 + at - r * heads;
        float s[8] = {};
        if (r < rows) {
          const uint16_t* q = static_cast<const uint16_t*>(a.q) + (row0 + r) * a.q_row_stride + static_cast<int64_t>(head * p.group) * a.q_head_stride + d;
#pragma unroll 8
          for (int h = 0; h < p.group; ++h) {
            float v[8];
            widen<kBf16>(*reinterpret_cast<const uint4*>(q + h * a.q_head_stride), v);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += v[e];
          }
        }
        float4* to = reinterpret_cast<float4*>(q_sum + static_cast<int64_t>(at) * a.dk + d);
        to[0] = make_float4(s[0], s[1], s[2], s[3]);
        to[1] = make_float4(s[4], s[5], s[6], s[7]);
      }
      // a warp's turn: 32 blocks of a head; neighbouring warps have the same blocks' next heads, which lie side by side
      const int turns = count * heads;
      const int32_t* table = p.R.block_table + request * p.R.table_stride;
      const auto page_of = [&](int turn) {
        const int j = (first + turn / heads) * kTurnBlocks + lane;
        return turn < turns && j < most ? table[j] : -1;
      };
      int32_t next = page_of(warp);
      __syncthreads();
      for (int turn = warp; turn < turns; turn += kFewWarps) {
        const int block0 = (first + turn / heads) * kTurnBlocks, at = turn - turn / heads * heads, head = head0 + at;
        const int32_t page = next;
        next = page_of(turn + kFewWarps);
        const bool in = page >= 0 && page < p.R.num_blocks;
        if (!in && block0 + lane < most) flags |= TOPK_DEV_BAD_BLOCK;
        const unsigned there = __ballot_sync(~0u, in);
        const uint16_t* mine = static_cast<const uint16_t*>(a.means) + static_cast<int64_t>(in ? page : 0) * a.mean_block_stride + head * a.mean_head_stride;
        // eight lanes to a mean, four means at a time: block 4 c + four in step c
        float s[8][kRows] = {};
#pragma unroll 1
        for (int piece0 = 0; piece0 < pieces; piece0 += 8 * kAtOnce) {
          uint4 x[8][kAtOnce];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int from = c * 4 + four;
            const uint16_t* mean = reinterpret_cast<const uint16_t*>(__shfl_sync(~0u, reinterpret_cast<uint64_t>(mine), from));
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
              const int piece = piece0 + i * 8 + sub;
              x[c][i] = (there >> from & 1) && piece < pieces ? *reinterpret_cast<const uint4*>(mean + piece * 8) : make_uint4(0, 0, 0, 0);
            }
          }
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            const int piece = piece0 + i * 8 + sub;
            if (piece >= pieces) break;
            const float* q = q_sum + at * a.dk + piece * 8;
            // four dims of some means at a time, for which every row's queries are read once
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
#pragma unroll
              for (int c = 0; c < 8; c += kMeans) {
                float2 lo[kMeans], hi[kMeans];
#pragma unroll
                for (int k = 0; k < kMeans; ++k) {
                  lo[k] = widen2<kBf16>(e == 0 ? x[c + k][i].x : x[c + k][i].z);
                  hi[k] = widen2<kBf16>(e == 0 ? x[c + k][i].y : x[c + k][i].w);
                }
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                  const float4 y = *reinterpret_cast<const float4*>(q + r * heads * a.dk + e);
#pragma unroll
                  for (int k = 0; k < kMeans; ++k) s[c + k][r] = fmaf(lo[k].x, y.x, fmaf(lo[k].y, y.y, fmaf(hi[k].x, y.z, fmaf(hi[k].y, y.w, s[c + k][r]))));
                }
              }
            }
          }
        }
        // sums over the eight lanes, of which lane `sub` ends with step c = sub's: block 4 sub + four
        const int j = block0 + 4 * sub + four;
        const bool read = there >> (4 * sub + four) & 1;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          float t8[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) t8[c] = s[c][r];
#pragma unroll
          for (int w = 4; w > 0; w >>= 1) {
            const bool up = sub & w;
#pragma unroll
            for (int i = 0; i < w; ++i) {
              const float keep = up ? t8[i + w] : t8[i], send = up ? t8[i] : t8[i + w];
              t8[i] = keep + __shfl_xor_sync(~0u, send, w);
            }
          }
          const int n = seen[r];
          if (r < rows && j < n) a.scores[(row0 + r) * a.score_row_stride + head * a.score_head_stride + j] = final_score(p, t8[0], read, j, n);
        }
      }
    }
    skip = 0;
  }
  if (flags) atomicOr(p.R.status, flags);
}

template <int kRows, bool kBf16>
int launch_few(ScoreParams& p, int sms, cudaStream_t stream) {
  const topk_block_scores_args& a = p.a;
  const int fit = kQueryBytes / (kRows * a.dk * static_cast<int>(sizeof(float)));
  p.heads = fit < kFewWarps ? (fit < a.kv_heads ? fit : a.kv_heads) : (kFewWarps < a.kv_heads ? kFewWarps : a.kv_heads);
  p.windows = (a.kv_heads + p.heads - 1) / p.heads;
  const int64_t columns = a.rows.max_blocks < a.max_columns ? a.rows.max_blocks : a.max_columns;
  const int64_t most = a.rows.num_rows * ((columns + kTurnBlocks - 1) / kTurnBlocks), ctas = (2ll * sms + p.windows - 1) / p.windows;
  p.slices = static_cast<int32_t>(ctas < most ? ctas : most);
  return launch(few_kernel<kRows, kBf16>, static_cast<const ScoreParams&>(p), static_cast<int64_t>(p.slices) * p.windows, kFewThreads, sizeof(float) * kRows * p.heads * a.dk, stream);
}

// -- many rows

constexpr int kManyThreads = 128;
constexpr int kManyDk = 256, kManyGroup = 32;
constexpr int kTile = 128;           // blocks, and columns (row, head) at most
constexpr int kChunk = kTile * 128;  // bytes of 64 dims

// kGroup: heads of a group, 0: any number.
template <int kGroup, bool kBf16>
__global__ void __launch_bounds__(kManyThreads, 3) many_kernel(const __grid_constant__ ScoreParams p) {
  using namespace umma;
  extern __shared__ __align__(1024) uint8_t raw[];
  const topk_block_scores_args& a = p.a;
  const int chunks = (a.dk + 63) / 64, pieces = (chunks + 1) / 2;
  const uint32_t q_at = (smem_addr(raw) + 1023) & ~1023u, means_at = q_at + chunks * kChunk;
  __shared__ __align__(16) int32_t seen[kTile];  // blocks of each row, 0 behind the last one
  __shared__ uint64_t done;
  __shared__ uint32_t tmem_at, gave_up;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = kGroup > 0 ? kGroup : p.group;
  const Guard guard{&gave_up, p.R.status};
  if (tid == 0) {
    mbar_init(smem_addr(&done), 1);
    gave_up = 0;
    fence_async();
  }
  if (warp == 0) tmem_alloc(smem_addr(&tmem_at), kTile);
  dependent_wait();
  dependent_launch();
  write_lens(p);
  const Share share = find_share<kManyThreads>(p, blockIdx.x, kTile, a.kv_heads);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_at;
  constexpr uint32_t kFormat = kBf16 ? kBF16 : kF16;
  uint32_t flags = 0, products = 0;
  int64_t skip = share.skip, left = share.left;
  TokenCopies copies(warp * 32, lane);
  for (int64_t tile = share.tile; left > 0; ++tile) {
    TileRows t(p, tile);
    while (left > 0 && t.row0 < t.end) {
      int64_t request;
      int most;
      const int64_t row0 = t.row0;
      const int rows = t.run(p, &request, &most), steps = steps_of(most, kTile);
      t.row0 += rows;
      if (skip >= static_cast<int64_t>(steps) * a.kv_heads) {
        skip -= static_cast<int64_t>(steps) * a.kv_heads;
        continue;
      }
      seen[tid] = tid < rows ? seen_blocks(p, seen_tokens(p.R, p.R.lengths[row0 + tid], request)) : 0;
      const int cols = rows * group;
      const uint32_t inst = instruction(kFormat, (cols + 15) / 16 * 16, false);
      const int32_t* table = p.R.block_table + request * p.R.table_stride;
      for (int head = static_cast<int>(skip / steps); left > 0 && head < a.kv_heads; ++head) {
        const int first = static_cast<int>(skip % steps), count = static_cast<int>(min(static_cast<int64_t>(steps - first), left));
        skip = 0;
        left -= count;
        // queries of the head's columns
        for (int n = tid >> 3; n < (cols + 15) / 16 * 16; n += kManyThreads / 8) {
          const int r = n / group;
          const bool real = n < cols;
          const uint16_t* q = static_cast<const uint16_t*>(a.q);
          if (real) q += (row0 + r) * a.q_row_stride + static_cast<int64_t>(head * group + n - r * group) * a.q_head_stride;
          for (int c = 0; c < chunks; ++c) {
            const int dim = c * 64 + (tid & 7) * 8;
            const bool in = real && dim < a.dk;
            copy16(q_at + c * kChunk + n * 128 + (((tid & 7) ^ (n & 7)) << 4), in ? q + dim : static_cast<const uint16_t*>(a.q), in ? 16 : 0);
          }
        }
        // a step's means; `in`: whether this thread's block has one
        const auto copy_means = [&](int step, uint32_t to, int32_t page) {
          const int j = step * kTile + tid;
          const bool in = j < most && page >= 0 && page < p.R.num_blocks;
          if (!in && j < most) flags |= TOPK_DEV_BAD_BLOCK;
          copies.aim(static_cast<const char*>(a.means) + 2 * (static_cast<int64_t>(in ? page : 0) * a.mean_block_stride + head * a.mean_head_stride), in, lane);
          for (int u = 0; u < pieces; ++u) copies.columns(to + u * 2 * kChunk, kChunk, u * 256, a.dk * 2, a.means);
          asm volatile("cp.async.commit_group;" ::: "memory");
          return in;
        };
        const auto page_of = [&](int step) { return step < first + count && step * kTile + tid < most ? table[step * kTile + tid] : -1; };
        int32_t page = page_of(first), next_page = page_of(first + 1);
        asm volatile("" ::"r"(page), "r"(next_page) : "memory");  // before the copies: a load waits behind those
        bool in = copy_means(first, means_at, page);
        for (int step = first; step < first + count; ++step) {
          const bool more = step + 1 < first + count;
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          fence_async();
          __syncthreads();
          if (warp == 0) {
            fence_after();
            uint32_t k = means_at, q = q_at;
            int dims = a.dk;
            bool add = false;
#pragma unroll 1
            for (; dims >= 64; dims -= 64, k += kChunk, q += kChunk, add = true) mma16_chunk(tmem, operand(k, 16), operand(q, 16), inst, add);
#pragma unroll 1
            for (; dims > 0; dims -= 16, k += 32, q += 32, add = true) mma16_step(tmem, operand(k, 16), operand(q, 16), inst, add);
            commit(smem_addr(&done));
          }
          mbar_wait_warp(smem_addr(&done), products++ & 1, guard);
          fence_after();
          const int j = step * kTile + tid;
          float* to = a.scores + row0 * a.score_row_stride + head * a.score_head_stride + j;
          const uint32_t from = tmem + (static_cast<uint32_t>(warp * 32) << 16);
          if constexpr (kGroup > 0) {
            constexpr int kSpan = kGroup >= 8 ? 64 : kGroup > 1 ? 32 : 16, kRows = kSpan / kGroup;  // columns at a time
            const float always = in ? INFINITY : -INFINITY;  // what the score is where it is not the sum
            const bool fixed = !in || j < a.sink_blocks;
#pragma unroll 1
            for (int c = 0; c < cols; c += kSpan) {
              float v[kSpan];
              if constexpr (kSpan == 64)
                tmem_load64(from + c, v);
              else
                tmem_load(from + c, v);
              const int32_t* n = seen + c / kGroup;
#pragma unroll
              for (int r = 0; r < kRows; ++r) {
                float* x = v + r * kGroup;
#pragma unroll
                for (int w = kGroup / 2; w > 0; w >>= 1)
#pragma unroll
                  for (int i = 0; i < w; ++i) x[i] += x[i + w];
                if (j < n[r]) to[r * a.score_row_stride] = fixed || j >= n[r] - a.recent_blocks ? always : x[0];
              }
              to += kRows * a.score_row_stride;
            }
          } else {
            int r = 0, held = 0;
            float sum = 0.f;
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) {
              float v[32];
              tmem_load(from + c, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                sum += v[i];
                if (++held == group) {
                  if (r < rows && j < seen[r]) *to = final_score(p, sum, in, j, seen[r]);
                  to += a.score_row_stride;
                  ++r;
                  held = 0;
                  sum = 0.f;
                }
              }
            }
          }
          fence_before();
          __syncthreads();  // the sums have been read, and the means' place may be filled again
          if (more) {
            page = next_page;
            next_page = page_of(step + 2);
            in = copy_means(step + 1, means_at, page);
          }
        }
      }
    }
    skip = 0;
  }
  if (flags) atomicOr(p.R.status, flags);
  settle(guard);
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) tmem_free(tmem, kTile);
}

template <int kGroup, bool kBf16>
int launch_many(ScoreParams& p, int device, const topk_device_props& props, cudaStream_t stream) {
  static int granted[kMaxDevices];
  const topk_block_scores_args& a = p.a;
  const size_t smem = 2 * ((a.dk + 63) / 64) * static_cast<size_t>(kChunk) + 1024;
  const int rc = allow_smem(many_kernel<kGroup, kBf16>, 2 * (kManyDk / 64) * static_cast<size_t>(kChunk) + 1024, device, granted);
  if (rc != TOPK_OK) return rc;
  const int64_t columns = a.rows.max_blocks < a.max_columns ? a.rows.max_blocks : a.max_columns;
  const int64_t most = a.rows.num_rows * a.kv_heads * ((columns + kTile - 1) / kTile);
  const int64_t held = props.max_smem_optin / (smem + 2048), ctas = props.num_sms * (held < 1 ? 1 : (held > 4 ? 4 : held));  // 4: of 512 columns of tensor memory
  p.slices = static_cast<int32_t>(ctas < most ? ctas : most);
  return launch(many_kernel<kGroup, kBf16>, static_cast<const ScoreParams&>(p), p.slices, kManyThreads, smem, stream);
}

template <bool kBf16>
int run_scores(ScoreParams& p, bool many, int device, const topk_device_props& props, cudaStream_t stream) {
  if (many) {
    switch (p.group) {
      case 1: return launch_many<1, kBf16>(p, device, props, stream);
      case 2: return launch_many<2, kBf16>(p, device, props, stream);
      case 4: return launch_many<4, kBf16>(p, device, props, stream);
      case 8: return launch_many<8, kBf16>(p, device, props, stream);
      case 16: return launch_many<16, kBf16>(p, device, props, stream);
      case 32: return launch_many<32, kBf16>(p, device, props, stream);
      default: return launch_many<0, kBf16>(p, device, props, stream);
    }
  }
  if (p.tile_rows <= 1) return launch_few<1, kBf16>(p, props.num_sms, stream);
  if (p.tile_rows <= 2) return launch_few<2, kBf16>(p, props.num_sms, stream);
  return launch_few<4, kBf16>(p, props.num_sms, stream);
}

static_assert(kFewRows * kMaxDk * sizeof(float) <= kQueryBytes, "queries of a tile");

bool two_bytes(int dtype) { return dtype == TOPK_DTYPE_F16 || dtype == TOPK_DTYPE_BF16; }

}  // namespace
}  // namespace paged
}  // namespace ltk

extern "C" int topk_block_means(const topk_block_means_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_block_means_args& a = *args;
  if (a.num_requests < 0 || a.num_requests > INT32_MAX || a.block_size < 1 || a.max_blocks < 1 || a.max_blocks > INT32_MAX ||
      a.table_stride < a.max_blocks || a.num_blocks < 0 || a.num_blocks > INT32_MAX || a.kv_heads < 1)
    return TOPK_ERR_INVALID_ARG;
  if (!two_bytes(a.dtype) || a.kv_heads > 1024 || a.dk < 8 || a.dk > kMaxDk || a.dk % 8) return TOPK_ERR_UNSUPPORTED;
  const int64_t widths = (a.kv_heads * (a.dk / 8) + kMeanColumns - 1) / kMeanColumns;
  if ((a.num_requests < kSegment ? a.num_requests : kSegment) * a.max_blocks > INT32_MAX / widths) return TOPK_ERR_UNSUPPORTED;
  if (a.num_requests == 0) return TOPK_OK;
  if (a.context_lens == nullptr || a.new_lens == nullptr || a.block_table == nullptr || a.k == nullptr || a.means == nullptr ||
      a.workspace == nullptr)
    return TOPK_ERR_INVALID_ARG;
  if (misaligned(a.context_lens, 4) || misaligned(a.new_lens, 4) || misaligned(a.block_table, 4) || misaligned(a.k, 16) ||
      a.k_block_stride % 8 || a.k_token_stride % 8 || a.k_head_stride % 8 || misaligned(a.means, 16) || a.mean_block_stride % 8 ||
      a.mean_head_stride % 8 || misaligned(a.workspace, 16))
    return TOPK_ERR_MISALIGNED;
  const int sms = num_sms();
  if (sms < 1) return TOPK_ERR_CUDA;
  MeanParams p{};
  p.a = a;
  topk_paged_rows rows{};
  rows.block_size = a.block_size;
  rows.max_blocks = a.max_blocks;
  p.R = make_rows(rows, INT32_MAX, a.workspace);
  p.columns = a.kv_heads * (a.dk / 8);
  p.widths = static_cast<uint32_t>(widths);
  // Pages are not known here: as many CTAs as the SMs hold, each with every so manieth unit.
  const int64_t grid = sms * 5;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.dtype == TOPK_DTYPE_BF16 ? launch(means_kernel<true>, static_cast<const MeanParams&>(p), grid, kMeanThreads, 0, s)
                                    : launch(means_kernel<false>, static_cast<const MeanParams&>(p), grid, kMeanThreads, 0, s);
}

extern "C" int topk_block_scores(const topk_block_scores_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_block_scores_args& a = *args;
  int rc = check_rows(a.rows);
  if (rc != TOPK_OK) return rc;
  if (a.heads < 1 || a.kv_heads < 1 || a.heads % a.kv_heads != 0 || a.sink_blocks < 0 || a.recent_blocks < 0 || a.max_columns < 1 ||
      a.score_row_stride < 0 || a.score_head_stride < 0)
    return TOPK_ERR_INVALID_ARG;
  if (!two_bytes(a.dtype) || a.heads > 1024 || a.dk < 8 || a.dk > kMaxDk || a.dk % 8) return TOPK_ERR_UNSUPPORTED;
  if (a.rows.num_rows == 0) return TOPK_OK;
  rc = check_row_pointers(a.rows);
  if (rc != TOPK_OK) return rc;
  if (a.q == nullptr || a.means == nullptr || a.scores == nullptr || a.score_lens == nullptr || a.workspace == nullptr) return TOPK_ERR_INVALID_ARG;
  if (misaligned(a.q, 16) || a.q_row_stride % 8 || a.q_head_stride % 8 || misaligned(a.means, 16) || a.mean_block_stride % 8 ||
      a.mean_head_stride % 8 || misaligned(a.scores, 4) || misaligned(a.score_lens, 4) || misaligned(a.workspace, 16))
    return TOPK_ERR_MISALIGNED;
  int device = 0;
  topk_device_props props{};
  if (cudaGetDevice(&device) != cudaSuccess || topk_query_device(device, &props) != TOPK_OK) {
    cudaGetLastError();
    return TOPK_ERR_CUDA;
  }
  ScoreParams p{};
  p.a = a;
  p.R = make_rows(a.rows, INT32_MAX, a.workspace);
  p.group = a.heads / a.kv_heads;
  const int64_t rows = a.rows.num_rows;
  // Rows that read the same means share them: the rows of a request; where each row brings its request, as many
  // neighbours as a request has rows on average. Two and more of them go to the tensor cores, as many as fill 128 columns, unless a
  // group is so large that a row's heads take most of those. (64 requests of 64 K tokens, 64 heads over 8: a row each 29 us this
  // way, 28 by fused multiply-adds; two 30, 32.5; four 32, 42. 16 requests, a row each: 10.5, 8.5. 128 heads over one, two rows each: 27, 18.) A
  // group that is no power of two has no kernel of its own there, and goes from four rows on (groups of 3, two rows: 43, 33; of 24,
  // three: 18, 13; of 7, four: 44, 51).
  int64_t share = a.rows.next_n;
  if (a.rows.row_request != nullptr) share = a.rows.num_requests > 0 ? (rows + a.rows.num_requests - 1) / a.rows.num_requests : 1;
  const int least = (p.group & (p.group - 1)) == 0 ? 2 : 4;
  const bool many = a.dk <= kManyDk && p.group <= kManyGroup && share >= least;
  const int most = many ? kTile / p.group : kFewRows;
  p.tile_rows = static_cast<int32_t>(share < most ? share : most);
  if (a.rows.row_request == nullptr) {
    p.request_tiles = (a.rows.next_n + p.tile_rows - 1) / p.tile_rows;
    p.tiles = rows / a.rows.next_n * p.request_tiles;
  } else {
    p.tiles = (rows + p.tile_rows - 1) / p.tile_rows;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.dtype == TOPK_DTYPE_BF16 ? run_scores<true>(p, many, device, props, s) : run_scores<false>(p, many, device, props, s);
}
