// Mean keys of pages (topk_block_means) and the scores that rows give blocks by them (topk_block_scores).
//
//   means[b, g, :] = 1/n sum_t k[b, t, g, :]           scores[r, g, j] = (sum_h q[r, h, :]) . means[page of j, g, :]
//
// The sum over a group's heads comes first, so that a score is one product of dk elements whatever the group's size.
//
// Means. The keys of a page are a matrix, tokens by (head, dim), and a unit is 512 bytes of its width; a thread sums 16 bytes of
// a token's row over every fourth token, eight loads at a time, and the threads of one column meet in shared memory, in
// a fixed order. Units are found as the map finds its tokens: every CTA sums the requests' pages up. Bound by HBM for
// prompts, by latency for the page or so that a decode step touches of each request.
//
// Scores. A warp has 32 blocks of one head and up to eight rows of a request: eight lanes read a mean, 128 bytes at a time,
// and multiply it with the rows' queries, whose sums over the group stand in shared memory. (A thread to each mean would read
// the same bytes, but 16 of every line at a time: 52 us against LEAVE for 64 rows.) The means, which are all there
// is to read for a few rows, stream from HBM; many rows of one request are bound by the fused multiply-adds.
#include "paged.cuh"

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
  int32_t widths;   // units of a page
};

// New pages of a request: the first one's column, and how many.
__device__ __forceinline__ int touched(const MeanParams& p, int64_t r, int32_t* first, int64_t* total) {
  const int64_t had = p.a.context_lens[r] > 0 ? p.a.context_lens[r] : 0, more = p.a.new_lens[r] > 0 ? p.a.new_lens[r] : 0;
  *total = had + more < INT32_MAX ? had + more : INT32_MAX;  // positions stay below 2^31
  *first = block_column(p.R, static_cast<int>(had));
  return more == 0 || *total <= had ? 0 : block_column(p.R, static_cast<int>(*total - 1)) - *first + 1;
}

template <bool kBf16>
__global__ void __launch_bounds__(kMeanThreads) means_kernel(const __grid_constant__ MeanParams p) {
  __shared__ uint32_t start[kSegment + 1];
  __shared__ uint32_t warp_sum[kMeanThreads / 32];
  __shared__ float4 part[kMeanThreads][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const topk_block_means_args& a = p.a;
  constexpr int kPer = kSegment / kMeanThreads;
  dependent_wait();
  dependent_launch();
  uint32_t flags = 0;
  int64_t before = 0;  // pages of earlier segments
  for (int64_t r0 = 0; r0 < a.num_requests; r0 += kSegment) {
    // the segment's new pages, and each request's first among them (32 bits do: they are entries of the table)
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
    // this CTA's first unit of the segment
    const int64_t units = static_cast<int64_t>(all) * p.widths, done = before * p.widths;
    const int64_t skipped = (done + gridDim.x - 1 - blockIdx.x) / gridDim.x * gridDim.x + blockIdx.x - done;
    for (int64_t v = skipped; v < units; v += gridDim.x) {
      const uint32_t u = static_cast<uint32_t>(v / p.widths);
      const int c = static_cast<int>(v - static_cast<int64_t>(u) * p.widths) * kMeanColumns + lane;
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
        constexpr int kAtOnce = 8;
        for (int t = warp; t < held; t += kAtOnce * kTeams) {
          uint4 x[kAtOnce];
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) x[i] = fetch(k + static_cast<int64_t>(min(t + i * kTeams, held - 1)) * a.k_token_stride);
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            if (t + i * kTeams >= held) break;
            float v8[8];
            widen<kBf16>(x[i], v8);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += v8[e];
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
    before += all;
    __syncthreads();  // the next segment writes the starts again
  }
  if (flags) atomicOr(p.R.status, flags);
}

// ---- scores -----------------------------------------------------------------

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kTileRows = 8;
constexpr int kQueryBytes = 48 * 1024;  // queries of a tile's rows and some of its heads

struct ScoreParams {
  topk_block_scores_args a;
  Rows R;
  int32_t group;
  int32_t tile_rows;      // rows of a tile: of one request where next_n says whose they are, else neighbours
  int32_t request_tiles;  // tiles of a request, 0: of all rows
  int64_t tiles;
  int32_t heads;    // of a window: those whose queries are held at a time
  int32_t windows;  // of the heads
  int32_t splits;   // CTAs that share a tile's blocks
};

__device__ __forceinline__ int seen_blocks(const ScoreParams& p, int tokens) {
  return tokens == 0 ? 0 : static_cast<int>(min(static_cast<int64_t>(block_column(p.R, tokens - 1)) + 1, p.a.max_columns));
}

template <int kRows, bool kBf16>
__global__ void __launch_bounds__(kScoreThreads, 2) scores_kernel(const __grid_constant__ ScoreParams p) {
  constexpr int kAtOnce = kRows > 2 ? 1 : 2;  // pieces of each mean
  constexpr int kMeans = kRows > 2 ? 4 : 8;
  extern __shared__ __align__(16) float q_sum[];  // [kRows][heads of the window][dk]
  __shared__ int32_t seen[kRows];
  const topk_block_scores_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane & 7, four = lane >> 3;
  const int split = blockIdx.x % p.splits, window = blockIdx.x / p.splits % p.windows;
  const int64_t tile = blockIdx.x / p.splits / p.windows;
  const int head0 = window * p.heads, heads = min(p.heads, a.kv_heads - head0), pieces = a.dk / 8;
  dependent_wait();
  dependent_launch();
  int64_t row0, row_end;  // of the tile
  if (p.request_tiles > 0) {
    const int64_t request = tile / p.request_tiles;
    row0 = request * p.R.next_n + (tile - request * p.request_tiles) * p.tile_rows;
    row_end = min(row0 + p.tile_rows, (request + 1) * p.R.next_n);
  } else {
    row0 = tile * p.tile_rows;
    row_end = min(row0 + p.tile_rows, p.R.num_rows);
  }
  uint32_t flags = 0;
  while (row0 < row_end) {
    // the rows from here on that have the same request
    const int64_t request = row_request(p.R, row0);
    int rows = 1;
    while (row0 + rows < row_end && row_request(p.R, row0 + rows) == request) ++rows;
    __syncthreads();  // the last rows' queries have been read
    if (tid < kRows) {
      const int n = tid < rows ? seen_tokens(p.R, p.R.lengths[row0 + tid], request) : 0;
      seen[tid] = seen_blocks(p, n);
      if (tid < rows && n > 0 && block_column(p.R, n - 1) >= a.max_columns) flags |= TOPK_DEV_LENGTH_CLAMPED;
    }
    for (int i = tid; i < kRows * heads * pieces; i += kScoreThreads) {
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
    __syncthreads();
    int most = 0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) most = max(most, seen[r]);
    if (split == 0)
      for (int i = tid; i < rows * heads; i += kScoreThreads) a.score_lens[(row0 + i / heads) * a.kv_heads + head0 + i % heads] = seen[i / heads];
    // a warp's turn: 32 blocks of a head; neighbouring warps have the same blocks' next heads, which lie side by side
    const int turns = (most + 31) / 32 * heads;
    for (int turn = split * kScoreWarps + warp; turn < turns; turn += p.splits * kScoreWarps) {
      const int block0 = turn / heads * 32, at = turn - turn / heads * heads, head = head0 + at;
      int64_t page = -1;
      if (block0 + lane < most) page = p.R.block_table[request * p.R.table_stride + block0 + lane];
      const bool in = page >= 0 && page < p.R.num_blocks;
      if (!in && block0 + lane < most) flags |= TOPK_DEV_BAD_BLOCK;
      const unsigned there = __ballot_sync(~0u, in);
      const uint16_t* mine = static_cast<const uint16_t*>(a.means) + (in ? page : 0) * a.mean_block_stride + head * a.mean_head_stride;
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
        float t[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) t[c] = s[c][r];
#pragma unroll
        for (int w = 4; w > 0; w >>= 1) {
          const bool up = sub & w;
#pragma unroll
          for (int i = 0; i < w; ++i) {
            const float keep = up ? t[i + w] : t[i], send = up ? t[i] : t[i + w];
            t[i] = keep + __shfl_xor_sync(~0u, send, w);
          }
        }
        const int n = seen[r];
        if (r >= rows || j >= n) continue;
        const bool kept = j < a.sink_blocks || j >= n - a.recent_blocks;
        a.scores[(row0 + r) * a.score_row_stride + head * a.score_head_stride + j] = !read ? -INFINITY : kept ? INFINITY : t[0];
      }
    }
    row0 += rows;
  }
  if (blockIdx.x == 0) report_rows(p.R, tid, kScoreThreads);
  if (flags) atomicOr(p.R.status, flags);
}

template <int kRows, bool kBf16>
int launch_scores(ScoreParams& p, int sms, cudaStream_t stream) {
  const topk_block_scores_args& a = p.a;
  const int fit = kQueryBytes / (kRows * a.dk * static_cast<int>(sizeof(float)));
  p.heads = fit < kScoreWarps ? (fit < a.kv_heads ? fit : a.kv_heads) : (kScoreWarps < a.kv_heads ? kScoreWarps : a.kv_heads);
  p.windows = (a.kv_heads + p.heads - 1) / p.heads;
  // CTAs for some rounds of the GPU, if there are blocks for as many: lengths are not known here, and those of a tile that reach
  // past its blocks end at once.
  const int64_t columns = a.rows.max_blocks < a.max_columns ? a.rows.max_blocks : a.max_columns;
  const int64_t units = p.tiles * p.windows, turns = (columns + 31) / 32 * p.heads, most = (turns + kScoreWarps - 1) / kScoreWarps;
  const int64_t wanted = (16ll * sms + units - 1) / units;
  p.splits = static_cast<int32_t>(wanted < most ? wanted : most);
  if (units * p.splits > INT32_MAX) return TOPK_ERR_UNSUPPORTED;
  return launch(scores_kernel<kRows, kBf16>, static_cast<const ScoreParams&>(p), units * p.splits, kScoreThreads, sizeof(float) * kRows * p.heads * a.dk, stream);
}

template <bool kBf16>
int run_scores(ScoreParams& p, int sms, cudaStream_t stream) {
  if (p.tile_rows <= 1) return launch_scores<1, kBf16>(p, sms, stream);
  if (p.tile_rows <= 2) return launch_scores<2, kBf16>(p, sms, stream);
  if (p.tile_rows <= 4) return launch_scores<4, kBf16>(p, sms, stream);
  return launch_scores<8, kBf16>(p, sms, stream);
}

static_assert(kTileRows * kMaxDk * sizeof(float) <= kQueryBytes, "queries of a tile");

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
  if ((a.num_requests < kSegment ? a.num_requests : kSegment) * a.max_blocks > UINT32_MAX) return TOPK_ERR_UNSUPPORTED;
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
  p.widths = (p.columns + kMeanColumns - 1) / kMeanColumns;
  // Pages are not known here: as many CTAs as the SMs hold, each with every so manieth unit.
  const int64_t grid = sms * 10;
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
  const int sms = num_sms();
  if (sms < 1) return TOPK_ERR_CUDA;
  ScoreParams p{};
  p.a = a;
  p.R = make_rows(a.rows, INT32_MAX, a.workspace);
  p.group = a.heads / a.kv_heads;
  const int64_t rows = a.rows.num_rows;
  // Rows that read the same means share them: the rows of a request; where each row brings its request, as many
  // neighbours as a request has rows on average.
  int64_t share = a.rows.next_n;
  if (a.rows.row_request != nullptr) share = a.rows.num_requests > 0 ? (rows + a.rows.num_requests - 1) / a.rows.num_requests : 1;
  p.tile_rows = static_cast<int32_t>(share < kTileRows ? share : kTileRows);
  if (a.rows.row_request == nullptr) {
    p.request_tiles = (a.rows.next_n + p.tile_rows - 1) / p.tile_rows;
    p.tiles = rows / a.rows.next_n * p.request_tiles;
  } else {
    p.tiles = (rows + p.tile_rows - 1) / p.tile_rows;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.dtype == TOPK_DTYPE_BF16 ? run_scores<true>(p, sms, s) : run_scores<false>(p, sms, s);
}
