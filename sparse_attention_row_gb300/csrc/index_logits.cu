// Logits of the sparse-attention indexer over a paged key cache
// (topk_index_logits), on the tensor cores:
//   logits[r, t] = s_t * sum_h w[r, h] * max(0, q[r, h, :] . k[t, :]).
//
// A unit is a few consecutive rows; those that belong to one request (drafted
// tokens, a prompt's piece) share a pass over its keys. A product takes 128 tokens,
//   S^T [128 tokens x N] = K [128 x dim] . Q^T [dim x N],  N = rows x heads <= 256,
// and puts a token's scores for all rows and heads in one lane of tensor memory, so
// that the weighted sum over the heads is one thread's own: no exchange at all.
// There are two places of 256 columns, so that one's sums run while the next is
// multiplied. Two tiles share a place where N <= 128. A step, what is copied at once, is
// two tiles, or one where all passes are wider; where each row brings its request, the
// kernel finds the passes, and a wide one multiplies a step's two tiles one after the other.
//
// The units' steps are dealt in equal runs to the CTAs, one on each SM; every CTA
// sums up the rows' steps to find its run. Rows are independent over the tokens,
// so nothing has to be joined.
//
// Roles in a CTA (19 warps): 2 bring the queries, and one of them (both, where
// pages are no multiples of 8 tokens) the keys by TMA into a ring of steps (cache_map.cuh), a
// warp issues the products, four groups of 4 warps sum: two a step, which take a
// tile each, or half of the rows of the one.
//
// What bounds it. Decoding reads every key once: 32 requests of two rows of 64 heads
// over 100 K to 160 K tokens take 174 us (6.3 TB/s, bf16), 64 rows over 8 K to 32 K
// 8-bit keys 39 us (4.6 TB/s: a step of 32 KB costs some 1400 cycles of hand-overs between
// its warps, about what its data takes). A prompt's piece keeps no unit busy (tensor pipe
// 44%, issue 48%): a place of 256 columns is multiplied in 1024 cycles, in which the
// warps that are to sum it wait, and summed while the other place is multiplied. 512
// rows of 64 heads over 16 K tokens take 122 us (1110 TFLOP/s). All of it depends on short
// loops: spills and unrolled look-ups in them showed (8-bit keys: 57 us with 80 registers
// a thread, 42 with 96, at which 20 bytes a thread are still spilled).
#include "cache_map.cuh"
#include "paged.cuh"
#include "umma.cuh"

namespace ltk {
namespace paged {
namespace {

using namespace ltk::umma;

constexpr int kTile = 128;
constexpr int kChunk = 128 * 128;  // bytes of 128 tokens x 128 bytes
constexpr int kSumWarps = 16, kCopyWarps = 2;
constexpr int kCopyThreads = kCopyWarps * 32;
constexpr int kMmaWarp = kSumWarps + kCopyWarps;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kMaxSlots = 8;
constexpr int kGroup = 4;        // steps whose blocks are looked up together
constexpr int kSegmentSlots = 4;  // a segment's weights are written when at most two segments are still being summed
constexpr int kMaxCols = 256, kMaxRows = 16;

struct Params {
  CacheMap map;
  topk_index_logits_args a;
  Rows R;
  int32_t pack;      // rows of a unit
  int32_t head_cols; // columns of a row: heads rounded up to 16
  int32_t row_bytes; // of a key
  int32_t chunks;    // of 128 bytes
  int32_t tiles;     // of a step: 1 or 2
  int32_t slots;
  int32_t slices;
  int64_t units;
  uint32_t q_bytes;
  uint32_t inst;     // instruction descriptor without N
};

struct Smem {
  float weight[kSegmentSlots][kMaxCols];
  int32_t length[kSegmentSlots][kMaxRows];
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t q_full, q_empty, s_full[2], s_empty[2], segment_full[kSegmentSlots], all_done;
  int64_t scan[kThreads / 32];
  int64_t start_unit, start_at, steps;
  uint32_t tmem, gave_up;
};

__device__ __forceinline__ int steps_of(const Params& p, int length) { return static_cast<int>((length + (p.tiles * kTile - 1u)) / (p.tiles * kTile)); }

// Steps of a unit: those of its passes, each a run of rows of one request (rows that see nothing do not part one).
__device__ __forceinline__ int64_t unit_steps(const Params& p, int64_t u) {
  const int64_t row0 = u * p.pack;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.pack), p.R.num_rows - row0));
  int longest = 0;
  int64_t request = -1, steps = 0;
  for (int j0 = 0; j0 < rows; j0 += 4) {  // four rows' entries on their way at once
    int32_t n[4];
    int64_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = row0 + min(j0 + i, rows - 1);
      n[i] = p.R.lengths[row];
      b[i] = row_request(p.R, row);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = j0 + i < rows ? seen_tokens(p.R, n[i], b[i]) : 0;
      if (c == 0) continue;
      if (b[i] != request) {
        steps += steps_of(p, longest);
        longest = 0;
      }
      request = b[i];
      longest = max(longest, c);
    }
  }
  return steps + steps_of(p, longest);
}

// A slice's run of steps, walked by whole warps segment by segment (a segment: the steps of one pass in the run).
struct Walk {
  int64_t unit, left;
  int64_t row0;      // of the pass
  int64_t request;
  int first, rows;   // the pass's rows within the unit
  int at, count, longest;
  __device__ void pass(const Params& p, int from) {  // the one of row `from` or of a later one; none: longest is 0
    const int lane = threadIdx.x & 31, unit_rows = static_cast<int>(min(static_cast<int64_t>(p.pack), p.R.num_rows - row0));
    int n = 0, b = 0;
    if (lane >= from && lane < unit_rows) {
      const int64_t of = row_request(p.R, row0 + lane);
      n = seen_tokens(p.R, p.R.lengths[row0 + lane], of);
      b = static_cast<int>(of);
    }
    const unsigned seen = __ballot_sync(~0u, n > 0);
    first = seen ? __ffs(seen) - 1 : unit_rows;
    b = n > 0 ? b : -1;
    const int mine = __shfl_sync(~0u, b, first & 31);
    const unsigned others = __ballot_sync(~0u, n > 0 && b != mine);
    const unsigned run = others ? seen & ((1u << (__ffs(others) - 1)) - 1) : seen;
    rows = run ? 32 - __clz(run) - first : 0;
    longest = __reduce_max_sync(~0u, (run >> lane) & 1 ? n : 0);
    request = mine;
  }
  __device__ void enter(const Params& p, int64_t u) {
    unit = u;
    row0 = u * p.pack;
    pass(p, 0);
  }
  __device__ void size(const Params& p) { count = static_cast<int>(min(static_cast<int64_t>(steps_of(p, longest) - at), left)); }
  __device__ void start(const Params& p, int64_t u, int64_t offset) {
    enter(p, u);
    while (offset >= steps_of(p, longest)) {
      offset -= steps_of(p, longest);
      pass(p, first + rows);
    }
    at = static_cast<int>(offset);
    size(p);
  }
  __device__ void next(const Params& p) {
    left -= count;
    at = 0;
    if (left <= 0) return;
    pass(p, first + rows);
    while (longest == 0) enter(p, unit + 1);  // there are steps left, so some later unit has them
    size(p);
  }
  // A product of the pass: both tiles of a step where their columns fit a place of tensor memory side by side, else one.
  __device__ int product_tiles(const Params& p) const { return p.tiles == 2 && rows * p.head_cols <= kMaxCols / 2 ? 2 : 1; }
};

// Where a pass's tokens lie: looked up by the copying warps, and by the summing ones for the scales.
__device__ __forceinline__ int table_entry(const Params& p, const Walk& w, int x) {
  return x < w.longest ? p.R.block_table[w.request * p.R.table_stride + block_column(p.R, x)] : 0;
}
__device__ __forceinline__ bool in_cache(const Params& p, const Walk& w, int x, int b) {
  return x < w.longest && b >= 0 && b < p.R.num_blocks;
}

__device__ __forceinline__ float relu(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}

// s += w * relu(x) for two columns at once.
__device__ __forceinline__ void add_two(uint64_t* s, float w0, float w1, float x0, float x1) {
  asm("{\n .reg .b64 w, x;\n mov.b64 w, {%1, %2};\n mov.b64 x, {%3, %4};\n fma.rn.f32x2 %0, w, x, %0;\n}"
      : "+l"(*s)
      : "f"(w0), "f"(w1), "f"(relu(x0)), "f"(relu(x1)));
}
__device__ __forceinline__ float sum_of_two(uint64_t s) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(s));
  return a + b;
}

// The weighted sums of rows [row, row_end) of one tile for this thread's token. `at`: the first row's columns. kWide: heads
// are a multiple of 32, and the columns are taken 32 at a time, none of which is without a head. (Two sets of 16, one on
// its way while the other is summed, took 147 us where this takes 136, at 512 rows of 64 heads and 16 K tokens: the other
// warps hide the wait as well.)
template <bool kWide>
__device__ __forceinline__ void sum_tile(const Params& p, uint32_t at, const float* weight, const int32_t* length, int row, int row_end,
                                         int pos, float scale, bool found, int64_t row0) {
  if (row >= row_end) return;
  const uint32_t end = at + (row_end - row) * p.head_cols;
  weight += row * p.head_cols;
  float* out = p.a.logits + (row0 + row) * p.a.logits_row_stride + pos;
  constexpr int C = kWide ? 32 : 16;
  int in_row = 0;
  uint64_t s0 = 0, s1 = 0;
#pragma unroll 1
  for (; at < end; at += C) {
    float x[C];
    tmem_load(at, x);
    if (kWide || p.a.heads - in_row >= C) {
#pragma unroll
      for (int i = 0; i < C; i += 4) {
        const float4 w = *reinterpret_cast<const float4*>(weight + i);
        add_two(&s0, w.x, w.y, x[i], x[i + 1]);
        add_two(&s1, w.z, w.w, x[i + 2], x[i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (i < p.a.heads - in_row) add_two(&s0, weight[i], 0.f, x[i], 0.f);
    }
    weight += C;
    in_row += C;
    if (in_row == p.head_cols) {
      if (pos < length[row]) *out = found ? (sum_of_two(s0) + sum_of_two(s1)) * scale : -INFINITY;
      out += p.a.logits_row_stride;
      ++row;
      in_row = 0;
      s0 = s1 = 0;
    }
  }
}

template <bool k8Bit>
__global__ void __launch_bounds__(kThreads, 1) index_logits_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const uint32_t q_at = base, ring = q_at + p.q_bytes, tile_bytes = p.chunks * kChunk, slot_bytes = p.tiles * tile_bytes;
  Smem& sm = *reinterpret_cast<Smem*>(raw + (ring + p.slots * slot_bytes - smem_addr(raw)));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, slice = blockIdx.x;
  const Guard guard{&sm.gave_up, p.R.status};
  if (tid == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(smem_addr(&sm.full[i]), p.map.run_rows ? 1 : kCopyWarps);
      mbar_init(smem_addr(&sm.empty[i]), 1);
    }
    mbar_init(smem_addr(&sm.q_full), kCopyThreads);
    mbar_init(smem_addr(&sm.q_empty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sm.s_full[i]), 1);
      mbar_init(smem_addr(&sm.s_empty[i]), kSumWarps / 2);
    }
    for (int i = 0; i < kSegmentSlots; ++i) mbar_init(smem_addr(&sm.segment_full[i]), kCopyThreads);
    mbar_init(smem_addr(&sm.all_done), 1);
    sm.gave_up = 0;
    fence_async();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&sm.tmem), 2 * kMaxCols);
  dependent_wait();
  dependent_launch();
  {  // where this slice's run begins
    const int64_t per = (p.units + kThreads - 1) / kThreads;
    const int64_t u0 = min(per * tid, p.units), u1 = min(u0 + per, p.units);
    int64_t mine = 0;
    for (int64_t u = u0; u < u1; ++u) mine += unit_steps(p, u);
    int64_t pre = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(~0u, pre, d);
      if (lane >= d) pre += x;
    }
    if (lane == 31) sm.scan[warp] = pre;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) pre += sm.scan[w];
      total += sm.scan[w];
    }
    const int64_t begin = total * slice / p.slices;
    int64_t at = pre - mine;
    if (begin >= at && begin < pre) {
      if (u1 - u0 == 1) {
        sm.start_unit = u0;
        sm.start_at = begin - at;
      }
      for (int64_t u = u0; u1 - u0 > 1 && u < u1; ++u) {
        const int64_t n = unit_steps(p, u);
        if (begin < at + n) {
          sm.start_unit = u;
          sm.start_at = begin - at;
          break;
        }
        at += n;
      }
    }
    if (tid == 0) sm.steps = total;
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;
  Walk walk;
  walk.left = sm.steps * (slice + 1) / p.slices - sm.steps * slice / p.slices;
  if (walk.left > 0) walk.start(p, sm.start_unit, sm.start_at);
  const int elem = k8Bit ? 1 : 2;

  if (warp >= kSumWarps && warp < kMmaWarp) {
    // ---- copies -----------------------------------------------------------
    const int me = tid - kSumWarps * 32, col = lane & 7;
    const char* q = static_cast<const char*>(p.a.q);
    uint32_t segment = 0, slot = 0, phase = 0;
    for (; walk.left > 0; walk.next(p), ++segment) {
      mbar_wait(smem_addr(&sm.q_empty), (segment & 1) ^ 1, guard);
      const int64_t row0 = walk.row0 + walk.first;
      for (int j = 0; j < walk.rows; ++j) {
        const char* row_q = q + (row0 + j) * p.a.q_row_stride * elem;
#pragma unroll 4
        for (int h = me >> 3; h < p.head_cols; h += kCopyThreads / 8) {
          const char* from = row_q + h * p.a.q_head_stride * elem;
          const int n = j * p.head_cols + h;
          for (int ch = 0; ch < p.chunks; ++ch) {
            const int byte = ch * 128 + col * 16;
            const bool in = h < p.a.heads && byte < p.row_bytes;
            copy16(q_at + ch * (p.pack * p.head_cols * 128) + n * 128 + ((col ^ (n & 7)) << 4), in ? from + byte : q, in ? 16 : 0);
          }
        }
      }
      copies_arrive(smem_addr(&sm.q_full));
      const int ss = segment % kSegmentSlots;
#pragma unroll 4
      for (int j = 0; j < walk.rows; ++j)
        for (int h = me; h < p.head_cols; h += kCopyThreads)
          sm.weight[ss][j * p.head_cols + h] = h < p.a.heads ? p.a.weights[(row0 + j) * p.a.weight_row_stride + h] : 0.f;
      for (int j = me; j < walk.rows; j += kCopyThreads) sm.length[ss][j] = row_length(p.R, row0 + j);
      mbar_arrive(smem_addr(&sm.segment_full[ss]));
      // The keys of a pass's last tokens and of what lies behind them come whole: a token's scores are its own.
      const int step_tokens = kTile * p.tiles;
      const auto place_of = [&](int token) { return ring + slot * slot_bytes + token / kTile * tile_bytes + token % kTile * 128; };
      const auto row_of = [&](int x, int b) {
        const bool here = in_cache(p, walk, x, b);
        const int place = x - block_column(p.R, x) * p.R.block_size;
        return p.map.run_rows ? run_row(p.map, here, b, place) : gather_row(p.map, here, b, place);
      };
      const auto next_slot = [&]() {
        if (++slot == static_cast<uint32_t>(p.slots)) {
          slot = 0;
          phase ^= 1;
        }
      };
      if (p.map.run_rows) {
        // one warp, a lane for each run of tokens; the runs' blocks are looked up a group of steps ahead
        if (warp == kSumWarps) {
          const int token = lane * p.map.run_rows;
          const auto position = [&](int t) { return t < walk.count && token < step_tokens ? (walk.at + t) * step_tokens + token : INT_MAX; };
          int blocks[kGroup];
#pragma unroll
          for (int i = 0; i < kGroup; ++i) blocks[i] = table_entry(p, walk, position(i));
          for (int t0 = 0; t0 < walk.count; t0 += kGroup) {
            int next[kGroup];
#pragma unroll
            for (int i = 0; i < kGroup; ++i) next[i] = table_entry(p, walk, position(t0 + kGroup + i));
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
              if (t0 + i >= walk.count) break;
              const uint32_t full = smem_addr(&sm.full[0]) + slot * 8;
              const int row = row_of(position(t0 + i), blocks[i]);
              mbar_wait(smem_addr(&sm.empty[0]) + slot * 8, phase ^ 1, guard);
              if (lane == 0) expect_bytes(full, slot_bytes);
              __syncwarp();
              if (token < step_tokens)
                for (int c = 0; c < p.chunks; ++c) fetch_run(p.map, place_of(token) + c * kChunk, c, row, full);
              next_slot();
            }
#pragma unroll
            for (int i = 0; i < kGroup; ++i) blocks[i] = next[i];
          }
        }
      } else {
        // pages of odd sizes: both warps, a lane for each four tokens
        const int token = (warp - kSumWarps) * (step_tokens / kCopyWarps) + lane * 4;
        const bool mine = lane * 4 < step_tokens / kCopyWarps;
        for (int t = 0; t < walk.count; ++t) {
          const uint32_t full = smem_addr(&sm.full[0]) + slot * 8;
          int row[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int x = (walk.at + t) * step_tokens + token + j;
            row[j] = row_of(x, table_entry(p, walk, x));
          }
          mbar_wait(smem_addr(&sm.empty[0]) + slot * 8, phase ^ 1, guard);
          if (lane == 0) expect_bytes(full, slot_bytes / kCopyWarps);
          __syncwarp();
          if (mine)
            for (int c = 0; c < p.chunks; ++c) fetch_four(p.map, place_of(token) + c * kChunk, c, row, full);
          next_slot();
        }
      }
    }
    copies_wait_all();
  } else if (warp == kMmaWarp) {
    // ---- products ---------------------------------------------------------
    const int chunks = p.row_bytes / 128, rest = (p.row_bytes % 128 + 31) / 32;  // whole chunks, and steps of 32 bytes after them
    const uint32_t q_chunk = p.pack * p.head_cols * 128;
    uint32_t step = 0, segment = 0, slot = 0, phase = 0;
    for (; walk.left > 0; walk.next(p), ++segment) {
      const uint32_t inst = p.inst | (static_cast<uint32_t>(walk.rows * p.head_cols >> 3) << 17);
      const int at_once = walk.product_tiles(p);
      mbar_wait_warp(smem_addr(&sm.q_full), segment & 1, guard);
      fence_async();
      for (int t = 0; t < walk.count; ++t) {
        int from = 0;  // of the step's tiles
        do {
          mbar_wait_warp(smem_addr(&sm.s_empty[0]) + (step & 1) * 8, ((step >> 1) & 1) ^ 1, guard);
          if (from == 0) mbar_wait_warp(smem_addr(&sm.full[0]) + slot * 8, phase, guard);
          fence_after();
#pragma unroll 1
          for (int m = 0; m < at_once; ++m) {
            const uint32_t d = tmem + (step & 1) * kMaxCols + m * (kMaxCols / 2), k_at = ring + slot * slot_bytes + (from + m) * tile_bytes;
            int c = 0;
#pragma unroll 1
            for (; c < chunks; ++c) {
              if (k8Bit)
                mma8_chunk(d, operand(k_at + c * kChunk, 16), operand(q_at + c * q_chunk, 16), inst, c > 0);
              else
                mma16_chunk(d, operand(k_at + c * kChunk, 16), operand(q_at + c * q_chunk, 16), inst, c > 0);
            }
#pragma unroll 1
            for (int i = 0; i < rest; ++i) {
              if (k8Bit)
                mma8_step(d, operand(k_at + c * kChunk + i * 32, 16), operand(q_at + c * q_chunk + i * 32, 16), inst, c + i > 0);
              else
                mma16_step(d, operand(k_at + c * kChunk + i * 32, 16), operand(q_at + c * q_chunk + i * 32, 16), inst, c + i > 0);
            }
          }
          commit(smem_addr(&sm.s_full[0]) + (step & 1) * 8);
          ++step;
          from += at_once;
        } while (from < p.tiles && ((walk.at + t) * p.tiles + from) * kTile < walk.longest);
        commit(smem_addr(&sm.empty[0]) + slot * 8);
        if (t + 1 == walk.count) commit(smem_addr(&sm.q_empty));
        if (++slot == static_cast<uint32_t>(p.slots)) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    commit(smem_addr(&sm.all_done));
    mbar_wait_warp(smem_addr(&sm.all_done), 0, guard);
    __syncwarp();
  } else {
    // ---- sums -------------------------------------------------------------
    const uint32_t turn = warp >> 3;     // every second product
    const int part = (warp >> 2) & 1;    // its tile, or its half of the rows
    const int quarter = warp & 3;
    uint32_t step = 0, segment = 0;
    for (; walk.left > 0; walk.next(p), ++segment) {
      const int ss = segment % kSegmentSlots;
      mbar_wait(smem_addr(&sm.segment_full[ss]), (segment / kSegmentSlots) & 1, guard);
      const bool both = walk.product_tiles(p) == 2;
      const int tokens = both ? 2 * kTile : kTile;  // of a product
      const int token = (both ? part * kTile : 0) + quarter * 32 + lane;
      const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + turn * kMaxCols + (both ? part * (kMaxCols / 2) : 0);
      const int middle = (walk.rows + 1) / 2;
      const int row = !both && part == 1 ? middle : 0, row_end = !both && part == 0 ? middle : walk.rows;
      // the segment's products
      const int first = walk.at * (p.tiles * kTile / tokens);
      const int count = min((walk.at + walk.count) * (p.tiles * kTile / tokens), static_cast<int>((walk.longest + (tokens - 1u)) / tokens)) - first;
      // The token's blocks and scales, two of this group's steps at a time: a group of two is looked up while the one before
      // it is summed, its blocks one earlier still. (Looked up a step ahead, the scales of 8-bit keys were waited for: they
      // come from HBM, behind a stream of keys.)
      const auto position = [&](int t) { return t < count ? (first + t) * tokens + token : INT_MAX; };
      const auto token_scale = [&](int x, int b) {
        return p.a.key_scales && in_cache(p, walk, x, b)
                   ? p.a.key_scales[b * p.a.scale_block_stride + (x - block_column(p.R, x) * p.R.block_size) * p.a.scale_token_stride]
                   : 1.f;
      };
      const int t_first = (step & 1) == turn ? 0 : 1;
      int b0[2], b1[2];
      float s0[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) b0[i] = table_entry(p, walk, position(t_first + i * 2));
#pragma unroll
      for (int i = 0; i < 2; ++i) b1[i] = table_entry(p, walk, position(t_first + 4 + i * 2));
#pragma unroll
      for (int i = 0; i < 2; ++i) s0[i] = token_scale(position(t_first + i * 2), b0[i]);
      for (int t0 = t_first; t0 < count; t0 += 4) {
        int b2[2];
        float s1[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) b2[i] = table_entry(p, walk, position(t0 + 8 + i * 2));
#pragma unroll
        for (int i = 0; i < 2; ++i) s1[i] = token_scale(position(t0 + 4 + i * 2), b1[i]);
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int t = t0 + i * 2, pos = position(t);
          if (t >= count) break;
          const bool found = in_cache(p, walk, pos, i ? b0[1] : b0[0]);
          const float scale = i ? s0[1] : s0[0];
          if (pos < walk.longest && !found) atomicOr(p.R.status, TOPK_DEV_BAD_BLOCK);
          mbar_wait(smem_addr(&sm.s_full[turn]), ((step + t) >> 1) & 1, guard);
          __syncwarp();
          fence_after();
          if (p.a.heads % 32 == 0)
            sum_tile<true>(p, at + row * p.head_cols, sm.weight[ss], sm.length[ss], row, row_end, pos, scale, found, walk.row0 + walk.first);
          else
            sum_tile<false>(p, at + row * p.head_cols, sm.weight[ss], sm.length[ss], row, row_end, pos, scale, found, walk.row0 + walk.first);
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sm.s_empty[turn]));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          b0[i] = b1[i];
          b1[i] = b2[i];
          s0[i] = s1[i];
        }
      }
      step += count;
    }
  }
  if (slice == 0) report_rows(p.R, tid, kThreads);
  settle(guard);
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp) tmem_free(tmem, 2 * kMaxCols);
}

template <bool k8Bit>
int run(Params& p, int device, int smem_limit, cudaStream_t stream) {
  const int extra = static_cast<int>(sizeof(Smem)) + 1024;
  const int slot = p.tiles * p.chunks * kChunk, room = smem_limit - extra - static_cast<int>(p.q_bytes);
  p.slots = room / slot < kMaxSlots ? room / slot : kMaxSlots;
  if (p.slots < 2) return TOPK_ERR_PLAN;
  const size_t smem = p.q_bytes + static_cast<size_t>(p.slots) * slot + extra;
  static int granted[kMaxDevices];
  const int rc = allow_smem(index_logits_kernel<k8Bit>, smem_limit, device, granted);
  if (rc != TOPK_OK) return rc;
  return launch(index_logits_kernel<k8Bit>, static_cast<const Params&>(p), p.slices, kThreads, smem, stream);
}

}  // namespace
}  // namespace paged
}  // namespace ltk

extern "C" int topk_index_logits(const topk_index_logits_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_index_logits_args& a = *args;
  int rc = check_rows(a.rows);
  if (rc != TOPK_OK) return rc;
  if (a.max_len < 1 || a.max_len > INT32_MAX || a.logits_row_stride < 0) return TOPK_ERR_INVALID_ARG;
  const int size = a.dtype == TOPK_DTYPE_F8E4M3 ? 1 : 2, piece = 16 / size;
  if (a.dtype != TOPK_DTYPE_F16 && a.dtype != TOPK_DTYPE_BF16 && a.dtype != TOPK_DTYPE_F8E4M3) return TOPK_ERR_UNSUPPORTED;
  if (a.heads < 1 || a.heads > 128 || a.dim < piece || a.dim > 128 || a.dim % piece != 0) return TOPK_ERR_UNSUPPORTED;
  if (a.rows.num_rows == 0) return TOPK_OK;
  rc = check_row_pointers(a.rows);
  if (rc != TOPK_OK) return rc;
  if (a.q == nullptr || a.weights == nullptr || a.keys == nullptr || a.logits == nullptr || a.workspace == nullptr)
    return TOPK_ERR_INVALID_ARG;
  if (misaligned(a.q, 16) || a.q_row_stride % piece || a.q_head_stride % piece || misaligned(a.keys, 16) ||
      a.key_block_stride % piece || a.key_token_stride % piece || misaligned(a.weights, 4) ||
      misaligned(a.key_scales, 4) || misaligned(a.logits, 4) || misaligned(a.workspace, 16))
    return TOPK_ERR_MISALIGNED;
  int dev = 0;
  topk_device_props props{};
  if (cudaGetDevice(&dev) != cudaSuccess || topk_query_device(dev, &props) != TOPK_OK) {
    cudaGetLastError();
    return TOPK_ERR_CUDA;
  }
  Params p{};
  p.a = a;
  p.R = make_rows(a.rows, a.max_len, a.workspace);
  p.head_cols = (a.heads + 15) / 16 * 16;
  // Rows of a unit: as many as a product takes, of one request (the largest divisor of next_n; given each row's request, the
  // kernel sees to it), but no more than leaves every SM a step where the rows are few and short. (22 rows of 32 heads over
  // 400 tokens: 9 us with one row a unit, 16 us with eight.)
  const int fit = kMaxCols / p.head_cols;
  for (int d = 1; d <= fit && d <= a.rows.num_rows; ++d) {
    if (a.rows.row_request != nullptr ? (d & (d - 1)) != 0 : a.rows.next_n % d != 0) continue;
    const int64_t tokens = kTile * (d * p.head_cols <= kMaxCols / 2 ? 2 : 1);
    if (d == 1 || (a.rows.num_rows + d - 1) / d * ((p.R.max_len + tokens - 1) / tokens) >= props.num_sms) p.pack = d;
  }
  // Two tiles a step where a unit's columns leave room for both in a place, and where rows bring their requests: passes may
  // then be of fewer rows. One of more columns multiplies a step's tiles one after the other.
  p.tiles = a.rows.row_request != nullptr || p.pack * p.head_cols <= kMaxCols / 2 ? 2 : 1;
  p.units = (a.rows.num_rows + p.pack - 1) / p.pack;
  rc = make_cache_map(&p.map, a.keys, size, a.dtype, a.rows.num_blocks, a.rows.block_size, a.dim, a.key_block_stride, a.key_token_stride,
                      64);
  if (rc != TOPK_OK) return rc;
  p.row_bytes = a.dim * size;
  p.chunks = (p.row_bytes + 127) / 128;
  p.q_bytes = static_cast<uint32_t>(p.pack * p.head_cols * 128 * p.chunks);
  const int64_t step = p.tiles * kTile, most = a.rows.num_rows * ((p.R.max_len + step - 1) / step);
  p.slices = static_cast<int32_t>(most < props.num_sms ? most : props.num_sms);
  using namespace ltk::umma;
  p.inst = instruction(size == 1 ? kE4M3 : a.dtype == TOPK_DTYPE_BF16 ? kBF16 : kF16, 0, false);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return size == 1 ? run<true>(p, dev, props.max_smem_optin, s) : run<false>(p, dev, props.max_smem_optin, s);
}
