// Logits of the sparse-attention indexer over a paged key cache
// (topk_index_logits), on the tensor cores:
//   logits[r, t] = s_t * sum_h w[r, h] * max(0, q[r, h, :] . k[t, :]).
//
// A unit is a few consecutive rows; where they belong to one request (drafted
// tokens, a prompt's piece) they share a pass over its keys, otherwise each has a
// pass of its own. A product takes 128 tokens,
//   S^T [128 tokens x N] = K [128 x dim] . Q^T [dim x N],  N = rows x heads <= 256,
// and puts a token's scores for all rows and heads in one lane of tensor memory, so
// that the weighted sum over the heads is one thread's own: no exchange at all.
// A step is two such tiles where N <= 128 and one where it is more: 256 columns of
// tensor memory, of which there are two places, so that one step's sums run while the
// next is multiplied. (One tile a step, and half as many warps for the sums: what a
// step costs beside its data, 1700 to 2000 cycles of waits and hand-overs, was all that
// the batch over 8-bit keys took.)
//
// The units' steps are dealt in equal runs to the CTAs, one on each SM; every CTA
// sums up the rows' steps to find its run. Rows are independent over the tokens,
// so nothing has to be joined.
//
// Roles in a CTA (21 warps): 4 fetch keys into a ring of steps by TMA (cache_map.cuh), a
// warp issues the products, four groups of 4 warps sum: two a step, which take a
// tile each, or half of the rows of the one.
#include "cache_map.cuh"
#include "paged.cuh"
#include "umma.cuh"

namespace ltk {
namespace paged {
namespace {

using namespace ltk::umma;

constexpr int kTile = 128;
constexpr int kChunk = 128 * 128;  // bytes of 128 tokens x 128 bytes
constexpr int kSumWarps = 16, kCopyWarps = 4;
constexpr int kCopyThreads = kCopyWarps * 32;
constexpr int kMmaWarp = kSumWarps + kCopyWarps;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kMaxSlots = 5;
constexpr int kTokenSlots = 8;   // more than the steps that the copies can be ahead of the sums: ring slots + 2
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
  float scale[kTokenSlots][2 * kTile];
  uint8_t found[kTokenSlots][2 * kTile];
  float weight[kSegmentSlots][kMaxCols];
  int32_t length[kSegmentSlots][kMaxRows];
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t q_full, q_empty, s_full[2], s_empty[2], token_full[kTokenSlots], segment_full[kSegmentSlots], all_done;
  int64_t scan[kThreads / 32];
  int64_t start_unit, start_at, steps;
  uint32_t tmem, gave_up;
};

__device__ __forceinline__ int steps_of(const Params& p, int length) { return (length + p.tiles * kTile - 1) / (p.tiles * kTile); }

// The rows of a unit: whether those that see anything have one request, and the unit's steps.
struct Unit {
  int64_t row0;
  int rows;
  bool shared;
  int64_t steps;
  __device__ Unit(const Params& p, int64_t u, bool report) {
    row0 = u * p.pack;
    rows = static_cast<int>(min(static_cast<int64_t>(p.pack), p.R.num_rows - row0));
    shared = true;
    int most = 0;
    int64_t sum = 0, request = -1;
    for (int j = 0; j < rows; ++j) {
      const int n = row_length(p.R, row0 + j, report);
      if (n == 0) continue;
      most = max(most, n);
      sum += steps_of(p, n);
      const int64_t b = row_request(p.R, row0 + j);
      if (request >= 0 && b != request) shared = false;
      request = b;
    }
    steps = shared ? steps_of(p, most) : sum;
  }
};

// A slice's run of steps, segment by segment (a segment: the steps of one pass in the run).
struct Walk {
  int64_t unit, left;
  int64_t row0;      // of the pass
  int64_t request;
  int first, rows;   // the pass's rows within the unit
  int unit_rows;
  bool shared;
  int at, count, longest;
  __device__ void pass(const Params& p, int from) {  // the pass that begins with the unit's row `from` or a later one
    longest = 0;
    first = from;
    rows = 0;
    if (shared) {
      if (from > 0) return;
      rows = unit_rows;
      for (int j = 0; j < rows; ++j) {
        const int n = row_length(p.R, row0 + j, false);
        if (n > 0) request = row_request(p.R, row0 + j);
        longest = max(longest, n);
      }
    } else {
      for (; first < unit_rows; ++first) {
        longest = row_length(p.R, row0 + first, false);
        if (longest > 0) {
          rows = 1;
          request = row_request(p.R, row0 + first);
          return;
        }
      }
    }
  }
  __device__ void enter(const Params& p, int64_t u) {
    const Unit x(p, u, false);
    unit = u;
    row0 = x.row0;
    unit_rows = x.rows;
    shared = x.shared;
    pass(p, 0);
  }
  __device__ void size(const Params& p) { count = static_cast<int>(min(static_cast<int64_t>(steps_of(p, longest) - at), left)); }
  __device__ void start(const Params& p, int64_t u, int64_t offset) {
    enter(p, u);
    while (offset >= steps_of(p, longest)) {
      offset -= steps_of(p, longest);
      pass(p, first + 1);
    }
    at = static_cast<int>(offset);
    size(p);
  }
  __device__ void next(const Params& p) {
    left -= count;
    at = 0;
    if (left <= 0) return;
    pass(p, shared ? 1 : first + 1);
    while (longest == 0) enter(p, unit + 1);  // there are steps left, so some later unit has them
    size(p);
  }
};

__device__ __forceinline__ float relu(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}

// The weighted sums of rows [row, row_end) of one tile for this thread's token, 16 columns at a time, the next ones on
// their way meanwhile. `at`: the first row's columns.
__device__ __forceinline__ void sum_tile(const Params& p, uint32_t at, const float* weight, const int32_t* length, int row, int row_end,
                                         int pos, float scale, bool found, int64_t row0) {
  constexpr int C = 16;
  if (row >= row_end) return;
  float v[2][C];
  const int cols = (row_end - row) * p.head_cols;
  weight += row * p.head_cols;
  tmem_load(at, v[0]);
  int in_row = 0;
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
  const auto take = [&](float (&x)[C], int c) {
    // columns past the heads hold zeros times a key: not numbers where the key is none
    const int real = p.a.heads - in_row;
    if (real >= C) {
#pragma unroll
      for (int i = 0; i < C; i += 4) {
        const float4 w = *reinterpret_cast<const float4*>(weight + c + i);
        s0 = fmaf(w.x, relu(x[i]), s0);
        s1 = fmaf(w.y, relu(x[i + 1]), s1);
        s2 = fmaf(w.z, relu(x[i + 2]), s2);
        s3 = fmaf(w.w, relu(x[i + 3]), s3);
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (i < real) s0 = fmaf(weight[c + i], relu(x[i]), s0);
    }
    in_row += C;
    if (in_row == p.head_cols) {
      if (pos < length[row]) p.a.logits[(row0 + row) * p.a.logits_row_stride + pos] = found ? ((s0 + s1) + (s2 + s3)) * scale : -INFINITY;
      ++row;
      in_row = 0;
      s0 = s1 = s2 = s3 = 0.f;
    }
  };
  for (int c = 0; c < cols; c += 2 * C) {
    load_wait(v[0]);
    if (c + C < cols) tmem_load(at + c + C, v[1]);
    take(v[0], c);
    if (c + C < cols) {
      load_wait(v[1]);
      if (c + 2 * C < cols) tmem_load(at + c + 2 * C, v[0]);
      take(v[1], c + C);
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
      mbar_init(smem_addr(&sm.full[i]), kCopyWarps * p.tiles);
      mbar_init(smem_addr(&sm.empty[i]), 1);
    }
    mbar_init(smem_addr(&sm.q_full), kCopyThreads);
    mbar_init(smem_addr(&sm.q_empty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sm.s_full[i]), 1);
      mbar_init(smem_addr(&sm.s_empty[i]), kSumWarps / 2);
    }
    for (int i = 0; i < kTokenSlots; ++i) mbar_init(smem_addr(&sm.token_full[i]), kCopyThreads);
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
    for (int64_t u = u0; u < u1; ++u) mine += Unit(p, u, slice == 0).steps;
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
      for (int64_t u = u0; u < u1; ++u) {
        const int64_t n = Unit(p, u, false).steps;
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
    TokenRows rows;
    uint32_t step = 0, segment = 0, slot = 0, phase = 0;
    for (; walk.left > 0; walk.next(p), ++segment) {
      mbar_wait(smem_addr(&sm.q_empty), (segment & 1) ^ 1, guard);
      const int cols = walk.rows * p.head_cols;
      const int64_t row0 = walk.row0 + walk.first;
      for (int n = me >> 3; n < cols; n += kCopyThreads / 8) {
        const int j = n / p.head_cols, h = n - j * p.head_cols;
        const char* from = q + ((row0 + j) * p.a.q_row_stride + h * p.a.q_head_stride) * elem;
        for (int ch = 0; ch < p.chunks; ++ch) {
          const int byte = ch * 128 + col * 16;
          const bool in = h < p.a.heads && byte < p.row_bytes;
          copy16(q_at + ch * (p.pack * p.head_cols * 128) + n * 128 + ((col ^ (n & 7)) << 4), in ? from + byte : q, in ? 16 : 0);
        }
      }
      copies_arrive(smem_addr(&sm.q_full));
      const int ss = segment % kSegmentSlots;
      for (int n = me; n < cols; n += kCopyThreads) {
        const int j = n / p.head_cols, h = n - j * p.head_cols;
        sm.weight[ss][n] = h < p.a.heads ? p.a.weights[(row0 + j) * p.a.weight_row_stride + h] : 0.f;
      }
      for (int j = me; j < walk.rows; j += kCopyThreads) sm.length[ss][j] = row_length(p.R, row0 + j, false);
      mbar_arrive(smem_addr(&sm.segment_full[ss]));
      // A step's tokens (this thread's: one of each tile) are found in stages, each a step earlier than its result is
      // used: the block, then the scale.
      const auto position = [&](int t, int m) { return t < walk.count ? ((walk.at + t) * p.tiles + m) * kTile + me : INT_MAX; };
      const auto column = [&](int x) { return p.R.block_shift >= 0 ? x >> p.R.block_shift : x / p.R.block_size; };
      const auto table_entry = [&](int x) {
        return x < walk.longest ? __ldg(p.R.block_table + walk.request * p.R.table_stride + column(x)) : 0;
      };
      const auto in_cache = [&](int x, int b) { return x < walk.longest && b >= 0 && b < p.R.num_blocks; };
      const auto token_scale = [&](int x, int b) {
        return p.a.key_scales && in_cache(x, b)
                   ? __ldg(p.a.key_scales + b * p.a.scale_block_stride + (x - column(x) * p.R.block_size) * p.a.scale_token_stride)
                   : 1.f;
      };
      int at_block[2], next_block[2], later_block[2];
      float scale[2], next_scale[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        at_block[m] = next_block[m] = later_block[m] = 0;
        scale[m] = next_scale[m] = 1.f;
        if (m < p.tiles) {
          at_block[m] = table_entry(position(0, m));
          next_block[m] = table_entry(position(1, m));
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (m < p.tiles) scale[m] = token_scale(position(0, m), at_block[m]);
      for (int t = 0; t < walk.count; ++t, ++step) {
        const uint32_t full = smem_addr(&sm.full[0]) + slot * 8, ts = step % kTokenSlots;
#pragma unroll
        for (int m = 0; m < 2; ++m)
          if (m < p.tiles) {
            later_block[m] = table_entry(position(t + 2, m));
            next_scale[m] = token_scale(position(t + 1, m), next_block[m]);
          }
        mbar_wait(smem_addr(&sm.empty[0]) + slot * 8, phase ^ 1, guard);
#pragma unroll
        for (int m = 0; m < 2; ++m)
          if (m < p.tiles) {
            const int x = position(t, m), place = x - column(x) * p.R.block_size;
            const bool here = in_cache(x, at_block[m]);
            if (x < walk.longest && !here) atomicOr(p.R.status, TOPK_DEV_BAD_BLOCK);
            if (p.map.run_rows && ((walk.at + t) * p.tiles + m + 1) * kTile <= walk.longest)  // before the pass's last tile
              rows.set(run_row(p.map, here, at_block[m], place, 0), p.map.run_rows, lane);
            else
              rows.set(gather_row(p.map, here, at_block[m], place, 0), 0, lane);
            rows.fetch(p.map, ring + slot * slot_bytes + m * tile_bytes + (warp - kSumWarps) * 32 * 128, 0, p.chunks, full, lane);
            sm.scale[ts][m * kTile + me] = scale[m];
            sm.found[ts][m * kTile + me] = here;
          }
        mbar_arrive(smem_addr(&sm.token_full[ts]));
        if (++slot == static_cast<uint32_t>(p.slots)) {
          slot = 0;
          phase ^= 1;
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          at_block[m] = next_block[m];
          next_block[m] = later_block[m];
          scale[m] = next_scale[m];
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
      mbar_wait_warp(smem_addr(&sm.q_full), segment & 1, guard);
      fence_async();
      for (int t = 0; t < walk.count; ++t, ++step) {
        mbar_wait_warp(smem_addr(&sm.s_empty[0]) + (step & 1) * 8, ((step >> 1) & 1) ^ 1, guard);
        mbar_wait_warp(smem_addr(&sm.full[0]) + slot * 8, phase, guard);
        fence_after();
#pragma unroll 1
        for (int m = 0; m < p.tiles; ++m) {
          const uint32_t d = tmem + (step & 1) * kMaxCols + m * (kMaxCols / 2), k_at = ring + slot * slot_bytes + m * tile_bytes;
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
    const uint32_t turn = warp >> 3;     // every second step
    const int part = (warp >> 2) & 1;    // its tile, or its half of the rows
    const int quarter = warp & 3, token = (p.tiles == 2 ? part * kTile : 0) + quarter * 32 + lane;
    const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + turn * kMaxCols + (p.tiles == 2 ? part * (kMaxCols / 2) : 0);
    uint32_t step = 0, segment = 0;
    for (; walk.left > 0; walk.next(p), ++segment) {
      const int ss = segment % kSegmentSlots;
      mbar_wait(smem_addr(&sm.segment_full[ss]), (segment / kSegmentSlots) & 1, guard);
      const int middle = (walk.rows + 1) / 2;
      const int row = p.tiles == 1 && part == 1 ? middle : 0, row_end = p.tiles == 1 && part == 0 ? middle : walk.rows;
      for (int t = 0; t < walk.count; ++t, ++step) {
        if ((step & 1) != turn) continue;
        const uint32_t ts = step % kTokenSlots;
        mbar_wait(smem_addr(&sm.token_full[ts]), (step / kTokenSlots) & 1, guard);
        const float scale = sm.scale[ts][token];
        const bool found = sm.found[ts][token];
        mbar_wait(smem_addr(&sm.s_full[turn]), (step >> 1) & 1, guard);
        fence_after();
        const int pos = (walk.at + t) * p.tiles * kTile + token;
        __syncwarp();
        sum_tile(p, at + row * p.head_cols, sm.weight[ss], sm.length[ss], row, row_end, pos, scale, found, walk.row0 + walk.first);
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.s_empty[turn]));
      }
    }
  }
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
  rc = make_cache_map(&p.map, a.keys, size, a.dtype, a.rows.num_blocks, a.rows.block_size, 1, a.dim, a.key_block_stride, a.key_token_stride, 0);
  if (rc != TOPK_OK) return rc;
  p.head_cols = (a.heads + 15) / 16 * 16;
  const int fit = kMaxCols / p.head_cols;  // rows that a product takes
  if (a.rows.row_request != nullptr) {
    p.pack = fit;
  } else {  // units that do not cross requests: the largest divisor of next_n that fits
    p.pack = 1;
    for (int d = 2; d <= fit; ++d)
      if (a.rows.next_n % d == 0) p.pack = d;
  }
  if (p.pack > a.rows.num_rows) p.pack = static_cast<int32_t>(a.rows.num_rows);
  p.units = (a.rows.num_rows + p.pack - 1) / p.pack;
  p.row_bytes = a.dim * size;
  p.chunks = (p.row_bytes + 127) / 128;
  p.q_bytes = static_cast<uint32_t>(p.pack * p.head_cols * 128 * p.chunks);
  p.tiles = p.pack * p.head_cols <= kMaxCols / 2 ? 2 : 1;
  const int64_t step = p.tiles * kTile, most = a.rows.num_rows * ((p.R.max_len + step - 1) / step);
  p.slices = static_cast<int32_t>(most < props.num_sms ? most : props.num_sms);
  p.inst = ltk::umma::instruction(a.dtype == TOPK_DTYPE_BF16 ? ltk::umma::kBF16 : ltk::umma::kF16, 0, false);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return size == 1 ? run<true>(p, dev, props.max_smem_optin, s) : run<false>(p, dev, props.max_smem_optin, s);
}
