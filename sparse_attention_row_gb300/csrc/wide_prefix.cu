// Attention over a prefix that many columns share (topk_shared_attention), joined with what rows see behind it.
//
// A unit is a run of rows that share a prefix and one key-value head: up to 256 columns (row, head), as two halves of 128.
// Unlike in paged_attention.cu, whose columns are few, the columns are the long side of both products, M = 128:
//   S [128 columns x 128 tokens]  = Q [128 x dk] . K^T
//   O [128 columns x dv]         += P [128 x 128 tokens] . V
// so that both run at the tensor core's full rate (N = 128: 64 cycles for 16 of the inner dimension), and a column's
// scores lie in one thread: its maximum and sum need no exchange. P goes back into the tensor memory that its scores stood
// in, and is the second product's A operand there. The two halves take turns: while the softmax of one is at work, the other's
// products run. Tensor memory holds S and O of both: all of its 512 columns.
//
// Order of the products: for each tile P_a V in two steps of 64 tokens, each as soon as its probabilities stand, Q_a K' of the
// next tile, P_b V, Q_b K'. A half's next scores are written over its
// probabilities; the tensor core takes products in the order in which one thread has issued them.
//
// Split: as in paged_attention.cu the units' tiles of 128 tokens, in order, are dealt in equal runs to the CTAs, one on
// each SM; parts of units go through the workspace and a second kernel.
//
// Roles (13 warps): 4 softmax warps to each half, a thread to a column; 4 copy keys and values (and the queries of
// later units) with 16-byte asynchronous copies, two places each; one issues the products.
//
// A column's maximum is taken from a unit's first 64 tokens; later the probabilities are taken with the maximum in use, and only
// where their sum comes out too large is that moved and O scaled (a warp at a time, for its own 32 columns). Statistics and O
// are in fp32; P is rounded to the input type for the second product (fp16: scaled by 2^7 first, sums of 64 below 2^15).
#include <cfloat>

#include "attention_forms.cuh"
#include "attention_parts.cuh"
#include "paged.cuh"
#include "token_copies.cuh"
#include "umma.cuh"

namespace ltk {
namespace paged {
namespace {

using namespace ltk::umma;

constexpr int kTile = 128;           // tokens
constexpr int kChunk = kTile * 128;  // bytes of 64 dims
constexpr int kPiece = 2 * kChunk;   // of a tile's keys or values: up to 128 dims
constexpr int kStep = 64;            // tokens whose probabilities are handed over at a time
constexpr int kHalf = 128;           // columns
constexpr int kCols = 2 * kHalf;
constexpr int kSoftmaxWarps = 8, kCopyWarps = 4, kCopyThreads = kCopyWarps * 32;
constexpr int kMmaWarp = kSoftmaxWarps + kCopyWarps;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kSeenSlots = 4;  // tiles that the copies can be ahead of the softmax, and one
constexpr int kMaxDim = 128;
static_assert(kCols == kWideCols);

struct Params {
  topk_attention_args a;
  Rows R;
  FormArgs f;
  int32_t group;   // heads a key-value head
  int32_t v_cols;  // dv, rounded up to 16
  int32_t slices;
  float scale2;    // scale * log2(e)
  float4* part;    // [slices][2][v_cols / 4][kCols]
  float2* stat;    // [slices][2][kCols]: maximum (in powers of two) and sum
  float* tail;     // [slices][2][kCols]: the logarithm of the sum behind the prefix
  Join* join;      // [slices]
  int32_t join_lanes;  // of the join's CTAs, which take the slices in turn
};

struct Smem {
  uint32_t seen[kSeenSlots][kCopyWarps];  // tokens of a tile that are there
  uint64_t key_full[2], key_empty[2], value_full[2], value_empty[2];
  uint64_t seen_full[2][kSeenSlots];  // for each half, by the tiles that it takes part in
  uint64_t q_first, q_full, q_empty, s_full[2], all_done;
  // For each half and step, by the tiles that the half takes part in: a parity tells no phase from the second one before it, so
  // the steps of a tile, which may both come before the first is waited for, have barriers of their own.
  uint64_t p_full[2][2], o_done[2][2];
  int64_t scan[kThreads / 32];
  int64_t start_group, start_at, tiles, run_begin, run_end;
  uint32_t tmem, gave_up;
};

// A slice's run of tiles, walked segment by segment (a segment: the tiles of one unit in the run).
struct Walk {
  int64_t group, left;     // tiles of the run from here on
  int kv_head, at, tiles;  // the unit, the segment's first tile, the unit's tiles
  int count;               // tiles of the segment
  __device__ void size() { count = static_cast<int>(min(static_cast<int64_t>(tiles - at), left)); }
};

__device__ __forceinline__ int run_tiles(const Params& p, int64_t g) { return static_cast<int>((p.f.runs[g].length + (kTile - 1u)) / kTile); }

__device__ __forceinline__ void next_segment(const Params& p, Walk& w) {
  w.left -= w.count;
  w.at = 0;
  if (++w.kv_head == p.a.kv_heads) {
    w.kv_head = 0;
    ++w.group;
    if (w.left > 0) w.tiles = run_tiles(p, w.group);
  }
  w.size();
}

// A unit's queries into their K-major tiles, a half after the other; zeros past its columns and past dk.
__device__ __noinline__ void copy_queries(const Params& p, uint32_t q_at, int64_t row0, int kv_head, int cols, int me, int threads) {
  const int piece = me & 7;
  const int halves = cols > kHalf ? 2 : 1, chunks = (p.a.dk + 63) / 64;
#pragma unroll 1
  for (int n = me >> 3; n < halves * kHalf; n += threads >> 3) {
    const int j = n / p.group, row = n & (kHalf - 1);
    const uint16_t* q = static_cast<const uint16_t*>(p.a.q);
    const bool real = n < cols;
    if (real) q += (row0 + j) * p.a.q_row_stride + static_cast<int64_t>(kv_head * p.group + n - j * p.group) * p.a.q_head_stride;
    const uint32_t dst = q_at + (n / kHalf) * kPiece + row * 128 + ((piece ^ (row & 7)) << 4);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (c >= chunks) break;
      const int dim = c * 64 + piece * 8;
      const bool in = real && dim < p.a.dk;
      copy16(dst + c * kChunk, in ? q + dim : static_cast<const uint16_t*>(p.a.q), in ? 16 : 0);
    }
  }
}

// S = Q K^T of a half: steps of 16 dims.
__device__ __forceinline__ void multiply_keys(uint32_t d, uint32_t q, uint32_t k, int dk, uint32_t inst) {
  if (dk == 128) {
    mma16_pair(d, operand(q, 16), kChunk >> 4, operand(k, 16), kChunk >> 4, inst, false);
    return;
  }
  bool add = false;
  int left = dk;
#pragma unroll 1
  for (; left >= 64; left -= 64, q += kChunk, k += kChunk, add = true) mma16_chunk(d, operand(q, 16), operand(k, 16), inst, add);
#pragma unroll 1
  for (; left > 0; left -= 16, q += 32, k += 32, add = true) mma16_step(d, operand(q, 16), operand(k, 16), inst, add);
}

__device__ __forceinline__ uint64_t two(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 apart(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  if constexpr (kBf16) return __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(x));
  else return __half22float2(reinterpret_cast<const __half2&>(x));
}

// The probabilities of a column for half a tile's tokens, packed, and their sum. All scores are loaded at once: with a wait for
// every 16 or 32 of them, each part's chain of latencies stands by itself (1700 cycles a tile against 1200).
template <bool kBf16>
__device__ __forceinline__ float probabilities(uint32_t s_at, float scale2, float in_use, uint32_t seen0, uint32_t seen1, uint32_t (&out)[kStep / 2]) {
  const uint64_t scale = two(scale2, scale2), base = two(-in_use, -in_use);
  float s[kStep];
  tmem_load64(s_at, s);
  if ((seen0 & seen1) != ~0u) {
#pragma unroll
    for (int i = 0; i < kStep; ++i)
      if (!((i < 32 ? seen0 : seen1) >> (i & 31) & 1)) s[i] = -INFINITY;
  }
  uint64_t l[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kStep; i += 2) {
    const float2 y = apart(fma2(two(s[i], s[i + 1]), scale, base));
    const float u = exp2_fast(y.x), v = exp2_fast(y.y);
    l[i / 2 & 3] = add2(l[i / 2 & 3], two(u, v));
    out[i / 2] = pack2<kBf16>(u, v);
  }
  const float2 both = apart(add2(add2(l[0], l[1]), add2(l[2], l[3])));
  return both.x + both.y;
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t raw[];
  const uint32_t q_at = (smem_addr(raw) + 1023) & ~1023u, key_at = q_at + 2 * kPiece, value_at = key_at + 2 * kPiece;
  Smem& sm = *reinterpret_cast<Smem*>(raw + (value_at + 2 * kPiece - smem_addr(raw)));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, slice = blockIdx.x;
  const Guard guard{&sm.gave_up, p.R.status};

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sm.key_full[i]), kCopyThreads);
      mbar_init(smem_addr(&sm.key_empty[i]), 1);
      mbar_init(smem_addr(&sm.value_full[i]), kCopyThreads);
      mbar_init(smem_addr(&sm.value_empty[i]), 1);
      for (int j = 0; j < kSeenSlots; ++j) mbar_init(smem_addr(&sm.seen_full[i][j]), kCopyWarps);
      mbar_init(smem_addr(&sm.s_full[i]), 1);
      for (int j = 0; j < 2; ++j) {
        mbar_init(smem_addr(&sm.p_full[i][j]), kSoftmaxWarps / 2);
        mbar_init(smem_addr(&sm.o_done[i][j]), 1);
      }
    }
    mbar_init(smem_addr(&sm.q_first), kSoftmaxWarps * 32);
    mbar_init(smem_addr(&sm.q_full), kCopyThreads);
    mbar_init(smem_addr(&sm.q_empty), 1);
    mbar_init(smem_addr(&sm.all_done), 1);
    sm.gave_up = 0;
    fence_async();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&sm.tmem), 512);
  dependent_wait();
  dependent_launch();

  // where this slice's run begins
  {
    const int64_t groups = *p.f.run_count, per = (groups + kThreads - 1) / kThreads;
    const int64_t g0 = min(per * tid, groups), g1 = min(g0 + per, groups);
    int64_t mine = 0;
    for (int64_t g = g0; g < g1; ++g) mine += run_tiles(p, g);
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
    total *= p.a.kv_heads;
    const int64_t begin = slice_begin(total, p.slices, slice);
    int64_t at = (pre - mine) * p.a.kv_heads;
    if (begin >= at && begin < pre * p.a.kv_heads) {
      for (int64_t g = g0; g < g1; ++g) {
        const int64_t n = static_cast<int64_t>(run_tiles(p, g)) * p.a.kv_heads;
        if (begin < at + n) {
          sm.start_group = g;
          sm.start_at = begin - at;
          break;
        }
        at += n;
      }
    }
    if (tid == 0) {
      sm.tiles = total;
      sm.run_begin = begin;
      sm.run_end = slice_begin(total, p.slices, slice + 1);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;
  const int64_t run_begin = sm.run_begin;
  Walk walk{};
  walk.left = sm.run_end - run_begin;
  if (walk.left > 0) {
    walk.group = sm.start_group;
    walk.tiles = run_tiles(p, walk.group);
    int64_t at = sm.start_at;
    for (; at >= walk.tiles; at -= walk.tiles) ++walk.kv_head;
    walk.at = static_cast<int>(at);
    walk.size();
  }
  const auto columns = [&]() { return p.f.runs[walk.group].rows * p.group; };

  // the first segment's queries, by the warps that have nothing to do yet
  if (walk.left > 0 && warp < kSoftmaxWarps) {
    copy_queries(p, q_at, p.f.runs[walk.group].row0, walk.kv_head, columns(), tid, kSoftmaxWarps * 32);
    copies_arrive(smem_addr(&sm.q_first));
  }
  if (warp >= kSoftmaxWarps && warp < kMmaWarp) {
    // ---- copies -----------------------------------------------------------
    const int me = tid - kSoftmaxWarps * 32;  // a thread's token of a tile
    TokenCopies copies((warp - kSoftmaxWarps) * 32, lane);
    uint32_t tile = 0, second = 0, segment = 0;  // second: tiles of which the second half takes part
    for (; walk.left > 0; next_segment(p, walk), ++segment) {
      const SharedRun run = p.f.runs[walk.group];
      const int cols = run.rows * p.group;
      const int32_t* pages = p.f.prefixes.table + run.prefix * p.f.prefixes.stride;
      const auto place = [&](int t) { return t < walk.count ? (walk.at + t) * kTile + me : INT_MAX; };
      const auto page_of = [&](int x) { return x < run.length ? pages[block_column(p.R, x)] : 0; };
      int x = place(0), page = page_of(x);
      asm volatile("" ::"r"(page) : "memory");  // here, before any copies are issued: a load waits behind those
      if (segment > 0) {                        // the first one's are copied by the softmax warps
        mbar_wait(smem_addr(&sm.q_empty), (segment & 1) ^ 1, guard);
        copy_queries(p, q_at, run.row0, walk.kv_head, cols, me, kCopyThreads);
        copies_arrive(smem_addr(&sm.q_full));
      }
      for (int t = 0; t < walk.count; ++t, ++tile) {
        const bool seen = x < run.length && page >= 0 && page < p.R.num_blocks;
        if (!seen && x < run.length) atomicOr(p.R.status, TOPK_DEV_BAD_BLOCK);
        const uint32_t who = __ballot_sync(~0u, seen);
        if (lane == 0) {
          sm.seen[tile % kSeenSlots][warp - kSoftmaxWarps] = who;
          mbar_arrive(smem_addr(&sm.seen_full[0][tile % kSeenSlots]));
          if (cols > kHalf) mbar_arrive(smem_addr(&sm.seen_full[1][second % kSeenSlots]));
        }
        second += cols > kHalf;
        const char *kp = static_cast<const char*>(p.a.k), *vp = static_cast<const char*>(p.a.v);
        if (seen) {
          const int in_page = x - block_column(p.R, x) * p.R.block_size;
          kp += 2 * (static_cast<int64_t>(page) * p.a.k_block_stride + in_page * p.a.k_token_stride + walk.kv_head * p.a.k_head_stride);
          vp += 2 * (static_cast<int64_t>(page) * p.a.v_block_stride + in_page * p.a.v_token_stride + walk.kv_head * p.a.v_head_stride);
        }
        x = place(t + 1);
        page = page_of(x);
        const uint32_t slot = tile & 1, phase = ((tile >> 1) & 1) ^ 1;
        copies.aim(kp, seen, lane);
        mbar_wait(smem_addr(&sm.key_empty[slot]), phase, guard);
        copies.columns(key_at + slot * kPiece, kChunk, 0, p.a.dk * 2, p.a.k);
        copies_arrive(smem_addr(&sm.key_full[slot]));
        copies.aim(vp, seen, lane);
        mbar_wait(smem_addr(&sm.value_empty[slot]), phase, guard);
        copies.columns(value_at + slot * kPiece, kChunk, 0, p.a.dv * 2, p.a.v);
        copies_arrive(smem_addr(&sm.value_full[slot]));
      }
    }
    copies_wait_all();
  } else if (warp == kMmaWarp) {
    // ---- products -----------------------------------------------------------
    constexpr uint32_t kKeys = instruction(kBf16 ? kBF16 : kF16, kTile, false);
    const uint32_t values = instruction_b_mn(kBf16 ? kBF16 : kF16, p.v_cols);
    uint32_t tile = 0, second = 0, segment = 0;
    const auto scores = [&](int half, uint32_t t) {
      multiply_keys(tmem + half * kTile, q_at + half * kPiece, key_at + (t & 1) * kPiece, p.a.dk, kKeys);
      commit(smem_addr(&sm.s_full[half]));
    };
    const auto outputs = [&](int half, uint32_t t, uint32_t turn, bool add) {
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        mbar_wait_warp(smem_addr(&sm.p_full[half][step]), turn & 1, guard);
        fence_after();
        mma16_held(tmem + kCols + half * kMaxDim, tmem + half * kTile + step * (kStep / 2), operand(value_at + (t & 1) * kPiece + step * kStep * 128, kChunk),
                   values, add || step > 0);
        commit(smem_addr(&sm.o_done[half][step]));
      }
    };
    const auto keys_come = [&](uint32_t t) {
      mbar_wait_warp(smem_addr(&sm.key_full[t & 1]), (t >> 1) & 1, guard);
      fence_async();
    };
    for (; walk.left > 0; next_segment(p, walk), ++segment) {
      const bool both = columns() > kHalf;
      if (segment == 0)
        mbar_wait_warp(smem_addr(&sm.q_first), 0, guard);
      else
        mbar_wait_warp(smem_addr(&sm.q_full), (segment & 1) ^ 1, guard);
      keys_come(tile);
      scores(0, tile);
      if (both) scores(1, tile);
      commit(smem_addr(&sm.key_empty[tile & 1]));
#pragma unroll 1
      for (int t = 0; t < walk.count; ++t, ++tile) {
        const bool more = t + 1 < walk.count;
        mbar_wait_warp(smem_addr(&sm.value_full[tile & 1]), (tile >> 1) & 1, guard);
        fence_async();
        outputs(0, tile, tile, t > 0);
        if (more) {
          keys_come(tile + 1);
          scores(0, tile + 1);
        }
        if (both) {
          outputs(1, tile, second, t > 0);
          ++second;
        }
        commit(smem_addr(&sm.value_empty[tile & 1]));
        if (more) {
          if (both) scores(1, tile + 1);
          commit(smem_addr(&sm.key_empty[(tile + 1) & 1]));
        }
      }
      commit(smem_addr(&sm.q_empty));
    }
    commit(smem_addr(&sm.all_done));
    mbar_wait_warp(smem_addr(&sm.all_done), 0, guard);
  } else {
    // ---- softmax and output ---------------------------------------------------
    constexpr float kShift = kBf16 ? 0.f : 7.f;  // fp16: probabilities use the upper half of its range, at most 2^15
    constexpr float kMostSum = kBf16 ? 1048576.f : 32768.f;  // of 64 probabilities, above which the maximum moves
    const int half = warp >> 2, column = tid;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + half * kTile, o_at = tmem + lanes + kCols + half * kMaxDim;
    uint32_t tile = 0, turn = 0;  // turn: tiles that this half took part in
    bool first_segment = true;
    for (; walk.left > 0; next_segment(p, walk)) {
      const SharedRun run = p.f.runs[walk.group];
      const int cols = run.rows * p.group;
      if (half == 1 && cols <= kHalf) {
        tile += walk.count;
        first_segment = false;
        continue;
      }
      const int j = column / p.group, head = walk.kv_head * p.group + column - j * p.group;
      const bool real = column < cols;
      // in powers of two: the maximum when it last moved, and what is taken off the scores; the lowest number until a finite
      // one has come, so that any such score makes the maximum move
      float m = -INFINITY, in_use = -FLT_MAX, l = 0.f;
      for (int t = 0; t < walk.count; ++t, ++tile, ++turn) {
        mbar_wait(smem_addr(&sm.seen_full[half][turn % kSeenSlots]), (turn / kSeenSlots) & 1, guard);
        mbar_wait_warp(smem_addr(&sm.s_full[half]), turn & 1, guard);
        fence_after();
#pragma unroll 1
        for (int step = 0; step < 2; ++step) {
          const uint32_t from = s_at + step * kStep, seen0 = sm.seen[tile % kSeenSlots][step * 2], seen1 = sm.seen[tile % kSeenSlots][step * 2 + 1];
          uint32_t out[kStep / 2];
          float sum = 0.f;
          // with the maximum in use, unless there is none yet or the probabilities come out too large: then that is moved first
          for (bool move_first = t == 0 && step == 0;; move_first = true) {
            if (move_first) {
              float top = -INFINITY;
#pragma unroll 1
              for (int c = 0; c < kStep; c += 16) {
                float x[16];
                tmem_load(from + c, x);
                const uint32_t who = (c < 32 ? seen0 : seen1) >> (c & 16);
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, who >> i & 1 ? x[i] : -INFINITY);
              }
              top *= p.scale2;
              const bool move = top > m, rescale = __any_sync(~0u, move && m > -INFINITY);
              const float factor = move && m > -INFINITY ? exp2_fast(m - top) : 1.f;
              if (move) {
                m = top;
                in_use = m - kShift;
              }
              if (rescale) {
                mbar_wait_warp(smem_addr(&sm.o_done[half][step ^ 1]), (turn & 1) ^ (step ^ 1), guard);  // the step before has been added
                fence_after();
                l *= factor;
#pragma unroll 1
                for (int c = 0; c < p.v_cols; c += 16) {
                  float o[16];
                  tmem_load(o_at + c, o);
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] *= factor;
                  tmem_store8(o_at + c, o);
                  tmem_store8(o_at + c + 8, o + 8);
                }
                store_wait();
              }
            }
            sum = probabilities<kBf16>(from, p.scale2, in_use, seen0, seen1, out);
            if (!__any_sync(~0u, !(sum <= kMostSum)) || move_first) break;
          }
          l += sum;
          tmem_store32(s_at + step * (kStep / 2), out);  // where scores stood that have been read
          store_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sm.p_full[half][step]));
        }
      }
      // the whole unit, or a part of it
      const bool whole = walk.count == walk.tiles;
      const int64_t slot = static_cast<int64_t>(slice) * 2 + (first_segment ? 0 : 1);
      float* lse = real ? p.a.lse + (run.row0 + j) * p.a.heads + head : nullptr;
      const float tail = real ? *lse : -INFINITY;
      const Weights both = weigh(l == 0.f ? -INFINITY : in_use + log2f(l), tail);
      const float factor = l == 0.f ? 0.f : both.prefix / l;
      if (whole) {
        if (real) *lse = both.lse;
      } else {
        p.stat[slot * kCols + column] = make_float2(m == -INFINITY ? -INFINITY : in_use, l);
        p.tail[slot * kCols + column] = tail;
      }
      mbar_wait_warp(smem_addr(&sm.o_done[half][1]), (turn & 1) ^ 1, guard);
      fence_after();
      uint16_t* out = static_cast<uint16_t*>(p.a.out) + (real ? (run.row0 + j) * p.a.out_row_stride + head * p.a.out_head_stride : 0);
#pragma unroll 1
      for (int c = 0; c < p.v_cols; c += 16) {
        float o[16];
        tmem_load(o_at + c, o);
        if (l == 0.f) {  // nothing seen: zeros, whatever stands in O
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0.f;
        }
        if (!whole) {
          float4* to = p.part + (slot * (p.v_cols / 4) + c / 4) * kCols + column;
#pragma unroll
          for (int i = 0; i < 4; ++i) to[i * kCols] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else if (real) {
#pragma unroll
          for (int i = 0; i < 16; i += 8) {
            if (c + i >= p.a.dv) break;
            uint4* at = reinterpret_cast<uint4*>(out + c + i);
            const uint4 x = *at;
            const uint32_t old[4] = {x.x, x.y, x.z, x.w};
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack2<kBf16>(old[e]);
              y[e] = pack2<kBf16>(o[i + 2 * e] * factor + both.tail * f.x, o[i + 2 * e + 1] * factor + both.tail * f.y);
            }
            *at = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
      fence_before();
      if (first_segment && tid == 0) {  // a unit that began before this slice and ends in it
        Join j{};
        j.last = -1;
        if (walk.at > 0 && walk.at + walk.count == walk.tiles) {
          const int64_t unit_begin = run_begin - walk.at;
          j.rowgroup = walk.group;
          j.kv_head = walk.kv_head;
          j.first = slice_of(sm.tiles, p.slices, unit_begin);
          j.last = slice;
          j.first_slot = slice_begin(sm.tiles, p.slices, j.first) == unit_begin ? 0 : 1;
          j.tiles = sm.tiles;
        }
        p.join[slice] = j;
      }
      first_segment = false;
    }
    if (first_segment && tid == 0) {  // an empty run
      Join j{};
      j.last = -1;
      p.join[slice] = j;
    }
  }
  settle(guard);
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp) tmem_free(tmem, 512);
}

// Joins the parts of the units that fell into several slices: 32 columns of a unit and some of its values a CTA, lanes along the
// columns, four values a thread at a time. kSplit CTAs share the values of 32 columns, and the warps that are then left the parts. Where units
// are few and have many parts, that is eight, and 16 CTAs look for the units among all slices; else two, and each slice has its own. (32 rows, 16
// heads over 2, a prefix of 32 K tokens, two units in 76 parts: 47 us, the other way 51, with a CTA to 32 columns 58; 32 rows, 32 heads over 8, 16 K,
// eight units in 19 parts: 45, 46, 48; 256 rows, 32 K, 32 units: 184, 172, 173.)
constexpr int kJoinCols = 32, kJoinWarps = 8, kMaxParts = 160;
static_assert(kMaxParts <= kJoinWarps * 32);

template <int kSplit, bool kBf16>
__device__ __forceinline__ void join_unit(const Params& p, const Join& jn, int col0, int part0) {
  constexpr int kQuads = kMaxDim / 4 / kSplit;                                // of four values, of this CTA
  constexpr int kAcross = kQuads < kJoinWarps ? kQuads : kJoinWarps;          // warps along them
  constexpr int kTeams = kJoinWarps / kAcross, kEach = kQuads / kAcross;      // teams that take the parts in turn; quads of a warp
  __shared__ int32_t place[kMaxParts];  // of each part
  __shared__ int32_t warp_parts[kJoinWarps];
  __shared__ float weight[kMaxParts][kJoinCols];
  __shared__ float4 sums[kJoinCols][kQuads + 1];
  __shared__ float of_tail[kJoinCols];
  __shared__ float2 stats[kJoinWarps][kJoinCols];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quads = p.v_cols / 4, quad0 = part0 * kQuads;
  const SharedRun run = p.f.runs[jn.rowgroup];
  const int cols = run.rows * p.group, spanned = jn.last - jn.first + 1;
  if (col0 >= cols || quad0 >= quads) return;
  int parts = 0;  // in order, without the slices that have no tiles
  __syncthreads();  // the last unit's places and sums have been read
  {
    const int s = jn.first + tid;
    const bool is = tid < spanned && slice_begin(jn.tiles, p.slices, s) != slice_begin(jn.tiles, p.slices, s + 1);
    const unsigned who = __ballot_sync(~0u, is);
    if (lane == 0) warp_parts[warp] = __popc(who);
    __syncthreads();
    int at = __popc(who & ((1u << lane) - 1));
    for (int w = 0; w < kJoinWarps; ++w) {
      if (w < warp) at += warp_parts[w];
      parts += warp_parts[w];
    }
    if (is) place[at] = s * 2 + (tid == 0 ? jn.first_slot : 0);
  }
  __syncthreads();
  // each column's maximum and sum: a warp's parts, then the warps' in order; and from them each part's weight in the whole
  {
    const int col = col0 + lane;
    float m = -INFINITY, sum = 0.f;
    constexpr int kAtOnce = 4;
    for (int i0 = warp; i0 < parts; i0 += kAtOnce * kJoinWarps) {
      float2 st[kAtOnce];
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) st[a] = p.stat[place[min(i0 + a * kJoinWarps, parts - 1)] * kCols + col];
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        const int i = i0 + a * kJoinWarps;
        if (i >= parts) break;
        weight[i][lane] = st[a].x;
        const float top = fmaxf(m, st[a].x), b = top == -INFINITY ? 0.f : top;
        sum = sum * exp2f(m - b) + st[a].y * exp2f(st[a].x - b);
        m = top;
      }
    }
    stats[warp][lane] = make_float2(m, sum);
    const float tail = p.tail[place[0] * kCols + col];
    __syncthreads();
    m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float2 st = stats[w][lane];
      const float top = fmaxf(m, st.x), b = top == -INFINITY ? 0.f : top;
      sum = sum * exp2f(m - b) + st.y * exp2f(st.x - b);
      m = top;
    }
    const Weights both = weigh(sum == 0.f ? -INFINITY : m + log2f(sum), tail);
    const float base = m == -INFINITY ? 0.f : m, factor = sum == 0.f ? 0.f : both.prefix / sum;
    for (int i = warp; i < parts; i += kJoinWarps) weight[i][lane] = factor == 0.f ? 0.f : exp2f(weight[i][lane] - base) * factor;
    if (warp == 0) {
      of_tail[lane] = both.tail;
      if (part0 == 0 && col < cols) {
        const int j = col / p.group;
        p.a.lse[(run.row0 + j) * p.a.heads + jn.kv_head * p.group + col - j * p.group] = both.lse;
      }
    }
  }
  __syncthreads();
  const int across = warp % kAcross, team = warp / kAcross;
  {
    constexpr int kAtOnce = kEach > 1 ? 4 : 8;
    float4 x[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = team; i0 < parts; i0 += kAtOnce * kTeams) {
      float4 y[kAtOnce][kEach];
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a)
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          y[a][k] = load_now(p.part + (static_cast<int64_t>(place[min(i0 + a * kTeams, parts - 1)]) * quads + min(quad0 + across + k * kAcross, quads - 1)) * kCols + col0 + lane);
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        const float w = i0 + a * kTeams < parts ? weight[i0 + a * kTeams][lane] : 0.f;
        if (w == 0.f) continue;  // nothing seen, whatever stands there
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          x[k].x += w * y[a][k].x;
          x[k].y += w * y[a][k].y;
          x[k].z += w * y[a][k].z;
          x[k].w += w * y[a][k].w;
        }
      }
    }
    for (int turn = 0; turn < kTeams; ++turn) {  // in the teams' order: the same sums every time
      if (turn > 0) __syncthreads();
      if (team != turn) continue;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        float4* to = &sums[lane][across + k * kAcross];
        const float4 y = turn == 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : *to;
        *to = make_float4(x[k].x + y.x, x[k].y + y.y, x[k].z + y.z, x[k].w + y.w);
      }
    }
  }
  __syncthreads();
  // along the values: four a thread
  for (int e = tid; e < kJoinCols * kQuads; e += kJoinWarps * 32) {
    const int n = e / kQuads, d = quad0 + e % kQuads, col = col0 + n, j = col / p.group;
    if (col >= cols || d * 4 >= p.a.dv) continue;
    uint2* at = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.a.out) + (run.row0 + j) * p.a.out_row_stride +
                                         static_cast<int64_t>(jn.kv_head * p.group + col - j * p.group) * p.a.out_head_stride + d * 4);
    const uint2 old = *at;
    const float2 f = unpack2<kBf16>(old.x), g = unpack2<kBf16>(old.y);
    const float4 x = sums[n][e % kQuads];
    const float w = of_tail[n];
    *at = make_uint2(pack2<kBf16>(x.x + w * f.x, x.y + w * f.y), pack2<kBf16>(x.z + w * g.x, x.w + w * g.y));
  }
}

template <int kSplit, bool kBf16>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ Params p) {
  const int at = blockIdx.x / kSplit, col0 = at % (kCols / kJoinCols) * kJoinCols;
  dependent_wait();
  dependent_launch();
  for (int s = at / (kCols / kJoinCols); s < p.slices; s += p.join_lanes) {
    const Join jn = p.join[s];
    if (jn.last >= 0) join_unit<kSplit, kBf16>(p, jn, col0, blockIdx.x % kSplit);
  }
}

constexpr int kManySplit = 8, kFewSplit = 2, kFewUnitLanes = 16, kFewUnitParts = 16;

constexpr size_t kSmem = 6 * kPiece + sizeof(Smem) + 1024;
static_assert(kSmem <= 232448, "keys, values and queries of 256 columns");

size_t parts_of(int sms) { return static_cast<size_t>(sms) * 2; }

template <bool kBf16>
int run_wide(const Params& p, int device, cudaStream_t stream) {
  static int granted[kMaxDevices];
  int rc = allow_smem(prefix_kernel<kBf16>, kSmem, device, granted);
  if (rc != TOPK_OK) return rc;
  rc = launch(prefix_kernel<kBf16>, p, p.slices, kThreads, kSmem, stream);
  if (rc != TOPK_OK) return rc;
  const int64_t ctas = static_cast<int64_t>(p.join_lanes) * (kCols / kJoinCols);
  if (p.join_lanes < p.slices) return launch(join_kernel<kManySplit, kBf16>, p, ctas * kManySplit, kJoinWarps * 32, 0, stream);
  return launch(join_kernel<kFewSplit, kBf16>, p, ctas * kFewSplit, kJoinWarps * 32, 0, stream);
}

}  // namespace

size_t wide_scratch(int sms) { return parts_of(sms) * kCols * (kMaxDim * sizeof(float) + sizeof(float2) + sizeof(float)) + static_cast<size_t>(sms) * sizeof(Join); }

int attend_wide(const topk_attention_args& a, const FormArgs& f, void* scratch, void* stream) {
  int device = 0;
  topk_device_props props{};
  if (cudaGetDevice(&device) != cudaSuccess || topk_query_device(device, &props) != TOPK_OK) {
    cudaGetLastError();
    return TOPK_ERR_CUDA;
  }
  Params p{};
  p.a = a;
  p.f = f;
  p.R = make_rows(a.rows, INT32_MAX, a.workspace);
  p.group = a.heads / a.kv_heads;
  p.v_cols = (a.dv + 15) / 16 * 16;
  p.scale2 = a.scale * 1.4426950408889634f;
  const int64_t most = a.rows.num_rows * a.kv_heads * ((f.prefixes.most + kTile - 1) / kTile);
  int64_t slices = props.num_sms < kMaxParts ? props.num_sms : kMaxParts;
  p.slices = static_cast<int32_t>(slices < most ? slices : most);
  // units if all rows share one prefix: where they have many parts each, more CTAs join each of them
  const int pack = rows_of_run(a);
  const int64_t units = (a.rows.num_rows + pack - 1) / pack * a.kv_heads;
  p.join_lanes = p.slices >= kFewUnitParts * units && p.slices > kFewUnitLanes ? kFewUnitLanes : p.slices;
  char* w = static_cast<char*>(scratch);
  const size_t parts = parts_of(props.num_sms) * kCols;
  p.part = reinterpret_cast<float4*>(w);
  p.stat = reinterpret_cast<float2*>(w + parts * kMaxDim * sizeof(float));
  p.tail = reinterpret_cast<float*>(p.stat + parts);
  p.join = reinterpret_cast<Join*>(p.tail + parts);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.dtype == TOPK_DTYPE_BF16 ? run_wide<true>(p, device, s) : run_wide<false>(p, device, s);
}

}  // namespace paged
}  // namespace ltk
