// Attention of each row's heads over a paged cache (topk_paged_attention), on
// the tensor cores.
//
//   s_t = scale * q . k_t,   out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m)
//
// Shape of the work. A unit is a group of rows that read the same tokens (one
// row, or a request's next_n rows where no index list tells them apart) and one
// key-value head; its queries are columns (row j, head h) and come in blocks of
// up to 64. Tokens come in tiles of 128. Both products are taken with the tokens
// and values as the long side, M = 128, and the queries as N = 16, 32 or 64:
//   S^T [128 tokens x N]     = K [128 x dk] . Q^T [dk x N]
//   O^T [128 values x N] (+)= V^T [128 x 128 tokens] . P^T [128 tokens x N]
// so that few heads waste no rows of the tensor core, a tile of the cache is
// read in the layout that it has in memory by both products (K-major for the
// first, MN-major for the second), and latent attention's O^T, 512 values of 64
// heads, takes 256 of the 512 columns of tensor memory.
//
// Split. The units' tiles, in order, are dealt in equal runs to the CTAs, one
// on each SM; a unit that falls into several runs leaves its sums and statistics in
// the workspace, and a second kernel joins them in the order of the tokens. The
// lengths are read on the device: every CTA sums up the rows' tiles to find its
// run. With more than 64 columns, neighbouring CTAs take the column blocks of one
// run and meet its tokens in L2.
//
// Roles in a CTA (14 warps): 4 copy tokens into a ring of 32 KB pieces (128
// tokens x 128 dims) with 16-byte asynchronous copies, which take any page size,
// stride and index list and write zeros for what is masked (whatever the cache
// holds there); one warp issues the scores' products and one the values'; 8 warps do
// the softmax, a thread per token and half of the columns. A column's maximum
// runs over the tokens, that is over threads: a butterfly of shuffles in each
// warp, then four numbers per column through shared memory. It is taken for a
// unit's first tile, and later only where a probability comes out above 2^8: then the
// maximum in use is moved, and the sums and O^T are scaled. Everything is held in fp32
// but P, which is rounded to the input type for the second product (for fp16, scaled
// by 2^7, so that small probabilities keep their bits).
//
// What bounds it. Grouped heads read every byte once: 64 rows of 32 heads over 4
// key-value heads and 8 K to 32 K tokens run at the speed of the memory (380 us on the
// device, 392 a call among others: 7.1 and 6.8 TB/s). Latent attention is bounded by the chain of a tile's steps. Its 147 KB of keys and
// 64 columns' queries fill shared memory, so the next tile's keys can only come while this
// one's values are multiplied and leave the ring: at N = 64 some 1850 cycles for the values'
// products, 1500 until the last keys are there, 950 for the scores that wait for them and
// 1150 for the softmax, 6000 in all, of which the products read shared memory for 3260 (48 to
// 50 cycles an instruction, 39 to 42 at N = 16). 1024 rows of 64 heads over 2048 tokens each
// take 372 us (786 TFLOP/s), 64 rows of 128 heads over 2048 of 8 K to 32 K tokens 64 us. Tiles of
// 64 tokens, of which two fit, were slower (540 and 90 us): their products read more shared
// memory a token, and copies and products meet there all the time.
#include <cfloat>

#include "paged.cuh"
#include "token_copies.cuh"
#include "umma.cuh"

namespace ltk {
namespace paged {
namespace {

using namespace ltk::umma;

constexpr int kTile = 128;            // tokens
constexpr int kChunk = kTile * 128;   // bytes of 64 dims
constexpr int kPiece = 2 * kChunk;    // a ring slot: 128 dims
// Places for P. A latent tile and the queries leave room for one; elsewhere the next tile's probabilities need not wait
// until the last one's have been multiplied.
template <bool kLatent>
constexpr int places = kLatent ? 1 : 2;
constexpr int kSoftmaxWarps = 8, kCopyWarps = 4;
constexpr int kCopyThreads = kCopyWarps * 32;
constexpr int kScoreWarp = kSoftmaxWarps + kCopyWarps, kValueWarp = kScoreWarp + 1;
constexpr int kThreads = (kValueWarp + 1) * 32;
constexpr int kTokenSlots = 8;  // more than the tiles that the copies can be ahead of the softmax: ring slots + 1
constexpr int kMaxSlots = 6;
constexpr int kMaxQk = 576, kMaxV = 512;
constexpr int kMaxBlockCols = 64;
constexpr int kTeam = 128, kJoinDims = 32;  // threads of a team
constexpr int kMaxTeams = 4;                // which take the parts in turn
constexpr int kMaxParts = 256;  // slices of a launch at most
constexpr float kMoveAbove = 8.f;  // in powers of two

struct Join {  // what the join kernel has to know of the unit that ends in a slice and began before it
  int64_t rowgroup;
  int32_t kv_head;
  int32_t first, last;  // slices
  int32_t first_slot;   // which of its two places the first slice used
  int64_t tiles;        // of all units
};

struct Params {
  topk_attention_args a;
  Rows R;
  int32_t pack;          // rows of a unit
  int32_t group;         // heads a key-value head
  int32_t cols;          // pack * group
  int32_t blocks;        // column blocks of a unit
  int32_t block_cols;    // columns of a block (the last one may have fewer)
  int32_t k_chunks;      // of 64 dims
  int32_t k_pieces, v_pieces;
  int32_t latent;        // values are the first dims of the keys
  int32_t rest;          // 1: the last 64 dims of latent keys, which are no values, have a buffer of their own
  int32_t rest_is_p;     // 1: which is P's place, free until the tile's probabilities are written
  int32_t slots;         // of the ring
  int32_t slices;
  int32_t row_tiles;     // tiles of every unit where index lists are given, else 0
  int32_t whole;         // 1: slices begin between units only (index lists)
  int64_t row_groups;
  uint32_t tmem_cols;
  uint32_t q_bytes;
  float scale2;          // scale * log2(e)
  float* part;           // [slices][2][blocks][v_pieces * 128][N]
  float2* stat;          // [slices][2][blocks][N]: maximum (in powers of two) and sum
  Join* join;            // [joins]
  int32_t joins;         // places for a unit's end: one for each unit, or where those are more, for each slice
  int32_t by_unit;
  int32_t teams;         // of the join
};

template <int N>
struct Smem {  // behind the tiles
  static constexpr int kHalf = N / 2;
  int32_t token[kTokenSlots][128];  // position of each token of a tile, INT_MAX where nothing is to be seen
  float column_max[2][4][kHalf];      // [half][warp]; a barrier stands between one tile's reads and the next one's writes
  float moved[kSoftmaxWarps][2][kHalf];  // maximum in use, factor of the old sums
  float column_sum[2][4][kHalf];
  int32_t limit[2][2][kHalf];  // [parity of the segment][half]: tokens that a column sees
  union {
    int64_t out_at[2][2][kHalf];  // and where its output lies
    int64_t scan[kThreads / 32];  // before the first segment
  };
  int32_t least[2][2], split[2][2];  // of those; and from where on not all of the unit's rows that see anything see a token
  uint32_t kept;                // 1 + the last of the tiles that begin a segment but add to what O holds
  // A slot of the ring is free (`empty`, by slots), or a piece has come: the keys' pieces by their number, and the values'.
  // Each is waited for by one warp, one after another: a parity tells no phase from the second one before it, so no wait may
  // skip a phase, and copies of later pieces do not say that the arrivals of earlier ones have been counted.
  uint64_t key_come[kMaxSlots], value_come[kMaxSlots], empty[kMaxSlots];
  uint64_t q_first, q_full, q_empty, rest_full, rest_empty, s_full[2], s_empty[2], p_full[2], o_done[2], token_full[kTokenSlots], all_done[2];
  int64_t start_group, tiles, run_begin, run_end;
  int64_t start_at;
  uint32_t tmem;
  uint32_t gave_up;
};

// Out of line: seven copies of it in a kernel that is already longer than the instruction caches like cost 3 to 5 % (and
// fetching tokens into L2 ahead of their copies, which was tried, cost more than it brought).
static __device__ __noinline__ int group_length(const Params& p, int64_t g) {
  int most = 0;
#pragma unroll 1
  for (int j = 0; j < p.pack; ++j) most = max(most, row_length(p.R, g * p.pack + j));
  return most;
}

// Tiles of a unit; one at least, so that every unit is met and its rows written.
__device__ __forceinline__ int group_tiles(const Params& p, int64_t g) {
  if (p.row_tiles) return p.row_tiles;
  const int n = group_length(p, g);
  return n == 0 ? 1 : static_cast<int>((n + kTile - 1u) / kTile);
}

// First tile of slice s, and the slice of tile x; in 32 bits where the products fit (a 64-bit division takes some
// hundreds of cycles, and a launch starts with several).
constexpr int64_t kSmallTiles = 1 << 22;
__device__ __forceinline__ int64_t slice_begin(int64_t tiles, int slices, int s) {
  if (tiles < kSmallTiles) return static_cast<uint32_t>(tiles) * static_cast<uint32_t>(s) / static_cast<uint32_t>(slices);
  return tiles * s / slices;
}
__device__ __forceinline__ int slice_of(int64_t tiles, int slices, int64_t x) {
  if (tiles < kSmallTiles)
    return static_cast<int>((static_cast<uint32_t>(x + 1) * static_cast<uint32_t>(slices) - 1) / static_cast<uint32_t>(tiles));
  return static_cast<int>(((x + 1) * slices - 1) / tiles);
}

// A slice's run of tiles, walked segment by segment (a segment: the tiles of one unit in the run).
struct Walk {
  int64_t group;
  int64_t left;  // tiles of the run from here on
  int kv_head, at, tiles;  // the unit, the segment's first tile, the unit's tiles
  int count;               // tiles of the segment
  __device__ void size() { count = static_cast<int>(min(static_cast<int64_t>(tiles - at), left)); }
  __device__ void next(const Params& p) {
    left -= count;
    at = 0;
    if (++kv_head == p.a.kv_heads) {
      kv_head = 0;
      ++group;
      if (left > 0) tiles = group_tiles(p, group);
    }
    size();
  }
};

// A place in the ring of pieces, or among barriers that are taken in turn, and the parity of its phase.
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void step(uint32_t slots) {
    if (++slot == slots) slot = 0, phase ^= 1;
  }
  __device__ __forceinline__ void step(uint32_t slots, uint32_t by) {
    for (slot += by; slot >= slots; slot -= slots) phase ^= 1;
  }
};

// Reduces v[c] over the warp's lanes; lane i gets column i % N.
template <int N, bool kMax>
__device__ __forceinline__ float reduce_columns(const float (&v)[N], int lane) {
  float t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = v[i];
#pragma unroll
  for (int w = N / 2; w > 0; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const float keep = up ? t[j + w] : t[j], send = up ? t[j] : t[j + w];
      const float other = __shfl_xor_sync(~0u, send, w);
      t[j] = kMax ? fmaxf(keep, other) : keep + other;
    }
  }
#pragma unroll
  for (int d = N; d < 32; d <<= 1) {
    const float other = __shfl_xor_sync(~0u, t[0], d);
    t[0] = kMax ? fmaxf(t[0], other) : t[0] + other;
  }
  return t[0];
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kBf16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return reinterpret_cast<const uint32_t&>(x);
  } else {
    const __half2 x = __floats2half2_rn(lo, hi);
    return reinterpret_cast<const uint32_t&>(x);
  }
}

// A segment's queries [N][dk] into their K-major tiles, by `threads` threads (a multiple of 8); zeros past the block's columns
// and past dk.
template <int N>
__device__ __noinline__ void copy_queries(const Params& p, uint32_t q_at, int64_t row0, int kv_head, int block, int block_cols, int me,
                                          int threads) {
  const int col = me & 7;
#pragma unroll 1
  for (int n = me >> 3; n < N; n += threads >> 3) {
    const int c = block * p.block_cols + n, j = c / p.group;
    const uint16_t* q = static_cast<const uint16_t*>(p.a.q);
    const bool real = n < block_cols;
    if (real) q += (row0 + j) * p.a.q_row_stride + static_cast<int64_t>(kv_head * p.group + c - j * p.group) * p.a.q_head_stride;
    const uint32_t dst = q_at + n * 128 + ((col ^ (n & 7)) << 4);
#pragma unroll 3
    for (int ch = 0; ch < p.k_chunks; ++ch) {
      const int dim = ch * 64 + col * 8;
      const bool in = real && dim < p.a.dk;
      copy16(dst + ch * (N * 128), in ? q + dim : static_cast<const uint16_t*>(p.a.q), in ? 16 : 0);
    }
  }
}

// Tokens that only some of a unit's rows see. For the other rows' columns their probability is zero, which does not keep a value
// that is NaN or infinite out of the product. Such values are looked for in these tokens, a unit's last few, and
// where there are any, they are added to O for the columns that see them, and replaced by zeros for the product. (The look
// costs a unit less than 1 us; a thread to each token, not a warp, cost 10 of 246 us with 16 requests of two rows. Tiles of
// their own for each row's last tokens would not do: they end in the same O.)
template <bool kBf16>
__device__ __forceinline__ bool no_number(uint32_t bits) {
  constexpr uint32_t kExponent = kBf16 ? 0x7F80 : 0x7C00;
  return (bits & kExponent) == kExponent;
}

struct Values {  // a tile's, in the ring
  uint32_t ring, piece, slots;  // the first piece, counted from the launch's first
  int dv;
  __device__ __forceinline__ uint32_t chunk(int c) const { return ring + (piece + c / 2) % slots * kPiece + c % 2 * kChunk; }
};

// Whether one of the tokens `who` of the warp's 32 has such a value; all lanes look at one token at a time. With `clear`, zeros
// take their places.
template <bool kBf16, bool kClear>
static __device__ __noinline__ bool find_no_numbers(Values v, int first_token, uint32_t who) {
  constexpr uint32_t kExponents = kBf16 ? 0x7F807F80 : 0x7C007C00, kLowest = kBf16 ? 0x00800080 : 0x04000400;
  const int lane = threadIdx.x & 31;
  uint32_t found = 0;
#pragma unroll 1
  for (; who; who &= who - 1) {
    const int token = first_token + __ffs(who) - 1;
#pragma unroll 1
    for (int c = lane >> 3; c * 64 < v.dv; c += 4) {
      const uint32_t at = v.chunk(c) + token * 128 + (lane & 7) * 16;
      uint32_t x[4];
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t bad = ((x[i] & kExponents) + kLowest) & 0x80008000;  // an exponent of all ones carries
        found |= bad;
        if (kClear) x[i] &= ~((bad >> 15) * 0xFFFF);
      }
      if (kClear) asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
    }
  }
  return found != 0;
}

// Adds them to O in this thread's lane: value `dim` of each piece, `columns` columns from `o` on, which see as many tokens as
// `limit` says.
template <bool kBf16, int kColumns>
static __device__ __noinline__ void add_no_numbers(Values v, uint32_t o, uint32_t n, int v_pieces, int dim, const int32_t* position, int split,
                                                   const int32_t* limit) {
#pragma unroll 1
  for (int token = 0; token < kTile; ++token) {
    const int pos = position[token];
    if (pos < split || pos == INT_MAX) continue;
#pragma unroll 1
    for (int u = 0; u < v_pieces; ++u) {
      uint16_t bits;
      asm volatile("ld.shared.u16 %0, [%1];"
                   : "=h"(bits)
                   : "r"(v.chunk(u * 2 + (dim >> 6)) + token * 128 + ((((dim & 63) >> 3) ^ (token & 7)) << 4) + (dim & 7) * 2)
                   : "memory");
      const bool mine = u * 128 + dim < v.dv && no_number<kBf16>(bits);
      if (!__any_sync(~0u, mine)) continue;
      const float x = !mine ? 0.f : (kBf16 ? __bfloat162float(__ushort_as_bfloat16(bits)) : __half2float(__ushort_as_half(bits)));
#pragma unroll 1
      for (int i = 0; i < kColumns; i += 8) {
        float y[8];
        tmem_load(o + u * n + i, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] += pos < limit[i + j] ? x : 0.f;
        tmem_store8(o + u * n + i, y);
        store_wait();
      }
    }
  }
}

// The softmax warps call it for a tile of such tokens, which has been scored and not yet been multiplied with its values.
template <int N, bool kBf16, bool kLatent>
static __device__ __noinline__ void protect(const Params& p, Smem<N>& sm, uint32_t ring, uint32_t tile, uint32_t segment, bool first, uint32_t tmem) {
  const int half = threadIdx.x >> 7, token = threadIdx.x & 127, split = sm.split[segment & 1][half];
  const int32_t* position = sm.token[tile % kTokenSlots];
  const Guard guard{&sm.gave_up, p.R.status};
  const uint32_t k_ring = p.k_pieces - p.rest;
  const Values v{ring, tile * (k_ring + (kLatent ? 0 : p.v_pieces)) + (kLatent ? 0 : k_ring), static_cast<uint32_t>(p.slots), p.a.dv};
  const uint32_t come = smem_addr(kLatent ? &sm.key_come[0] : &sm.value_come[0]), number = tile * (kLatent ? k_ring : p.v_pieces);
  const uint32_t who = __ballot_sync(~0u, position[token] >= split && position[token] != INT_MAX);
  // the last tile's values are through, so that what is waited for is this tile's
  if (!first) mbar_wait(smem_addr(&sm.o_done[(tile & 1) ^ 1]), ((tile - 1) >> 1) & 1, guard);
#pragma unroll 1
  for (int u = 0; u < p.v_pieces; ++u) mbar_wait(come + (number + u) % kMaxSlots * 8, (number + u) / kMaxSlots & 1, guard);
  __syncwarp();
  // both halves of the warps, of which the first looks, decide the same
  if (!named_any(3, kSoftmaxWarps * 32, half == 0 && find_no_numbers<kBf16, false>(v, token & ~31, who))) return;
  const uint32_t o = tmem + ((token & ~31u) << 16) + half * (N / 2);
  __syncwarp();
  if (!first) {
    fence_after();
  } else {
    const float zeros[8] = {};
    for (int u = 0; u < p.v_pieces; ++u)
      for (int i = 0; i < N / 2; i += 8) tmem_store8(o + u * N + i, zeros);
    store_wait();
    if (threadIdx.x == 0) sm.kept = tile + 1;
  }
  add_no_numbers<kBf16, N / 2>(v, o, N, p.v_pieces, token, position, split, sm.limit[segment & 1][half]);
  named_sync(3, kSoftmaxWarps * 32);
  if (half == 0) find_no_numbers<kBf16, true>(v, token & ~31, who);
  __syncwarp();
}

template <int N, bool kBf16, bool kLatent>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ Params p) {
  constexpr int kPlaces = places<kLatent>;
  extern __shared__ __align__(1024) uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const uint32_t q_at = base, ring = q_at + p.q_bytes, rest = ring + p.slots * kPiece;
  const uint32_t p_at = rest + (p.rest && !p.rest_is_p ? kChunk : 0);
  Smem<N>& sm = *reinterpret_cast<Smem<N>*>(raw + (p_at + kPlaces * kChunk - smem_addr(raw)));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int block = blockIdx.x % p.blocks, slice = blockIdx.x / p.blocks;
  const Guard guard{&sm.gave_up, p.R.status};

  if (tid == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(smem_addr(&sm.key_come[i]), kCopyThreads);
      mbar_init(smem_addr(&sm.value_come[i]), kCopyThreads);
      mbar_init(smem_addr(&sm.empty[i]), 1);
    }
    mbar_init(smem_addr(&sm.q_first), kSoftmaxWarps * 32);
    mbar_init(smem_addr(&sm.q_full), kCopyThreads);
    mbar_init(smem_addr(&sm.q_empty), 1);
    mbar_init(smem_addr(&sm.rest_full), kCopyThreads);
    mbar_init(smem_addr(&sm.rest_empty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sm.s_full[i]), 1);
      mbar_init(smem_addr(&sm.s_empty[i]), kSoftmaxWarps);
      mbar_init(smem_addr(&sm.p_full[i]), kSoftmaxWarps);
      mbar_init(smem_addr(&sm.o_done[i]), 1);
      mbar_init(smem_addr(&sm.all_done[i]), 1);
    }
    for (int i = 0; i < kTokenSlots; ++i) mbar_init(smem_addr(&sm.token_full[i]), kCopyThreads);
    sm.gave_up = 0;
    sm.kept = 0;
    fence_async();
  }
  if (warp == kScoreWarp) tmem_alloc(smem_addr(&sm.tmem), p.tmem_cols);
  dependent_wait();
  dependent_launch();

  // where this slice's run begins
  if (p.row_tiles) {
    if (tid == 0) {
      const int64_t units = p.row_groups * p.a.kv_heads;
      sm.tiles = units * p.row_tiles;
      if (p.whole) {
        const int64_t unit = slice_begin(units, p.slices, slice);
        sm.run_begin = unit * p.row_tiles;
        sm.run_end = slice_begin(units, p.slices, slice + 1) * p.row_tiles;
        sm.start_group = p.a.kv_heads == 1 ? unit : unit / p.a.kv_heads;
      } else {
        sm.run_begin = slice_begin(sm.tiles, p.slices, slice);
        sm.run_end = slice_begin(sm.tiles, p.slices, slice + 1);
        const int64_t per = static_cast<int64_t>(p.row_tiles) * p.a.kv_heads;
        sm.start_group = sm.run_begin < kSmallTiles ? static_cast<uint32_t>(sm.run_begin) / static_cast<uint32_t>(per) : sm.run_begin / per;
      }
      sm.start_at = sm.run_begin - sm.start_group * p.a.kv_heads * p.row_tiles;
    }
  } else {
    const int64_t per = (p.row_groups + kThreads - 1) / kThreads;
    const int64_t g0 = min(per * tid, p.row_groups), g1 = min(g0 + per, p.row_groups);
    int64_t mine = 0;
    for (int64_t g = g0; g < g1; ++g) mine += group_tiles(p, g);
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
      if (g1 - g0 == 1) {
        sm.start_group = g0;
        sm.start_at = begin - at;
      }
      for (int64_t g = g0; g1 - g0 > 1 && g < g1; ++g) {
        const int64_t n = static_cast<int64_t>(group_tiles(p, g)) * p.a.kv_heads;
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
  const int64_t all_tiles = sm.tiles, run_begin = sm.run_begin;
  Walk walk;
  walk.left = sm.run_end - run_begin;
  walk.group = sm.start_group;
  walk.count = 0;
  if (walk.left > 0) {
    walk.tiles = group_tiles(p, walk.group);
    walk.kv_head = 0;
    int64_t at = sm.start_at;
    for (; at >= walk.tiles; at -= walk.tiles) ++walk.kv_head;
    walk.at = static_cast<int>(at);
    walk.size();
  }
  const int k_ring = p.k_pieces - p.rest;                       // pieces of the keys in the ring
  const uint32_t s_cols = static_cast<uint32_t>(p.v_pieces) * N;  // columns before the scores'
  const int block_cols = min(p.block_cols, p.cols - block * p.block_cols);

  // the first segment's queries, by the warps that have nothing to do yet
  if (walk.left > 0 && warp < kSoftmaxWarps) {
    copy_queries<N>(p, q_at, walk.group * p.pack, walk.kv_head, block, block_cols, tid, kSoftmaxWarps * 32);
    copies_arrive(smem_addr(&sm.q_first));
  }
  if (warp >= kSoftmaxWarps && warp < kScoreWarp) {
    // ---- copies -----------------------------------------------------------
    const int me = tid - kSoftmaxWarps * 32;  // a thread's token of a tile
    const uint32_t empty = smem_addr(&sm.empty[0]);
    Ring at, keys, values;
    TokenCopies copies((warp - kSoftmaxWarps) * 32, lane);
    const auto copy_slot = [&](int first, int bytes, const void* cache, uint64_t* come, Ring& number) {
      mbar_wait(empty + at.slot * 8, at.phase ^ 1, guard);
      copies.columns(ring + at.slot * kPiece, kChunk, first, bytes, cache);
      copies_arrive(smem_addr(come + number.slot));
      at.step(p.slots);
      number.step(kMaxSlots);
    };
    uint32_t tile = 0, segment = 0;
    for (; walk.left > 0; walk.next(p), ++segment) {
      const int64_t row0 = walk.group * p.pack;
      const int length = group_length(p, walk.group);
      const int64_t request = length > 0 ? row_request(p.R, row0) : 0;
      const int32_t* list = p.a.indices ? p.a.indices + row0 * p.a.index_row_stride : nullptr;
      // A tile's tokens are found in two steps, each a tile earlier than its result is used: the position (from
      // the list), then the block (from the table).
      const auto listed = [&](int t) {
        const int i = (walk.at + t) * kTile + me;
        if (t >= walk.count) return -1;
        return !list ? i : (i < p.a.num_indices ? list[i] : -1);
      };
      const auto table_entry = [&](int x) {
        return x >= 0 && x < length ? p.R.block_table[request * p.R.table_stride + block_column(p.R, x)] : 0;
      };
      const auto address = [&](const void* cache, int x, int x_block, int64_t block_stride, int64_t token_stride, int64_t head_stride) {
        return static_cast<const char*>(cache) + 2 * (static_cast<int64_t>(x_block) * block_stride +
                                                      (x - block_column(p.R, x) * p.R.block_size) * token_stride + walk.kv_head * head_stride);
      };
      const auto in_cache = [&](int x, int x_block) { return x >= 0 && x < length && x_block >= 0 && x_block < p.R.num_blocks; };
      int at_token = listed(0), next_token = listed(1);
      int at_block = table_entry(at_token);
      asm volatile("" ::"r"(at_block) : "memory");  // here, before any copies are issued: a load waits behind those
      if (segment > 0) {  // the first one's are copied by the softmax warps
        mbar_wait(smem_addr(&sm.q_empty), (segment & 1) ^ 1, guard);
        copy_queries<N>(p, q_at, row0, walk.kv_head, block, block_cols, me, kCopyThreads);
        copies_arrive(smem_addr(&sm.q_full));
      }
      for (int t = 0; t < walk.count; ++t, ++tile) {
        const bool seen = in_cache(at_token, at_block);
        if (!seen && at_token >= 0 && at_token < length) atomicOr(p.R.status, TOPK_DEV_BAD_BLOCK);
        sm.token[tile % kTokenSlots][me] = seen ? at_token : INT_MAX;
        mbar_arrive(smem_addr(&sm.token_full[tile % kTokenSlots]));
        const char *kp = static_cast<const char*>(p.a.k), *vp = static_cast<const char*>(p.a.v);
        if (seen) {
          kp = address(kp, at_token, at_block, p.a.k_block_stride, p.a.k_token_stride, p.a.k_head_stride);
          if (!kLatent) vp = address(vp, at_token, at_block, p.a.v_block_stride, p.a.v_token_stride, p.a.v_head_stride);
        }
        const int next_block = table_entry(next_token), later_token = listed(t + 2);
        copies.aim(kp, seen, lane);
        const auto copy_rest = [&]() {
          mbar_wait(smem_addr(&sm.rest_empty), (tile & 1) ^ 1, guard);
          copies.columns(rest, kChunk, k_ring * 2 * 128, p.a.dk * 2, p.a.k);
          copies_arrive(smem_addr(&sm.rest_full));
        };
        // the rest first where its buffer is free since the last tile was scored
        if (kLatent && p.rest && !p.rest_is_p) copy_rest();
        for (int u = 0; u < k_ring; ++u) copy_slot(u * 2 * 128, p.a.dk * 2, p.a.k, sm.key_come, keys);
        if (kLatent && p.rest && p.rest_is_p) copy_rest();
        if constexpr (!kLatent) {
          copies.aim(vp, seen, lane);
          for (int u = 0; u < p.v_pieces; ++u) copy_slot(u * 2 * 128, p.a.dv * 2, p.a.v, sm.value_come, values);
        }
        at_token = next_token;
        at_block = next_block;
        next_token = later_token;
      }
    }
    copies_wait_all();
  } else if (warp == kScoreWarp) {
    // ---- S^T = K Q^T, into one of two places ---------------------------------
    constexpr uint32_t kInst = instruction(kBf16 ? kBF16 : kF16, N, false);
    const uint32_t come = smem_addr(&sm.key_come[0]), empty = smem_addr(&sm.empty[0]);
    const int whole_pieces = p.a.dk / (2 * 64);
    const bool rest_first = kLatent && p.rest && !p.rest_is_p;
    Ring at, keys;
    uint32_t tile = 0, segment = 0;
    for (; walk.left > 0; walk.next(p), ++segment) {
      if (segment == 0)
        mbar_wait_warp(smem_addr(&sm.q_first), 0, guard);
      else
        mbar_wait_warp(smem_addr(&sm.q_full), (segment & 1) ^ 1, guard);
      fence_async();
#pragma unroll 1
      for (int t = 0; t < walk.count; ++t, ++tile) {
        const uint32_t b = tile & 1, d = tmem + s_cols + b * N;
        // the keys' last dims where they fill no piece
        const auto last_dims = [&](bool add) {
          uint32_t k_at, q_piece = q_at + whole_pieces * 2 * (N * 128);
          if (kLatent && p.rest) {
            k_at = rest;
            mbar_wait_warp(smem_addr(&sm.rest_full), tile & 1, guard);
          } else {
            k_at = ring + at.slot * kPiece;
            mbar_wait_warp(come + keys.slot * 8, keys.phase, guard);
            keys.step(kMaxSlots);
          }
          fence_async();
          int left = p.a.dk - whole_pieces * (2 * 64);
#pragma unroll 1
          for (; left >= 64; left -= 64, k_at += kChunk, q_piece += N * 128, add = true)
            mma16_chunk(d, operand(k_at, 16), operand(q_piece, 16), kInst, add);
#pragma unroll 1
          for (; left > 0; left -= 16, k_at += 32, q_piece += 32, add = true) mma16_step(d, operand(k_at, 16), operand(q_piece, 16), kInst, add);
          if (kLatent && p.rest) {
            if (!p.rest_is_p) commit(smem_addr(&sm.rest_empty));
          } else {
            if (!kLatent || whole_pieces >= p.v_pieces) commit(empty + at.slot * 8);
            at.step(p.slots);
          }
        };
        mbar_wait_warp(smem_addr(&sm.s_empty[b]), ((tile >> 1) & 1) ^ 1, guard);
        fence_after();
        if (rest_first) last_dims(false);
        uint32_t q_piece = q_at;
#pragma unroll 1
        for (int u = 0; u < whole_pieces; ++u) {
          mbar_wait_warp(come + keys.slot * 8, keys.phase, guard);
          keys.step(kMaxSlots);
          fence_async();
          const uint32_t slot = at.slot;
          at.step(p.slots);
          mma16_pair(d, operand(ring + slot * kPiece, 16), kChunk >> 4, operand(q_piece, 16), (N * 128) >> 4, kInst, rest_first || u > 0);
          q_piece += 2 * N * 128;
          if (!kLatent || u >= p.v_pieces) commit(empty + slot * 8);  // keys that are no values are done with
        }
        if (!rest_first && whole_pieces < p.k_pieces) last_dims(whole_pieces > 0);
        if (!kLatent) at.step(p.slots, p.v_pieces);
        commit(smem_addr(&sm.s_full[b]));
      }
      commit(smem_addr(&sm.q_empty));
    }
    commit(smem_addr(&sm.all_done[0]));
    mbar_wait_warp(smem_addr(&sm.all_done[0]), 0, guard);
  } else if (warp == kValueWarp) {
    // ---- O^T += V^T P^T --------------------------------------------------------
    constexpr uint32_t kInst = instruction(kBf16 ? kBF16 : kF16, N, true);
    const uint32_t come = smem_addr(&sm.value_come[0]), empty = smem_addr(&sm.empty[0]);
    Ring at, values;
    uint32_t tile = 0;
    for (; walk.left > 0; walk.next(p)) {
#pragma unroll 1
      for (int t = 0; t < walk.count; ++t, ++tile) {
        const uint32_t b = tile & 1;
        mbar_wait_warp(smem_addr(&sm.p_full[b]), (tile >> 1) & 1, guard);
        fence_after();
        if (!kLatent) at.step(p.slots, k_ring);
        const bool add = t > 0 || *const_cast<volatile uint32_t*>(&sm.kept) == tile + 1;
        const uint32_t p_tile = operand(p_at + (kPlaces == 2 ? b * kChunk : 0), 1024);
#pragma unroll 1
        for (int u = 0; u < p.v_pieces; ++u) {
          if (!kLatent) {
            mbar_wait_warp(come + values.slot * 8, values.phase, guard);
            values.step(kMaxSlots);
            fence_async();
          }
          mma16_tokens(tmem + u * N, operand(ring + at.slot * kPiece, kChunk), p_tile, kInst, add);
          commit(empty + at.slot * 8);
          at.step(p.slots);
        }
        if (kLatent) at.step(p.slots, k_ring - p.v_pieces);
        if (kLatent && p.rest_is_p) commit(smem_addr(&sm.rest_empty));
        commit(smem_addr(&sm.o_done[b]));
      }
    }
    commit(smem_addr(&sm.all_done[1]));
    mbar_wait_warp(smem_addr(&sm.all_done[1]), 0, guard);
  } else {
    // ---- softmax and output ------------------------------------------------
    constexpr int H = N / 2;
    constexpr float kMostProbability = kBf16 ? 256.f : 32768.f;  // 2^(kMoveAbove + kShift)
    constexpr float kShift = kBf16 ? 0.f : 7.f;  // fp16: probabilities use the upper half of its range, at most 2^15
    const int half = warp >> 2, quarter = warp & 3, token = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int my_col = half * H + (lane & (H - 1));  // the column whose statistics this lane keeps
    uint32_t tile = 0, segment = 0;
    bool first_segment = true;
    for (; walk.left > 0; walk.next(p), ++segment) {
      const int64_t row0 = walk.group * p.pack;
      if (quarter == 0) {  // what each column sees
        const int c = block * p.block_cols + my_col;
        int n = INT_MAX;
        if (my_col < block_cols) {
          const int j = c / p.group;
          n = row_length(p.R, row0 + j);
          if (lane < H)
            sm.out_at[segment & 1][half][lane] = (row0 + j) * p.a.out_row_stride + static_cast<int64_t>(walk.kv_head * p.group + c - j * p.group) * p.a.out_head_stride;
        }
        int least = n, split = INT_MAX;
        if (p.pack > 1) {
#pragma unroll 1
          for (int j = lane; j < p.pack; j += 32) {
            const int seen = row_length(p.R, row0 + j);
            if (seen > 0) split = min(split, seen);
          }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
          least = min(least, __shfl_xor_sync(~0u, least, d));
          split = min(split, __shfl_xor_sync(~0u, split, d));
        }
        if (lane < H) sm.limit[segment & 1][half][lane] = n == INT_MAX ? 0 : n;
        if (lane == 0) {
          sm.least[segment & 1][half] = least;
          sm.split[segment & 1][half] = split;
        }
      }
      named_sync(1 + half, 128);
      const int least = sm.least[segment & 1][half], split_at = sm.split[segment & 1][half] / kTile - walk.at;
      // of my_col, in powers of two: its maximum when that last moved, and what is taken off its scores; the lowest
      // number until a finite one has come, so that any such score makes the maximum move
      float m = -INFINITY, in_use = -FLT_MAX;
      float l[H];
#pragma unroll
      for (int i = 0; i < H; ++i) l[i] = 0.f;
      for (int t = 0; t < walk.count; ++t, ++tile) {
        mbar_wait(smem_addr(&sm.token_full[tile % kTokenSlots]), (tile / kTokenSlots) & 1, guard);
        const int pos = sm.token[tile % kTokenSlots][token];
        mbar_wait(smem_addr(&sm.s_full[tile & 1]), (tile >> 1) & 1, guard);
        fence_after();
        if (t >= split_at) protect<N, kBf16, kLatent>(p, sm, ring, tile, segment, t == 0, tmem);
        float s[H];
        tmem_load(tmem + lanes + s_cols + (tile & 1) * N + half * H, s);
        const auto mask = [&]() {
          if (pos >= least) {
#pragma unroll
            for (int i = 0; i < H; ++i)
              if (pos >= sm.limit[segment & 1][half][i]) s[i] = -INFINITY;
          }
        };
        const auto probabilities = [&]() {
#pragma unroll
          for (int i = 0; i < H; i += 4) {
            const float4 u = *reinterpret_cast<const float4*>(&sm.moved[warp][0][i]);
            s[i] = exp2_fast(fmaf(s[i], p.scale2, -u.x));
            s[i + 1] = exp2_fast(fmaf(s[i + 1], p.scale2, -u.y));
            s[i + 2] = exp2_fast(fmaf(s[i + 2], p.scale2, -u.z));
            s[i + 3] = exp2_fast(fmaf(s[i + 3], p.scale2, -u.w));
          }
        };
        mask();
        // With the maxima in use: is any of the probabilities so large that its column's has to move?
        bool move_any = t == 0;
        if (t > 0) {
          probabilities();
          float x = 0.f;
#pragma unroll
          for (int i = 0; i < H; i += 2) x = fmaxf(x, fmaxf(s[i], s[i + 1]));
          move_any = named_any(1 + half, 128, x > kMostProbability);
        }
        bool rescale = false;
        if (move_any) {
          if (t > 0) {
            tmem_load(tmem + lanes + s_cols + (tile & 1) * N + half * H, s);
            mask();
          }
          const float warp_max = reduce_columns<H, true>(s, lane);
          if (lane < H) sm.column_max[half][quarter][lane] = warp_max;
          named_sync(1 + half, 128);
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) top = fmaxf(top, sm.column_max[half][w][lane & (H - 1)]);
          top *= p.scale2;
          const bool move = top > m + kMoveAbove || (m == -INFINITY && top > m);
          rescale = __any_sync(~0u, move && m > -INFINITY);
          const float factor = move && m > -INFINITY ? exp2_fast(m - top) : 1.f;
          if (move) {
            m = top;
            in_use = m - kShift;
          }
          if (lane < H) {
            sm.moved[warp][0][lane] = in_use;
            sm.moved[warp][1][lane] = factor;
          }
          __syncwarp();
          probabilities();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.s_empty[tile & 1]));
        if (rescale) {  // the same for all warps of this half: they hold the same maxima
          mbar_wait(smem_addr(&sm.o_done[(tile & 1) ^ 1]), ((tile - 1) >> 1) & 1, guard);  // the tile before has been added
          __syncwarp();
          fence_after();
#pragma unroll
          for (int i = 0; i < H; ++i) l[i] *= sm.moved[warp][1][i];
          for (int u = 0; u < p.v_pieces; ++u) {
#pragma unroll 1
            for (int i = 0; i < H; i += 8) {
              float o[8];
              const uint32_t at = tmem + lanes + u * N + half * H + i;
              tmem_load(at, o);
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] *= sm.moved[warp][1][i + j];
              tmem_store8(at, o);
            }
          }
          store_wait();
        }
        // the product that read this place of P is done
        if (tile >= kPlaces) mbar_wait(smem_addr(&sm.o_done[(tile - kPlaces) & 1]), ((tile - kPlaces) >> 1) & 1, guard);
        const uint32_t row = p_at + (kPlaces == 2 ? (tile & 1) * kChunk : 0) + token * 128;
        {
#pragma unroll
          for (int i = 0; i < H; i += 8) {
            const uint32_t at = row + ((((half * H + i) >> 3) ^ (token & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(pack2<kBf16>(s[i], s[i + 1])),
                         "r"(pack2<kBf16>(s[i + 2], s[i + 3])), "r"(pack2<kBf16>(s[i + 4], s[i + 5])),
                         "r"(pack2<kBf16>(s[i + 6], s[i + 7]))
                         : "memory");
          }
        }
        fence_async();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.p_full[tile & 1]));
#pragma unroll
        for (int i = 0; i < H; ++i) l[i] += s[i];
      }
      const float part_l = reduce_columns<H, false>(l, lane);
      if (lane < H) sm.column_sum[half][quarter][lane] = part_l;
      named_sync(1 + half, 128);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) sum += sm.column_sum[half][w][lane & (H - 1)];
      const bool whole = walk.count == walk.tiles;
      const int64_t slot = ((static_cast<int64_t>(slice) * 2 + (first_segment ? 0 : 1)) * p.blocks + block) * N;
      const float inverse = sum == 0.f ? 0.f : 1.f / sum;
      const bool blank = __any_sync(~0u, sum == 0.f);  // some column saw nothing: its values are zeros, whatever stands in O
      if (lane < H) sm.moved[warp][0][lane] = inverse;
      if (quarter == 0 && lane < H) {
        if (!whole) {
          p.stat[slot + my_col] = make_float2(m == -INFINITY ? -INFINITY : in_use, sum);
        } else if (p.a.lse && my_col < block_cols) {
          const int c = block * p.block_cols + my_col, j = c / p.group;
          p.a.lse[(row0 + j) * p.a.heads + walk.kv_head * p.group + c - j * p.group] =
              sum == 0.f ? -INFINITY : (in_use + log2f(sum)) * 0.69314718055994531f;
        }
      }
      __syncwarp();
      mbar_wait(smem_addr(&sm.o_done[(tile & 1) ^ 1]), ((tile - 1) >> 1) & 1, guard);
      __syncwarp();
      fence_after();
#pragma unroll 1
      for (int u = 0; u < p.v_pieces; ++u) {
        float o[H];
        tmem_load(tmem + lanes + u * N + half * H, o);
        const int dim = u * 128 + token;
        if (blank) {
#pragma unroll
          for (int i = 0; i < H; ++i)
            if (sm.moved[warp][0][i] == 0.f) o[i] = 0.f;
        }
        if (!whole) {  // [dim][column]: a thread's columns side by side
          float4* to = reinterpret_cast<float4*>(p.part + slot * (p.v_pieces * 128) + dim * N + half * H);
#pragma unroll
          for (int i = 0; i < H; i += 4) to[i / 4] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        } else {
          // two columns at a time: neighbouring lanes exchange them and store pairs of dims
          const int odd = lane & 1, d = dim - odd, real = d < p.a.dv ? block_cols - half * H - odd : 0;
          const int64_t* out_at = sm.out_at[segment & 1][half] + odd;
          uint16_t* out = static_cast<uint16_t*>(p.a.out) + d;
#pragma unroll
          for (int i = 0; i < H; i += 2) {
            const float2 f = *reinterpret_cast<const float2*>(&sm.moved[warp][0][i]);
            const uint32_t mine = pack2<kBf16>(o[i] * f.x, o[i + 1] * f.y), other = __shfl_xor_sync(~0u, mine, 1);
            // the even lane has this column of both dims, the odd lane the next one
            const uint32_t both = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
            if (i < real) *reinterpret_cast<uint32_t*>(out + out_at[i]) = both;
          }
        }
      }
      fence_before();
      const bool ends = walk.at + walk.count == walk.tiles;
      if (tid == 0 && block == 0 && (p.by_unit ? ends : first_segment)) {  // a unit that began before this slice and ends in it
        Join j{};
        j.last = -1;
        if (walk.at > 0 && ends) {
          const int64_t unit_begin = run_begin - walk.at;
          j.rowgroup = walk.group;
          j.kv_head = walk.kv_head;
          j.first = slice_of(all_tiles, p.slices, unit_begin);
          j.last = slice;
          j.first_slot = slice_begin(all_tiles, p.slices, j.first) == unit_begin ? 0 : 1;
          j.tiles = all_tiles;
        }
        p.join[p.by_unit ? walk.group * p.a.kv_heads + walk.kv_head : slice] = j;
      }
      first_segment = false;
    }
    if (first_segment && !p.by_unit && tid == 0 && block == 0) {  // an empty run
      Join j{};
      j.last = -1;
      p.join[slice] = j;
    }
  }
  if (blockIdx.x == 0) report_rows(p.R, tid, kThreads);
  settle(guard);
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kScoreWarp) tmem_free(tmem, p.tmem_cols);
}

// A load that stays where it is written: left to the compiler, the join's loads move to their uses, one latency each
// (4 parts of eight loads a thread: 17 000 cycles against 4300).
__device__ __forceinline__ float4 load_now(const float4* at) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(at) : "memory");
  return v;
}

// Joins the parts of the units that fell into several slices: kJoinDims values of a unit's columns a CTA. Every thread
// has four columns of some values and sums them over its team's parts, four parts' loads at a time; the teams' sums meet in
// shared memory, to be stored along the values.
template <int N, bool kBf16>
__global__ void __launch_bounds__(kTeam * kMaxTeams) join_kernel(const __grid_constant__ Params p) {
  __shared__ int32_t place[kMaxParts];  // of each part, in columns; -1: the slice was empty
  __shared__ float base[N], inverse[N];
  __shared__ float sums[kJoinDims][N + 4];
  const int tid = threadIdx.x, per = p.v_pieces * 128 / kJoinDims;
  const int dim0 = blockIdx.x % per * kJoinDims, block = blockIdx.x / per % p.blocks, at_join = blockIdx.x / per / p.blocks;
  const int block_cols = min(p.block_cols, p.cols - block * p.block_cols);
  dependent_wait();
  dependent_launch();
  const Join jn = p.join[at_join];
  if (jn.last < 0 || dim0 >= p.a.dv) return;
  const int parts = jn.last - jn.first + 1, width = p.v_pieces * 128;
  const int64_t row0 = jn.rowgroup * p.pack;
  for (int i = tid; i < parts; i += kTeam * p.teams) {
    const int s = jn.first + i;
    const bool empty = slice_begin(jn.tiles, p.slices, s) == slice_begin(jn.tiles, p.slices, s + 1);
    place[i] = empty ? -1 : ((s * 2 + (i == 0 ? jn.first_slot : 0)) * p.blocks + block) * N;
  }
  __syncthreads();
  {  // each column's maximum and sum
    const int lanes_each = kTeam / N * p.teams;
    const int col = tid / lanes_each, sub = tid % lanes_each;
    float m = -INFINITY, sum = 0.f;
    for (int i = sub; i < parts; i += lanes_each) {
      if (place[i] < 0) continue;
      const float2 st = p.stat[place[i] + col];
      const float top = fmaxf(m, st.x), b = top == -INFINITY ? 0.f : top;
      sum = sum * exp2f(m - b) + st.y * exp2f(st.x - b);
      m = top;
    }
#pragma unroll
    for (int d = lanes_each / 2; d; d >>= 1) {
      const float m2 = __shfl_xor_sync(~0u, m, d), sum2 = __shfl_xor_sync(~0u, sum, d);
      const float top = fmaxf(m, m2), b = top == -INFINITY ? 0.f : top;
      sum = sum * exp2f(m - b) + sum2 * exp2f(m2 - b);
      m = top;
    }
    if (sub == 0) {
      base[col] = m == -INFINITY ? 0.f : m;
      inverse[col] = sum == 0.f ? 0.f : 1.f / sum;
      const int c = block * p.block_cols + col, j = c / p.group;
      if (p.a.lse && dim0 == 0 && col < block_cols)
        p.a.lse[(row0 + j) * p.a.heads + jn.kv_head * p.group + c - j * p.group] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994531f;
    }
  }
  __syncthreads();
  constexpr int kRow = N / 4, kEach = kJoinDims * kRow / kTeam, kAtOnce = 4;
  const int team = tid / kTeam, col = tid % kRow * 4, dim = tid % kTeam / kRow;  // and every kTeam / kRow dims on
  float4 x[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 b = make_float4(base[col], base[col + 1], base[col + 2], base[col + 3]);
  for (int i0 = team; i0 < parts; i0 += kAtOnce * p.teams) {
    float4 y[kAtOnce][kEach], st[kAtOnce][2];
#pragma unroll
    for (int a = 0; a < kAtOnce; ++a) {
      const int i = i0 + a * p.teams, at = max(i < parts ? place[i] : 0, 0);
      st[a][0] = load_now(reinterpret_cast<const float4*>(p.stat + at + col));
      st[a][1] = load_now(reinterpret_cast<const float4*>(p.stat + at + col) + 1);
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        y[a][k] = load_now(reinterpret_cast<const float4*>(p.part + static_cast<int64_t>(at) * width + (dim0 + dim + k * (kTeam / kRow)) * N + col));
    }
#pragma unroll
    for (int a = 0; a < kAtOnce; ++a) {
      const int i = i0 + a * p.teams;
      if (i >= parts || place[i] < 0) continue;
      const float4 w = make_float4(exp2f(st[a][0].x - b.x), exp2f(st[a][0].z - b.y), exp2f(st[a][1].x - b.z), exp2f(st[a][1].z - b.w));
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        x[k].x += w.x * y[a][k].x;
        x[k].y += w.y * y[a][k].y;
        x[k].z += w.z * y[a][k].z;
        x[k].w += w.w * y[a][k].w;
      }
    }
  }
  for (int turn = 0; turn < p.teams; ++turn) {  // in the teams' order: the same sums every time
    if (team == turn) {
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        float4* to = reinterpret_cast<float4*>(&sums[dim + k * (kTeam / kRow)][col]);
        const float4 y = turn == 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : *to;
        *to = make_float4(x[k].x + y.x, x[k].y + y.y, x[k].z + y.z, x[k].w + y.w);
      }
    }
    if (turn + 1 < min(parts, p.teams)) __syncthreads();
    else break;
  }
  __syncthreads();
  for (int e = tid; e < block_cols * (kJoinDims / 2); e += kTeam * p.teams) {
    const int n = e / (kJoinDims / 2), d = e % (kJoinDims / 2) * 2, c = block * p.block_cols + n, j = c / p.group;
    if (dim0 + d < p.a.dv)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.a.out) + (row0 + j) * p.a.out_row_stride +
                                   static_cast<int64_t>(jn.kv_head * p.group + c - j * p.group) * p.a.out_head_stride + dim0 + d) =
          inverse[n] == 0.f ? 0u : pack2<kBf16>(sums[d][n] * inverse[n], sums[d + 1][n] * inverse[n]);
  }
}

constexpr size_t kJoinBytes = sizeof(Join);

// CTAs of a launch: one on each SM, or one for each column block where there are more of those.
int most_ctas(int sms) { return sms > 16 ? sms : 16; }

size_t workspace_for(int sms) {
  const size_t slots = static_cast<size_t>(most_ctas(sms)) * 2;
  return TOPK_PAGED_WORKSPACE_BYTES + (most_ctas(sms) * kJoinBytes + 255) / 256 * 256 + slots * kMaxBlockCols * (kMaxV * sizeof(float) + sizeof(float2));
}

static_assert(sizeof(Smem<64>) + 1024 + 9 * 64 * 128 + 4 * kPiece + kChunk <= 232448, "a latent tile beside 64 columns");

template <int N, bool kBf16, bool kLatent>
int run(Params& p, int device, int smem_limit, bool joins, cudaStream_t stream) {
  const int extra = static_cast<int>(sizeof(Smem<N>)) + 1024;
  p.q_bytes = p.k_chunks * N * 128;
  p.rest_is_p = 0;
  constexpr int kPBytes = places<kLatent> * kChunk;
  int room = smem_limit - extra - static_cast<int>(p.q_bytes) - kPBytes;  // for the ring and, where it is not P, the rest
  if (p.rest) {
    // a buffer of its own for the rest lets the next tile's last keys come early, if the ring loses nothing by it
    p.rest_is_p = (room - kChunk) / kPiece < room / kPiece;
    if (!p.rest_is_p) room -= kChunk;
  }
  p.slots = room / kPiece < kMaxSlots ? room / kPiece : kMaxSlots;
  const int k_ring = p.k_pieces - p.rest;
  if (p.slots < (p.latent && k_ring > 2 ? k_ring : 2) || (!p.latent && p.pack > 1 && p.slots < p.v_pieces)) return TOPK_ERR_PLAN;
  p.tmem_cols = 32;
  while (p.tmem_cols < static_cast<uint32_t>((p.v_pieces + 2) * N)) p.tmem_cols *= 2;
  const size_t smem = p.q_bytes + static_cast<size_t>(p.slots) * kPiece + (p.rest && !p.rest_is_p ? kChunk : 0) + kPBytes + extra;
  static int granted[kMaxDevices];
  int rc = allow_smem(attention_kernel<N, kBf16, kLatent>, smem_limit, device, granted);
  if (rc != TOPK_OK) return rc;
  rc = launch(attention_kernel<N, kBf16, kLatent>, static_cast<const Params&>(p), static_cast<int64_t>(p.slices) * p.blocks, kThreads, smem, stream);
  if (rc != TOPK_OK || !joins) return rc;
  return launch(join_kernel<N, kBf16>, static_cast<const Params&>(p), static_cast<int64_t>(p.joins) * p.blocks * (p.v_pieces * 128 / kJoinDims), kTeam * p.teams, 0, stream);
}

template <int N>
int run_columns(Params& p, int device, int smem_limit, bool joins, cudaStream_t stream) {
  const bool bf16 = p.a.dtype == TOPK_DTYPE_BF16;
  if (p.latent) return bf16 ? run<N, true, true>(p, device, smem_limit, joins, stream) : run<N, false, true>(p, device, smem_limit, joins, stream);
  return bf16 ? run<N, true, false>(p, device, smem_limit, joins, stream) : run<N, false, false>(p, device, smem_limit, joins, stream);
}

}  // namespace
}  // namespace paged
}  // namespace ltk

extern "C" size_t topk_attention_workspace_size(int device) {
  topk_device_props p{};
  if (topk_query_device(device, &p) != TOPK_OK) return 0;
  return ltk::paged::workspace_for(p.num_sms);
}

extern "C" int topk_paged_attention(const topk_attention_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_attention_args& a = *args;
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
  int dev = 0;
  topk_device_props props{};
  if (cudaGetDevice(&dev) != cudaSuccess || topk_query_device(dev, &props) != TOPK_OK) {
    cudaGetLastError();
    return TOPK_ERR_CUDA;
  }
  const int sms = props.num_sms;
  if (a.workspace_bytes < workspace_for(sms)) return TOPK_ERR_WORKSPACE_TOO_SMALL;

  Params p{};
  p.a = a;
  p.R = make_rows(a.rows, INT32_MAX, a.workspace);
  p.group = a.heads / a.kv_heads;
  // The rows of a request share its tokens, unless index lists tell them apart. (Even where that makes no fewer column blocks:
  // 16 requests of two rows of 128 heads over 8 K to 32 K tokens take 247 us, each row by itself 255.)
  // Not where a tile's values are more pieces than the ring may hold, which have to be there together before the product of
  // tokens that only some rows see.
  p.latent = a.v == nullptr;
  p.k_chunks = (a.dk + 63) / 64;
  p.v_pieces = (a.dv + 127) / 128;
  const int held = (props.max_smem_optin - static_cast<int>(sizeof(Smem<64>)) - 1024 - p.k_chunks * 64 * 128 - 2 * kChunk) / kPiece;
  const bool together = a.indices == nullptr && a.rows.row_request == nullptr && a.rows.next_n * static_cast<int64_t>(p.group) <= 1024 &&
                        (p.latent || p.v_pieces <= held);
  p.pack = together ? a.rows.next_n : 1;
  p.cols = p.pack * p.group;
  p.blocks = (p.cols + kMaxBlockCols - 1) / kMaxBlockCols;
  p.block_cols = (p.cols + p.blocks - 1) / p.blocks;
  p.k_pieces = (p.k_chunks + 1) / 2;
  p.rest = p.latent && p.k_chunks % 2 == 1 && p.k_pieces > p.v_pieces;
  p.row_groups = a.rows.num_rows / p.pack;
  p.row_tiles = a.indices ? (a.num_indices + kTile - 1) / kTile : 0;
  p.scale2 = a.scale * 1.4426950408889634f;
  const int64_t units = p.row_groups * a.kv_heads;
  const int64_t most = units * (a.indices ? p.row_tiles : (p.R.max_len + static_cast<int64_t>(kTile) - 1) / kTile);
  int64_t slices = sms / p.blocks < 1 ? 1 : sms / p.blocks;
  if (slices > most) slices = most;
  if (slices > kMaxParts) slices = kMaxParts;
  p.slices = static_cast<int32_t>(slices);
  bool joins = true;
  if (p.row_tiles) {  // every unit has as many tiles
    // Whole units, if the longest run then takes no longer than an equal share with what a split costs: the parts' way
    // through memory and the join take about as long as a tile for every 16 columns.
    const int split_tiles = (p.block_cols + 15) / 16;
    const int64_t equal = (units * p.row_tiles + p.slices - 1) / p.slices, even = (units + p.slices - 1) / p.slices * p.row_tiles;
    p.whole = even <= equal + split_tiles;
    if (p.whole && p.slices > units) p.slices = static_cast<int32_t>(units);
    joins = !p.whole;
  }
  p.by_unit = units <= p.slices;
  // Units in many parts are joined by more threads each; units in a few by more CTAs at once. (One unit in about 100 parts,
  // 64 columns: 35 us with four teams, 55 with one; 64 units in two or three, 16 columns: 39 us with one, 45 with four.)
  p.teams = p.slices >= 8 * units ? kMaxTeams : 1;
  p.joins = p.by_unit ? static_cast<int32_t>(units) : p.slices;
  char* w = static_cast<char*>(a.workspace) + TOPK_PAGED_WORKSPACE_BYTES;
  p.join = reinterpret_cast<Join*>(w);
  w += (most_ctas(sms) * kJoinBytes + 255) / 256 * 256;
  p.stat = reinterpret_cast<float2*>(w);
  w += static_cast<size_t>(most_ctas(sms)) * 2 * kMaxBlockCols * sizeof(float2);
  p.part = reinterpret_cast<float*>(w);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.block_cols <= 16) return run_columns<16>(p, dev, props.max_smem_optin, joins, s);
  if (p.block_cols <= 32) return run_columns<32>(p, dev, props.max_smem_optin, joins, s);
  return run_columns<64>(p, dev, props.max_smem_optin, joins, s);
}
