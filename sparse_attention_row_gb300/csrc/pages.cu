// The pages of a pool: forking and freeing requests, compacting the pool, and copying pages.
//
// Forking and freeing change three things that have to agree: rows of the table, the holders of each page beyond its first, and
// the stack of free pages whose pointer is `taken`. What comes out has to be the same every time, so nothing is handed out or
// handed back in the order of atomics: places come from exclusive sums over the lists, as in the map (kv_map.cu).
//
//   fork     a CTA has some of the forks and counts the new pages of all before them; its threads go along the rows.
//   free     a page that several of the call's rows hold goes back once, at the first of its places. Three steps, a cluster's
//            barrier between them: every place takes a holder off; of a page without holders, the places
//            meet in its word of `shares` by their number's minimum; and the places whose number stands there are counted, summed up
//            and written.
//   compact  marks of what the table and the list name; the free pages in rising and the named ones in falling order by
//            sums over the pool; their pairs are the moves, as long as they lower a number.
//   copy     every cache's pages in pieces of 16 KB over all CTAs, 16 bytes a thread and four loads at a time: bound by HBM.
//
// Free and compact are one cluster of 16 CTAs, whose barrier in hardware takes the place of further launches. They are bound by
// latency (a step is 1 to 2 us) up to some 10 000 entries of the table and by 16 SMs' loads and atomics above: freeing 256 requests
// of about 64 pages, most of them shared, takes 15 us (22 with 8 CTAs); compacting 18 K pages with 16 K entries 15 us (17), 1.1 M pages with
// 1 M entries 169 us. The copy of 1024 pages of 32 KB takes 8 us.
#include "paged.cuh"

namespace ltk {
namespace paged {
namespace {

constexpr int kTicketWord = 8;  // of the workspace, as in the map

// ---- fork -------------------------------------------------------------------

constexpr int kForkThreads = 256;

struct ForkParams {
  topk_page_fork_args a;
  Rows R;  // for the division by block_size
};

struct Fork {
  int64_t parent, child;  // rows of the table
  int32_t whole;          // pages shared
  int32_t source;         // page of what is left, -1: nothing
};

__device__ __forceinline__ Fork read_fork(const ForkParams& p, int64_t i, uint32_t* flags) {
  const topk_page_pool& t = p.a.pool;
  Fork f{p.a.parents[i], p.a.children[i], 0, -1};
  if (f.parent < 0 || f.parent >= t.num_requests || f.child < 0 || f.child >= t.num_requests) {
    *flags |= TOPK_DEV_BAD_BLOCK;
    f.child = -1;
    return f;
  }
  const int n = min(max(p.a.kept_lens[i], 0), p.R.max_len);
  f.whole = block_column(p.R, n);
  if (n > f.whole * p.R.block_size) {
    f.source = t.block_table[f.parent * t.table_stride + f.whole];
    if (f.source < 0 || f.source >= t.num_blocks) {
      *flags |= TOPK_DEV_BAD_BLOCK;
      f.source = -1;
    }
  }
  return f;
}

__global__ void __launch_bounds__(kForkThreads) fork_kernel(const __grid_constant__ ForkParams p) {
  __shared__ Fork forks[kForkThreads];
  __shared__ int32_t rank[kForkThreads], warp_sum[kForkThreads / 32], all_before;
  const topk_page_fork_args& a = p.a;
  const topk_page_pool& t = a.pool;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t flags = 0, none = 0;
  dependent_wait();
  dependent_launch();
  const int64_t taken = *t.taken;
  const int64_t per = (a.num_forks + gridDim.x - 1) / gridDim.x;
  const int64_t i0 = min(per * blockIdx.x, a.num_forks), i1 = min(i0 + per, a.num_forks);
  if (tid == 0) all_before = 0;
  __syncthreads();
  int32_t count = 0;
  for (int64_t i = tid; i < i0; i += kForkThreads) count += read_fork(p, i, &none).source >= 0;
  for (int d = 16; d; d >>= 1) count += __shfl_xor_sync(~0u, count, d);
  if (lane == 0 && count > 0) atomicAdd(&all_before, count);  // a sum of whole numbers: any order
  __syncthreads();
  int64_t before = all_before;
  for (int64_t base = i0; base < i1; base += kForkThreads) {
    const int here = static_cast<int>(min(i1 - base, static_cast<int64_t>(kForkThreads)));
    Fork f{0, -1, 0, -1};
    if (tid < here) f = read_fork(p, base + tid, &flags);
    const unsigned who = __ballot_sync(~0u, f.source >= 0);
    if (lane == 0) warp_sum[warp] = __popc(who);
    __syncthreads();
    int32_t at = __popc(who & ((1u << lane) - 1)), total = 0;
    for (int w = 0; w < kForkThreads / 32; ++w) {
      if (w < warp) at += warp_sum[w];
      total += warp_sum[w];
    }
    forks[tid] = f;
    rank[tid] = at;
    __syncthreads();
    for (int k = 0; k < here; ++k) {
      const Fork g = forks[k];
      const int64_t n = taken + before + rank[k];
      int32_t target = -1;
      if (g.source >= 0) {
        if (n >= 0 && n < t.num_free) {
          target = t.free_blocks[n];
          if (target < 0 || target >= t.num_blocks) {  // no page of the pool
            target = -1;
            flags |= TOPK_DEV_BAD_BLOCK;
          }
        } else {
          flags |= TOPK_DEV_BLOCKS_EXHAUSTED;
        }
      }
      if (tid == 0) {
        a.source[base + k] = target < 0 ? -1 : g.source;
        a.target[base + k] = target;
      }
      if (g.child < 0) continue;
      const int32_t* from = t.block_table + g.parent * t.table_stride;
      int32_t* to = t.block_table + g.child * t.table_stride;
      for (int64_t c = tid; c < t.max_blocks; c += kForkThreads) {
        int32_t page = c == g.whole ? target : -1;
        if (c < g.whole) {
          page = from[c];
          if (page >= 0 && page < t.num_blocks) {
            atomicAdd(t.shares + page, 1);
          } else {
            page = -1;
            flags |= TOPK_DEV_BAD_BLOCK;
          }
        }
        to[c] = page;
      }
    }
    before += total;
    __syncthreads();  // the next forks are written
  }
  if (flags) atomicOr(p.R.status, flags);
  // the CTA with the last forks knows how many pages went; it is the last to have read `taken` if all others have drawn their
  // tickets, and the last one writes what that CTA left
  __shared__ bool last;
  uint32_t* ticket = p.R.status + kTicketWord;
  if (tid == 0) {
    if (blockIdx.x == gridDim.x - 1) ticket[1] = static_cast<uint32_t>(before);
    __threadfence();
    last = gridDim.x == 1 || atomicAdd(ticket, 1u) + 1 == gridDim.x;
    if (last) {
      __threadfence();
      const int64_t after = taken + static_cast<int64_t>(*const_cast<volatile uint32_t*>(ticket + 1));
      ticket[0] = 0;
      ticket[1] = 0;
      *t.taken = static_cast<int32_t>(after < t.num_free ? after : (taken > t.num_free ? taken : t.num_free));
    }
  }
}

// ---- one cluster ------------------------------------------------------------

constexpr int kCluster = 16;  // CTAs at most; 8 where the device takes no more
constexpr int kPageThreads = 1024;
constexpr int kPageWarps = kPageThreads / 32;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}

// All threads of the cluster meet; what they wrote before is seen behind it. In one step, or in two with other work between them.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

__device__ __forceinline__ int32_t read_peer(const int32_t* mine, uint32_t rank) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  uint32_t there;
  int32_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(there) : "memory");
  return v;
}

// What other CTAs of the cluster wrote: from L2.
__device__ __forceinline__ int32_t look(const int32_t* at) { return __ldcg(at); }

__device__ __forceinline__ int4 look4(const int32_t* at) { return __ldcg(reinterpret_cast<const int4*>(at)); }

// Of two counts of every thread: those of the threads before it in `a` and `b`, and the CTA's in `all_a` and `all_b`.
struct Counts {
  int32_t a, b, all_a, all_b;
};
__device__ __forceinline__ Counts count_before(int32_t a, int32_t b, int2 (&warp_sum)[kPageWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t x = a, y = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t u = __shfl_up_sync(~0u, x, d), v = __shfl_up_sync(~0u, y, d);
    if (lane >= d) x += u, y += v;
  }
  __syncthreads();  // the last sums have been read
  if (lane == 31) warp_sum[warp] = make_int2(x, y);
  __syncthreads();
  int2 mine = warp_sum[lane];  // every warp sums them up for itself
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t u = __shfl_up_sync(~0u, mine.x, d), v = __shfl_up_sync(~0u, mine.y, d);
    if (lane >= d) mine.x += u, mine.y += v;
  }
  Counts c;
  c.all_a = __shfl_sync(~0u, mine.x, 31);
  c.all_b = __shfl_sync(~0u, mine.y, 31);
  const int32_t before_a = __shfl_sync(~0u, mine.x, warp ? warp - 1 : 0), before_b = __shfl_sync(~0u, mine.y, warp ? warp - 1 : 0);
  c.a = x - a + (warp ? before_a : 0);
  c.b = y - b + (warp ? before_b : 0);
  return c;
}

// Sums over the cluster of what each CTA has in *mine: those before this one, and all.
__device__ __forceinline__ void sum_of_cluster(const int32_t* mine, int64_t* before, int64_t* all) {
  *before = *all = 0;
  const uint32_t me = cluster_rank(), ctas = cluster_ctas();
  int32_t x[kCluster];
#pragma unroll
  for (uint32_t r = 0; r < kCluster; ++r) x[r] = r < ctas ? read_peer(mine, r) : 0;
#pragma unroll
  for (uint32_t r = 0; r < kCluster; ++r) {
    if (r < me) *before += x[r];
    *all += x[r];
  }
}

// ---- free -------------------------------------------------------------------

constexpr int64_t kMostFreed = 1 << 20;  // requests of a call
constexpr int kOnceWords = kMostFreed / 8 / 32 + 2;
// Requests that were listed before: up to kCompared of them are compared one with another. More are compared within pieces of a CTA's
// share only, and for those before a piece there is a bit for each row of the table, kRowBits rows at a time: the steps then grow with the
// number of requests and not with its square, unless the table's rows are so many more that they make the passes dear. (A call's us, all compared
// and with bits: 1 K requests 23, 21; 4 K 50, 25; 16 K 470, 66; 262 K 119 000, 660.)
constexpr int kCompared = 1024;
constexpr int kRowBits = 24 * 1024 * 8;
constexpr int kEach = 8;                       // places of a thread at a time, side by side
constexpr int kRound = kEach * kPageThreads;  // places of a CTA

struct FreeParams {
  topk_page_free_args a;
  uint32_t* status;
};

__global__ void __launch_bounds__(kPageThreads, 1) free_kernel(const __grid_constant__ FreeParams p) {
  __shared__ int2 warp_sum[kPageWarps];
  __shared__ int32_t mine;
  __shared__ uint32_t again[kOnceWords];  // bits of the requests of this CTA that were listed before
  __shared__ uint32_t listed[kRowBits / 32];  // bits of rows that were
  const topk_page_free_args& a = p.a;
  const topk_page_pool& t = a.pool;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t flags = 0;
  // this CTA's requests, and places: a request's columns in order
  const int64_t per = (a.num_freed + cluster_ctas() - 1) / cluster_ctas(), i0 = min(per * cluster_rank(), a.num_freed), i1 = min(i0 + per, a.num_freed);
  for (int i = tid; i < (i1 - i0 + 31) / 32; i += kPageThreads) again[i] = 0;
  dependent_wait();
  dependent_launch();
  const int64_t taken = min(max(static_cast<int64_t>(*t.taken), int64_t{0}), t.num_free);
  __syncthreads();
  const bool many = a.num_freed > kCompared && a.num_freed > 16 * ((t.num_requests + kRowBits - 1) / kRowBits);
  for (int64_t i = i0 + warp; i < i1; i += kPageWarps) {
    const int32_t request = a.requests[i];
    bool found = false;
#pragma unroll 8
    for (int64_t j = (many ? i - (i - i0) % kPageThreads : 0) + lane; j < i; j += 32) found |= a.requests[j] == request;
    if (__any_sync(~0u, found) && lane == 0) atomicOr(&again[(i - i0) >> 5], 1u << ((i - i0) & 31));
  }
  for (int64_t row0 = 0; many && row0 < t.num_requests; row0 += kRowBits) {
    for (int i = tid; i < kRowBits / 32; i += kPageThreads) listed[i] = 0;
    const auto place = [&](int64_t i) {  // of a request's row in the bits, negative where it has none
      const int64_t row = a.requests[i] - row0;
      return row >= 0 && row < kRowBits ? static_cast<int>(row) : -1;
    };
    __syncthreads();
#pragma unroll 8
    for (int64_t i = tid; i < i0; i += kPageThreads) {
      const int at = place(i);
      if (at >= 0) atomicOr(&listed[at >> 5], 1u << (at & 31));
    }
    __syncthreads();
    for (int64_t piece = i0; piece < i1; piece += kPageThreads) {
      const int64_t i = piece + tid;
      const int at = i < i1 ? place(i) : -1;
      if (at >= 0 && (listed[at >> 5] >> (at & 31) & 1)) atomicOr(&again[(i - i0) >> 5], 1u << ((i - i0) & 31));
      __syncthreads();
      if (at >= 0) atomicOr(&listed[at >> 5], 1u << (at & 31));
      __syncthreads();
    }
  }
  __syncthreads();
  const int64_t places = (i1 - i0) * t.max_blocks;
  const uint32_t columns = static_cast<uint32_t>(t.max_blocks);
  // The pages at this thread's places of a round, -1 where there is none. They stay in registers where there is one round only.
  int32_t page[kEach];
  const auto read = [&](int64_t round) {
    const int64_t first = round * kRound + tid * kEach;
    uint32_t i = static_cast<uint32_t>(first) / columns, c = static_cast<uint32_t>(first) - i * columns;
    int64_t entry[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      entry[k] = -1;
      if (first + k < places && !(again[i >> 5] >> (i & 31) & 1)) {
        const int64_t request = a.requests[i0 + i];
        if (request < 0 || request >= t.num_requests)
          flags |= TOPK_DEV_BAD_BLOCK;
        else
          entry[k] = request * t.table_stride + c;
      }
      if (++c == columns) c = 0, ++i;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) page[k] = entry[k] >= 0 ? t.block_table[entry[k]] : -1;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      if (page[k] >= t.num_blocks) {
        flags |= TOPK_DEV_BAD_BLOCK;
        page[k] = -1;
      }
    }
  };
  const auto number = [&](int64_t round, int k) { return INT32_MIN + static_cast<int32_t>(i0 * t.max_blocks + round * kRound + tid * kEach + k); };
  // Bits of the places whose pages go back: those whose number their page's word holds.
  const auto going_back = [&](int64_t round) {
    int32_t word[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) word[k] = page[k] >= 0 ? look(t.shares + page[k]) : 0;
    uint32_t back = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) back |= (page[k] >= 0 && word[k] == number(round, k) ? 1u : 0u) << k;
    return back;
  };
  const int64_t rounds = (places + kRound - 1) / kRound;
  for (int64_t r = 0; r < rounds; ++r) {
    read(r);
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (page[k] >= 0) atomicSub(t.shares + page[k], 1);
  }
  cluster_sync();
  for (int64_t r = 0; r < rounds; ++r) {
    if (rounds > 1) read(r);
    int32_t word[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) word[k] = page[k] >= 0 ? look(t.shares + page[k]) : 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (word[k] < 0) atomicMin(t.shares + page[k], number(r, k));
  }
  cluster_sync();
  int32_t count = 0;
  for (int64_t r = 0; r < rounds; ++r) {
    if (rounds > 1) read(r);
    count += __popc(going_back(r));
  }
  const Counts sums = count_before(count, 0, warp_sum);
  if (tid == 0) mine = sums.all_a;
  cluster_sync();
  int64_t before, all;
  sum_of_cluster(&mine, &before, &all);
  const int64_t first = taken - all;  // where the pages go, in front of the others
  if (first < 0) flags |= TOPK_DEV_BLOCKS_EXHAUSTED;
  for (int64_t r = 0; r < rounds; ++r) {
    if (rounds > 1) read(r);
    // (a page's word, once cleared here, is no place's number, as it was none of its other places' before)
    const uint32_t back = going_back(r);
    const Counts here = count_before(__popc(back), 0, warp_sum);
    int64_t to = first + before + here.a;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      if (!(back >> k & 1)) continue;
      if (to >= 0) t.free_blocks[to] = page[k];
      t.shares[page[k]] = 0;
      ++to;
    }
    before += here.all_a;
  }
  // the rows hold nothing any more
#pragma unroll 4
  for (int64_t x = tid; x < places; x += kPageThreads) {
    const uint32_t i = static_cast<uint32_t>(x) / columns, c = static_cast<uint32_t>(x) - i * columns;
    const int64_t request = a.requests[i0 + i];
    if (request >= 0 && request < t.num_requests && !(again[i >> 5] >> (i & 31) & 1)) t.block_table[request * t.table_stride + c] = -1;
  }
  if (flags) atomicOr(p.status, flags);
  cluster_sync();  // no CTA leaves before its sums are read; and `taken` has been read by all
  if (cluster_rank() == 0 && tid == 0) *t.taken = static_cast<int32_t>(first > 0 ? first : 0);
}

// ---- compact ----------------------------------------------------------------

enum Mark : int32_t { kNothing = 0, kNamed = 1, kFree = 2, kBoth = 3, kArrived = 4 };  // and ~target for a page that moves

struct CompactParams {
  topk_page_compact_args a;
  uint32_t* status;
};

// Pages of a CTA at a time: four side by side for each thread.
constexpr int kPages = 4 * kPageThreads;

__device__ __forceinline__ void count4(const int4& m, bool (*is)(int32_t), bool (&hit)[4]) {
  hit[0] = is(m.x), hit[1] = is(m.y), hit[2] = is(m.z), hit[3] = is(m.w);
}
__device__ __forceinline__ bool is_free_now(int32_t m) { return m == kFree; }
__device__ __forceinline__ bool is_named(int32_t m) { return (m & kNamed) != 0; }
__device__ __forceinline__ bool is_free_after(int32_t m) { return m == kFree || m < 0; }
__device__ __forceinline__ int32_t ones(const bool (&hit)[4]) { return hit[0] + hit[1] + hit[2] + hit[3]; }

// The counts of all CTAs of the cluster, summed up: first[r] of those before CTA r, first[ctas] of all. Every thread calls it, after
// the cluster has met.
__device__ __forceinline__ void gather_counts(const int32_t* mine, int32_t (&first)[kCluster + 1]) {
  const int tid = threadIdx.x;
  if (tid < 32) {
    const int32_t x = tid < static_cast<int>(cluster_ctas()) ? read_peer(mine, tid) : 0;
    int32_t sum = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t y = __shfl_up_sync(~0u, sum, d);
      if (tid >= d) sum += y;
    }
    if (tid <= kCluster) first[tid] = sum - x;
  }
  __syncthreads();
}

// The CTA that has the i-th of what is counted.
__device__ __forceinline__ int holder(const int32_t (&first)[kCluster + 1], int64_t i) {
  int r = 0;
#pragma unroll
  for (int step = kCluster / 2; step > 0; step >>= 1)
    if (first[r + step] <= i) r += step;
  return r;
}

__global__ void __launch_bounds__(kPageThreads, 1) compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ int2 warp_sum[kPageWarps];
  __shared__ int32_t mine[3], free_first[kCluster + 1], named_first[kCluster + 1], left_first[kCluster + 1];
  const topk_page_compact_args& a = p.a;
  const topk_page_pool& t = a.pool;
  const int tid = threadIdx.x;
  const int64_t rank = cluster_rank(), all_threads = cluster_ctas() * kPageThreads, me = rank * kPageThreads + tid;
  const int64_t padded = (t.num_blocks + 3) / 4 * 4;  // marks are read four at a time; those past the last page are kNothing
  int32_t* mark = static_cast<int32_t*>(a.scratch);
  int32_t *low = mark + padded, *high = low + t.num_blocks;  // each CTA's free and named pages, from its first page's place on
  uint32_t flags = 0;
  dependent_wait();
  dependent_launch();
  const int64_t taken = min(max(static_cast<int64_t>(*t.taken), int64_t{0}), t.num_free);
  const int64_t entries = t.num_requests * t.max_blocks;
  const uint32_t columns = static_cast<uint32_t>(t.max_blocks);
  for (int64_t b = me * 4; b < padded; b += all_threads * 4) *reinterpret_cast<int4*>(mark + b) = make_int4(kNothing, kNothing, kNothing, kNothing);
  cluster_sync();
#pragma unroll 4
  for (int64_t e = me; e < entries; e += all_threads) {
    const uint32_t r = static_cast<uint32_t>(e) / columns, c = static_cast<uint32_t>(e) - r * columns;
    const int32_t page = t.block_table[r * t.table_stride + c];
    if (page >= 0 && page < t.num_blocks) atomicOr(mark + page, static_cast<int32_t>(kNamed));
    if (page >= t.num_blocks) flags |= TOPK_DEV_BAD_BLOCK;
  }
#pragma unroll 4
  for (int64_t f = taken + me; f < t.num_free; f += all_threads) {
    const int32_t page = t.free_blocks[f];
    if (page < 0 || page >= t.num_blocks || (atomicOr(mark + page, static_cast<int32_t>(kFree)) & kFree)) flags |= TOPK_DEV_BAD_BLOCK;
  }
  cluster_sync();
  // this CTA's pages
  const int64_t per = (padded / 4 + cluster_ctas() - 1) / cluster_ctas() * 4, b0 = min(per * rank, padded), b1 = min(b0 + per, padded);
  const auto marks = [&](int64_t x) { return x + tid * 4 < b1 ? look4(mark + x + tid * 4) : make_int4(kNothing, kNothing, kNothing, kNothing); };
  int64_t free_here = b0, named_here = b0;
  for (int64_t x = b0; x < b1; x += kPages) {
    const int4 m = marks(x);
    if (m.x == kBoth || m.y == kBoth || m.z == kBoth || m.w == kBoth) flags |= TOPK_DEV_BAD_BLOCK;
    bool is_free[4], named[4];
    count4(m, is_free_now, is_free);
    count4(m, is_named, named);
    const Counts here = count_before(ones(is_free), ones(named), warp_sum);
    int64_t at_free = free_here + here.a, at_named = named_here + here.b;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int32_t b = static_cast<int32_t>(x + tid * 4 + k);
      if (is_free[k]) low[at_free++] = b;
      if (named[k]) high[at_named++] = b;
    }
    free_here += here.all_a;
    named_here += here.all_b;
  }
  if (tid == 0) {
    mine[0] = static_cast<int32_t>(free_here - b0);
    mine[1] = static_cast<int32_t>(named_here - b0);
  }
  cluster_sync();
  gather_counts(&mine[0], free_first);
  gather_counts(&mine[1], named_first);
  const int64_t free_all = free_first[kCluster], named_all = named_first[kCluster], pairs = min(free_all, named_all);
  // the i-th free page from below, and the i-th named one from above
  const auto free_at = [&](int64_t i) {
    const int r = holder(free_first, i);
    return look(low + min(per * r, padded) + (i - free_first[r]));
  };
  const auto named_at = [&](int64_t i) {
    const int r = holder(named_first, named_all - 1 - i);
    return look(high + min(per * r, padded) + (named_all - 1 - i - named_first[r]));
  };
#pragma unroll 2
  for (int64_t i = me; i < a.max_copies; i += all_threads) {
    const int32_t from = i < pairs ? named_at(i) : -1, to = i < pairs ? free_at(i) : -1;
    const bool moves = to < from;
    const int32_t source = moves ? from : -1, target = moves ? to : -1;
    a.source[i] = source;
    a.target[i] = target;
    if (moves) {
      const int32_t n = t.shares[source];
      mark[source] = ~target;
      mark[target] = kArrived;
      a.shares_out[target] = n;
      a.shares_out[source] = 0;
    }
  }
  cluster_sync();
  // the free pages that each CTA has now, while the table is rewritten
  int32_t count = 0;
  for (int64_t x = b0; x < b1; x += kPages) {
    const int4 m = marks(x);
    bool hit[4];
    count4(m, is_free_after, hit);
    count += ones(hit);
    if (a.shares_out != t.shares) {
      const int32_t word[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t b = x + tid * 4 + k;
        if (b < min(b1, t.num_blocks) && word[k] >= 0 && word[k] != kArrived) a.shares_out[b] = t.shares[b];
      }
    }
  }
  const Counts left = count_before(count, 0, warp_sum);
  if (tid == 0) mine[2] = left.all_a;
  cluster_arrive();
#pragma unroll 4
  for (int64_t e = me; e < entries; e += all_threads) {
    const uint32_t r = static_cast<uint32_t>(e) / columns, c = static_cast<uint32_t>(e) - r * columns;
    int32_t page = t.block_table[r * t.table_stride + c];
    if (page >= 0 && page < t.num_blocks) {
      const int32_t m = look(mark + page);
      if (m < 0) page = ~m;
    }
    a.block_table_out[r * a.table_out_stride + c] = page;
  }
  cluster_wait();
  gather_counts(&mine[2], left_first);
  const int64_t taken_out = t.num_free - left_first[kCluster];  // the list holds every free page once, so there are no more than it has places
  int64_t before = left_first[rank];
  for (int64_t x = b0; x < b1; x += kPages) {
    const int4 m = marks(x);
    bool hit[4];
    count4(m, is_free_after, hit);
    const Counts here = count_before(ones(hit), 0, warp_sum);
    int64_t at = taken_out + before + here.a;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (hit[k]) a.free_blocks_out[at++] = static_cast<int32_t>(x + tid * 4 + k);
    before += here.all_a;
  }
  if (a.free_blocks_out != t.free_blocks)
    for (int64_t f = me; f < taken_out; f += all_threads) a.free_blocks_out[f] = t.free_blocks[f];
  if (flags) atomicOr(p.status, flags);
  cluster_sync();  // no CTA leaves before its sums are read, and `taken` has been read by all
  if (me == 0) *a.taken_out = static_cast<int32_t>(taken_out);
}

// A cluster of `ctas` for this kernel, as a launch without its stream.
template <typename Args>
cudaLaunchConfig_t cluster_config(void (*kernel)(Args), int ctas, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPageThreads);
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent_launch_default() ? 2 : 1;
  return cfg;
}

// CTAs of the cluster: 16 where the device can hold one of those, else 8. Asked for once for each kernel and device.
template <typename Args>
int cluster_size(void (*kernel)(Args), int* known) {
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (device < kMaxDevices && __atomic_load_n(&known[device], __ATOMIC_ACQUIRE) > 0) return known[device];
  int size = 8, clusters = 0;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = cluster_config(kernel, kCluster, attr);
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0)
    size = kCluster;
  cudaGetLastError();
  if (device < kMaxDevices) __atomic_store_n(&known[device], size, __ATOMIC_RELEASE);
  return size;
}

template <typename Args>
int launch_cluster(void (*kernel)(Args), const Args& args, int* known, cudaStream_t stream) {
  const int ctas = cluster_size(kernel, known);
  if (ctas == 0) return TOPK_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = cluster_config(kernel, ctas, attr);
  cfg.stream = stream;
  if (cudaLaunchKernelEx(&cfg, kernel, args) != cudaSuccess) {
    cudaGetLastError();
    return TOPK_ERR_CUDA;
  }
  return TOPK_OK;
}

// ---- copy -------------------------------------------------------------------

constexpr int kCopyThreads = 256;
constexpr int kAtOnce = 4;  // loads of a thread
constexpr int kFewCaches = 16;

struct Cache {
  char* base;
  int64_t block_stride, stride0, stride1;
  int32_t num_blocks, n1;
  uint32_t pieces;      // of a page
  uint32_t run_pieces;  // of a run
  uint32_t first;       // chunk of a pair at which this cache's begin
  int32_t shift;        // a piece is 2^shift bytes
};

template <int kCaches>
struct CopyParams {
  const int32_t *source, *target;
  int64_t num_copies;
  uint32_t* status;
  int32_t num_caches;
  uint32_t chunks;  // of a pair
  Cache cache[kCaches];
};

// One piece of each of kAtOnce places of a page, on which both pages agree; T has the piece's size. Places of pages that are one run
// are told apart from the others once, not piece by piece.
template <typename T, bool kOneRun>
__device__ __forceinline__ void copy_pieces(const Cache& c, const char* from, char* to, uint32_t x0) {
  const auto place = [&](uint32_t x) -> int64_t {
    if (kOneRun) return static_cast<int64_t>(x) * sizeof(T);
    const uint32_t run = x / c.run_pieces, n0 = run / c.n1;
    return n0 * c.stride0 + (run - n0 * c.n1) * c.stride1 + static_cast<int64_t>(x - run * c.run_pieces) * sizeof(T);
  };
  T v[kAtOnce];
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i)
    if (x0 + i * kCopyThreads < c.pieces) v[i] = *reinterpret_cast<const T*>(from + place(x0 + i * kCopyThreads));
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i)
    if (x0 + i * kCopyThreads < c.pieces) *reinterpret_cast<T*>(to + place(x0 + i * kCopyThreads)) = v[i];
}

template <typename T>
__device__ __forceinline__ void copy_chunk(const Cache& c, const char* from, char* to, uint32_t x0) {
  if (c.run_pieces == c.pieces)
    copy_pieces<T, true>(c, from, to, x0);
  else
    copy_pieces<T, false>(c, from, to, x0);
}

template <int kCaches>
__global__ void __launch_bounds__(kCopyThreads, 4) copy_kernel(const __grid_constant__ CopyParams<kCaches> p) {
  dependent_wait();
  dependent_launch();
  uint32_t flags = 0;
  for (int64_t u = blockIdx.x; u < p.num_copies * p.chunks; u += gridDim.x) {
    const int64_t pair = u / p.chunks;
    const uint32_t chunk = static_cast<uint32_t>(u - pair * p.chunks);
    const int32_t source = p.source[pair], target = p.target[pair];
    if (source < 0 || target < 0) continue;
    int k = 0;  // the last cache whose first chunk is at or before this one
    for (int step = kCaches / 2; step > 0; step >>= 1)
      if (k + step < p.num_caches && p.cache[k + step].first <= chunk) k += step;
    const Cache& c = p.cache[k];
    if (source >= c.num_blocks || target >= c.num_blocks) {
      flags |= TOPK_DEV_BAD_BLOCK;
      continue;
    }
    const uint32_t x0 = (chunk - c.first) * (kCopyThreads * kAtOnce) + threadIdx.x;
    const char* from = c.base + source * c.block_stride;
    char* to = c.base + target * c.block_stride;
    switch (c.shift) {
      case 4: copy_chunk<uint4>(c, from, to, x0); break;
      case 3: copy_chunk<uint2>(c, from, to, x0); break;
      case 2: copy_chunk<uint32_t>(c, from, to, x0); break;
      case 1: copy_chunk<uint16_t>(c, from, to, x0); break;
      default: copy_chunk<uint8_t>(c, from, to, x0);
    }
  }
  if (flags && threadIdx.x == 0) atomicOr(p.status, flags);
}

template <int kCaches>
int run_copy(const topk_page_copy_args& a, const Cache* caches, uint32_t chunks, int sms, cudaStream_t stream) {
  CopyParams<kCaches> p{};
  p.source = a.source;
  p.target = a.target;
  p.num_copies = a.num_copies;
  p.status = static_cast<uint32_t*>(a.workspace);
  p.num_caches = a.num_caches;
  p.chunks = chunks;
  for (int i = 0; i < a.num_caches; ++i) p.cache[i] = caches[i];
  const int64_t units = a.num_copies * chunks, most = 8ll * sms;
  return launch(copy_kernel<kCaches>, static_cast<const CopyParams<kCaches>&>(p), units < most ? units : most, kCopyThreads, 0, stream);
}

int check_pool(const topk_page_pool& t) {
  if (t.num_requests < 0 || t.num_requests > INT32_MAX || t.max_blocks < 1 || t.max_blocks > INT32_MAX || t.table_stride < t.max_blocks ||
      t.num_blocks < 0 || t.num_blocks > INT32_MAX || t.num_free < 0 || t.num_free > INT32_MAX || t.num_requests * t.max_blocks > INT32_MAX)
    return TOPK_ERR_INVALID_ARG;
  if (t.taken == nullptr || t.workspace == nullptr || (t.num_requests > 0 && t.block_table == nullptr) || (t.num_blocks > 0 && t.shares == nullptr) ||
      (t.num_free > 0 && t.free_blocks == nullptr))
    return TOPK_ERR_INVALID_ARG;
  if (misaligned(t.block_table, 4) || misaligned(t.shares, 4) || misaligned(t.free_blocks, 4) || misaligned(t.taken, 4) || misaligned(t.workspace, 16))
    return TOPK_ERR_MISALIGNED;
  return TOPK_OK;
}

}  // namespace
}  // namespace paged
}  // namespace ltk

extern "C" int topk_page_fork(const topk_page_fork_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_page_fork_args& a = *args;
  const int rc = check_pool(a.pool);
  if (rc != TOPK_OK) return rc;
  if (a.num_forks < 0 || a.num_forks > INT32_MAX || a.block_size < 1) return TOPK_ERR_INVALID_ARG;
  if (a.num_forks == 0) return TOPK_OK;
  if (a.parents == nullptr || a.children == nullptr || a.kept_lens == nullptr || a.source == nullptr || a.target == nullptr) return TOPK_ERR_INVALID_ARG;
  if (misaligned(a.parents, 4) || misaligned(a.children, 4) || misaligned(a.kept_lens, 4) || misaligned(a.source, 4) || misaligned(a.target, 4))
    return TOPK_ERR_MISALIGNED;
  const int sms = num_sms();
  if (sms < 1) return TOPK_ERR_CUDA;
  ForkParams p{};
  p.a = a;
  topk_paged_rows rows{};
  rows.block_size = a.block_size;
  rows.max_blocks = a.pool.max_blocks;
  p.R = make_rows(rows, INT32_MAX, a.pool.workspace);
  const int64_t grid = a.num_forks < 2ll * sms ? a.num_forks : 2ll * sms;
  return launch(fork_kernel, static_cast<const ForkParams&>(p), grid, kForkThreads, 0, static_cast<cudaStream_t>(stream));
}

extern "C" int topk_page_free(const topk_page_free_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_page_free_args& a = *args;
  const int rc = check_pool(a.pool);
  if (rc != TOPK_OK) return rc;
  if (a.num_freed < 0 || a.num_freed > kMostFreed || a.num_freed * a.pool.max_blocks >= INT32_MAX - 65536) return TOPK_ERR_INVALID_ARG;
  if (a.num_freed == 0) return TOPK_OK;
  if (a.requests == nullptr) return TOPK_ERR_INVALID_ARG;
  if (misaligned(a.requests, 4)) return TOPK_ERR_MISALIGNED;
  FreeParams p{};
  p.a = a;
  p.status = static_cast<uint32_t*>(a.pool.workspace);
  static int known[kMaxDevices];
  return launch_cluster(free_kernel, static_cast<const FreeParams&>(p), known, static_cast<cudaStream_t>(stream));
}

extern "C" int topk_page_compact(const topk_page_compact_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_page_compact_args& a = *args;
  const int rc = check_pool(a.pool);
  if (rc != TOPK_OK) return rc;
  const topk_page_pool& t = a.pool;
  if (a.max_copies < 0 || a.max_copies > INT32_MAX || a.table_out_stride < t.max_blocks) return TOPK_ERR_INVALID_ARG;
  if ((a.max_copies > 0 && (a.source == nullptr || a.target == nullptr)) || (t.num_requests > 0 && a.block_table_out == nullptr) ||
      (t.num_blocks > 0 && (a.shares_out == nullptr || a.scratch == nullptr)) || (t.num_free > 0 && a.free_blocks_out == nullptr) || a.taken_out == nullptr)
    return TOPK_ERR_INVALID_ARG;
  if (misaligned(a.source, 4) || misaligned(a.target, 4) || misaligned(a.block_table_out, 4) || misaligned(a.shares_out, 4) ||
      misaligned(a.free_blocks_out, 4) || misaligned(a.taken_out, 4) || misaligned(a.scratch, 16))
    return TOPK_ERR_MISALIGNED;
  if (a.scratch_bytes < static_cast<size_t>(t.num_blocks) * 3 * sizeof(int32_t) + 16) return TOPK_ERR_WORKSPACE_TOO_SMALL;
  CompactParams p{};
  p.a = a;
  p.status = static_cast<uint32_t*>(t.workspace);
  static int known[kMaxDevices];
  return launch_cluster(compact_kernel, static_cast<const CompactParams&>(p), known, static_cast<cudaStream_t>(stream));
}

extern "C" int topk_page_copy(const topk_page_copy_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_page_copy_args& a = *args;
  if (a.num_copies < 0 || a.num_copies > INT32_MAX || a.num_caches < 0 || a.num_caches > TOPK_MAX_PAGE_CACHES || (a.num_caches > 0 && a.caches == nullptr))
    return TOPK_ERR_INVALID_ARG;
  Cache caches[TOPK_MAX_PAGE_CACHES];
  int64_t chunks = 0;
  for (int i = 0; i < a.num_caches; ++i) {
    const topk_page_cache& c = a.caches[i];
    if (c.num_blocks < 0 || c.num_blocks > INT32_MAX || c.n0 < 1 || c.n1 < 1 || c.run_bytes < 1 || (c.num_blocks > 0 && c.base == nullptr)) return TOPK_ERR_INVALID_ARG;
    const uint64_t all = reinterpret_cast<uint64_t>(c.base) | static_cast<uint64_t>(c.block_stride) | static_cast<uint64_t>(c.run_bytes) |
                         (c.n0 > 1 ? static_cast<uint64_t>(c.stride0) : 0) | (c.n1 > 1 ? static_cast<uint64_t>(c.stride1) : 0);
    int shift = 0;
    while (shift < 4 && !(all >> shift & 1)) ++shift;
    const int64_t run = c.run_bytes >> shift;
    if (run > INT32_MAX || run * c.n0 > INT32_MAX || run * c.n0 * c.n1 > INT32_MAX - kCopyThreads * kAtOnce) return TOPK_ERR_UNSUPPORTED;
    const int64_t pieces = run * c.n0 * c.n1;
    caches[i] = Cache{static_cast<char*>(c.base), c.block_stride, c.stride0, c.stride1, static_cast<int32_t>(c.num_blocks), c.n1,
                      static_cast<uint32_t>(pieces), static_cast<uint32_t>(run), static_cast<uint32_t>(chunks), shift};
    chunks += (pieces + kCopyThreads * kAtOnce - 1) / (kCopyThreads * kAtOnce);
    if (chunks > INT32_MAX) return TOPK_ERR_UNSUPPORTED;
  }
  if (a.num_copies == 0 || a.num_caches == 0) return TOPK_OK;
  if (a.source == nullptr || a.target == nullptr || a.workspace == nullptr) return TOPK_ERR_INVALID_ARG;
  if (misaligned(a.source, 4) || misaligned(a.target, 4) || misaligned(a.workspace, 16)) return TOPK_ERR_MISALIGNED;
  const int sms = num_sms();
  if (sms < 1) return TOPK_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.num_caches <= kFewCaches ? run_copy<kFewCaches>(a, caches, static_cast<uint32_t>(chunks), sms, s)
                                    : run_copy<TOPK_MAX_PAGE_CACHES>(a, caches, static_cast<uint32_t>(chunks), sms, s);
}
