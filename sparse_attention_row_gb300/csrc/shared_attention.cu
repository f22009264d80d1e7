// topk_shared_attention: attention over everything cached, for requests of which some begin with the same pages.
//
//   softmax over a row's tokens, split in two:  out = w_p out_p + w_t out_t,  w = exp(lse - log(exp(lse_p) + exp(lse_t)))
//
// for the prefix's tokens p and those behind it, t. Three steps, in order on the stream:
//   plan    which rows share what, from the rows' lengths and requests, on the device: a run is as many neighbouring rows
//           with the same prefix as fill a unit's columns, and every row gets its length behind the prefix.
//   tails   attention over what is behind the prefixes, each request by itself (kTail): bound by HBM. Its results stand in
//           `out` and `lse`. It reports requests whose prefix is none.
//   prefix  attention over the prefixes, a run of rows at a time, which joins its results with those of the tails as it writes
//           them: wide_prefix.cu, 256 columns a run, or kShared of the kernel of all forms, 64.
// Small calls take none of them, but one launch in which every row finds the prefix's pages in their table (kWhole).
#include <cfloat>

#include "attention_forms.cuh"
#include "paged.cuh"

namespace ltk {
namespace paged {
namespace {

constexpr int kMostThreads = 1024;

struct PlanParams {
  Rows R;
  Prefixes prefixes;
  int32_t run_rows;     // of a run at most
  int32_t* tail_lengths;
  int32_t* skip;
  SharedRun* runs;
  int32_t* run_count;
};

// One CTA: up to 1024 rows at a time, a thread each, with the start of the run that the last segment ended in.
__global__ void __launch_bounds__(kMostThreads) plan_kernel(const PlanParams p) {
  __shared__ int64_t key[kMostThreads + 2];  // prefix and tokens of each row of the segment, and of its neighbours
  __shared__ int32_t warp_start[kMostThreads / 32], warp_ends[kMostThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads / 32;
  dependent_wait();
  dependent_launch();
  const auto key_of = [&](int64_t row) -> int64_t {
    int32_t prefix = -1;
    const int n = row_prefix_tokens(p.prefixes, p.R, row, &prefix);
    return n == 0 ? -1 : static_cast<int64_t>(prefix) << 32 | n;
  };
  uint32_t bits = 0;
  int64_t start = 0;  // of the run so far
  int32_t count = 0;  // runs listed
  for (int64_t row0 = 0; row0 < p.R.num_rows; row0 += threads) {
    const int64_t row = row0 + tid;
    const bool real = row < p.R.num_rows;
    const int64_t mine = key_of(row);
    key[tid + 1] = mine;
    // the neighbours' keys, by a warp each, as every key is found
    if (warp == 0) {
      const int64_t k = key_of(row0 - 1);
      if (lane == 0) key[0] = k;
    }
    if (warp == warps - 1) {
      const int64_t k = key_of(row0 + threads);
      if (lane == 0) key[threads + 1] = k;
    }
    if (real) {
      const int64_t request = row_request(p.R, row);
      const int32_t n = p.R.lengths[row];
      if (request >= p.R.num_requests) bits |= TOPK_DEV_BAD_BLOCK;
      if (request >= 0 && request < p.R.num_requests && (n < 0 || n > p.R.max_len)) bits |= TOPK_DEV_LENGTH_CLAMPED;
      const int shared = mine < 0 ? 0 : static_cast<int32_t>(mine);
      p.tail_lengths[row] = seen_tokens(p.R, n, request) - shared;
      p.skip[row] = block_column(p.R, shared);
    }
    __syncthreads();
    // the start of each row's run: the last row at or before it whose key is another than the row's before
    int32_t from = real && key[tid] != mine ? tid : -1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t x = __shfl_up_sync(~0u, from, d);
      if (lane >= d) from = max(from, x);
    }
    if (lane == 31) warp_start[warp] = from;
    __syncthreads();
    int32_t before = -1;
    for (int w = 0; w < warp; ++w) before = max(before, warp_start[w]);
    from = max(from, before);
    const int64_t run_start = from >= 0 ? row0 + from : start;
    const int64_t at = row - run_start;
    const bool ends = real && mine >= 0 && (key[tid + 2] != mine || at % p.run_rows == p.run_rows - 1);
    const unsigned who = __ballot_sync(~0u, ends);
    if (lane == 0) warp_ends[warp] = __popc(who);
    __syncthreads();
    int32_t place = count + __popc(who & ((1u << lane) - 1)), total = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) place += warp_ends[w];
      total += warp_ends[w];
    }
    if (ends) {
      const int rows = static_cast<int>(at % p.run_rows) + 1;
      p.runs[place] = SharedRun{static_cast<int32_t>(row - rows + 1), rows, static_cast<int32_t>(mine >> 32), static_cast<int32_t>(mine)};
    }
    count += total;
    int32_t last = -1;
    for (int w = 0; w < warps; ++w) last = max(last, warp_start[w]);
    if (last >= 0) start = row0 + last;
    __syncthreads();  // the next segment writes the sums again
  }
  if (tid == 0) *p.run_count = count;
  if (bits) atomicOr(p.R.status, bits);
}

// Bytes that all rows together read up to which each reads the prefix for itself, out of L2. (In us alone against shared. 32 heads over
// 8: 134 MB 25 to 28 against 31 to 34, 268 MB 38 to 44 against 34 to 44, 537 MB 62 to 77 against 36 to 52. 16 heads over 2, wide units: 134 MB
// 26 against 33, 268 MB 38 against 35 to 40; units of up to 64 columns, of which there are two, 268 MB 38 against 45. 16 latent heads: 151 MB 29 to
// 35 against 55 to 61; 302 MB 46 to 50 against 61 to 69; 604 MB 74 to 77 against 70 to 81. 128 latent heads fill the columns by themselves: 604 MB
// 194 against 221. All of one prefix for all rows, and with a table as wide as the prefix: a wider one is taken for a longer prefix.)
double read_alone(const topk_attention_args& a) {
  if (takes_wide(a)) return 256e6;
  if (a.heads / a.kv_heads >= kSharedCols) return DBL_MAX;
  const int pack = rows_of_run(a);
  const int64_t units = (a.rows.num_rows + pack - 1) / pack * a.kv_heads;
  return a.v != nullptr && units >= 8 ? 256e6 : 512e6;
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

// Scratch: the number of runs, the runs, rows' lengths behind the prefix and their first columns, the tails' statistics or the
// parts of the wide kernel.
struct Scratch {
  size_t runs, lengths, skip, tail_lse, end;
  Scratch(int sms, int64_t rows) {
    runs = 256;
    lengths = runs + round_up(sizeof(SharedRun) * rows);
    skip = lengths + round_up(sizeof(int32_t) * rows);
    tail_lse = skip + round_up(sizeof(int32_t) * rows);
    const size_t few = static_cast<size_t>(sms > 16 ? sms : 16) * 2 * kSharedCols * sizeof(float), many = wide_scratch(sms);
    end = tail_lse + (few > many ? few : many);
  }
};

}  // namespace
}  // namespace paged
}  // namespace ltk

extern "C" size_t topk_shared_attention_scratch_size(int device, int64_t num_rows) {
  topk_device_props p{};
  if (topk_query_device(device, &p) != TOPK_OK) return 0;
  return ltk::paged::Scratch(p.num_sms, num_rows < 0 ? 0 : num_rows).end;
}

extern "C" int topk_shared_attention(const topk_shared_attention_args* args, void* stream) {
  using namespace ltk::paged;
  if (args == nullptr) return TOPK_ERR_INVALID_ARG;
  const topk_shared_attention_args& s = *args;
  const topk_attention_args& a = s.attention;
  if (a.indices != nullptr || s.num_prefixes < 0 || s.num_prefixes > INT32_MAX || s.prefix_blocks < 1 || s.prefix_blocks > INT32_MAX ||
      s.prefix_stride < s.prefix_blocks)
    return TOPK_ERR_INVALID_ARG;
  int rc = check_attention(a);
  if (rc != TOPK_OK || a.rows.num_rows == 0) return rc;
  if (a.lse == nullptr || s.prefix_of == nullptr || s.scratch == nullptr || (s.num_prefixes > 0 && (s.prefix_lens == nullptr || s.prefix_table == nullptr)))
    return TOPK_ERR_INVALID_ARG;
  if (misaligned(s.prefix_of, 4) || misaligned(s.prefix_lens, 4) || misaligned(s.prefix_table, 4) || misaligned(s.scratch, 16)) return TOPK_ERR_MISALIGNED;
  int device = 0;
  topk_device_props props{};
  if (cudaGetDevice(&device) != cudaSuccess || topk_query_device(device, &props) != TOPK_OK) {
    cudaGetLastError();
    return TOPK_ERR_CUDA;
  }
  const Scratch at(props.num_sms, a.rows.num_rows);
  if (s.scratch_bytes < at.end || a.workspace_bytes < topk_attention_workspace_size(device)) return TOPK_ERR_WORKSPACE_TOO_SMALL;
  char* scratch = static_cast<char*>(s.scratch);
  const int64_t held = s.prefix_blocks > INT32_MAX / a.rows.block_size ? INT32_MAX : s.prefix_blocks * a.rows.block_size;

  FormArgs f{};
  f.prefixes = Prefixes{s.prefix_of, s.prefix_lens, s.prefix_table, s.num_prefixes, s.prefix_stride, held};
  // Of the prefixes' lengths the host knows what their table can hold.
  const double bytes = 2.0 * a.rows.num_rows * held * a.kv_heads * (a.dk + (a.v != nullptr ? a.dv : 0));
  if (bytes <= read_alone(a)) return attend_whole(a, f, stream);

  PlanParams p{};
  p.R = make_rows(a.rows, INT32_MAX, a.workspace);
  p.prefixes = f.prefixes;
  p.run_rows = rows_of_run(a);
  p.tail_lengths = reinterpret_cast<int32_t*>(scratch + at.lengths);
  p.skip = reinterpret_cast<int32_t*>(scratch + at.skip);
  p.runs = reinterpret_cast<SharedRun*>(scratch + at.runs);
  p.run_count = reinterpret_cast<int32_t*>(scratch);
  const int threads = a.rows.num_rows < kMostThreads ? static_cast<int>((a.rows.num_rows + 31) / 32 * 32) : kMostThreads;
  rc = launch(plan_kernel, p, 1, threads, 0, static_cast<cudaStream_t>(stream));
  if (rc != TOPK_OK) return rc;

  f.skip = p.skip;
  topk_attention_args tail = a;
  tail.rows.lengths = p.tail_lengths;
  rc = attend_tail(tail, f, stream);
  if (rc != TOPK_OK || s.num_prefixes == 0) return rc;
  f.runs = p.runs;
  f.run_count = p.run_count;
  f.tail_lse = reinterpret_cast<float*>(scratch + at.tail_lse);
  return takes_wide(a) ? attend_wide(tail, f, f.tail_lse, stream) : attend_shared(tail, f, stream);
}
