// What the attention kernels share: the deal of tiles to slices, parts of units and their join, probabilities.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace ltk {
namespace paged {

struct Join {  // what a join has to know of the unit that ends in a slice and began before it
  int64_t rowgroup;
  int32_t kv_head;
  int32_t first, last;  // slices
  int32_t first_slot;   // which of its two places the first slice used
  int64_t tiles;        // of all units
};

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
// The group of tile x where every group has `per` of them: lists of blocks may be so long that 32 bits do not hold `per`, and its lower
// ones are zero.
__host__ __device__ __forceinline__ int64_t group_of(int64_t x, int64_t per) {
  if (x < per) return 0;
  return x < kSmallTiles ? static_cast<uint32_t>(x) / static_cast<uint32_t>(per) : x / per;
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

// What a prefix and the tokens behind it weigh in the whole: from the logarithms of their sums, the prefix's in powers of
// two, the other's a natural one.
struct Weights {
  float prefix, tail, lse;
};
__device__ __forceinline__ Weights weigh(float prefix2, float tail_lse) {
  const float tail2 = tail_lse * 1.4426950408889634f, top = fmaxf(prefix2, tail2), b = top == -INFINITY ? 0.f : top;
  const float x = exp2f(prefix2 - b), y = exp2f(tail2 - b), sum = x + y, r = sum == 0.f ? 0.f : 1.f / sum;
  return {x * r, y * r, sum == 0.f ? -INFINITY : (b + log2f(sum)) * 0.69314718055994531f};
}

// Two values of a row and `weight` times those behind the prefix, which stand at `at`.
template <bool kBf16>
__device__ __forceinline__ uint32_t add_tail(float lo, float hi, const uint16_t* at, float weight) {
  const uint32_t bits = *reinterpret_cast<const uint32_t*>(at);
  float2 t;
  if constexpr (kBf16)
    t = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(bits));
  else
    t = __half22float2(reinterpret_cast<const __half2&>(bits));
  return pack2<kBf16>(lo + weight * t.x, hi + weight * t.y);
}

// A load that stays where it is written: left to the compiler, the join's loads move to their uses, one latency each
// (4 parts of eight loads a thread: 17 000 cycles against 4300).
__device__ __forceinline__ float4 load_now(const float4* at) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(at) : "memory");
  return v;
}

}  // namespace paged
}  // namespace ltk
