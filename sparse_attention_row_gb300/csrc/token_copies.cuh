// Copies of a tile's tokens from a paged cache into shared memory, in 16-byte
// cp.async: any page size, stride and order of tokens, and zeros for a token that
// is masked, whatever the cache holds there.
//
// Measured beside TMA (rows by number four at a time, or runs of a page): a warp's TMA
// instruction takes some 70 cycles to issue for 512 bytes and 180 for 8 KB, one CTA's
// four copying warps bring 26 to 45 bytes a cycle; cp.async brings 72 (both from L2, all
// SMs at once), 44 beside the tensor cores' own reads of shared memory.
#pragma once

#include "umma.cuh"

namespace ltk {
namespace paged {

// A copying warp's 32 tokens of a tile: eight lanes to each 128 bytes, four tokens an instruction.
struct TokenCopies {
  static constexpr int kEach = 8, kColumns = 2;
  const char* from[kEach];
  uint32_t seen;   // bit i: from[i] is to be read
  uint32_t to[2];  // place in the tile of the even and odd instructions, whose tokens differ by four
  int byte;        // of a 128-byte row
  bool all;        // every one of the warp's tokens is to be read
  __device__ TokenCopies(int first_token, int lane) : seen(0), all(false) {
    const int token = first_token + (lane >> 3), col = lane & 7;
    byte = col * 16;
    to[0] = token * 128 + ((col ^ (token & 7)) << 4);
    to[1] = (token + 4) * 128 + ((col ^ ((token + 4) & 7)) << 4);
  }
  // Each lane brings the address of a token, lane by lane in the order of the tile.
  __device__ __forceinline__ void aim(const char* mine, bool on, int lane) {
    const unsigned who = __ballot_sync(~0u, on);
    all = who == ~0u;
    seen = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int lane_from = i * 4 + (lane >> 3);
      from[i] = reinterpret_cast<const char*>(__shfl_sync(~0u, reinterpret_cast<uint64_t>(mine), lane_from)) + byte;
      seen |= ((who >> lane_from) & 1) << i;
    }
  }
  // Up to 256 bytes of each token from `first` on, a token having `bytes` in all: 128-byte columns (swizzled
  // tiles, `column` bytes apart), the last one filled up with zeros.
  __device__ __forceinline__ void columns(uint32_t dst, uint32_t column, int first, int bytes, const void* anywhere) const {
    if (all && first + kColumns * 128 <= bytes) {  // nearly always: no selections, a third of the instructions
      const uint32_t even = dst + to[0], odd = dst + to[1];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const char* at = from[i] + first;
#pragma unroll
        for (int c = 0; c < kColumns; ++c) umma::copy16((i & 1 ? odd : even) + c * column + (i >> 1) * 1024, at + c * 128, 16);
      }
      return;
    }
#pragma unroll 1
    for (int c = 0; c < kColumns; ++c) {
      if (first + c * 128 >= bytes) break;
      const bool in = first + c * 128 + byte < bytes;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const bool on = in && ((seen >> i) & 1);
        umma::copy16(dst + c * column + to[i & 1] + (i >> 1) * 1024, on ? from[i] + (first + c * 128) : anywhere, on ? 16 : 0);
      }
    }
  }
};

}  // namespace paged
}  // namespace ltk
