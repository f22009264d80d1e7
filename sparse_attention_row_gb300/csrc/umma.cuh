// The instructions that the tensor-core kernels of the paged calls use:
// mbarriers, asynchronous copies into shared memory, tcgen05 products with
// their operands in shared memory and their sums in tensor memory.
//
// Operand tiles are stored as the 128-byte swizzle wants them: rows of 128
// bytes, in groups of eight rows (1024 bytes, aligned to that), the 16-byte
// piece c of row r at place c ^ (r & 7). Such a tile serves as a K-major operand
// (its rows run along M or N, its bytes along K) and as an MN-major one (its rows
// run along K): the same keys are the A operand of K Q^T and, read the other
// way, of V^T P^T.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "libtopk.h"

namespace ltk {
namespace umma {

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// The same, suspended for up to 20 us where the phase is not over yet.
__device__ __forceinline__ bool mbar_try_long(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return done != 0;
}

// A CTA's waits. One that runs out sets the flag, after which every wait of the CTA returns at once: the
// loops run to their end without waiting, over memory that stays in bounds, and the launch's status says
// that its results are void.
struct Guard {
  volatile uint32_t* gave_up;  // shared memory
  uint32_t* status;
};

constexpr uint64_t kWaitLimitNs = 1000ull * 1000ull * 1000ull;

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

static __device__ __noinline__ void mbar_wait_slow(uint32_t bar, uint32_t parity, volatile uint32_t* gave_up, uint32_t* status) {
  const uint64_t t0 = now_ns();
  while (!mbar_try_long(bar, parity)) {
    if (*gave_up) return;
    if (now_ns() - t0 > kWaitLimitNs) {
      *gave_up = 1;
      atomicOr(status, TOPK_DEV_PIPELINE_TIMEOUT);
      return;
    }
  }
}

__device__ __forceinline__ void mbar_wait(uint32_t bar, uint32_t parity, const Guard& g) {
  if (!mbar_try(bar, parity)) mbar_wait_slow(bar, parity, g.gave_up, g.status);
}

// Before a CTA that gave up ends: its copies and products in flight, of which no one waits for the end any more,
// take microseconds; 2 ms are waited.
__device__ __forceinline__ void settle(const Guard& g) {
  if (!*g.gave_up) return;
  const uint64_t t0 = now_ns();
  while (now_ns() - t0 < 2000000) __nanosleep(1000);
}

// mbar_wait for a whole warp, which goes on in step.
__device__ __forceinline__ void mbar_wait_warp(uint32_t bar, uint32_t parity, const Guard& g) {
  mbar_wait(bar, parity, g);
  __syncwarp();
}

// 16 bytes into shared memory; `bytes` 0 writes zeros and reads nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// One arrival on `bar` when every copy that this thread has begun has landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void copies_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Orders this thread's (and, after a barrier, others') writes to shared memory before the tensor cores' reads.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Instructions marked .aligned, and bar.sync, which is, want their whole warp in step. Branches and waits before them can
// leave its lanes apart (each lane leaves mbar_wait() by itself), so each such function brings them together first; what
// follows within it is straight-line code.
__device__ __forceinline__ void named_sync(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Whether `x` holds for any of the threads that meet at the barrier.
__device__ __forceinline__ bool named_any(int id, int threads, bool x) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n barrier.cta.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(x))
      : "memory");
  return any != 0;
}

// ---- tensor memory --------------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t where, uint32_t columns) {  // a whole warp
  __syncwarp();
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns) {  // the same warp
  __syncwarp();
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void store_wait() {
  __syncwarp();
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Columns [addr, addr + N) of this warp's 32 lanes; a thread gets its lane's, when they have come.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[N]) {
  static_assert(N == 8 || N == 16 || N == 32);
  __syncwarp();
  if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(addr));
  if constexpr (N == 16)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
                   "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(addr));
  if constexpr (N == 32)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));  // used from here on, not before
}

__device__ __forceinline__ void tmem_store8(uint32_t addr, const float* v) {
  __syncwarp();
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// ---- products -------------------------------------------------------------

// Descriptor of an operand tile, 128-byte swizzle, groups of eight rows 1024 bytes apart: its low word, from the
// tile's shared-memory address (16-byte aligned). `leading` matters to MN-major operands of more than 64 elements
// only: bytes from one 128-byte column of the tile to the next. The high word is the same for all.
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t leading) { return (addr >> 4) | (leading >> 4 << 16); }
constexpr uint32_t kOperandHigh = (1024u >> 4) | (1u << 14) | (2u << 29);

enum Format : uint32_t { kF16 = 0, kBF16 = 1, kE4M3 = 0 };

// Instruction descriptor: fp32 sums, M = 128, N columns, both operands of one format; `mn_major`: both are MN-major.
__host__ __device__ constexpr uint32_t instruction(uint32_t format, uint32_t n, bool mn_major) {
  return (1u << 4) | (format << 7) | (format << 10) | (mn_major ? (1u << 15) | (1u << 16) : 0u) | ((n >> 3) << 17) |
         ((128u >> 4) << 24);
}

// The same value in every lane, and known to be: it can live in a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(~0u, x, 0); }

// Products, by a whole warp in step, of which one thread issues: D (tensor memory) = A B, or D += A B where `add`
// (or a later step of the same call). Every lane of the warp runs the code around them, so that addresses stay in
// uniform registers, which the instruction wants: one thread alone, with a register moved over for every operand, takes
// about 120 cycles an instruction (N = 16 and N = 64 alike) where the tensor core takes 36 to 48.
// 32 bytes of both K-major operands: 16 elements of two bytes.
__device__ __forceinline__ void mma16_step(uint32_t d, uint32_t a, uint32_t b, uint32_t inst, bool add) {
  d = uniform(d), a = uniform(a), b = uniform(b);
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b32 x, y;\n .reg .b64 a, b;\n"
      " setp.ne.u32 p, %5, 0;\n setp.eq.u32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n"
      " add.u32 x, %1, 0; add.u32 y, %2, 0; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n"
      "}" ::"r"(d), "r"(a), "r"(b), "r"(kOperandHigh), "r"(inst), "r"(static_cast<uint32_t>(add))
      : "memory");
}

// 128 bytes of both: four such steps.
__device__ __forceinline__ void mma16_chunk(uint32_t d, uint32_t a, uint32_t b, uint32_t inst, bool add) {
  d = uniform(d), a = uniform(a), b = uniform(b);
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b32 x, y;\n .reg .b64 a, b;\n"
      " setp.ne.u32 p, %5, 0;\n setp.eq.u32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n"
      " add.u32 x, %1, 0; add.u32 y, %2, 0; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n"
      " add.u32 x, %1, 2; add.u32 y, %2, 2; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %1, 4; add.u32 y, %2, 4; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %1, 6; add.u32 y, %2, 6; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      "}" ::"r"(d), "r"(a), "r"(b), "r"(kOperandHigh), "r"(inst), "r"(static_cast<uint32_t>(add))
      : "memory");
}

// 256 bytes of both, in two chunks, the second ones `a_next` and `b_next` (in 16 bytes) behind the first.
__device__ __forceinline__ void mma16_pair(uint32_t d, uint32_t a, uint32_t a_next, uint32_t b, uint32_t b_next, uint32_t inst, bool add) {
  d = uniform(d), a = uniform(a), b = uniform(b);
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b32 x, y;\n .reg .b64 a, b;\n"
      " setp.ne.u32 p, %5, 0;\n setp.eq.u32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n"
      " add.u32 x, %1, 0; add.u32 y, %2, 0; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n"
      " add.u32 x, %1, 2; add.u32 y, %2, 2; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %1, 4; add.u32 y, %2, 4; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %1, 6; add.u32 y, %2, 6; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %6, 0; add.u32 y, %7, 0; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %6, 2; add.u32 y, %7, 2; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %6, 4; add.u32 y, %7, 4; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %6, 6; add.u32 y, %7, 6; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      "}" ::"r"(d), "r"(a), "r"(b), "r"(kOperandHigh), "r"(inst), "r"(static_cast<uint32_t>(add)), "r"(a + a_next), "r"(b + b_next)
      : "memory");
}

// MN-major operands, 128 rows: eight steps of 16 rows.
__device__ __forceinline__ void mma16_tokens(uint32_t d, uint32_t a, uint32_t b, uint32_t inst, bool add) {
  d = uniform(d), a = uniform(a), b = uniform(b);
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b32 x, y;\n .reg .b64 a, b;\n"
      " setp.ne.u32 p, %5, 0;\n setp.eq.u32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n"
      " add.u32 x, %1, 0; add.u32 y, %2, 0; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n"
      " add.u32 x, %1, 128; add.u32 y, %2, 128; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %1, 256; add.u32 y, %2, 256; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %1, 384; add.u32 y, %2, 384; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %1, 512; add.u32 y, %2, 512; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %1, 640; add.u32 y, %2, 640; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %1, 768; add.u32 y, %2, 768; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      " add.u32 x, %1, 896; add.u32 y, %2, 896; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      "}" ::"r"(d), "r"(a), "r"(b), "r"(kOperandHigh), "r"(inst), "r"(static_cast<uint32_t>(add))
      : "memory");
}

// 32 bytes of both K-major operands: 32 elements of one byte.
__device__ __forceinline__ void mma8_step(uint32_t d, uint32_t a, uint32_t b, uint32_t inst, bool add) {
  d = uniform(d), a = uniform(a), b = uniform(b);
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b32 x, y;\n .reg .b64 a, b;\n"
      " setp.ne.u32 p, %5, 0;\n setp.eq.u32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n"
      " add.u32 x, %1, 0; add.u32 y, %2, 0; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n"
      "}" ::"r"(d), "r"(a), "r"(b), "r"(kOperandHigh), "r"(inst), "r"(static_cast<uint32_t>(add))
      : "memory");
}

// 128 bytes of both.
__device__ __forceinline__ void mma8_chunk(uint32_t d, uint32_t a, uint32_t b, uint32_t inst, bool add) {
  d = uniform(d), a = uniform(a), b = uniform(b);
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b32 x, y;\n .reg .b64 a, b;\n"
      " setp.ne.u32 p, %5, 0;\n setp.eq.u32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n"
      " add.u32 x, %1, 0; add.u32 y, %2, 0; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n"
      " add.u32 x, %1, 2; add.u32 y, %2, 2; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, t;\n"
      " add.u32 x, %1, 4; add.u32 y, %2, 4; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, t;\n"
      " add.u32 x, %1, 6; add.u32 y, %2, 6; mov.b64 a, {x, %3}; mov.b64 b, {y, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, t;\n"
      "}" ::"r"(d), "r"(a), "r"(b), "r"(kOperandHigh), "r"(inst), "r"(static_cast<uint32_t>(add))
      : "memory");
}

// One arrival on `bar` when every product that this warp has issued is done.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar)
      : "memory");
}

}  // namespace umma
}  // namespace ltk
