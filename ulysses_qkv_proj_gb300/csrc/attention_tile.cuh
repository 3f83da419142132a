// attention_tile.cuh -- what the attention kernels over the paged cache share: bounded waits, TMA and tensor-memory
// instructions, packed arithmetic, visible tokens as words, and the care for values that a row must not see.
#pragma once

#include "cache.cuh"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace qnre {
namespace attention {

constexpr int kTile = 128;     // cached tokens a tile, rows a unit
constexpr uint64_t kWaitLimitNs = 1000ull * 1000ull * 1000ull;
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;  // log2 of the factor on P, O and the sum alike; a part's "maximum" is less it
constexpr float kRescale = 8.f;  // log2 growth of a row's maximum that O is rescaled at

// Where columns [4 * i, 4 * i + 4) of row r of a part lie, in 16-byte pieces.  The threads that write hold a row each, so
// GROUPED has eight rows side by side, 128 bytes, and a warp's store touches 4 lines instead of 32; with few rows the
// join wants a row's columns together.
template <int D, bool GROUPED>
__device__ __forceinline__ long long part_at(int slot, int r, int i) {
  return GROUPED ? ((static_cast<long long>(slot) * 16 + r / 8) * (D / 4) + i) * 8 + r % 8
                 : (static_cast<long long>(slot) * 128 + r) * (D / 4) + i;
}

// Waits for a phase; false (and the abort word set) after the time limit or an abort elsewhere.
static __device__ __noinline__ bool slow_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t* status) {
  const uint64_t t0 = ptx::global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((i & 31u) == 0) {
      if (*abort_flag) return false;
      if (ptx::global_timer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1u;
        atomicOr(status, QNRE_CACHE_WAIT_TIMEOUT);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t* status) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  return slow_wait(bar, parity, abort_flag, status);
}

__device__ __forceinline__ void pair_sync(int quarter) { asm volatile("bar.sync %0, 64;" ::"r"(2 + quarter) : "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

template <bool BF16>
__device__ __forceinline__ float to_float(uint32_t bits16) {
  if (BF16) return __uint_as_float(bits16 << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(bits16)));
}

// Non-finite halves of a word as a mask of 0xFFFF fields.
template <bool BF16>
__device__ __forceinline__ uint32_t nonfinite_mask(uint32_t w) {
  const uint32_t e = BF16 ? 0x7F80u : 0x7C00u;
  return ((w & e) == e ? 0xFFFFu : 0u) | (((w >> 16) & e) == e ? 0xFFFF0000u : 0u);
}

__device__ __forceinline__ void tmem_fence_regs(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem desc].
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t smem_dst, const void* tmap, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// The same load into every CTA of `mask` at the same place, each one's barrier told of its bytes.
__device__ __forceinline__ void tma_load_4d_multicast(uint32_t smem_dst, const void* tmap, uint32_t bar, int c0, int c1,
                                                      int c2, int c3, uint16_t mask) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.multicast::cluster"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "h"(mask)
      : "memory");
}

// One arrival on the barrier at this place in every CTA of `mask` when this thread's products are done.
__device__ __forceinline__ void umma_commit_multicast(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

// The low word of a shared-memory descriptor moves with the address; the rest is fixed.  (Built
// whole for each instruction, a descriptor cost its one thread more than the instruction.)
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t bytes) { return base + (bytes >> 4); }

// Lets the products issued so far end before the thread leaves its loop early.
__device__ __forceinline__ void drain_mma(uint32_t bar) {
  ptx::umma_commit(bar);
  const uint64_t t0 = ptx::global_timer_ns();
  while (!ptx::mbar_try_wait(bar, 0) && ptx::global_timer_ns() - t0 < kWaitLimitNs) {
  }
}

// Packed pairs of floats (one instruction for two).
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bits of the 32 tokens from d0 on (relative to the row's length) that a row sees: the context, then `bits`.
__device__ __forceinline__ uint32_t seen_word(int d0, uint64_t bits) {
  if (d0 <= -32) return 0xFFFFFFFFu;
  if (d0 < 0) return (1u << -d0) - 1u | static_cast<uint32_t>(bits << -d0);
  return d0 < 64 ? static_cast<uint32_t>(bits >> d0) : 0u;
}

// x + the non-finite elements in column c of V over the drafts in `seen` (all below slot `last`).
template <bool BF16>
__device__ __noinline__ float add_nonfinite(const CacheView& cache, int layer, int row, int kvh, int len, int first, int last,
                                            uint64_t seen, int c, float x) {
  for (; seen != 0; seen &= seen - 1) {
    const int pos = len + __ffsll(static_cast<long long>(seen)) - 1;
    if (pos < first || pos >= last) continue;
    const int page = cache.page_of(row, pos);
    if (page < 0) continue;
    const uint16_t w = *reinterpret_cast<const uint16_t*>(cache.v + cache.token_offset(layer, page, kvh, pos) + c * 2);
    if (nonfinite_mask<BF16>(w) & 0xFFFFu) x += to_float<BF16>(w);
  }
  return x;
}

// Which of the 32 channels from `c` on hold +inf, -inf or NaN in V of the tokens [first, last) (a whole warp).
struct Kinds {
  uint32_t plus, minus, nan;
};
template <bool BF16>
__device__ __noinline__ Kinds search_context(const CacheView& cache, int layer, int row, int kvh, int first, int last, int c) {
  Kinds k{0, 0, 0};
  for (int pos = first + static_cast<int>(threadIdx.x % 32); pos < last; pos += 32) {
    const int page = cache.page_of(row, pos);
    if (page < 0) continue;
    const uint4* at = reinterpret_cast<const uint4*>(cache.v + cache.token_offset(layer, page, kvh, pos) + c * 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 w = at[i];
      const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t x = words[e / 2] >> (e % 2 * 16) & 0xFFFFu;
        if (nonfinite_mask<BF16>(x) & 0xFFFFu) {
          const float f = to_float<BF16>(x);
          const uint32_t bit = 1u << (8 * i + e);
          k.plus |= f > 0.f ? bit : 0u;
          k.minus |= f < 0.f ? bit : 0u;
          k.nan |= f != f ? bit : 0u;
        }
      }
    }
  }
  __syncwarp();
  return Kinds{__reduce_or_sync(0xFFFFFFFFu, k.plus), __reduce_or_sync(0xFFFFFFFFu, k.minus),
               __reduce_or_sync(0xFFFFFFFFu, k.nan)};
}

// Pieces [first, last) of a V row of a tile past the context: slots without a token are zeroed; in drafted ones the non-finite
// elements are, and true is returned.
template <int D, bool BF16>
__device__ __noinline__ bool clean_v_row(char* row, bool token, int first, int last) {
  bool found = false;
#pragma unroll 4
  for (int i = first; i < last; ++i) {
    // each lane its own order of the row's pieces: rows are 128 bytes apart, so equal pieces share banks
    uint4* at = reinterpret_cast<uint4*>(row + (i / 8) * (kTile * 128) + ((i ^ threadIdx.x) % 8) * 16);
    if (!token) {
      *at = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4 w = *at;
    const uint4 z = make_uint4(nonfinite_mask<BF16>(w.x), nonfinite_mask<BF16>(w.y), nonfinite_mask<BF16>(w.z),
                               nonfinite_mask<BF16>(w.w));
    if (z.x | z.y | z.z | z.w) {
      found = true;
      *at = make_uint4(w.x & ~z.x, w.y & ~z.y, w.z & ~z.z, w.w & ~z.w);
    }
  }
  ptx::fence_proxy_async_smem();
  return found;
}

// 2^x for the join of parts, x <= 0: never 0, so that a part with an infinite sum stays one under a far larger maximum.
__device__ __forceinline__ float part_weight(float x) { return fmaxf(exp2_fast(x), 1.4e-45f); }

// Memory of device `dev` itself: K and V of more than one row tile come by cluster multicast, which is for a GPU's own
// memory alone, so pools of another device or of the host are refused, whatever the number of nodes.
inline bool own_memory(const void* p, int dev) {
  cudaPointerAttributes at{};
  return cudaPointerGetAttributes(&at, p) == cudaSuccess && at.type == cudaMemoryTypeDevice && at.device == dev;
}

}  // namespace attention
}  // namespace qnre
