// seq_tile.cuh -- pieces that the tensor-core kernels of the token-sequence
// operators share: TMA loads of 128-row tiles from strided tensors, visibility
// masks of a row over 128 keys, descriptors by element type, and the clearing
// of tile rows that no row of a block may see.
#pragma once
#include <cuda.h>

#include "sm100_ptx.cuh"
#include "sta_common.cuh"
#include "seq_common.cuh"

namespace sta {

constexpr int kTileRows = 128;
constexpr uint32_t kTilePanel = kTileRows * 128;  // 128 rows x 64 elements, 128-byte swizzle

// Instruction descriptor of tcgen05.mma kind::f16 for operands of type T (the
// format fields are 1 for bf16 and 0 for f16), fp32 accumulator.
template <class T>
__host__ __device__ constexpr uint32_t idesc_for(int M, int N, bool a_mn_major, bool b_mn_major) {
  const uint32_t both_bf16 = (1u << 7) | (1u << 10);
  const uint32_t d = idesc_bf16_f32(M, N, a_mn_major, b_mn_major);
  return std::is_same<T, __half>::value ? d & ~both_bf16 : d;
}

// Rows [row, row + 128) of head `head` of batch entry `slice`, all D columns,
// as D / 64 panels.  Rows past the tensor's end arrive as zero.
template <int D>
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *map, int row, int head, int slice,
                                          uint64_t *bar) {
  if constexpr (D == 128) tma_load_5d(dst, map, 0, row, head, slice, 0, bar);
  else tma_load_4d(dst, map, 0, row, head, slice, bar);
}

__device__ __forceinline__ void fence_proxy_async_cta() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Zero rows [from, to) of a D / 64 panel tile, by one warp, before tensor-core
// reads of them.
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t *tile, int from, int to, int lane) {
  const int n = (to - from) * 8;  // 16-byte pieces of a panel
  for (int i = lane; i < n; i += 32)
#pragma unroll
    for (int pn = 0; pn < D / 64; ++pn)
      *reinterpret_cast<uint4 *>(tile + pn * kTilePanel + (from + (i >> 3)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_cta();
  __syncwarp();
}

// Bits [0, n) of a word, for any n.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Bit i: the query at `pos` sees key base + 32 w + i, of the first `valid`
// keys from base on.
__device__ __forceinline__ uint32_t visible_bits(int pos, int base, int valid, int window, int sinks, int w) {
  const int hi = min(valid - 1, pos - base) + 1 - 32 * w;  // keys below
  const int lo = pos - window + 1 - base - 32 * w, sk = sinks - base - 32 * w;
  return bits_below(hi) & (~bits_below(lo) | bits_below(sk));
}

}  // namespace sta
