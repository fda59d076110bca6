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

// ------------------------------------------------------- work items on demand
// Each kernel below is launched with one CTA per work item, but a running CTA
// takes over items whose CTAs have not started yet (cluster launch control), so
// items of uneven cost spread over the SMs while the pipelines of one CTA run
// from item to item without a restart.  The producer thread asks for the next
// item when it starts one, and leaves what the other roles need of an item in
// a ring of two, ahead of them.  Item::stop marks the end.
template <class Item>
struct ItemRing {
  Item *items;              // [2]
  uint64_t *full, *empty;   // [2] each; empty: one arrival per consumer warp
  uint4 *answer;
  uint64_t *answered;
  static constexpr uint32_t kBytes = 16 + 5 * 8 + 2 * sizeof(Item) + 15;

  __device__ __forceinline__ explicit ItemRing(void *smem) {
    answer = reinterpret_cast<uint4 *>((reinterpret_cast<uintptr_t>(smem) + 15) & ~uintptr_t(15));
    full = reinterpret_cast<uint64_t *>(answer + 1);
    empty = full + 2, answered = full + 4;
    items = reinterpret_cast<Item *>(full + 5);
  }
  __device__ __forceinline__ void init(int consumers) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], consumers);
    }
    mbar_init(answered, 1);
  }

  // ---- the producer thread
  __device__ __forceinline__ bool put(uint32_t n, const Item &it, const WaitCtl &ctl, int code) {
    if (!mbar_wait(&empty[n & 1], ((n >> 1) & 1) ^ 1, ctl, code)) return false;
    items[n & 1] = it;
    mbar_arrive(&full[n & 1]);
    return true;
  }
  // ask for the item after the n-th (not after an answer of none)
  __device__ __forceinline__ void ask() {
    fence_proxy_async_cta();  // the answer before has been read
    mbar_arrive_expect_tx(answered, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(answered))
                 : "memory");
  }
  __device__ __forceinline__ int read() const {
    uint32_t some, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(some), "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    return some ? (int)x : -1;
  }
  // the item after the n-th, or -1: there is none left; n counts on only once
  // the answer is there (discard waits for the one that is not)
  __device__ __forceinline__ bool take(uint32_t &n, int &item, const WaitCtl &ctl, int code) {
    if (!mbar_wait(answered, n & 1, ctl, code)) return false;
    item = read();
    ++n;
    return true;
  }
  // After an abort in the n-th item (`asked`: its successor has been asked for):
  // take the items that are left, so that no CTA starts on them only to wait in
  // vain.
  __device__ __forceinline__ void discard(uint32_t n, bool asked) {
    while (true) {
      if (!asked) ask();
      asked = false;
      if (!drain_wait(answered, n & 1) || read() < 0) return;
      ++n;
    }
  }

  // ---- a consumer warp
  // The n-th item, or none: the end, or a wait that ran out (ok = false).
  __device__ __forceinline__ const Item *get(uint32_t n, bool &ok, const WaitCtl &ctl, int code) const {
    if (!mbar_wait_w(&full[n & 1], (n >> 1) & 1, ctl, code)) {
      ok = false;
      return nullptr;
    }
    const Item *it = &items[n & 1];
    return it->stop ? nullptr : it;
  }
  __device__ __forceinline__ void release(uint32_t n, int lane) const {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[n & 1]);
  }
};

// Four 16-byte pieces of this lane's row, columns 64 bytes wide, stored so that
// four lanes write a row's 64 bytes together (a 4 x 4 exchange among them): a
// lane for a row would touch 32 lines with every store.  `first`: the row of the
// quad's first lane at those columns; rows `pitch` bytes apart, `rows` of the
// quad there.
__device__ __forceinline__ void store_quad(uint4 (&w)[4], char *first, long long pitch, int rows, int lane) {
  auto swap = [&](uint4 &a, uint4 &b, int bit) {
    const bool up = lane & bit;
    uint4 give = up ? a : b;
    give.x = __shfl_xor_sync(0xffffffffu, give.x, bit);
    give.y = __shfl_xor_sync(0xffffffffu, give.y, bit);
    give.z = __shfl_xor_sync(0xffffffffu, give.z, bit);
    give.w = __shfl_xor_sync(0xffffffffu, give.w, bit);
    if (up) a = give;
    else b = give;
  };
  swap(w[0], w[1], 1);
  swap(w[2], w[3], 1);
  swap(w[0], w[2], 2);
  swap(w[1], w[3], 2);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < rows) *reinterpret_cast<uint4 *>(first + k * pitch + 16 * (lane & 3)) = w[k];
}

}  // namespace sta
