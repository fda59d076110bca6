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
// from item to item without a restart.  The producer warp asks for the next
// item when it starts one; every role reads the answer when it is done with
// its own.  Two answers are in flight at most.
struct Tickets {
  uint4 *answer;  // [2], shared memory
  uint64_t *full, *empty;  // [2] each; empty: one arrival per consumer warp
};
constexpr uint32_t kTicketBytes = 2 * 16 + 4 * 8;

__device__ __forceinline__ Tickets tickets_at(void *smem16) {
  uint4 *a = static_cast<uint4 *>(smem16);
  uint64_t *b = reinterpret_cast<uint64_t *>(a + 2);
  return Tickets{a, b, b + 2};
}
__device__ __forceinline__ void tickets_init(const Tickets &t, int consumers) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(&t.full[i], 1);
    mbar_init(&t.empty[i], consumers);
  }
}

__device__ __forceinline__ void ticket_cancel(const Tickets &t, uint32_t k) {
  mbar_arrive_expect_tx(&t.full[k & 1], 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(&t.answer[k & 1])),
               "r"(smem_u32(&t.full[k & 1]))
               : "memory");
}

// Ask for the k-th answer (the producer thread; not after an answer of none).
__device__ __forceinline__ bool ticket_ask(const Tickets &t, uint32_t k, const WaitCtl &ctl, int code) {
  if (!mbar_wait(&t.empty[k & 1], ((k >> 1) & 1) ^ 1, ctl, code)) return false;
  ticket_cancel(t, k);
  return true;
}

// The item in the k-th answer, or -1: there is none left.
__device__ __forceinline__ int ticket_read(const Tickets &t, uint32_t k) {
  uint32_t some, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(some), "=r"(x)
      : "r"(smem_u32(&t.answer[k & 1]))
      : "memory");
  fence_proxy_async_cta();  // the next answer is written by the async proxy
  return some ? (int)x : -1;
}

// The k-th answer for a whole consumer warp (-1: none, or a wait ran out).
__device__ __forceinline__ int ticket_next(const Tickets &t, uint32_t &k, bool &ok, const WaitCtl &ctl, int code, int lane) {
  if (!mbar_wait_w(&t.full[k & 1], (k >> 1) & 1, ctl, code)) {
    ok = false;
    return -1;
  }
  const int item = ticket_read(t, k);
  __syncwarp();
  if (lane == 0) mbar_arrive(&t.empty[k & 1]);
  ++k;
  return item;
}

// The k-th answer for the producer thread, which is not counted as a consumer.
__device__ __forceinline__ int ticket_take(const Tickets &t, uint32_t &k, bool &ok, const WaitCtl &ctl, int code) {
  if (!mbar_wait(&t.full[k & 1], (k >> 1) & 1, ctl, code)) {
    ok = false;
    return -1;
  }
  return ticket_read(t, k++);
}

// After an abort (the producer thread; `asked` answers asked for, `taken`
// read): take the items that are left, so that no CTA starts on them only to
// wait in vain.  The consumers have left, so their arrivals are not waited for.
__device__ __forceinline__ void tickets_discard(const Tickets &t, uint32_t asked, uint32_t taken, bool none) {
  while (!none) {
    if (asked == taken) ticket_cancel(t, asked++);
    if (!drain_wait(&t.full[taken & 1], (taken >> 1) & 1)) return;
    none = ticket_read(t, taken++) < 0;
  }
}

}  // namespace sta
