// seq_common.cuh -- device helpers shared by the token-sequence kernels:
// element conversions, the rows of a (packed or dense) sequence, and the
// addressing of a paged cache.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <atomic>
#include <cstdint>

#include "seq_kernels.h"

namespace sta {

// Raise a kernel's limit of dynamic shared memory, once per device.  `done` is
// the caller's record of the devices it has been raised on.
template <class Kernel>
cudaError_t allow_shared(Kernel *kernel, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// fp32 <-> the 16-bit types, two at a time; lo in bits 0..15.
template <class T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static constexpr float kMax = 3.3895313892515355e38f;
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
template <> struct Elem<__half> {
  static constexpr float kMax = 65504.f;
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// Rows [q0, q0 + nq) of the query tensors and [k0, k0 + nk) of the key tensors
// hold sequence b; `slice` is its batch index in the tensors (0 when packed).
struct Sequence {
  int slice, q0, nq, k0, nk;
};

__device__ __forceinline__ void packed_range(const int32_t *cu, int b, int rows, int longest, int &first, int &n) {
  first = min(max(__ldg(cu + b), 0), rows);
  const int end = min(max(__ldg(cu + b + 1), first), rows);
  n = min(end - first, longest);
}

__device__ __forceinline__ Sequence sequence(const WinParams &p, int b) {
  Sequence s{b, 0, p.q_len, 0, p.kv_len};
  if (p.cu_q) {
    s.slice = 0;
    packed_range(p.cu_q, b, p.q_rows, p.q_len, s.q0, s.nq);
    packed_range(p.cu_kv, b, p.kv_rows, p.kv_len, s.k0, s.nk);
  }
  return s;
}

// Index of a query row in lse and D.
__device__ __forceinline__ long long stat_row(const WinParams &p, const Sequence &s, int h, int row) {
  return p.cu_q ? (long long)h * p.q_rows + s.q0 + row : ((long long)s.slice * p.heads + h) * p.q_len + row;
}

__device__ __forceinline__ bool visible(int pos, int key, int window, int sinks) {
  return key <= pos && (key > pos - window || key < sinks);
}

// Whether a row of a packed tensor is in a sequence.  Exact where the starts
// ascend; of starts that do not, some rows of sequences are called outside.
__device__ __forceinline__ bool in_sequence(const int32_t *cu, int batch, int rows, int longest, int row) {
  int lo = 0, hi = batch - 1;  // the last sequence that starts at or before the row
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (__ldg(cu + mid) <= row) lo = mid;
    else hi = mid - 1;
  }
  int first, n;
  packed_range(cu, lo, rows, longest, first, n);
  return row >= first && row < first + n;
}

// Rows [32 i, 32 i + 32) of up to two packed tensors (and lse) that no sequence
// holds become zeros (-inf), by one warp.  What writes the sequences' rows runs
// afterwards.
__device__ __forceinline__ void clear_outside(const int32_t *cu, int batch, int rows, int longest, int i, int heads, int d,
                                              const Rows &x, const Rows &y, float *lse) {
  const int lane = threadIdx.x & 31, row0 = 32 * i, mine = row0 + lane;
  uint32_t out = __ballot_sync(0xffffffffu, mine < rows && !in_sequence(cu, batch, rows, longest, mine));
  const int per = d / 8, pieces = heads * per;  // 16 bytes each
  for (; out; out &= out - 1) {
    const long long row = row0 + __ffs(out) - 1;
    for (int j = lane; j < pieces; j += 32) {
      const int h = j / per, at = 16 * (j % per);
      *reinterpret_cast<uint4 *>(x.p + 2 * (h * x.h + row * x.r) + at) = make_uint4(0u, 0u, 0u, 0u);
      if (y.p) *reinterpret_cast<uint4 *>(y.p + 2 * (h * y.h + row * y.r) + at) = make_uint4(0u, 0u, 0u, 0u);
    }
    if (lse)
      for (int h = lane; h < heads; h += 32) lse[(long long)h * rows + row] = -INFINITY;
  }
}

// Page that holds token `pos` of sequence b, or -1 (absent, or past the table).
__device__ __forceinline__ int page_of(const CacheParams &c, int b, int pos) {
  const int i = pos / c.page_size;
  if (pos < 0 || i >= c.table_pages) return -1;
  const int page = __ldg(c.table + (long long)b * c.table_pages + i);
  return (unsigned)page < (unsigned)c.pages ? page : -1;
}

}  // namespace sta
