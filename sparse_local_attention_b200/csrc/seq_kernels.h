// seq_kernels.h -- parameter blocks and launchers of the token-sequence
// operators, shared by their host API (seq_api.cpp) and the CUDA kernels.
// Internal to libsta.so.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/sta.h"

namespace sta {

// A window that hides nothing: every position minus it is far below zero.
constexpr int kNoWindow = 1 << 30;

uint64_t wait_limit_ns();  // sta_set_wait_limit_ns's value

// Strides of a tensor of rows, in elements.
struct Rows {
  char *p;
  long long b, h, r;
};

// One problem of sta_window_forward / sta_window_backward.
struct WinParams {
  int batch, heads, kv_heads, group, d;
  int q_len, kv_len;    // rows of every sequence, or of the longest one (packed)
  int q_rows, kv_rows;  // packed: rows of the tensors
  int window, sinks;    // window >= 1
  const int32_t *cu_q, *cu_kv;
  float scale, scale_log2;
  Rows q, k, v, o, dout, dq, dk, dv;
  float *lse;
  // backward
  float *dd;       // D = rowsum(dO o O), laid out like lse
  uint8_t *aug;    // operand panels of -LSE and -D: 256 bytes per 8 query rows
  int aug_rows;    // panel rows per head
  float *norms;    // largest row norm of dO per pre_rows(d) rows (fp16)
  int n_norms;
  float *parts;    // fp32 sums of dK and dV of the parts of key blocks
  int seg_chunks;  // chunks of 128 queries per part
  int sink_blocks, sink_segs, norm_segs;  // key blocks that hold sinks; parts per block there and elsewhere, at most
  bool zero;       // packed: rows outside every sequence become zeros (-inf in lse)
  int *status;
  unsigned long long wait_limit_ns;
};

// Query rows per block of the backward's first pass.
__host__ __device__ constexpr int pre_rows(int d) { return d == 128 ? 64 : 128; }

// The cache of sta_cache, with its pages addressed through a table.
struct CacheParams {
  int pages, kv_heads, page_size, block, d;
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  const int32_t *table;
  int table_pages;
};

// sta_cache_write / sta_cache_read.
struct CacheMove {
  CacheParams c;
  int batch, rows;
  Rows k, v;
  const int32_t *start, *count;
  bool zero;  // reading: rows without a token become zeros
};

cudaError_t launch_cache_write(const CacheMove &m, int cache_type, int io_type, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheMove &m, int cache_type, int io_type, cudaStream_t stream);

// sta_cache_attention.
struct CacheAttn {
  CacheParams c;
  int batch, heads, group, q_len, window, sinks;
  float scale_log2;
  Rows q, o;
  float *lse;
  const int32_t *lengths;
  int blocks, block_shift;   // scales per page and head, log2(block)
};
cudaError_t launch_cache_attention(const CacheAttn &a, int cache_type, int io_type, cudaStream_t stream);

// o and lse of rows outside every sequence (p.zero).
cudaError_t launch_window_clear(const WinParams &p, cudaStream_t stream);
// Forward on 128-row tiles; maps: q, k, v.  With p.zero, after launch_window_clear.
cudaError_t launch_window_tiles(const WinParams &p, int type, const CUtensorMap *maps, cudaStream_t stream);
// Forward of a few query rows per key head, the keys split over the GPU.
cudaError_t launch_window_split(const WinParams &p, int type, cudaStream_t stream);
// Backward; maps: q, k, v, dO.
cudaError_t launch_window_backward(const WinParams &p, int type, const CUtensorMap *maps, cudaStream_t stream);

}  // namespace sta
