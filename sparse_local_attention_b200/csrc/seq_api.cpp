// seq_api.cpp -- host side of the token-sequence calls of include/sta.h:
// argument checks, workspace sizes, parameter blocks and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/sta.h"
#include "seq_kernels.h"

namespace {

constexpr size_t kStatusBytes = 256;
constexpr float kLeastScale = 7.888609052210118e-31f;  // 2^-100: |LSE / scale| is finite
constexpr long long kMaxRows = (1ll << 31) - 1024;
constexpr long long kMaxBlocks = 1ll << 30;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t round256(size_t b) { return (b + 255) & ~size_t(255); }

// A tensor of `batch` x `heads` x `rows` rows: its pointer and strides.
sta_status check_rows(const sta_rows *x, long long batch, long long heads, long long rows) {
  if (!x || !x->data) return STA_ERR_INVALID_ARG;
  const int64_t s[3] = {x->batch, x->head, x->row};
  const long long n[3] = {batch, heads, rows};
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;  // an extent of one: the stride is not used
    if (s[i] <= 0 || s[i] >= (1ll << 38)) return STA_ERR_INVALID_ARG;
    if (s[i] % 8) return STA_ERR_ALIGNMENT;
  }
  return aligned16(x->data) ? STA_OK : STA_ERR_ALIGNMENT;
}

sta::Rows rows_of(const sta_rows *x) {
  return sta::Rows{static_cast<char *>(x->data), x->batch, x->head, x->row};
}

bool io_type_ok(int32_t t) { return t == STA_TYPE_BF16 || t == STA_TYPE_FP16; }

sta_status check_problem(const sta_window_problem *p, bool packed) {
  if (!p) return STA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->heads < 1 || p->kv_heads < 1 || p->q_len < 0 || p->kv_len < 0 || p->q_rows < 0 ||
      p->kv_rows < 0 || p->heads % p->kv_heads || p->batch > 65534 || p->heads > 65535)
    return STA_ERR_SHAPE;
  if (p->head_dim != 64 && p->head_dim != 128) return STA_ERR_UNSUPPORTED;
  if (!io_type_ok(p->type)) return STA_ERR_UNSUPPORTED;
  if (p->window < 0 || p->sinks < 0 || !(p->scale == p->scale) || std::isinf(p->scale)) return STA_ERR_INVALID_ARG;
  // positions reach kv_len and -q_len: kept clear of kNoWindow
  if (p->q_len >= sta::kNoWindow / 2 || p->kv_len >= sta::kNoWindow / 2) return STA_ERR_SHAPE;
  // rows of the tensors, and blocks of the work lists; packed sequences share
  // their rows, so that q_len and kv_len count for the blocks only
  const long long bh = (long long)p->batch * p->heads, bk = (long long)p->batch * p->kv_heads;
  if ((packed ? (long long)p->heads * p->q_rows : bh * p->q_len) >= kMaxRows ||
      (packed ? (long long)p->kv_heads * p->kv_rows : bk * p->kv_len) >= kMaxRows ||
      bh * (p->q_len / 128 + 1) >= kMaxBlocks || bk * (p->kv_len / 128 + 1) >= kMaxBlocks)
    return STA_ERR_SHAPE;
  return STA_OK;
}

// Rows of lse and D.
size_t stat_rows(const sta_window_problem *p, bool packed) {
  return packed ? (size_t)p->heads * p->q_rows : (size_t)p->batch * p->heads * p->q_len;
}

// Whether a forward call splits the keys over the GPU (16 query rows of a key
// head at a time) or runs on 128-row tiles: what takes less by the rates of
// either on a B200.  The split form does 1400 steps of 16 keys a microsecond at
// head dim 64 and 550 at 128; a tile item takes 2.1 or 2.4 us for each 128 keys
// of its pair of blocks, in rounds of 148, or 1.1 or 1.3 us with the keys of one
// block split in its CTA, where all blocks fit in one round.  Measured, split
// against tiles, in us: 8 sequences, 24 heads over 8, d 128, window 1024: 3 rows
// 11 / 26, 24 rows 17 / 28, 96 rows 46 / 28; 1 sequence, 16 heads over 4, 8192
// keys, d 128: 4 rows 11 / 86, 256 rows 52 / 87, 512 rows 102 / 87.
bool splits_keys(const sta_window_problem *p) {
  auto up = [](long long n, long long m) { return (n + m - 1) / m; };
  const long long group = p->heads / p->kv_heads, slices = (long long)p->batch * p->kv_heads;
  const long long rows = p->q_len * group, blocks = up(p->q_len, 128) * group;
  if (rows > 256) return false;
  const long long span = (long long)p->window + p->q_len - 1 + p->sinks;
  const long long keys = p->window > 0 && span < p->kv_len ? span : p->kv_len;
  const bool small = p->head_dim == 64;
  const double split = (double)up(rows, 16) * slices * up(keys, 16) / (small ? 1400 : 550);
  const double per = blocks * slices <= 148 ? (small ? 1.1 : 1.3) : (small ? 2.1 : 2.4) * up(up(blocks, 2) * slices, 148);
  return rows <= 16 || split < per * (up(keys, 128) + 1);
}

size_t window_fwd_bytes(const sta_window_problem *) { return kStatusBytes; }

// How the backward's key blocks are cut into parts, and its workspace.  A part
// is at least 8 chunks of 128 queries (its 128 KB of sums are written and read
// once, about the time of two chunks) and otherwise 1 / (2 SMs) of the work, so
// that no block is one CTA's work for longer than the rest together.
struct BackwardLayout {
  int seg_chunks, sink_blocks, sink_segs, norm_segs, aug_rows, n_norms;
  size_t dd, aug, norms, parts, bytes;
};

BackwardLayout backward_layout(const sta_window_problem *p, bool packed) {
  constexpr long long kTargets = 2 * 148;
  BackwardLayout l{};
  auto up = [](long long n, long long m) { return (n + m - 1) / m; };
  const long long group = p->heads / p->kv_heads, slices = (long long)p->batch * p->kv_heads;
  const long long nkb = up(p->kv_len, 128);
  const bool windowed = p->window > 0 && p->window < p->kv_len;
  const long long all = up(p->q_len + 7ll, 128), seen = windowed ? up(p->window + 135ll, 128) : all;
  const long long norm = (seen < all ? seen : all) * group;
  l.sink_blocks = windowed && p->sinks > 0 ? (int)(up(p->sinks, 128) < nkb ? up(p->sinks, 128) : nkb) : 0;
  const long long work = slices * (nkb * norm / (windowed ? 1 : 2) + (l.sink_blocks ? l.sink_blocks * all * group : 0));
  const long long per = up(work, kTargets) > 8 ? up(work, kTargets) : 8;
  l.seg_chunks = (int)(per < 0x7fffffff ? per : 0x7fffffff);
  l.norm_segs = (int)(norm > per ? up(norm, per) : 1);
  l.sink_segs = (int)(l.sink_blocks && all * group > per ? up(all * group, per) : 1);
  // a packed sequence begins at a multiple of 8 panel rows, and at a place of its own among the norms
  l.aug_rows = (int)(packed ? up(p->q_rows, 8) * 8 + 8ll * p->batch + 8 : up(p->q_len, 8) * 8);
  const size_t aug_rows = (size_t)l.aug_rows * p->heads * (packed ? 1 : p->batch);
  const int pre = sta::pre_rows(p->head_dim);
  l.n_norms = (int)(packed ? (p->q_rows / pre + p->batch + 1ll) * p->heads : up(p->q_len, pre) * p->heads * p->batch);
  size_t slots = 0;
  if (l.norm_segs > 1) slots = (size_t)slices * (l.sink_blocks * l.sink_segs + (nkb - l.sink_blocks) * l.norm_segs);
  else if (l.sink_segs > 1) slots = (size_t)slices * l.sink_blocks * l.sink_segs;
  l.dd = kStatusBytes;
  l.aug = l.dd + round256(stat_rows(p, packed) * 4);
  l.norms = l.aug + (aug_rows + 128) * 32;  // a chunk reads 128 rows from any multiple of 8 on
  l.parts = l.norms + round256((size_t)l.n_norms * 4);
  l.bytes = l.parts + slots * 2 * 128 * p->head_dim * 4;
  return l;
}

// A problem without packed rows may still be that of a packed call over empty tensors.
size_t window_bwd_bytes(const sta_window_problem *p) {
  const size_t packed = backward_layout(p, true).bytes, dense = p->q_rows > 0 ? 0 : backward_layout(p, false).bytes;
  return packed > dense ? packed : dense;
}

sta::WinParams window_params(const sta_window_problem *p, const int32_t *cu_q, const int32_t *cu_kv, void *ws) {
  sta::WinParams w{};
  w.batch = p->batch, w.heads = p->heads, w.kv_heads = p->kv_heads, w.group = p->heads / p->kv_heads, w.d = p->head_dim;
  w.q_len = p->q_len, w.kv_len = p->kv_len, w.q_rows = p->q_rows, w.kv_rows = p->kv_rows;
  w.window = p->window == 0 || p->window > sta::kNoWindow ? sta::kNoWindow : p->window;
  w.sinks = p->sinks < sta::kNoWindow ? p->sinks : sta::kNoWindow;
  w.cu_q = cu_q, w.cu_kv = cu_kv;
  w.scale = p->scale > 0.f ? p->scale : 1.f / std::sqrt((float)p->head_dim);
  w.scale_log2 = w.scale * 1.4426950408889634f;
  w.status = static_cast<int *>(ws);
  w.wait_limit_ns = sta::wait_limit_ns();
  return w;
}

sta_status finish(void *ws, cudaStream_t stream, uint32_t flags) {
  if (flags & STA_CALL_CHECK) {
    if (cudaStreamSynchronize(stream) != cudaSuccess) return STA_ERR_CUDA;
    int st = 0;
    if (ws && cudaMemcpy(&st, ws, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return STA_ERR_CUDA;
    if (st != 0) return STA_ERR_TIMEOUT;
  }
  return STA_OK;
}

bool bad_window_call(uint32_t flags, const int32_t *cu_q, const int32_t *cu_kv) {
  return (flags & ~(STA_CALL_CHECK | (cu_q ? STA_PACKED_ZERO : 0u))) || (cu_q == nullptr) != (cu_kv == nullptr);
}

sta_status check_tensors(const sta_window_problem *p, bool packed, const sta_rows *const *q_side, int nq,
                         const sta_rows *const *kv_side, int nkv) {
  const long long batch = packed ? 1 : p->batch;
  for (int i = 0; i < nq; ++i)
    if (const sta_status st = check_rows(q_side[i], batch, p->heads, packed ? p->q_rows : p->q_len)) return st;
  for (int i = 0; i < nkv; ++i)
    if (const sta_status st = check_rows(kv_side[i], batch, p->kv_heads, packed ? p->kv_rows : p->kv_len)) return st;
  return STA_OK;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return reinterpret_cast<EncodeTiledFn>(ok ? ptr : nullptr);
  }();
  return fn;
}

// A tensor of rows viewed as (64, rows, heads, batch[, 2 panels of head dim
// 128]); a box is 128 rows of one head, all panels.
bool tile_map(CUtensorMap *m, const sta_rows *x, int32_t type, int d, long long rows, long long heads, long long batch) {
  const EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  // strides of extents of one are not used, but must be valid
  auto bytes = [](long long n, int64_t stride) { return (cuuint64_t)(n > 1 ? stride * 2 : 256); };
  const cuuint64_t dims[5] = {64, (cuuint64_t)(rows > 0 ? rows : 1), (cuuint64_t)heads, (cuuint64_t)batch, 2};
  const cuuint64_t strides[4] = {bytes(rows, x->row), bytes(heads, x->head), bytes(batch, x->batch), 128};
  const cuuint32_t box[5] = {64, 128, 1, 1, 2}, estr[5] = {1, 1, 1, 1, 1};
  return enc(m, type == STA_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             d == 128 ? 5 : 4, x->data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

bool q_map(CUtensorMap *m, const sta_rows *x, const sta_window_problem *p, bool packed) {
  return tile_map(m, x, p->type, p->head_dim, packed ? p->q_rows : p->q_len, p->heads, packed ? 1 : p->batch);
}
bool kv_map(CUtensorMap *m, const sta_rows *x, const sta_window_problem *p, bool packed) {
  return tile_map(m, x, p->type, p->head_dim, packed ? p->kv_rows : p->kv_len, p->kv_heads, packed ? 1 : p->batch);
}

// Make the current device's context current for this thread, too: a thread that
// has not used the device before (such as an autograd worker) has none, and
// encoding a tensor map needs it.
bool open_device() {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
}

sta_status check_workspace(const void *ws, size_t have, size_t need) {
  if (!ws || have < need) return STA_ERR_WORKSPACE;
  return aligned16(ws) ? STA_OK : STA_ERR_ALIGNMENT;
}

sta_status check_cache(const sta_cache *c, int32_t batch, int32_t table_pages) {
  if (!c) return STA_ERR_INVALID_ARG;
  if (c->pages < 1 || c->kv_heads < 1 || c->kv_heads > 65535 || c->page_size < 1 || batch < 1 || batch > 32767 ||
      table_pages < 1 || (long long)table_pages * c->page_size >= sta::kNoWindow / 2 ||
      (long long)c->pages * c->page_size > 0x7fffffffll)
    return STA_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return STA_ERR_UNSUPPORTED;
  if (c->type != STA_TYPE_E4M3 && c->type != STA_TYPE_INT8) return STA_ERR_UNSUPPORTED;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return STA_ERR_UNSUPPORTED;
  if (c->page_size % c->block) return STA_ERR_SHAPE;
  return STA_OK;
}

sta_status check_cache_pointers(const sta_cache *c, const int32_t *table, const int32_t *per_sequence) {
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !table || !per_sequence) return STA_ERR_INVALID_ARG;
  const void *p[] = {c->k, c->v, c->k_scale, c->v_scale};
  for (const void *x : p)
    if (!aligned16(x)) return STA_ERR_ALIGNMENT;
  return STA_OK;
}

sta::CacheParams cache_params(const sta_cache *c, const int32_t *table, int32_t table_pages) {
  sta::CacheParams p{};
  p.pages = c->pages, p.kv_heads = c->kv_heads, p.page_size = c->page_size, p.block = c->block, p.d = c->head_dim;
  p.k = static_cast<uint8_t *>(c->k), p.v = static_cast<uint8_t *>(c->v);
  p.k_scale = c->k_scale, p.v_scale = c->v_scale;
  p.table = table, p.table_pages = table_pages;
  return p;
}

sta_status move_call(bool write, const sta_cache *c, int32_t batch, int32_t rows, const sta_rows *k, const sta_rows *v,
                     int32_t type, const int32_t *table, int32_t table_pages, const int32_t *start,
                     const int32_t *count, void *stream_, uint32_t flags) {
  if (const sta_status st = check_cache(c, batch, table_pages)) return st;
  if (rows < 0 || (long long)batch * c->kv_heads * rows >= kMaxRows) return STA_ERR_SHAPE;
  if (!io_type_ok(type)) return STA_ERR_UNSUPPORTED;
  if (flags & ~(STA_CALL_CHECK | (write ? 0u : STA_READ_ZERO))) return STA_ERR_INVALID_ARG;
  if (const sta_status st = check_cache_pointers(c, table, start)) return st;
  if (const sta_status st = check_rows(k, batch, c->kv_heads, rows)) return st;
  if (const sta_status st = check_rows(v, batch, c->kv_heads, rows)) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (rows > 0) {
    const sta::CacheMove m{cache_params(c, table, table_pages), batch, rows, rows_of(k), rows_of(v), start, count,
                           (flags & STA_READ_ZERO) != 0};
    const cudaError_t e = write ? sta::launch_cache_write(m, c->type, type, stream)
                                : sta::launch_cache_read(m, c->type, type, stream);
    if (e != cudaSuccess) return STA_ERR_CUDA;
  }
  return finish(nullptr, stream, flags);
}

}  // namespace

extern "C" {

sta_status sta_window_workspace_size(const sta_window_problem *p, size_t *fwd, size_t *bwd) {
  if (const sta_status st = check_problem(p, p && p->q_rows > 0)) return st;
  if (fwd) *fwd = window_fwd_bytes(p);
  if (bwd) *bwd = window_bwd_bytes(p);
  return STA_OK;
}

sta_status sta_window_forward(const sta_window_problem *p, const sta_rows *q, const sta_rows *k, const sta_rows *v,
                              const sta_rows *o, float *lse, const int32_t *cu_q, const int32_t *cu_kv, void *ws,
                              size_t ws_bytes, void *stream_, uint32_t flags) {
  if (const sta_status st = check_problem(p, cu_q != nullptr)) return st;
  if (bad_window_call(flags, cu_q, cu_kv)) return STA_ERR_INVALID_ARG;
  const sta_rows *qs[] = {q, o}, *ks[] = {k, v};
  if (const sta_status st = check_tensors(p, cu_q, qs, 2, ks, 2)) return st;
  if (const sta_status st = check_workspace(ws, ws_bytes, window_fwd_bytes(p))) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  sta::WinParams w = window_params(p, cu_q, cu_kv, ws);
  w.q = rows_of(q), w.k = rows_of(k), w.v = rows_of(v), w.o = rows_of(o), w.lse = lse;
  if ((flags & STA_CALL_CHECK) && cudaMemsetAsync(ws, 0, sizeof(int), stream) != cudaSuccess) return STA_ERR_CUDA;
  w.zero = (flags & STA_PACKED_ZERO) != 0;
  if (w.zero && p->q_rows > 0 && sta::launch_window_clear(w, stream) != cudaSuccess) return STA_ERR_CUDA;
  if (p->q_len > 0) {
    if (splits_keys(p)) {
      if (sta::launch_window_split(w, p->type, stream) != cudaSuccess) return STA_ERR_CUDA;
      return finish(ws, stream, flags);
    }
    CUtensorMap maps[3];
    if (!open_device() || !q_map(&maps[0], q, p, cu_q) || !kv_map(&maps[1], k, p, cu_q) ||
        !kv_map(&maps[2], v, p, cu_q) || sta::launch_window_tiles(w, p->type, maps, stream) != cudaSuccess)
      return STA_ERR_CUDA;
  }
  return finish(ws, stream, flags);
}

sta_status sta_window_backward(const sta_window_problem *p, const sta_rows *q, const sta_rows *k, const sta_rows *v,
                               const sta_rows *o, const float *lse, const sta_rows *dout, const sta_rows *dq,
                               const sta_rows *dk, const sta_rows *dv, const int32_t *cu_q, const int32_t *cu_kv,
                               void *ws, size_t ws_bytes, void *stream_, uint32_t flags) {
  if (const sta_status st = check_problem(p, cu_q != nullptr)) return st;
  if (bad_window_call(flags, cu_q, cu_kv) || !lse) return STA_ERR_INVALID_ARG;
  if (p->scale > 0.f && p->scale < kLeastScale) return STA_ERR_INVALID_ARG;
  const sta_rows *qs[] = {q, o, dout, dq}, *ks[] = {k, v, dk, dv};
  if (const sta_status st = check_tensors(p, cu_q, qs, 4, ks, 4)) return st;
  const BackwardLayout l = backward_layout(p, cu_q != nullptr);
  if (const sta_status st = check_workspace(ws, ws_bytes, l.bytes)) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  sta::WinParams w = window_params(p, cu_q, cu_kv, ws);
  w.q = rows_of(q), w.k = rows_of(k), w.v = rows_of(v), w.o = rows_of(o), w.dout = rows_of(dout);
  w.dq = rows_of(dq), w.dk = rows_of(dk), w.dv = rows_of(dv);
  w.lse = const_cast<float *>(lse);
  w.zero = (flags & STA_PACKED_ZERO) != 0;
  char *base = static_cast<char *>(ws);
  w.dd = reinterpret_cast<float *>(base + l.dd);
  w.aug = reinterpret_cast<uint8_t *>(base + l.aug), w.aug_rows = l.aug_rows;
  w.norms = reinterpret_cast<float *>(base + l.norms), w.n_norms = l.n_norms;
  w.parts = reinterpret_cast<float *>(base + l.parts);
  w.seg_chunks = l.seg_chunks, w.sink_blocks = l.sink_blocks, w.sink_segs = l.sink_segs, w.norm_segs = l.norm_segs;
  if ((flags & STA_CALL_CHECK) && cudaMemsetAsync(ws, 0, sizeof(int), stream) != cudaSuccess) return STA_ERR_CUDA;
  CUtensorMap maps[4];
  if (!open_device() || !q_map(&maps[0], q, p, cu_q) || !kv_map(&maps[1], k, p, cu_q) ||
      !kv_map(&maps[2], v, p, cu_q) || !q_map(&maps[3], dout, p, cu_q) ||
      sta::launch_window_backward(w, p->type, maps, stream) != cudaSuccess)
    return STA_ERR_CUDA;
  return finish(ws, stream, flags);
}

sta_status sta_cache_write(const sta_cache *c, int32_t batch, int32_t rows, const sta_rows *k, const sta_rows *v,
                           int32_t in_type, const int32_t *table, int32_t table_pages, const int32_t *start,
                           const int32_t *count, void *stream, uint32_t flags) {
  return move_call(true, c, batch, rows, k, v, in_type, table, table_pages, start, count, stream, flags);
}

sta_status sta_cache_read(const sta_cache *c, int32_t batch, int32_t rows, const sta_rows *k, const sta_rows *v,
                          int32_t out_type, const int32_t *table, int32_t table_pages, const int32_t *start,
                          const int32_t *count, void *stream, uint32_t flags) {
  return move_call(false, c, batch, rows, k, v, out_type, table, table_pages, start, count, stream, flags);
}

sta_status sta_cache_attention(const sta_cache *c, int32_t batch, int32_t heads, int32_t q_len, int32_t window,
                               int32_t sinks, float scale, int32_t type, const sta_rows *q, const sta_rows *o,
                               float *lse, const int32_t *table, int32_t table_pages, const int32_t *lengths,
                               void *stream_, uint32_t flags) {
  if (const sta_status st = check_cache(c, batch, table_pages)) return st;
  if (heads < 1 || heads > 65535 || heads % c->kv_heads || q_len < 0 || (long long)batch * heads * q_len >= kMaxRows ||
      (long long)q_len * (heads / c->kv_heads) > 16 * 65535)
    return STA_ERR_SHAPE;
  if (!io_type_ok(type)) return STA_ERR_UNSUPPORTED;
  if ((flags & ~STA_CALL_CHECK) || window < 0 || sinks < 0 || !(scale == scale) || std::isinf(scale))
    return STA_ERR_INVALID_ARG;
  if (const sta_status st = check_cache_pointers(c, table, lengths)) return st;
  if (const sta_status st = check_rows(q, batch, heads, q_len)) return st;
  if (const sta_status st = check_rows(o, batch, heads, q_len)) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  sta::CacheAttn a{};
  a.c = cache_params(c, table, table_pages);
  a.batch = batch, a.heads = heads, a.group = heads / c->kv_heads, a.q_len = q_len;
  a.window = window == 0 || window > sta::kNoWindow ? sta::kNoWindow : window;
  a.sinks = sinks < sta::kNoWindow ? sinks : sta::kNoWindow;
  a.scale_log2 = (scale > 0.f ? scale : 1.f / std::sqrt((float)c->head_dim)) * 1.4426950408889634f;
  a.q = rows_of(q), a.o = rows_of(o), a.lse = lse, a.lengths = lengths;
  a.blocks = c->page_size / c->block;
  while ((1 << a.block_shift) < c->block) ++a.block_shift;
  if (q_len > 0 && sta::launch_cache_attention(a, c->type, type, stream) != cudaSuccess) return STA_ERR_CUDA;
  return finish(nullptr, stream, flags);
}

}  // extern "C"
