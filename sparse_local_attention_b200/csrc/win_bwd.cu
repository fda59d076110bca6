// win_bwd.cu -- backward of causal sliding-window attention with sinks on
// 128-row tiles (sm_100a tensor cores).
//
// With P = exp(S - LSE) over the visible pairs and D_i = sum_c dO_ic O_ic:
//   dV = P^T dO,  dS = P o (dO V^T - D),  dK = scale dS^T Q,  dQ = scale dS K,
// dK and dV summed over the query heads of a key head.  No atomics: every sum
// has one order.
//
//   1. window_pre: D per row; per 8 query rows the operand panel that carries
//      -LSE / scale and -D into the dK / dV kernel's products; for fp16 the
//      largest row norm of dO per block.
//   2. window_dkdv: an item is a 128-row key block of a key head (or a part of
//      its queries): K and V stay in shared memory; the 128-row chunks of the
//      queries that see the block, head after head of the group, stream
//      through rings.  S^T = K Q^T and dP^T = V dO^T land in tensor memory,
//      the elementwise warps (thread = key row) turn them into P^T and dS^T,
//      then dV += P^T dO and dK += dS^T Q accumulate in tensor memory.  Blocks
//      that many queries see (sinks; long sequences of few heads) are cut into
//      parts of at most seg_chunks chunks, whose fp32 sums window_join adds up
//      in order: without it one sink block of a long sequence is one CTA's
//      work for longer than all the others together.
//   3. window_dq: an item is a 128-row query block of a head; its keys come as
//      in the forward (sinks, then the window from its own first key on).
//
// Chunks that all rows see whole take no mask.  A contraction runs over the
// valid rows of a chunk rounded up to 16, and the "clear" warp zeroes the rows
// in between, so that another sequence's rows never meet a zero as NaN.
//
// P and dS are rounded to the tensors' type, the precision of the tensor
// core's A operand.  fp16 has 5 exponent bits: P is held times 2^8 and dS times
// a power of two near 4 / max_i |dO_i| over the finite rows that see a key, so that
// neither falls below its normal range where it matters (|dS| <= 2 |dO_i| |V_j|:
// rows of V up to a norm of 8192 do not overflow).  D is taken from O as it was
// stored, in the tensors' type; -LSE and -D enter as three bf16 numbers each, which
// keep fp32's precision and range.
//
// Measured on a B200, in us: 2 x 4096 tokens, 16 heads, d 64, window 512: 149;
// 8192 tokens, 24 heads, d 128, window 2048: 706 (0.64 PFLOP/s over the visible
// pairs), without a window 1359 (0.76); packed, 9 sequences up to 701, 16 heads
// over 8, d 128, window 256: 110.  dK / dV waits for its next Q and dO (two stages of each fit
// beside K and V at d 128) about 400 cycles of a chunk's 2600.
#include "seq_tile.cuh"

namespace sta {
namespace {

constexpr int kBM = kTileRows;
constexpr uint32_t kAugBytes = 4096;  // panel of 128 query rows
constexpr float kLog2e = 1.4426950408889634f;

// Elementwise warps of NG warpgroups (warpgroup e: columns [e kBM / NG, (e + 1)
// kBM / NG) of each chunk; thread = TMEM lane = row), then the TMA producer, the
// MMA issuer and the clear warp.
template <int NG>
struct Roles {
  static constexpr int kGroups = NG;
  static constexpr int kMathWarps = 4 * NG;
  static constexpr int kProducerWarp = kMathWarps, kMmaWarp = kMathWarps + 1, kClearWarp = kMathWarps + 2;
  static constexpr int kThreads = 32 * (kMathWarps + 3);
  static constexpr int kCols = kBM / NG;
};

template <class T> constexpr bool kIsHalf = std::is_same<T, __half>::value;
template <class T> constexpr float kPShift = kIsHalf<T> ? 8.f : 0.f;  // log2 of P's factor

// x as three bf16 numbers, lo in bits 0..15 of r[0]: 24 bits, as many as x has
// (two leave 2^-18 of x, 4% of P at a log-sum-exp of 10 000).
__device__ __forceinline__ void three_parts(float x, uint32_t (&r)[2]) {
  using E = Elem<__nv_bfloat16>;
  x = fabsf(x) > E::kMax ? copysignf(E::kMax, x) : x;  // does not round to infinity
  const float rest = x - E::unpack(E::pack(x, 0.f)).x;
  r[0] = E::pack(x, rest);
  r[1] = E::pack(rest - E::unpack(r[0]).y, 0.f);
}

// The panel row of one query, in bf16 whatever T is (fp16 would end at a
// |LSE / scale| of 2^20): elements 0 -- 2 carry -LSE / scale, 3 -- 5 -D.

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Panel row of query `row` of head h: rows of a sequence are consecutive and
// its first one a multiple of 8.
__device__ __forceinline__ long long aug_row(const WinParams &p, const Sequence &s, int b, int h) {
  if (p.cu_q) return (long long)h * p.aug_rows + (s.q0 & ~7) + 8 * b;
  return ((long long)s.slice * p.heads + h) * p.aug_rows;
}

// The factor of dS (1 unless T is fp16), by a whole CTA.
template <class T>
__device__ __forceinline__ float ds_factor(const WinParams &p, float *smem_word) {
  if constexpr (!kIsHalf<T>) return 1.f;
  int *word = reinterpret_cast<int *>(smem_word);
  if (threadIdx.x == 0) *word = 0;
  __syncthreads();
  float m = 0.f;
  for (int i = threadIdx.x; i < p.n_norms; i += blockDim.x) m = fmaxf(m, p.norms[i]);
  atomicMax(word, __float_as_int(m));  // nonnegative floats order like integers
  __syncthreads();
  const float top = __int_as_float(*word);
  if (!(top > 0.f) || isinf(top)) return 1.f;
  const int e = ((__float_as_int(top) >> 23) & 0xff) - 127;
  return exp2f((float)max(-100, min(100, 2 - e)));
}

// ----------------------------------------------------------------------- 1. preprocess
// Sums of four rows' values over a group of kLanes lanes; lane `part` gets row
// 2 (part & 1) + (part >> 1 & 1)'s.  The group's lanes share the rows after two
// exchanges, so that what follows runs once for four rows.
template <int kLanes>
__device__ __forceinline__ float sum_rows(const float (&v)[4], int part) {
  const bool up = part & 1, upper = part & 2;
  const float a = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 1);
  const float b = (up ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 1);
  float x = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 2);
#pragma unroll
  for (int off = 4; off < kLanes; off *= 2) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// A group of D / 8 lanes per row, a CTA per pre_rows(D) rows of a head: four
// rows per lane group, all of them in flight at once.
template <int D, class T>
__global__ void __launch_bounds__(256) window_pre_kernel(const WinParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, part = lane % kLanes, h = blockIdx.y;
  int b = blockIdx.z;
  if (p.zero && b-- == 0) {
    // the first blocks: gradients of rows outside every sequence
    const int q_parts = (p.q_rows + 31ll) / 32, kv_parts = (p.kv_rows + 31ll) / 32, warps = gridDim.x * gridDim.y * 8;
    for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * 8 + (threadIdx.x >> 5); i < q_parts + kv_parts; i += warps) {
      if (i < q_parts) clear_outside(p.cu_q, p.batch, p.q_rows, p.q_len, i, p.heads, D, p.dq, Rows{}, nullptr);
      else clear_outside(p.cu_kv, p.batch, p.kv_rows, p.kv_len, i - q_parts, p.kv_heads, D, p.dk, p.dv, nullptr);
    }
    return;
  }
  const Sequence s = sequence(p, b);
  const long long aug0 = aug_row(p, s, b, h);
  constexpr int kPass = 8 * kRows;
  static_assert(pre_rows(D) == 4 * kPass, "four rows per lane group");
  const int row0 = blockIdx.x * pre_rows(D) + (threadIdx.x >> 5) * kRows + sub;
  const char *o_at = p.o.p + 2 * (s.slice * p.o.b + h * p.o.h + (long long)(s.q0 + row0) * p.o.r) + 16 * part;
  const char *g_at =
      p.dout.p + 2 * (s.slice * p.dout.b + h * p.dout.h + (long long)(s.q0 + row0) * p.dout.r) + 16 * part;
  // the row that this lane (and those that differ from it in the upper bits) finishes
  const int row = row0 + (2 * (part & 1) + (part >> 1 & 1)) * kPass;
  const bool valid = row < s.nq;
  uint4 a[4], g[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = g[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row0 + i * kPass < s.nq) {
      a[i] = __ldg(reinterpret_cast<const uint4 *>(o_at + 2ll * i * kPass * p.o.r));
      g[i] = __ldg(reinterpret_cast<const uint4 *>(g_at + 2ll * i * kPass * p.dout.r));
    }
  }
  const float lse = valid ? __ldg(p.lse + stat_row(p, s, h, row)) : 0.f;
  float accs[4], sqs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    accs[i] = 0.f, sqs[i] = 0.f;
    const uint32_t av[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, gv[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 af = Elem<T>::unpack(av[e]), gf = Elem<T>::unpack(gv[e]);
      accs[i] = fmaf(af.x, gf.x, fmaf(af.y, gf.y, accs[i]));
      sqs[i] = fmaf(gf.x, gf.x, fmaf(gf.y, gf.y, sqs[i]));
    }
  }
  const float acc = sum_rows<kLanes>(accs, part);
  if (valid && part < 8) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (part < 4) {
      p.dd[stat_row(p, s, h, row)] = acc;
      // a row that sees nothing has LSE = -inf; all its pairs are masked
      uint32_t a[2], d[2];
      three_parts(lse == -INFINITY ? 0.f : -lse / p.scale, a);
      three_parts(-acc, d);
      w[0] = a[0], w[1] = a[1] | d[0] << 16, w[2] = d[0] >> 16 | d[1] << 16;
    }
    const long long ar = aug0 + row;  // two halves of 16 bytes, the second one zero
    *reinterpret_cast<uint4 *>(p.aug + ar / 8 * 256 + part / 4 * 128 + ar % 8 * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if constexpr (kIsHalf<T>) {
    __shared__ int top;
    if (threadIdx.x == 0) top = 0;
    __syncthreads();
    // rows that see nothing have no gradients, those of others are not finite
    const float sq = sum_rows<kLanes>(sqs, part);
    const bool counts = valid && lse > -INFINITY && sq < INFINITY;
    const int most = __reduce_max_sync(0xffffffffu, counts ? __float_as_int(sqrtf(sq)) : 0);
    if (lane == 0) atomicMax(&top, most);  // nonnegative floats order like integers
    __syncthreads();
    if (threadIdx.x == 0) {
      if (!p.cu_q) p.norms[((long long)b * p.heads + h) * gridDim.x + blockIdx.x] = __int_as_float(top);
      // packed: of the rows that are there; the others have been zeroed
      else if ((int)blockIdx.x * pre_rows(D) < s.nq)
        p.norms[(long long)h * (p.n_norms / p.heads) + s.q0 / pre_rows(D) + b + blockIdx.x] = __int_as_float(top);
    }
  }
}

// ----------------------------------------------------------------------- 2. dK, dV
// A key block and the part [c0, c1) of its chunks; chunk c is rows [qa + 128
// (c % per_head), ...) of head c / per_head of the group.
struct KeyItem {
  bool stop;
  Sequence s;
  int b, hk, key0, rows;  // rows: 0 for a part that is not there
  int qa, qe, per_head, c0, c1, segs;
  int lead;  // rows of a head's first chunk before the first one that sees the block
  long long slot;  // of the part's sums, or -1: the block is one part
  __device__ __forceinline__ int first(int c) const { return qa + c % per_head * kBM; }
  __device__ __forceinline__ int valid(int c) const { return min(kBM, qe - first(c)); }
  __device__ __forceinline__ int hidden(int c) const { return c % per_head == 0 ? lead : 0; }
  // Rows of a chunk that the contraction meets and that do not see the block (the
  // first `hidden`, and those past `valid` up to a multiple of 16) are cleared:
  // NaN there would not stay behind a P of zero.
  __device__ __forceinline__ bool clears(int c) const { return valid(c) % 16 != 0 || hidden(c) > 0; }
};

// The queries that see a key block, and its number of parts.
__device__ __forceinline__ void block_queries(const WinParams &p, KeyItem &it) {
  const int off = it.s.nk - it.s.nq;
  it.rows = min(kBM, it.s.nk - it.key0);
  it.qa = max(0, it.key0 - off) & ~7;  // panels start at multiples of 8
  it.lead = max(0, it.key0 - off) & 7;
  const int past = it.key0 + it.rows - 1 + p.window - off;  // first row past the window of the last key
  it.qe = it.rows <= 0 ? 0 : it.key0 < p.sinks ? it.s.nq : min(it.s.nq, past);
  it.per_head = max(0, (it.qe - it.qa + kBM - 1) / kBM);
  const int total = it.per_head * p.group;
  it.segs = max(1, (total + p.seg_chunks - 1) / p.seg_chunks);
}

// Parts are numbered sink blocks first (sink_blocks of them with sink_segs
// slots each), then the others (norm_segs each), key blocks ascending, the
// sequences and key heads innermost.
__device__ __forceinline__ KeyItem key_item(const WinParams &p, int item) {
  KeyItem it;
  it.stop = item < 0;
  if (it.stop) return it;
  const int slices = p.batch * p.kv_heads;
  const int slice = item % slices, unit = item / slices, sink_units = p.sink_blocks * p.sink_segs;
  int kb, seg;
  if (unit < sink_units) {
    kb = unit / p.sink_segs, seg = unit % p.sink_segs;
  } else {
    kb = p.sink_blocks + (unit - sink_units) / p.norm_segs, seg = (unit - sink_units) % p.norm_segs;
  }
  it.b = slice / p.kv_heads, it.hk = slice % p.kv_heads;
  it.s = sequence(p, it.b);
  it.key0 = kb * kBM;
  block_queries(p, it);
  if (seg >= it.segs) it.rows = 0;
  const int total = it.rows > 0 ? it.per_head * p.group : 0, per = (total + it.segs - 1) / it.segs;
  it.c0 = min(total, seg * per), it.c1 = min(total, it.c0 + per);
  it.slot = it.segs > 1 ? item : -1;
  return it;
}

// S^T, dP^T, dV and dK fill tensor memory at head dim 128, so P^T and dS^T lie
// over the S^T and dP^T they come from, and each of the two takes its turn
// while the other one's products run:
//   tensor core:  dV(i)  S^T(i + 1)  dK(i)  dP^T(i + 1)  dV(i + 1) ...
//   warps:        dS^T(i) -------->  P^T(i + 1) ------>  dS^T(i + 1) ...
// A thread's columns lie over its own, so no warp waits for another one to
// have read: the P^T of columns [kCols e, kCols (e + 1)) takes the first half
// of them.
template <int D>
struct DkvCfg {
  static constexpr uint32_t kTile = kBM * D * 2;
  using R = Roles<D == 64 ? 4 : 2>;
  static constexpr int kStages = D == 128 ? 2 : 4;    // of each ring
  static constexpr uint32_t kQStage = kTile + kAugBytes;  // Q and the rows' panel
  static constexpr uint32_t kSel = 2 * kAugBytes;         // selector panels of -LSE / scale and -D
  // q_full[S] q_empty[S] q_raw[S] do_full[S] do_empty[S] do_raw[S]
  // kv_full kv_free s_full dp_full p_ready ds_ready acc_done acc_free drain
  static constexpr int kNumBars = 6 * kStages + 9;
  static constexpr uint32_t kSmem =
      2 * kTile + kStages * (kQStage + kTile) + kSel + kNumBars * 8 + 64 + ItemRing<KeyItem>::kBytes + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  static constexpr uint32_t kTmS = 0, kTmDP = 128, kTmDV = 256, kTmDK = kTmDV + D;
  static_assert(kTmDK + D <= 512, "TMEM budget");
  // tensor-memory column of the kk-th 16 queries of P^T (or dS^T) within its 128
  static __device__ __forceinline__ constexpr uint32_t p_col(int kk) {
    return 16 * kk / R::kCols * R::kCols + 16 * kk % R::kCols / 2;
  }
};

template <int D, class T>
__global__ void __launch_bounds__(DkvCfg<D>::R::kThreads, 1)
    window_dkdv_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_do,
                       const WinParams p) {
  using C = DkvCfg<D>;
  using R = typename C::R;
  constexpr int kCW = R::kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *k_s = smem, *v_s = smem + C::kTile;
  uint8_t *q_st = smem + 2 * C::kTile;  // [stage]{Q tile, panel}
  uint8_t *do_st = q_st + C::kStages * C::kQStage;
  uint8_t *sel_s = do_st + C::kStages * C::kTile;
  uint64_t *bars = reinterpret_cast<uint64_t *>(sel_s + C::kSel);
  // full, empty, raw of the Q ring, then of the dO ring
  uint64_t *q_full = bars, *q_empty = bars + C::kStages, *q_raw = bars + 2 * C::kStages;
  uint64_t *do_full = bars + 3 * C::kStages, *do_empty = bars + 4 * C::kStages, *do_raw = bars + 5 * C::kStages;
  uint64_t *kv_full = bars + 6 * C::kStages, *kv_free = kv_full + 1;
  uint64_t *s_full = kv_full + 2, *dp_full = kv_full + 3;    // S^T, dP^T of a chunk are in TMEM
  uint64_t *p_ready = kv_full + 4, *ds_ready = kv_full + 5;  // P^T, dS^T written
  uint64_t *acc_done = kv_full + 6, *acc_free = kv_full + 7, *drain = kv_full + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kNumBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  ItemRing<KeyItem> ring(tmem_slot + 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    ring.init(R::kMathWarps + 2);
    for (int i = 0; i < C::kNumBars; ++i) {
      uint64_t *bar = bars + i;
      mbar_init(bar, bar == p_ready || bar == ds_ready || bar == acc_free ? R::kMathWarps : 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == R::kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // selector panels, every row alike: (1, 1, 1, 0, ...) picks -LSE / scale, (0, 0, 0,
  // 1, 1, 1, 0, ...) -D
  for (int c = threadIdx.x; c < (int)(C::kSel / 16); c += blockDim.x) {
    const bool first_half = ((c * 16) % 256) < 128, d_panel = c * 16 >= (int)kAugBytes;
    const uint32_t one = 0x3f80u;  // bf16
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (first_half && !d_panel) w.x = one | one << 16, w.y = one;
    if (first_half && d_panel) w.y = one << 16, w.z = one | one << 16;
    reinterpret_cast<uint4 *>(sel_s)[c] = w;
  }
  fence_proxy_async_cta();
  // window_dq may take the SMs that find no item any more
  asm volatile("griddepcontrol.launch_dependents;");
  const float fac = ds_factor<T>(p, reinterpret_cast<float *>(tmem_slot + 2));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};

  if (warp == R::kProducerWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tmap_q);
      tma_prefetch_desc(&tmap_k);
      tma_prefetch_desc(&tmap_v);
      tma_prefetch_desc(&tmap_do);
      uint32_t ld = 0, items = 0, n = 0;
      // loads begun of each ring; per stage: parity of raw, last load went to raw
      uint32_t q_bits = 0, do_bits = 0, raw_par = 0, raw_last = 0;
      int item = blockIdx.x;
      bool ok = true, asked = false;
      while (true) {
        const KeyItem it = key_item(p, item);
        if (!ring.put(n, it, ctl, kErrBwdWait)) { ok = false; break; }
        if (it.stop) break;
        ring.ask();
        asked = true;
        if (it.c0 == it.c1) {
          if (!ring.take(n, item, ctl, kErrBwdWait)) { ok = false; break; }
          asked = false;
          continue;
        }
        if (!mbar_wait(kv_free, (items & 1) ^ 1, ctl, kErrBwdWait)) { ok = false; break; }
        mbar_arrive_expect_tx(kv_full, 2 * C::kTile);
        load_tile<D>(k_s, &tmap_k, it.s.k0 + it.key0, it.hk, it.s.slice, kv_full);
        load_tile<D>(v_s, &tmap_v, it.s.k0 + it.key0, it.hk, it.s.slice, kv_full);
        ++items;
        for (int c = it.c0; c < it.c1; ++c) {
          const uint32_t st = ld % C::kStages, ph = (ld / C::kStages) & 1, bit = 1u << st;
          const int h = it.hk * p.group + c / it.per_head, first = it.first(c);
          const bool clear = it.clears(c);
          if (!mbar_wait(&q_empty[st], ph ^ 1, ctl, kErrBwdWait)) { ok = false; break; }
          raw_last = clear ? raw_last | bit : raw_last & ~bit;
          if (clear) raw_par ^= bit;
          uint64_t *bar = clear ? &q_raw[st] : &q_full[st];
          mbar_arrive_expect_tx(bar, C::kQStage);
          load_tile<D>(q_st + st * C::kQStage, &tmap_q, it.s.q0 + first, h, it.s.slice, bar);
          bulk_load(q_st + st * C::kQStage + C::kTile, p.aug + (aug_row(p, it.s, it.b, h) + first) / 8 * 256, kAugBytes, bar);
          ++q_bits;
          if (!mbar_wait(&do_empty[st], ph ^ 1, ctl, kErrBwdWait)) { ok = false; break; }
          bar = clear ? &do_raw[st] : &do_full[st];
          mbar_arrive_expect_tx(bar, C::kTile);
          load_tile<D>(do_st + st * C::kTile, &tmap_do, it.s.q0 + first, h, it.s.slice, bar);
          ++do_bits;
          ++ld;
        }
        if (!ok || !ring.take(n, item, ctl, kErrBwdWait)) { ok = false; break; }
        asked = false;
      }
      if (!ok) {
        // let the copies already issued land before the CTA exits
        for (int r = 0; r < 2; ++r) {
          const uint32_t begun = r ? do_bits : q_bits, start = begun > (uint32_t)C::kStages ? begun - C::kStages : 0;
          uint64_t *f = r ? do_full : q_full, *w = r ? do_raw : q_raw;
          for (uint32_t i = start; i < begun; ++i) {
            const uint32_t st = i % C::kStages;
            if (raw_last >> st & 1) drain_wait(&w[st], (raw_par >> st & 1) ^ 1);
            else drain_wait(&f[st], (i / C::kStages) & 1);
          }
        }
        if (items > 0) drain_wait(kv_full, (items - 1) & 1);
        if (item >= 0) ring.discard(n, asked);
      }
    }
  } else if (warp == R::kClearWarp) {
    uint32_t ld = 0, raw_par = 0;
    bool ok = true;
    for (uint32_t n = 0;; ++n) {
      const KeyItem *at = ring.get(n, ok, ctl, kErrBwdWait);
      if (!at) break;
      const KeyItem it = *at;
      ring.release(n, lane);
      for (int c = it.c0; c < it.c1 && ok; ++c, ++ld) {
        if (!it.clears(c)) continue;
        const int valid = it.valid(c), hidden = it.hidden(c);
        const uint32_t st = ld % C::kStages, par = raw_par >> st & 1;
        const int upto = (valid + 15) & ~15;
        ok = mbar_wait_w(&q_raw[st], par, ctl, kErrBwdWait);
        if (!ok) break;
        clear_rows<D>(q_st + st * C::kQStage, 0, hidden, lane);
        clear_rows<D>(q_st + st * C::kQStage, valid, upto, lane);
        if (lane == 0) mbar_arrive(&q_full[st]);
        ok = mbar_wait_w(&do_raw[st], par, ctl, kErrBwdWait);
        raw_par ^= 1u << st;
        if (!ok) break;
        clear_rows<D>(do_st + st * C::kTile, 0, hidden, lane);
        clear_rows<D>(do_st + st * C::kTile, valid, upto, lane);
        if (lane == 0) mbar_arrive(&do_full[st]);
      }
      if (!ok) break;
    }
  } else if (warp == R::kMmaWarp) {
    constexpr uint32_t idesc_ss = idesc_for<T>(kBM, kBM, false, false);
    constexpr uint32_t idesc_aug = idesc_for<__nv_bfloat16>(kBM, kBM, false, false);  // the panels'
    constexpr uint32_t idesc_acc = idesc_for<T>(kBM, D, false, true);
    const uint64_t kd = smem_desc_sw128(smem_u32(k_s), 16, 1024), vd = smem_desc_sw128(smem_u32(v_s), 16, 1024);
    const uint64_t qk0 = smem_desc_sw128(smem_u32(q_st), 16, 1024), qm0 = smem_desc_sw128(smem_u32(q_st), kTilePanel, 1024);
    const uint64_t gk0 = smem_desc_sw128(smem_u32(do_st), 16, 1024), gm0 = smem_desc_sw128(smem_u32(do_st), kTilePanel, 1024);
    const uint64_t sel_l = smem_desc_plain(smem_u32(sel_s), 128, 256);
    const uint64_t sel_d = smem_desc_plain(smem_u32(sel_s) + kAugBytes, 128, 256);
    const uint64_t aug0 = smem_desc_plain(smem_u32(q_st + C::kTile), 128, 256);
    uint32_t ld = 0, items = 0, waits = 0;
    bool ok = true, issued = false;
    auto issue_s = [&](uint32_t st) {  // S^T = K Q^T - LSE / scale
      const uint32_t so = (st * C::kQStage) >> 4;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk / 4) * kTilePanel + (kk % 4) * 32) >> 4;
        mma_ss_w(tmem + C::kTmS, kd + off, qk0 + so + off, idesc_ss, kk > 0 ? 1u : 0u);
      }
      mma_ss_w(tmem + C::kTmS, sel_l, aug0 + so, idesc_aug, 1u);
      mma_commit_w(s_full);
    };
    auto issue_dp = [&](uint32_t st) {  // dP^T = V dO^T - D
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk / 4) * kTilePanel + (kk % 4) * 32) >> 4;
        mma_ss_w(tmem + C::kTmDP, vd + off, gk0 + ((st * C::kTile) >> 4) + off, idesc_ss, kk > 0 ? 1u : 0u);
      }
      mma_ss_w(tmem + C::kTmDP, sel_d, aug0 + ((st * C::kQStage) >> 4), idesc_aug, 1u);
      mma_commit_w(dp_full);
    };
    auto wait_full = [&](uint64_t *full, uint32_t l) -> bool {
      if (!mbar_wait_w(&full[l % C::kStages], (l / C::kStages) & 1, ctl, kErrBwdWait)) return false;
      tc_fence_after();
      return true;
    };
    for (uint32_t rn = 0;; ++rn) {
      const KeyItem *at = ring.get(rn, ok, ctl, kErrBwdWait);
      if (!at) break;
      const KeyItem it = *at;
      ring.release(rn, lane);
      const int n = it.c1 - it.c0;
      if (n == 0) continue;
      if (!mbar_wait_w(kv_full, items & 1, ctl, kErrBwdWait)) { ok = false; break; }
      tc_fence_after();
      if (!wait_full(q_full, ld)) { ok = false; break; }
      issue_s(ld % C::kStages);
      issued = true;
      if (!wait_full(do_full, ld)) { ok = false; break; }
      issue_dp(ld % C::kStages);
      if (n == 1) mma_commit_w(kv_free);
      for (int i = 0; i < n && ok; ++i, ++waits) {
        const uint32_t cur = ld + i, st = cur % C::kStages, st1 = (cur + 1) % C::kStages;
        const bool more = i + 1 < n;
        const int steps = (it.valid(it.c0 + i) + 15) / 16;
        if (more && !wait_full(q_full, cur + 1)) { ok = false; break; }
        if (!mbar_wait_w(p_ready, waits & 1, ctl, kErrBwdWait)) { ok = false; break; }
        if (i == 0 && items > 0 && !mbar_wait_w(acc_free, (items - 1) & 1, ctl, kErrBwdWait)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kBM / 16; ++kk)
          if (kk < steps)
            mma_ts_w(tmem + C::kTmDV, tmem + C::kTmS + C::p_col(kk), gm0 + ((st * C::kTile + kk * 16 * 128) >> 4), idesc_acc,
                     (i > 0 || kk > 0) ? 1u : 0u);
        mma_commit_w(&do_empty[st]);
        if (more) {
          issue_s(st1);  // over the P^T just read
          if (!wait_full(do_full, cur + 1)) { ok = false; break; }
        }
        if (!mbar_wait_w(ds_ready, waits & 1, ctl, kErrBwdWait)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kBM / 16; ++kk)
          if (kk < steps)
            mma_ts_w(tmem + C::kTmDK, tmem + C::kTmDP + C::p_col(kk), qm0 + ((st * C::kQStage + kk * 16 * 128) >> 4), idesc_acc,
                     (i > 0 || kk > 0) ? 1u : 0u);
        mma_commit_w(&q_empty[st]);
        if (more) issue_dp(st1);  // over the dS^T just read
        if (i + 2 == n) mma_commit_w(kv_free);  // K and V are no longer read
      }
      if (!ok) break;
      ld += n;
      mma_commit_w(acc_done);
      ++items;
    }
    if (!ok && issued) {
      mma_commit_w(drain);
      drain_wait(drain, 0);
    }
  } else {
    // elementwise: thread = key row; warpgroup e owns query columns [kCW e, kCW e + kCW) of each chunk
    const int e = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2), shift = make_float2(kPShift<T>, kPShift<T>);
    // dS = P (dP - D), with P's own factor taken out again
    const float ds_mul = kIsHalf<T> ? fac * exp2f(-kPShift<T>) : 1.f;
    const float2 dsm = make_float2(ds_mul, ds_mul);
    const uint32_t s_tm = tmem + lane_off + C::kTmS + kCW * e, d_tm = tmem + lane_off + C::kTmDP + kCW * e;
    uint32_t waits = 0, items = 0;
    bool ok = true;
    for (uint32_t n = 0;; ++n) {
      const KeyItem *at = ring.get(n, ok, ctl, kErrBwdWait);
      if (!at) break;
      const KeyItem it = *at;
      ring.release(n, lane);
      const int key = it.key0 + row, off = it.s.nk - it.s.nq;
      for (int c = it.c0; c < it.c1; ++c, ++waits) {
        const int valid = it.valid(c), qpos = it.first(c) + off;
        // whole: all 128 queries see all 128 keys
        const bool whole = valid == kBM && qpos >= it.key0 + kBM - 1 &&
                           (qpos + kBM - 1 < it.key0 + p.window || it.key0 + kBM <= p.sinks);
        const int c_lo = key - qpos - kCW * e;  // columns below do not see this key
        const int c_hi = min(valid, key < p.sinks ? kBM : min(kBM, key - qpos + p.window)) - kCW * e;
        if (!mbar_wait_w(s_full, waits & 1, ctl, kErrBwdWait)) { ok = false; break; }
        tc_fence_after();
        float2 pr[kCW / 2];
        uint32_t bits[kCW / 32];
        uint32_t r[kCW / 32][32];
#pragma unroll
        for (int g = 0; g < kCW / 32; ++g) tmem_ld32(s_tm + 32 * g, r[g]);
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < kCW / 32; ++g) reg_fence32(r[g]);
#pragma unroll
        for (int g = 0; g < kCW / 32; ++g) {
          bits[g] = whole ? 0xffffffffu : bits_below(c_hi - 32 * g) & ~bits_below(c_lo - 32 * g);
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 sv = make_float2(__uint_as_float(r[g][2 * k]), __uint_as_float(r[g][2 * k + 1]));
            const float2 t = kIsHalf<T> ? fma2(sv, sl2, shift) : mul2(sv, sl2);
            float2 x = make_float2(ex2_approx(t.x), ex2_approx(t.y));
            if (!whole) {
              if (!(bits[g] & (1u << (2 * k)))) x.x = 0.f;
              if (!(bits[g] & (2u << (2 * k)))) x.y = 0.f;
            }
            pr[16 * g + k] = x;
            w[k] = Elem<T>::pack(x.x, x.y);
          }
          tmem_st16(s_tm + 16 * g, w);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(p_ready, lane);
        if (!mbar_wait_w(dp_full, waits & 1, ctl, kErrBwdWait)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < kCW / 32; ++g) tmem_ld32(d_tm + 32 * g, r[g]);
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < kCW / 32; ++g) reg_fence32(r[g]);
#pragma unroll
        for (int g = 0; g < kCW / 32; ++g) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float2 x = mul2(pr[16 * g + k], make_float2(__uint_as_float(r[g][2 * k]), __uint_as_float(r[g][2 * k + 1])));
            if (kIsHalf<T>) x = mul2(x, dsm);
            if (!whole) {
              // what is not seen may be anything, times a P of zero
              if (!(bits[g] & (1u << (2 * k)))) x.x = 0.f;
              if (!(bits[g] & (2u << (2 * k)))) x.y = 0.f;
            }
            w[k] = Elem<T>::pack(x.x, x.y);
          }
          tmem_st16(d_tm + 16 * g, w);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(ds_ready, lane);
      }
      if (!ok) break;
      if (it.rows <= 0) continue;
      const bool any = it.c0 < it.c1;
      if (any) {
        if (!mbar_wait_w(acc_done, items & 1, ctl, kErrBwdWait)) { ok = false; break; }
        tc_fence_after();
      }
      // epilogue: the first half of the warpgroups writes dV, the second half dK, kOut columns each
      constexpr int kHalf = R::kGroups / 2, kOut = D / kHalf;
      static_assert(kOut % 32 == 0, "whole 32-column TMEM loads");
      const int which = e / kHalf, part = e % kHalf;
      const uint32_t col = (which ? C::kTmDK : C::kTmDV) + part * kOut;
      const float mul = which ? p.scale / fac : exp2f(-kPShift<T>);
      const Rows &out = which ? p.dk : p.dv;
      char *dst = out.p + 2 * (it.s.slice * out.b + it.hk * out.h + (long long)(it.s.k0 + (key & ~3)) * out.r + part * kOut);
      const int quad_rows = it.rows - (row & ~3);
      // the parts' sums, four columns of all rows behind one another
      float4 *sums = reinterpret_cast<float4 *>(p.parts) + ((it.slot * 2 + which) * (D / 4) + part * kOut / 4) * kBM + row;
#pragma unroll
      for (int c = 0; c < kOut / 32; ++c) {
        uint32_t r[32];
        if (any) {
          tmem_ld32(tmem + lane_off + col + c * 32, r);
          tmem_ld_wait();
          reg_fence32(r);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = 0u;
        }
        if (it.slot >= 0) {
#pragma unroll
          for (int v = 0; v < 8; ++v)
            sums[(c * 8 + v) * kBM] = make_float4(__uint_as_float(r[4 * v]) * mul, __uint_as_float(r[4 * v + 1]) * mul,
                                                  __uint_as_float(r[4 * v + 2]) * mul, __uint_as_float(r[4 * v + 3]) * mul);
        } else {
          uint4 w[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            auto pair = [&](int i) {
              return Elem<T>::pack(__uint_as_float(r[8 * v + 2 * i]) * mul, __uint_as_float(r[8 * v + 2 * i + 1]) * mul);
            };
            w[v] = make_uint4(pair(0), pair(1), pair(2), pair(3));
          }
          store_quad(w, dst + 64 * c, 2 * out.r, quad_rows, lane);
        }
      }
      if (any) {
        tc_fence_before();
        warp_arrive(acc_free, lane);
        ++items;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == R::kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The parts of a key block added up in order, four columns of a row per thread.
template <int D, class T>
__global__ void __launch_bounds__(256) window_join_kernel(const WinParams p) {
  const int kb = blockIdx.x, slice = blockIdx.y, slices = gridDim.y;
  KeyItem it;
  it.b = slice / p.kv_heads, it.hk = slice % p.kv_heads;
  it.s = sequence(p, it.b);
  it.key0 = kb * kBM;
  block_queries(p, it);
  if (it.rows <= 0 || it.segs == 1) return;
  const bool sink = kb < p.sink_blocks;
  const int unit = sink ? kb * p.sink_segs : p.sink_blocks * p.sink_segs + (kb - p.sink_blocks) * p.norm_segs;
  constexpr int kPer = D / 4;
  for (int i = blockIdx.z * 256 + threadIdx.x; i < 2 * kBM * kPer; i += gridDim.z * 256) {
    const int row = i % kBM, col = i / kBM % kPer, which = i / (kBM * kPer);
    if (row >= it.rows) continue;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int seg = 0; seg < it.segs; ++seg) {
      const long long slot = (long long)(unit + seg) * slices + slice;
      const float4 u = reinterpret_cast<const float4 *>(p.parts)[((slot * 2 + which) * kPer + col) * kBM + row];
      a.x += u.x, a.y += u.y, a.z += u.z, a.w += u.w;
    }
    const Rows &out = which ? p.dk : p.dv;
    char *row_at = out.p + 2 * (it.s.slice * out.b + it.hk * out.h + (long long)(it.s.k0 + it.key0 + row) * out.r);
    *reinterpret_cast<uint2 *>(row_at + 8 * col) =
        make_uint2(Elem<T>::pack(a.x, a.y), Elem<T>::pack(a.z, a.w));
  }
}

// ----------------------------------------------------------------------- 3. dQ
struct QueryItem {
  bool stop;
  Sequence s;
  int h, qb, rows, pos0, base, last, nsink, ns, nc;  // rows: 0 for a block that is not there
  __device__ __forceinline__ void chunk(int j, int &first, int &valid) const {
    first = j < ns ? j * kBM : base + (j - ns) * kBM;
    valid = min(kBM, (j < ns ? nsink : last + 1) - first);
  }
};

// The warpgroups share each chunk of 128 keys (64 or 32 columns each); dS has
// columns of its own.  At head dim 128 S and dP take turns: P is formed while dP
// is being computed, dS while the next chunk's S is.  At head dim 64 the products
// are short and the waits are what counts, so both are handed over at once (2
// sequences of 4096, 16 heads, window 512: 149 against 152 us, dK and dV
// included; at 128, 8192 tokens, 24 heads without a window: 1425 in turns
// against 1562 us).  (Halves of 64 keys, as in window_dkdv, were slower here: 867 against
// 796 us at 8192 tokens, 24 heads, d 128, window 2048, dK and dV included: the
// products of 64 columns run at 60% of the rate, and nothing waits for room.)
template <int D>
struct DqCfg {
  static constexpr uint32_t kTile = kBM * D * 2;
  // Slots of a chunk's K and of its V: K is held until dQ has read it, and the
  // one after the next must be there by then.
  static constexpr int kSlotsK = D == 128 ? 3 : 4, kSlotsV = D == 128 ? 2 : 4, kSlots = kSlotsK + kSlotsV;
  using R = Roles<D == 64 ? 4 : 2>;
  // full[S] empty[S] raw[S] q_full q_free s_full s_read dp_full dp_read ds_ready ds_free acc_done acc_free drain
  static constexpr int kNumBars = 3 * kSlots + 11;
  static constexpr uint32_t kSmem = (2 + kSlots) * kTile + kNumBars * 8 + 64 + ItemRing<QueryItem>::kBytes + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  static constexpr uint32_t kTmS = 0, kTmDP = 128, kTmDS = 256, kTmDQ = 320;
  static_assert(kTmDQ + D <= 512, "TMEM budget");
  static constexpr bool kTurns = D == 128;
  // Load l is K (even) or V (odd) of chunk l / 2 of the CTA's.
  static __device__ __forceinline__ uint32_t slot(uint32_t l) { return l & 1 ? kSlotsK + l / 2 % kSlotsV : l / 2 % kSlotsK; }
  static __device__ __forceinline__ uint32_t phase(uint32_t l) { return l / 2 / (l & 1 ? kSlotsV : kSlotsK) & 1; }
};

__device__ __forceinline__ QueryItem query_item(const WinParams &p, int item) {
  QueryItem it;
  it.stop = item < 0;
  if (it.stop) return it;
  const int slices = p.batch * p.heads, nqb = (p.q_len + kBM - 1) / kBM, slice = item % slices;
  it.qb = nqb - 1 - item / slices;  // the last blocks have the most keys
  it.h = slice % p.heads;
  it.s = sequence(p, slice / p.heads);
  it.rows = max(0, min(kBM, it.s.nq - it.qb * kBM));
  it.pos0 = it.qb * kBM + it.s.nk - it.s.nq;
  it.last = it.rows > 0 ? min(it.s.nk - 1, it.pos0 + it.rows - 1) : -1;
  const int lo = max(0, it.pos0 - p.window + 1);
  it.base = p.sinks >= lo ? 0 : lo;
  it.nsink = min(p.sinks, it.base);
  it.ns = (it.nsink + kBM - 1) / kBM;
  it.nc = it.last >= 0 ? it.ns + (it.last - it.base + kBM) / kBM : 0;
  return it;
}

template <int D, class T>
__global__ void __launch_bounds__(DqCfg<D>::R::kThreads, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_do,
                     const WinParams p) {
  using C = DqCfg<D>;
  using R = typename C::R;
  constexpr int kCW = R::kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *q_s = smem, *do_s = smem + C::kTile, *slots = smem + 2 * C::kTile;
  uint64_t *bars = reinterpret_cast<uint64_t *>(slots + C::kSlots * C::kTile);
  uint64_t *full = bars, *empty = bars + C::kSlots, *raw = bars + 2 * C::kSlots;
  uint64_t *q_full = bars + 3 * C::kSlots, *q_free = q_full + 1;
  uint64_t *s_full = q_full + 2, *s_read = q_full + 3;    // S of a chunk is in TMEM, has been read
  uint64_t *dp_full = q_full + 4, *dp_read = q_full + 5;  // dP
  uint64_t *ds_ready = q_full + 6;                        // dS written
  uint64_t *ds_free = q_full + 7;                         // the dQ products have read it
  uint64_t *acc_done = q_full + 8, *acc_free = q_full + 9, *drain = q_full + 10;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kNumBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  ItemRing<QueryItem> ring(tmem_slot + 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    ring.init(R::kMathWarps + 2);
    for (int i = 0; i < C::kNumBars; ++i) {
      uint64_t *bar = bars + i;
      const bool by_math = bar == s_read || bar == dp_read || bar == ds_ready || bar == acc_free;
      mbar_init(bar, by_math ? R::kMathWarps : 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == R::kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  const float fac = ds_factor<T>(p, reinterpret_cast<float *>(tmem_slot + 2));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};

  if (warp == R::kProducerWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tmap_q);
      tma_prefetch_desc(&tmap_k);
      tma_prefetch_desc(&tmap_v);
      tma_prefetch_desc(&tmap_do);
      uint32_t ld = 0, items = 0, raw_par = 0, raw_last = 0, n = 0;
      int item = blockIdx.x;
      bool ok = true, asked = false;
      while (true) {
        const QueryItem it = query_item(p, item);
        if (!ring.put(n, it, ctl, kErrBwdWait)) { ok = false; break; }
        if (it.stop) break;
        ring.ask();
        asked = true;
        if (it.nc == 0) {
          if (!ring.take(n, item, ctl, kErrBwdWait)) { ok = false; break; }
          asked = false;
          continue;
        }
        if (!mbar_wait(q_free, (items & 1) ^ 1, ctl, kErrBwdWait)) { ok = false; break; }
        mbar_arrive_expect_tx(q_full, 2 * C::kTile);
        load_tile<D>(q_s, &tmap_q, it.s.q0 + it.qb * kBM, it.h, it.s.slice, q_full);
        load_tile<D>(do_s, &tmap_do, it.s.q0 + it.qb * kBM, it.h, it.s.slice, q_full);
        ++items;
        for (int s = 0; s < 2 * it.nc; ++s) {  // K0 V0 K1 V1 ...
          int first, valid;
          it.chunk(s >> 1, first, valid);
          const uint32_t slot = C::slot(ld), bit = 1u << slot;
          if (!mbar_wait(&empty[slot], C::phase(ld) ^ 1, ctl, kErrBwdWait)) { ok = false; break; }
          const bool clear = !(s & 1) && valid % 16 != 0;
          uint64_t *bar = clear ? &raw[slot] : &full[slot];
          raw_last = clear ? raw_last | bit : raw_last & ~bit;
          if (clear) raw_par ^= bit;
          mbar_arrive_expect_tx(bar, C::kTile);
          load_tile<D>(slots + slot * C::kTile, (s & 1) ? &tmap_v : &tmap_k, it.s.k0 + first, it.h / p.group, it.s.slice, bar);
          ++ld;
        }
        if (!ok || !ring.take(n, item, ctl, kErrBwdWait)) { ok = false; break; }
        asked = false;
      }
      if (!ok) {
        const uint32_t start = ld > 2u * C::kSlotsK ? ld - 2 * C::kSlotsK : 0;
        for (uint32_t i = start; i < ld; ++i) {
          const uint32_t slot = C::slot(i);
          if (ld - i > 2u * (i % 2 ? C::kSlotsV : C::kSlotsK)) continue;  // its slot has been loaded again
          if (raw_last >> slot & 1) drain_wait(&raw[slot], (raw_par >> slot & 1) ^ 1);
          else drain_wait(&full[slot], C::phase(i));
        }
        if (items > 0) drain_wait(q_full, (items - 1) & 1);
        if (item >= 0) ring.discard(n, asked);
      }
    }
  } else if (warp == R::kClearWarp) {
    uint32_t ld = 0, raw_par = 0;
    bool ok = true;
    for (uint32_t n = 0;; ++n) {
      const QueryItem *at = ring.get(n, ok, ctl, kErrBwdWait);
      if (!at) break;
      const QueryItem it = *at;
      ring.release(n, lane);
      for (int j = 0; j < it.nc && ok; ++j) {
        int first, valid;
        it.chunk(j, first, valid);
        if (valid % 16 == 0) continue;
        const uint32_t slot = C::slot(ld + 2 * j);
        ok = mbar_wait_w(&raw[slot], raw_par >> slot & 1, ctl, kErrBwdWait);
        raw_par ^= 1u << slot;
        if (!ok) break;
        clear_rows<D>(slots + slot * C::kTile, valid, (valid + 15) & ~15, lane);
        if (lane == 0) mbar_arrive(&full[slot]);
      }
      if (!ok) break;
      ld += 2 * it.nc;
    }
  } else if (warp == R::kMmaWarp) {
    constexpr uint32_t idesc_ss = idesc_for<T>(kBM, kBM, false, false);
    constexpr uint32_t idesc_dq = idesc_for<T>(kBM, D, false, true);
    const uint64_t qd = smem_desc_sw128(smem_u32(q_s), 16, 1024), dod = smem_desc_sw128(smem_u32(do_s), 16, 1024);
    const uint64_t sk0 = smem_desc_sw128(smem_u32(slots), 16, 1024);         // K-major K / V
    const uint64_t sm0 = smem_desc_sw128(smem_u32(slots), kTilePanel, 1024);  // MN-major K
    uint32_t ld = 0, items = 0, ds_waits = 0, r_waits = 0;
    bool ok = true, issued = false;
    auto wait_slot = [&](uint32_t l) -> bool {
      if (!mbar_wait_w(&full[C::slot(l)], C::phase(l), ctl, kErrBwdWait)) return false;
      tc_fence_after();
      return true;
    };
    // S = Q K^T of the K in load l, dP = dO V^T of the V in load l
    auto issue = [&](uint32_t tm, uint64_t a, uint32_t l, uint64_t *done) {
      const uint32_t so = (C::slot(l) * C::kTile) >> 4;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk / 4) * kTilePanel + (kk % 4) * 32) >> 4;
        mma_ss_w(tm, a + off, sk0 + so + off, idesc_ss, kk > 0 ? 1u : 0u);
      }
      if (done) mma_commit_w(done);
    };
    auto issue_s = [&](uint32_t lk) { issue(tmem + C::kTmS, qd, lk, C::kTurns ? s_full : nullptr); };
    auto issue_dp = [&](uint32_t lv) {
      issue(tmem + C::kTmDP, dod, lv, dp_full);
      mma_commit_w(&empty[C::slot(lv)]);  // V is read by dP only
    };
    for (uint32_t n = 0;; ++n) {
      const QueryItem *at = ring.get(n, ok, ctl, kErrBwdWait);
      if (!at) break;
      const QueryItem it = *at;
      ring.release(n, lane);
      if (it.nc == 0) continue;
      if (!mbar_wait_w(q_full, items & 1, ctl, kErrBwdWait)) { ok = false; break; }
      tc_fence_after();
      if (!wait_slot(ld)) { ok = false; break; }
      issue_s(ld);
      issued = true;
      if (!wait_slot(ld + 1)) { ok = false; break; }
      issue_dp(ld + 1);
      if (it.nc == 1) mma_commit_w(q_free);
      for (int j = 0; j < it.nc && ok; ++j) {
        const uint32_t lk = ld + 2 * j, ks = C::slot(lk);
        int first, valid;
        it.chunk(j, first, valid);
        const int steps = (valid + 15) / 16;
        if (j + 1 < it.nc) {
          // the next chunk's S and dP as soon as this chunk's have been read
          if (!wait_slot(lk + 2) || (!C::kTurns && !wait_slot(lk + 3))) { ok = false; break; }
          if (!mbar_wait_w(C::kTurns ? s_read : dp_read, r_waits & 1, ctl, kErrBwdWait)) { ok = false; break; }
          tc_fence_after();
          issue_s(lk + 2);
          if (C::kTurns && (!wait_slot(lk + 3) || !mbar_wait_w(dp_read, r_waits & 1, ctl, kErrBwdWait))) {
            ok = false;
            break;
          }
          ++r_waits;
          tc_fence_after();
          issue_dp(lk + 3);
          if (j + 2 == it.nc) mma_commit_w(q_free);  // Q and dO are no longer read
        }
        if (!mbar_wait_w(ds_ready, ds_waits & 1, ctl, kErrBwdWait)) { ok = false; break; }
        ++ds_waits;
        if (j == 0 && items > 0 && !mbar_wait_w(acc_free, (items - 1) & 1, ctl, kErrBwdWait)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kBM / 16; ++kk)
          if (kk < steps)
            mma_ts_w(tmem + C::kTmDQ, tmem + C::kTmDS + kk * 8, sm0 + ((ks * C::kTile + kk * 16 * 128) >> 4), idesc_dq,
                     (j > 0 || kk > 0) ? 1u : 0u);
        mma_commit_w(&empty[ks]);
        mma_commit_w(ds_free);
      }
      if (!ok) break;
      ld += 2 * it.nc;
      mma_commit_w(acc_done);
      ++items;
    }
    if (!ok && issued) {
      mma_commit_w(drain);
      drain_wait(drain, 0);
    }
  } else {
    // elementwise: thread = query row; warpgroup e owns key columns [kCW e, kCW e + kCW)
    const int e = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2), fac2 = make_float2(fac, fac);
    uint32_t s_waits = 0, items = 0;
    bool ok = true;
    for (uint32_t n = 0;; ++n) {
      const QueryItem *at = ring.get(n, ok, ctl, kErrBwdWait);
      if (!at) break;
      const QueryItem it = *at;
      ring.release(n, lane);
      if (it.rows == 0) continue;
      const int qrow = it.qb * kBM + row;
      float lse2 = 0.f, dd = 0.f;
      if (row < it.rows && it.nc > 0) {
        const long long at_stat = stat_row(p, it.s, it.h, qrow);
        lse2 = p.lse[at_stat] * kLog2e, dd = p.dd[at_stat];
      }
      const float2 nlse2 = make_float2(-lse2, -lse2), ndd = make_float2(-dd, -dd);
      for (int j = 0; j < it.nc; ++j) {
        int first, valid;
        it.chunk(j, first, valid);
        const bool whole = valid == kBM && first + kBM - 1 <= it.pos0 &&
                           (first > it.pos0 + kBM - 1 - p.window || first + kBM <= p.sinks);
        if (!mbar_wait_w(C::kTurns ? s_full : dp_full, s_waits & 1, ctl, kErrBwdWait)) { ok = false; break; }
        ++s_waits;
        tc_fence_after();
        uint32_t r[kCW / 32][32], rd[kCW / 32][32];
        const uint32_t base = tmem + lane_off + kCW * e;
        auto load = [&](uint32_t(&v)[kCW / 32][32], uint32_t tm) {
#pragma unroll
          for (int g = 0; g < kCW / 32; ++g) tmem_ld32(tm + 32 * g, v[g]);
        };
        // the loads are done: what they read may be written once every warp says so
        auto loaded = [&](uint64_t *read) {
          tmem_ld_wait();
#pragma unroll
          for (int g = 0; g < kCW / 32; ++g) {
            if (!C::kTurns || read == s_read) reg_fence32(r[g]);
            if (!C::kTurns || read == dp_read) reg_fence32(rd[g]);
          }
          if (j + 1 < it.nc) {
            tc_fence_before();
            warp_arrive(read, lane);
          }
        };
        load(r, base + C::kTmS);
        if (!C::kTurns) load(rd, base + C::kTmDP);
        loaded(C::kTurns ? s_read : dp_read);
        float2 pr[kCW / 2];
        uint32_t bits[kCW / 32];
#pragma unroll
        for (int g = 0; g < kCW / 32; ++g) {
          bits[g] = whole ? 0xffffffffu : visible_bits(it.pos0 + row, first, valid, p.window, p.sinks, (kCW / 32) * e + g);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 t = fma2(make_float2(__uint_as_float(r[g][2 * k]), __uint_as_float(r[g][2 * k + 1])), sl2, nlse2);
            pr[16 * g + k] = make_float2(ex2_approx(t.x), ex2_approx(t.y));
          }
        }
        if constexpr (C::kTurns) {
          if (!mbar_wait_w(dp_full, (s_waits - 1) & 1, ctl, kErrBwdWait)) { ok = false; break; }
          tc_fence_after();
          load(rd, base + C::kTmDP);
          loaded(dp_read);
        }
        uint32_t pd[kCW / 32][16];
#pragma unroll
        for (int g = 0; g < kCW / 32; ++g)
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 dp = make_float2(__uint_as_float(rd[g][2 * k]), __uint_as_float(rd[g][2 * k + 1]));
            float2 dr = mul2(pr[16 * g + k], add2(dp, ndd));
            if (kIsHalf<T>) dr = mul2(dr, fac2);
            if (!whole) {
              if (!(bits[g] & (1u << (2 * k)))) dr.x = 0.f;
              if (!(bits[g] & (2u << (2 * k)))) dr.y = 0.f;
            }
            pd[g][k] = Elem<T>::pack(dr.x, dr.y);
          }
        if (s_waits > 1) {
          // the dQ products of the chunk before have read its dS
          if (!mbar_wait_w(ds_free, s_waits & 1, ctl, kErrBwdWait)) { ok = false; break; }
          tc_fence_after();
        }
#pragma unroll
        for (int hf = 0; hf < kCW / 32; ++hf) tmem_st16(tmem + lane_off + C::kTmDS + (kCW / 2) * e + 16 * hf, pd[hf]);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(ds_ready, lane);
      }
      if (!ok) break;
      if (it.nc > 0) {
        if (!mbar_wait_w(acc_done, items & 1, ctl, kErrBwdWait)) { ok = false; break; }
        tc_fence_after();
      }
      // warpgroup e < D / 32 writes dQ's columns [32 e, 32 e + 32), then 32 kGroups further
      const float mul = p.scale / fac;
#pragma unroll
      for (int c = 0; c < (D / 32 + R::kGroups - 1) / R::kGroups; ++c) {
        const int col = 32 * (e + c * R::kGroups);
        if (col >= D) break;
        uint32_t r[32];
        if (it.nc > 0) {
          tmem_ld32(tmem + lane_off + C::kTmDQ + col, r);
          tmem_ld_wait();
          reg_fence32(r);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = 0u;
        }
        uint4 w[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          auto pair = [&](int i) {
            return Elem<T>::pack(__uint_as_float(r[8 * v + 2 * i]) * mul, __uint_as_float(r[8 * v + 2 * i + 1]) * mul);
          };
          w[v] = make_uint4(pair(0), pair(1), pair(2), pair(3));
        }
        char *dst = p.dq.p + 2 * (it.s.slice * p.dq.b + it.h * p.dq.h + (long long)(it.s.q0 + (qrow & ~3)) * p.dq.r + col);
        store_quad(w, dst, 2 * p.dq.r, it.rows - (row & ~3), lane);
      }
      if (it.nc > 0) {
        tc_fence_before();
        warp_arrive(acc_free, lane);
        ++items;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == R::kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // this grid does not end before window_dkdv, which may still be running
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D, class T>
cudaError_t launch(const WinParams &p, const CUtensorMap *m, cudaStream_t stream) {
  using K = DkvCfg<D>;
  using Q = DqCfg<D>;
  static std::atomic<uint64_t> done_kv{0}, done_q{0};
  if (const cudaError_t e = allow_shared(window_dkdv_kernel<D, T>, (int)K::kSmem, done_kv)) return e;
  if (const cudaError_t e = allow_shared(window_dq_kernel<D, T>, (int)Q::kSmem, done_q)) return e;
  const int nqb = (p.q_len + kBM - 1) / kBM, nkb = (p.kv_len + kBM - 1) / kBM, slices = p.batch * p.kv_heads;
  if (kIsHalf<T> && p.cu_q)
    if (const cudaError_t e = cudaMemsetAsync(p.norms, 0, (size_t)p.n_norms * 4, stream)) return e;
  if (nqb > 0)
    window_pre_kernel<D, T>
        <<<dim3((p.q_len + pre_rows(D) - 1) / pre_rows(D), p.heads, p.batch + p.zero), 256, 0, stream>>>(p);
  const int kv_items = (p.sink_blocks * p.sink_segs + (nkb - p.sink_blocks) * p.norm_segs) * slices;
  const int q_items = nqb * p.batch * p.heads;
  if (kv_items > 0) window_dkdv_kernel<D, T><<<kv_items, K::R::kThreads, K::kSmem, stream>>>(m[0], m[1], m[2], m[3], p);
  if (q_items > 0) {
    // It needs nothing of window_dkdv, so it starts while that one's last items
    // run (their SMs free up one by one over about an item's time).
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(q_items), cfg.blockDim = dim3(Q::R::kThreads), cfg.dynamicSmemBytes = Q::kSmem, cfg.stream = stream;
    cfg.attrs = &early, cfg.numAttrs = kv_items > 0 ? 1 : 0;
    if (const cudaError_t e = cudaLaunchKernelEx(&cfg, window_dq_kernel<D, T>, m[0], m[1], m[2], m[3], p)) return e;
  }
  const int joined = kv_items == 0 ? 0 : p.norm_segs > 1 ? nkb : p.sink_segs > 1 ? p.sink_blocks : 0;
  if (joined > 0) window_join_kernel<D, T><<<dim3(joined, slices, 2 * kBM * D / 4 / 256), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_backward(const WinParams &p, int type, const CUtensorMap *maps, cudaStream_t stream) {
  if (p.d == 128)
    return type == STA_TYPE_BF16 ? launch<128, __nv_bfloat16>(p, maps, stream)
                                 : launch<128, __half>(p, maps, stream);
  return type == STA_TYPE_BF16 ? launch<64, __nv_bfloat16>(p, maps, stream)
                               : launch<64, __half>(p, maps, stream);
}

}  // namespace sta
