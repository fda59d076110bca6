// win_fwd.cu -- forward of causal sliding-window attention with sinks on
// 128-row tiles (sm_100a tensor cores).
//
// For each query row i at position pos_i: O_i = sum_j P_ij V_j, P_ij =
// exp(s_ij - LSE_i) over the visible keys j (j <= pos_i, and j > pos_i -
// window or j < sinks), by one pass over the keys with the running maximum and
// sum of the softmax in fp32.
//
//   * A unit is a 128-row query block of one head.  The units of a key head
//     are numbered block by block, the heads of the group within a block, and
//     a work item is two consecutive units (A, B): every key chunk in shared
//     memory serves 256 query rows, with any number of heads per key head.
//     The blocks with the most keys come first, on whichever SM is free.
//   * An item's keys are its sinks, then its window [lo, hi], each in chunks
//     of 128 from its own first key on (TMA rows need no alignment), so no
//     chunk holds keys below every row's window.  Where A and B are blocks of
//     different rows, chunks also end where A's keys end and begin where B's
//     window begins, so that a unit sees all of a chunk's keys or is left out
//     of it: a V row that only the other one sees would reach it as 0 x NaN.
//     Chunks that every row of a unit sees whole take no mask; others apply a
//     128-bit mask per row.
//   * Keys of a chunk past its valid ones (another sequence's, or the future)
//     must not meet P = 0 as NaN: the product P V runs over the valid keys
//     rounded up to 16, and the "clear" warp zeroes the V rows in between.
//   * Warps: 0-3 / 4-7 softmax of A / B (thread = row = TMEM lane), 8 TMA
//     producer, 9 MMA issuer, 10 clear.  S_X = Q_X K^T and O_X += P_X V with P
//     over the first 64 columns of S (tensor memory: S_A, S_B, O_A, O_B); the
//     part of P V whose P is written first is issued before the rest is
//     formed; O is rescaled only when a row's maximum grows by more than 2^8.
// P is rounded to the tensors' type, the precision of the tensor core's A
// operand; statistics and O are fp32 until the final rounding.
//
// Bound by the chain of a chunk pair, S -> softmax -> P V, of which the two units
// hide each other's: about 3900 cycles at head dim 128 (the products alone take
// 2100), and 1.5 pairs more for an item's start and end.  8192 tokens, 24 heads,
// d 128: without a window 414 us (1.0 PFLOP/s, 60% of a library product's rate),
// window 2048 224 us (0.80); window 512, d 64, 2 x 4096 tokens, 16 heads: 61 us.
// (A V of its own for each unit in the chunks that they see different keys of took
// 64 us there, and 150 us instead of 145 for 8192 tokens with a window of 1024,
// where chunks of their own cost 0 -- 2%.)
#include "seq_tile.cuh"

namespace sta {
namespace {

constexpr int kBM = kTileRows;
constexpr int kThreads = 352;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kClearWarp = 10;

struct Item {
  bool stop;
  Sequence s;
  int hk;
  int h[2], qb[2];   // query head and query block of A and B
  bool has[2];
  int pos0[2], lo[2], hi[2];  // position of row 0; first window key; last key (below 0: none)
  int nsink, base, edge, past; // sink keys [0, nsink), window keys [base, edge); only B sees [edge, past)
  int gap, tail;              // chunks apart from the rest: keys [nsink, base + kBM) that only A sees, and [edge, past)
  int ns, nc;                 // sink chunks, chunks
  int n0;                     // split: chunks [0, n0) are warpgroup 0's, [n0, nc) warpgroup 1's
  __device__ __forceinline__ int begin(int x) const { return x ? n0 : 0; }
  __device__ __forceinline__ int end(int x) const { return x ? nc : n0; }
  template <bool kSplit>
  __device__ __forceinline__ void chunk(int j, int &first, int &valid) const {
    first = j < ns ? j * kBM : base + (j - ns) * kBM;
    valid = min(kBM, (j < ns ? nsink : edge) - first);
    if (!kSplit && (j == gap || j == tail)) {
      first = j == gap ? nsink : edge;
      valid = (j == gap ? base + kBM : past) - first;
    }
  }
};

// P = 2^(s - m) with m the maximum less kHead when it last moved: in fp16 P stays
// below 2^15 and the smallest number stands for 2^-31 of the row's largest.
template <class T> constexpr float kHead = std::is_same<T, __half>::value ? 7.f : 0.f;

// The chunks of an item in the order of their loads, K and V, until f(x, chunk,
// is_v) is false.  Shared: K0 V0 K1 V1 ...; split: the first K of each
// warpgroup, then V(j) and K(j + 1) of the one and of the other.
template <bool kSplit, class F>
__device__ __forceinline__ bool for_loads(const Item &it, F &&f) {
  if constexpr (!kSplit) {
    for (int c = 0; c < it.nc; ++c)
      if (!f(0, c, false) || !f(0, c, true)) return false;
  } else {
    for (int j = -1; j < it.n0; ++j)
      for (int x = 0; x < 2; ++x) {
        const int c = it.begin(x) + j, end = it.end(x);
        if (j >= 0 && c < end && !f(x, c, true)) return false;
        if (c + 1 < end && !f(x, c + 1, false)) return false;
      }
  }
  return true;
}

template <int D>
struct Cfg {
  static constexpr uint32_t kTile = kBM * D * 2;
  static constexpr int kSlots = D == 128 ? 4 : 8;  // ring of K and V chunks
  static constexpr uint32_t kTmO = 256;            // O_X at kTmO + X * D; S_X at 128 * X
  static constexpr uint32_t kTmCols = 512;
  static constexpr int kLead = D == 128 ? 96 : 64;  // keys of the first part of P V
  // full[S] empty[S] raw[S] q_full q_free s_full[2] p_ready[2] pv_done[2] o_free[2] drain p_lead[2]
  static constexpr int kNumBars = 3 * kSlots + 13;
  static constexpr uint32_t kSmem = (2 + kSlots) * kTile + kNumBars * 8 + 64 + 4 * kBM * 4 + ItemRing<Item>::kBytes + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

// Whether unit x sees a key of a chunk (hi is below 0 for a unit that is not there).
__device__ __forceinline__ bool sees(const Item &it, int x, int first, int valid, int sinks) {
  return first <= it.hi[x] && (first + valid > it.lo[x] || first < sinks);
}

template <bool kSplit>
__device__ __forceinline__ Item decode(const WinParams &p, int item) {
  Item it;
  it.stop = item < 0;
  if (it.stop) return it;
  const int slices = p.batch * p.kv_heads, nqb = (p.q_len + kBM - 1) / kBM;
  const int per = kSplit ? 1 : 2, rounds = (nqb * p.group + per - 1) / per;  // units of an item, items of a key head
  const int round = rounds - 1 - item / slices, slice = item % slices;  // the last blocks have the most keys
  const int b = slice / p.kv_heads;
  it.hk = slice % p.kv_heads;
  it.s = sequence(p, b);
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int unit = kSplit ? round : 2 * round + x;
    it.qb[x] = unit / p.group;
    it.h[x] = it.hk * p.group + unit % p.group;
    const int rows = min(kBM, it.s.nq - it.qb[x] * kBM);
    it.has[x] = it.qb[x] < nqb && rows > 0;
    it.pos0[x] = it.qb[x] * kBM + it.s.nk - it.s.nq;
    it.lo[x] = max(0, it.pos0[x] - p.window + 1);
    it.hi[x] = it.has[x] ? min(it.s.nk - 1, it.pos0[x] + rows - 1) : -1;
  }
  it.base = p.sinks >= it.lo[0] ? 0 : it.lo[0];
  it.nsink = min(p.sinks, it.base);
  it.edge = it.past = max(it.hi[0], it.hi[1]) + 1;
  it.gap = it.tail = -1;
  // A block of rows each: B's keys end at most 128 behind A's, and its window
  // begins 128 behind A's, where a chunk does, or nearer if the sequence's start
  // or the sinks cut A's.
  const bool two = !kSplit && it.has[1] && it.qb[1] > it.qb[0] && it.hi[0] >= 0, cut = two && it.base == 0 && p.sinks < it.lo[1];
  if (two) it.edge = it.hi[0] + 1;
  if (cut) it.nsink = p.sinks, it.base = it.lo[1] - kBM;
  it.ns = (it.nsink + kBM - 1) / kBM;
  it.nc = it.has[0] && it.past > 0 ? it.ns + (it.edge - it.base + kBM - 1) / kBM + two : 0;
  if (cut) it.gap = it.ns;
  if (two) it.tail = it.nc - 1;
  it.n0 = (it.nc + 1) / 2;
  return it;
}

template <int D, class T, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const WinParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *q_smem = smem, *slots = smem + 2 * C::kTile;
  uint64_t *bars = reinterpret_cast<uint64_t *>(slots + C::kSlots * C::kTile);
  uint64_t *full = bars, *empty = bars + C::kSlots;
  uint64_t *raw = bars + 2 * C::kSlots;  // a V chunk landed whose last rows are still to be cleared
  uint64_t *q_full = bars + 3 * C::kSlots, *q_free = q_full + 1;
  uint64_t *s_full = q_free + 1, *p_ready = s_full + 2, *pv_done = p_ready + 2, *o_free = pv_done + 2;
  uint64_t *drain = o_free + 2, *p_lead = drain + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kNumBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  float *ml_s = reinterpret_cast<float *>(tmem_slot + 16);  // split: m of both warpgroups' rows, then l
  ItemRing<Item> ring(ml_s + 4 * kBM);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    ring.init(10);  // softmax warps, MMA, clear
    for (int i = 0; i < 3 * C::kSlots; ++i) mbar_init(&bars[i], 1);
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_ready[x], 4);
      mbar_init(&p_lead[x], 4);
      mbar_init(&pv_done[x], 1);
      mbar_init(&o_free[x], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, C::kTmCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};

  if (warp == kProducerWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tmap_q);
      tma_prefetch_desc(&tmap_k);
      tma_prefetch_desc(&tmap_v);
      uint32_t ld = 0, items = 0, raw_par = 0, raw_last = 0;  // per slot: parity of raw, last load went to raw
      uint32_t n = 0;
      int item = blockIdx.x;
      bool ok = true, asked = false;
      while (true) {
        const Item it = decode<kSplit>(p, item);
        if (!ring.put(n, it, ctl, kErrWaitProducer)) { ok = false; break; }
        if (it.stop) break;
        ring.ask();
        asked = true;
        if (it.nc == 0) {
          if (!ring.take(n, item, ctl, kErrWaitProducer)) { ok = false; break; }
          asked = false;
          continue;
        }
        if (!mbar_wait(q_free, (items & 1) ^ 1, ctl, kErrWaitProducer)) { ok = false; break; }
        const int n_q = !kSplit && it.has[1] ? 2 : 1;
        mbar_arrive_expect_tx(q_full, n_q * C::kTile);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (x < n_q) load_tile<D>(q_smem + x * C::kTile, &tmap_q, it.s.q0 + it.qb[x] * kBM, it.h[x], it.s.slice, q_full);
        ++items;
        ok = for_loads<kSplit>(it, [&](int, int c, bool is_v) {
          int first, valid;
          it.chunk<kSplit>(c, first, valid);
          const uint32_t slot = ld % C::kSlots, phase = (ld / C::kSlots) & 1, bit = 1u << slot;
          if (!mbar_wait(&empty[slot], phase ^ 1, ctl, kErrWaitProducer)) return false;
          const bool clear = is_v && valid % 16 != 0;
          uint64_t *bar = clear ? &raw[slot] : &full[slot];
          raw_last = clear ? raw_last | bit : raw_last & ~bit;
          if (clear) raw_par ^= bit;
          mbar_arrive_expect_tx(bar, C::kTile);
          load_tile<D>(slots + slot * C::kTile, is_v ? &tmap_v : &tmap_k, it.s.k0 + first, it.hk, it.s.slice, bar);
          ++ld;
          return true;
        });
        if (!ok || !ring.take(n, item, ctl, kErrWaitProducer)) { ok = false; break; }
        asked = false;
      }
      if (!ok) {
        // let the copies already issued land before the CTA exits
        const uint32_t start = ld > (uint32_t)C::kSlots ? ld - C::kSlots : 0;
        for (uint32_t i = start; i < ld; ++i) {
          const uint32_t slot = i % C::kSlots;
          if (raw_last >> slot & 1) drain_wait(&raw[slot], (raw_par >> slot & 1) ^ 1);
          else drain_wait(&full[slot], (i / C::kSlots) & 1);
        }
        if (items > 0) drain_wait(q_full, (items - 1) & 1);
        if (item >= 0) ring.discard(n, asked);
      }
    }
  } else if (warp == kClearWarp) {
    uint32_t ld = 0, raw_par = 0;
    bool ok = true;
    for (uint32_t n = 0;; ++n) {
      const Item *at = ring.get(n, ok, ctl, kErrWaitProducer);
      if (!at) break;
      const Item &it = *at;
      uint32_t l = ld;
      ok = for_loads<kSplit>(it, [&](int, int c, bool is_v) {
        const uint32_t slot = l++ % C::kSlots;
        int first, valid;
        it.chunk<kSplit>(c, first, valid);
        if (!is_v || valid % 16 == 0) return true;
        if (!mbar_wait_w(&raw[slot], raw_par >> slot & 1, ctl, kErrWaitProducer)) return false;
        raw_par ^= 1u << slot;
        clear_rows<D>(slots + slot * C::kTile, valid, (valid + 15) & ~15, lane);
        if (lane == 0) mbar_arrive(&full[slot]);
        return true;
      });
      if (!ok) break;
      ld += 2 * it.nc;
      ring.release(n, lane);
    }
  } else if (warp == kMmaWarp) {
    constexpr uint32_t idesc_qk = idesc_for<T>(kBM, kBM, false, false);
    constexpr uint32_t idesc_pv = idesc_for<T>(kBM, D, false, true);
    const uint32_t slots_addr = smem_u32(slots);
    const uint64_t qdesc0 = smem_desc_sw128(smem_u32(q_smem), 16, 1024);
    const uint64_t kdesc0 = smem_desc_sw128(slots_addr, 16, 1024);
    const uint64_t vdesc0 = smem_desc_sw128(slots_addr, kTilePanel, 1024);
    uint32_t ld = 0, items = 0;
    uint32_t p_waits[2] = {0, 0}, o_waits[2] = {0, 0}, used[2] = {0, 0};
    bool ok = true, issued = false;
    auto mma_s = [&](int x, uint32_t slot) {
      const uint64_t qd = qdesc0 + (((kSplit ? 0 : x) * C::kTile) >> 4), kd = kdesc0 + ((slot * C::kTile) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk / 4) * kTilePanel + (kk % 4) * 32) >> 4;
        mma_ss_w(tmem + 128 * x, qd + off, kd + off, idesc_qk, kk > 0 ? 1u : 0u);
      }
      mma_commit_w(&s_full[x]);
    };
    // O_X += P_X V over the first `steps` groups of 16 keys: the part whose P
    // is written first as soon as it is there, then the rest
    auto mma_pv = [&](int x, uint32_t slot, bool first, uint32_t ph, int steps) -> bool {
      const uint64_t vd = vdesc0 + ((slot * C::kTile) >> 4);
      const uint32_t o_tm = tmem + C::kTmO + x * D, p_tm = tmem + 128 * x;
#pragma unroll
      for (int kk = 0; kk < C::kLead / 16; ++kk)
        if (kk < steps) mma_ts_w(o_tm, p_tm + kk * 8, vd + ((kk * 16 * 128) >> 4), idesc_pv, (first && kk == 0) ? 0u : 1u);
      if (!mbar_wait_w(&p_ready[x], ph, ctl, kErrWaitMma)) return false;
      tc_fence_after();
#pragma unroll
      for (int kk = C::kLead / 16; kk < kBM / 16; ++kk)
        if (kk < steps) mma_ts_w(o_tm, p_tm + kk * 8, vd + ((kk * 16 * 128) >> 4), idesc_pv, 1u);
      mma_commit_w(&pv_done[x]);
      return true;
    };
    auto wait_slot = [&](uint32_t l) -> bool {
      if (!mbar_wait_w(&full[l % C::kSlots], (l / C::kSlots) & 1, ctl, kErrWaitMma)) return false;
      tc_fence_after();
      return true;
    };
    for (uint32_t n = 0;; ++n) {
      const Item *at = ring.get(n, ok, ctl, kErrWaitMma);
      if (!at) break;
      const Item it = *at;
      if (it.nc == 0) {
        ring.release(n, lane);
        continue;
      }
      if (!mbar_wait_w(q_full, items & 1, ctl, kErrWaitMma)) { ok = false; break; }
      tc_fence_after();
      ++items;
      const uint32_t k0 = ld;
      bool begun[2] = {false, false};
      // P V of unit x's chunk whose V is in `slot`
      auto attend = [&](int x, uint32_t slot, int steps) -> bool {
        const uint32_t ph = p_waits[x] & 1;
        ++p_waits[x];
        if (!mbar_wait_w(&p_lead[x], ph, ctl, kErrWaitMma)) return false;
        tc_fence_after();
        if (!begun[x] && used[x] > 0) {
          // the epilogue of the previous item here has read O_X
          if (!mbar_wait_w(&o_free[x], o_waits[x] & 1, ctl, kErrWaitMma)) return false;
          ++o_waits[x];
          tc_fence_after();
        }
        const bool first = !begun[x];
        begun[x] = true;
        return mma_pv(x, slot, first, ph, steps);
      };
      if constexpr (!kSplit) {
        if (!wait_slot(k0)) { ok = false; break; }
        int first, valid;
        it.chunk<kSplit>(0, first, valid);
        bool act[2] = {sees(it, 0, first, valid, p.sinks), sees(it, 1, first, valid, p.sinks)};
        issued = true;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (act[x]) mma_s(x, k0 % C::kSlots);
        mma_commit_w(&empty[k0 % C::kSlots]);
        if (it.nc == 1) mma_commit_w(q_free);
        for (int j = 0; j < it.nc && ok; ++j) {
          const uint32_t vj = k0 + 2 * j + 1, kn = vj + 1;
          const bool more = j + 1 < it.nc;
          const int steps = (valid + 15) / 16;
          it.chunk<kSplit>(j + 1, first, valid);
          const bool next[2] = {more && sees(it, 0, first, valid, p.sinks), more && sees(it, 1, first, valid, p.sinks)};
          if (!wait_slot(vj) || (more && !wait_slot(kn))) { ok = false; break; }
  #pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (act[x]) {
              if (!attend(x, vj % C::kSlots, steps)) { ok = false; break; }
            }
            act[x] = next[x];
            if (act[x]) mma_s(x, kn % C::kSlots);
          }
          if (!ok) break;
          mma_commit_w(&empty[vj % C::kSlots]);
          if (more) mma_commit_w(&empty[kn % C::kSlots]);
          if (j + 2 == it.nc) mma_commit_w(q_free);
        }
      } else {
        uint32_t l = k0;
        int s_left = it.nc;
        // S of warpgroup x's next chunk from its K, which is load l
        auto score = [&](int x) -> bool {
          if (!wait_slot(l)) return false;
          mma_s(x, l % C::kSlots);
          issued = true;
          mma_commit_w(&empty[l++ % C::kSlots]);
          if (--s_left == 0) mma_commit_w(q_free);
          return true;
        };
        ok = score(0) && (it.n0 == it.nc || score(1));
        for (int j = 0; j < it.n0 && ok; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int c = it.begin(x) + j;
            if (c >= it.end(x)) continue;
            int first, valid;
            it.chunk<kSplit>(c, first, valid);
            const uint32_t vl = l++;
            // the next K, too, while the softmax works
            if (!wait_slot(vl) || (c + 1 < it.end(x) && !wait_slot(l)) || !attend(x, vl % C::kSlots, (valid + 15) / 16)) {
              ok = false;
              break;
            }
            mma_commit_w(&empty[vl % C::kSlots]);
            if (c + 1 < it.end(x) && !score(x)) { ok = false; break; }
          }
      }
      if (!ok) break;
      ld = k0 + 2 * it.nc;
      ring.release(n, lane);
#pragma unroll
      for (int x = 0; x < 2; ++x) used[x] += begun[x] ? 1 : 0;
    }
    if (!ok && issued) {
      mma_commit_w(drain);
      drain_wait(drain, 0);
    }
  } else {
    // softmax warpgroup x: row `row` of unit x
    const int x = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_off + 128 * x, o_tm = tmem + lane_off + C::kTmO + x * D;
    const float sl2 = p.scale_log2;
    uint32_t s_waits = 0;
    bool ok = true;
    for (uint32_t n = 0;; ++n) {
      const Item *at = ring.get(n, ok, ctl, kErrWaitSoftmax);
      // The warpgroups of a split item meet at its end, at barriers without a
      // limit: they begin it together or not at all (a wait of one warp may run
      // out before the item is there, and another one's find it).
      if (kSplit && !named_bar_and(1, 256, at != nullptr)) break;
      if (!at) break;
      const Item &it = *at;  // stays in shared memory: beside a row of scores registers are short
      const int u = kSplit ? 0 : x;  // its unit
      if (!it.has[u]) {
        ring.release(n, lane);
        continue;
      }
      float m = -INFINITY, l = 0.f;
      bool seen = false;
      for (int j = kSplit ? it.begin(x) : 0; j < (kSplit ? it.end(x) : it.nc); ++j) {
        int first, valid;
        it.chunk<kSplit>(j, first, valid);
        if (!kSplit && !sees(it, x, first, valid, p.sinks)) continue;
        // whole: every row of the unit sees all 128 keys
        const int pos0 = it.pos0[u];
        const bool whole = valid == kBM && first + kBM - 1 <= pos0 &&
                           (first > pos0 + kBM - 1 - p.window || first + kBM <= p.sinks);
        if (!mbar_wait_w(&s_full[x], s_waits & 1, ctl, kErrWaitSoftmax)) { ok = false; break; }
        ++s_waits;
        tc_fence_after();
        // O_X holds every chunk before this one: S was issued after their P V
        auto mask = [&](uint32_t(&r)[32], int w) {
          if (whole) return;
          const uint32_t bits = visible_bits(pos0 + row, first, valid, p.window, p.sinks, w);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(bits & (1u << i))) r[i] = 0xff800000u;  // -inf
        };
        // The row maximum takes all 128 scores; the second half is then read
        // from tensor memory again while P of the second quarter is formed: held
        // throughout, the scores would not fit (272 us where this takes 222, 8190
        // tokens, 24 heads, d 128, window 2048).
        uint32_t r0[32], r1[32];
        float mloc;
        {
          uint32_t r2[32], r3[32];
          auto top = [](float t, const uint32_t(&r)[32]) {
            float a = max3(t, __uint_as_float(r[0]), __uint_as_float(r[1]));
            float b = max3(__uint_as_float(r[2]), __uint_as_float(r[3]), __uint_as_float(r[4]));
#pragma unroll
            for (int i = 5; i < 29; i += 4) {
              a = max3(a, __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
              b = max3(b, __uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]));
            }
            a = max3(a, __uint_as_float(r[29]), __uint_as_float(r[30]));
            return max3(a, b, __uint_as_float(r[31]));
          };
          tmem_ld32(s_tm + 64, r2);
          tmem_ld32(s_tm + 96, r3);
          tmem_ld_wait();
          reg_fence32(r2);
          reg_fence32(r3);
          tmem_ld32(s_tm, r0);
          mask(r2, 2);
          float t = top(-INFINITY, r2);
          tmem_ld32(s_tm + 32, r1);
          mask(r3, 3);
          t = top(t, r3);
          tmem_ld_wait();
          reg_fence32(r0);
          reg_fence32(r1);
          mask(r0, 0);
          t = top(t, r0);
          mask(r1, 1);
          mloc = top(t, r1) * sl2;
        }
        const bool resc = mloc > m + (kHead<T> + 8.0f);  // also the first finite maximum
        const float m_new = resc ? mloc - kHead<T> : m;
        const float alpha = resc ? ex2_approx(m - m_new) : 1.f;
        const bool warp_resc = __any_sync(0xffffffffu, resc) && seen;
        m = m_new;
        const float ms = m == -INFINITY ? 0.f : m;  // a row without a visible key so far: P = 0
        const float2 sl2x2 = make_float2(sl2, sl2), nms = make_float2(-ms, -ms);
        float2 ls[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) ls[a] = make_float2(0.f, 0.f);
        // P of 32 keys from their scores: written over S, added to the row sum
        auto form = [&](const uint32_t(&r)[32], int c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x = fma2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), sl2x2, nms);
            const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            ls[i & 3] = add2(ls[i & 3], e);
            pk[i] = Elem<T>::pack(e.x, e.y);
          }
          tmem_st16(s_tm + c * 16, pk);
        };
        auto lead = [&]() {
          tmem_st_wait();
          tc_fence_before();
          warp_arrive(&p_lead[x], lane);
        };
        form(r0, 0);
        uint32_t r2[32], r3[32];
        tmem_ld32(s_tm + 64, r2);
        tmem_ld32(s_tm + 96, r3);
        form(r1, 1);
        if (warp_resc) {
#pragma unroll 1
          for (int oc = 0; oc < D / 16; ++oc) {
            uint32_t r[16];
            tmem_ld16(o_tm + oc * 16, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
            tmem_st16(o_tm + oc * 16, r);
          }
        }
        if constexpr (C::kLead == 64) lead();
        tmem_ld_wait();
        reg_fence32(r2);
        reg_fence32(r3);
        mask(r2, 2);
        form(r2, 2);
        if constexpr (C::kLead == 96) lead();
        mask(r3, 3);
        form(r3, 3);
        const float2 sum = add2(add2(ls[0], ls[1]), add2(ls[2], ls[3]));
        l = l * alpha + (sum.x + sum.y);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&p_ready[x], lane);
        seen = true;
      }
      if (!kSplit && !ok) break;
      if (seen && ok) {
        // one P V per chunk so far: the last one's phase
        ok = mbar_wait_w(&pv_done[x], (s_waits - 1) & 1, ctl, kErrWaitEpilogue);
        tc_fence_after();
      }
      if (!kSplit && !ok) break;
      const int qrow = it.qb[u] * kBM + row;
      const bool row_valid = qrow < it.s.nq;
      float f[2] = {1.f, 0.f};  // split: the weights of the two partial O
      if constexpr (kSplit) {
        // join the two halves of the keys: each warpgroup writes half of the columns
        ml_s[x * kBM + row] = m, ml_s[(2 + x) * kBM + row] = l;
        ok = named_bar_and(1, 256, ok);
        if (!ok) break;
        tc_fence_after();
        const float m0 = ml_s[row], m1 = ml_s[kBM + row], top = fmaxf(m0, m1);
        f[0] = m0 == -INFINITY ? 0.f : ex2_approx(m0 - top), f[1] = m1 == -INFINITY ? 0.f : ex2_approx(m1 - top);
        m = top, l = ml_s[2 * kBM + row] * f[0] + ml_s[3 * kBM + row] * f[1];
      }
      const bool none = l == 0.f;
      const float inv_l = none ? 0.f : 1.f / l;
      f[0] *= inv_l, f[1] *= inv_l;
      // rows outside the sequences have been cleared
      asm volatile("griddepcontrol.wait;" ::: "memory");
      // the quad's first row, and how many of its rows there are
      char *dst = p.o.p + 2 * ((long long)it.s.slice * p.o.b + (long long)it.h[u] * p.o.h +
                               (long long)(it.s.q0 + (qrow & ~3)) * p.o.r);
      const int quad_rows = it.s.nq - (qrow & ~3);
      constexpr int kOut = kSplit ? D / 2 : D;  // columns of this warpgroup
      const uint32_t from = tmem + lane_off + C::kTmO + (kSplit ? x * kOut : x * D);
#pragma unroll
      for (int c = 0; c < kOut / 32; ++c) {
        uint32_t r[32], r1[32];
        if (kSplit ? it.nc > 0 : seen) tmem_ld32(from + c * 32, r);
        if (kSplit && it.nc > it.n0) tmem_ld32(from + D + c * 32, r1);
        tmem_ld_wait();
        reg_fence32(r);
        if constexpr (kSplit) {
          reg_fence32(r1);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float y = __uint_as_float(r[i]) * f[0];
            if (it.nc > it.n0) y = fmaf(__uint_as_float(r1[i]), f[1], y);
            r[i] = __float_as_uint(y);
          }
        }
        uint4 w[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          auto pair = [&](int e) {
            const float k = kSplit ? 1.f : f[0];
            return none ? 0u : Elem<T>::pack(__uint_as_float(r[8 * v + 2 * e]) * k, __uint_as_float(r[8 * v + 2 * e + 1]) * k);
          };
          w[v] = make_uint4(pair(0), pair(1), pair(2), pair(3));
        }
        store_quad(w, dst + 64 * c + (kSplit ? 2 * x * kOut : 0), 2 * p.o.r, quad_rows, lane);
      }
      if (kSplit) {
        tc_fence_before();
        named_bar_sync(2, 256);  // both warpgroups have read both O, m and l
      }
      if (seen) {
        tc_fence_before();
        warp_arrive(&o_free[x], lane);
      }
      if (row_valid && p.lse && (!kSplit || x == 0))
        p.lse[stat_row(p, it.s, it.h[u], qrow)] = none ? -INFINITY : (m + __log2f(l)) * 0.69314718055994530942f;
      ring.release(n, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmCols);
  }
  // this grid does not end before window_clear
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A warp per 32 rows.
__global__ void __launch_bounds__(256) window_clear_kernel(const WinParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i * 32ll < p.q_rows) clear_outside(p.cu_q, p.batch, p.q_rows, p.q_len, i, p.heads, p.d, p.o, Rows{}, p.lse);
}

template <int D, class T, bool kSplit>
cudaError_t launch_mode(const WinParams &p, const CUtensorMap *maps, long long items, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  if (const cudaError_t e = allow_shared(window_fwd_kernel<D, T, kSplit>, (int)Cfg<D>::kSmem, done)) return e;
  // beside window_clear: only its stores wait for that
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)items), cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::kSmem, cfg.stream = stream;
  cfg.attrs = &early, cfg.numAttrs = p.zero ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, window_fwd_kernel<D, T, kSplit>, maps[0], maps[1], maps[2], p);
}

// Pairs of units share their keys; where one round of the GPU has room for
// every unit on its own, the two warpgroups take half of its keys each.
// Measured, pairs / halves, in us (24 heads over 8, d 128, window 1024): 72 units
// 30 / 23, 144 units 31 / 25, 168 units 31 / 38, 288 units 33 / 41; 16 heads, d 64,
// no window: 128 units 71 / 47, 176 units 72 / 77.
template <int D, class T>
cudaError_t launch(const WinParams &p, const CUtensorMap *maps, cudaStream_t stream) {
  const long long units = (long long)((p.q_len + kBM - 1) / kBM) * p.group, slices = (long long)p.batch * p.kv_heads;
  if (units * slices <= 148) return launch_mode<D, T, true>(p, maps, units * slices, stream);
  return launch_mode<D, T, false>(p, maps, (units + 1) / 2 * slices, stream);
}

}  // namespace

cudaError_t launch_window_clear(const WinParams &p, cudaStream_t stream) {
  window_clear_kernel<<<(unsigned)((p.q_rows + 255ll) / 256), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_window_tiles(const WinParams &p, int type, const CUtensorMap *maps, cudaStream_t stream) {
  if (p.d == 128)
    return type == STA_TYPE_BF16 ? launch<128, __nv_bfloat16>(p, maps, stream)
                                 : launch<128, __half>(p, maps, stream);
  return type == STA_TYPE_BF16 ? launch<64, __nv_bfloat16>(p, maps, stream)
                               : launch<64, __half>(p, maps, stream);
}

}  // namespace sta
