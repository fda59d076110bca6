// split_attn.cu -- attention of a few query rows: the keys are split over the
// warps of a thread block cluster and the parts joined through its shared
// memory.  Serves attention over the 8-bit cache and sliding-window attention of few
// query rows (up to 256 of a key head, by the rule beside its call).
//
// For each query row i with visible keys j: O_i = sum_j P_ij V_j / sum_j P_ij,
// P_ij = 2^(s_ij - m_i).  The query rows of one key head (group x q_len of them,
// kRows per block) are the N side of warp-wide products of 16 keys:
//   S^T[key][row] = K Q^T,   O^T[d][row] += V^T P^T
// in an order of d and of the keys under which a lane's 16-byte pieces of K and V
// are what it multiplies.  Each warp copies its own steps into a ring of its own
// in shared memory (asynchronous copies, several steps ahead: what is in flight
// is not held in registers, and hidden keys arrive as zeros), so no warp waits
// for another one until the join.  8-bit codes widen to fp16, which holds them
// all; a 16-key step lies in one scale block, so its scales are two numbers.  The
// query rows are scaled by a power of two each, so that fp16 holds them as well
// as bf16 did.  Sums, statistics and O are fp32; P is rounded to the operand type,
// which the matrix instructions take.
//
// With one row per sequence the bound is reading the keys: 64 sequences up to
// 8192 tokens, 8 key heads, d 128, e4m3: 121 us for 0.70 GB, 5.8 TB/s (89% of a
// copy's rate; 118 us with one maximum for P and P s).  With 16 rows and d 64 it is
// the latency of a step, one chain of some 300 instructions per warp, most of them
// the widening of the codes and the softmax, on 14 -- 16 warps per SM (32 sequences x
// 4 tokens, 16 heads over 4, window 4096, int8: 31 us for 68 MB, with the issue slots
// 44% busy).  Small calls are latency: 8 us for one token of one sequence over 1031.
#include <cooperative_groups.h>

#include "seq_common.cuh"
#include "sm100_ptx.cuh"

namespace sta {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8, kThreads = 32 * kWarps, kStep = 16;  // keys per step
// P = 2^(x - m) with m set to the maximum less kHead, and moved when a score
// exceeds m by kHead + 8: P stays below 2^15 and the smallest fp16 stands for 2^-31.
// Where the values have scales s, what meets their codes is P s, and it has a
// maximum of its own: 2^(x + log2 s - n), n set and moved like m and held as m - n,
// which stays small.  (With P s over the largest s, a block's values were lost
// beside one of 2^31 their scale, however little weight that one had.)
constexpr float kHead = 7.f;
// m of a row without a key so far: no score is below it
constexpr float kNoMax = -3.4028234663852886e38f;
constexpr float kNoScale = 200.f;
constexpr int kMaxSplits = 16;  // blocks of a cluster

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                         __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 16-bit matrix, a row per 4 lanes, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four codes as two pairs of fp16 numbers.
template <int kType> struct Code16;
template <> struct Code16<STA_TYPE_E4M3> {
  static __device__ __forceinline__ uint32_t prepare(uint32_t w) { return w; }
  static __device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
};
template <> struct Code16<STA_TYPE_INT8> {
  // b ^ 0x80 in the low bits of 1024 is 1024 + b + 128; less 1152 it is b
  static __device__ __forceinline__ uint32_t prepare(uint32_t w) { return w ^ 0x80808080u; }
  static __device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off), y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
    lo = *reinterpret_cast<const uint32_t *>(&x), hi = *reinterpret_cast<const uint32_t *>(&y);
  }
};

// 16 bytes from global to shared memory, zeros where !there
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

// The keys that some query row of a block sees: others are not read, so that
// whatever they hold never meets P = 0.
struct Seen {
  int end, low, sinks;  // below end, and from low on or below sinks
  __device__ __forceinline__ bool operator()(int key) const { return key < end && (key >= low || key < sinks); }
  // all 16 keys of a step
  __device__ __forceinline__ bool whole(int k0) const {
    return k0 + kStep <= end && (k0 >= low || k0 + kStep <= sinks);
  }
};

// Lane (g, c) = (lane / 4, lane % 4) multiplies, of 16 keys: K rows g and g + 8,
// a quarter of d each; V rows 2c, 2c + 1, 2c + 8, 2c + 9, an eighth of d each.
// A step's rows lie in shared memory with their 16-byte pieces exchanged such
// that the lanes of one access touch all banks (8-byte rows of V: half of them).
struct Source {
  const char *k, *v;  // first key
  const float *k_scale, *v_scale;
};

// The 8-bit cache.
template <int D, int kType, class T>
struct CacheKeys {
  using Io = T;
  using Op = __half;
  static constexpr bool kScaled = true;
  CacheAttn a;
  int b, hk, nk, nq;
  static constexpr int kRowBytes = D;
  __device__ __forceinline__ int length(int i) const {
    return min(max(__ldg(a.lengths + i), 0), a.c.table_pages * a.c.page_size);
  }
  __device__ __forceinline__ void open(int slice) {
    b = slice / a.c.kv_heads, hk = slice % a.c.kv_heads, nq = a.q_len;
    nk = length(b);
  }
  __device__ __forceinline__ int batch() const { return a.batch; }
  __device__ __forceinline__ int kv_heads() const { return a.c.kv_heads; }
  __device__ __forceinline__ const char *q_row(int h, int i) const {
    return a.q.p + 2 * (b * a.q.b + h * a.q.h + i * a.q.r);
  }
  __device__ __forceinline__ char *o_row(int h, int i) const { return a.o.p + 2 * (b * a.o.b + h * a.o.h + i * a.o.r); }
  __device__ __forceinline__ float *lse_at(int h, int i) const {
    return a.lse ? a.lse + ((long long)b * a.heads + h) * a.q_len + i : nullptr;
  }
  // Where a step's keys lie, looked up a step before the loads that need it: from
  // the first key of the page on (-1: absent) and of its scales, its place in the
  // table, and the steps before it in the page.
  struct Place {
    long long row, scale;
    int index, in_page;
  };
  __device__ __forceinline__ void look_up(Place &p) const {
    const int page = __ldg(a.c.table + (long long)b * a.c.table_pages + p.index);
    const long long ph = (long long)page * a.c.kv_heads + hk;
    p.row = (unsigned)page < (unsigned)a.c.pages ? ph * a.c.page_size * D : -1;
    p.scale = ph * a.blocks;
  }
  __device__ __forceinline__ Place place(int step) const {
    const int per = a.c.page_size / kStep;
    Place p{-1, 0, step / per, step % per};
    look_up(p);
    return p;
  }
  __device__ __forceinline__ void advance(Place &p) const {
    if (++p.in_page < a.c.page_size / kStep) return;
    p.in_page = 0;
    ++p.index;
    look_up(p);
  }
  static __device__ __forceinline__ constexpr int k_pitch() { return D; }
  static __device__ __forceinline__ constexpr int v_pitch() { return D; }
  __device__ __forceinline__ bool there(const Place &p) const { return p.row >= 0; }
  __device__ __forceinline__ Source source(const Place &p, int) const {
    const int at = p.in_page * kStep;
    const long long row = p.row + at * D, sc = p.scale + (at >> a.block_shift);
    return Source{reinterpret_cast<const char *>(a.c.k + row), reinterpret_cast<const char *>(a.c.v + row),
                  a.c.k_scale + sc, a.c.v_scale + sc};
  }
  // A operand of the s-th 16 columns of d, from 64 bytes' pieces of rows g and g + 8
  static constexpr int kPerPiece = 4;
  static __device__ __forceinline__ void k_frag(const uint32_t (&w)[2][4], int i, uint32_t (&f)[4]) {
    Code16<kType>::widen(Code16<kType>::prepare(w[0][i]), f[0], f[2]);
    Code16<kType>::widen(Code16<kType>::prepare(w[1][i]), f[1], f[3]);
  }
  static __device__ __forceinline__ int k_col(int s, int c) { return 64 * (s / 4) + 16 * c + 4 * (s % 4); }
  // A operand of the t-th 16 rows of V^T
  static __device__ __forceinline__ void v_frag(const uint32_t (&w)[4][kRowBytes / 32], int t, uint32_t (&f)[4]) {
    const uint32_t sel = t % 2 ? 0x7362 : 0x5140;
    Code16<kType>::widen(Code16<kType>::prepare(__byte_perm(w[0][t / 2], w[1][t / 2], sel)), f[0], f[1]);
    Code16<kType>::widen(Code16<kType>::prepare(__byte_perm(w[2][t / 2], w[3][t / 2], sel)), f[2], f[3]);
  }
  static __device__ __forceinline__ int v_col(int t, int g) { return D / 8 * g + 2 * t; }
};

// K and V in the tensors' own type.
template <int D, class T>
struct RowKeys {
  using Io = T;
  using Op = T;
  static constexpr bool kScaled = false;
  WinParams p;
  Sequence s;
  int hk, nk, nq;
  static constexpr int kRowBytes = 2 * D;
  __device__ __forceinline__ int length(int i) const { return sequence(p, i).nk; }
  __device__ __forceinline__ int batch() const { return p.batch; }
  __device__ __forceinline__ int kv_heads() const { return p.kv_heads; }
  __device__ __forceinline__ void open(int slice) {
    hk = slice % p.kv_heads;
    s = sequence(p, slice / p.kv_heads);
    nk = s.nk, nq = s.nq;
  }
  __device__ __forceinline__ const char *q_row(int h, int i) const {
    return p.q.p + 2 * (s.slice * p.q.b + h * p.q.h + (long long)(s.q0 + i) * p.q.r);
  }
  __device__ __forceinline__ char *o_row(int h, int i) const {
    return p.o.p + 2 * (s.slice * p.o.b + h * p.o.h + (long long)(s.q0 + i) * p.o.r);
  }
  __device__ __forceinline__ float *lse_at(int h, int i) const { return p.lse ? p.lse + stat_row(p, s, h, i) : nullptr; }
  struct Place {};
  __device__ __forceinline__ Place place(int) const { return Place{}; }
  __device__ __forceinline__ void advance(Place &) const {}
  __device__ __forceinline__ bool there(const Place &) const { return true; }
  __device__ __forceinline__ Source source(const Place &, int step) const {
    const long long row = s.k0 + step * kStep;
    return Source{p.k.p + 2 * (s.slice * p.k.b + hk * p.k.h + row * p.k.r),
                  p.v.p + 2 * (s.slice * p.v.b + hk * p.v.h + row * p.v.r), nullptr, nullptr};
  }
  __device__ __forceinline__ long long k_pitch() const { return 2 * p.k.r; }
  __device__ __forceinline__ long long v_pitch() const { return 2 * p.v.r; }
  static constexpr int kPerPiece = 2;
  static __device__ __forceinline__ void k_frag(const uint32_t (&w)[2][4], int i, uint32_t (&f)[4]) {
    f[0] = w[0][2 * i], f[2] = w[0][2 * i + 1], f[1] = w[1][2 * i], f[3] = w[1][2 * i + 1];
  }
  static __device__ __forceinline__ int k_col(int s, int c) { return 32 * (s / 2) + 8 * c + 4 * (s % 2); }
  static __device__ __forceinline__ void v_frag(const uint32_t (&w)[4][kRowBytes / 32], int t, uint32_t (&f)[4]) {
    f[0] = __byte_perm(w[0][t], w[1][t], 0x5410), f[1] = __byte_perm(w[0][t], w[1][t], 0x7632);
    f[2] = __byte_perm(w[2][t], w[3][t], 0x5410), f[3] = __byte_perm(w[2][t], w[3][t], 0x7632);
  }
  static __device__ __forceinline__ int v_col(int t, int g) { return 64 * (t / 4) + 8 * g + 2 * (t % 4); }
};

template <int D, int NT, class Keys>
struct SplitCfg {
  static constexpr int kRows = 8 * NT, kPitch = D + 4;
  static constexpr int kHalf = kStep * Keys::kRowBytes;  // K (or V) of a step
  static constexpr int kStage = 2 * kHalf + 16;          // and its two scales
  // CTAs per SM, and steps of a warp's ring: as many as shared memory holds
  static constexpr int kCtas = Keys::kRowBytes == 256 || (NT == 2 && D == 128) ? 1 : 2;
  static constexpr int kFit = (kCtas == 2 ? 100 : 200) * 1024 / (kWarps * kStage), kStages = kFit > 6 ? 6 : kFit;
  static_assert(kStages >= 2, "a step ahead");
  // the join's sums lie over the rings
  static constexpr int kSums = kWarps * kRows * kPitch * 4, kRings = kWarps * kStages * kStage;
  static constexpr int kStats = 4 * kRows * 2 * (kWarps + 1 + kMaxSplits);
  static constexpr int kSmem = (kSums > kRings ? kSums : kRings) + kStats;
};

// Where piece `col` (16 bytes) of row `row` lies.
template <int kRowBytes>
__device__ __forceinline__ int k_place(int row, int col) {
  return row * kRowBytes + 16 * (kRowBytes >= 128 ? col ^ ((row & 1) << 2) : col);
}
template <int kRowBytes>
__device__ __forceinline__ int v_place(int row, int col) {
  return row * kRowBytes + 16 * (kRowBytes >= 128 ? col ^ (row & 6) : col ^ (row & 2));
}

struct SplitShape {
  int splits, group, window, sinks;
  int span;      // keys that the rows of a sequence may see, at most
  bool by_keys;  // slices in the order of their keys, most first
  float scale_log2;
};

// The slice'th slice (sequence and key head) by the keys it reads, most first, so
// that the longest do not start last.  By the whole CTA, for at most kThreads
// sequences; `words` holds kThreads + 1 of them.
template <class Keys>
__device__ __forceinline__ int by_keys(const Keys &keys, int slice, int span, uint32_t *words) {
  const int t = threadIdx.x, n = keys.batch(), want = slice / keys.kv_heads();
  // steps up to 2^23 and the sequence's number: no two are equal
  const uint32_t mine =
      t < n ? (uint32_t)min(min(keys.length(t), span) / kStep + 1, (1 << 23) - 1) << 8 | (uint32_t)(kThreads - 1 - t) : 0u;
  words[t] = mine;
  __syncthreads();
  if (mine) {
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 4) {
      const uint4 w = *reinterpret_cast<const uint4 *>(words + j);  // zeros past the last one
      rank += (w.x > mine) + (w.y > mine) + (w.z > mine) + (w.w > mine);
    }
    if (rank == want) words[kThreads] = t;
  }
  __syncthreads();
  const int b = words[kThreads];
  __syncthreads();  // before anything else is written there
  return b * keys.kv_heads() + slice % keys.kv_heads();
}

// NT groups of 8 query rows.  Grid: (splits x slices, row blocks), a cluster
// per slice.
template <int D, int NT, class Keys>
__global__ void __launch_bounds__(kThreads, SplitCfg<D, NT, Keys>::kCtas)
    split_attn_kernel(const Keys keys_in, const SplitShape shape) {
  using T = typename Keys::Io;
  using Op = typename Keys::Op;
  using C = SplitCfg<D, NT, Keys>;
  constexpr int kRows = C::kRows, kPitch = C::kPitch, kRow = Keys::kRowBytes, kAhead = C::kStages - 1;
  extern __shared__ __align__(16) float smem[];
  float *o_s = smem;                             // [kWarps][kRows][kPitch], over the rings
  float *m_s = reinterpret_cast<float *>(reinterpret_cast<char *>(smem) + (C::kSmem - C::kStats));  // [kWarps][kRows]
  float *l_s = m_s + kWarps * kRows;             // [kWarps][kRows]
  float *cta_m = l_s + kWarps * kRows, *cta_l = cta_m + kRows;
  float *all_m = cta_l + kRows, *all_l = all_m + kMaxSplits * kRows;  // [splits][kRows]
  Keys keys = keys_in;
  const int rank = blockIdx.x % shape.splits;
  int slice = blockIdx.x / shape.splits;
  if (shape.by_keys) slice = by_keys(keys, slice, shape.span, reinterpret_cast<uint32_t *>(smem));
  keys.open(slice);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int group = shape.group, row0 = blockIdx.y * kRows, rows = min(kRows, keys.nq * group - row0);
  // row r is query r / group of head r % group of the key head's
  const int first_pos = row0 / group + keys.nk - keys.nq, last_pos = (row0 + rows - 1) / group + keys.nk - keys.nq;

  // steps of the sinks, then of the window
  int n_steps = 0, sink_steps = 0, base_step = 0;
  Seen seen{0, 0, shape.sinks};
  if (rows > 0 && last_pos >= 0 && keys.nk > 0) {
    const int lo = max(0, first_pos - shape.window + 1);
    base_step = lo / kStep;
    seen.low = lo, seen.end = min(last_pos, keys.nk - 1) + 1;
    sink_steps = min((min(shape.sinks, lo) + kStep - 1) / kStep, base_step);
    n_steps = sink_steps + (seen.end - 1) / kStep - base_step + 1;
  }
  // a warp's steps, one behind another
  const int parts = shape.splits * kWarps, part = rank * kWarps + warp;
  const int begin = (int)((long long)n_steps * part / parts), end = (int)((long long)n_steps * (part + 1) / parts);
  const int skipped = base_step - sink_steps;  // steps between the sinks and the window
  auto step_of = [&](int i) { return i < sink_steps ? i : i + skipped; };

  float o[NT][D / 16][4], m[NT][2], l[NT][2];
  float mn[NT][2];  // m - n, where the values have scales
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = kNoMax, l[nt][0] = l[nt][1] = 0.f;
    mn[nt][0] = mn[nt][1] = 0.f;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) o[nt][t][0] = o[nt][t][1] = o[nt][t][2] = o[nt][t][3] = 0.f;
  }

  char *ring = reinterpret_cast<char *>(smem) + warp * C::kStages * C::kStage;
  const uint32_t ring_at = smem_u32(ring);
  uint32_t here_bits = 0;  // stages whose keys are there
  typename Keys::Place next{};
  // a lane's 16-byte pieces of a step: kPieces to a row, kPass rows apart
  constexpr int kPieces = kRow / 16, kPass = 32 / kPieces;
  const int lane_row = lane / kPieces, lane_col = lane % kPieces;
  const long long k_off = lane_row * keys.k_pitch() + 16 * lane_col, v_off = lane_row * keys.v_pitch() + 16 * lane_col;
  // the copies of the step at i into a stage (a group of them, empty past the end)
  auto fetch = [&](int i, int stage) {
    if (i < end) {
      const int k0 = step_of(i) * kStep;
      if (keys.there(next)) {
        const Source src = keys.source(next, step_of(i));
        const uint32_t at = ring_at + stage * C::kStage;
        const char *k = src.k + k_off, *v = src.v + v_off;
        if (seen.whole(k0)) {
#pragma unroll
          for (int j = 0; j < kStep / kPass; ++j) {
            const int row = lane_row + kPass * j;
            copy16(at + k_place<kRow>(row, lane_col), k + kPass * j * keys.k_pitch(), true);
            copy16(at + C::kHalf + v_place<kRow>(row, lane_col), v + kPass * j * keys.v_pitch(), true);
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < kStep / kPass; ++j) {
            const int row = lane_row + kPass * j;
            const bool there = seen(k0 + row);
            // a row that is not there is not addressed either
            copy16(at + k_place<kRow>(row, lane_col), there ? k + kPass * j * keys.k_pitch() : src.k, there);
            copy16(at + C::kHalf + v_place<kRow>(row, lane_col), there ? v + kPass * j * keys.v_pitch() : src.v, there);
          }
        }
        if (Keys::kScaled && lane < 2) copy4(at + 2 * C::kHalf + 4 * lane, lane ? src.v_scale : src.k_scale);
        here_bits |= 1u << stage;
      } else {
        here_bits &= ~(1u << stage);
      }
      if (i + 1 < end) {
        if (i + 1 == sink_steps) next = keys.place(sink_steps + skipped);
        else keys.advance(next);
      }
    }
    copies_commit();
  };
  int i = begin, ahead = i, stage = 0, into = 0;
  if (i < end) next = keys.place(step_of(i));
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    fetch(ahead, into++);
    ++ahead;
  }
  // Q as the B operand: lane (g, c) holds row g, columns k_col(s, c) .. + 3
  uint32_t qf[NT][D / 16][2];
  float fac[NT][2];  // of this lane's score columns 2c, 2c + 1
  int pos[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = row0 + 8 * nt + g;
    const bool has = 8 * nt + g < rows;
    const char *q = keys.q_row(keys.hk * group + (has ? r % group : 0), has ? r / group : 0);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const uint2 w = has ? *reinterpret_cast<const uint2 *>(q + 2 * Keys::k_col(s, c)) : make_uint2(0u, 0u);
      qf[nt][s][0] = w.x, qf[nt][s][1] = w.y;
    }
    float row_fac = shape.scale_log2;
    if constexpr (Keys::kScaled) {
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 f = Elem<T>::unpack(qf[nt][s][e]);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // largest element into [2^8, 2^9)
      const int exponent = ((__float_as_int(top) >> 23) & 0xff) - 127;
      const int e = top > 0.f && top < INFINITY ? min(max(8 - exponent, -119), 119) : 0;
      const float up = __int_as_float((127 + e) << 23);
      row_fac *= __int_as_float((127 - e) << 23);
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 f = Elem<T>::unpack(qf[nt][s][x]);
          qf[nt][s][x] = Elem<__half>::pack(f.x * up, f.y * up);
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int n = 2 * c + x;
      fac[nt][x] = __shfl_sync(0xffffffffu, row_fac, n * 4);
      pos[nt][x] = 8 * nt + n < rows ? (row0 + 8 * nt + n) / group + keys.nk - keys.nq : -1;
    }
  }

  for (; i < end; ++i) {
    const int step = step_of(i);
    fetch(ahead, into);  // into the stage read last
    ++ahead;
    into = into + 1 == C::kStages ? 0 : into + 1;
    copies_wait<kAhead>();
    __syncwarp();
    const bool here = here_bits >> stage & 1;
    const char *k_s = ring + stage * C::kStage, *v_s = k_s + C::kHalf;
    stage = stage + 1 == C::kStages ? 0 : stage + 1;
    if (here) {
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
      for (int u = 0; u < kRow / 64; ++u) {
        uint32_t w[2][4];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint4 q = *reinterpret_cast<const uint4 *>(k_s + k_place<kRow>(g + 8 * y, c + 4 * u));
          w[y][0] = q.x, w[y][1] = q.y, w[y][2] = q.z, w[y][3] = q.w;
        }
#pragma unroll
        for (int j = 0; j < Keys::kPerPiece; ++j) {
          uint32_t a[4];
          Keys::k_frag(w, j, a);
          const int s = u * Keys::kPerPiece + j;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(x[nt], a, qf[nt][s][0], qf[nt][s][1], Op{});
        }
      }
      float ks = 1.f, vs = 1.f, vs_log = 0.f;
      if constexpr (Keys::kScaled) {
        const float2 f = *reinterpret_cast<const float2 *>(k_s + 2 * C::kHalf);
        ks = f.x, vs = f.y;
        vs_log = __log2f(fabsf(vs));
      }
      // whole: every row sees the 16 keys (rows that are not there are not read)
      const int k0 = step * kStep;
      const bool whole = k0 + kStep - 1 <= first_pos && k0 + kStep <= keys.nk &&
                         (k0 > last_pos - shape.window || k0 + kStep <= shape.sinks);
      bool grows = false;
      float z[NT][4];  // x - m
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 f = mul2(make_float2(fac[nt][0], fac[nt][1]), make_float2(ks, ks));
        float most[2] = {kHead + 8.f, kHead + 8.f};  // above m, or n - log2 s
        if constexpr (Keys::kScaled)
          for (int e = 0; e < 2; ++e) most[e] -= fmaxf(0.f, mn[nt][e] + vs_log);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float2 y = mul2(make_float2(x[nt][e], x[nt][e + 1]), f);
          x[nt][e] = y.x, x[nt][e + 1] = y.y;
          if (!whole) {
            const int key = k0 + g + 4 * e;
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2)
              if (key >= keys.nk || !visible(pos[nt][c2], key, shape.window, shape.sinks)) x[nt][e + c2] = -INFINITY;
          }
          z[nt][e] = x[nt][e] - m[nt][0], z[nt][e + 1] = x[nt][e + 1] - m[nt][1];
          grows = grows || z[nt][e] > most[0] || z[nt][e + 1] > most[1];
        }
      }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(x[nt][e], x[nt][2 + e]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float most = top - kHead;
            top = fmaxf(most, m[nt][e]);
            const float down = m[nt][e] - top;
            float alpha = ex2_approx(down);
            m[nt][e] = top;
            z[nt][e] = x[nt][e] - top, z[nt][2 + e] = x[nt][2 + e] - top;
            l[nt][e] *= alpha;
            if constexpr (Keys::kScaled) {
              // no scale but 0 so far: kNoScale, more than any other
              const float now = fminf(fminf(top - most - vs_log, mn[nt][e] - down), kNoScale);
              alpha = ex2_approx(now - mn[nt][e] + down);
              mn[nt][e] = now;
            }
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[nt][t][e] *= alpha, o[nt][t][2 + e] *= alpha;
          }
      }
      const uint32_t sign = Keys::kScaled && vs < 0.f ? 0x80008000u : 0u;
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          float2 y = make_float2(ex2_approx(z[nt][e]), ex2_approx(z[nt][e + 1]));
          const float2 sum = add2(make_float2(l[nt][0], l[nt][1]), y);
          l[nt][0] = sum.x, l[nt][1] = sum.y;
          if constexpr (Keys::kScaled) {
            y = add2(make_float2(z[nt][e], z[nt][e + 1]), make_float2(mn[nt][0] + vs_log, mn[nt][1] + vs_log));
            y = make_float2(ex2_approx(y.x), ex2_approx(y.y));
          }
          x[nt][e] = y.x, x[nt][e + 1] = y.y;
        }
        pb[nt][0] = transpose8(Elem<Op>::pack(x[nt][0], x[nt][1]) ^ sign);
        pb[nt][1] = transpose8(Elem<Op>::pack(x[nt][2], x[nt][3]) ^ sign);
      }
      uint32_t w[4][kRow / 32];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int row = 2 * c + (y & 1) + 8 * (y >> 1);
        if constexpr (kRow == 64) {
          const uint2 q = *reinterpret_cast<const uint2 *>(v_s + v_place<kRow>(row, g / 2) + 8 * (g & 1));
          w[y][0] = q.x, w[y][1] = q.y;
        } else {
#pragma unroll
          for (int u = 0; u < kRow / 128; ++u) {
            const uint4 q = *reinterpret_cast<const uint4 *>(v_s + v_place<kRow>(row, g + 8 * u));
            w[y][4 * u] = q.x, w[y][4 * u + 1] = q.y, w[y][4 * u + 2] = q.z, w[y][4 * u + 3] = q.w;
          }
        }
      }
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        uint32_t a[4];
        Keys::v_frag(w, t, a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][t], a, pb[nt][0], pb[nt][1], Op{});
      }
    }
    __syncwarp();  // the stage may be copied over
  }
  copies_wait<0>();
  __syncthreads();  // the sums take the rings' place

  // join the warps
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off *= 2) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
      if (g == 0) {
        m_s[warp * kRows + 8 * nt + 2 * c + e] = m[nt][e];
        l_s[warp * kRows + 8 * nt + 2 * c + e] = l[nt][e];
      }
    }
  __syncthreads();
  auto weight = [](float part, float top) { return ex2_approx(part - top); };
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * nt + 2 * c + e;
      float top = kNoMax;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w * kRows + r]);
      float f = m[nt][e] - top;
      if constexpr (Keys::kScaled) f -= mn[nt][e];
      f = ex2_approx(f);
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
        *reinterpret_cast<float2 *>(&o_s[(warp * kRows + r) * kPitch + Keys::v_col(t, g)]) =
            make_float2(o[nt][t][e] * f, o[nt][t][2 + e] * f);
      if (warp == 0 && g == 0) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += l_s[w * kRows + r] * weight(m_s[w * kRows + r], top);
        cta_m[r] = top, cta_l[r] = sum;
      }
    }
  __syncthreads();
  constexpr int kQuads = kRows * D / 4;  // four columns each
  for (int q = threadIdx.x; q < kQuads; q += kThreads) {
    float4 *at = reinterpret_cast<float4 *>(&o_s[q / (D / 4) * kPitch + q % (D / 4) * 4]);
    float4 sum = *at;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 y = at[w * kRows * kPitch / 4];
      sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
    }
    *at = sum;
  }
  // join the cluster: each block finishes its share of the columns, with every
  // block's statistics copied first
  cg::cluster_group cluster = cg::this_cluster();
  const int splits = shape.splits;
  if (splits > 1) {
    cluster.sync();
    for (int x = threadIdx.x; x < kRows * splits; x += kThreads) {
      all_m[x] = *cluster.map_shared_rank(&cta_m[x % kRows], x / kRows);
      all_l[x] = *cluster.map_shared_rank(&cta_l[x % kRows], x / kRows);
    }
  }
  __syncthreads();
  for (int q = threadIdx.x * splits + rank; q < kQuads; q += splits * kThreads) {
    const int r = q / (D / 4), col = q % (D / 4) * 4;
    if (r >= rows) continue;
    float top = kNoMax, sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (splits > 1) {
      for (int x = 0; x < splits; ++x) top = fmaxf(top, all_m[x * kRows + r]);
#pragma unroll 4
      for (int x = 0; x < splits; ++x) {
        const float f = weight(all_m[x * kRows + r], top);
        const float4 z = *reinterpret_cast<float4 *>(cluster.map_shared_rank(&o_s[r * kPitch + col], x));
        sum = fmaf(all_l[x * kRows + r], f, sum);
        y.x = fmaf(z.x, f, y.x), y.y = fmaf(z.y, f, y.y), y.z = fmaf(z.z, f, y.z), y.w = fmaf(z.w, f, y.w);
      }
    } else {
      top = cta_m[r], sum = cta_l[r];
      y = *reinterpret_cast<float4 *>(&o_s[r * kPitch + col]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int h = keys.hk * group + (row0 + r) % group, qi = (row0 + r) / group;
    const bool none = sum == 0.f;
    *reinterpret_cast<uint2 *>(keys.o_row(h, qi) + 2 * col) =
        none ? make_uint2(0u, 0u) : make_uint2(Elem<T>::pack(y.x * inv, y.y * inv), Elem<T>::pack(y.z * inv, y.w * inv));
    if (col == 0)
      if (float *lse = keys.lse_at(h, qi)) *lse = none ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994530942f;
  }
  if (splits > 1) cluster.sync();  // no block leaves while others read its part
}

// Blocks per slice (units: slices and row blocks).  As many as fill the GPU
// once, with a step for each warp; and twice that where the slices are no more
// than the GPU holds and each warp is left 16 steps.  Measured with 1 / 2 / 4 / 8
// / 16 blocks, in us (* chosen):
//   1 x 1031 tokens, d 128, cache:              14.0  11.4   9.4   8.5*  8.6
//   1 x 8192, 16 heads over 4, d 128, bf16:     63.4  36.7  22.3  15.6  12.2*
//   8 x 1024, 24 heads over 8, d 128, bf16:     14.5  12.3* 18.5  36.2  63.4
//   32 x 4096, 4 key heads, d 64, cache:        41.0  32.0* 40.0  57.6   111
//   64 x 1500, 16 heads over 4, d 64, bf16:     17.2* 22.5  32.1  55.2   107
//   32 x up to 8192, 8 key heads, d 128, cache: 87.5  76.3* 88.0
//   64 x up to 8192, 8 key heads, d 128, cache:  124* 136   166   223   378
int splits_for(long long units, long long most_keys, int ctas) {
  const long long steps = (most_keys + kStep - 1) / kStep, room = 148ll * ctas;
  int s = 1;
  while (s < kMaxSplits && ((units * 2 * s <= room && steps >= 2ll * s * kWarps) ||
                            (units * s <= room && steps >= 2ll * s * kWarps * 16)))
    s *= 2;
  return s;
}

// Clusters of 16 blocks, once per device.
template <class Kernel>
cudaError_t allow_wide_clusters(Kernel *kernel, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

template <int D, int NT, class Keys>
cudaError_t launch(const Keys &keys, SplitShape shape, long long slices, int rows, long long longest,
                   cudaStream_t stream) {
  auto *kernel = split_attn_kernel<D, NT, Keys>;
  const long long most_keys = longest < shape.span ? longest : shape.span;
  const int blocks = (rows + 8 * NT - 1) / (8 * NT);
  shape.splits = splits_for(slices * blocks, most_keys, SplitCfg<D, NT, Keys>::kCtas);
  // Sequences in the order of their keys where that shortens the end: more blocks
  // than the GPU holds, but not many rounds of them (the order costs each 1.5 us);
  // keys enough for a difference; and no window that makes most of them equal.
  // Measured as they come / most first, in us, 8 key heads, d 128, cache: 64 x up
  // to 8192 159 / 124, 100 x 3000 89 / 80, 64 x 1000 32 / 30; left as they come:
  // 200 x 1500 89 / 98, 256 x 300 53 / 69, 64 x 8192 with a window of 2000 57 / 60.
  const long long room = 148 * SplitCfg<D, NT, Keys>::kCtas, all = slices * blocks * shape.splits;
  shape.by_keys = shape.by_keys && all > room && all <= 4 * room && most_keys >= 512 && 2ll * shape.span >= longest;
  constexpr size_t smem = SplitCfg<D, NT, Keys>::kSmem;
  static std::atomic<uint64_t> done{0}, wide{0};
  if (const cudaError_t e = allow_shared(kernel, (int)smem, done)) return e;
  if (shape.splits > 8)
    if (const cudaError_t e = allow_wide_clusters(kernel, wide)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(slices * shape.splits), blocks), cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem, cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = shape.splits, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, keys, shape);
}

// Up to 8 rows take one group (64 x up to 8192 above, as they come in two blocks:
// 149 us, with two groups 227; 64 x 1500: 16.9 and 20.7).
template <int D, class Keys>
cudaError_t launch_rows(const Keys &keys, const SplitShape &shape, long long slices, int rows, long long longest,
                        cudaStream_t stream) {
  return rows <= 8 ? launch<D, 1>(keys, shape, slices, rows, longest, stream)
                   : launch<D, 2>(keys, shape, slices, rows, longest, stream);
}

// `uneven`: sequences of lengths that only the device knows.
SplitShape shape_of(int group, long long q_len, int window, int sinks, bool uneven, int batch, float scale_log2) {
  const long long span = window + q_len - 1 + sinks;
  return SplitShape{1, group, window, sinks, (int)(span < 0x7fffffff ? span : 0x7fffffff),
                    uneven && batch > 1 && batch <= kThreads, scale_log2};
}

template <int D, int kType, class T>
cudaError_t cache_launch(const CacheAttn &a, const SplitShape &shape, cudaStream_t stream) {
  CacheKeys<D, kType, T> keys{};
  keys.a = a;
  return launch_rows<D>(keys, shape, (long long)a.batch * a.c.kv_heads, a.q_len * a.group,
                        (long long)a.c.table_pages * a.c.page_size, stream);
}

template <int D, class T>
cudaError_t window_launch(const WinParams &p, const SplitShape &shape, cudaStream_t stream) {
  RowKeys<D, T> keys{};
  keys.p = p;
  return launch_rows<D>(keys, shape, (long long)p.batch * p.kv_heads, p.q_len * p.group, p.kv_len, stream);
}

}  // namespace

cudaError_t launch_cache_attention(const CacheAttn &a, int cache_type, int io_type, cudaStream_t stream) {
  const SplitShape shape = shape_of(a.group, a.q_len, a.window, a.sinks, true, a.batch, a.scale_log2);
  auto io = [&](auto d, auto code) {
    constexpr int D = decltype(d)::value, kType = decltype(code)::value;
    return io_type == STA_TYPE_BF16 ? cache_launch<D, kType, __nv_bfloat16>(a, shape, stream)
                                    : cache_launch<D, kType, __half>(a, shape, stream);
  };
  auto code = [&](auto d) {
    return cache_type == STA_TYPE_E4M3 ? io(d, std::integral_constant<int, STA_TYPE_E4M3>{})
                                       : io(d, std::integral_constant<int, STA_TYPE_INT8>{});
  };
  return a.c.d == 128 ? code(std::integral_constant<int, 128>{}) : code(std::integral_constant<int, 64>{});
}

cudaError_t launch_window_split(const WinParams &p, int type, cudaStream_t stream) {
  const SplitShape shape = shape_of(p.group, p.q_len, p.window, p.sinks, p.cu_q, p.batch, p.scale_log2);
  if (p.d == 128)
    return type == STA_TYPE_BF16 ? window_launch<128, __nv_bfloat16>(p, shape, stream)
                                 : window_launch<128, __half>(p, shape, stream);
  return type == STA_TYPE_BF16 ? window_launch<64, __nv_bfloat16>(p, shape, stream)
                               : window_launch<64, __half>(p, shape, stream);
}

}  // namespace sta
