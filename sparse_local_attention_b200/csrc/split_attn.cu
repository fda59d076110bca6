// split_attn.cu -- attention of a few query rows: the keys are split over the
// warps of a thread block cluster and the parts joined through its shared
// memory.  Serves attention over the 8-bit cache and the single-token form of
// sliding-window attention.
//
// Bound by reading the keys and values once.  The query rows of one key head
// (group x q_len of them, kRows per block) are the N side of warp-wide
// products of 16 keys:
//   S^T[key][row] = K Q^T,   O^T[d][row] += V^T P^T
// so that K and V go from global memory straight into the A operand's
// registers, in an order of d and of the keys under which each lane's 16-byte
// loads are what it multiplies: nothing is staged in shared memory and no warp
// waits for another one until the join.  8-bit codes widen to fp16, which holds
// them all; a 16-key step lies in one scale block, so its scales are two
// numbers per warp.  The query rows are scaled by a power of two each, so that
// fp16 holds them as well as bf16 did.  Sums, statistics and O are fp32, P is
// rounded to the operand type.
#include <cooperative_groups.h>

#include "seq_common.cuh"
#include "sm100_ptx.cuh"

namespace sta {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8, kThreads = 32 * kWarps, kStep = 16;  // keys per step
// P = 2^(x - m) with m set to the maximum less kHead, and moved when a score
// exceeds m by kHead + 8: P stays below 2^15 and the smallest fp16 stands for 2^-31.
constexpr float kHead = 7.f;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16) {
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

// Two codes (bits 0..15) as fp16, times Code16::kUnit.
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

template <int kWords>
__device__ __forceinline__ void load_words(uint32_t *dst, const void *src) {
  if constexpr (kWords == 4) {
    const uint4 w = __ldg(static_cast<const uint4 *>(src));
    dst[0] = w.x, dst[1] = w.y, dst[2] = w.z, dst[3] = w.w;
  } else {
    const uint2 w = __ldg(static_cast<const uint2 *>(src));
    dst[0] = w.x, dst[1] = w.y;
  }
}

// The keys that some query row of a block sees: others are not read, so that
// whatever they hold never meets P = 0.
struct Seen {
  int end, low, sinks;  // below end, and from low on or below sinks
  __device__ __forceinline__ bool operator()(int key) const { return key < end && (key >= low || key < sinks); }
};

// Lane (g, c) = (lane / 4, lane % 4) holds, of 16 keys: K rows g and g + 8,
// a quarter of d each; V rows 2c, 2c + 1, 2c + 8, 2c + 9, an eighth of d each.

// The 8-bit cache.
template <int D, int kType, class T>
struct CacheKeys {
  using Io = T;
  using Op = __half;
  static constexpr bool kScaled = true;
  CacheAttn a;
  int b, hk, nk, nq;
  struct Raw {
    uint32_t k[2][D / 16], v[4][D / 32];
    float ks, vs;
  };
  __device__ __forceinline__ void open(int slice) {
    b = slice / a.c.kv_heads, hk = slice % a.c.kv_heads, nq = a.q_len;
    nk = min(max(__ldg(a.lengths + b), 0), a.c.table_pages * a.c.page_size);
  }
  __device__ __forceinline__ const char *q_row(int h, int i) const {
    return a.q.p + 2 * (b * a.q.b + h * a.q.h + i * a.q.r);
  }
  __device__ __forceinline__ char *o_row(int h, int i) const { return a.o.p + 2 * (b * a.o.b + h * a.o.h + i * a.o.r); }
  __device__ __forceinline__ float *lse_at(int h, int i) const {
    return a.lse ? a.lse + ((long long)b * a.heads + h) * a.q_len + i : nullptr;
  }
  // the page of a step, looked up a step before its loads
  __device__ __forceinline__ int place(int step) const { return page_of(a.c, b, step * kStep); }
  __device__ __forceinline__ bool there(int page) const { return page >= 0; }
  __device__ __forceinline__ void load(Raw &r, int page, int step, const Seen &seen, int g, int c) const {
    const int k0 = step * kStep, at = k0 % a.c.page_size;
    const bool here = page >= 0;
    const long long row = ((long long)page * a.c.kv_heads + hk) * a.c.page_size + at;
    const long long sc = ((long long)page * a.c.kv_heads + hk) * (a.c.page_size / a.c.block) + at / a.c.block;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
        if (here && seen(k0 + g + 8 * x)) load_words<4>(&r.k[x][4 * u], a.c.k + (row + g + 8 * x) * D + 16 * c + 64 * u);
        else r.k[x][4 * u] = r.k[x][4 * u + 1] = r.k[x][4 * u + 2] = r.k[x][4 * u + 3] = 0u;
      }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int key = 2 * c + (x & 1) + 8 * (x >> 1);
      if (here && seen(k0 + key)) load_words<D / 32>(r.v[x], a.c.v + (row + key) * D + D / 8 * g);
      else
#pragma unroll
        for (int j = 0; j < D / 32; ++j) r.v[x][j] = 0u;
    }
    r.ks = here ? __ldg(a.c.k_scale + sc) : 0.f;
    r.vs = here ? __ldg(a.c.v_scale + sc) : 0.f;
  }
  // A operand of the s-th 16 columns of d
  static __device__ __forceinline__ void k_frag(const Raw &r, int s, uint32_t (&f)[4]) {
    Code16<kType>::widen(Code16<kType>::prepare(r.k[0][s]), f[0], f[2]);
    Code16<kType>::widen(Code16<kType>::prepare(r.k[1][s]), f[1], f[3]);
  }
  static __device__ __forceinline__ int k_col(int s, int c) { return 64 * (s / 4) + 16 * c + 4 * (s % 4); }
  // A operand of the t-th 16 rows of V^T
  static __device__ __forceinline__ void v_frag(const Raw &r, int t, uint32_t (&f)[4]) {
    const int j = t / 2;
    const uint32_t sel = t % 2 ? 0x7362 : 0x5140;
    Code16<kType>::widen(Code16<kType>::prepare(__byte_perm(r.v[0][j], r.v[1][j], sel)), f[0], f[1]);
    Code16<kType>::widen(Code16<kType>::prepare(__byte_perm(r.v[2][j], r.v[3][j], sel)), f[2], f[3]);
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
  struct Raw {
    uint32_t k[2][D / 8], v[4][D / 16];
  };
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
  __device__ __forceinline__ int place(int) const { return 0; }
  __device__ __forceinline__ bool there(int) const { return true; }
  __device__ __forceinline__ void load(Raw &r, int, int step, const Seen &seen, int g, int c) const {
    const int k0 = step * kStep;
    const long long row = s.k0 + k0;
    const char *k = p.k.p + 2 * (s.slice * p.k.b + hk * p.k.h + row * p.k.r);
    const char *v = p.v.p + 2 * (s.slice * p.v.b + hk * p.v.h + row * p.v.r);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int u = 0; u < D / 32; ++u) {
        if (seen(k0 + g + 8 * x)) load_words<4>(&r.k[x][4 * u], k + 2 * (g + 8 * x) * p.k.r + 16 * c + 64 * u);
        else r.k[x][4 * u] = r.k[x][4 * u + 1] = r.k[x][4 * u + 2] = r.k[x][4 * u + 3] = 0u;
      }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int key = 2 * c + (x & 1) + 8 * (x >> 1);
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
        if (seen(k0 + key)) load_words<4>(&r.v[x][4 * u], v + 2 * key * p.v.r + 16 * g + 128 * u);
        else r.v[x][4 * u] = r.v[x][4 * u + 1] = r.v[x][4 * u + 2] = r.v[x][4 * u + 3] = 0u;
      }
    }
  }
  static __device__ __forceinline__ void k_frag(const Raw &r, int s, uint32_t (&f)[4]) {
    f[0] = r.k[0][2 * s], f[2] = r.k[0][2 * s + 1], f[1] = r.k[1][2 * s], f[3] = r.k[1][2 * s + 1];
  }
  static __device__ __forceinline__ int k_col(int s, int c) { return 32 * (s / 2) + 8 * c + 4 * (s % 2); }
  static __device__ __forceinline__ void v_frag(const Raw &r, int t, uint32_t (&f)[4]) {
    f[0] = __byte_perm(r.v[0][t], r.v[1][t], 0x5410), f[1] = __byte_perm(r.v[0][t], r.v[1][t], 0x7632);
    f[2] = __byte_perm(r.v[2][t], r.v[3][t], 0x5410), f[3] = __byte_perm(r.v[2][t], r.v[3][t], 0x7632);
  }
  static __device__ __forceinline__ int v_col(int t, int g) { return 64 * (t / 4) + 8 * g + 2 * (t % 4); }
};

struct SplitShape {
  int splits, group, window, sinks;
  float scale_log2;
};

// NT groups of 8 query rows.  Grid: (splits x slices, row blocks), a cluster
// per slice.
template <int D, int NT, class Keys>
__global__ void __launch_bounds__(kThreads) split_attn_kernel(const Keys keys_in, const SplitShape shape) {
  using T = typename Keys::Io;
  using Op = typename Keys::Op;
  constexpr int kRows = 8 * NT, kPitch = D + 4;
  extern __shared__ float smem[];
  float *o_s = smem;                             // [kWarps][kRows][kPitch]
  float *m_s = o_s + kWarps * kRows * kPitch;    // [kWarps][kRows]
  float *l_s = m_s + kWarps * kRows;             // [kWarps][kRows]
  float *cta_m = l_s + kWarps * kRows, *cta_l = cta_m + kRows;
  Keys keys = keys_in;
  const int rank = blockIdx.x % shape.splits;
  keys.open(blockIdx.x / shape.splits);
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
  const int begin = (int)((long long)n_steps * rank / shape.splits);
  const int end = (int)((long long)n_steps * (rank + 1) / shape.splits);
  auto step_of = [&](int i) { return i < sink_steps ? i : base_step + i - sink_steps; };

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
      const int e = top > 0.f && top < INFINITY ? min(max(8 - (((__float_as_int(top) >> 23) & 0xff) - 127), -119), 119) : 0;
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

  float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) o[nt][t][0] = o[nt][t][1] = o[nt][t][2] = o[nt][t][3] = 0.f;
  }

  typename Keys::Raw cur, next;
  int i = begin + warp, page = 0, page_next = 0;
  if (i < end) {
    page = keys.place(step_of(i));
    keys.load(cur, page, step_of(i), seen, g, c);
    if (i + kWarps < end) page_next = keys.place(step_of(i + kWarps));
  }
  for (; i < end; i += kWarps) {
    const int step = step_of(i);
    const bool here = keys.there(page);
    if (i + kWarps < end) {
      keys.load(next, page_next, step_of(i + kWarps), seen, g, c);
      page = page_next;
      if (i + 2 * kWarps < end) page_next = keys.place(step_of(i + 2 * kWarps));
    }
    if (here) {
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        uint32_t a[4];
        Keys::k_frag(cur, s, a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(x[nt], a, qf[nt][s][0], qf[nt][s][1], Op{});
      }
      float ks = 1.f;
      if constexpr (Keys::kScaled) ks = cur.ks;
      // whole: every row sees the 16 keys (rows that are not there are not read)
      const int k0 = step * kStep;
      const bool whole = k0 + kStep - 1 <= first_pos && k0 + kStep <= keys.nk &&
                         (k0 > last_pos - shape.window || k0 + kStep <= shape.sinks);
      bool grows = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[nt][e] *= fac[nt][e & 1] * ks;
          if (!whole) {
            const int key = k0 + g + 8 * (e >> 1);
            if (key >= keys.nk || !visible(pos[nt][e & 1], key, shape.window, shape.sinks)) x[nt][e] = -INFINITY;
          }
          grows = grows || x[nt][e] > m[nt][e & 1] + (kHead + 8.f);
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
            top = fmaxf(top - kHead, m[nt][e]);
            const float alpha = top == m[nt][e] ? 1.f : ex2_approx(m[nt][e] - top);
            m[nt][e] = top;
            l[nt][e] *= alpha;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[nt][t][e] *= alpha, o[nt][t][2 + e] *= alpha;
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float mm = m[nt][e & 1];
          x[nt][e] = ex2_approx(x[nt][e] - (mm == -INFINITY ? 0.f : mm));
          l[nt][e & 1] += x[nt][e];
        }
        pb[nt][0] = transpose8(Elem<Op>::pack(x[nt][0], x[nt][1]));
        pb[nt][1] = transpose8(Elem<Op>::pack(x[nt][2], x[nt][3]));
      }
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        uint32_t a[4];
        Keys::v_frag(cur, t, a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (Keys::kScaled) {
            float y[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816(y, a, pb[nt][0], pb[nt][1], Op{});
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][t][e] = fmaf(y[e], cur.vs, o[nt][t][e]);
          } else {
            mma16816(o[nt][t], a, pb[nt][0], pb[nt][1], Op{});
          }
        }
      }
    }
    cur = next;
  }

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
  auto weight = [](float part, float top) { return part == -INFINITY ? 0.f : ex2_approx(part - top); };
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * nt + 2 * c + e;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w * kRows + r]);
      const float f = weight(m[nt][e], top);
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
  // join the cluster: each block finishes its share of the columns
  cg::cluster_group cluster = cg::this_cluster();
  if (shape.splits > 1) cluster.sync();
  else __syncthreads();
  for (int q = threadIdx.x + rank * kThreads; q < kQuads; q += shape.splits * kThreads) {
    const int r = q / (D / 4), col = q % (D / 4) * 4;
    if (r >= rows) continue;
    float top = -INFINITY, sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (shape.splits > 1) {
      for (int s = 0; s < shape.splits; ++s) top = fmaxf(top, *cluster.map_shared_rank(&cta_m[r], s));
      for (int s = 0; s < shape.splits; ++s) {
        const float f = weight(*cluster.map_shared_rank(&cta_m[r], s), top);
        sum += *cluster.map_shared_rank(&cta_l[r], s) * f;
        const float4 z = *reinterpret_cast<float4 *>(cluster.map_shared_rank(&o_s[r * kPitch + col], s));
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
  if (shape.splits > 1) cluster.sync();  // no block leaves while others read its part
}

constexpr size_t split_smem(int d, int nt) {
  return sizeof(float) * (kWarps * 8 * nt * (d + 4) + 2 * kWarps * 8 * nt + 2 * 8 * nt);
}

// Blocks per slice: enough for two per SM, but at least two steps for each warp.
int splits_for(long long units, long long most_keys) {
  const long long steps = (most_keys + kStep - 1) / kStep;
  int s = 1;
  while (s < 16 && units * s < 2 * 148 && steps >= 2ll * s * kWarps * 2) s *= 2;
  return s;
}

template <int D, int NT, class Keys>
cudaError_t launch(const Keys &keys, SplitShape shape, long long slices, int rows, long long most_keys, cudaStream_t stream) {
  auto *kernel = split_attn_kernel<D, NT, Keys>;
  const int blocks = (rows + 8 * NT - 1) / (8 * NT);
  shape.splits = splits_for(slices * blocks, most_keys);
  const size_t smem = split_smem(D, NT);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(slices * shape.splits), blocks), cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem, cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = shape.splits, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, keys, shape);
}

template <int D, class Keys>
cudaError_t launch_rows(const Keys &keys, const SplitShape &shape, long long slices, int rows, long long most_keys,
                        cudaStream_t stream) {
  return rows <= 8 ? launch<D, 1>(keys, shape, slices, rows, most_keys, stream)
                   : launch<D, 2>(keys, shape, slices, rows, most_keys, stream);
}

// keys that one query row may see
long long visible_keys(long long nk, long long q_len, long long window, long long sinks) {
  const long long w = window + q_len - 1 + sinks;
  return w < nk ? w : nk;
}

template <int D, int kType, class T>
cudaError_t cache_launch(const CacheAttn &a, const SplitShape &shape, cudaStream_t stream) {
  CacheKeys<D, kType, T> keys{};
  keys.a = a;
  const long long nk = (long long)a.c.table_pages * a.c.page_size;
  return launch_rows<D>(keys, shape, (long long)a.batch * a.c.kv_heads, a.q_len * a.group,
                        visible_keys(nk, a.q_len, a.window, a.sinks), stream);
}

template <int D, class T>
cudaError_t window_launch(const WinParams &p, const SplitShape &shape, cudaStream_t stream) {
  RowKeys<D, T> keys{};
  keys.p = p;
  return launch_rows<D>(keys, shape, (long long)p.batch * p.kv_heads, p.q_len * p.group,
                        visible_keys(p.kv_len, p.q_len, p.window, p.sinks), stream);
}

}  // namespace

cudaError_t launch_cache_attention(const CacheAttn &a, int cache_type, int io_type, cudaStream_t stream) {
  const SplitShape shape{1, a.group, a.window, a.sinks, a.scale_log2};
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
  const SplitShape shape{1, p.group, p.window, p.sinks, p.scale_log2};
  if (p.d == 128)
    return type == STA_TYPE_BF16 ? window_launch<128, __nv_bfloat16>(p, shape, stream)
                                 : window_launch<128, __half>(p, shape, stream);
  return type == STA_TYPE_BF16 ? window_launch<64, __nv_bfloat16>(p, shape, stream)
                               : window_launch<64, __half>(p, shape, stream);
}

}  // namespace sta
