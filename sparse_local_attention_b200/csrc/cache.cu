// cache.cu -- writing to and reading from the 8-bit key/value cache.
//
// Every `block` tokens of a page and key head share one fp32 scale s, and a
// code c stands for c * s.  Writing rows x into a block:
//   s = max(scale of the block's earlier tokens, max |x| / qmax, 2^-100),
//   c = round(x * (1 / s)),  and where s grew by earlier tokens: their codes
//   become round(c * s_old * (1 / s)).
// Bound by memory: 2 bytes read and 1 written per element, 1 read and 2 written
// on the way back (prompts of 8 sequences up to 4096 tokens, 8 key heads, d 128:
// written in 22.4 us and read in 24.7, 5.6 and 5.1 TB/s); a few rows are two
// latencies of memory, 3.2 us.
#include "seq_common.cuh"
#include "sm100_ptx.cuh"

namespace sta {
namespace {

constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100: its reciprocal is finite

template <int kType> struct Code;  // STA_TYPE_E4M3 / STA_TYPE_INT8
template <> struct Code<STA_TYPE_E4M3> {
  static constexpr float kMax = 448.f;
  // two codes of two values (lo in bits 0..7), to nearest even, cut to +-448;
  // NaN becomes 0
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    lo = lo == lo ? lo : 0.f;
    hi = hi == hi ? hi : 0.f;
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
  // four finite values of at most the largest code (but for a rounding)
  static __device__ __forceinline__ uint32_t pack_finite(float2 a, float2 b) {
    uint16_t x, y;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(x) : "f"(a.y), "f"(a.x));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(b.y), "f"(b.x));
    return uint32_t(x) | (uint32_t(y) << 16);
  }
  static __device__ __forceinline__ void unpack4(uint32_t w, float2 &a, float2 &b) {
    a = unpack(w & 0xffffu), b = unpack(w >> 16);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
    return __half22float2(*reinterpret_cast<__half2 *>(&h));
  }
};
template <> struct Code<STA_TYPE_INT8> {
  static constexpr float kMax = 127.f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    // __float2int_rn of NaN is 0
    const int a = __float2int_rn(fminf(fmaxf(lo, -127.f), 127.f)), b = __float2int_rn(fminf(fmaxf(hi, -127.f), 127.f));
    return (lo == lo ? (uint32_t)a & 0xffu : 0u) | ((hi == hi ? (uint32_t)b & 0xffu : 0u) << 8);
  }
  // Adding 1.5 * 2^23 rounds to the nearest even integer, whose two's complement
  // is the sum's low byte.
  static __device__ __forceinline__ uint32_t pack_finite(float2 a, float2 b) {
    const float2 magic = make_float2(12582912.f, 12582912.f), x = add2(a, magic), y = add2(b, magic);
    return __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                       __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
  }
  static __device__ __forceinline__ void unpack4(uint32_t w, float2 &a, float2 &b) {
    // c ^ 0x80 in the low byte of 2^23 is 2^23 + 128 + c
    w ^= 0x80808080u;
    const float2 off = make_float2(-8388736.f, -8388736.f);
    auto at = [&](int s) { return __uint_as_float(__byte_perm(w, 0x4b000000u, s)); };
    a = add2(make_float2(at(0x7440), at(0x7441)), off), b = add2(make_float2(at(0x7442), at(0x7443)), off);
  }
};

__device__ __forceinline__ int clamp_count(const CacheMove &m, int b) {
  return m.count ? min(max(__ldg(m.count + b), 0), m.rows) : m.rows;
}

// Largest magnitude of packed pairs: without their sign, 16-bit floats order
// like unsigned integers, with infinity and NaN on top.
__device__ __forceinline__ uint32_t top_pair(uint32_t top, uint32_t w) { return __vmaxu2(top, w & 0x7fff7fffu); }
template <class T> constexpr uint32_t kInfBits = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;

// One CTA per (block of tokens touched, key head, sequence and tensor).  The new
// rows stay in registers between the maximum and the codes: one pass over them.
template <int D, int kBlock, int kType, class T>
__global__ void __launch_bounds__(128) cache_write_kernel(const CacheMove m) {
  const CacheParams &c = m.c;
  const bool is_v = blockIdx.z & 1;
  const int b = blockIdx.z >> 1, h = blockIdx.y;
  const int start = __ldg(m.start + b), count = clamp_count(m, b);
  if (start < 0 || count == 0) return;
  const long long end = (long long)start + count;
  const long long first = ((long long)start / kBlock + blockIdx.x) * kBlock;  // first token of the block
  if (first >= end || first + kBlock > (long long)c.table_pages * c.page_size) return;
  const int page = page_of(c, b, (int)first);
  if (page < 0) return;
  const int in_page = (int)first % c.page_size;
  const long long ph = (long long)page * c.kv_heads + h;
  uint8_t *codes = (is_v ? c.v : c.k) + (ph * c.page_size + in_page) * D;
  float *scale = (is_v ? c.v_scale : c.k_scale) + ph * (c.page_size / kBlock) + in_page / kBlock;
  const Rows &x = is_v ? m.v : m.k;
  const int lo = (int)max(0ll, start - first), hi = (int)min((long long)kBlock, end - first);  // new tokens of the block
  constexpr int kPer = D / 8;  // 16-byte pieces per row
  constexpr int kPieces = kBlock * kPer / 128 > 0 ? kBlock * kPer / 128 : 1, kPass = 128 / kPer;
  const int row0 = lo + threadIdx.x / kPer, col = threadIdx.x % kPer * 8;
  const char *src = x.p + 2 * ((long long)b * x.b + (long long)h * x.h + (first - start + row0) * x.r + col);
  const float old = lo > 0 ? *scale : 0.f;
  const long long src_step = 2 * kPass * x.r;
  uint4 held[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    held[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row0 + kPass * i < hi) held[i] = __ldg(reinterpret_cast<const uint4 *>(src));
    src += src_step;
  }
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    top = top_pair(top_pair(top_pair(top_pair(top, held[i].x), held[i].y), held[i].z), held[i].w);
  top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  __shared__ uint32_t part[4];
  __shared__ float part_f[4];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();  // every thread has read the old scale, too
  top = max(max(part[0], part[1]), max(part[2], part[3]));
  float amax = Elem<T>::unpack(top).x;
  const bool plain = top < kInfBits<T>;
  if (!plain) {
    // infinities count as the type's largest value, NaN as nothing
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (row0 + kPass * i < hi) {
        const uint32_t w[4] = {held[i].x, held[i].y, held[i].z, held[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = Elem<T>::unpack(w[e]);
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));  // fmaxf drops NaN
        }
      }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if ((threadIdx.x & 31) == 0) part_f[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = fminf(fmaxf(fmaxf(part_f[0], part_f[1]), fmaxf(part_f[2], part_f[3])), Elem<T>::kMax);
  }
  const float s = fmaxf(old, fmaxf(amax / Code<kType>::kMax, kScaleFloor));
  const float inv = 1.f / s;
  const float2 inv2 = make_float2(inv, inv);
  if (threadIdx.x == 0) *scale = s;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if (row0 + kPass * i < hi) {
      const uint32_t w[4] = {held[i].x, held[i].y, held[i].z, held[i].w};
      uint32_t q[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 f = mul2(Elem<T>::unpack(w[2 * e]), inv2), z = mul2(Elem<T>::unpack(w[2 * e + 1]), inv2);
        q[e] = plain ? Code<kType>::pack_finite(f, z)
                     : Code<kType>::pack(f.x, f.y) | (Code<kType>::pack(z.x, z.y) << 16);
      }
      *reinterpret_cast<uint2 *>(codes + (row0 + kPass * i) * D + col) = make_uint2(q[0], q[1]);
    }
  }
  if (lo > 0 && s > old) {
    // the block's earlier tokens at the new scale
    for (int i = threadIdx.x; i < lo * D / 4; i += 128) {
      uint32_t *w = reinterpret_cast<uint32_t *>(codes) + i;
      float2 a, z;
      Code<kType>::unpack4(*w, a, z);
      *w = Code<kType>::pack(a.x * old * inv, a.y * old * inv) | (Code<kType>::pack(z.x * old * inv, z.y * old * inv) << 16);
    }
  }
}

// A warp per 16 tokens that begin at a multiple of 16: one page and one scale,
// a run of 16 D codes, of which a lane takes 8 at a time so that a warp's stores
// are whole lines (a lookup per row and lane, and stores of half sectors: 26.7 us
// where this takes 24.7, prompts of 8 sequences up to 4096; 512 tokens of 16
// sequences, d 64: 4.7 and 3.7).
constexpr int kReadTokens = 16, kReadWarps = 4;
template <int D, int kType, class T>
__global__ void __launch_bounds__(32 * kReadWarps) cache_read_kernel(const CacheMove m) {
  const CacheParams &c = m.c;
  constexpr int kPer = D / 8, kRows = 32 / kPer, kLoads = kReadTokens / kRows;  // lanes per row, rows per load
  const bool is_v = blockIdx.z & 1;
  const int b = blockIdx.z >> 1, h = blockIdx.y, lane = threadIdx.x & 31;
  const int start = __ldg(m.start + b), count = clamp_count(m, b), base = max(start, 0);
  const long long first = (base / kReadTokens + (long long)blockIdx.x * kReadWarps + (threadIdx.x >> 5)) * kReadTokens;
  const bool none = first - base >= count;  // rows that get no token
  if (first - base >= m.rows || (none && !m.zero)) return;
  const int row0 = (int)(first - base) + lane / kPer, col = lane % kPer * 8;  // row0: from -15 on
  int page = -1, in_page = 0;
  const Rows &x = is_v ? m.v : m.k;
  char *out = x.p + 2 * ((long long)b * x.b + (long long)h * x.h + (long long)row0 * x.r + col);
  const long long out_step = 2 * kRows * x.r;
  if (none) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i, out += out_step)
      if (row0 + kRows * i < m.rows) *reinterpret_cast<uint4 *>(out) = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  if (start >= 0 && first < (long long)c.table_pages * c.page_size) {
    const int index = (int)first / c.page_size;
    page = __ldg(c.table + (long long)b * c.table_pages + index);
    if ((unsigned)page >= (unsigned)c.pages) page = -1;
    in_page = (int)first - index * c.page_size;
  }
  const long long ph = (long long)page * c.kv_heads + h;
  const uint8_t *codes = (is_v ? c.v : c.k) + (ph * c.page_size + in_page) * D + 8 * lane;
  uint2 w[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = row0 + kRows * i;
    w[i] = make_uint2(0u, 0u);
    if (page >= 0 && row >= 0 && row < count) w[i] = __ldg(reinterpret_cast<const uint2 *>(codes + 256 * i));
  }
  float s = 0.f;
  if (page >= 0) s = __ldg((is_v ? c.v_scale : c.k_scale) + ph * (c.page_size / c.block) + in_page / c.block);
  const float2 s2 = make_float2(s, s);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = row0 + kRows * i;
    const bool there = page >= 0 && row < count;
    const float2 by = there ? s2 : make_float2(0.f, 0.f);  // whatever the scale of a block without tokens
    uint32_t v[4];
    const uint32_t in[2] = {w[i].x, w[i].y};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float2 f, g;
      Code<kType>::unpack4(in[e], f, g);
      f = mul2(f, by), g = mul2(g, by);
      v[2 * e] = Elem<T>::pack(f.x, f.y), v[2 * e + 1] = Elem<T>::pack(g.x, g.y);
    }
    if (row >= 0 && row < m.rows && (there || m.zero))
      *reinterpret_cast<uint4 *>(out) = make_uint4(v[0], v[1], v[2], v[3]);
    out += out_step;
  }
}

template <int D, int kType, class T>
cudaError_t write_launch(const CacheMove &m, cudaStream_t stream) {
  // a run of `rows` tokens that starts anywhere touches at most this many blocks
  const dim3 grid((m.rows + m.c.block - 2) / m.c.block + 1, m.c.kv_heads, 2 * m.batch);
  switch (m.c.block) {
    case 16: cache_write_kernel<D, 16, kType, T><<<grid, 128, 0, stream>>>(m); break;
    case 32: cache_write_kernel<D, 32, kType, T><<<grid, 128, 0, stream>>>(m); break;
    case 64: cache_write_kernel<D, 64, kType, T><<<grid, 128, 0, stream>>>(m); break;
    default: cache_write_kernel<D, 128, kType, T><<<grid, 128, 0, stream>>>(m);
  }
  return cudaGetLastError();
}
template <int D, int kType, class T>
cudaError_t read_launch(const CacheMove &m, cudaStream_t stream) {
  // a run of `rows` tokens that starts anywhere touches at most this many groups
  const int groups = (m.rows + kReadTokens - 2) / kReadTokens + 1;
  const dim3 grid((groups + kReadWarps - 1) / kReadWarps, m.c.kv_heads, 2 * m.batch);
  cache_read_kernel<D, kType, T><<<grid, 32 * kReadWarps, 0, stream>>>(m);
  return cudaGetLastError();
}

template <class F>
cudaError_t by_types(int d, int cache_type, int io_type, F &&f) {
  auto io = [&](auto dim, auto code) {
    return io_type == STA_TYPE_BF16 ? f(dim, code, __nv_bfloat16{}) : f(dim, code, __half{});
  };
  auto cache = [&](auto dim) {
    return cache_type == STA_TYPE_E4M3 ? io(dim, std::integral_constant<int, STA_TYPE_E4M3>{})
                                       : io(dim, std::integral_constant<int, STA_TYPE_INT8>{});
  };
  return d == 128 ? cache(std::integral_constant<int, 128>{}) : cache(std::integral_constant<int, 64>{});
}

}  // namespace

cudaError_t launch_cache_write(const CacheMove &m, int cache_type, int io_type, cudaStream_t stream) {
  return by_types(m.c.d, cache_type, io_type, [&](auto d, auto code, auto t) {
    return write_launch<decltype(d)::value, decltype(code)::value, decltype(t)>(m, stream);
  });
}

cudaError_t launch_cache_read(const CacheMove &m, int cache_type, int io_type, cudaStream_t stream) {
  return by_types(m.c.d, cache_type, io_type, [&](auto d, auto code, auto t) {
    return read_launch<decltype(d)::value, decltype(code)::value, decltype(t)>(m, stream);
  });
}

}  // namespace sta
