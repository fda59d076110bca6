// seq_attn.cu -- attention over the 8-bit cache, one warp per query row.
#include "seq_common.cuh"

namespace sta {
namespace {

template <class T>
__device__ __forceinline__ float to_f(const char *row, int e) {
  return (float)reinterpret_cast<const T *>(row)[e];
}

__device__ __forceinline__ const char *row_ptr(const Rows &x, int b, int h, long long r) {
  return x.p + 2 * ((long long)b * x.b + (long long)h * x.h + r * x.r);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Online softmax over the visible keys of one row; load(key, kf, vf) gives the
// lane's elements and says whether the key is there.
template <int D, class Load>
__device__ __forceinline__ void attend(const float (&q)[D / 32], int pos, int nk, int window, int sinks, float sl2,
                                       float (&o)[D / 32], float &m, float &l, Load &&load) {
  m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  const int lo = max(0, pos - window + 1), s_end = min(min(sinks, lo), nk);
  const int last = min(pos, nk - 1);
  for (int i = 0; i < s_end + max(0, last - lo + 1); ++i) {
    const int key = i < s_end ? i : lo + i - s_end;
    float kf[D / 32], vf[D / 32];
    if (!load(key, kf, vf)) continue;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) s = fmaf(q[e], kf[e], s);
    s = warp_sum(s) * sl2;
    const float mn = fmaxf(m, s), a = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * a + p;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = fmaf(o[e], a, p * vf[e]);
  }
}

template <int D, class T>
__device__ __forceinline__ void finish(const float (&o)[D / 32], float m, float l, char *dst, float *lse, int lane) {
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) reinterpret_cast<T *>(dst)[lane + 32 * e] = (T)(o[e] * inv);
  if (lse && lane == 0) *lse = l > 0.f ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

template <int D, int kType, class T>
__global__ void __launch_bounds__(256) cache_rows_kernel(const CacheAttn a) {
  const CacheParams &c = a.c;
  const int lane = threadIdx.x & 31, h = blockIdx.y, row = blockIdx.x * 8 + (threadIdx.x >> 5), b = blockIdx.z;
  if (row >= a.q_len) return;
  const int nk = min(max(a.lengths[b], 0), c.table_pages * c.page_size);
  float q[D / 32], o[D / 32], m, l;
  const char *qr = row_ptr(a.q, b, h, row);
  for (int e = 0; e < D / 32; ++e) q[e] = to_f<T>(qr, lane + 32 * e);
  attend<D>(q, row + nk - a.q_len, nk, a.window, a.sinks, a.scale_log2, o, m, l, [&](int key, auto &kf, auto &vf) {
    const int page = page_of(c, b, key);
    if (page < 0) return false;
    const int in_page = key % c.page_size;
    const long long ph = (long long)page * c.kv_heads + h / a.group;
    const long long at = (ph * c.page_size + in_page) * D, sc = ph * (c.page_size / c.block) + in_page / c.block;
    for (int e = 0; e < D / 32; ++e) {
      const int i = lane + 32 * e;
      if (kType == STA_TYPE_INT8) {
        kf[e] = (float)(int8_t)c.k[at + i] * c.k_scale[sc], vf[e] = (float)(int8_t)c.v[at + i] * c.v_scale[sc];
      } else {
        __nv_fp8_e4m3 kk, vv;
        kk.__x = c.k[at + i], vv.__x = c.v[at + i];
        kf[e] = (float)kk * c.k_scale[sc], vf[e] = (float)vv * c.v_scale[sc];
      }
    }
    return true;
  });
  finish<D, T>(o, m, l, const_cast<char *>(row_ptr(a.o, b, h, row)),
               a.lse ? a.lse + ((long long)b * a.heads + h) * a.q_len + row : nullptr, lane);
}

template <int D, int kType>
cudaError_t cache_d(const CacheAttn &a, int io_type, cudaStream_t stream) {
  const dim3 grid((a.q_len + 7) / 8, a.heads, a.batch);
  if (io_type == STA_TYPE_BF16) cache_rows_kernel<D, kType, __nv_bfloat16><<<grid, 256, 0, stream>>>(a);
  else cache_rows_kernel<D, kType, __half><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attention(const CacheAttn &a, int cache_type, int io_type, cudaStream_t stream) {
  if (a.c.d == 128)
    return cache_type == STA_TYPE_E4M3 ? cache_d<128, STA_TYPE_E4M3>(a, io_type, stream)
                                       : cache_d<128, STA_TYPE_INT8>(a, io_type, stream);
  return cache_type == STA_TYPE_E4M3 ? cache_d<64, STA_TYPE_E4M3>(a, io_type, stream)
                                     : cache_d<64, STA_TYPE_INT8>(a, io_type, stream);
}

}  // namespace sta
