// seq_attn.cu -- token-sequence attention, one warp per query (or key) row:
// forward and backward of the sliding window with sinks, and the forward over
// the 8-bit cache.
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

// dQ and D of one query row per warp.
template <int D, class T>
__global__ void __launch_bounds__(256) window_dq_rows_kernel(const WinParams p) {
  const int lane = threadIdx.x & 31, h = blockIdx.y, row = blockIdx.x * 8 + (threadIdx.x >> 5);
  const Sequence s = sequence(p, blockIdx.z);
  if (row >= s.nq) return;
  float q[D / 32], g[D / 32], dq[D / 32], dd = 0.f;
  const char *qr = row_ptr(p.q, s.slice, h, s.q0 + row), *gr = row_ptr(p.dout, s.slice, h, s.q0 + row),
             *orow = row_ptr(p.o, s.slice, h, s.q0 + row);
  for (int e = 0; e < D / 32; ++e) {
    q[e] = to_f<T>(qr, lane + 32 * e), g[e] = to_f<T>(gr, lane + 32 * e), dq[e] = 0.f;
    dd = fmaf(g[e], to_f<T>(orow, lane + 32 * e), dd);
  }
  dd = warp_sum(dd);
  const long long at = stat_row(p, s, h, row);
  if (lane == 0) p.dd[at] = dd;
  const float lse2 = p.lse[at] * 1.4426950408889634f;
  const int pos = row + s.nk - s.nq;
  for (int key = 0; key <= min(pos, s.nk - 1); ++key) {
    if (!visible(pos, key, p.window, p.sinks)) continue;
    const char *kr = row_ptr(p.k, s.slice, h / p.group, s.k0 + key), *vr = row_ptr(p.v, s.slice, h / p.group, s.k0 + key);
    float x = 0.f, dp = 0.f, kf[D / 32];
    for (int e = 0; e < D / 32; ++e) {
      kf[e] = to_f<T>(kr, lane + 32 * e);
      x = fmaf(q[e], kf[e], x), dp = fmaf(g[e], to_f<T>(vr, lane + 32 * e), dp);
    }
    x = warp_sum(x), dp = warp_sum(dp);
    const float ds = exp2f(x * p.scale_log2 - lse2) * (dp - dd);
    for (int e = 0; e < D / 32; ++e) dq[e] = fmaf(ds, kf[e], dq[e]);
  }
  char *dst = const_cast<char *>(row_ptr(p.dq, s.slice, h, s.q0 + row));
  for (int e = 0; e < D / 32; ++e) reinterpret_cast<T *>(dst)[lane + 32 * e] = (T)(dq[e] * p.scale);
}

// dK and dV of one key row per warp, summed over the query heads of its group.
template <int D, class T>
__global__ void __launch_bounds__(256) window_dkdv_rows_kernel(const WinParams p) {
  const int lane = threadIdx.x & 31, h = blockIdx.y, key = blockIdx.x * 8 + (threadIdx.x >> 5);
  const Sequence s = sequence(p, blockIdx.z);
  if (key >= s.nk) return;
  float k[D / 32], v[D / 32], dk[D / 32], dv[D / 32];
  const char *kr = row_ptr(p.k, s.slice, h, s.k0 + key), *vr = row_ptr(p.v, s.slice, h, s.k0 + key);
  for (int e = 0; e < D / 32; ++e)
    k[e] = to_f<T>(kr, lane + 32 * e), v[e] = to_f<T>(vr, lane + 32 * e), dk[e] = dv[e] = 0.f;
  for (int hq = h * p.group; hq < (h + 1) * p.group; ++hq)
    for (int row = max(0, key - (s.nk - s.nq)); row < s.nq; ++row) {
      if (!visible(row + s.nk - s.nq, key, p.window, p.sinks)) continue;
      const char *qr = row_ptr(p.q, s.slice, hq, s.q0 + row), *gr = row_ptr(p.dout, s.slice, hq, s.q0 + row);
      const long long at = stat_row(p, s, hq, row);
      float x = 0.f, dp = 0.f, q[D / 32], g[D / 32];
      for (int e = 0; e < D / 32; ++e) {
        q[e] = to_f<T>(qr, lane + 32 * e), g[e] = to_f<T>(gr, lane + 32 * e);
        x = fmaf(q[e], k[e], x), dp = fmaf(g[e], v[e], dp);
      }
      x = warp_sum(x), dp = warp_sum(dp);
      const float pr = exp2f(x * p.scale_log2 - p.lse[at] * 1.4426950408889634f), ds = pr * (dp - p.dd[at]);
      for (int e = 0; e < D / 32; ++e) dv[e] = fmaf(pr, g[e], dv[e]), dk[e] = fmaf(ds, q[e], dk[e]);
    }
  char *dst = const_cast<char *>(row_ptr(p.dk, s.slice, h, s.k0 + key));
  char *dst_v = const_cast<char *>(row_ptr(p.dv, s.slice, h, s.k0 + key));
  for (int e = 0; e < D / 32; ++e) {
    reinterpret_cast<T *>(dst)[lane + 32 * e] = (T)(dk[e] * p.scale);
    reinterpret_cast<T *>(dst_v)[lane + 32 * e] = (T)dv[e];
  }
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

template <int D, class T>
cudaError_t backward_d(const WinParams &p, cudaStream_t stream) {
  window_dq_rows_kernel<D, T><<<dim3((p.q_len + 7) / 8, p.heads, p.batch), 256, 0, stream>>>(p);
  window_dkdv_rows_kernel<D, T><<<dim3((p.kv_len + 7) / 8, p.kv_heads, p.batch), 256, 0, stream>>>(p);
  return cudaGetLastError();
}
template <int D, int kType>
cudaError_t cache_d(const CacheAttn &a, int io_type, cudaStream_t stream) {
  const dim3 grid((a.q_len + 7) / 8, a.heads, a.batch);
  if (io_type == STA_TYPE_BF16) cache_rows_kernel<D, kType, __nv_bfloat16><<<grid, 256, 0, stream>>>(a);
  else cache_rows_kernel<D, kType, __half><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_backward(const WinParams &p, int type, cudaStream_t stream) {
  if (p.d == 128)
    return type == STA_TYPE_BF16 ? backward_d<128, __nv_bfloat16>(p, stream) : backward_d<128, __half>(p, stream);
  return type == STA_TYPE_BF16 ? backward_d<64, __nv_bfloat16>(p, stream) : backward_d<64, __half>(p, stream);
}
cudaError_t launch_cache_attention(const CacheAttn &a, int cache_type, int io_type, cudaStream_t stream) {
  if (a.c.d == 128)
    return cache_type == STA_TYPE_E4M3 ? cache_d<128, STA_TYPE_E4M3>(a, io_type, stream)
                                       : cache_d<128, STA_TYPE_INT8>(a, io_type, stream);
  return cache_type == STA_TYPE_E4M3 ? cache_d<64, STA_TYPE_E4M3>(a, io_type, stream)
                                     : cache_d<64, STA_TYPE_INT8>(a, io_type, stream);
}

}  // namespace sta
