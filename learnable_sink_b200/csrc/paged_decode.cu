// Single-token attention with a learnable sink over a paged cache, 16-bit or
// E4M3 with a scale for each page and KV head:
//   x_j = scale <q, k_j>,  l = sum_j e^{x_j - m},  O = sum_j e^{x_j - m} v_j / (l + e^{a - m})
// over the visible positions j < n, and with a window also j < n_sink or
// j >= n - window.
#include <cuda_fp8.h>

#include "internal.h"
#include "paged.cuh"

namespace sk {

namespace {

constexpr int kTile = 128;  // positions per step

template <class E>
__device__ __forceinline__ float cell(const void* pages, long long at, bool fp8) {
  if (fp8) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(pages)[at], __NV_E4M3);
    return __half2float(__half(h));
  }
  return (float)static_cast<const typename E::T*>(pages)[at];
}

// One CTA per (sequence, KV head); thread i scores position i of a tile and sums
// column i of the values.
template <class E, int D>
__global__ void __launch_bounds__(kTile) paged_decode_kernel(PagedDecodeProblem p) {
  const PagedView& c = p.c;
  const int b = blockIdx.x / c.Hkv, kvh = blockIdx.x % c.Hkv, G = p.Hq / c.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ float sq[kPagedMaxGroup * D], sp[kPagedMaxGroup * kTile], red[4];
  __shared__ long long s_row[kTile];
  __shared__ float s_vs[kTile];
  const long long cap = (long long)c.max_pages << c.page_log2;
  int n = max(__ldg(c.seqlens + b), 0);
  if (n > cap) {
    if (tid == 0) set_status(c.status, SINKATTN_ERR_BOUNDS);
    n = (int)cap;
  }
  const typename E::T* q = static_cast<const typename E::T*>(p.q) + ((long long)b * p.Hq + kvh * G) * D;
  for (int i = tid; i < G * D; i += kTile) sq[i] = (float)q[i];
  float m[kPagedMaxGroup], l[kPagedMaxGroup], acc[kPagedMaxGroup];
#pragma unroll
  for (int h = 0; h < kPagedMaxGroup; ++h) { m[h] = -INFINITY; l[h] = 0.f; acc[h] = 0.f; }
  __syncthreads();
  for (int j0 = 0; j0 < n; j0 += kTile) {
    const int j = j0 + tid;
    bool seen = j < n && (p.window <= 0 || j < p.n_sink || j >= n - p.window);
    long long row = 0;
    float ks = 1.f, vs = 1.f;
    if (seen) {
      const int page = __ldg(c.table + (long long)b * c.max_pages + (j >> c.page_log2));
      if (page < 0 || page >= c.n_pages) {
        set_status(c.status, SINKATTN_ERR_BOUNDS);
        seen = false;
      } else {
        const long long blk = (long long)page * c.Hkv + kvh;
        row = (blk << c.page_log2) + (j & (c.page_size - 1));
        if (p.fp8) { ks = c.k_scale[blk]; vs = c.v_scale[blk]; }
      }
    }
    float x[kPagedMaxGroup];
#pragma unroll
    for (int h = 0; h < kPagedMaxGroup; ++h) x[h] = 0.f;
    if (seen)
      for (int d = 0; d < D; ++d) {
        const float kv = cell<E>(c.k_pages, row * D + d, p.fp8);
#pragma unroll
        for (int h = 0; h < kPagedMaxGroup; ++h)
          if (h < G) x[h] += sq[h * D + d] * kv;
      }
    s_row[tid] = seen ? row : -1;
    s_vs[tid] = vs;
#pragma unroll
    for (int h = 0; h < kPagedMaxGroup; ++h) {
      if (h >= G) break;
      x[h] = seen ? x[h] * ks * (p.scale * kLog2e) : -INFINITY;
      float mx = x[h];
      for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      __syncthreads();
      if (lane == 0) red[warp] = mx;
      __syncthreads();
      mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
      const float mn = fmaxf(m[h], mx);
      const float corr = m[h] == -INFINITY ? 0.f : exp2f(m[h] - mn);
      const float pr = x[h] == -INFINITY ? 0.f : exp2f(x[h] - mn);
      l[h] = l[h] * corr + pr;
      acc[h] *= corr;
      m[h] = mn;
      sp[h * kTile + tid] = pr;
    }
    __syncthreads();
    if (tid < D)
      for (int i = 0; i < kTile; ++i)
        if (s_row[i] >= 0) {
          const float v = cell<E>(c.v_pages, s_row[i] * D + tid, p.fp8) * s_vs[i];
#pragma unroll
          for (int h = 0; h < kPagedMaxGroup; ++h)
            if (h < G) acc[h] += sp[h * kTile + i] * v;
        }
    __syncthreads();
  }
#pragma unroll
  for (int h = 0; h < kPagedMaxGroup; ++h) {
    if (h >= G) break;
    float t = l[h];
    for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    __syncthreads();
    if (lane == 0) red[warp] = t;
    __syncthreads();
    t = (red[0] + red[1]) + (red[2] + red[3]);
    const float a2 = p.sink ? p.sink[kvh * G + h] * kLog2e : -INFINITY;
    const float mt = fmaxf(m[h], a2);
    const float w = m[h] == -INFINITY ? 0.f : exp2f(m[h] - mt);
    const float den = t * w + (a2 == -INFINITY ? 0.f : exp2f(a2 - mt));
    const long long row = (long long)b * p.Hq + kvh * G + h;
    if (tid < D)
      static_cast<typename E::T*>(p.out)[row * D + tid] =
          (typename E::T)(den != 0.f ? acc[h] * w / den : 0.f);
    if (tid == 0) {
      p.lse[row] = den != 0.f ? (mt + log2f(den)) * kLn2 : -INFINITY;
      if (p.sink_s) p.sink_s[row] = den != 0.f ? t * w / den : 0.f;
    }
  }
}

template <class E, int D>
int decode_typed(const PagedDecodeProblem& p, cudaStream_t stream) {
  paged_decode_kernel<E, D><<<p.c.B * p.c.Hkv, kTile, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SINKATTN_OK : SINKATTN_ERR_CUDA;
}

}  // namespace

size_t paged_decode_part_floats(int B, int Hq, int Hkv, int D, int sms) {
  return ((size_t)2 * sms + (size_t)B * Hkv) * (Hq / Hkv) * (D + 2);
}

int launch_paged_decode(const PagedDecodeProblem& p, cudaStream_t s) {
  if (p.dt == SINKATTN_FP16)
    return p.D == 128 ? decode_typed<ElemF16, 128>(p, s) : decode_typed<ElemF16, 64>(p, s);
  return p.D == 128 ? decode_typed<ElemBf16, 128>(p, s) : decode_typed<ElemBf16, 64>(p, s);
}

}  // namespace sk
