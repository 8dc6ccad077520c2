// Dense GQA of a batch's new tokens over the whole paged cache, bf16 or
// one-byte (E4M3) KV.
//
// For row r at position t, head h, group g = h / 16:
//   out = sum_{j <= t} softmax_j(sm_scale q.K_j) V_j,  lse = log sum_j exp(sm_scale q.K_j)
// One CTA per (row, KV group, split of the row's pages); the splits of a row
// are joined by their log-sum-exp in split order.
#include <cuda.h>

#include "s5_common.cuh"
#include "s5_kernels.h"

namespace s5 {

namespace {

constexpr int kDnThreads = 256;

template <bool KV8>
__device__ __forceinline__ float kv_value(const void *pool, size_t i) {
  if (KV8) {
    float f0, f1, f2, f3;
    e4m3x4_to_float(reinterpret_cast<const uint8_t *>(pool)[i], f0, f1, f2, f3);
    return f0;
  }
  return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(pool)[i]);
}

// K / V pools are read with plain loads (written before this call).
template <bool KV8>
__global__ void __launch_bounds__(kDnThreads) dense_simple_kernel(const DenseArgs a) {
  __shared__ float q_s[kHpg][kD];
  __shared__ float p_s[kHpg][kPage];
  __shared__ float corr_s[kHpg], m_s[kHpg], l_s[kHpg];
  const int tid = threadIdx.x;
  const int split = blockIdx.x % a.n_split;
  const int rg = blockIdx.x / a.n_split;
  const int g = rg % kKv, r = rg / kKv;
  const int s = seq_of_row(a.cu_q, a.batch, r);
  if (s < 0) {  // behind the batch: left as it was
    return;
  }
  const int lo = ld_cg(a.cu_q + s), hi = ld_cg(a.cu_q + s + 1), ctx = ld_cg(a.ctx_lens + s);
  const bool bad = lo < 0 || hi > a.total_q || ctx < 0 || ctx > a.max_len - (hi - lo);
  if (bad && tid == 0 && r == max(lo, 0) && g == 0 && split == 0) record_error(a.err, S5_ERR_DEVICE_BOUNDS, r);
  const int t = bad ? -1 : ctx + (r - lo);
  for (int i = tid; i < kHpg * kD; i += kDnThreads)
    q_s[i / kD][i % kD] = __bfloat162float(
        reinterpret_cast<const __nv_bfloat16 *>(a.q)[((size_t)r * kHeads + g * kHpg) * kD + i]);
  if (tid < kHpg) {
    m_s[tid] = -INFINITY;
    l_s[tid] = 0.f;
  }
  const int pages = t / kPage + (t >= 0 ? 1 : 0);
  const int per = (pages + a.n_split - 1) / a.n_split;
  const int p0 = min(pages, split * per), p1 = min(pages, p0 + per);
  const int oh = tid / 16, od = (tid % 16) * 12;  // this thread's head and 12 dims of O
  float o[12];
#pragma unroll
  for (int e = 0; e < 12; ++e) o[e] = 0.f;
  for (int p = p0; p < p1; ++p) {
    const int page = ld_cg(a.page_table + (size_t)s * a.max_pages + p);
    const bool page_ok = page >= 0 && page < a.num_pages;
    if (!page_ok && tid == 0) record_error(a.err, S5_ERR_DEVICE_BOUNDS, r);
    const size_t base = ((size_t)max(page, 0) * kKv + g) * kPage * kD;
    __syncthreads();
    const int tok = tid % kPage, h0 = (tid / kPage) * 4;
    const bool seen = page_ok && p * kPage + tok <= t;
    float sc[4] = {0.f, 0.f, 0.f, 0.f};
    if (seen)
      for (int d = 0; d < kD; ++d) {
        const float k = kv_value<KV8>(a.k_pool, base + (size_t)tok * kD + d);
#pragma unroll
        for (int h = 0; h < 4; ++h) sc[h] = fmaf(q_s[h0 + h][d], k, sc[h]);
      }
#pragma unroll
    for (int h = 0; h < 4; ++h) p_s[h0 + h][tok] = seen ? sc[h] * a.scale_log2 : -INFINITY;
    __syncthreads();
    if (tid < kHpg) {
      float m = m_s[tid];
      for (int x = 0; x < kPage; ++x) m = fmaxf(m, p_s[tid][x]);
      const float mu = m == -INFINITY ? 0.f : m;
      const float c = exp2f(m_s[tid] - mu);
      float l = l_s[tid] * c;
      for (int x = 0; x < kPage; ++x) {
        const float w = exp2f(p_s[tid][x] - mu);
        p_s[tid][x] = w;
        l += w;
      }
      m_s[tid] = m;
      l_s[tid] = l;
      corr_s[tid] = c;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 12; ++e) o[e] *= corr_s[oh];
    const int n = page_ok ? min(kPage, t + 1 - p * kPage) : 0;
    for (int x = 0; x < n; ++x) {
      const float w = p_s[oh][x];
#pragma unroll
      for (int e = 0; e < 12; ++e) o[e] = fmaf(w, kv_value<KV8>(a.v_pool, base + (size_t)x * kD + od + e), o[e]);
    }
  }
  __syncthreads();
  const size_t rh = (size_t)r * kHeads + g * kHpg + oh;
  float *po = a.part_o + (rh * a.n_split + split) * kD + od;
#pragma unroll
  for (int e = 0; e < 12; ++e) po[e] = o[e];
  if (tid % 16 == 0) {
    a.part_ml[(rh * a.n_split + split) * 2] = m_s[oh];
    a.part_ml[(rh * a.n_split + split) * 2 + 1] = l_s[oh];
  }
}

__global__ void __launch_bounds__(kD) dense_join_kernel(const DenseArgs a) {
  const size_t rh = blockIdx.x;
  if (seq_of_row(a.cu_q, a.batch, (int)(rh / kHeads)) < 0) return;
  const float *ml = a.part_ml + rh * a.n_split * 2;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int p = 0; p < a.n_split; ++p) m = fmaxf(m, ml[2 * p]);
  const float mu = m == -INFINITY ? 0.f : m;
  for (int p = 0; p < a.n_split; ++p) {
    const float w = exp2f(ml[2 * p] - mu);
    l += w * ml[2 * p + 1];
    if (ml[2 * p] != -INFINITY) o += w * a.part_o[(rh * a.n_split + p) * kD + threadIdx.x];
  }
  // (l == 0: no visible token with a finite score; NaN passes through)
  reinterpret_cast<__nv_bfloat16 *>(a.out)[rh * kD + threadIdx.x] = __float2bfloat16(l == 0.f ? 0.f : o / l * a.v_scale);
  if (threadIdx.x == 0 && a.lse != nullptr) a.lse[rh] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_dense(const DenseArgs &a, cudaStream_t st) {
  const long long n = (long long)a.total_q * kKv * a.n_split;
  if (n > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.kv8) dense_simple_kernel<true><<<(unsigned)n, kDnThreads, 0, st>>>(a);
  else dense_simple_kernel<false><<<(unsigned)n, kDnThreads, 0, st>>>(a);
  dense_join_kernel<<<(unsigned)a.total_q * kHeads, kD, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace s5
