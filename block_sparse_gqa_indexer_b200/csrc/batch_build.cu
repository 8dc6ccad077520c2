// s5_build_batch: a step's page table, row offsets, slots and positions, built
// on the GPU from the lengths of the requests in the batch.
//
// With held = ceil(ctx / 64), need = ceil((ctx + new) / 64) of each sequence,
// two exclusive sums over the sequences give everything else: that of
// need - held the place of a sequence's new pages in the free list, that of
// the new tokens its first row.  Every table entry, row and new page is then an
// independent lookup.
//
// The work is small (about 4 bytes read and written per table entry), so the
// launch and the dependent steps inside it bound all but the largest calls: one
// launch, in which every CTA repeats the sums over the batch (1,024 sequences
// at a time, 4 per thread, 12 bytes read per sequence, in L2 after the first
// CTA) instead of waiting for another CTA's; then its warps take 256 columns of a
// table row at a time, all their loads in flight together, and its threads a new
// token each.  Measured (replayed graph): 3.3 us for 8 requests, 4.6 us for 16
// prefill chunks of up to 2,048 tokens, 7.1 us for 1,024 requests of up to 131,072
// tokens (12.6 MB), where a table entry per thread and step took 9.5 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "s5_common.cuh"
#include "s5_kernels.h"

using namespace s5;

namespace {

constexpr int kBThreads = 256;
constexpr int kBPer = 4;                       // sequences per thread and round
constexpr int kBSeqs = kBThreads * kBPer;      // sequences per round
constexpr int kBCols = 256;                    // table columns per warp and step
constexpr int kBMaxBatch = 65535;              // page sums stay below 2^31 (32,768 pages per sequence)

struct BuildArgs {
  int32_t *req_pages;
  const int32_t *free_pages;
  int32_t num_reqs, req_stride, num_free;
  const int32_t *req_ids, *ctx_lens, *new_lens;
  int32_t batch, max_pages, total_q;
  int32_t *page_table, *cu_q, *slots, *positions, *pages_used;
  int32_t *err;
};

// inclusive sum over the block of one value per thread; `buf` holds 8 partial sums
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) buf[warp] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kBThreads / 32 - 1; ++w)
    if (w < warp) v += buf[w];
  return v;
}

// VEC: table and request rows are whole 16-byte units (both widths load and store whole 128-byte
// lines; rows of other lengths cannot be read 16 bytes at a time)
template <bool VEC>
__global__ void __launch_bounds__(kBThreads) build_batch_kernel(const BuildArgs a) {
  __shared__ int s_id[kBSeqs], s_held[kBSeqs], s_need[kBSeqs], s_take[kBSeqs], s_ctx[kBSeqs];
  __shared__ int s_cu[kBSeqs + 1];
  __shared__ int pbuf[kBThreads / 32];
  __shared__ long long rbuf[kBThreads / 32];
  __shared__ int tot_pages;
  __shared__ long long tot_rows;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  int pages0 = 0;       // sums over the rounds before
  long long rows0 = 0;
  for (int s0 = 0; s0 < a.batch; s0 += kBSeqs) {
    const int n = min(kBSeqs, a.batch - s0);
    int id[kBPer], ctx[kBPer], nw[kBPer];
#pragma unroll
    for (int i = 0; i < kBPer; ++i) {
      const int s = s0 + tid * kBPer + i;
      const bool in = s < a.batch;
      id[i] = in ? ld_cg(a.req_ids + s) : -1;
      ctx[i] = in ? ld_cg(a.ctx_lens + s) : 0;
      nw[i] = in ? ld_cg(a.new_lens + s) : 0;
    }
    int held[kBPer], need[kBPer], pages = 0;
    long long rows = 0;
#pragma unroll
    for (int i = 0; i < kBPer; ++i) {
      bool ok = id[i] >= 0 && id[i] < a.num_reqs && ctx[i] >= 0 && nw[i] >= 0 && ctx[i] <= S5_MAX_LEN &&
                nw[i] <= S5_MAX_LEN - ctx[i];
      if (ok) {
        held[i] = (ctx[i] + kPage - 1) / kPage;
        need[i] = (ctx[i] + nw[i] + kPage - 1) / kPage;
        ok = need[i] <= a.max_pages && need[i] <= a.req_stride;
      }
      if (!ok) {
        if (id[i] != -1 && blockIdx.x == 0) record_error(a.err, S5_ERR_DEVICE_BOUNDS, s0 + tid * kBPer + i);
        id[i] = -1;
        held[i] = need[i] = ctx[i] = nw[i] = 0;
      }
      pages += need[i] - held[i];
      rows += nw[i];
    }
    int pages_end = pages0 + block_scan(pages, pbuf);
    long long rows_end = rows0 + block_scan(rows, rbuf);
    if (tid == kBThreads - 1) {
      tot_pages = pages_end;
      tot_rows = rows_end;
    }
    pages_end -= pages;
    rows_end -= rows;
#pragma unroll
    for (int i = 0; i < kBPer; ++i) {
      const int k = tid * kBPer + i;
      s_id[k] = id[i];
      s_ctx[k] = ctx[i];
      s_held[k] = held[i];
      s_need[k] = need[i];
      s_take[k] = pages_end;
      s_cu[k] = (int)min(rows_end, (long long)a.total_q);
      if (blockIdx.x == 0 && k < n) {
        a.cu_q[s0 + k] = s_cu[k];
        if (rows_end <= a.total_q && rows_end + nw[i] > a.total_q) record_error(a.err, S5_ERR_DEVICE_BOUNDS, s0 + k);
        if (pages_end <= a.num_free && pages_end + need[i] - held[i] > a.num_free)
          record_error(a.err, S5_ERR_DEVICE_BOUNDS, s0 + k);
      }
      pages_end += need[i] - held[i];
      rows_end += nw[i];
    }
    __syncthreads();
    pages0 = tot_pages;
    rows0 = tot_rows;
    if (tid == 0) s_cu[kBSeqs] = (int)min(rows0, (long long)a.total_q);
    __syncthreads();

    // ---- table entries: a warp takes 256 columns of a row, their loads in flight together ----
    const int segs = (a.max_pages + kBCols - 1) / kBCols;
    const int units = n * segs;  // <= 1,024 * 2^12 (the host bounds max_pages)
    for (int u = blockIdx.x * (kBThreads / 32) + warp; u < units; u += gridDim.x * (kBThreads / 32)) {
      const int k = u / segs, c0 = (u - k * segs) * kBCols;
      const int h = s_held[k], nd = s_need[k], take = s_take[k] - h;
      int32_t *req = a.req_pages + (size_t)max(s_id[k], 0) * a.req_stride;
      int32_t *dst = a.page_table + (size_t)(s0 + k) * a.max_pages;
      constexpr int W = VEC ? 4 : 1, N = kBCols / (32 * W);  // columns of a piece, pieces of a lane
      alignas(16) int32_t v[N][W];  // (pieces of W = 4 go in and out as one int4)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = c0 + (i * 32 + lane) * W;
        if (VEC) {
          if (c < h) *reinterpret_cast<int4 *>(v[i]) = *reinterpret_cast<const int4 *>(req + c);
        } else if (c < h) {
          v[i][0] = req[c];
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = c0 + (i * 32 + lane) * W;
        if (c >= a.max_pages) continue;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          if (c + e < h) continue;
          v[i][e] = -1;
          if (c + e < nd) {  // a page taken now
            if (take + c + e < a.num_free) v[i][e] = ld_cg(a.free_pages + take + c + e);
            req[c + e] = v[i][e];
          }
        }
        if (VEC) *reinterpret_cast<int4 *>(dst + c) = *reinterpret_cast<const int4 *>(v[i]);
        else dst[c] = v[i][0];
      }
    }
    // ---- rows ----
    if (a.slots != nullptr || a.positions != nullptr) {
      // (unsigned: a row number may be next to 2^31, and the step behind the last row passes it)
      const uint32_t end = (uint32_t)s_cu[kBSeqs], step = gridDim.x * kBThreads;
      for (uint32_t u = (uint32_t)s_cu[0] + blockIdx.x * kBThreads + tid; u < end; u += step) {
        const int r = (int)u;
        int lo = 0, hi = n;  // the last k with s_cu[k] <= r: the sequence that has row r
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_cu[mid] <= r) lo = mid;
          else hi = mid;
        }
        const int t = s_ctx[lo] + (r - s_cu[lo]);
        const int p = t / kPage;
        if (a.positions != nullptr) a.positions[r] = t;
        if (a.slots != nullptr) {
          int page = -1;
          if (p < s_held[lo]) {
            page = a.req_pages[(size_t)s_id[lo] * a.req_stride + p];
          } else {
            const int f = s_take[lo] + p - s_held[lo];
            if (f < a.num_free) page = ld_cg(a.free_pages + f);
          }
          a.slots[r] = page >= 0 && page <= (INT32_MAX - kPage) / kPage ? page * kPage + t % kPage : -1;
        }
      }
    }
    __syncthreads();  // the next round rewrites the shared arrays
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.cu_q[a.batch] = (int)min(rows0, (long long)a.total_q);
    if (a.pages_used != nullptr) *a.pages_used = min(pages0, a.num_free);
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

extern "C" s5_status s5_build_batch(const s5_request_desc *requests, const int32_t *req_ids, const int32_t *new_lens,
                                    const s5_batch_desc *batch, int32_t *slots, int32_t *positions,
                                    int32_t *pages_used, void *workspace, size_t workspace_bytes, s5_stream_t stream) {
  if (requests == nullptr || batch == nullptr || req_ids == nullptr || new_lens == nullptr) return S5_ERR_INVALID_ARG;
  if (requests->req_pages == nullptr || requests->num_reqs < 1 || requests->req_stride < 1 || requests->num_free < 0 ||
      (requests->num_free > 0 && requests->free_pages == nullptr))
    return S5_ERR_INVALID_ARG;
  if (batch->batch < 1 || batch->max_pages < 1 || batch->total_q < 0) return S5_ERR_INVALID_ARG;
  if (batch->page_table == nullptr || batch->ctx_lens == nullptr || batch->cu_q == nullptr) return S5_ERR_INVALID_ARG;
  if (batch->batch > kBMaxBatch || batch->max_pages > (1 << 20)) return S5_ERR_UNSUPPORTED;
  {  // page_table and req_pages must not overlap
    const uintptr_t t0 = reinterpret_cast<uintptr_t>(batch->page_table);
    const uintptr_t t1 = t0 + (size_t)batch->batch * batch->max_pages * sizeof(int32_t);
    const uintptr_t r0 = reinterpret_cast<uintptr_t>(requests->req_pages);
    const uintptr_t r1 = r0 + (size_t)requests->num_reqs * requests->req_stride * sizeof(int32_t);
    if (t0 < r1 && r0 < t1) return S5_ERR_INVALID_ARG;
  }
  if (workspace == nullptr || workspace_bytes < S5_WS_FIXED_BYTES) return S5_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 3u) != 0) return S5_ERR_INVALID_ARG;  // the error record's words

  BuildArgs a{};
  a.req_pages = requests->req_pages;
  a.free_pages = requests->free_pages;
  a.num_reqs = requests->num_reqs;
  a.req_stride = requests->req_stride;
  a.num_free = requests->num_free;
  a.req_ids = req_ids;
  a.ctx_lens = batch->ctx_lens;
  a.new_lens = new_lens;
  a.batch = batch->batch;
  a.max_pages = batch->max_pages;
  a.total_q = batch->total_q;
  // the table and the offsets are written: the descriptor's const covers the calls that read them
  a.page_table = const_cast<int32_t *>(batch->page_table);
  a.cu_q = const_cast<int32_t *>(batch->cu_q);
  a.slots = slots;
  a.positions = positions;
  a.pages_used = pages_used;
  a.err = static_cast<int32_t *>(workspace);
  const bool vec = batch->max_pages % 4 == 0 && requests->req_stride % 4 == 0 && aligned16(batch->page_table) &&
                   aligned16(requests->req_pages);
  const int rounds_seqs = batch->batch < kBSeqs ? batch->batch : kBSeqs;
  constexpr int kWarps = kBThreads / 32;
  const long long by_table = ((long long)rounds_seqs * ((batch->max_pages + kBCols - 1) / kBCols) + kWarps - 1) / kWarps;
  const long long by_rows = ((long long)batch->total_q + kBThreads - 1) / kBThreads;
  long long grid = by_table > by_rows ? by_table : by_rows;
  if (grid > 148 * 4) grid = 148 * 4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kBThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      vec ? cudaLaunchKernelEx(&cfg, build_batch_kernel<true>, a) : cudaLaunchKernelEx(&cfg, build_batch_kernel<false>, a);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? S5_OK : S5_ERR_CUDA;
}
