// Dense GQA of a batch's new tokens over the whole paged cache, bf16 or
// one-byte (E4M3) KV, on the 5th-generation tensor cores.
//
// For row r at position t, head h, group g = h / 16:
//   out = sum_{j <= t} softmax_j(sm_scale q.K_j) V_j,  lse = log sum_j exp(sm_scale q.K_j)
// computed in one pass over the cache with a running reference maximum and sum
// per (row, head); parts of a row's cache are joined by
//   M = max_p m_p,  O = sum_p 2^(m_p - M) O_p,  L = sum_p 2^(m_p - M) l_p.
//
// Bound: HBM.  A cached token costs 3,072 bytes (bf16) for 16 FLOPs per byte and
// query row, far below the tensor cores' ratio even for the 8 rows of a tile, so
// the aim is a full stream of pages on every SM.
//
// Split.  The work is a list of page units: sequences in order, in each its KV
// groups, in each group its tiles of `tile_rows` query rows, in each tile the
// pages up to its last row.  Every CTA (one per SM, persistent) finds its equal
// share of the list from the device's lengths by prefix sums, so ragged batches
// balance to within a page and one long sequence spreads over every SM.  A tile
// that spans CTAs leaves a part per CTA; the last CTA of a group of parts to
// arrive joins the group, the last group joins the groups (in CTA order, so
// results do not depend on who is last).
//
// One CTA works in chunks of two pages (128 tokens): warp 4 streams K and warp
// 5 V, one TMA copy per page and KV group, through rings of kStages chunks; warp
// 6 issues S = Q K^T (M = N = 128) and warp 7 O += P V (N = 192), both with A (Q,
// P) in tensor memory; warps 0-3, one thread per MMA row, load Q, run the softmax
// and finish each tile.  (N = 64 products take 56 cycles instead of 32, so single
// pages would cost the tensor pipe almost as much per page as chunks do per two.)
//
// The M = 128 rows for fewer than 128 (row, head) pairs.  MMA row
//   m = ((c * kSlots + slot) * RT + j) * 16 + h
// stands for tile row j, head h, copy c and slot.  A copy owns a run of 128 /
// copies tokens of every chunk: its P is zero elsewhere, it has its own reference
// and sum, and the copies are joined at the end; so all 128 threads work on
// the softmax of one decode row and none needs another's maximum.  A slot holds
// one term of the weights, the remainder of the terms before it, at no cost in
// MMAs: two terms carry a weight to 2^-15 in bf16 (8 rows: one term, 2^-8).  One
// byte: the weight in f16 (2^-12), whose upper byte is an E5M2 value; four such
// bytes, each of what the ones before leave, hold an f16 above 2^-16 exactly.
// (E4M3 terms took 7 conversions per pair of weights, at 8 cycles each: 2,000
// cycles of a chunk, against 370 for these.)
#include <cuda.h>

#include "s5_common.cuh"
#include "s5_kernels.h"
#include "s5_tcgen05.cuh"

namespace s5 {

namespace {

constexpr int kDnSoft = 128;  // softmax threads: warps 0-3
constexpr int kDnThreads = 256;
constexpr int kWarpK = 4, kWarpV = 5, kWarpS = 6, kWarpPv = 7;
constexpr int kChunk = 2 * kPage;               // tokens
constexpr int kScanPer = 4;                      // sequences per thread and round of the prefix sums
constexpr int kScanSeqs = kDnThreads * kScanPer;
constexpr uint64_t kDnWaitNs = 2000000000ull;    // 2 s per wait
constexpr uint32_t kDnHintNs = 1000;
constexpr int kMaxJoin = 16;                     // parts joined at a time (16 * 16 >= CTAs)
constexpr float kLn2 = 0.69314718055994531f;

// tensor memory columns
constexpr uint32_t kTmS = 0;    // 128: S of a chunk
constexpr uint32_t kTmP = 128;  // 64: P of a chunk (one byte: 32 per term)
constexpr uint32_t kTmO = 192;  // 192: O
constexpr uint32_t kTmQ = 384;  // 96: Q (bf16: two dims per column; one byte: two terms of 48 columns)
constexpr uint32_t kTmCols = 512;

template <bool KV8, int RT>
struct Cfg {
  // term slots.  bf16: the weight and its remainder, unless 8 rows take every MMA row.
  // One byte: 4 one-term slots, or (2 and 4 rows) 2 slots of two terms each.
  static constexpr int kSlots = KV8 ? (RT == 1 ? 4 : 2) : (RT == 8 ? 1 : 2);
  static constexpr int kTerms = KV8 ? 4 / kSlots : 1;  // unscaled terms per slot (MMA passes of P V)
  static constexpr int kCopies = 8 / (RT * kSlots);
  static constexpr int kTok = kChunk / kCopies;        // tokens of a chunk per softmax thread
  static constexpr int kPageBytes = kPage * kD * (KV8 ? 1 : 2);
  // a page in shared memory: [8 groups of 8 tokens][3 planes of 64 dims][8 tokens][kRowB], so
  // that 8-token groups are evenly spaced across the pages of a chunk
  static constexpr int kRowB = KV8 ? 64 : 128;
  static constexpr int kPlane = 8 * kRowB;
  static constexpr int kGroup = 3 * kPlane;
  static constexpr int kStages = KV8 ? 4 : 2;          // chunks per ring
  static constexpr int kStageBytes = 2 * kPageBytes;
  // The reference sits kOff binades under the maximum it was taken from and moves when a weight
  // would exceed 2^kTop.  One byte: f16 weights reach 2^15, E5M2 ones go down to 2^-16, so
  // weights of 2^-28 of the largest still count.
  static constexpr float kOff = KV8 ? 12.f : 0.f;
  static constexpr float kTop = KV8 ? 15.f : 8.f;
  static_assert(kCopies >= 1 && kCopies * kSlots * RT == 8, "128 MMA rows");
  // shared memory (from a 1,024-byte aligned base)
  static constexpr int kOffV = kStages * kStageBytes;
  static constexpr int kOffStage = 2 * kStages * kStageBytes; // float [2][128][20]: epilogue; join weights
  static constexpr int kOffMl = kOffStage + 2 * 128 * 20 * 4; // float [2][128]: references and sums
  static constexpr int kOffBad = kOffMl + 2 * 128 * 4;        // uint32 [48]: per dim, rows that saw a non-finite value
  static constexpr int kOffBar = kOffBad + 192;
  static constexpr int kNumBars = 4 * kStages + 16;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffMisc + 256 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

// ---------------------------------------------------------------- the list of page units

// Sum over i < n of floor(i / w): full groups of w, then the rest.
__device__ __forceinline__ long long floor_sum(long long n, int w) {
  const long long q = n / w;
  return w * (q * (q - 1) / 2) + q * (n - w * q);
}

// Pages of the first m tiles of a sequence with ctx cached tokens when those
// tiles are full: sum over k < m of ceil((ctx + RT (k + 1)) / 64).
template <int RT>
__device__ __forceinline__ long long full_tile_pages(int ctx, int m) {
  constexpr int w = kPage / RT;
  const long long b = ((long long)ctx + kPage - 1 + RT) / RT;
  return floor_sum(b + m, w) - floor_sum(b, w);
}

struct Seq {
  int lo, n, ctx;  // first row, rows (0: none to compute), cached tokens
  bool bad;
};

__device__ __forceinline__ Seq load_seq(const DenseArgs &a, int s) {
  Seq q;
  q.lo = ld_cg(a.cu_q + s);
  const int hi = ld_cg(a.cu_q + s + 1);
  q.ctx = ld_cg(a.ctx_lens + s);
  q.bad = q.lo < 0 || hi < q.lo || hi > a.total_q;
  q.n = q.bad ? 0 : hi - q.lo;
  if (q.n > 0 && (q.ctx < 0 || q.ctx > a.max_len - q.n)) {
    q.bad = true;
    q.n = 0;
  }
  return q;
}

template <int RT>
__device__ __forceinline__ long long group_pages(const Seq &q) {  // of one KV group of the sequence
  if (q.n <= 0) return 0;
  const int tiles = (q.n + RT - 1) / RT;
  const long long last = (q.ctx + q.n + kPage - 1) / kPage;
  return tiles == 1 ? last : full_tile_pages<RT>(q.ctx, tiles - 1) + last;
}

// A run of pages of one tile.
struct Seg {
  int s, g, row0, nr, t0;    // sequence, KV group, first row, rows, position of the first row
  int p0, np, tile_pages;    // first page, pages, pages of the whole tile
  long long tile_u;          // unit of the tile's first page
};

// The runs of one CTA in order.  Every warp walks them by itself.
template <int RT>
struct Walk {
  const DenseArgs &a;
  Seq q;
  int s, g, k, p;
  long long u, rem;

  __device__ Walk(const DenseArgs &args, int s0, long long off, long long u0, long long count)
      : a(args), s(s0), u(u0), rem(count) {
    q = load_seq(a, s);
    const long long per = group_pages<RT>(q);
    g = (int)(off / per);
    const long long o = off - g * per;
    int lo = 0, hi = (q.n + RT - 1) / RT;  // the last tile k whose pages before are <= o
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (full_tile_pages<RT>(q.ctx, mid) <= o) lo = mid;
      else hi = mid;
    }
    k = lo;
    p = (int)(o - full_tile_pages<RT>(q.ctx, k));
  }

  __device__ bool next(Seg &x) {
    if (rem <= 0) return false;
    const int nr = min(RT, q.n - k * RT);
    x.s = s;
    x.g = g;
    x.row0 = q.lo + k * RT;
    x.nr = nr;
    x.t0 = q.ctx + k * RT;
    x.tile_pages = (x.t0 + nr + kPage - 1) / kPage;
    x.p0 = p;
    x.np = (int)min((long long)(x.tile_pages - p), rem);
    x.tile_u = u - p;
    u += x.np;
    rem -= x.np;
    p += x.np;
    if (p == x.tile_pages) {
      p = 0;
      if (++k * RT >= q.n) {
        k = 0;
        if (++g == kKv) {
          g = 0;
          q.n = 0;
          while (rem > 0 && q.n == 0 && ++s < a.batch) q = load_seq(a, s);
          if (q.n == 0) rem = 0;
        }
      }
    }
    return true;
  }
};

// ---------------------------------------------------------------- small arithmetic

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)), "l"(*reinterpret_cast<uint64_t *>(&c)));
  return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
  return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// two f16 values to two E4M3 codes (nearest, saturating) and back (exact)
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t h) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
  return c;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return h;
}
__device__ __forceinline__ uint32_t float2_to_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  const __half2 v = __hsub2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Q of one MMA row into tensor memory, negated when the scale is negative: bf16 as
// it is.
__device__ __forceinline__ void load_q_bf16(const DenseArgs &a, size_t qrow, bool on, uint32_t tq) {
  const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
  const uint4 *src = reinterpret_cast<const uint4 *>(a.q) + qrow * (kD / 8);
#pragma unroll
  for (int x = 0; x < kD / 32; ++x) {
    uint32_t w[16];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const uint4 v = on ? ld_cg(src + 4 * x + y) : make_uint4(0, 0, 0, 0);
      w[4 * y] = v.x ^ flip;
      w[4 * y + 1] = v.y ^ flip;
      w[4 * y + 2] = v.z ^ flip;
      w[4 * y + 3] = v.w ^ flip;
    }
    tc::st_16cols(tq + 16 * x, w);
  }
}

// Q of one MMA row as two E4M3 terms (the value and its remainder) of q times a
// power of two that puts the row's largest magnitude in [2^7, 2^8); returns the
// inverse of that power.  Two 4-bit terms hold a bf16's 8 bits exactly down to
// 2^-10 of the largest magnitude; smaller values are rounded to 2^-17 of it.
__device__ __forceinline__ float load_q_e4m3(const DenseArgs &a, size_t qrow, bool on, uint32_t tq) {
  const uint4 *src = reinterpret_cast<const uint4 *>(a.q) + qrow * (kD / 8);
  float top = 0.f;
  bool finite = true;
  if (on) {
#pragma unroll 4
    for (int x = 0; x < kD / 8; ++x) {
      const uint4 v = ld_cg(src + x);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float f0 = fabsf(bf16lo(w[y])), f1 = fabsf(bf16hi(w[y]));
        finite = finite && f0 < INFINITY && f1 < INFINITY;
        top = max3(top, f0, f1);
      }
    }
  }
  const int e = (int)(__float_as_uint(top) >> 23);  // biased exponent of the largest magnitude
  float up = finite ? __uint_as_float((uint32_t)min(261 - e, 254) << 23) : __uint_as_float(0x7FC00000u);
  if (a.scale_log2 < 0.f) up = -up;
  const float down = e > 7 ? __uint_as_float((uint32_t)(e - 7) << 23) : __uint_as_float(0x00400000u);
#pragma unroll
  for (int x = 0; x < kD / 32; ++x) {
    uint32_t t0[8], t1[8];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const uint4 v = on ? ld_cg(src + 4 * x + y) : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int z = 0; z < 4; z += 2) {
        uint32_t c0 = 0, c1 = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t h = float2_to_f16x2(bf16lo(w[z + i]) * up, bf16hi(w[z + i]) * up);
          const uint32_t c = f16x2_to_e4m3x2(h);
          c0 |= c << (16 * i);
          c1 |= f16x2_to_e4m3x2(sub_f16x2(h, e4m3x2_to_f16x2(c))) << (16 * i);
        }
        t0[2 * y + z / 2] = c0;
        t1[2 * y + z / 2] = c1;
      }
    }
    tc::st_8cols(tq + 8 * x, t0);
    tc::st_8cols(tq + 48 + 8 * x, t1);
  }
  return down;
}

// ---------------------------------------------------------------- the kernel

template <bool KV8, int RT>
__global__ void __launch_bounds__(kDnThreads, 1)
    dense_kernel(const DenseArgs a, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<KV8, RT>;
  constexpr int NS = C::kStages, PB = C::kPageBytes, SB = C::kStageBytes, kPairs = RT * kHpg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sk = smem, *sv = smem + C::kOffV;
  float *stage = reinterpret_cast<float *>(smem + C::kOffStage);
  float *ml_s = reinterpret_cast<float *>(smem + C::kOffMl);
  uint32_t *bad_s = reinterpret_cast<uint32_t *>(smem + C::kOffBad);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
  uint64_t *k_full = bars, *k_empty = bars + NS, *v_full = bars + 2 * NS, *v_empty = bars + 3 * NS;
  uint64_t *s_full = bars + 4 * NS, *s_empty = s_full + 1, *p_full = s_full + 2, *p_free = s_full + 3;
  uint64_t *q_full = s_full + 4, *q_empty = s_full + 5, *o_empty = s_full + 6, *b_soft = s_full + 7,
           *b_flag = s_full + 8, *b_final = s_full + 9;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
  int *abort_flag = reinterpret_cast<int *>(smem + C::kOffMisc + 4);
  int *flag_s = reinterpret_cast<int *>(smem + C::kOffMisc + 8);
  int *start_s = reinterpret_cast<int *>(smem + C::kOffMisc + 12);
  int *n_bad_s = reinterpret_cast<int *>(smem + C::kOffMisc + 16);
  long long *off_s = reinterpret_cast<long long *>(smem + C::kOffMisc + 24);
  long long *sum_s = reinterpret_cast<long long *>(smem + C::kOffMisc + 32);  // [8]
  int *bad_list = reinterpret_cast<int *>(stage);                             // [kScanSeqs], before the pipeline runs

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 4 * NS; ++i) mbar_init(bars + i, 1);
    mbar_init(s_full, 1);
    mbar_init(s_empty, 4);
    mbar_init(p_full, 4);
    mbar_init(p_free, 1);
    mbar_init(q_full, 4);
    mbar_init(q_empty, 1);
    mbar_init(o_empty, 4);
    mbar_init(b_soft, kDnSoft);
    mbar_init(b_flag, 1);
    mbar_init(b_final, 2);
    *abort_flag = 0;
    *n_bad_s = 0;
    *start_s = -1;
  }
  if (tid < 48) bad_s[tid] = 0;
  fence_mbar_init();
  __syncthreads();
  pdl_wait();  // (programmatic launch) global memory is read from here on

  // ---- this CTA's share: prefix sums of the sequences' page units ----
  const int rounds = (a.batch + kScanSeqs - 1) / kScanSeqs;
  long long total = 0, units[kScanPer], before = 0;
  auto scan_round = [&](int r, bool report) {  // units[] of this thread's sequences; exclusive prefix in `before`
    long long mine = 0;
#pragma unroll
    for (int i = 0; i < kScanPer; ++i) {
      const int s = r * kScanSeqs + tid * kScanPer + i;
      units[i] = 0;
      if (s < a.batch) {
        const Seq q = load_seq(a, s);
        units[i] = kKv * group_pages<RT>(q);
        if (q.bad && report && s % (int)gridDim.x == (int)blockIdx.x) {
          record_error(a.err, S5_ERR_DEVICE_BOUNDS, max(q.lo, 0));
          bad_list[atomicAdd(n_bad_s, 1)] = s;
        }
      }
      mine += units[i];
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sum_s[warp] = incl;
    __syncthreads();
    before = incl - mine;
    long long all = 0;
#pragma unroll
    for (int w = 0; w < kDnThreads / 32; ++w) {
      if (w < warp) before += sum_s[w];
      all += sum_s[w];
    }
    // rows of bad sequences: zeros
    const int nb = *n_bad_s;
    for (int b = 0; b < nb; ++b) {
      const int s = bad_list[b];
      const int lo = max(ld_cg(a.cu_q + s), 0), hi = min(ld_cg(a.cu_q + s + 1), a.total_q);
      for (long long i = (long long)lo * kHeads * (kD / 8) + tid; i < (long long)hi * kHeads * (kD / 8); i += kDnThreads)
        reinterpret_cast<uint4 *>(a.out)[i] = make_uint4(0, 0, 0, 0);
      if (a.lse != nullptr)
        for (long long i = (long long)lo * kHeads + tid; i < (long long)hi * kHeads; i += kDnThreads) a.lse[i] = -INFINITY;
    }
    __syncthreads();
    if (tid == 0) *n_bad_s = 0;
    __syncthreads();
    return all;
  };
  for (int r = 0; r < rounds; ++r) total += scan_round(r, true);
  const long long chunk = max((total + gridDim.x - 1) / gridDim.x, 1LL);
  const long long u0 = chunk * blockIdx.x;
  if (u0 >= total) return;
  const long long count = min(chunk, total - u0);
  {
    long long base = 0;
    for (int r = 0; r < rounds; ++r) {
      const long long all = rounds > 1 ? scan_round(r, false) : total;
      long long at = base + before;
#pragma unroll
      for (int i = 0; i < kScanPer; ++i) {
        if (at <= u0 && u0 < at + units[i]) {
          *start_s = r * kScanSeqs + tid * kScanPer + i;
          *off_s = u0 - at;
        }
        at += units[i];
      }
      base += all;
      if (base > u0) break;
    }
  }
  if (warp == 0) tc::tmem_alloc(tmem_slot, kTmCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  Walk<RT> walk(a, *start_s, *off_s, u0, count);
  Seg x;

  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (*reinterpret_cast<volatile int *>(abort_flag)) return false;
    if (mbar_wait_bounded_hint(bar, parity, kDnWaitNs, kDnHintNs)) return true;
    *reinterpret_cast<volatile int *>(abort_flag) = 1;
    record_error(a.err, S5_ERR_TIMEOUT, 0);
    return false;
  };

  if (warp == kWarpK || warp == kWarpV) {
    // ---------------- TMA producers ----------------
    const bool is_k = warp == kWarpK;
    uint8_t *ring = is_k ? sk : sv;
    const CUtensorMap *map = is_k ? &tm_k : &tm_v;
    uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
    const uint64_t policy = a.reread ? policy_evict_normal() : policy_evict_first();
    int gc = 0;
    bool ok = true;
    while (ok && walk.next(x)) {
      const int32_t *pt = a.page_table + (size_t)x.s * a.max_pages + x.p0;
      int ids = lane < x.np ? ld_cg(pt + lane) : -1;  // pages c .. c + 31, one per lane; the next 32 in flight
      for (int c = 0; c < x.np && ok; c += 32) {
        const int nxt = c + 32 + lane < x.np ? ld_cg(pt + c + 32 + lane) : -1;
        const int m = min(32, x.np - c);
        for (int i = 0; i < m; i += 2, ++gc) {
          const int page[2] = {__shfl_sync(0xffffffffu, ids, i), __shfl_sync(0xffffffffu, ids, i + 1)};
          int go = 1;
          if (lane == 0) {
            const int st = gc % NS;
            if (gc >= NS) go = wait(empty + st, ((gc / NS) - 1) & 1) ? 1 : 0;
            if (go) {
              bool page_ok[2];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                page_ok[y] = page[y] >= 0 && page[y] < a.num_pages;
                if (!page_ok[y] && is_k && i + y < m) record_error(a.err, S5_ERR_DEVICE_BOUNDS, x.row0);
              }
              mbar_arrive_expect_tx(full + st, (page_ok[0] ? PB : 0) + (page_ok[1] ? PB : 0));
#pragma unroll
              for (int y = 0; y < 2; ++y)
                if (page_ok[y])
                  tma_load_4d(ring + st * SB + y * PB, map, 0, 0, 0, (page[y] * kKv + x.g) * (kPage / 8), full + st, policy);
            }
          }
          if (!__shfl_sync(0xffffffffu, go, 0)) {
            ok = false;
            break;
          }
        }
        ids = nxt;
      }
    }
    // no copy may still be writing shared memory when the CTA retires
    if (lane == 0)
      for (int c = max(0, gc - NS); c < gc; ++c) mbar_wait_bounded(full + c % NS, (c / NS) & 1, kDnWaitNs);
  } else if (warp == kWarpS) {
    // ---------------- S = Q K^T ----------------
    if (lane == 0) {
      const uint32_t k_base = smem_u32(sk);
      int gc = 0, qi = 0;
      bool ok = true;
      while (ok && walk.next(x)) {
        if (!wait(q_full, qi & 1)) break;
        for (int c = 0; c < x.np; c += 2, ++gc) {
          const int st = gc % NS;
          if (!wait(k_full + st, (gc / NS) & 1) || (gc >= 1 && !wait(s_empty, (gc - 1) & 1))) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint32_t kb = k_base + st * SB;
          const int n = c + 1 < x.np ? 2 * kPage : kPage;  // (a run's last page may stand alone)
          if constexpr (KV8) {
            const uint32_t idesc = tc::idesc_f8_f32(128, n, 0, false);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int kk = 0; kk < kD / 32; ++kk)
                tc::mma_f8_ts(tmem + kTmS, tmem + kTmQ + t * 48 + kk * 8,
                                tc::smem_desc_sw64(kb + (kk >> 1) * C::kPlane + (kk & 1) * 32, 16, C::kGroup), idesc,
                                t + kk > 0);
          } else {
            const uint32_t idesc = tc::idesc_bf16_f32(128, n);
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk)
              tc::mma_bf16_ts(tmem + kTmS, tmem + kTmQ + kk * 8,
                              tc::smem_desc_k_sw128_stride(kb + (kk >> 2) * C::kPlane + (kk & 3) * 32, C::kGroup), idesc,
                              kk > 0);
          }
          tc::commit(k_empty + st);
          tc::commit(s_full);
          if (c + 2 >= x.np) tc::commit(q_empty);
        }
        ++qi;
      }
      tc::commit(b_final);  // arrives once every MMA issued above has completed
    }
  } else if (warp == kWarpPv) {
    // ---------------- O += P V ----------------
    if (lane == 0) {
      const uint32_t v_base = smem_u32(sv);
      int gc = 0, qi = 0;
      bool ok = true;
      while (ok && walk.next(x)) {
        for (int c = 0; c < x.np; c += 2, ++gc) {
          const int st = gc % NS;
          if (!wait(p_full, gc & 1) || !wait(v_full + st, (gc / NS) & 1) ||
              (c == 0 && qi > 0 && !wait(o_empty, (qi - 1) & 1))) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint32_t vb = v_base + st * SB, pa = tmem + kTmP;
          const int m = c + 1 < x.np ? 2 : 1;
          if constexpr (KV8) {
            constexpr uint32_t idesc = tc::idesc_f8_f32(128, kD, 1, true);
#pragma unroll
            for (int t = 0; t < C::kTerms; ++t)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                if (ks < 2 * m)
                  tc::mma_f8_ts(tmem + kTmO, pa + t * 32 + ks * 8,
                                  tc::smem_desc_sw64(vb + ks * 4 * C::kGroup, C::kPlane, C::kGroup), idesc, c + t + ks > 0);
          } else {
            constexpr uint32_t idesc = tc::idesc_bf16_f32_bmn(128, kD);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              if (ks < 4 * m)
                tc::mma_bf16_ts(tmem + kTmO, pa + ks * 8,
                                tc::smem_desc_mn_sw128(vb + ks * 2 * C::kGroup, C::kPlane, C::kGroup), idesc, c + ks > 0);
          }
          tc::commit(v_empty + st);
          tc::commit(p_free);
        }
        ++qi;
      }
      tc::commit(b_final);
    }
  } else {
    // ---------------- softmax and epilogue: one thread per MMA row ----------------
    const int h = tid & 15, j = (tid >> 4) % RT, slot = (tid / kPairs) % C::kSlots, cp = tid / (kPairs * C::kSlots);
    const int pr = tid % kPairs;  // (row, head) pair of the tile
    const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
    constexpr int TOK = C::kTok;
    int gc = 0, qi = 0, n_soft = 0, n_flag = 0;
    bool ok = true;
    // a warp leaves together: if any lane gave up, all do
    auto wait_warp = [&](uint64_t *bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait(bar, parity));
    };
    auto soft_sync = [&]() -> bool {  // the 128 threads of these warps
      mbar_arrive(b_soft);
      return wait_warp(b_soft, n_soft++ & 1);
    };
    {  // P is zero outside each copy's tokens, for good
      const uint32_t z[16] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) tc::st_16cols(tl + kTmP + 16 * i, z);
      tc::wait_st();
    }
    while (ok && walk.next(x)) {
      const bool row_ok = j < x.nr;
      const int t_row = x.t0 + j, t_last = x.t0 + x.nr - 1;
      float m_ref = -INFINITY, l = 0.f, sl2 = fabsf(a.scale_log2);
      // (a score of -inf, masked or not, has weight 0 with a scale of 0 too)
      if (qi > 0 && !wait_warp(q_empty, (qi - 1) & 1)) break;
      {
        const size_t qrow = (size_t)(x.row0 + j) * kHeads + x.g * kHpg + h;
        if constexpr (KV8) sl2 *= load_q_e4m3(a, qrow, row_ok, tl + kTmQ);
        else load_q_bf16(a, qrow, row_ok, tl + kTmQ);
        sl2 = fmaxf(sl2, 1e-37f);
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      const int32_t *pt = a.page_table + (size_t)x.s * a.max_pages + x.p0;
      int ids = -1, nxt = lane < x.np ? ld_cg(pt + lane) : -1;
      for (int c = 0; c < x.np; c += 2, ++gc) {
        if ((c & 31) == 0) {
          ids = nxt;
          nxt = c + 32 + lane < x.np ? ld_cg(pt + c + 32 + lane) : -1;
        }
        // (a page behind the run's last reads as -1: no token of it is visible)
        const int pa = __shfl_sync(0xffffffffu, ids, c & 31), pb = __shfl_sync(0xffffffffu, ids, (c & 31) + 1);
        const bool ok_a = pa >= 0 && pa < a.num_pages, ok_b = pb >= 0 && pb < a.num_pages;
        const int base = (x.p0 + c) * kPage;
        const bool masked = !ok_a || !ok_b || base + kChunk - 1 > x.t0;
        // tokens 0 .. lim of this thread's run are visible to its row, past the 64th those to lim_b
        const int lim0 = t_row - base - cp * TOK;
        const int lim = (TOK == kChunk || cp * TOK < kPage ? ok_a : ok_b) ? lim0 : -1;
        const int lim_b = ok_b ? lim0 : -1;
        if (!wait_warp(s_full, gc & 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        uint32_t v[TOK];
#pragma unroll
        for (int i = 0; i < TOK / 32; ++i)
          tc::ld_32cols(tl + kTmS + cp * TOK + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * i));
        tc::wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty);
        if (masked) {
#pragma unroll
          for (int i = 0; i < TOK; ++i)
            if (i > (i < kPage ? lim : lim_b)) v[i] = 0xFF800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < TOK; i += 2)
          mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
        // scores in log2 units are sl2 * S (sl2 >= 0: a negative scale's sign is in Q)
        const float raw = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const float top = raw * sl2;
        // the reference moves only when a weight would exceed 2^kTop (or with the first finite score)
        const bool first = m_ref == -INFINITY;
        const bool grow = first ? top > -INFINITY : top - m_ref > C::kTop;
        const bool resc = grow && !first;
        const float m_old = m_ref;
        if (grow) m_ref = top - C::kOff;
        if (__any_sync(0xffffffffu, resc)) {
          const float corr = resc ? hw_exp2(m_old - m_ref) : 1.f;
          if (c > 0) {  // O holds the chunks before: after their last product
            if (!wait_warp(p_free, (gc - 1) & 1)) {
              ok = false;
              break;
            }
            tc::fence_after_sync();
#pragma unroll 1
            for (int cb = 0; cb < kD / 16; ++cb) {
              uint32_t o[16];
              tc::ld_16cols(tl + kTmO + cb * 16, o);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
              tc::st_16cols(tl + kTmO + cb * 16, o);
            }
            tc::wait_st();
          }
          l *= corr;
        }
        const float mu = (m_ref == -INFINITY) ? 0.f : m_ref;
        float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // this slot's term of the weights: the upper half (one byte: E5M2 byte) of what the slots
        // before it, taking the same toward zero, leave
        uint32_t pk[C::kTerms][TOK / (KV8 ? 4 : 2)];
#pragma unroll
        for (int i = 0; i < TOK; i += KV8 ? 4 : 2) {
          float2 p2[2];
#pragma unroll
          for (int y = 0; y < (KV8 ? 2 : 1); ++y) {
            const float2 s2 = fma2(make_float2(__uint_as_float(v[i + 2 * y]), __uint_as_float(v[i + 2 * y + 1])),
                                   make_float2(sl2, sl2), make_float2(-mu, -mu));
            p2[y] = make_float2(hw_exp2(s2.x), hw_exp2(s2.y));
            ps[y ^ ((i >> 1) & 1)] = add2(ps[y ^ ((i >> 1) & 1)], p2[y]);
          }
          if constexpr (KV8) {
            uint32_t r[2] = {float2_to_f16x2(p2[0].x, p2[0].y), float2_to_f16x2(p2[1].x, p2[1].y)};
#pragma unroll
            for (int y = 0; y < (C::kSlots - 1) * C::kTerms; ++y)
#pragma unroll
              for (int z = 0; z < 2; ++z) r[z] = sub_f16x2(r[z], r[z] & (slot * C::kTerms > y ? 0xFF00FF00u : 0u));
#pragma unroll
            for (int t = 0; t < C::kTerms; ++t) {
              pk[t][i / 4] = __byte_perm(r[0], r[1], 0x7531);
              if (t + 1 < C::kTerms)
#pragma unroll
                for (int z = 0; z < 2; ++z) r[z] = sub_f16x2(r[z], r[z] & 0xFF00FF00u);
            }
          } else if constexpr (C::kSlots == 2) {
            const uint32_t cut = slot ? 0xFFFF0000u : 0u;
            const float2 r = fma2(make_float2(__uint_as_float(__float_as_uint(p2[0].x) & cut),
                                              __uint_as_float(__float_as_uint(p2[0].y) & cut)),
                                  make_float2(-1.f, -1.f), p2[0]);
            pk[0][i / 2] = __byte_perm(__float_as_uint(r.x), __float_as_uint(r.y), 0x7632);
          } else {
            pk[0][i / 2] = pack_bf16(p2[0].x, p2[0].y);
          }
        }
        l += (ps[0].x + ps[1].x) + (ps[0].y + ps[1].y);
        // P, last read by the product of the chunk before
        if (gc >= 1 && !wait_warp(p_free, (gc - 1) & 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        constexpr int PC = TOK / (KV8 ? 4 : 2);  // columns of a term
#pragma unroll
        for (int t = 0; t < C::kTerms; ++t) {
          const uint32_t tp = tl + kTmP + t * 32 + cp * PC;
          if constexpr (PC == 8) tc::st_8cols(tp, *reinterpret_cast<const uint32_t(*)[8]>(pk[t]));
          else
#pragma unroll
            for (int i = 0; i < PC / 16; ++i) tc::st_16cols(tp + 16 * i, *reinterpret_cast<const uint32_t(*)[16]>(pk[t] + 16 * i));
        }
        if (masked) {
          // V of tokens that a row of the tile does not see must not be NaN or infinite (P is 0 there,
          // but 0 * NaN is NaN): tokens that no row sees become zeros; in tokens that some rows see, a
          // value that is not finite becomes zero and is noted for the rows that see it
          const int st = gc % NS;
          if (!wait_warp(v_full + st, (gc / NS) & 1)) {
            ok = false;
            break;
          }
          uint8_t *vb = sv + st * SB;
          constexpr int kPieces = C::kRowB / 16;  // 16-byte pieces of a token in a plane
          const int n_tok = c + 1 < x.np ? kChunk : kPage;
          // from the first token of a bad page, or the first that some row does not see
          const int first_tok = !ok_a ? 0 : min(max(x.t0 + 1 - base, 0), ok_b ? kChunk : kPage);
          for (int i = first_tok * 3 * kPieces + tid; i < n_tok * 3 * kPieces; i += kDnSoft) {
            const int tok = i / (3 * kPieces), y = i % (3 * kPieces), plane = y / kPieces, piece = y % kPieces;
            uint4 *at = reinterpret_cast<uint4 *>(vb + (tok >> 3) * C::kGroup + plane * C::kPlane + (tok & 7) * C::kRowB +
                                                  piece * 16);
            if (!(tok < kPage ? ok_a : ok_b) || base + tok > t_last) {
              *at = make_uint4(0, 0, 0, 0);
            } else if (base + tok > x.t0) {
              const int swz = KV8 ? (tok >> 1) & 3 : tok & 7;
              const int d0 = plane * 64 + (piece ^ swz) * (KV8 ? 16 : 8);
              // rows whose position is at least the token's
              const uint32_t rows = (0xFFu << (base + tok - x.t0)) & 0xFFu;
              uint32_t w[4] = {at->x, at->y, at->z, at->w};
              bool hit = false;
#pragma unroll
              for (int e = 0; e < (KV8 ? 16 : 8); ++e) {
                const int sh = KV8 ? 8 * (e & 3) : 16 * (e & 1);
                uint32_t &word = w[KV8 ? e >> 2 : e >> 1];
                const uint32_t bits = word >> sh;
                if (KV8 ? (bits & 0x7Fu) == 0x7Fu : (bits & 0x7F80u) == 0x7F80u) {
                  hit = true;
                  word &= ~((KV8 ? 0xFFu : 0xFFFFu) << sh);
                  atomicOr(bad_s + (d0 + e) / 4, rows << (8 * ((d0 + e) & 3)));
                }
              }
              if (hit) *at = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          fence_proxy_async_smem();
        }
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (!ok) break;

      // ---- the run's result: copies and slots summed ----
      ml_s[tid] = m_ref;
      ml_s[128 + tid] = l;
      if (!soft_sync()) {
        ok = false;
        break;
      }
      float M = -INFINITY;
#pragma unroll
      for (int i = 0; i < C::kCopies; ++i) M = fmaxf(M, ml_s[i * kPairs * C::kSlots + pr]);
      const float Mu = (M == -INFINITY) ? 0.f : M;
      float L = 0.f;
#pragma unroll
      for (int i = 0; i < C::kCopies; ++i)
        L += hw_exp2(ml_s[i * kPairs * C::kSlots + pr] - Mu) * ml_s[128 + i * kPairs * C::kSlots + pr];
      const bool whole = x.np == x.tile_pages;
      const float own = hw_exp2(m_ref - Mu) * (whole ? (L == 0.f ? 0.f : a.v_scale / L) : 1.f);
      // parts of a tile: CTA index within the tile, its slot of partial results
      const int c_first = whole ? 0 : (int)(x.tile_u / chunk);
      const int n_parts = whole ? 1 : (int)((x.tile_u + x.tile_pages - 1) / chunk) - c_first + 1;
      const int me = whole ? 0 : (int)blockIdx.x - c_first;
      auto part_slot = [&](int i) { return 2 * (c_first + i) + (i == 0 ? 1 : 0); };
      float *po = a.part_o + (size_t)part_slot(me) * kPairs * kD;
      if (tid < kPairs && row_ok) {
        if (whole) {
          if (a.lse != nullptr)
            a.lse[(size_t)(x.row0 + j) * kHeads + x.g * kHpg + h] = L == 0.f ? -INFINITY : (M + hw_log2(L)) * kLn2;
        } else {
          float *ml = a.part_ml + (size_t)part_slot(me) * 2 * kPairs;
          ml[pr] = M;
          ml[kPairs + pr] = L;
        }
      }
      if (!wait_warp(p_free, (gc - 1) & 1)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
#pragma unroll 1
      for (int cb = 0; cb < kD / 16; ++cb) {
        float *sg = stage + (cb & 1) * 128 * 20;
        uint32_t o[16];
        tc::ld_16cols(tl + kTmO + cb * 16, o);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4 *>(sg + tid * 20 + i) =
              make_float4(__uint_as_float(o[i]) * own, __uint_as_float(o[i + 1]) * own, __uint_as_float(o[i + 2]) * own,
                          __uint_as_float(o[i + 3]) * own);
        if (!soft_sync()) {
          ok = false;
          break;
        }
        for (int i = tid; i < kPairs * 4; i += kDnSoft) {
          const int q = i >> 2, d = cb * 16 + (i & 3) * 4, jj = q >> 4;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int z = 0; z < C::kCopies * C::kSlots; ++z) {
            const float4 y = *reinterpret_cast<const float4 *>(sg + (z * kPairs + q) * 20 + (i & 3) * 4);
            acc.x += y.x;
            acc.y += y.y;
            acc.z += y.z;
            acc.w += y.w;
          }
          const uint32_t nf = bad_s[d / 4] >> jj;  // byte e: dim d + e, bit 0: this row saw a value that is not finite
          if (nf & 0x01010101u) {
            if (nf & 1u) acc.x = __uint_as_float(0x7FC00000u);
            if (nf & 0x100u) acc.y = __uint_as_float(0x7FC00000u);
            if (nf & 0x10000u) acc.z = __uint_as_float(0x7FC00000u);
            if (nf & 0x1000000u) acc.w = __uint_as_float(0x7FC00000u);
          }
          if (jj < x.nr) {
            if (whole) {
              uint2 w2;
              w2.x = pack_bf16(acc.x, acc.y);
              w2.y = pack_bf16(acc.z, acc.w);
              *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) +
                                         ((size_t)(x.row0 + jj) * kHeads + x.g * kHpg + (q & 15)) * kD + d) = w2;
            } else {
              *reinterpret_cast<float4 *>(po + (size_t)q * kD + d) = acc;
            }
          }
        }
      }
      if (!ok) break;
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty);
      ++qi;
      if (!soft_sync()) {  // bad_s, stage and ml_s are free again
        ok = false;
        break;
      }
      if (tid < 48) bad_s[tid] = 0;
      if (whole) continue;

      // ---- join the tile's parts: groups of `gs` consecutive CTAs, then the groups ----
      int gs = n_parts;
      if (n_parts > 8) {
        gs = 3;
        while (gs * gs < n_parts) ++gs;
      }
      const int n_groups = (n_parts + gs - 1) / gs, grp = me / gs;
      int level = 0;
      while (true) {
        // level 0: the parts of group grp; level 1: the groups
        const int lead = level == 0 ? grp * gs : 0;
        const int n = level == 0 ? min(gs, n_parts - lead) : n_groups;
        __threadfence();
        mbar_arrive(b_soft);
        if (tid == 0) {
          int last = 0;
          if (wait(b_soft, n_soft & 1)) {
            __threadfence();
            uint32_t *cnt = a.cnt + (level == 0 ? part_slot(lead) : 2 * (int)gridDim.x + c_first);
            last = atomicAdd(cnt, 1u) == (uint32_t)n - 1 ? 1 : 0;
            if (last) atomicExch(cnt, 0u);  // every part has arrived: ready for the next call
          }
          *flag_s = last;
          __threadfence();
          mbar_arrive(b_flag);
        }
        ++n_soft;
        if (!wait_warp(b_flag, n_flag++ & 1)) {
          ok = false;
          break;
        }
        if (!*flag_s) break;
        __threadfence();
        const bool final = level == 1 || n_groups == 1;
        const int step = level == 0 ? 1 : gs;
        // (a group's joined reference and sum lie behind the parts', its joined O in its first part)
        auto ml_of = [&](int i) {
          return a.part_ml + ((size_t)part_slot(lead + i * step) + (level == 0 ? 0 : 2 * (size_t)gridDim.x)) * 2 * kPairs;
        };
        float *wt = stage;  // [n][kPairs] weights
        if (tid < kPairs && row_ok) {
          float mv[kMaxJoin], lv[kMaxJoin], top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int i = 0; i < kMaxJoin; ++i) {
            mv[i] = i < n ? ld_cg(ml_of(i) + pr) : -INFINITY;
            lv[i] = i < n ? ld_cg(ml_of(i) + kPairs + pr) : 0.f;
          }
#pragma unroll
          for (int i = 0; i < kMaxJoin; ++i) top = fmaxf(top, mv[i]);
          const float tu = (top == -INFINITY) ? 0.f : top;
#pragma unroll
          for (int i = 0; i < kMaxJoin; ++i)
            if (i < n) {
              mv[i] = hw_exp2(mv[i] - tu);
              sum += mv[i] * lv[i];
            }
          const float inv = final ? (sum == 0.f ? 0.f : a.v_scale / sum) : 1.f;
#pragma unroll
          for (int i = 0; i < kMaxJoin; ++i)
            if (i < n) wt[i * kPairs + pr] = mv[i] * inv;
          if (final) {
            if (a.lse != nullptr)
              a.lse[(size_t)(x.row0 + j) * kHeads + x.g * kHpg + h] = sum == 0.f ? -INFINITY : (top + hw_log2(sum)) * kLn2;
          } else {
            float *ml = a.part_ml + ((size_t)part_slot(lead) + 2 * (size_t)gridDim.x) * 2 * kPairs;
            ml[pr] = top;
            ml[kPairs + pr] = sum;
          }
        }
        if (!soft_sync()) {
          ok = false;
          break;
        }
        for (int i = tid; i < x.nr * kHpg * (kD / 4); i += kDnSoft) {
          const int q = i / (kD / 4), d = (i % (kD / 4)) * 4;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int z0 = 0; z0 < n; z0 += 8) {
            float4 y[8];
#pragma unroll
            for (int z = 0; z < 8; ++z)
              if (z0 + z < n)
                y[z] = ld_cg(reinterpret_cast<const float4 *>(
                    a.part_o + ((size_t)part_slot(lead + (z0 + z) * step) * kPairs + q) * kD + d));
#pragma unroll
            for (int z = 0; z < 8; ++z)
              if (z0 + z < n) {
                const float wz = wt[(z0 + z) * kPairs + q];
                acc.x = fmaf(wz, y[z].x, acc.x);
                acc.y = fmaf(wz, y[z].y, acc.y);
                acc.z = fmaf(wz, y[z].z, acc.z);
                acc.w = fmaf(wz, y[z].w, acc.w);
              }
          }
          if (final) {
            uint2 w2;
            w2.x = pack_bf16(acc.x, acc.y);
            w2.y = pack_bf16(acc.z, acc.w);
            *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) +
                                       ((size_t)(x.row0 + (q >> 4)) * kHeads + x.g * kHpg + (q & 15)) * kD + d) = w2;
          } else {
            *reinterpret_cast<float4 *>(a.part_o + ((size_t)part_slot(lead) * kPairs + q) * kD + d) = acc;
          }
        }
        if (final) {
          if (!soft_sync()) ok = false;  // the weights are read before the next epilogue writes there
          break;
        }
        level = 1;
      }
    }
  }

  // ---- teardown: no MMA may be writing tensor memory when it is released ----
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) {
    mbar_wait_bounded(b_final, 0, kDnWaitNs);
    tc::tmem_dealloc(tmem, kTmCols);
  }
}

template <bool KV8, int RT>
cudaError_t launch(const DenseArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t st) {
  auto kernel = dense_kernel<KV8, RT>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), Cfg<KV8, RT>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.n_ctas);
  cfg.blockDim = dim3(kDnThreads);
  cfg.dynamicSmemBytes = Cfg<KV8, RT>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, tk, tv);
}

}  // namespace

cudaError_t launch_dense(const DenseArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t st) {
  switch (a.tile_rows + (a.kv8 ? 16 : 0)) {
    case 1: return launch<false, 1>(a, tk, tv, st);
    case 2: return launch<false, 2>(a, tk, tv, st);
    case 4: return launch<false, 4>(a, tk, tv, st);
    case 8: return launch<false, 8>(a, tk, tv, st);
    case 17: return launch<true, 1>(a, tk, tv, st);
    case 18: return launch<true, 2>(a, tk, tv, st);
    case 20: return launch<true, 4>(a, tk, tv, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace s5
