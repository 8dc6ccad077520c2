// Dense GQA of a batch's new tokens over the whole paged cache, bf16 or
// one-byte (E4M3) KV, on the 5th-generation tensor cores.
//
// For row r at position t, head h, group g = h / 16:
//   out = sum_{j <= t} softmax_j(sm_scale q.K_j) V_j,  lse = log sum_j exp(sm_scale q.K_j)
// computed in one pass over the cache with a running reference maximum and sum
// per (row, head); parts of a row's cache are joined by
//   M = max_p m_p,  O = sum_p 2^(m_p - M) O_p,  L = sum_p 2^(m_p - M) l_p.
//
// Bound: HBM.  A cached token costs 3 KB (bf16) for 16 FLOPs per byte and
// query row, far below the tensor cores' ratio even for the 4 rows of a tile, so
// the aim is a full stream of pages on every SM: 32 requests x 131,072 bf16 tokens
// take 1.81 to 1.85 ms = 7.1 to 7.0 TB/s, 64 x 30,000 to 65,536 one-byte tokens 0.71 ms = 6.6 TB/s in a replayed graph
// and 0.77 to 0.80 ms in calls in sequence with other inputs (the power limit holds the SM clock at 1.4 to 1.8 GHz,
// and times follow it).
//
// Split.  The work is a list of page units: sequences in order, in each its KV
// groups, in each group its tiles of `tile_rows` query rows, in each tile the
// pages up to its last row.  Every CTA (one per SM, persistent) finds its equal
// share of the list from the device's lengths by prefix sums, so ragged batches
// balance to within a page and one long sequence spreads over every SM.  A tile
// that spans CTAs leaves a part per CTA, and a second kernel joins the parts; in
// batches of short sequences a tile belongs whole to the CTA in whose share it
// begins, and there is nothing to join.
// (Joined by the last CTA to arrive, in two levels, a tile of 37 parts took 14 us,
// of 4 rows 21 us: two counters' round trips, and the parts read by one SM.  The
// second kernel takes 4 to 5 us.)
//
// One CTA works in chunks of two pages (128 tokens): a warp streams K and another
// V, one TMA copy per page and KV group, through rings in shared memory; one warp
// issues S^T = K Q^T (M = 128 tokens, N = heads of the tile) into tensor memory;
// the softmax warps, a thread per token (2 or 4 rows: two), turn a row of S^T into
// weights P and store them as the N operand of O^T += V^T P^T, which a fourth warp
// issues (M = 128 + 64 dims); O^T stays in tensor memory until the tile's run of
// pages ends.
//
// Tokens and dims are the M side so that no product is wasted: a decode row has
// only 16 heads per KV group, and with heads as M = 128 rows (copies of the heads
// in the spare rows, each working on a run of tokens) the same stream ran at 2.18
// ms for 32 x 131,072 bf16 tokens with the clock down to 1.06 GHz for the
// power that the redundant products drew.  An MMA of N <= 32 takes 45 cycles, N =
// 64 takes 50, N = 128 66, whatever the types.
//
// Weights are held in terms, each a column of P: bf16 KV the upper half of the
// fp32 weight and the upper half of the remainder (2^-15); one-byte KV the weight
// in f16, whose upper byte is an E5M2 value, as bytes of what the terms before
// leave: four hold an f16 exactly above 2^-16 (weights to 2^-12), three with the
// last rounded are within 2^-9.  Column sums need no split: fp32 in registers.
#include <cuda.h>

#include "s5_common.cuh"
#include "s5_kernels.h"
#include "s5_tcgen05.cuh"

namespace s5 {

namespace {

constexpr int kChunk = 2 * kPage;                // tokens
constexpr int kScanPer = 4;                      // sequences per thread and round of the prefix sums
constexpr uint64_t kDnWaitNs = 2000000000ull;    // 2 s per wait
constexpr float kLn2 = 0.69314718055994531f;

template <bool KV8, int RT>
struct Cfg {
  static constexpr int kPairs = RT * kHpg;            // (row, head) pairs of a tile: columns of S^T and O^T
  // Softmax warps: 4, a thread per token, or (2 and 4 rows) 8, two threads per token with half of the
  // columns each (one-byte KV, 16 x 16,384 tokens, 2 rows: 80 against 73 us; 4 rows: 121 against 86 to 93 us).
  static constexpr int kSoftWarps = RT >= 2 ? 8 : 4, kSoft = 32 * kSoftWarps, kThreads = kSoft + 128;
  static constexpr int kHalves = kSoftWarps / 4, kCols = kPairs / kHalves;  // threads per token, their columns
  static constexpr int kWarpK = kSoftWarps, kWarpV = kWarpK + 1, kWarpS = kWarpK + 2, kWarpPv = kWarpK + 3;
  static constexpr int kQTerms = KV8 ? 2 : 1;         // terms of q (rows of the N operand)
  static constexpr int kS = kPairs * kQTerms;         // columns of S^T
  static constexpr int kTerms = KV8 ? (RT == 4 ? 3 : 4) : 2;
  static constexpr int kP = kPairs * kTerms;          // columns of P and O^T
  static constexpr int kSBuf = 2 * kS + 2 * kP <= 512 ? 2 : 1;
  // tensor memory: S^T buffers, O^T of dims 0-127, O^T of dims 128-191 (M = 64)
  static constexpr uint32_t kTmO = kSBuf * kS, kTmO2 = kTmO + kP;
  static constexpr uint32_t kTmNeed = kTmO2 + kP;
  static constexpr uint32_t kTmCols = kTmNeed <= 128 ? 128 : kTmNeed <= 256 ? 256 : 512;
  static_assert(kTmNeed <= 512, "tensor memory columns");
  static constexpr int kPageBytes = kPage * kD * (KV8 ? 1 : 2);
  // a page in shared memory: [8 groups of 8 tokens][3 planes of 64 dims][8 tokens][kRowB], so
  // that 8-token groups are evenly spaced across the pages of a chunk
  static constexpr int kRowB = KV8 ? 64 : 128;
  static constexpr int kPlane = 8 * kRowB;
  static constexpr int kGroup = 3 * kPlane;
  // Rings of 172 KB (one byte: 123 KB).  Deeper ones do not stream faster but less evenly: with four
  // V pages (bf16) the first SM ended 32 x 131,072 tokens 180 us before the last and the call took
  // 1.89 ms, with three 1.83 ms.
  static constexpr int kKStages = KV8 ? 3 : 2;                        // chunks in the K ring
  static constexpr int kVPages = KV8 ? 4 : 3;                         // pages in the V ring
  static constexpr int kChunkBytes = 2 * kPageBytes;
  // P: [16 groups of 8 tokens][atoms][8 tokens][kAtom bytes], swizzled over an atom's rows
  static constexpr int kPRow = kP * (KV8 ? 1 : 2);
  static constexpr int kAtom = kPRow % 128 == 0 ? 128 : 64;
  static constexpr int kPGroup = 8 * kPRow;
  static constexpr int kPBuf = KV8 || RT <= 2 ? 2 : 1;  // buffers (bf16, 4 rows: no room for two)
  // Q: [3 planes][kS rows][kRowB]
  static constexpr int kQPlane = kS * kRowB;
  static constexpr int kQThreads = kSoft / kPairs, kQPieces = kD / 8 / kQThreads;  // threads of a row, 8-dim pieces of each
  // the reference sits kOff binades under the maximum it was taken from and moves when a weight
  // would exceed 2^kTop.  One byte: f16 weights reach 2^15, E5M2 ones go down to 2^-16, so
  // weights of 2^-28 of the largest still count.
  static constexpr float kOff = KV8 ? 12.f : 0.f;
  static constexpr float kTop = KV8 ? 15.f : 8.f;
  // What a run costs besides its pages, in pages, for equal shares: 2 us a run were measured on 64 ragged
  // requests (1 row), 7 us on 16 verified ones (4 rows); a bf16 page takes about 1 us.
  static constexpr int kStart = (RT == 1 ? 2 : RT == 2 ? 4 : 6) * (KV8 ? 2 : 1);
  // shared memory (from a 1,024-byte aligned base)
  static constexpr int kOffV = kKStages * kChunkBytes;
  static constexpr int kOffQ = kOffV + kVPages * kPageBytes;
  static constexpr int kOffP = kOffQ + 3 * kQPlane;
  static constexpr int kOffCol = kOffP + kPBuf * 16 * kPGroup;        // float [6][kPairs]: per-column values
  static constexpr int kOffBad = kOffCol + 6 * kPairs * 4;            // uint32 [48]: per dim, rows that saw a non-finite value
  static constexpr int kOffBar = kOffBad + 192;
  static constexpr int kNumBars = 2 * kKStages + 2 * kVPages + 13;
  static constexpr int kOffMisc = kOffBar + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kSmem = kOffMisc + 128 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  static_assert(16 * kPGroup >= kThreads * kScanPer * 4, "the list of bad sequences lies in P's room");
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

__device__ __forceinline__ Seq load_seq(const int32_t *cu_q, const int32_t *ctx_lens, int total_q, int max_len, int s) {
  Seq q;
  q.lo = ld_cg(cu_q + s);
  const int hi = ld_cg(cu_q + s + 1);
  q.ctx = ld_cg(ctx_lens + s);
  q.bad = q.lo < 0 || hi < q.lo || hi > total_q;
  q.n = q.bad ? 0 : hi - q.lo;
  if (q.n > 0 && (q.ctx < 0 || q.ctx > max_len - q.n)) {
    q.bad = true;
    q.n = 0;
  }
  return q;
}
__device__ __forceinline__ Seq load_seq(const DenseArgs &a, int s) {
  return load_seq(a.cu_q, a.ctx_lens, a.total_q, a.max_len, s);
}

// The first sequence from s on that has rows (batch: none).  The warp looks at 32 at a time, a lane each: one
// after the other they are dependent reads of L2, and a call of 18 us took 44 with 100 sequences without
// rows between two with rows (padded places of a batch), 757 with 3,000; 20 and 51 this way.  (A call for the
// same reason as fill_bad: inlined, one-byte calls took up to 9% longer.)
__device__ __noinline__ int next_live(const int32_t *cu_q, const int32_t *ctx_lens, int batch, int total_q, int max_len,
                                      int s) {
  const int lane = threadIdx.x & 31;
  for (; s < batch; s += 32) {
    const uint32_t live =
        __ballot_sync(0xffffffffu, lane < batch - s && load_seq(cu_q, ctx_lens, total_q, max_len, s + lane).n > 0);
    if (live != 0) return s + __ffs(live) - 1;
  }
  return batch;
}

// Units of the first m tiles, full ones: a tile counts its pages and, before them, START units for
// what beginning and ending a run costs.
template <int RT, int START>
__device__ __forceinline__ long long full_tile_units(int ctx, int m) {
  return full_tile_pages<RT>(ctx, m) + (long long)START * m;
}

template <int RT, int START>
__device__ __forceinline__ long long group_units(const Seq &q) {  // of one KV group of the sequence
  if (q.n <= 0) return 0;
  const int tiles = (q.n + RT - 1) / RT;
  const long long last = (q.ctx + q.n + kPage - 1) / kPage + START;
  return tiles == 1 ? last : full_tile_units<RT, START>(q.ctx, tiles - 1) + last;
}

// Where a CTA's share begins: unit `off` of sequence s.
struct Start {
  Seq q;
  int s;
  long long off;
};

// A run of pages of one tile.
struct Seg {
  int s, g, row0, nr, t0;    // sequence, KV group, first row, rows, position of the first row
  int p0, np, tile_pages;    // first page, pages, pages of the whole tile
  long long tile_u;          // unit of the tile's first page (after its START units)
};

// The runs of one CTA in order.  Every warp walks them by itself.
template <int RT, int START>
struct Walk {
  const DenseArgs &a;
  Seq q;
  int s, g, k, o;  // sequence, group, tile, unit of the tile that comes next
  long long u, rem;

  // unit u0 is unit `off` of sequence s0
  __device__ Walk(const DenseArgs &args, const Seq &q0, int s0, long long off, long long u0, long long count)
      : a(args), q(q0), s(s0), g(0), u(u0), rem(count) {
    const long long per = group_units<RT, START>(q);
    long long left = off;
    while (left >= per) {
      left -= per;
      ++g;
    }
    int lo = 0, hi = (q.n + RT - 1) / RT;  // the last tile k whose units before are <= left
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (full_tile_units<RT, START>(q.ctx, mid) <= left) lo = mid;
      else hi = mid;
    }
    k = lo;
    o = (int)(left - full_tile_units<RT, START>(q.ctx, k));
    if (a.whole && o > 0) {  // the tile that lies across the share's begin is the CTA's before
      const int n = tile_pages() + START - o;
      u += n;
      rem -= n;
      advance();
    }
    skip_start();
  }

  __device__ int tile_pages() const { return (q.ctx + min((k + 1) * RT, q.n) + kPage - 1) / kPage; }

  __device__ void advance() {  // to the next tile
    o = 0;
    if (++k * RT >= q.n) {
      k = 0;
      if (++g == kKv) {
        g = 0;
        q.n = 0;
        while (rem > 0 && q.n == 0 && ++s < a.batch) {
          q = load_seq(a, s);
          if (q.n == 0) s = next_live(a.cu_q, a.ctx_lens, a.batch, a.total_q, a.max_len, s + 1) - 1;
        }
        if (q.n == 0) rem = 0;
      }
    }
  }

  __device__ void skip_start() {
    const long long n = a.whole ? START : min((long long)max(START - o, 0), max(rem, 0LL));
    if (a.whole && rem <= 0) return;
    o += (int)n;
    u += n;
    rem -= a.whole ? 0 : n;
  }

  __device__ void run(Seg &x) const {  // the run that starts here (rem > 0)
    const int nr = min(RT, q.n - k * RT);
    x.s = s;
    x.g = g;
    x.row0 = q.lo + k * RT;
    x.nr = nr;
    x.t0 = q.ctx + k * RT;
    x.tile_pages = tile_pages();
    x.p0 = o - START;
    x.np = a.whole ? x.tile_pages : (int)min((long long)(x.tile_pages - x.p0), rem);
    x.tile_u = u - x.p0;
  }

  __device__ bool next(Seg &x) {
    if (rem <= 0) return false;
    run(x);
    u += x.np;
    rem -= a.whole ? x.np + START : x.np;
    o += x.np;
    if (o == x.tile_pages + START) {
      advance();
      skip_start();
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
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, float f) {
  const __half2 v = __hmul2(*reinterpret_cast<__half2 *>(&a), __float2half2_rn(f));
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  const __half2 v = __hsub2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Barrier of the softmax warps (named barrier 1).  They always run the same sequence
// of these: a warp whose bounded wait expired goes on to the next one, where all learn of it.
template <int THREADS>
__device__ __forceinline__ bool soft_or_n(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(THREADS)
      : "memory");
  return r != 0;
}
template <int THREADS>
__device__ __forceinline__ void soft_sync_n() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// D[tmem] (+)= A[smem] * B[smem]^T, one K step; KV8: kind::f8f6f4, else kind::f16.
template <bool KV8>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, bool accumulate) {
  if constexpr (KV8) tc::mma_f8(d_tmem, a_desc, b_desc, idesc, accumulate);
  else tc::mma_bf16(d_tmem, a_desc, b_desc, idesc, accumulate);
}

// The tile's queries as the N operand, K-major: row j * 16 + h; thread `tid` takes a run of
// dims of one row.  bf16: as they are.  One byte: two E4M3 terms (rows n and kPairs + n) of q
// times a power of two that puts the tile's largest finite magnitude in [2^7, 2^8): the nearest
// code and 16 times the remainder, together a bf16's 8 bits exactly down to 2^-14 of that
// magnitude; smaller values are rounded to multiples of 2^-21 of it, which changes a score by at
// most 2^-22 of what the largest magnitude makes of the same K.  (One power per row instead
// needs a factor per column in the softmax.)  Returns the factor of the scores.
template <bool KV8, int RT>
__device__ __forceinline__ void fetch_q(const DenseArgs &a, const Seg &x, int tid, uint4 (&v)[Cfg<KV8, RT>::kQPieces]) {
  using C = Cfg<KV8, RT>;
  const int n = tid / C::kQThreads, part = tid % C::kQThreads;
  const uint4 *src = reinterpret_cast<const uint4 *>(a.q) +
                     ((size_t)(x.row0 + n / kHpg) * kHeads + x.g * kHpg + n % kHpg) * (kD / 8) + part * C::kQPieces;
#pragma unroll
  for (int i = 0; i < C::kQPieces; ++i) v[i] = n / kHpg < x.nr ? ld_cg(src + i) : make_uint4(0, 0, 0, 0);
}

template <bool KV8, int RT>
__device__ __forceinline__ float store_q(const DenseArgs &a, const uint4 (&v)[Cfg<KV8, RT>::kQPieces], uint8_t *sq,
                                         float *max_s, int tid) {
  using C = Cfg<KV8, RT>;
  constexpr int kPer = C::kQThreads, kPieces = C::kQPieces;
  const int n = tid / kPer, part = tid % kPer;
  const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale's sign goes into q
  if constexpr (!KV8) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = part * kPieces + i;  // dims 8 p ..
      *reinterpret_cast<uint4 *>(sq + (p >> 3) * C::kQPlane + n * 128 + (((p & 7) ^ (n & 7)) << 4)) =
          make_uint4(v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
    }
    return fabsf(a.scale_log2);
  } else {
    float top = 0.f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float f0 = fabsf(bf16lo(w[y])), f1 = fabsf(bf16hi(w[y]));
        finite = finite && f0 < INFINITY && f1 < INFINITY;
        top = max3(top, f0 < INFINITY ? f0 : 0.f, f1 < INFINITY ? f1 : 0.f);
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
    for (int o = 1; o < kPer; o <<= 1) finite = __shfl_xor_sync(0xffffffffu, (int)finite, o) != 0 && finite;
    if (tid % 32 == 0) max_s[tid / 32] = top;
    soft_sync_n<C::kSoft>();
#pragma unroll
    for (int i = 0; i < C::kSoftWarps; ++i) top = fmaxf(top, max_s[i]);
    const int e = (int)(__float_as_uint(top) >> 23);  // biased exponent of the largest magnitude
    // (a row with a value that is not finite: NaN)
    float up = finite ? __uint_as_float((uint32_t)min(261 - e, 254) << 23) : __uint_as_float(0x7FC00000u);
    const float down = e > 7 ? __uint_as_float((uint32_t)(e - 7) << 23) : __uint_as_float(0x00400000u);
    if (flip) up = -up;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = part * kPieces + i;
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t c0[2] = {0, 0}, c1[2] = {0, 0};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint32_t x = float2_to_f16x2(bf16lo(w[y]) * up, bf16hi(w[y]) * up);
        const uint32_t c = f16x2_to_e4m3x2(x);
        c0[y >> 1] |= c << (16 * (y & 1));
        c1[y >> 1] |= f16x2_to_e4m3x2(mul_f16x2(sub_f16x2(x, e4m3x2_to_f16x2(c)), 16.f)) << (16 * (y & 1));
      }
      uint8_t *at = sq + (p >> 3) * C::kQPlane + n * 64 + ((((p >> 1) & 3) ^ ((n >> 1) & 3)) << 4) + (p & 1) * 8;
      *reinterpret_cast<uint2 *>(at) = make_uint2(c0[0], c0[1]);
      *reinterpret_cast<uint2 *>(at + C::kPairs * 64) = make_uint2(c1[0], c1[1]);
    }
    return fabsf(a.scale_log2) * down;
  }
}

// The parts of a tile that spans CTAs: its first CTA, their number, and the slot of partial results
// of the i-th (a CTA's second slot holds the tile that begins in its share and ends behind it).
struct Parts {
  int first, n;
  __device__ int slot(int i) const { return 2 * (first + i) + (i == 0 ? 1 : 0); }
};
__device__ __forceinline__ Parts parts_of(const Seg &x, long long chunk) {
  Parts p;
  p.first = (int)(x.tile_u / chunk);
  p.n = (int)((x.tile_u + x.tile_pages - 1) / chunk) - p.first + 1;
  return p;
}
// row of out and lse of the tile's (row, head) pair q
__device__ __forceinline__ size_t out_row(const Seg &x, int q) {
  return (size_t)(x.row0 + q / kHpg) * kHeads + x.g * kHpg + q % kHpg;
}

// V of tokens that a row of the tile does not see must not be NaN or infinite (P is 0 there, but
// 0 * NaN is NaN): tokens that no row sees (after t_last, or all of a page that is none) become zeros;
// in tokens that only some rows see (after t0), a value that is not finite becomes zero and is noted
// in bad_s for the rows that see it.  Positions are relative to the page's first token.
template <bool KV8, int RT>
__device__ __forceinline__ void clean_v(uint8_t *vb, uint32_t *bad_s, bool page_ok, int t0, int t_last, int tid) {
  using C = Cfg<KV8, RT>;
  constexpr int kPieces = C::kRowB / 16;  // 16-byte pieces of a token in a plane
  const int from = page_ok ? max(t0 + 1, 0) : 0;
  for (int i = from * 3 * kPieces + tid; i < kPage * 3 * kPieces; i += C::kSoft) {
    const int tok = i / (3 * kPieces), z = i % (3 * kPieces), plane = z / kPieces, pc = z % kPieces;
    uint4 *at = reinterpret_cast<uint4 *>(vb + (tok >> 3) * C::kGroup + plane * C::kPlane + (tok & 7) * C::kRowB + pc * 16);
    if (!page_ok || tok > t_last) {
      *at = make_uint4(0, 0, 0, 0);
    } else {
      const int d0 = plane * 64 + (pc ^ (KV8 ? (tok >> 1) & 3 : tok & 7)) * (KV8 ? 16 : 8);
      // rows whose position is at least the token's
      const uint32_t rows = (0xFFu << (tok - t0)) & 0xFFu;
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
}

// Rows of the bad sequences in `list`: zeros, in the rows that no sequence with good offsets has, since other
// CTAs write those.  Such a sequence before s ends at or before the largest offset up to s, one behind it
// begins at or behind the smallest from s + 1 on (offsets outside [0, total_q] are no good sequence's),
// so the rows between the two are only s's.  All threads of the CTA.  (A call: inlined, it changed
// the code behind it, and one-byte calls took up to 3% longer, 32 x 1,000 tokens 20.0 instead of 19.0 us.)
__device__ __noinline__ void fill_bad(const int32_t *cu_q, int batch, int total_q, void *out, float *lse, const int *list,
                                      int nb, int *range_s) {
  const int tid = threadIdx.x, nt = blockDim.x;
  for (int b = 0; b < nb; ++b) {
    const int s = list[b];
    if (tid == 0) {
      range_s[0] = 0;
      range_s[1] = total_q;
    }
    __syncthreads();
    int lo = 0, hi = total_q;
    if (ld_cg(cu_q + s) < hi && ld_cg(cu_q + s + 1) > 0)  // (else it has no rows in the batch)
      for (int i = tid; i <= batch; i += nt) {
        const int c = ld_cg(cu_q + i);
        if (c < 0 || c > total_q) continue;
        if (i <= s) lo = max(lo, c);
        else hi = min(hi, c);
      }
    else hi = 0;
    lo = __reduce_max_sync(0xffffffffu, lo);
    hi = __reduce_min_sync(0xffffffffu, hi);
    if (tid % 32 == 0) {
      atomicMax(range_s, lo);
      atomicMin(range_s + 1, hi);
    }
    __syncthreads();
    lo = range_s[0];
    hi = range_s[1];
    for (long long i = (long long)lo * kHeads * (kD / 8) + tid; i < (long long)hi * kHeads * (kD / 8); i += nt)
      reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
    if (lse != nullptr)
      for (long long i = (long long)lo * kHeads + tid; i < (long long)hi * kHeads; i += nt) lse[i] = -INFINITY;
    __syncthreads();  // range_s is written again
  }
}

// ---------------------------------------------------------------- the kernel

template <bool KV8, int RT>
__global__ void __launch_bounds__(Cfg<KV8, RT>::kThreads, 1)
    dense_kernel(const DenseArgs a, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<KV8, RT>;
  constexpr int KS = C::kKStages, VP = C::kVPages, PB = C::kPageBytes, NQ = C::kPairs, NT = C::kThreads;
  constexpr int kWarpK = C::kWarpK, kWarpV = C::kWarpV, kWarpS = C::kWarpS, kWarpPv = C::kWarpPv;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sk = smem, *sv = smem + C::kOffV, *sq = smem + C::kOffQ, *sp = smem + C::kOffP;
  float *col_s = reinterpret_cast<float *>(smem + C::kOffCol);
  float *ref_s = col_s, *max_s = col_s + NQ;                    // reference (0: none yet); warps' largest |q|
  float *warp_s = col_s + 2 * NQ;                               // [4][NQ]: the warps' maxima or sums
  // what a move of the reference changes (thread i reads column i of warp_s, then writes there)
  float *shift_s = warp_s, *corr_s = warp_s + NQ;
  uint32_t *bad_s = reinterpret_cast<uint32_t *>(smem + C::kOffBad);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
  uint64_t *k_full = bars, *k_empty = bars + KS, *v_full = bars + 2 * KS, *v_empty = v_full + VP;
  uint64_t *s_full = v_empty + VP, *s_empty = s_full + 2, *p_full = s_full + 4, *p_free = s_full + 6;
  uint64_t *q_full = s_full + 8, *q_empty = s_full + 9, *o_empty = s_full + 10, *b_final = s_full + 11;
  uint64_t *b_stall = s_full + 12;  // nothing ever arrives on it (expired-wait test hook)
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
  int *abort_flag = reinterpret_cast<int *>(smem + C::kOffMisc + 4);
  int *n_bad_s = reinterpret_cast<int *>(smem + C::kOffMisc + 12);
  Start *start_s = reinterpret_cast<Start *>(smem + C::kOffMisc + 16);
  int *range_s = reinterpret_cast<int *>(smem + C::kOffMisc + 16 + sizeof(Start));  // [2], before the pipeline runs
  long long *sum_s = reinterpret_cast<long long *>(col_s);                    // [warps], before the pipeline runs
  int *bad_list = reinterpret_cast<int *>(sp);                                // [NT * kScanPer], before the pipeline runs

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2 * KS + 2 * VP; ++i) mbar_init(bars + i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(s_empty + i, C::kSoftWarps);
      mbar_init(p_full + i, C::kSoftWarps);
      mbar_init(p_free + i, 1);
    }
    mbar_init(q_full, C::kSoftWarps);
    mbar_init(q_empty, 1);
    mbar_init(o_empty, C::kSoftWarps);
    mbar_init(b_final, 2);
    mbar_init(b_stall, 1);
    *abort_flag = 0;
    *n_bad_s = 0;
  }
  if (tid < 48) bad_s[tid] = 0;
  fence_mbar_init();
  if (warp == kWarpPv) tc::tmem_alloc(tmem_slot, C::kTmCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  if (tid == kWarpK * 32) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
  if (tid == kWarpV * 32) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
  pdl_wait();  // (programmatic launch) global memory is read from here on
  if (tid == 0) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);

  // ---- this CTA's share: prefix sums of the sequences' page units ----
  const int per = a.batch <= NT ? 1 : kScanPer;  // sequences per thread
  const int rounds = (a.batch + NT * per - 1) / (NT * per);
  long long total = 0, units[kScanPer], before = 0;
  Seq seqs[kScanPer];
  auto scan_round = [&](int r, bool report) {  // units[] of this thread's sequences; exclusive prefix in `before`
    long long mine = 0;
    bool any_bad = false;
#pragma unroll
    for (int i = 0; i < kScanPer; ++i) {
      const int s = (r * NT + tid) * per + i;
      seqs[i].n = 0;
      seqs[i].bad = false;
      if (i < per && s < a.batch) seqs[i] = load_seq(a, s);
    }
#pragma unroll
    for (int i = 0; i < kScanPer; ++i) {
      const int s = (r * NT + tid) * per + i;
      units[i] = kKv * group_units<RT, C::kStart>(seqs[i]);
      mine += units[i];
      if (seqs[i].bad && report && s % (int)gridDim.x == (int)blockIdx.x) {
        record_error(a.err, S5_ERR_DEVICE_BOUNDS, max(seqs[i].lo, 0));
        bad_list[atomicAdd(n_bad_s, 1)] = s;
        any_bad = true;
      }
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sum_s[warp] = incl;
    any_bad = __syncthreads_or(any_bad);
    before = incl - mine;
    long long all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) before += sum_s[w];
      all += sum_s[w];
    }
    if (any_bad) {
      fill_bad(a.cu_q, a.batch, a.total_q, a.out, a.lse, bad_list, *n_bad_s, range_s);
      if (tid == 0) *n_bad_s = 0;
    }
    if (rounds > 1) __syncthreads();  // sum_s and the list are written again
    return all;
  };
  // Up to 32 sequences: every warp has the sums by itself, a lane per sequence, and none waits for
  // another (a bad sequence, whose rows are to be filled, takes the other way)
  Start start;
  bool by_warp = false;
  long long incl_w = 0, units_w = 0;
  if (a.batch <= 32) {
    start.q.n = 0;
    start.q.bad = false;
    if (lane < a.batch) start.q = load_seq(a, lane);
    by_warp = !__any_sync(0xffffffffu, start.q.bad);
    units_w = kKv * group_units<RT, C::kStart>(start.q);
    incl_w = units_w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl_w, o);
      if (lane >= o) incl_w += v;
    }
    total = __shfl_sync(0xffffffffu, incl_w, 31);
  }
  if (!by_warp) {
    total = 0;
    for (int r = 0; r < rounds; ++r) total += scan_round(r, true);
  }
  long long chunk = total < (1LL << 31) ? max(((uint32_t)total + gridDim.x - 1) / gridDim.x, 1u)
                                        : (total + gridDim.x - 1) / gridDim.x;
  // (short shares take as long for a page as for a chunk, and have fewer parts to join)
  if (chunk < 16) chunk += chunk & 1;
  const long long u0 = chunk * blockIdx.x;
  const bool idle = u0 >= total;
  const long long count = min(chunk, total - u0);
  if (by_warp) {
    const int src = __popc(__ballot_sync(0xffffffffu, incl_w <= u0));  // sequences that end at or before u0
    const long long off = u0 - (incl_w - units_w);
    start.s = src;
    start.off = __shfl_sync(0xffffffffu, off, src & 31);
    start.q.lo = __shfl_sync(0xffffffffu, start.q.lo, src & 31);
    start.q.n = __shfl_sync(0xffffffffu, start.q.n, src & 31);
    start.q.ctx = __shfl_sync(0xffffffffu, start.q.ctx, src & 31);
  } else if (!idle) {
    long long base = 0;
    for (int r = 0; r < rounds; ++r) {
      const long long all = rounds > 1 ? scan_round(r, false) : total;
      long long at = base + before;
#pragma unroll
      for (int i = 0; i < kScanPer; ++i) {
        if (at <= u0 && u0 < at + units[i]) {
          start_s->s = (r * NT + tid) * per + i;
          start_s->off = u0 - at;
          start_s->q = seqs[i];
        }
        at += units[i];
      }
      base += all;
      if (base > u0) break;
    }
  }
  if (idle) {
    if (warp == kWarpPv) tc::tmem_dealloc(tmem, C::kTmCols);
    return;
  }
  if (!by_warp) {
    __syncthreads();
    start = *start_s;
  }
  Walk<RT, C::kStart> walk(a, start.q, start.s, start.off, u0, count);
  Seg x;

  // Bounded wait.  (Polling with test_wait instead, without suspension, was 3% slower: the
  // stream leaves most warps waiting, and their polls cost issue slots and power.)
  auto wait = [&](uint64_t *bar, uint32_t parity, uint64_t limit_ns = kDnWaitNs) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!*reinterpret_cast<volatile int *>(abort_flag)) {
      if (mbar_try_wait(bar, parity)) return true;
      if (globaltimer_ns() - t0 > limit_ns) {
        *reinterpret_cast<volatile int *>(abort_flag) = 1;
        record_error(a.err, S5_ERR_TIMEOUT, 0);
      }
    }
    return false;
  };

  if (warp == kWarpK || warp == kWarpV) {
    // ---------------- TMA producers: K a chunk at a time, V a page at a time ----------------
    const bool is_k = warp == kWarpK;
    const uint64_t policy = a.reread ? policy_evict_normal() : policy_evict_first();
    int n = 0;  // chunks (K) or pages (V) so far
    bool ok = true;
    while (ok && walk.next(x)) {
      const int32_t *pt = a.page_table + (size_t)x.s * a.max_pages + x.p0;
      int ids = lane < x.np ? ld_cg(pt + lane) : -1;  // pages c .. c + 31, one per lane; the next 32 in flight
      for (int c = 0; c < x.np && ok; c += 32) {
        const int nxt = c + 32 + lane < x.np ? ld_cg(pt + c + 32 + lane) : -1;
        const int m = min(32, x.np - c), step = is_k ? 2 : 1;
        for (int i = 0; i < m; i += step, ++n) {
          const int page0 = __shfl_sync(0xffffffffu, ids, i), page1 = __shfl_sync(0xffffffffu, ids, min(i + 1, 31));
          int go = 1;
          if (lane == 0) {
            const int depth = is_k ? KS : VP, st = n % depth;
            uint64_t *full = (is_k ? k_full : v_full) + st;
            if (n >= depth) go = wait((is_k ? k_empty : v_empty) + st, ((n / depth) - 1) & 1) ? 1 : 0;
            if (go) {
              const bool ok0 = page0 >= 0 && page0 < a.num_pages;
              if (is_k) {
                const bool ok1 = i + 1 < m && page1 >= 0 && page1 < a.num_pages;
                if (!ok0 || (i + 1 < m && !ok1)) record_error(a.err, S5_ERR_DEVICE_BOUNDS, x.row0);
                mbar_arrive_expect_tx(full, (ok0 ? PB : 0) + (ok1 ? PB : 0));
                uint8_t *dst = sk + st * C::kChunkBytes;
                if (ok0) tma_load_4d(dst, &tm_k, 0, 0, 0, (page0 * kKv + x.g) * (kPage / 8), full, policy);
                if (ok1) tma_load_4d(dst + PB, &tm_k, 0, 0, 0, (page1 * kKv + x.g) * (kPage / 8), full, policy);
              } else {
                mbar_arrive_expect_tx(full, ok0 ? PB : 0);
                if (ok0) tma_load_4d(sv + st * PB, &tm_v, 0, 0, 0, (page0 * kKv + x.g) * (kPage / 8), full, policy);
              }
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
    if (lane == 0) {
      const int depth = is_k ? KS : VP;
      for (int c = max(0, n - depth); c < n; ++c)
        mbar_wait_bounded((is_k ? k_full : v_full) + c % depth, (c / depth) & 1, kDnWaitNs);
    }
  } else if (warp == kWarpS) {
    // ---------------- S^T = K Q^T ----------------
    // (The issuing warps stay converged, with counters instead of divisions and one elected lane only
    // around the instructions, so that descriptors are built in uniform registers.)
    constexpr uint32_t idesc = KV8 ? tc::idesc_f8_f32(128, C::kS, 0, 0) : tc::idesc_bf16_f32(128, C::kS);
    const uint64_t kd0 = tc::smem_desc_sw(smem_u32(sk), 16, C::kGroup, C::kRowB);
    const uint64_t qd0 = tc::smem_desc_sw(smem_u32(sq), 16, C::kPlane, C::kRowB);
    const bool leader = elect_one();
    // test hook (workspace header, zero in normal use): wait that many ns for nothing, then give up
    uint64_t stall_ns = a.err != nullptr ? ld_cg_u64(reinterpret_cast<const uint64_t *>(a.err) + kWsStallWord) : 0;
    int st = 0, sb = 0;                        // K stage, S^T buffer
    uint32_t k_par = 0, s_par = 1, q_par = 0;  // (an unused buffer counts as released)
    bool ok = true;
    while (ok && walk.next(x)) {
      const int np = __shfl_sync(0xffffffffu, x.np, 0);
      ok = __all_sync(0xffffffffu, wait(q_full, q_par));
      q_par ^= 1;
      for (int c = 0; c < np && ok; c += 2) {
        ok = __all_sync(0xffffffffu, wait(k_full + st, k_par) && wait(s_empty + sb, s_par));
        if (ok && stall_ns != 0) ok = __all_sync(0xffffffffu, wait(b_stall, 0, stall_ns));
        if (!ok) break;
        tc::fence_after_sync();
        if (leader) {
          const uint64_t kd = kd0 + (uint32_t)(st * (C::kChunkBytes >> 4));
          const uint32_t d = tmem + sb * C::kS;
          // a K step is 32 bytes of a row: 4 (bf16) or 2 (one byte) per plane
          constexpr int kSteps = KV8 ? 6 : 12, kPer = kSteps / 3;
#pragma unroll
          for (int kk = 0; kk < kSteps; ++kk)
            mma_ss<KV8>(d, kd + (((kk / kPer) * C::kPlane + (kk % kPer) * 32) >> 4),
                        qd0 + (((kk / kPer) * C::kQPlane + (kk % kPer) * 32) >> 4), idesc, kk > 0);
          tc::commit(k_empty + st);
          tc::commit(s_full + sb);
          if (c + 2 >= np) tc::commit(q_empty);
        }
        __syncwarp();
        if (++st == KS) {
          st = 0;
          k_par ^= 1;
        }
        if (++sb == C::kSBuf) {
          sb = 0;
          s_par ^= 1;
        }
      }
    }
    if (leader) tc::commit(b_final);  // arrives once every MMA issued above has completed
  } else if (warp == kWarpPv) {
    // ---------------- O^T += V^T P^T ----------------
    constexpr uint32_t base = (KV8 ? tc::idesc_f8_f32(0, C::kP, 0, 1) : tc::idesc_bf16_f32(0, C::kP)) | tc::kIdescMnA |
                              tc::kIdescMnB;
    constexpr uint32_t id1 = base | (128u >> 4) << 24, id2 = base | (64u >> 4) << 24;
    const uint64_t vd0 = tc::smem_desc_sw(smem_u32(sv), C::kPlane, C::kGroup, C::kRowB);
    const uint64_t pd0 = tc::smem_desc_sw(smem_u32(sp), 8 * C::kAtom, C::kPGroup, C::kAtom);
    const bool leader = elect_one();
    int st = 0, pb = 0;                       // V page, P buffer
    uint32_t v_par = 0, p_par = 0, o_par = 1;
    bool ok = true;
    auto page = [&](int y, bool first) {  // page y of the chunk
      if (leader) {
        constexpr int kSteps = KV8 ? 2 : 4, kGrp = 8 / kSteps;  // K steps of a page, 8-token groups of a step
        const uint64_t vd = vd0 + (uint32_t)(st * (PB >> 4));
        const uint64_t pd = pd0 + (uint32_t)((2 * pb + y) * (8 * C::kPGroup >> 4));
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
          const uint64_t vk = vd + (ks * kGrp * C::kGroup >> 4), pk = pd + (ks * kGrp * C::kPGroup >> 4);
          mma_ss<KV8>(tmem + C::kTmO, vk, pk, id1, !first || ks > 0);
          mma_ss<KV8>(tmem + C::kTmO2, vk + (2 * C::kPlane >> 4), pk, id2, !first || ks > 0);
        }
        tc::commit(v_empty + st);
      }
      __syncwarp();
      if (++st == VP) {
        st = 0;
        v_par ^= 1;
      }
    };
    while (ok && walk.next(x)) {
      const int np = __shfl_sync(0xffffffffu, x.np, 0);
      for (int c = 0; c < np; c += 2) {
        // V first: it is there long before P (unless the stream is behind)
        ok = __all_sync(0xffffffffu, wait(v_full + st, v_par) && wait(p_full + pb, p_par) && (c > 0 || wait(o_empty, o_par)));
        if (!ok) break;
        tc::fence_after_sync();
        page(0, c == 0);
        if (c + 1 < np) {  // (a run's last page may stand alone)
          ok = __all_sync(0xffffffffu, wait(v_full + st, v_par));
          if (!ok) break;
          page(1, false);
        }
        if (leader) tc::commit(p_free + pb);
        __syncwarp();
        if (++pb == C::kPBuf) {
          pb = 0;
          p_par ^= 1;
        }
      }
      o_par ^= 1;
    }
    if (leader) tc::commit(b_final);
  } else {
    // ---------------- softmax and epilogue: a thread is token tok of the chunk, then dim tok ----------------
    constexpr int NC = C::kCols;  // its columns, from c0
    const int tok = (warp & 3) * 32 + lane, half = warp >> 2, c0 = half * NC;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    auto soft_or = [](bool v) { return soft_or_n<C::kSoft>(v); };
    auto soft_sync = [] { soft_sync_n<C::kSoft>(); };
    int gc = 0, vp = 0, qi = 0;  // chunks, V pages, runs so far
    bool ok = true;              // this thread's waits so far; all decide at the barriers
    // Q of a run, once the products of the run before have read theirs
    float scale = 0.f;
    uint4 qv[C::kQPieces];
    constexpr bool kEarlyQ = RT == 1;  // (registers for it: 3 pieces a thread)
    auto stage_q = [&]() {
      scale = fmaxf(store_q<KV8, RT>(a, qv, sq, max_s, tid), 1e-37f);
      // (a scale of 0 must not make a score of -inf NaN)
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    };
    if (walk.rem > 0) {
      walk.run(x);
      fetch_q<KV8, RT>(a, x, tid, qv);
      stage_q();
    }
    while (walk.next(x)) {
      const int t_last = x.t0 + x.nr - 1;
      if (tid < NQ) ref_s[tid] = 0.f;
      bool had = false;  // (thread i < NQ) column i has a reference
      if (soft_or(!ok)) {
        ok = false;
        break;
      }
      if (kEarlyQ && walk.rem > 0) {  // the next run's Q is under way during this one
        Seg y;
        walk.run(y);
        fetch_q<KV8, RT>(a, y, tid, qv);
      }
      float2 l[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) l[i] = make_float2(0.f, 0.f);
      bool force = true;  // some column has no reference yet
      const int32_t *pt = a.page_table + (size_t)x.s * a.max_pages + x.p0;
      int nxt = lane < x.np ? ld_cg(pt + lane) : -1;
      uint32_t good = 0;  // bit i: page i of the current 32 is in the pool (none behind the run's last)
      for (int c = 0; c < x.np; c += 2, ++gc) {
        if ((c & 31) == 0) {
          good = __ballot_sync(0xffffffffu, nxt >= 0 && nxt < a.num_pages);
          nxt = c + 32 + lane < x.np ? ld_cg(pt + c + 32 + lane) : -1;
        }
        const bool ok_a = (good >> (c & 31)) & 1, ok_b = (good >> (c & 31)) & 2;
        const int base = (x.p0 + c) * kPage;
        const bool masked = !ok_a || !ok_b || base + kChunk - 1 > x.t0;
        const int sb = gc % C::kSBuf;
        // (the references are fetched before the wait: while products run, they take most of shared
        // memory's bandwidth, and these loads took 800 cycles of a 4-row tile's chunk after it)
        float4 ref[NC / 4];
#pragma unroll
        for (int i = 0; i < NC / 4; ++i) ref[i] = *reinterpret_cast<const float4 *>(ref_s + c0 + 4 * i);
        ok = ok && wait(s_full + sb, (gc / C::kSBuf) & 1);
        __syncwarp();
        tc::fence_after_sync();
        // the token's scores, two columns per element
        float2 sc[NC / 2];
        {
          const uint32_t ts = tl + sb * C::kS + c0;
          if constexpr (!KV8) {
#pragma unroll
            for (int i = 0; i < NC / 16; ++i)
              tc::ld_16cols(ts + 16 * i, *reinterpret_cast<uint32_t(*)[16]>(reinterpret_cast<uint32_t *>(sc) + 16 * i));
            tc::wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < NC / 16; ++i) {
              uint32_t lo[16];
              tc::ld_16cols(ts + 16 * i, *reinterpret_cast<uint32_t(*)[16]>(reinterpret_cast<uint32_t *>(sc) + 16 * i));
              tc::ld_16cols(ts + NQ + 16 * i, lo);
              tc::wait_ld();
#pragma unroll
              for (int y = 0; y < 8; ++y)
                sc[8 * i + y] = fma2(make_float2(__uint_as_float(lo[2 * y]), __uint_as_float(lo[2 * y + 1])),
                                     make_float2(0.0625f, 0.0625f), sc[8 * i + y]);
            }
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty + sb);
        if (masked) {
          const int pos = (tok < kPage ? ok_a : ok_b) ? base + tok : 0x7fffffff;
#pragma unroll
          for (int j = 0; j < NC / kHpg; ++j)
            if (pos > min(x.t0 + c0 / kHpg + j, t_last))
#pragma unroll
              for (int i = 0; i < 8; ++i) sc[8 * j + i] = make_float2(-INFINITY, -INFINITY);
        }
        // relative to the references, in log2 units
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < NC / 2; i += 2) {
          const float4 r = ref[i / 2];
          sc[i] = fma2(sc[i], make_float2(scale, scale), make_float2(-r.x, -r.y));
          sc[i + 1] = fma2(sc[i + 1], make_float2(scale, scale), make_float2(-r.z, -r.w));
          mx[0] = max3(mx[0], sc[i].x, sc[i].y);
          mx[1] = max3(mx[1], sc[i + 1].x, sc[i + 1].y);
        }
        // a reference moves only when a weight would exceed 2^kTop (or with its first finite score)
        if (soft_or(force || !ok || fmaxf(mx[0], mx[1]) > C::kTop)) {
          // maxima of the columns over the chunk's tokens
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            int b = __float_as_int(fmaxf((i & 1) ? sc[i / 2].y : sc[i / 2].x, -INFINITY));  // (NaN: -inf)
            b = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7fffffff));
            if (lane == i) warp_s[(warp & 3) * NQ + c0 + i] = __int_as_float(b ^ ((b >> 31) & 0x7fffffff));
          }
          if (soft_or(!ok)) {
            ok = false;
            break;
          }
          bool none = false;
          if (tid < NQ) {
            const float top = fmaxf(fmaxf(warp_s[tid], warp_s[NQ + tid]), fmaxf(warp_s[2 * NQ + tid], warp_s[3 * NQ + tid]));
            const bool grow = had ? top > C::kTop : top > -INFINITY;
            const float shift = grow ? top - C::kOff : 0.f;
            shift_s[tid] = shift;
            corr_s[tid] = grow && had ? hw_exp2(-shift) : 1.f;
            ref_s[tid] += shift;
            had = had || grow;
            none = !had;
          }
          force = soft_or(none);
#pragma unroll
          for (int i = 0; i < NC / 2; ++i) {
            const float2 sh = *reinterpret_cast<const float2 *>(shift_s + c0 + 2 * i);
            const float2 co = *reinterpret_cast<const float2 *>(corr_s + c0 + 2 * i);
            sc[i] = add2(sc[i], make_float2(-sh.x, -sh.y));
            l[i].x *= co.x;
            l[i].y *= co.y;
          }
          if (c > 0) {  // O^T holds the chunks before: after their last product
            ok = ok && wait(p_free + (gc - 1) % C::kPBuf, ((gc - 1) / C::kPBuf) & 1);
            __syncwarp();
            tc::fence_after_sync();
#pragma unroll 1
            for (int cb = half; cb < 2 * C::kP / 16; cb += C::kHalves) {
              uint32_t o[16];
              tc::ld_16cols(tl + C::kTmO + cb * 16, o);
              tc::wait_ld();
              const float *co = corr_s + (cb * 16) % NQ;
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * co[i]);
              tc::st_16cols(tl + C::kTmO + cb * 16, o);
            }
            tc::wait_st();
          }
        }
        // P, last read by the products of the chunk kPBuf before
        const int pbuf = gc % C::kPBuf;
        if (gc >= C::kPBuf) ok = ok && wait(p_free + pbuf, (gc / C::kPBuf - 1) & 1);
        {
          uint8_t *row = sp + pbuf * 16 * C::kPGroup + (tok >> 3) * C::kPGroup + (tok & 7) * C::kAtom;
          const int sw = C::kAtom == 128 ? tok & 7 : (tok >> 1) & 3;
          constexpr int kPer = C::kAtom / 16;  // 16-byte pieces of an atom's row
          auto piece = [&](int i) {
            return reinterpret_cast<uint4 *>(row + (i / kPer) * 8 * C::kAtom + (((i % kPer) ^ sw) << 4));
          };
          constexpr int kPc = KV8 ? 16 : 8;  // columns of a piece
#pragma unroll
          for (int i0 = 0; i0 < NC; i0 += kPc) {
            uint32_t w[C::kTerms][4];
#pragma unroll
            for (int i = 0; i < kPc; i += KV8 ? 4 : 2) {
              float2 p2[2];
#pragma unroll
              for (int y = 0; y < (KV8 ? 2 : 1); ++y) {
                const int at = (i0 + i) / 2 + y;
                p2[y] = make_float2(hw_exp2(sc[at].x), hw_exp2(sc[at].y));
                l[at] = add2(l[at], p2[y]);
              }
              if constexpr (KV8) {
                uint32_t r0 = float2_to_f16x2(p2[0].x, p2[0].y), r1 = float2_to_f16x2(p2[1].x, p2[1].y);
#pragma unroll
                for (int t = 0; t < C::kTerms; ++t) {
                  if (t == C::kTerms - 1 && C::kTerms < 4) {  // the last term to nearest
                    r0 += 0x00800080u;
                    r1 += 0x00800080u;
                  }
                  w[t][i / 4] = __byte_perm(r0, r1, 0x7531);
                  if (t + 1 < C::kTerms) {
                    r0 = sub_f16x2(r0, r0 & 0xFF00FF00u);
                    r1 = sub_f16x2(r1, r1 & 0xFF00FF00u);
                  }
                }
              } else {
                const uint32_t b0 = __float_as_uint(p2[0].x), b1 = __float_as_uint(p2[0].y);
                const float2 r = fma2(make_float2(__uint_as_float(b0 & 0xFFFF0000u), __uint_as_float(b1 & 0xFFFF0000u)),
                                      make_float2(-1.f, -1.f), p2[0]);
                w[0][i / 2] = __byte_perm(b0, b1, 0x7632);
                w[1][i / 2] = __byte_perm(__float_as_uint(r.x), __float_as_uint(r.y), 0x7632);
              }
            }
#pragma unroll
            for (int t = 0; t < C::kTerms; ++t)
              *piece((t * NQ + c0 + i0) / kPc) = make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
          }
        }
        if (masked) {
          // V of tokens that a row of the tile does not see must not be NaN or infinite.  (The chunk before
          // must be done: until its pages have been consumed, a wait for this chunk's pages could take
          // the ring slot's phase before last for the one it waits for.)
          if (gc >= 1) ok = ok && wait(p_free + (gc - 1) % C::kPBuf, ((gc - 1) / C::kPBuf) & 1);
#pragma unroll 1
          for (int y = 0; y < min(2, x.np - c); ++y) {
            const int st = (vp + y) % VP, first = base + y * kPage;
            const bool ok_y = y == 0 ? ok_a : ok_b;
            if (ok_y && first + kPage - 1 <= x.t0) continue;
            ok = ok && wait(v_full + st, ((vp + y) / VP) & 1);
            clean_v<KV8, RT>(sv + st * PB, bad_s, ok_y, x.t0 - first, t_last - first, tid);
          }
        }
        vp += min(2, x.np - c);
        fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + pbuf);
      }

      // ---- the run's result ----
      if (walk.rem > 0) {  // the next run's Q first, so that its first scores are there after this epilogue
        ok = ok && wait(q_empty, qi & 1);
        if (!kEarlyQ) {
          Seg y;
          walk.run(y);
          fetch_q<KV8, RT>(a, y, tid, qv);
        }
        stage_q();
      }
      // column sums over the warp: halves of the columns are exchanged until a lane has one
      {
        float v[NC];
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) {
          v[2 * i] = l[i].x;
          v[2 * i + 1] = l[i].y;
        }
        int n = NC, at = 0;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
          if (n > 1) {
            n >>= 1;
            const bool up = (lane & o) != 0;
            if (up) at += n;
#pragma unroll
            for (int i = 0; i < NC / 2; ++i)
              if (i < n) v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + n], o);
          } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
          }
        }
        // the last products: once they are done, no warp reads what a moved reference left in warp_s
        ok = ok && wait(p_free + (gc - 1) % C::kPBuf, ((gc - 1) / C::kPBuf) & 1);
        warp_s[(warp & 3) * NQ + c0 + at] = v[0];
      }
      if (soft_or(!ok)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const bool whole = x.np == x.tile_pages;
      const Parts parts = parts_of(x, chunk);
      const size_t my_slot = parts.slot((int)blockIdx.x - parts.first);
      float *po = a.part_o + my_slot * NQ * kD;
      if (tid < NQ) {
        const float L = (warp_s[tid] + warp_s[NQ + tid]) + (warp_s[2 * NQ + tid] + warp_s[3 * NQ + tid]);
        const float M = had ? ref_s[tid] : -INFINITY;
        corr_s[tid] = whole ? (L == 0.f ? 0.f : a.v_scale / L) : 1.f;
        if (tid / kHpg < x.nr) {
          if (whole) {
            if (a.lse != nullptr) a.lse[out_row(x, tid)] = L == 0.f ? -INFINITY : (M + hw_log2(L)) * kLn2;
          } else {
            float *ml = a.part_ml + my_slot * 2 * NQ;
            ml[tid] = M;
            ml[NQ + tid] = L;
            // the CTA where a tile begins tells the joining kernel about it
            if (tid == 0 && parts.first == (int)blockIdx.x) a.joins[blockIdx.x] = make_int4(parts.n, x.row0, x.nr, x.g);
          }
        }
      }
      soft_sync();
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {  // dims 0-127, then 128-191 (M = 64: 16 lanes of a lane quarter)
        const int d = part == 0 ? tok : 128 + (warp & 3) * 16 + lane;
        const bool on = part == 0 || lane < 16;
        const uint32_t nf = on ? bad_s[d >> 2] >> (8 * (d & 3)) : 0;  // bit j: row j saw a value that is not finite
#pragma unroll 1
        for (int j = c0 / kHpg; j < min(x.nr, (c0 + NC) / kHpg); ++j) {
          float v[16];
          uint32_t o[C::kTerms][16];
#pragma unroll
          for (int t = 0; t < C::kTerms; ++t)
            tc::ld_16cols(tl + (part == 0 ? C::kTmO : C::kTmO2) + t * NQ + j * 16, o[t]);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] = __uint_as_float(o[0][i]);
#pragma unroll
            for (int t = 1; t < C::kTerms; ++t) v[i] += __uint_as_float(o[t][i]);
            v[i] *= corr_s[j * 16 + i];
            if ((nf >> j) & 1u) v[i] = __uint_as_float(0x7FC00000u);
          }
          if (on) {
            if (whole) {
              __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(a.out) + out_row(x, j * kHpg) * kD + d;
#pragma unroll
              for (int i = 0; i < 16; ++i) out[i * kD] = __float2bfloat16(v[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) po[(size_t)(j * 16 + i) * kD + d] = v[i];
            }
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty);
      ++qi;
      soft_sync();  // the columns' values and bad_s are free again
      if (tid < 48) bad_s[tid] = 0;
    }
  }

  // ---- teardown: no MMA may be writing tensor memory when it is released ----
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kWarpPv) {
    mbar_wait_bounded(b_final, 0, kDnWaitNs);
    tc::tmem_dealloc(tmem, C::kTmCols);
  }
}

// ---------------------------------------------------------------- the joining kernel

// Work items: of a tile of at most kFewParts parts four (row, head) pairs, a warp each; of a tile of more
// parts one pair, whose parts the CTA's warps share (warp w takes parts w, w + 4, ...; their sums are
// added in warp order).  Few parts come with many tiles and many parts with few tiles, so either way the
// SMs have enough items and a few rounds of loads end each.  4 to 5 us behind the first kernel, for 4
// tiles of 37 parts as for 130 of 2 or 3; latency-bound (records, then references, sums and parts, one
// round trip each, and the launch).  Four CTAs per SM: six hold a thread to 80 registers, which spills 100
// bytes and makes the calls 0.4 to 0.9 us longer (1 x 1,000 tokens 10.7 against 10.3 us).
constexpr int kJoinThreads = 128, kJoinWarps = kJoinThreads / 32, kJoinCtasPerSm = 4;
constexpr int kFewParts = 4, kMaxCtas = 256;
static_assert(kMaxCtas == 2 * kJoinThreads, "two records per thread");

__device__ __forceinline__ void store_joined(const DenseArgs &a, size_t row, int lane, const float2 (&o)[3], float top,
                                             float sum) {
  const float inv = sum == 0.f ? 0.f : a.v_scale / sum;
#pragma unroll
  for (int e = 0; e < 3; ++e)
    reinterpret_cast<uint32_t *>(a.out)[row * (kD / 2) + lane + 32 * e] = pack_bf16(o[e].x * inv, o[e].y * inv);
  if (lane == 0 && a.lse != nullptr) a.lse[row] = sum == 0.f ? -INFINITY : (top + hw_log2(sum)) * kLn2;
}

template <int RT>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtasPerSm) dense_join_kernel(const DenseArgs a) {
  constexpr int NQ = RT * kHpg;
  __shared__ int4 rec_s[kMaxCtas];
  __shared__ int first_s[kMaxCtas + 1];  // first item of a CTA's tile
  __shared__ int sum_s[kJoinWarps];
  __shared__ float w_s[kMaxCtas], red_s[2][kJoinWarps];
  __shared__ float2 acc_s[kJoinWarps][kD / 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  int items[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = 2 * tid + i;
    uint4 r = make_uint4(0, 0, 0, 0);
    if (c < a.n_ctas) r = ld_cg(reinterpret_cast<const uint4 *>(a.joins + c));
    rec_s[c] = make_int4((int)r.x, (int)r.y, (int)r.z, (int)r.w);
    items[i] = r.x == 0 ? 0 : (int)r.z * (r.x <= kFewParts ? kHpg / kJoinWarps : kHpg);
  }
  int incl = items[0] + items[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sum_s[warp] = incl;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w)
    if (w < warp) incl += sum_s[w];
  first_s[2 * tid + 1] = incl - items[1];
  first_s[2 * tid + 2] = incl;
  if (tid == 0) first_s[0] = 0;
  __syncthreads();
  const int total = first_s[kMaxCtas];
  for (int it = blockIdx.x; it < total; it += gridDim.x) {
    int c = 0;  // the last c with first_s[c] <= it: its tile has the item
#pragma unroll
    for (int o = kMaxCtas / 2; o >= 1; o >>= 1)
      if (first_s[c + o] <= it) c += o;
    const int n = rec_s[c].x, row0 = rec_s[c].y, g = rec_s[c].w, i0 = it - first_s[c];
    const Parts parts{c, n};
    if (n <= kFewParts) {
      const int q = i0 * kJoinWarps + warp;
      float m[kFewParts], l[kFewParts], top = -INFINITY, sum = 0.f;
      float2 v[kFewParts][3], o[3] = {};
#pragma unroll
      for (int i = 0; i < kFewParts; ++i) {
        m[i] = -INFINITY;
        if (i < n) {
          const float *ml = a.part_ml + (size_t)parts.slot(i) * 2 * NQ + q;
          m[i] = ld_cg(ml);
          l[i] = ld_cg(ml + NQ);
          const float *src = a.part_o + ((size_t)parts.slot(i) * NQ + q) * kD + 2 * lane;
#pragma unroll
          for (int e = 0; e < 3; ++e) v[i][e] = ld_cg2(src + 64 * e);
        }
      }
#pragma unroll
      for (int i = 0; i < kFewParts; ++i) top = fmaxf(top, m[i]);
      const float tu = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int i = 0; i < kFewParts; ++i)
        if (i < n) {
          const float w = hw_exp2(m[i] - tu);
          sum = fmaf(w, l[i], sum);
#pragma unroll
          for (int e = 0; e < 3; ++e) o[e] = fma2(make_float2(w, w), v[i][e], o[e]);
        }
      store_joined(a, (size_t)(row0 + q / kHpg) * kHeads + g * kHpg + q % kHpg, lane, o, top, sum);
    } else {
      const int q = i0;
      float m[2], l[2], top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int p = tid + i * kJoinThreads;
        const float *ml = a.part_ml + (size_t)parts.slot(p) * 2 * NQ + q;
        m[i] = p < n ? ld_cg(ml) : -INFINITY;
        l[i] = p < n ? ld_cg(ml + NQ) : 0.f;
        top = fmaxf(top, m[i]);
      }
      float2 o[3] = {};
      for (int p0 = warp; p0 < n; p0 += 8 * kJoinWarps) {
        float2 v[8][3];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (p0 + i * kJoinWarps < n) {
            const float *src = a.part_o + ((size_t)parts.slot(p0 + i * kJoinWarps) * NQ + q) * kD + 2 * lane;
#pragma unroll
            for (int e = 0; e < 3; ++e) v[i][e] = ld_cg2(src + 64 * e);
          }
        if (p0 == warp) {  // (every warp has a part: n > kFewParts) the weights, while the first parts come
#pragma unroll
          for (int x = 16; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          if (lane == 0) red_s[0][warp] = top;
          __syncthreads();
#pragma unroll
          for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, red_s[0][w]);
          const float tu = top == -INFINITY ? 0.f : top;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float w = hw_exp2(m[i] - tu);
            w_s[tid + i * kJoinThreads] = w;
            sum = fmaf(w, l[i], sum);
          }
#pragma unroll
          for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          if (lane == 0) red_s[1][warp] = sum;
          __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (p0 + i * kJoinWarps < n) {
            const float w = w_s[p0 + i * kJoinWarps];
#pragma unroll
            for (int e = 0; e < 3; ++e) o[e] = fma2(make_float2(w, w), v[i][e], o[e]);
          }
      }
#pragma unroll
      for (int e = 0; e < 3; ++e) acc_s[warp][lane + 32 * e] = o[e];
      __syncthreads();
      if (warp == 0) {
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
          sum += red_s[1][w];
          if (w > 0)
#pragma unroll
            for (int e = 0; e < 3; ++e) o[e] = add2(o[e], acc_s[w][lane + 32 * e]);
        }
        store_joined(a, (size_t)(row0 + q / kHpg) * kHeads + g * kHpg + q % kHpg, lane, o, top, sum);
      }
      __syncthreads();  // the shared arrays are written again
    }
  }
}

template <bool KV8, int RT>
cudaError_t launch(const DenseArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t st) {
  auto kernel = dense_kernel<KV8, RT>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), Cfg<KV8, RT>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.n_ctas);
  cfg.blockDim = dim3(Cfg<KV8, RT>::kThreads);
  cfg.dynamicSmemBytes = Cfg<KV8, RT>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a, tk, tv);
  if (e != cudaSuccess || a.n_ctas == 1 || a.whole) return e;
  cfg.gridDim = dim3((unsigned)(a.n_ctas * kJoinCtasPerSm));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, dense_join_kernel<RT>, a);
}

}  // namespace

cudaError_t launch_dense(const DenseArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t st) {
  switch (a.tile_rows + (a.kv8 ? 16 : 0)) {
    case 1: return launch<false, 1>(a, tk, tv, st);
    case 2: return launch<false, 2>(a, tk, tv, st);
    case 4: return launch<false, 4>(a, tk, tv, st);
    case 17: return launch<true, 1>(a, tk, tv, st);
    case 18: return launch<true, 2>(a, tk, tv, st);
    case 20: return launch<true, 4>(a, tk, tv, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace s5
