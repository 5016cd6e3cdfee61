// Accumulated attention weights of cached keys (fa_kv_accumulate): for each sequence, kv head and key j
//   weight[j] = (j is a new token's ? 0 : weight[j]) + sum over new tokens i and heads h of the group,
//               where i sees j, of exp(scale q_ih . k_j - lse_ih).
//
// One pass over K; the log-sum-exps are the attention call's, so nothing has to be known of other keys.
// S^T = K Q^T on the tensor core: the keys are the 128 rows of the instruction, a row of tensor memory and a thread
// each, so that a key's sum needs no exchange between threads, and a single token's few query heads are the
// narrow side (16, 32 or 64 columns; 128 for chunks).  One kernel serves both:
//   * a unit is 256 keys (two tiles) of one sequence and kv head; a persistent CTA takes its units one after the
//     other and streams, for each, the query blocks that see its keys.  No atomics, the same bits in every call.
//   * few rows (decoding): the bytes of K bound it.  A CTA has a run of units, most of them of one head, whose
//     queries stay in shared memory; a ring of K tiles is kept full.  64 sequences, 284k keys, 8 kv heads of 128:
//     E4M3 55 us (85 % of the copy rate), BF16 95 us (93 %).
//   * chunks: 256 x 128 pairs of a head take 1024 clocks of tensor work, and as many for their exponentials (32 a clock
//     and SM); both together, with the sums between them, bound it.  2048 tokens over 34k keys, 32 heads of 128: 388
//     to 411 us, 1350 to 1430 TFLOP/s, from run to run (without the products 339).  Units are dealt round by round, early
//     keys, which most tokens see, first.  Where there are few of them each is cut into parts by its query blocks, whose sums
//     a second kernel joins in order.
// E4M3 caches, few rows: the codes are the operand as they are (kind::f8f6f4).  A query vector goes into three E5M2
// vectors that add up to it: BF16 has 8 significant bits, E5M2 3, and its smallest step is 2^-30 of the largest entry or
// less.  Entries of at least 2^-23 of the largest are exact, smaller ones off by 2^-31 of it at most.  Chunks: a warpgroup
// turns the codes into BF16, once for all the query blocks of a unit.  The key's scale multiplies S in FP32.
#include <limits.h>
#include <stdlib.h>

#include <algorithm>

#include "paged_attn.cuh"

namespace fa {
namespace paged {

constexpr int kAccKeys = 256;        // of a unit
constexpr int kAccTile = 128;        // keys of a tile
constexpr int kPieces = 3;           // E5M2 vectors of a query vector
constexpr float kLog2e = 1.4426950408889634f, kLog2eRest = (float)(1.4426950408889634 - (double)kLog2e);
constexpr int kColStages = 4;        // blocks of queries whose log-sum-exps are in shared memory
// Chunks: units are cut into parts until there are about eight for each of 152 SMs, none of less than four
// query blocks.
constexpr int kMostParts = 1216, kPartBlocks = 4;

struct Acc {
  Attn a;                  // queries, cache, lengths (o and lse are not used)
  const float* lse;        // [T, Hq]
  float* weights;          // [pages][Hkv][page_size]
  long long weight_stride;
  const float* q_scale;    // E4M3, few rows: [T, Hq], what the pieces are to be multiplied by
  float scale_log2;        // scale log2(e)
  float* part;             // chunks: [kMostParts][kAccKeys], the parts' sums
  int max_parts;           // of a unit
};

template <int D, bool kFp8, int N>
struct AccCfg {
  static constexpr bool kChunk = N == 128;
  static constexpr bool kPieced = kFp8 && !kChunk, kConvert = kFp8 && kChunk;
  // the pieces side by side, 3 N columns of S that are added afterwards: the tensor core then reads K once.  (64
  // columns leave no room for that: S takes the pieces one after the other.)
  static constexpr bool kWide = kPieced && N <= 32;
  // chunks: two sets of warps take the blocks in turn, the one with an even place (of its tile) the first buffer of S, the
  // other the second, and add their sums at the end of a unit.  2048 tokens over 34k keys 390 us (at best, as the
  // other figures here); two sets with half of each block's columns 406, one set 423.  Not with converters beside them: 80
  // registers are too few (466 us, 431).
  static constexpr int kHalves = kChunk && !kConvert ? 2 : 1;
  static constexpr int kSumWarps = 8 * kHalves, kThreads = 32 * (kSumWarps + (kConvert ? 8 : 4));
  // CTAs on an SM: two where each holds three units' keys or more.  (A unit's hand-offs take longer than its 16 or 32 KB:
  // decoding over 284k E4M3 keys, d = 128, 61 us with one.)
  static constexpr int kCtas = N == 16 && D * (kFp8 ? 1 : 2) <= 128 ? 2 : 1;
  // operands
  static constexpr int kRowBytes = D * (kPieced ? 1 : 2);
  static constexpr int kAtomBytes = kRowBytes < 128 ? kRowBytes : 128;   // swizzle atom row
  static constexpr int kAtoms = kRowBytes / kAtomBytes, kAtomElems = D / kAtoms;
  static constexpr int kTileBytes = kAccTile * kRowBytes, kPairBytes = 2 * kTileBytes;
  static constexpr int kQTile = N * kRowBytes, kQBytes = (kPieced ? kPieces : 1) * kQTile;
  static constexpr int kQStages = kChunk ? (kConvert ? 3 : 4) : 2;
  static constexpr int kCodeBytes = kConvert ? kAccKeys * D : 0;         // a unit's codes
  static constexpr int kColBytes = (kPieced ? 2 : 1) * N * 4;            // a block's columns: -lse, and pieces: the factor
  static constexpr int kSideStages = kChunk ? 2 : 8 / kCtas;
  static constexpr int kSideBytes = kAccKeys * 4 * (kFp8 ? 2 : 1) + 64;  // a unit's weights, scales and pages
  static constexpr int kQOff = 0;
  static constexpr int kCodeOff = kQOff + kQStages * kQBytes, kKOff = kCodeOff + kCodeBytes;
  static constexpr int kHalfBytes = kHalves == 2 ? 2 * kAccKeys * 4 : 0; // two units' sums of the second set
  static constexpr int kRest = kColStages * kColBytes + kSideStages * kSideBytes + kHalfBytes;
  static constexpr int kRoom = (kCtas == 2 ? 112 : 226) * 1024 - kKOff - kRest;
  static constexpr int kKStages = kRoom / kPairBytes < 6 ? kRoom / kPairBytes : 6;
  static constexpr int kColOff = kKOff + kKStages * kPairBytes, kSideOff = kColOff + kColStages * kColBytes;
  static constexpr int kHalfOff = kSideOff + kSideStages * kSideBytes;
  static constexpr int kSharedOff = kColOff + kRest;
  // S: buffers of a tile, each kBufCols columns of tensor memory
  static constexpr int kSCols = kWide ? kPieces * N : N, kBufCols = kWide ? 4 * N : N;
  static constexpr int kBufs = 2 * 4 * kBufCols * kCtas <= 512 ? 4 : 2;
  static constexpr int kTmemCols = 2 * kBufs * kBufCols;
  static constexpr uint32_t kIdesc = kPieced ? idesc_e4m3(128, kSCols, false, false) | (1u << 10)   // B: E5M2
                                             : idesc_bf16(128, N, false, false);
  static_assert(kKStages >= 1 && kTmemCols * kCtas <= 512 && kTmemCols >= 32, "shared or tensor memory");
};

constexpr int kMaxKStages = 6, kMaxQStages = 4, kMaxBufs = 4, kMaxSideStages = 8, kMaxWarps = 20;

struct AccShared {
  uint64_t k_full[kMaxKStages], k_empty[kMaxKStages], q_full[kMaxQStages], q_empty[kMaxQStages];
  uint64_t col_full[kColStages], col_empty[kColStages], side_full[kMaxSideStages], side_empty[kMaxSideStages];
  uint64_t s_full[2][kMaxBufs], s_empty[2][kMaxBufs];
  uint64_t code_full, code_empty;  // E4M3 chunks: a unit's codes have landed / have been read
  uint64_t half_full[2][2], half_empty[2][2];  // sums of the second set of warps: by tile, two units'
  uint64_t mma_done;
  uint64_t never;                  // test builds only: a barrier nothing arrives on
  long long scan[kMaxWarps];
  long long first;                 // this CTA's first unit (or part) within its sequence
  uint32_t tmem_base, abort_flag;
  int first_b;                     // that sequence; -1: none
};

template <int D, bool kFp8, int N>
constexpr int acc_smem() {
  return AccCfg<D, kFp8, N>::kSharedOff + (int)sizeof(AccShared);
}
template <int D, bool kFp8>
constexpr bool acc_fits() {
  return AccCfg<D, kFp8, 16>::kCtas * (acc_smem<D, kFp8, 16>() + 1024) <= 228 * 1024 &&
         acc_smem<D, kFp8, 32>() <= 227 * 1024 && acc_smem<D, kFp8, 64>() <= 227 * 1024 &&
         acc_smem<D, kFp8, 128>() <= 227 * 1024;
}
static_assert(acc_fits<64, false>() && acc_fits<64, true>() && acc_fits<128, false>() && acc_fits<128, true>(),
              "shared-memory layout exceeds 227 KB");

// A sequence's units: its walk's blocks of keys for each kv head.
struct AccSeq {
  Seq s;
  KeyWalk<kAccKeys> w;
  __device__ __forceinline__ AccSeq(const Attn& p, int b) : s(load_seq(p, b)), w(p, s.pos0, s.kv - 1) {
    if (s.n == 0 || w.hi == 0) w.steps = 0;
  }
  __device__ __forceinline__ long long units(const Attn& p) const { return (long long)w.steps * p.c.Hkv; }
};

// Sums the sequences' units over the CTA, settles into how many parts each is cut, and finds what `range`
// asks for: the sequence (first_b, -1: none) that holds number `want` of the launch's parts, the number within it
// (first) and how many are wanted (count).  Returns the parts of a unit.
template <int kThreads, class Range>
__device__ __forceinline__ int find_units(const Attn& p, int max_parts, long long* scan, int& first_b, long long& first,
                                          long long& count, Range range) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int per = (p.c.B + kThreads - 1) / kThreads;
  const int b_from = min((int)threadIdx.x * per, p.c.B), b_to = min(b_from + per, p.c.B);
  long long mine = 0;
  for (int b = b_from; b < b_to; ++b) mine += AccSeq(p, b).units(p);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) scan[warp] = incl;
  if (threadIdx.x == 0) first_b = -1;
  __syncthreads();
  long long from = incl - mine, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) from += scan[w];
    all += scan[w];
  }
  const int parts = all > 0 ? (int)max(min((long long)max_parts, kMostParts / all), 1ll) : 1;
  long long want;
  count = range(all, parts, want);
  from *= parts;
  if (count > 0 && want >= from && want < from + mine * parts) {
    for (int b = b_from; b < b_to; ++b) {
      const long long n = AccSeq(p, b).units(p) * parts;
      if (want < from + n) {
        first = want - from;
        first_b = b;
        break;
      }
      from += n;
    }
  }
  __syncthreads();
  return parts;
}

// A CTA's units, in order.  Every role walks them with a copy of its own.  Few rows: a run of them, ordered by
// sequence, kv head and block of keys.  Chunks: every gridDim.x-th part, ordered by sequence, block of keys,
// kv head and part.
template <bool kChunk>
struct AccCursor {
  int b, h, j, part;       // sequence (B: no unit is left), kv head, step of the walk, part
  bool fresh;              // the first of its head in this CTA
  long long left;          // few rows: units until the end of the run; chunks: number within the sequence
  Seq s;
  KeyWalk<kAccKeys> w;
  __device__ __forceinline__ AccCursor(const Attn& p, int parts, int first_b, long long first, long long n)
      : b(first_b), h(0), j(0), part(0), fresh(true), left(kChunk ? first : n), s{}, w(p, 0, -1) {
    if (b < 0) {
      b = p.c.B;
      return;
    }
    const AccSeq x(p, b);
    s = x.s;
    w = x.w;
    if constexpr (kChunk) {
      place(p, parts);
    } else {
      h = (int)(first / w.steps);
      j = (int)(first - (long long)h * w.steps);
    }
  }
  __device__ __forceinline__ void place(const Attn& p, int parts) {
    const int r = (int)(left / parts);   // (a sequence's units are under 2^27)
    part = (int)(left - (long long)r * parts);
    j = r / p.c.Hkv;
    h = r - j * p.c.Hkv;
  }
  __device__ __forceinline__ bool valid(const Attn& p) const { return b < p.c.B; }
  __device__ __forceinline__ void next(const Attn& p, int parts) {
    if constexpr (kChunk) {
      left += gridDim.x;
      for (long long n = (long long)w.steps * p.c.Hkv * parts; left >= n; n = (long long)w.steps * p.c.Hkv * parts) {
        left -= n;
        if (++b >= p.c.B) return;
        const AccSeq x(p, b);
        s = x.s;
        w = x.w;
      }
      place(p, parts);
    } else {
      fresh = false;
      if (--left == 0) {
        b = p.c.B;
        return;
      }
      if (++j < w.steps) return;
      j = 0;
      fresh = true;
      if (++h < p.c.Hkv) return;
      h = 0;
      for (++b; b < p.c.B; ++b) {
        const AccSeq x(p, b);
        if (x.w.steps == 0) continue;
        s = x.s;
        w = x.w;
        return;
      }
    }
  }
  // whether the next unit has another head's queries, or there is none
  __device__ __forceinline__ bool last() const { return left == 1 || j + 1 == w.steps; }
  __device__ __forceinline__ int key() const { return w.at(j); }
  // the blocks of queries that see a key of the unit, or this part's share of them: [from, to).  (Few rows: one.)
  __device__ __forceinline__ void blocks(const Attn& p, int parts, int tokens, int& from, int& to) const {
    from = 0;
    to = 1;
    if constexpr (kChunk) {
      const int lo = max(key() - s.pos0, 0) / tokens;
      int hi = (s.n + tokens - 1) / tokens;
      if (p.window && key() >= p.sinks) {
        const long long t = (long long)key() + kAccKeys - 1 + p.window - 1 - s.pos0;   // the last token that sees one
        hi = t < 0 ? 0 : (int)min((long long)hi, t / tokens + 1);
      }
      const int n = max(hi - lo, 0);
      from = lo + (int)((long long)n * part / parts);
      to = lo + (int)((long long)n * (part + 1) / parts);
    }
  }
  // whether tile t of the unit has keys
  __device__ __forceinline__ bool tile(int t) const { return key() + t * kAccTile < w.hi; }
};

// sum += of the columns: 2^(S f factor - l), of those in `mask` alone where kMasked; l is lse log2(e), and the factors
// hold scale log2(e), so that an exponential takes one product and sum.  (A product with log2(e) behind the difference
// of natural logarithms costs two instructions more for four columns: 2048 tokens over 34k keys 428 us, this 406.)
// kPieced: the query's factor first: codes times q stays in FP32's range, where pieces times a large key's scale
// would not.
template <int W, bool kPieced, bool kMasked>
__device__ __forceinline__ void acc_columns(const uint32_t (&r)[W], const float* neg_lse, const float* factor, float f,
                                            uint32_t mask, float (&sum)[4]) {
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const float4 l = *reinterpret_cast<const float4*>(neg_lse + i);
    float s0 = __uint_as_float(r[i]), s1 = __uint_as_float(r[i + 1]), s2 = __uint_as_float(r[i + 2]), s3 = __uint_as_float(r[i + 3]);
    if constexpr (kPieced) {
      const float4 y = *reinterpret_cast<const float4*>(factor + i);
      mul2(s0, s1, s0, s1, y.x, y.y);
      mul2(s2, s3, s2, s3, y.z, y.w);
    }
    fma2(s0, s1, s0, s1, f, f, l.x, l.y);
    fma2(s2, s3, s2, s3, f, f, l.z, l.w);
    float e0 = ex2_approx(s0), e1 = ex2_approx(s1), e2 = ex2_approx(s2), e3 = ex2_approx(s3);
    if constexpr (kMasked) {
      e0 = mask >> i & 1 ? e0 : 0.f;
      e1 = mask >> (i + 1) & 1 ? e1 : 0.f;
      e2 = mask >> (i + 2) & 1 ? e2 : 0.f;
      e3 = mask >> (i + 3) & 1 ? e3 : 0.f;
    }
    add2(sum[0], sum[1], sum[0], sum[1], e0, e1);
    add2(sum[2], sum[3], sum[2], sum[3], e2, e3);
  }
}

#ifdef FA_DEBUG_BOUNDS
// Whether a page whose keys sequence b's new tokens see is one of another sequence's: the CTAs of both would read and
// write its weights, and one of the sums be lost.
__device__ __forceinline__ void check_not_shared(const Attn& p, int b, int page) {
  const int shift = p.c.page_shift;
  for (int x = 0; x < p.c.B; ++x) {
    const AccSeq other(p, x);
    if (x == b || other.w.steps == 0) continue;
    for (int i = 0; i << shift < other.w.hi; ++i)
      if (other.w.any(i << shift, 1 << shift) && __ldg(p.c.table + x * p.c.table_stride + i) == page)
        report_bounds(p.c.status, kSitePagedShared, page);
  }
}
#endif

// The pages of a unit's boxes, one for each lane (num_pages where there is nothing to read): one access to the table
// serves as many of a sequence's units as the lanes hold.
struct AccPages {
  int b = -1, from = 0, page = 0;
  // boxes of a unit, of 1 << shift keys each
  template <class Cursor>
  __device__ __forceinline__ int get(const Attn& p, const Cursor& c, int boxes, int shift) {
    const int lane = threadIdx.x % 32, units = 32 / boxes;
    if (c.b != b || c.j < from || c.j >= from + units) {
      b = c.b;
      from = c.j;
      const int j = c.j + lane / boxes, key = c.w.at(j) + (lane % boxes << shift);
      page = p.c.num_pages;
      // (the walk ends at the sequence's length, which the table holds)
      if (j < c.w.steps && c.w.any(key, 1 << shift)) {
        page = __ldg(p.c.table + c.b * p.c.table_stride + (key >> p.c.page_shift));
        if (page < 0 || page >= p.c.num_pages) {
          report_bounds(p.c.status, kSitePagedPage, page);
          page = p.c.num_pages;
        }
      }
    }
    return __shfl_sync(0xffffffffu, page, (c.j - from) * boxes + lane % boxes);
  }
};

template <int D, bool kFp8, int N>
__global__ void __launch_bounds__(AccCfg<D, kFp8, N>::kThreads, AccCfg<D, kFp8, N>::kCtas)
    fa_accumulate_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ Acc g) {
  using C = AccCfg<D, kFp8, N>;
  using Cursor = AccCursor<C::kChunk>;
  constexpr int kKWarp = C::kSumWarps, kQWarp = kKWarp + 1, kMmaWarp = kKWarp + 2, kColWarp = kKWarp + 3, kConvertWarp = kKWarp + 4;
  constexpr int W = N < 32 ? N : 32;    // columns taken at a time
  extern __shared__ __align__(1024) uint8_t smem[];
  const Attn& p = g.a;
  if (smem_u32(smem) & 1023u) {         // the swizzled tiles need it
    if (threadIdx.x == 0) report_bounds(p.c.status, kSiteSmemAlign, (long long)smem_u32(smem));
    return;
  }
  if constexpr (C::kChunk) cudaTriggerProgrammaticLaunchCompletion();   // the joining kernel may get ready
  AccShared& sh = *reinterpret_cast<AccShared*>(smem + C::kSharedOff);
  volatile uint32_t* abort_flag = &sh.abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int tokens = N / p.group;       // of a block of queries
  // keys come in boxes of a page, of half a page of 256
  const int page_size = 1 << p.c.page_shift, box_shift = min(p.c.page_shift, 7), boxes = kAccKeys >> box_shift;

  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(&sh.k_full[s], C::kConvert ? 128 : 1);
      mbar_init(&sh.k_empty[s], 1);
    }
    for (int s = 0; s < C::kQStages; ++s) {
      mbar_init(&sh.q_full[s], 1);
      mbar_init(&sh.q_empty[s], 1);
    }
    for (int s = 0; s < kColStages; ++s) {
      mbar_init(&sh.col_full[s], 32);
      mbar_init(&sh.col_empty[s], 8);    // four warps for each tile
    }
    for (int s = 0; s < C::kSideStages; ++s) {
      mbar_init(&sh.side_full[s], 32);  // the loading warp's lanes (pages), one of them with the expected bytes
      mbar_init(&sh.side_empty[s], C::kSumWarps);
    }
    for (int t = 0; t < 2; ++t)
      for (int s = 0; s < C::kBufs; ++s) {
        mbar_init(&sh.s_full[t][s], 1);
        mbar_init(&sh.s_empty[t][s], 4);
      }
    for (int t = 0; t < 2; ++t)
      for (int s = 0; s < 2; ++s) {
        mbar_init(&sh.half_full[t][s], 4);
        mbar_init(&sh.half_empty[t][s], 4);
      }
    mbar_init(&sh.code_full, 1);
    mbar_init(&sh.code_empty, 128);
    mbar_init(&sh.mma_done, 1);
    mbar_init(&sh.never, 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  if (tokens * p.group < N) {
    // rows of a block that no token fills: S = 0 there, and a log-sum-exp of infinity, so that full blocks need no mask
    for (int i = threadIdx.x; i < C::kQStages * C::kQBytes / 16; i += C::kThreads)
      *reinterpret_cast<uint4*>(smem + C::kQOff + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  long long count;
  const int parts = find_units<C::kThreads>(p, C::kChunk ? g.max_parts : 1, sh.scan, sh.first_b, sh.first, count,
                                            [&](long long all, int parts, long long& want) {
    if (C::kChunk) {
      want = blockIdx.x;
      return all * parts - want;     // (every gridDim.x-th from there on)
    }
    const long long share = (all + gridDim.x - 1) / gridDim.x;
    want = blockIdx.x * share;
    return min(share, all - want);
  });
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  // (a CTA without a unit walks none; all of them free their tensor memory below)
  Cursor cur(p, parts, sh.first_b, sh.first, count);

  if (warp == kKWarp) {
    // ------------------------------------------------------------ K tiles (or their codes), page by page
    const uint32_t base = smem_u32(smem);
    if (lane == 0) tma_prefetch_desc(&tmK);
    AccPages pages;
    int n = 0;
    for (; cur.valid(p); cur.next(p, parts), ++n) {
      const int s = n % C::kKStages, tiles = cur.tile(1) ? 2 : 1;
      const int page = pages.get(p, cur, boxes, box_shift);
#ifdef FA_DEBUG_BOUNDS
      if (lane < boxes && page < p.c.num_pages) check_not_shared(p, cur.b, page);
      __syncwarp();
#endif
      uint64_t* full = C::kConvert ? &sh.code_full : &sh.k_full[s];
      if (!__all_sync(0xffffffffu, C::kConvert ? mbar_wait(&sh.code_empty, (n & 1) ^ 1, abort_flag, p.c.status)
                                               : mbar_wait(&sh.k_empty[s], ((n / C::kKStages) & 1) ^ 1, abort_flag, p.c.status)))
        break;
      if (lane == 0) mbar_arrive_expect_tx(full, tiles * kAccTile * D * (kFp8 ? 1 : 2));
      __syncwarp();
      const int row = lane << box_shift, slot = (cur.key() + row) & (page_size - 1);
      if (lane < boxes && row < tiles * kAccTile) {
        if constexpr (C::kConvert) {
          tma_load_page(base + C::kCodeOff + row * D, &tmK, full, 0, slot, cur.h, page);
        } else {
          const uint32_t dst =
              base + C::kKOff + s * C::kPairBytes + (row / kAccTile) * C::kTileBytes + (row % kAccTile) * C::kAtomBytes;
#pragma unroll
          for (int a = 0; a < C::kAtoms; ++a)
            tma_load_page(dst + a * kAccTile * C::kAtomBytes, &tmK, full, a * C::kAtomElems, slot, cur.h, page);
        }
      }
    }
    if (*abort_flag) {
      // let copies still in flight land before the CTA's shared memory goes away
      volatile uint32_t ignore_abort = 0;
      if constexpr (C::kConvert) {
        if (n > 0) mbar_wait(&sh.code_full, (n - 1) & 1, &ignore_abort, p.c.status);
      } else {
        for (int i = max(0, n - C::kKStages); i < n; ++i)
          mbar_wait(&sh.k_full[i % C::kKStages], (i / C::kKStages) & 1, &ignore_abort, p.c.status);
      }
    }
  } else if (warp == kQWarp) {
    // ------------------------------------------------------------ blocks of queries
    if constexpr (C::kPieced) cudaGridDependencySynchronize();   // the pieces are there (in every CTA: what follows
                                                                 // in the stream waits for this launch only)
    if (elect_one()) {
      tma_prefetch_desc(&tmQ);
      int n = 0;
      bool ok = true;
      for (; ok && cur.valid(p); cur.next(p, parts)) {
        if (!C::kChunk && !cur.fresh) continue;
        int i, last;
        for (cur.blocks(p, parts, tokens, i, last); i < last; ++i, ++n) {
          const int s = n % C::kQStages;
          if (!(ok = mbar_wait(&sh.q_empty[s], ((n / C::kQStages) & 1) ^ 1, abort_flag, p.c.status))) break;
          mbar_arrive_expect_tx(&sh.q_full[s], tokens * p.group * C::kRowBytes * (C::kPieced ? kPieces : 1));
          uint8_t* dst = smem + C::kQOff + s * C::kQBytes;
          const int token = cur.s.q0 + i * tokens, head = cur.h * p.group;
          if constexpr (C::kPieced) {
            for (int x = 0; x < kPieces; ++x) tma_load_page(smem_u32(dst + x * C::kQTile), &tmQ, &sh.q_full[s], 0, head, token, x);
          } else {
            for (int a = 0; a < C::kAtoms; ++a)
              tma_load_3d(dst + a * N * C::kAtomBytes, &tmQ, &sh.q_full[s], a * C::kAtomElems, head, token);
          }
        }
      }
      if (*abort_flag) {
        volatile uint32_t ignore_abort = 0;
        for (int i = max(0, n - C::kQStages); i < n; ++i)
          mbar_wait(&sh.q_full[i % C::kQStages], (i / C::kQStages) & 1, &ignore_abort, p.c.status);
      }
    }
  } else if (warp == kColWarp) {
    // ------------------------------------------------------------ a unit's weights, scales and pages; its blocks' log-sum-exps
    constexpr int kPer = (N + 31) / 32, kAhead = C::kChunk ? 4 : 1;
    if constexpr (C::kPieced) cudaGridDependencySynchronize();
    int tr[kPer], off[kPer];               // a column's token within its block, its place behind the block's first row
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int r = e * 32 + lane;
      tr[e] = r < tokens * p.group ? r / p.group : INT_MAX;
      off[e] = r / p.group * p.Hq + r % p.group;
    }
    AccPages pages;
    int n = 0, nu = 0;
    bool ok = true;
    for (; ok && cur.valid(p); cur.next(p, parts)) {
      {
        const int x = nu % C::kSideStages, row = lane << box_shift;
        const int page = pages.get(p, cur, boxes, box_shift);
        const bool real = lane < boxes && page < p.c.num_pages;
        const int reals = __popc(__ballot_sync(0xffffffffu, real));
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.side_empty[x], ((nu / C::kSideStages) & 1) ^ 1, abort_flag, p.c.status));
        if (!ok) break;
        uint8_t* side = smem + C::kSideOff + x * C::kSideBytes;
        if (lane < 16) reinterpret_cast<int*>(side + C::kSideBytes - 64)[lane] = real ? page : -1;
        if (lane == 0)
          mbar_arrive_expect_tx(&sh.side_full[x], (reals << box_shift) * 4 * (kFp8 ? 2 : 1));
        else
          mbar_arrive(&sh.side_full[x]);
        __syncwarp();
        if (real) {
          const long long at = (long long)cur.h * page_size + ((cur.key() + row) & (page_size - 1));
          bulk_load(side + row * 4, g.weights + page * g.weight_stride + at, 4 << box_shift, &sh.side_full[x]);
          if constexpr (kFp8)
            bulk_load(side + (kAccKeys + row) * 4, p.c.k_scale + page * p.c.scale_stride + at, 4 << box_shift, &sh.side_full[x]);
        }
        ++nu;
      }
      if (!C::kChunk && !cur.fresh) continue;
      int i, last;
      for (cur.blocks(p, parts, tokens, i, last); ok && i < last; i += kAhead) {
        float neg[kAhead][kPer], factor[kAhead][kPer];
#pragma unroll
        for (int x = 0; x < kAhead; ++x)
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            neg[x][e] = -INFINITY;         // columns without a row weigh nothing, nor do rows that saw no key
            factor[x][e] = 0.f;
            const int t0 = (i + x) * tokens;
            if (i + x < last && tr[e] < cur.s.n - t0) {
              const long long row = (long long)(cur.s.q0 + t0) * p.Hq + cur.h * p.group + off[e];
              neg[x][e] = __ldg(g.lse + row);
              if constexpr (C::kPieced) factor[x][e] = __ldg(g.q_scale + row);
            }
          }
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
          if (i + x >= last) break;
          const int s = n % kColStages;
          ok = __all_sync(0xffffffffu, mbar_wait(&sh.col_empty[s], ((n / kColStages) & 1) ^ 1, abort_flag, p.c.status));
          if (!ok) break;
          float* col = reinterpret_cast<float*>(smem + C::kColOff + s * C::kColBytes);
#pragma unroll
          for (int e = 0; e < kPer; ++e)
            if (e * 32 + lane < N) {
              // -lse log2(e), the constant in two parts: its rounding would be the same for all
              const float l = neg[x][e];
              col[e * 32 + lane] = isinf(l) ? -INFINITY : -fmaf(l, kLog2e, l * kLog2eRest);
              if constexpr (C::kPieced) col[N + e * 32 + lane] = g.scale_log2 * factor[x][e];
            }
          mbar_arrive(&sh.col_full[s]);
          ++n;
        }
      }
    }
    if (*abort_flag) {
      volatile uint32_t ignore_abort = 0;
      for (int i = max(0, nu - C::kSideStages); i < nu; ++i)
        mbar_wait(&sh.side_full[i % C::kSideStages], (i / C::kSideStages) & 1, &ignore_abort, p.c.status);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    if (elect_one()) {
      const uint32_t sK = smem_u32(smem + C::kKOff), sQ = smem_u32(smem + C::kQOff);
      int nk = 0, nq = 0, ns[2] = {0, 0};
      bool ok = true;
#ifdef FA_TEST_HOOKS
      // failure-detection test: as in the few-rows kernel
      if (p.inject_stall) ok = mbar_wait(&sh.never, 0, abort_flag, p.c.status);
#endif
      for (; ok && cur.valid(p); cur.next(p, parts), ++nk) {
        const int ks = nk % C::kKStages, tiles = cur.tile(1) ? 2 : 1;
        if (!(ok = mbar_wait(&sh.k_full[ks], (nk / C::kKStages) & 1, abort_flag, p.c.status))) break;
        int i, last;
        for (cur.blocks(p, parts, tokens, i, last); ok && i < last; ++i) {
          const int qs = nq % C::kQStages;
          // few rows: a head's queries stay for all its units
          if ((C::kChunk || cur.fresh) && !(ok = mbar_wait(&sh.q_full[qs], (nq / C::kQStages) & 1, abort_flag, p.c.status))) break;
          for (int t = 0; t < tiles; ++t) {
            const int buf = ns[t] % C::kBufs;
            if (!(ok = mbar_wait(&sh.s_empty[t][buf], ((ns[t] / C::kBufs) & 1) ^ 1, abort_flag, p.c.status))) break;
            tc_fence_after();
            const uint32_t d = tmem + (t * C::kBufs + buf) * C::kBufCols;
            const uint32_t a0 = sK + ks * C::kPairBytes + t * C::kTileBytes, b0 = sQ + qs * C::kQBytes;
            if constexpr (C::kPieced) {
#pragma unroll
              for (int x = 0; x < (C::kWide ? 1 : kPieces); ++x)
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk) {
                  // one after the other: the smallest piece first, so that few steps cut a sum of full size (d = 128,
                  // products of one sign: S low by 0.18 2^-23 of it on average, the largest first 0.40)
                  const uint32_t a = a0 + kk * 32, b = b0 + (C::kWide ? 0 : kPieces - 1 - x) * C::kQTile + kk * 32;
                  if constexpr (C::kAtomBytes == 128)
                    mma_ss_f8(d, sdesc_sw128(a, 16, 1024), sdesc_sw128(b, 16, 1024), C::kIdesc, x + kk > 0);
                  else
                    mma_ss_f8(d, sdesc_sw64(a, 16, 512), sdesc_sw64(b, 16, 512), C::kIdesc, x + kk > 0);
                }
            } else {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(d, sdesc_sw128(a0 + (kk / 4) * kAccTile * 128 + (kk % 4) * 32, 16, 1024),
                       sdesc_sw128(b0 + (kk / 4) * N * 128 + (kk % 4) * 32, 16, 1024), C::kIdesc, kk > 0);
            }
            tc_commit(&sh.s_full[t][buf]);
            ++ns[t];
          }
          if (ok && (C::kChunk || cur.last())) {
            tc_commit(&sh.q_empty[qs]);
            ++nq;
          }
        }
        if (ok) tc_commit(&sh.k_empty[ks]);
      }
      tc_commit(&sh.mma_done);
      {
        // products still in flight must finish before tensor memory is released, even after an abort
        volatile uint32_t ignore_abort = 0;
        mbar_wait(&sh.mma_done, 0, &ignore_abort, p.c.status);
      }
    }
  } else if (warp < C::kSumWarps) {
    // ------------------------------------------------------------ exponentials and sums: a thread (chunks: two) per key
    const int t = warp / (4 * C::kHalves), half = warp / 4 % C::kHalves;
    const int row = t * kAccTile + (warp % 4) * 32 + lane;   // the thread's key within a unit
    const uint32_t tS = tmem + t * C::kBufs * C::kBufCols + ((uint32_t)((warp % 4) * 32) << 16);
    int nq = 0, ns = 0, nu = 0;
    long long number = blockIdx.x;                   // chunks: of the part in the launch
    bool ok = true;
    auto wait = [&](uint64_t* bar, int n, int stages) {
      return __all_sync(0xffffffffu, mbar_wait(bar, (n / stages) & 1, abort_flag, p.c.status));
    };
    auto give = [&](int buf) {                       // a buffer of S has been read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.s_empty[t][buf]);
    };
    auto columns = [&](int n) {
      return reinterpret_cast<const float*>(smem + C::kColOff + n % kColStages * C::kColBytes);
    };
    for (; ok && cur.valid(p); cur.next(p, parts), ++nu, number += gridDim.x) {
      const int x = nu % C::kSideStages;
      const uint8_t* side = smem + C::kSideOff + x * C::kSideBytes;
      if (!(ok = wait(&sh.side_full[x], nu, C::kSideStages))) break;
      const int page = reinterpret_cast<const int*>(side + C::kSideBytes - 64)[row >> box_shift];
      const float old = reinterpret_cast<const float*>(side)[row];
      const float key_scale = kFp8 ? reinterpret_cast<const float*>(side)[kAccKeys + row] : 1.f;
      const float f = C::kPieced ? key_scale : key_scale * g.scale_log2;   // (a power of two: exact)
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.side_empty[x]);
      const bool active = cur.tile(t);
      const int key = cur.key() + row, ahead = key - cur.s.pos0;   // the first token that sees the key, but for 0
      float total = 0.f;
      int i, last;
      cur.blocks(p, parts, tokens, i, last);
      // chunks: the blocks [i_all, last_all) of which every row sees every key of the warp
      int i_all = INT_MAX, last_all = 0;
      if (C::kChunk && active) {
        const int lo = ahead - lane, hi = lo + 31;   // (of the warp's first key and of its last)
        i_all = (max(hi, 0) + tokens - 1) / tokens;
        last_all = cur.s.n / tokens;
        if (p.window && key - lane + 31 >= p.sinks)
          last_all = (int)max(min((long long)last_all, ((long long)lo + p.window) / tokens), 0ll);
        last_all = min(last_all, last);
      }
      while (i < last) {
        if (C::kChunk && i >= i_all && i < last_all) {
          for (; i < last_all; ++i, ++nq, ++ns) {
            if (C::kHalves == 2 && ns % 2 != half) continue;   // the other set's
            const int buf = ns % C::kBufs;
            const float* col = columns(nq);
            if (!(ok = wait(&sh.s_full[t][buf], ns, C::kBufs))) break;
            tc_fence_after();
            uint32_t r[32];
            tmem_ld32(tS + buf * C::kBufCols, r);
            if (!(ok = wait(&sh.col_full[nq % kColStages], nq, kColStages))) break;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < N / 32; ++c) {
              tmem_ld_wait();
              reg_fence(r);
              if (c + 1 == N / 32) give(buf);
              acc_columns<32, false, false>(r, col + c * 32, nullptr, f, 0, sum);
              if (c + 1 < N / 32) tmem_ld32(tS + buf * C::kBufCols + (c + 1) * 32, r);
            }
            total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.col_empty[nq % kColStages]);
          }
          tmem_ld_wait();   // (where a wait gave up)
          if (!ok) break;
          continue;
        }
        if (C::kHalves == 2 && (active ? ns % 2 : 0) != half) {   // (a tile without keys: the first set's)
          ns += active;
          ++nq;
          ++i;
          continue;
        }
        if ((C::kChunk || cur.fresh) && !(ok = wait(&sh.col_full[nq % kColStages], nq, kColStages))) break;
        if (active) {
          const int buf = ns % C::kBufs;
          if (!(ok = wait(&sh.s_full[t][buf], ns, C::kBufs))) break;
          tc_fence_after();
          // the rows that see the key: its own token's on, up to the last one whose window holds it
          const int t0 = i * tokens, here = min(cur.s.n - t0, tokens);
          const int lo = min(max(ahead - t0, 0), here) * p.group;
          int end = here;
          if (p.window && key >= p.sinks) end = (int)min((long long)here, max((long long)ahead + p.window - t0, 0ll));
          const int hi = end * p.group;
          const float* col = columns(nq);
          const uint32_t at = tS + buf * C::kBufCols;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c0 = 0; c0 < N; c0 += W) {
            if (__all_sync(0xffffffffu, hi <= c0 || lo >= c0 + W)) continue;
            uint32_t r[W];
            auto get = [&](uint32_t (&to)[W], int c) {
              if constexpr (W == 16)
                tmem_ld16(at + c, to);
              else
                tmem_ld32(at + c, to);
            };
            get(r, c0);
            if constexpr (C::kWide) {
              uint32_t r1[W], r2[W];
              get(r1, N + c0);
              get(r2, 2 * N + c0);
              tmem_ld_wait();
              reg_fence(r);
              reg_fence(r1);
              reg_fence(r2);
#pragma unroll
              for (int e = 0; e < W; ++e)   // the smaller ones first
                r[e] = __float_as_uint(__uint_as_float(r[e]) + (__uint_as_float(r1[e]) + __uint_as_float(r2[e])));
            } else {
              tmem_ld_wait();
              reg_fence(r);
            }
            acc_columns<W, C::kPieced, true>(r, col + c0, col + N + c0, f, low_bits(hi - c0) & ~low_bits(lo - c0), sum);
          }
          give(buf);
          ++ns;
          total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        } else {
          __syncwarp();
        }
        if (C::kChunk || cur.last()) {
          if (lane == 0) mbar_arrive(&sh.col_empty[nq % kColStages]);
          ++nq;
        }
        ++i;
      }
      if constexpr (C::kHalves == 2) {
        // the second set's sums go to the first
        if (!ok) break;
        const int y = nu % 2;
        float* sums = reinterpret_cast<float*>(smem + C::kHalfOff) + y * kAccKeys;
        if (half == 1) {
          if (!(ok = wait(&sh.half_empty[t][y], nu + 2, 2))) break;   // (free at first)
          sums[row] = total;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.half_full[t][y]);
          continue;
        }
        if (!(ok = wait(&sh.half_full[t][y], nu, 2))) break;
        total += sums[row];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.half_empty[t][y]);
      }
      if (ok && cur.w.seen(key)) {
        if (parts > 1)
          g.part[number * kAccKeys + row] = total;
        else if (page >= 0)
          g.weights[page * g.weight_stride + ((long long)cur.h << p.c.page_shift) + (key & ((1 << p.c.page_shift) - 1))] =
              (ahead >= 0 ? 0.f : old) + total;
      }
    }
  }

  if constexpr (C::kConvert) {
    if (warp >= kConvertWarp) {
      // ---------------------------------------------------------- codes -> BF16 operand tiles
      // D / 16 neighbouring threads take one key's row, 16 codes each: two 16-byte chunks of a 64-column block,
      // swizzled; the second block's threads take theirs in the other order, so that a row's threads meet
      // different banks.  The scales are left to the sums.
      constexpr int kPer = D / 16, kRowStep = 128 / kPer, kRows = kAccTile / kRowStep;
      const int r0 = (threadIdx.x - 32 * kConvertWarp) / kPer, x = threadIdx.x % kPer, flip = x / 4;
      const uint32_t c0 = (uint32_t)(flip * kAccTile * 128 + r0 * 128 + ((((x % 4) * 2 + flip) ^ (r0 & 7)) << 4));
      const uint32_t c1 = (uint32_t)(flip * kAccTile * 128 + r0 * 128 + ((((x % 4) * 2 + 1 - flip) ^ (r0 & 7)) << 4));
      static_assert(kRowStep % 8 == 0, "a thread's rows share one swizzle phase");
      bool ok = true;
      for (int n = 0; ok && cur.valid(p); cur.next(p, parts), ++n) {
        const int s = n % C::kKStages, tiles = cur.tile(1) ? 2 : 1;
        if (!(ok = mbar_wait(&sh.code_full, n & 1, abort_flag, p.c.status))) break;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
          uint4 codes[kRows];
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            codes[i] = *reinterpret_cast<const uint4*>(smem + C::kCodeOff + (t * kAccTile + r0 + i * kRowStep) * D + x * 16);
          if (t + 1 == tiles) mbar_arrive(&sh.code_empty);
          if (t == 0 && !(ok = mbar_wait(&sh.k_empty[s], ((n / C::kKStages) & 1) ^ 1, abort_flag, p.c.status))) break;
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const uint4 u = codes[i];
            const uint32_t w[4] = {flip ? u.z : u.x, flip ? u.w : u.y, flip ? u.x : u.z, flip ? u.y : u.w};
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 f = e4m3x2_to_float2(w[e / 2] >> (16 * (e & 1)));
              y[e] = pack_bf16x2(f.x, f.y);   // exact
            }
            const uint32_t tile = smem_u32(smem) + C::kKOff + s * C::kPairBytes + t * C::kTileBytes + i * kRowStep * 128;
            sts128(tile + c0, make_uint4(y[0], y[1], y[2], y[3]));
            sts128(tile + c1, make_uint4(y[4], y[5], y[6], y[7]));
          }
        }
        if (!ok) break;
        fence_proxy_async_smem();
        mbar_arrive(&sh.k_full[s]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Chunks whose units were cut: a unit's weights from its parts' sums, in their order.  A CTA has a unit, a thread a
// key.  A programmatic launch: its CTAs find their units beside the first kernel, which lets them start, and wait for its end
// (300 tokens over 1000 E4M3 keys 17.5 -> 17.2 us).
__global__ void __launch_bounds__(kAccKeys) fa_accumulate_join(const __grid_constant__ Acc g) {
  __shared__ long long scan[kAccKeys / 32], first;
  __shared__ int first_b;
  const Attn& p = g.a;
  long long count;
  const int parts = find_units<kAccKeys>(p, g.max_parts, scan, first_b, first, count, [&](long long all, int parts, long long& want) {
    want = (long long)blockIdx.x * parts;
    return parts > 1 && blockIdx.x < all ? 1 : 0;
  });
  cudaGridDependencySynchronize();   // before any exit: what follows must find the first kernel complete
  if (first_b < 0) return;
  const AccCursor<true> c(p, parts, first_b, first, 1);
  const int key = c.key() + (int)threadIdx.x;
  if (!c.w.seen(key)) return;
  const int page = __ldg(p.c.table + c.b * p.c.table_stride + (key >> p.c.page_shift));
  if (page < 0 || page >= p.c.num_pages) return;   // (recorded by the first kernel)
  float sum = 0.f;
  for (int i = 0; i < parts; ++i) sum += g.part[((long long)blockIdx.x * parts + i) * kAccKeys + threadIdx.x];
  float* w = g.weights + page * g.weight_stride + ((long long)c.h << p.c.page_shift) + (key & ((1 << p.c.page_shift) - 1));
  *w = (key >= c.s.pos0 ? 0.f : *w) + sum;
}

// The three E5M2 vectors of a query vector x: x = 2^e (p0 + p1 + p2), e such that the largest entry is in
// [2^14, 2^15).  Each takes what is left, rounded to nearest.  D / 8 lanes have a vector.
template <int D>
__global__ void __launch_bounds__(256) split_queries_kernel(const __nv_bfloat16* __restrict__ q, long long q_stride, int T,
                                                            int Hq, uint8_t* __restrict__ pieces, float* __restrict__ scale) {
  constexpr int kLanes = D / 8, kVecs = 256 / kLanes;
  cudaTriggerProgrammaticLaunchCompletion();   // the kernel that reads the pieces may get ready
  const long long vec = (long long)blockIdx.x * kVecs + threadIdx.x / kLanes, all = (long long)T * Hq;
  const int j = threadIdx.x % kLanes;
  const long long v = vec < all ? vec : all - 1;
  const long long token = v / Hq;
  const uint4 u = *reinterpret_cast<const uint4*>(q + token * q_stride + (v - token * Hq) * D + j * 8);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float x[8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    amax = max(amax, max(__float_as_uint(x[2 * i]) & 0x7FFFFFFFu, __float_as_uint(x[2 * i + 1]) & 0x7FFFFFFFu));
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  // 2^e and 2^-e stay normal: vectors under 2^-112 keep a smaller largest entry
  const int e = amax == 0 ? 0 : max((int)(amax >> 23) - 127 - 14, -126);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
  const bool bad = amax >= 0x7F800000u;
  uint2 out[kPieces];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= inv;
#pragma unroll
  for (int n = 0; n < kPieces; ++n) {
    uint32_t codes[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      asm("{\n .reg .b16 c;\n cvt.rn.satfinite.e5m2x2.f32 c, %2, %1;\n mov.b32 %0, {c, 0};\n}"
          : "=r"(codes[i])
          : "f"(x[2 * i]), "f"(x[2 * i + 1]));
      // an E5M2 code is the upper byte of the FP16 number
      uint32_t half = (codes[i] & 0xFFu) << 8 | (codes[i] & 0xFF00u) << 16;
      float lo, hi;
      asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
          : "=f"(lo), "=f"(hi)
          : "r"(half));
      x[2 * i] -= lo;
      x[2 * i + 1] -= hi;
    }
    out[n] = make_uint2(codes[0] | codes[1] << 16, codes[2] | codes[3] << 16);
    if (bad) out[n] = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);   // NaN or Inf in the vector: NaN
  }
  if (vec >= all) return;
#pragma unroll
  for (int n = 0; n < kPieces; ++n) *reinterpret_cast<uint2*>(pieces + (n * all + vec) * D + j * 8) = out[n];
  if (j == 0) scale[vec] = __uint_as_float((uint32_t)(e + 127) << 23);
}

// A launch that may start before the one before it in the stream has ended.
template <typename... Args, typename... Given>
static int launch_early(const char* what, void (*kern)(Args...), int grid, int threads, int smem, cudaStream_t s,
                        const Given&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return check_cuda(cudaLaunchKernelEx(&cfg, kern, args...), what);
}

template <int D, bool kFp8, int N>
static int launch_acc(const CUtensorMap& tq, const CUtensorMap& tk, const Acc& g, cudaStream_t s) {
  using C = AccCfg<D, kFp8, N>;
  constexpr int smem = acc_smem<D, kFp8, N>();
  auto kern = fa_accumulate_kernel<D, kFp8, N>;
  static std::atomic<uint64_t> prepared{0};
  int rc = prepare_kernel(reinterpret_cast<const void*>(kern), smem, C::kThreads, 0, "accumulate kernel", &prepared);
  if (rc) return rc;
  const int grid = C::kCtas * sm_count();
  if (C::kPieced) return launch_early("launch fa_accumulate_kernel", kern, grid, C::kThreads, smem, s, tq, tk, g);
  kern<<<grid, C::kThreads, smem, s>>>(tq, tk, g);
  if ((rc = check_cuda(cudaGetLastError(), "launch fa_accumulate_kernel"))) return rc;
  if (!C::kChunk || g.max_parts == 1) return FA_OK;
  // (units are cut in two at least where there are half as many as parts at most)
  return launch_early("launch fa_accumulate_join", fa_accumulate_join, kMostParts / 2, kAccKeys, 0, s, g);
}

template <int D, bool kFp8>
static int launch_columns(int columns, const CUtensorMap& tq, const CUtensorMap& tk, const Acc& g, cudaStream_t s) {
  if (columns == 16) return launch_acc<D, kFp8, 16>(tq, tk, g, s);
  if (columns == 32) return launch_acc<D, kFp8, 32>(tq, tk, g, s);
  if (columns == 64) return launch_acc<D, kFp8, 64>(tq, tk, g, s);
  return launch_acc<D, kFp8, 128>(tq, tk, g, s);
}

// Columns of S, which hold all of a sequence's rows for a kv head, or a block of them.
static int columns_of(int max_q, int group) {
  const long long rows = (long long)max_q * group;
  return rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 64 ? 64 : 128));
}

// Chunks: the most parts that a unit may be cut into.
static int parts_of(int max_q, int group) {
  const int tokens = 128 / group;
  return (int)std::max(1ll, std::min(16ll, ((long long)max_q + tokens - 1) / tokens / kPartBlocks));
}

static int check_accumulate(int T, int max_q, int Hq, int Hkv, int d) {
  if (T < 0 || max_q < 0) return set_error(FA_ERR_INVALID_ARG, "T, max_q must be >= 0 (got %d, %d)", T, max_q);
  if (Hkv < 1 || Hq < 1) return set_error(FA_ERR_INVALID_ARG, "Hq, Hkv must be >= 1 (got %d, %d)", Hq, Hkv);
  if (Hq % Hkv) return set_error(FA_ERR_INVALID_ARG, "Hq = %d is not a multiple of Hkv = %d", Hq, Hkv);
  if (Hq / Hkv > 128) return set_error(FA_ERR_UNSUPPORTED, "more than 128 query heads for a kv head (%d)", Hq / Hkv);
  if (d != 64 && d != 128) return set_error(FA_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
  if ((long long)T * Hq >= (1ll << 31)) return set_error(FA_ERR_INVALID_ARG, "T*Hq must be < 2^31");
  return FA_OK;
}

// Few rows over E4M3: the queries' pieces, then their factors.  Chunks: the parts' sums.
static size_t pieces_bytes(int T, int Hq, int d) { return round_up((size_t)kPieces * T * Hq * d, 256); }
static size_t accumulate_bytes(int T, int max_q, int Hq, int Hkv, int d, int dtype) {
  const int group = Hq / Hkv;
  if (columns_of(max_q, group) == 128) return parts_of(max_q, group) > 1 ? (size_t)kMostParts * kAccKeys * 4 : 0;
  return dtype == FA_KV_E4M3 ? pieces_bytes(T, Hq, d) + round_up((size_t)T * Hq * 4, 256) : 0;
}

}  // namespace paged
}  // namespace fa

extern "C" size_t fa_kv_accumulate_workspace_size(int T, int max_q, int Hq, int Hkv, int d, int dtype) {
  using namespace fa;
  clear_error();
  if (paged::check_accumulate(T, max_q, Hq, Hkv, d) || T == 0) return 0;
  return paged::accumulate_bytes(T, max_q, Hq, Hkv, d, dtype);
}

extern "C" int fa_kv_accumulate(const fa_paged_kv* kv, float* weights, int64_t weight_stride, const void* q, int64_t q_stride,
                                const float* lse, const int32_t* q_indptr, int T, int max_q, int Hq, int window, int sinks,
                                float scale, void* workspace, size_t workspace_bytes, void* stream) {
  fa::NvtxRange nvtx_range("fa_kv_accumulate");
  using namespace fa;
  clear_error();
  paged::Acc g{};
  paged::Attn& p = g.a;
  int rc;
  if ((rc = paged::check_cache(kv, &p.c)) || (rc = paged::check_accumulate(T, max_q, Hq, kv->Hkv, kv->d))) return rc;
  if ((rc = paged::check_weights(kv, weights, weight_stride))) return rc;
  if ((rc = check_ptr(q, "q")) || (rc = paged::check_indptr(q_indptr, "q_indptr"))) return rc;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3)) return set_error(FA_ERR_INVALID_ARG, "lse must be a 4-byte aligned device pointer");
  if (q_stride < (int64_t)Hq * kv->d || q_stride % 8)
    return set_error(FA_ERR_INVALID_ARG, "q_stride %lld must be a multiple of 8 and at least Hq*d = %d", (long long)q_stride, Hq * kv->d);
  if (!(scale > 0.f) || !isfinite(scale)) return set_error(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (window < 0 || sinks < 0) return set_error(FA_ERR_INVALID_ARG, "window and sinks must be >= 0 (got %d, %d)", window, sinks);
  if (!window && sinks) return set_error(FA_ERR_INVALID_ARG, "sinks need a window");
  const bool fp8 = kv->dtype == FA_KV_E4M3;
  const int max_kv = kv->max_pages * kv->page_size;
  if (kv->B > (1 << 30)) return set_error(FA_ERR_INVALID_ARG, "B must be <= 2^30 (got %d)", kv->B);
  // a sequence's units are counted in 32 bits
  if ((long long)kv->Hkv * (max_kv / paged::kAccKeys + 1) >= (1ll << 31) / 16)
    return set_error(FA_ERR_INVALID_ARG, "Hkv * max_pages * page_size must be < 2^35");
  if (T == 0 || max_q == 0) return FA_OK;
  const size_t need = paged::accumulate_bytes(T, max_q, Hq, kv->Hkv, kv->d, kv->dtype);
  if (need) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
      return set_error(FA_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
    if (workspace_bytes < need)
      return set_error(FA_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed", workspace_bytes, need);
  }
  p.c.status = device_status_word();
  if (!p.c.status) return set_error(FA_ERR_CUDA, "could not allocate the device status record");
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.q_indptr = q_indptr;
  p.T = T;
  p.Hq = Hq;
  p.group = Hq / kv->Hkv;
  const int columns = paged::columns_of(max_q, p.group);
  p.max_rows = (int)((long long)max_q * p.group < INT32_MAX ? max_q * p.group : INT32_MAX);
  p.window = window >= max_kv ? 0 : window;
  p.sinks = std::min(sinks, max_kv);
  // The tensor core cuts a sum to FP32 after every 16 products instead of rounding it: half a unit of the last place
  // each time, 0.36 2^-23 of the sum so far on average, which grows evenly.  (Weights of 2048 tokens over 34k keys were low
  // by 7.7e-7 on average.)  The scale is raised by that for BF16 keys, so that a weight is what its formula says of the
  // log-sum-exp that it is given: 1024 tokens over 16k keys, d = 128: 1.1e-7 off, without 5.5e-7.  (The attention call cuts its
  // sums alike, and its log-sum-exps are 8e-7 low of values near 10: rows sum to 1 + 8e-7 for it, without the raise
  // 1 + 2e-7.)  Of E4M3 codes' products, 12 bits wide, little is cut: 0 to 0.5 2^-23, and no raise.
  const double cut = fp8 ? 0 : (kv->d / 16 + 1) / 2. * 0.36 * 0x1p-23;
  g.scale_log2 = (float)(scale * 1.4426950408889634 * (1 + cut));
#ifdef FA_TEST_HOOKS
  const char* inject = getenv("FA_TEST_INJECT_STALL");
  p.inject_stall = (inject && inject[0] == '1') ? 1 : 0;
#endif
  g.lse = lse;
  g.weights = weights;
  g.weight_stride = weight_stride;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int d = kv->d, box = kv->page_size < paged::kAccTile ? kv->page_size : paged::kAccTile;
  const bool chunk = columns == 128;
  g.max_parts = chunk ? paged::parts_of(max_q, p.group) : 1;
  g.part = static_cast<float*>(workspace);
  CUtensorMap tq, tk;
  if ((rc = make_tmap_pages(&tk, kv->k, fp8, d, kv->page_size, kv->Hkv, kv->num_pages, kv->page_stride, box, fp8 && chunk)))
    return rc;
  if (fp8 && !chunk) {
    uint8_t* pieces = static_cast<uint8_t*>(workspace);
    float* factors = reinterpret_cast<float*>(pieces + paged::pieces_bytes(T, Hq, d));
    g.q_scale = factors;
    const int vecs = 256 / (d / 8);
    const unsigned grid = (unsigned)(((long long)T * Hq + vecs - 1) / vecs);
    if (d == 64)
      paged::split_queries_kernel<64><<<grid, 256, 0, s>>>(p.q, q_stride, T, Hq, pieces, factors);
    else
      paged::split_queries_kernel<128><<<grid, 256, 0, s>>>(p.q, q_stride, T, Hq, pieces, factors);
    if ((rc = check_cuda(cudaGetLastError(), "launch split_queries_kernel"))) return rc;
    rc = make_tmap_pieces(&tq, pieces, T, Hq, d, paged::kPieces, p.group, columns / p.group);
  } else {
    rc = make_tmap_rows(&tq, q, T, Hq, d, q_stride, p.group, columns / p.group);
  }
  if (rc) return rc;
  if (fp8)
    return d == 64 ? paged::launch_columns<64, true>(columns, tq, tk, g, s) : paged::launch_columns<128, true>(columns, tq, tk, g, s);
  return d == 64 ? paged::launch_columns<64, false>(columns, tq, tk, g, s) : paged::launch_columns<128, false>(columns, tq, tk, g, s);
}
