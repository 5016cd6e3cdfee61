// Accumulated attention weights of cached keys (fa_kv_accumulate): for each sequence, kv head and key j
//   weight[j] = (j is a new token's ? 0 : weight[j]) + sum over new tokens i and heads h of the group,
//               where i sees j, of exp(scale q_ih . k_j - lse_ih).
//
// One pass over K; the log-sum-exps are the attention call's, so nothing has to be known of other keys.
// S^T = K Q^T on the tensor core: the keys are the 128 rows of the instruction, a row of tensor memory and a thread
// each, so that a key's sum needs no exchange between threads, and a single token's few query heads are the
// narrow side (16, 32 or 64 columns; 128 for chunks).  One kernel serves both:
//   * a unit is 256 keys (two tiles) of one sequence and kv head; a persistent CTA takes a share of the
//     units and streams, for each, the query blocks that see its keys.  A key belongs to one CTA: no atomics,
//     the same bits in every call.
//   * few rows (decoding): the bytes of K bound it; a ring of K tiles is kept full.
//   * chunks: one exponential per pair and head, 32 a clock and SM, against 512 clocks of tensor work for
//     256 x 128 x 128: the exponentials bound it.
// E4M3 caches: the codes are the operand as they are (kind::f8f6f4).  A query vector goes into three E5M2 vectors
// that add up to it: BF16 has 8 significant bits, E5M2 3, and its exponents reach 2^-31 of the largest
// entry, so the sum is exact down to entries of 2^-24 of it.  The key's scale multiplies S in FP32.
#include <stdlib.h>

#include <algorithm>

#include "paged_attn.cuh"

namespace fa {
namespace paged {

constexpr int kAccThreads = 384;
constexpr int kAccKeys = 256;        // of a unit
constexpr int kAccTile = 128;        // keys of a tile
constexpr int kPieces = 3;           // E5M2 vectors of a query vector

struct Acc {
  Attn a;                  // queries, cache, lengths (o and lse are not used)
  const float* lse;        // [T, Hq]
  float* weights;          // [pages][Hkv][page_size]
  long long weight_stride;
  const float* q_scale;    // E4M3: [T, Hq], what the pieces are to be multiplied by
};

template <int D, bool kFp8, int N>
struct AccCfg {
  static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
  static constexpr int kAtomBytes = kRowBytes < 128 ? kRowBytes : 128;   // swizzle atom row
  static constexpr int kAtoms = kRowBytes / kAtomBytes, kAtomElems = D / kAtoms;
  static constexpr int kTileBytes = kAccTile * kRowBytes, kPairBytes = 2 * kTileBytes;
  static constexpr int kQTile = N * kRowBytes, kQBytes = (kFp8 ? kPieces : 1) * kQTile;
  static constexpr int kQStages = N == 128 ? 2 : 3;
  static constexpr int kRoom = 220 * 1024 - kQStages * kQBytes;
  static constexpr int kKStages = kRoom / kPairBytes < 6 ? kRoom / kPairBytes : 6;
  static constexpr int kBufs = N == 128 ? 2 : 4;                 // S buffers of a tile
  static constexpr int kTmemCols = 2 * kBufs * N;
  static constexpr int kQOff = kKStages * kPairBytes;
  static constexpr int kColOff = kQOff + kQStages * kQBytes;     // per stage: -lse log2e, factor
  static constexpr int kSharedOff = kColOff + kQStages * 2 * N * 4;
  static constexpr uint32_t kIdesc = kFp8 ? idesc_e4m3(128, N, false, false) | (1u << 10)   // B: E5M2
                                          : idesc_bf16(128, N, false, false);
  static_assert(kKStages >= 2 && kTmemCols <= 512 && kTmemCols >= 32, "shared or tensor memory");
};

constexpr int kMaxKStages = 6, kMaxQStages = 3, kMaxBufs = 4;

struct AccShared {
  uint64_t k_full[kMaxKStages], k_empty[kMaxKStages], q_full[kMaxQStages], q_empty[kMaxQStages];
  uint64_t s_full[2][kMaxBufs], s_empty[2][kMaxBufs];
  uint64_t mma_done;
  uint64_t never;                  // test builds only: a barrier nothing arrives on
  uint32_t tmem_base, abort_flag;
  long long scan[kAccThreads / 32];
  int first_b, first_unit;         // this CTA's first unit; first_b = -1: none
  long long first_cost;            // what lies before it
};

template <int D, bool kFp8, int N>
constexpr int acc_smem() {
  return AccCfg<D, kFp8, N>::kSharedOff + (int)sizeof(AccShared);
}
static_assert(acc_smem<128, false, 128>() <= 227 * 1024 && acc_smem<128, true, 128>() <= 227 * 1024 &&
                  acc_smem<128, false, 64>() <= 227 * 1024 && acc_smem<128, true, 64>() <= 227 * 1024 &&
                  acc_smem<128, false, 16>() <= 227 * 1024 && acc_smem<128, true, 16>() <= 227 * 1024,
              "shared-memory layout exceeds 227 KB");

// A sequence's units: (kv head, block of its walk), the block fastest.  A unit costs kUnitCost for its keys
// and one for each block of queries of the sequence.
constexpr int kUnitCost = 2;

template <int N>
struct AccSeq {
  Seq s;
  KeyWalk<kAccKeys> w;
  int blocks;              // of queries, `tokens` tokens each
  __device__ __forceinline__ AccSeq(const Attn& p, int b) : s(load_seq(p, b)), w(p, s.pos0, s.kv - 1) {
    const int tokens = N / p.group;
    blocks = (s.n + tokens - 1) / tokens;
    if (s.n == 0 || w.hi == 0) w.steps = 0;
  }
  __device__ __forceinline__ int cost() const { return kUnitCost + blocks; }
  __device__ __forceinline__ long long total(const Attn& p) const { return (long long)w.steps * p.c.Hkv * cost(); }
};

// The units of a CTA's share, in order.  Every role walks them with a copy of its own.
template <int N>
struct AccCursor {
  int b, h, j;             // sequence (B: no unit is left), kv head, step of the walk
  long long left;          // cost until the end of the share
  Seq s;
  KeyWalk<kAccKeys> w;
  int cost;
  __device__ __forceinline__ void take(const AccSeq<N>& x) {
    s = x.s;
    w = x.w;
    cost = x.cost();
  }
  __device__ __forceinline__ AccCursor(const Attn& p, int first_b, int first_unit, long long share)
      : b(first_b), left(share), s{}, w(p, 0, -1), cost(0) {
    const AccSeq<N> x(p, b);
    take(x);
    h = first_unit / max(w.steps, 1);
    j = first_unit - h * max(w.steps, 1);
    if (h >= p.c.Hkv) next_sequence(p);
    if (left <= 0) b = p.c.B;
  }
  __device__ __forceinline__ void next_sequence(const Attn& p) {
    h = j = 0;
    for (++b; b < p.c.B; ++b) {
      const AccSeq<N> x(p, b);
      if (x.w.steps == 0) continue;
      take(x);
      return;
    }
  }
  __device__ __forceinline__ bool valid(const Attn& p) const { return b < p.c.B; }
  __device__ __forceinline__ void next(const Attn& p) {
    left -= cost;
    if (left <= 0) {
      b = p.c.B;
      return;
    }
    if (++j == w.steps) {
      j = 0;
      if (++h == p.c.Hkv) next_sequence(p);
    }
  }
  __device__ __forceinline__ int key() const { return w.at(j); }
  // the blocks of queries that see a key of the unit: [first, last)
  __device__ __forceinline__ int first_block(int tokens) const { return max(key() - s.pos0, 0) / tokens; }
  __device__ __forceinline__ int last_block(const Attn& p, int tokens) const {
    const int all = (s.n + tokens - 1) / tokens;
    if (!p.window || key() < p.sinks) return all;
    const long long t = (long long)key() + kAccKeys - 1 + p.window - 1 - s.pos0;   // the last token that sees one
    return t < 0 ? 0 : (int)min((long long)all, t / tokens + 1);
  }
  // whether tile t of the unit has keys
  __device__ __forceinline__ bool tile(int t) const { return key() + t * kAccTile < w.hi; }
};

// A thread's key of a unit: where its weight lies, what was there.
struct AccKey {
  bool mine, fresh;        // a new token sees it; it is a new token's
  int page;
  long long at;            // slot within the page's head
  float old, scale;
};

// sum += of the columns c0 .. c0 + W - 1 of S: exp2(S f - lse log2e), of those in `mask` alone where kMasked.
template <int W, bool kFp8, bool kMasked>
__device__ __forceinline__ void acc_columns(const uint32_t (&r)[W], const float* neg_lse, const float* factor, float scale,
                                            uint32_t mask, float (&sum)[4]) {
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const float4 l = *reinterpret_cast<const float4*>(neg_lse + i);
    float s0 = __uint_as_float(r[i]), s1 = __uint_as_float(r[i + 1]), s2 = __uint_as_float(r[i + 2]), s3 = __uint_as_float(r[i + 3]);
    if constexpr (kFp8) {
      const float4 f = *reinterpret_cast<const float4*>(factor + i);
      mul2(s0, s1, s0, s1, scale, scale);
      mul2(s2, s3, s2, s3, scale, scale);
      fma2(s0, s1, s0, s1, f.x, f.y, l.x, l.y);
      fma2(s2, s3, s2, s3, f.z, f.w, l.z, l.w);
    } else {
      fma2(s0, s1, s0, s1, scale, scale, l.x, l.y);
      fma2(s2, s3, s2, s3, scale, scale, l.z, l.w);
    }
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

template <int D, bool kFp8, int N>
__global__ void __launch_bounds__(kAccThreads, 1)
    fa_accumulate_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ Acc g) {
  using C = AccCfg<D, kFp8, N>;
  constexpr int kKWarp = 8, kQWarp = 9, kMmaWarp = 10;
  constexpr int W = N < 32 ? N : 32;    // columns taken at a time
  extern __shared__ __align__(1024) uint8_t smem[];
  const Attn& p = g.a;
  if (smem_u32(smem) & 1023u) {         // the swizzled tiles need it
    if (threadIdx.x == 0) report_bounds(p.c.status, kSiteSmemAlign, (long long)smem_u32(smem));
    return;
  }
  AccShared& sh = *reinterpret_cast<AccShared*>(smem + C::kSharedOff);
  volatile uint32_t* abort_flag = &sh.abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int tokens = N / p.group;       // of a block of queries

  // ---- this CTA's share: every thread sums the costs of a few sequences, the CTA scans the sums
  const int per = (p.c.B + kAccThreads - 1) / kAccThreads;
  const int b_from = min((int)threadIdx.x * per, p.c.B), b_to = min(b_from + per, p.c.B);
  long long mine = 0;
  for (int b = b_from; b < b_to; ++b) mine += AccSeq<N>(p, b).total(p);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sh.scan[warp] = incl;
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    sh.first_b = -1;
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(&sh.k_full[s], 1);
      mbar_init(&sh.k_empty[s], 1);
    }
    for (int s = 0; s < C::kQStages; ++s) {
      mbar_init(&sh.q_full[s], 33);     // the loading warp's lanes (column data) and the expected bytes
      mbar_init(&sh.q_empty[s], 9);     // eight warps that sum and the products
    }
    for (int t = 0; t < 2; ++t)
      for (int s = 0; s < C::kBufs; ++s) {
        mbar_init(&sh.s_full[t][s], 1);
        mbar_init(&sh.s_empty[t][s], 4);
      }
    mbar_init(&sh.mma_done, 1);
    mbar_init(&sh.never, 1);
    fence_barrier_init();
  }
  __syncthreads();
  long long from = incl - mine, all = 0;
#pragma unroll
  for (int w = 0; w < kAccThreads / 32; ++w) {
    if (w < warp) from += sh.scan[w];
    all += sh.scan[w];
  }
  const long long share = (all + gridDim.x - 1) / gridDim.x;
  const long long c_first = blockIdx.x * share, c_end = min(c_first + share, all);
  if (c_first < c_end && c_first >= from && c_first < from + mine) {
    // the sequence that holds the share's first cost; a unit belongs to the share that its own first lies in
    for (int b = b_from; b < b_to; ++b) {
      const AccSeq<N> x(p, b);
      const long long n = x.total(p);
      if (c_first < from + n) {
        sh.first_unit = (int)((c_first - from + x.cost() - 1) / x.cost());
        sh.first_cost = from + (long long)sh.first_unit * x.cost();
        sh.first_b = b;
        break;
      }
      from += n;
    }
  }
  __syncwarp();
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  // (a CTA without a unit walks none; all of them free their tensor memory below)
  AccCursor<N> cur(p, max(sh.first_b, 0), sh.first_b < 0 ? 0 : sh.first_unit, sh.first_b < 0 ? 0 : c_end - sh.first_cost);

  if (warp == kKWarp) {
    // ------------------------------------------------------------ K tiles, page by page
    const int page_size = 1 << p.c.page_shift, box = min(page_size, kAccTile), boxes = kAccKeys / box;
    const uint32_t base = smem_u32(smem);
    auto look = [&](const AccCursor<N>& c) {
      int page = p.c.num_pages;         // out of range: zeros
      if (c.valid(p) && lane < boxes && c.w.any(c.key() + lane * box, box)) {
        const int x = find_page(p.c, c.b, c.key() + lane * box, kSitePagedPage);
        if (x >= 0) page = x;
      }
      return page;
    };
    if (lane == 0) tma_prefetch_desc(&tmK);
    int n = 0, page = look(cur);
    bool ok = true;
    while (cur.valid(p)) {
      AccCursor<N> ahead = cur;
      ahead.next(p);
      const int page_ahead = look(ahead);
      const int s = n % C::kKStages;
      ok = __all_sync(0xffffffffu, mbar_wait(&sh.k_empty[s], ((n / C::kKStages) & 1) ^ 1, abort_flag, p.c.status));
      if (!ok) break;
      const int tiles = cur.tile(1) ? 2 : 1;
      if (lane == 0) mbar_arrive_expect_tx(&sh.k_full[s], tiles * C::kTileBytes);
      __syncwarp();
      if (lane < boxes && lane * box < tiles * kAccTile) {
        const int row = lane * box;
        const uint32_t dst = base + s * C::kPairBytes + (row / kAccTile) * C::kTileBytes + (row % kAccTile) * C::kAtomBytes;
#pragma unroll
        for (int a = 0; a < C::kAtoms; ++a)
          tma_load_page(dst + a * kAccTile * C::kAtomBytes, &tmK, &sh.k_full[s], a * C::kAtomElems,
                        (cur.key() + row) & (page_size - 1), cur.h, page);
      }
      ++n;
      cur = ahead;
      page = page_ahead;
    }
    if (*abort_flag) {
      // let copies still in flight land before the CTA's shared memory goes away
      volatile uint32_t ignore_abort = 0;
      for (int i = max(0, n - C::kKStages); i < n; ++i)
        mbar_wait(&sh.k_full[i % C::kKStages], (i / C::kKStages) & 1, &ignore_abort, p.c.status);
    }
  } else if (warp == kQWarp) {
    // ------------------------------------------------------------ blocks of queries and their log-sum-exps
    if (lane == 0) tma_prefetch_desc(&tmQ);
    constexpr int kPer = (N + 31) / 32;
    int n = 0;
    bool ok = true;
    for (; ok && cur.valid(p); cur.next(p)) {
      const int last = cur.last_block(p, tokens);
      for (int i = cur.first_block(tokens); i < last; ++i, ++n) {
        float neg[kPer], factor[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const int r = e * 32 + lane, t = i * tokens + r / p.group;
          neg[e] = -INFINITY;
          factor[e] = 0.f;
          if (r < tokens * p.group && t < cur.s.n) {
            const long long row = (long long)(cur.s.q0 + t) * p.Hq + cur.h * p.group + r % p.group;
            const float lse = __ldg(g.lse + row);
            // a row that saw no key weighs nothing
            neg[e] = lse == -INFINITY ? -INFINITY : -1.4426950408889634f * lse;
            if constexpr (kFp8) factor[e] = p.scale_log2 * __ldg(g.q_scale + row);
          }
        }
        const int s = n % C::kQStages;
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.q_empty[s], ((n / C::kQStages) & 1) ^ 1, abort_flag, p.c.status));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.q_full[s], tokens * p.group * C::kRowBytes * (kFp8 ? kPieces : 1));
          uint8_t* dst = smem + C::kQOff + s * C::kQBytes;
          const int token = cur.s.q0 + i * tokens, head = cur.h * p.group;
          if constexpr (kFp8) {
            for (int x = 0; x < kPieces; ++x) tma_load_page(smem_u32(dst + x * C::kQTile), &tmQ, &sh.q_full[s], 0, head, token, x);
          } else {
            for (int a = 0; a < C::kAtoms; ++a)
              tma_load_3d(dst + a * N * C::kAtomBytes, &tmQ, &sh.q_full[s], a * C::kAtomElems, head, token);
          }
        }
        __syncwarp();
        float* col = reinterpret_cast<float*>(smem + C::kColOff) + s * 2 * N;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (e * 32 + lane < N) {
            col[e * 32 + lane] = neg[e];
            if constexpr (kFp8) col[N + e * 32 + lane] = factor[e];
          }
        mbar_arrive(&sh.q_full[s]);
      }
    }
    if (*abort_flag) {
      volatile uint32_t ignore_abort = 0;
      for (int i = max(0, n - C::kQStages); i < n; ++i)
        mbar_wait(&sh.q_full[i % C::kQStages], (i / C::kQStages) & 1, &ignore_abort, p.c.status);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    if (elect_one()) {
      const uint32_t sK = smem_u32(smem), sQ = smem_u32(smem + C::kQOff);
      int nk = 0, nq = 0, ns[2] = {0, 0};
      bool ok = true;
#ifdef FA_TEST_HOOKS
      // failure-detection test: as in the few-rows kernel
      if (p.inject_stall) ok = mbar_wait(&sh.never, 0, abort_flag, p.c.status);
#endif
      for (; ok && cur.valid(p); cur.next(p), ++nk) {
        const int ks = nk % C::kKStages, tiles = cur.tile(1) ? 2 : 1, last = cur.last_block(p, tokens);
        if (!(ok = mbar_wait(&sh.k_full[ks], (nk / C::kKStages) & 1, abort_flag, p.c.status))) break;
        for (int i = cur.first_block(tokens); ok && i < last; ++i, ++nq) {
          const int qs = nq % C::kQStages;
          if (!(ok = mbar_wait(&sh.q_full[qs], (nq / C::kQStages) & 1, abort_flag, p.c.status))) break;
          for (int t = 0; t < tiles; ++t) {
            const int buf = ns[t] % C::kBufs;
            if (!(ok = mbar_wait(&sh.s_empty[t][buf], ((ns[t] / C::kBufs) & 1) ^ 1, abort_flag, p.c.status))) break;
            tc_fence_after();
            const uint32_t d = tmem + (t * C::kBufs + buf) * N;
            const uint32_t a0 = sK + ks * C::kPairBytes + t * C::kTileBytes, b0 = sQ + qs * C::kQBytes;
            if constexpr (kFp8) {
#pragma unroll
              for (int x = 0; x < kPieces; ++x)
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk) {
                  const uint32_t a = a0 + kk * 32, b = b0 + x * C::kQTile + kk * 32;
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
          if (ok) tc_commit(&sh.q_empty[qs]);
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
  } else if (warp < 8) {
    // ------------------------------------------------------------ exponentials and sums: a thread per key
    const int t = warp / 4, row = t * kAccTile + (warp % 4) * 32 + lane;   // the thread's key within a unit
    const uint32_t tS = tmem + t * C::kBufs * N + ((uint32_t)((warp % 4) * 32) << 16);
    // the page of a unit's key is looked up two units ahead, what lies there is loaded one ahead
    auto look = [&](const AccCursor<N>& c) {
      AccKey k{false, false, -1, 0, 0.f, 0.f};
      if (!c.valid(p)) return k;
      const int key = c.key() + row;
      k.mine = c.w.seen(key);
      k.fresh = key >= c.s.pos0;
      if (k.mine) k.page = __ldg(p.c.table + c.b * p.c.table_stride + (key >> p.c.page_shift));   // hi is within the table
      k.at = ((long long)c.h << p.c.page_shift) + (key & ((1 << p.c.page_shift) - 1));
      return k;
    };
    auto load = [&](AccKey& k) {
      if (!k.mine) return;
      if (k.page < 0 || k.page >= p.c.num_pages) {
        report_bounds(p.c.status, kSitePagedPage, k.page);
        k.mine = false;
        return;
      }
      if (!k.fresh) k.old = g.weights[k.page * g.weight_stride + k.at];
      if constexpr (kFp8) k.scale = __ldg(p.c.k_scale + k.page * p.c.scale_stride + k.at);
    };
    AccKey k0 = look(cur);
    load(k0);
    AccCursor<N> c1 = cur;
    if (cur.valid(p)) c1.next(p);
    AccKey k1 = look(c1);
    int nq = 0, ns = 0;
    bool ok = true;
    while (ok && cur.valid(p)) {
      load(k1);
      AccCursor<N> c2 = c1;
      if (c1.valid(p)) c2.next(p);
      const AccKey k2 = look(c2);
      const int last = cur.last_block(p, tokens);
      const bool active = cur.tile(t);
      const int key = cur.key() + row;
      const float scale = kFp8 ? k0.scale : p.scale_log2;
      float total = 0.f;
      for (int i = cur.first_block(tokens); i < last; ++i, ++nq) {
        const int qs = nq % C::kQStages;
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.q_full[qs], (nq / C::kQStages) & 1, abort_flag, p.c.status));
        if (!ok) break;
        if (active) {
          const int buf = ns % C::kBufs;
          ok = __all_sync(0xffffffffu, mbar_wait(&sh.s_full[t][buf], (ns / C::kBufs) & 1, abort_flag, p.c.status));
          if (!ok) break;
          tc_fence_after();
          // the rows that see the key: its own token's on, up to the last one whose window holds it
          const int t0 = i * tokens, here = min(cur.s.n - t0, tokens);
          const int lo = min(max(key - cur.s.pos0 - t0, 0), here) * p.group;
          int end = here;
          if (p.window && key >= p.sinks) end = (int)min((long long)here, max((long long)key + p.window - cur.s.pos0 - t0, 0ll));
          const int hi = end * p.group;
          const float* col = reinterpret_cast<const float*>(smem + C::kColOff) + qs * 2 * N;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c0 = 0; c0 < N; c0 += W) {
            if (__all_sync(0xffffffffu, hi <= c0 || lo >= c0 + W)) continue;
            uint32_t r[W];
            if constexpr (W == 16)
              tmem_ld16(tS + buf * N + c0, r);
            else
              tmem_ld32(tS + buf * N + c0, r);
            tmem_ld_wait();
            reg_fence(r);
            if (__all_sync(0xffffffffu, lo <= c0 && hi >= c0 + W))
              acc_columns<W, kFp8, false>(r, col + c0, col + N + c0, scale, 0, sum);
            else
              acc_columns<W, kFp8, true>(r, col + c0, col + N + c0, scale, low_bits(hi - c0) & ~low_bits(lo - c0), sum);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.s_empty[t][buf]);
          ++ns;
          total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        } else {
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&sh.q_empty[qs]);
      }
      if (ok && k0.mine) g.weights[k0.page * g.weight_stride + k0.at] = k0.old + total;
      cur = c1;
      c1 = c2;
      k0 = k1;
      k1 = k2;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// The three E5M2 vectors of a query vector x: x = 2^e (p0 + p1 + p2), e such that the largest entry is in
// [2^14, 2^15).  Each takes what is left, rounded to nearest.  D / 8 lanes have a vector.
template <int D>
__global__ void __launch_bounds__(256) split_queries_kernel(const __nv_bfloat16* __restrict__ q, long long q_stride, int T,
                                                            int Hq, uint8_t* __restrict__ pieces, float* __restrict__ scale) {
  constexpr int kLanes = D / 8, kVecs = 256 / kLanes;
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

template <int D, bool kFp8, int N>
static int launch_acc(const CUtensorMap& tq, const CUtensorMap& tk, const Acc& g, cudaStream_t s) {
  auto kern = fa_accumulate_kernel<D, kFp8, N>;
  static std::atomic<uint64_t> prepared{0};
  const int rc = prepare_kernel(reinterpret_cast<const void*>(kern), acc_smem<D, kFp8, N>(), kAccThreads, 0, "accumulate kernel",
                                &prepared);
  if (rc) return rc;
  kern<<<sm_count(), kAccThreads, acc_smem<D, kFp8, N>(), s>>>(tq, tk, g);
  return check_cuda(cudaGetLastError(), "launch fa_accumulate_kernel");
}

template <int D, bool kFp8>
static int launch_columns(int columns, const CUtensorMap& tq, const CUtensorMap& tk, const Acc& g, cudaStream_t s) {
  if (columns == 16) return launch_acc<D, kFp8, 16>(tq, tk, g, s);
  if (columns == 32) return launch_acc<D, kFp8, 32>(tq, tk, g, s);
  if (columns == 64) return launch_acc<D, kFp8, 64>(tq, tk, g, s);
  return launch_acc<D, kFp8, 128>(tq, tk, g, s);
}

static int check_accumulate(int T, int Hq, int Hkv, int d) {
  if (T < 0) return set_error(FA_ERR_INVALID_ARG, "T must be >= 0 (got %d)", T);
  if (Hkv < 1 || Hq < 1) return set_error(FA_ERR_INVALID_ARG, "Hq, Hkv must be >= 1 (got %d, %d)", Hq, Hkv);
  if (Hq % Hkv) return set_error(FA_ERR_INVALID_ARG, "Hq = %d is not a multiple of Hkv = %d", Hq, Hkv);
  if (Hq / Hkv > 128) return set_error(FA_ERR_UNSUPPORTED, "more than 128 query heads for a kv head (%d)", Hq / Hkv);
  if (d != 64 && d != 128) return set_error(FA_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
  if ((long long)T * Hq >= (1ll << 31)) return set_error(FA_ERR_INVALID_ARG, "T*Hq must be < 2^31");
  return FA_OK;
}

// E4M3: the queries' pieces, then their factors.
static size_t pieces_bytes(int T, int Hq, int d) { return round_up((size_t)kPieces * T * Hq * d, 256); }

}  // namespace paged
}  // namespace fa

extern "C" size_t fa_kv_accumulate_workspace_size(int T, int Hq, int Hkv, int d, int dtype) {
  using namespace fa;
  clear_error();
  if (paged::check_accumulate(T, Hq, Hkv, d)) return 0;
  return dtype == FA_KV_E4M3 ? paged::pieces_bytes(T, Hq, d) + round_up((size_t)T * Hq * 4, 256) : 0;
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
  if ((rc = paged::check_cache(kv, &p.c)) || (rc = paged::check_accumulate(T, Hq, kv->Hkv, kv->d))) return rc;
  if (max_q < 0) return set_error(FA_ERR_INVALID_ARG, "max_q must be >= 0 (got %d)", max_q);
  if (!weights || (reinterpret_cast<uintptr_t>(weights) & 3))
    return set_error(FA_ERR_INVALID_ARG, "weights must be a 4-byte aligned device pointer");
  const long long page = (long long)kv->Hkv * kv->page_size;
  if (weight_stride < page)
    return set_error(FA_ERR_INVALID_ARG, "weight_stride %lld must be at least Hkv*page_size = %lld", (long long)weight_stride, page);
  if ((rc = check_ptr(q, "q")) || (rc = paged::check_indptr(q_indptr, "q_indptr"))) return rc;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3)) return set_error(FA_ERR_INVALID_ARG, "lse must be a 4-byte aligned device pointer");
  if (q_stride < (int64_t)Hq * kv->d || q_stride % 8)
    return set_error(FA_ERR_INVALID_ARG, "q_stride %lld must be a multiple of 8 and at least Hq*d = %d", (long long)q_stride, Hq * kv->d);
  if (!(scale > 0.f) || !isfinite(scale)) return set_error(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (window < 0 || sinks < 0) return set_error(FA_ERR_INVALID_ARG, "window and sinks must be >= 0 (got %d, %d)", window, sinks);
  if (!window && sinks) return set_error(FA_ERR_INVALID_ARG, "sinks need a window");
  const bool fp8 = kv->dtype == FA_KV_E4M3;
  const size_t need = fp8 ? fa_kv_accumulate_workspace_size(T, Hq, kv->Hkv, kv->d, kv->dtype) : 0;
  if (T == 0 || max_q == 0) return FA_OK;
  if (need) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
      return set_error(FA_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
    if (workspace_bytes < need)
      return set_error(FA_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed", workspace_bytes, need);
  }
  p.c.status = device_status_word();
  if (!p.c.status) return set_error(FA_ERR_CUDA, "could not allocate the device status record");
  const int max_kv = kv->max_pages * kv->page_size;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.q_indptr = q_indptr;
  p.T = T;
  p.Hq = Hq;
  p.group = Hq / kv->Hkv;
  p.max_rows = (int)((long long)max_q * p.group < INT32_MAX ? max_q * p.group : INT32_MAX);
  p.window = window >= max_kv ? 0 : window;
  p.sinks = std::min(sinks, max_kv);
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
#ifdef FA_TEST_HOOKS
  const char* inject = getenv("FA_TEST_INJECT_STALL");
  p.inject_stall = (inject && inject[0] == '1') ? 1 : 0;
#endif
  g.lse = lse;
  g.weights = weights;
  g.weight_stride = weight_stride;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int d = kv->d, box = kv->page_size < paged::kAccTile ? kv->page_size : paged::kAccTile;
  const int columns = p.max_rows <= 16 ? 16 : (p.max_rows <= 32 ? 32 : (p.max_rows <= 64 ? 64 : 128));
  CUtensorMap tq, tk;
  if ((rc = make_tmap_pages(&tk, kv->k, fp8, d, kv->page_size, kv->Hkv, kv->num_pages, kv->page_stride, box))) return rc;
  if (fp8) {
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
    if ((rc = make_tmap_pieces(&tq, pieces, T, Hq, d, paged::kPieces, p.group, columns / p.group))) return rc;
    return d == 64 ? paged::launch_columns<64, true>(columns, tq, tk, g, s) : paged::launch_columns<128, true>(columns, tq, tk, g, s);
  }
  if ((rc = make_tmap_rows(&tq, q, T, Hq, d, q_stride, p.group, columns / p.group))) return rc;
  return d == 64 ? paged::launch_columns<64, false>(columns, tq, tk, g, s) : paged::launch_columns<128, false>(columns, tq, tk, g, s);
}
