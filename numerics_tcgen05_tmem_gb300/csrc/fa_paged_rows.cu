// Paged attention for few rows (decoding): at most 64 rows for a kv head.
//
// With so few rows a key and its value are used for a handful of products only, so the kernel's
// bound is reading the cache: the rest has to stay out of the way of that stream.
//   * The keys of all sequences and kv heads are one list of 64-key blocks, sequence by sequence,
//     dealt to the CTAs in equal contiguous shares: two CTAs per SM, whatever the lengths, and no
//     long sequence that keeps one CTA busy after the others are done.  A share may end inside a
//     sequence; such a piece leaves its normalised output and log-sum-exp in the workspace and
//     fa_rows_combine joins the pieces in their order, so results do not depend on timing.
//   * One warp loads: page numbers from the table, 32 at a time, then TMA boxes into a ring of K and
//     V blocks (swizzled, so that the fragment loads meet no bank conflicts).  A page that no row
//     sees is taken out of range, which fills zeros without a read.
//   * Four warps compute with mma.sync: at 1 to 64 rows a tcgen05 tile (128 rows) would be mostly
//     empty, and its softmax would hold one row per thread.  The products are taken transposed,
//     S^T = K Q^T and O^T = V^T P^T, so that the rows are the instruction's narrow side: 8 of them
//     where 16 x 8 tiles of S would have 16.  A head's K and V fragments, and E4M3's conversions, are
//     then spent on 8 rows (kNR = 1) or 16 (2).  Row groups are dealt to the warps first, the block's
//     keys to the rest: for up to 16 rows each warp takes 16 keys of every block with its own running
//     maximum and sum, joined once at the end of a piece.
//   * E4M3: codes become FP16 with one conversion for two (exact), the vectors' scales multiply the
//     FP32 scores (K) and the FP32 probabilities (V, signs included).  Q goes to FP16 with a power of two per row
//     that brings its largest magnitude into [1, 2): exact but for elements 2^-14 below it, whose
//     error stays under 2^-25 of that magnitude, the size of an FP32 product's rounding.  The
//     weights, probability times scale, are rounded to FP16 relative to the piece's largest scale, or
//     where scales differ much to the row's largest weight so far: a large vector that a row does not see, or
//     gives next to no weight, would push all its other keys out of FP16's range.
// Softmax statistics and sums are FP32; P is rounded to BF16 (FP16 with E4M3) for the product with V,
// as the tensor core takes it.
// 64 sequences with 284k keys in all, 32 query heads and 8 kv heads, d = 128: E4M3 99 us, 92 % of the
// measured copy rate (605 MB read once; tensor pipe 16 %), BF16 173 us, at the copy rate; d = 64: 74 us, 63 %,
// and 92 us, 95 %.  One sequence of 4k keys, BF16: 7 us, of which the bytes take 2.5: what is left is one
// block's chain of load, products and softmax, and the join.
#include "paged_attn.cuh"

namespace fa {
namespace paged {

constexpr int kRowsBlk = 64;
// A warpgroup computes, one warp of a second one loads.  The second is a whole warpgroup because
// setmaxnreg moves registers between warpgroups: the computing threads hold Q, O and the scores of
// two blocks (with 168 registers the E4M3 form spilled and was 7 % slower).
constexpr int kRowsWarps = 4;
constexpr int kRowsLoadWarp = 4;
constexpr int kRowsThreads = 256;
constexpr int kRowsRegLaunch = 128, kRowsRegCompute = 208, kRowsRegLoad = 48;
static_assert(kRowsRegCompute + kRowsRegLoad <= 2 * kRowsRegLaunch, "register split exceeds the launch allocation");

// E4M3: the weights P~ (scale of V) go to FP16 with their reference at 2^kWeightExp, half of what FP16
// holds: weights down to 2^-29 of it keep 11 bits, and one under 2^-40 of it is lost.  A piece's scales that
// lie within kWideSpread of each other share the largest one as reference, at most that much above any row's
// largest weight (the key with the largest score has P~ = 1); with others each row takes the largest weight
// itself.  64 sequences of 4.4k keys, 8 kv heads, d = 128, at 8, 16, 32 and 64 rows: 99, 128, 199, 310 us; with a
// reference for each row in all pieces 104, 151, 230, 348; with the largest scale alone, which loses keys, 98,
// 123, 190, 302.
constexpr int kWeightExp = 15;
constexpr float kWideSpread = 1024.f;
constexpr float kLeastRef = 3.8518598887744717e-34f;   // 2^-111: 2^kWeightExp over it stays finite

template <int D, bool kFp8>
struct RowsCfg {
  static constexpr int kElem = kFp8 ? 1 : 2;
  static constexpr int kRowBytes = D * kElem;                          // 64, 128 or 256
  static constexpr int kAtomBytes = kRowBytes >= 128 ? 128 : 64;       // swizzle atom row
  static constexpr int kAtoms = kRowBytes / kAtomBytes;
  static constexpr int kAtomElems = kAtomBytes / kElem;
  static constexpr int kTile = kRowsBlk * kRowBytes;                   // K or V of one block
  static constexpr int kFit = 96 * 1024 / (2 * kTile);
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kScaleOff = kStages * 2 * kTile;
  static constexpr int kScaleBytes = kFp8 ? 2 * kRowsBlk * 4 : 0;      // per stage
  static constexpr int kBufOff = kScaleOff + kStages * kScaleBytes;    // joining: four rows of each warp
  static constexpr int kBufRow = D + 8;                                // floats; the pad spreads rows over banks
  static constexpr int kSmemBytes = kBufOff + kRowsWarps * 4 * kBufRow * 4 + 1024;
  static_assert(2 * (kSmemBytes + 2048) <= 228 * 1024, "two CTAs must fit one SM's shared memory");
  // shared-memory address of 16-byte chunk x of row r of a tile
  __device__ static uint32_t chunk(uint32_t base, int r, int x) {
    constexpr int kPer = kAtomBytes / 16;
    const int sw = kAtomBytes == 128 ? (r & 7) : ((r >> 1) & 3);
    return base + (x / kPer) * (kRowsBlk * kAtomBytes) + r * kAtomBytes + (((x % kPer) ^ sw) << 4);
  }
};

struct RowsShared {
  uint64_t full[8], empty[8], sync;
  uint64_t never;            // test builds only: a barrier nothing arrives on
  uint32_t abort_flag;
  float m[kRowsWarps][16], l[kRowsWarps][16];   // by warp and row of its group
  int scan[kRowsThreads / 32];
  int first_b;               // the sequence of this CTA's first unit
  long long first_unit;      // ... and that unit's number within the sequence
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// The 8 x 8 matrix of 16-bit elements that the warp holds (row lane / 4, two columns per lane), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two E4M3 codes (low 16 bits of w) as FP16 pairs.
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t w) {
  uint32_t h;
  asm("{\n .reg .b16 c, x;\n mov.b32 {c, x}, %1;\n cvt.rn.f16x2.e4m3x2 %0, c;\n}" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t codes_hi_f16x2(uint32_t w) {
  uint32_t h;
  asm("{\n .reg .b16 c, x;\n mov.b32 {x, c}, %1;\n cvt.rn.f16x2.e4m3x2 %0, c;\n}" : "=r"(h) : "r"(w));
  return h;
}

// A sequence as the few-rows kernel sees it: its walk, or no steps where it is not this kernel's.
struct RowsItem {
  Seq s;
  int rows;
  KeyWalk<kRowsBlk> w;
  __device__ __forceinline__ RowsItem(const Attn& p, int b) : s(load_seq(p, b)), rows(s.n * p.group), w(p, s.pos0, s.kv - 1) {
    if (rows == 0 || rows > p.few_rows) w.steps = 0;
  }
};

// Work is dealt in units: an item (sequence, kv head) takes kItemUnits for loading its queries and
// writing its rows, then one per 64-key block.  Unit u of the launch is (b, h, unit within the item),
// the last fastest; a CTA's share is [u_first, u_end).
// On 64 sequences of 500 to 16k keys, E4M3, two units for an item were 9 % faster than none, six 15 %
// (the CTAs with short sequences were last).
constexpr int kItemUnits = 6;
constexpr int kMinShare = 2;   // for a batch of few keys: as many CTAs as there are pairs of blocks

// Units of the sequences [b0, b1), for one kv head.
__device__ __forceinline__ int count_units(const Attn& p, int b0, int b1) {
  int n = 0;
  for (int b = b0; b < b1; ++b) {
    const int steps = RowsItem(p, b).w.steps;
    n += steps ? steps + kItemUnits : 0;
  }
  return n;
}

// kRG row groups of 8 kNR rows: warp w takes row group w / (4 / kRG) and the keys of group w % (4 / kRG).
template <int D, bool kFp8, int kRG, int kNR>
__global__ void __launch_bounds__(kRowsThreads, 2)
    fa_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Attn p) {
  using C = RowsCfg<D, kFp8>;
  constexpr int kKG = kRowsWarps / kRG;        // key groups
  constexpr int kKeys = kRowsBlk / kKG;        // keys of a block for one warp
  constexpr int kKT = kKeys / 16;              // 16-key tiles of S^T
  constexpr int kPair = kRG == 1 ? 2 : 1;      // blocks taken at a time
  constexpr int kRows = 8 * kNR * kRG;         // rows of a slot
  static_assert(C::kStages >= kPair, "the ring must hold every block that is waited for at once");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ RowsShared sh;
  volatile uint32_t* abort_flag = &sh.abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  // ---- shares: every thread counts the units of a few sequences, the CTA scans the counts
  const int per = (p.c.B + kRowsThreads - 1) / kRowsThreads;
  const int b_from = min((int)threadIdx.x * per, p.c.B), b_to = min(b_from + per, p.c.B);
  const int mine = count_units(p, b_from, b_to);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sh.scan[warp] = incl;
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    sh.first_b = -1;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], kRowsWarps);
    }
    mbar_init(&sh.sync, 32 * kRowsWarps);
    mbar_init(&sh.never, 1);
    fence_barrier_init();
  }
  __syncthreads();
  int before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kRowsThreads / 32; ++w) {
    if (w < warp) before += sh.scan[w];
    total += sh.scan[w];
  }
  const long long units = (long long)total * p.c.Hkv;
  const int share = (int)max((units + gridDim.x - 1) / gridDim.x, (long long)kMinShare);
  const long long u_first = (long long)blockIdx.x * share;
  const long long u_end = min(u_first + share, units);
  {
    // the thread whose sequences hold the share's first unit finds the sequence
    const long long from = (long long)before * p.c.Hkv, to = from + (long long)mine * p.c.Hkv;
    if (u_first < u_end && u_first >= from && u_first < to) {
      long long u = from;
      for (int b = b_from; b < b_to; ++b) {
        const long long n = (long long)count_units(p, b, b + 1) * p.c.Hkv;
        if (u_first < u + n) {
          sh.first_b = b;
          sh.first_unit = u_first - u;
          break;
        }
        u += n;
      }
    }
  }
  __syncthreads();
  // Launched beside a chunk kernel, this launch must not end before it (what follows in the stream
  // waits for this launch only): one idle warp waits for it.
  const bool waits = blockIdx.x == 0 && warp == kRowsThreads / 32 - 1;
  if (u_first >= u_end || sh.first_b < 0) {
    if (waits) cudaGridDependencySynchronize();
    return;
  }

  if (warp >= kRowsWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRowsRegLoad));
    if (warp != kRowsLoadWarp) {
      if (waits) cudaGridDependencySynchronize();
      return;
    }
    // ------------------------------------------------------------------ loading warp
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    const int page_size = 1 << p.c.page_shift;
    const int box = min(page_size, kRowsBlk), ppb = kRowsBlk / box;  // box rows, boxes per block
    const int per_group = 32 / ppb;                                  // blocks whose pages one look-up covers
    const uint32_t base = smem_u32(smem);
    int n = 0;
    bool ok = true;
    int b = sh.first_b;
    long long unit = sh.first_unit;
    for (long long u = u_first; ok && u < u_end && b < p.c.B; ++b, unit = 0) {
      const RowsItem it(p, b);
      if (it.w.steps == 0) continue;
      const int n_units = it.w.steps + kItemUnits;
      int h = (int)(unit / n_units), x0 = (int)(unit - (long long)h * n_units);
      for (; ok && h < p.c.Hkv && u < u_end; ++h, x0 = 0) {
        const int x1 = (int)min((long long)n_units, x0 + (u_end - u));
        u += x1 - x0;
        const int j0 = max(x0 - kItemUnits, 0), j1 = max(x1 - kItemUnits, 0);  // this piece's blocks, if any
        for (int jg = j0; ok && jg < j1; jg += per_group) {
          const int jl = jg + lane / ppb;
          int page = p.c.num_pages;  // out of range: zeros
          if (jl < j1) {
            const int key = it.w.at(jl) + (lane % ppb) * box;
            if (it.w.any(key, box)) {
              const int x = find_page(p.c, b, key, kSitePagedPage);
              if (x >= 0) page = x;
            }
          }
          for (int jj = 0; jj < per_group && jg + jj < j1; ++jj, ++n) {
            const int s = n % C::kStages;
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&sh.empty[s], ((n / C::kStages) & 1) ^ 1, abort_flag, p.c.status));
            if (!ok) break;
            const int pg = __shfl_sync(0xffffffffu, page, jj * ppb + lane % ppb);
            const bool loads = lane < ppb, real = loads && pg < p.c.num_pages;
            const int scaled = kFp8 ? __popc(__ballot_sync(0xffffffffu, real)) : 0;
            if (lane == 0) mbar_arrive_expect_tx(&sh.full[s], 2 * C::kTile + scaled * 2 * box * 4);
            __syncwarp();
            if (loads) {
              const int slot = (it.w.at(jg + jj) + lane * box) & (page_size - 1);
              const uint32_t dst = base + s * 2 * C::kTile + lane * box * C::kAtomBytes;
#pragma unroll
              for (int a = 0; a < C::kAtoms; ++a) {
                tma_load_page(dst + a * kRowsBlk * C::kAtomBytes, &tmK, &sh.full[s], a * C::kAtomElems, slot, h, pg);
                tma_load_page(dst + C::kTile + a * kRowsBlk * C::kAtomBytes, &tmV, &sh.full[s], a * C::kAtomElems, slot,
                              h, pg);
              }
              if (kFp8 && real) {
                uint8_t* sc = smem + C::kScaleOff + s * C::kScaleBytes + lane * box * 4;
                const long long row = pg * p.c.scale_stride + (long long)h * page_size + slot;
                bulk_load(sc, p.c.k_scale + row, box * 4, &sh.full[s]);
                bulk_load(sc + kRowsBlk * 4, p.c.v_scale + row, box * 4, &sh.full[s]);
              }
            }
          }
        }
      }
    }
    if (*abort_flag) {
      // let copies still in flight land before the CTA's shared memory goes away
      volatile uint32_t ignore_abort = 0;
      for (int i = max(0, n - C::kStages); i < n; ++i)
        mbar_wait(&sh.full[i % C::kStages], (i / C::kStages) & 1, &ignore_abort, p.c.status);
    }
    return;
  }

  // -------------------------------------------------------------------- computing warps
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowsRegCompute));
  const int rg = warp / kKG, kg = warp % kKG;     // row group, key group
  const int l4 = lane / 4, t4 = lane % 4;
  const int row0 = rg * 8 * kNR;                  // first row of the group
  const int row_k = kg * kKeys;                   // this warp's first key within a block
  const uint32_t base = smem_u32(smem);
  float* buf = reinterpret_cast<float*>(smem + C::kBufOff);
  // the lane's row and 16-byte chunk within the 8 x 8 matrices of a fragment load: (8 keys, chunk)
  // in the order (low, 0) (high, 0) (low, 1) (high, 1); V in BF16 takes (low, 0) (low, 1) (high, 0) ..
  const int f_key = (lane & 7) + ((lane >> 3) & 1) * 8, f_chunk = lane >> 4;
  const int v_key = kFp8 ? f_key : (lane & 7) + (lane >> 4) * 8, v_chunk = kFp8 ? f_chunk : (lane >> 3) & 1;
  int n = 0, syncs = 0;
  bool ok = true;
  auto warps_sync = [&]() {
    mbar_arrive(&sh.sync);
    return mbar_wait(&sh.sync, syncs++ & 1, abort_flag, p.c.status);
  };
#ifdef FA_TEST_HOOKS
  // failure-detection test: wait on a barrier nothing arrives on; the bounded wait runs out, raises
  // the CTA's abort flag and records a timeout, and every warp unwinds
  if (p.inject_stall) ok = __all_sync(0xffffffffu, mbar_wait(&sh.never, 0, abort_flag, p.c.status));
#endif
  int b = sh.first_b;
  long long unit = sh.first_unit;
  bool first_piece = true;
  for (long long u = u_first; ok && u < u_end && b < p.c.B; ++b, unit = 0) {
    const RowsItem it(p, b);
    if (it.w.steps == 0) continue;
    const int steps = it.w.steps, n_units = steps + kItemUnits;
    int h = (int)(unit / n_units), x0 = (int)(unit - (long long)h * n_units);
    for (; ok && h < p.c.Hkv && u < u_end; ++h, x0 = 0) {
      const int x1 = (int)min((long long)n_units, x0 + (u_end - u));
      const long long u_blocks = u - x0 + kItemUnits;   // the unit of the item's first block
      u += x1 - x0;
      const int j0 = max(x0 - kItemUnits, 0), j1 = max(x1 - kItemUnits, 0);  // this piece's blocks
      if (j1 == j0) continue;                                                // (the next CTA's)
      // ---- Q fragments (the B operand, columns = rows of the group): lane's column l4 of each 8
      float c_row[kNR][2];   // score factors of the rows 2 t4, 2 t4 + 1 that the lane's scores belong to
      int pos[kNR][2];       // their positions; -1 (sees nothing) past the last row
      uint32_t qf[kNR][D / 16][2];
#pragma unroll
      for (int nr = 0; nr < kNR; ++nr) {
        const int r = row0 + 8 * nr + l4, t = r / p.group;
        const bool valid = r < it.rows;
        const __nv_bfloat16* qr =
            p.q + (long long)(it.s.q0 + t) * p.q_stride + (long long)(h * p.group + (r - t * p.group)) * D;
        float factor = p.scale_log2;
        if constexpr (!kFp8) {
          // BF16: columns 2t, 2t + 1 and 2t + 8, 2t + 9 of each 16
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            qf[nr][kk][0] = valid ? __ldg(reinterpret_cast<const uint32_t*>(qr + kk * 16 + 2 * t4)) : 0u;
            qf[nr][kk][1] = valid ? __ldg(reinterpret_cast<const uint32_t*>(qr + kk * 16 + 8 + 2 * t4)) : 0u;
          }
        } else {
          // E4M3: columns 4t .. 4t + 3 of each 16, the order in which K's codes arrive
          uint2 w[D / 16];
          uint32_t amax = 0;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            w[kk] = valid ? __ldg(reinterpret_cast<const uint2*>(qr + kk * 16 + 4 * t4)) : make_uint2(0, 0);
            amax = max(amax, max(max((w[kk].x & 0x7FFFu) << 16, w[kk].x & 0x7FFF0000u),
                                 max((w[kk].y & 0x7FFFu) << 16, w[kk].y & 0x7FFF0000u)));
          }
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          int e = (int)(amax >> 23) - 127;
          // zero rows and rows with Inf or NaN go unscaled; 2^-e and 2^e stay normal
          if (amax == 0 || amax >= 0x7F800000u) e = 0;
          e = min(max(e, -126), 126);
          const float down = __uint_as_float((uint32_t)(127 - e) << 23);
          factor *= __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            qf[nr][kk][0] = pack_f16x2(__uint_as_float(w[kk].x << 16) * down, __uint_as_float(w[kk].x & 0xFFFF0000u) * down);
            qf[nr][kk][1] = pack_f16x2(__uint_as_float(w[kk].y << 16) * down, __uint_as_float(w[kk].y & 0xFFFF0000u) * down);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = row0 + 8 * nr + 2 * t4 + e;
          pos[nr][e] = rr < it.rows ? it.s.pos0 + rr / p.group : -1;
          c_row[nr][e] = kFp8 ? __shfl_sync(0xffffffffu, factor, (2 * t4 + e) * 4) : factor;
        }
      }
      float o[D / 16][kNR][4];   // O^T: 16 columns of O by 8 rows
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][nr][e] = 0.f;
      float m[kNR][2], l[kNR][2];
#pragma unroll
      for (int nr = 0; nr < kNR; ++nr) m[nr][0] = m[nr][1] = -INFINITY, l[nr][0] = l[nr][1] = 0.f;
      // E4M3: O is in units of v_ref / 2^kWeightExp, and v_inv is its reciprocal; once the scales seen
      // spread too far (wide), each row has a reference of its own, w_ref.  v_low: the least scale seen
      float v_ref = 0.f, v_inv = 0.f, v_low = INFINITY, w_ref[kNR][2];
      bool wide = false;
      // kPair blocks at a time: their products are independent of each other, and the bookkeeping of
      // the running maximum is paid once for both
      for (int j = j0; j < j1; j += kPair) {
        const int nb = min(kPair, j1 - j);
        bool edge = false;
#pragma unroll
        for (int x = 0; x < kPair; ++x) {
          if (x >= nb) break;
          ok = __all_sync(0xffffffffu, mbar_wait(&sh.full[(n + x) % C::kStages], ((n + x) / C::kStages) & 1, abort_flag,
                                                 p.c.status));
          if (!ok) break;
          edge |= !it.w.all(p, it.w.at(j + x), it.s.pos0, it.s.kv - 1);
        }
        if (!ok) break;
        // ---- S^T = K Q^T; an odd last block's missing partner repeats it and is masked (a uniform
        // body keeps the accumulation chains interleaved)
        float sc[kPair * kKT][kNR][4];
#pragma unroll
        for (int i = 0; i < kPair * kKT; ++i)
#pragma unroll
          for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[i][nr][e] = 0.f;
        uint32_t sK[kPair];
#pragma unroll
        for (int x = 0; x < kPair; ++x) sK[x] = base + ((n + (x < nb ? x : 0)) % C::kStages) * 2 * C::kTile;
#pragma unroll
        for (int c0 = 0; c0 < C::kRowBytes / 16; c0 += 2) {
#pragma unroll
          for (int i = 0; i < kPair * kKT; ++i) {
            uint32_t f[4];
            ldsm4(f, C::chunk(sK[i / kKT], row_k + (i % kKT) * 16 + f_key, c0 + f_chunk));
            if constexpr (!kFp8) {
#pragma unroll
              for (int nr = 0; nr < kNR; ++nr) mma16816<false>(sc[i][nr], f, qf[nr][c0 / 2][0], qf[nr][c0 / 2][1]);
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t a[4] = {codes_f16x2(f[2 * e]), codes_f16x2(f[2 * e + 1]), codes_hi_f16x2(f[2 * e]),
                                       codes_hi_f16x2(f[2 * e + 1])};
#pragma unroll
                for (int nr = 0; nr < kNR; ++nr) mma16816<true>(sc[i][nr], a, qf[nr][c0 + e][0], qf[nr][c0 + e][1]);
              }
            }
          }
        }
        // ---- scores in units of log2, scales of K (a lane's keys: l4 and l4 + 8 of each 16)
#pragma unroll
        for (int i = 0; i < kPair * kKT; ++i) {
          float k0 = 1.f, k1 = 1.f;
          if constexpr (kFp8) {
            const float* ks = reinterpret_cast<const float*>(
                smem + C::kScaleOff + ((n + (i / kKT < nb ? i / kKT : 0)) % C::kStages) * C::kScaleBytes);
            k0 = ks[row_k + (i % kKT) * 16 + l4];
            k1 = ks[row_k + (i % kKT) * 16 + l4 + 8];
          }
#pragma unroll
          for (int nr = 0; nr < kNR; ++nr) {
            float (&v)[4] = sc[i][nr];
            mul2(v[0], v[1], v[0], v[1], k0 * c_row[nr][0], k0 * c_row[nr][1]);
            mul2(v[2], v[3], v[2], v[3], k1 * c_row[nr][0], k1 * c_row[nr][1]);
          }
        }
        if (kPair > 1 && nb < kPair) {
#pragma unroll
          for (int i = kKT; i < kPair * kKT; ++i)
#pragma unroll
            for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[i][nr][e] = -INFINITY;
        }
        if (edge) {
#pragma unroll
          for (int x = 0; x < kPair; ++x) {
            if (x >= nb) break;
            const int key0 = it.w.at(j + x) + row_k;
            // V rows that no row sees may hold anything: 0 * NaN must not reach the product
            const uint32_t sV = base + ((n + x) % C::kStages) * 2 * C::kTile + C::kTile;
            for (int i = lane; i < kKeys * (C::kRowBytes / 16); i += 32) {
              const int r = i / (C::kRowBytes / 16);
              if (!it.w.seen(key0 + r))
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                 C::chunk(sV, row_k + r, i % (C::kRowBytes / 16))),
                             "r"(0)
                             : "memory");
            }
#pragma unroll
            for (int i = 0; i < kKT; ++i)
#pragma unroll
              for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int key = key0 + i * 16 + l4 + (e >> 1) * 8, at = pos[nr][e & 1];
                  const bool see = key <= at && (!p.window || at - key < p.window || key < p.sinks);
                  if (!see) sc[x * kKT + i][nr][e] = -INFINITY;
                }
          }
          __syncwarp();
        }
        // ---- running maximum and sum of each row; the lanes of one t4 hold a row's keys
        float f_row[kNR][2];
        bool moved = false;
#pragma unroll
        for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = m[nr][e];
#pragma unroll
            for (int i = 0; i < kPair * kKT; ++i) mx = max3f(mx, sc[i][nr][e], sc[i][nr][e + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mu = mx == -INFINITY ? 0.f : mx;
            f_row[nr][e] = ex2_approx(m[nr][e] - mu);
            m[nr][e] = mx;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < kPair * kKT; ++i) {
              float &a = sc[i][nr][e], &c = sc[i][nr][e + 2];
              add2(a, c, a, c, -mu, -mu);
              a = ex2_approx(a);
              c = ex2_approx(c);
              sum += a + c;
            }
            l[nr][e] = l[nr][e] * f_row[nr][e] + sum;
            moved |= f_row[nr][e] != 1.f;
          }
        if constexpr (kFp8) {
          // ---- weights P~ (scale of V), for FP16
          float v0[kPair * kKT], v1[kPair * kKT], top = 0.f, low = INFINITY;
#pragma unroll
          for (int i = 0; i < kPair * kKT; ++i) {
            const int x = i / kKT;
            const float* vs = reinterpret_cast<const float*>(smem + C::kScaleOff + ((n + x) % C::kStages) * C::kScaleBytes) +
                              kRowsBlk + row_k + (i % kKT) * 16 + l4;
            v0[i] = v1[i] = 0.f;
            if (x < nb) {
              v0[i] = vs[0];
              v1[i] = vs[8];
              if (edge) {   // slots that no row sees may hold anything
                const int key = it.w.at(j + x) + row_k + (i % kKT) * 16 + l4;
                if (!it.w.seen(key)) v0[i] = 0.f;
                if (!it.w.seen(key + 8)) v1[i] = 0.f;
              }
            }
            top = max3f(top, fabsf(v0[i]), fabsf(v1[i]));
            low = min3f(low, v0[i] == 0.f ? INFINITY : fabsf(v0[i]), v1[i] == 0.f ? INFINITY : fabsf(v1[i]));
          }
          // scales alike: the largest one so far is the reference of all rows
          if (!wide && __any_sync(0xffffffffu, top > v_ref || low < v_low)) {
#pragma unroll
            for (int off = 4; off < 32; off *= 2) {
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
              low = fminf(low, __shfl_xor_sync(0xffffffffu, low, off));
            }
            top = fmaxf(fmaxf(top, v_ref), kLeastRef);
            v_low = fminf(low, v_low);
            wide = v_low * kWideSpread < top;
            if (wide) {
#pragma unroll
              for (int nr = 0; nr < kNR; ++nr) w_ref[nr][0] = w_ref[nr][1] = v_ref;
            } else if (top > v_ref) {
              const float ratio = v_ref / top;
#pragma unroll
              for (int nr = 0; nr < kNR; ++nr) {
                f_row[nr][0] *= ratio;
                f_row[nr][1] *= ratio;
              }
              v_ref = top;
              v_inv = (float)(1 << kWeightExp) / top;
              moved = true;
            }
          }
          if (!wide) {
#pragma unroll
            for (int i = 0; i < kPair * kKT; ++i) {
              const float a = v0[i] * v_inv, c = v1[i] * v_inv;
#pragma unroll
              for (int nr = 0; nr < kNR; ++nr) {
                float (&v)[4] = sc[i][nr];
                mul2(v[0], v[1], v[0], v[1], a, a);
                mul2(v[2], v[3], v[2], v[3], c, c);
              }
            }
          } else {
            // a row's reference is its largest weight so far (or above it); it falls with m's rise as O
            // does, so O is rescaled only where a weight exceeds it
            moved = false;
#pragma unroll
            for (int nr = 0; nr < kNR; ++nr) {
              float most[2] = {0.f, 0.f};
#pragma unroll
              for (int i = 0; i < kPair * kKT; ++i) {
                float (&v)[4] = sc[i][nr];
                mul2(v[0], v[1], v[0], v[1], v0[i], v0[i]);
                mul2(v[2], v[3], v[2], v[3], v1[i], v1[i]);
                most[0] = max3f(most[0], fabsf(v[0]), fabsf(v[2]));
                most[1] = max3f(most[1], fabsf(v[1]), fabsf(v[3]));
              }
#pragma unroll
              for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int off = 4; off < 32; off *= 2)
                  most[e] = fmaxf(most[e], __shfl_xor_sync(0xffffffffu, most[e], off));
                const float was = w_ref[nr][e] * f_row[nr][e];
                w_ref[nr][e] = fmaxf(fmaxf(most[e], was), kLeastRef);
                f_row[nr][e] = was / w_ref[nr][e];
                moved |= f_row[nr][e] != 1.f;
              }
              const float inv0 = (float)(1 << kWeightExp) / w_ref[nr][0], inv1 = (float)(1 << kWeightExp) / w_ref[nr][1];
#pragma unroll
              for (int i = 0; i < kPair * kKT; ++i) {
                float (&v)[4] = sc[i][nr];
                mul2(v[0], v[1], v[0], v[1], inv0, inv1);
                mul2(v[2], v[3], v[2], v[3], inv0, inv1);
              }
            }
          }
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int nr = 0; nr < kNR; ++nr) {
              float (&v)[4] = o[i][nr];
              mul2(v[0], v[1], v[0], v[1], f_row[nr][0], f_row[nr][1]);
              mul2(v[2], v[3], v[2], v[3], f_row[nr][0], f_row[nr][1]);
            }
        }
        // ---- O^T += V^T P^T: 16 keys per step
#pragma unroll
        for (int x = 0; x < kPair; ++x) {
          if (x >= nb) break;
          const int s = (n + x) % C::kStages;
          const uint32_t sV = base + s * 2 * C::kTile + C::kTile;
#pragma unroll
          for (int i = 0; i < kKT; ++i) {
            uint32_t pb[kNR][2];   // P^T as the B operand: keys along k, rows along n
#pragma unroll
            for (int nr = 0; nr < kNR; ++nr) {
              const float (&v)[4] = sc[x * kKT + i][nr];
              pb[nr][0] = transpose8(kFp8 ? pack_f16x2(v[0], v[1]) : pack_bf16x2(v[0], v[1]));
              pb[nr][1] = transpose8(kFp8 ? pack_f16x2(v[2], v[3]) : pack_bf16x2(v[2], v[3]));
            }
#pragma unroll
            for (int c0 = 0; c0 < C::kRowBytes / 16; c0 += 2) {
              uint32_t f[4];
              ldsm4_t(f, C::chunk(sV, row_k + i * 16 + v_key, c0 + v_chunk));
              if constexpr (!kFp8) {
#pragma unroll
                for (int nr = 0; nr < kNR; ++nr) mma16816<false>(o[c0 / 2][nr], f, pb[nr][0], pb[nr][1]);
              } else {
                // each 16-bit element is two columns' codes, bytes (key, col) (key, col + 1) (key + 1, ..):
                // the even columns become the tile's rows 0-7, the odd ones 8-15
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t lo = __byte_perm(f[2 * e], 0, 0x3120), hi = __byte_perm(f[2 * e + 1], 0, 0x3120);
                  const uint32_t a[4] = {codes_f16x2(lo), codes_hi_f16x2(lo), codes_f16x2(hi), codes_hi_f16x2(hi)};
#pragma unroll
                  for (int nr = 0; nr < kNR; ++nr) mma16816<true>(o[c0 + e][nr], a, pb[nr][0], pb[nr][1]);
                }
              }
            }
          }
          if (edge) fence_proxy_async_smem();  // the zeroed rows precede the stage's next TMA write
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.empty[s]);
        }
        n += nb;
      }
      if (!ok) break;
      // ---- join the key groups and write
#pragma unroll
      for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int off = 4; off < 32; off *= 2) l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], off);
          if (l4 == 0) {
            sh.m[warp][8 * nr + 2 * t4 + e] = m[nr][e];
            sh.l[warp][8 * nr + 2 * t4 + e] = l[nr][e];
          }
        }
      if (!(ok = __all_sync(0xffffffffu, warps_sync()))) break;
      const bool whole = j0 == 0 && j1 == steps;
      const int slot = 2 * blockIdx.x + (first_piece ? 0 : 1);
      first_piece = false;
      float w_row[kNR][2];
#pragma unroll
      for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int in = 8 * nr + 2 * t4 + e, r = row0 + in;
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int k = 0; k < kKG; ++k) top = fmaxf(top, sh.m[rg * kKG + k][in]);
          const float tu = top == -INFINITY ? 0.f : top;
#pragma unroll
          for (int k = 0; k < kKG; ++k) sum += sh.l[rg * kKG + k][in] * ex2_approx(sh.m[rg * kKG + k][in] - tu);
          const bool empty = top == -INFINITY && sum == 0.f;   // no visible key (a NaN score is not that)
          w_row[nr][e] = empty ? 0.f : ex2_approx(m[nr][e] - tu) / sum;
          if constexpr (kFp8) w_row[nr][e] *= 1.f / (1 << kWeightExp);
          const float lse = empty ? -INFINITY : top * 0.6931471805599453f + logf(sum);
          const bool mine = kg == 0 && l4 == 0 && r < it.rows;
          if (mine) {
            if (!whole) {
              p.part_lse[(long long)slot * kRows + r] = lse;
            } else if (p.lse) {
              const int t = r / p.group;
              p.lse[(long long)(it.s.q0 + t) * p.Hq + h * p.group + (r - t * p.group)] = lse;
            }
          }
          if (whole) report_nonfinite((mine && !empty && !(fabsf(lse) < INFINITY)) ? 1u : 0u, p.c.status, kOutLse);
        }
      uint32_t bad = 0;
      for (int rr = 0; rr < min(8 * kNR, it.rows); rr += 4) {   // four rows of every row group at a time
#pragma unroll
        for (int nr = 0; nr < kNR; ++nr) {
          if (rr / 8 != nr || (t4 & 2) != ((rr & 4) >> 1)) continue;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* dst = buf + (warp * 4 + (2 * t4 & 3) + e) * C::kBufRow;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              float a = o[i][nr][e] * w_row[nr][e], c = o[i][nr][e + 2] * w_row[nr][e];
              if constexpr (kFp8) {
                const float ref = wide ? w_ref[nr][e] : v_ref;
                a *= ref;   // (a product of its own: the factors' may be subnormal)
                c *= ref;
                *reinterpret_cast<float2*>(dst + i * 16 + 2 * l4) = make_float2(a, c);
              } else {
                dst[i * 16 + l4] = a;
                dst[i * 16 + l4 + 8] = c;
              }
            }
          }
        }
        if (!(ok = __all_sync(0xffffffffu, warps_sync()))) break;
#pragma unroll
        for (int e = 0; e < (kRG * D + 127) / 128; ++e) {
          const int idx = threadIdx.x + e * 128;          // of 4 kRG rows x D / 4 groups of four columns
          if (kRG * D < 128 && idx >= kRG * D) break;
          const int q4 = idx / (D / 4), c4 = (idx % (D / 4)) * 4, g = q4 / 4;
          const int r = g * 8 * kNR + rr + q4 % 4;
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < kKG; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(buf + ((g * kKG + k) * 4 + q4 % 4) * C::kBufRow + c4);
            sum.x += x.x;
            sum.y += x.y;
            sum.z += x.z;
            sum.w += x.w;
          }
          if (r < it.rows) {
            if (!whole) {
              *reinterpret_cast<float4*>(p.part_o + ((long long)slot * kRows + r) * D + c4) = sum;
            } else {
              const int t = r / p.group;
              const uint2 v = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
              bad += nonfinite_bf16x2(v.x) + nonfinite_bf16x2(v.y);
              *reinterpret_cast<uint2*>(
                  p.o + ((long long)(it.s.q0 + t) * p.Hq + h * p.group + (r - t * p.group)) * D + c4) = v;
            }
          }
        }
        if (!(ok = __all_sync(0xffffffffu, warps_sync()))) break;
      }
      if (!ok) break;
      report_nonfinite(bad, p.c.status, kOutO);
      // the CTA with an item's first step tells the joining kernel where its pieces are
      if (j0 == 0 && threadIdx.x == 0) {
        const int last_cta = (int)((u_blocks + steps - 1) / share);
        p.part_info[b * p.c.Hkv + h] = make_int4((int)blockIdx.x, last_cta, slot, 0);
      }
    }
  }
}

// Joins the pieces of split items: out = sum_i w_i o_i, w_i = exp(lse_i - lse), lse = log sum exp(lse_i).
// A warp per row, four rows per CTA.  The first piece is in the slot that its CTA recorded, the others
// are the first pieces of the CTAs that follow.  A programmatic launch: its CTAs start where the pieces' CTAs
// have ended (none of those triggers before), and what they read of the pieces comes after the wait.
template <int D>
__global__ void __launch_bounds__(128) fa_rows_combine(const Attn p, int slot_rows) {
  const int groups = slot_rows / 4;
  const int item = blockIdx.x / groups, b = item / p.c.Hkv, h = item - b * p.c.Hkv;
  const RowsItem it(p, b);
  const int r = (blockIdx.x % groups) * 4 + threadIdx.x / 32, lane = threadIdx.x % 32;
  // before any exit: the launch that follows this one must find the pieces' kernel complete
  cudaGridDependencySynchronize();
  if (it.w.steps == 0 || r >= it.rows) return;
  const int4 info = p.part_info[item];
  // a launch that gave up (a wait that ran out) may have left the record unwritten
  if (info.x < 0 || info.y < info.x || info.y >= kRowsMaxCtas || (info.z >> 1) != info.x) {
    if (lane == 0) report_bounds(p.c.status, kSitePagedPieces, info.x);
    return;
  }
  const int pieces = info.y - info.x + 1;
  if (pieces < 2) return;
  constexpr int kPer = D / 32;   // columns per lane: 2 or 4
  auto row_of = [&](int i) { return (i == 0 ? (long long)info.z : 2ll * (info.x + i)) * slot_rows + r; };
  float top = -INFINITY;
  for (int i = lane; i < pieces; i += 32) top = fmaxf(top, p.part_lse[row_of(i)]);
#pragma unroll
  for (int off = 16; off > 0; off /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  const float tu = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int i = 0; i < pieces; ++i) {
    const long long row = row_of(i);
    const float w = ex2_approx((p.part_lse[row] - tu) * 1.4426950408889634f);
    const float* src = p.part_o + row * D + lane * kPer;
    sum += w;
    if constexpr (kPer == 4) {
      const float4 x = *reinterpret_cast<const float4*>(src);
      acc[0] = fmaf(w, x.x, acc[0]);
      acc[1] = fmaf(w, x.y, acc[1]);
      acc[2] = fmaf(w, x.z, acc[2]);
      acc[3] = fmaf(w, x.w, acc[3]);
    } else {
      const float2 x = *reinterpret_cast<const float2*>(src);
      acc[0] = fmaf(w, x.x, acc[0]);
      acc[1] = fmaf(w, x.y, acc[1]);
    }
  }
  const bool empty = top == -INFINITY && sum == 0.f;
  const float inv = empty ? 0.f : 1.f / sum;
  const int t = r / p.group;
  const long long row = (long long)(it.s.q0 + t) * p.Hq + h * p.group + (r - t * p.group);
  uint32_t w2[kPer / 2], bad = 0;
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e) {
    w2[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    bad += nonfinite_bf16x2(w2[e]);
  }
  if constexpr (kPer == 4)
    *reinterpret_cast<uint2*>(p.o + row * D + lane * 4) = make_uint2(w2[0], w2[1]);
  else
    *reinterpret_cast<uint32_t*>(p.o + row * D + lane * 2) = w2[0];
  report_nonfinite(bad, p.c.status, kOutO);
  const float lse = empty ? -INFINITY : top + logf(sum);
  report_nonfinite((lane == 0 && !empty && !(fabsf(lse) < INFINITY)) ? 1u : 0u, p.c.status, kOutLse);
  if (lane == 0 && p.lse) p.lse[row] = lse;
}

// A launch that may start before the one before it in the stream has ended.
template <typename... Args, typename... Given>
static cudaError_t launch_early(void (*kern)(Args...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                                const Given&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, bool kFp8, int kRG, int kNR>
static int launch(const CUtensorMap& tk, const CUtensorMap& tv, const Attn& p, int grid, bool beside, cudaStream_t s) {
  using C = RowsCfg<D, kFp8>;
  auto kern = fa_rows_kernel<D, kFp8, kRG, kNR>;
  static std::atomic<uint64_t> prepared{0};
  int rc = prepare_kernel(reinterpret_cast<const void*>(kern), C::kSmemBytes, kRowsThreads,
                          128 * (kRowsRegCompute + kRowsRegLoad), "few-rows kernel", &prepared);
  if (rc) return rc;
  if (beside)
    return check_cuda(launch_early(kern, grid, kRowsThreads, C::kSmemBytes, s, tk, tv, p), "launch fa_rows_kernel");
  kern<<<grid, kRowsThreads, C::kSmemBytes, s>>>(tk, tv, p);
  return check_cuda(cudaGetLastError(), "launch fa_rows_kernel");
}

template <int D, bool kFp8>
static int launch_groups(const CUtensorMap& tk, const CUtensorMap& tv, const Attn& p, int grid, bool beside,
                         cudaStream_t s) {
  if (p.few_rows == 8) return launch<D, kFp8, 1, 1>(tk, tv, p, grid, beside, s);
  if (p.few_rows == 16) return launch<D, kFp8, 1, 2>(tk, tv, p, grid, beside, s);
  if (p.few_rows == 32) return launch<D, kFp8, 2, 2>(tk, tv, p, grid, beside, s);
  return launch<D, kFp8, 4, 2>(tk, tv, p, grid, beside, s);
}

// beside: after a chunk kernel of the same call, without waiting for it.
int launch_rows(const Attn& p, int d, bool fp8, bool beside, cudaStream_t s) {
  const int page_size = 1 << p.c.page_shift, box = page_size < kRowsBlk ? page_size : kRowsBlk;
  CUtensorMap tk, tv;
  int rc;
  if ((rc = make_tmap_pages(&tk, p.c.k, fp8, d, page_size, p.c.Hkv, p.c.num_pages, p.c.page_stride, box)) ||
      (rc = make_tmap_pages(&tv, p.c.v, fp8, d, page_size, p.c.Hkv, p.c.num_pages, p.c.page_stride, box)))
    return rc;
  int grid = 2 * sm_count();
  if (grid > kRowsMaxCtas) grid = kRowsMaxCtas;
  if (d == 64)
    return fp8 ? launch_groups<64, true>(tk, tv, p, grid, beside, s) : launch_groups<64, false>(tk, tv, p, grid, beside, s);
  return fp8 ? launch_groups<128, true>(tk, tv, p, grid, beside, s) : launch_groups<128, false>(tk, tv, p, grid, beside, s);
}

int launch_rows_combine(const Attn& p, int d, cudaStream_t s) {
  const unsigned grid = (unsigned)(p.c.B * p.c.Hkv * (p.few_rows / 4));
  return check_cuda(launch_early(d == 64 ? fa_rows_combine<64> : fa_rows_combine<128>, grid, 128, 0, s, p, p.few_rows),
                    "launch fa_rows_combine");
}

}  // namespace paged
}  // namespace fa
