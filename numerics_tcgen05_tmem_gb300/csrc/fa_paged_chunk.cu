// Paged attention for chunks of new tokens: sequences with more rows for a kv head than the few-rows
// kernel takes.
//
// The products dominate here, so they run on the tensor core as in the dense forward: two tiles of
// 128 rows per CTA against a shared stream of 128-key blocks, S and O in tensor memory, P~ fed back
// from tensor memory, one softmax warpgroup per tile, a correction warpgroup, one MMA thread.
//   * A tile's rows are (token, head of the group) pairs of one kv head, 128 / group tokens of
//     `group` rows each: TMA brings Q in that order from the packed rows (a box of group heads by
//     tokens), and K and V are read once for the whole group.  With a group that does not divide 128
//     the last rows of a tile stay unused.
//   * K and V blocks come page by page.  E4M3 codes land in slots of their own, from which a warpgroup
//     multiplies them by their vector's scale and writes the BF16 operand tiles (exact for power-of-two
//     scales) beside the softmax.  Where enough tiles read each key, kv_copy_kernel does that once, into
//     BF16 pages in the workspace, and this kernel reads those (copy_pays).
//   * With rows for one tile only the tensor core would wait for each block's softmax and the softmax for
//     each product.  Both warpgroups then work on that tile: one on the even blocks, the other on the odd
//     ones, each with its own running maximum, sum and O, joined at the end (a mixed batch of eight
//     sequences, E4M3, window 1024: 45 us with one chain, 37 with two).
//   * V rows that no row of the CTA sees (slots behind the sequence's end, keys before the window)
//     may hold anything, and 0 * NaN is NaN: they are zeroed in shared memory before the product.
//   * The tiles that are left after whole rounds of one CTA per SM would leave SMs idle: their keys are
//     split over several CTAs, whose normalised FP32 results fa_chunk_combine joins (in order, whatever
//     the timing).
// Softmax: running maximum and sum in FP32 per row (one thread per row), P~ rounded to BF16 for the
// product as the tensor core takes it.  Plain shift: the stabilised rule guards the training
// backward, and the output does not depend on the shift.
#include <stdlib.h>

#include <algorithm>

#include "paged_attn.cuh"

namespace fa {
namespace paged {

constexpr int kM = 128;             // rows per tile (TMEM lanes)
constexpr int kN = 128;             // keys per block
constexpr int kStages = 2;
constexpr int kSplitSteps = 4;      // fewest key blocks worth a split of their own

template <int D, bool kFp8>
struct ChunkCfg {
  static constexpr int kThreads = kFp8 ? 640 : 512;
  static constexpr int kMmaWarp = 12, kLoadWarp = 13, kGuardWarp = 14, kConvertWarp = 16;
  // registers per thread after the launch: softmax, correction, MMA/TMA, conversion
  static constexpr int kRegLaunch = kFp8 ? 96 : 128;
  static constexpr int kRegSoftmax = kFp8 ? 160 : 176, kRegCorr = kFp8 ? 48 : 96, kRegOther = kFp8 ? 40 : 56,
                       kRegConvert = 72;
  static constexpr int kSplit =
      256 * kRegSoftmax + 128 * kRegCorr + 128 * kRegOther + (kFp8 ? 128 * kRegConvert : 0);
  static_assert(kSplit <= kThreads * kRegLaunch, "register split exceeds the launch allocation");
  static constexpr int kAtoms = D / 64;              // 128-byte column blocks of a BF16 tile
  static constexpr int kAtomBlock = 128 * 128;       // bytes of one
  static constexpr int kTileBytes = kAtoms * kAtomBlock;
  static constexpr int kQOff = 0, kKOff = 2 * kTileBytes, kVOff = kKOff + kStages * kTileBytes;
  // E4M3: slots for the codes of a tile (K and V of a block in turn) and their vectors' scales; at
  // d = 128 two fill what the tiles leave
  static constexpr int kSlots = kFp8 ? (D == 128 ? 2 : 4) : 0;
  static constexpr int kCodeOff = kVOff + kStages * kTileBytes, kCodeBytes = kN * D;
  static constexpr int kScaleOff = kCodeOff + kSlots * kCodeBytes;
  static constexpr int kBarOff = kScaleOff + kSlots * kN * 4;
  static constexpr uint32_t kTmemO = 256;            // S0 | S1 | O0 | O1
  static constexpr uint32_t kIdescS = idesc_bf16(128, kN, false, false);
  static constexpr uint32_t kIdescO = idesc_bf16(128, D, false, true);
};

constexpr int kMaxSlots = 4;

struct ChunkShared {
  uint64_t q_full, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  // a V block with unseen rows: the MMA thread, which has seen it land, asks for the zeroing and
  // waits for it (one request at a time, so the parities cannot alias)
  uint64_t v_dirty, v_clean;
  uint64_t code_full[kMaxSlots], code_empty[kMaxSlots];   // E4M3: a slot has landed / has been read
  uint64_t s_full[2], p_half[2], p_full[2], pv_done[2], o_done[2], alpha_ready[2], o_ready[2], l_ready[2];
  uint64_t mma_done;
  uint64_t never;                  // test builds only: a barrier nothing arrives on
  float alpha[2][kM];
  uint32_t tmem_base, abort_flag;
  int b, tile;                     // this CTA's sequence and pair of tiles; b = -1: none
};

template <int D, bool kFp8>
constexpr int chunk_smem() {
  return ChunkCfg<D, kFp8>::kBarOff + (int)sizeof(ChunkShared);
}
static_assert(chunk_smem<128, true>() <= 227 * 1024, "shared-memory layout exceeds 227 KB");

// The work of one CTA: a pair of tiles of sequence b for kv head h, steps [js, je) of its walk.
struct ChunkWork {
  Seq s;
  int tok0, tokens;      // first token of the pair, tokens per tile
  int last;              // position of its last token
  int splits;            // pieces that the pair's keys are split into
  KeyWalk<kN> w;
  __device__ __forceinline__ ChunkWork(const Attn& p, int b, int tile, int max_splits)
      : s(load_seq(p, b)),
        tokens(kM / p.group),
        w(p, s.pos0 + tile * 2 * (kM / p.group), s.pos0 + min((tile + 1) * 2 * (kM / p.group), s.n) - 1) {
    tok0 = tile * 2 * tokens;
    last = s.pos0 + min(tok0 + 2 * tokens, s.n) - 1;
    splits = min(max_splits, max(1, w.steps / kSplitSteps));
  }
  // steps of tile t alone: up to the block of its last token
  __device__ __forceinline__ int steps(int t) const {
    const int t0 = tok0 + t * tokens;
    if (t0 >= s.n) return 0;
    const int hi = max(s.pos0 + min(t0 + tokens, s.n), 0);
    return max(w.n_sink + (hi + kN - 1) / kN - w.b_lo, 1);
  }
};

__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// How the launch's tiles (pair of tiles, kv head) are dealt: the first `whole` to one CTA each, every
// other one to `splits` CTAs that take a share of its keys.
struct ChunkGrid {
  int whole, splits;
};

// Pairs of tiles of sequence b that are the chunk kernel's.
__device__ __forceinline__ int chunk_tiles(const Attn& p, int b) {
  const int n = load_seq(p, b).n, per = 2 * (kM / p.group);
  return n * p.group <= p.few_rows ? 0 : (n + per - 1) / per;
}

// The sequence and pair of tiles that is number `want` of the launch (-1: none), 32 sequences at a
// time; a sequence's last (longest) tiles come first.  The whole warp calls it.
__device__ __forceinline__ void find_tiles(const Attn& p, int want, int& found, int& tile) {
  const int lane = threadIdx.x % 32;
  found = -1;
  tile = 0;
  for (int b0 = 0; b0 < p.c.B && found < 0; b0 += 32) {
    const int mine = b0 + lane < p.c.B ? chunk_tiles(p, b0 + lane) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, want < incl);
    const int at = hit ? __ffs(hit) - 1 : 31;
    const int upto = __shfl_sync(0xffffffffu, incl, at), n = __shfl_sync(0xffffffffu, mine, at);
    if (hit) {
      found = b0 + at;
      tile = n - 1 - (want - (upto - n));
    } else {
      want -= upto;
    }
  }
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(ChunkCfg<D, kFp8>::kThreads, 1)
    fa_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const Attn p, const ChunkGrid g) {
  using C = ChunkCfg<D, kFp8>;
  // a few-rows launch of the same call, which touches none of this one's rows, may run beside it
  cudaTriggerProgrammaticLaunchCompletion();
  extern __shared__ __align__(1024) uint8_t smem[];
  // the swizzled tiles need a 1024-byte aligned base (there is no slack for E4M3, d = 128)
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) report_bounds(p.c.status, kSiteSmemAlign, (long long)smem_u32(smem));
    return;
  }
  ChunkShared& sh = *reinterpret_cast<ChunkShared*>(smem + C::kBarOff);
  volatile uint32_t* abort_flag = &sh.abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // blockIdx.x = (pair of tiles, kv head, split), split fastest
  const int extra = (int)blockIdx.x - g.whole;   // number among the split tiles' CTAs; negative: a whole tile
  const int max_splits = extra < 0 ? 1 : g.splits;
  const int split = extra < 0 ? 0 : extra % g.splits;
  const int unit = extra < 0 ? (int)blockIdx.x : g.whole + extra / g.splits;
  const int h = unit % p.c.Hkv;

  if (warp == 0) {
    int found, tile;
    find_tiles(p, unit / p.c.Hkv, found, tile);
    if (lane == 0) {
      sh.b = found;
      sh.tile = tile;
    }
  }
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    mbar_init(&sh.q_full, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh.k_full[s], kFp8 ? 128 : 1);
      mbar_init(&sh.k_empty[s], 1);
      mbar_init(&sh.v_full[s], kFp8 ? 128 : 1);
      mbar_init(&sh.v_empty[s], 1);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&sh.code_full[s], 1);
      mbar_init(&sh.code_empty[s], 128);
    }
    mbar_init(&sh.v_dirty, 1);
    mbar_init(&sh.v_clean, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.p_half[t], kM);
      mbar_init(&sh.p_full[t], kM);
      mbar_init(&sh.pv_done[t], 1);
      mbar_init(&sh.o_done[t], 1);
      mbar_init(&sh.alpha_ready[t], kM);
      mbar_init(&sh.o_ready[t], kM);
      mbar_init(&sh.l_ready[t], kM);
    }
    mbar_init(&sh.mma_done, 1);
    mbar_init(&sh.never, 1);
    fence_barrier_init();
  }
  __syncthreads();
  const int b = sh.b;
  if (b < 0) return;
  const ChunkWork wk(p, b, sh.tile, max_splits);
  if (split >= wk.splits) return;
  const int js = (int)((long long)wk.w.steps * split / wk.splits);
  const int je = (int)((long long)wk.w.steps * (split + 1) / wk.splits);
  // steps of this CTA for each tile (0 where the tile ends before the piece)
  const int nbmax = je - js;
  // rows for one tile only: chain t (its warpgroup, S and O) takes the blocks 2 i + t of that tile
  const bool dual = wk.steps(1) == 0 && nbmax > 1;
  const int nb0 = dual ? (nbmax + 1) / 2 : max(0, min(je, wk.steps(0)) - js);
  const int nb1 = dual ? nbmax / 2 : max(0, min(je, wk.steps(1)) - js);
  // block of step i of tile (or chain) t
  auto block = [&](int t, int i) { return dual ? 2 * i + t : i; };
  // the rows' sums for the last step, +inf for rows that saw nothing (O / l = 0), and with two chains
  // their maxima: in the tile's Q, which its last S has read by then (two chains: in the unused tile)
  auto fin = [&](int t) {
    return reinterpret_cast<float*>(smem + C::kQOff + (dual ? C::kTileBytes + t * 2 * kM * 4 : t * C::kTileBytes));
  };
  // whether the block at `key` has rows that no row of the CTA sees
  auto unseen = [&](int key) {
    return key + kN > wk.w.hi || (key < wk.w.lo && key + kN > wk.w.sinks);
  };

  if (warp == C::kMmaWarp) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  if (kFp8 && warp >= C::kConvertWarp) {
    if constexpr (kFp8) {
    // ------------------------------------------------------------ E4M3 -> BF16 operand tiles
    // D / 16 neighbouring threads take one key's row, 16 codes each; a thread has D / 16 rows.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegConvert));
    constexpr int kPer = D / 16, kRowStep = 128 / kPer;
    const int r0 = (threadIdx.x - 32 * C::kConvertWarp) / kPer, x = threadIdx.x % kPer;
    // a row's 16 codes become two 16-byte chunks of a 64-column block, swizzled; the second block's
    // threads take theirs in the other order, so that a row's threads meet different banks
    const int flip = x / 4;
    const uint32_t c0 = (uint32_t)((x / 4) * C::kAtomBlock + r0 * 128 + ((((x % 4) * 2 + flip) ^ (r0 & 7)) << 4));
    const uint32_t c1 = (uint32_t)((x / 4) * C::kAtomBlock + r0 * 128 + ((((x % 4) * 2 + 1 - flip) ^ (r0 & 7)) << 4));
    static_assert(kRowStep % 8 == 0, "a thread's rows share one swizzle phase");
    bool ok = true;
    int n = 0;   // tiles converted
    for (int step = 0; ok && step <= nbmax; ++step) {
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const int j = step - kv;   // K of block `step`, then V of the block before
        if (j < 0 || j >= nbmax) continue;
        const int s = j % kStages, key0 = wk.w.at(js + j);
        const bool gaps = unseen(key0);
        const uint32_t tile = smem_u32(smem) + (kv ? C::kVOff : C::kKOff) + s * C::kTileBytes;
        const int slot = n % C::kSlots;
        if (!(ok = mbar_wait(&sh.code_full[slot], (n / C::kSlots) & 1, abort_flag, p.c.status))) break;
        uint4 codes[kPer];
        float scale[kPer];
        const uint4* src = reinterpret_cast<const uint4*>(smem + C::kCodeOff + slot * C::kCodeBytes + r0 * D) + x;
        const float* sc = reinterpret_cast<const float*>(smem + C::kScaleOff) + slot * kN + r0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          codes[i] = src[i * kRowStep * D / 16];
          scale[i] = sc[i * kRowStep];
        }
        if (gaps) {  // slots that no row sees may hold anything
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (!wk.w.seen(key0 + i * kRowStep + r0)) {
              codes[i] = make_uint4(0, 0, 0, 0);
              scale[i] = 0.f;
            }
        }
        mbar_arrive(&sh.code_empty[slot]);
        // the products that read this stage's previous tile are done
        if (!(ok = mbar_wait(kv ? &sh.v_empty[s] : &sh.k_empty[s], ((j / kStages) & 1) ^ 1, abort_flag, p.c.status))) break;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const uint32_t w[4] = {flip ? codes[i].z : codes[i].x, flip ? codes[i].w : codes[i].y,
                                 flip ? codes[i].x : codes[i].z, flip ? codes[i].y : codes[i].w};
          uint4 o[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t y[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 f = e4m3x2_to_float2(w[2 * e + q / 2] >> (16 * (q & 1)));
              float a, c;
              mul2(a, c, f.x, f.y, scale[i], scale[i]);
              y[q] = pack_bf16x2(a, c);
            }
            o[e] = make_uint4(y[0], y[1], y[2], y[3]);
          }
          sts128(tile + c0 + i * kRowStep * 128, o[0]);
          sts128(tile + c1 + i * kRowStep * 128, o[1]);
        }
        fence_proxy_async_smem();
        mbar_arrive(kv ? &sh.v_full[s] : &sh.k_full[s]);
        ++n;
      }
    }
    }
  } else if (warp >= C::kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegOther));
    if (warp == C::kLoadWarp) {
      // ---------------------------------------------------------- loads: Q, and K and V page by page
      const uint32_t base = smem_u32(smem);
      const int ntiles = nb1 > 0 && !dual ? 2 : 1;
      if (elect_one()) {
        tma_prefetch_desc(&tmQ);
        mbar_arrive_expect_tx(&sh.q_full, ntiles * wk.tokens * p.group * 128 * C::kAtoms);
        for (int t = 0; t < ntiles; ++t)
          for (int c = 0; c < C::kAtoms; ++c)
            tma_load_3d(smem + C::kQOff + t * C::kTileBytes + c * C::kAtomBlock, &tmQ, &sh.q_full, c * 64, h * p.group,
                        wk.s.q0 + wk.tok0 + t * wk.tokens);
      }
      __syncwarp();
      {
        const int page_size = 1 << p.c.page_shift;
        const int box = min(page_size, kN), ppb = kN / box, per_group = 32 / ppb;
        int nk = 0, nv = 0, n = 0;   // K and V tiles, or slots of codes, loaded
        bool ok = true;
        // K of block j, then V of the block before it: a K load never waits behind the V of a block
        // whose P~ V has yet to free the stage
        int v_page = 0, v_slot = 0;   // of the block before
        for (int jg = 0; ok && jg <= nbmax; jg += per_group) {
          const int jl = jg + lane / ppb;
          int page = p.c.num_pages;  // out of range: zeros
          if (jl < nbmax) {
            const int key = wk.w.at(js + jl) + (lane % ppb) * box;
            if (wk.w.any(key, box)) {
              const int x = find_page(p.c, b, key, kSitePagedPage);
              if (x >= 0) page = x;
            }
          }
          for (int jj = 0; ok && jj < per_group && jg + jj <= nbmax; ++jj) {
            const int k_page = __shfl_sync(0xffffffffu, page, jj * ppb + lane % ppb);
            const int k_slot = jg + jj < nbmax ? (wk.w.at(js + jg + jj) + lane * box) & (page_size - 1) : 0;
            for (int kv = 0; kv < 2; ++kv) {
              const int j = jg + jj - kv, s = j & (kStages - 1);
              if (j < 0 || j >= nbmax) continue;
              const int pg = kv ? v_page : k_page, slot = kv ? v_slot : k_slot;
              const CUtensorMap* map = kv ? &tmV : &tmK;
              if constexpr (kFp8) {
                const bool real = lane < ppb && pg < p.c.num_pages;
                const int scaled = __popc(__ballot_sync(0xffffffffu, real));
                const int x = n % C::kSlots;
                ok = __all_sync(0xffffffffu, mbar_wait(&sh.code_empty[x], ((n / C::kSlots) & 1) ^ 1, abort_flag, p.c.status));
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&sh.code_full[x], C::kCodeBytes + scaled * box * 4);
                __syncwarp();
                if (lane < ppb)
                  tma_load_page(base + C::kCodeOff + x * C::kCodeBytes + lane * box * D, map, &sh.code_full[x], 0, slot, h, pg);
                if (real)
                  bulk_load(smem + C::kScaleOff + (x * kN + lane * box) * 4,
                            (kv ? p.c.v_scale : p.c.k_scale) + pg * p.c.scale_stride + (long long)h * page_size + slot, box * 4,
                            &sh.code_full[x]);
                ++n;
              } else {
                uint64_t* full = kv ? &sh.v_full[s] : &sh.k_full[s];
                ok = __all_sync(0xffffffffu, mbar_wait(kv ? &sh.v_empty[s] : &sh.k_empty[s], ((j / kStages) & 1) ^ 1,
                                                       abort_flag, p.c.status));
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(full, C::kTileBytes);
                __syncwarp();
                const uint32_t tile = base + (kv ? C::kVOff : C::kKOff) + s * C::kTileBytes + lane * box * 128;
                if (lane < ppb)
                  for (int c = 0; c < C::kAtoms; ++c)
                    tma_load_page(tile + c * C::kAtomBlock, map, full, c * 64, slot, h, pg);
                (kv ? nv : nk) = j + 1;
              }
            }
            v_page = k_page;
            v_slot = k_slot;
          }
        }
        if (*abort_flag) {
          // let copies still in flight land before the CTA's shared memory goes away
          volatile uint32_t ignore_abort = 0;
          for (int j = max(0, nk - kStages); j < nk; ++j)
            mbar_wait(&sh.k_full[j % kStages], (j / kStages) & 1, &ignore_abort, p.c.status);
          for (int j = max(0, nv - kStages); j < nv; ++j)
            mbar_wait(&sh.v_full[j % kStages], (j / kStages) & 1, &ignore_abort, p.c.status);
          if constexpr (kFp8)
            for (int i = max(0, n - C::kSlots); i < n; ++i)
              mbar_wait(&sh.code_full[i % C::kSlots], (i / C::kSlots) & 1, &ignore_abort, p.c.status);
        }
      }
      if (*abort_flag) {
        volatile uint32_t ignore_abort = 0;
        mbar_wait(&sh.q_full, 0, &ignore_abort, p.c.status);
      }
    } else if (warp == C::kGuardWarp) {
      // ---------------------------------------------------------- zero V rows that no row sees
      if constexpr (!kFp8) {
        bool ok = true;
        int n = 0;
        for (int j = 0; ok && j < nbmax; ++j) {
          const int key0 = wk.w.at(js + j), s = j % kStages;
          if (!unseen(key0)) continue;
          ok = __all_sync(0xffffffffu, mbar_wait(&sh.v_dirty, n++ & 1, abort_flag, p.c.status));
          if (!ok) break;
          for (int r = lane; r < kN; r += 32) {
            if (wk.w.seen(key0 + r)) continue;
            uint8_t* row = smem + C::kVOff + s * C::kTileBytes + r * 128;
#pragma unroll
            for (int x = 0; x < C::kAtoms * 8; ++x)   // a lane's chunks in an order that spreads the banks
              *reinterpret_cast<uint4*>(row + (x / 8) * C::kAtomBlock + ((x ^ lane) & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.v_clean);
        }
      }
    } else if (warp == C::kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer
      if (elect_one()) {
        const uint32_t sQ = smem_u32(smem + C::kQOff), sK = smem_u32(smem + C::kKOff), sV = smem_u32(smem + C::kVOff);
        const int nb[2] = {nb0, nb1};
        bool ok = mbar_wait(&sh.q_full, 0, abort_flag, p.c.status);
#ifdef FA_TEST_HOOKS
        // failure-detection test: as in the few-rows kernel
        if (p.inject_stall) ok = ok && mbar_wait(&sh.never, 0, abort_flag, p.c.status);
#endif
        tc_fence_after();
        int cleaned = 0;  // V blocks that had rows zeroed
        auto issue_s = [&](int t, int s) {
          const uint32_t a0 = sQ + (dual ? 0 : t * C::kTileBytes), b0 = sK + s * C::kTileBytes;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk / 4) * C::kAtomBlock + (kk % 4) * 32;
            mma_ss(tmem + t * 128, sdesc_sw128(a0 + off, 16, 1024), sdesc_sw128(b0 + off, 16, 1024), C::kIdescS, kk > 0);
          }
          tc_commit(&sh.s_full[t]);
        };
        auto issue_pv = [&](int t, int s, int j, int k_lo, int k_hi) {
          const uint32_t d = tmem + C::kTmemO + t * D, b0 = sV + s * C::kTileBytes;
#pragma unroll
          for (int kk = k_lo; kk < k_hi; ++kk)
            mma_ts(d, tmem + t * 128 + kk * 8, sdesc_sw128(b0 + kk * 2048, C::kAtomBlock, 1024), C::kIdescO,
                   (j > 0 || kk > 0) ? 1u : 0u);
          if (k_hi == kN / 16) {
            tc_commit(&sh.pv_done[t]);
            if (j == nb[t] - 1) tc_commit(&sh.o_done[t]);
          }
        };
        // S0_0 S1_0 | PV0_0 S0_1 PV1_0 S1_1 | ... ; P~ V in two halves over the keys, the first as
        // soon as the softmax has stored it.  Two chains on one tile: S0_0 | S1_1 | PV0_0 S0_2 |
        // PV1_1 S1_3 | ... (chain _ block), each block's P~ V two blocks later.
        const int lag = dual ? 2 : 1;
        for (int j = 0; ok && j < nbmax + lag; ++j) {
          const int s = j % kStages, jp = j - lag, sp = jp & (kStages - 1);   // block jp's P~ V
          const bool has_s = j < nbmax, has_pv = jp >= 0 && jp < nbmax;
          if (has_s) {
            if (!(ok = mbar_wait(&sh.k_full[s], (j / kStages) & 1, abort_flag, p.c.status))) break;
            tc_fence_after();
          }
          if (has_pv) {
            if (!(ok = mbar_wait(&sh.v_full[sp], (jp / kStages) & 1, abort_flag, p.c.status))) break;
            if (!kFp8 && unseen(wk.w.at(js + jp))) {
              mbar_arrive(&sh.v_dirty);
              if (!(ok = mbar_wait(&sh.v_clean, cleaned++ & 1, abort_flag, p.c.status))) break;
            }
            tc_fence_after();
          }
          for (int t = 0; t < 2; ++t) {
            if (dual && t != (j & 1)) continue;
            const int i = dual ? j / 2 : j, ip = i - 1;   // the tile's (chain's) step, and the one whose P~ V is due
            if (has_pv && ip < nb[t]) {
              if (!(ok = mbar_wait(&sh.p_half[t], ip & 1, abort_flag, p.c.status))) break;
              if (ip > 0 && !(ok = mbar_wait(&sh.o_ready[t], (ip - 1) & 1, abort_flag, p.c.status))) break;
              tc_fence_after();
              issue_pv(t, sp, ip, 0, kN / 32);
              if (!(ok = mbar_wait(&sh.p_full[t], ip & 1, abort_flag, p.c.status))) break;
              tc_fence_after();
              issue_pv(t, sp, ip, kN / 32, kN / 16);
            }
            if (has_s && i < nb[t]) issue_s(t, s);
          }
          if (!ok) break;
          if (has_s) tc_commit(&sh.k_empty[s]);
          if (has_pv) tc_commit(&sh.v_empty[sp]);
        }
        tc_commit(&sh.mma_done);
        {
          // MMAs still in flight must finish before TMEM is released, even after an abort
          volatile uint32_t ignore_abort = 0;
          mbar_wait(&sh.mma_done, 0, &ignore_abort, p.c.status);
        }
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax warpgroups
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegSoftmax));
    const int t = warp / 4, r = (warp % 4) * 32 + lane;
    const int nb = t == 0 ? nb0 : nb1;
    const int tr = r / p.group, tok = wk.tok0 + (dual ? 0 : t * wk.tokens) + tr;
    const bool valid = tr < wk.tokens && tok < wk.s.n;
    // rows past the last token count as that token's: nothing of theirs is stored, and they must not
    // send their warp through the masked path in every block
    const int pos = valid ? wk.s.pos0 + tok : wk.last;
    const bool idle = !__any_sync(0xffffffffu, valid);   // no row of the warp: only keeps the barriers going
    const uint32_t tS = tmem + t * 128 + ((uint32_t)((warp % 4) * 32) << 16);
    const float c = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nb; ++j) {
      if (!(ok = mbar_wait(&sh.s_full[t], j & 1, abort_flag, p.c.status))) break;
      if (idle) {
        if (j > 0) {
          sh.alpha[t][r] = 1.f;
          mbar_arrive(&sh.alpha_ready[t]);
        }
        mbar_arrive(&sh.p_half[t]);
        mbar_arrive(&sh.p_full[t]);
        continue;
      }
      tc_fence_after();
      uint32_t raw[kN];
      float pmax[kN / 32];
#pragma unroll
      for (int c0 = 0; c0 < kN; c0 += 32)
        tmem_ld32_max(tS + c0, *reinterpret_cast<uint32_t(*)[32]>(raw + c0), pmax[c0 / 32]);
      tmem_ld_wait();
      reg_fence(raw);
      reg_fence(pmax);
      float sv[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) sv[i] = __uint_as_float(raw[i]);
      // mask: keys after the row's token, and keys before its window that are no sinks
      const int col0 = wk.w.at(js + block(t, j));
      const int lim = pos - col0 + 1, w_lo = p.window ? pos - p.window + 1 - col0 : 0, s_hi = p.sinks - col0;
      const bool open = lim >= kN && (w_lo <= 0 || s_hi >= kN);
      float bm;
      if (__all_sync(0xffffffffu, open)) {
        bm = fmaxf(max3f(pmax[0], pmax[1], pmax[2]), pmax[3]);
      } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) sv[i] = (i < lim && (i >= w_lo || i < s_hi)) ? sv[i] : -INFINITY;
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kN; i += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3f(mx[e], sv[i + 2 * e], sv[i + 2 * e + 1]);
        bm = fmaxf(max3f(mx[0], mx[1], mx[2]), mx[3]);
      }
      const float m_new = fmaxf(m, bm);
      const float mu = m_new == -INFINITY ? 0.f : m_new;   // nothing seen yet
      const float alpha = ex2_approx((m - mu) * c);
      m = m_new;
      if (j > 0) {
        sh.alpha[t][r] = alpha;
        mbar_arrive(&sh.alpha_ready[t]);
      }
      const float nmc = -mu * c;
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float x0, x1;
          fma2(x0, x1, sv[half * 64 + i], sv[half * 64 + i + 1], c, c, nmc, nmc);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          add2(sum0, sum1, sum0, sum1, p0, p1);
          pk[i / 2] = pack_bf16x2(p0, p1);
        }
        __syncwarp();
        tmem_st32(tS + half * 32, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(half == 0 ? &sh.p_half[t] : &sh.p_full[t]);
      }
      l = l * alpha + (sum0 + sum1);
    }
    if (ok) {
      const bool empty = m == -INFINITY && l == 0.f;  // no visible key in this piece (a NaN score is not that)
      fin(t)[r] = empty && !dual ? INFINITY : l;
      if (dual) fin(t)[kM + r] = m;
      mbar_arrive(&sh.l_ready[t]);
      const float lse = empty ? -INFINITY : m * p.scale + logf(l);
      const long long row = (long long)(wk.s.q0 + tok) * p.Hq + h * p.group + (r - tr * p.group);
      if (valid && !dual) {
        if (wk.splits > 1)
          p.part_lse[(long long)extra * (2 * kM) + t * kM + r] = lse;
        else if (p.lse)
          p.lse[row] = lse;
      }
      if (wk.splits == 1 && !dual)
        report_nonfinite((valid && !empty && !(fabsf(lse) < INFINITY)) ? 1u : 0u, p.c.status, kOutLse);
    }
  } else {
    // ------------------------------------------------------------ correction warpgroup
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegCorr));
    const int r = (warp % 4) * 32 + lane;
    const uint32_t tO = tmem + C::kTmemO + ((uint32_t)((warp % 4) * 32) << 16);
    const int nb[2] = {nb0, nb1};
    bool ok = true;
    for (int j = 1; ok && j < max(nb0, nb1); ++j) {
      for (int t = 0; t < 2; ++t) {
        if (j >= nb[t]) continue;
        if (!(ok = mbar_wait(&sh.alpha_ready[t], (j - 1) & 1, abort_flag, p.c.status))) break;
        const float alpha = sh.alpha[t][r];
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
          if (!(ok = mbar_wait(&sh.pv_done[t], (j - 1) & 1, abort_flag, p.c.status))) break;
          tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t w[32];
            tmem_ld32(tO + t * D + c0, w);
            tmem_ld_wait();
            reg_fence(w);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float a0, a1;
              mul2(a0, a1, __uint_as_float(w[i]), __uint_as_float(w[i + 1]), alpha, alpha);
              w[i] = __float_as_uint(a0);
              w[i + 1] = __float_as_uint(a1);
            }
            tmem_st32(tO + t * D + c0, w);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(&sh.o_ready[t]);
      }
    }
    // Two chains: their O weighted by exp(max - joint max) over the joint sum, and the row's lse
    if (ok && dual) {
      for (int t = 0; ok && t < 2; ++t)
        ok = mbar_wait(&sh.o_done[t], 0, abort_flag, p.c.status) && mbar_wait(&sh.l_ready[t], 0, abort_flag, p.c.status);
      if (ok) {
        tc_fence_after();
        const float m0 = fin(0)[kM + r], m1 = fin(1)[kM + r], top = fmaxf(m0, m1), tu = top == -INFINITY ? 0.f : top;
        float w0 = ex2_approx((m0 - tu) * p.scale_log2), w1 = ex2_approx((m1 - tu) * p.scale_log2);
        const float sum = fin(0)[r] * w0 + fin(1)[r] * w1;
        const bool empty = top == -INFINITY && sum == 0.f;
        const float lse = empty ? -INFINITY : top * p.scale + logf(sum);
        w0 = empty ? 0.f : w0 / sum;
        w1 = empty ? 0.f : w1 / sum;
        const int tr = r / p.group, tok = wk.tok0 + tr;
        const bool valid = tr < wk.tokens && tok < wk.s.n;
        const long long row = valid ? (long long)(wk.s.q0 + tok) * p.Hq + h * p.group + (r - tr * p.group) : 0;
        uint32_t bad = 0;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 16) {
          uint32_t x[16], y[16];
          tmem_ld16(tO + c0, x);
          tmem_ld16(tO + D + c0, y);
          tmem_ld_wait();
          reg_fence(x);
          reg_fence(y);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), w0, __uint_as_float(y[i]) * w1));
          if (wk.splits > 1) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + ((long long)extra * (2 * kM) + r) * D + c0);
            if (valid)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                dst[i] = make_float4(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1]), __uint_as_float(x[4 * i + 2]),
                                     __uint_as_float(x[4 * i + 3]));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              x[i] = pack_bf16x2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
              bad += nonfinite_bf16x2(x[i]);
            }
            uint4* dst = reinterpret_cast<uint4*>(p.o + row * D + c0);
            if (valid) {
              dst[0] = make_uint4(x[0], x[1], x[2], x[3]);
              dst[1] = make_uint4(x[4], x[5], x[6], x[7]);
            }
          }
        }
        if (valid && wk.splits > 1)
          p.part_lse[(long long)extra * (2 * kM) + r] = lse;
        else if (valid && p.lse)
          p.lse[row] = lse;
        if (wk.splits == 1) {
          report_nonfinite(valid ? bad : 0u, p.c.status, kOutO);
          report_nonfinite((valid && !empty && !(fabsf(lse) < INFINITY)) ? 1u : 0u, p.c.status, kOutLse);
        }
      }
    }
    // O / l, to the output or to this piece's partial result
    for (int t = 0; ok && !dual && t < 2; ++t) {
      if (nb[t] == 0) continue;
      if (!(ok = mbar_wait(&sh.o_done[t], 0, abort_flag, p.c.status))) break;
      if (!(ok = mbar_wait(&sh.l_ready[t], 0, abort_flag, p.c.status))) break;
      tc_fence_after();
      const float inv_l = 1.f / fin(t)[r];
      const int tr = r / p.group, tok = wk.tok0 + t * wk.tokens + tr;
      const bool valid = tr < wk.tokens && tok < wk.s.n;
      const long long row = valid ? (long long)(wk.s.q0 + tok) * p.Hq + h * p.group + (r - tr * p.group) : 0;
      uint32_t bad = 0;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t w[32];
        tmem_ld32(tO + t * D + c0, w);
        tmem_ld_wait();
        reg_fence(w);
        if (wk.splits > 1) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + ((long long)extra * (2 * kM) + t * kM + r) * D + c0);
          if (valid)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(__uint_as_float(w[4 * i]) * inv_l, __uint_as_float(w[4 * i + 1]) * inv_l,
                                   __uint_as_float(w[4 * i + 2]) * inv_l, __uint_as_float(w[4 * i + 3]) * inv_l);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.o + row * D + c0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[e] = pack_bf16x2(__uint_as_float(w[8 * i + 2 * e]) * inv_l, __uint_as_float(w[8 * i + 2 * e + 1]) * inv_l);
              bad += nonfinite_bf16x2(x[e]);
            }
            if (valid) dst[i] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      }
      if (wk.splits == 1) report_nonfinite(valid ? bad : 0u, p.c.status, kOutO);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Row `row` of the output from the `pieces` partial rows that are 2 kM apart from `base` on.
template <int D>
__device__ __forceinline__ void join_row(const Attn& p, long long base, int pieces, long long row, int lane) {
  constexpr int kPer = D / 32;
  const float mine = lane < pieces ? p.part_lse[base + lane * (2 * kM)] : -INFINITY;
  float top = mine;
#pragma unroll
  for (int off = 16; off > 0; off /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  const float tu = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int i = 0; i < pieces; ++i) {
    const float part = __shfl_sync(0xffffffffu, mine, i);
    if (part == -INFINITY) continue;  // saw nothing: its output may not have been written
    const float w = ex2_approx((part - tu) * 1.4426950408889634f);
    sum += w;
    const float* src = p.part_o + (base + i * (2 * kM)) * D + lane * kPer;
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

// Joins the pieces of tiles whose keys were split: 32 rows of a tile per CTA, four per warp.  A programmatic
// launch: it starts while the pieces are still being computed, or, with a few-rows launch between, where
// that one's CTAs have ended.
constexpr int kJoinRows = 32;

template <int D>
__global__ void __launch_bounds__(256) fa_chunk_combine(const Attn p, const ChunkGrid g) {
  // before any exit: the launch that follows this one must find the pieces' kernel complete
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x % 32;
  constexpr int kParts = 2 * kM / kJoinRows;
  const int unit = g.whole + blockIdx.x / kParts, h = unit % p.c.Hkv;
  int b, tile;
  find_tiles(p, unit / p.c.Hkv, b, tile);
  if (b < 0) return;
  const ChunkWork wk(p, b, tile, g.splits);
  const int pieces = wk.splits;
  if (pieces < 2) return;
  for (int i = threadIdx.x / 32; i < kJoinRows; i += 8) {
    const int x = (blockIdx.x % kParts) * kJoinRows + i, t = x / kM, r = x % kM, tr = r / p.group;
    const int tok = wk.tok0 + t * wk.tokens + tr;
    if (tr >= wk.tokens || tok >= wk.s.n) continue;   // the same for the whole warp
    const long long row = (long long)(wk.s.q0 + tok) * p.Hq + h * p.group + (r - tr * p.group);
    join_row<D>(p, (long long)(unit - g.whole) * g.splits * (2 * kM) + x, pieces, row, lane);
  }
}

template <int D, bool kFp8>
static int launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const Attn& p, int whole, int splits,
                  cudaStream_t s) {
  using C = ChunkCfg<D, kFp8>;
  auto kern = fa_chunk_kernel<D, kFp8>;
  static std::atomic<uint64_t> prepared{0};
  int rc = prepare_kernel(reinterpret_cast<const void*>(kern), chunk_smem<D, kFp8>(), C::kThreads, C::kSplit, "chunk kernel",
                          &prepared);
  if (rc) return rc;
  const long long tiles = chunk_pairs(p.T, p.c.B, p.group) * p.c.Hkv;
  const long long grid = whole + (tiles - whole) * splits;
  if (grid >= (1ll << 31)) return set_error(FA_ERR_INVALID_ARG, "too many tiles for one launch");
  const ChunkGrid g{whole, splits};
  kern<<<(unsigned)grid, C::kThreads, chunk_smem<D, kFp8>(), s>>>(tq, tk, tv, p, g);
  return check_cuda(cudaGetLastError(), "launch fa_chunk_kernel");
}

template <int D>
static int join(const Attn& p, int whole, int splits, cudaStream_t s) {
  const long long tiles = chunk_pairs(p.T, p.c.B, p.group) * p.c.Hkv;
  const ChunkGrid g{whole, splits};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((tiles - whole) * (2 * kM / kJoinRows)));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return check_cuda(cudaLaunchKernelEx(&cfg, fa_chunk_combine<D>, p, g), "launch fa_chunk_combine");
}

int launch_chunk(const Attn& p, int d, bool fp8, int whole, int splits, cudaStream_t s) {
  const int page_size = 1 << p.c.page_shift;
  CUtensorMap tq, tk, tv;
  int rc;
  if ((rc = make_tmap_rows(&tq, p.q, p.T, p.Hq, d, p.q_stride, p.group, kM / p.group))) return rc;
  const int box = page_size < kN ? page_size : kN;
  if ((rc = make_tmap_pages(&tk, p.c.k, fp8, d, page_size, p.c.Hkv, p.c.num_pages, p.c.page_stride, box, fp8)) ||
      (rc = make_tmap_pages(&tv, p.c.v, fp8, d, page_size, p.c.Hkv, p.c.num_pages, p.c.page_stride, box, fp8)))
    return rc;
  if (d == 64) return fp8 ? launch<64, true>(tq, tk, tv, p, whole, splits, s) : launch<64, false>(tq, tk, tv, p, whole, splits, s);
  return fp8 ? launch<128, true>(tq, tk, tv, p, whole, splits, s) : launch<128, false>(tq, tk, tv, p, whole, splits, s);
}

int launch_chunk_combine(const Attn& p, int d, int whole, int splits, cudaStream_t s) {
  return d == 64 ? join<64>(p, whole, splits, s) : join<128>(p, whole, splits, s);
}

}  // namespace paged
}  // namespace fa

namespace {

using fa::paged::kMaxFewRows;

// Which kernels a call launches and how: from sizes that the host knows.
struct Plan {
  int few_rows;   // sequences of up to this many rows go to the few-rows kernel (0: it is not launched)
  int splits;     // chunk kernel: most pieces of the keys of a tile past the first `whole` (0: not launched)
  int whole;
  long long extra;   // CTAs of split tiles
  int copy_pages;    // an E4M3 cache is copied to BF16 pages first: pages per sequence (0: it is not)
};

// Whether an E4M3 cache is copied to BF16 pages before the chunk kernel runs.  Else each tile of 256 rows
// multiplies the codes of all its keys by their scales, which takes longer than its products: 2048
// tokens (4 heads of a group, d = 128) over 16k keys 684 us, with the copy 428 (21 of them the copy's);
// over 60k 2233 and 1344.  The copy costs a launch and three times a key's bytes in memory traffic: over
// 16k keys 128 tokens (two tiles per kv head) take 72 us without, 77 with it, 200 tokens (three tiles)
// 109 and 98, 512 (eight) 199 and 146; 12 sequences, one of them with most of 828 tokens (7 heads of a
// group, d = 64), window 2000, 41 and 35; 16 sequences of some 75 tokens 142 and 151.  So: where 2.5 tiles or
// more read a copied key, with the mean sequence taken as half the longest one, of a copy of at most
// 2 GiB.
bool copy_pays(int T, int B, int group, int Hkv, int d, int max_kv, int window, long long pages) {
  constexpr long long kMostBytes = 1ll << 31;
  if (4 * pages * B * Hkv * d > kMostBytes >> fa::paged::kCopyShift) return false;
  const double tiles = (double)T * group / (2 * fa::paged::kM);
  const double by_tile = window ? window : max_kv;                              // keys
  const double copied = (B + 1) / 2.0 * by_tile + (window ? T : 0);             // of all sequences
  return tiles * by_tile >= 2.5 * copied;
}

Plan make_plan(int T, int B, int max_q, int group, int Hkv, int d, int max_kv, int window, int sinks, int dtype) {
  Plan pl{0, 0, 0, 0, 0};
  const long long rows = (long long)max_q * group;
  if (rows <= kMaxFewRows) {
    pl.few_rows = rows <= 8 ? 8 : (rows <= 16 ? 16 : (rows <= 32 ? 32 : 64));
    return pl;
  }
  // A batch of chunks may hold sequences with a token or two: those go to the few-rows kernel with one
  // row group (its fastest forms), everything else to the chunk kernel.
  if (B > 1 && group <= 16) pl.few_rows = group <= 8 ? 8 : 16;
  // One CTA per SM at a time.  Whole rounds of tiles stay whole; the rest is split so that its pieces
  // fill the SMs: the number of pieces that makes rounds * (steps of a piece + kPieceSteps) least, with
  // kPieceSteps for a CTA's start and end and one more step for each piece's partial result.  (2048
  // tokens over 32k keys, 256 tiles: 755 us whole, 700 with the last 104 in four pieces each.)
  // More than four rounds of pieces are not planned: the steps are counted from the table's width, and a
  // piece that finds its sequence too short for it still costs a CTA's start (four sequences of up to
  // 512 new tokens and 1.5k keys in a table for 128k: 56 us, without the limit 79).
  constexpr int kPieceSteps = 4, kMostRounds = 4;
  using fa::paged::kChunkSms;
  const long long tiles = fa::paged::chunk_pairs(T, B, group) * Hkv;
  const long long rest = tiles % kChunkSms;
  long long steps = (max_kv + 127) / 128;
  if (window && window / 128 + 3 < steps) steps = window / 128 + 3;
  pl.splits = 1;
  if (rest) {
    long long best = 0;
    for (int n = 1; n <= fa::paged::kMaxSplits && (n == 1 || steps / n >= fa::paged::kSplitSteps); ++n) {
      const long long rounds = (rest * n + kChunkSms - 1) / kChunkSms;
      if (n > 1 && rounds > kMostRounds) break;
      const long long cost = rounds * ((steps + n - 1) / n + kPieceSteps) + (n > 1 ? n : 0);
      if (best == 0 || cost < best) {
        best = cost;
        pl.splits = n;
      }
    }
  }
  pl.whole = (int)(pl.splits > 1 ? tiles - rest : tiles);
  pl.extra = pl.splits > 1 ? rest * pl.splits : 0;
  if (dtype == FA_KV_E4M3) {
    constexpr long long kBlk = 1 << fa::paged::kCopyShift;
    long long pages = (max_kv + kBlk - 1) / kBlk;
    if (window) {
      const long long seen = (sinks + kBlk - 1) / kBlk + ((long long)window + max_q) / kBlk + 2;
      if (seen < pages) pages = seen;
    }
    if (copy_pays(T, B, group, Hkv, d, max_kv, window, pages)) pl.copy_pages = (int)pages;
  }
  return pl;
}

struct Parts {
  size_t o, lse, info, k, v, table, total;   // offsets
};

// The workspace: FP32 partial outputs, their log-sum-exps, the few-rows kernel's records, the copied
// cache.  The two kernels of a mixed batch have parts of their own.
Parts carve(const Plan& pl, int B, int Hkv, int d, int max_kv, Parts* chunk) {
  const size_t rows = pl.few_rows ? (size_t)2 * fa::paged::kRowsMaxCtas * pl.few_rows : 0;
  Parts f{};
  f.o = 0;
  f.lse = fa::round_up(rows * d * 4, 256);
  f.info = f.lse + fa::round_up(rows * 4, 256);
  f.total = f.info + (rows ? fa::round_up((size_t)B * Hkv * sizeof(int4), 256) : 0);
  const size_t c_rows = (size_t)pl.extra * 2 * fa::paged::kM;
  chunk->o = f.total;
  chunk->lse = chunk->o + fa::round_up(c_rows * d * 4, 256);
  chunk->info = 0;
  constexpr size_t kBlk = 1 << fa::paged::kCopyShift;
  const size_t pool = fa::round_up((size_t)pl.copy_pages * B * kBlk * Hkv * d * 2, 256);
  chunk->k = chunk->lse + fa::round_up(c_rows * 4, 256);
  chunk->v = chunk->k + pool;
  chunk->table = chunk->v + pool;
  chunk->total = chunk->table + (pl.copy_pages ? fa::round_up((max_kv + kBlk - 1) / kBlk * B * 4, 256) : 0);
  return f;
}

int check_attn(int T, int B, int max_q, int Hq, int Hkv, int d) {
  using namespace fa;
  if (T < 0 || max_q < 0) return set_error(FA_ERR_INVALID_ARG, "T, max_q must be >= 0 (got %d, %d)", T, max_q);
  if (B < 1 || Hkv < 1 || Hq < 1) return set_error(FA_ERR_INVALID_ARG, "B, Hq, Hkv must be >= 1 (got %d, %d, %d)", B, Hq, Hkv);
  if (Hq % Hkv) return set_error(FA_ERR_INVALID_ARG, "Hq = %d is not a multiple of Hkv = %d", Hq, Hkv);
  if (Hq / Hkv > 128) return set_error(FA_ERR_UNSUPPORTED, "more than 128 query heads for a kv head (%d)", Hq / Hkv);
  if (d != 64 && d != 128) return set_error(FA_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
  // the few-rows join has up to kMaxFewRows / 4 CTAs for each sequence and kv head
  constexpr long long kMostItems = (1ll << 31) / (kMaxFewRows / 4);
  if ((long long)T * Hq >= (1ll << 31) || (long long)B * Hkv >= kMostItems)
    return set_error(FA_ERR_INVALID_ARG, "T*Hq must be < 2^31 and B*Hkv < %lld", kMostItems);
  return FA_OK;
}

}  // namespace

extern "C" size_t fa_fwd_paged_workspace_size(int T, int B, int max_q, int Hq, int Hkv, int d, int max_kv, int window,
                                               int sinks, int dtype) {
  fa::clear_error();
  if (check_attn(T, B, max_q, Hq, Hkv, d) || max_kv < 0 || window < 0 || sinks < 0 || T == 0) return 0;
  Parts chunk;
  carve(make_plan(T, B, max_q, Hq / Hkv, Hkv, d, max_kv, window < max_kv ? window : 0, std::min(sinks, max_kv), dtype), B, Hkv,
        d, max_kv, &chunk);
  return chunk.total;
}

extern "C" int fa_fwd_paged(const fa_paged_kv* kv, const void* q, int64_t q_stride, const int32_t* q_indptr, int T,
                            int max_q, int Hq, void* o, float* lse, int window, int sinks, float scale, void* workspace,
                            size_t workspace_bytes, void* stream) {
  fa::NvtxRange nvtx_range("fa_fwd_paged");
  using namespace fa;
  clear_error();
  paged::Attn p{};
  int rc;
  if ((rc = paged::check_cache(kv, &p.c)) || (rc = check_attn(T, kv->B, max_q, Hq, kv->Hkv, kv->d))) return rc;
  if ((rc = check_ptr(q, "q")) || (rc = check_ptr(o, "o"))) return rc;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3)) return set_error(FA_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  if (!q_indptr || (reinterpret_cast<uintptr_t>(q_indptr) & 3))
    return set_error(FA_ERR_INVALID_ARG, "q_indptr must be a 4-byte aligned device pointer");
  if (q_stride < (int64_t)Hq * kv->d || q_stride % 8)
    return set_error(FA_ERR_INVALID_ARG, "q_stride %lld must be a multiple of 8 and at least Hq*d = %d",
                     (long long)q_stride, Hq * kv->d);
  if (!(scale > 0.f) || !isfinite(scale)) return set_error(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (window < 0 || sinks < 0) return set_error(FA_ERR_INVALID_ARG, "window and sinks must be >= 0 (got %d, %d)", window, sinks);
  if (!window && sinks) return set_error(FA_ERR_INVALID_ARG, "sinks need a window");
  if (T == 0 || max_q == 0) return FA_OK;
  const int max_kv = kv->max_pages * kv->page_size;
  if (window >= max_kv) window = 0;   // a window of the whole cache is none
  sinks = std::min(sinks, max_kv);
  const Plan pl = make_plan(T, kv->B, max_q, Hq / kv->Hkv, kv->Hkv, kv->d, max_kv, window, sinks, kv->dtype);
  Parts chunk;
  const Parts few = carve(pl, kv->B, kv->Hkv, kv->d, max_kv, &chunk);
  if (chunk.total) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
      return set_error(FA_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
    if (workspace_bytes < chunk.total)
      return set_error(FA_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed", workspace_bytes, chunk.total);
  }
  p.c.status = device_status_word();
  if (!p.c.status) return set_error(FA_ERR_CUDA, "could not allocate the device status record");
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.q_indptr = q_indptr;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.T = T;
  p.Hq = Hq;
  p.group = Hq / kv->Hkv;
  p.max_rows = (int)((long long)max_q * p.group < INT32_MAX ? max_q * p.group : INT32_MAX);
  p.few_rows = pl.few_rows;
  p.window = window;
  p.sinks = sinks;
  p.copy_pages = pl.copy_pages;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
#ifdef FA_TEST_HOOKS
  const char* inject = getenv("FA_TEST_INJECT_STALL");
  p.inject_stall = (inject && inject[0] == '1') ? 1 : 0;
#endif
  const bool fp8 = kv->dtype == FA_KV_E4M3, copy = pl.copy_pages > 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  // Chunks first; the few-rows kernel of a mixed batch then starts beside them, on SMs that they leave
  // free; the joining kernels come last.
  paged::Attn c = p;
  c.part_o = reinterpret_cast<float*>(ws + chunk.o);
  c.part_lse = reinterpret_cast<float*>(ws + chunk.lse);
  p.part_o = reinterpret_cast<float*>(ws + few.o);
  p.part_lse = reinterpret_cast<float*>(ws + few.lse);
  p.part_info = reinterpret_cast<int4*>(ws + few.info);
  if (copy) {
    c.c.k = ws + chunk.k;
    c.c.v = ws + chunk.v;
    c.c.table = reinterpret_cast<const int32_t*>(ws + chunk.table);
    c.c.page_shift = paged::kCopyShift;
    c.c.max_pages = (max_kv + (1 << paged::kCopyShift) - 1) >> paged::kCopyShift;
    c.c.table_stride = c.c.max_pages;
    c.c.num_pages = pl.copy_pages * kv->B;
    c.c.page_stride = (long long)kv->Hkv * kv->d << paged::kCopyShift;
    if ((rc = paged::launch_copy(p, c.c, kv->d, s))) return rc;
  }
  if (pl.splits && (rc = paged::launch_chunk(c, kv->d, fp8 && !copy, pl.whole, pl.splits, s))) return rc;
  if (pl.few_rows && (rc = paged::launch_rows(p, kv->d, fp8, pl.splits > 0, s))) return rc;
  if (pl.splits > 1 && (rc = paged::launch_chunk_combine(c, kv->d, pl.whole, pl.splits, s))) return rc;
  return pl.few_rows ? paged::launch_rows_combine(p, kv->d, s) : FA_OK;
}
