// What the two paged attention kernels and their host side share: parameters, the part of a
// sequence that its new tokens see, and the partial results of rows whose keys were split.
//
// A kv head serves `group` = Hq / Hkv query heads.  A sequence's rows for it are numbered
// r = t * group + g (t: new token, g: head within the group), so one pass over a head's K and V
// serves the whole group.  Token t sits at position pos0 + t, pos0 = kv_len - new tokens, and sees
//   key <= position  and  (no window, or position - key < window, or key < sinks).
#pragma once

#include "paged.cuh"

namespace fa {
namespace paged {

// The few-rows kernel takes sequences of up to this many rows for a kv head (four groups of 16).
constexpr int kMaxFewRows = 64;

struct Attn {   // arguments of both kernels
  Cache c;
  const __nv_bfloat16* q;
  long long q_stride;        // elements between tokens
  const int32_t* q_indptr;
  __nv_bfloat16* o;          // [T, Hq, d]
  float* lse;                // [T, Hq] or NULL
  float* part_o;             // partial results, see the kernels
  float* part_lse;
  int4* part_info;
  int T, Hq, group;
  int max_rows;              // largest number of rows of a sequence (the caller's max_q)
  int few_rows;              // sequences of up to this many rows (8, 16, 32, 64) are the few-rows kernel's; 0: none
  int copy_pages;            // pages of a sequence in the BF16 copy of an E4M3 cache (see launch_copy)
  int window, sinks;         // window 0: none
  float scale, scale_log2;   // scale_log2 = scale log2(e)
  int inject_stall;          // test builds only (FA_TEST_HOOKS): make a warp's first wait run out
};

// The new tokens of one sequence and the keys they see.
struct Seq {
  int q0, n;      // first packed row, new tokens
  int kv, pos0;   // keys, position of the first new token (negative: its first rows see nothing)
};

__device__ __forceinline__ Seq load_seq(const Attn& p, int b) {
  Seq s;
  s.q0 = __ldg(p.q_indptr + b);
  const int q1 = __ldg(p.q_indptr + b + 1);
  s.kv = __ldg(p.c.kv_len + b);
  s.n = q1 - s.q0;
  if (s.q0 < 0 || q1 < s.q0 || q1 > p.T || (long long)s.n * p.group > p.max_rows) {
    report_bounds(p.c.status, kSitePagedLen, q1);
    s.n = 0;
  }
  const int cap = p.c.max_pages << p.c.page_shift;
  if (s.kv < 0 || s.kv > cap) {
    report_bounds(p.c.status, kSitePagedLen, s.kv);
    s.kv = min(max(s.kv, 0), cap);
  }
  s.pos0 = s.kv - s.n;
  return s;
}

// The kBlk-key blocks that the tokens first .. last (positions) see, in order: step j takes the
// block at key at(j).  With a window: the blocks that hold sinks, then those from the window of the
// first token on.  At least one step, so that rows without keys are written too.
template <int kBlk>
struct KeyWalk {
  int lo, hi, sinks;   // keys some row sees: [lo, hi) and [0, sinks)
  int n_sink, b_lo, steps;
  __device__ __forceinline__ KeyWalk(const Attn& p, int first, int last) {
    hi = max(last + 1, 0);
    lo = p.window ? max(0, first - p.window + 1) : 0;
    sinks = p.window ? min(p.sinks, hi) : 0;
    b_lo = lo / kBlk;
    n_sink = min((sinks + kBlk - 1) / kBlk, b_lo);
    steps = max(n_sink + (hi + kBlk - 1) / kBlk - b_lo, 1);
  }
  __device__ __forceinline__ int at(int j) const { return (j < n_sink ? j : j - n_sink + b_lo) * kBlk; }
  // whether any row sees a key of [key, key + n)
  __device__ __forceinline__ bool any(int key, int n) const {
    return key < hi && (key + n > lo || key < sinks);
  }
  __device__ __forceinline__ bool seen(int key) const { return key < hi && (key >= lo || key < sinks); }
  // whether every key of [key, key + kBlk) is seen by every token first .. last
  __device__ __forceinline__ bool all(const Attn& p, int key, int first, int last) const {
    return key + kBlk <= first + 1 && (!p.window || key > last - p.window || key + kBlk <= sinks);
  }
};

// 4-D tiled load (d, slot, head, page) of one box of a page pool.
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int slot,
                                              int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(slot), "r"(head), "r"(page)
      : "memory");
}

// Few rows: the most CTAs that fa_rows_kernel is launched with, and its partial results: two slots of
// few_rows rows (8, 16, 32 or 64) for each CTA: the item that it continues, the item that it leaves
// unfinished.
constexpr int kRowsMaxCtas = 304;

// Chunks: an upper bound of the pairs of tiles that T packed rows of B sequences need.
constexpr int kChunkSms = 152;   // CTAs that run at once, one per SM
constexpr int kMaxSplits = 16;
inline long long chunk_pairs(int T, int B, int group) {
  const int per = 2 * (128 / group), seqs = T < B ? T : B;   // each sequence may end inside a pair
  return (T - seqs) / per + seqs;
}

constexpr int kCopyShift = 7;    // tokens of a page of the copied cache: 128, the chunk kernel's block

int launch_copy(const Attn& p, const Cache& to, int d, cudaStream_t s);
int launch_rows(const Attn& p, int d, bool fp8, bool beside, cudaStream_t s);
int launch_rows_combine(const Attn& p, int d, cudaStream_t s);
int launch_chunk(const Attn& p, int d, bool fp8, int whole, int splits, cudaStream_t s);
int launch_chunk_combine(const Attn& p, int d, int whole, int splits, cudaStream_t s);

}  // namespace paged
}  // namespace fa
