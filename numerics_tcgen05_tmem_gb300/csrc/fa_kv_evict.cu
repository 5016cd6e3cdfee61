// Eviction from a paged cache by accumulated attention weight (fa_kv_evict): of each sequence and kv head `keep`
// keys stay -- the first `sinks`, the newest `recent`, and of the others those with the largest weights (of equal
// ones the first) -- and move, in order, to the first positions of the sequence in another block table, or
// in the same one.
//
//   select  a CTA per (sequence, kv head): the smallest weight that stays, by three passes over the weights' bits
//           (11, 11 and 10 of them, a histogram each in shared memory), then one pass in order that writes the
//           kept positions.
//   move    the kept vectors, their scales and weights: bandwidth work, 16 bytes a thread; by the selecting CTAs or in a
//           launch of its own.
// Measured: 64 sequences of 4.4k keys on average, 8 heads of 128, cut to 2000 in other pages, E4M3 87 us (66 at the
// copy rate; the selection alone takes 29, for its longest sequence), BF16 145; one sequence of 4.5k to 2k 12 us.
// In place a vector only ever moves to a lower position, to where nothing is that is still to be read as long
// as the vectors are taken in order: a CTA takes all of one head's K or V, 64 (or 32) bytes wide, step by step,
// and waits between a step's loads and its stores.
#include <algorithm>

#include "overlap.h"
#include "paged_attn.cuh"

namespace fa {
namespace paged {

constexpr int kDigit = 11, kBins = 1 << kDigit;

struct Evict {
  Cache c;
  float* weights;
  long long weight_stride;
  const int32_t* table_out;      // [B][..], rows table_out_stride apart
  long long table_out_stride;
  int max_pages_out;
  int keep, sinks, recent;
  int32_t* kept_len;             // [B]
  int32_t* kept;                 // [B][Hkv][keep]
};

// Weights in the order of unsigned integers; NaN is the largest, -0 is 0.
__device__ __forceinline__ uint32_t weight_order(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ ((int)u < 0 ? 0xFFFFFFFFu : 0x80000000u);
}

// A sequence's length: 0, recorded, where it is out of range.
__device__ __forceinline__ int evict_length(const Cache& c, int b) {
  const int n = __ldg(c.kv_len + b);
  if (n < 0 || n > c.max_pages << c.page_shift) {
    if (threadIdx.x == 0) report_bounds(c.status, kSitePagedLen, n);
    return 0;
  }
  return n;
}

// Where a key lies: its page and its offset within a page's head; page -1, recorded, where there is none.
struct Spot {
  int page, slot;
};
__device__ __forceinline__ Spot spot_of(const Cache& c, const int32_t* table, long long stride, int max_pages, int b, int key) {
  const int i = key >> c.page_shift;
  Spot s{-1, key & ((1 << c.page_shift) - 1)};
  if (key < 0 || i >= max_pages) {
    report_bounds(c.status, kSitePagedEvict, key);
    return s;
  }
  s.page = __ldg(table + b * stride + i);
  if (s.page < 0 || s.page >= c.num_pages) {
    report_bounds(c.status, kSitePagedEvict, s.page);
    s.page = -1;
  }
  return s;
}

// The kept keys first .. first + here - 1 of a (sequence, kv head), at most kVecs, to their places in table_out: a lane of the
// warp looks one up and moves its scales and weight, then kRow / 16 lanes move a vector, kMost loads of a lane in flight.
template <int kRow, int kVecs, int kMost>    // kRow: bytes of a vector
__device__ __forceinline__ void move_keys(const Evict& g, int item, int first, int here) {
  constexpr int kLanes = kRow / 16, kGroups = 32 / kLanes, kSteps = kVecs / kGroups;
  constexpr int kUnroll = 2 * kSteps < kMost ? 2 * kSteps : kMost;
  static_assert(2 * kSteps % kUnroll == 0, "K and V in whole rounds");
  const int lane = threadIdx.x % 32;
  const int b = item / g.c.Hkv, h = item - b * g.c.Hkv;
  const long long page_size = 1ll << g.c.page_shift;
  const int elem = g.c.k_scale != nullptr ? 1 : 2;
  long long from = -1, to = -1;       // the lane's vector: bytes from the pool's start
  if (lane < here) {
    const int key = g.kept[(long long)item * g.keep + first + lane];
    const Spot f = spot_of(g.c, g.c.table, g.c.table_stride, g.c.max_pages, b, key);
    Spot t = spot_of(g.c, g.table_out, g.table_out_stride, g.max_pages_out, b, first + lane);
    // a page of the sequence's own, as in a copy of its table: other keys of the page are still to be read
    if (t.page >= 0 && t.page == __ldg(g.c.table + b * g.c.table_stride + ((first + lane) >> g.c.page_shift))) {
      if (key != first + lane) report_bounds(g.c.status, kSitePagedEvict, t.page);   // (else it is there)
      t.page = -1;
    }
    if (f.page >= 0 && t.page >= 0) {
      const long long f_at = h * page_size + f.slot, t_at = h * page_size + t.slot;
      from = f.page * g.c.page_stride * elem + f_at * kRow;
      to = t.page * g.c.page_stride * elem + t_at * kRow;
      g.weights[t.page * g.weight_stride + t_at] = g.weights[f.page * g.weight_stride + f_at];
      if (g.c.k_scale != nullptr) {
        const long long f_s = f.page * g.c.scale_stride + f_at, t_s = t.page * g.c.scale_stride + t_at;
        const float ks = g.c.k_scale[f_s], vs = g.c.v_scale[f_s];
        g.c.k_scale[t_s] = ks;
        g.c.v_scale[t_s] = vs;
      }
    }
  }
  const int col = lane % kLanes * 16;
#pragma unroll
  for (int s0 = 0; s0 < 2 * kSteps; s0 += kUnroll) {
    uint4 x[kUnroll];
    bool moves[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int s = s0 + u, v = s / 2 * kGroups + lane / kLanes;      // K and V of the same vectors in turn
      const long long src = __shfl_sync(0xffffffffu, from, v);
      moves[u] = src >= 0;
      if (moves[u]) x[u] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>((s & 1) ? g.c.v : g.c.k) + src + col);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int s = s0 + u;
      const long long dst = __shfl_sync(0xffffffffu, to, s / 2 * kGroups + lane / kLanes);
      if (moves[u]) *reinterpret_cast<uint4*>(static_cast<uint8_t*>((s & 1) ? g.c.v : g.c.k) + dst + col) = x[u];
    }
  }
}

// kCached weights stay in shared memory between the passes.  512 threads and 8192 weights, three CTAs on an SM beside
// the moving kernel's first ones (with 16384: the selection 2 us faster, the call on 64 sequences of 4.4k keys 117 us
// instead of 105); 1024 and 40960 for long sequences where there are fewer CTAs than two for each SM (one of 40k
// keys: 49 us with the smaller form).
// kRow > 0: the CTA also moves its keys, vectors of kRow bytes, into other pages.  Two CTAs on an SM, four loads of a lane in
// flight (three and two: 90 us where these take 87; 256 threads 112).  The longest sequences, of kMostSorted at most,
// come first, so that the CTAs that start last have little to do (64 of 0.5k to 16k keys: 101 -> 87 us).
constexpr int kMostSorted = 256;

template <int kSelectThreads, int kCached, int kRow>
__global__ void __launch_bounds__(kSelectThreads, kRow > 0 ? 2 : 1536 / kSelectThreads)
    evict_select_kernel(const __grid_constant__ Evict g) {
  constexpr int kWarps = kSelectThreads / 32, kStep = 4 * kSelectThreads;   // a thread has four keys at a time
  extern __shared__ __align__(16) uint32_t cached[];
  __shared__ uint32_t bins[kBins];
  __shared__ int warp_sum[kWarps];
  __shared__ int found_bin, found_above;
  cudaTriggerProgrammaticLaunchCompletion();   // a moving kernel may get ready; it waits for this one's end
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int b = blockIdx.x / g.c.Hkv;
  const int h = blockIdx.x - b * g.c.Hkv;
  if constexpr (kRow > 0) {
    // the sequence that comes in this place
    __shared__ int place;
    if (g.c.B <= kMostSorted) {
      int* len = reinterpret_cast<int*>(cached);
      for (int i = threadIdx.x; i < g.c.B; i += kSelectThreads) len[i] = __ldg(g.c.kv_len + i);
      __syncthreads();
      for (int i = threadIdx.x; i < g.c.B; i += kSelectThreads) {
        const int mine = len[i];
        int before = 0;
        for (int x = 0; x < g.c.B; ++x) before += len[x] > mine || (len[x] == mine && x < i) ? 1 : 0;
        if (before == b) place = i;
      }
      __syncthreads();
      b = place;
    }
  }
  const int item = b * g.c.Hkv + h;
  const int n = evict_length(g.c, b), kept = min(n, g.keep);
  int32_t* out = g.kept + (long long)item * g.keep;
  if (h == 0 && threadIdx.x == 0) g.kept_len[b] = kept;
  for (uint32_t i = (uint32_t)kept + threadIdx.x; i < (uint32_t)g.keep; i += kSelectThreads) out[i] = -1;   // (keep: any int)
  if (n <= g.keep) {
    for (int i = threadIdx.x; i < n; i += kSelectThreads) out[i] = i;
    if constexpr (kRow > 0) {
      __syncthreads();
      for (int first = 32 * warp; first < kept; first += 32 * kWarps)
        move_keys<kRow, 32, 4>(g, item, first, min(kept - first, 32));
    }
    return;
  }
  const int page_mask = (1 << g.c.page_shift) - 1;
  const int32_t* table = g.c.table + b * g.c.table_stride;
  // the order of the four weights at `key`, which lie in one page
  auto page_at = [&](int key) { return key < n ? __ldg(table + (key >> g.c.page_shift)) : -1; };
  auto read_page = [&](int key, int page) {
    if (page < 0 || page >= g.c.num_pages) {
      if (key < n) report_bounds(g.c.status, kSitePagedEvict, page);
      return make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return *reinterpret_cast<const float4*>(g.weights + page * g.weight_stride + ((long long)h << g.c.page_shift) +
                                            (key & page_mask));
  };
  auto ordered = [](const float4& w) {
    return make_uint4(weight_order(w.x), weight_order(w.y), weight_order(w.z), weight_order(w.w));
  };
  auto read = [&](int key) { return ordered(read_page(key, page_at(key))); };
  auto again = [&](int key) { return key < kCached ? *reinterpret_cast<const uint4*>(cached + key) : read(key); };
  // the candidates [lo, hi), of which `want` stay: those above `limit`, and the first `ties` that equal it
  const int lo = g.sinks, hi = n - g.recent, want = g.keep - g.sinks - g.recent;
  uint32_t limit = 0xFFFFFFFFu;
  int ties = 0;
  if (want > 0) {
    uint32_t prefix = 0;
    int left = want, shift = 32;
    for (int pass = 0; pass < 3; ++pass) {
      const int digit = pass < 2 ? kDigit : 32 - 2 * kDigit;
      const int above = shift;          // bits from here on are settled
      shift -= digit;
      for (int i = threadIdx.x; i < kBins; i += kSelectThreads) bins[i] = 0;
      __syncthreads();
      auto count = [&](int key, const uint4& u) {
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key + e >= lo && key + e < hi && (pass == 0 || (x[e] >> above) == prefix))
            atomicAdd(&bins[x[e] >> shift & ((1 << digit) - 1)], 1u);
      };
      int key = 4 * (int)threadIdx.x;
      if (pass > 0)
        for (; key < min(hi, kCached); key += kStep) count(key, *reinterpret_cast<const uint4*>(cached + key));
      constexpr int kFlight = 4;        // accesses of a thread on their way
      for (; key < hi; key += kFlight * kStep) {
        int page[kFlight];
        float4 w[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) page[i] = page_at(key + i * kStep);
#pragma unroll
        for (int i = 0; i < kFlight; ++i) w[i] = read_page(key + i * kStep, page[i]);
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const int at = key + i * kStep;
          if (at >= hi) break;
          const uint4 u = ordered(w[i]);
          if (pass == 0 && at < kCached) *reinterpret_cast<uint4*>(cached + at) = u;   // read back by this thread
          count(at, u);
        }
      }
      __syncthreads();
      // from the largest bin down: the one in which the count reaches `left`.  A thread has kBins / threads bins.
      constexpr int kPer = kBins / kSelectThreads;
      const int top = kBins - 1 - (int)threadIdx.x * kPer;
      int mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) mine += (int)bins[top - i];
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      int before = incl - mine;
      for (int w = 0; w < warp; ++w) before += warp_sum[w];
      if (before < left && before + mine >= left) {
        int i = 0;
        while (before + (int)bins[top - i] < left) before += (int)bins[top - i++];
        found_bin = top - i;
        found_above = before;
      }
      __syncthreads();
      prefix = prefix << digit | (uint32_t)found_bin;
      left -= found_above;
    }
    limit = prefix;
    ties = left;
  }
  // in order: what stays.  A key's place is the number of those before it that stay for sure, and of those that
  // equal the limit, `ties` at most.
  int sure_before = 0, equal_before = 0;    // before this step
  auto get = [&](int key) { return want > 0 && key < hi ? again(key) : make_uint4(0, 0, 0, 0); };
  uint4 next = get(4 * (int)threadIdx.x);
  for (int base = 0; base < n; base += kStep) {
    const int key = base + 4 * (int)threadIdx.x;
    const uint32_t x[4] = {next.x, next.y, next.z, next.w};
    next = get(key + kStep);
    bool sure[4], equal[4];
    int counts = 0;                          // equal ones in the upper half
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool inside = key + e >= lo && key + e < hi;
      sure[e] = key + e < n && (!inside || (want > 0 && x[e] > limit));
      equal[e] = inside && want > 0 && x[e] == limit;
      counts += (sure[e] ? 1 : 0) + (equal[e] ? 1 << 16 : 0);
    }
    int incl = counts;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int excl = incl - counts, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) excl += warp_sum[w];
      all += warp_sum[w];
    }
    int at_sure = sure_before + (excl & 0xFFFF), at_equal = equal_before + (excl >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int place = at_sure + min(at_equal, ties);   // (under keep, unless weights change during the call)
      if ((sure[e] || (equal[e] && at_equal < ties)) && place < kept) out[place] = key + e;
      at_sure += sure[e] ? 1 : 0;
      at_equal += equal[e] ? 1 : 0;
    }
    sure_before += all & 0xFFFF;
    equal_before += all >> 16;
    __syncthreads();
  }
  if constexpr (kRow > 0)
    for (int first = 32 * warp; first < kept; first += 32 * kWarps)
      move_keys<kRow, 32, 4>(g, item, first, min(kept - first, 32));
}

// Into other pages: a warp has kVecs kept keys of one (sequence, kv head).  32 keys; 8 where that would leave SMs with a few
// warps (one sequence cut from 4.5k keys to 2k: 14.2 us with 32, 12.0 with 8).
constexpr int kMoveThreads = 256;

template <int kRow, int kVecs>    // kRow: bytes of a vector
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ Evict g, int chunks, long long warps) {
  cudaGridDependencySynchronize();
  const long long w = (long long)blockIdx.x * (kMoveThreads / 32) + threadIdx.x / 32;
  if (w >= warps) return;
  const int item = (int)(w / chunks), first = (int)(w - (long long)item * chunks) * kVecs;
  const int here = min(g.kept_len[item / g.c.Hkv] - first, kVecs);
  if (here <= 0) return;
  move_keys<kRow, kVecs, 8>(g, item, first, here);
}

// Within the same pages.  A CTA has one (sequence, kv head), K or V, kSlice bytes of each vector; the first slice's
// CTAs also move the scales, that of K the weights.  While a step's vectors are on their way the next step's places
// are looked up.
template <int kSlice>
__global__ void __launch_bounds__(kMoveThreads) evict_shift_kernel(const __grid_constant__ Evict g, int row_bytes) {
  constexpr int kLanes = kSlice / 16, kGroups = kMoveThreads / kLanes, kUnroll = 4, kStep = kGroups * kUnroll;
  const int slices = row_bytes / kSlice;
  const int slice = blockIdx.x % slices, is_v = blockIdx.x / slices % 2, item = blockIdx.x / slices / 2;
  const int b = item / g.c.Hkv, h = item - b * g.c.Hkv;
  cudaGridDependencySynchronize();
  const int kept = g.kept_len[b];
  const int32_t* keys = g.kept + (long long)item * g.keep;
  const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes, col = slice * kSlice + lane * 16;
  const long long page_size = 1ll << g.c.page_shift;
  const long long page_bytes = g.c.page_stride * (g.c.k_scale != nullptr ? 1 : 2);
  uint8_t* pool = static_cast<uint8_t*>(is_v ? g.c.v : g.c.k);
  float* scales = is_v ? g.c.v_scale : g.c.k_scale;
  const bool moves_scale = scales != nullptr && slice == 0 && lane == 0, moves_weight = !is_v && slice == 0 && lane == 1;
  Spot from[kUnroll], to[kUnroll];    // to: -1 where nothing moves
  auto look = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kGroups + group;
      to[u].page = -1;
      const int key = i < kept ? keys[i] : i;
      if (key == i) continue;          // it stays where it is
      from[u] = spot_of(g.c, g.c.table, g.c.table_stride, g.c.max_pages, b, key);
      if (from[u].page >= 0) to[u] = spot_of(g.c, g.c.table, g.c.table_stride, g.c.max_pages, b, i);
    }
  };
  look(0);
  for (int i0 = 0; i0 < kept; i0 += kStep) {
    uint4 x[kUnroll];
    float s[kUnroll];
    Spot here[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      here[u] = to[u];
      if (to[u].page < 0) continue;
      const long long at = h * page_size + from[u].slot;
      x[u] = *reinterpret_cast<const uint4*>(pool + from[u].page * page_bytes + at * row_bytes + col);
      if (moves_scale) s[u] = scales[from[u].page * g.c.scale_stride + at];
      if (moves_weight) s[u] = g.weights[from[u].page * g.weight_stride + at];
    }
    look(i0 + kStep);
    __syncthreads();   // every load of this step comes before its stores; those of the next step read higher positions
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (here[u].page < 0) continue;
      const long long at = h * page_size + here[u].slot;
      *reinterpret_cast<uint4*>(pool + here[u].page * page_bytes + at * row_bytes + col) = x[u];
      if (moves_scale) scales[here[u].page * g.c.scale_stride + at] = s[u];
      if (moves_weight) g.weights[here[u].page * g.weight_stride + at] = s[u];
    }
  }
}

}  // namespace paged
}  // namespace fa

extern "C" int fa_kv_evict(const fa_paged_kv* kv, float* weights, int64_t weight_stride, const int32_t* table_out,
                           int64_t table_out_stride, int max_pages_out, int keep, int sinks, int recent, int32_t* kept_len,
                           int32_t* kept, void* stream) {
  fa::NvtxRange nvtx_range("fa_kv_evict");
  using namespace fa;
  clear_error();
  paged::Evict g{};
  int rc;
  if ((rc = paged::check_cache(kv, &g.c))) return rc;
  if ((rc = paged::check_weights(kv, weights, weight_stride))) return rc;
  if (keep < 1 || sinks < 0 || recent < 0)
    return set_error(FA_ERR_INVALID_ARG, "keep must be >= 1, sinks and recent >= 0 (got %d, %d, %d)", keep, sinks, recent);
  if ((long long)sinks + recent > keep)
    return set_error(FA_ERR_INVALID_ARG, "sinks + recent = %lld must be at most keep = %d", (long long)sinks + recent, keep);
  const bool in_place = !table_out || table_out == kv->block_table;
  const long long max_kv = (long long)kv->max_pages * kv->page_size;
  if (!in_place) {
    if (reinterpret_cast<uintptr_t>(table_out) & 3) return set_error(FA_ERR_INVALID_ARG, "table_out is not 4-byte aligned");
    if (max_pages_out < 1 || table_out_stride < max_pages_out)
      return set_error(FA_ERR_INVALID_ARG, "table_out_stride %lld is less than max_pages_out %d, or that is under 1",
                       (long long)table_out_stride, max_pages_out);
    const long long need = keep < max_kv ? keep : max_kv;
    if ((long long)max_pages_out * kv->page_size < need)
      return set_error(FA_ERR_INVALID_ARG, "table_out has room for %lld keys of a sequence, %lld may be kept",
                       (long long)max_pages_out * kv->page_size, need);
  }
  if (!kept_len || !kept || ((reinterpret_cast<uintptr_t>(kept_len) | reinterpret_cast<uintptr_t>(kept)) & 3))
    return set_error(FA_ERR_INVALID_ARG, "kept_len and kept must be 4-byte aligned device pointers");
  if (kept_len == kv->kv_len)   // every head's CTA reads the length
    return set_error(FA_ERR_INVALID_ARG, "kept_len must not be kv_len itself");
  const long long items = (long long)kv->B * kv->Hkv, most = keep < max_kv ? keep : max_kv;
  const int vecs = items * ((most + 31) / 32) >= 32ll * sm_count() ? 32 : 8;   // of a warp that moves
  const long long chunks = (most + vecs - 1) / vecs;
  if (items * std::max(chunks, 8ll) >= (1ll << 31)) return set_error(FA_ERR_INVALID_ARG, "B*Hkv*keep/32 must be < 2^31");
  const auto ints = [](const void* p, long long rows, long long n, long long stride) { return Pieces{p, 4 * n, {rows, 1, 1}, {4 * stride, 0, 0}}; };
  const Pieces out[2] = {ints(kept_len, 1, kv->B, 0), ints(kept, 1, items * keep, 0)};
  const Pieces in[3] = {ints(kv->kv_len, 1, kv->B, 0), ints(kv->block_table, kv->B, kv->max_pages, kv->table_stride),
                        ints(table_out, kv->B, max_pages_out, table_out_stride)};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < (in_place ? 2 : 3); ++j)
      if (pieces_overlap(out[i], in[j]))
        return set_error(FA_ERR_INVALID_ARG, "%s overlaps another tensor of the call", i == 0 ? "kept_len" : "kept");
  if (pieces_overlap(out[0], out[1])) return set_error(FA_ERR_INVALID_ARG, "kept overlaps another tensor of the call, kept_len");
  g.c.status = device_status_word();
  if (!g.c.status) return set_error(FA_ERR_CUDA, "could not allocate the device status record");
  g.weights = weights;
  g.weight_stride = weight_stride;
  g.table_out = in_place ? kv->block_table : table_out;
  g.table_out_stride = in_place ? kv->table_stride : table_out_stride;
  g.max_pages_out = in_place ? kv->max_pages : max_pages_out;
  g.keep = keep;
  g.sinks = sinks;
  g.recent = recent;
  g.kept_len = kept_len;
  g.kept = kept;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // One launch where there is a CTA for each SM at least: a CTA moves its own keys, while others still select.  8 heads of 128, to
  // 2000 keys, E4M3: 64 sequences of 0.5k to 16k keys 106 -> 87 us (BF16 157 -> 145), to 500 keys 57 -> 41, of 4.4k each
  // 116 -> 109; 32 sequences 58 -> 52; 40 of 4.4k each, a few CTAs more than run at once, 76 -> 84.  Long sequences
  // where CTAs of 512 threads leave room select with 1024 (20 of 5k to 40k keys: 93 us, moving their own 106).
  const int row = kv->d * (kv->dtype == FA_KV_E4M3 ? 1 : 2);
  const bool wide = items < 2ll * sm_count() && max_kv > 16384, own = items >= sm_count() && !in_place && !wide;
  const int cache = (wide ? 40960 : 8192) * 4, threads = wide ? 1024 : 512;
  auto select = wide              ? paged::evict_select_kernel<1024, 40960, 0>
                : !own            ? paged::evict_select_kernel<512, 8192, 0>
                : row == 64       ? paged::evict_select_kernel<512, 8192, 64>
                : row == 128      ? paged::evict_select_kernel<512, 8192, 128>
                                  : paged::evict_select_kernel<512, 8192, 256>;
  static std::atomic<uint64_t> prepared[5];
  if ((rc = prepare_kernel(reinterpret_cast<const void*>(select), cache, threads, 0, "evict_select_kernel",
                           &prepared[wide ? 0 : !own ? 1 : row == 64 ? 2 : row == 128 ? 3 : 4])))
    return rc;
  select<<<(unsigned)items, threads, cache, s>>>(g);
  if ((rc = check_cuda(cudaGetLastError(), "launch evict_select_kernel")) || own) return rc;
  const long long warps = items * chunks, per = paged::kMoveThreads / 32;
  cudaLaunchConfig_t cfg{};
  // in place: 64 bytes of a vector, 32 where that leaves SMs without a CTA
  const int slice = items * 2 * (row / 64) < 2ll * sm_count() ? 32 : 64;
  cfg.gridDim = dim3((unsigned)(in_place ? items * 2 * (row / slice) : (warps + per - 1) / per));
  cfg.blockDim = dim3(paged::kMoveThreads);
  cfg.stream = s;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  if (in_place)
    return check_cuda(cudaLaunchKernelEx(&cfg, slice == 32 ? paged::evict_shift_kernel<32> : paged::evict_shift_kernel<64>, g, row),
                      "launch evict_shift_kernel");
  auto kern = row == 64    ? (vecs == 8 ? paged::evict_move_kernel<64, 8> : paged::evict_move_kernel<64, 32>)
              : row == 128 ? (vecs == 8 ? paged::evict_move_kernel<128, 8> : paged::evict_move_kernel<128, 32>)
                           : (vecs == 8 ? paged::evict_move_kernel<256, 8> : paged::evict_move_kernel<256, 32>);
  return check_cuda(cudaLaunchKernelEx(&cfg, kern, g, (int)chunks, warps), "launch evict_move_kernel");
}
