// Eviction from a paged cache by accumulated attention weight (fa_kv_evict): of each sequence and kv head `keep`
// keys stay -- the first `sinks`, the newest `recent`, and of the others those with the largest weights (of equal
// ones the first) -- and move, in order, to the first positions of the sequence in another block table, or
// in the same one.
//
//   select  a CTA per (sequence, kv head): the smallest weight that stays, by three passes over the weights' bits
//           (11, 11 and 10 of them, a histogram each in shared memory), then one pass in order that writes the
//           kept positions.
//   move    the kept vectors, their scales and weights: bandwidth work, 16 bytes a thread.
// In place a vector only ever moves to a lower position, to where nothing is that is still to be read as long
// as the vectors are taken in order: a CTA takes all of one head's K or V, 64 bytes wide, step by step, and
// waits between a step's loads and its stores.
#include <algorithm>

#include "paged_attn.cuh"

namespace fa {
namespace paged {

constexpr int kSelectThreads = 512;
constexpr int kDigit = 11, kBins = 1 << kDigit;
constexpr int kCached = 16384;   // weights that stay in shared memory between the passes

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

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const __grid_constant__ Evict g) {
  constexpr int kWarps = kSelectThreads / 32, kStep = 4 * kSelectThreads;   // a thread has four keys at a time
  extern __shared__ __align__(16) uint32_t cached[];
  __shared__ uint32_t bins[kBins];
  __shared__ int warp_sum[kWarps];
  __shared__ int found_bin, found_above;
  cudaTriggerProgrammaticLaunchCompletion();   // the moving kernel may get ready; it waits for this one's end
  const int b = blockIdx.x / g.c.Hkv, h = blockIdx.x - b * g.c.Hkv;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int n = evict_length(g.c, b), kept = min(n, g.keep);
  int32_t* out = g.kept + (long long)blockIdx.x * g.keep;
  if (h == 0 && threadIdx.x == 0) g.kept_len[b] = kept;
  for (int i = kept + (int)threadIdx.x; i < g.keep; i += kSelectThreads) out[i] = -1;
  if (n <= g.keep) {
    for (int i = threadIdx.x; i < n; i += kSelectThreads) out[i] = i;
    return;
  }
  const int page_mask = (1 << g.c.page_shift) - 1;
  const int32_t* table = g.c.table + b * g.c.table_stride;
  // the order of the four weights at `key`, which lie in one page
  auto read = [&](int key) {
    const int page = __ldg(table + (key >> g.c.page_shift));
    if (page < 0 || page >= g.c.num_pages) {
      report_bounds(g.c.status, kSitePagedEvict, page);
      return make_uint4(0, 0, 0, 0);
    }
    const float4 w = *reinterpret_cast<const float4*>(g.weights + page * g.weight_stride + ((long long)h << g.c.page_shift) +
                                                      (key & page_mask));
    return make_uint4(weight_order(w.x), weight_order(w.y), weight_order(w.z), weight_order(w.w));
  };
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
      for (int key = 4 * (int)threadIdx.x; key < hi; key += kStep) {
        const uint4 u = pass == 0 ? read(key) : again(key);
        if (pass == 0 && key < kCached) *reinterpret_cast<uint4*>(cached + key) = u;   // read back by this thread
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key + e >= lo && key + e < hi && (pass == 0 || (x[e] >> above) == prefix))
            atomicAdd(&bins[x[e] >> shift & ((1 << digit) - 1)], 1u);
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
  for (int base = 0; base < n; base += kStep) {
    const int key = base + 4 * (int)threadIdx.x;
    uint32_t x[4] = {0, 0, 0, 0};
    if (want > 0 && key < hi) {
      const uint4 u = again(key);
      x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    }
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
      if (sure[e] || (equal[e] && at_equal < ties)) out[at_sure + min(at_equal, ties)] = key + e;
      at_sure += sure[e] ? 1 : 0;
      at_equal += equal[e] ? 1 : 0;
    }
    sure_before += all & 0xFFFF;
    equal_before += all >> 16;
    __syncthreads();
  }
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

// Into other pages.  A warp has 32 kept keys of one (sequence, kv head): a lane looks one up and moves its scales and
// weight, then kRow / 16 lanes move a vector, eight loads of each lane in flight.
constexpr int kMoveThreads = 256, kMoveVecs = 32;

template <int kRow>    // bytes of a vector
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ Evict g, int chunks, long long warps) {
  constexpr int kLanes = kRow / 16, kGroups = 32 / kLanes, kSteps = kMoveVecs / kGroups, kUnroll = 8;
  static_assert(2 * kSteps % kUnroll == 0, "K and V in whole rounds");
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x % 32;
  const long long w = (long long)blockIdx.x * (kMoveThreads / 32) + threadIdx.x / 32;
  if (w >= warps) return;
  const int item = (int)(w / chunks), first = (int)(w - (long long)item * chunks) * kMoveVecs;
  const int b = item / g.c.Hkv, h = item - b * g.c.Hkv;
  const int here = min(g.kept_len[b] - first, kMoveVecs);
  if (here <= 0) return;
  const long long page_size = 1ll << g.c.page_shift;
  const int elem = g.c.k_scale != nullptr ? 1 : 2;
  long long from = -1, to = -1;       // the lane's vector: bytes from the pool's start
  if (lane < here) {
    const Spot f = spot_of(g.c, g.c.table, g.c.table_stride, g.c.max_pages, b, g.kept[(long long)item * g.keep + first + lane]);
    const Spot t = spot_of(g.c, g.table_out, g.table_out_stride, g.max_pages_out, b, first + lane);
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
    long long dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int s = s0 + u, v = s / 2 * kGroups + lane / kLanes;      // K and V of the same vectors in turn
      const long long src = __shfl_sync(0xffffffffu, from, v);
      dst[u] = __shfl_sync(0xffffffffu, to, v);
      if (dst[u] >= 0) x[u] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>((s & 1) ? g.c.v : g.c.k) + src + col);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (dst[u] >= 0) *reinterpret_cast<uint4*>(static_cast<uint8_t*>(((s0 + u) & 1) ? g.c.v : g.c.k) + dst[u] + col) = x[u];
  }
}

// Within the same pages.  A CTA has one (sequence, kv head), K or V, 64 bytes of each vector; the first slice's
// CTAs also move the scales, that of K the weights.
constexpr int kSlice = 64;

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
  for (int i0 = 0; i0 < kept; i0 += kStep) {
    uint4 x[kUnroll];
    float s[kUnroll];
    Spot to[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kGroups + group;
      to[u].page = -1;
      if (i >= kept) continue;
      const int key = keys[i];
      if (key == i) continue;            // it stays where it is
      const Spot f = spot_of(g.c, g.c.table, g.c.table_stride, g.c.max_pages, b, key);
      if (f.page < 0) continue;
      to[u] = spot_of(g.c, g.c.table, g.c.table_stride, g.c.max_pages, b, i);
      const long long at = h * page_size + f.slot;
      x[u] = *reinterpret_cast<const uint4*>(pool + f.page * page_bytes + at * row_bytes + col);
      if (moves_scale) s[u] = scales[f.page * g.c.scale_stride + at];
      if (moves_weight) s[u] = g.weights[f.page * g.weight_stride + at];
    }
    __syncthreads();   // every load of this step comes before its stores; those of the next step read higher positions
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (to[u].page < 0) continue;
      const long long at = h * page_size + to[u].slot;
      *reinterpret_cast<uint4*>(pool + to[u].page * page_bytes + at * row_bytes + col) = x[u];
      if (moves_scale) scales[to[u].page * g.c.scale_stride + at] = s[u];
      if (moves_weight) g.weights[to[u].page * g.weight_stride + at] = s[u];
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
  if (keep < 1 || sinks < 0 || recent < 0) return set_error(FA_ERR_INVALID_ARG, "keep must be >= 1, sinks and recent >= 0 (got %d, %d, %d)", keep, sinks, recent);
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
  const long long chunks = (most + paged::kMoveVecs - 1) / paged::kMoveVecs;
  if (items * std::max(chunks, 8ll) >= (1ll << 31))
    return set_error(FA_ERR_INVALID_ARG, "B*Hkv*keep/%d must be < 2^31", paged::kMoveVecs);
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
  constexpr int cache = paged::kCached * 4;
  static std::atomic<uint64_t> prepared{0};
  if ((rc = prepare_kernel(reinterpret_cast<const void*>(paged::evict_select_kernel), cache, paged::kSelectThreads, 0,
                           "evict_select_kernel", &prepared)))
    return rc;
  paged::evict_select_kernel<<<(unsigned)items, paged::kSelectThreads, cache, s>>>(g);
  if ((rc = check_cuda(cudaGetLastError(), "launch evict_select_kernel"))) return rc;
  const int row = kv->d * (kv->dtype == FA_KV_E4M3 ? 1 : 2);
  const long long warps = items * chunks, per = paged::kMoveThreads / 32;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(in_place ? items * 2 * (row / paged::kSlice) : (warps + per - 1) / per));
  cfg.blockDim = dim3(paged::kMoveThreads);
  cfg.stream = s;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  if (in_place) return check_cuda(cudaLaunchKernelEx(&cfg, paged::evict_shift_kernel, g, row), "launch evict_shift_kernel");
  auto kern = row == 64 ? paged::evict_move_kernel<64> : (row == 128 ? paged::evict_move_kernel<128> : paged::evict_move_kernel<256>);
  return check_cuda(cudaLaunchKernelEx(&cfg, kern, g, (int)chunks, warps), "launch evict_move_kernel");
}
