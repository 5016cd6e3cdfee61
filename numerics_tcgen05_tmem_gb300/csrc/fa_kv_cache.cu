// Writing new tokens' keys and values into a paged cache (fa_kv_append) and reading a cache back
// as packed BF16 rows (fa_kv_read).
//
// Both move each vector (one head's key or value of one token, d elements) once: bandwidth work.
// The threads of a CTA look its tokens up, one each (sequence, page, slot: four loads that wait for one
// another), then its warps walk the tokens' vectors, eight loads of each lane in flight, so dealt
// that neighbouring lanes take neighbouring slots of one head, which follow one another in the cache, as do
// their scales.  26k tokens of 8 heads, d = 128: into E4M3 30 us, 80 % of the measured copy rate,
// into BF16 34 us, 93 %; 53k tokens back from E4M3 54 us, 91 %, from BF16 67 us, 97 %; half the
// elements (d = 64) 18, 19, 30, 36 us.  With a warp for each token and its 2 Hkv vectors instead: 33, 34,
// 64, 67 us, at d = 64 21, 19, 47, 58, and 8 to 27 us with one head (now 4 to 9).
// E4M3 caches: scale = least power of two with max|x| <= 448 scale, code = E4M3(x / scale) (the
// division is exact, one rounding to nearest even), value = code * scale (exact in BF16, whose 8
// significant bits hold the code's 4; only with scales under 2^-124 do the smallest codes fall
// between BF16's subnormals and are rounded).  A vector that holds a NaN or an Inf gets a NaN scale and
// reads back as NaN.
#include <type_traits>

#include "paged_attn.cuh"

namespace fa {
namespace paged {

constexpr int kThreads = 256;

// Largest magnitude of a vector whose 8-element parts (BF16) are with kLanes neighbouring lanes, as
// FP32 bits: magnitudes order like unsigned integers (Inf and NaN above the rest), two per operation.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
template <int kLanes>
__device__ __forceinline__ uint32_t vector_amax(const uint4& u) {
  uint32_t m = max_u16x2(max_u16x2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), max_u16x2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
  return max(m << 16, m & 0xFFFF0000u);
}

__device__ __forceinline__ uint32_t quant4(uint32_t w0, uint32_t w1, float inv) {
  float a, b, c, d;
  mul2(a, b, __uint_as_float(w0 << 16), __uint_as_float(w0 & 0xFFFF0000u), inv, inv);
  mul2(c, d, __uint_as_float(w1 << 16), __uint_as_float(w1 & 0xFFFF0000u), inv, inv);
  return pack_e4m3x4(a, b, c, d);
}

// Magnitudes above 1.875 * 2^127 to that value: with the largest scale their code would be
// 256 = 2^8, whose value 2^128 overflows.
__device__ __forceinline__ uint4 clamp_top(const uint4& u) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = min(w[i] & 0x7FFFu, 0x7F70u), hi = min(w[i] & 0x7FFF0000u, 0x7F700000u);
    w[i] = (w[i] & 0x80008000u) | lo | hi;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Where a CTA's tokens lie in the cache: page (negative: skip the token) and slot.
struct Places {
  int page[kThreads], slot[kThreads];
};

// D / 8 lanes take 8 elements each of a vector, a warp kVecs vectors at a time, each lane kUnroll
// of those in flight.
template <int D>
struct Deal {
  static constexpr int kLanes = D / 8;
  static constexpr int kVecs = 32 / kLanes;
  static constexpr int kUnroll = 8;
  static constexpr int kStep = kVecs * (kThreads / 32);   // vectors of the CTA's warps together
};

// k_new, v_new: [T, Hkv, d] with `stride` elements between tokens; 2^shift of them per CTA, where
// 2^shift divides Deal::kStep: a thread's vectors are all of one token, K and V of every per_step-th
// head, whose addresses cost an addition.  (Any deal over the CTA's tokens, as in read_tokens: 37 us.)
template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const Cache c, const __nv_bfloat16* __restrict__ k_new,
                                                             const __nv_bfloat16* __restrict__ v_new,
                                                             long long stride, const int32_t* __restrict__ q_indptr,
                                                             int T, int shift) {
  using L = Deal<D>;
  __shared__ Places at;
  const int lane = threadIdx.x % 32, tokens = 1 << shift, first = blockIdx.x << shift;
  const int page_size = 1 << c.page_shift;
  if ((int)threadIdx.x < tokens) {
    const int token = first + threadIdx.x;
    int page = -1, pos = 0;
    const int b = token < T ? find_sequence(q_indptr, c.B, token) : -1;
    if (b >= 0) {
      pos = __ldg(c.kv_len + b) - __ldg(q_indptr + b + 1) + token;
      page = find_page(c, b, pos, kSitePagedAppend);
    }
    at.page[threadIdx.x] = page;
    at.slot[threadIdx.x] = pos & (page_size - 1);
  }
  __syncthreads();
  const int col = (lane % L::kLanes) * 8, v = threadIdx.x / L::kLanes, t = v & (tokens - 1);
  const int page = at.page[t], slot = at.slot[t], per_step = L::kStep >> shift;
  const int h_lane = v >> shift, h_warp = (threadIdx.x / 32 * L::kVecs) >> shift;   // the warp's least
  const long long src = (first + t) * stride + col, dst = page * c.page_stride + (long long)slot * D + col;
  const long long head = (long long)page_size * D, s_dst = page * c.scale_stride + slot;
  for (int j0 = 0; j0 + h_warp < c.Hkv; j0 += L::kUnroll / 2 * per_step) {
    uint4 x[L::kUnroll];
#pragma unroll
    for (int u = 0; u < L::kUnroll; ++u) {
      const int h = j0 + u / 2 * per_step + h_lane;
      x[u] = make_uint4(0, 0, 0, 0);
      if (h < c.Hkv && page >= 0) x[u] = __ldg(reinterpret_cast<const uint4*>((u & 1 ? v_new : k_new) + src + h * D));
    }
#pragma unroll
    for (int u = 0; u < L::kUnroll; ++u) {
      const int h = j0 + u / 2 * per_step + h_lane;
      if (j0 + u / 2 * per_step + h_warp >= c.Hkv) break;  // the same for the whole warp
      const bool mine = h < c.Hkv && page >= 0;
      if constexpr (!kFp8) {
        __nv_bfloat16* base = static_cast<__nv_bfloat16*>(u & 1 ? c.v : c.k);
        if (mine) *reinterpret_cast<uint4*>(base + dst + h * head) = x[u];
      } else {
        const uint32_t amax = vector_amax<L::kLanes>(x[u]);
        float scale = 1.f, inv = 1.f;
        int e = 0;
        if (amax != 0) {
          e = scale_exponent(amax);
          scale = __uint_as_float((uint32_t)(e + 127) << 23);
          inv = __uint_as_float((uint32_t)(127 - e) << 23);
        }
        if (e == kMaxScaleExp) x[u] = clamp_top(x[u]);
        uint2 q = make_uint2(quant4(x[u].x, x[u].y, inv), quant4(x[u].z, x[u].w, inv));
        if (amax >= 0x7F800000u) {  // Inf or NaN in the vector
          scale = __uint_as_float(0x7FC00000u);
          q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        }
        if (mine) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(u & 1 ? c.v : c.k) + dst + h * head) = q;
          if (col == 0) (u & 1 ? c.v_scale : c.k_scale)[s_dst + (long long)h * page_size] = scale;
        }
      }
    }
  }
}

// The K and V rows of a CTA's 2^shift tokens as BF16: token t's of head h go to k_out and v_out +
// t * token_stride + h * head_stride.  Vector v is the one of token v % 2^shift and of head i / 2, K where
// i = v / 2^shift is even: up to 256 tokens fill the warps' loads however few heads there are.
template <int D, bool kFp8>
__device__ __forceinline__ void read_tokens(const Cache& c, const Places& at, int shift, __nv_bfloat16* k_out,
                                            __nv_bfloat16* v_out, long long token_stride, long long head_stride) {
  // 8 elements per lane: a warp's stores then cover whole lines (with 16 codes per lane each 16-byte
  // store left half of its sector to the next one)
  using L = Deal<D>;
  constexpr int kBytes = kFp8 ? 1 : 2;
  using Part = std::conditional_t<kFp8, uint2, uint4>;   // a lane's elements in the cache
  const int lane = threadIdx.x % 32, sub = lane / L::kLanes, col = (lane % L::kLanes) * 8;
  const int tokens = 1 << shift, all = 2 * c.Hkv << shift, page_size = 1 << c.page_shift;
  for (int v0 = threadIdx.x / 32 * L::kVecs; v0 < all; v0 += L::kUnroll * L::kStep) {
    Part x[L::kUnroll];
    float sc[L::kUnroll];
#pragma unroll
    for (int u = 0; u < L::kUnroll; ++u) {
      const int v = v0 + u * L::kStep + sub, t = v & (tokens - 1), i = v >> shift;
      const int page = v < all ? at.page[t] : -1;
      x[u] = Part{};
      sc[u] = 0.f;
      if (page >= 0) {
        const long long row = (long long)(i >> 1) * page_size + at.slot[t];
        const uint8_t* base = static_cast<const uint8_t*>((i & 1) ? c.v : c.k);
        x[u] = __ldg(reinterpret_cast<const Part*>(base + (page * c.page_stride + row * D + col) * kBytes));
        if constexpr (kFp8) sc[u] = __ldg(((i & 1) ? c.v_scale : c.k_scale) + page * c.scale_stride + row);
      }
    }
#pragma unroll
    for (int u = 0; u < L::kUnroll; ++u) {
      const int v = v0 + u * L::kStep + sub, t = v & (tokens - 1), i = v >> shift;
      if (v >= all || at.page[t] < 0) continue;
      uint4* dst = reinterpret_cast<uint4*>(((i & 1) ? v_out : k_out) + t * token_stride + (i >> 1) * head_stride + col);
      if constexpr (!kFp8) {
        *dst = x[u];
      } else {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = e4m3x2_to_float2((e < 2 ? x[u].x : x[u].y) >> (16 * (e & 1)));
          float lo, hi;
          mul2(lo, hi, f.x, f.y, sc[u], sc[u]);
          o[e] = pack_bf16x2(lo, hi);
        }
        *dst = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// k_out, v_out: [rows, Hkv, d] contiguous; 2^shift rows per CTA.
template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const Cache c, const int32_t* __restrict__ kv_indptr,
                                                           __nv_bfloat16* __restrict__ k_out,
                                                           __nv_bfloat16* __restrict__ v_out, int rows, int shift) {
  __shared__ Places at;
  const int first = blockIdx.x << shift;
  if (threadIdx.x < 1 << shift) {
    const int r = first + threadIdx.x;
    int page = -1, pos = 0;
    const int b = r < rows ? find_sequence(kv_indptr, c.B, r) : -1;
    if (b >= 0) {
      pos = r - __ldg(kv_indptr + b);
      // past the sequence the row stays as it was
      if (pos < __ldg(c.kv_len + b)) page = find_page(c, b, pos, kSitePagedRead);
    }
    at.page[threadIdx.x] = page;
    at.slot[threadIdx.x] = pos & ((1 << c.page_shift) - 1);
  }
  __syncthreads();
  const long long stride = (long long)c.Hkv * D;
  read_tokens<D, kFp8>(c, at, shift, k_out + first * stride, v_out + first * stride, stride, D);
}

// The E4M3 keys and values that the chunk kernel's sequences see, as a BF16 cache of its own (pages of 128
// tokens, a table and a pool in the workspace): a tile would multiply every code by its scale anew.
// Sequence b's seen blocks of 128 keys have p.copy_pages pages from b * p.copy_pages on: those that
// hold sinks, then those from its window on.  per_seq CTAs share them, 2^shift <= 128 tokens of a page at
// a time: their number follows the sequences, not the table's width, whose unused part costs nothing.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_copy_kernel(const Attn p, const Cache to, int shift, int per_seq) {
  constexpr int kBlk = 1 << kCopyShift;
  __shared__ Places at;
  const int b = blockIdx.x / per_seq, parts = kBlk >> shift;
  const Seq s = load_seq(p, b);
  if (s.n == 0 || s.n * p.group <= p.few_rows) return;
  const KeyWalk<kBlk> walk(p, s.pos0, s.kv - 1);
  const int n_sink = (walk.sinks + kBlk - 1) / kBlk, from = max(walk.b_lo, n_sink);
  const int pages = min(n_sink + max((walk.hi + kBlk - 1) / kBlk - from, 0), p.copy_pages);
  for (int x = blockIdx.x - b * per_seq; x < pages * parts; x += per_seq) {
    const int slot = x / parts, i = slot < n_sink ? slot : from + slot - n_sink;
    const int part = (x - slot * parts) << shift, first = i * kBlk + part;
    if (i >= to.max_pages) return;
    const int page_to = b * p.copy_pages + slot;
    if (part == 0 && threadIdx.x == 0) const_cast<int32_t*>(to.table)[b * to.table_stride + i] = page_to;
    if (!walk.any(first, 1 << shift)) continue;
    __syncthreads();   // the last part's places have been read
    if (threadIdx.x < 1 << shift) {
      const int key = first + threadIdx.x;
      at.page[threadIdx.x] = walk.seen(key) ? find_page(p.c, b, key, kSitePagedPage) : -1;
      at.slot[threadIdx.x] = key & ((1 << p.c.page_shift) - 1);
    }
    __syncthreads();
    const long long row = page_to * to.page_stride + (long long)part * D;
    read_tokens<D, true>(p.c, at, shift, static_cast<__nv_bfloat16*>(to.k) + row, static_cast<__nv_bfloat16*>(to.v) + row, D,
                         (long long)kBlk * D);
  }
}

// log2 of the tokens of a CTA: as many as give it 32768 elements (two steps of eight loads for each
// lane), a lookup per thread at most; fewer, but not under 8, where that leaves SMs without a CTA.
static int tokens_shift(int Hkv, int d, long long rows) {
  int shift = 8;
  while (shift > 0 && (2ll * Hkv * d << shift) > 32768) --shift;
  while (shift > 3 && rows < (long long)sm_count() << shift) --shift;
  return shift;
}

int launch_copy(const Attn& p, const Cache& to, int d, cudaStream_t s) {
  const int tokens = tokens_shift(p.c.Hkv, d, (long long)p.copy_pages * p.c.B << kCopyShift);
  const int shift = tokens < kCopyShift ? tokens : kCopyShift;
  // eight CTAs per SM over all sequences, but 64 for each, one of which may hold most keys
  const long long most = (long long)p.copy_pages << (kCopyShift - shift);
  const long long share = (8ll * sm_count() + p.c.B - 1) / p.c.B, wanted = share > 64 ? share : 64;
  const int per_seq = (int)(wanted < most ? wanted : most);
  const unsigned grid = (unsigned)per_seq * p.c.B;
  if (d == 64)
    kv_copy_kernel<64><<<grid, kThreads, 0, s>>>(p, to, shift, per_seq);
  else
    kv_copy_kernel<128><<<grid, kThreads, 0, s>>>(p, to, shift, per_seq);
  return check_cuda(cudaGetLastError(), "launch kv_copy_kernel");
}

int check_cache(const fa_paged_kv* kv, Cache* c) {
  if (!kv) return set_error(FA_ERR_INVALID_ARG, "kv is NULL");
  if (kv->B < 1 || kv->Hkv < 1) return set_error(FA_ERR_INVALID_ARG, "B, Hkv must be >= 1 (got %d, %d)", kv->B, kv->Hkv);
  if (kv->d != 64 && kv->d != 128)
    return set_error(FA_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", kv->d);
  if (kv->page_size < 16 || kv->page_size > 256 || (kv->page_size & (kv->page_size - 1)))
    return set_error(FA_ERR_UNSUPPORTED, "page_size=%d not supported (16, 32, 64, 128 or 256)", kv->page_size);
  if (kv->num_pages < 1 || kv->max_pages < 1)
    return set_error(FA_ERR_INVALID_ARG, "num_pages, max_pages must be >= 1 (got %d, %d)", kv->num_pages, kv->max_pages);
  // positions, and differences of two of them, stay within 32 bits
  if ((long long)kv->max_pages * kv->page_size > (1ll << 30))
    return set_error(FA_ERR_INVALID_ARG, "max_pages * page_size must be <= 2^30");
  if (kv->dtype != FA_KV_BF16 && kv->dtype != FA_KV_E4M3)
    return set_error(FA_ERR_UNSUPPORTED, "cache dtype %d not supported (FA_KV_BF16 or FA_KV_E4M3)", kv->dtype);
  int rc;
  if ((rc = check_ptr(kv->k, "kv->k")) || (rc = check_ptr(kv->v, "kv->v"))) return rc;
  const long long page = (long long)kv->Hkv * kv->page_size;
  const int align = kv->dtype == FA_KV_E4M3 ? 16 : 8;  // 16 bytes
  if (kv->page_stride < page * kv->d || kv->page_stride % align)
    return set_error(FA_ERR_INVALID_ARG, "page_stride %lld must be a multiple of %d and at least Hkv*page_size*d = %lld",
                     (long long)kv->page_stride, align, page * kv->d);
  if (kv->dtype == FA_KV_E4M3) {
    if ((rc = check_ptr(kv->k_scale, "kv->k_scale")) || (rc = check_ptr(kv->v_scale, "kv->v_scale"))) return rc;
    if (kv->scale_stride < page || kv->scale_stride % 4)
      return set_error(FA_ERR_INVALID_ARG, "scale_stride %lld must be a multiple of 4 and at least Hkv*page_size = %lld",
                       (long long)kv->scale_stride, page);
  }
  if (!kv->block_table || (reinterpret_cast<uintptr_t>(kv->block_table) & 3))
    return set_error(FA_ERR_INVALID_ARG, "block_table must be a 4-byte aligned device pointer");
  if (kv->table_stride < kv->max_pages)
    return set_error(FA_ERR_INVALID_ARG, "table_stride %lld is less than max_pages %d", (long long)kv->table_stride,
                     kv->max_pages);
  if (!kv->kv_len || (reinterpret_cast<uintptr_t>(kv->kv_len) & 3))
    return set_error(FA_ERR_INVALID_ARG, "kv_len must be a 4-byte aligned device pointer");
  int shift = 4;
  while ((1 << shift) < kv->page_size) ++shift;
  *c = Cache{kv->k,     kv->v,     kv->k_scale, kv->v_scale, kv->page_stride, kv->scale_stride, kv->block_table,
             kv->table_stride, kv->kv_len, kv->B, kv->Hkv, shift, kv->num_pages, kv->max_pages, nullptr};
  return FA_OK;
}

int check_weights(const fa_paged_kv* kv, const float* weights, long long stride) {
  const int rc = check_ptr(weights, "weights");
  if (rc) return rc;
  const long long page = (long long)kv->Hkv * kv->page_size;
  if (stride < page || stride % 4)
    return set_error(FA_ERR_INVALID_ARG, "weight_stride %lld must be a multiple of 4 and at least Hkv*page_size = %lld", stride, page);
  return FA_OK;
}

int check_indptr(const int32_t* p, const char* name) {
  if (!p || (reinterpret_cast<uintptr_t>(p) & 3))
    return set_error(FA_ERR_INVALID_ARG, "%s must be a 4-byte aligned device pointer", name);
  return FA_OK;
}

}  // namespace paged
}  // namespace fa

extern "C" int fa_kv_append(const fa_paged_kv* kv, const void* k_new, const void* v_new, int64_t new_stride,
                            const int32_t* q_indptr, int T, void* stream) {
  fa::NvtxRange nvtx_range("fa_kv_append");
  using namespace fa;
  clear_error();
  paged::Cache c;
  int rc;
  if ((rc = paged::check_cache(kv, &c))) return rc;
  if (T < 0) return set_error(FA_ERR_INVALID_ARG, "T must be >= 0 (got %d)", T);
  if ((rc = check_ptr(k_new, "k_new")) || (rc = check_ptr(v_new, "v_new")) ||
      (rc = paged::check_indptr(q_indptr, "q_indptr")))
    return rc;
  if (new_stride < (int64_t)kv->Hkv * kv->d || new_stride % 8)
    return set_error(FA_ERR_INVALID_ARG, "new_stride %lld must be a multiple of 8 and at least Hkv*d = %d",
                     (long long)new_stride, kv->Hkv * kv->d);
  if (T == 0) return FA_OK;
  c.status = device_status_word();
  if (!c.status) return set_error(FA_ERR_CUDA, "could not allocate the device status record");
  const int most = kv->d == 64 ? 5 : 4, wanted = paged::tokens_shift(kv->Hkv, kv->d, T);   // kStep tokens
  const int shift = wanted < most ? wanted : most;
  const unsigned grid = (unsigned)((((long long)T - 1) >> shift) + 1);
  const __nv_bfloat16 *k = static_cast<const __nv_bfloat16*>(k_new), *v = static_cast<const __nv_bfloat16*>(v_new);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool fp8 = kv->dtype == FA_KV_E4M3;
  auto kern = kv->d == 64 ? (fp8 ? paged::kv_append_kernel<64, true> : paged::kv_append_kernel<64, false>)
                          : (fp8 ? paged::kv_append_kernel<128, true> : paged::kv_append_kernel<128, false>);
  kern<<<grid, paged::kThreads, 0, s>>>(c, k, v, new_stride, q_indptr, T, shift);
  return check_cuda(cudaGetLastError(), "launch fa_kv_append");
}

extern "C" int fa_kv_read(const fa_paged_kv* kv, const int32_t* kv_indptr, void* k_out, void* v_out, int rows,
                          void* stream) {
  fa::NvtxRange nvtx_range("fa_kv_read");
  using namespace fa;
  clear_error();
  paged::Cache c;
  int rc;
  if ((rc = paged::check_cache(kv, &c))) return rc;
  if (rows < 0) return set_error(FA_ERR_INVALID_ARG, "rows must be >= 0 (got %d)", rows);
  if ((rc = check_ptr(k_out, "k_out")) || (rc = check_ptr(v_out, "v_out")) ||
      (rc = paged::check_indptr(kv_indptr, "kv_indptr")))
    return rc;
  if (rows == 0) return FA_OK;
  c.status = device_status_word();
  if (!c.status) return set_error(FA_ERR_CUDA, "could not allocate the device status record");
  const int shift = paged::tokens_shift(kv->Hkv, kv->d, rows);
  const unsigned grid = (unsigned)((((long long)rows - 1) >> shift) + 1);
  __nv_bfloat16 *k = static_cast<__nv_bfloat16*>(k_out), *v = static_cast<__nv_bfloat16*>(v_out);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool fp8 = kv->dtype == FA_KV_E4M3;
  auto kern = kv->d == 64 ? (fp8 ? paged::kv_read_kernel<64, true> : paged::kv_read_kernel<64, false>)
                          : (fp8 ? paged::kv_read_kernel<128, true> : paged::kv_read_kernel<128, false>);
  kern<<<grid, paged::kThreads, 0, s>>>(c, kv_indptr, k, v, rows, shift);
  return check_cuda(cudaGetLastError(), "launch fa_kv_read");
}
