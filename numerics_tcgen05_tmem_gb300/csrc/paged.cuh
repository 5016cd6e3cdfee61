// What the paged key/value cache kernels share: the cache's description, the lookup of a packed
// row's sequence and of a position's page, and the E4M3 vector format.
//
// A cache is a pool of pages [num_pages][Hkv][page_size][d] for K and one for V.  Position t of
// sequence b lies in page block_table[b][t / page_size] at slot t % page_size.  The lengths, the
// table and the offsets are read on the device, so a call captured into a graph follows them; each
// entry is checked where it is used (a bad one is recorded and skipped, never followed).
#pragma once

#include <cuda_bf16.h>
#include <math.h>

#include "fa_host.h"
#include "sm103.cuh"

namespace fa {
namespace paged {

struct Cache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  long long page_stride;   // elements from one page to the next
  long long scale_stride;  // floats from one page's scales to the next
  const int32_t* table;
  long long table_stride;
  const int32_t* kv_len;
  int B, Hkv, page_shift, num_pages, max_pages;
  DevStatus* status;
};

// Largest E4M3 magnitude 448 = 1.75 * 2^8.  The scale of a vector is the least power of two that
// brings its largest magnitude within it, so x / scale, and a code times the scale, are exact.
constexpr uint32_t kMant448 = 0x600000;  // mantissa bits of 1.75
constexpr int kMinScaleExp = -126;       // scales and their reciprocals stay normal
constexpr int kMaxScaleExp = 120;        // of the largest finite vectors

// The scale exponent of a vector whose largest magnitude has these FP32 bits (finite, not zero).
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127;  // a subnormal's -127 ends at the clamp like its true one
  const int k = (amax_bits & 0x7FFFFFu) <= kMant448 ? e - 8 : e - 7;
  return max(k, kMinScaleExp);
}

// Two E4M3 codes (low 16 bits) as FP32; every code is exact in half precision.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  uint32_t h;
  asm("{\n .reg .b16 c, hi;\n mov.b32 {c, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, c;\n}" : "=r"(h) : "r"(codes));
  float lo, hi;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}

// The sequence of packed row `row`: the b with offsets[b] <= row < offsets[b + 1]; -1 when there is
// none (a row behind the last sequence).
__device__ __forceinline__ int find_sequence(const int32_t* offsets, int B, int row) {
  int lo = 0, hi = B + 1;   // offsets[0 .. lo) <= row < offsets[hi ..)
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (__ldg(offsets + mid) <= row)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo - 1 < B ? lo - 1 : -1;
}

// The page of position `pos` of sequence b; -1, recorded at `site`, where the table or the
// position is out of range.
__device__ __forceinline__ int find_page(const Cache& c, int b, int pos, uint32_t site) {
  const int i = pos >> c.page_shift;
  if (pos < 0 || i >= c.max_pages) {
    report_bounds(c.status, site, pos);
    return -1;
  }
  const int page = __ldg(c.table + b * c.table_stride + i);
  if (page < 0 || page >= c.num_pages) {
    report_bounds(c.status, site, page);
    return -1;
  }
  return page;
}

// Host side: checks a public cache description and fills `c`.
int check_cache(const fa_paged_kv* kv, Cache* c);

}  // namespace paged
}  // namespace fa
