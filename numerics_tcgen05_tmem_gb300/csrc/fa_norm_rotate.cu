// Norm of queries and keys for each head and position rotation in one pass: dense with gradients
// (fa_norm_rotate, fa_norm_rotate_bwd), and for packed rows with the write into a paged cache (fa_qkv_append).
//
// A vector x is one head of one token, d elements; its first `rot` are rotated in pairs (a, b):
//   r = 1 / sqrt(mean x^2 + eps), y = w o x r,  z_a = y_a cos - y_b sin,  z_b = y_b cos + y_a sin.
// Backward: dy is dz rotated by the opposite angle, g = w o dy, dw = sum of dy o x r over the vectors,
//   dx = r g - x r^3 / d sum(x o g).
// r is computed again from x, which the backward reads in any case.
//
// Memory bounds all three: about 7 issue slots of a sub-partition go to a vector, while the copy rate gives
// an SM 20 clocks for its 512 bytes.  d / 16 lanes take a vector, each two 16-byte parts that hold both
// entries of its pairs, so that the rotation needs no exchange and the sums three (two) shuffles.
//
// Angles: position times frequency modulo one turn.  In FP32 a position of 2^20 would leave 0.06 rad of error.
// A frequency is kept as a fraction of a turn in 64 bits; the product with a 32-bit position wraps at whole
// turns by itself, and its upper 32 bits are the angle (error: pos * 2^-54 turns, from the double it comes from).
#include <cuda_bf16.h>
#include <math.h>

#include "paged_attn.cuh"

namespace fa {
namespace rotate {

using paged::Cache;

constexpr int kThreads = 256;
constexpr int kUnroll = 4;    // vectors in flight for each lane group (backward: kUnrollBwd)
constexpr int kUnrollBwd = 1;

// Lane groups: kLanes neighbouring lanes hold a vector, lane j the 8-element parts a(j) and b(j).
template <int D>
struct Lanes {
  static constexpr int kLanes = D / 16;
  static constexpr int kGroups = kThreads / kLanes;   // of a CTA
};

// How vectors are normed and rotated.
struct Plan {
  const double* inv_freq;
  int rot, norm;
  float eps;
};

// Queries or keys: where they lie and which CTAs have them.  2^shift lane groups share a token's heads.
struct Side {
  const __nv_bfloat16* x;
  long long x_b, x_h, x_n;     // strides of batch, head, token
  const __nv_bfloat16* dz;
  long long dz_b, dz_h, dz_n;
  __nv_bfloat16* out;          // forward: z; backward: dx
  long long out_b, out_h, out_n;
  const void* w;               // [d] or NULL
  int w_bf16, H, shift, ctas;
};

struct Parts {                 // a lane's parts of one vector
  float a[8], b[8];
};

__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// The first elements of lane j's parts.  Pairs (i, i + rot / 2): a and b lie rot / 2 apart.  Neighbouring
// pairs, and lanes behind the rotated entries: 16 elements in a row.
template <bool kInter>
__device__ __forceinline__ void part_columns(int j, int rot, int& a, int& b) {
  const bool split = !kInter && 16 * j < rot;
  a = split ? 8 * j : 16 * j;
  b = split ? 8 * j + rot / 2 : 16 * j + 8;
}

__device__ __forceinline__ void load_weights(const void* w, int is_bf16, int col, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = w == nullptr ? 1.f
                        : (is_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[col + i])
                                   : static_cast<const float*>(w)[col + i]);
}

// Sum over the lanes of a group.
template <int kLanes>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float inverse_rms(float sum, int d, const Plan& p) {
  return p.norm ? __frsqrt_rn(sum * (1.f / d) + p.eps) : 1.f;
}

// The pairs of a lane turned by its eight angles (kSign = -1: back).
template <bool kInter, int kSign>
__device__ __forceinline__ void turn(Parts& v, const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& x = kInter ? (i < 4 ? v.a[2 * i] : v.b[2 * i - 8]) : v.a[i];
    float& y = kInter ? (i < 4 ? v.a[2 * i + 1] : v.b[2 * i - 7]) : v.b[i];
    const float sn = kSign * s[i], x0 = x, y0 = y;
    x = x0 * c[i] - y0 * sn;
    y = y0 * c[i] + x0 * sn;
  }
}

// cos and sin of a tile's tokens.  The tables start behind the frequencies, kFreq of them.
struct Table {
  uint64_t* turns;   // [rot / 2] turns for each position, in units of 2^-64
  float* cos;        // [tokens][rot / 2]
  float* sin;
};
template <int D>
__device__ __forceinline__ Table table_at(void* smem, int tokens, int rot) {
  uint64_t* t = static_cast<uint64_t*>(smem);
  float* c = reinterpret_cast<float*>(t + D / 2);
  return Table{t, c, c + tokens * (rot / 2)};
}
// bytes for `tokens` tokens at a time
template <int D>
constexpr int table_bytes(int tokens) {
  return D / 2 * 8 + tokens * D * 4;
}

__device__ __forceinline__ void fill_turns(const Table& t, const Plan& p) {
  if ((int)threadIdx.x < p.rot / 2) {
    double f = p.inv_freq[threadIdx.x] * 0.15915494309189533577;   // 1 / (2 pi)
    f -= floor(f);
    t.turns[threadIdx.x] = f < 1.0 ? (uint64_t)__double2ull_rd(f * 18446744073709551616.0) : 0;
  }
}

// position(i): that of the tile's token i.  Every thread of the CTA calls it; a barrier has to follow.
template <class Position>
__device__ __forceinline__ void fill_angles(const Table& t, int rot, int tokens, Position position) {
  const int half = rot / 2;
  for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
    const int token = i / half, f = i - token * half;
    const uint64_t at = (uint64_t)(int64_t)position(token) * t.turns[f];
    // the nearest quarter turn apart, the rest is within an eighth: its rounding to FP32 stays under 2^-25 rad
    const uint32_t u = (uint32_t)(at >> 32), quarter = (u + 0x20000000u) >> 30;
    float s0, c0;
    sincospif((float)(int32_t)(u - (quarter << 30)) * 0x1p-31f, &s0, &c0);   // a turn is 2^32, sincospi's is 2
    float s = quarter & 1 ? c0 : s0, c = quarter & 1 ? s0 : c0;
    if (quarter & 2) s = -s;
    if ((quarter + 1) & 2) c = -c;
    t.cos[i] = c;
    t.sin[i] = s;
  }
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 u = reinterpret_cast<const float4*>(p)[0], v = reinterpret_cast<const float4*>(p)[1];
  f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
}
// A lane's angles of a token: 1 and 0 behind the rotated entries.
__device__ __forceinline__ void load_angles(const Table& t, int rot, int token, int j, float (&c)[8], float (&s)[8]) {
  if (16 * j < rot) {
    load8(t.cos + token * (rot / 2) + 8 * j, c);
    load8(t.sin + token * (rot / 2) + 8 * j, s);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  }
}

// One vector's parts normed and turned, in place.
template <int D, bool kInter>
__device__ __forceinline__ void forward_vector(Parts& v, const Plan& p, const float (&wa)[8], const float (&wb)[8],
                                               const float (&c)[8], const float (&s)[8]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += v.a[i] * v.a[i] + v.b[i] * v.b[i];
  const float r = inverse_rms(group_sum<Lanes<D>::kLanes>(sum), D, p);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v.a[i] = v.a[i] * r * wa[i];
    v.b[i] = v.b[i] * r * wb[i];
  }
  turn<kInter, 1>(v, c, s);
}

// (not through the read-only path: an output may be its input, every vector is read before it is written)
__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }

// The token of a dense batch: batch entry and place in it.
struct Place {
  long long b, n;
};
__device__ __forceinline__ Place place_of(long long token, int N) {
  const long long b = token / N;
  return Place{b, token - b * N};
}

struct Dense {
  Plan p;
  const int32_t* positions;   // NULL: 0, 1, ..
  long long pos_b;            // entries between two sequences' positions
  long long tokens;           // B * N
  int N;
};

__device__ __forceinline__ int dense_position(const Dense& g, long long token) {
  if (token >= g.tokens) return 0;
  const Place at = place_of(token, g.N);
  return g.positions == nullptr ? (int)at.n : __ldg(g.positions + at.b * g.pos_b + at.n);
}

// A CTA has kGroups >> shift tokens of one side; the first q.ctas CTAs are the queries'.
template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 2) norm_rotate_kernel(const __grid_constant__ Dense g,
                                                                  const __grid_constant__ Side q,
                                                                  const __grid_constant__ Side k) {
  using L = Lanes<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  const bool is_q = (int)blockIdx.x < q.ctas;
  const Side& side = is_q ? q : k;
  const int tokens = L::kGroups >> side.shift, groups = 1 << side.shift;
  const long long first = (long long)((int)blockIdx.x - (is_q ? 0 : q.ctas)) * tokens;
  const int group = threadIdx.x / L::kLanes, j = threadIdx.x % L::kLanes;
  const int mine = group >> side.shift, head0 = group & (groups - 1);
  const long long token = first + mine;
  const bool valid = token < g.tokens;
  const Place at = place_of(valid ? token : 0, g.N);
  int ca, cb;
  part_columns<kInter>(j, g.p.rot, ca, cb);
  const __nv_bfloat16* x = side.x + at.b * side.x_b + at.n * side.x_n;
  __nv_bfloat16* z = side.out + at.b * side.out_b + at.n * side.out_n;

  uint4 xa[kUnroll], xb[kUnroll];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * groups;
      if (valid && h < side.H) {
        xa[u] = load16(x + h * side.x_h + ca);
        xb[u] = load16(x + h * side.x_h + cb);
      }
    }
  };
  load(head0);   // in flight while the angles are computed
  const Table t = table_at<D>(smem, tokens, g.p.rot);
  fill_turns(t, g.p);
  float wa[8], wb[8], c[8], s[8];
  load_weights(side.w, side.w_bf16, ca, wa);
  load_weights(side.w, side.w_bf16, cb, wb);
  __syncthreads();
  fill_angles(t, g.p.rot, tokens, [&](int i) { return dense_position(g, first + i); });
  __syncthreads();
  load_angles(t, g.p.rot, mine, j, c, s);
  for (int h0 = head0; h0 - head0 < side.H; h0 += kUnroll * groups) {
    if (h0 != head0) load(h0);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * groups;
      if (h - head0 >= side.H) break;   // the same for the whole CTA: the shuffles need every lane
      Parts v;
      unpack(xa[u], v.a);
      unpack(xb[u], v.b);
      forward_vector<D, kInter>(v, g.p, wa, wb, c, s);
      if (valid && h < side.H) {
        *reinterpret_cast<uint4*>(z + h * side.out_h + ca) = pack(v.a);
        *reinterpret_cast<uint4*>(z + h * side.out_h + cb) = pack(v.b);
      }
    }
  }
}

// CTA i of a side takes its tiles i, i + ctas, ..; the weights' gradients are summed in registers, then
// over the CTA's groups, and the CTA's sum goes to part[CTA][d].
template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 2) norm_rotate_bwd_kernel(const __grid_constant__ Dense g,
                                                                      const __grid_constant__ Side q,
                                                                      const __grid_constant__ Side k,
                                                                      float* __restrict__ part) {
  using L = Lanes<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  const bool is_q = (int)blockIdx.x < q.ctas;
  const Side& side = is_q ? q : k;
  const int tokens = L::kGroups >> side.shift, groups = 1 << side.shift;
  const int cta = (int)blockIdx.x - (is_q ? 0 : q.ctas);
  const int group = threadIdx.x / L::kLanes, j = threadIdx.x % L::kLanes;
  const int mine = group >> side.shift, head0 = group & (groups - 1);
  int ca, cb;
  part_columns<kInter>(j, g.p.rot, ca, cb);
  const Table t = table_at<D>(smem, tokens, g.p.rot);
  fill_turns(t, g.p);
  float wa[8], wb[8], dwa[8], dwb[8];
  load_weights(side.w, side.w_bf16, ca, wa);
  load_weights(side.w, side.w_bf16, cb, wb);
#pragma unroll
  for (int i = 0; i < 8; ++i) dwa[i] = dwb[i] = 0.f;

  const long long tiles = (g.tokens + tokens - 1) / tokens;
  for (long long tile = cta; tile < tiles; tile += side.ctas) {
    const long long token = tile * tokens + mine;
    const bool valid = token < g.tokens;
    const Place at = place_of(valid ? token : 0, g.N);
    const __nv_bfloat16* x = side.x + at.b * side.x_b + at.n * side.x_n;
    const __nv_bfloat16* dz = side.dz + at.b * side.dz_b + at.n * side.dz_n;
    __nv_bfloat16* dx = side.out + at.b * side.out_b + at.n * side.out_n;
    uint4 xa[kUnrollBwd], xb[kUnrollBwd], za[kUnrollBwd], zb[kUnrollBwd];
    auto load = [&](int h0) {
#pragma unroll
      for (int u = 0; u < kUnrollBwd; ++u) {
        const int h = h0 + u * groups;
        xa[u] = xb[u] = za[u] = zb[u] = make_uint4(0, 0, 0, 0);   // adds nothing to the weights' gradient
        if (valid && h < side.H) {
          xa[u] = load16(x + h * side.x_h + ca);
          xb[u] = load16(x + h * side.x_h + cb);
          za[u] = load16(dz + h * side.dz_h + ca);
          zb[u] = load16(dz + h * side.dz_h + cb);
        }
      }
    };
    load(head0);
    __syncthreads();   // the turns are there; the last tile's angles have been read
    fill_angles(t, g.p.rot, tokens, [&](int i) { return dense_position(g, tile * tokens + i); });
    __syncthreads();
    float c[8], s[8];
    load_angles(t, g.p.rot, mine, j, c, s);
    for (int h0 = head0; h0 - head0 < side.H; h0 += kUnrollBwd * groups) {
      if (h0 != head0) load(h0);
#pragma unroll
      for (int u = 0; u < kUnrollBwd; ++u) {
        const int h = h0 + u * groups;
        if (h - head0 >= side.H) break;
        Parts v, dy;
        unpack(xa[u], v.a);
        unpack(xb[u], v.b);
        unpack(za[u], dy.a);
        unpack(zb[u], dy.b);
        turn<kInter, -1>(dy, c, s);
        float sum = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum += v.a[i] * v.a[i] + v.b[i] * v.b[i];
          dot += v.a[i] * (wa[i] * dy.a[i]) + v.b[i] * (wb[i] * dy.b[i]);
        }
        sum = group_sum<L::kLanes>(sum);
        dot = group_sum<L::kLanes>(dot);
        const float r = inverse_rms(sum, D, g.p);
        const float back = g.p.norm ? dot * r * r * (1.f / D) : 0.f;   // sum(x o g) r^2 / d
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float ua = v.a[i] * r, ub = v.b[i] * r;
          if (valid && h < side.H) {
            dwa[i] += dy.a[i] * ua;
            dwb[i] += dy.b[i] * ub;
          }
          v.a[i] = r * (wa[i] * dy.a[i]) - ua * back;
          v.b[i] = r * (wb[i] * dy.b[i]) - ub * back;
        }
        if (valid && h < side.H) {
          *reinterpret_cast<uint4*>(dx + h * side.out_h + ca) = pack(v.a);
          *reinterpret_cast<uint4*>(dx + h * side.out_h + cb) = pack(v.b);
        }
      }
    }
  }
  if (part == nullptr) return;
  // the groups' sums: one row of d for each group in shared memory, summed in order
  __syncthreads();
  float* rows = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    rows[group * D + ca + i] = dwa[i];
    rows[group * D + cb + i] = dwb[i];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f;
    for (int i = 0; i < L::kGroups; ++i) sum += rows[i * D + threadIdx.x];
    part[(long long)blockIdx.x * D + threadIdx.x] = sum;
  }
}

// The weights' gradients: the CTAs' sums, always in the same order.  A CTA has 32 columns of one side; its
// 32 warps take every 32nd part each.
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float* __restrict__ part, int d, int q_ctas, int k_ctas,
                                                           float* __restrict__ dqw, float* __restrict__ dkw) {
  __shared__ float sums[32][33];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const bool is_q = (int)blockIdx.x < d / 32;
  const int col = ((int)blockIdx.x - (is_q ? 0 : d / 32)) * 32 + lane;
  const float* from = part + (is_q ? 0 : (long long)q_ctas * d) + col;
  const int n = is_q ? q_ctas : k_ctas;
  float sum = 0.f;
#pragma unroll 4
  for (int i = warp; i < n; i += 32) sum += from[(long long)i * d];
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp == 0) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += sums[i][lane];
    (is_q ? dqw : dkw)[col] = sum;
  }
}

// ------------------------------------------------------------------ packed rows into a paged cache

struct Packed {
  Plan p;
  Cache c;
  const int32_t* q_indptr;
  const int32_t* positions;   // [T] or NULL: the places in the cache
  int T;
};

// A vector's parts as E4M3 codes with the scale rule of fa_kv_append; the FP32 values are rounded once.
template <int kLanes>
__device__ __forceinline__ void quantize(const Parts& v, uint2& ca, uint2& cb, float& scale) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    amax = max(amax, max(__float_as_uint(v.a[i]) & 0x7FFFFFFFu, __float_as_uint(v.b[i]) & 0x7FFFFFFFu));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  scale = 1.f;
  float inv = 1.f, top = __uint_as_float(0x7F7FFFFFu);
  if (amax != 0) {
    const int e = paged::scale_exponent(amax);
    scale = __uint_as_float((uint32_t)(e + 127) << 23);
    inv = __uint_as_float((uint32_t)(127 - e) << 23);
    if (e == paged::kMaxScaleExp) top = __uint_as_float(0x7F700000u);   // 1.875 2^127: see fa_kv_append
  }
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = fminf(fmaxf(v.a[i], -top), top) * inv;
    b[i] = fminf(fmaxf(v.b[i], -top), top) * inv;
  }
  ca = make_uint2(pack_e4m3x4(a[0], a[1], a[2], a[3]), pack_e4m3x4(a[4], a[5], a[6], a[7]));
  cb = make_uint2(pack_e4m3x4(b[0], b[1], b[2], b[3]), pack_e4m3x4(b[4], b[5], b[6], b[7]));
  if (amax >= 0x7F800000u) {   // Inf or NaN in the vector
    scale = __uint_as_float(0x7FC00000u);
    ca = cb = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  }
}

// A CTA has kGroups >> shift tokens of the queries, the keys or the values (in the order of the CTAs).
template <int D, bool kInter, bool kFp8>
__global__ void __launch_bounds__(kThreads, 2) qkv_append_kernel(const __grid_constant__ Packed g,
                                                                 const __grid_constant__ Side q, const __grid_constant__ Side k,
                                                                 const __grid_constant__ Side v) {
  using L = Lanes<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int at_page[L::kGroups], at_slot[L::kGroups], at_pos[L::kGroups];
  int cta = blockIdx.x;
  const int which = cta < q.ctas ? 0 : (cta < q.ctas + k.ctas ? 1 : 2);
  cta -= which == 0 ? 0 : (which == 1 ? q.ctas : q.ctas + k.ctas);
  const Side& side = which == 0 ? q : (which == 1 ? k : v);
  const int tokens = L::kGroups >> side.shift, groups = 1 << side.shift;
  const long long first = (long long)cta * tokens;
  const int group = threadIdx.x / L::kLanes, j = threadIdx.x % L::kLanes;
  const int mine = group >> side.shift, head0 = group & (groups - 1);
  const long long token = first + mine;
  const bool there = token < g.T;
  const int rot = which == 2 ? 0 : g.p.rot;
  int ca, cb;
  part_columns<kInter>(j, rot, ca, cb);
  const __nv_bfloat16* x = side.x + (there ? token : 0) * side.x_n;

  uint4 xa[kUnroll], xb[kUnroll];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * groups;
      if (there && h < side.H) {
        xa[u] = load16(x + h * side.x_h + ca);
        xb[u] = load16(x + h * side.x_h + cb);
      }
    }
  };
  load(head0);
  const Table t = table_at<D>(smem, tokens, rot);
  if (which != 2) fill_turns(t, g.p);
  if ((int)threadIdx.x < tokens) {
    const long long i = first + threadIdx.x;
    int page = -1, pos = 0;
    const int b = i < g.T ? paged::find_sequence(g.q_indptr, g.c.B, (int)i) : -1;
    if (b >= 0) {
      pos = __ldg(g.c.kv_len + b) - __ldg(g.q_indptr + b + 1) + (int)i;
      page = which == 0 ? 0 : paged::find_page(g.c, b, pos, kSitePagedAppend);
    }
    at_page[threadIdx.x] = page;
    at_slot[threadIdx.x] = pos & ((1 << g.c.page_shift) - 1);
    at_pos[threadIdx.x] = b >= 0 && g.positions != nullptr ? __ldg(g.positions + i) : pos;
  }
  float wa[8], wb[8], c[8], s[8];
  load_weights(side.w, side.w_bf16, ca, wa);
  load_weights(side.w, side.w_bf16, cb, wb);
  __syncthreads();
  fill_angles(t, rot, tokens, [&](int i) { return at_pos[i]; });
  __syncthreads();
  load_angles(t, rot, mine, j, c, s);
  const int page = at_page[mine];
  const bool valid = there && page >= 0;
  const long long page_size = 1ll << g.c.page_shift;
  const long long to = which == 0 ? token * side.out_n : page * g.c.page_stride + at_slot[mine] * (long long)D;
  const long long to_scale = page * g.c.scale_stride + at_slot[mine];
  for (int h0 = head0; h0 - head0 < side.H; h0 += kUnroll * groups) {
    if (h0 != head0) load(h0);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * groups;
      if (h - head0 >= side.H) break;
      const bool stores = valid && h < side.H;
      Parts y;
      unpack(xa[u], y.a);
      unpack(xb[u], y.b);
      if (which != 2) forward_vector<D, kInter>(y, g.p, wa, wb, c, s);
      if (which == 0) {
        if (stores) {
          *reinterpret_cast<uint4*>(side.out + to + h * side.out_h + ca) = pack(y.a);
          *reinterpret_cast<uint4*>(side.out + to + h * side.out_h + cb) = pack(y.b);
        }
      } else if constexpr (!kFp8) {
        if (stores) {
          __nv_bfloat16* row = static_cast<__nv_bfloat16*>(which == 1 ? g.c.k : g.c.v) + to + h * page_size * D;
          *reinterpret_cast<uint4*>(row + ca) = which == 2 ? xa[u] : pack(y.a);
          *reinterpret_cast<uint4*>(row + cb) = which == 2 ? xb[u] : pack(y.b);
        }
      } else {
        uint2 qa, qb;
        float scale;
        quantize<L::kLanes>(y, qa, qb, scale);
        if (stores) {
          uint8_t* row = static_cast<uint8_t*>(which == 1 ? g.c.k : g.c.v) + to + h * page_size * D;
          *reinterpret_cast<uint2*>(row + ca) = qa;
          *reinterpret_cast<uint2*>(row + cb) = qb;
          if (j == 0) (which == 1 ? g.c.k_scale : g.c.v_scale)[to_scale + h * page_size] = scale;
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------------ host side

// Lane groups for a token's H heads: as many as leave each group kUnroll heads, so that the angles are read
// once for those; more where the batch is too small for that to fill the SMs.
static int pick_shift(int H, int groups, int unroll, long long tokens) {
  int shift = 0;
  while ((unroll << shift) < H && (2 << shift) <= groups) ++shift;
  while ((1 << shift) < H && (2 << shift) <= groups && tokens * (1 << shift) < (long long)groups * 2 * sm_count()) ++shift;
  return shift;
}

static int check_rotation(const fa_rotation* r, int d, Plan* p) {
  if (!r) return set_error(FA_ERR_INVALID_ARG, "rotation is NULL");
  if (d != 64 && d != 128) return set_error(FA_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
  if (r->rot < 0 || r->rot > d || r->rot % 16)
    return set_error(FA_ERR_INVALID_ARG, "rot must be a multiple of 16 from 0 to d=%d (got %d)", d, r->rot);
  if (r->rot > 0 && (!r->inv_freq || (reinterpret_cast<uintptr_t>(r->inv_freq) & 7)))
    return set_error(FA_ERR_INVALID_ARG, "inv_freq must be an 8-byte aligned device pointer");
  if (r->norm && !(r->eps >= 0.f && isfinite(r->eps)))
    return set_error(FA_ERR_INVALID_ARG, "eps must be finite and >= 0 (got %g)", r->eps);
  if (!r->norm && (r->q_weight || r->k_weight)) return set_error(FA_ERR_INVALID_ARG, "weights need the norm");
  const int align = r->weight_bf16 ? 1 : 3;
  if ((reinterpret_cast<uintptr_t>(r->q_weight) & align) || (reinterpret_cast<uintptr_t>(r->k_weight) & align))
    return set_error(FA_ERR_INVALID_ARG, "q_weight, k_weight are not aligned to their type");
  *p = Plan{r->inv_freq, r->rot, r->norm != 0, r->eps};
  return FA_OK;
}

// Strides of a [B, H, N, d] view, in elements; those of dimensions with one entry are not used.
static int check_heads(const fa_heads* x, const char* name, int B, int H, int N, bool written, int d) {
  if (!x) return set_error(FA_ERR_INVALID_ARG, "%s is NULL", name);
  int rc = check_ptr(x->p, name);
  if (rc) return rc;
  const long long strides[3] = {B > 1 ? x->stride_b : 0, H > 1 ? x->stride_h : 0, N > 1 ? x->stride_n : 0};
  for (long long s : strides)
    if (s < 0 || s % 8) return set_error(FA_ERR_INVALID_ARG, "%s: strides must be multiples of 8, not negative (got %lld)", name, s);
  // two vectors that are written may not overlap: each stride passes what the smaller ones span
  if (written) {
    long long n[3] = {B, H, N}, s[3] = {strides[0], strides[1], strides[2]};
    for (int i = 0; i < 3; ++i)
      for (int j = i + 1; j < 3; ++j)
        if (s[j] < s[i]) {
          const long long a = s[i], b = n[i];
          s[i] = s[j], n[i] = n[j], s[j] = a, n[j] = b;
        }
    long long span = d;
    for (int i = 0; i < 3; ++i) {
      if (n[i] == 1) continue;
      if (s[i] < span) return set_error(FA_ERR_INVALID_ARG, "%s: heads of tokens must not overlap", name);
      span += s[i] * (n[i] - 1);
    }
  }
  return FA_OK;
}

static int check_sizes(int B, int Hq, int Hkv, int N) {
  if (B < 1 || Hq < 1 || Hkv < 1 || N < 1)
    return set_error(FA_ERR_INVALID_ARG, "B, Hq, Hkv, N must be >= 1 (got %d, %d, %d, %d)", B, Hq, Hkv, N);
  if ((long long)B * N * (Hq > Hkv ? Hq : Hkv) >= (1ll << 31)) return set_error(FA_ERR_INVALID_ARG, "B*H*N must be < 2^31");
  return FA_OK;
}

static int check_positions(const int32_t* p) {
  if (reinterpret_cast<uintptr_t>(p) & 3) return set_error(FA_ERR_INVALID_ARG, "positions is not 4-byte aligned");
  return FA_OK;
}

template <int D>
static Side make_side(const fa_heads* x, const fa_heads* dz, const fa_heads* out, const void* w, int w_bf16, int H,
                      long long tokens, int unroll, int most_ctas) {
  Side s = {};
  s.x = static_cast<const __nv_bfloat16*>(x->p);
  s.x_b = x->stride_b, s.x_h = x->stride_h, s.x_n = x->stride_n;
  if (dz) {
    s.dz = static_cast<const __nv_bfloat16*>(dz->p);
    s.dz_b = dz->stride_b, s.dz_h = dz->stride_h, s.dz_n = dz->stride_n;
  }
  s.out = static_cast<__nv_bfloat16*>(out->p);
  s.out_b = out->stride_b, s.out_h = out->stride_h, s.out_n = out->stride_n;
  s.w = w;
  s.w_bf16 = w_bf16;
  s.H = H;
  s.shift = pick_shift(H, Lanes<D>::kGroups, unroll, tokens);
  const int per = Lanes<D>::kGroups >> s.shift;
  const long long tiles = (tokens + per - 1) / per;
  s.ctas = (int)(tiles < most_ctas ? tiles : most_ctas);
  return s;
}

// CTAs of the backward, two for each of 152 SMs; each side gets a share by its heads (together at most all).
constexpr int kBwdCtas = 304;
static int bwd_ctas(int H, int others) {
  const int n = (int)((long long)kBwdCtas * H / ((long long)H + others));
  return n < 1 ? 1 : n;
}

constexpr int kNoLimit = 0x7FFFFFFF;

template <int D>
static int launch_forward(const fa_rotation* r, const Dense& g, const fa_heads* q, const fa_heads* k, const fa_heads* qo,
                          const fa_heads* ko, int Hq, int Hkv, cudaStream_t s) {
  const Side sq = make_side<D>(q, nullptr, qo, r->q_weight, r->weight_bf16, Hq, g.tokens, kUnroll, kNoLimit);
  const Side sk = make_side<D>(k, nullptr, ko, r->k_weight, r->weight_bf16, Hkv, g.tokens, kUnroll, kNoLimit);
  const int most = sq.shift < sk.shift ? sq.shift : sk.shift;
  const int smem = table_bytes<D>(Lanes<D>::kGroups >> most);
  const unsigned grid = (unsigned)sq.ctas + (unsigned)sk.ctas;
  auto kern = r->interleaved ? norm_rotate_kernel<D, true> : norm_rotate_kernel<D, false>;
  kern<<<grid, kThreads, smem, s>>>(g, sq, sk);
  return check_cuda(cudaGetLastError(), "launch fa_norm_rotate");
}

template <int D>
static int launch_backward(const fa_rotation* r, const Dense& g, const fa_heads* q, const fa_heads* k, const fa_heads* dzq,
                           const fa_heads* dzk, const fa_heads* dq, const fa_heads* dk, float* dqw, float* dkw, float* part,
                           int Hq, int Hkv, cudaStream_t s) {
  const Side sq = make_side<D>(q, dzq, dq, r->q_weight, r->weight_bf16, Hq, g.tokens, kUnrollBwd, bwd_ctas(Hq, Hkv));
  const Side sk = make_side<D>(k, dzk, dk, r->k_weight, r->weight_bf16, Hkv, g.tokens, kUnrollBwd, bwd_ctas(Hkv, Hq));
  const int most = sq.shift < sk.shift ? sq.shift : sk.shift;
  const int table = table_bytes<D>(Lanes<D>::kGroups >> most), rows = Lanes<D>::kGroups * D * 4;
  const int smem = table > rows ? table : rows;
  auto kern = r->interleaved ? norm_rotate_bwd_kernel<D, true> : norm_rotate_bwd_kernel<D, false>;
  kern<<<sq.ctas + sk.ctas, kThreads, smem, s>>>(g, sq, sk, part);
  const int rc = check_cuda(cudaGetLastError(), "launch fa_norm_rotate_bwd");
  if (rc || !part) return rc;
  weight_grad_kernel<<<2 * D / 32, 1024, 0, s>>>(part, D, sq.ctas, sk.ctas, dqw, dkw);
  return check_cuda(cudaGetLastError(), "launch fa_norm_rotate_bwd weights");
}

template <int D>
static int launch_append(const fa_rotation* r, const Packed& g, const fa_heads* q, const fa_heads* k, const fa_heads* v,
                         const fa_heads* qo, int Hq, int Hkv, bool fp8, cudaStream_t s) {
  const Side sq = make_side<D>(q, nullptr, qo, r->q_weight, r->weight_bf16, Hq, g.T, kUnroll, kNoLimit);
  const Side sk = make_side<D>(k, nullptr, k, r->k_weight, r->weight_bf16, Hkv, g.T, kUnroll, kNoLimit);
  const Side sv = make_side<D>(v, nullptr, v, nullptr, 0, Hkv, g.T, kUnroll, kNoLimit);
  const int most = sq.shift < sk.shift ? sq.shift : sk.shift;
  const int smem = table_bytes<D>(Lanes<D>::kGroups >> most);
  const unsigned grid = (unsigned)sq.ctas + (unsigned)sk.ctas + (unsigned)sv.ctas;
  auto kern = r->interleaved ? (fp8 ? qkv_append_kernel<D, true, true> : qkv_append_kernel<D, true, false>)
                             : (fp8 ? qkv_append_kernel<D, false, true> : qkv_append_kernel<D, false, false>);
  kern<<<grid, kThreads, smem, s>>>(g, sq, sk, sv);
  return check_cuda(cudaGetLastError(), "launch fa_qkv_append");
}

}  // namespace rotate
}  // namespace fa

extern "C" int fa_norm_rotate(const fa_rotation* rotation, const fa_heads* q, const fa_heads* k, const fa_heads* q_out,
                              const fa_heads* k_out, int B, int Hq, int Hkv, int N, int d, const int32_t* positions,
                              int64_t positions_stride, void* stream) {
  fa::NvtxRange nvtx_range("fa_norm_rotate");
  using namespace fa;
  clear_error();
  rotate::Plan p;
  int rc;
  if ((rc = rotate::check_sizes(B, Hq, Hkv, N)) || (rc = rotate::check_rotation(rotation, d, &p)) ||
      (rc = rotate::check_heads(q, "q", B, Hq, N, false, d)) || (rc = rotate::check_heads(k, "k", B, Hkv, N, false, d)) ||
      (rc = rotate::check_heads(q_out, "q_out", B, Hq, N, true, d)) ||
      (rc = rotate::check_heads(k_out, "k_out", B, Hkv, N, true, d)) || (rc = rotate::check_positions(positions)))
    return rc;
  const rotate::Dense g{p, positions, positions_stride, (long long)B * N, N};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return d == 64 ? rotate::launch_forward<64>(rotation, g, q, k, q_out, k_out, Hq, Hkv, s)
                 : rotate::launch_forward<128>(rotation, g, q, k, q_out, k_out, Hq, Hkv, s);
}

extern "C" size_t fa_norm_rotate_bwd_workspace_size(int B, int Hq, int Hkv, int N, int d) {
  fa::clear_error();
  if (fa::rotate::check_sizes(B, Hq, Hkv, N)) return 0;
  if (d != 64 && d != 128) {
    fa::set_error(FA_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
    return 0;
  }
  return (size_t)fa::rotate::kBwdCtas * d * sizeof(float);   // a row of d for each CTA
}

extern "C" int fa_norm_rotate_bwd(const fa_rotation* rotation, const fa_heads* q, const fa_heads* k, const fa_heads* dzq,
                                  const fa_heads* dzk, const fa_heads* dq, const fa_heads* dk, float* dq_weight,
                                  float* dk_weight, int B, int Hq, int Hkv, int N, int d, const int32_t* positions,
                                  int64_t positions_stride, void* workspace, size_t workspace_bytes, void* stream) {
  fa::NvtxRange nvtx_range("fa_norm_rotate_bwd");
  using namespace fa;
  clear_error();
  rotate::Plan p;
  int rc;
  if ((rc = rotate::check_sizes(B, Hq, Hkv, N)) || (rc = rotate::check_rotation(rotation, d, &p)) ||
      (rc = rotate::check_heads(q, "q", B, Hq, N, false, d)) || (rc = rotate::check_heads(k, "k", B, Hkv, N, false, d)) ||
      (rc = rotate::check_heads(dzq, "dzq", B, Hq, N, false, d)) || (rc = rotate::check_heads(dzk, "dzk", B, Hkv, N, false, d)) ||
      (rc = rotate::check_heads(dq, "dq", B, Hq, N, true, d)) || (rc = rotate::check_heads(dk, "dk", B, Hkv, N, true, d)) ||
      (rc = rotate::check_positions(positions)))
    return rc;
  if (!dq_weight != !dk_weight) return set_error(FA_ERR_INVALID_ARG, "dq_weight and dk_weight are given together or not at all");
  if ((reinterpret_cast<uintptr_t>(dq_weight) & 3) || (reinterpret_cast<uintptr_t>(dk_weight) & 3))
    return set_error(FA_ERR_INVALID_ARG, "dq_weight, dk_weight are not 4-byte aligned");
  if (dq_weight && !p.norm) return set_error(FA_ERR_INVALID_ARG, "weight gradients need the norm");
  float* part = nullptr;
  if (dq_weight) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
      return set_error(FA_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
    const size_t need = fa_norm_rotate_bwd_workspace_size(B, Hq, Hkv, N, d);
    if (workspace_bytes < need)
      return set_error(FA_ERR_INVALID_ARG, "workspace too small: %zu bytes, %zu needed", workspace_bytes, need);
    part = static_cast<float*>(workspace);
  }
  const rotate::Dense g{p, positions, positions_stride, (long long)B * N, N};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return d == 64 ? rotate::launch_backward<64>(rotation, g, q, k, dzq, dzk, dq, dk, dq_weight, dk_weight, part, Hq, Hkv, s)
                 : rotate::launch_backward<128>(rotation, g, q, k, dzq, dzk, dq, dk, dq_weight, dk_weight, part, Hq, Hkv, s);
}

extern "C" int fa_qkv_append(const fa_paged_kv* kv, const fa_rotation* rotation, const void* q, int64_t q_stride, void* q_out,
                             int Hq, const void* k_new, const void* v_new, int64_t new_stride, const int32_t* q_indptr,
                             const int32_t* positions, int T, void* stream) {
  fa::NvtxRange nvtx_range("fa_qkv_append");
  using namespace fa;
  clear_error();
  rotate::Packed g = {};
  int rc;
  if ((rc = paged::check_cache(kv, &g.c)) || (rc = rotate::check_rotation(rotation, kv->d, &g.p))) return rc;
  if (T < 0) return set_error(FA_ERR_INVALID_ARG, "T must be >= 0 (got %d)", T);
  if (Hq < 1) return set_error(FA_ERR_INVALID_ARG, "Hq must be >= 1 (got %d)", Hq);
  const int d = kv->d, Hkv = kv->Hkv;
  if ((long long)T * (Hq > Hkv ? Hq : Hkv) >= (1ll << 31)) return set_error(FA_ERR_INVALID_ARG, "T*H must be < 2^31");
  if ((rc = check_ptr(q, "q")) || (rc = check_ptr(q_out, "q_out")) || (rc = check_ptr(k_new, "k_new")) ||
      (rc = check_ptr(v_new, "v_new")) || (rc = paged::check_indptr(q_indptr, "q_indptr")) ||
      (rc = rotate::check_positions(positions)))
    return rc;
  if (q_stride < (int64_t)Hq * d || q_stride % 8)
    return set_error(FA_ERR_INVALID_ARG, "q_stride %lld must be a multiple of 8 and at least Hq*d = %lld", (long long)q_stride,
                     (long long)Hq * d);
  if (new_stride < (int64_t)Hkv * d || new_stride % 8)
    return set_error(FA_ERR_INVALID_ARG, "new_stride %lld must be a multiple of 8 and at least Hkv*d = %lld",
                     (long long)new_stride, (long long)Hkv * d);
  if (T == 0) return FA_OK;
  g.c.status = device_status_word();
  if (!g.c.status) return set_error(FA_ERR_CUDA, "could not allocate the device status record");
  g.q_indptr = q_indptr;
  g.positions = positions;
  g.T = T;
  const fa_heads hq{const_cast<void*>(q), 0, d, q_stride}, ho{q_out, 0, d, (int64_t)Hq * d};
  const fa_heads hk{const_cast<void*>(k_new), 0, d, new_stride}, hv{const_cast<void*>(v_new), 0, d, new_stride};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool fp8 = kv->dtype == FA_KV_E4M3;
  return d == 64 ? rotate::launch_append<64>(rotation, g, &hq, &hk, &hv, &ho, Hq, Hkv, fp8, s)
                 : rotate::launch_append<128>(rotation, g, &hq, &hk, &hv, &ho, Hq, Hkv, fp8, s);
}
