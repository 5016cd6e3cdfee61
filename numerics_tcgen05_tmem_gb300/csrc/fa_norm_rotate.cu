// Norm of queries and keys for each head and position rotation in one pass: dense with gradients
// (fa_norm_rotate, fa_norm_rotate_bwd), and for packed rows with the write into a paged cache (fa_qkv_append).
//
// A vector x is one head of one token, d elements; its first `rot` are rotated in pairs (a, b):
//   r = 1 / sqrt(mean x^2 + eps), y = w o x r,  z_a = y_a cos - y_b sin,  z_b = y_b cos + y_a sin.
// Backward: dy is dz rotated by the opposite angle, g = w o dy, dw = sum of dy o x r over the vectors,
//   dx = r g - x r^3 / d sum(x o g)   (without the norm dx = dy).
// r is computed again from x, which the backward reads in any case.  Where the squares leave FP32's range
// (entries past 2^56, or all under 2^-38 and eps as small) x is multiplied by a power of two first: y does not change, and
// dx takes the factor at its end.
//
// Memory bounds all three.  d / 16 lanes take a vector, each two 16-byte parts that hold both entries of its
// pairs, so that the rotation needs no exchange and the sums three (two) shuffles.  Persistent CTAs, and a
// thread's copies (cp.async) run two vectors ahead, into slots that only it reads: registers as the store of
// what is on its way left the backward at 4.7 TB/s, where it now moves 6.1.
//   8192 tokens, 32 + 32 heads, d = 128: forward 45 us, backward 66 us and 3 us for the weights' gradients, without the
//   norm 48 us (268, 403 and 268 MB: 6.0, 6.1 and 5.6 TB/s of the 6.8 of a plain copy); 8 x 1024 tokens, 12 + 12 heads,
//   d = 64: 14.5 and 19 + 3 us, where a third is the start (frequencies, angles) and the last, partly filled round of tiles;
//   23100 packed tokens, 32 + 8 + 8 heads, into a BF16 cache 61 us, 6.2 TB/s.
//
// Angles: position times frequency modulo one turn.  In FP32 a position of 2^20 would leave 0.06 rad of error.
// A frequency is kept as a fraction of a turn in 64 bits; the product with a 32-bit position wraps at whole
// turns by itself, and its upper 32 bits are the angle (error: pos * 2^-54 turns, from the double it comes from).
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "overlap.h"
#include "paged_attn.cuh"

namespace fa {
namespace rotate {

using paged::Cache;

constexpr int kThreads = 256;
// Measured on 8192 tokens, 32 and 32 heads, d = 128 (forward and backward together), and on 23100 packed tokens, 32 and 8
// heads, into BF16: as chosen 113 and 61 us; with two CTAs for the forward 118 and 66 (registers as the store of
// what is on its way), with four of two stages 119 and 64, with one CTA for the backward 138; two heads for a
// lane group 126 and 74, eight 113 and 73.
constexpr int kCtas = 3;       // forward and append: CTAs on an SM
constexpr int kBwdCtas = 2;    // backward
constexpr int kStages = 3;     // vectors of a lane group that are worked on or on their way
constexpr int kHeads = 4;      // heads of a token for one lane group, where there are enough tokens

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
  float least_sum;   // of a lane's squares, from which on their rounding is FP32's (0 where eps is far above what is lost)
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

// The first elements of lane j's parts.  Neighbouring lanes take neighbouring 16 bytes, so that an access of the
// lanes covers whole sectors (with 32 bytes in a row for each lane the forward took 59 us where it takes 45).
// Pairs (i, i + rot / 2): a and b lie rot / 2 apart, and half the rest behind the rotated entries.  Neighbouring
// pairs lie within a part.
template <int D, bool kInter>
__device__ __forceinline__ void part_columns(int j, int rot, int& a, int& b) {
  const bool rest = !kInter && 16 * j >= rot;
  a = rest ? 8 * j + rot / 2 : 8 * j;              // (rot + 8 (j - rot / 16))
  b = a + (kInter ? D : (rest ? D - rot : rot)) / 2;
}

// Sum over the lanes of a group.
template <int kLanes>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The pairs of a lane turned by its eight angles (kSign = -1: back).
template <bool kInter, int kSign>
__device__ __forceinline__ void turn(Parts& v, const float (&c)[8], const float (&s)[8]) {
  if constexpr (kInter) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float& x = i < 4 ? v.a[2 * i] : v.b[2 * i - 8];
      float& y = i < 4 ? v.a[2 * i + 1] : v.b[2 * i - 7];
      float p, q;
      mul2(p, q, y, x, -kSign * s[i], kSign * s[i]);
      fma2(x, y, x, y, c[i], c[i], p, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float p0, p1, q0, q1;   // s y, s x
      mul2(p0, p1, s[i], s[i + 1], v.b[i], v.b[i + 1]);
      mul2(q0, q1, s[i], s[i + 1], v.a[i], v.a[i + 1]);
      fma2(v.a[i], v.a[i + 1], v.a[i], v.a[i + 1], c[i], c[i + 1], -kSign * p0, -kSign * p1);
      fma2(v.b[i], v.b[i + 1], v.b[i], v.b[i + 1], c[i], c[i + 1], kSign * q0, kSign * q1);
    }
  }
}

// Shared memory of a CTA.  Lane j reads 16 bytes at j of a row of lanes, so that no two lanes meet in a bank.
template <int D>
struct Tables {
  static constexpr int kLanes = Lanes<D>::kLanes, kMaxTokens = Lanes<D>::kGroups;
  uint64_t turns[D / 2];                   // of a position, in units of 2^-64
  float4 weight[4][kLanes];                // of the parts a and b, four each
  float4 angle[2][kMaxTokens][4][kLanes];  // cos and sin of a tile's tokens, of this tile and of the next
};

template <int D, bool kInter>
__device__ __forceinline__ void fill_weights(Tables<D>& t, const void* w, int is_bf16, int rot) {
  if (threadIdx.x < D) {
    const int j = threadIdx.x / 16, e = threadIdx.x % 16;
    int a, b;
    part_columns<D, kInter>(j, rot, a, b);
    const int col = e < 8 ? a + e : b + e - 8;
    float f = 1.f;
    if (w != nullptr)
      f = is_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[col]) : static_cast<const float*>(w)[col];
    reinterpret_cast<float*>(&t.weight[e / 4][j])[e % 4] = f;
  }
}

// Which angles a thread computes: those of frequency f, kThreads >> shift threads for each.
struct Mine {
  int f, shift;
  __device__ __forceinline__ explicit Mine(int rot) : shift(0) {
    while ((2 << shift) < rot) ++shift;   // 2^shift >= rot / 2
    f = threadIdx.x & ((1 << shift) - 1);
  }
};

// The thread's frequency as a fraction of a turn.  (All threads of a frequency write the same, each reads
// it back itself.)
template <int D>
__device__ __forceinline__ void fill_turns(Tables<D>& t, const Plan& p, int rot) {
  const Mine m(rot);
  if (2 * m.f >= rot) return;
  double x = __ldg(p.inv_freq + m.f) * 0.15915494309189533577;   // 1 / (2 pi)
  x -= floor(x);
  t.turns[m.f] = x < 1.0 ? (uint64_t)__double2ull_rd(x * 18446744073709551616.0) : 0;   // (NaN: 0)
}

// position(i): that of the tile's token i.  A barrier has to follow.
template <int D, bool kInter, class Position>
__device__ __forceinline__ void fill_angles(Tables<D>& t, int buf, int rot, int tokens, Position position) {
  const Mine m(rot);
  if (2 * m.f >= rot) return;
  // a lane's eight: of its eight pairs between a and b, or of four pairs in a and four in b
  const int row = kInter ? m.f / (D / 4) : m.f % 8 / 4, lane = kInter ? m.f % (D / 4) / 4 : m.f / 8;
  float* to = reinterpret_cast<float*>(&t.angle[buf][0][row][lane]) + m.f % 4;
  for (int token = threadIdx.x >> m.shift; token < tokens; token += kThreads >> m.shift) {
    const uint64_t at = (uint64_t)(int64_t)position(token) * t.turns[m.f];
    // the nearest quarter turn apart, the rest is within an eighth: its rounding to FP32 stays under 2^-25 rad
    const uint32_t u = (uint32_t)(at >> 32), quarter = (u + 0x20000000u) >> 30;
    float s0, c0;
    sincospif((float)(int32_t)(u - (quarter << 30)) * 0x1p-31f, &s0, &c0);   // a turn is 2^32, sincospi's is 2
    const float s = quarter & 1 ? c0 : s0, c = quarter & 1 ? s0 : c0;
    constexpr int kRow = 4 * Lanes<D>::kLanes;   // floats of a row of lanes; cos has rows 0 and 1, sin 2 and 3
    to[token * 4 * kRow] = (quarter + 1) & 2 ? -c : c;
    to[token * 4 * kRow + 2 * kRow] = quarter & 2 ? -s : s;
  }
}

__device__ __forceinline__ void spread8(const float4& u, const float4& v, float (&f)[8]) {
  f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
}
// A lane's angles of a token: 1 and 0 behind the rotated entries.
template <int D, bool kInter>
__device__ __forceinline__ void load_angles(const Tables<D>& t, int buf, int rot, int token, int j, float (&c)[8], float (&s)[8]) {
  const float4 one = make_float4(1.f, 1.f, 1.f, 1.f), zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool first = kInter ? 8 * j < rot : 16 * j < rot, second = kInter ? D / 2 + 8 * j < rot : first;
  const auto& at = t.angle[buf][token];
  spread8(first ? at[0][j] : one, second ? at[1][j] : one, c);
  spread8(first ? at[2][j] : zero, second ? at[3][j] : zero, s);
}

// A thread's own copies of its 16-byte parts, kParts of a vector, on their way to slots of its own: no other
// thread reads them, so that a wait for the thread's own copies is all it takes.  Every vector is copied before
// anything is written in its place: an output may be its input.
template <int kParts>
struct Ring {
  uint4 slot[kStages][kParts][kThreads];
  __device__ __forceinline__ void copy(int stage, int part, const __nv_bfloat16* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&slot[stage][part][threadIdx.x])), "l"(from) : "memory");
  }
  __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // the oldest of kStages groups has landed
  __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory"); }
  __device__ __forceinline__ uint4 get(int stage, int part) const { return slot[stage][part][threadIdx.x]; }
};

// Sum of squares of a lane's parts.
__device__ __forceinline__ float squares(const Parts& v) {
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    fma2(s[0], s[1], v.a[i], v.a[i + 1], v.a[i], v.a[i + 1], s[0], s[1]);
    fma2(s[2], s[3], v.b[i], v.b[i + 1], v.b[i], v.b[i + 1], s[2], s[3]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __forceinline__ void scale_vector(Parts& v, float f) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    mul2(v.a[i], v.a[i + 1], v.a[i], v.a[i + 1], f, f);
    mul2(v.b[i], v.b[i + 1], v.b[i], v.b[i + 1], f, f);
  }
}

// What 1 / rms is computed from: a lane's sum of squares and eps, of the vector times `factor`.
struct Squares {
  float sum, eps, factor;
  bool scaled;   // whether a vector of the warp has a factor that may not be 1
};
constexpr float kLargestSum = 0x1p116f;   // of a lane; eight of them stay in range

// The factor is 1 but for vectors of which a lane's sum is out of [p.least_sum, kLargestSum): theirs is the power of two that
// brings the largest entry to [1, 2) (and eps under 4, where it is more than that entry's square).  Zeros, and vectors with
// an entry that is not finite, stay.  real: whether it is a vector, not what its slot held before.  The vote takes 1 % (8192
// tokens, 32 + 32 heads, both passes 113.3 -> 114.6 us; neighbouring pairs 2 to 4 %); a vote on 1 / rms itself, behind the sums
// over the lanes, 3 %.
template <int D>
__device__ __forceinline__ Squares vector_squares(Parts& v, const Plan& p, bool real) {
  constexpr int kLanes = Lanes<D>::kLanes;
  Squares q{squares(v), p.eps, 1.f, false};
  const bool out = real && !(q.sum >= p.least_sum && q.sum < kLargestSum);
  if (__any_sync(0xffffffffu, out)) {
    q.scaled = true;
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      amax = max(amax, max(__float_as_uint(v.a[i]) & 0x7FFFFFFFu, __float_as_uint(v.b[i]) & 0x7FFFFFFFu));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const unsigned mine = __ballot_sync(0xffffffffu, out) >> (threadIdx.x % 32 / kLanes * kLanes) & ((1u << kLanes) - 1);
    if (mine != 0 && amax != 0 && amax < 0x7F800000u) {
      const int e_eps = p.eps > 0.f ? ((int)(__float_as_uint(p.eps) >> 23) - 127) >> 1 : -127;
      const int e = min(max(max((int)(amax >> 23) - 127, e_eps), -126), 126);   // both 2^e and 2^-e are normal numbers
      q.factor = __uint_as_float((uint32_t)(127 - e) << 23);
      scale_vector(v, q.factor);
      q.sum = squares(v);
      q.eps = p.eps * q.factor * q.factor;
    }
  }
  return q;
}

template <int D>
__device__ __forceinline__ float inverse_rms(const Squares& q) {
  return __frsqrt_rn(group_sum<Lanes<D>::kLanes>(q.sum) * (1.f / D) + q.eps);
}

// One vector's parts normed and turned, in place.
template <int D, bool kInter>
__device__ __forceinline__ void forward_vector(Parts& v, const Plan& p, const Tables<D>& t, int j, const float (&c)[8],
                                               const float (&s)[8], bool real) {
  if (p.norm) {
    const float r = inverse_rms<D>(vector_squares<D>(v, p, real));
    float w[8];
    spread8(t.weight[0][j], t.weight[1][j], w);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      mul2(v.a[i], v.a[i + 1], v.a[i], v.a[i + 1], r, r);
      mul2(v.a[i], v.a[i + 1], v.a[i], v.a[i + 1], w[i], w[i + 1]);
    }
    spread8(t.weight[2][j], t.weight[3][j], w);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      mul2(v.b[i], v.b[i + 1], v.b[i], v.b[i + 1], r, r);
      mul2(v.b[i], v.b[i + 1], v.b[i], v.b[i + 1], w[i], w[i + 1]);
    }
  }
  turn<kInter, 1>(v, c, s);
}

// The token of a dense batch: batch entry and place in it.
struct Place {
  unsigned b, n;
};
__device__ __forceinline__ Place place_of(unsigned token, int N) {
  const unsigned b = token / (unsigned)N;
  return Place{b, token - b * N};
}

struct Dense {
  Plan p;
  const int32_t* positions;   // NULL: 0, 1, ..
  long long pos_b;            // entries between two sequences' positions
  unsigned tokens;            // B * N, under 2^31
  int N;
};

__device__ __forceinline__ int dense_position(const Dense& g, unsigned token) {
  if (token >= g.tokens) return 0;
  const Place at = place_of(token, g.N);
  return g.positions == nullptr ? (int)at.n : __ldg(g.positions + at.b * g.pos_b + at.n);
}

// How a side's tokens are dealt: a tile has kGroups >> shift tokens, CTA i takes the tiles i, i + ctas, ..
// Lane group x of a CTA has token x >> shift of the tile and the heads (x & groups - 1), + groups, ..
struct Deal {
  int groups, tokens, mine, head0;
  unsigned tiles;
  __device__ __forceinline__ Deal(int shift, int all_groups, int group, unsigned all)
      : groups(1 << shift), tokens(all_groups >> shift), mine(group >> shift), head0(group & ((1 << shift) - 1)),
        tiles((all + tokens - 1) / tokens) {}
};

// The vectors of a lane group, in the order in which it works on them; one of these runs ahead for the copies.
struct Ahead {
  unsigned tile;
  int h, stage;
};

template <int D, int kParts>
struct Shared {
  Tables<D> t;
  Ring<kParts> ring;
};

// The first q.ctas CTAs have the queries.  Copies run kStages - 1 vectors ahead, and the next tile's angles are
// computed beside the current one's vectors: one barrier for a tile.
template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads, kCtas) norm_rotate_kernel(const __grid_constant__ Dense g,
                                                                      const __grid_constant__ Side q,
                                                                      const __grid_constant__ Side k) {
  using L = Lanes<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  Tables<D>& t = reinterpret_cast<Shared<D, 2>*>(smem)->t;
  Ring<2>& ring = reinterpret_cast<Shared<D, 2>*>(smem)->ring;
  const bool is_q = (int)blockIdx.x < q.ctas;
  const Side& side = is_q ? q : k;
  const int j = threadIdx.x % L::kLanes, H = side.H;
  const Deal d(side.shift, L::kGroups, threadIdx.x / L::kLanes, g.tokens);
  int ca, cb;
  part_columns<D, kInter>(j, g.p.rot, ca, cb);
  unsigned tile = blockIdx.x - (is_q ? 0 : q.ctas);

  Ahead next{tile, d.head0, 0};
  const __nv_bfloat16* from = nullptr;
  const long long x_step = d.groups * side.x_h, out_step = d.groups * side.out_h;
  auto seek = [&] {   // the first vector of next.tile
    const unsigned token = next.tile * d.tokens + d.mine;
    from = nullptr;
    if (next.tile < d.tiles && token < g.tokens) {
      const Place at = place_of(token, g.N);
      from = side.x + at.b * side.x_b + at.n * side.x_n + d.head0 * side.x_h + ca;
    }
  };
  auto copy = [&] {
    if (from != nullptr && next.h < H) {
      ring.copy(next.stage, 0, from);
      ring.copy(next.stage, 1, from + (cb - ca));
      from += x_step;
    }
    ring.commit();
    next.stage = next.stage + 1 == kStages ? 0 : next.stage + 1;
    next.h += d.groups;
    if (next.h - d.head0 >= H) {
      next.h = d.head0;
      next.tile += side.ctas;
      seek();
    }
  };
  seek();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) copy();
  fill_turns(t, g.p, g.p.rot);
  fill_weights<D, kInter>(t, side.w, side.w_bf16, g.p.rot);
  fill_angles<D, kInter>(t, 0, g.p.rot, d.tokens, [&](int i) { return dense_position(g, tile * d.tokens + i); });
  __syncthreads();
  int stage = 0;
  for (int buf = 0; tile < d.tiles; tile += side.ctas, buf ^= 1) {
    const unsigned after = tile + side.ctas, token = tile * d.tokens + d.mine;
    if (after < d.tiles)
      fill_angles<D, kInter>(t, buf ^ 1, g.p.rot, d.tokens, [&](int i) { return dense_position(g, after * d.tokens + i); });
    const bool valid = token < g.tokens;
    const Place at = place_of(valid ? token : 0, g.N);
    __nv_bfloat16* z = side.out + at.b * side.out_b + at.n * side.out_n + d.head0 * side.out_h + ca;
    float c[8], s[8];
    load_angles<D, kInter>(t, buf, g.p.rot, d.mine, j, c, s);
    for (int h = d.head0; h - d.head0 < H; h += d.groups) {   // the same number of steps for the whole CTA
      copy();
      ring.wait();
      Parts v;
      unpack(ring.get(stage, 0), v.a);
      unpack(ring.get(stage, 1), v.b);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      const bool real = valid && h < H;
      forward_vector<D, kInter>(v, g.p, t, j, c, s, real);
      if (real) {
        *reinterpret_cast<uint4*>(z) = pack(v.a);
        *reinterpret_cast<uint4*>(z + (cb - ca)) = pack(v.b);
      }
      z += out_step;
    }
    __syncthreads();
  }
}

// Without the norm dx is dz turned back: x is not read, so that what it holds (NaN in an unused row) stays out of dx.
// The weights' gradients are summed in registers, then over the CTA's groups, and the CTA's sum goes to
// part[CTA][d].
template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads, kBwdCtas) norm_rotate_bwd_kernel(const __grid_constant__ Dense g,
                                                                             const __grid_constant__ Side q,
                                                                             const __grid_constant__ Side k,
                                                                             float* __restrict__ part) {
  using L = Lanes<D>;
  cudaTriggerProgrammaticLaunchCompletion();   // the weights' kernel may get ready; it waits for this one's end
  extern __shared__ __align__(16) uint8_t smem[];
  Tables<D>& t = reinterpret_cast<Shared<D, 4>*>(smem)->t;
  Ring<4>& ring = reinterpret_cast<Shared<D, 4>*>(smem)->ring;
  const bool is_q = (int)blockIdx.x < q.ctas;
  const Side& side = is_q ? q : k;
  const int j = threadIdx.x % L::kLanes, group = threadIdx.x / L::kLanes, H = side.H;
  const Deal d(side.shift, L::kGroups, group, g.tokens);
  int ca, cb;
  part_columns<D, kInter>(j, g.p.rot, ca, cb);
  unsigned tile = blockIdx.x - (is_q ? 0 : q.ctas);
  float dwa[8], dwb[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dwa[i] = dwb[i] = 0.f;

  Ahead next{tile, d.head0, 0};
  const __nv_bfloat16 *from = nullptr, *from_dz = nullptr;
  const long long x_step = d.groups * side.x_h, dz_step = d.groups * side.dz_h, out_step = d.groups * side.out_h;
  auto seek = [&] {
    const unsigned token = next.tile * d.tokens + d.mine;
    from = nullptr;
    if (next.tile < d.tiles && token < g.tokens) {
      const Place at = place_of(token, g.N);
      from = side.x + at.b * side.x_b + at.n * side.x_n + d.head0 * side.x_h + ca;
      from_dz = side.dz + at.b * side.dz_b + at.n * side.dz_n + d.head0 * side.dz_h + ca;
    }
  };
  auto copy = [&] {
    if (from != nullptr && next.h < H) {
      if (g.p.norm) {
        ring.copy(next.stage, 0, from);
        ring.copy(next.stage, 1, from + (cb - ca));
        from += x_step;
      }
      ring.copy(next.stage, 2, from_dz);
      ring.copy(next.stage, 3, from_dz + (cb - ca));
      from_dz += dz_step;
    }
    ring.commit();
    next.stage = next.stage + 1 == kStages ? 0 : next.stage + 1;
    next.h += d.groups;
    if (next.h - d.head0 >= H) {
      next.h = d.head0;
      next.tile += side.ctas;
      seek();
    }
  };
  seek();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) copy();
  fill_turns(t, g.p, g.p.rot);
  fill_weights<D, kInter>(t, side.w, side.w_bf16, g.p.rot);
  fill_angles<D, kInter>(t, 0, g.p.rot, d.tokens, [&](int i) { return dense_position(g, tile * d.tokens + i); });
  __syncthreads();
  int stage = 0;
  for (int buf = 0; tile < d.tiles; tile += side.ctas, buf ^= 1) {
    const unsigned after = tile + side.ctas, token = tile * d.tokens + d.mine;
    if (after < d.tiles)
      fill_angles<D, kInter>(t, buf ^ 1, g.p.rot, d.tokens, [&](int i) { return dense_position(g, after * d.tokens + i); });
    const bool valid = token < g.tokens;
    const Place at = place_of(valid ? token : 0, g.N);
    __nv_bfloat16* dx = side.out + at.b * side.out_b + at.n * side.out_n + d.head0 * side.out_h + ca;
    float c[8], s[8];
    load_angles<D, kInter>(t, buf, g.p.rot, d.mine, j, c, s);
    for (int h = d.head0; h - d.head0 < H; h += d.groups) {   // the same number of steps for the whole CTA
      copy();
      ring.wait();
      Parts dy;
      unpack(ring.get(stage, 2), dy.a);
      unpack(ring.get(stage, 3), dy.b);
      const bool real = valid && h < H;   // (else its slot holds what was there)
      turn<kInter, -1>(dy, c, s);
      if (g.p.norm) {
        Parts v;
        unpack(ring.get(stage, 0), v.a);
        unpack(ring.get(stage, 1), v.b);
        const Squares sq = vector_squares<D>(v, g.p, real);
        float dot[4] = {0.f, 0.f, 0.f, 0.f}, w[8], m0, m1;
        spread8(t.weight[0][j], t.weight[1][j], w);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          mul2(m0, m1, w[i], w[i + 1], dy.a[i], dy.a[i + 1]);
          fma2(dot[0], dot[1], v.a[i], v.a[i + 1], m0, m1, dot[0], dot[1]);
        }
        spread8(t.weight[2][j], t.weight[3][j], w);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          mul2(m0, m1, w[i], w[i + 1], dy.b[i], dy.b[i + 1]);
          fma2(dot[2], dot[3], v.b[i], v.b[i + 1], m0, m1, dot[2], dot[3]);
        }
        const float all = group_sum<L::kLanes>((dot[0] + dot[1]) + (dot[2] + dot[3]));
        const float r = inverse_rms<D>(sq);
        const float back = -all * r * r * (1.f / D);   // -sum(x o g) r^2 / d
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          mul2(v.a[i], v.a[i + 1], v.a[i], v.a[i + 1], r, r);   // x r
          mul2(v.b[i], v.b[i + 1], v.b[i], v.b[i + 1], r, r);
        }
        if (real) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            fma2(dwa[i], dwa[i + 1], dy.a[i], dy.a[i + 1], v.a[i], v.a[i + 1], dwa[i], dwa[i + 1]);
            fma2(dwb[i], dwb[i + 1], dy.b[i], dy.b[i + 1], v.b[i], v.b[i + 1], dwb[i], dwb[i + 1]);
          }
        }
        // dx = r w dy - (x r) sum(x o g) r^2 / d
        spread8(t.weight[0][j], t.weight[1][j], w);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          mul2(dy.a[i], dy.a[i + 1], dy.a[i], dy.a[i + 1], w[i], w[i + 1]);
          mul2(dy.a[i], dy.a[i + 1], dy.a[i], dy.a[i + 1], r, r);
          fma2(dy.a[i], dy.a[i + 1], v.a[i], v.a[i + 1], back, back, dy.a[i], dy.a[i + 1]);
        }
        spread8(t.weight[2][j], t.weight[3][j], w);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          mul2(dy.b[i], dy.b[i + 1], dy.b[i], dy.b[i + 1], w[i], w[i + 1]);
          mul2(dy.b[i], dy.b[i + 1], dy.b[i], dy.b[i + 1], r, r);
          fma2(dy.b[i], dy.b[i + 1], v.b[i], v.b[i + 1], back, back, dy.b[i], dy.b[i + 1]);
        }
        if (sq.scaled) scale_vector(dy, sq.factor);
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
      if (real) {
        *reinterpret_cast<uint4*>(dx) = pack(dy.a);
        *reinterpret_cast<uint4*>(dx + (cb - ca)) = pack(dy.b);
      }
      dx += out_step;
    }
    __syncthreads();
  }
  if (part == nullptr) return;
  // the groups' sums: one row of d for each group in shared memory, summed in order
  float* rows = reinterpret_cast<float*>(t.angle);
  static_assert(sizeof(t.angle) >= L::kGroups * D * sizeof(float), "room for the groups' sums");
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
// 32 warps take every 32nd part each.  A programmatic launch: it starts beside the last CTAs and waits for them.
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float* __restrict__ part, int d, int q_ctas, int k_ctas,
                                                           float* __restrict__ dqw, float* __restrict__ dkw) {
  __shared__ float sums[32][33];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const bool is_q = (int)blockIdx.x < d / 32;
  const int col = ((int)blockIdx.x - (is_q ? 0 : d / 32)) * 32 + lane;
  const float* from = part + (is_q ? 0 : (long long)q_ctas * d) + col;
  const int n = is_q ? q_ctas : k_ctas;
  cudaGridDependencySynchronize();
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

// Where a tile's tokens lie: page (negative: not written) and slot in the cache, position for the rotation.
template <int kTokens>
struct Places {
  int page[3][kTokens], slot[3][kTokens], pos[3][kTokens];   // of this tile and the next two
};

// The CTAs have the queries, the keys and the values, in this order; the loop is norm_rotate_kernel's.
template <int D, bool kInter, bool kFp8>
__global__ void __launch_bounds__(kThreads, kCtas) qkv_append_kernel(const __grid_constant__ Packed g,
                                                                     const __grid_constant__ Side q,
                                                                     const __grid_constant__ Side k,
                                                                     const __grid_constant__ Side v) {
  using L = Lanes<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  Tables<D>& t = reinterpret_cast<Shared<D, 2>*>(smem)->t;
  Ring<2>& ring = reinterpret_cast<Shared<D, 2>*>(smem)->ring;
  __shared__ Places<L::kGroups> at;
  unsigned tile = blockIdx.x;
  const int which = (int)tile < q.ctas ? 0 : ((int)tile < q.ctas + k.ctas ? 1 : 2);
  tile -= which == 0 ? 0 : (which == 1 ? q.ctas : q.ctas + k.ctas);
  const Side& side = which == 0 ? q : (which == 1 ? k : v);
  const int j = threadIdx.x % L::kLanes, H = side.H, T = g.T;
  const Deal d(side.shift, L::kGroups, threadIdx.x / L::kLanes, T);
  const int rot = which == 2 ? 0 : g.p.rot;
  int ca, cb;
  part_columns<D, kInter>(j, rot, ca, cb);

  Ahead next{tile, d.head0, 0};
  const __nv_bfloat16* from = nullptr;
  auto seek = [&] {
    const unsigned token = next.tile * d.tokens + d.mine;
    from = nullptr;
    if (next.tile < d.tiles && token < (unsigned)T) from = side.x + token * side.x_n + d.head0 * D + ca;
  };
  auto copy = [&] {
    if (from != nullptr && next.h < H) {
      ring.copy(next.stage, 0, from);
      ring.copy(next.stage, 1, from + (cb - ca));
      from += d.groups * D;
    }
    ring.commit();
    next.stage = next.stage + 1 == kStages ? 0 : next.stage + 1;
    next.h += d.groups;
    if (next.h - d.head0 >= H) {
      next.h = d.head0;
      next.tile += side.ctas;
      seek();
    }
  };
  seek();
  // the places of a tile's tokens, by one thread each: four loads that wait for one another
  auto look = [&](unsigned at_tile, int slot) {
    if ((int)threadIdx.x >= d.tokens || at_tile >= d.tiles) return;
    const long long i = (long long)at_tile * d.tokens + threadIdx.x;
    int page = -1, pos = 0;
    const int b = i < T ? paged::find_sequence(g.q_indptr, g.c.B, (int)i) : -1;
    if (b >= 0) {
      pos = __ldg(g.c.kv_len + b) - __ldg(g.q_indptr + b + 1) + (int)i;
      page = which == 0 ? 0 : paged::find_page(g.c, b, pos, kSitePagedAppend);
    }
    at.page[slot][threadIdx.x] = page;
    at.slot[slot][threadIdx.x] = pos & ((1 << g.c.page_shift) - 1);
    at.pos[slot][threadIdx.x] = b >= 0 && g.positions != nullptr ? __ldg(g.positions + i) : pos;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) copy();
  look(tile, 0);
  look(tile + side.ctas, 1);
  fill_turns(t, g.p, rot);
  if (which != 2) fill_weights<D, kInter>(t, side.w, side.w_bf16, rot);
  __syncthreads();
  fill_angles<D, kInter>(t, 0, rot, d.tokens, [&](int i) { return at.pos[0][i]; });
  __syncthreads();
  const long long page_size = 1ll << g.c.page_shift;
  int stage = 0;
  for (int buf = 0, here = 0; tile < d.tiles; tile += side.ctas, buf ^= 1) {
    const unsigned after = tile + side.ctas, token = tile * d.tokens + d.mine;
    const int ahead = here == 2 ? 0 : here + 1;
    look(after + side.ctas, ahead == 2 ? 0 : ahead + 1);
    if (after < d.tiles) fill_angles<D, kInter>(t, buf ^ 1, rot, d.tokens, [&](int i) { return at.pos[ahead][i]; });
    const int page = at.page[here][d.mine], slot = at.slot[here][d.mine];
    const bool valid = token < (unsigned)T && page >= 0;
    const long long to = which == 0 ? token * side.out_n : page * g.c.page_stride + slot * (long long)D;
    const long long to_h = which == 0 ? D : page_size * D, to_scale = page * g.c.scale_stride + slot;
    float c[8], s[8];
    load_angles<D, kInter>(t, buf, rot, d.mine, j, c, s);
    for (int h = d.head0; h - d.head0 < H; h += d.groups) {
      copy();
      ring.wait();
      uint4 a = ring.get(stage, 0), b = ring.get(stage, 1);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      const bool stores = valid && h < H;
      Parts y;
      unpack(a, y.a);
      unpack(b, y.b);
      if (which != 2) forward_vector<D, kInter>(y, g.p, t, j, c, s, stores);
      if (!kFp8 || which == 0) {
        if (which != 2) {
          a = pack(y.a);
          b = pack(y.b);
        }
        if (stores) {
          __nv_bfloat16* row = (which == 0 ? side.out : static_cast<__nv_bfloat16*>(which == 1 ? g.c.k : g.c.v)) + to + h * to_h;
          *reinterpret_cast<uint4*>(row + ca) = a;
          *reinterpret_cast<uint4*>(row + cb) = b;
        }
      } else {
        uint2 qa, qb;
        float scale;
        quantize<L::kLanes>(y, qa, qb, scale);
        if (stores) {
          uint8_t* row = static_cast<uint8_t*>(which == 1 ? g.c.k : g.c.v) + to + h * to_h;
          *reinterpret_cast<uint2*>(row + ca) = qa;
          *reinterpret_cast<uint2*>(row + cb) = qb;
          if (j == 0) (which == 1 ? g.c.k_scale : g.c.v_scale)[to_scale + h * page_size] = scale;
        }
      }
    }
    __syncthreads();   // everyone has read this tile's tables and written those that come
    here = ahead;
  }
}

// ------------------------------------------------------------------------------------ host side

// log2 of the lane groups for a token's H heads.  kHeads to 2 kHeads heads for each group, which reads the angles
// once for them, dealt as evenly as one of the two numbers allows; more groups where the batch is too small for
// that to fill the SMs.
static int pick_shift(int H, int groups, long long tokens) {
  int shift = 0;
  while ((kHeads << shift) < H && (2 << shift) <= groups) ++shift;
  const auto idle = [H](int x) { return (-H & ((1 << x) - 1)) << (8 - x); };   // of a round of the groups, in 1/256
  if (shift > 0 && idle(shift - 1) < idle(shift)) --shift;
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
  *p = Plan{r->inv_freq, r->rot, r->norm != 0, r->eps, r->eps >= 0x1p-80f ? 0.f : 0x1p-76f};
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

static Pieces pieces_of(const fa_heads* x, int B, int H, int N, int d) {
  return Pieces{x->p, 2ll * d, {B, H, N}, {B > 1 ? 2 * x->stride_b : 0, H > 1 ? 2 * x->stride_h : 0, N > 1 ? 2 * x->stride_n : 0}};
}

// A tensor of a call and its heads.
struct Named {
  const fa_heads* x;
  int H;
};

// An output of H heads may be one of its `own` inputs, with the same strides, and shares no memory with the call's other
// tensors.
static int check_out(const fa_heads* out, const char* name, int B, int H, int N, int d, std::initializer_list<const fa_heads*> own,
                     std::initializer_list<Named> others) {
  const Pieces o = pieces_of(out, B, H, N, d);
  for (const fa_heads* x : own) {
    const bool same = x->p == out->p && (B == 1 || x->stride_b == out->stride_b) && (H == 1 || x->stride_h == out->stride_h) &&
                      (N == 1 || x->stride_n == out->stride_n);
    if (!same && pieces_overlap(o, pieces_of(x, B, H, N, d)))
      return set_error(FA_ERR_INVALID_ARG, "%s overlaps an input: it may be that input, with the same strides, only", name);
  }
  for (const Named& t : others)
    if (pieces_overlap(o, pieces_of(t.x, B, t.H, N, d)))
      return set_error(FA_ERR_INVALID_ARG, "%s overlaps another tensor of the call", name);
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

// What a token of H heads costs, in quarters of a vector; its angles, computed once, as much as `angles` quarters for whole
// heads.  Measured as the split that is fastest: forward 24 (15003 tokens, 28 + 4 heads, d = 128: 43.7 us, with 16 46.9; 16384
// tokens, 32 + 8: 57.6 and 57.1), backward and append 16 (8192 tokens, 32 + 8, both passes: 78.8 us, with 24 80.5;
// 23100 tokens into BF16 61.1, with 12 62.6, with 24 63.0).
constexpr int kForwardAngles = 24, kAngles = 16;
static long long token_cost(int H, int rot, int d, int angles) { return 4ll * H + angles * rot / d; }

// A side with its share of `all` CTAs, at least one: cost of `costs`.
template <int D>
static Side make_side(const fa_heads* x, const fa_heads* dz, const fa_heads* out, const void* w, int w_bf16, int H,
                      long long tokens, long long cost, long long costs, int all) {
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
  s.shift = pick_shift(H, Lanes<D>::kGroups, tokens);
  const int per = Lanes<D>::kGroups >> s.shift;
  const long long tiles = (tokens + per - 1) / per, share = std::max(1ll, all * cost / costs);
  s.ctas = (int)std::min(tiles, share);
  return s;
}

constexpr int kParts = 152 * kBwdCtas;   // CTAs of the backward at most, and its partial sums

template <int D, int kRingParts>
static int prepare(const void* kern, std::atomic<uint64_t>* done) {
  constexpr int bytes = (int)sizeof(Shared<D, kRingParts>);
  static_assert(kCtas * (sizeof(Shared<D, 2>) + sizeof(Places<Lanes<D>::kGroups>) + 1024) <= 228 * 1024 &&
                    kBwdCtas * (sizeof(Shared<D, 4>) + 1024) <= 228 * 1024,
                "an SM's CTAs fit its shared memory");
  return prepare_kernel(kern, bytes, kThreads, 0, "norm and rotation", done);
}

template <int D>
static int launch_forward(const fa_rotation* r, const Dense& g, const fa_heads* q, const fa_heads* k, const fa_heads* qo,
                          const fa_heads* ko, int Hq, int Hkv, cudaStream_t s) {
  const int all = kCtas * sm_count();
  const long long cq = token_cost(Hq, r->rot, D, kForwardAngles), ck = token_cost(Hkv, r->rot, D, kForwardAngles);
  const Side sq = make_side<D>(q, nullptr, qo, r->q_weight, r->weight_bf16, Hq, g.tokens, cq, cq + ck, all);
  const Side sk = make_side<D>(k, nullptr, ko, r->k_weight, r->weight_bf16, Hkv, g.tokens, ck, cq + ck, all);
  auto kern = r->interleaved ? norm_rotate_kernel<D, true> : norm_rotate_kernel<D, false>;
  static std::atomic<uint64_t> prepared[2];
  const int rc = prepare<D, 2>(reinterpret_cast<const void*>(kern), &prepared[r->interleaved != 0]);
  if (rc) return rc;
  kern<<<sq.ctas + sk.ctas, kThreads, sizeof(Shared<D, 2>), s>>>(g, sq, sk);
  return check_cuda(cudaGetLastError(), "launch fa_norm_rotate");
}

template <int D>
static int launch_backward(const fa_rotation* r, const Dense& g, const fa_heads* q, const fa_heads* k, const fa_heads* dzq,
                           const fa_heads* dzk, const fa_heads* dq, const fa_heads* dk, float* dqw, float* dkw, float* part,
                           int Hq, int Hkv, cudaStream_t s) {
  // (rounded down, but one CTA at least for each side: together kParts at most)
  const long long cq = token_cost(Hq, r->rot, D, kAngles), ck = token_cost(Hkv, r->rot, D, kAngles);
  const Side sq = make_side<D>(q, dzq, dq, r->q_weight, r->weight_bf16, Hq, g.tokens, cq, cq + ck, kParts);
  const Side sk = make_side<D>(k, dzk, dk, r->k_weight, r->weight_bf16, Hkv, g.tokens, ck, cq + ck, kParts);
  auto kern = r->interleaved ? norm_rotate_bwd_kernel<D, true> : norm_rotate_bwd_kernel<D, false>;
  static std::atomic<uint64_t> prepared[2];
  int rc = prepare<D, 4>(reinterpret_cast<const void*>(kern), &prepared[r->interleaved != 0]);
  if (rc) return rc;
  kern<<<sq.ctas + sk.ctas, kThreads, sizeof(Shared<D, 4>), s>>>(g, sq, sk, part);
  rc = check_cuda(cudaGetLastError(), "launch fa_norm_rotate_bwd");
  if (rc || !part) return rc;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return check_cuda(cudaLaunchKernelEx(&cfg, weight_grad_kernel, (const float*)part, D, sq.ctas, sk.ctas, dqw, dkw),
                    "launch fa_norm_rotate_bwd weights");
}

template <int D>
static int launch_append(const fa_rotation* r, const Packed& g, const fa_heads* q, const fa_heads* k, const fa_heads* v,
                         const fa_heads* qo, int Hq, int Hkv, bool fp8, cudaStream_t s) {
  const int all = kCtas * sm_count();
  const long long cq = token_cost(Hq, r->rot, D, kAngles), ck = token_cost(Hkv, r->rot, D, kAngles),
                  cv = token_cost(Hkv, 0, D, kAngles);
  const Side sq = make_side<D>(q, nullptr, qo, r->q_weight, r->weight_bf16, Hq, g.T, cq, cq + ck + cv, all);
  const Side sk = make_side<D>(k, nullptr, k, r->k_weight, r->weight_bf16, Hkv, g.T, ck, cq + ck + cv, all);
  const Side sv = make_side<D>(v, nullptr, v, nullptr, 0, Hkv, g.T, cv, cq + ck + cv, all);
  auto kern = r->interleaved ? (fp8 ? qkv_append_kernel<D, true, true> : qkv_append_kernel<D, true, false>)
                             : (fp8 ? qkv_append_kernel<D, false, true> : qkv_append_kernel<D, false, false>);
  static std::atomic<uint64_t> prepared[4];
  const int rc = prepare<D, 2>(reinterpret_cast<const void*>(kern), &prepared[2 * (r->interleaved != 0) + fp8]);
  if (rc) return rc;
  kern<<<sq.ctas + sk.ctas + sv.ctas, kThreads, sizeof(Shared<D, 2>), s>>>(g, sq, sk, sv);
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
      (rc = rotate::check_heads(k_out, "k_out", B, Hkv, N, true, d)) ||
      (rc = rotate::check_positions(positions)) || (rc = rotate::check_out(q_out, "q_out", B, Hq, N, d, {q}, {{k, Hkv}, {k_out, Hkv}})) ||
      (rc = rotate::check_out(k_out, "k_out", B, Hkv, N, d, {k}, {{q, Hq}})))
    return rc;
  const rotate::Dense g{p, positions, positions_stride, (unsigned)((long long)B * N), N};
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
  return (size_t)fa::rotate::kParts * d * sizeof(float);   // a row of d for each CTA
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
      (rc = rotate::check_out(dq, "dq", B, Hq, N, d, {q, dzq}, {{k, Hkv}, {dzk, Hkv}, {dk, Hkv}})) ||
      (rc = rotate::check_out(dk, "dk", B, Hkv, N, d, {k, dzk}, {{q, Hq}, {dzq, Hq}})) ||
      (rc = rotate::check_positions(positions)))
    return rc;
  if (!dq_weight != !dk_weight) return set_error(FA_ERR_INVALID_ARG, "dq_weight and dk_weight are given together or not at all");
  if (dq_weight && pieces_overlap({dq_weight, 4ll * d, {1, 1, 1}, {}}, {dk_weight, 4ll * d, {1, 1, 1}, {}}))
    return set_error(FA_ERR_INVALID_ARG, "dq_weight and dk_weight are one tensor, or overlap");
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
  const rotate::Dense g{p, positions, positions_stride, (unsigned)((long long)B * N), N};
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
  if (kv->B > (1 << 30)) return set_error(FA_ERR_INVALID_ARG, "B must be <= 2^30 (got %d)", kv->B);
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
  const auto rows = [T](const void* p, long long elems, long long stride) { return Pieces{p, 2 * elems, {T, 1, 1}, {2 * stride, 0, 0}}; };
  const Pieces out = rows(q_out, (long long)Hq * d, (long long)Hq * d);
  if ((!(q_out == q && (T == 1 || q_stride == (int64_t)Hq * d)) && pieces_overlap(out, rows(q, (long long)Hq * d, q_stride))) ||
      pieces_overlap(out, rows(k_new, (long long)Hkv * d, new_stride)) || pieces_overlap(out, rows(v_new, (long long)Hkv * d, new_stride)))
    return set_error(FA_ERR_INVALID_ARG, "q_out may be q, where that is contiguous, and overlaps no input otherwise");
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
