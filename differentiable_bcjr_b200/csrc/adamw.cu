// adamw.cu -- one AdamW step of many tensors in one launch (bcjr_adamw_step).
//
// An elementwise pass: every byte of p, g and the two states is read once and
// p and the states are written once, so memory bandwidth bounds it (28 B an
// element for float32 with 32-bit states, 10.06 B for bf16 with 8-bit ones).
// Measured: 16.8 M float32 elements with 32-bit states 73.8 us (6.4 TB/s, 98 %
// of the copy rate); 134 M bf16 elements with 8-bit states 352 us (3.8 TB/s; 361
// without the packed float32 operations on pairs).  These issue 67 instructions
// an element, nine of them the hash, which alone would take 240 us; the rest is
// latency that too few warps hide (42 % of them, issue 71 %): the loads of a block
// wait behind the arithmetic of the one before.  With a count on the device every
// CTA takes two powers before its first load, 395 us.
// The flat states are cut into blocks of 256 elements, the blocks that 8-bit
// scales belong to; a warp takes one block at a time, 8 elements a lane, and
// finds its tensor by bisection in a table that travels as a kernel
// parameter, so a call needs no device memory of its own and no copy.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>

#include "layer_util.cuh"

namespace {

using namespace bcjr;

constexpr int kBlock = 256;     // elements of a state block
constexpr int kWarps = 8;
constexpr float kTiny = 0x1p-100f;

struct Scalars {
  float b1, c1, b2, c2, eps, decay;  // c = 1 - b, decay = 1 - lr wd
  float lr_bc1, inv_sqrt_bc2;        // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t mix;                      // of step and seed
};

template <int CAP>
struct Table {
  void* p[CAP];
  const void* g[CAP];
  int64_t numel[CAP];
  int first_block[CAP];  // relative to the launch's first block
  int n;
  int blocks;            // of the launch
  int each;              // blocks of a warp
};

struct Common {
  void* first;
  void* second;
  float* scales;           // [2][all blocks] (8-bit states)
  size_t all_blocks;
  size_t block0;           // of the launch within the flat states
  const int64_t* step_ptr;
  const float* grad_scale;
  double lr, beta1, beta2;
  uint32_t seed;
  bool small_eps;          // a subnormal second moment's root counts beside eps
  Scalars s;
};

__host__ __device__ inline uint32_t mix_of(uint32_t step, uint32_t seed) {
  return step * 0x632BE5ABu + seed * 0x85157AF5u;
}

__host__ __device__ inline void bias_scalars(double lr, double b1, double b2, double t, Scalars& s) {
  s.lr_bc1 = static_cast<float>(lr / (1.0 - pow(b1, t)));
  s.inv_sqrt_bc2 = static_cast<float>(1.0 / sqrt(1.0 - pow(b2, t)));
}

// 32 bits a (step, seed, element), 16 for either rounding: a multiply and
// xor-shift mix of h = element * kHashA + mix_of(step, seed); multipliers and
// shifts of C. Wellons, "Prospecting for Hash Functions", 2018.
constexpr uint32_t kHashA = 0x9E3779B1u;
__device__ __forceinline__ uint32_t hash_bits(uint32_t h) {
  h = (h ^ (h >> 15)) * 0x2C1B3C6Du;
  h = (h ^ (h >> 12)) * 0x297A2D39u;
  return h ^ (h >> 15);
}

// The code of the magnitude of x (a float's bits), scaled so that its block's largest is 448 2^-120:
// a float's exponent field is then e4m3's, so the code is the float's bits cut
// after three mantissa bits; the 20 bits that fall away decide the rounding
// together with `random`, 16 bits and a half.  Sixteen times their sum has the
// code in its upper byte (a sign bit of x leaves at the top).  The largest (at most a few places off 448) does not
// round up, since random is at least eight places short of a whole step.
__device__ __forceinline__ uint32_t e4m3_upper(uint32_t x, uint32_t random) {
  uint32_t d;  // (a multiply-add, where a shift and an add would load the busier integer pipe)
  asm("mad.lo.u32 %0, %1, 16, %2;" : "=r"(d) : "r"(x), "r"(random));
  return d;
}

// The upper bytes of four words.
__device__ __forceinline__ uint32_t upper_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// Byte i of a word as a float times 2^-120, exactly (subnormal codes are subnormal floats).
template <bool SIGNED>
__device__ __forceinline__ float e4m3_small(uint32_t w, int i) {
  if (SIGNED) return __uint_as_float(static_cast<uint32_t>(static_cast<int32_t>(w << (24 - 8 * i)) >> 4) & 0x87F00000u);
  return __uint_as_float((i == 3 ? w >> 4 : w << (20 - 8 * i)) & 0x07F00000u);
}

__device__ __forceinline__ float sqrt_approx(float v) {  // within 2^-23 of the root, denormals included
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_approx(float v) {  // within 2^-23; 0 above 2^126
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Two sums.  Packed ones are contracted with packed products here, whatever
// rounding is asked for (scales then differ by one place); these are not.
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }

// The roots of two v in [2^-126, 2^128) correctly rounded but for a case in
// millions: y = 1 / sqrt(v) gives g = v y, whose square is v up to a few places,
// and one Newton step g + (v - g^2) y / 2 with the exact residual of a fused
// multiply-add (P. Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990).  A few operations without a branch, where
// __fsqrt_rn takes twice as long here.  0 gives 0; another v below 2^-126 a root
// that is positive but too small (y stops at 2^63), under 2^-62; infinity a NaN.
// block_step8 looks for what these come to; their blocks take roots_of_all.
__device__ __forceinline__ float2 roots(float2 v) {
  float2 y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(fmaxf(v.x, 0x1p-126f)));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(fmaxf(v.y, 0x1p-126f)));
  const float2 g = __fmul2_rn(v, y);
  return __ffma2_rn(__ffma2_rn(g, g, __fmul2_rn(v, both(-1.f))), __fmul2_rn(y, both(-0.5f)), g);
}

// The same for every v: a power of four brings what is below 2^-126 into range, and its root takes it back out.
__device__ __forceinline__ float2 roots_of_all(float2 v) {
  const bool sx = v.x < 0x1p-126f, sy = v.y < 0x1p-126f;
  float2 r = roots(__fmul2_rn(v, make_float2(sx ? 0x1p64f : 1.f, sy ? 0x1p64f : 1.f)));
  r = __fmul2_rn(r, make_float2(sx ? 0x1p-32f : 1.f, sy ? 0x1p-32f : 1.f));
  const float inf = __uint_as_float(0x7F800000u);
  return make_float2(v.x == inf ? inf : r.x, v.y == inf ? inf : r.y);
}

// Which elements of its block a lane holds: COALESCED 4 at 4 lane and 4 at
// 128 + 4 lane (16-byte loads of float32); PACKED 8 at 8 lane (16-byte loads
// of 16-bit types); STRIDED lane, lane + 32, ... one by one, for tensors that
// are not 16-byte aligned and for the last block of a tensor.
enum Map { COALESCED, PACKED, STRIDED };

template <Map MAP>
__device__ __forceinline__ int element_of(int lane, int i) {
  if (MAP == COALESCED) return (i >> 2) * 128 + lane * 4 + (i & 3);
  if (MAP == PACKED) return lane * 8 + i;
  return i * 32 + lane;
}

template <int BYTES>
struct Raw;
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<8> { using type = uint2; };
template <>
struct Raw<16> { using type = uint4; };

template <typename T, Map MAP>
__device__ __forceinline__ void load8(const T* base, int lane, int limit, T (&v)[8]) {
  if constexpr (MAP == STRIDED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = element_of<MAP>(lane, i);
      if (e < limit) v[i] = base[e];
      else memset(&v[i], 0, sizeof(T));
    }
  } else {
    constexpr int RUN = MAP == PACKED ? 8 : 4;
    static_assert(RUN * sizeof(T) <= 16, "one vector access a run");
    using V = typename Raw<RUN * sizeof(T)>::type;
#pragma unroll
    for (int i = 0; i < 8; i += RUN) {
      const V x = *reinterpret_cast<const V*>(base + element_of<MAP>(lane, i));
      memcpy(&v[i], &x, sizeof(V));
    }
  }
}

template <typename T, Map MAP>
__device__ __forceinline__ void store8(T* base, int lane, int limit, const T (&v)[8]) {
  if constexpr (MAP == STRIDED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = element_of<MAP>(lane, i);
      if (e < limit) base[e] = v[i];
    }
  } else {
    constexpr int RUN = MAP == PACKED ? 8 : 4;
    using V = typename Raw<RUN * sizeof(T)>::type;
#pragma unroll
    for (int i = 0; i < 8; i += RUN) {
      V x;
      memcpy(&x, &v[i], sizeof(V));
      *reinterpret_cast<V*>(base + element_of<MAP>(lane, i)) = x;
    }
  }
}

// m, v and p of one element.
__device__ __forceinline__ float advance(float& m, float& v, float g, float p, const Scalars& s) {
  m = fmaf(m, s.b1, g * s.c1);
  v = fmaf(v, s.b2, g * g * s.c2);
  const float step = m * rcp_approx(fmaf(sqrt_approx(v), s.inv_sqrt_bc2, s.eps));
  return fmaf(-s.lr_bc1, step, p * s.decay);
}

// m, r = sqrt(v) and p of two elements.  8-bit codes are rounded from m and r:
// every operation on the way is rounded by itself and correctly, so that a
// code does not hang on how the compiler contracts products and sums (one
// code more or less is a sixteenth of the value, far over what the parameter's
// float32 arithmetic leaves).
template <bool ALL>
__device__ __forceinline__ float2 advance2(float2& m, float2& r, float2 g, float2 p, const Scalars& s) {
  m = add2(__fmul2_rn(m, both(s.b1)), __fmul2_rn(g, both(s.c1)));
  const float2 v = add2(__fmul2_rn(__fmul2_rn(r, r), both(s.b2)), __fmul2_rn(__fmul2_rn(g, g), both(s.c2)));
  r = ALL ? roots_of_all(v) : roots(v);
  const float2 d = __ffma2_rn(r, both(s.inv_sqrt_bc2), both(s.eps));
  const float2 step = __fmul2_rn(m, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
  return __ffma2_rn(step, both(-s.lr_bc1), __fmul2_rn(p, both(s.decay)));
}

// One block of one tensor.  `limit`: elements of the block that exist.
template <typename P, typename G, Map MAP>
__device__ __forceinline__ void block_step32(P* p, const G* g, const Common& c, const Scalars& s, float gs,
                                             size_t block, int lane, int limit) {
  float* const first = static_cast<float*>(c.first) + block * kBlock;
  float* const second = static_cast<float*>(c.second) + block * kBlock;
  P pv[8];
  G gv[8];
  float m[8], v[8];
  load8<float, MAP>(first, lane, kBlock, m);
  load8<float, MAP>(second, lane, kBlock, v);
  load8<G, MAP>(g, lane, limit, gv);
  load8<P, MAP>(p, lane, limit, pv);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    pv[i] = from_f32<P>(advance(m[i], v[i], __fmul_rn(to_f32(gv[i]), gs), to_f32(pv[i]), s));
  }
  store8<P, MAP>(p, lane, limit, pv);
  store8<float, MAP>(first, lane, MAP == STRIDED ? limit : kBlock, m);
  store8<float, MAP>(second, lane, MAP == STRIDED ? limit : kBlock, v);
}

// ALL: for every second moment; otherwise false, and nothing stored, where the
// block holds one that roots() does not do.
template <typename P, typename G, Map MAP, bool ALL>
__device__ __forceinline__ bool block_step8(P* p, const G* g, const Common& c, const Scalars& s, float gs,
                                            size_t block, int lane, int limit) {
  uint8_t* const first = static_cast<uint8_t*>(c.first) + block * kBlock;
  uint8_t* const second = static_cast<uint8_t*>(c.second) + block * kBlock;
  P pv[8];
  float2 m[4], r[4];
  G gv[8];
  uint8_t a[8], b[8];
  load8<uint8_t, MAP>(first, lane, kBlock, a);
  load8<uint8_t, MAP>(second, lane, kBlock, b);
  load8<G, MAP>(g, lane, limit, gv);
  load8<P, MAP>(p, lane, limit, pv);
  const float sa = c.scales[block], sb = c.scales[c.all_blocks + block];
  uint32_t wa[2], wb[2];
  memcpy(wa, a, 8);
  memcpy(wb, b, 8);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    m[i / 2] = make_float2(e4m3_small<true>(wa[i >> 2], i & 3), e4m3_small<true>(wa[i >> 2], (i & 3) + 1));
    r[i / 2] = make_float2(e4m3_small<false>(wb[i >> 2], i & 3), e4m3_small<false>(wb[i >> 2], (i & 3) + 1));
  }
  // A code is its float times 2^-120; bringing that back and the scale are one
  // product where 2^120 times the scale is a float (a uniform choice: scales
  // of 128 and more stand for moments beyond 2^15).
  float fa = sa * 0x1p120f, fb = sb * 0x1p120f;
  if (!(sa < 128.f && sb < 128.f)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = __fmul2_rn(m[i], both(0x1p120f));
      r[i] = __fmul2_rn(r[i], both(0x1p120f));
    }
    fa = sa;
    fb = sb;
  }
  // the order of the magnitudes' bits is that of the values, NaN above all
  uint32_t ta = 0, tb = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = __fmul2_rn(m[i], both(fa));
    r[i] = __fmul2_rn(r[i], both(fb));
    const float2 g2 = __fmul2_rn(make_float2(to_f32(gv[2 * i]), to_f32(gv[2 * i + 1])), both(gs));
    const float2 p2 = advance2<ALL>(m[i], r[i], g2, make_float2(to_f32(pv[2 * i]), to_f32(pv[2 * i + 1])), s);
    pv[2 * i] = from_f32<P>(p2.x);
    pv[2 * i + 1] = from_f32<P>(p2.y);
    if (MAP == STRIDED) {
      if (element_of<MAP>(lane, 2 * i) >= limit) m[i].x = r[i].x = 0.f;
      if (element_of<MAP>(lane, 2 * i + 1) >= limit) m[i].y = r[i].y = 0.f;
    }
    ta = max(ta, max(__float_as_uint(m[i].x) << 1, __float_as_uint(m[i].y) << 1));
    tb = max(tb, max(__float_as_uint(r[i].x), __float_as_uint(r[i].y)));
  }
  const uint32_t most_b = __reduce_max_sync(~0u, tb) & 0x7FFFFFFFu;
  if constexpr (!ALL) {
    // roots() does not do (uniform, and rare):
    // - an infinite v, whose root came out as a NaN (as a NaN's does);
    // - subnormal ones (whose roots are under 2^-63) where they reach codes.  Beside
    //   a largest root of 2^-45 they have the smallest code whatever they are exactly;
    // - subnormal ones where they reach parameters, which they do beside a small eps.
    if (most_b > 0x7F800000u || (most_b != 0 && most_b < __float_as_uint(0x1p-45f))) return false;
    if (c.small_eps) {
      bool some = false;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        some = some || __float_as_uint(r[i].x) - 1u < __float_as_uint(0x1p-62f) || __float_as_uint(r[i].y) - 1u < __float_as_uint(0x1p-62f);
      if (__any_sync(~0u, some)) return false;
    }
  }
  store8<P, MAP>(p, lane, limit, pv);
  const float top_a = __uint_as_float(__reduce_max_sync(~0u, ta) >> 1);
  const float top_b = __uint_as_float(most_b);
  const bool held_a = !(top_a < kTiny), held_b = !(top_b < kTiny);
  float inv_a = held_a ? __fmul_rn(__frcp_rn(top_a), 448.f) : 0.f, inv_b = held_b ? __fmul_rn(__frcp_rn(top_b), 448.f) : 0.f;
  const uint32_t least_b = held_b ? 1u << 24 : 0u;  // r > 0 (then it is at least 2^-75) does not become 0
  // The factor 2^-120 goes into the reciprocal where that stays a normal float.
  float small = 1.f;
  if (inv_a >= 0x1p-5f && inv_b >= 0x1p-5f) {
    inv_a *= 0x1p-120f;
    inv_b *= 0x1p-120f;
  } else {
    small = 0x1p-120f;
  }
  uint32_t h0 = (static_cast<uint32_t>(block * kBlock) + element_of<MAP>(lane, 0)) * kHashA + s.mix;
  uint32_t ua[8], ub[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x = __fmul2_rn(m[i], both(inv_a)), y = __fmul2_rn(r[i], both(inv_b));
    if (small != 1.f) {
      x = __fmul2_rn(x, both(small));
      y = __fmul2_rn(y, both(small));
    }
    const uint32_t two[2][4] = {{__float_as_uint(x.x), __float_as_uint(y.x), __float_as_uint(m[i].x), __float_as_uint(r[i].x)},
                                {__float_as_uint(x.y), __float_as_uint(y.y), __float_as_uint(m[i].y), __float_as_uint(r[i].y)}};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t h = hash_bits(h0 + static_cast<uint32_t>(element_of<MAP>(0, 2 * i + q) - element_of<MAP>(0, 0)) * kHashA);
      const uint32_t a4 = e4m3_upper(two[q][0], __byte_perm(h, 0x80u, 0x5324));  // h's upper half between 0 and 0x80
      const uint32_t b4 = e4m3_upper(two[q][1], __byte_perm(h, 0x80u, 0x5104));  // and its lower half
      ua[2 * i + q] = (a4 & 0x7FFFFFFFu) | (two[q][2] & 0x80000000u);
      ub[2 * i + q] = max(b4, min(two[q][3], least_b));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    wa[i >> 2] = upper_bytes(ua[i], ua[i + 1], ua[i + 2], ua[i + 3]);
    wb[i >> 2] = upper_bytes(ub[i], ub[i + 1], ub[i + 2], ub[i + 3]);
  }
  memcpy(a, wa, 8);
  memcpy(b, wb, 8);
  if (lane == 0) {
    c.scales[block] = held_a ? __fmul_rn(top_a, 1.f / 448.f) : 0.f;
    // an infinite second moment would hold its block's parameters still for good: a NaN shows instead
    c.scales[c.all_blocks + block] = !held_b ? 0.f : top_b <= 3.402823466e38f ? __fmul_rn(top_b, 1.f / 448.f) : __uint_as_float(0x7FC00000u);
  }
  store8<uint8_t, MAP>(first, lane, MAP == STRIDED ? limit : kBlock, a);
  store8<uint8_t, MAP>(second, lane, MAP == STRIDED ? limit : kBlock, b);
  return true;
}

// False: not done (see block_step8).
template <typename P, typename G, int BITS, Map MAP>
__device__ __forceinline__ bool block_step(P* p, const G* g, const Common& c, const Scalars& s, float gs,
                                           size_t block, int lane, int limit) {
  if constexpr (BITS == 32) {
    block_step32<P, G, MAP>(p, g, c, s, gs, block, lane, limit);
    return true;
  } else {
    return block_step8<P, G, MAP, false>(p, g, c, s, gs, block, lane, limit);
  }
}

template <typename P, typename G, int BITS, int CAP>
__global__ void __launch_bounds__(kWarps * 32) adamw_kernel(const __grid_constant__ Table<CAP> t,
                                                            const __grid_constant__ Common c) {
  Scalars s = c.s;
  if (c.step_ptr) {  // uniform: the step count is only known now
    __shared__ Scalars shared;
    if (threadIdx.x == 0) {
      const int64_t step = *c.step_ptr;
      shared = c.s;
      bias_scalars(c.lr, c.beta1, c.beta2, static_cast<double>(step), shared);
      shared.mix = mix_of(static_cast<uint32_t>(step), c.seed);
    }
    __syncthreads();
    s = shared;
  }
  const float gs = c.grad_scale ? *c.grad_scale : 1.f;
  const int lane = threadIdx.x & 31;
  const int b0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * t.each, end = min(b0 + t.each, t.blocks);
  if (b0 >= end) return;
  int lo = 0, hi = t.n - 1;  // the last tensor that starts at or before b0
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first_block[mid] <= b0) lo = mid;
    else hi = mid - 1;
  }
  constexpr Map FULL = (BITS == 8 && sizeof(P) == 2 && sizeof(G) == 2) ? PACKED : COALESCED;
  uint32_t left_out = 0;  // which of the warp's blocks (32 at most) are not done
  for (int b = b0; b < end; ++b) {
    while (lo + 1 < t.n && t.first_block[lo + 1] <= b) ++lo;
    if (!t.g[lo]) continue;
    const int64_t at = static_cast<int64_t>(b - t.first_block[lo]) * kBlock;
    const int64_t left = t.numel[lo] - at;
    P* const p = static_cast<P*>(t.p[lo]) + at;
    const G* const g = static_cast<const G*>(t.g[lo]) + at;
    const size_t block = c.block0 + b;
    bool done;
    if (left >= kBlock && ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(g)) & 15) == 0)
      done = block_step<P, G, BITS, FULL>(p, g, c, s, gs, block, lane, kBlock);
    else
      done = block_step<P, G, BITS, STRIDED>(p, g, c, s, gs, block, lane, left < kBlock ? static_cast<int>(left) : kBlock);
    if (!done) left_out |= 1u << (b - b0);
  }
  if constexpr (BITS == 8) {
    // A loop of its own, which shares registers with the one above: within that
    // one it costs every block some (80 and more a thread, two layers of bf16 410
    // us; so 352, and 348 without it).
    for (; left_out; left_out &= left_out - 1) {
      const int b = b0 + __ffs(static_cast<int>(left_out)) - 1;
      for (lo = t.n - 1; t.first_block[lo] > b;) --lo;
      const int64_t at = static_cast<int64_t>(b - t.first_block[lo]) * kBlock, left = t.numel[lo] - at;
      block_step8<P, G, STRIDED, true>(static_cast<P*>(t.p[lo]) + at, static_cast<const G*>(t.g[lo]) + at, c, s, gs, c.block0 + b, lane,
                                       left < kBlock ? static_cast<int>(left) : kBlock);
    }
  }
}

template <typename P, typename G, int BITS, int CAP>
bcjr_status launch(const bcjr_adamw_tensor* ts, int n, Common& c, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return BCJR_ERR_CUDA;
  Table<CAP> t;
  t.n = 0;
  int64_t blocks = 0;
  for (int i = 0; i <= n; ++i) {
    const int64_t more = i < n ? (ts[i].numel + kBlock - 1) / kBlock : 0;
    // a launch's blocks are counted in an int
    if (t.n > 0 && (i == n || t.n == CAP || blocks + more > (int64_t{1} << 30))) {
      t.blocks = static_cast<int>(blocks);
      // finding a block's tensor and the step's constants costs as much as some
      // elements do: several blocks a warp once there are enough for all warps
      t.each = BITS == 8 && blocks >= int64_t{4} * 64 * sms ? 4 : 1;  // at most 32
      const int64_t per_cta = int64_t{kWarps} * t.each;
      const unsigned grid = static_cast<unsigned>((blocks + per_cta - 1) / per_cta);
      adamw_kernel<P, G, BITS, CAP><<<grid, kWarps * 32, 0, stream>>>(t, c);
      const bcjr_status st = launched();
      if (st != BCJR_OK) return st;
      c.block0 += static_cast<size_t>(blocks);
      t.n = 0;
      blocks = 0;
    }
    if (i == n || more == 0) continue;
    t.p[t.n] = ts[i].param;
    t.g[t.n] = ts[i].grad;
    t.numel[t.n] = ts[i].numel;
    t.first_block[t.n] = static_cast<int>(blocks);
    ++t.n;
    blocks += more;
  }
  return BCJR_OK;
}

// Tables of 128 tensors fit the classic 4 KB of kernel parameters, which are
// cheaper to launch with; 1024 tensors take 28 KB.
template <typename P, typename G, int BITS>
bcjr_status launch_any(const bcjr_adamw_tensor* ts, int n, Common& c, cudaStream_t stream) {
  return n <= 128 ? launch<P, G, BITS, 128>(ts, n, c, stream) : launch<P, G, BITS, 1024>(ts, n, c, stream);
}

template <typename P, typename G>
bcjr_status launch_bits(const bcjr_adamw_tensor* ts, int n, int bits, Common& c, cudaStream_t stream) {
  return bits == 8 ? launch_any<P, G, 8>(ts, n, c, stream) : launch_any<P, G, 32>(ts, n, c, stream);
}

struct Span {
  uintptr_t begin, end;
};

// Whether no two of the parameters share memory.  Sorted in place (a heap sort: no allocation, no exception).
bool apart(Span* spans, int n) {
  auto less = [](const Span& a, const Span& b) { return a.begin < b.begin; };
  bool sorted = true;
  for (int i = 1; i < n; ++i) sorted = sorted && spans[i - 1].end <= spans[i].begin;
  if (sorted) return true;
  std::make_heap(spans, spans + n, less);
  std::sort_heap(spans, spans + n, less);
  for (int i = 1; i < n; ++i) {
    if (spans[i - 1].end > spans[i].begin) return false;
  }
  return true;
}

}  // namespace

extern "C" bcjr_status bcjr_adamw_step(const bcjr_adamw_tensor* tensors, int n_tensors, int param_dtype,
                                       int grad_dtype, int state_bits, void* first, void* second, float* scales,
                                       const bcjr_adamw_options* o, bcjr_stream_t stream) {
  if (n_tensors < 0 || (n_tensors > 0 && !tensors) || !o) return BCJR_ERR_INVALID_ARG;
  if (!dtype_ok(param_dtype) || !dtype_ok(grad_dtype)) return BCJR_ERR_INVALID_ARG;
  if (state_bits != 8 && state_bits != 32) return BCJR_ERR_UNSUPPORTED;
  if (param_dtype != BCJR_F32 && grad_dtype != BCJR_F32 && grad_dtype != param_dtype) return BCJR_ERR_UNSUPPORTED;
  if (!std::isfinite(o->lr) || o->lr < 0 || !(o->beta1 >= 0 && o->beta1 < 1) || !(o->beta2 >= 0 && o->beta2 < 1) ||
      !(o->eps >= 0) || !std::isfinite(o->eps) || !std::isfinite(o->weight_decay) || o->weight_decay < 0)
    return BCJR_ERR_INVALID_ARG;
  if (!o->step_ptr && o->step < 1) return BCJR_ERR_INVALID_ARG;
  int64_t blocks = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const bcjr_adamw_tensor& t = tensors[i];
    if (t.numel < 0 || t.numel > (int64_t{1} << 37)) return BCJR_ERR_INVALID_ARG;
    if (t.numel > 0 && (!t.param || !ptr_aligned(t.param, dtype_size(param_dtype)) ||
                        !ptr_aligned(t.grad, dtype_size(grad_dtype))))
      return BCJR_ERR_INVALID_ARG;
    blocks += (t.numel + kBlock - 1) / kBlock;
  }
  if (blocks == 0) return BCJR_OK;
  {
    Span few[256];
    std::unique_ptr<Span[]> many;
    Span* spans = few;
    if (n_tensors > 256) {
      many.reset(new (std::nothrow) Span[n_tensors]);
      if (!many) return BCJR_ERR_WORKSPACE;
      spans = many.get();
    }
    int n = 0;
    for (int i = 0; i < n_tensors; ++i) {
      if (tensors[i].numel == 0) continue;
      const uintptr_t at = reinterpret_cast<uintptr_t>(tensors[i].param);
      spans[n++] = {at, at + static_cast<uintptr_t>(tensors[i].numel) * dtype_size(param_dtype)};
    }
    if (!apart(spans, n)) return BCJR_ERR_INVALID_ARG;
  }
  if (!first || !second || !ptr_aligned(first, 16) || !ptr_aligned(second, 16)) return BCJR_ERR_INVALID_ARG;
  if ((state_bits == 8) != (scales != nullptr) || !ptr_aligned(scales, 4) || !ptr_aligned(o->grad_scale, 4) ||
      !ptr_aligned(o->step_ptr, 8))
    return BCJR_ERR_INVALID_ARG;
  {
    // nor may the states share memory with one another, a parameter or a gradient
    auto span = [](const void* p, int64_t bytes) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      return Span{at, p ? at + static_cast<uintptr_t>(bytes) : at};
    };
    auto meet = [](const Span& a, const Span& b) { return a.begin < b.end && b.begin < a.end; };
    const int64_t bytes = blocks * kBlock * (state_bits / 8);
    const Span s[3] = {span(first, bytes), span(second, bytes), span(scales, blocks * 8)};
    if (meet(s[0], s[1]) || meet(s[0], s[2]) || meet(s[1], s[2])) return BCJR_ERR_INVALID_ARG;
    const Span all = {std::min({s[0].begin, s[1].begin, scales ? s[2].begin : s[1].begin}), std::max({s[0].end, s[1].end, s[2].end})};
    const uintptr_t p_size = dtype_size(param_dtype), g_size = dtype_size(grad_dtype);
    for (int i = 0; i < n_tensors; ++i) {
      const uintptr_t n = static_cast<uintptr_t>(tensors[i].numel);
      const uintptr_t p_at = reinterpret_cast<uintptr_t>(tensors[i].param), g_at = reinterpret_cast<uintptr_t>(tensors[i].grad);
      const Span p = {p_at, p_at + n * p_size}, g = {g_at, g_at + n * g_size};
      if (n == 0 || (!meet(all, p) && !meet(all, g))) continue;
      for (const Span& state : s)
        if (meet(state, p) || (g_at && meet(state, g))) return BCJR_ERR_INVALID_ARG;
    }
  }
  Common c = {};
  c.first = first;
  c.second = second;
  c.scales = scales;
  c.all_blocks = static_cast<size_t>(blocks);
  c.step_ptr = o->step_ptr;
  c.grad_scale = o->grad_scale;
  c.lr = o->lr;
  c.beta1 = o->beta1;
  c.beta2 = o->beta2;
  c.seed = o->seed;
  c.s.b1 = static_cast<float>(o->beta1);
  c.s.c1 = static_cast<float>(1.0 - o->beta1);
  c.s.b2 = static_cast<float>(o->beta2);
  c.s.c2 = static_cast<float>(1.0 - o->beta2);
  // a subnormal denominator's approximate reciprocal is infinite, and 0 times it a NaN; beside the root of a v > 0
  // (2^-75 at least) what is added here does not show
  c.s.eps = o->eps > 0 && o->eps < 0x1p-126 ? 0x1p-126f : static_cast<float>(o->eps);
  c.s.decay = static_cast<float>(1.0 - o->lr * o->weight_decay);
  // a root of a subnormal v is under 2^-63, and its bias correction is largest in the first step; what is left out
  // beside an eps 2^24 times as large does not show
  c.small_eps = o->eps < 0x1p-39 / std::sqrt(1.0 - o->beta2);
  if (!o->step_ptr) {
    bias_scalars(o->lr, o->beta1, o->beta2, static_cast<double>(o->step), c.s);
    c.s.mix = mix_of(static_cast<uint32_t>(o->step), o->seed);
  }
  cudaStream_t s = as_stream(stream);
  if (param_dtype == BCJR_F32) {
    if (grad_dtype == BCJR_F32) return launch_bits<float, float>(tensors, n_tensors, state_bits, c, s);
    if (grad_dtype == BCJR_F16) return launch_bits<float, __half>(tensors, n_tensors, state_bits, c, s);
    return launch_bits<float, __nv_bfloat16>(tensors, n_tensors, state_bits, c, s);
  }
  if (param_dtype == BCJR_F16)
    return grad_dtype == BCJR_F32 ? launch_bits<__half, float>(tensors, n_tensors, state_bits, c, s)
                                  : launch_bits<__half, __half>(tensors, n_tensors, state_bits, c, s);
  return grad_dtype == BCJR_F32 ? launch_bits<__nv_bfloat16, float>(tensors, n_tensors, state_bits, c, s)
                                : launch_bits<__nv_bfloat16, __nv_bfloat16>(tensors, n_tensors, state_bits, c, s);
}
