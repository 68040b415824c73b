// int4_matmul.cuh -- a few tokens times 4-bit weights (bcjr_int4_matmul).
//
// Weights are the 16-row operand of mma.m16n8k16 and tokens its 8 columns, so
// eight tokens cost what one does.  A lane's 16-byte load of a packed tile
// holds, word by word, the codes of its fragment positions in columns 32 j +
// 8 t .. + 7: (word >> 4 i) & 0x000F000F is the fragment register of columns
// 8 t + 2 i and + 1, which or-ed with the bits of 128 (bf16; 1024 in half)
// is exactly 128 + q, and one packed subtraction gives q - zero, exactly.
// Group sums stay in float32 and are scaled in float32, so the only rounding
// is that of the sums.  float32 tokens are cut into three bf16 parts of 8
// bits (exact, the lower ones held 2^8 and 2^16 times as large), which take three
// of the eight columns.
//
// Global loads return in the order they were issued, so inputs and scales are
// staged in shared memory first and only the weights, two tiles ahead, are
// loaded beside the products.
//
// Up to four columns (tokens, or parts of them): a CTA owns 16 or 32 rows, its 16
// warps split the columns of the matrix and add their sums in a fixed order.
// More: a CTA owns 128 rows, 16 a warp, so that staged tokens serve more rows;
// the CTAs of a cluster split the columns of the matrix and add their sums
// through distributed shared memory in a fixed order.
//
// Measured, device time a call with the weights in memory (in the L2 cache): 8192 x
// 8192 in groups of 128, one bf16 token 11.4 us (10.7; 34.6 MB: 3.0 TB/s; reading
// them alone takes 6.4 us from memory with as many threads), 8 tokens 13.1 (12.4),
// 32 tokens 22.9 (22.3), one float32 token 13.1 (12.3), ten 23.7 (22.6); 16384 x
// 8192 in groups of 32, 16 half tokens 36.8 (33.9).  No pipe is full: one token
// issues half of the time, the integer pipe (masks and shifts) is busy 42 %, the
// matrix instruction 19 %, and 16 tokens less.  It is latency: two tiles of weights
// are on their way for a warp, and for several tokens every chunk's staging is
// waited for.  More than 32 tokens take as many passes over the weights (256
// tokens 152 us, 2048 tokens 1.0 ms).
#pragma once
#include <cooperative_groups.h>

#include <cstring>

#include "int4_internal.h"
#include "layer_util.cuh"

namespace cg = cooperative_groups;

namespace bcjr {
namespace {

using Params = Int4MatmulParams;

// (a & mask) | bits in one instruction (two immediates would take two)
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
  return d;
}

template <typename T>
struct Half2;  // the packed 16-bit type that multiplies T

template <>
struct Half2<__half> {
  static constexpr uint32_t kMagic = 0x64006400u;
  // The eight codes of a word less the zero point.  In the mantissa's low bits
  // beside the bits of 1024 a code is 1024 + q; four bits higher 1024 + 16 q,
  // which one fused multiply-add brings down, saving two of the three shifts.
  static __device__ __forceinline__ uint32_t zero_pair(uint32_t z) { return 0x64006400u + z * 0x00010001u; }  // 1024 + z
  static __device__ __forceinline__ void words(uint32_t w, uint32_t off, uint32_t magic, uint32_t (&out)[4]) {
    const uint32_t off16 = off * 16 + (0xD400D400u - 0x40064000u);  // -(64 + z): the last place of 64 in half is 1/16
    const uint32_t v = w >> 8;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(out[0]) : "r"(and_or(w, 0x000F000Fu, magic)), "r"(off));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(out[1]) : "r"(and_or(w, 0x00F000F0u, magic)), "r"(0x2C002C00u), "r"(off16));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(out[2]) : "r"(and_or(v, 0x000F000Fu, magic)), "r"(off));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(out[3]) : "r"(and_or(v, 0x00F000F0u, magic)), "r"(0x2C002C00u), "r"(off16));
  }
  static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  // the same onto nothing
  static __device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  }
};

template <>
struct Half2<__nv_bfloat16> {
  static constexpr uint32_t kMagic = 0x43004300u;
  static __device__ __forceinline__ uint32_t zero_pair(uint32_t z) { return 0x43004300u + z * 0x00010001u; }  // 128 + z
  static __device__ __forceinline__ void words(uint32_t w, uint32_t off, uint32_t magic, uint32_t (&out)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(out[i]) : "r"(and_or(w >> (4 * i), 0x000F000Fu, magic)), "r"(off));
  }
  static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  // the same onto nothing
  static __device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  }
};

template <>
struct Half2<float> : Half2<__nv_bfloat16> {};

// A float as three bf16's bits: the upper 8 bits of its mantissa, the next 8
// times 2^8, the last 8 times 2^16, each cut off exactly (where they are they may
// lie below bf16's smallest number, 2^-133).  An infinity is its own first part
// and leaves 0 for the others; a NaN, also one of the lowest bits alone, has one there.
constexpr float kPart = 0x1p8f, kPartDown = 0x1p-8f;
__device__ __forceinline__ bool finite(float v) { return fabsf(v) <= 3.402823466e38f; }
__device__ __forceinline__ void parts_of(float v, uint32_t (&out)[3]) {
  const float top = __uint_as_float((v == v ? __float_as_uint(v) : 0x7FFF0000u) & 0xFFFF0000u);
  const float rest = top == v ? 0.f : __fmul_rn(v - top, kPart);
  const float mid = __uint_as_float(__float_as_uint(rest) & 0xFFFF0000u);
  const float low = __fmul_rn(rest - mid, kPart);
  out[0] = __float_as_uint(top) >> 16;
  out[1] = __float_as_uint(mid) >> 16;
  out[2] = __float_as_uint(low) >> 16;
}

// A sum over values or over one of their parts, of mma column `column`, as it
// counts in the values' sum.  What is not finite comes with the first part: a
// lower part's 0 times an infinite scale is a NaN that the value has not.  (Done
// where sums are written: where they are added up it keeps their loads from
// running ahead, 4.9 us a call for 4.5.)
template <int PARTS>
__device__ __forceinline__ float part_sum(float v, int column) {
  return column % PARTS == 0 ? v : (finite(v) ? v : 0.f) * (column % PARTS == 1 ? kPartDown : kPartDown * kPartDown);
}

// Weights are read once: they would only push the inputs out of the L1 cache.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

constexpr int kWarps = 16;

struct Group {  // of one row
  float scale;
  uint32_t zero;  // what the codes' bits less their zero point start from
};

// A group's sums, scaled, onto the total: rows g (the first two) and g + 8.
__device__ __forceinline__ void scaled_add(float (&total)[4], const float (&acc)[4], float lo, float hi) {
  const float2 a = __ffma2_rn(make_float2(acc[0], acc[1]), make_float2(lo, lo), make_float2(total[0], total[1]));
  const float2 b = __ffma2_rn(make_float2(acc[2], acc[3]), make_float2(hi, hi), make_float2(total[2], total[3]));
  total[0] = a.x;
  total[1] = a.y;
  total[2] = b.x;
  total[3] = b.y;
}

// Bytes of a staged mma column of `blocks` blocks of 128 columns: the odd 64
// keep the lanes' reads of different columns off one another's banks.
__host__ __device__ constexpr int x_row(int blocks) { return blocks * 256 + 64; }

// Stages blocks base .. base + n - 1: the tokens as mma columns `xrow` bytes
// apart from `xs`, the scales and zero points of ROWS rows as [group][row],
// four rows a thread where they are aligned for it.  MANY tokens divide the
// threads by a power of two not below the pieces of one; up to four are told
// apart by comparing.  Both save the division.
template <typename XT, int THREADS, int ROWS, int FLUSH, bool MANY>
__device__ __forceinline__ void stage(const Params& p, unsigned char* xs, int xrow, Group (*groups)[ROWS], int base, int n,
                                      int token0, int tokens, int row0) {
  constexpr int PARTS = sizeof(XT) == 4 ? 3 : 1;
  constexpr int NF = 128 / FLUSH;
  const int tid = threadIdx.x;
  const int log = MANY ? 36 - __clz(n - 1) : 0, all = MANY ? 1 << log : n * 16;
  for (int i = tid; i < tokens * all; i += THREADS) {  // 8 columns of a token
    const int token = MANY ? i >> log : (i >= all) + (i >= 2 * all) + (i >= 3 * all);
    const int piece = i - token * all, col = base * 128 + piece * 8;
    if (MANY && piece >= n * 16) continue;
    const XT* const from = static_cast<const XT*>(p.x) + static_cast<size_t>(token0 + token) * p.cols + col;
    unsigned char* const to = xs + token * PARTS * xrow + piece * 16;
    if (PARTS == 1 && p.fast_x && col + 8 <= p.cols) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from) : "memory");
      continue;
    }
    XT v[8];
    if (PARTS == 3 && p.fast_x && col + 8 <= p.cols) {
#pragma unroll
      for (int o = 0; o < 8; o += 16 / sizeof(XT)) {
        const uint4 some = *reinterpret_cast<const uint4*>(from + o);
        memcpy(v + o, &some, 16);
      }
    } else {
#pragma unroll
      for (int o = 0; o < 8; ++o) v[o] = col + o < p.cols ? from[o] : from_f32<XT>(0.f);
    }
    if constexpr (PARTS == 1) {
      memcpy(to, v, 16);
    } else {
      uint32_t out[3][4];
#pragma unroll
      for (int o = 0; o < 8; o += 2) {
        uint32_t a[3], b[3];
        parts_of(v[o], a);
        parts_of(v[o + 1], b);
#pragma unroll
        for (int q = 0; q < 3; ++q) out[q][o / 2] = a[q] | (b[q] << 16);
      }
#pragma unroll
      for (int q = 0; q < 3; ++q) *reinterpret_cast<uint4*>(to + q * xrow) = make_uint4(out[q][0], out[q][1], out[q][2], out[q][3]);
    }
  }
  // columns behind the last group are padding, whose sums of 0 are scaled by 0
  auto group_of = [&](int i) {
    if (FLUSH == 128 && p.long_groups) return __float2int_rz((static_cast<float>(base + i) + 0.5f) * p.inv_group);
    return min(base * NF + i, p.groups - 1);
  };
  auto in_use = [&](int i) { return FLUSH == 128 || base * NF + i < p.groups; };
  // With 64 registers a thread, four rows pay only for long groups (8192 x 8192
  // in groups of 128, one token: 10.8 us against 11.2; 16384 x 4096 in groups of
  // 64 with zero points: 13.4 against 13.0).
  if ((MANY || FLUSH == 128) && p.fast_groups) {
    const int at_row = tid % (ROWS / 4) * 4;
    const size_t row = static_cast<size_t>(min(row0 + at_row, p.rows - 4));
#pragma unroll(MANY ? 4 : 1)
    for (int i = tid / (ROWS / 4); i < n * NF; i += THREADS / (ROWS / 4)) {
      const size_t at = static_cast<size_t>(group_of(i)) * p.rows + row;
      const uint32_t z = p.zeros ? *reinterpret_cast<const uint32_t*>(p.zeros + at) : 0x08080808u;
      const float4 scale = load4_as_f32(p.scales, p.scale_dtype, at);
      const float f[4] = {scale.x, scale.y, scale.z, scale.w};
      uint32_t word[8];
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        word[2 * o] = in_use(i) ? __float_as_uint(f[o]) : 0u;
        word[2 * o + 1] = Half2<XT>::zero_pair(z >> (8 * o) & 0xFFu);
      }
      uint4* const to = reinterpret_cast<uint4*>(&groups[i][at_row]);
      to[0] = make_uint4(word[0], word[1], word[2], word[3]);
      to[1] = make_uint4(word[4], word[5], word[6], word[7]);
    }
  } else {
    const int at_row = tid & (ROWS - 1);
    const size_t row = static_cast<size_t>(min(row0 + at_row, p.rows - 1));
#pragma unroll 4
    for (int i = tid / ROWS; i < n * NF; i += THREADS / ROWS) {
      const size_t at = static_cast<size_t>(group_of(i)) * p.rows + row;
      Group put;
      put.scale = in_use(i) ? load_as_f32(p.scales, p.scale_dtype, at) : 0.f;
      put.zero = Half2<XT>::zero_pair(p.zeros ? p.zeros[at] : 8u);
      groups[i][at_row] = put;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
}

// Up to 8 mma columns.  FLUSH: matrix columns after which the sums are scaled
// (the group, or 128 of a longer one).  TILES: row tiles of a CTA, whose warps
// take every kWarps-th block of 128 columns.
template <typename XT, int FLUSH, int TILES>
__global__ void __launch_bounds__(kWarps * 32, 2) int4_matmul_kernel(const __grid_constant__ Params p) {
  constexpr int PARTS = sizeof(XT) == 4 ? 3 : 1;
  constexpr int NF = 128 / FLUSH;  // scalings of a block of 128 columns
  constexpr int AHEAD = 2;         // tiles in flight
  constexpr int ROWS = 16 * TILES;
  using H = Half2<XT>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int row0 = blockIdx.x * ROWS;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int token0 = blockIdx.z * p.pass_tokens;
  const int tokens = min(p.pass_tokens, p.tokens - token0);
  const int xrow = x_row(p.chunk);
  unsigned char* const xs = smem;                                                            // [tokens * PARTS][xrow]
  Group(*const groups)[ROWS] = reinterpret_cast<Group(*)[ROWS]>(smem + tokens * PARTS * xrow);  // [chunk * NF][ROWS]

  // a warp takes every kWarps-th block, and of it one row tile after the other
  const int tiles = min(TILES, (p.rows - row0 + 15) / 16);
  const uint4* const weights = reinterpret_cast<const uint4*>(p.packed) + static_cast<size_t>(row0 / 16) * p.blocks * 64 + lane;
  uint4 ring[AHEAD][2];
  auto fetch = [&](int slot, int block, int tile) {
    if (block >= p.blocks) return;
    const uint4* const from = weights + (static_cast<size_t>(tile < tiles ? tile : 0) * p.blocks + block) * 64;
    ring[slot][0] = load_once(from);
    ring[slot][1] = load_once(from + 32);
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) fetch(i, warp + i / TILES * kWarps, i % TILES);

  // mma columns behind the last token compute with it too; nobody reads their sums
  const unsigned char* const xcol = xs + min(g, tokens * PARTS - 1) * xrow + t * 16;

  uint32_t magic;  // kept in a register
  asm volatile("mov.b32 %0, %1;" : "=r"(magic) : "n"(H::kMagic));
  float total[TILES][4] = {};
  for (int base = 0; base < p.blocks; base += p.chunk) {
    const int n = min(p.chunk, p.blocks - base);
    if (base != 0) __syncthreads();
    stage<XT, kWarps * 32, ROWS, FLUSH, false>(p, xs, xrow, groups, base, n, token0, tokens, row0);

    constexpr int TURN = AHEAD > TILES ? AHEAD : TILES;  // tiles of one pass of the unrolled loop
    static_assert(TURN % TILES == 0 && TURN % AHEAD == 0, "whole blocks, whole rings");
#pragma unroll 1
    for (int b = warp; b < n; b += TURN / TILES * kWarps) {
#pragma unroll
      for (int i = 0; i < TURN; ++i) {
        const int at = b + i / TILES * kWarps, tile = i % TILES, slot = i % AHEAD;
        if (at >= n) break;
        const uint32_t lo[4] = {ring[slot][0].x, ring[slot][0].y, ring[slot][0].z, ring[slot][0].w};
        const uint32_t hi[4] = {ring[slot][1].x, ring[slot][1].y, ring[slot][1].z, ring[slot][1].w};
        float acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int f = j * 32 / FLUSH;
          const Group gl = groups[at * NF + f][tile * 16 + g], gh = groups[at * NF + f][tile * 16 + g + 8];
          uint32_t al[4], ah[4];
          H::words(lo[j], gl.zero, magic, al);
          H::words(hi[j], gh.zero, magic, ah);
          const uint4 x = *reinterpret_cast<const uint4*>(xcol + at * 256 + j * 64);
          if (j * 32 % FLUSH == 0) H::mma_first(acc, al[0], ah[0], al[1], ah[1], x.x, x.y);
          else H::mma(acc, al[0], ah[0], al[1], ah[1], x.x, x.y);
          H::mma(acc, al[2], ah[2], al[3], ah[3], x.z, x.w);
          if ((j + 1) * 32 % FLUSH == 0) {
            scaled_add(total[tile], acc, gl.scale, gh.scale);
          }
        }
        fetch(slot, base + at + (i % TILES + AHEAD) / TILES * kWarps, (i + AHEAD) % TILES);
      }
    }
  }

  // [warp][mma column][row], where the tokens were
  __syncthreads();
  float* const sums = reinterpret_cast<float*>(smem);
  constexpr int PITCH = ROWS + 4, PLANE = 8 * PITCH;
#pragma unroll
  for (int tile = 0; tile < TILES; ++tile) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int col = 2 * t + (c & 1);
      sums[warp * PLANE + col * PITCH + tile * 16 + g + (c >> 1) * 8] = part_sum<PARTS>(total[tile][c], col);
    }
  }
  __syncthreads();
  for (int i = tid; i < ROWS * tokens; i += kWarps * 32) {
    const int token = i / ROWS, at = i % ROWS;
    float v = 0.f;
#pragma unroll
    for (int part = PARTS - 1; part >= 0; --part) {
#pragma unroll 8
      for (int w = 0; w < kWarps; ++w) v += sums[w * PLANE + (token * PARTS + part) * PITCH + at];
    }
    if (row0 + at < p.rows)
      static_cast<XT*>(p.y)[static_cast<size_t>(token0 + token) * p.rows + row0 + at] = from_f32<XT>(v);
  }
}

constexpr int kRowWarps = 8;
constexpr int kRows = 16 * kRowWarps;  // rows of a CTA whose warps split the rows
constexpr int kChunk = 8;              // blocks of 128 columns that it stages at a time

// NT: tiles of 8 mma columns.  FLUSH: matrix columns after which the sums are
// scaled (the group, or 128 of a longer one).  128 registers for 9 and more mma
// columns: with 80 and a third CTA 16 tokens take 46 us, not 35.
template <typename XT, int NT, int FLUSH>
__global__ void __launch_bounds__(kRowWarps * 32, NT == 1 ? 4 : 2) int4_matmul_rows_kernel(const __grid_constant__ Params p) {
  constexpr int PARTS = sizeof(XT) == 4 ? 3 : 1;
  constexpr int NF = 128 / FLUSH;  // scalings of a block of 128 columns
  constexpr int AHEAD = 2;         // blocks in flight
  using H = Half2<XT>;
  extern __shared__ __align__(16) unsigned char smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int split = static_cast<int>(cluster.num_blocks()), part_k = static_cast<int>(cluster.block_rank());
  const int row0 = static_cast<int>(blockIdx.x) / split * kRows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int token0 = blockIdx.z * p.pass_tokens;
  const int tokens = min(p.pass_tokens, p.tokens - token0);
  unsigned char* const xs = smem;                                                               // [tokens * PARTS][x_row(kChunk)]
  Group(*const groups)[kRows] = reinterpret_cast<Group(*)[kRows]>(smem + tokens * PARTS * x_row(kChunk));  // [kChunk * NF][kRows]

  const int share = (p.blocks + split - 1) / split;
  const int first = min(part_k * share, p.blocks), last = min(first + share, p.blocks);
  // rows behind the last tile compute with it; nobody reads their sums
  const int tile = min(row0 / 16 + warp, (p.rows - 1) / 16);
  const uint4* weights = reinterpret_cast<const uint4*>(p.packed) + (static_cast<size_t>(tile) * p.blocks + first) * 64 + lane;

  uint4 ring[AHEAD][2];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    if (first + i < last) {
      ring[i][0] = load_once(weights + i * 64);
      ring[i][1] = load_once(weights + i * 64 + 32);
    }
  }

  // mma columns behind the last token compute with it too
  const unsigned char* xcol[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) xcol[nt] = xs + min(nt * 8 + g, tokens * PARTS - 1) * x_row(kChunk) + t * 16;
  const Group* const g_lo = &groups[0][warp * 16 + g];

  uint32_t magic;  // kept in a register
  asm volatile("mov.b32 %0, %1;" : "=r"(magic) : "n"(H::kMagic));
  float total[NT][4] = {};
  for (int base = first; base < last; base += kChunk) {
    const int n = min(kChunk, last - base);
    if (base != first) __syncthreads();
    stage<XT, kRowWarps * 32, kRows, FLUSH, true>(p, xs, x_row(kChunk), groups, base, n, token0, tokens, row0);

#pragma unroll 1
    for (int b = 0; b < n; b += AHEAD) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (b + i < n) {
          const uint32_t lo[4] = {ring[i][0].x, ring[i][0].y, ring[i][0].z, ring[i][0].w};
          const uint32_t hi[4] = {ring[i][1].x, ring[i][1].y, ring[i][1].z, ring[i][1].w};
          float acc[NT][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int f = j * 32 / FLUSH;
            const Group gl = g_lo[((b + i) * NF + f) * kRows], gh = g_lo[((b + i) * NF + f) * kRows + 8];
            uint32_t al[4], ah[4];
            H::words(lo[j], gl.zero, magic, al);
            H::words(hi[j], gh.zero, magic, ah);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4 x = *reinterpret_cast<const uint4*>(xcol[nt] + (b + i) * 256 + j * 64);
              if (j * 32 % FLUSH == 0) H::mma_first(acc[nt], al[0], ah[0], al[1], ah[1], x.x, x.y);
              else H::mma(acc[nt], al[0], ah[0], al[1], ah[1], x.x, x.y);
              H::mma(acc[nt], al[2], ah[2], al[3], ah[3], x.z, x.w);
            }
            if ((j + 1) * 32 % FLUSH == 0) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) scaled_add(total[nt], acc[nt], gl.scale, gh.scale);
            }
          }
          if (base + b + i + AHEAD < last) {
            ring[i][0] = load_once(weights + (i + AHEAD) * 64);
            ring[i][1] = load_once(weights + (i + AHEAD) * 64 + 32);
          }
        }
      }
      weights += AHEAD * 64;
    }
  }

  // [mma column][row], where the tokens were
  __syncthreads();
  float* const sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int col = nt * 8 + 2 * t + (c & 1), at = warp * 16 + g + (c >> 1) * 8;
      const float sum = part_sum<PARTS>(total[nt][c], col);  // (not within the branch: 4.7 us a call for 4.5)
      if (col < tokens * PARTS) sums[col * (kRows + 4) + at] = sum;
    }
  }
  if (split > 1) cluster.sync();
  else __syncthreads();
  const int rows_each = kRows / split;
  for (int i = tid; i < rows_each * tokens; i += kRowWarps * 32) {
    const int token = i / rows_each, at = part_k * rows_each + i - token * rows_each;
    float v = 0.f;
    for (int q = 0; q < split; ++q) {
      const float* const from = split == 1 ? sums : cluster.map_shared_rank(sums, q);
#pragma unroll
      for (int part = PARTS - 1; part >= 0; --part) v += from[(token * PARTS + part) * (kRows + 4) + at];
    }
    if (row0 + at < p.rows)
      static_cast<XT*>(p.y)[static_cast<size_t>(token0 + token) * p.rows + row0 + at] = from_f32<XT>(v);
  }
  if (split > 1) cluster.sync();  // nobody leaves while its shared memory is read
}

template <typename XT, int FLUSH, int TILES>
bcjr_status launch(Params p, int passes, cudaStream_t s) {
  constexpr int PARTS = sizeof(XT) == 4 ? 3 : 1;
  constexpr int NF = 128 / FLUSH, ROWS = 16 * TILES;
  const int columns = (p.tokens < p.pass_tokens ? p.tokens : p.pass_tokens) * PARTS;
  // as many blocks at a time as leave room for a second CTA, an even number for
  // each warp (its ring of two starts anew with each chunk)
  const int each = columns * 256 + NF * ROWS * static_cast<int>(sizeof(Group));
  static_assert(32 * (8 * 256 + NF * ROWS * sizeof(Group)) + 8 * 64 <= 100 * 1024, "two blocks a warp fit");
  int chunk = (100 * 1024 - columns * 64) / each / (2 * kWarps) * (2 * kWarps);
  if (chunk > p.blocks) chunk = p.blocks;
  p.chunk = chunk;
  const int staged = columns * x_row(chunk) + chunk * NF * ROWS * static_cast<int>(sizeof(Group));
  constexpr int sums = kWarps * 8 * (ROWS + 4) * static_cast<int>(sizeof(float));
  const int bytes = staged > sums ? staged : sums;
  auto* const kernel = int4_matmul_kernel<XT, FLUSH, TILES>;
  static PerDevice done;
  if (!allow_shared(reinterpret_cast<const void*>(kernel), done)) return BCJR_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>((p.rows + ROWS - 1) / ROWS), 1, static_cast<unsigned>(passes));
  kernel<<<grid, kWarps * 32, static_cast<size_t>(bytes), s>>>(p);
  return launched();
}

template <typename XT, int NT, int FLUSH>
bcjr_status launch_rows(const Params& p, int passes, int sms, cudaStream_t s) {
  constexpr int PARTS = sizeof(XT) == 4 ? 3 : 1;
  const int columns = (p.tokens < p.pass_tokens ? p.tokens : p.pass_tokens) * PARTS;
  const int staged = columns * x_row(kChunk) + kChunk * (128 / FLUSH) * kRows * static_cast<int>(sizeof(Group));
  static_assert(x_row(kChunk) >= (kRows + 4) * 4, "the sums fit where the tokens were");
  // Columns are split over the CTAs of a cluster while the rows alone do not
  // give every multiprocessor its CTAs: two for 8 columns, which wait for
  // weights, one for more, which the matrix instruction holds up (8192 x 8192, 32
  // tokens: 24.1 us with one, 28.0 with two; 8 tokens: 14.9 and 12.8).
  const long long tiles = (p.rows + kRows - 1) / kRows;
  int split = 1;
  while (split < 8 && tiles * passes * split < (NT == 1 ? 2 : 1) * sms && p.blocks >= 2 * split) split *= 2;
  auto* const kernel = int4_matmul_rows_kernel<XT, NT, FLUSH>;
  static PerDevice done;
  if (!allow_shared(reinterpret_cast<const void*>(kernel), done)) return BCJR_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * split), 1, static_cast<unsigned>(passes));
  cfg.blockDim = dim3(kRowWarps * 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(staged);
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(split);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return BCJR_ERR_CUDA;
  }
  return BCJR_OK;
}

template <typename XT, int FLUSH>
bcjr_status launch_tokens(Params p, int sms, cudaStream_t s) {
  constexpr int PARTS = sizeof(XT) == 4 ? 3 : 1;
  const int nt = p.tokens * PARTS <= 8 ? 1 : p.tokens * PARTS <= 16 ? 2 : 4;
  p.pass_tokens = nt * 8 / PARTS;
  const int passes = (p.tokens + p.pass_tokens - 1) / p.pass_tokens;
  // With more than four columns the staged tokens cost the CTAs of few rows more
  // than their warps save by sharing no sums (8192 x 8192, 8 bf16 tokens: 16.1 us
  // against 12.8; 3 tokens: 12.6 against 12.5; 1 token of 2048 x 8192: 4.5 against 6.4).
  if (nt == 1 && p.tokens * PARTS > 4) return launch_rows<XT, 1, FLUSH>(p, passes, sms, s);
  if (nt == 2) return launch_rows<XT, 2, FLUSH>(p, passes, sms, s);
  if (nt == 4) return launch_rows<XT, 4, FLUSH>(p, passes, sms, s);
  // two row tiles a CTA once that leaves every multiprocessor more than one
  return static_cast<long long>(p.rows / 32) * 2 >= sms * 3 ? launch<XT, FLUSH, 2>(p, passes, s) : launch<XT, FLUSH, 1>(p, passes, s);
}

template <typename XT>
bcjr_status launch_groups(const Params& p, int group, int sms, cudaStream_t s) {
  if (group == 32) return launch_tokens<XT, 32>(p, sms, s);
  if (group == 64) return launch_tokens<XT, 64>(p, sms, s);
  return launch_tokens<XT, 128>(p, sms, s);
}

}  // namespace
}  // namespace bcjr
