// int4_quantize.cu -- 4-bit group quantisation into tensor-core tiles (bcjr_int4_quantize).
//
// A warp takes two rows of a 128-column block at a time: lane l holds columns
// 8 (l mod 16) .. + 7 of row l / 16, which are the eight codes of one 32-bit
// word of the packed tile, so a lane reads 16 or 32 contiguous bytes and
// writes one word, two blocks' loads ahead of the work on them.  Groups of 32,
// 64 and 128 columns are 4, 8 and 16 neighbouring lanes, their extremes a few
// shuffles.  Reading w bounds the call for float32 (4.5 B a weight moved in all):
// 2048 x 8192 in groups of 128 takes 13.7 us from memory (5.5 TB/s; whole rows,
// read twice, 18.3).  16-bit types (2.5 B a weight) take 16.2 us, because a lane
// has eight columns whatever their type: half the bytes on the way for the same
// shuffles, reciprocals and codes.  Persistent CTAs with the next blocks' loads on
// the way were slower.
#include <cmath>
#include <cstring>

#include "layer_util.cuh"

namespace {

using namespace bcjr;

constexpr int kWarps = 8;  // two rows each: a tile of 16 rows

struct Params {
  const void* w;
  int rows, cols, blocks;   // blocks of 128 columns
  int group_blocks;         // of a group; 0: groups shorter than a block
  int lanes_log2;           // of the lanes of a group within its block (4, 8 or 16)
  int groups;
  unsigned units;           // CTAs of a tile's columns
  uint8_t* packed;
  void* scales;
  int scale_dtype;
  uint8_t* zeros;
};

template <typename T>
__device__ __forceinline__ void load8(const T* row, int col, int cols, bool fast, float (&v)[8]) {
  if (fast && col + 8 <= cols) {
    if constexpr (sizeof(T) == 4) {
      const float4 a = *reinterpret_cast<const float4*>(row + col), b = *reinterpret_cast<const float4*>(row + col + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(row + col);
      T t[8];
      memcpy(t, &a, sizeof a);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = to_f32(t[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col + i < cols ? to_f32(row[col + i]) : 0.f;
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN is not lost, as fmaxf would
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Extremes of a group so far, with zero among the values: the largest and the
// largest negated value, or (no zero points) the largest magnitude alone.
template <bool ZERO>
struct Extremes {
  float hi = 0.f, minus_lo = 0.f;
  __device__ __forceinline__ void add(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi = max_nan(hi, ZERO ? v[i] : fabsf(v[i]));
      if (ZERO) minus_lo = max_nan(minus_lo, -v[i]);
    }
  }
  __device__ __forceinline__ void over(int lanes_log2) {
#pragma unroll
    for (int step = 0; step < 4; ++step) {
      if (step >= lanes_log2) break;
      const int d = 1 << step;
      hi = max_nan(hi, __shfl_xor_sync(~0u, hi, d));
      if (ZERO) minus_lo = max_nan(minus_lo, __shfl_xor_sync(~0u, minus_lo, d));
    }
  }
};

struct Code {
  float inv;
  int zero;
  bool tiny;  // inv is of 2^64 times the scale
};

constexpr float kUp = 0x1p64f;

// The group's scale (rounded to its type and stored by one lane) and how to
// take codes with it.  Multiplying by the reciprocal instead of dividing by
// the scale differs from the quotient's rounding only next to a tie.  Scales up
// to 2^-128, whose reciprocals overflow, and weights are taken 2^64 times as large.
template <bool ZERO, bool HALF>
__device__ __forceinline__ Code group_code(const Params& p, const Extremes<ZERO>& e, int row, int group, bool writes) {
  float s = ZERO ? __fmul_rn(__fadd_rn(e.hi, e.minus_lo), 1.f / 15.f) : __fmul_rn(e.hi, 1.f / 7.f);
  if (HALF) s = __half2float(__float2half_rn(s));
  else if (p.scale_dtype == BCJR_BF16) s = __bfloat162float(__float2bfloat16_rn(s));
  Code c;
  float minus_lo = e.minus_lo;
  c.inv = s > 0.f ? __frcp_rn(s) : 0.f;
  c.tiny = !HALF && c.inv > 3.402823466e38f;
  if (c.tiny) {
    c.inv = __frcp_rn(__fmul_rn(s, kUp));
    minus_lo = __fmul_rn(minus_lo, kUp);
  }
  c.zero = ZERO ? static_cast<int>(fminf(fmaxf(rintf(__fmul_rn(minus_lo, c.inv)), 0.f), 15.f)) : 8;
  if (writes && row < p.rows) {
    const size_t i = static_cast<size_t>(group) * p.rows + row;
    store_from_f32(p.scales, HALF ? BCJR_F16 : p.scale_dtype, i, s);
    if (ZERO) p.zeros[i] = static_cast<uint8_t>(c.zero);
  }
  return c;
}

// Eight columns of a row as the word of the tile that holds them.  Adding
// 1.5 2^23 rounds to the nearest integer, ties to even, and leaves it in the
// low bits (together with an even zero point; an odd one would turn the ties).
// What can leave 0..15: with zero points, both ends of a range may round up,
// which makes 16; a subnormal half scale, or one of the tiny ones, may be half of
// what it stands for, so either end (LOOSE).  0 times an infinity, a NaN, takes
// some code of a group whose scale says so.
template <bool ZERO, bool LOOSE>
__device__ __forceinline__ void put_codes(const Params& p, const float (&v)[8], const Code& c, int tile, int block,
                                         int row16, int l16, bool row_ok, int col) {
  uint32_t word = 0;
#pragma unroll
  for (int o = 0; o < 8; ++o) {
    const float t = __fmul_rn(v[o], c.inv);
    uint32_t q;
    if (ZERO || LOOSE) {
      int i = __float_as_int(__fadd_rn(t, 12582912.f)) - 0x4B400000 + c.zero;
      i = min(i, 15);
      if (LOOSE) i = max(i, 0);
      q = static_cast<uint32_t>(i);
    } else {
      q = __float_as_uint(__fadd_rn(t, 12582920.f));
    }
    const int at = 4 * (o >> 1) + 16 * (o & 1);
    word |= (q << at) & (15u << at);
  }
  if (!row_ok) word = 0x88888888u;
  else if (col + 8 > p.cols) {
#pragma unroll
    for (int o = 0; o < 8; ++o) {
      const int at = 4 * (o >> 1) + 16 * (o & 1);
      if (col + o >= p.cols) word = (word & ~(15u << at)) | (8u << at);
    }
  }
  const size_t at = (static_cast<size_t>(tile) * p.blocks + block) * 1024 + (row16 >> 3) * 512 + (row16 & 7) * 64 +
                    (l16 & 3) * 16 + (l16 >> 2) * 4;
  *reinterpret_cast<uint32_t*>(p.packed + at) = word;
}

template <bool ZERO, bool HALF>
__device__ __forceinline__ void put_word(const Params& p, float (&v)[8], const Code& c, int tile, int block, int row16, int l16,
                                         bool row_ok, int col) {
  if (!HALF && c.tiny) {
#pragma unroll
    for (int o = 0; o < 8; ++o) v[o] = __fmul_rn(v[o], kUp);
    put_codes<ZERO, true>(p, v, c, tile, block, row16, l16, row_ok, col);
  } else {
    put_codes<ZERO, HALF>(p, v, c, tile, block, row16, l16, row_ok, col);
  }
}

// Blocks that a thread loads before it works on them.  Measured when it was chosen
// (2048 x 8192 float32): two 15.6 us, one 19.2, four 16.3 (fewer warps), eight 24.1.
constexpr int kAtOnce = 2;

template <typename T, bool ZERO, bool HALF>
__global__ void __launch_bounds__(kWarps * 32) int4_quantize_kernel(const __grid_constant__ Params p) {
  const int lane = threadIdx.x & 31, l16 = lane & 15;
  const int row16 = (threadIdx.x >> 5) * 2 + (lane >> 4);
  const int tile = static_cast<int>(blockIdx.x / p.units);
  const int row = tile * 16 + row16;
  const bool ok = row < p.rows;
  const T* const src = static_cast<const T*>(p.w) + static_cast<size_t>(ok ? row : p.rows - 1) * p.cols;
  const bool fast = (p.cols * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(p.w) & 15) == 0;
  const int b0 = static_cast<int>(blockIdx.x % p.units) * kAtOnce;
  float v[kAtOnce][8];
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i) load8(src, (b0 + i) * 128 + l16 * 8, p.cols, fast, v[i]);
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i) {
    const int block = b0 + i, col = block * 128 + l16 * 8;
    if (block >= p.blocks) break;
    Extremes<ZERO> e;
    e.add(v[i]);
    e.over(p.lanes_log2);
    const int group = (block << (4 - p.lanes_log2)) + (l16 >> p.lanes_log2);
    const Code c = group_code<ZERO, HALF>(p, e, row, group, (l16 & ((1 << p.lanes_log2) - 1)) == 0 && group < p.groups);
    put_word<ZERO, HALF>(p, v[i], c, tile, block, row16, l16, ok, col);
  }
}

// Groups longer than a block: a CTA takes two rows of a group, its warps every
// kWarps-th block; the extremes meet in shared memory, and the second pass
// reads the blocks from the cache.
template <typename T, bool ZERO, bool HALF>
__global__ void __launch_bounds__(kWarps * 32) int4_quantize_long_kernel(const __grid_constant__ Params p) {
  __shared__ float hi[kWarps][2], minus_lo[kWarps][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l16 = lane & 15, half = lane >> 4;
  const int pair = static_cast<int>(blockIdx.x / p.units), tile = pair >> 3, row16 = (pair & 7) * 2 + half;
  const int row = tile * 16 + row16;
  const bool ok = row < p.rows;
  const T* const src = static_cast<const T*>(p.w) + static_cast<size_t>(ok ? row : p.rows - 1) * p.cols;
  const bool fast = (p.cols * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(p.w) & 15) == 0;
  const int group = static_cast<int>(blockIdx.x % p.units);
  const int b0 = group * p.group_blocks, b1 = min(b0 + p.group_blocks, p.blocks);
  float v[8];
  Extremes<ZERO> e;
#pragma unroll 4
  for (int block = b0 + warp; block < b1; block += kWarps) {
    load8(src, block * 128 + l16 * 8, p.cols, fast, v);
    e.add(v);
  }
  e.over(4);
  if (l16 == 0) {
    hi[warp][half] = e.hi;
    minus_lo[warp][half] = e.minus_lo;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    e.hi = max_nan(e.hi, hi[w][half]);
    if (ZERO) e.minus_lo = max_nan(e.minus_lo, minus_lo[w][half]);
  }
  const Code c = group_code<ZERO, HALF>(p, e, row, group, warp == 0 && l16 == 0);
#pragma unroll 4
  for (int block = b0 + warp; block < b1; block += kWarps) {
    const int col = block * 128 + l16 * 8;
    load8(src, col, p.cols, fast, v);
    put_word<ZERO, HALF>(p, v, c, tile, block, row16, l16, ok, col);
  }
}

template <typename T, bool ZERO, bool HALF>
void launch(const Params& p, unsigned grid, cudaStream_t s) {
  if (p.group_blocks) int4_quantize_long_kernel<T, ZERO, HALF><<<grid, kWarps * 32, 0, s>>>(p);
  else int4_quantize_kernel<T, ZERO, HALF><<<grid, kWarps * 32, 0, s>>>(p);
}

template <typename T>
void launch_kind(const Params& p, unsigned grid, cudaStream_t s) {
  const bool half = p.scale_dtype == BCJR_F16;
  if (p.zeros) half ? launch<T, true, true>(p, grid, s) : launch<T, true, false>(p, grid, s);
  else half ? launch<T, false, true>(p, grid, s) : launch<T, false, false>(p, grid, s);
}

}  // namespace

extern "C" bcjr_status bcjr_int4_quantize(const void* w, int w_dtype, int rows, int cols, int group_size,
                                          void* packed, void* scales, int scale_dtype, uint8_t* zeros,
                                          bcjr_stream_t stream) {
  if (!dtype_ok(w_dtype) || !dtype_ok(scale_dtype) || rows < 0 || cols < 1 || group_size < 0) return BCJR_ERR_INVALID_ARG;
  if (group_size % 128 != 0 && group_size != 32 && group_size != 64) return BCJR_ERR_UNSUPPORTED;
  // columns as in the product
  if (rows > (1 << 30) || cols > (1 << 27)) return BCJR_ERR_UNSUPPORTED;
  if (rows == 0) return BCJR_OK;
  if (!w || !packed || !scales || !ptr_aligned(w, dtype_size(w_dtype)) || !ptr_aligned(packed, 16) ||
      !ptr_aligned(scales, dtype_size(scale_dtype)))
    return BCJR_ERR_INVALID_ARG;
  Params p = {};
  p.w = w;
  p.rows = rows;
  p.cols = cols;
  p.blocks = (cols + 127) / 128;
  p.packed = static_cast<uint8_t*>(packed);
  p.scales = scales;
  p.scale_dtype = scale_dtype;
  p.zeros = zeros;
  if (group_size == 0 || group_size >= cols) {
    // one group: shorter than a block only where its columns are
    p.group_blocks = p.blocks;
    p.groups = 1;
  } else if (group_size <= 128) {
    p.lanes_log2 = group_size == 32 ? 2 : group_size == 64 ? 3 : 4;
    p.groups = (cols + group_size - 1) / group_size;
  } else {
    p.group_blocks = group_size / 128;
    p.groups = (cols + group_size - 1) / group_size;
  }
  p.units = static_cast<unsigned>(p.group_blocks ? p.groups : (p.blocks + kAtOnce - 1) / kAtOnce);
  const long long grid = static_cast<long long>((rows + 15) / 16) * (p.group_blocks ? 8 : 1) * p.units;
  if (grid > 0x7FFFFFFFll) return BCJR_ERR_UNSUPPORTED;
  cudaStream_t s = as_stream(stream);
  if (w_dtype == BCJR_F32) launch_kind<float>(p, static_cast<unsigned>(grid), s);
  else if (w_dtype == BCJR_F16) launch_kind<__half>(p, static_cast<unsigned>(grid), s);
  else launch_kind<__nv_bfloat16>(p, static_cast<unsigned>(grid), s);
  return launched();
}
