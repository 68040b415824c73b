// int4_quantize.cu -- 4-bit group quantisation into tensor-core tiles (bcjr_int4_quantize).
//
// A warp takes two rows of a 128-column block at a time: lane l holds columns
// 8 (l mod 16) .. + 7 of row l / 16, which are the eight codes of one 32-bit
// word of the packed tile, so a lane reads 16 or 32 contiguous bytes and
// writes one word.  Groups of 32, 64 and 128 columns are 4, 8 and 16
// neighbouring lanes, their extremes a few shuffles.  Longer groups take two
// passes over their blocks, the second from the cache.  Reading w bounds the
// call (4.5 B a weight for float32 moved in all, 2.5 B for 16-bit types).
#include <cmath>

#include "layer_util.cuh"

namespace {

using namespace bcjr;

constexpr int kWarps = 8;  // two rows each: a tile of 16 rows

struct Params {
  const void* w;
  int rows, cols, blocks;   // blocks of 128 columns
  int group_blocks;         // of a group; 0: groups shorter than a block
  int lanes;                // lanes of a group within its block (4, 8 or 16)
  int groups;
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

// Extremes of a group so far.  Zero is always among the values (lo <= 0 <= hi);
// a NaN must not be lost, which fminf and fmaxf would do, so it is tracked.
struct Extremes {
  float lo = 0.f, hi = 0.f;
  bool nan = false;
  __device__ void add(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, v[i]);
      hi = fmaxf(hi, v[i]);
      nan |= v[i] != v[i];
    }
  }
  __device__ void over(int lanes) {
    for (int d = 1; d < lanes; d <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(~0u, lo, d));
      hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, d));
      nan |= __shfl_xor_sync(~0u, static_cast<int>(nan), d) != 0;
    }
  }
};

struct Code {
  float inv, zero;
};

// The group's scale (rounded to its type and stored by one lane) and how to
// take codes with it.  Multiplying by the reciprocal instead of dividing by
// the scale differs from the quotient's rounding only next to a tie.
__device__ __forceinline__ Code group_code(const Params& p, const Extremes& e, int row, int group, bool writes) {
  const float range = p.zeros ? __fsub_rn(e.hi, e.lo) : fmaxf(e.hi, -e.lo);
  float s = e.nan ? NAN : __fmul_rn(range, p.zeros ? 1.f / 15.f : 1.f / 7.f);
  if (p.scale_dtype == BCJR_F16) s = __half2float(__float2half_rn(s));
  else if (p.scale_dtype == BCJR_BF16) s = __bfloat162float(__float2bfloat16_rn(s));
  Code c;
  c.inv = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
  c.zero = p.zeros ? fminf(fmaxf(rintf(__fmul_rn(-e.lo, c.inv)), 0.f), 15.f) : 8.f;
  if (writes && row < p.rows) {
    const size_t i = static_cast<size_t>(group) * p.rows + row;
    store_from_f32(p.scales, p.scale_dtype, i, s);
    if (p.zeros) p.zeros[i] = static_cast<uint8_t>(c.zero);
  }
  return c;
}

// Eight columns of a row as the word of the tile that holds them.
__device__ __forceinline__ void put_word(const Params& p, const float (&v)[8], const Code& c, int tile, int block,
                                         int row16, int l16, bool row_ok, int col) {
  uint32_t word = 0;
#pragma unroll
  for (int o = 0; o < 8; ++o) {
    uint32_t q = 8;
    if (row_ok && col + o < p.cols) {
      const float f = __fadd_rn(rintf(__fmul_rn(v[o], c.inv)), c.zero);
      q = static_cast<uint32_t>(fminf(fmaxf(f, 0.f), 15.f));  // a NaN gives 0
    }
    word |= q << (4 * (o >> 1) + 16 * (o & 1));
  }
  const size_t at = (static_cast<size_t>(tile) * p.blocks + block) * 1024 + (row16 >> 3) * 512 + (row16 & 7) * 64 +
                    (l16 & 3) * 16 + (l16 >> 2) * 4;
  *reinterpret_cast<uint32_t*>(p.packed + at) = word;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) int4_quantize_kernel(const __grid_constant__ Params p) {
  const int lane = threadIdx.x & 31, l16 = lane & 15;
  const int row16 = (threadIdx.x >> 5) * 2 + (lane >> 4);
  const int tile = blockIdx.y;
  const int row = tile * 16 + row16;
  const bool ok = row < p.rows;
  const T* const src = static_cast<const T*>(p.w) + static_cast<size_t>(ok ? row : p.rows - 1) * p.cols;
  const bool fast = (p.cols * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(p.w) & 15) == 0;
  float v[8];
  if (p.group_blocks == 0) {
    for (int block = blockIdx.x; block < p.blocks; block += gridDim.x) {
      const int col = block * 128 + l16 * 8;
      load8(src, col, p.cols, fast, v);
      Extremes e;
      e.add(v);
      e.over(p.lanes);
      const int group = block * (16 / p.lanes) + l16 / p.lanes;
      const Code c = group_code(p, e, row, group, l16 % p.lanes == 0 && group < p.groups);
      put_word(p, v, c, tile, block, row16, l16, ok, col);
    }
  } else {
    for (int group = blockIdx.x; group < p.groups; group += gridDim.x) {
      const int b0 = group * p.group_blocks, b1 = min(b0 + p.group_blocks, p.blocks);
      Extremes e;
      for (int block = b0; block < b1; ++block) {
        load8(src, block * 128 + l16 * 8, p.cols, fast, v);
        e.add(v);
      }
      e.over(16);
      const Code c = group_code(p, e, row, group, l16 == 0);
      for (int block = b0; block < b1; ++block) {
        const int col = block * 128 + l16 * 8;
        load8(src, col, p.cols, fast, v);
        put_word(p, v, c, tile, block, row16, l16, ok, col);
      }
    }
  }
}

}  // namespace

extern "C" bcjr_status bcjr_int4_quantize(const void* w, int w_dtype, int rows, int cols, int group_size,
                                          void* packed, void* scales, int scale_dtype, uint8_t* zeros,
                                          bcjr_stream_t stream) {
  if (!dtype_ok(w_dtype) || !dtype_ok(scale_dtype) || rows < 0 || cols < 1 || group_size < 0) return BCJR_ERR_INVALID_ARG;
  if (group_size % 128 != 0 && group_size != 32 && group_size != 64) return BCJR_ERR_UNSUPPORTED;
  // tiles are the second grid dimension; columns as in the product
  if (rows > 16 * 65535 || cols > (1 << 27)) return BCJR_ERR_UNSUPPORTED;
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
    p.lanes = group_size / 8;
    p.groups = (cols + group_size - 1) / group_size;
  } else {
    p.group_blocks = group_size / 128;
    p.groups = (cols + group_size - 1) / group_size;
  }
  const int units = p.group_blocks ? p.groups : p.blocks;
  const dim3 grid(static_cast<unsigned>(units), static_cast<unsigned>((rows + 15) / 16));
  cudaStream_t s = as_stream(stream);
  if (w_dtype == BCJR_F32) int4_quantize_kernel<float><<<grid, kWarps * 32, 0, s>>>(p);
  else if (w_dtype == BCJR_F16) int4_quantize_kernel<__half><<<grid, kWarps * 32, 0, s>>>(p);
  else int4_quantize_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, s>>>(p);
  return launched();
}
