// int4_matmul.cu -- a few tokens times 4-bit weights (bcjr_int4_matmul).
//
// Weights are the 16-row operand of mma.m16n8k16 and tokens its 8 columns, so
// eight tokens cost what one does.  A lane's 16-byte load of a packed tile
// holds, word by word, the codes of its fragment positions in columns 32 j +
// 8 t .. + 7: (word >> 4 i) & 0x000F000F is the fragment register of columns
// 8 t + 2 i and + 1, which or-ed with the bits of 128 (bf16; 1024 in half)
// is exactly 128 + q, and one packed subtraction gives q - zero, exactly.
// Group sums stay in float32 and are scaled in float32, so the only rounding
// is that of the sums.  float32 tokens are cut into three bf16 parts of 8
// bits (exact), which take three of the eight columns.
//
// A CTA owns 16 rows; its warps, and the CTAs of its cluster, split the
// columns and add their sums through (distributed) shared memory in a fixed
// order.  Reading the packed weights bounds the call.
#include <cmath>
#include <cooperative_groups.h>

#include "layer_util.cuh"

namespace cg = cooperative_groups;

namespace {

using namespace bcjr;

struct Params {
  const void* x;
  const uint8_t* packed;
  const void* scales;
  const uint8_t* zeros;
  void* y;
  int tokens, rows, cols, blocks;
  int group;        // columns of a group
  int scale_dtype;
  int pass_tokens;  // tokens of a pass (grid z)
  bool fast_x;      // x may be read 16 bytes at a time
};

template <typename T>
struct Half2;  // the packed 16-bit type that multiplies T

template <>
struct Half2<__half> {
  static constexpr uint32_t kMagic = 0x64006400u;  // 1024 in either half
  static __device__ uint32_t zero_pair(uint32_t z) { return kMagic | z | (z << 16); }
  static __device__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

template <>
struct Half2<__nv_bfloat16> {
  static constexpr uint32_t kMagic = 0x43004300u;  // 128 in either half
  static __device__ uint32_t zero_pair(uint32_t z) { return kMagic | z | (z << 16); }
  static __device__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

template <>
struct Half2<float> : Half2<__nv_bfloat16> {};

// Part `part` (0, 1, 2) of a float as a bf16's bits: the upper 8 bits of its
// mantissa, the next 8, the last 8, each cut off exactly.  What is not finite
// is its own first part, and the others are 0, so that an infinity stays one.
__device__ __forceinline__ uint32_t part_of(float v, int part) {
  const uint32_t top = __float_as_uint(v) & 0xFFFF0000u;
  if (part == 0) return (v == v ? top : 0x7FC00000u) >> 16;
  if (!(fabsf(v) < INFINITY)) return 0u;
  const float rest = v - __uint_as_float(top);
  const uint32_t mid = __float_as_uint(rest) & 0xFFFF0000u;
  if (part == 1) return mid >> 16;
  return __float_as_uint(rest - __uint_as_float(mid)) >> 16;
}

// The eight columns col .. col + 7 of one mma column (a token, or a part of
// one) as four packed pairs.
template <typename XT>
__device__ __forceinline__ void load_x(const Params& p, const XT* row, int part, int col, uint32_t (&v)[4]) {
  if constexpr (sizeof(XT) == 2) {
    if (p.fast_x && col + 8 <= p.cols) {
      const uint4 a = *reinterpret_cast<const uint4*>(row + col);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else {
      const uint16_t* const raw = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = col + 2 * i < p.cols ? raw[col + 2 * i] : 0u;
        const uint32_t hi = col + 2 * i + 1 < p.cols ? raw[col + 2 * i + 1] : 0u;
        v[i] = lo | (hi << 16);
      }
    }
  } else {
    float f[8];
    if (p.fast_x && col + 8 <= p.cols) {
      const float4 a = *reinterpret_cast<const float4*>(row + col), b = *reinterpret_cast<const float4*>(row + col + 4);
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = col + i < p.cols ? row[col + i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = part_of(f[2 * i], part) | (part_of(f[2 * i + 1], part) << 16);
  }
}

constexpr int kWarps = 8;

// NT: tiles of 8 mma columns.  FLUSH: columns after which the sums are scaled
// (the group, or 128 of a longer one).
template <typename XT, int NT, int FLUSH>
__global__ void __launch_bounds__(kWarps * 32) int4_matmul_kernel(const __grid_constant__ Params p) {
  constexpr int PARTS = sizeof(XT) == 4 ? 3 : 1;
  constexpr int NF = 128 / FLUSH;             // scalings of a block of 128 columns
  constexpr int AHEAD = FLUSH == 128 ? 4 : 2; // blocks in flight
  using H = Half2<XT>;
  cg::cluster_group cluster = cg::this_cluster();
  const int split = static_cast<int>(cluster.num_blocks()), part_k = static_cast<int>(cluster.block_rank());
  const int tile = static_cast<int>(blockIdx.x) / split;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int token0 = blockIdx.z * p.pass_tokens;
  const int tokens = min(p.pass_tokens, p.tokens - token0);
  const int r_lo = min(tile * 16 + g, p.rows - 1), r_hi = min(tile * 16 + g + 8, p.rows - 1);

  const XT* xrow[NT];
  int xpart[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int n = nt * 8 + g, token = n / PARTS;
    xrow[nt] = token < tokens ? static_cast<const XT*>(p.x) + static_cast<size_t>(token0 + token) * p.cols : nullptr;
    xpart[nt] = n % PARTS;
  }

  float total[NT][4] = {};
  const uint4* const weights = reinterpret_cast<const uint4*>(p.packed) + static_cast<size_t>(tile) * p.blocks * 64 + lane;
  const int stride = kWarps * split;
  uint4 ring[AHEAD][2];
  float scale[AHEAD][NF][2];
  uint32_t zero[AHEAD][NF][2];
  auto fetch = [&](int slot, int block) {
    if (block >= p.blocks) return;
    ring[slot][0] = weights[static_cast<size_t>(block) * 64];
    ring[slot][1] = weights[static_cast<size_t>(block) * 64 + 32];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      // columns behind the last group are padding: the last group's scale will do
      const size_t at = static_cast<size_t>(min(block * 128 + f * FLUSH, p.cols - 1) / p.group) * p.rows;
      scale[slot][f][0] = load_as_f32(p.scales, p.scale_dtype, at + r_lo);
      scale[slot][f][1] = load_as_f32(p.scales, p.scale_dtype, at + r_hi);
      zero[slot][f][0] = p.zeros ? p.zeros[at + r_lo] : 8u;
      zero[slot][f][1] = p.zeros ? p.zeros[at + r_hi] : 8u;
    }
  };
  const int first = part_k * kWarps + warp;
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) fetch(i, first + i * stride);
  for (int base = first; base < p.blocks; base += AHEAD * stride) {
#pragma unroll
    for (int slot = 0; slot < AHEAD; ++slot) {
      const int block = base + slot * stride;
      if (block >= p.blocks) break;
      const uint32_t lo[4] = {ring[slot][0].x, ring[slot][0].y, ring[slot][0].z, ring[slot][0].w};
      const uint32_t hi[4] = {ring[slot][1].x, ring[slot][1].y, ring[slot][1].z, ring[slot][1].w};
      float acc[NT][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int f = j * 32 / FLUSH;
        const uint32_t zlo = H::zero_pair(zero[slot][f][0]), zhi = H::zero_pair(zero[slot][f][1]);
        uint32_t xv[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (xrow[nt]) load_x<XT>(p, xrow[nt], xpart[nt], block * 128 + j * 32 + t * 8, xv[nt]);
          else xv[nt][0] = xv[nt][1] = xv[nt][2] = xv[nt][3] = 0u;
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          uint32_t a[4];
          a[0] = H::sub(((lo[j] >> (4 * i)) & 0x000F000Fu) | H::kMagic, zlo);
          a[1] = H::sub(((hi[j] >> (4 * i)) & 0x000F000Fu) | H::kMagic, zhi);
          a[2] = H::sub(((lo[j] >> (4 * i + 4)) & 0x000F000Fu) | H::kMagic, zlo);
          a[3] = H::sub(((hi[j] >> (4 * i + 4)) & 0x000F000Fu) | H::kMagic, zhi);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) H::mma(acc[nt], a, xv[nt][i], xv[nt][i + 1]);
        }
        if ((j + 1) * 32 % FLUSH == 0) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              total[nt][c] = fmaf(acc[nt][c], scale[slot][f][c >> 1], total[nt][c]);
              acc[nt][c] = 0.f;
            }
          }
        }
      }
      fetch(slot, block + AHEAD * stride);
    }
  }

  __shared__ float sums[kWarps][16][NT * 8 + 1];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    sums[warp][g][nt * 8 + 2 * t] = total[nt][0];
    sums[warp][g][nt * 8 + 2 * t + 1] = total[nt][1];
    sums[warp][g + 8][nt * 8 + 2 * t] = total[nt][2];
    sums[warp][g + 8][nt * 8 + 2 * t + 1] = total[nt][3];
  }
  __syncthreads();
  // warp 0's plane takes the CTA's sum
  for (int i = threadIdx.x; i < 16 * NT * 8; i += kWarps * 32) {
    const int row = i & 15, n = i >> 4;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sums[w][row][n];
    sums[0][row][n] = v;
  }
  if (split > 1) cluster.sync();
  else __syncthreads();
  if (part_k == 0) {
    for (int i = threadIdx.x; i < 16 * tokens; i += kWarps * 32) {
      const int row = i & 15, token = i >> 4;
      if (tile * 16 + row >= p.rows) continue;
      float v = 0.f;
      for (int q = 0; q < split; ++q) {
        const float* const from = q == 0 ? &sums[0][row][0] : cluster.map_shared_rank(&sums[0][row][0], q);
#pragma unroll
        for (int part = PARTS - 1; part >= 0; --part) v += from[token * PARTS + part];
      }
      static_cast<XT*>(p.y)[static_cast<size_t>(token0 + token) * p.rows + tile * 16 + row] = from_f32<XT>(v);
    }
  }
  if (split > 1) cluster.sync();  // nobody leaves while its shared memory is read
}

template <typename XT, int NT, int FLUSH>
bcjr_status launch(const Params& p, int split, int passes, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.rows + 15) / 16 * split), 1, static_cast<unsigned>(passes));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(split);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, int4_matmul_kernel<XT, NT, FLUSH>, p) != cudaSuccess) {
    cudaGetLastError();
    return BCJR_ERR_CUDA;
  }
  return BCJR_OK;
}

template <typename XT, int NT>
bcjr_status launch_flush(const Params& p, int split, int passes, cudaStream_t s) {
  if (p.group == 32) return launch<XT, NT, 32>(p, split, passes, s);
  if (p.group == 64) return launch<XT, NT, 64>(p, split, passes, s);
  return launch<XT, NT, 128>(p, split, passes, s);
}

template <typename XT>
bcjr_status launch_tokens(Params p, int sms, cudaStream_t s) {
  constexpr int PARTS = sizeof(XT) == 4 ? 3 : 1;
  const int nt = p.tokens * PARTS <= 8 ? 1 : p.tokens * PARTS <= 16 ? 2 : 4;
  p.pass_tokens = nt * 8 / PARTS;
  const int passes = (p.tokens + p.pass_tokens - 1) / p.pass_tokens;
  // columns are split over the CTAs of a cluster while that leaves every warp
  // a block and the rows alone do not give two CTAs a multiprocessor
  const int tiles = (p.rows + 15) / 16;
  int split = 1;
  while (split < 8 && static_cast<long long>(tiles) * passes * split < 2 * sms && p.blocks >= 2 * split * kWarps) split *= 2;
  if (nt == 1) return launch_flush<XT, 1>(p, split, passes, s);
  if (nt == 2) return launch_flush<XT, 2>(p, split, passes, s);
  return launch_flush<XT, 4>(p, split, passes, s);
}

}  // namespace

extern "C" bcjr_status bcjr_int4_matmul(const void* x, int x_dtype, int tokens, int rows, int cols, const void* packed,
                                        const void* scales, int scale_dtype, const uint8_t* zeros, int group_size,
                                        void* y, bcjr_stream_t stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(scale_dtype) || tokens < 0 || rows < 0 || cols < 1 || group_size < 0)
    return BCJR_ERR_INVALID_ARG;
  if (group_size % 128 != 0 && group_size != 32 && group_size != 64) return BCJR_ERR_UNSUPPORTED;
  // passes are the third grid dimension; row tiles times the split the first
  if (tokens > 65535 || rows > (1 << 30) || cols > (1 << 30)) return BCJR_ERR_UNSUPPORTED;
  if (tokens == 0 || rows == 0) return BCJR_OK;
  if (!x || !packed || !scales || !y || !ptr_aligned(packed, 16) || !ptr_aligned(x, dtype_size(x_dtype)) ||
      !ptr_aligned(y, dtype_size(x_dtype)) || !ptr_aligned(scales, dtype_size(scale_dtype)))
    return BCJR_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0) return BCJR_ERR_CUDA;
  Params p = {};
  p.x = x;
  p.packed = static_cast<const uint8_t*>(packed);
  p.scales = scales;
  p.zeros = zeros;
  p.y = y;
  p.tokens = tokens;
  p.rows = rows;
  p.cols = cols;
  p.blocks = (cols + 127) / 128;
  p.group = group_size == 0 || group_size >= cols ? p.blocks * 128 : group_size;
  p.scale_dtype = scale_dtype;
  p.fast_x = ptr_aligned(x, 16) && (cols * dtype_size(x_dtype)) % 16 == 0;
  cudaStream_t s = as_stream(stream);
  if (x_dtype == BCJR_F32) return launch_tokens<float>(p, sms, s);
  if (x_dtype == BCJR_F16) return launch_tokens<__half>(p, sms, s);
  return launch_tokens<__nv_bfloat16>(p, sms, s);
}
