// int4_api.cu -- the C entry of the product with 4-bit weights: checks, then the kernels of int4_matmul_*.cu.
#include "int4_internal.h"
#include "layer_util.cuh"

using namespace bcjr;

extern "C" bcjr_status bcjr_int4_matmul(const void* x, int x_dtype, int tokens, int rows, int cols, const void* packed,
                                        const void* scales, int scale_dtype, const uint8_t* zeros, int group_size,
                                        void* y, bcjr_stream_t stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(scale_dtype) || tokens < 0 || rows < 0 || cols < 1 || group_size < 0)
    return BCJR_ERR_INVALID_ARG;
  if (group_size % 128 != 0 && group_size != 32 && group_size != 64) return BCJR_ERR_UNSUPPORTED;
  // passes (of at least 10 tokens) are the third grid dimension, row tiles times the split the first;
  // a block's group comes out of a float product, exact below 2^21 blocks
  if (tokens > 10 * 65535 || rows > (1 << 30) || cols > (1 << 27)) return BCJR_ERR_UNSUPPORTED;
  if (tokens == 0 || rows == 0) return BCJR_OK;
  if (!x || !packed || !scales || !y || !ptr_aligned(packed, 16) || !ptr_aligned(x, dtype_size(x_dtype)) ||
      !ptr_aligned(y, dtype_size(x_dtype)) || !ptr_aligned(scales, dtype_size(scale_dtype)))
    return BCJR_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0) return BCJR_ERR_CUDA;
  Int4MatmulParams p = {};
  p.x = x;
  p.packed = static_cast<const uint8_t*>(packed);
  p.scales = scales;
  p.zeros = zeros;
  p.y = y;
  p.tokens = tokens;
  p.rows = rows;
  p.cols = cols;
  p.blocks = (cols + 127) / 128;
  p.fast_x = ptr_aligned(x, 16) && (cols * dtype_size(x_dtype)) % 16 == 0;
  p.fast_groups = rows % 4 == 0 && ptr_aligned(scales, 4 * dtype_size(scale_dtype)) && ptr_aligned(zeros, 4);
  const int group = group_size == 0 || group_size >= cols ? p.blocks * 128 : group_size;
  p.groups = (cols + group - 1) / group;
  p.inv_group = group >= 128 ? 1.f / static_cast<float>(group / 128) : 0.f;
  p.long_groups = group > 128;
  p.scale_dtype = scale_dtype;
  cudaStream_t s = as_stream(stream);
  if (x_dtype == BCJR_F32) return int4_matmul_f32(p, group, sms, s);
  if (x_dtype == BCJR_F16) return int4_matmul_f16(p, group, sms, s);
  return int4_matmul_bf16(p, group, sms, s);
}
