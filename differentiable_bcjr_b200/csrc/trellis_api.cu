// trellis_api.cu -- the C entry of the product with packed trellis weights: checks, then the kernels of trellis_matmul_k*.cu.
#include "layer_util.cuh"
#include "trellis_internal.h"

using namespace bcjr;

extern "C" bcjr_status bcjr_trellis_matmul(const void* x, int x_dtype, int tokens, int rows, int cols,
                                           const uint32_t* packed, const void* codebook, int codebook_dtype,
                                           int state_bits, int k, int seq_len, const float* scales, int group_size,
                                           void* y, bcjr_stream_t stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(codebook_dtype) || tokens < 0 || rows < 0 || cols < 1 || seq_len < 1 ||
      state_bits < 1 || k < 1 || k > state_bits || (scales && group_size < 0))
    return BCJR_ERR_INVALID_ARG;
  if (cols % seq_len != 0) return BCJR_ERR_INVALID_ARG;
  // passes of 8 tokens are the second grid dimension; columns and bits are counted in ints
  if (k > 4 || state_bits > 16 || tokens > 8 * 65535 || rows > (1 << 30) || cols > (1 << 28)) return BCJR_ERR_UNSUPPORTED;
  int group = cols;
  if (scales && group_size > 0) {
    group = group_size;
    const bool whole = group % seq_len == 0 && cols % group == 0;
    const bool part = group % 16 == 0 && seq_len % group == 0;
    if (!whole && !part) return BCJR_ERR_UNSUPPORTED;
  }
  if (tokens == 0 || rows == 0) return BCJR_OK;
  if (!x || !packed || !codebook || !y || !ptr_aligned(x, dtype_size(x_dtype)) || !ptr_aligned(y, dtype_size(x_dtype)) ||
      !ptr_aligned(packed, 4) || !ptr_aligned(codebook, dtype_size(codebook_dtype)) || !ptr_aligned(scales, 4))
    return BCJR_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0) return BCJR_ERR_CUDA;
  TrellisMatmulParams p = {};
  p.x = x;
  p.packed = packed;
  p.codebook = codebook;
  p.scales = scales;
  p.y = y;
  p.x_dtype = x_dtype;
  p.c_dtype = codebook_dtype;
  p.tokens = tokens;
  p.rows = rows;
  p.cols = cols;
  p.n = seq_len;
  p.words = static_cast<int>((static_cast<long long>(seq_len) * k + state_bits - k + 31) / 32);
  p.L = state_bits;
  p.group = group;
  p.seqs = cols / seq_len;
  cudaStream_t s = as_stream(stream);
  switch (k) {
    case 1: return trellis_matmul_k1(p, sms, s);
    case 2: return trellis_matmul_k2(p, sms, s);
    case 3: return trellis_matmul_k3(p, sms, s);
    default: return trellis_matmul_k4(p, sms, s);
  }
}
