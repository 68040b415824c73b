// trellis_internal.h -- launch parameters shared by the C-ABI layer and the trellis product's kernels.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "bcjr_layer.h"

namespace bcjr {

struct TrellisMatmulParams {
  const void* x;
  const uint32_t* packed;
  const void* codebook;
  const float* scales;
  void* y;
  int x_dtype, c_dtype;
  int tokens, rows, cols, n, words;
  int L, group;
  int seqs;         // sequences of a row
  int per_seq;      // chunks of a sequence
  int chunks;       // of a row
  int wide;         // warps that share a row
  int copies_log2;  // of the codebook
  int unit_chunks;  // chunks of a scale (of a row without scales)
  int unit_steps;   // of four chunks, of a scale
  int steps;        // of a row
  bool padded;      // some chunks have fewer steps, or some fours fewer chunks
  uint64_t seq_inverse, unit_inverse;  // 2^40 / per_seq and / unit_steps, rounded up
};

// One translation unit for each number of bits a step.
bcjr_status trellis_matmul_k1(const TrellisMatmulParams& p, int sms, cudaStream_t s);
bcjr_status trellis_matmul_k2(const TrellisMatmulParams& p, int sms, cudaStream_t s);
bcjr_status trellis_matmul_k3(const TrellisMatmulParams& p, int sms, cudaStream_t s);
bcjr_status trellis_matmul_k4(const TrellisMatmulParams& p, int sms, cudaStream_t s);

}  // namespace bcjr
