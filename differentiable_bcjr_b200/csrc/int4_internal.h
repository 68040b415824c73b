// int4_internal.h -- launch parameters shared by the C-ABI layer and the 4-bit product's kernels.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "bcjr_layer.h"

namespace bcjr {

struct Int4MatmulParams {
  const void* x;
  const uint8_t* packed;
  const void* scales;
  const uint8_t* zeros;
  void* y;
  int tokens, rows, cols, blocks;
  bool fast_x;         // x may be read 16 bytes at a time
  bool fast_groups;    // scales and zero points may be read four rows at a time
  int groups;
  float inv_group;     // 1 / (blocks of a group), for groups of 128 columns and more
  bool long_groups;    // groups of more than 128 columns
  int scale_dtype;
  int chunk;           // blocks staged at a time
  int pass_tokens;     // tokens of a pass (grid z)
};

// One translation unit for each type of x.  `group`: columns of a group.
bcjr_status int4_matmul_f32(Int4MatmulParams p, int group, int sms, cudaStream_t s);
bcjr_status int4_matmul_f16(Int4MatmulParams p, int group, int sms, cudaStream_t s);
bcjr_status int4_matmul_bf16(Int4MatmulParams p, int group, int sms, cudaStream_t s);

}  // namespace bcjr
