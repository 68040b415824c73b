// int4_matmul_f32.cu -- the 4-bit product's kernels for float32 inputs.
#include "int4_matmul.cuh"

bcjr_status bcjr::int4_matmul_f32(Int4MatmulParams p, int group, int sms, cudaStream_t s) {
  return launch_groups<float>(p, group, sms, s);
}
