// int4_matmul_bf16.cu -- the 4-bit product's kernels for bfloat16 inputs.
#include "int4_matmul.cuh"

bcjr_status bcjr::int4_matmul_bf16(Int4MatmulParams p, int group, int sms, cudaStream_t s) {
  return launch_groups<__nv_bfloat16>(p, group, sms, s);
}
