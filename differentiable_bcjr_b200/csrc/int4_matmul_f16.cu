// int4_matmul_f16.cu -- the 4-bit product's kernels for half inputs.
#include "int4_matmul.cuh"

bcjr_status bcjr::int4_matmul_f16(Int4MatmulParams p, int group, int sms, cudaStream_t s) {
  return launch_groups<__half>(p, group, sms, s);
}
