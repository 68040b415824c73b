// trellis_matmul_k4.cu -- the trellis product's kernels for 4 bits a step.
#include "trellis_matmul.cuh"

bcjr_status bcjr::trellis_matmul_k4(const TrellisMatmulParams& p, int sms, cudaStream_t s) {
  return launch_held<4>(p, sms, s);
}
