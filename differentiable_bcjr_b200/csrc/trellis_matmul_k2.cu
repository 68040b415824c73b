// trellis_matmul_k2.cu -- the trellis product's kernels for 2 bits a step.
#include "trellis_matmul.cuh"

bcjr_status bcjr::trellis_matmul_k2(const TrellisMatmulParams& p, int sms, cudaStream_t s) {
  return launch_held<2>(p, sms, s);
}
