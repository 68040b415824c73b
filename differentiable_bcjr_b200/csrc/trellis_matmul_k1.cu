// trellis_matmul_k1.cu -- the trellis product's kernels for 1 bit a step.
#include "trellis_matmul.cuh"

bcjr_status bcjr::trellis_matmul_k1(const TrellisMatmulParams& p, int sms, cudaStream_t s) {
  return launch_held<1>(p, sms, s);
}
