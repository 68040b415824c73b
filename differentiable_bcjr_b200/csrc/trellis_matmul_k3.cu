// trellis_matmul_k3.cu -- the trellis product's kernels for 3 bits a step.
#include "trellis_matmul.cuh"

bcjr_status bcjr::trellis_matmul_k3(const TrellisMatmulParams& p, int sms, cudaStream_t s) {
  return launch_held<3>(p, sms, s);
}
