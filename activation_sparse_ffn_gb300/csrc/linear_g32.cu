// The 4-bit linear layer's kernels for groups of 32.
#define SFFN_LINEAR_GROUP 32
#include "linear.cuh"

namespace sffn {

cudaError_t prepare_linear_g32(int nt, int fmt, LinearFit* fit) { return prepare<32>(nt, fmt, fit); }

cudaError_t run_linear_g32(int nt, int fmt, int cluster, const LinearArgs& a, int blocks, int smem, cudaStream_t st) {
  return run<32>(nt, fmt, cluster, a, blocks, smem, st);
}

}  // namespace sffn
