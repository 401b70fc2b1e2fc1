// Cross attention on tensor cores: instantiations for bf16 pools.
#include "cross_tc.cuh"

int pkv_launch_cross_tc_bf16(const pkv::CrossParams& p, int num_seqs, int dim,
                           const pkv::CrossMaps& maps, cudaStream_t stream) {
  using T = __nv_bfloat16;
  return dim == 64 ? pkv::launch_cross_tc<T, 64, 1, false>(p, num_seqs, maps, stream)
                   : pkv::launch_cross_tc<T, 128, 1, false>(p, num_seqs, maps, stream);
}
