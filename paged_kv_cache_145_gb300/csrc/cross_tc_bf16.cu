// Cross attention on tensor cores: instantiations for bf16 pools.
#include "cross_stream.cuh"

int pkv_launch_cross_tc_bf16(const pkv::CrossParams& p, int num_seqs, int dim, pkv::CrossRows rows,
                           const pkv::CrossMaps& maps, cudaStream_t stream) {
  using T = __nv_bfloat16;
  return dim == 64 ? pkv::launch_cross_rows<T, 64, false>(p, num_seqs, rows, maps, stream)
                   : pkv::launch_cross_rows<T, 128, false>(p, num_seqs, rows, maps, stream);
}
