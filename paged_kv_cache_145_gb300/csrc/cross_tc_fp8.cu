// Cross attention on tensor cores: instantiations for FP8 pools (head_dim
// 128), q and out in fp16 or bf16.
#include "cross_stream.cuh"

int pkv_launch_cross_tc_fp8(const pkv::CrossParams& p, int io_dtype, int num_seqs,
                            pkv::CrossRows rows, const pkv::CrossMaps& maps, cudaStream_t stream) {
  return io_dtype == PKV_F16
             ? pkv::launch_cross_rows<__half, 128, true>(p, num_seqs, rows, maps, stream)
             : pkv::launch_cross_rows<__nv_bfloat16, 128, true>(p, num_seqs, rows, maps, stream);
}
