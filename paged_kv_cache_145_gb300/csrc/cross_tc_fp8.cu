// Cross attention on tensor cores: instantiations for FP8 pools (head_dim
// 128), q and out in fp16 or bf16.
#include "cross_tc.cuh"

int pkv_launch_cross_tc_fp8(const pkv::CrossParams& p, int io_dtype, int num_seqs, bool wide,
                            const pkv::CrossMaps& maps, cudaStream_t stream) {
  if (io_dtype == PKV_F16)
    return wide ? pkv::launch_cross_tc<__half, 128, 2, true>(p, num_seqs, maps, stream)
                : pkv::launch_cross_tc<__half, 128, 1, true>(p, num_seqs, maps, stream);
  return wide ? pkv::launch_cross_tc<__nv_bfloat16, 128, 2, true>(p, num_seqs, maps, stream)
              : pkv::launch_cross_tc<__nv_bfloat16, 128, 1, true>(p, num_seqs, maps, stream);
}
