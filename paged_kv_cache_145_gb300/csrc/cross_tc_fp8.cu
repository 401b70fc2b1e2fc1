// Cross attention on tensor cores: instantiations for FP8 pools (head_dim
// 128), q and out in fp16 or bf16.
#include "cross_tc.cuh"

namespace {

template <typename T>
int launch(const pkv::CrossParams& p, int num_seqs, bool wide, const pkv::CrossMaps& maps,
           cudaStream_t stream) {
  return wide ? pkv::launch_cross_tc<T, 128, 2, true>(p, num_seqs, maps, stream)
              : pkv::launch_cross_tc<T, 128, 1, true>(p, num_seqs, maps, stream);
}

}  // namespace

int pkv_launch_cross_tc_fp8(const pkv::CrossParams& p, int io_dtype, int num_seqs, bool wide,
                            const pkv::CrossMaps& maps, cudaStream_t stream) {
  return io_dtype == PKV_F16 ? launch<__half>(p, num_seqs, wide, maps, stream)
                             : launch<__nv_bfloat16>(p, num_seqs, wide, maps, stream);
}
