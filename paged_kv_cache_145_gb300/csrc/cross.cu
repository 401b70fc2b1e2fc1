// Cross attention on CUDA cores: instantiations and launch.
#include <type_traits>

#include "cross.cuh"

namespace {

template <typename T, typename TC, int D>
int launch(const pkv::CrossParams& p, int num_seqs, cudaStream_t stream) {
  const int64_t tiles =
      ((int64_t)p.max_queries * p.group + pkv::kCrossRows - 1) / pkv::kCrossRows;
  if (tiles * p.kv_heads > INT32_MAX) return PKV_ERR_ARG;
  const dim3 grid((unsigned)(tiles * p.kv_heads), (unsigned)num_seqs, (unsigned)p.parts);
  pkv::cross_kernel<T, TC, D><<<grid, pkv::kCrossWarps * 32, 0, stream>>>(p);
  return pkv::launch_cross_merge<T, D>(p, num_seqs, stream);
}

}  // namespace

// fp32 pools (head_dim 64 or 128) and FP8 pools of head_dim 64.
int pkv_launch_cross(const pkv::CrossParams& p, int dtype, int io_dtype, int num_seqs, int dim,
                     cudaStream_t stream) {
  switch (dtype) {
    case PKV_F32:
      return dim == 64 ? launch<float, float, 64>(p, num_seqs, stream)
                       : launch<float, float, 128>(p, num_seqs, stream);
    case PKV_FP8_E4M3:  // (head_dim 64)
      return io_dtype == PKV_F16 ? launch<__half, __nv_fp8_e4m3, 64>(p, num_seqs, stream)
                                 : launch<__nv_bfloat16, __nv_fp8_e4m3, 64>(p, num_seqs, stream);
  }
  return PKV_ERR_ARG;
}
