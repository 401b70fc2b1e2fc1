// Windowed attention for single tokens: instantiations for 16-bit and FP8 pools.
#include "window_token.cuh"

namespace {

template <typename T, typename TC>
int launch(const pkv::WindowParams& p, int num_seqs, int dim, const pkv::CrossMaps& maps,
           cudaStream_t stream) {
  return dim == 64 ? pkv::launch_window_token<T, TC, 64>(p, num_seqs, maps, stream)
                   : pkv::launch_window_token<T, TC, 128>(p, num_seqs, maps, stream);
}

}  // namespace

int pkv_launch_window_token(const pkv::WindowParams& p, int dtype, int io_dtype, int num_seqs, int dim,
                            const pkv::CrossMaps& maps, cudaStream_t stream) {
  using F16 = __half;
  using BF16 = __nv_bfloat16;
  using FP8 = __nv_fp8_e4m3;
  switch (dtype) {
    case PKV_F16: return launch<F16, F16>(p, num_seqs, dim, maps, stream);
    case PKV_BF16: return launch<BF16, BF16>(p, num_seqs, dim, maps, stream);
    case PKV_FP8_E4M3:
      return io_dtype == PKV_F16 ? launch<F16, FP8>(p, num_seqs, dim, maps, stream)
                                 : launch<BF16, FP8>(p, num_seqs, dim, maps, stream);
  }
  return PKV_ERR_ARG;
}
