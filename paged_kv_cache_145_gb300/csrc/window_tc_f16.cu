// Windowed attention on tensor cores: instantiations for f16 pools.
#include "window_tc.cuh"

int pkv_launch_window_tc_f16(const pkv::WindowParams& p, int dim, const pkv::WindowMaps& maps, int sms,
                             cudaStream_t stream) {
  using T = __half;
  return dim == 64 ? pkv::launch_window_tc<T, 64>(p, maps, sms, stream)
                   : pkv::launch_window_tc<T, 128>(p, maps, sms, stream);
}
