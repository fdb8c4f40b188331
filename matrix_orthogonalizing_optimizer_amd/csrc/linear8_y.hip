// Forward product of the linear layer on 8-bit rows.
#include "linear8_few.hpp"
#include "linear8_inst.hpp"

namespace muon {

namespace {
template <int T> hipError_t few(int odt, const Linear8Args& a, hipStream_t s) {
  const dim3 g((unsigned)((a.N + 15) / 16));
  if (odt == DT_BF16) hipLaunchKernelGGL((linear8_few_kernel<T, bf16>), g, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((linear8_few_kernel<T, float>), g, dim3(512), 0, s, a);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_linear8_few(int odt, const Linear8Args& a, hipStream_t s) {
  return a.M <= 16 ? few<1>(odt, a, s) : a.M <= 32 ? few<2>(odt, a, s) : few<4>(odt, a, s);
}

hipError_t launch_linear8_planes(int dt, const PlanesArgs& a, hipStream_t s) {
  const int64_t groups = (a.rows + 3) / 4;
  const dim3 g((unsigned)(groups < (1 << 20) ? groups : (1 << 20)), (unsigned)((a.cols + 511) / 512));
  if (dt == DT_BF16) hipLaunchKernelGGL((linear8_planes_kernel<bf16>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((linear8_planes_kernel<float>), g, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_linear8_forward(int tile, int odt, const Linear8Args& a, hipStream_t s) {
  return tile == 256 ? linear8_go<L8_Y, B_Q8, 256>(odt, a, s)
                     : linear8_go<L8_Y, B_Q8, 128>(odt, a, s);
}
}  // namespace muon
