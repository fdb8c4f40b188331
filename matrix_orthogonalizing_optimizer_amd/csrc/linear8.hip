// Linear layer on 8-bit rows.
#include "launch.hpp"
#include "linear8.hpp"

namespace muon {

hipError_t launch_linear8_forward(int dt, const Linear8Args& a, hipStream_t s) {
  const dim3 g((unsigned)((a.out + 63) / 64), (unsigned)((a.tokens + 63) / 64));
  if (dt == DT_BF16) hipLaunchKernelGGL((linear8_forward_kernel<bf16>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((linear8_forward_kernel<float>), g, dim3(256), 0, s, a);
  return hipGetLastError();
}

namespace {
template <bool WG, typename TD> hipError_t grad(int dt, const Linear8Args& a, hipStream_t s) {
  const int rows = WG ? a.out : a.tokens;
  const dim3 g((unsigned)((a.in + 63) / 64), (unsigned)((rows + 63) / 64));
  if (dt == DT_BF16) hipLaunchKernelGGL((linear8_grad_kernel<WG, TD, bf16>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((linear8_grad_kernel<WG, TD, float>), g, dim3(256), 0, s, a);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_linear8_grad(bool weight, int dy_dt, int out_dt, const Linear8Args& a, hipStream_t s) {
  if (weight) return dy_dt == DT_BF16 ? grad<true, bf16>(out_dt, a, s) : grad<true, float>(out_dt, a, s);
  return dy_dt == DT_BF16 ? grad<false, bf16>(out_dt, a, s) : grad<false, float>(out_dt, a, s);
}

}  // namespace muon
