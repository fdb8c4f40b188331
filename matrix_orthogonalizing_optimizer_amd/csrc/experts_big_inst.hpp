// Launch of one pass of the large products grouped by expert.
#pragma once

#include "experts_big.hpp"
#include "launch.hpp"

namespace muon {

template <int MODE> hipError_t experts_big_go(int odt, const ExpertsArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((experts_list_kernel<MODE>), dim3(8), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 g(256), b(512);  // a workgroup on every CU
  if (odt == DT_BF16) hipLaunchKernelGGL((experts_big_kernel<MODE, bf16>), g, b, 0, s, a);
  else hipLaunchKernelGGL((experts_big_kernel<MODE, float>), g, b, 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess || MODE != EX_DW || a.rows <= a.chunk) return e;
  if (odt == DT_BF16) hipLaunchKernelGGL((experts_sum_kernel<bf16>), dim3(512), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((experts_sum_kernel<float>), dim3(512), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
