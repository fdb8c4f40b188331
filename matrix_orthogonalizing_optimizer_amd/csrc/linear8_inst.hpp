// Launch of one mode of the tiled 8-bit linear products.
#pragma once

#include "launch.hpp"
#include "linear8.hpp"

namespace muon {

template <int MODE, int ASRC, int T, int NW = T / 32> hipError_t linear8_go(int odt, const Linear8Args& a, hipStream_t s) {
  const dim3 g((unsigned)(a.tilesM * a.tilesN * a.splits)), b(64 * NW);
  if (a.splits > 1) {
    hipLaunchKernelGGL((linear8_kernel<MODE, ASRC, T, NW, float, true>), g, b, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t pieces = (int64_t)a.M * ((a.N + 7) / 8);
    const dim3 gj((unsigned)((pieces + 255) / 256));
    if (odt == DT_BF16) hipLaunchKernelGGL((linear8_join_kernel<MODE == L8_Y, bf16>), gj, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((linear8_join_kernel<MODE == L8_Y, float>), gj, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  if (odt == DT_BF16) hipLaunchKernelGGL((linear8_kernel<MODE, ASRC, T, NW, bf16, false>), g, b, 0, s, a);
  else hipLaunchKernelGGL((linear8_kernel<MODE, ASRC, T, NW, float, false>), g, b, 0, s, a);
  return hipGetLastError();
}

template <int MODE> hipError_t linear8_grad_any(int tile, int asrc, int odt, const Linear8Args& a, hipStream_t s) {
  if (tile == 256) {
    if (asrc == A_DIRECT) return linear8_go<MODE, A_DIRECT, 256>(odt, a, s);
    if (asrc == A_REG16) return linear8_go<MODE, A_REG16, 256>(odt, a, s);
    return linear8_go<MODE, A_REG32, 256>(odt, a, s);
  }
  if (asrc == A_DIRECT) return linear8_go<MODE, A_DIRECT, 128>(odt, a, s);
  if (asrc == A_REG16) return linear8_go<MODE, A_REG16, 128>(odt, a, s);
  return linear8_go<MODE, A_REG32, 128>(odt, a, s);
}

}  // namespace muon
