// Launch of one mode of the tiled 8-bit linear products.
#pragma once

#include "launch.hpp"
#include "linear8.hpp"

namespace muon {

template <int MODE, int BSRC, int T> hipError_t linear8_go(int odt, const Linear8Args& a, hipStream_t s) {
  constexpr int NW = 8;  // waves per workgroup, for both tiles (see linear8.hpp)
  const int tiles = a.tilesM * a.tilesN, rem = a.splits > 1 ? tiles - a.whole : 0;
  const dim3 g((unsigned)(tiles - rem + rem * a.splits)), b(64 * NW);
  if (odt == DT_BF16) hipLaunchKernelGGL((linear8_kernel<MODE, BSRC, T, NW, bf16>), g, b, 0, s, a);
  else hipLaunchKernelGGL((linear8_kernel<MODE, BSRC, T, NW, float>), g, b, 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || rem == 0) return e;
  const dim3 gj((unsigned)(rem * (T * T / 2048)));
  if (odt == DT_BF16) hipLaunchKernelGGL((linear8_join_kernel<MODE == L8_Y, T, bf16>), gj, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((linear8_join_kernel<MODE == L8_Y, T, float>), gj, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int MODE>
hipError_t linear8_grad_any(int tile, bool expanded, bool dy_f32, int odt, const Linear8Args& a, hipStream_t s) {
  if (dy_f32) return linear8_go<MODE, B_Q8_A_F32, 128>(odt, a, s);
  if (tile == 128) return linear8_go<MODE, B_Q8, 128>(odt, a, s);
  return expanded ? linear8_go<MODE, B_BF16, 256>(odt, a, s) : linear8_go<MODE, B_Q8, 256>(odt, a, s);
}

}  // namespace muon
