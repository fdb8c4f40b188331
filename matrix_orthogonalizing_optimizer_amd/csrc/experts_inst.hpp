// Launch of one pass of the tiled products grouped by expert.
#pragma once

#include "experts.hpp"
#include "launch.hpp"

namespace muon {

template <int MODE, bool DIRECT, typename TI, typename TO>
hipError_t experts_go(int64_t tiles, int64_t joined, const ExpertsArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((experts_kernel<MODE, DIRECT, TI, TO>), dim3((unsigned)(tiles * a.splits)), dim3(512), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || joined == 0) return e;
  hipLaunchKernelGGL((experts_join_kernel<MODE, TO>), dim3((unsigned)(joined * (EXPERTS_T * EXPERTS_T / 2048))), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int MODE, typename TO> hipError_t experts_in(bool direct, int dt, int64_t tiles, int64_t joined, const ExpertsArgs& a, hipStream_t s) {
  if (dt == DT_F32) return experts_go<MODE, false, float, TO>(tiles, joined, a, s);
  if (!direct) return experts_go<MODE, false, bf16, TO>(tiles, joined, a, s);
  return experts_go<MODE, true, bf16, TO>(tiles, joined, a, s);
}

template <int MODE> hipError_t experts_any(bool direct, int dt, int odt, int64_t tiles, int64_t joined, const ExpertsArgs& a, hipStream_t s) {
  return odt == DT_BF16 ? experts_in<MODE, bf16>(direct, dt, tiles, joined, a, s)
                        : experts_in<MODE, float>(direct, dt, tiles, joined, a, s);
}

}  // namespace muon
