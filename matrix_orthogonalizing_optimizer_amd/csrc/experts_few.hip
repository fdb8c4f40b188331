// Forward product grouped by expert for few rows an expert.
#include "experts_few.hpp"

#include "experts_plan.hpp"
#include "launch.hpp"

namespace muon {

namespace {
template <int T, int CG, int U, bool WHOLE, typename TI> hipError_t go(int odt, const ExpertsArgs& a, hipStream_t s) {
  const dim3 g((unsigned)((a.N + 16 * CG - 1) / (16 * CG)), (unsigned)(a.experts < a.rows ? a.experts : a.rows)), b(512);
  if (odt == DT_BF16) hipLaunchKernelGGL((experts_few_kernel<T, CG, U, WHOLE, TI, bf16>), g, b, 0, s, a);
  else hipLaunchKernelGGL((experts_few_kernel<T, CG, U, WHOLE, TI, float>), g, b, 0, s, a);
  return hipGetLastError();
}
template <bool WHOLE, typename TI> hipError_t few(const ExpertsFewShape& p, int odt, const ExpertsArgs& a, hipStream_t s) {
  if (p.row_tiles == 2) return go<2, 2, 4, WHOLE, TI>(odt, a, s);
  return p.row_tiles == 1 ? go<1, 1, 4, WHOLE, TI>(odt, a, s) : go<4, 1, 1, WHOLE, TI>(odt, a, s);
}
}  // namespace

hipError_t launch_experts_few(int dt, int odt, const ExpertsArgs& a, hipStream_t s) {
  const ExpertsFewShape p = experts_few_shape(a.rows, a.experts, a.N, a.K, dt == DT_F32 ? MUON_F32 : MUON_BF16);
  if (dt == DT_F32) return p.whole ? few<true, float>(p, odt, a, s) : few<false, float>(p, odt, a, s);
  return p.whole ? few<true, bf16>(p, odt, a, s) : few<false, bf16>(p, odt, a, s);
}

}  // namespace muon
