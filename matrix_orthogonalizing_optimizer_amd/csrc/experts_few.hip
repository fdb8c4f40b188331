// Forward product grouped by expert for few rows an expert.
#include "experts_few.hpp"

#include "launch.hpp"

namespace muon {

namespace {
template <int T, int CG, int U, bool WHOLE, typename TI> hipError_t go(int odt, const ExpertsArgs& a, hipStream_t s) {
  const dim3 g((unsigned)((a.N + 16 * CG - 1) / (16 * CG)), (unsigned)(a.experts < a.rows ? a.experts : a.rows)), b(512);
  if (odt == DT_BF16) hipLaunchKernelGGL((experts_few_kernel<T, CG, U, WHOLE, TI, bf16>), g, b, 0, s, a);
  else hipLaunchKernelGGL((experts_few_kernel<T, CG, U, WHOLE, TI, float>), g, b, 0, s, a);
  return hipGetLastError();
}
// Rows of an expert on average -> rows and channels of a workgroup at a time.
// Two tiles of rows and two groups of channels read the rows half as often, and
// leave enough workgroups where the channels of all experts make 512 (us, one
// of each against two: 64 experts of 1408 x 2048, 384 rows 82 and 76, 1024 rows
// 131 and 103, before experts of at most 16 rows left the second tile out; but 64 rows, one an expert, 38 and 39, 16 rows of one expert of
// 768 x 768 6.0 and 7.5).  Where they do not, 4 tiles of rows from 8 rows an
// expert up (256 rows over 16 experts of 512 x 513: 25 and 14 us).
template <bool WHOLE, typename TI> hipError_t few(int odt, const ExpertsArgs& a, hipStream_t s) {
  const int64_t some = a.experts < a.rows ? a.experts : a.rows;
  if (a.rows > 2 * some && some * ((a.N + 31) / 32) >= 512) return go<2, 2, 4, WHOLE, TI>(odt, a, s);
  return a.rows <= 8 * some ? go<1, 1, 4, WHOLE, TI>(odt, a, s) : go<4, 1, 1, WHOLE, TI>(odt, a, s);
}
}  // namespace

hipError_t launch_experts_few(int dt, int odt, const ExpertsArgs& a, hipStream_t s) {
  if (dt == DT_F32) return a.K % 16 == 0 ? few<true, float>(odt, a, s) : few<false, float>(odt, a, s);
  return a.K % 32 == 0 ? few<true, bf16>(odt, a, s) : few<false, bf16>(odt, a, s);
}

}  // namespace muon
