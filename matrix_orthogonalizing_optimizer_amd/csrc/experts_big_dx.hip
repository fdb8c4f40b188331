// Large products grouped by expert: input gradient.
#include "experts_big_inst.hpp"

namespace muon {
hipError_t launch_experts_big_dx(int odt, const ExpertsArgs& a, hipStream_t s) { return experts_big_go<EX_DX>(odt, a, s); }
}  // namespace muon
