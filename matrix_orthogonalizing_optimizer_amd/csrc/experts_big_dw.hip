// Large products grouped by expert: weight gradient.
#include "experts_big_inst.hpp"

namespace muon {
hipError_t launch_experts_big_dw(int odt, const ExpertsArgs& a, hipStream_t s) { return experts_big_go<EX_DW>(odt, a, s); }
}  // namespace muon
