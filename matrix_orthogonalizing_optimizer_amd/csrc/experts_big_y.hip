// Large products grouped by expert: forward product.
#include "experts_big_inst.hpp"

namespace muon {
hipError_t launch_experts_big_y(int odt, const ExpertsArgs& a, hipStream_t s) { return experts_big_go<EX_Y>(odt, a, s); }
}  // namespace muon
