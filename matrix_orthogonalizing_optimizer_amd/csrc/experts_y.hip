// Forward product of the products grouped by expert.
#include "experts_inst.hpp"

namespace muon {
hipError_t launch_experts_y(bool direct, int dt, int odt, int64_t tiles, int64_t joined, const ExpertsArgs& a, hipStream_t s) {
  return experts_any<EX_Y>(direct, dt, odt, tiles, joined, a, s);
}
}  // namespace muon
