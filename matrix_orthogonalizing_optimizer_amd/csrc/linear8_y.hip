// Forward product of the linear layer on 8-bit rows.
#include "linear8_inst.hpp"

namespace muon {
hipError_t launch_linear8_forward(int tile, int odt, const Linear8Args& a, hipStream_t s) {
  return tile == 256 ? linear8_go<L8_Y, A_DIRECT, 256>(odt, a, s) : linear8_go<L8_Y, A_DIRECT, 128>(odt, a, s);
}
}  // namespace muon
