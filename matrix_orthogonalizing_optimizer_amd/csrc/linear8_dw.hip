// Weight gradient of the linear layer on 8-bit rows.
#include "linear8_inst.hpp"

namespace muon {
hipError_t launch_linear8_dw(int tile, bool expanded, bool dy_f32, int odt, const Linear8Args& a, hipStream_t s) {
  return linear8_grad_any<L8_DW>(tile, expanded, dy_f32, odt, a, s);
}
}  // namespace muon
