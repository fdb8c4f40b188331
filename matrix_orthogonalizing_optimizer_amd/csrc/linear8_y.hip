// Forward product of the linear layer on 8-bit rows.
#include "linear8_few.hpp"
#include "linear8_inst.hpp"

namespace muon {

namespace {
// A product over no channels: y is the bias, or zero, whatever the scales hold
// (0 times a scale that is not finite would be NaN in the kernels above, and
// asking there costs 1% of a large product).  8 columns of a row per thread.
template <typename TO> __global__ __launch_bounds__(256) void linear8_bias_kernel(const Linear8Args a) {
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= a.N) return;
  float v[8] = {};
  if (a.bias) vec_load(a.bias, a.bias_dtype, (int)c, a.N, v);
  for (int64_t r = blockIdx.y; r < a.M; r += gridDim.y)
    piece_store(static_cast<TO*>(a.o) + r * a.ldo, (int)c, a.N, v);
}

template <int T, int CG> hipError_t few(int odt, const Linear8Args& a, hipStream_t s) {
  const dim3 g((unsigned)((a.N + 16 * CG - 1) / (16 * CG)));
  if (odt == DT_BF16) hipLaunchKernelGGL((linear8_few_kernel<T, CG, bf16>), g, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((linear8_few_kernel<T, CG, float>), g, dim3(512), 0, s, a);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_linear8_few(int odt, const Linear8Args& a, hipStream_t s) {
  if (a.M > 16) return a.M <= 32 ? few<2, 1>(odt, a, s) : few<4, 1>(odt, a, s);
  // short rows leave 8 parts of K one or two steps each: 2 parts for 4 groups
  // of channels, if the groups still fill the chip (us, 1 and 16 tokens:
  // 50304 x 768 13.3 -> 11.0 and 15.2 -> 14.9, 16384 x 1024 6.1 -> 5.4 and 7.0
  // -> 6.5, 50304 x 1024 14.7 -> 13.3 and 17.7 -> 18.7; but 8192 x 768 3.9 ->
  // 4.3, 50304 x 2048 20.5 -> 24.2)
  return a.K <= 1024 && a.N >= 16384 ? few<1, 4>(odt, a, s) : few<1, 1>(odt, a, s);
}

hipError_t launch_linear8_bias(int odt, const Linear8Args& a, hipStream_t s) {
  const dim3 g((unsigned)((a.N + 2047) / 2048), (unsigned)(a.M < 65535 ? a.M : 65535));
  if (odt == DT_BF16) hipLaunchKernelGGL((linear8_bias_kernel<bf16>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((linear8_bias_kernel<float>), g, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_linear8_planes(int dt, const PlanesArgs& a, hipStream_t s) {
  const int64_t groups = (a.rows + 3) / 4;
  const dim3 g((unsigned)(groups < (1 << 20) ? groups : (1 << 20)), (unsigned)((a.cols + 511) / 512));
  if (dt == DT_BF16) hipLaunchKernelGGL((linear8_planes_kernel<bf16>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((linear8_planes_kernel<float>), g, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_linear8_forward(int tile, int odt, const Linear8Args& a, hipStream_t s) {
  return tile == 256 ? linear8_go<L8_Y, B_Q8, 256>(odt, a, s)
                     : linear8_go<L8_Y, B_Q8, 128>(odt, a, s);
}
}  // namespace muon
