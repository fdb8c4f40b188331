// Launchers of the row operators.
#include <type_traits>

#include "consts.hpp"
#include "launch.hpp"
#include "row_ops.hpp"

namespace muon {

namespace {

// Grid of at least `blocks` workgroups (row_block() numbers them).
dim3 row_grid(int64_t blocks) {
  const int64_t x = blocks < (1 << 20) ? blocks : (1 << 20);
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}

// (threads per row, pieces per thread) for a row of `cols` values.  Smaller
// groups leave fewer lanes idle and have fewer waves to launch, larger ones need
// fewer registers.  Measured, forward / backward: 57 columns 13.9 / 30.7 us with
// a wave per row, 5.2 / 14.4 with 8 lanes; 200 columns 10.2 / 22.2 and 7.6 / 16.0
// with 32; 768 columns (8192 rows) 9.5 / 19.9 and 8.9 / 18.0 with 32 x 3 pieces;
// but 512 columns 12.3 / 19.2 and 12.3 / 21.1 with 32 x 2, 1001 columns 34.4 /
// 66.7 and 35.4 / 83.1 with 32 x 4.
template <typename F> hipError_t by_width(int cols, F&& f) {
  if (cols <= 64) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  if (cols <= 256) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
  if (cols <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  if (cols <= 768) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 3>{});
  if (cols <= 1024) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  if (cols <= 2048) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  if (cols <= 4096) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  if (cols <= 8192) return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}

template <typename T, int KIND> hipError_t forward(const RowArgs& a, hipStream_t s) {
  if (a.cols > ROW_MAX_COLS) {
    hipLaunchKernelGGL((row_forward_long_kernel<T, KIND>), row_grid(a.rows), dim3(1024), 0, s, a);
    return hipGetLastError();
  }
  return by_width(a.cols, [&](auto g, auto nv) {
    constexpr int G = decltype(g)::value, NV = decltype(nv)::value;
    constexpr int RPW = G < 256 ? 256 / G : 1;
    hipLaunchKernelGGL((row_forward_kernel<T, KIND, G, NV>), row_grid((a.rows + RPW - 1) / RPW),
                       dim3(G < 256 ? 256 : G), 0, s, a);
    return hipGetLastError();
  });
}

template <typename T, int KIND> hipError_t backward(const NormBwdArgs& a, int parts, hipStream_t s) {
  if (a.cols > NORM_BWD_MAX_COLS) {
    // the column sums first: dx may overwrite dy
    if (a.partials) {
      hipLaunchKernelGGL((norm_columns_long_kernel<T, KIND>), dim3((unsigned)((a.cols + 2047) / 2048), (unsigned)parts),
                         dim3(256), 0, s, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((norm_backward_long_kernel<T, KIND == 0 ? 0 : 1>), row_grid(a.rows), dim3(1024), 0, s, a);
    return hipGetLastError();
  }
  return by_width(a.cols, [&](auto g, auto nv) {
    constexpr int G = decltype(g)::value, NV = decltype(nv)::value;
    if constexpr (G <= 512) {  // 512 x 2 pieces cover NORM_BWD_MAX_COLS
      hipLaunchKernelGGL((norm_backward_kernel<T, KIND, G, NV>), dim3((unsigned)parts), dim3(G < 256 ? 256 : G), 0, s,
                         a);
      return hipGetLastError();
    }
    return hipErrorInvalidValue;
  });
}

}  // namespace

hipError_t launch_row_forward(int kind, int dt, const RowArgs& a, hipStream_t s) {
  if (dt == DT_BF16)
    return kind == 0 ? forward<bf16, 0>(a, s) : kind == 1 ? forward<bf16, 1>(a, s) : forward<bf16, ROW_COPY>(a, s);
  return kind == 0 ? forward<float, 0>(a, s) : kind == 1 ? forward<float, 1>(a, s) : forward<float, ROW_COPY>(a, s);
}

namespace {
template <typename T> hipError_t restore(const RestoreArgs& a, hipStream_t s) {
  return by_width(a.cols, [&](auto g, auto nv) {
    constexpr int G = decltype(g)::value, NV = decltype(nv)::value;
    constexpr int RPW = G < 256 ? 256 / G : 1;
    hipLaunchKernelGGL((row_restore_kernel<T, G, NV>), row_grid((a.rows + RPW - 1) / RPW),
                       dim3(G < 256 ? 256 : G), 0, s, a);
    return hipGetLastError();
  });
}
}  // namespace

hipError_t launch_row_restore(int dt, const RestoreArgs& a, hipStream_t s) {
  return dt == DT_BF16 ? restore<bf16>(a, s) : restore<float>(a, s);
}

hipError_t launch_norm_backward(int kind, int dt, const NormBwdArgs& a, int parts, hipStream_t s) {
  const bool rms_beta = kind != 0 && a.sum_dy;
  if (dt == DT_BF16)
    return kind == 0 ? backward<bf16, 0>(a, parts, s)
           : rms_beta ? backward<bf16, NORM_RMS_BETA>(a, parts, s)
                      : backward<bf16, 1>(a, parts, s);
  return kind == 0 ? backward<float, 0>(a, parts, s)
         : rms_beta ? backward<float, NORM_RMS_BETA>(a, parts, s)
                    : backward<float, 1>(a, parts, s);
}

hipError_t launch_norm_join(int vec_dtype, const JoinArgs& a, hipStream_t s) {
  const dim3 g((unsigned)((a.cols + 63) / 64), a.dbeta ? 2 : 1);
  if (vec_dtype == DT_BF16) hipLaunchKernelGGL((norm_columns_join_kernel<bf16>), g, dim3(1024), 0, s, a);
  else hipLaunchKernelGGL((norm_columns_join_kernel<float>), g, dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
