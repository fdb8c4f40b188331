// Forward product of the 8-bit linear layer for few tokens, gfx950.
//
// With few tokens the product reads each weight byte once and does little
// with it: it is bound by HBM.  A workgroup owns 16 channels and all tokens
// (T tiles of 16), its 8 waves share K in contiguous parts, and their sums
// (exact in 32-bit integers) join in LDS.  v_mfma_i32_16x16x64_i8 with the
// weights as its rows: a lane loads 16 bytes of channel lane % 16, so a
// wave-wide load takes 64 bytes of 16 rows, and two steps in a row take whole
// 128-byte lines; a lane's four results are four neighbouring channels of one
// token.  Weights and activations go to registers directly: no wave shares a
// weight, and the activations come from L2.  One token, 14336 x 4096: 14.2 us
// (4.1 TB/s of weights, about 3 us of it launch and ramp); T channel tiles
// per workgroup, to use an activation fragment T times, was slower below 8192
// channels (too few workgroups: 64 tokens, 4096 x 4096: 29.5 against 14.9 us).
#pragma once

#include "device_common.hpp"
#include "kernel_args.hpp"
#include "row_ops.hpp"

namespace muon {

typedef int32_t i32x4v __attribute__((ext_vector_type(4)));

template <int T, typename TO>
__global__ __launch_bounds__(512) void linear8_few_kernel(const Linear8Args a) {
  constexpr int U = 8 / T;    // steps of 64 in flight
  __shared__ i32x4v part[4][T][64];
  const int lane = threadIdx.x & 63, l16 = lane & 15, kq = (lane >> 4) * 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int steps = (a.K + 63) / 64;
  const int per = (steps + 7) / 8;
  const int s1 = min(steps, (wave + 1) * per);
  const bool wok = n0 + l16 < a.N;
  const int8_t* wrow = static_cast<const int8_t*>(a.B) + (n0 + l16) * a.ldb + kq;
  const int8_t* xrow[T];
  bool xok[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    xok[t] = 16 * t + l16 < a.M;
    xrow[t] = static_cast<const int8_t*>(a.A) + (int64_t)(16 * t + l16) * a.lda + kq;
  }
  i32x4v acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) acc[t] = i32x4v{0, 0, 0, 0};
  for (int s = wave * per; s < s1; s += U) {
    i32x4v w[U], x[U][T];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + u) * 64;
      // a 16-byte piece that starts before K lies in its row's storage
      const bool in = s + u < s1 && k + kq < a.K;
      w[u] = i32x4v{0, 0, 0, 0};
      if (in && wok) w[u] = *as_global(reinterpret_cast<const i32x4v*>(wrow + k));
#pragma unroll
      for (int t = 0; t < T; ++t) {
        x[u][t] = i32x4v{0, 0, 0, 0};
        if (in && xok[t]) x[u][t] = *as_global(reinterpret_cast<const i32x4v*>(xrow[t] + k));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < T; ++t) acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u], x[u][t], acc[t], 0, 0, 0);
  }
  // waves 4..7 to 0..3, then 2, 3 to 0, 1, then 1 to 0
#pragma unroll
  for (int h = 4; h >= 1; h >>= 1) {
    if (wave >= h && wave < 2 * h) {
#pragma unroll
      for (int i = 0; i < T; ++i) part[wave - h][i][lane] = acc[i];
    }
    __syncthreads();
    if (wave < h) {
#pragma unroll
      for (int i = 0; i < T; ++i) acc[i] += part[wave][i][lane];
    }
    if (h > 1) __syncthreads();
  }
  if (wave != 0) return;
  const int64_t n = n0 + 4 * (lane >> 4);
  float ws[4], b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    ws[e] = n + e < a.N ? as_global(a.sb)[n + e] : 0.f;
    b[e] = 0.f;
    if (a.bias && n + e < a.N)
      b[e] = a.bias_dtype == DT_F32 ? as_global(static_cast<const float*>(a.bias))[n + e]
                                    : to_f32(as_global(static_cast<const bf16*>(a.bias))[n + e]);
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int64_t tok = 16 * t + l16;
    if (tok >= a.M) continue;
    const float sx = as_global(a.sa)[tok];
    TO* y = static_cast<TO*>(a.o) + tok * a.ldo + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = (float)acc[t][e] * sx * ws[e];
      if (a.bias) v += b[e];
      if (n + e < a.N) as_global(y)[e] = from_f32<TO>(v);
    }
  }
}

}  // namespace muon
