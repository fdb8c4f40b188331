// Forward product of the 8-bit linear layer for few tokens, gfx950.
//
// With few tokens the product reads each weight byte once and does little
// with it: it is bound by HBM.  A workgroup owns CG groups of 16 channels and
// all tokens (T tiles of 16), the 8 / CG waves of a group share K in contiguous
// parts, and their sums (exact in 32-bit integers) join in LDS.  v_mfma_i32_16x16x64_i8 with the
// weights as its rows: a lane loads 16 bytes of channel lane % 16, so a
// wave-wide load takes 64 bytes of 16 rows, and two steps in a row take whole
// 128-byte lines; a lane's four results are four neighbouring channels of one
// token.  Weights and activations go to registers directly: no wave shares a
// weight, and the activations come from L2.  One token, 14336 x 4096: 14.2 us
// (4.1 TB/s of weights, about 3 us of it launch and ramp).  More tokens cost
// the activations' way from L2 to the registers of every workgroup (16 tokens
// there 20.5 us); sharing them among four groups of a workgroup saves 0.4 to 2 us
// of that and costs more elsewhere (too few workgroups: 4096 x 4096, 16 tokens
// 6.8 -> 16.5 us), so more than one group is left to short rows.
#pragma once

#include "device_common.hpp"
#include "kernel_args.hpp"
#include "row_ops.hpp"

namespace muon {

typedef int32_t i32x4v __attribute__((ext_vector_type(4)));

struct __attribute__((packed, aligned(2))) u32x2_e2 {
  u32x2 v;
};
template <typename TO> __device__ __forceinline__ void store4(TO* y, const float (&v)[4]) {
  if constexpr (sizeof(TO) == 2)
    as_global(reinterpret_cast<u32x2_e2*>(y))->v = u32x2{pack2<TO>(v[0], v[1]), pack2<TO>(v[2], v[3])};
  else
    as_global(reinterpret_cast<f32x4_e4*>(y))->v = f32x4{v[0], v[1], v[2], v[3]};
}

template <int T, int CG, typename TO>
__global__ __launch_bounds__(512) void linear8_few_kernel(const Linear8Args a) {
  constexpr int U = 8 / T;    // steps of 64 in flight
  constexpr int KP = 8 / CG;  // parts of K
  __shared__ i32x4v part[4][T][64];
  const int lane = threadIdx.x & 63, l16 = lane & 15, kq = (lane >> 4) * 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cg = wave % CG, kp = wave / CG;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * CG) + 16 * cg;
  const int steps = (a.K + 63) / 64;
  const int per = (steps + KP - 1) / KP;
  const int s1 = min(steps, (kp + 1) * per);
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
  for (int s = kp * per; s < s1; s += U) {
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
  // the upper half of the parts of K to the lower half, until one is left
#pragma unroll
  for (int h = KP / 2; h >= 1; h >>= 1) {
    if (kp >= h && kp < 2 * h) {
#pragma unroll
      for (int i = 0; i < T; ++i) part[(kp - h) * CG + cg][i][lane] = acc[i];
    }
    __syncthreads();
    if (kp < h) {
#pragma unroll
      for (int i = 0; i < T; ++i) acc[i] += part[kp * CG + cg][i][lane];
    }
    if (h > 1) __syncthreads();
  }
  if (kp != 0) return;
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
    float sx, sx2;
    split_scale(as_global(a.sa)[tok], sx, sx2);
    TO* y = static_cast<TO*>(a.o) + tok * a.ldo + n;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = (float)acc[t][e] * sx * ws[e] * sx2;
      if (a.bias) v[e] += b[e];
    }
    if (n + 4 <= a.N) {
      store4(y, v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < a.N) as_global(y)[e] = from_f32<TO>(v[e]);
    }
  }
}

}  // namespace muon
