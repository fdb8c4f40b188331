// Linear layer on 8-bit rows, gfx950.
//
//   y[t][n]  = scale[t] wscale[n] sum_k q[t][k] w[n][k] + bias[n]
//   dW[n][k] = sum_t dy[t][n] scale[t] q[t][k]
//   dX[t][k] = sum_n dy[t][n] wscale[n] w[n][k]
// Simple forms: the forward product with one 32 x 32 tile per wave and
// fragments straight from global memory; the gradients with 64 x 64 tiles in
// shared memory and fp32 FMAs.
#pragma once

#include "device_common.hpp"
#include "kernel_args.hpp"

namespace muon {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float any_f32(const void* p, int dt, int64_t i) {
  return dt == DT_F32 ? as_global(static_cast<const float*>(p))[i] : to_f32(as_global(static_cast<const bf16*>(p))[i]);
}

template <typename TO>
__global__ __launch_bounds__(256) void linear8_forward_kernel(const Linear8Args a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l32 = lane & 31, half = lane >> 5;
  const int64_t t0 = (int64_t)blockIdx.y * 64 + (wave >> 1) * 32;
  const int64_t n0 = (int64_t)blockIdx.x * 64 + (wave & 1) * 32;
  const bool tok = t0 + l32 < a.tokens, ch = n0 + l32 < a.out;
  const int8_t* qa = a.q + (t0 + l32) * a.ldq;
  const int8_t* wb = a.w + (n0 + l32) * a.ldw;
  i32x16 acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0;
  for (int k = 0; k < a.in; k += 32) {
    const int kk = k + 16 * half;
    i32x4 fa = {0, 0, 0, 0}, fb = {0, 0, 0, 0};
    // a 16-byte chunk that starts before the end of the row is inside its storage
    if (tok && kk < a.in) fa = *as_global(reinterpret_cast<const i32x4*>(qa + kk));
    if (ch && kk < a.in) fb = *as_global(reinterpret_cast<const i32x4*>(wb + kk));
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa, fb, acc, 0, 0, 0);
  }
  if (!ch) return;
  const int64_t n = n0 + l32;
  const float ws = as_global(a.wscale)[n];
  const float b = a.bias ? any_f32(a.bias, a.bias_dtype, n) : 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int64_t t = t0 + 8 * (e >> 2) + 4 * half + (e & 3);
    if (t < a.tokens)
      as_global(static_cast<TO*>(a.o))[t * a.ldo + n] = from_f32<TO>((float)acc[e] * as_global(a.scale)[t] * ws + b);
  }
}

// WG: rows of the result are outputs n, summed over tokens; else rows are
// tokens, summed over outputs.
template <bool WG, typename TD, typename TO>
__global__ __launch_bounds__(256) void linear8_grad_kernel(const Linear8Args a) {
  __shared__ float sa[16][65], sq[16][65];
  const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
  const int64_t rows = WG ? a.out : a.tokens, sum = WG ? a.tokens : a.out;
  const int8_t* q = WG ? a.q : a.w;
  const float* sc = WG ? a.scale : a.wscale;
  const int64_t ldq = WG ? a.ldq : a.ldw;
  const TD* dy = static_cast<const TD*>(a.dy);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t s0 = 0; s0 < sum; s0 += 16) {
    for (int i = threadIdx.x; i < 16 * 64; i += 256) {
      int ss, rr;
      if (WG) { ss = i >> 6; rr = i & 63; } else { ss = i & 15; rr = i >> 4; }
      const int64_t s = s0 + ss, r = r0 + rr;
      sa[ss][rr] = s < sum && r < rows ? to_f32(as_global(dy)[WG ? s * a.lddy + r : r * a.lddy + s]) : 0.f;
      const int64_t sq_ = s0 + (i >> 6), c = c0 + (i & 63);
      sq[i >> 6][i & 63] =
          sq_ < sum && c < a.in ? (float)as_global(q)[sq_ * ldq + c] * as_global(sc)[sq_] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sq[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = r0 + ty * 4 + i, c = c0 + tx * 4 + j;
      if (r < rows && c < a.in) {
        TO* o = static_cast<TO*>(a.o) + r * a.ldo + c;
        const float old = WG && a.accumulate ? to_f32(*as_global(o)) : 0.f;
        *as_global(o) = from_f32<TO>(acc[i][j] + old);
      }
    }
}

}  // namespace muon
