// Forward product grouped by expert for few rows an expert, gfx950.
//
// With few rows the product reads every weight of the experts that have any
// once and does little with it: it is bound by HBM.  A workgroup owns CG groups
// of 16 channels of one expert and all its rows, T tiles of 16 at a time; its 8
// waves share K in contiguous parts and their sums join in LDS.  The weights are the rows of
// v_mfma_f32_16x16x32_bf16 (fp32: v_mfma_f32_16x16x4_f32): a lane loads 16 bytes
// of channel lane % 16, two steps in a row take whole 128-byte lines, and a
// lane's four results are four neighbouring channels of one row.  Weights and
// rows go to registers directly: no wave shares a weight, and the rows come from
// L2.  Only experts with rows get workgroups: the j-th of the grid's row takes
// the j-th such expert.
//
// Measured, bf16: 6 rows of 64 experts of 1408 x 2048 9.0 to 10.2 us a call (the kernel
// 8.0 on average, 7.6 at least: 64 KB of weights a workgroup, two trips to HBM in
// series for each of its waves); 384 rows of all 64 experts 71 us a call, 5.2 TB/s of
// weights (a large copy: 5.4 to 6.0; the kernel traced over 23 calls 77 to 117 us, 81 on
// average); 900 rows 92: the rows, which every workgroup reads from L2, begin to count.
// An expert's rows are one loop: 384 rows that all go to one of the 64 experts take 95
// us instead of 73.
#pragma once

#include "experts.hpp"

namespace muon {

template <typename TI> struct FewMfma;
template <> struct FewMfma<bf16> {
  static constexpr int STEP = 32;  // K of a step: 16 bytes in each quarter of the wave
  __device__ __forceinline__ static void run(f32x4& c, const u32x4& a, const u32x4& b) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
template <> struct FewMfma<float> {
  static constexpr int STEP = 16;
  __device__ __forceinline__ static void run(f32x4& c, const u32x4& a, const u32x4& b) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], c, 0, 0, 0);
  }
};

struct __attribute__((packed, aligned(2))) u32x2_e2x {
  u32x2 v;
};

// Rows r0 .. r0 + 16 T - 1 of the expert (those below `count`) times its
// channels n0 .. n0 + 16 CG - 1.  ROOM: tiles of sums that `part` has room for.
template <int T, int CG, int U, bool WHOLE, bool SHORT, int ROOM, typename TI, typename TO>
__device__ __forceinline__ void experts_few_rows(const ExpertsArgs& a, const TI* W, const TI* X, TO* Y, int n0, int r0,
                                                 int count, f32x4 (*part)[ROOM][64]) {
  constexpr int STEP = FewMfma<TI>::STEP, PER = STEP / 4;
  const int lane = threadIdx.x & 63, l16 = lane & 15, kq = (lane >> 4) * PER;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int steps = (a.K + STEP - 1) / STEP;
  const int per = (steps + 7) / 8;
  const int s0 = wave * per, s1 = min(steps, s0 + per);
  const TI *wrow[CG], *xrow[T];
  bool wok[CG], xok[T];
#pragma unroll
  for (int c = 0; c < CG; ++c) {
    wok[c] = n0 + 16 * c + l16 < a.N;
    wrow[c] = W + (int64_t)min(n0 + 16 * c + l16, a.N - 1) * a.ldb;
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    xok[t] = r0 + 16 * t + l16 < count;
    xrow[t] = X + (int64_t)min(r0 + 16 * t + l16, count - 1) * a.lda;
  }
  f32x4 acc[CG][T];
#pragma unroll
  for (int c = 0; c < CG; ++c)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[c][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto steps_from = [&](int s, auto uc) __attribute__((always_inline)) {
    constexpr int UN = decltype(uc)::value;
    Piece<TI, SHORT> w[UN][CG], x[UN][T];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int k = (s + u) * STEP + kq;
#pragma unroll
      for (int c = 0; c < CG; ++c) w[u][c].load(wrow[c], k, a.K);
#pragma unroll
      for (int t = 0; t < T; ++t) x[u][t].load(xrow[t], k, a.K);
      // bf16: a step's loads before the next one's, or the compiler moves them to their
      // uses (64 experts of 1408 x 2048, 384 rows: 84 us instead of 77 then; fp32, whose
      // products are dearer: 184 without, 215 with)
      if constexpr (sizeof(TI) == 2) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      if (!WHOLE) {  // clear what reaches past the rows' ends
        const int k = (s + u) * STEP + kq;
#pragma unroll
        for (int c = 0; c < CG; ++c) w[u][c].settle(k, a.K, wok[c]);
#pragma unroll
        for (int t = 0; t < T; ++t) x[u][t].settle(k, a.K, xok[t]);
      }
#pragma unroll
      for (int c = 0; c < CG; ++c)
#pragma unroll
        for (int t = 0; t < T; ++t) FewMfma<TI>::run(acc[c][t], w[u][c].w, x[u][t].w);
    }
  };
  // the last steps by twos and ones: a step past the end that is loaded all the same
  // cost 384 rows of 64 experts of 2048 x 1408 91 us instead of 77
  int s = s0;
  for (; s + U <= s1; s += U) steps_from(s, std::integral_constant<int, U>{});
  if constexpr (U > 2)
    if (s + 2 <= s1) {
      steps_from(s, std::integral_constant<int, 2>{});
      s += 2;
    }
  if constexpr (U > 1)
    if (s < s1) steps_from(s, std::integral_constant<int, 1>{});
  // the upper half of the parts of K to the lower half, until one is left
#pragma unroll
  for (int h = 4; h >= 1; h >>= 1) {
    if (wave >= h && wave < 2 * h) {
#pragma unroll
      for (int i = 0; i < T * CG; ++i) part[wave - h][i][lane] = acc[i / T][i % T];
    }
    __syncthreads();
    if (wave < h) {
#pragma unroll
      for (int i = 0; i < T * CG; ++i) acc[i / T][i % T] += part[wave][i][lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int c = 0; c < CG; ++c) {
    const int n = n0 + 16 * c + 4 * (lane >> 4);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if (!xok[t]) continue;
      TO* y = Y + (int64_t)(r0 + 16 * t + l16) * a.ldo + n;
      const f32x4 v = acc[c][t];
      if (n + 4 <= a.N) {
        if constexpr (sizeof(TO) == 2)
          as_global(reinterpret_cast<u32x2_e2x*>(y))->v = u32x2{pack2<TO>(v[0], v[1]), pack2<TO>(v[2], v[3])};
        else
          as_global(reinterpret_cast<f32x4_e4*>(y))->v = v;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < a.N) as_global(y)[e] = from_f32<TO>(v[e]);
      }
    }
  }
}

// WHOLE: K a multiple of a step.  Rows and channels past the end then repeat the
// last ones, and their results are dropped: a result takes no value of
// another row or channel.  T: tiles of 16 rows, CG: groups of 16 channels at a
// time; U: steps of K in flight.
template <int T, int CG, int U, bool WHOLE, typename TI, typename TO>
__global__ __launch_bounds__(512) void experts_few_kernel(const ExpertsArgs a) {
  __shared__ f32x4 part[4][T * CG][64];
  const int lane = threadIdx.x & 63;
  // the j-th expert with rows
  int left = blockIdx.y, e = -1, begin = 0, count = 0;
  for (int c = 0; c < a.experts; c += 64) {
    ExpertRows r = {0, 0};
    if (c + lane < a.experts) r = experts_rows(a, c + lane);
    const uint64_t some = __ballot(r.count > 0);
    const int n = __popcll(some);
    if (left < n) {
      // its place among the bits: how many set bits lie below each lane's
      const int below = __popcll(some & ((1ull << lane) - 1));
      const int l = __builtin_amdgcn_readfirstlane(__builtin_ctzll(__ballot((some >> lane & 1) && below == left)));
      e = c + l;
      begin = __builtin_amdgcn_readlane(r.begin, l);
      count = __builtin_amdgcn_readlane(r.count, l);
      break;
    }
    left -= n;
  }
  if (e < 0) return;
  const TI* W = static_cast<const TI*>(a.B) + (int64_t)e * a.se;
  const TI* X = static_cast<const TI*>(a.A) + (int64_t)begin * a.lda;
  TO* Y = static_cast<TO*>(a.o) + (int64_t)begin * a.ldo;
  const int n0 = (int)blockIdx.x * (16 * CG);
  if constexpr (!WHOLE) {
    if (a.K < 16 / (int)sizeof(TI)) {  // rows shorter than a piece
      for (int r0 = 0; r0 < count; r0 += 16 * T) experts_few_rows<T, CG, 1, false, true, T * CG, TI, TO>(a, W, X, Y, n0, r0, count, part);
      return;
    }
  }
  if (T == 2 && count <= 16) {  // one tile of rows: 64 experts of 1408 x 2048, 384 rows 74 us instead of 78
    experts_few_rows<1, CG, U, WHOLE, false, T * CG, TI, TO>(a, W, X, Y, n0, 0, count, part);
    return;
  }
  for (int r0 = 0; r0 < count; r0 += 16 * T) experts_few_rows<T, CG, U, WHOLE, false, T * CG, TI, TO>(a, W, X, Y, n0, r0, count, part);
}

}  // namespace muon
