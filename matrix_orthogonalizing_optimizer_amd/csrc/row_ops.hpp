// Row operators on gfx950: norms, their gradients, and 8-bit rows.
//
// Per row x of `cols` values,
//   mu = mean(x) or 0,  r = 1 / sqrt(mean((x - mu)^2) + eps),  h = (x - mu) r,
//   y = h gamma + beta;
//   g = dy gamma,  dx = r (g - mean(g) - h mean(g h)),
//   dgamma = sum_rows dy h,  dbeta = sum_rows dy;
//   8-bit rows: s = 2^e with max|y| <= 127 s, q = rne(y / s).
// All of it is bound by HBM: a row is read once and kept in registers (fp32)
// by a group of G threads: a part of a wave or a wave up to 1024 columns (no
// barrier), 256 to 1024 threads with one or two pieces of 8 columns each above.
// Rows longer than that allows are read again for each pass.
#pragma once

#include "device_common.hpp"
#include "kernel_args.hpp"

namespace muon {

constexpr int ROW_VE = 8;  // columns per piece

// Vectors at the alignment of their elements only: global accesses may be
// unaligned on gfx950, so rows of odd widths and odd starts take the same
// path as aligned ones.
struct __attribute__((packed, aligned(2))) u32x4_e2 {
  u32x4 v;
};
struct __attribute__((packed, aligned(4))) f32x4_e4 {
  f32x4 v;
};

template <typename T> __device__ __forceinline__ void row_load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    const u32x4 w = as_global(reinterpret_cast<const u32x4_e2*>(p))->v;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = __builtin_bit_cast(float, (e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
  } else {
    const f32x4 a = as_global(reinterpret_cast<const f32x4_e4*>(p))->v;
    const f32x4 b = as_global(reinterpret_cast<const f32x4_e4*>(p + 4))->v;
#pragma unroll
    for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[e + 4] = b[e]; }
  }
}

template <typename T> __device__ __forceinline__ void row_store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack2<T>(v[2 * j], v[2 * j + 1]);
    as_global(reinterpret_cast<u32x4_e2*>(p))->v = w;
  } else {
    as_global(reinterpret_cast<f32x4_e4*>(p))->v = f32x4{v[0], v[1], v[2], v[3]};
    as_global(reinterpret_cast<f32x4_e4*>(p + 4))->v = f32x4{v[4], v[5], v[6], v[7]};
  }
}

// Piece at column c of a row of `cols`: columns past the end read as zero
// and are not written.
template <typename T> __device__ __forceinline__ void piece_load(const T* row, int c, int cols, float (&v)[8]) {
  if (c + 8 <= cols) {
    row_load8(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? to_f32(as_global(row)[c + e]) : 0.f;
  }
}

// 8 elements of a row as they lie in memory, loaded and settled apart: what is
// under way takes a 16-bit row half the registers of its fp32 values, and no
// branch stands behind the load.  (A branch that clears the registers of the
// lanes past the row's end waits for the loads of the others: 8192 x 2040
// bf16, whose last wave is partly past the end, norm backward 38 against 28 us
// of 8192 x 2048.)  A piece that reaches past the end loads the row's last 8
// elements, and settle() moves its own to the front and clears the others.
// SHORT: rows may have less than 8 elements, which are loaded one by one.
template <typename T, bool SHORT> struct RowRaw {
  static constexpr int PER = 4 / sizeof(T), NW = 8 / PER;  // elements per register, registers
  uint32_t w[NW];
  __device__ __forceinline__ void load(const T* row, int c, int cols) {
    if (!SHORT || cols >= 8) {
      const T* p = row + min(c, cols - 8);
      if constexpr (sizeof(T) == 2) {
        const u32x4 a = as_global(reinterpret_cast<const u32x4_e2*>(p))->v;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = a[j];
      } else {
        const f32x4 a = as_global(reinterpret_cast<const f32x4_e4*>(p))->v;
        const f32x4 b = as_global(reinterpret_cast<const f32x4_e4*>(p + 4))->v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j] = __builtin_bit_cast(uint32_t, (float)a[j]);
          w[j + 4] = __builtin_bit_cast(uint32_t, (float)b[j]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NW; ++j) w[j] = 0u;
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (c + e < cols) {
          if constexpr (sizeof(T) == 2)
            w[e >> 1] |= (uint32_t)as_global(reinterpret_cast<const uint16_t*>(row))[c + e] << (16 * (e & 1));
          else
            w[e] = as_global(reinterpret_cast<const uint32_t*>(row))[c + e];
        }
    }
  }
  __device__ __forceinline__ void settle(int c, int cols) {
    if ((SHORT && cols < 8) || c + 8 <= cols) return;
    const int off = min(c + 8 - cols, 8);  // elements to drop at the front
    const int regs = off / PER;
    // registers by powers of two, then half a register
#pragma unroll
    for (int b = NW; b >= 1; b >>= 1) {
      const bool take = (regs & b) != 0;
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        const uint32_t from = j + b < NW ? w[j + b] : 0u;
        w[j] = take ? from : w[j];
      }
    }
    if constexpr (PER == 2) {
      const bool take = (off & 1) != 0;
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        const uint32_t from = (w[j] >> 16) | (j + 1 < NW ? w[j + 1] << 16 : 0u);
        w[j] = take ? from : w[j];
      }
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 2)
      return __builtin_bit_cast(float, (e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
    else
      return __builtin_bit_cast(float, w[e]);
  }
};
// Piece at column c of a row of at least 8 elements that may be overwritten
// from here on: what reaches past the row's end is taken from `last`, the
// thread's last piece as it was loaded and settled before.  A select in the
// load's registers, so no branch stands behind the load.
template <typename T>
__device__ __forceinline__ void row_piece_reload(const T* row, int c, int cols, const RowRaw<T, false>& last,
                                                 float (&v)[8]) {
  RowRaw<T, false> x = last;
  if (c + 8 <= cols) x.load(row, c, cols);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = x.get(e);
}
// A piece of a row of at least 8 elements, widened.
template <typename T> __device__ __forceinline__ void row_piece_load(const T* row, int c, int cols, float (&v)[8]) {
  RowRaw<T, false> x;
  x.load(row, c, cols);
  x.settle(c, cols);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = x.get(e);
}
// Piece of a vector whose dtype is known at run time only.
template <bool SHORT = true>
__device__ __forceinline__ void vec_load(const void* p, int dt, int c, int cols, float (&v)[8]) {
  if constexpr (SHORT) {
    if (dt == DT_F32) piece_load(static_cast<const float*>(p), c, cols, v);
    else piece_load(static_cast<const bf16*>(p), c, cols, v);
  } else {
    if (dt == DT_F32) row_piece_load(static_cast<const float*>(p), c, cols, v);
    else row_piece_load(static_cast<const bf16*>(p), c, cols, v);
  }
}
template <typename T> __device__ __forceinline__ void piece_store(T* row, int c, int cols, const float (&v)[8]) {
  if (c + 8 <= cols) {
    row_store8(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < cols) as_global(row)[c + e] = from_f32<T>(v[e]);
  }
}

// Workgroup number: grids of rows are two-dimensional, since a launch holds
// fewer than 2^32 threads along x.
__device__ __forceinline__ int64_t row_block() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Deterministic sums over a group of G threads (a part of a wave, or whole
// waves): butterfly inside a wave, waves in order.  G > 64: all threads of the
// workgroup take part and `red` is one of two alternating buffers, so one
// barrier per sum is enough (a wave writes a buffer again only after the
// barrier of the sum in between, which every reader of it has passed).
template <int G, int N> struct GroupRed {
  float slot[2][G < 64 ? 1 : G / 64][N];
};
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], GroupRed<G, N>& red, int buf) {
#pragma unroll
  for (int off = (G < 64 ? G : 64) / 2; off >= 1; off >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], off, 64);
  if constexpr (G > 64) {
    const int w = (threadIdx.x % G) >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) red.slot[buf][w][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if constexpr (G <= 256) {
        float s = red.slot[buf][0][k];
#pragma unroll
        for (int i = 1; i < G / 64; ++i) s += red.slot[buf][i][k];
        v[k] = s;
      } else {  // many waves: one read per lane and a butterfly, not a register per wave
        v[k] = red.slot[buf][threadIdx.x & (G / 64 - 1)][k];
#pragma unroll
        for (int off = G / 128; off >= 1; off >>= 1) v[k] += __shfl_xor(v[k], off, 64);
      }
    }
  }
}
template <int G>
__device__ __forceinline__ uint32_t group_umax(uint32_t v, GroupRed<G, 1>& red, int buf) {
#pragma unroll
  for (int off = (G < 64 ? G : 64) / 2; off >= 1; off >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, off, 64);
    v = v > o ? v : o;
  }
  if constexpr (G > 64) {
    const int w = (threadIdx.x % G) >> 6;
    if ((threadIdx.x & 63) == 0) red.slot[buf][w][0] = __builtin_bit_cast(float, v);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < G / 64; ++i) {
      const uint32_t o = __builtin_bit_cast(uint32_t, red.slot[buf][i][0]);
      v = v > o ? v : o;
    }
  }
  return v;
}

// Magnitude bits of a float: as unsigned integers they order like the
// magnitudes, infinities above every finite value and NaNs above those, so
// one integer maximum finds both the scale and a non-finite row.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

// Scale of a row whose largest magnitude has the bits m: the smallest power
// of two with max <= 127 s.  max = f 2^k, 1 <= f < 2: s = 2^(k - 6) if
// f <= 127/64, else 2^(k - 5); 127/64 has the fraction bits 0x7e0000, and
// adding 0x1ffff carries into the exponent exactly above it.  inv = 1 / s is
// a normal number (s is at least 2^-126 and below 2^123).
// lim: 127, or 63 for the largest scale, 2^122, where 64 s is out of range.
__device__ __forceinline__ void row_scale(uint32_t m, float& s, float& inv, float& lim) {
  int e = (int)((m + 0x1ffffu) >> 23) - 6;
  e = e < 1 ? 1 : e;
  s = __builtin_bit_cast(float, (uint32_t)e << 23);
  inv = __builtin_bit_cast(float, (uint32_t)(254 - e) << 23);
  lim = e == 122 + 127 ? 63.f : 127.f;
  if (m >= 0x7f800000u) {
    s = __builtin_bit_cast(float, 0x7fc00000u);
    inv = 0.f;
  }
}
// A sum of products of 8-bit values times the scale s of its row and a second
// scale c, v = sum * a * c * b with s = a b.  Left to right, sum * s leaves
// fp32's range from s = 2^97 on (|sum| < 2^31) though a small c may bring the
// result back: there s gives 2^32 to b.  Nothing is lost below: c is at least
// 2^-126, so from s = 2^96 on sum * a * c is zero or at least 2^-62.  Below, a is s
// and b is 1.
__device__ __forceinline__ void split_scale(float s, float& a, float& b) {
  const bool large = __builtin_fabsf(s) >= 0x1p96f;
  a = large ? s * 0x1p-32f : s;
  b = large ? 0x1p32f : 1.f;
}
// 8 values -> 8 bytes; x * inv is exact (a power of two) wherever it matters:
// what falls below the normal range rounds to 0 either way.
__device__ __forceinline__ u32x2 quant8(const float (&v)[8], float inv, float lim, bool fine) {
  u32x2 w = {0u, 0u};
  if (fine) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = __builtin_amdgcn_fmed3f(__builtin_rintf(v[e] * inv), -lim, lim);
      w[e >> 2] |= ((uint32_t)(int)r & 0xffu) << (8 * (e & 3));
    }
  }
  return w;
}

enum : int { ROW_COPY = 2 };  // next to MUON_NORM_LAYER = 0 and MUON_NORM_RMS = 1: no norm, quantize only

// Norm forward / quantize, a row per group of G threads, NV pieces each.
// Two reductions for the layer norm (the variance is taken around the mean
// from registers, not as a difference of sums), one more for the 8-bit scale.
template <typename T, int KIND, int G, int NV>
__global__ __launch_bounds__(G < 256 ? 256 : G) void row_forward_kernel(const RowArgs a) {
  constexpr int RPW = G < 256 ? 256 / G : 1;  // rows per workgroup
  __shared__ GroupRed<G, 1> red;
  const int t = threadIdx.x % G;
  const int64_t row = row_block() * RPW + threadIdx.x / G;
  if (row >= a.rows) return;  // whole groups; no barrier below when G < 256
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  float v[NV][8];
  RowRaw<T, G == 8> raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) raw[i].load(x, (i * G + t) * ROW_VE, a.cols);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    raw[i].settle((i * G + t) * ROW_VE, a.cols);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = raw[i].get(e);
  }
  if constexpr (KIND != ROW_COPY) {
    float mean = 0.f;
    if constexpr (KIND == 0) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += v[i][e];
      group_sum<G, 1>(s, red, 0);
      mean = s[0] / (float)a.cols;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = (i * G + t) * ROW_VE + e < a.cols ? v[i][e] - mean : 0.f;
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] = fmaf(v[i][e], v[i][e], s[0]);
    group_sum<G, 1>(s, red, 1);
    const float r = 1.f / sqrtf(s[0] / (float)a.cols + a.eps);
    if (t == 0) {
      if (a.mean) as_global(a.mean)[row] = mean;
      if (a.rstd) as_global(a.rstd)[row] = r;
    }
    if (!a.y && !a.scale) return;  // uniform
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + t) * ROW_VE;
      float w[8];
      vec_load<G == 8>(a.gamma, a.vec_dtype, c, a.cols, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * r * w[e];
      if (a.beta) {
        vec_load<G == 8>(a.beta, a.vec_dtype, c, a.cols, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] += w[e];
      }
    }
    if (a.y) {
      T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
      for (int i = 0; i < NV; ++i) piece_store(y, (i * G + t) * ROW_VE, a.cols, v[i]);
    }
  }
  if (a.scale) {  // 8-bit rows (q may be null when there are no columns)
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // a NaN's padding products (0 * NaN) sit in columns past the end
        const uint32_t b = (i * G + t) * ROW_VE + e < a.cols ? mag_bits(v[i][e]) : 0u;
        m = m > b ? m : b;
      }
    m = group_umax<G>(m, red, 0);
    float s, inv, lim;
    row_scale(m, s, inv, lim);
    const bool fine = m < 0x7f800000u;
    if (t == 0) as_global(a.scale)[row] = s;
    int8_t* q = a.q + row * a.ldq;
    const int cpad = (a.cols + 15) & ~15;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + t) * ROW_VE;
      if (c < cpad) *as_global(reinterpret_cast<u32x2*>(q + c)) = quant8(v[i], inv, lim, fine);
    }
  }
}

// The same for rows of any length, which are read again for every pass.  y may
// be x: in the pass that writes, a thread reads only what it alone writes.  Its
// piece at the row's end, which is loaded with columns of its neighbour, is kept
// from the pass before (loading it element by element behind that loop took
// 2048 x 20001 bf16 from 51 to 56 us).
template <typename T, int KIND>
__global__ __launch_bounds__(1024) void row_forward_long_kernel(const RowArgs a) {
  constexpr int G = 1024;
  __shared__ GroupRed<G, 1> red;
  const int t = threadIdx.x;
  const int64_t row = row_block();
  if (row >= a.rows) return;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  float mean = 0.f, r = 1.f;
  RowRaw<T, false> last;
  if constexpr (KIND != ROW_COPY) {
    if constexpr (KIND == 0) {
      float s[1] = {0.f};
      for (int64_t c = (int64_t)t * ROW_VE; c < a.cols; c += G * ROW_VE) {
        float v[8];
        row_piece_load(x, (int)c, a.cols, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += v[e];
      }
      group_sum<G, 1>(s, red, 0);
      mean = s[0] / (float)a.cols;
    }
    float s[1] = {0.f};
    for (int64_t c = (int64_t)t * ROW_VE; c < a.cols; c += G * ROW_VE) {
      last.load(x, (int)c, a.cols);
      last.settle((int)c, a.cols);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = c + e < a.cols ? last.get(e) - mean : 0.f;
        s[0] = fmaf(d, d, s[0]);
      }
    }
    group_sum<G, 1>(s, red, 1);
    r = 1.f / sqrtf(s[0] / (float)a.cols + a.eps);
    if (t == 0) {
      if (a.mean) as_global(a.mean)[row] = mean;
      if (a.rstd) as_global(a.rstd)[row] = r;
    }
    if (!a.y && !a.scale) return;
  }
  auto norm = [&](int64_t c, float (&v)[8]) {
    if constexpr (KIND != ROW_COPY) {
      float w[8];
      vec_load<false>(a.gamma, a.vec_dtype, (int)c, a.cols, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (v[e] - mean) * r * w[e];
      if (a.beta) {
        vec_load<false>(a.beta, a.vec_dtype, (int)c, a.cols, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += w[e];
      }
    }
  };
  float s = 0.f, inv = 0.f, lim = 0.f;
  bool fine = false;
  if (a.scale) {  // 8-bit rows (q may be null when there are no columns)
    uint32_t m = 0;
    for (int64_t c = (int64_t)t * ROW_VE; c < a.cols; c += G * ROW_VE) {
      float v[8];
      row_piece_load(x, (int)c, a.cols, v);
      norm(c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = c + e < a.cols ? mag_bits(v[e]) : 0u;
        m = m > b ? m : b;
      }
    }
    m = group_umax<G>(m, red, 0);
    row_scale(m, s, inv, lim);
    fine = m < 0x7f800000u;
    if (t == 0) as_global(a.scale)[row] = s;
  }
  const int64_t cpad = ((int64_t)a.cols + 15) & ~(int64_t)15;
  for (int64_t c = (int64_t)t * ROW_VE; c < cpad; c += G * ROW_VE) {
    float v[8];  // past the row's end: anything, and not written
    if constexpr (KIND == ROW_COPY) row_piece_load(x, (int)c, a.cols, v);
    else row_piece_reload(x, (int)c, a.cols, last, v);
    norm(c, v);
    if (a.scale) {  // 8-bit rows (q may be null when there are no columns)
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = c + e < a.cols ? v[e] : 0.f;
      *as_global(reinterpret_cast<u32x2*>(a.q + row * a.ldq + c)) = quant8(z, inv, lim, fine);
    }
    if (KIND != ROW_COPY && a.y) piece_store(static_cast<T*>(a.y) + row * a.ldy, (int)c, a.cols, v);
  }
}

// Restore: y = q * scale.  A row per group of G threads, NV pieces of 8
// columns each at a time (8-byte loads, 16- or 32-byte stores).
template <typename T, int G, int NV>
__global__ __launch_bounds__(G < 256 ? 256 : G) void row_restore_kernel(const RestoreArgs a) {
  constexpr int RPW = G < 256 ? 256 / G : 1;
  const int t = threadIdx.x % G;
  const int64_t row = row_block() * RPW + threadIdx.x / G;
  if (row >= a.rows) return;
  const int8_t* q = a.q + row * a.ldq;
  T* y = static_cast<T*>(a.y) + row * a.ldy;
  const float s = as_global(a.scale)[row];
  for (int64_t c0 = (int64_t)t * ROW_VE; c0 < a.cols; c0 += NV * G * ROW_VE) {
    u32x2 w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (c0 + i * G * ROW_VE < a.cols) w[i] = *as_global(reinterpret_cast<const u32x2*>(q + c0 + i * G * ROW_VE));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)(w[i][e >> 2] >> (8 * (e & 3))) * s;
      if (c0 + i * G * ROW_VE < a.cols) piece_store(y, (int)(c0 + i * G * ROW_VE), a.cols, v);
    }
  }
}

// The backward kernels' KIND is that of the norm, and NORM_RMS_BETA for an RMS
// norm whose bias gradient is asked for: the others keep no sum of dy that
// nobody reads (a layer norm needs it for dx's mean in any case).
enum : int { NORM_RMS_BETA = 3 };
constexpr bool norm_sums_dy(int kind) { return kind != 1; }

// Norm backward: workgroups loop over rows; a thread keeps its columns' gamma
// and its sums of dy h and dy in registers over all of them, and the sums go
// to workspace once per workgroup (partials[2][workgroups][cols]).  The next
// row's loads are issued before this row's sums, so that few workgroups
// (and few partial rows) keep enough bytes in flight.
template <typename T, int KIND, int G, int NV>
__global__ __launch_bounds__(G < 256 ? 256 : G) void norm_backward_kernel(const NormBwdArgs a) {
  constexpr int RPW = G < 256 ? 256 / G : 1;
  __shared__ GroupRed<G, 2> red;
  __shared__ float comb[RPW > 1 ? RPW * G * NV * 8 : 1];
  const int t = threadIdx.x % G;
  const int sub = threadIdx.x / G;
  float gam[NV][8], sg[NV][8], sb[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    vec_load<G == 8>(a.gamma, a.vec_dtype, (i * G + t) * ROW_VE, a.cols, gam[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) sg[i][e] = sb[i][e] = 0.f;
  }
  const int64_t stride = (int64_t)gridDim.x * RPW;
  int64_t row = (int64_t)blockIdx.x * RPW + sub;
  RowRaw<T, G == 8> x[NV], dy[NV];
  float r = 0.f, mean = 0.f;
  auto fetch = [&](int64_t at) {
    const T* xp = static_cast<const T*>(a.x) + at * a.ldx;
    const T* dp = static_cast<const T*>(a.dy) + at * a.lddy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i].load(xp, (i * G + t) * ROW_VE, a.cols);
      dy[i].load(dp, (i * G + t) * ROW_VE, a.cols);
    }
    r = as_global(a.rstd)[at];
    if (KIND == 0) mean = as_global(a.mean)[at];
  };
  if (row < a.rows) fetch(row);
  int buf = 0;
  while (row < a.rows) {
    const int64_t next = row + stride;
    RowRaw<T, G == 8> cx[NV], cd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cx[i] = x[i];
      cd[i] = dy[i];
    }
    const float cr = r, cm = mean;
    if (next < a.rows) fetch(next);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cx[i].settle((i * G + t) * ROW_VE, a.cols);
      cd[i].settle((i * G + t) * ROW_VE, a.cols);
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float h = (cx[i].get(e) - cm) * cr, d = cd[i].get(e);
        sg[i][e] = fmaf(d, h, sg[i][e]);
        if (norm_sums_dy(KIND)) sb[i][e] += d;
        const float g = d * gam[i][e];
        s[0] = fmaf(g, h, s[0]);
        if (KIND == 0) s[1] += g;
      }
    group_sum<G, 2>(s, red, buf);
    buf ^= 1;
    const float c2 = s[0] / (float)a.cols, c1 = KIND == 0 ? s[1] / (float)a.cols : 0.f;
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + t) * ROW_VE;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float h = (cx[i].get(e) - cm) * cr;
        o[e] = cr * (cd[i].get(e) * gam[i][e] - c1 - h * c2);
      }
      if (c < a.cols) piece_store(dx, c, a.cols, o);
    }
    row = next;
  }
  if (!a.partials) return;
  auto put = [&](float (&v)[NV][8], int which) {
    float* p = a.partials + ((int64_t)which * gridDim.x + blockIdx.x) * a.cols;
    if constexpr (RPW > 1) {  // the workgroup's rows join in order
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) comb[((sub * NV + i) * 8 + e) * G + t] = v[i][e];
      __syncthreads();
      if (sub == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float s = comb[(i * 8 + e) * G + t];
#pragma unroll
            for (int w = 1; w < RPW; ++w) s += comb[((w * NV + i) * 8 + e) * G + t];
            v[i][e] = s;
          }
      }
      __syncthreads();
      if (sub != 0) return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * G + t) * ROW_VE < a.cols) piece_store(p, (i * G + t) * ROW_VE, a.cols, v[i]);
  };
  put(sg, 0);
  if constexpr (norm_sums_dy(KIND)) put(sb, 1);
}

// Rows above NORM_BWD_MAX_COLS (a thread would hold too much of one): dx with
// the row read twice, and the column sums on their own.
template <typename T, int KIND>
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(const NormBwdArgs a) {
  constexpr int G = 1024;
  __shared__ GroupRed<G, 2> red;
  const int t = threadIdx.x;
  const int64_t row = row_block();
  if (row >= a.rows) return;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
  T* dx = static_cast<T*>(a.dx) + row * a.lddx;
  const float r = as_global(a.rstd)[row];
  const float mean = KIND == 0 ? as_global(a.mean)[row] : 0.f;
  float s[2] = {0.f, 0.f};
  RowRaw<T, false> last;  // dx may be dy (see row_forward_long_kernel)
  for (int64_t c = (int64_t)t * ROW_VE; c < a.cols; c += G * ROW_VE) {
    float h[8], w[8];
    row_piece_load(x, (int)c, a.cols, h);
    last.load(dy, (int)c, a.cols);
    last.settle((int)c, a.cols);
    vec_load<false>(a.gamma, a.vec_dtype, (int)c, a.cols, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float ge = last.get(e) * w[e];
      s[0] = fmaf(ge, (h[e] - mean) * r, s[0]);
      s[1] += ge;
    }
  }
  group_sum<G, 2>(s, red, 0);
  const float c2 = s[0] / (float)a.cols, c1 = KIND == 0 ? s[1] / (float)a.cols : 0.f;
  for (int64_t c = (int64_t)t * ROW_VE; c < a.cols; c += G * ROW_VE) {
    float h[8], g[8], w[8];
    row_piece_load(x, (int)c, a.cols, h);
    row_piece_reload(dy, (int)c, a.cols, last, g);
    vec_load<false>(a.gamma, a.vec_dtype, (int)c, a.cols, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = r * (g[e] * w[e] - c1 - (h[e] - mean) * r * c2);
    piece_store(dx, (int)c, a.cols, g);
  }
}

// partials[2][gridDim.y][cols]: 8 columns per thread, every gridDim.y-th row.
template <typename T, int KIND>
__global__ __launch_bounds__(256) void norm_columns_long_kernel(const NormBwdArgs a) {
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * ROW_VE;
  if (c >= a.cols) return;
  float sg[8] = {}, sb[8] = {};
#pragma unroll 2
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    float g[8], x[8];
    row_piece_load(static_cast<const T*>(a.dy) + row * a.lddy, (int)c, a.cols, g);
    row_piece_load(static_cast<const T*>(a.x) + row * a.ldx, (int)c, a.cols, x);
    const float mean = KIND == 0 ? as_global(a.mean)[row] : 0.f, r = as_global(a.rstd)[row];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sg[e] = fmaf(g[e], (x[e] - mean) * r, sg[e]);
      sb[e] += g[e];
    }
  }
  piece_store(a.partials + (int64_t)blockIdx.y * a.cols, (int)c, a.cols, sg);
  if (norm_sums_dy(KIND)) piece_store(a.partials + ((int64_t)gridDim.y + blockIdx.y) * a.cols, (int)c, a.cols, sb);
}

// Joins the workgroups' column sums in order: 64 columns per workgroup, 16
// waves each a sixteenth of the partials.
template <typename TV>
__global__ __launch_bounds__(1024) void norm_columns_join_kernel(const JoinArgs a) {
  __shared__ float part[16][64];
  const int which = blockIdx.y;
  TV* out = static_cast<TV*>(which == 0 ? a.dgamma : a.dbeta);
  if (!out) return;  // uniform
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + l;
  const float* p = a.partials + (int64_t)which * a.parts * a.cols;
  const int per = (a.parts + 15) / 16;
  const int hi = min(a.parts, (w + 1) * per);
  float s = 0.f;
  if (c < a.cols) {
#pragma unroll 8
    for (int i = w * per; i < hi; ++i) s += as_global(p)[(int64_t)i * a.cols + c];
  }
  part[w][l] = s;
  __syncthreads();
  if (w == 0 && c < a.cols) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][l];
    if (a.accumulate) s += to_f32(as_global(out)[c]);
    as_global(out)[c] = from_f32<TV>(s);
  }
}

}  // namespace muon
