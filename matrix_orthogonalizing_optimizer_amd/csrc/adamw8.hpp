// AdamW on moments kept in 8 bits, gfx950: one grouped launch over the tensors
// of a step.
//
// Per element, in fp32 with every operation rounded by itself (no fused
// multiply-add in the moments, so that their codes follow from the formula):
//   m' = m + (1 - b1) (g - m),   v' = v + (1 - b2) (g g - v)
//   w' = w (1 - lr wd) - step m' / (eps + sqrt(v'))
// w' uses m' and v' as computed; what is kept of them is 8 bits each.
//
// Codes.  The bits u(x) of a float x >= 0 grow with x, and u >> 20 is its
// exponent and 3 bits of its mantissa.  A block of 256 elements keeps one
// 16-bit offset
//   o = max(0, ceil(max u / 2^20) - K),   K = 127 (m), 255 (v)
// and per element k = floor((u + r) / 2^20) - o, which stands for the float of
// bits (k + o) << 20, or zero where k is 0; the code of m has its sign in bit 7.
// So the largest value of a block always fits, steps are 1/8 to 1/16 of a value,
// and codes reach 2^15.9 (m) and 2^31.9 (v, the square root's 2^15.9) down.
// r is uniform in [0, 2^20): a value goes up or down with the probabilities
// that keep its mean.  Rounding to nearest would freeze v: 1 - b2 = 0.05 takes
// at most 5% off v in a step, and half a step of the codes is 3 to 6% of it.
// It is v and not its root that is rounded, since the error of a root's mean
// would add up over 1 / (1 - b2) steps.
// Below the smallest code lo, m becomes lo with probability m / lo and else 0
// (its mean is kept), v becomes lo: a second moment of zero would make the
// update as large as m / eps.
// r is 16 bits of a hash of the step and of the element's index, so a step
// gives the same result wherever and however often it is computed.
//
// Bound by HBM: w and g once, two codes read and written, 10 bytes per bf16
// element against 22 with fp32 moments.  A wave owns blocks of 256 elements, 4
// per lane: one load or store instruction per array and block, and the block's
// largest value is a reduction over the wave's registers.  128256 x 4096 in bf16:
// 902 us a call, 5.8 TB/s; traced over 23 calls in a row 897 to 1006 us, 944 on
// average (3.2 GB read and 2.1 GB written by the counters, what it cannot do
// without).  50257 x 768 and 74 vectors: 66 us, 5.9 TB/s with what the caches keep
// of the step before.
#pragma once

#include "consts.hpp"
#include "kernel_args.hpp"
#include "row_ops.hpp"

namespace muon {

constexpr uint32_t A8_NAN = 0x7fc00000u;

// A 32-bit mixer: shifts fold the high bits down, the odd factors (fractional
// bits of the square roots of 2 and 3) carry low bits up.
__host__ __device__ __forceinline__ uint32_t adamw8_mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6a09e667u;
  x ^= x >> 15;
  x *= 0xbb67ae85u;
  return x ^ (x >> 16);
}
// The step's part of the hash.
inline uint32_t adamw8_key(int64_t step) {
  return adamw8_mix((uint32_t)step ^ adamw8_mix((uint32_t)((uint64_t)step >> 32)));
}
// Hash of group q (4 elements) of a block's 64; the block's part of it is uniform.
__device__ __forceinline__ uint32_t adamw8_hash(int64_t block, int q, uint32_t key) {
  const uint64_t group = (uint64_t)block * 64;
  return adamw8_mix(((uint32_t)group + (uint32_t)q) ^ ((uint32_t)(group >> 32) * 0x9e3779b1u) ^ key);
}
// Random bits of element e of a group: low half for m, high half for v.
__device__ __forceinline__ uint32_t adamw8_turn(uint32_t h, int e) { return e ? (h >> (8 * e)) | (h << (32 - 8 * e)) : h; }

// Largest of the wave's values in a scalar register: rows of 16 lanes, then
// across rows (lanes without a source see 0).
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  auto step = [&](auto ctl) {
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctl)::value, 0xf, 0xf, false));
  };
  step(std::integral_constant<int, 0x111>{});  // row_shr:1
  step(std::integral_constant<int, 0x112>{});
  step(std::integral_constant<int, 0x114>{});
  step(std::integral_constant<int, 0x118>{});
  step(std::integral_constant<int, 0x142>{});  // row_bcast:15
  step(std::integral_constant<int, 0x143>{});  // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

__device__ __forceinline__ uint32_t adamw8_offset(uint32_t top, int K) {
  return (uint32_t)max(0, (int)((top + 0xfffffu) >> 20) - K);
}
// |x| as bits; a NaN, whatever its payload, as one that rounding keeps a NaN.
__device__ __forceinline__ uint32_t adamw8_bits(float x) {
  return x == x ? __builtin_bit_cast(uint32_t, x) & 0x7fffffffu : A8_NAN;
}
// The same for the result of an arithmetic instruction, whose NaNs are quiet.
__device__ __forceinline__ uint32_t adamw8_result_bits(float x) {
  return min(__builtin_bit_cast(uint32_t, x) & 0x7fffffffu, A8_NAN);
}
// Code of |m| for values from the smallest code up.
__device__ __forceinline__ uint32_t adamw8_round_m(uint32_t u, uint32_t h, uint32_t off) {
  return ((u + ((h & 0xffffu) << 4)) >> 20) - off;
}
__device__ __forceinline__ uint32_t adamw8_encode_m(float x, uint32_t u, uint32_t h, uint32_t off) {
  const uint32_t r = h & 0xffffu, first = (off + 1) << 20;
  const float lo = __builtin_bit_cast(float, first);
  const uint32_t low = __builtin_fabsf(x) > lo * fmaf((float)r, 0x1p-16f, 0x1p-17f) ? 1u : 0u;
  return (u < first ? low : adamw8_round_m(u, h, off)) | ((__builtin_bit_cast(uint32_t, x) >> 24) & 0x80u);
}
__device__ __forceinline__ uint32_t adamw8_encode_v(uint32_t u, uint32_t h, uint32_t off) {
  // a value below the smallest code rounds to -off, ..., 0 or 1
  return (uint32_t)max((int)((u + ((h >> 12) & 0xffff0u)) >> 20) - (int)off, (int)min(u, 1u));
}
__device__ __forceinline__ float adamw8_decode_m(uint32_t c, uint32_t off) {
  const uint32_t k = c & 127u;
  return __builtin_bit_cast(float, (k ? (k + off) << 20 : 0u) | ((c & 128u) << 24));
}
__device__ __forceinline__ float adamw8_decode_v(uint32_t c, uint32_t off) {
  return __builtin_bit_cast(float, c ? (c + off) << 20 : 0u);
}

// The buffer of one moment: codes of whole blocks, then a 16-bit offset per block.
__device__ __forceinline__ int64_t adamw8_blocks(int64_t numel) { return (numel + ADAMW8_BLOCK - 1) / ADAMW8_BLOCK; }

// Loads and stores, past the caches' replacement order (STREAM) or not.
template <bool STREAM, typename P> __device__ __forceinline__ auto adamw8_get(P p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool STREAM, typename P, typename X> __device__ __forceinline__ void adamw8_put(P p, X x) {
  if constexpr (STREAM) __builtin_nontemporal_store(x, p);
  else *p = x;
}

// 4 elements of T at the alignment of one (global accesses may be unaligned).
typedef u32x2 u32x2_u __attribute__((aligned(2)));
typedef f32x4 f32x4_u __attribute__((aligned(4)));
template <typename T, bool STREAM> struct Four;
template <bool STREAM> struct Four<bf16, STREAM> {
  u32x2 w;
  __device__ __forceinline__ void load(const bf16* p) {
    const auto* q = (const __attribute__((address_space(1))) u32x2_u*)p;
    if constexpr (STREAM) w = __builtin_nontemporal_load(q);
    else w = *q;
  }
  __device__ __forceinline__ void store(bf16* p) const {
    auto* q = (__attribute__((address_space(1))) u32x2_u*)p;
    if constexpr (STREAM) __builtin_nontemporal_store(w, q);
    else *q = w;
  }
  __device__ __forceinline__ float get(int e) const {
    return __builtin_bit_cast(float, (e & 1) ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[4]) { w = u32x2{pack2<bf16>(v[0], v[1]), pack2<bf16>(v[2], v[3])}; }
};
template <bool STREAM> struct Four<float, STREAM> {
  f32x4 w;
  __device__ __forceinline__ void load(const float* p) {
    const auto* q = (const __attribute__((address_space(1))) f32x4_u*)p;
    if constexpr (STREAM) w = __builtin_nontemporal_load(q);
    else w = *q;
  }
  __device__ __forceinline__ void store(float* p) const {
    auto* q = (__attribute__((address_space(1))) f32x4_u*)p;
    if constexpr (STREAM) __builtin_nontemporal_store(w, q);
    else *q = w;
  }
  __device__ __forceinline__ float get(int e) const { return w[e]; }
  __device__ __forceinline__ void set(const float (&v)[4]) { w = f32x4{v[0], v[1], v[2], v[3]}; }
};

// One element; m and v are left as computed, before they are rounded.
// EXACT: root and quotient correctly rounded; otherwise by the instructions of
// 1 ulp, 24 instructions less.  Those take a v under 2^-126 as zero: next to an eps of
// 2^-38 or more its root is less than half an ulp.
template <bool EXACT> __device__ __forceinline__ float adamw8_elem(float w, float g, float& m, float& v, const Adamw8Args& a) {
  {
#pragma clang fp contract(off)
    m = m + (g - m) * a.one_minus_b1;
    v = v + (g * g - v) * a.one_minus_b2;
  }
  const float q = EXACT ? m / (a.eps + sqrtf(v)) : m * __builtin_amdgcn_rcpf(a.eps + __builtin_amdgcn_sqrtf(v));
  return w * a.keep - a.step * q;
}

// Blocks first, ..., first + NB - 1 of one tensor.  WHOLE: all of them lie in
// the tensor, so the loads of all go out first and no branch stands between
// them.  Otherwise NB is 1, and lanes past the tensor's end take zeros and
// write nothing.
template <typename T, int NB, bool WHOLE, bool EXACT, bool STREAM>
__device__ __forceinline__ void adamw8_tile(const Adamw8Desc& d, int64_t first, const Adamw8Args& a) {
  const int lane = threadIdx.x & 63;
  const int64_t i0 = first * ADAMW8_BLOCK + 4 * lane;
  T* W = static_cast<T*>(d.w) + i0;
  const T* G = static_cast<const T*>(d.g) + i0;
  auto* M = as_global(reinterpret_cast<uint32_t*>(d.m + i0));
  auto* V = as_global(reinterpret_cast<uint32_t*>(d.v + i0));
  const int64_t codes = adamw8_blocks(d.numel) * ADAMW8_BLOCK;
  auto* mo = as_global(reinterpret_cast<uint16_t*>(d.m + codes)) + first;
  auto* vo = as_global(reinterpret_cast<uint16_t*>(d.v + codes)) + first;
  static_assert(WHOLE || NB == 1, "one block at the tensor's end");
  const int64_t rest = d.numel - i0;
  const int left = WHOLE || rest >= 4 ? 4 : rest > 0 ? (int)rest : 0;  // of the lane's elements, those in the tensor
  Four<T, STREAM> w[NB], g[NB];
  uint32_t mc[NB], vc[NB], om[NB], ov[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (left == 4) {
      g[b].load(G + b * ADAMW8_BLOCK);
      w[b].load(W + b * ADAMW8_BLOCK);
    } else {
      float x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = e < left ? to_f32(as_global(W)[e]) : 0.f;
        y[e] = e < left ? to_f32(as_global(G)[e]) : 0.f;
      }
      w[b].set(x);
      g[b].set(y);
    }
    mc[b] = adamw8_get<STREAM>(M + b * (ADAMW8_BLOCK / 4));
    vc[b] = adamw8_get<STREAM>(V + b * (ADAMW8_BLOCK / 4));
    om[b] = mo[b];
    ov[b] = vo[b];
  }
  float x[NB][4], m[NB][4], v[NB][4];
  uint32_t um[NB], uv[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    um[b] = uv[b] = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m[b][e] = adamw8_decode_m(mc[b] >> (8 * e) & 255u, om[b]);
      v[b][e] = adamw8_decode_v(vc[b] >> (8 * e) & 255u, ov[b]);
      x[b][e] = adamw8_elem<EXACT>(w[b].get(e), g[b].get(e), m[b][e], v[b][e], a);
      if (!WHOLE && e >= left) m[b][e] = v[b][e] = 0.f;
      um[b] = max(um[b], adamw8_result_bits(m[b][e]));
      uv[b] = max(uv[b], adamw8_result_bits(v[b][e]));
    }
  }
  uint32_t nm[NB], nv[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    nm[b] = adamw8_offset(wave_max(um[b]), 127);
    nv[b] = adamw8_offset(wave_max(uv[b]), 255);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const uint32_t h = adamw8_hash(first + b, lane, a.key);
    uint32_t cm = 0, cv = 0;
    bool low = false;  // a first moment under the smallest code: few blocks have any
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t r = adamw8_turn(h, e), u = adamw8_result_bits(m[b][e]);
      low |= u < (nm[b] + 1) << 20;
      cm |= (adamw8_round_m(u, r, nm[b]) | ((__builtin_bit_cast(uint32_t, m[b][e]) >> 24) & 0x80u)) << (8 * e);
      cv |= adamw8_encode_v(adamw8_result_bits(v[b][e]), r, nv[b]) << (8 * e);
    }
    if (__ballot(low)) {
      cm = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        cm |= adamw8_encode_m(m[b][e], adamw8_result_bits(m[b][e]), adamw8_turn(h, e), nm[b]) << (8 * e);
    }
    if (left == 4) {
      w[b].set(x[b]);
      w[b].store(W + b * ADAMW8_BLOCK);
    } else {
      // the codes of the last block behind the tensor's end stay as they are
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) as_global(W)[e] = from_f32<T>(x[b][e]);
      const uint32_t mine = (1u << (8 * left)) - 1u;
      cm = (cm & mine) | (mc[b] & ~mine);
      cv = (cv & mine) | (vc[b] & ~mine);
    }
    adamw8_put<STREAM>(M + b * (ADAMW8_BLOCK / 4), cm);
    adamw8_put<STREAM>(V + b * (ADAMW8_BLOCK / 4), cv);
    if (lane == 0) {
      mo[b] = (uint16_t)nm[b];
      vo[b] = (uint16_t)nv[b];
    }
  }
}

// Number of the tensor that owns workgroup b: how many of the others start at
// or before it.
__device__ __forceinline__ int adamw8_owner(const Adamw8Args& a, uint32_t b) {
  int n = -1;
#pragma unroll
  for (int p = 0; p < (ADAMW8_TENSORS + 63) / 64; ++p) {
    const int i = 64 * p + (int)(threadIdx.x & 63);
    const bool at = i < a.tensors && a.first[i < ADAMW8_TENSORS ? i : 0] <= b;
    n += __popcll(__ballot(at));
  }
  return __builtin_amdgcn_readfirstlane(n);
}

template <typename T, bool EXACT, bool STREAM> __device__ __forceinline__ void adamw8_blocks_of(const Adamw8Desc& d, int64_t first, const Adamw8Args& a) {
  if ((first + ADAMW8_WAVE_BLOCKS) * ADAMW8_BLOCK <= d.numel) {
    adamw8_tile<T, ADAMW8_WAVE_BLOCKS, true, EXACT, STREAM>(d, first, a);
  } else {
    const int64_t end = min(first + ADAMW8_WAVE_BLOCKS, adamw8_blocks(d.numel));
    for (int64_t b = first; b < end; ++b) adamw8_tile<T, 1, false, EXACT, STREAM>(d, b, a);
  }
}

template <bool EXACT, bool STREAM> __global__ __launch_bounds__(256) void adamw8_kernel(const Adamw8Args a) {
  const uint32_t b = a.wg_base + blockIdx.x;
  const int t = adamw8_owner(a, b);
  const Adamw8Desc& d = a.desc[t];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t first = ((int64_t)(b - a.first[t]) * 4 + wave) * ADAMW8_WAVE_BLOCKS;
  if (d.dtype == DT_BF16) adamw8_blocks_of<bf16, EXACT, STREAM>(d, first, a);
  else adamw8_blocks_of<float, EXACT, STREAM>(d, first, a);
}

// fp32 values -> codes (rounded as in a step of number `step`), and back.  A
// wave per block, element by element, as they are for conversions now and then:
// 128256 x 4096 values packed in 530 us (5.0 TB/s), unpacked in 955 (2.8 TB/s: a
// lane's 4 values go out in 4 stores), where a large copy's rate would take 438.
template <bool SECOND> __global__ __launch_bounds__(256) void adamw8_pack_kernel(const Adamw8PackArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t nblk = adamw8_blocks(a.numel);
  auto* offs = as_global(reinterpret_cast<uint16_t*>(a.state + nblk * ADAMW8_BLOCK));
  for (int64_t blk = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); blk < nblk; blk += (int64_t)gridDim.x * 4) {
    const int64_t i = blk * ADAMW8_BLOCK + 4 * lane;
    float x[4];
    uint32_t u = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = i + e < a.numel ? as_global(a.x)[i + e] : 0.f;
      u = max(u, adamw8_bits(x[e]));
    }
    const uint32_t off = adamw8_offset(wave_max(u), SECOND ? 255 : 127);
    const uint32_t h = adamw8_hash(blk, lane, a.key);
    uint32_t c = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t r = adamw8_turn(h, e);
      c |= (SECOND ? adamw8_encode_v(adamw8_bits(x[e]), r, off) : adamw8_encode_m(x[e], adamw8_bits(x[e]), r, off))
           << (8 * e);
    }
    *as_global(reinterpret_cast<uint32_t*>(a.state + i)) = c;
    if (lane == 0) offs[blk] = (uint16_t)off;
  }
}
template <bool SECOND> __global__ __launch_bounds__(256) void adamw8_unpack_kernel(const Adamw8PackArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t nblk = adamw8_blocks(a.numel);
  const auto* offs = as_global(reinterpret_cast<const uint16_t*>(a.state + nblk * ADAMW8_BLOCK));
  for (int64_t blk = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); blk < nblk; blk += (int64_t)gridDim.x * 4) {
    const int64_t i = blk * ADAMW8_BLOCK + 4 * lane;
    const uint32_t c = *as_global(reinterpret_cast<const uint32_t*>(a.state + i)), off = offs[blk];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t k = c >> (8 * e) & 255u;
      if (i + e < a.numel) as_global(a.x)[i + e] = SECOND ? adamw8_decode_v(k, off) : adamw8_decode_m(k, off);
    }
  }
}

}  // namespace muon
