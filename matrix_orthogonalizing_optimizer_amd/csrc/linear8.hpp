// Linear layer on 8-bit rows, gfx950: three tiled matrix products
//   L8_Y   y[t][n]  = scale[t] wscale[n] sum_k q[t][k] w[n][k] + bias[n]
//   L8_DW  dW[n][k] = sum_t dy[t][n] (scale[t] q[t][k])
//   L8_DX  dX[t][k] = sum_n dy[t][n] (wscale[n] w[n][k])
// Written below as C (M x N) = sum over K of A B.
//
// A workgroup of 8 waves owns a T x T tile of C (T = 256: 128 x 64 outputs per
// wave, one workgroup per CU; T = 128: 64 x 32 per wave, two workgroups per CU; 4
// waves of 64 x 64 read less LDS but were 10% slower with one workgroup on a CU
// and no faster with two) and walks K in stages of 128 bytes per row: 128 values of int8, or 64 of bf16.  Two stages live in LDS.
//
// L8_Y: both operands row-major int8, copied global -> LDS without a register
// round trip; v_mfma_i32_32x32x32_i8, sums exact in 32-bit integers.
//
// L8_DW, L8_DX: v_mfma_f32_32x32x16_bf16.  The 8-bit operand lies K-major
// (row s of the storage is summation index s) with one scale per summation
// row, which no epilogue can apply.  It is loaded to registers, turned into
// bf16 (q * scale; exact, the scale being a power of two) once per workgroup
// and written to LDS, between the MFMAs of the stage before; converting in
// front of the MFMAs instead would repeat it in every wave that shares the
// columns.  Fragments come out of LDS transposed (ds_read_b64_tr_b16).  dy is
// row-major for dX, K-major for dW.
// Where many tile rows share the 8-bit operand it is turned into bf16 in the
// workspace first (B_BF16; row_restore_kernel) and then copied to LDS like
// dy: that takes 3 bytes of HBM traffic per element once, and saves every
// workgroup the conversion and its register writes to LDS (1.88 -> 1.62 us per
// 256 x 256 x 64 stage of random data).  linear8_plan (linear8_plan.hpp) chooses.
// dy is copied to LDS directly as well, which takes bf16 rows in whole
// 16-byte pieces.  Any other dy is laid out so in the workspace first
// (linear8_planes_kernel): bf16 rows of odd widths or addresses as they are,
// fp32 as three bf16 planes that sum to it (8 significant bits each; see bf16_piece);
// K is then walked once per plane.  The planes are 6 bytes written and read
// next to 4 of dy.  Where few tile columns share them, the 128 tiles cut fp32 dy
// themselves (B_Q8_A_F32): it is loaded to registers once per K-stage, each of
// the stage's three walks writes the next piece to LDS and keeps what is left.
// A stage takes 0.2 to 0.4 us more for that; 5451 x 64 x 11904 98 instead of 228 us.
//
// The first `whole` tiles, as many as fill the chip in full rounds, are computed
// by one workgroup each; the K of the others (all of them, if the product has
// few) is split over workgroups that leave partial tiles in the workspace, and
// linear8_join_kernel adds those in order.
#pragma once

#include "device_common.hpp"
#include "gemm.hpp"
#include "kernel_args.hpp"
#include "row_ops.hpp"

namespace muon {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

enum : int { L8_Y = 0, L8_DW = 1, L8_DX = 2 };
enum : int { B_Q8 = 0, B_BF16 = 1, B_Q8_A_F32 = 2 };

template <bool INT> struct Acc8;
template <> struct Acc8<true> {
  typedef i32x16 type;
  __device__ __forceinline__ static void mma(i32x16& c, const u32x4& a, const u32x4& b) {
    c = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
};
template <> struct Acc8<false> {
  typedef f32x16 type;
  __device__ __forceinline__ static void mma(f32x16& c, const u32x4& a, const u32x4& b) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                0, 0);
  }
};

// Piece p (0, 1, 2) of fp32 x as bf16 bits in the high half of the result.
// Cutting off mantissa bits leaves at most 24 - 8 - 8 = 8 significant bits
// for the last piece, so the three add up to x exactly, except for bits under
// 2^-133, which bf16 does not have (so from |x| = 2^-110 up nothing is lost); an
// infinity or NaN is all in the first piece (a NaN keeps a mantissa bit).
__device__ __forceinline__ uint32_t bf16_piece(float x, int p) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  uint32_t hi = u & 0xffff0000u;
  if ((u & 0x7f800000u) == 0x7f800000u) return p ? 0u : (hi | ((u & 0x7fffffu) ? 0x400000u : 0u));
  if (p == 0) return hi;
  float r = x - __builtin_bit_cast(float, hi);
  hi = __builtin_bit_cast(uint32_t, r) & 0xffff0000u;
  if (p == 1) return hi;
  r -= __builtin_bit_cast(float, hi);
  return __builtin_bit_cast(uint32_t, r) & 0xffff0000u;
}

// dy (rows x cols, any alignment) -> PIECES planes of bf16, rows ldo apart (a
// multiple of 8), zero up to a multiple of 8 columns; 8 columns per thread, 4
// rows of 64 pieces per workgroup at a time.
template <typename T>
__global__ __launch_bounds__(256) void linear8_planes_kernel(const PlanesArgs a) {
  const int c = (int)(blockIdx.y * 64 + (threadIdx.x & 63)) * 8;
  if (c >= a.cols) return;
  for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < a.rows; row += (int64_t)gridDim.x * 4) {
    RowRaw<T, true> x;
    x.load(static_cast<const T*>(a.dy) + row * a.ld, c, a.cols);
    x.settle(c, a.cols);
    bf16* o = static_cast<bf16*>(a.o) + row * a.ldo + c;
    if constexpr (sizeof(T) == 2) {
      *as_global(reinterpret_cast<u32x4*>(o)) = u32x4{x.w[0], x.w[1], x.w[2], x.w[3]};
    } else {
#pragma unroll
      for (int pc = 0; pc < 3; ++pc) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = (bf16_piece(x.get(2 * j), pc) >> 16) | bf16_piece(x.get(2 * j + 1), pc);
        *as_global(reinterpret_cast<u32x4*>(o + pc * a.plane)) = w;
      }
    }
  }
}

// Workgroups are spread over the XCDs in chunks of S consecutive pieces of
// work, as the optimizer's products are (gemm.hpp): a bijection of [0, tot).
__device__ __forceinline__ int linear8_deal(int b, int tot, int S) {
  const int xcd = b & 7, loc = b >> 3;
  const int full = tot / (8 * S);
  if (loc < full * S) return (loc / S) * 8 * S + xcd * S + loc % S;
  const int rest = tot - full * 8 * S, q = rest >> 3, r = rest & 7;
  return full * 8 * S + xcd * q + (xcd < r ? xcd : r) + (loc - full * S);
}
// Tile number -> tile row and column: groups of 4 tile rows, column by column.
__device__ __forceinline__ void linear8_tile(const Linear8Args& a, int tile, int& bi, int& bj) {
  constexpr int GROUP = 4;
  const int g = tile / (GROUP * a.tilesN);
  const int first = g * GROUP;
  const int gm = min(a.tilesM - first, GROUP);
  const int w = tile - g * GROUP * a.tilesN;
  bi = first + w % gm;
  bj = w / gm;
}

// Partial tile of a split: [splits][tiles from `whole` on][T][T] in the workspace.
template <int T> __device__ __forceinline__ int64_t linear8_part(const Linear8Args& a, int tile, int split) {
  return ((int64_t)split * (a.tilesM * a.tilesN - a.whole) + (tile - a.whole)) * (T * T);
}

template <int MODE, int BSRC, int T, int NW, typename TO>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(T == 128 ? NW / 2 : NW / 4, T == 128 ? NW / 2 : NW / 4)))
void linear8_kernel(const Linear8Args a) {
  constexpr bool INT = MODE == L8_Y;
  constexpr bool CVT = !INT && BSRC != B_BF16;  // the 8-bit operand is converted here
  constexpr bool AF32 = BSRC == B_Q8_A_F32;     // dy is fp32 and cut into its pieces here
  constexpr bool AKM = MODE == L8_DW;      // A lies K-major
  constexpr int ES = INT ? 1 : 2;
  constexpr int EPC = 16 / ES;             // elements per 16-byte chunk
  constexpr int BK = 8 * EPC;              // K per stage
  constexpr int WGN = NW / 2;              // waves: 2 along M, NW / 2 along N
  constexpr int WTM = T / 64, WN = T / WGN, WTN = WN / 32;
  constexpr int OPS = T * 8;               // chunks of one operand's stage
  constexpr int STG = 2 * OPS;
  constexpr int NQ = OPS / (64 * NW);      // 16-byte pieces of one operand a thread moves per stage
  constexpr int NDR = WTM + WTN, NPAIR = WTM * WTN;
  constexpr int RPP = (NDR + NPAIR - 1) / NPAIR;  // fragment reads issued per MFMA
  constexpr int CR = T / 8;                // chunks per K-row of a K-major stage
  constexpr int RPC = 64 / CR;             // K-rows per wave-wide copy
  constexpr int RSTEP = 64 * NW / CR;      // rows between a thread's pieces of the 8-bit operand
  static_assert(NQ * 8 * NW == T && RSTEP % 4 == 0, "chunks shared out evenly");
  __shared__ u32x4 ring[2][STG];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / WGN, wn = wid % WGN;
  const int half = lane >> 5, l32 = lane & 31;
  // the division runs on the vector unit: results back to scalar registers
  const bool part = a.splits > 1 && (int)blockIdx.x >= a.whole;
  int split = 0, tile, bi, bj;
  if (!part) {
    tile = linear8_deal(blockIdx.x, a.splits > 1 ? a.whole : a.tilesM * a.tilesN, 8 * a.tilesN);
  } else {
    const int rem = a.tilesM * a.tilesN - a.whole;
    const int w = linear8_deal(blockIdx.x - a.whole, rem * a.splits, 8 * a.tilesN);
    split = w / rem;
    tile = a.whole + w % rem;
  }
  split = __builtin_amdgcn_readfirstlane(split);
  tile = __builtin_amdgcn_readfirstlane(tile);
  linear8_tile(a, tile, bi, bj);
  bi = __builtin_amdgcn_readfirstlane(bi);
  bj = __builtin_amdgcn_readfirstlane(bj);
  const int row0 = bi * T, col0 = bj * T;

  // stages of this split: K-stages [ks0, ks1), walked once per piece of dy
  const int nks = (a.K + BK - 1) / BK;
  const int per = part ? a.per_split : nks;
  const int ks0 = min(split * per, nks), ks1 = min(ks0 + per, nks);
  const int nst = (ks1 - ks0) * a.planes;

  auto swz_t = [](int krow) { return ((krow & 1) << 2) ^ (((krow >> 1) & 1) * 10); };

  // summation rows of K-stage ks.  The clamp compiles to a vector instruction:
  // back to a scalar register, or the buffer resources built from it count as
  // divergent and each load runs in a waterfall loop (0.2 us of a
  // 1.06 us stage of a 128 tile)
  auto stage_rows = [&](int ks) { return __builtin_amdgcn_readfirstlane(max(0, min(BK, a.K - ks * BK))); };
  // ---- operand A (and B for L8_Y), row-major: rows of the tile
  const int rows_a = min(T, a.M - row0);
  const char* Abase = static_cast<const char*>(a.A) + (AKM ? 0 : (int64_t)row0 * a.lda * ES);
  // 8-bit rows have all their ld bytes, the last row of dy whole 16-byte pieces
  const uint32_t Abytes = INT ? (uint32_t)((int64_t)rows_a * a.lda)
                              : (uint32_t)((((int64_t)rows_a - 1) * a.lda + ((a.K + 7) & ~7)) * 2);
  const int rows_b = min(T, a.N - col0);
  const __amdgpu_buffer_rsrc_t brs =
      make_rsrc(static_cast<const int8_t*>(a.B) + (INT ? (int64_t)col0 * a.ldb : 0), (uint32_t)((int64_t)rows_b * a.ldb));
  const int crow = wid * (8 * NQ) + (lane >> 3);              // tile row of copy 0
  const int ck[2] = {((lane & 7) ^ (lane >> 3)) * EPC, ((lane & 7) ^ (lane >> 3) ^ 1) * EPC};
  auto copy_row_major = [&](__amdgpu_buffer_rsrc_t r, int64_t ld, int region, int q, int v, int ks) {
    const int k = ks * BK + ck[q & 1];
    const uint32_t off = k < a.K ? (uint32_t)(((crow + 8 * q) * ld + k) * ES) : OOB;
    copy16_to_lds(r, &ring[v & 1][region + (wid * NQ + q) * 64], off);
  };
  // ---- operand A of dW, K-major: rows of the stage, columns row0 .. of dy
  // (and B when it is bf16): a lane's K-row and chunk of copy q depend on q
  // only through q & 1, as in gemm.hpp
  auto km_offset = [&](int par, int64_t ld, int c0, int cols) {
    const int krow = (wid * NQ + par) * RPC + lane / CR;
    const int col = c0 + ((lane % CR) ^ swz_t(krow)) * 8;
    return col < cols ? (uint32_t)(((int64_t)krow * ld + col) * 2) : OOB;
  };
  const uint32_t ta[2] = {km_offset(0, a.lda, row0, a.M), km_offset(1, a.lda, row0, a.M)};
  const uint32_t tbb[2] = {km_offset(0, a.ldb, col0, a.N), km_offset(1, a.ldb, col0, a.N)};
  auto copy_k_major = [&](const void* base, int64_t ld, int cols, const uint32_t(&t)[2], int region, int q, int v, int ks) {
    const int nk = stage_rows(ks);
    const char* p = static_cast<const char*>(base) + (int64_t)ks * BK * ld * 2;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(p, nk ? (uint32_t)((((int64_t)nk - 1) * ld + cols) * 2) : 0u);
    copy16_to_lds(r, &ring[v & 1][region + (wid * NQ + q) * 64], t[q & 1] + (uint32_t)((int64_t)((q & ~1) * RPC) * ld * 2));
  };
  auto copy_a = [&](int q, int v, int ks, int plane) {
    const char* base = Abase + (INT ? 0 : plane * a.plane * 2);
    if constexpr (AKM) copy_k_major(base, a.lda, (a.M + 7) & ~7, ta, 0, q, v, ks);
    else copy_row_major(make_rsrc(base, Abytes), a.lda, 0, q, v, ks);
  };
  // expanded B has whole 16-byte chunks behind its last column
  auto copy_b = [&](int q, int v, int ks) {
    copy_k_major(a.B, a.ldb, (a.N + 7) & ~7, tbb, OPS, q, v, ks);
  };
  // ---- 8-bit operand of the gradients: piece i of a thread is row RSTEP i +
  // tid / CR of the stage, columns 8 (tid % CR) .. + 7 of the tile
  u32x2 bq[NQ];
  float bs[NQ];
  const int brow = tid / CR, bcol = (tid % CR) * 8;
  const uint32_t boff = col0 + bcol < a.ldb ? (uint32_t)(brow * a.ldb + col0 + bcol) : OOB;
  const int bslot = OPS + brow * CR + ((tid % CR) ^ swz_t(brow));
  auto load_b = [&](int ks) {
    if constexpr (CVT) {
      const int nk = stage_rows(ks);
      const __amdgpu_buffer_rsrc_t r =
          make_rsrc(static_cast<const int8_t*>(a.B) + (int64_t)ks * BK * a.ldb, (uint32_t)((int64_t)nk * a.ldb));
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.sb + (int64_t)ks * BK, (uint32_t)(nk * 4));
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        bq[i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, boff + (uint32_t)(i * RSTEP * a.ldb), 0, 0));
        bs[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, (uint32_t)(RSTEP * i + brow) * 4, 0, 0));
      }
    }
  };
  // ---- fp32 dy of the gradients, where the copies above would put its pieces:
  // the registers hold what the pieces made so far have left of the values
  float xa[AF32 ? NQ : 1][8];
  int xlim[AF32 ? NQ : 1];  // dX: elements of the piece before the end of K
  auto load_a = [&](int ks) {
    if constexpr (AF32) {
      const int nk = stage_rows(ks);
      const char* base = static_cast<const char*>(a.A) + (AKM ? (int64_t)ks * BK * a.lda * 4 : (int64_t)row0 * a.lda * 4);
      const __amdgpu_buffer_rsrc_t r = make_rsrc(
          base, AKM ? (nk ? (uint32_t)((((int64_t)nk - 1) * a.lda + a.M) * 4) : 0u)
                    : (uint32_t)((((int64_t)rows_a - 1) * a.lda + a.K) * 4));
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        uint32_t off;
        if constexpr (AKM) {
          const int krow = (wid * NQ + i) * RPC + lane / CR, col = row0 + ((lane % CR) ^ swz_t(krow)) * 8;
          off = col < a.M ? (uint32_t)(((int64_t)krow * a.lda + col) * 4) : OOB;
        } else {
          const int k = ks * BK + ck[i & 1];
          off = k < a.K ? (uint32_t)(((crow + 8 * i) * a.lda + k) * 4) : OOB;
          xlim[i] = a.K - k;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 x = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 16 * h, 0, 0));
#pragma unroll
          for (int e = 0; e < 4; ++e) xa[i][4 * h + e] = x[e];
        }
      }
    }
  };
  u32x4 aw;
  auto convert_a = [&](int idx, int v) {  // as convert_b
    if constexpr (AF32) {
      const int i = idx >> 2, j = idx & 3;
      uint32_t hi[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = xa[i][2 * j + e];
        if constexpr (!AKM) x = 2 * j + e < xlim[i] ? x : 0.f;
        x = __builtin_canonicalizef(x);  // a NaN keeps a bit among the high ones
        hi[e] = __builtin_bit_cast(uint32_t, x) & 0xffff0000u;
        const float rest = x - __builtin_bit_cast(float, hi[e]);
        xa[i][2 * j + e] = rest == rest ? rest : 0.f;  // infinities and NaN are all in the first piece
      }
      aw[j] = (hi[0] >> 16) | hi[1];
      if (j == 3) ring[v & 1][(wid * NQ + i) * 64 + lane] = aw;
    }
  };
  u32x4 bw;
  auto convert_b = [&](int idx, int v) {  // pair idx of the thread's 8 NQ values; the fourth pair of a piece stores it
    if constexpr (CVT) {
      const int i = idx >> 2, j = idx & 3;
      const uint32_t w = bq[i][j >> 1] >> (16 * (j & 1));
      bw[j] = pack2<bf16>((float)(int8_t)w * bs[i], (float)(int8_t)(w >> 8) * bs[i]);
      if (j == 3) ring[v & 1][bslot + i * RSTEP * CR] = bw;
    }
  };

  typename Acc8<INT>::type acc[WTM][WTN];
#pragma unroll
  for (int i = 0; i < WTM; ++i)
#pragma unroll
    for (int j = 0; j < WTN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  // ---- fragments, double buffered by k-step
  u32x4 fa[2][WTM], fb[2][WTN];
  const int rswz = (l32 & 7) ^ ((l32 >> 3) & 1);
  constexpr int ROWB = CR * 16;
  uint32_t tbase[NDR];
#pragma unroll
  for (int r = 0; r < NDR; ++r) {
    const int e = (lane >> 2) & 3, q = lane & 3;
    const int region = r < WTM ? 0 : OPS;
    const int rb = r < WTM ? wm * (T / 2) + r * 32 : wn * WN + (r - WTM) * 32;
    const int col = rb + 16 * ((lane >> 4) & 1) + 4 * q;
    tbase[r] = (uint32_t)(uintptr_t)(lds_ptr_t)&ring[0][0] +
               (uint32_t)(region * 16 + (8 * half + e) * ROWB + ((col >> 3) ^ swz_t(e)) * 16 + (col & 7) * 2);
  }
  auto read_one = [&](int r, int v, int s, int slot) {
    const bool isA = r < WTM;
    const int rb = isA ? wm * (T / 2) + r * 32 : wn * WN + (r - WTM) * 32;
    u32x4 f;
    if (INT || (isA && !AKM)) {
      f = ring[v & 1][(isA ? 0 : OPS) + (rb + l32) * 8 + ((2 * s + half) ^ rswz)];
    } else {
      const uint32_t p = tbase[r] + (uint32_t)((v & 1) * STG * 16);
#pragma unroll
      for (int kq = 0; kq < 2; ++kq) {
        const uint2 w = lds_read_tr16_step<ROWB>(p, 2 * s + kq);
        f[2 * kq] = w.x;
        f[2 * kq + 1] = w.y;
      }
    }
    if (isA) fa[slot][r] = f;
    else fb[slot][r - WTM] = f;
  };
  // reads in the order of first use: A0, B0 .. B(WTN-1), A1 .. A(WTM-1)
  auto ro = [](int p) { return p == 0 ? 0 : (p <= WTN ? WTM + p - 1 : p - WTN); };
  // The compiler does not track the transposed reads.  LDS instructions of a
  // wave complete in order, so before MFMA p it is enough that at most as
  // many are outstanding as were issued after the fragment that p is the
  // first to use: this step's later fragments and the next step's first p
  // ones (two instructions each; untransposed reads and register writes are
  // not counted, which only waits for more).  Waiting for all of them once
  // per step took 1.95 instead of 1.89 us for a stage of the weight gradient.
  auto wait_frag = [&](auto pc) {
    if constexpr (!INT) {
      constexpr int p = decltype(pc)::value;
      constexpr int i = p / WTN, j = p % WTN;
      constexpr bool needA = j == 0 && AKM, needB = i == 0;  // first uses among the transposed
      if constexpr (needA || needB) {
        // position of that fragment in the reading order
        constexpr int at = needB ? (j + 1) : (i == 0 ? 0 : WTN + i);
        constexpr int later_a = AKM ? (WTM - 1 - (at > WTN ? at - WTN : 0)) : 0;
        constexpr int later_b = at <= WTN ? WTN - at : 0;
        constexpr int now = p * RPP < NDR ? p * RPP : NDR;  // reads issued so far in this step
        constexpr int now_a = AKM ? (now > 0 ? 1 : 0) + (now > WTN + 1 ? now - WTN - 1 : 0) : 0;
        constexpr int now_b = now <= 1 ? 0 : (now - 1 < WTN ? now - 1 : WTN);
        constexpr int n = 2 * (later_a + later_b + now_a + now_b);
        __builtin_amdgcn_s_waitcnt(0xc07f | ((n < 15 ? n : 15) << 8));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  auto mfma_pair = [&](int p, int slot) {
    Acc8<INT>::mma(acc[p / WTN][p % WTN], fa[slot][p / WTN], fb[slot][p % WTN]);
  };
  // K-stage and plane of the stage that is loaded next; past the end the loads
  // only refill a slot that nobody reads
  int ksn = ks0, pcn = 0;
  auto advance = [&] {
    if constexpr (AF32) {  // all pieces of a stage in a row
      if (++pcn == a.planes) {
        pcn = 0;
        ++ksn;
      }
      return;
    }
    if (++ksn == ks1 && pcn + 1 < a.planes) {
      ksn = ks0;
      ++pcn;
    }
  };

  if (nst > 0) {
    // ---- prologue: stages 0 and 1 in LDS (of converted operands, stage 1's values in registers)
    auto copies = [&](int v) {
#pragma unroll
      for (int q = 0; q < NQ; ++q)
        if constexpr (!AF32) copy_a(q, v, ksn, pcn);
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if constexpr (INT) copy_row_major(brs, a.ldb, OPS, q, v, ksn);
        else if constexpr (!CVT) copy_b(q, v, ksn);
      }
    };
    load_b(ksn);
    load_a(ksn);
    copies(0);
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) convert_b(i, 0);
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) convert_a(i, 0);
    advance();
    load_b(ksn);
    copies(1);
    // All of it, stage 1 too: a wait for stage 0 alone would count on an order of
    // issue that nothing holds the compiler to, and the barrier waits for every
    // copy to LDS anyway.
    if constexpr (!AF32) wait_vmcnt_lgkm0<0>();
    __syncthreads();
#pragma unroll
    for (int r = 0; r < NDR; ++r) read_one(ro(r), 0, 0, 0);

    for (int v = 0; v < nst; ++v) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        static_for<0, NPAIR>([&](auto pc) __attribute__((always_inline)) {
          constexpr int p = decltype(pc)::value;
          wait_frag(pc);
          mfma_pair(p, s & 1);
          // the fragment reads of a step before its register writes: those wait
#pragma unroll
          for (int r = p * RPP; r < NDR && r < (p + 1) * RPP; ++r) read_one(ro(r), v, s + 1, (s + 1) & 1);
          if constexpr (CVT) {
            // 4 NQ pairs of B over the 3 NPAIR MFMAs, after a head start for the loads
            constexpr int SLOTS = 3 * NPAIR, HEAD = NPAIR >= 8 ? 6 : 2;
            constexpr int PER = (4 * NQ + SLOTS - HEAD - 1) / (SLOTS - HEAD);
            const int at = s * NPAIR + p - HEAD;
#pragma unroll
            for (int c = 0; c < PER; ++c)
              if (at >= 0 && at * PER + c < 4 * NQ) {
                convert_b(at * PER + c, v + 1);
                convert_a(at * PER + c, v + 1);
              }
          }
          __builtin_amdgcn_sched_barrier(0);
        });
      }
      // stage v + 1 is whole and this wave is done reading stage v; after the
      // barrier that holds for every wave
      wait_vmcnt_lgkm0<0>();
      __syncthreads();
      __builtin_amdgcn_sched_barrier(0);
      advance();
      load_b(ksn);
      if (AF32 && pcn == 0) load_a(ksn);
#pragma unroll
      for (int p = 0; p < NPAIR; ++p) {
        mfma_pair(p, 1);
#pragma unroll
        for (int c = p; c < 2 * NQ; c += NPAIR) {
          if constexpr (AF32) continue;
          else if (c < NQ) copy_a(c, v + 2, ksn, pcn);
          else if constexpr (INT) copy_row_major(brs, a.ldb, OPS, c - NQ, v + 2, ksn);
          else if constexpr (!CVT) copy_b(c - NQ, v + 2, ksn);
        }
#pragma unroll
        for (int r = p * RPP; r < NDR && r < (p + 1) * RPP; ++r) read_one(ro(r), v + 1, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    wait_vmcnt_lgkm0<0>();  // trailing copies and reads
    __builtin_amdgcn_sched_barrier(0);
  }
  __syncthreads();

  // ---- epilogue: 32-row strips of a wave through its part of the ring, then
  // rows of 8 values per lane
  constexpr int SROW = WN + 8;
  static_assert(NW * 32 * SROW * 4 <= 2 * STG * 16, "strips fit in the ring");
  constexpr int CW = WN / 8, DRS = 64 / CW, NT = 32 / DRS;
  float* strip = reinterpret_cast<float*>(&ring[0][0]) + wid * (32 * SROW);
  const int dr0 = lane / CW, dc8 = (lane % CW) * 8;
  const int gj = col0 + wn * WN + dc8;
  float cs[8], cb[8];
  if constexpr (INT) {
    if (!part && gj < a.N) {
      piece_load(a.sb, gj, a.N, cs);
      if (a.bias) vec_load(a.bias, a.bias_dtype, gj, a.N, cb);
    }
  }
  static_for<0, WTM>([&](auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value;
    const int gr0 = row0 + wm * (T / 2) + i * 32;
#pragma unroll
    for (int j = 0; j < WTN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const auto x = acc[i][j][e];
        strip[((e >> 2) * 8 + half * 4 + (e & 3)) * SROW + j * 32 + l32] = __builtin_bit_cast(float, x);
      }
    wave_lds_sync();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = gr0 + dr0 + DRS * t;
      const float* sp = strip + (dr0 + DRS * t) * SROW + dc8;
      const f32x4 lo = *reinterpret_cast<const f32x4*>(sp);
      const f32x4 hi = *reinterpret_cast<const f32x4*>(sp + 4);
      float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      if (r < a.M && gj < a.N) {
        if (part) {
          float* o = a.ws + linear8_part<T>(a, tile, split) + (r - row0) * T + (gj - col0);
          *as_global(reinterpret_cast<f32x4*>(o)) = lo;
          *as_global(reinterpret_cast<f32x4*>(o + 4)) = hi;
        } else {
          TO* o = static_cast<TO*>(a.o) + (int64_t)r * a.ldo;
          if constexpr (INT) {
            float sr, sr2;
            split_scale(as_global(a.sa)[r], sr, sr2);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)__builtin_bit_cast(int32_t, v[e]) * sr * cs[e];
            if (sr2 != 1.f) {  // multiplied for every row: 8192 x 14336 x 4096 417 instead of 414 us
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] *= sr2;
            }
            if (a.bias) {
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] += cb[e];
            }
          } else if (a.accumulate) {
            float old[8];
            piece_load(o, gj, a.N, old);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += old[e];
          }
          piece_store(o, gj, a.N, v);
        }
      }
    }
    wave_lds_sync();
  });
}

// Adds the partial tiles of a split product in order and finishes it as the
// epilogue above does.  8 columns per thread, T * T / 2048 workgroups per tile.
template <bool INT, int T, typename TO>
__global__ __launch_bounds__(256) void linear8_join_kernel(const Linear8Args a) {
  constexpr int WGS = T * T / 2048;
  const int tile = a.whole + (int)(blockIdx.x / WGS);
  const int in = (int)(blockIdx.x % WGS) * 2048 + threadIdx.x * 8;  // first value within the tile
  int bi, bj;
  linear8_tile(a, tile, bi, bj);
  const int64_t r = (int64_t)bi * T + in / T;
  const int c = bj * T + in % T;
  if (r >= a.M || c >= a.N) return;
  const float* w = a.ws + linear8_part<T>(a, tile, 0) + in;
  const int64_t step = (int64_t)(a.tilesM * a.tilesN - a.whole) * (T * T);
  float v[8];
  if constexpr (INT) {
    int32_t s[8] = {};
    for (int z = 0; z < a.splits; ++z)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const i32x4 x = *as_global(reinterpret_cast<const i32x4*>(w + z * step + 4 * h));
#pragma unroll
        for (int e = 0; e < 4; ++e) s[4 * h + e] += x[e];
      }
    float sr, sr2, cs[8];
    split_scale(as_global(a.sa)[r], sr, sr2);
    piece_load(a.sb, c, a.N, cs);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)s[e] * sr * cs[e] * sr2;
    if (a.bias) {
      vec_load(a.bias, a.bias_dtype, c, a.N, cs);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += cs[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll 4
    for (int z = 0; z < a.splits; ++z)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 x = *as_global(reinterpret_cast<const f32x4*>(w + z * step + 4 * h));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * h + e] += x[e];
      }
  }
  TO* o = static_cast<TO*>(a.o) + r * a.ldo;
  if (!INT && a.accumulate) {
    float old[8];
    piece_load(o, c, a.N, old);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += old[e];
  }
  piece_store(o, c, a.N, v);
}

}  // namespace muon
