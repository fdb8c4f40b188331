// Matrix products grouped by expert, gfx950.  Rows offsets[e] .. offsets[e+1]-1
// belong to expert e:
//   EX_Y   y[r]  = x[r] W[e]^T
//   EX_DX  dx[r] = dy[r] W[e]
//   EX_DW  dW[e] = sum over the rows r of e of dy[r]^T x[r]
// Written below as C (M x N) = sum over K of A B, sums in fp32.
//
// The offsets lie on the device, so the host does not know how many rows an
// expert has.  EX_Y and EX_DX launch as many workgroups as any offsets can
// need (rows / 128 + experts tile rows); each finds its tile from a prefix sum
// over the experts' tile rows (experts_tile), and those past the last tile
// end at once.  EX_DW has a workgroup per tile and unit of at most `chunk` rows
// of an expert (one unit for an expert without rows).  Offsets are clamped to 0 .. rows, so no value of theirs
// leads outside the operands.
//
// A workgroup of 8 waves owns a 128 x 128 tile of C (64 x 32 outputs per wave,
// two workgroups per CU) and walks K in stages of 128 bytes per row: 64 values of
// bf16, 32 of fp32.  Two stages live in LDS.  v_mfma_f32_32x32x16_bf16, or
// v_mfma_f32_32x32x2_f32.
//
// An operand lies row-major (K contiguous: x and w of EX_Y, dy of EX_DX) or
// K-major (w of EX_DX, both of EX_DW).  K-major bf16 fragments come out of LDS
// transposed (ds_read_b64_tr_b16), fp32 ones element by element.
//
// DIRECT: bf16 rows of whole 16-byte pieces are copied global -> LDS without a
// register round trip.  Otherwise (odd widths, any alignment, fp32) the pieces go
// through registers, and what reaches past a row's end becomes zero there.
//
// Parts of a tile's K (`splits` of them, or chunks of an expert's rows in the
// weight gradient) go to workgroups of their own, which leave partial tiles in
// the workspace; experts_join_kernel adds those in order.
//
// Measured: fp32, 8192 rows of 8 experts of 2048 x 2048, weight gradient 555 us, 124
// of the 154 TFLOP/s of a large fp32 product, forward 657, input gradient 676; weight
// gradient of 3001 rows of 7 of 513 x 767 51 us a call (kernels traced one by one 46
// and 8 to join), bound by 480 workgroups of unequal length, up to 14 us, dealt in
// table order on 256 CUs, and by 31 MB of partial tiles; bf16 input gradient at any
// address, 1531 rows of 13 of 701 x 301 17 us a call (14 and 4 to join): K's 11 stages
// in two parts make 108 workgroups on 256 CUs, bound by the latency of their 6 stages
// through registers and by two launches.  With one odd width large bf16 products
// come here too: 49152 rows of 64 experts of 1407 x 2048, input gradient 489 us,
// weight gradient 522 (302 and 342 with 1408 in the large tiles); of 1408 x 2047
// forward 566, input gradient 484, weight gradient 529.
// A workgroup scans the offsets of all experts for its tile, so that part grows with
// the square of their number: weight gradient of 40000 rows of 2048 experts of 512 x
// 512 2.1 ms, of 4096 7.4 ms, where the results' bytes alone would take 0.2 and 0.4.
#pragma once

#include "device_common.hpp"
#include "gemm.hpp"
#include "kernel_args.hpp"
#include "row_ops.hpp"

namespace muon {

enum : int { EX_Y = 0, EX_DW = 1, EX_DX = 2 };
constexpr int EXPERTS_T = 128;  // edge of a tile

// First row of expert e and their number.
struct ExpertRows {
  int begin, count;
};
__device__ __forceinline__ ExpertRows experts_rows(const ExpertsArgs& a, int e) {
  const auto* off = as_global(a.offsets);
  const int b = min(max(off[e], 0), a.rows);
  return {b, min(max(off[e + 1], b), a.rows) - b};
}

// Inclusive prefix sum over the wave.
__device__ __forceinline__ int wave_prefix(int v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(v, d, 64);
    if ((int)(threadIdx.x & 63) >= d) v += up;
  }
  return v;
}

// A tile of C: its expert and that one's rows (or a chunk of them), tile row and
// column within it.
struct ExpertTile {
  int expert, begin, count, bi, bj;
  int64_t slot;  // partial tile that it leaves in the workspace; -1: C itself
  int split;     // forward, input gradient: part of its K
  int parts;     // joining: partial tiles, from slot on `stride` apart
  int64_t stride;
};

// Workgroups are spread over the XCDs in chunks of S consecutive pieces of
// work, as the optimizer's products are (gemm.hpp): a bijection of [0, tot).
__device__ __forceinline__ int experts_deal(int b, int tot, int S) {
  const int xcd = b & 7, loc = b >> 3;
  const int full = tot / (8 * S);
  if (loc < full * S) return (loc / S) * 8 * S + xcd * S + loc % S;
  const int rest = tot - full * 8 * S, q = rest >> 3, r = rest & 7;
  return full * 8 * S + xcd * q + (xcd < r ? xcd : r) + (loc - full * S);
}

// Tile number -> tile row and column: groups of 4 tile rows, column by column.
__device__ __forceinline__ void experts_place(int w, int tilesM, int tilesN, int& bi, int& bj) {
  constexpr int GROUP = 4;
  const int g = w / (GROUP * tilesN);
  const int first = g * GROUP;
  const int gm = min(tilesM - first, GROUP);
  const int in = w - g * GROUP * tilesN;
  bi = first + in % gm;
  bj = in / gm;
}

// The tile of workgroup b; false if there is none.  JOIN: the b-th tile that was
// left in parts.
//   forward, input gradient: tiles of 128 rows of the experts; all in `splits` parts
//   weight gradient: units of at most `chunk` rows of an expert; experts of
//   several units leave parts
template <int MODE, bool JOIN> __device__ __forceinline__ bool experts_tile(const ExpertsArgs& a, int b, ExpertTile& t) {
  constexpr int T = EXPERTS_T;
  constexpr bool DW = MODE == EX_DW;
  const int lane = threadIdx.x & 63;
  const int tiles = DW ? a.tilesM * a.tilesN : a.tilesN;  // of a unit, or of a tile row
  // units or tile rows of the wave's 64 experts, and those in parts (joining: experts in parts)
  ExpertRows r = {0, 0};
  int mine = 0, pre = 0, cut = 0, cutpre = 0;
  auto look = [&](int c) {
    r = {0, 0};
    if (c + lane < a.experts) r = experts_rows(a, c + lane);
    mine = c + lane >= a.experts ? 0 : DW ? max(1, (r.count + a.chunk - 1) / a.chunk) : (r.count + T - 1) / T;
    pre = wave_prefix(mine);
    if constexpr (DW) {
      cut = mine > 1 ? mine : 0;
      cutpre = wave_prefix(cut);
    }
  };
  int64_t sum = 0;
  for (int c = 0; c < a.experts; c += 64) {
    look(c);
    sum += __builtin_amdgcn_readlane(pre, 63);
  }
  // more than the rows allow: the offsets go back, and the groups overlap
  if (sum > (DW ? a.experts + a.rows / a.chunk : a.rows / T + min(a.experts, a.rows))) return false;
  const int tot = (int)sum * tiles;
  t.split = 0;
  t.slot = -1;
  int before = 0, cutbefore = 0;
  if constexpr (DW && JOIN) {
    int left = b / tiles;
    for (int c = 0; c < a.experts; c += 64) {
      if (a.experts > 64) look(c);
      const uint64_t some = __ballot(cut > 0);
      const int n = __popcll(some);
      if (left < n) {
        const int below = __popcll(some & ((1ull << lane) - 1));
        const int l = __builtin_ctzll(__ballot((some >> lane & 1) && below == left));
        t.expert = c + l;
        t.parts = __builtin_amdgcn_readlane(cut, l);
        const int in = b % tiles;
        t.slot = (int64_t)(cutbefore + __builtin_amdgcn_readlane(cutpre, l) - t.parts) * tiles + in;
        t.stride = tiles;
        t.begin = t.count = 0;
        experts_place(in, a.tilesM, a.tilesN, t.bi, t.bj);
        return true;
      }
      left -= n;
      cutbefore += __builtin_amdgcn_readlane(cutpre, 63);
    }
    return false;
  }
  const int splits = DW || JOIN ? 1 : a.splits;
  if (b >= tot * splits) return false;
  int w = JOIN ? b : experts_deal(b, tot * splits, 8 * a.tilesN);
  t.split = __builtin_amdgcn_readfirstlane(w / tot);
  w = __builtin_amdgcn_readfirstlane(w % tot);
  const int at = __builtin_amdgcn_readfirstlane(w / tiles);  // unit or tile row, counted over all experts
  int unit = 0, units = 0, cuts = 0;
  for (int c = 0; c < a.experts; c += 64) {
    if (a.experts > 64) look(c);  // otherwise they are still there
    const uint64_t past = __ballot(before + pre > at);
    if (past) {
      const int l = __builtin_amdgcn_readfirstlane(__builtin_ctzll(past));
      t.expert = c + l;
      t.begin = __builtin_amdgcn_readlane(r.begin, l);
      t.count = __builtin_amdgcn_readlane(r.count, l);
      units = __builtin_amdgcn_readlane(mine, l);
      unit = at - (before + __builtin_amdgcn_readlane(pre, l) - units);
      if constexpr (DW) cuts = cutbefore + __builtin_amdgcn_readlane(cutpre, l) - units;
      break;
    }
    before += __builtin_amdgcn_readlane(pre, 63);
    if constexpr (DW) cutbefore += __builtin_amdgcn_readlane(cutpre, 63);
  }
  if constexpr (DW) {
    experts_place(w % tiles, a.tilesM, a.tilesN, t.bi, t.bj);
    t.begin += unit * a.chunk;
    t.count = min(a.chunk, t.count - unit * a.chunk);
    if (units > 1) t.slot = (int64_t)(cuts + unit) * tiles + w % tiles;
  } else {
    experts_place(w - (at - unit) * tiles, units, a.tilesN, t.bi, t.bj);
    if (a.splits > 1) t.slot = JOIN ? (int64_t)w * a.splits : (int64_t)w * a.splits + t.split;
    t.parts = a.splits;
    t.stride = 1;
  }
  t.bi = __builtin_amdgcn_readfirstlane(t.bi);
  t.bj = __builtin_amdgcn_readfirstlane(t.bj);
  return true;
}

// Stages of K of a part of a tile: [ks0, ks1).
template <int MODE, int BK> __device__ __forceinline__ void experts_stages(const ExpertsArgs& a, const ExpertTile& t, int& ks0, int& ks1) {
  const int K = MODE == EX_DW ? t.count : a.K;
  const int nks = (K + BK - 1) / BK;
  const int per = (nks + a.splits - 1) / a.splits;
  ks0 = __builtin_amdgcn_readfirstlane(min(t.split * per, nks));
  ks1 = __builtin_amdgcn_readfirstlane(min(ks0 + per, nks));
}

// A 16-byte piece of a row at column c, through registers.  load() takes the
// row's last piece where c reaches past its end, settle() moves its own
// elements to the front and clears the others (all of them where !ok), so no
// branch stands behind the load.  SHORT: rows shorter than a piece, element by
// element (with both in one loop the loads of a stage cost 3 - 15% more).
template <typename T, bool SHORT> struct Piece {
  static constexpr int PER = 16 / sizeof(T);
  u32x4 w;
  __device__ __forceinline__ void load(const T* row, int c, int cols) {
    if constexpr (!SHORT) {
      const T* p = row + min(c, cols - PER);
      if constexpr (sizeof(T) == 2) w = as_global(reinterpret_cast<const u32x4_e2*>(p))->v;
      else w = __builtin_bit_cast(u32x4, as_global(reinterpret_cast<const f32x4_e4*>(p))->v);
    } else {
      w = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (c + e < cols) {
          if constexpr (sizeof(T) == 2) w[e >> 1] |= (uint32_t)as_global(reinterpret_cast<const uint16_t*>(row))[c + e] << (16 * (e & 1));
          else w[e] = as_global(reinterpret_cast<const uint32_t*>(row))[c + e];
        }
    }
  }
  __device__ __forceinline__ void settle(int c, int cols, bool ok) {
    const int over = SHORT ? 0 : max(c + PER - cols, 0);
    const int off = ok ? min(over, PER) : PER;  // elements to drop at the front
    if (__ballot(off != 0) == 0) return;
    const int regs = off * (int)sizeof(T) / 4;
#pragma unroll
    for (int b = 4; b >= 1; b >>= 1) {
      const bool take = (regs & b) != 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t from = j + b < 4 ? w[j + b] : 0u;
        w[j] = take ? from : w[j];
      }
    }
    if constexpr (sizeof(T) == 2) {
      const bool take = (off & 1) != 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t from = (w[j] >> 16) | (j + 1 < 4 ? w[j + 1] << 16 : 0u);
        w[j] = take ? from : w[j];
      }
    }
  }
};

// 16 bytes from LDS at a constant offset from addr, in inline assembly: for a
// read that the compiler sees it waits for all copies to LDS under way, as
// they might write what is read (the last quarter of every stage then took the
// time of its copies).
template <int OFF> __device__ __forceinline__ u32x4 lds_read_b128(uint32_t addr) {
  static_assert(OFF >= 0 && OFF < 65536, "ds offset field");
  u32x4 r;
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(r) : "v"(addr), "i"(OFF) : "memory");
  return r;
}

// Row block r (0 .. 3) of 32 rows of 128 bytes.
__device__ __forceinline__ u32x4 lds_read_b128_block(uint32_t addr, int r) {
  switch (r) {
    case 0: return lds_read_b128<0>(addr);
    case 1: return lds_read_b128<4096>(addr);
    case 2: return lds_read_b128<8192>(addr);
    default: return lds_read_b128<12288>(addr);
  }
}

// Waits for the fragments that MFMA p of a step is the first to use.  The
// compiler does not track reads in inline assembly.  LDS instructions of a wave
// complete in order, so it is enough that at most as many are outstanding as were
// issued after that fragment: this step's later fragments and the next step's
// first ones, IA or IB instructions each (0: reads that the compiler tracks; those
// and register writes are not counted, which only waits for more).  Reads come in
// the order A0, B0 .. B(NB-1), A1 .. A(NA-1).
template <int NA, int NB, int IA, int IB, typename P> __device__ __forceinline__ void experts_wait_frag(P) {
  constexpr int NDR = NA + NB, NPAIR = NA * NB, RPP = (NDR + NPAIR - 1) / NPAIR;
  constexpr int p = P::value, i = p / NB, j = p % NB;
  constexpr bool needA = j == 0 && IA > 0, needB = i == 0 && IB > 0;  // first uses
  if constexpr (needA || needB) {
    // position of that fragment in the reading order
    constexpr int at = needB ? j + 1 : (i == 0 ? 0 : NB + i);
    constexpr int later_a = NA - 1 - (at > NB ? at - NB : 0);
    constexpr int later_b = at <= NB ? NB - at : 0;
    constexpr int now = p * RPP < NDR ? p * RPP : NDR;  // reads issued so far in this step
    constexpr int now_a = (now > 0 ? 1 : 0) + (now > NB + 1 ? now - NB - 1 : 0);
    constexpr int now_b = now <= 1 ? 0 : (now - 1 < NB ? now - 1 : NB);
    constexpr int n = IA * (later_a + now_a) + IB * (later_b + now_b);
    __builtin_amdgcn_s_waitcnt(0xc07f | ((n < 15 ? n : 15) << 8));
    __builtin_amdgcn_sched_barrier(0);
  }
}

// One tile, of which the first 64 MA rows are computed (the others lie outside
// C): MA is the number of 32 x 32 blocks of a wave along M.  SKIP: waves whose
// blocks lie outside C leave their products out.
template <int MODE, int MA, bool DIRECT, bool SHORT, bool SKIP, typename TI, typename TO>
__device__ __forceinline__ void experts_compute(const ExpertsArgs& a, const ExpertTile& t, u32x4 (*ring)[2 * EXPERTS_T * 8]) {
  constexpr int T = EXPERTS_T;
  constexpr int NA = 1;                    // 32 x 32 blocks of a wave along N
  constexpr int NW = 8;
  constexpr bool AKM = MODE == EX_DW;      // A lies K-major
  constexpr bool BKM = MODE != EX_Y;       // B lies K-major
  constexpr int ES = (int)sizeof(TI);
  constexpr int EPC = 16 / ES;             // elements per 16-byte chunk
  constexpr int BK = 8 * EPC;              // K per stage
  constexpr int WGN = NW / 2;              // waves: 2 along M, NW / 2 along N
  constexpr int WN = 32 * NA;              // columns of a wave
  constexpr int OPS = T * 8;               // chunks of one operand's stage
  constexpr int STG = 2 * OPS;
  constexpr int NQ = OPS / (64 * NW);      // 16-byte pieces of one operand a thread moves per stage
  constexpr int NDR = MA + NA, NPAIR = MA * NA;
  constexpr int RPP = (NDR + NPAIR - 1) / NPAIR;  // fragment reads issued per MFMA
  constexpr int CR = T * ES / 16;          // chunks per K-row of a K-major stage
  constexpr int RPC = 64 / CR;             // K-rows per wave-wide copy
  static_assert(!DIRECT || ES == 2, "direct copies are bf16");
  static_assert(RPC >= 1 && BK * CR == OPS, "K-major stage");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  // SKIP: the lower half's waves turned by two, so that those inside a narrow C are on
  // all four SIMDs
  const int wm = wid / WGN, wn = SKIP ? (wid + wm * (WGN / 2)) % WGN : wid % WGN;
  const int half = lane >> 5, l32 = lane & 31;
  const int row0 = t.bi * T, col0 = t.bj * T;
  int ks0, ks1;
  experts_stages<MODE, BK>(a, t, ks0, ks1);
  const int nst = ks1 - ks0;
  const int M = MODE == EX_DW ? a.M : t.count;  // rows of C
  const int K = MODE == EX_DW ? t.count : a.K;
  const TI* A = static_cast<const TI*>(a.A) + (int64_t)t.begin * a.lda;
  const TI* B = static_cast<const TI*>(a.B) + (MODE == EX_DW ? (int64_t)t.begin * a.ldb : (int64_t)t.expert * a.se);

  // K-major chunk swizzle, see gemm.hpp
  auto swz_t = [](int krow) {
    return ES == 2 ? (((krow & 1) << 2) ^ (((krow >> 1) & 1) * 10)) : ((krow >> 2) & 1) << 3;
  };
  // the clamp compiles to a vector instruction: back to a scalar register, or
  // the loads' buffer resources count as divergent
  auto stage_rows = [&](int ks) { return __builtin_amdgcn_readfirstlane(max(0, min(BK, K - ks * BK))); };

  // Chunk q of a thread: row-major, tile row crow + 8 q at k ck[q & 1] of the
  // stage; K-major, K-row (wid NQ + q) RPC + lane / CR at column 8 ((lane % CR) ^ swz).
  const int rows_a = min(T, M - row0), rows_b = min(T, a.N - col0);
  const int crow = wid * (8 * NQ) + (lane >> 3);
  const int ck[2] = {((lane & 7) ^ (lane >> 3)) * EPC, ((lane & 7) ^ (lane >> 3) ^ 1) * EPC};
  auto km_row = [&](int q) { return (wid * NQ + q) * RPC + lane / CR; };
  auto km_col = [&](int q) { return ((lane % CR) ^ swz_t(km_row(q))) * EPC; };

  // ---- direct copies
  auto km_offset = [&](int par, int64_t ld, int c0, int cols) {
    const int col = c0 + km_col(par);
    return col < cols ? (uint32_t)(((int64_t)km_row(par) * ld + col) * ES) : OOB;
  };
  const uint32_t ta[2] = {km_offset(0, a.lda, row0, M), km_offset(1, a.lda, row0, M)};
  const uint32_t tb[2] = {km_offset(0, a.ldb, col0, a.N), km_offset(1, a.ldb, col0, a.N)};
  const TI* Arow = A + (AKM ? 0 : (int64_t)row0 * a.lda);
  const TI* Brow = B + (BKM ? 0 : (int64_t)col0 * a.ldb);
  auto copy_row_major = [&](const TI* base, int64_t ld, int rows, int region, int q, int v, int ks) {
    const __amdgpu_buffer_rsrc_t r = make_rsrc(base, (uint32_t)((((int64_t)rows - 1) * ld + K) * ES));
    const int k = ks * BK + ck[q & 1];
    const uint32_t off = k < K ? (uint32_t)(((crow + 8 * q) * ld + k) * ES) : OOB;
    copy16_to_lds(r, &ring[v & 1][region + (wid * NQ + q) * 64], off);
  };
  auto copy_k_major = [&](const TI* base, int64_t ld, int cols, const uint32_t(&o)[2], int region, int q, int v, int ks) {
    const int nk = stage_rows(ks);
    const __amdgpu_buffer_rsrc_t r =
        make_rsrc(base + (int64_t)ks * BK * ld, nk ? (uint32_t)((((int64_t)nk - 1) * ld + cols) * ES) : 0u);
    copy16_to_lds(r, &ring[v & 1][region + (wid * NQ + q) * 64],
                  o[q & 1] + (uint32_t)((int64_t)((q & ~1) * RPC) * ld * ES));
  };
  auto copy_a = [&](int q, int v, int ks) {
    if constexpr (AKM) copy_k_major(A, a.lda, M, ta, 0, q, v, ks);
    else if (MA == T / 64 || wid * (8 * NQ) < 64 * MA) copy_row_major(Arow, a.lda, rows_a, 0, q, v, ks);
  };
  auto copy_b = [&](int q, int v, int ks) {
    if constexpr (BKM) copy_k_major(B, a.ldb, a.N, tb, OPS, q, v, ks);
    else copy_row_major(Brow, a.ldb, rows_b, OPS, q, v, ks);
  };

  // ---- the same chunks through registers
  Piece<TI, SHORT> pa[DIRECT ? 1 : NQ], pb[DIRECT ? 1 : NQ];
  auto load_pieces = [&](int ks) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        // rows past the end: a row that is there, cleared by settle()
        if constexpr (AKM) pa[q].load(A + (int64_t)min(ks * BK + km_row(q), K - 1) * a.lda, row0 + km_col(q), M);
        else pa[q].load(Arow + (int64_t)min(crow + 8 * q, rows_a - 1) * a.lda, ks * BK + ck[q & 1], K);
        if constexpr (BKM) pb[q].load(B + (int64_t)min(ks * BK + km_row(q), K - 1) * a.ldb, col0 + km_col(q), a.N);
        else pb[q].load(Brow + (int64_t)min(crow + 8 * q, rows_b - 1) * a.ldb, ks * BK + ck[q & 1], K);
      }
    }
  };
  auto write_pieces = [&](int q, int v, int ks) {  // q < NQ: A, else B
    if constexpr (!DIRECT) {
      const int i = q < NQ ? q : q - NQ;
      Piece<TI, SHORT>& p = q < NQ ? pa[i] : pb[i];
      if (q < NQ ? AKM : BKM)
        p.settle((q < NQ ? row0 : col0) + km_col(i), q < NQ ? M : a.N, ks * BK + km_row(i) < K);
      else
        p.settle(ks * BK + ck[i & 1], K, crow + 8 * i < (q < NQ ? rows_a : rows_b));
      ring[v & 1][(q < NQ ? 0 : OPS) + (wid * NQ + i) * 64 + lane] = p.w;
    }
  };

  f32x16 acc[MA][NA];
#pragma unroll
  for (int i = 0; i < MA; ++i)
#pragma unroll
    for (int j = 0; j < NA; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  // ---- fragments, double buffered by k-step
  u32x4 fa[2][MA], fb[2][NA];
  const int rswz = (l32 & 7) ^ ((l32 >> 3) & 1);
  constexpr int ROWB = CR * 16;
  const uint32_t rd[2] = {
      (uint32_t)(uintptr_t)(lds_ptr_t)&ring[0][(wm * (32 * MA) + l32) * 8 + (half ^ rswz)],
      (uint32_t)(uintptr_t)(lds_ptr_t)&ring[0][OPS + (wn * WN + l32) * 8 + (half ^ rswz)]};
  uint32_t tbase[NDR];
#pragma unroll
  for (int r = 0; r < NDR; ++r) {
    const int e = (lane >> 2) & 3, q = lane & 3;
    const int region = r < MA ? 0 : OPS;
    const int rb = r < MA ? wm * (32 * MA) + r * 32 : wn * WN + (r - MA) * 32;
    const int col = rb + 16 * ((lane >> 4) & 1) + 4 * q;
    tbase[r] = (uint32_t)(uintptr_t)(lds_ptr_t)&ring[0][0] +
               (uint32_t)(region * 16 + (8 * half + e) * ROWB + ((col >> 3) ^ swz_t(e)) * 16 + (col & 7) * 2);
  }
  auto read_one = [&](int r, int v, int s, int slot) {
    const bool isA = r < MA;
    const int rb = isA ? wm * (32 * MA) + r * 32 : wn * WN + (r - MA) * 32;
    const u32x4* st = &ring[v & 1][isA ? 0 : OPS];
    u32x4 f;
    if (!(isA ? AKM : BKM)) {
      // chunk 2 s + half of the row, swizzled
      f = lds_read_b128_block((rd[isA ? 0 : 1] ^ (uint32_t)(32 * s)) + (uint32_t)((v & 1) * STG * 16), isA ? r : r - MA);
    } else if constexpr (ES == 2) {
      const uint32_t p = tbase[r] + (uint32_t)((v & 1) * STG * 16);
#pragma unroll
      for (int kq = 0; kq < 2; ++kq) {
        const uint2 w = lds_read_tr16_step<ROWB>(p, 2 * s + kq);
        f[2 * kq] = w.x;
        f[2 * kq + 1] = w.y;
      }
    } else {
      // 4 consecutive k of one column
      const int c = rb + l32;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 8 * s + 4 * half + e;
        f[e] = reinterpret_cast<const uint32_t*>(st)[(k * CR + ((c >> 2) ^ swz_t(k))) * 4 + (c & 3)];
      }
    }
    if (isA) fa[slot][r] = f;
    else fb[slot][r - MA] = f;
  };
  // reads in the order of first use: A0, B0 .. B(NA-1), A1 .. A(MA-1)
  auto ro = [](int p) { return p == 0 ? 0 : (p <= NA ? MA + p - 1 : p - NA); };
  auto wait_frag = [&](auto pc) {
    experts_wait_frag<MA, NA, AKM ? (ES == 2 ? 2 : 0) : 1, BKM ? (ES == 2 ? 2 : 0) : 1>(pc);
  };
  const bool inside = row0 + wm * (32 * MA) < M && col0 + wn * WN < a.N;
  auto mfma_pair = [&](int p, int slot) {
    if (SKIP && !inside) return;
    Mfma<TI>::run(acc[p / NA][p % NA], fa[slot][p / NA], fb[slot][p % NA]);
  };

  if (nst > 0) {
    // ---- prologue: stages 0 and 1 in LDS (through registers: stage 1 in those)
    if constexpr (DIRECT) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) copy_a(q, s, ks0 + s);
#pragma unroll
        for (int q = 0; q < NQ; ++q) copy_b(q, s, ks0 + s);
      }
    } else {
      load_pieces(ks0);
#pragma unroll
      for (int q = 0; q < 2 * NQ; ++q) write_pieces(q, 0, ks0);
      load_pieces(ks0 + 1);
    }
    if constexpr (DIRECT) wait_vmcnt_lgkm0<0>();
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
          if constexpr (!DIRECT) {
            // 2 NQ pieces over the last 2 of the 3 steps, after a head start for the loads
            constexpr int SLOTS = 2 * NPAIR, PER = (2 * NQ + SLOTS - 1) / SLOTS;
            const int at = (s - 1) * NPAIR + p;
#pragma unroll
            for (int c = 0; c < PER; ++c)
              if (at >= 0 && at * PER + c < 2 * NQ) write_pieces(at * PER + c, v + 1, ks0 + v + 1);
          }
          __builtin_amdgcn_sched_barrier(0);
        });
      }
      // stage v + 1 is whole and this wave is done reading stage v; after the
      // barrier that holds for every wave
      wait_vmcnt_lgkm0<0>();
      __syncthreads();
      __builtin_amdgcn_sched_barrier(0);
      load_pieces(ks0 + v + 2);
#pragma unroll
      for (int p = 0; p < NPAIR; ++p) {
        mfma_pair(p, 1);
        if constexpr (DIRECT) {
#pragma unroll
          for (int c = p; c < 2 * NQ; c += NPAIR) {
            if (c < NQ) copy_a(c, v + 2, ks0 + v + 2);
            else copy_b(c - NQ, v + 2, ks0 + v + 2);
          }
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
  TO* C = static_cast<TO*>(a.o) + (MODE == EX_DW ? (int64_t)t.expert * a.se : (int64_t)t.begin * a.ldo);
  static_for<0, MA>([&](auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value;
    const int gr0 = row0 + wm * (32 * MA) + i * 32;
#pragma unroll
    for (int j = 0; j < NA; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) strip[((e >> 2) * 8 + half * 4 + (e & 3)) * SROW + j * 32 + l32] = acc[i][j][e];
    wave_lds_sync();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = gr0 + dr0 + DRS * n;
      const float* sp = strip + (dr0 + DRS * n) * SROW + dc8;
      const f32x4 lo = *reinterpret_cast<const f32x4*>(sp);
      const f32x4 hi = *reinterpret_cast<const f32x4*>(sp + 4);
      float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      if (r < M && gj < a.N) {
        if (t.slot >= 0) {
          float* o = a.ws + t.slot * (T * T) + (r - row0) * T + (gj - col0);
          *as_global(reinterpret_cast<f32x4*>(o)) = lo;
          *as_global(reinterpret_cast<f32x4*>(o + 4)) = hi;
        } else {
          TO* o = C + (int64_t)r * a.ldo;
          if (MODE == EX_DW && a.accumulate) {
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

template <int MODE, bool DIRECT, typename TI, typename TO>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(4, 4)))
void experts_kernel(const ExpertsArgs a) {
  constexpr int T = EXPERTS_T;
  __shared__ u32x4 ring[2][2 * T * 8];
  ExpertTile t;
  if (!experts_tile<MODE, false>(a, blockIdx.x, t)) return;
  // a tile at C's edge of which half or less is inside computes that half: 64
  // experts of 1408 x 2048, 49152 rows lose a tenth of their work to edges
  // instead of a quarter
  const bool low = (MODE == EX_DW ? a.M : t.count) - t.bi * T <= T / 2;
  if constexpr (!DIRECT) {
    // one operand's rows are shorter than a 16-byte piece
    constexpr int PER = 16 / (int)sizeof(TI);
    if ((MODE != EX_Y && a.N < PER) || (MODE == EX_DW ? a.M : a.K) < PER) {
      experts_compute<MODE, 2, false, true, false, TI, TO>(a, t, ring);
      return;
    }
  }
  if constexpr (sizeof(TI) == 4) {
    // fp32, bound by its products: where blocks of waves lie outside C (us with and without:
    // 541 rows of 128 experts of 586 x 3008, input gradient 245 and 318; forward 29597 rows
    // of 3 of 59 x 9472 423 and 642; but 4000 of 64 of 1408 x 2048, few of them outside,
    // 463 and 392 with the branch in every tile)
    if ((MODE == EX_DW ? a.M : t.count) - t.bi * T <= 32 || a.N - t.bj * T <= 96) {
      if (low) experts_compute<MODE, 1, DIRECT, false, true, TI, TO>(a, t, ring);
      else experts_compute<MODE, 2, DIRECT, false, true, TI, TO>(a, t, ring);
      return;
    }
  }
  if (low) experts_compute<MODE, 1, DIRECT, false, false, TI, TO>(a, t, ring);
  else experts_compute<MODE, 2, DIRECT, false, false, TI, TO>(a, t, ring);
}

// Adds the partial tiles of a tile in order.  8 columns per thread, WGS
// workgroups per tile.  Parts without stages were written as zeros.
template <int MODE, typename TO> __global__ __launch_bounds__(256) void experts_join_kernel(const ExpertsArgs a) {
  constexpr int T = EXPERTS_T, WGS = T * T / 2048;
  ExpertTile t;
  if (!experts_tile<MODE, true>(a, (int)(blockIdx.x / WGS), t)) return;
  const int in = (int)(blockIdx.x % WGS) * 2048 + threadIdx.x * 8;  // first value within the tile
  const int r = t.bi * T + in / T, c = t.bj * T + in % T;
  if (r >= (MODE == EX_DW ? a.M : t.count) || c >= a.N) return;
  const float* w = a.ws + t.slot * (T * T) + in;
  float v[8] = {};
#pragma unroll 4
  for (int z = 0; z < t.parts; ++z)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 x = *as_global(reinterpret_cast<const f32x4*>(w + z * t.stride * (T * T) + 4 * h));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * h + e] += x[e];
    }
  TO* o = static_cast<TO*>(a.o) +
          (MODE == EX_DW ? (int64_t)t.expert * a.se : (int64_t)t.begin * a.ldo) + (int64_t)r * a.ldo;
  if (MODE == EX_DW && a.accumulate) {
    float old[8];
    piece_load(o, c, a.N, old);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += old[e];
  }
  piece_store(o, c, a.N, v);
}

}  // namespace muon
