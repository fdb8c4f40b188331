// Large products grouped by expert, gfx950: bf16 operands of whole 16-byte
// pieces, 256 x 256 tiles, one workgroup of 8 waves on each CU that computes tile
// after tile (see experts.hpp for the products and the layout of a stage).
//
// Between two tiles of a workgroup that starts anew lie its launch, the search for its
// tile, the way of its first stage from HBM and its epilogue: 11 us next to the
// 1.6 us of a stage of K, with 12 stages in the weight gradient of 768 rows an
// expert.  Here the copies run on into the next tile: after the last stages
// of a tile its successor's first two are under way while the sums are
// stored (through LDS of its own), and the matrix instructions go on with the
// first barrier.
//
// experts_list_kernel writes the tiles into a list per XCD first.  A workgroup
// begins with the places k, 32 + k and 64 + k of its XCD's list and then takes the
// next one that nobody has, asking for it two tiles ahead.  Chunks of neighbouring tiles
// share an XCD's L2.  What the last round of an XCD's 32 workgroups would compute
// with a few of them is cut into halves or quarters of tiles.  The weight gradient's lists begin with the experts
// of most rows, and those with more than `chunk` rows come in pieces that
// experts_sum_kernel adds up.  (The cheaper tiles at C's edges last in the other
// products' lists balanced the workgroups better and lost more by reading the
// weights of all experts once again: 49152 rows of 64 experts of 1408 x 2048 355
// instead of 310 us.)
//
// Measured at 49152 rows of 64 experts of 1408 x 2048, where a large library product's
// 1.36 PFLOP/s would take 208 us: forward 322 us a call, input gradient 302, weight
// gradient 342, with the matrix pipes busy 44 to 48, 49 to 55 and 41 to 42% at 1.8 to
// 2.06 GHz; traced over 23 calls in a row, without lists and sums, 363 (317 to 395),
// 329 (286 to 358) and 353 us (337 to 367).  16384 rows of 8 experts of 14336 x 4096:
// 1646 us a call, 1.17 PFLOP/s; 1713 traced (1608 to 1961), bound by power (busy 67 to
// 70%, the clock falls to 1.34 to 1.74 GHz).  In a stage the reads and copies of LDS
// take as many cycles as the matrix instructions (2048 of a CU's 128 bytes a cycle for
// operands that all lie K-major) in both; what the first has more of is tiles' ends,
// one in 32, 22 or 12 stages instead of 64, half-empty last tiles (8%) and the last
// round of workgroups.  A weight gradient that is added to reads C in an epilogue
// whose end the next tile waits for: 424 us (fp32 C 496, written 390).  Storing a tile by
// exchanges between lanes instead of through LDS changed nothing (forward 314 and 317).
// The list takes 5 us at 64 experts (weight gradient 8), 7 at 1024 and 11 at 2048; the
// weight gradient's, which compares every unit with every other, 11 at 256 experts
// and 113 at 1024.
#pragma once

#include "experts.hpp"

namespace muon {

constexpr int BIG_T = 256;
constexpr int BIG_EXPERTS = 2048;  // experts of a large product, at most: their sums lie in LDS
constexpr int BIG_UNITS = 2048;    // the same for experts + rows / chunk

// Inclusive prefix sums of the workgroup's 256 values; *total their sum.
__device__ __forceinline__ int block_prefix(int v, int* wave_sums, int* total) {
  const int wave = threadIdx.x >> 6;
  v = wave_prefix(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) wave_sums[wave] = v;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    before += w < wave ? wave_sums[w] : 0;
    all += wave_sums[w];
  }
  *total = all;
  return v + before;
}

// Place p of XCD x's list among tot tiles dealt in chunks of S, there and back; the
// rest that is no full round of chunks in equal parts.
__device__ __forceinline__ int big_deal(int x, int p, int tot, int S) {
  const int full = tot / (8 * S);
  if (p < full * S) {
    const int round = p / S;
    return (round * 8 + ((round & 1) ? 7 - x : x)) * S + p % S;
  }
  const int rest = tot - full * 8 * S, q = rest >> 3, r = rest & 7;
  return full * 8 * S + x * q + min(x, r) + (p - full * S);
}
__device__ __forceinline__ int big_count(int x, int tot, int S) {
  const int full = tot / (8 * S);
  const int rest = tot - full * 8 * S;
  return full * S + (rest >> 3) + (x < (rest & 7));
}
// Last index with sums[index] <= at, of n + 1 ascending sums from 0.
__device__ __forceinline__ int big_find(const int* sums, int n, int at) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sums[mid] <= at) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Workgroup x writes the list of XCD x.
template <int MODE> __global__ __launch_bounds__(256) void experts_list_kernel(const ExpertsArgs a) {
  constexpr int T = BIG_T;
  __shared__ int wave_sums[4];
  const int x = blockIdx.x, tid = threadIdx.x;
  ExpertsItem* out = a.items + (int64_t)x * a.cap;
  if (tid == 0) a.head->taken[x][0] = 96;  // three for each workgroup
  if constexpr (MODE != EX_DW) {
    __shared__ int first[BIG_EXPERTS + 1];  // tile rows of the experts before
    int sum = 0;
    for (int c = 0; c < a.experts; c += 256) {
      const int n = c + tid < a.experts ? experts_rows(a, c + tid).count : 0;
      int tot;
      const int pre = block_prefix((n + T - 1) / T, wave_sums, &tot);
      // more tile rows than the rows allow: the offsets go back, and the groups overlap
      if (tot > a.rows / T + min(a.experts, a.rows) - sum) {
        if (tid == 0) a.head->count[x] = 0;
        return;
      }
      if (c + tid < a.experts) first[c + tid + 1] = sum + pre;
      sum += tot;
    }
    if (tid == 0) first[0] = 0;
    __syncthreads();
    const int S = 4 * a.tilesN, n = big_count(x, sum * a.tilesN, S);
    // what is left over full rounds of 32 workgroups
    const int rest = n % 32, parts = rest == 0 || rest > 16 ? 1 : rest > 8 ? 2 : 4, cut = parts > 1 ? rest : 0;
    for (int p = tid; p < n; p += 256) {
      const int at = big_deal(x, p, sum * a.tilesN, S);
      const int e = big_find(first, a.experts, at / a.tilesN);
      const ExpertRows r = experts_rows(a, e);
      int bi, bj;
      experts_place(at - first[e] * a.tilesN, (r.count + T - 1) / T, a.tilesN, bi, bj);
      const ExpertsItem t = {r.begin, r.count, bi * T, bj * T, T | T << 16, e, -1, 0};
      if (p < n - cut) {
        out[p] = t;
      } else {
        for (int q = 0; q < parts; ++q) {  // halves along N, quarters along both
          ExpertsItem h = t;
          h.col0 += (q & 1) * (T / 2);
          h.row0 += (q >> 1) * (T / 2);
          h.size = (parts == 2 ? T : T / 2) | (T / 2) << 16;
          out[n - cut + (p - (n - cut)) * parts + q] = h;
        }
      }
    }
    if (tid == 0) a.head->count[x] = n + cut * (parts - 1);
  } else {
    // units: an expert, or a chunk of one
    __shared__ int first[BIG_EXPERTS + 1], slots[BIG_EXPERTS + 1];  // units and partial units of the experts before
    __shared__ int order[BIG_UNITS];
    const int tiles = a.tilesM * a.tilesN;
    int units = 0, parts = 0, split = 0;
    for (int c = 0; c < a.experts; c += 256) {
      const int n = c + tid < a.experts ? experts_rows(a, c + tid).count : 0;
      const int k = c + tid < a.experts ? max(1, (n + a.chunk - 1) / a.chunk) : 0;
      int tot, totp, tots;
      const int pre = block_prefix(k, wave_sums, &tot);
      const int prep = block_prefix(k > 1 ? k : 0, wave_sums, &totp);
      const int pres = block_prefix(k > 1, wave_sums, &tots);
      // More units than the rows allow: the offsets go back.  Within this there are no
      // more partial ones than 2 (rows / chunk) and no more experts in parts than
      // rows / chunk, as those have two units or more; lists and workspace have
      // room for them.
      if (units + tot > a.experts + a.rows / a.chunk || split + tots > EXPERTS_SPLIT) {
        if (tid == 0) {
          a.head->count[x] = 0;
          if (x == 0) a.head->splits = 0;
        }
        return;
      }
      if (c + tid < a.experts) {
        first[c + tid + 1] = units + pre;
        slots[c + tid + 1] = parts + prep;
        if (x == 0 && k > 1) {
          a.head->split[split + pres - 1].expert = c + tid;
          a.head->split[split + pres - 1].slot = (parts + prep - k) * tiles;
          a.head->split[split + pres - 1].chunks = k;
        }
      }
      units += tot;
      parts += totp;
      split += tots;
    }
    if (tid == 0) first[0] = slots[0] = 0;
    if (x == 0 && tid == 0) a.head->splits = split;
    __syncthreads();
    // unit u: expert, rows
    auto rows_of = [&](int u, int& e, int& j) {
      e = big_find(first, a.experts, u);
      j = u - first[e];
      const ExpertRows r = experts_rows(a, e);
      return ExpertRows{r.begin + j * a.chunk, min(a.chunk, r.count - j * a.chunk)};
    };
    __shared__ int rows[BIG_UNITS];
    for (int u = tid; u < units; u += 256) {
      int e, j;
      rows[u] = rows_of(u, e, j).count;
    }
    __syncthreads();
    for (int u = tid; u < units; u += 256) {
      int rank = 0;
      for (int v = 0; v < units; ++v) rank += rows[v] > rows[u] || (rows[v] == rows[u] && v < u);
      order[rank] = u;
    }
    __syncthreads();
    // chunks of the list: a unit's tiles, or at least 32 in groups of 4 tile rows
    const int S = tiles <= 96 ? tiles : 4 * a.tilesN * ((32 + 4 * a.tilesN - 1) / (4 * a.tilesN));
    const int n = big_count(x, units * tiles, S);
    for (int p = tid; p < n; p += 256) {
      const int at = big_deal(x, p, units * tiles, S);
      const int u = order[at / tiles];
      int e, j, bi, bj;
      const ExpertRows r = rows_of(u, e, j);
      experts_place(at % tiles, a.tilesM, a.tilesN, bi, bj);
      const bool part = first[e + 1] - first[e] > 1;
      out[p] = {r.begin, r.count, bi * T, bj * T, T | T << 16, e, part ? (slots[e] + j) * tiles + bi * a.tilesN + bj : -1, 0};
    }
    if (tid == 0) a.head->count[x] = n;
  }
}

// What an earlier kernel wrote, for scalar loads.
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef const __attribute__((address_space(4))) i32x8* item_ptr;
typedef const __attribute__((address_space(4))) int32_t* const_int_ptr;

// A word of LDS that is the same for all lanes.
__device__ __forceinline__ int lds_read_uniform(const int* p) {
  int r;
  asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(r) : "v"((uint32_t)(uintptr_t)(lds_ptr_t)p) : "memory");
  return __builtin_amdgcn_readfirstlane(r);
}

// The workgroup's barrier without the waits of __syncthreads(), which are for all
// memory instructions under way, the stores of the tile before among them.
// What has to be complete has been waited for in front of it.
__device__ __forceinline__ void big_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

template <int MODE, typename TO>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void experts_big_kernel(const ExpertsArgs a) {
  constexpr int T = BIG_T, NW = 8;
  constexpr bool AKM = MODE == EX_DW, BKM = MODE != EX_Y;  // operands that lie K-major
  constexpr int ES = 2, EPC = 8, BK = 64;
  constexpr int WGN = NW / 2;
  constexpr int OPS = T * 8, STG = 2 * OPS, NQ = OPS / (64 * NW);
  constexpr int CR = T / 8, RPC = 64 / CR, ROWB = CR * 16;
  constexpr int SROWS = 8;                 // rows of an epilogue strip
  __shared__ u32x4 ring[2][STG];
  __shared__ float strips[NW][SROWS * 64];
  __shared__ int mail[2];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / WGN, wn = wid % WGN;
  const int half = lane >> 5, l32 = lane & 31;
  const int x = blockIdx.x & 7, k0 = blockIdx.x >> 3;
  const int count = ((const_int_ptr)a.head)[x];
  const item_ptr list = (item_ptr)a.items + (int64_t)x * a.cap;
  auto item = [&](int p) {  // (the first one again past the end)
    return __builtin_bit_cast(ExpertsItem, (i32x8)list[p < count ? p : 0]);
  };
  if (k0 >= count) return;

  auto swz_t = [](int krow) { return ((krow & 1) << 2) ^ (((krow >> 1) & 1) * 10); };
  const int crow = wid * (8 * NQ) + (lane >> 3);
  const int ck[2] = {((lane & 7) ^ (lane >> 3)) * EPC, ((lane & 7) ^ (lane >> 3) ^ 1) * EPC};
  const int kmr[2] = {(wid * NQ) * RPC + lane / CR, (wid * NQ + 1) * RPC + lane / CR};
  const int kmc[2] = {((lane % CR) ^ swz_t(kmr[0])) * EPC, ((lane % CR) ^ swz_t(kmr[1])) * EPC};

  // ---- the copies' side: which stage of which item goes to the ring next
  // Items are opened in the order they are taken.  When one is opened, the place of
  // the next but one is asked for: one atomic of wave 0, which comes back by the
  // end of the stage; it goes to the other waves through `mail` before that stage's
  // barrier, and is read when the next item is opened.  The first three places
  // are fixed, as two items may be opened before the first barrier.
  int cks = 0, cn = 0, cg = 0;  // stage of the item, its stages, ring slot
  int opened = 0, next = 32 + k0, got = 0;
  bool cdone = false, asked = false;
  ExpertsItem nitem = item(next);
  int q0 = 0, q1 = 0, q2 = 0, queued = 0;  // places of the items opened and not computed yet
  const bf16 *cA = nullptr, *cB = nullptr;
  int crows_a = 0, crows_b = 0, cK = 0;
  uint32_t ta[2] = {OOB, OOB}, tb[2] = {OOB, OOB};
  auto ask = [&] {
    asked = true;
    if (tid == 0) got = (int)atomicAdd((uint32_t*)&a.head->taken[x][0], 1u);
  };
  auto open_item = [&](const ExpertsItem& t, int p) {
    q0 = queued == 0 ? p : q0;
    q1 = queued == 1 ? p : q1;
    q2 = queued == 2 ? p : q2;
    ++queued;
    cK = MODE == EX_DW ? t.count : a.K;
    cn = max(1, (cK + BK - 1) / BK);  // an expert without rows: a stage of zeros
    cks = 0;
    const int M = MODE == EX_DW ? a.M : t.count;
    crows_a = min(t.size & 0xffff, M - t.row0);
    crows_b = min(t.size >> 16, a.N - t.col0);
    cA = static_cast<const bf16*>(a.A) + (int64_t)t.begin * a.lda + (AKM ? 0 : (int64_t)t.row0 * a.lda);
    cB = static_cast<const bf16*>(a.B) +
         (MODE == EX_DW ? (int64_t)t.begin * a.ldb : (int64_t)t.expert * a.se + (BKM ? 0 : (int64_t)t.col0 * a.ldb));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if constexpr (AKM) ta[q] = kmc[q] < crows_a ? (uint32_t)(((int64_t)kmr[q] * a.lda + t.row0 + kmc[q]) * ES) : OOB;
      if constexpr (BKM) tb[q] = kmc[q] < crows_b ? (uint32_t)(((int64_t)kmr[q] * a.ldb + t.col0 + kmc[q]) * ES) : OOB;
    }
  };
  // buffer resources of the stage; of no bytes once all items are copied
  __amdgpu_buffer_rsrc_t ra, rb;
  auto open_stage = [&] {
    auto res = [&](const bf16* base, int64_t ld, int rows, int cols, bool km) {
      const int nk = __builtin_amdgcn_readfirstlane(max(0, min(BK, cK - cks * BK)));
      const int64_t last = km ? ((int64_t)nk - 1) * ld + cols : ((int64_t)rows - 1) * ld + cK;
      return make_rsrc(km ? base + (int64_t)cks * BK * ld : base,
                       cdone || nk == 0 || rows <= 0 ? 0u : (uint32_t)(last * ES));
    };
    ra = res(cA, a.lda, crows_a, a.M, AKM);
    rb = res(cB, a.ldb, crows_b, a.N, BKM);
    // row-major: copy q is 8 q rows further on than these
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = cks * BK + ck[q];
      if constexpr (!AKM) ta[q] = k < cK ? (uint32_t)(((int64_t)crow * a.lda + k) * ES) : OOB;
      if constexpr (!BKM) tb[q] = k < cK ? (uint32_t)(((int64_t)crow * a.ldb + k) * ES) : OOB;
    }
  };
  auto copy_one = [&](int c) {  // c < NQ: A, else B
    const int q = c < NQ ? c : c - NQ;
    const bool km = c < NQ ? AKM : BKM;
    const int64_t ld = c < NQ ? a.lda : a.ldb;
    const uint32_t off = (c < NQ ? ta : tb)[q & 1] + (uint32_t)((km ? (q & ~1) * RPC : 8 * q) * (int)ld * ES);
    copy16_to_lds(c < NQ ? ra : rb, &ring[cg & 1][(c < NQ ? 0 : OPS) + (wid * NQ + q) * 64], off);
  };
  auto close_stage = [&] {  // on to the next one
    ++cg;
    if (++cks >= cn && !cdone) {
      if (next >= count) {
        cdone = true;
      } else {
        const ExpertsItem t = nitem;
        const int p = next;
        next = ++opened == 1 ? 64 + k0 : lds_read_uniform(&mail[opened & 1]);
        nitem = item(next);
        ask();
        open_item(t, p);
      }
    }
  };
  auto post = [&] {  // before a stage's barrier, after its wait for the copies
    if (asked) {
      if (tid == 0) mail[(opened + 1) & 1] = got;
      wait_lgkm0();
      asked = false;
    }
  };

  // ---- fragments
  const int rswz = (l32 & 7) ^ ((l32 >> 3) & 1);
  const uint32_t ring0 = (uint32_t)(uintptr_t)(lds_ptr_t)&ring[0][0];

  int g = 0;  // ring slot of the stage that is computed next
  // C in whole 16-byte pieces, written and not added to: a strip is ST stores,
  // whichever of its lanes lie inside C
  constexpr int ST = sizeof(TO) / 2;
  const bool pieces = !(MODE == EX_DW && a.accumulate) && a.N % 8 == 0 && a.ldo % 8 == 0 &&
                      (MODE != EX_DW || a.se % 8 == 0) && (uintptr_t)a.o % 16 == 0;
  bool stored = false;  // the tile before was written so
  ExpertsItem now = item(k0);
  auto tile = [&](const ExpertsItem& t, int nst, auto mc, auto nc) __attribute__((always_inline)) {
    constexpr int MA = decltype(mc)::value, NA = decltype(nc)::value;  // 32 x 32 blocks of a wave along M and N
    constexpr int WN = 32 * NA, NDR = MA + NA, NPAIR = MA * NA, RPP = (NDR + NPAIR - 1) / NPAIR;
    f32x16 acc[MA][NA];
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
      for (int j = 0; j < NA; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    u32x4 fa[2][MA], fb[2][NA];
    const uint32_t rd[2] = {ring0 + (uint32_t)(((wm * (32 * MA) + l32) * 8 + (half ^ rswz)) * 16),
                            ring0 + (uint32_t)((OPS + (wn * WN + l32) * 8 + (half ^ rswz)) * 16)};
    uint32_t tbase[NDR];
#pragma unroll
    for (int r = 0; r < NDR; ++r) {
      const int e = (lane >> 2) & 3, q = lane & 3;
      const int rb_ = r < MA ? wm * (32 * MA) + r * 32 : wn * WN + (r - MA) * 32;
      const int col = rb_ + 16 * ((lane >> 4) & 1) + 4 * q;
      tbase[r] = ring0 + (uint32_t)((r < MA ? 0 : OPS) * 16 + (8 * half + e) * ROWB + ((col >> 3) ^ swz_t(e)) * 16 +
                                    (col & 7) * 2);
    }
    auto read_one = [&](int r, int v, int s, int slot) {
      const bool isA = r < MA;
      u32x4 f;
      if (!(isA ? AKM : BKM)) {
        // chunk 2 s + half of the row, swizzled
        f = lds_read_b128_block((rd[isA ? 0 : 1] ^ (uint32_t)(32 * s)) + (uint32_t)(((g + v) & 1) * STG * 16),
                                isA ? r : r - MA);
      } else {
        const uint32_t p = tbase[r] + (uint32_t)(((g + v) & 1) * STG * 16);
#pragma unroll
        for (int kq = 0; kq < 2; ++kq) {
          const uint2 w = lds_read_tr16_step<ROWB>(p, 2 * s + kq);
          f[2 * kq] = w.x;
          f[2 * kq + 1] = w.y;
        }
      }
      if (isA) fa[slot][r] = f;
      else fb[slot][r - MA] = f;
    };
    auto ro = [](int p) { return p == 0 ? 0 : (p <= NA ? MA + p - 1 : p - NA); };
    auto wait_frag = [&](auto pc) { experts_wait_frag<MA, NA, AKM ? 2 : 1, BKM ? 2 : 1>(pc); };
    auto mfma_pair = [&](int p, int slot) { Mfma<bf16>::run(acc[p / NA][p % NA], fa[slot][p / NA], fb[slot][p % NA]); };

    {
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
#pragma unroll
            for (int r = p * RPP; r < NDR && r < (p + 1) * RPP; ++r) read_one(ro(r), v, s + 1, (s + 1) & 1);
            // the scalar work for this stage's copies, here between MFMAs: behind the
            // barrier, where all waves would do it at once, it took 5% of the stage
            if (s == 1 && p == 0) {
              close_stage();
              open_stage();
            }
            __builtin_amdgcn_sched_barrier(0);
          });
        }
        // the next stage is whole and this wave is done reading this one; after
        // the barrier that holds for every wave
        // The stores of the tile before, 8 ST of a wave or more, were issued after the
        // copies of the next stage: as many may still be under way.
        wait_vmcnt<8 * ST>();
        if (v > 0 || !stored) wait_vmcnt<0>();
        wait_lgkm0();
        post();
        big_barrier();
#pragma unroll
        for (int p = 0; p < NPAIR; ++p) {
          mfma_pair(p, 1);
#pragma unroll
          for (int c = p; c < 2 * NQ; c += NPAIR) copy_one(c);
          // past the tile's last stage these read what the next tile begins with, and
          // are not used
#pragma unroll
          for (int r = p * RPP; r < NDR && r < (p + 1) * RPP; ++r) read_one(ro(r), v + 1, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      // the unused reads land before their registers are given to anything else
      wait_lgkm0();
      __builtin_amdgcn_sched_barrier(0);
    }
    g += nst;
    now = item(q0);  // the next one, on its way during the epilogue

    // ---- epilogue: strips of 8 rows of a wave, then 8 values of a row per lane
    constexpr int CW = WN / 8, DRS = 64 / CW;
    static_assert(DRS >= SROWS, "a lane takes one piece of a strip");
    float* strip = strips[wid];
    const int dr0 = lane / CW, dc8 = (lane % CW) * 8;
    const int gj = t.col0 + wn * WN + dc8;
    const int M = MODE == EX_DW ? a.M : t.count;
    const bool mine = dr0 < SROWS && gj < a.N;
    TO* C = static_cast<TO*>(a.o) + (MODE == EX_DW ? (int64_t)t.expert * a.se : (int64_t)t.begin * a.ldo) +
            (int64_t)t.row0 * a.ldo;
    // put(lo, hi): the lane's values of a strip; strips come in the order of their rows
    auto each_strip = [&](auto put) __attribute__((always_inline)) {
      static_for<0, 4 * MA>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value / 4, h = decltype(ic)::value % 4;
#pragma unroll
        for (int j = 0; j < NA; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) strip[(half * 4 + e) * WN + j * 32 + l32] = acc[i][j][4 * h + e];
        wave_lds_sync();
        const float* sp = strip + (dr0 % SROWS) * WN + dc8;
        put(*reinterpret_cast<const f32x4*>(sp), *reinterpret_cast<const f32x4*>(sp + 4));
        wave_lds_sync();
      });
    };
    if (pieces && (MODE != EX_DW || t.slot < 0)) {
      // through a resource that drops what lies outside C
      const int rows = min(T, M - t.row0);
      const __amdgpu_buffer_rsrc_t rc =
          make_rsrc(C, rows > 0 ? (uint32_t)((((int64_t)rows - 1) * a.ldo + a.N) * (int)sizeof(TO)) : 0u);
      const uint32_t step = (uint32_t)(SROWS * a.ldo * (int)sizeof(TO));
      uint32_t off = mine ? (uint32_t)(((int64_t)(wm * (32 * MA) + dr0) * a.ldo + gj) * (int)sizeof(TO)) : OOB;
      each_strip([&](const f32x4& lo, const f32x4& hi) __attribute__((always_inline)) {
        const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        buffer_store8<TO>(rc, off, v);
        off += step;
        asm volatile("" : "+v"(off));  // one register, not one per strip
      });
      static_assert(4 * MA >= 8, "strips of a tile");
      stored = true;
    } else {
      int r = wm * (32 * MA) + dr0;
      each_strip([&](const f32x4& lo, const f32x4& hi) __attribute__((always_inline)) {
        if (mine && t.row0 + r < M) {
          if (MODE == EX_DW && t.slot >= 0) {
            float* o = a.ws + (int64_t)t.slot * (T * T) + r * T + (gj - t.col0);
            *as_global(reinterpret_cast<f32x4*>(o)) = lo;
            *as_global(reinterpret_cast<f32x4*>(o + 4)) = hi;
          } else {
            float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
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
        r += SROWS;
        asm volatile("" : "+v"(r));
      });
      stored = false;
    }
  };

  // ---- the first two stages, then item by item
  open_item(item(k0), k0);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    open_stage();
#pragma unroll
    for (int c = 0; c < 2 * NQ; ++c) copy_one(c);
    if (s == 0) close_stage();  // the second one's follows in the first stage computed
  }
  wait_vmcnt_lgkm0<0>();
  post();
  big_barrier();
  while (queued > 0) {
    const ExpertsItem t = now;
    q0 = q1;
    q1 = q2;
    --queued;
    const int nst = max(1, ((MODE == EX_DW ? t.count : a.K) + BK - 1) / BK);
    const bool low = min(t.size & 0xffff, (MODE == EX_DW ? a.M : t.count) - t.row0) <= T / 2;
    const bool narrow = min(t.size >> 16, a.N - t.col0) <= T / 2;
    std::integral_constant<int, 1> c1;
    std::integral_constant<int, 2> c2;
    std::integral_constant<int, 4> c4;
    if (low && narrow) tile(t, nst, c2, c1);
    else if (low) tile(t, nst, c2, c2);
    else if (narrow) tile(t, nst, c4, c1);
    else tile(t, nst, c4, c2);
  }
  wait_vmcnt_lgkm0<0>();  // the copies that found nothing more
}

// Weight gradient: adds the partial tiles of the experts that were summed in
// chunks, in order.  8 columns per thread, 2048 values per workgroup at a time.
template <typename TO> __global__ __launch_bounds__(256) void experts_sum_kernel(const ExpertsArgs a) {
  constexpr int T = BIG_T, PER = T * T / 2048;
  const int tiles = a.tilesM * a.tilesN;
  const int64_t n = (int64_t)a.head->splits * tiles * PER;
  for (int64_t b = blockIdx.x; b < n; b += gridDim.x) {
    const int s = (int)(b / (tiles * PER)), tile = (int)(b / PER % tiles);
    const int in = (int)(b % PER) * 2048 + threadIdx.x * 8;
    const int bi = tile / a.tilesN, bj = tile % a.tilesN;
    const int r = bi * T + in / T, c = bj * T + in % T;
    if (r >= a.M || c >= a.N) continue;
    const auto& sp = a.head->split[s];
    const float* w = a.ws + ((int64_t)sp.slot + tile) * (T * T) + in;
    float v[8] = {};
    for (int z = 0; z < sp.chunks; ++z)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 p = *as_global(reinterpret_cast<const f32x4*>(w + (int64_t)z * tiles * (T * T) + 4 * h));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * h + e] += p[e];
      }
    TO* o = static_cast<TO*>(a.o) + (int64_t)sp.expert * a.se + (int64_t)r * a.ldo;
    if (a.accumulate) {
      float old[8];
      piece_load(o, c, a.N, old);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += old[e];
    }
    piece_store(o, c, a.N, v);
  }
}

}  // namespace muon
