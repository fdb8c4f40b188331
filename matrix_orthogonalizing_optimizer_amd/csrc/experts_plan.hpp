// Host side of the products grouped by expert: which kernel a product takes.
// No HIP in here, so that a host program can ask for the choice.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "libmuon.h"
#include "plan.hpp"

namespace muon {

struct ExpertsPlan {
  bool few;       // forward, few rows an expert: no tiles
  bool big;       // 256 x 256 tiles from lists
  int tile, splits;
  int64_t tiles;  // most that any offsets need
  int64_t joined; // of them, those that are left in parts
  int64_t chunk;  // weight gradient: rows of an expert summed at once
  int64_t cap;    // big: room of a list
  size_t items_off, ws_off;  // workspace: lists, partial tiles
  size_t bytes;
};

// The few-row kernel's shape: tiles of 16 rows that a workgroup takes at a time,
// with two of them two groups of 16 channels; whole: K a multiple of a step.
// Two tiles of rows and two groups of channels read the rows half as often, and
// leave enough workgroups where the channels of all experts make 512 (us, one
// of each against two: 64 experts of 1408 x 2048, 384 rows 82 and 76, 1024 rows
// 131 and 103, before experts of at most 16 rows left the second tile out; but 64
// rows, one an expert, 38 and 39, 16 rows of one expert of 768 x 768 6.0 and 7.5).
// Where they do not, 4 tiles of rows from 8 rows an expert up (256 rows over 16
// experts of 512 x 513: 25 and 14 us).
struct ExpertsFewShape {
  int row_tiles;
  bool whole;
};
inline ExpertsFewShape experts_few_shape(int64_t rows, int64_t experts, int64_t out, int64_t in, int32_t dtype) {
  const int64_t some = std::min(experts, rows);
  const bool whole = in % (dtype == MUON_F32 ? 16 : 32) == 0;
  if (rows > 2 * some && some * ((out + 31) / 32) >= 512) return {2, whole};
  return {rows <= 8 * some ? 1 : 4, whole};
}

// direct: all operands are bf16 rows of whole 16-byte pieces.  out and in are 2^21
// at most, so that no product here overflows.
inline ExpertsPlan experts_plan(int pass, int64_t rows, int64_t experts, int64_t out, int64_t in, int32_t dtype,
                                bool direct) {
  const bool dw = pass == MUON_EXPERTS_WEIGHT_GRAD;
  const int64_t N = pass == MUON_EXPERTS_FORWARD ? out : in;
  const int64_t some = std::min(experts, rows);
  ExpertsPlan p{};
  p.tile = 128;
  p.splits = 1;
  // Few rows: the kernel that streams the weights is ahead of the tiles up to 12
  // rows an expert, where the products are dear (fp32) or the tiles do not fill
  // the chip up to 24, and up to 64 rows at all (us, against the tiles: 64 experts of
  // 1408 x 2048, 384 rows 74 and 87, 900 rows 88 and 84; 8 of 14336 x 4096, 96 rows
  // 204 and 206; 8 of 1024 x 1024, 200 rows 10.6 and 13.7, 500 rows 18.1 and 15.7;
  // fp32, 8 of 4096 x 4096, 150 rows 146 and 151, 190 rows 153 and 151, 64 of 1408 x
  // 2048, 1024 rows 193 and 208, 1500 rows 212 and 200; one of 768 x 768, 80 rows 10.3
  // and 11.2; odd widths: 8 of 1023 x 1025, 60 rows 14.9 and 17.1, 100 rows 23 and 18).
  // These rows are spread over the experts; the counts lie on the device, so the rule
  // cannot see them.  All of them on one expert of 64 of 1408 x 2048 (us, and the same
  // rows spread): 384 rows 95 and 73; 768 rows 190 and 82, where the tiles take 23 for
  // 769; fp32 1536 rows 723 and 220, the tiles 144 for 1537.
  const bool dear = dtype == MUON_F32 || (direct && some * ((out + 31) / 32) < 512);
  p.few = pass == MUON_EXPERTS_FORWARD && some <= 65535 && (out + 15) / 16 * some <= 1 << 22 &&
          (rows <= (dear ? 24 : 12) * some || rows <= 64);
  if (p.few) {
    p.tiles = (out + 15) / 16 * some;
    return p;
  }
  // forward, input gradient: tile rows that the offsets need at most; tiles when
  // every expert's last tile row is half full
  auto most = [&](int64_t t) { return rows / t + some; };
  auto tiles = [&](int64_t t) { return (dw ? experts * ((out + t - 1) / t) : rows / t + (some + 1) / 2) * ((N + t - 1) / t); };
  const int64_t per = ((out + 255) / 256) * ((N + 255) / 256);  // weight gradient: tiles of an expert
  // an expert with more rows than a CU sums over all is cut
  const int64_t share = (rows + 63) / 64 * per / 256;
  // (at most 2^29: the kernels add it to an expert's rows, up to 2^30, in 32 bits)
  constexpr int64_t MAX_CHUNK = (int64_t)1 << 29;
  p.chunk = std::min(MAX_CHUNK, 64 * std::max<int64_t>(8, share));
  // 256 x 256 tiles where there is about one for every CU.  us, against tiles of 128:
  // forward 4096 rows of 8 experts of 1408 x 2048, 120 tiles 43 and 34; weight
  // gradient 4096 rows of 8 of 512 x 1024, 64 tiles 34 and 25; from about 260 on
  // ahead: forward 16384 rows of 8 of 4096 x 4096 497 and 587, weight gradient 1024
  // rows of 2 of 4096 x 4096, 512 tiles 46 and 61, 4096 rows of 64 of 1408 x 2048 103
  // and 176 (but the forward product of the latter 120 and 102).  The lists hold 2048
  // experts, in the weight gradient experts and units: past that come the tiles of 128,
  // whose search for a tile is dear by then (40000 rows of 512 x 512: weight gradient at
  // 1900 experts 612, at 2048 2110; forward at 2048 257, at 4096 1357).
  p.big = direct && tiles(256) >= 240 && experts + (dw ? rows / p.chunk : 0) <= 2048;
  if (p.big) {
    p.tile = 256;
    p.tiles = dw ? (experts + rows / p.chunk) * per : most(256) * ((N + 255) / 256);
    p.cap = p.tiles / 8 + 32;  // 8 equal lists, the last tiles in up to 24 more parts
    p.items_off = 8192;  // behind the head
    p.ws_off = p.items_off + (size_t)p.cap * 8 * 32;
    p.bytes = p.ws_off + (dw ? (size_t)(2 * (rows / p.chunk) * per) * 256 * 256 * sizeof(float) : 0) + WS_ALIGN;
    return p;
  }
  // tiles of 128: two workgroups on a CU
  const int64_t bk = dtype == MUON_F32 ? 32 : 64, slots = 512;
  if (dw) {
    // Units as above, of 12 stages at least (us, against 8: 1000 rows of 2 experts of
    // 1024 x 1024 14 and 18, 49152 of one of 64 x 64 20 and 21, 10000 of 4 of 300 x 300
    // 23 and 22).  fp32 products fill the time of a CU: of 8 to 16, or of one to two
    // times its share, the stages of a unit with which the busiest CU has the least
    // to do (8, 12 and 16: 3001 rows of 7 of 513 x 767 53, 70 and 75; 2000 of 2 of
    // 768 x 768 52, 43 and 49).
    const int64_t mine = ((out + 127) / 128) * ((N + 127) / 128);
    int64_t unit = std::max<int64_t>(dtype == MUON_F32 ? 8 : 12, ((rows + bk - 1) / bk) * mine / slots);
    if (dtype == MUON_F32) {
      const int64_t from = unit, step = std::max<int64_t>(1, from / 16);
      double least = 0.0;
      for (int64_t s = from; s <= 2 * from; s += step) {
        const double units = (double)rows / (double)(bk * s) + 0.5 * (double)experts;  // the last ones half full
        const double work = std::ceil(units * (double)mine / 256.0) * (double)(s + 2);
        if (s == from || work < least) {
          least = work;
          unit = s;
        }
      }
    }
    p.chunk = std::min(MAX_CHUNK, bk * unit);
    p.tiles = (experts + rows / p.chunk) * mine;
    p.joined = rows / p.chunk * mine;
    p.bytes = p.joined ? (size_t)(2 * p.joined) * 128 * 128 * sizeof(float) + WS_ALIGN : 0;
    return p;
  }
  const int64_t K = pass == MUON_EXPERTS_FORWARD ? in : out;
  const int64_t stages = (K + bk - 1) / bk, n = std::max<int64_t>(1, tiles(p.tile));
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({slots / n, stages / 4, 32}));
  p.tiles = most(p.tile) * ((N + p.tile - 1) / p.tile);
  p.joined = p.splits > 1 ? p.tiles : 0;
  p.bytes = p.joined ? (size_t)p.joined * (size_t)p.splits * 128 * 128 * sizeof(float) + WS_ALIGN : 0;
  return p;
}

}  // namespace muon
