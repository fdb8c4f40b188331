// Host side of the linear layer on 8-bit rows: which kernel a product takes.
// No HIP in here, so that a host program can ask for the choice.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "libmuon.h"
#include "plan.hpp"

namespace muon {

// Tile, split and workspace of a product of the 8-bit linear layer.
struct Linear8Plan {
  bool few;       // few tokens: no tiles
  bool expanded;  // gradients: the 8-bit operand as bf16 in the workspace first
  bool dy_f32;    // gradients: the product itself cuts fp32 dy into its pieces
  int tile, splits, per_split;
  int64_t whole;  // tiles that are not split
  int64_t ldx, lddy;
  size_t dy_off, ws_off;  // workspace: expanded operand, planes of dy, partial results
  size_t bytes;
};
// Estimated time of a tiled product in us: what the choice between tiles,
// splits and expansion rests on.  The constants come from a fit to 1018 timings
// on one MI355X (21 shapes from 512 x 512 x 512 to 8192 x 4096 x 14336, all
// three passes; 10% rms; the choice cost 3% against the best one timed then);
// those of the 128 tiles were lowered by hand by what going from 4 to 8 waves
// gained afterwards, and the choice as a whole has not been timed since.
// Per stage of K (128 bytes of a row):
//   128 tiles  0.77 with one workgroup on a CU, 1.21 with two (forward 0.53,
//              0.90): bound by issue and LDS, not by memory (a ring of four
//              stages in LDS was no faster)
//   256 tiles  1.71 converting the 8-bit operand, 1.32 on the expanded one (forward
//              1.44) with all CUs at work, down to 0.84 (0.69) of it with few:
//              bound by power at full load
//   128 tiles  1.0 and 1.6 cutting fp32 dy into its pieces (input gradient 1.1
//              and 1.8)
// and a constant per round of workgroups; a second launch and partial tiles for
// a split; a launch and 3 bytes per element for the expansion; a launch and 4 or
// 10 bytes per element where dy is laid out as planes.  Cutting fp32 dy in the
// product saves those, and costs each stage (us against planes: 701 x 301 x
// 1531 20.2 and 25.0, 5451 x 64 x 11904 98 and 228, 4096 x 256 x 8192 94 and
// 147, but 1500 x 1500 x 1500 53.8 and 51.3).
// z parts of the tiles that do not fill a round (the chip holds 256 workgroups of
// 256 tiles, 512 of 128): 14336 x 4096 has 3.5 rounds of 256 tiles, and its last
// half round takes as long as a whole one unless it is split.
inline double linear8_cost(int pass, int tile, bool expanded, bool dy_f32, int64_t M, int64_t N, int64_t K,
                           int64_t nks, int64_t z, int planes) {
  const bool fwd = pass == MUON_LINEAR8_FORWARD, dw = pass == MUON_LINEAR8_WEIGHT_GRAD;
  const int64_t slots = tile == 128 ? 512 : 256;
  const int64_t tiles = ((M + tile - 1) / tile) * ((N + tile - 1) / tile);
  const int64_t rounds = tiles / slots, rem = tiles % slots;
  auto round = [&](int64_t wgs, double stages) {
    if (dy_f32) return stages * (wgs <= 256 ? (dw ? 1.0 : 1.1) : (dw ? 1.6 : 1.8)) + 5.0;
    if (tile == 128)
      return stages * (wgs <= 256 ? (fwd ? 0.53 : 0.77) : (fwd ? 0.90 : 1.21)) + (fwd ? 5.0 : 4.7);
    const double low = fwd ? 0.69 : 0.84, fill = (double)std::min<int64_t>(wgs, 256) / 256.0;
    return stages * (fwd ? 1.44 : expanded ? 1.32 : 1.71) * (low + (1.0 - low) * fill) + (fwd ? 9.3 : 7.6);
  };
  const double pieces = planes ? planes : 1;
  const double all = (double)nks * pieces, part = (double)((nks + z - 1) / z) * pieces;
  double us = (double)rounds * round(slots, all);
  for (int64_t left = rem * z; left > 0; left -= slots) us += round(std::min(left, slots), part);
  if (z > 1 && rem > 0)
    us += (fwd ? 3.3 : 5.9) + 8.0 * (double)z * (double)rem * (double)(tile * tile) / (fwd ? 7.7e6 : 9.0e6);
  if (planes && !dy_f32) us += 3.0 + (double)M * (double)K * (planes == 3 ? 10.0 : 4.0) / 5.0e6;
  if (expanded) us += 3.3 + 3.0 * (double)K * (double)N / 5.3e6;
  return us;
}

inline Linear8Plan linear8_plan(int pass, int64_t tokens, int64_t out, int64_t in, int planes) {
  const int64_t M = pass == MUON_LINEAR8_WEIGHT_GRAD ? out : tokens;
  const int64_t N = pass == MUON_LINEAR8_FORWARD ? out : in;
  const int64_t K = pass == MUON_LINEAR8_FORWARD ? in : pass == MUON_LINEAR8_WEIGHT_GRAD ? tokens : out;
  const int64_t nks = (K + (pass == MUON_LINEAR8_FORWARD ? 128 : 64) - 1) / (pass == MUON_LINEAR8_FORWARD ? 128 : 64);
  Linear8Plan p;
  // Few tokens: up to 16 the kernel bound by the weights is ahead at every size
  // measured (14336 x 4096, 16 tokens: 20.5 against 25 us in tiles).  Up to 64
  // it is while the weights are few, there are not so many channels that all
  // workgroups reading all tokens counts, and a workgroup's own share of them
  // stays short.  Against the tiles, us: 4096 x 4096, 64 tokens 13.0 / 14.8, 2048
  // x 8192, 32 tokens 13.9 / 14.2; beyond each bound 5120 x 5120, 32 tokens 20.5 /
  // 16.3, 16384 x 1024, 32 tokens 9.3 / 8.8, 2048 x 8192, 64 tokens 21.5 / 16.4,
  // 1024 x 14336, 64 tokens 34.3 / 17.6.
  p.few = pass == MUON_LINEAR8_FORWARD &&
          (tokens <= 16 || (tokens <= 64 && out <= 8192 && out * in <= ((int64_t)1 << 24) &&
                            tokens * in <= ((int64_t)1 << 18)));
  p.expanded = p.dy_f32 = false;
  p.ldx = p.lddy = 0;
  p.dy_off = p.ws_off = 0;
  if (p.few) {
    p.tile = 128;
    p.splits = 1;
    p.per_split = (int)nks;
    p.whole = 0;
    p.bytes = 0;
    return p;
  }
  const bool fwd = pass == MUON_LINEAR8_FORWARD;
  double best = 0.0;
  int64_t z = 0;
  for (int option = 0; option < (fwd ? 2 : planes == 3 ? 4 : 3); ++option) {
    const int tile = option == 0 || option == 3 ? 128 : 256;
    const bool expanded = option == 2, dy_f32 = option == 3;
    for (int64_t t = 1; t <= std::max<int64_t>(1, std::min<int64_t>(nks, 32)); ++t) {
      const double us = linear8_cost(pass, tile, expanded, dy_f32, M, N, K, nks, t, planes);
      if (z == 0 || us < best) {
        best = us;
        p.tile = tile;
        p.expanded = expanded;
        p.dy_f32 = dy_f32;
        z = t;
      }
    }
  }
  p.per_split = (int)std::max<int64_t>(1, (nks + z - 1) / z);
  p.splits = (int)std::max<int64_t>(1, (nks + p.per_split - 1) / p.per_split);
  const int64_t tiles = ((M + p.tile - 1) / p.tile) * ((N + p.tile - 1) / p.tile);
  const int64_t rem = tiles % (p.tile == 128 ? 512 : 256);
  if (rem == 0) p.splits = 1;
  p.whole = tiles - rem;
  if (p.expanded) {
    p.ldx = (N + 63) / 64 * 64;
    p.dy_off = (size_t)K * (size_t)p.ldx * 2;
  }
  p.ws_off = p.dy_off;
  if (planes && !p.dy_f32) {
    p.lddy = (out + 63) / 64 * 64;
    p.ws_off += (size_t)planes * (size_t)tokens * (size_t)p.lddy * 2;
  }
  p.bytes = p.ws_off + (p.splits > 1 ? (size_t)p.splits * (size_t)rem * (size_t)(p.tile * p.tile) * sizeof(float) : 0);
  if (p.bytes) p.bytes += WS_ALIGN;
  return p;
}

}  // namespace muon
