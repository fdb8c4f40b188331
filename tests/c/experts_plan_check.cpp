// Host driver of the planner of the products grouped by expert
// (csrc/experts_plan.hpp, no HIP).  Reads lines "pass rows experts out in dtype
// direct" and prints "kernel tile splits tiles joined chunk cap bytes row_tiles
// whole" for each (the last two: shape of the few-row kernel, or 0).
#include <cstdio>

#include "experts_plan.hpp"

int main() {
  int pass, dtype, direct;
  long long r, e, o, i;
  while (std::scanf("%d %lld %lld %lld %lld %d %d", &pass, &r, &e, &o, &i, &dtype, &direct) == 7) {
    const muon::ExpertsPlan p = muon::experts_plan(pass, r, e, o, i, dtype, direct != 0);
    const muon::ExpertsFewShape f = p.few ? muon::experts_few_shape(r, e, o, i, dtype) : muon::ExpertsFewShape{};
    std::printf("%s %d %d %lld %lld %lld %lld %zu %d %d\n", p.few ? "few" : p.big ? "big" : "tiles", p.tile, p.splits,
                (long long)p.tiles, (long long)p.joined, (long long)p.chunk, (long long)p.cap, p.bytes, f.row_tiles, f.whole);
  }
  return 0;
}
