// Host driver of the planner of the linear layer on 8-bit rows
// (csrc/linear8_plan.hpp, no HIP).  Reads lines "pass tokens out in planes" and
// prints "tile form share splits per_split whole bytes" for each.
#include <cstdio>

#include "linear8_plan.hpp"

int main() {
  int pass, planes;
  long long t, n, k;
  while (std::scanf("%d %lld %lld %lld %d", &pass, &t, &n, &k, &planes) == 5) {
    const muon::Linear8Plan p = muon::linear8_plan(pass, t, n, k, planes);
    std::printf("%d %s %s %d %d %lld %zu\n", p.few ? 0 : p.tile,
                p.expanded ? "expanded" : p.dy_f32 ? "cut" : "converted",
                p.splits == 1 ? "none" : p.whole ? "some" : "all", p.splits, p.per_split, (long long)p.whole, p.bytes);
  }
  return 0;
}
