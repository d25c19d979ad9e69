// Walks the items that a grid's units take of a linear map's backward products, as the
// kernels do, for `shapes` drawn sizes and the SM counts given, and prints how many
// shapes leave an item out or take one twice.  Arguments: shapes, SM counts...
// With "turns rows in out": how often dw's early items go round.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <cmath>
#include <random>
#include <vector>

#include "linear_plan.hpp"

using namespace zeroadam;

static bool every_item_once(const Plan& p, int sms) {
  const int64_t items = p.whole + int64_t{p.tail} * p.splits;
  if (items == 0) return true;
  const int64_t units = p.gather ? items : grid_units(p, sms);
  const Turns turns{early_units_on(p, units), p.early_tiles, static_cast<int>(units)};
  std::vector<int> taken(items, 0);
  for (int u = 0; u < units; ++u)
    for (int t = turns.first(u); t < items; t = turns.after(t)) ++taken[t];
  for (int n : taken)
    if (n != 1) return false;
  return true;
}

int main(int argc, char** argv) {
  if (std::strcmp(argv[1], "turns") == 0) {
    const Plan dw = plan_backward({std::atoll(argv[2]), std::atoll(argv[3]), std::atoll(argv[4]), 0, 0, 0, 0,
                                   0, 0, 0, 0}, true, true).dw;
    std::printf("%d\n", dw.early_units > 0 ? dw.early_tiles / dw.early_units : 0);
    return 0;
  }
  std::mt19937 rng(1);
  std::uniform_real_distribution<double> d(0.0, 1.0);
  const auto draw = [&](double low, double high) {
    return static_cast<int64_t>(std::lround(std::exp(std::log(low) + d(rng) * std::log(high / low))));
  };
  std::vector<zero_linear_t> shapes;
  const int64_t known[][3] = {{8192, 2048, 8192}, {8192, 768, 50304}, {2048, 4096, 11008},
                              {713, 6493, 678},   {4341, 2240, 9408}, {2180, 4288, 9280},
                              {1024, 1024, 1024}, {1, 1, 1}};
  for (const auto& k : known) shapes.push_back({k[0], k[1], k[2], 0, 0, 0, 0, 0, 0, 0, 0});
  for (int i = 0; i < std::atoi(argv[1]); ++i)
    shapes.push_back({draw(1, 16384), draw(64, 12000), draw(64, 52000), 0, 0, 0, 0, 0, 0, 0, 0});
  std::vector<BackwardPlan> plans;
  int turns = 0;  // plans whose early items go round more than once
  for (const zero_linear_t& s : shapes) {
    plans.push_back(plan_backward(s, true, true));
    turns += plans.back().dw.early_tiles > plans.back().dw.early_units;
  }
  std::printf("turns %d\n", turns);
  for (int a = 2; a < argc; ++a) {
    int wrong = 0;
    for (const BackwardPlan& p : plans)
      wrong += !every_item_once(p.dx, std::atoi(argv[a])) || !every_item_once(p.dw, std::atoi(argv[a]));
    std::printf("%s %d\n", argv[a], wrong);
  }
}
