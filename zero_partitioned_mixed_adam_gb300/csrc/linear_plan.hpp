// linear_plan.hpp -- how a product of a linear map is cut into tiles and parts, and
// which of them each unit of the grid takes.  Host code, but for the shapes and the
// turns that the kernel shares; it compiles without CUDA.
#pragma once

#include <cstdint>

#include "zeroadam.h"

#ifdef __CUDACC__
#define ZERO_HD __host__ __device__
#else
#define ZERO_HD
#endif

namespace zeroadam {
namespace {

constexpr int kDepth = 64;         // steps of the reduction in one swizzled tile: 128 bytes
constexpr int kSub = 2;            // such tiles of each operand in one stage
constexpr int kStep = kSub * kDepth;
constexpr int kBlockRows = 128;    // rows of D per CTA: the lanes of tensor memory
constexpr int kEpilogueWarps = 8;  // two per quarter of the lanes
constexpr int kProductThreads = 64 + 32 * kEpilogueWarps;

// One tile of D is CG * 128 rows by bn columns (a multiple of 32, 256 or 128 at
// most), made by CG CTAs: each brings its own 128 rows of A and bn/CG rows of B,
// the tensor cores read both CTAs' B (half the shared-memory traffic of two
// tiles of their own), and each CTA's tensor memory ends up with its 128 rows.
// The ring has as many stages as fit.  Where D has fewer rows than a tile, only
// a_rows of A (a multiple of 8) are brought and given room: the tensor cores read
// on into whatever lies behind, and nothing is made of those rows of D.
constexpr int kStaging = kEpilogueWarps * 32 * 32 * 4;
constexpr int kMaxStages = 8;
constexpr int kBarriers = 256;
constexpr int kSmem = 227 * 1024;
static_assert((2 * kMaxStages + 5) * 8 <= kBarriers, "barriers, and two words");

template <int CG>
struct ProductShape {
  static constexpr int kMaxCols = CG == 2 ? 256 : 128;
  static constexpr int kColumns = 2 * kMaxCols;  // of tensor memory: two tiles
};
// Bytes of kDepth steps of one CTA's rows of A and B, and stages of the ring.
ZERO_HD constexpr int pair_bytes(int a_rows, int b_rows) {
  return (a_rows + b_rows) * kDepth * 2;
}
ZERO_HD constexpr int ring_stages(int a_rows, int b_rows) {
  const int n = (kSmem - 1024 - kStaging - kBarriers) / (kSub * pair_bytes(a_rows, b_rows));
  return n < kMaxStages ? n : kMaxStages;
}
static_assert(kStaging >= kBlockRows * kDepth * 2, "reads behind the last stage's A end in it");

ZERO_HD constexpr int64_t round_up(int64_t x, int64_t k) { return (x + k - 1) / k * k; }
ZERO_HD constexpr int64_t round_up4(int64_t x) { return round_up(x, 4); }

// The items of a unit (a CTA, or a pair): the early ones go round among the units that
// are there early, the rest among all.
struct Turns {
  int early_units, early_tiles, units;
  ZERO_HD inline int first(int unit) const {
    return unit < early_units ? unit : early_tiles + unit;
  }
  ZERO_HD inline int after(int t) const {
    return t + (t < early_tiles ? early_units : units);
  }
};

// Planned for the part's 152 SMs wherever it runs, so that the sums' order and
// the workspace follow from the sizes alone; a grid of other units takes the same
// items (early_units_on).
constexpr int kSms = 152;

// Rows of A that a CTA brings.
inline int a_rows_of(int64_t rows, int cg, bool a_mn) {
  return cg == 1 && !a_mn && rows < kBlockRows ? static_cast<int>(round_up(rows, 8)) : kBlockRows;
}

struct Plan {
  int cg, bn;
  int whole, splits;  // as in ProductArgs
  int tail;           // tiles split
  bool gather;        // the parts are a cluster's
  int early_units, early_tiles;  // as in ProductArgs
  double us;          // the estimate, with the wait for what it follows
  double last_us;     // of the last round, where that has whole tiles only
  int last_tiles;     // tiles of that round
  int64_t part_bytes() const {
    return splits > 1 && !gather ? int64_t{4} * tail * splits * cg * kBlockRows * bn : 0;
  }
};

// The shape of the tiles, and how the last round of them is spread: with T tiles
// on U units (pairs of SMs, or SMs) the tiles past the last multiple of U would
// leave most units idle, so their reduction may be cut into parts, which are
// joined by one more launch and two passes over them.  The least estimate in
// microseconds is taken, fitted to a sweep of 20 shapes: a stage of 256 x 256 on
// two SMs takes 0.65, of 256 x 128 0.47, of 128 x 128 on one SM 0.47, and no
// narrower tile less than 0.42; a stage's distinct rows of A and B come from HBM
// at 6.5 TB/s at best and 1.3 after they are asked for, a ring ahead, which is
// what counts for a few rows; 3 for a kernel's beginning and end, 0.9 for each 64
// columns of its last epilogue, 3 for the join's launch.
//
// follows: the product that is launched just before and does not have to end
// first, so that this one's tiles fill its last round: units without a tile there
// take theirs early, as many as they can do meanwhile (the first blocks of a grid
// get the first units that are free).  split: whether tiles past the last whole
// round may be.  most_parts: of a tile's reduction.
inline Plan plan_product(int64_t rows, int64_t cols, int64_t depth, bool a_mn, bool b_mn,
                  const Plan* follows = nullptr, bool split = true, int most_parts = 16) {
  Plan best{2, 256, 0, 1, 0, false, 0, 0, 0.0, 0.0, 0};
  if (rows < 1 || cols < 1) return best;
  const int steps = static_cast<int>((depth + kStep - 1) / kStep);
  best.us = 1e300;
  for (int cg = 2; cg >= 1; --cg) {
    const int most = cg == 2 ? 256 : 128;
    // MN-major operands come in columns of 64 per CTA
    const int unit = b_mn ? 64 * cg : 32;
    const int units = kSms / cg, a_rows = a_rows_of(rows, cg, a_mn);
    const int64_t tm = (rows + 128 * cg - 1) / (128 * cg);
    for (int bn = most; bn >= unit; bn -= unit) {
      const int64_t tn = (cols + bn - 1) / bn;
      if (tm * tn > INT32_MAX / 64) continue;
      const int tiles = static_cast<int>(tm * tn);
      const double share = static_cast<double>(bn) / most;
      const double mma = cg == 2 ? 0.40 + 0.25 * share * share : 0.42 + 0.055 * share * share;
      const double wait = 1.3 / ring_stages(a_rows, bn / cg);
      const double floor = mma > wait ? mma : wait;
      const auto stage = [&](int active) {
        const double distinct = static_cast<double>(active < tn ? active : tn) * bn +
                                static_cast<double>(active < tm ? active : tm) * 128 * cg;
        const double read = distinct * (2 * kStep) / 6.5e6;
        return floor > read ? floor : read;
      };
      const double tile = steps * stage(units), ends = 3.0 + 0.9 * bn / 64;
      const int taken = follows != nullptr ? follows->last_tiles * follows->cg : 0;  // SMs
      const int free = (kSms - taken) / cg;
      const bool fills = taken > 0 && free > 0;
      const double begin = follows != nullptr ? follows->last_us : 0.0;
      const int ahead = fills ? static_cast<int>(begin / tile) : 0;
      for (int turn = ahead; turn <= ahead + (fills ? 1 : 0); ++turn) {
        if (turn > 0 && turn > tiles / free) break;
        const int early = turn * free, rest = (tiles - early) % units;
        const int whole = tiles - rest;
        const double rounds_us = (whole - early) / units * tile;
        const double late_us = begin + rounds_us, early_us = turn * tile + rounds_us;
        const double all_us = late_us > early_us ? late_us : early_us;
        for (int parts = 1; parts <= most_parts; ++parts) {
          // (past two rounds of parts nothing was ever gained)
          if (parts > 1 && (rest == 0 || parts * 2 > steps || rest * parts > 2 * units ||
                            (!split && whole > 0)))
            break;
          Plan p{cg, bn, parts > 1 ? whole : tiles, parts, parts > 1 ? rest : 0, false,
                 fills ? free : 0, early, 0.0, 0.0, 0};
          if (p.part_bytes() > (int64_t{64} << 20)) break;
          const int items = rest * parts, rounds = (items + units - 1) / units;
          const double last =
              items > 0 ? rounds * ((steps + parts - 1) / parts) * stage(items < units ? items : units) : 0.0;
          if (parts == 1) {
            p.last_us = rest > 0 ? last : 0.0;
            p.last_tiles = rest;
          }
          const double end = fills && items <= free ? early_us + last : all_us + last;
          p.us = (end > late_us ? end : late_us) + ends;
          if (parts > 1) p.us += 3.0 + p.part_bytes() * 2 / 5.0e6;
          if (p.us < best.us) best = p;
          // A cluster's parts: 2.5 for the exchange.  (36 clusters of 4 fit.)
          if (cg == 1 && !a_mn && whole == 0 && ((parts == 2 && items <= 152) || (parts == 4 && items <= 144))) {
            p.gather = true;
            p.us = end + ends + 2.5;
            if (p.us < best.us) best = p;
          }
        }
      }
    }
  }
  return best;
}

// Units of a plan's grid on `sms` SMs: at most an item each.
inline int64_t grid_units(const Plan& p, int sms) {
  const int64_t units = sms / p.cg, items = p.whole + int64_t{p.tail} * p.splits;
  return items < units ? items : units;
}
// The units that its early items go round among: where fewer than the plan counts on
// are there, all of them.
inline int early_units_on(const Plan& p, int64_t units) {
  return p.early_units < units ? p.early_units : static_cast<int>(units);
}

inline Plan plan_forward(const zero_linear_t& s) {
  return plan_product(s.rows, s.out, s.in, false, false);
}

// dw's tiles fill dx's last round, or dx's last round is split.
struct BackwardPlan {
  Plan dx, dw;
};
inline BackwardPlan plan_backward(const zero_linear_t& s, bool dx, bool dw) {
  const auto first = [&](bool split) {
    return plan_product(s.rows, s.in, s.out, false, true, nullptr, split);
  };
  const auto second = [&](const Plan* follows) {
    return plan_product(s.out, s.in, s.rows, true, true, follows);
  };
  if (!dw) return {first(true), Plan{2, 256, 0, 1, 0, false, 0, 0, 0.0, 0.0, 0}};
  if (!dx) return {Plan{2, 256, 0, 1, 0, false, 0, 0, 0.0, 0.0, 0}, second(nullptr)};
  BackwardPlan filled{first(false), {}}, split{first(true), second(nullptr)};
  filled.dw = second(&filled.dx);
  return filled.dx.us - filled.dx.last_us + filled.dw.us <= split.dx.us + split.dw.us ? filled
                                                                                      : split;
}

}  // namespace
}  // namespace zeroadam
