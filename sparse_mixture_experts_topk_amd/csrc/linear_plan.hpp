// Host side of the tiled dense product: the choice of tile and schedule.
#pragma once
#include <algorithm>

#include "linear_tiles.hpp"

namespace moe {

// Tile shapes (columns x rows), all 8 wavefronts.  A smaller tile reads more
// bytes per product but leaves fewer CUs idle and needs less splitting.
// kSlice: us per slice of 64 terms once the stream runs, by how many operands are
// stored [t][r] (0 forward, 1 dx, 2 dw: the transposing reads take LDS twice as
// long per byte, which binds the smaller tiles); kTile: us a tile costs beyond
// its slices.  Measured on MI355X: 4096^3 gives the slices (256 x 256: 1362 / 1322
// / 1241 TFLOP/s, 128 x 64: 723 / 488 / 406), 4099 x 4096 x 256 the tiles.
struct Tile256x256 { static constexpr int NS = 2, WR = 4, WC = 2, WA = 4, WB = 8; static constexpr double kSlice[3] = {1.45, 1.50, 1.61}, kTile = 4.5; };
struct Tile256x128 { static constexpr int NS = 3, WR = 4, WC = 2, WA = 4, WB = 4; static constexpr double kSlice[3] = {0.86, 0.93, 1.02}, kTile = 2.7; };
struct Tile128x128 { static constexpr int NS = 4, WR = 4, WC = 2, WA = 2, WB = 4; static constexpr double kSlice[3] = {0.51, 0.66, 0.76}, kTile = 1.6; };
struct Tile128x64 { static constexpr int NS = 6, WR = 4, WC = 2, WA = 2, WB = 2; static constexpr double kSlice[3] = {0.355, 0.535, 0.645}, kTile = 1.2; };
template <class C> using GeomOf = ProductGeom<C::NS, C::WR, C::WC, C::WA, C::WB>;

// Splitting a tail costs a second launch, and its partial tiles are written and
// read once: 509 x 4096 x 2048 split in two with 128 x 128 tiles, 17 MB: 8 us
// longer than its slices; with 256 x 256 tiles, 67 MB: 25 us.
constexpr double kJoinFixed = 4.0, kJoinPerByte = 0.32e-6;
// Slices of a split run, at least (8 against 4, us: 33 x 256 x 4096 10.2 / 11.7, 1 x
// 8176 x 408 backward 19.5 / 22.7).
constexpr int kMinSlices = 8;

struct ProductPlan {
  double cost = 1e30;                // us, without what all candidates share
  int row_tiles = 0, col_tiles = 0, KT = 0, grid = 0;
  bool split = false;
  size_t workspace = 0;

  template <class C>
  static ProductPlan of(int rows, int cols, int len, int slow, int64_t cus) {
    using G = GeomOf<C>;
    ProductPlan best;
    for (int split = 0; split < 2; ++split) {
      ProductPlan p;
      p.row_tiles = (rows + G::TB - 1) / G::TB;
      p.col_tiles = (cols + G::TA - 1) / G::TA;
      p.KT = (len + G::BK - 1) / G::BK;
      p.split = split != 0;
      const int64_t tiles = (int64_t)p.row_tiles * p.col_tiles;
      const int64_t per_xcd = (tiles + 7) / 8, most = 8 * (p.split ? per_xcd * p.KT / kMinSlices : per_xcd);
      p.grid = (int)std::max<int64_t>(8, std::min<int64_t>(cus, most));
      const TileShare s = TileShare::of((int)tiles, 0, p.grid / 8, p.KT, p.split);      // the largest share
      const double parts = p.split ? 8.0 * (p.grid / 8 + s.tail) * G::PARTIAL * 4 : 0;
      p.cost = ((double)s.R * p.KT + (p.split ? s.P : s.tail > 0 ? p.KT : 0)) * C::kSlice[slow] +
               (s.R + (s.tail > 0 ? 1 : 0)) * C::kTile + (p.split ? kJoinFixed + kJoinPerByte * parts : 0);
      p.workspace = p.split ? (size_t)p.grid * 2 * G::PARTIAL * 4 : 0;
      if (p.cost < best.cost) best = p;
    }
    return best;
  }
};

// A product's plan in each of the four shapes, and the cheapest.
struct ProductPlans {
  ProductPlan p[4];
  int best = 0;

  static ProductPlans of(int rows, int cols, int len, int slow, int64_t cus) {
    ProductPlans s{{ProductPlan::of<Tile256x256>(rows, cols, len, slow, cus),
                    ProductPlan::of<Tile256x128>(rows, cols, len, slow, cus),
                    ProductPlan::of<Tile128x128>(rows, cols, len, slow, cus),
                    ProductPlan::of<Tile128x64>(rows, cols, len, slow, cus)}};
    for (int i = 1; i < 4; ++i)
      if (s.p[i].cost < s.p[s.best].cost) s.best = i;
    return s;
  }
  const ProductPlan& least() const { return p[best]; }
};
inline int64_t plan_cus(int cus) { return std::min<int64_t>(cus, kMaxPersistentGroups) / 8 * 8; }

// Calls run(tile shape) with shape i of the four.
template <class F>
auto with_tile(int i, F&& run) {
  if (i == 0) return run(Tile256x256{});
  if (i == 1) return run(Tile256x128{});
  if (i == 2) return run(Tile128x128{});
  return run(Tile128x64{});
}

// Workgroups of a join: every tail tile there may be (fewer than the slots of an XCD), all its rows.
template <class C>
unsigned join_blocks_of(const ProductPlan& p) {
  return (unsigned)(p.grid * (GeomOf<C>::TB / kJoinRows<GeomOf<C>::TA>));
}

template <bool PSLOW, bool QSLOW, int ACT>
hipError_t launch_product(const uint16_t* P, int64_t ldp, const uint16_t* Q, int64_t ldq, int rows, int cols,
                          int len, const ProductPlans& plans, void* partials, const Epilogue& ep, hipStream_t st) {
  const ProductPlan& p = plans.least();
  return with_tile(plans.best, [&](auto tile) {
    using C = decltype(tile);
    using G = GeomOf<C>;
    const ProductArgs a{P, Q, ldp, ldq, rows, cols, len, p.row_tiles, p.col_tiles, p.split,
                        static_cast<float*>(partials), ep};
    hipLaunchKernelGGL((linear_product_kernel<PSLOW, QSLOW, ACT, C::NS, C::WR, C::WC, C::WA, C::WB>),
                       dim3((unsigned)p.grid), dim3(G::THREADS), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.split) return e;
    hipLaunchKernelGGL((linear_join_kernel<ACT, G::TA, G::TB>), dim3(join_blocks_of<C>(p)), dim3(256), 0, st, a,
                       p.grid / 8);
    return hipGetLastError();
  });
}

}  // namespace moe
