// Host side of the feed-forward block's tiled products: the choice of tile and schedule.
#pragma once
#include <algorithm>

#include "ffn_tiles.hpp"
#include "linear_plan.hpp"

namespace moe {

// How the rows of the groups fall is known to the device alone: the plan takes them as
// even, each group half a tile short of its last.
struct FfnPlan {
  double cost = 1e30;      // us
  int shape = 0;           // tile, as with_tile counts them
  int row_tiles = 0, col_tiles = 0, grid = 0, split_ns = 0;
  size_t workspace = 0;

  // Rounds of tiles from which on a tail is not worth a join's launch.
  static constexpr int kNoTail = 24;

  template <class C>
  static FfnPlan of_tile(const moe_ffn_t& f, int kind, int shape, int64_t cus) {
    using G = GeomOf<C>;
    FfnPlan p;
    p.shape = shape;
    const bool over_rows = ffn_over_rows(kind);
    const int slow = kind == kGateUp ? 0 : over_rows ? 2 : 1;
    const int cols = kind == kGateUp ? 2 * f.d_ff : kind == kDh || kind == kDw2 ? f.d_ff : f.d_model;
    const int rows = kind == kDw2 ? f.d_model : f.d_ff, halves = kind == kDw13 ? 2 : 1;
    p.col_tiles = (cols + G::TA - 1) / G::TA;
    const double slice = C::kSlice[slow], tile = C::kTile;
    const int64_t row_tiles = (f.M + G::TB - 1) / G::TB, touched = std::min(f.groups, f.M);
    double tiles;
    int64_t most;            // tiles that any offsets can give
    int KT;
    if (over_rows) {
      p.row_tiles = (rows + G::TB - 1) / G::TB;
      most = (int64_t)f.groups * halves * p.row_tiles * p.col_tiles;
      tiles = (double)most;
      KT = std::max(slices_of((f.M + f.groups - 1) / f.groups), 1);
    } else {
      most = std::min<int64_t>(row_tiles + touched - 1, f.M) * p.col_tiles;
      tiles = (std::max<double>((double)f.M / G::TB + 0.5 * (touched - 1), f.groups == 1 ? row_tiles : 1)) * p.col_tiles;
      KT = (kind == kDx ? 2 : 1) * slices_of(kind == kDx ? f.d_ff : f.d_model);
    }
    const bool may_split = (!over_rows || f.groups == 1) && KT > kFfnMinSlices && tiles < (double)kNoTail * cus;
    const int64_t per_xcd = (most + 7) / 8;
    p.grid = (int)std::max<int64_t>(8, std::min<int64_t>(cus, 8 * (may_split ? per_xcd * KT / kFfnMinSlices : per_xcd)));
    const int slots = p.grid / 8;
    if (f.groups == 1) {
      const int ns = may_split ? (int)(slice * 1000) : 0;
      const FfnShare s = FfnShare::even((int)tiles, KT, 0, slots, ns, G::PARTIAL);      // the largest share
      p.cost = ((double)s.R * KT + (s.P > 0 ? s.P : s.tail > 0 ? KT : 0)) * slice + (s.R + (s.tail > 0 ? 1 : 0)) * tile;
      if (s.P > 0) p.cost += (kFfnJoinNs + 8.0 * (slots + s.tail) * G::PARTIAL / 256 * kFfnJoinNsPer100KiB / 100) * 1e-3;
    } else {
      const double rounds = tiles / p.grid;
      p.cost = may_split && rounds < 4 ? std::max(rounds, 0.25) * (KT * slice + tile) + 8
                                       : std::max(rounds + (rounds < 4 ? 0.5 : 0.0), 1.0) * (KT * slice + tile);
    }
    if (may_split) {
      p.split_ns = (int)(slice * 1000);
      p.workspace = (size_t)p.grid * 2 * G::PARTIAL * 4;
    }
    return p;
  }
  static FfnPlan of(const moe_ffn_t& f, int kind) {
    const int64_t cus = plan_cus(device_cu_count());
    const FfnPlan s[4] = {of_tile<Tile256x256>(f, kind, 0, cus), of_tile<Tile256x128>(f, kind, 1, cus),
                          of_tile<Tile128x128>(f, kind, 2, cus), of_tile<Tile128x64>(f, kind, 3, cus)};
    int best = 0;
    for (int i = 1; i < 4; ++i)
      if (s[i].cost < s[best].cost) best = i;
    return s[best];
  }
  // Whether a join has work to do, where the rows are known: one group of all M.
  template <class C>
  bool cuts(const moe_ffn_t& f, int kind) const {
    const bool over_rows = ffn_over_rows(kind);
    const int64_t total = over_rows ? (int64_t)(kind == kDw13 ? 2 : 1) * row_tiles * col_tiles
                                    : (int64_t)((f.M + GeomOf<C>::TB - 1) / GeomOf<C>::TB) * col_tiles;
    const int KT = over_rows ? slices_of(f.M) : (kind == kDx ? 2 : 1) * slices_of(kind == kDx ? f.d_ff : f.d_model);
    bool cut = false;
    for (int x = 0; x < 8; ++x)
      cut = cut || FfnShare::even((int)total, KT, x, grid / 8, split_ns, GeomOf<C>::PARTIAL).P > 0;
    return cut;
  }
};

template <int KIND>
hipError_t launch_ffn_tiles(const moe_ffn_t& f, FfnTileArgs a, void* partials, hipStream_t st) {
  const FfnPlan p = FfnPlan::of(f, KIND);
  a.M = f.M;
  a.groups = f.groups;
  a.act = f.act;
  a.row_tiles = p.row_tiles;
  a.col_tiles = p.col_tiles;
  a.split_ns = p.split_ns;
  a.partials = static_cast<float*>(partials);
  return with_tile(p.shape, [&](auto tile) {
    using C = decltype(tile);
    using G = GeomOf<C>;
    hipLaunchKernelGGL((ffn_tiles_kernel<KIND, C::NS, C::WR, C::WC, C::WA, C::WB>), dim3((unsigned)p.grid),
                       dim3(G::THREADS), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.split_ns == 0 || (a.offsets == nullptr && !p.template cuts<C>(f, KIND))) return e;
    constexpr int per_tile = G::TB / kFfnJoinRows<KIND, G::TA>;
    hipLaunchKernelGGL((ffn_join_kernel<KIND, G::TA, G::TB>), dim3((unsigned)(p.grid * per_tile)), dim3(256), 0, st, a,
                       p.grid / 8);
    return hipGetLastError();
  });
}

}  // namespace moe
