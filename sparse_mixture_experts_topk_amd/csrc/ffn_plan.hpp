// Host side of the feed-forward block's tiled products: the choice of tile and schedule.
#pragma once
#include <algorithm>

#include "ffn_tiles.hpp"
#include "linear_plan.hpp"

namespace moe {

// How the rows of the groups fall is known to the device alone: the plan takes them as
// even, each group half a tile short of its last.  For several groups the last round is
// therefore priced by fractions: where it may be cut and there are few rounds, by its part of a round
// (a quarter at least) and a join of 8 us; elsewhere few rounds are taken as half a
// round longer.  All gradients, us, so / by the rounds alone: 7080 rows of 2 groups of 1352 x
// 280 148 / 168, 600 of 4 of 2048 x 512 53 / 56, 1024 of 8 of 4096 x 2048 289 / 271; gate/up,
// 3000 of 4 of 1024 x 1408 39 / 41, 1024 of 8 of 4096 x 2048 81 / 87; 21 other cases the same.
struct FfnPlan {
  double cost = 1e30;      // us
  int row_tiles = 0, col_tiles = 0, grid = 0, split_ns = 0, cuts = 1;
  size_t workspace = 0;

  // Rounds of tiles from which on a tail is not worth a join's launch: what it saves, half a
  // round on average, is under 2%.  (All gradients, us, this / always a join / never: 8192 rows of
  // 8 groups of 4096 x 4096 1653 / 1655 / 1895, 4096 of 8 of 2048 x 4096 575 / 573 / 646, 509 x 4096 x
  // 2048 100 / 98 / 113.  Rows of several groups have a join launched that may find nothing to do:
  // 3000 of 4 of 1024 x 1408 126 / 126 / 117, gate/up of 2000 of 32 of 768 x 1024 40 / 40 / 27.)
  static constexpr int kNoTail = 24;

  template <class C>
  static FfnPlan of_tile(const moe_ffn_t& f, int kind, int64_t cus) {
    using G = GeomOf<C>;
    FfnPlan p;
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
      tiles = (double)touched * halves * p.row_tiles * p.col_tiles;
      KT = slices_of((f.M + touched - 1) / touched);
    } else {
      most = std::min<int64_t>(row_tiles + touched - 1, f.M) * p.col_tiles;
      tiles = (std::max<double>((double)f.M / G::TB + 0.5 * (touched - 1), f.groups == 1 ? row_tiles : 1)) * p.col_tiles;
      KT = (kind == kDx ? 2 : 1) * slices_of(kind == kDx ? f.d_ff : f.d_model);
    }
    const bool may_split = (!over_rows || f.groups == 1) && KT > kFfnMinSlices && tiles < (double)kNoTail * cus;
    if (over_rows && f.groups > 1) {             // few tiles: parts of them that fill the CUs once
      p.cuts = (int)std::max<int64_t>(1, std::min<int64_t>(cus / (int64_t)tiles, KT / kFfnMinSlices));
      most *= p.cuts;
    }
    const int64_t per_xcd = (most + 7) / 8;
    p.grid = (int)std::max<int64_t>(8, std::min<int64_t>(cus, 8 * (may_split ? per_xcd * KT / kFfnMinSlices : per_xcd)));
    const int slots = p.grid / 8;
    if (f.groups == 1) {
      const int ns = may_split ? (int)(slice * 1000) : 0;
      const FfnShare s = FfnShare::even((int)tiles, KT, 0, slots, ns, G::PARTIAL);      // the largest share
      p.cost = ((double)s.R * KT + (s.P > 0 ? s.P : s.tail > 0 ? KT : 0)) * slice + (s.R + (s.tail > 0 ? 1 : 0)) * tile;
      if (s.P > 0) p.cost += (kFfnJoinNs + 8.0 * (slots + s.tail) * G::PARTIAL / 256 * kFfnJoinNsPer100KiB / 100) * 1e-3;
    } else if (p.cuts > 1) {
      const double bytes = tiles * p.cuts * G::PARTIAL * 4;
      p.cost = (double)((KT + p.cuts - 1) / p.cuts) * slice + tile + kFfnJoinNs * 1e-3 + bytes / 1024 / 100 * kFfnJoinNsPer100KiB * 1e-3;
      p.workspace = (size_t)bytes;
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
  // Whether a join has work to do, where the rows are known: one group of all M.
  template <class C>
  bool has_tail(const moe_ffn_t& f, int kind) const {
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

// A product's plan in each of the four shapes, and the cheapest.
struct FfnPlans {
  FfnPlan p[4];
  int best = 0;

  static FfnPlans of(const moe_ffn_t& f, int kind) {
    const int64_t cus = plan_cus(device_cu_count());
    FfnPlans s{{FfnPlan::of_tile<Tile256x256>(f, kind, cus), FfnPlan::of_tile<Tile256x128>(f, kind, cus),
                FfnPlan::of_tile<Tile128x128>(f, kind, cus), FfnPlan::of_tile<Tile128x64>(f, kind, cus)}};
    for (int i = 1; i < 4; ++i)
      if (s.p[i].cost < s.p[s.best].cost) s.best = i;
    return s;
  }
  const FfnPlan& least() const { return p[best]; }
};

// Two products in one launch, with one tile shape: the second's workgroups fill the
// CUs that the first's last round leaves, and a launch is saved.  Worth kFfnOneLaunch
// us against each in its best shape.
constexpr double kFfnOneLaunch = 2.5;
// Its small tiles have two stages, so that a CU holds a workgroup of each product and one's
// start and epilogue fall under the other's products, which saves a share of short products' time, at most
// kPairSaves us.  All gradients, us, deep stages / two / two and this in the choice: 2108 x
// 1736 x 704 102 / 81 / 80; 509 x 4096 x 2048 108 / 107 / 101; 33 rows in 256 groups of 424 x 776
// 178 / 168 / 145; 3000 rows in 4 groups of 1024 x 1408 151 / 149 / 131.  (The share without a bound: 7351 rows in 256
// groups of 4096 x 2048 4590 -> 6310.)  Also where both products together leave every workgroup a CU of
// its own two stages are the faster, deep / two: 64 x 512 x 512 26.2 / 24.2, 300 x 1024 x 1024 42.0 / 34.1,
// 128 rows in 8 groups of 256 x 512 30.1 / 28.0.
constexpr double kPairOverlap = 0.28, kPairSaves = 25;
template <class C> constexpr int kPairStages = GeomOf<C>::TA * GeomOf<C>::TB <= 128 * 128 ? 2 : C::NS;
struct FfnPairPlan {
  FfnPlans a, b;
  int tile = 0;                      // the shape for both
  bool one;

  static FfnPairPlan of(const moe_ffn_t& f, int kind_a, int kind_b) {
    FfnPairPlan p{FfnPlans::of(f, kind_a), FfnPlans::of(f, kind_b)};
    for (int i = 1; i < 4; ++i)
      if (p.cost(i) < p.cost(p.tile)) p.tile = i;
    p.one = p.cost(p.tile) <= p.a.least().cost + p.b.least().cost + kFfnOneLaunch;
    return p;
  }
  double cost(int i) const {
    const double each = a.p[i].cost + b.p[i].cost;
    return i >= 2 ? each - std::min(kPairOverlap * each, kPairSaves) : each;
  }
  // partial tiles: both products', or those of one at a time
  size_t workspace() const {
    const size_t each = std::max(a.least().workspace, b.least().workspace);
    return one ? std::max(each, a.p[tile].workspace + b.p[tile].workspace) : each;
  }
};

inline FfnTileArgs planned(const moe_ffn_t& f, const FfnPlan& p, FfnTileArgs a, void* partials) {
  a.M = f.M;
  a.groups = f.groups;
  a.act = f.act;
  a.row_tiles = p.row_tiles;
  a.col_tiles = p.col_tiles;
  a.split_ns = p.split_ns;
  a.cuts = p.cuts;
  a.partials = static_cast<float*>(partials);
  return a;
}
// Workgroups of a product's join: every tail tile there may be (fewer than the slots of an XCD).
template <int KIND, class C>
unsigned ffn_join_blocks(const moe_ffn_t& f, const FfnPlan& p, const int32_t* offsets) {
  constexpr int per_tile = GeomOf<C>::TB / kFfnJoinRows<KIND, GeomOf<C>::TA>;
  if (p.cuts > 1) return (unsigned)((KIND == kDw13 ? 2 : 1) * std::min(f.groups, f.M) * p.row_tiles * p.col_tiles * per_tile);
  if (p.split_ns == 0 || (offsets == nullptr && !p.has_tail<C>(f, KIND))) return 0;
  return (unsigned)(p.grid * per_tile);
}

template <int KIND>
hipError_t launch_ffn_tiles(const moe_ffn_t& f, const FfnPlans& plans, const FfnTileArgs& args, void* partials,
                            hipStream_t st) {
  const FfnPlan& p = plans.least();
  const FfnTileArgs a = planned(f, p, args, partials);
  return with_tile(plans.best, [&](auto tile) {
    using C = decltype(tile);
    using G = GeomOf<C>;
    hipLaunchKernelGGL((ffn_tiles_kernel<KIND, C::NS, C::WR, C::WC, C::WA, C::WB>),
                       dim3((unsigned)p.grid), dim3(G::THREADS), 0, st, a);
    const hipError_t e = hipGetLastError();
    const unsigned joins = ffn_join_blocks<KIND, C>(f, p, a.offsets);
    if (e != hipSuccess || joins == 0) return e;
    hipLaunchKernelGGL((ffn_join_kernel<KIND, G::TA, G::TB>), dim3(joins), dim3(256), 0, st, a, p.grid / 8);
    return hipGetLastError();
  });
}

template <int KA, int KB>
hipError_t launch_ffn_pair(const moe_ffn_t& f, const FfnPairPlan& plan, const FfnTileArgs& args_a,
                           const FfnTileArgs& args_b, void* partials, hipStream_t st) {
  if (!plan.one) {
    const hipError_t e = launch_ffn_tiles<KA>(f, plan.a, args_a, partials, st);
    return e != hipSuccess ? e : launch_ffn_tiles<KB>(f, plan.b, args_b, partials, st);
  }
  const FfnPlan &pa = plan.a.p[plan.tile], &pb = plan.b.p[plan.tile];
  const FfnTileArgs a = planned(f, pa, args_a, partials);
  const FfnTileArgs b = planned(f, pb, args_b, static_cast<uint8_t*>(partials) + pa.workspace);
  return with_tile(plan.tile, [&](auto tile) {
    using C = decltype(tile);
    using G = GeomOf<C>;
    hipLaunchKernelGGL((ffn_pair_kernel<KA, KB, kPairStages<C>, C::WR, C::WC, C::WA, C::WB>),
                       dim3((unsigned)(pa.grid + pb.grid)), dim3(G::THREADS), 0, st, a, b, pa.grid);
    const hipError_t e = hipGetLastError();
    const unsigned ja = ffn_join_blocks<KA, C>(f, pa, a.offsets), jb = ffn_join_blocks<KB, C>(f, pb, b.offsets);
    if (e != hipSuccess || ja + jb == 0) return e;
    hipLaunchKernelGGL((ffn_pair_join_kernel<KA, KB, G::TA, G::TB>), dim3(ja + jb), dim3(256), 0, st, a, b, pa.grid / 8,
                       pb.grid / 8, (int)ja);
    return hipGetLastError();
  });
}

}  // namespace moe
