// The products of the feed-forward block (FfnKind) as streams of bf16 matrix-core tiles
// (tile_stream of linear_tiles.hpp) over groups of rows that only the device knows.
//
//   kind      rows (P)              columns (Q)                    terms
//   kGateUp   x [r][t]              w1, w3 [r][t], 16 + 16 in turn  d_model
//   kDh       dy [r][t]             w2 [t][r]                      d_model
//   kDx       dg then du [r][t]     w1 then w3 [t][r]              2 d_ff
//   kDw13     dg or du [t][r]       x [t][r]                       the group's rows
//   kDw2      dy [t][r]             h [t][r]                       the group's rows
//
// Nothing is transposed in memory and dh never goes there: kDh's epilogue meets each
// element of it with g and u and stores dg and du.  Every workgroup reads the offsets
// and finds its own tiles: they are cut into 8 contiguous shares, one per XCD, and its
// workgroups take full rounds of them.  The last, partial round is cut along the
// contraction where that is shorter by the plan's costs (FfnShare), its partial tiles
// joined in order by a second kernel; weight gradients of several groups have tiles of
// as many slices as their group has rows, so there the shares are even by slices, and
// where there are few tiles each is cut into as many parts (7080 rows in 2 groups of 1352
// x 280, all gradients: 227 -> 141 us); groups without rows have no tiles, and every workgroup of
// the launch clears a part of their gradients after its tiles (33 rows in 256 groups of 424 x 776, all gradients:
// 417 us as tiles of zeros, 184 by workgroups of their own, 178 so; 141 by now, with the pairs' two stages).
#pragma once
#include "device_common.hpp"
#include "ffn_groups.hpp"
#include "linear_tiles.hpp"

namespace moe {

// A split's join and its partial tiles in ns, and the least slices of a run (as in the
// dense product's plan).
constexpr int kFfnJoinNs = 4000, kFfnJoinNsPer100KiB = 33;
constexpr int kFfnMinSlices = 8;
// A tile's epilogue in slices, for shares that are even by slices.
constexpr int kFfnTileSlices = 3;

struct FfnTileArgs {
  const uint16_t *P0, *P1, *Q0, *Q1;      // P1, Q1: the second half where there are two
  const int32_t* offsets;
  int M, groups;
  int rows, cols, len;                    // kDw13, kDw2: rows of the weight; columns (kGateUp: channels); terms of a half
  int row_tiles, col_tiles;               // row_tiles: kDw13, kDw2, of a half
  int split_ns;                           // a slice, where there is room for partial tiles; else 0
  int cuts;                               // kDw13, kDw2 of several groups: parts of each contraction
  float* partials;
  const uint16_t *g, *u;                  // kDh
  uint16_t *o0, *o1, *o2;
  int act;
};

__host__ __device__ __forceinline__ int slices_of(int terms) { return (terms + 63) / 64; }

template <int KIND>
__device__ __forceinline__ void load_groups(FfnGroups& groups, const FfnTileArgs& a, int rows_per_tile) {
  // rows: tiles; weights: slices and the epilogue of one tile
  if constexpr (ffn_over_rows(KIND))
    groups.load(a.offsets, a.groups, a.M, [](int rows) { return slices_of(rows) + kFfnTileSlices; });
  else
    groups.load(a.offsets, a.groups, a.M, [=](int rows) { return (rows + rows_per_tile - 1) / rows_per_tile; });
}

// The XCD's share of the tile list: tiles begin .., R full rounds of its `slots`
// workgroups, then `tail` < slots tiles, taken whole (P = 0) or cut into runs of P slices,
// one per workgroup, each covering parts of at most two tiles.
struct FfnShare {
  int begin, R, tail, P, KT;              // KT: slices of a tile; 0: not the same for all

  // Of `total` tiles of KT slices (whole numbers, so that host and device agree).
  __host__ __device__ static FfnShare even(int total, int KT, int xcd, int slots, int split_ns, int tile_floats) {
    FfnShare s;
    const int per_xcd = (total + 7) >> 3;
    s.KT = KT;
    s.begin = xcd * per_xcd;
    const int end = s.begin + per_xcd < total ? s.begin + per_xcd : total, len = end > s.begin ? end - s.begin : 0;
    s.R = len / slots;
    s.tail = len - s.R * slots;
    s.P = 0;
    if (split_ns > 0 && s.tail > 0 && KT > kFfnMinSlices) {
      const int even = (s.tail * KT + slots - 1) / slots, P = even > kFfnMinSlices ? even : kFfnMinSlices;
      const int64_t parts = (int64_t)8 * (slots + s.tail) * tile_floats / 256;      // KiB
      if ((int64_t)P * split_ns + kFfnJoinNs + parts * kFfnJoinNsPer100KiB / 100 < (int64_t)KT * split_ns) s.P = P;
    }
    return s;
  }
  template <int KIND>
  __device__ static FfnShare of(const FfnTileArgs& a, const FfnGroups& groups, int xcd, int slots, int tile_floats) {
    const int per_group = (KIND == kDw13 ? 2 : 1) * a.row_tiles * a.col_tiles;
    if (!ffn_over_rows(KIND))
      return even(groups.before(a.groups) * a.col_tiles, (KIND == kDx ? 2 : 1) * slices_of(a.len), xcd, slots, a.split_ns,
                  tile_floats);
    if (a.groups == 1)
      return even(per_group, max(slices_of(groups.first(1) - groups.first(0)), 1), xcd, slots, a.split_ns, tile_floats);
    FfnShare s;
    s.KT = s.P = 0;
    s.begin = bound(groups, a.groups, per_group * a.cuts, xcd);
    const int len = bound(groups, a.groups, per_group * a.cuts, xcd + 1) - s.begin;
    s.R = len / slots;
    s.tail = len - s.R * slots;
    return s;
  }

 private:
  // First tile of XCD x's share, tiles counted over the groups that have rows: an eighth
  // of all slices each, to a tile.
  __device__ static int bound(const FfnGroups& groups, int n, int per_group, int x) {
    if (groups.full_before(n) == 0) return 0;
    if (x == 8) return groups.full_before(n) * per_group;
    const int64_t to = (int64_t)x * per_group * groups.before(n) / 8;      // slices before it
    const int e = groups.of((int)(to / per_group), n);
    const int w = groups.before(e + 1) - groups.before(e);
    const int in = (int)((to - (int64_t)per_group * groups.before(e) + w - 1) / w);
    return groups.full_before(e) * per_group + min(in, per_group);
  }
};

// Four values as bf16.
template <class V>
__device__ __forceinline__ u32x2_t pack4(const V& v) {
  return u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// A product leaves lane (i, g) with 4 columns of row i from each block; a store wants
// neighbouring lanes on neighbouring columns, for memory takes whole 128-byte lines far
// better than 64 scattered pieces of 16 bytes (the weight gradients of 8 groups of 1024
// rows, 4096 x 14336: 2 x 1875 us against 2120, 935 against 1010).  A row block goes
// through 1 KiB of LDS of the wavefront's own: one wavefront's LDS operations execute in
// order, so nothing waits but the reads' results.
//
// `Columns` = 64: 8 rows of 128 bytes at a time, 8 lanes a row; 32: 16 rows of 64 bytes, 4
// lanes a row.  The 16-byte chunks are swizzled by row.
template <int Columns>
struct RowStore {
  static constexpr int ROWS = 512 / Columns, LANES = Columns / 8, TIMES = 16 / ROWS;
  static_assert(Columns == 64 || Columns == 32, "a wavefront's columns");
  __device__ static __forceinline__ int key(int row) { return Columns == 64 ? row : row >> 2; }
  // This lane's row and first column in time 0.
  __device__ static __forceinline__ int row(int lane) { return lane / LANES; }
  __device__ static __forceinline__ int column(int lane) { return lane % LANES * 8; }
  // w: 4 columns of each 16-column block of row i; v[n]: 8 columns of row n ROWS + row(lane).
  __device__ static __forceinline__ void turn(uint8_t* lds, const u32x2_t (&w)[Columns / 16], int lane,
                                              u32x4_t (&v)[TIMES]) {
    const int i = lane & 15, g = lane >> 4, r = i % ROWS;
    uint8_t* to = lds + r * (Columns * 2) + (g & 1) * 8;
    const uint8_t* from = lds + row(lane) * (Columns * 2) + ((lane % LANES ^ key(row(lane))) << 4);
#pragma unroll
    for (int n = 0; n < TIMES; ++n) {
      if (TIMES == 1 || i / ROWS == n) {
#pragma unroll
        for (int x = 0; x < Columns / 16; ++x)
          *reinterpret_cast<u32x2_t*>(to + ((2 * x + (g >> 1)) ^ key(r)) * 16) = w[x];
      }
      asm volatile("" ::: "memory");             // (every lane's part, before any lane's read)
      v[n] = *reinterpret_cast<const u32x4_t*>(from);
      asm volatile("" ::: "memory");
    }
  }
};

// A tile's part of a bf16 output: a store outside the tile's rows or columns is dropped.
struct TileOut {
  __amdgpu_buffer_rsrc_t desc;
  // rows, cols: what there is from the tile's first row r0 and column c0 on
  __device__ __forceinline__ TileOut(uint16_t* out, int64_t ld, int r0, int c0, int rows, int cols)
      : desc(__builtin_amdgcn_make_buffer_rsrc(out + r0 * ld + c0, 0, (int)(((rows - 1) * ld + cols) * 2), kRawBufferFlags)) {}
  template <bool STREAM>
  __device__ __forceinline__ void store(int off, u32x4_t v) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, desc, off, 0, STREAM ? 2 : 0);      // 2: non-temporal
  }
  __device__ __forceinline__ void store(int off, u32x2_t v) const {
    __builtin_amdgcn_raw_buffer_store_b64(v, desc, off, 0, 0);
  }
};

// dg and du of 8 elements of dh, rounded to bf16, for the matrix cores take both operands in
// one type: dx, dw1 and dw3 are then 2.35e-3 of their size from the exact ones, where their
// own rounding alone makes 1.66e-3.  (Nothing else is lost: elementary products with the
// same rounding have the same bits in over 99% of the elements.)  Their low halves as
// further operands would take that away and double the terms of dx, dw1 and dw3, 3600 of
// 5700 us at 8192 rows of 8 groups of 4096 x 14336; fp32 operands keep all of it.
template <int KIND>
__device__ __forceinline__ void gated_gradients(const FfnTileArgs& a, const float (&dh)[8], uint4 g, uint4 u, uint4& dg,
                                                uint4& du) {
  float vg[8], vu[8];
  unpack8(g, vg);
  unpack8(u, vu);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float value, slope;
    act_both<false>(vg[k], a.act, value, slope);
    vg[k] = dh[k] * vu[k] * slope;
    vu[k] = dh[k] * value;
  }
  dg = pack8(vg);
  du = pack8(vu);
}

struct FfnLds {
  __attribute__((aligned(16))) uint8_t turned[8][1024];
  FfnGroups groups;
};

// The job of workgroup `block` of `blocks` (a multiple of 8).
template <int KIND, class G>
struct FfnJob {
  static constexpr bool kOverRows = ffn_over_rows(KIND), kPair = KIND == kGateUp;
  static constexpr bool kNt = G::STREAM && (KIND == kDw13 || KIND == kDw2);
  static constexpr int kStores = kPair ? G::WB : KIND == kDh ? G::WA * G::WB : G::WA * G::WB / 2;
  // e: group; r0, r_end: rows (of the weight for its gradients); first, terms: kDw13, kDw2,
  // the group's rows; half: kDw13, of w3
  struct Item { int e, r0, r_end, c0, first, terms, half, kb, ke, part; };
  const FfnTileArgs& a;
  const FfnGroups& groups;
  uint8_t* turned;                        // 1 KiB of LDS of this wavefront's
  FfnShare sp;
  int slots, xcd, slot, n_whole, run0, run1, n_items, wave, half_slices;
  int load_e = 0, tile_e = 0;             // groups of the two cursors

  __device__ __forceinline__ FfnJob(const FfnTileArgs& args, FfnLds& lds, int block, int blocks)
      : a(args), groups(lds.groups), turned(lds.turned[__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)]) {
    slots = blocks >> 3;
    xcd = block & 7;
    slot = block >> 3;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    half_slices = slices_of(a.len);
    sp = FfnShare::of<KIND>(a, groups, xcd, slots, G::PARTIAL);
    n_whole = sp.R + (sp.P == 0 && slot < sp.tail ? 1 : 0);
    run0 = slot * sp.P;
    run1 = min(run0 + sp.P, sp.tail * sp.KT);
    n_items = n_whole + (run0 < run1 ? (run1 - 1) / sp.KT - run0 / sp.KT + 1 : 0);
    if (kOverRows && a.groups > 1 && n_items > 0)
      load_e = tile_e = groups.full_of((sp.begin + slot) / ((KIND == kDw13 ? 2 : 1) * a.row_tiles * a.col_tiles * a.cuts), a.groups);
  }
  __device__ __forceinline__ Item item(int i, int& e) const {
    Item it{};
    int t;
    it.ke = sp.KT;
    it.part = -1;
    if (i < n_whole) {
      t = sp.begin + slot + i * slots;
    } else {
      const int j = run0 / sp.KT + (i - n_whole);
      t = sp.begin + sp.R * slots + j;
      it.kb = max(run0 - j * sp.KT, 0);
      it.ke = min(run1 - j * sp.KT, sp.KT);
      it.part = xcd * 2 * slots + slot + j;
    }
    int rt, ct;
    if constexpr (kOverRows) {
      const int per_half = a.row_tiles * a.col_tiles, per_group = (KIND == kDw13 ? 2 : 1) * per_half;
      const bool cut = a.groups > 1 && a.cuts > 1;
      int c = 0;
      if (cut) {
        it.part = t;
        c = t % a.cuts;
        t /= a.cuts;
      }
      const int n = t / per_group;                             // of the groups that have rows
      int in = t - n * per_group;
      if (a.groups > 1)
        while (groups.full_before(e + 1) <= n) ++e;            // tiles ascend
      if (KIND == kDw13 && in >= per_half) {
        in -= per_half;
        it.half = 1;
      }
      tile_at(in, a.row_tiles, a.col_tiles, rt, ct);
      it.first = groups.first(e);
      it.terms = groups.first(e + 1) - it.first;
      if (sp.KT == 0) {
        const int KT = slices_of(it.terms);
        it.kb = cut ? (int)((int64_t)KT * c / a.cuts) : 0;
        it.ke = cut ? (int)((int64_t)KT * (c + 1) / a.cuts) : KT;
        if (it.kb == it.ke) {                                  // fewer slices than parts: one slice of nothing
          it.terms = 0;
          it.kb = 0;
          it.ke = 1;
        }
      }
      it.r0 = rt * G::TB;
      it.r_end = a.rows;
    } else {
      if (a.groups > 1) e = groups.next(e, t / a.col_tiles, a.groups);      // tiles ascend
      const int before = groups.before(e);
      tile_at(t - before * a.col_tiles, groups.before(e + 1) - before, a.col_tiles, rt, ct);
      it.r0 = groups.first(e) + rt * G::TB;
      it.r_end = groups.first(e + 1);
    }
    it.e = e;
    it.c0 = ct * (kPair ? G::TA / 2 : G::TA);
    it.e = __builtin_amdgcn_readfirstlane(it.e);
    it.r0 = __builtin_amdgcn_readfirstlane(it.r0);
    if constexpr (!kOverRows) it.r_end = __builtin_amdgcn_readfirstlane(it.r_end);
    it.c0 = __builtin_amdgcn_readfirstlane(it.c0);
    it.half = __builtin_amdgcn_readfirstlane(it.half);
    it.kb = __builtin_amdgcn_readfirstlane(it.kb);
    it.ke = __builtin_amdgcn_readfirstlane(it.ke);
    it.part = __builtin_amdgcn_readfirstlane(it.part);
    return it;
  }
  __device__ __forceinline__ Item load_item(int i) { return item(i, load_e); }
  __device__ __forceinline__ Item tile_item(int i) { return item(i, tile_e); }
  __device__ __forceinline__ const void* base() const { return a.Q0; }
  __device__ __forceinline__ int64_t ldp() const { return kOverRows ? a.rows : a.len; }
  __device__ __forceinline__ int64_t ldq() const { return kPair ? a.len : a.cols; }
  __device__ __forceinline__ int row_slice(int kt) const { return KIND == kDx && kt >= half_slices ? kt - half_slices : kt; }
  __device__ __forceinline__ int row_terms() const { return a.len; }
  __device__ __forceinline__ void descs(const Item& it, int kt, bool first, i32x4_t& dq, i32x4_t& dp) const {
    const bool second = KIND == kDx && kt >= half_slices;
    const int64_t t0 = (int64_t)row_slice(kt) * G::BK;
    if constexpr (kPair) {
      const uint16_t* q = (wave >> 1) & 1 ? a.Q1 : a.Q0;
      if (first) dq = make_desc(q + ((int64_t)it.e * a.cols + it.c0) * a.len, min(G::TA / 2, a.cols - it.c0) * ldq() * 2);
    } else if constexpr (kOverRows) {
      dq = make_desc(a.Q0 + (it.first + t0) * ldq() + it.c0, ((it.terms - t0) * ldq() - it.c0) * 2);
    } else {
      const uint16_t* q = (second ? a.Q1 : a.Q0) + (int64_t)it.e * a.len * a.cols;
      dq = make_desc(q + t0 * ldq() + it.c0, ((a.len - t0) * ldq() - it.c0) * 2);
    }
    if constexpr (kOverRows) {
      const uint16_t* p = it.half != 0 ? a.P1 : a.P0;
      dp = make_desc(p + (it.first + t0) * ldp() + it.r0, ((it.terms - t0) * ldp() - it.r0) * 2);
    } else if (first || (KIND == kDx && kt == half_slices)) {
      dp = make_desc((second ? a.P1 : a.P0) + it.r0 * ldp(), min(G::TB, it.r_end - it.r0) * ldp() * 2);
    }
  }

  template <int WA, int WB>
  __device__ __forceinline__ void epilogue(const Item& it, f32x4_t (&acc)[WA][WB], int wr, int wc, int lane) const {
    asm volatile("" : "+v"(lane));          // (places in rows are formed here: kept, they would cost the product loop registers)
    int i = lane & 15, g = lane >> 4;
    float* part = it.part >= 0 ? a.partials + (int64_t)it.part * G::PARTIAL : nullptr;
    if (part != nullptr) {
#pragma unroll
      for (int o = 0; o < WA * WB; ++o) {
        const int x = o % WA, y = o / WA;
        asm volatile("" : "+v"(i), "+v"(g), "+s"(part));
        *reinterpret_cast<f32x4_t*>(part + ((wc * WB + y) * 16 + i) * G::TA + (wr * WA + x) * 16 + 4 * g) = acc[x][y];
        acc[x][y] = f32x4_t{};
        __builtin_amdgcn_sched_barrier(0);
      }
      return;
    }
    // Offsets from the tile's corner: one per pair of column blocks, out of range where
    // there is no such column; a row block adds `step`.
    const int rows = min(it.r_end - it.r0, G::TB), cols = a.cols - it.c0, step = 16 * a.cols * 2;
    constexpr int kPast = (int)0x80000000u;
    if constexpr (kPair) {
      // Blocks 2 n and 2 n + 1 of a wavefront are g and u of the same 16 channels.
      const TileOut h(a.o0, a.cols, it.r0, it.c0, rows, cols);
      const bool keep = a.o1 != nullptr;
      const TileOut pg(keep ? a.o1 : a.o0, a.cols, it.r0, it.c0, rows, cols);
      const TileOut pu(keep ? a.o2 : a.o0, a.cols, it.r0, it.c0, rows, cols);
      using Rows = RowStore<32>;
      const int c = WA == 4 ? wr * 32 + Rows::column(lane) : wr * 16 + 4 * g, r = WA == 4 ? Rows::row(lane) : i;
      int off = c < cols ? ((wc * WB * 16 + r) * a.cols + c) * 2 : kPast;
#pragma unroll
      for (int y = 0; y < WB; ++y) {
        asm volatile("" : "+v"(off));             // (or the row blocks' offsets are all formed at once)
        u32x2_t wh[WA / 2], wg[WA / 2], wu[WA / 2];
#pragma unroll
        for (int n = 0; n < WA / 2; ++n) {
          const f32x4_t vg = acc[2 * n][y], vu = acc[2 * n + 1][y];
          float vh[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) vh[k] = act_value<false>(vg[k], a.act) * vu[k];
          wh[n] = pack4(vh);
          wg[n] = pack4(vg);
          wu[n] = pack4(vu);
        }
        if constexpr (WA == 4) {
          u32x4_t v[1];
          Rows::turn(turned, wh, lane, v);
          h.template store<kNt>(off, v[0]);
          if (keep) {
            Rows::turn(turned, wg, lane, v);
            pg.template store<kNt>(off, v[0]);
            Rows::turn(turned, wu, lane, v);
            pu.template store<kNt>(off, v[0]);
          }
        } else {
          static_assert(WA == 2, "one pair of blocks, or two");
          h.store(off, wh[0]);
          if (keep) {
            pg.store(off, wg[0]);
            pu.store(off, wu[0]);
          }
        }
#pragma unroll
        for (int x = 0; x < WA; ++x) acc[x][y] = f32x4_t{};
        off += step;
        __builtin_amdgcn_sched_barrier(0);
      }
    } else if constexpr (KIND == kDh) {
      store_gradients(it, acc, wr, wc, i, g);
    } else {
      using Rows = RowStore<16 * WA>;
      uint16_t* to = it.half != 0 ? a.o1 : a.o0;
      if constexpr (kOverRows) to += (int64_t)it.e * a.rows * a.cols;
      const TileOut out(to, a.cols, it.r0, it.c0, rows, cols);
      const int c = wr * WA * 16 + Rows::column(lane), time = Rows::ROWS * a.cols * 2;
      int off = c < cols ? ((wc * WB * 16 + Rows::row(lane)) * a.cols + c) * 2 : kPast;
#pragma unroll
      for (int y = 0; y < WB; ++y) {
        asm volatile("" : "+v"(off));
        u32x2_t w[WA];
#pragma unroll
        for (int x = 0; x < WA; ++x) {
          w[x] = pack4(acc[x][y]);
          acc[x][y] = f32x4_t{};
        }
        u32x4_t v[Rows::TIMES];
        Rows::turn(turned, w, lane, v);
#pragma unroll
        for (int n = 0; n < Rows::TIMES; ++n) out.template store<kNt>(off + n * time, v[n]);
        off += step;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  // dg and du: g and u of D pieces (8 channels of a row per lane) are on their way.
  template <int WA, int WB>
  __device__ __forceinline__ void store_gradients(const Item& it, f32x4_t (&acc)[WA][WB], int wr, int wc, int i, int g) const {
    constexpr int NB = WA / 2, N = NB * WB, D = N < 4 ? N : 4;
    const int rows = min(it.r_end - it.r0, G::TB), cols = a.cols - it.c0, step = 16 * a.cols * 2;
    const TileOut og(a.o0, a.cols, it.r0, it.c0, rows, cols), ou(a.o1, a.cols, it.r0, it.c0, rows, cols);
    // (what is out of range loads as zero)
    const TileOut pg(const_cast<uint16_t*>(a.g), a.cols, it.r0, it.c0, rows, cols);
    const TileOut pu(const_cast<uint16_t*>(a.u), a.cols, it.r0, it.c0, rows, cols);
    u32x4_t vg[D], vu[D];
    int off[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int c = (wr * WA + 2 * n) * 16 + 8 * g;
      off[n] = c < cols ? ((wc * WB * 16 + i) * a.cols + c) * 2 : (int)0x80000000u;
    }
    auto fetch = [&](int o) __attribute__((always_inline)) {
      const int at = off[o % NB] + (o / NB) * step;
      vg[o % D] = __builtin_amdgcn_raw_buffer_load_b128(pg.desc, at, 0, 2);
      vu[o % D] = __builtin_amdgcn_raw_buffer_load_b128(pu.desc, at, 0, 2);
    };
#pragma unroll
    for (int o = 0; o < D; ++o) fetch(o);
#pragma unroll
    for (int o = 0; o < N; ++o) {
      const int n = o % NB, y = o / NB;
      asm volatile("" : "+v"(off[n]));
      float v[8];
      uint4 dg, du;
      join_blocks(acc[2 * n][y], acc[2 * n + 1][y], v);
      gated_gradients<KIND>(a, v, __builtin_bit_cast(uint4, vg[o % D]), __builtin_bit_cast(uint4, vu[o % D]), dg, du);
      const int at = off[n] + y * step;
      og.template store<kNt>(at, __builtin_bit_cast(u32x4_t, dg));
      ou.template store<kNt>(at, __builtin_bit_cast(u32x4_t, du));
      if (o + D < N) fetch(o + D);
      acc[2 * n][y] = acc[2 * n + 1][y] = f32x4_t{};
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

template <int KIND, int NS, int WR, int WC, int WA, int WB>
__device__ __forceinline__ void ffn_workgroup(const FfnTileArgs& a, uint8_t* smem, FfnLds& lds, int block,
                                              int blocks) {
  using G = ProductGeom<NS, WR, WC, WA, WB>;
  load_groups<KIND>(lds.groups, a, G::TB);
  FfnJob<KIND, G> job(a, lds, block, blocks);
  if (job.n_items > 0)
    tile_stream<ffn_over_rows(KIND), KIND != kGateUp, NS, WR, WC, WA, WB>(job, job.ldp(), job.ldq(), smem);
}

// Clears the gradients of groups without rows, of several: workgroup `block` of `blocks`,
// after its tiles (the groups are loaded).
template <int KIND, int THREADS>
__device__ __forceinline__ void clear_workgroup(const FfnTileArgs& a, const FfnGroups& groups, int block, int blocks) {
  const int halves = KIND == kDw13 ? 2 : 1, empty = (a.groups - groups.full_before(a.groups)) * halves;
  if (a.groups == 1 || empty == 0) return;
  constexpr int PART = THREADS * 8;                                  // 16-byte parts of a piece
  const int64_t n = (int64_t)a.rows * a.cols / 8;                    // (columns are a multiple of 8)
  const int64_t pieces = (n + PART - 1) / PART;
  for (int64_t i = block; i < empty * pieces; i += blocks) {
    const int q = (int)(i / pieces), e = groups.empty_of(q / halves, a.groups);
    const int64_t v0 = i % pieces * PART, v1 = v0 + PART < n ? v0 + PART : n;
    uint4* to = reinterpret_cast<uint4*>((q % halves != 0 ? a.o1 : a.o0) + (int64_t)e * a.rows * a.cols);
    for (int64_t v = v0 + threadIdx.x; v < v1; v += THREADS) store16<true>(to + v, make_uint4(0, 0, 0, 0));
  }
}

template <int KIND, int NS, int WR, int WC, int WA, int WB>
__global__ __launch_bounds__(64 * WR * WC, 1) void ffn_tiles_kernel(const FfnTileArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * ProductGeom<NS, WR, WC, WA, WB>::STAGE];
  __shared__ FfnLds lds;
  ffn_workgroup<KIND, NS, WR, WC, WA, WB>(a, smem, lds, blockIdx.x, gridDim.x);
  if constexpr (ffn_over_rows(KIND)) clear_workgroup<KIND, 64 * WR * WC>(a, lds.groups, blockIdx.x, gridDim.x);
}

// Sums the partial tiles of the cut tiles in contraction order and applies the epilogue.
// One workgroup per (XCD, tail tile, ROWS rows of it), or, if all are cut, (tile, ROWS rows), 8 columns (kGateUp:
// channels, 16 columns) of a row to a lane; four partials are in flight at a time.
template <int KIND, int TA> constexpr int kFfnJoinRows = (KIND == kGateUp ? 512 : 256) * 8 / TA;

template <int KIND, int TA, int TB>
__device__ __forceinline__ void ffn_join_workgroup(const FfnTileArgs& a, FfnGroups& groups, int slots, int block) {
  constexpr int ROWS = kFfnJoinRows<KIND, TA>, RG = TB / ROWS, LANES = 256 / ROWS;
  load_groups<KIND>(groups, a, TB);
  const int rg = block % RG;
  int t, first, parts;                       // the tile, and where its partial tiles lie
  bool cut = false;
  if constexpr (ffn_over_rows(KIND)) cut = a.groups > 1;
  if (cut) {
    t = block / RG;
    first = t * a.cuts;
    parts = a.cuts;
  } else {
    const int xcd = (block / RG) & 7, j = block / RG >> 3;
    const FfnShare sp = FfnShare::of<KIND>(a, groups, xcd, slots, TA * TB);
    if (sp.P == 0 || j >= sp.tail) return;
    t = sp.begin + sp.R * slots + j;
    const int s_lo = j * sp.KT / sp.P, s_hi = min(((j + 1) * sp.KT - 1) / sp.P, slots - 1);
    first = xcd * 2 * slots + j + s_lo;
    parts = s_hi - s_lo + 1;
  }
  int rt, ct, r0, r_end, half = 0, e = 0;
  if constexpr (ffn_over_rows(KIND)) {
    const int per_half = a.row_tiles * a.col_tiles, per_group = (KIND == kDw13 ? 2 : 1) * per_half;
    if (cut) {
      const int n = t / per_group;
      if (n >= groups.full_before(a.groups)) return;
      e = groups.full_of(n, a.groups);
      t -= n * per_group;
    }
    half = t >= per_half ? 1 : 0;
    tile_at(t - half * per_half, a.row_tiles, a.col_tiles, rt, ct);
    r0 = rt * TB;
    r_end = a.rows;
  } else {
    e = groups.of(t / a.col_tiles, a.groups);
    const int before = groups.before(e);
    tile_at(t - before * a.col_tiles, groups.before(e + 1) - before, a.col_tiles, rt, ct);
    r0 = groups.first(e) + rt * TB;
    r_end = groups.first(e + 1);
  }
  const int rl = rg * ROWS + threadIdx.x / LANES, cl = threadIdx.x % LANES * 8;
  const int r = r0 + rl, c = ct * (KIND == kGateUp ? TA / 2 : TA) + cl;
  if (r >= r_end || c >= a.cols) return;
  const int64_t at = (int64_t)r * a.cols + c;
  auto sum = [&](int col, float (&v)[8]) __attribute__((always_inline)) {
    const float* base = a.partials + (int64_t)first * (TA * TB) + rl * TA + col;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
    for (int s = 0; s < parts; s += 4) {
      float p[4][8];
#pragma unroll
      for (int q = 0; q < 4; ++q) load8f(base + (int64_t)min(s + q, parts - 1) * (TA * TB), p[q]);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += s + q < parts ? p[q][k] : 0.0f;
    }
  };
  float v[8];
  if constexpr (KIND == kGateUp) {
    float w[8];
    const int col = cl / 16 * 32 + cl % 16;
    sum(col, v);
    sum(col + 16, w);
    if (a.o1 != nullptr) {
      store16<false>(a.o1 + at, pack8(v));
      store16<false>(a.o2 + at, pack8(w));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = act_value<false>(v[k], a.act) * w[k];
    store16<false>(a.o0 + at, pack8(v));
  } else if constexpr (KIND == kDh) {
    const uint4 g = *reinterpret_cast<const uint4*>(a.g + at), u = *reinterpret_cast<const uint4*>(a.u + at);
    sum(cl, v);
    uint4 dg, du;
    gated_gradients<KIND>(a, v, g, u, dg, du);
    store16<false>(a.o0 + at, dg);
    store16<false>(a.o1 + at, du);
  } else {
    sum(cl, v);
    store16<false>((half != 0 ? a.o1 : a.o0) + (ffn_over_rows(KIND) ? (int64_t)e * a.rows * a.cols : 0) + at, pack8(v));
  }
}

// A's product on the first a_blocks workgroups, B's (a weight gradient) on the others; all clear.
template <int KA, int KB, int NS, int WR, int WC, int WA, int WB>
__global__ __launch_bounds__(64 * WR * WC, 1) void ffn_pair_kernel(const FfnTileArgs a, const FfnTileArgs b, int a_blocks) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * ProductGeom<NS, WR, WC, WA, WB>::STAGE];
  __shared__ FfnLds lds;
  const int i = blockIdx.x;
  if (i < a_blocks) ffn_workgroup<KA, NS, WR, WC, WA, WB>(a, smem, lds, i, a_blocks);
  else ffn_workgroup<KB, NS, WR, WC, WA, WB>(b, smem, lds, i - a_blocks, gridDim.x - a_blocks);
  clear_workgroup<KB, 64 * WR * WC>(b, lds.groups, i, gridDim.x);
}

template <int KA, int KB, int TA, int TB>
__global__ __launch_bounds__(256) void ffn_pair_join_kernel(const FfnTileArgs a, const FfnTileArgs b, int a_slots,
                                                            int b_slots, int a_blocks) {
  __shared__ FfnGroups groups;
  const int i = blockIdx.x;
  if (i < a_blocks) ffn_join_workgroup<KA, TA, TB>(a, groups, a_slots, i);
  else ffn_join_workgroup<KB, TA, TB>(b, groups, b_slots, i - a_blocks);
}

template <int KIND, int TA, int TB>
__global__ __launch_bounds__(256) void ffn_join_kernel(const FfnTileArgs a, int slots) {
  __shared__ FfnGroups groups;
  ffn_join_workgroup<KIND, TA, TB>(a, groups, slots, blockIdx.x);
}

}  // namespace moe
